// Prompt attention over ragged sequences: causal, within a sliding window,
// with the first tokens (sinks) always visible.
//
//   visible(i, j): j <= pos_i and (window < 0 or j > pos_i - window or j < sinks),  pos_i = nk - nq + i
//   s_ij = scale q_i . k_j;  lse_i = log sum_j exp(s_ij);  out_i = sum_j exp(s_ij - lse_i) v_j
//
// What bounds it: 4 x 128 flops per visible pair and head on the tensor cores
// and one exp2; every key tile is read from L2 by the items that see it.
//
// window_kernel (tcgen05). A work item is one KV head and two query tiles of
// 128 rows of one sequence; a tile's rows are consecutive tokens times the
// query heads that share the KV head, so that the heads of a group share every
// key tile and a narrow window wastes little. Keys and values come in tiles of
// 128 through a ring of 4. One CTA per SM, 16 warps:
//
//   8 softmax warps   a query tile each four, a thread owns a row
//   1 MMA warp        all tcgen05.mma; the warp runs as one with one lane
//                     elected per instruction: with the whole loop inside one
//                     lane's branch the operands of every MMA had to be moved to
//                     uniform registers first (a fifth slower when it was changed)
//   1 copy warp       items, and the tensor copies of queries, keys and values
//   4 output warps    O out of TMEM, normalised, staged and stored in 128-byte rows
//
//   S = Q K^T   both from shared memory (128-byte swizzle), into TMEM
//   P           2^(c S - c m), c = scale log2(e): registers, rounded once to the
//               inputs' type, back to TMEM over S, in two halves so that the
//               product with the values begins after the first
//   O += P V    P from TMEM, V from shared memory as stored (keys by d, the
//               d-contiguous operand form), into TMEM
//
// The two query tiles alternate: while one tile's softmax runs, the tensor
// cores run the other's P V and the next S. (An MMA warp per tile was a sixth
// slower when it was tried: the two then fall into step.) The running maximum m is a
// lazy reference: O is rescaled only when a row's maximum grew by more than
// 2^8 (weights then reach 2^8, whose relative rounding is the same), and the
// first weights of a tile are taken before its maximum is known.
//
// CTAs that have finished an item take the next from those of the grid that
// have not started (cluster launch control, asked with the copies of the last tile: the
// chunks below were 8 % slower when it was asked with those of the second): longest rows
// first, balanced whatever the lengths, and the next item's copies and first
// products run while the last one's results leave. With few items per SM each item's keys
// are split into parts whose partial sums window_join_kernel adds.
//
// The keys that an item's rows see are the sinks and one contiguous range.
// They are numbered without a gap (sinks rounded up to 16 rows, the extra rows
// masked), so a few sinks do not cost a tile of their own: the tile that
// holds both parts is copied in pieces of 16 rows.
//
// Rows that are not visible get weight 0, but 0 times an infinity or NaN in
// such a row's values would reach the sums. Columns of a row that are not finite
// are therefore looked into again from its visible keys alone (mend_row), when
// the CTA is done with its items: a row takes as long as its keys are many, and
// the pipeline's waits have a limit. Strides that a tensor map cannot express go
// row by row altogether (attend_row).
//
// Measured (GB300, 32 heads on 8 KV heads): 8,192 tokens causal 333 us in a short
// CUDA graph, 1.65 PFLOP/s of the visible pairs, 0.86 of the measured cuBLAS burst, and
// 375 us in a long loop of calls under the power limit, 0.77; in a window of 1,024 110
// us, 0.62 (masked edges, and about 2.5 us per item that its 9 key tiles do not hide);
// 8 ragged prompts of up to 2,048 tokens in a window of 512 76 us; chunks of up to 512
// tokens over 7,000 to 16,000 keys 215 us, of which the join takes 18. Code that the
// warps' loops do not need costs all of them: values past a sequence's end made zeros in
// shared memory, by the MMA, the copy or a spare warp, took 2 to 4 % of every prompt.
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "attn_row.cuh"
#include "cache_internal.cuh"
#include "qsa_internal.cuh"
#include "tensor_map.cuh"

namespace qsa {
namespace {

__device__ uint32_t g_window_error;

constexpr int ROWS = 128;                   // rows of a query tile, keys of a key tile
constexpr int HALF = ROWS * 128;            // bytes of 128 rows x 64 elements
constexpr int TILE_BYTES = 2 * HALF;
constexpr int STAGES = 4;                   // key and value tiles in flight
constexpr int PIECE = 16;                   // rows of a copy in the tile where sinks and window meet
constexpr int MMA_WARP = 8, COPY_WARP = 9, OUT_WARP = 12, WTHREADS = 512;
// 128 registers a thread at launch: 8 softmax warps x 168 + 8 x 88 = 16 x 128.
constexpr int MORE_REGISTERS = 168, FEW_REGISTERS = 88;
constexpr int STAGING = 32 * 128;           // bytes of an output warp's staging: 128 bytes of each of its rows
constexpr int SLOT_ROW = 132;               // 128 sums, reference, weight sum, padding
constexpr float LAZY = 8.0f;
constexpr uint32_t S_COL = 0, O_COL = 256, TMEM_COLS = 512;

// A tile quarter (32 rows) of an item with rows to mend: which, and the quarter of another item before it.
struct Odd {
    int before;         // its item's slot, or -1
    uint32_t rows[2];   // of both query tiles
};

struct WindowParams {
    CUtensorMap q, k, v, k_piece, v_piece;
    WindowAttnArgs a;
    int group, tokens;      // query heads per KV head; tokens of a query tile
    int k_has_heads, v_has_heads;   // 0: all KV heads at one address
    int pairs, splits;      // pairs of query tiles of the batch; parts that an item's keys are split into at most
    int part_tiles;         // key tiles of a part, at least on average
    int falling;            // parts fall in size
    Divider per_split, per_part;   // by splits, by part_tiles
    float *slots;           // [pairs][nkv][splits][2 x 128 rows][SLOT_ROW]
    Odd *odd;               // [pairs][nkv][splits][4]: lists of what output warps found, see mend_row
    uint64_t wait_ns;
    int stall;              // diagnostics only: CTA 0 never copies its first key tile
};

// The keys one query row sees: [0, sinks) and [lo, end).
struct RowKeys {
    int sinks, lo, end;
};
__device__ __forceinline__ RowKeys row_keys(const WindowAttnArgs &a, int nk, int pos) {
    RowKeys r;
    r.end = max(0, pos + 1);
    r.lo = a.window < 0 || a.window > nk ? 0 : max(0, r.end - a.window);
    r.sinks = min(a.sinks, r.lo);
    return r;
}

// One row by one warp in fp32. True: the weights' sum is finite, a result is not.
template <typename T>
__device__ bool attend_row(const WindowAttnArgs &a, int q_row, int h, int k0, int nk, int pos) {
    const int lane = threadIdx.x & 31, kvh = h / (a.nheads / a.nkv);
    const float4 q = load4(static_cast<const T *>(a.q) + q_row * a.q_tok + h * a.q_head + 4 * lane);
    const T *kp = static_cast<const T *>(a.k) + k0 * a.k_tok + kvh * a.k_head + 4 * lane;
    const T *vp = static_cast<const T *>(a.v) + k0 * a.v_tok + kvh * a.v_head + 4 * lane;
    const float c = a.scale * LOG2E;
    const RowKeys w = row_keys(a, nk, pos);
    RowState r;
    for (int part = 0; part < 2; ++part) {
        const int j1 = part == 0 ? w.sinks : w.end;
        for (int j = part == 0 ? 0 : w.lo; j < j1; ++j)
            r.add(c * warp_sum(dot4(q, load4(kp + j * a.k_tok))), load4(vp + j * a.v_tok));
    }
    const size_t row = static_cast<size_t>(q_row) * a.nheads + h;
    const float4 y = r.result();
    store4(static_cast<T *>(a.out) + row * 128 + 4 * lane, y);
    if (a.lse != nullptr && lane == 0) a.lse[row] = (r.m + log2f(r.l)) * LN2;
    const float odd = (y.x * 0.0f + y.y * 0.0f) + (y.z * 0.0f + y.w * 0.0f);
    return r.l - r.l == 0.0f && __any_sync(FULL_MASK, !(odd == 0.0f));
}

// A row in `out` whose weights have a finite sum but whose results are not all
// finite: there is an infinity or NaN among the values. Where a column has one in a key
// that the row sees, the result is the formula's (weights are positive): NaN, or that
// infinity. Where it is only in keys that the row does not see, which the tensor cores
// multiplied by 0, the column is summed again from the visible keys alone. By one
// warp; the values are looked through first, no further than needed, so that a NaN
// that every row sees costs little.
template <typename T, int kLook, int kAdd>   // keys looked through, and summed, at once
__device__ __forceinline__ void mend_row(const WindowAttnArgs &a, int q_row, int h, int k0, int nk, int pos) {
    const int lane = threadIdx.x & 31, kvh = h / (a.nheads / a.nkv);
    const T *kp = static_cast<const T *>(a.k) + k0 * a.k_tok + kvh * a.k_head + 4 * lane;
    const T *vp = static_cast<const T *>(a.v) + k0 * a.v_tok + kvh * a.v_head + 4 * lane;
    T *row = static_cast<T *>(a.out) + (static_cast<size_t>(q_row) * a.nheads + h) * 128 + 4 * lane;
    const RowKeys w = row_keys(a, nk, pos);
    const int n = w.sinks + w.end - w.lo;
    auto key = [&](int i) { return i < w.sinks ? i : i - w.sinks + w.lo; };
    const float4 y4 = load4(row);
    float y[4] = {y4.x, y4.y, y4.z, y4.w};
    uint32_t odd = 0, nan = 0, up = 0, down = 0;   // bits of this lane's columns
#pragma unroll
    for (int e = 0; e < 4; ++e) odd |= (y[e] - y[e] == 0.0f ? 0u : 1u) << e;
    for (int i0 = 0; i0 < n && !__all_sync(FULL_MASK, (odd & ~nan) == 0u); i0 += kLook) {
        float4 v[kLook];
#pragma unroll
        for (int b = 0; b < kLook; ++b) v[b] = load4(vp + key(min(i0 + b, n - 1)) * a.v_tok);
#pragma unroll
        for (int b = 0; b < kLook; ++b) {
            const float x[4] = {v[b].x, v[b].y, v[b].z, v[b].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                nan |= (x[e] != x[e] ? 1u : 0u) << e;
                up |= (x[e] == INFINITY ? 1u : 0u) << e;
                down |= (x[e] == -INFINITY ? 1u : 0u) << e;
            }
        }
        nan |= up & down;
    }
    RowState r;
    if (__any_sync(FULL_MASK, (odd & ~(nan | up | down)) != 0u)) {
        const float4 q = load4(static_cast<const T *>(a.q) + q_row * a.q_tok + h * a.q_head + 4 * lane);
        const float c = a.scale * LOG2E;
        for (int i0 = 0; i0 < n; i0 += kAdd) {
            float4 v[kAdd];
            float x[kAdd];
#pragma unroll
            for (int b = 0; b < kAdd; ++b) {
                const int j = key(min(i0 + b, n - 1));
                x[b] = dot4(q, load4(kp + j * a.k_tok));
                v[b] = load4(vp + j * a.v_tok);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                for (int b = 0; b < kAdd; ++b) x[b] += __shfl_xor_sync(FULL_MASK, x[b], o);
#pragma unroll
            for (int b = 0; b < kAdd; ++b)
                if (i0 + b < n) r.add(c * x[b], v[b]);
        }
    }
    const float4 s = r.result();
    const float again[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if ((odd >> e) & 1u)
            y[e] = (nan >> e) & 1u ? NAN : (up >> e) & 1u ? INFINITY : (down >> e) & 1u ? -INFINITY : again[e];
    store4(row, make_float4(y[0], y[1], y[2], y[3]));
}

// The sequence's ranges, clamped to the tensors.
struct Sequence {
    int q0, nq, k0, nk;
};
__device__ __forceinline__ Sequence sequence(const WindowAttnArgs &a, int s) {
    Sequence x;
    x.q0 = min(max(ld_in(a.cu_q + s), 0), a.total_q);
    x.nq = min(max(ld_in(a.cu_q + s + 1), x.q0), a.total_q) - x.q0;
    x.k0 = min(max(ld_in(a.cu_k + s), 0), a.total_k);
    x.nk = min(max(ld_in(a.cu_k + s + 1), x.k0), a.total_k) - x.k0;
    return x;
}

template <typename T>
__global__ void __launch_bounds__(256) window_rows_kernel(const WindowAttnArgs a) {
    grid_dependency_wait();
    const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
    const Sequence x = sequence(a, blockIdx.z);
    if (i >= x.nq) return;
    const int pos = x.nk - x.nq + i;
    // An infinity whose weight has since underflowed has become NaN.
    if (attend_row<T>(a, x.q0 + i, blockIdx.y, x.k0, x.nk, pos)) mend_row<T, 8, 4>(a, x.q0 + i, blockIdx.y, x.k0, x.nk, pos);
}

// An item's keys, numbered without gaps: numbers below `front` are keys
// 0 .. front-1 (front = the sinks rounded up to whole pieces), number i from
// there on is key i - front + lo. Row limits are in these numbers.
struct ItemKeys {
    int front, lo, count;
    int sink_end;            // numbers below it are sinks of every row
    int window;
    ItemKeys() = default;
    __device__ __forceinline__ ItemKeys(const WindowAttnArgs &a, int nk, int pos_first, int pos_last) {
        window = a.window < 0 || a.window > nk ? nk : a.window;
        lo = max(0, pos_first + 1 - window);
        const int sinks = min(a.sinks, nk);
        front = 0;
        if (sinks >= lo) {
            lo = 0;
        } else {
            front = (sinks + PIECE - 1) / PIECE * PIECE;
            // Rounded up, the front would reach the window: then from 0 on without a gap.
            if (front >= lo) front = lo = 0;
        }
        sink_end = sinks;
        const int end = max(0, pos_last + 1);
        count = end > lo ? front + end - lo : (end > 0 ? front : 0);
    }
    __device__ __forceinline__ int tiles() const { return (count + ROWS - 1) / ROWS; }
    // Row at pos sees number i iff i <= last(pos) and (i < sink_end or i >= first(pos)).
    __device__ __forceinline__ int last(int pos) const { return pos < 0 ? -1 : pos - lo + front; }
    __device__ __forceinline__ int first(int pos) const { return max(pos + 1 - window, lo) - lo + front; }
};

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two fp32 values in one 64-bit register, worked on by one instruction.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t r, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
template <typename T>
__device__ __forceinline__ uint32_t pack2_rn(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2_rn<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2_rn<__half>(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// A work item: two query tiles of one sequence and KV head, and (when items
// are split over their keys) one part of their key tiles.
struct Item {
    int q0, nq, k0, nk, t0, kvh, part, slot;   // t0: first token; slot: of the partial results
};

// What all roles need of an item, worked out once by the copying warp.
struct Work {
    Item it;
    int tokens0, tokens1, pos0, pos1;   // tokens and first row of the two tiles
    ItemKeys keys;
    int last0, first0, last1, first1;   // limits of the tiles' last and first rows
    int parts, j0, j1;                  // parts that have key tiles (at least 1), this part's tiles
    Work() = default;
    __device__ __forceinline__ Work(const WindowParams &p, const Item &it)
        : it(it), tokens0(min(p.tokens, it.nq - it.t0)), tokens1(min(p.tokens, max(0, it.nq - it.t0 - p.tokens))),
          pos0(it.nk - it.nq + it.t0), pos1(pos0 + p.tokens), keys(p.a, it.nk, pos0, pos0 + tokens0 + tokens1 - 1) {
        last0 = keys.last(pos0 + tokens0 - 1);
        first0 = keys.first(pos0);
        last1 = tokens1 > 0 ? keys.last(pos1 + tokens1 - 1) : -1;
        first1 = keys.first(pos1);
        const int n = keys.tiles();
        parts = 1;
        j0 = 0;
        j1 = n;
        if (p.splits > 1 && n > 0) {
            if (p.falling) {
                parts = min(p.splits, divide(p.per_part, n - 1) + 1);
                j0 = falling_begin(it.part, n);
                j1 = falling_begin(it.part + 1, n);
            } else {
                const int each = max(divide(p.per_split, n - 1) + 1, p.part_tiles);
                parts = (n + each - 1) / each;
                j0 = min(it.part * each, n);
                j1 = min(j0 + each, n);
            }
        }
    }
    // First key tile of part k of parts that fall in size, in the ratio m - 0.3, m - 1.3, .. 0.7 of m
    // parts (each has a tile), so that all items' large parts run first and the small ones fill
    // the ends.
    __device__ __forceinline__ int falling_begin(int k, int n) const {
        if (k == 0) return 0;
        if (k >= parts) return n;
        const uint32_t of = parts * (5 * parts + 2), at = k * (10 * parts - 5 * k + 2);
        const uint32_t whole = n / of, left = n - whole * of;   // n x at / of, where n x at might not fit
        return static_cast<int>(whole * at + left * at / of);
    }
    // Does any row of query tile i see a key of key tile j?
    __device__ __forceinline__ bool needed(int i, int j) const {
        const int n = j * ROWS;
        return n <= (i == 0 ? last0 : last1) && (n < keys.sink_end || n + ROWS - 1 >= (i == 0 ? first0 : first1));
    }
};

struct WindowBarriers {
    uint4 next;             // the answer about the next item
    Work work[2];
    uint64_t q_full[2], q_empty[2], kv_full[STAGES], kv_empty[STAGES], s_full[2], p_half[2], p_full[2];
    uint64_t o_full[2], o_empty[2], sum_full[2], sum_empty[2], item_full[2], item_empty[2], next_full, drain;
    uint32_t tmem, abort;
    uint32_t any[2];        // whether the tile's O was written
    float2 sum[2][ROWS];    // reference (base 2) and weight sum of each row
};
constexpr size_t WINDOW_SMEM = 1024 + (2 + STAGES) * static_cast<size_t>(TILE_BYTES) + 4 * STAGING + sizeof(WindowBarriers);
static_assert(WINDOW_SMEM <= 232448, "shared memory per CTA");

// The item number `n` of the grid, found by a whole warp; false when there is
// nothing to do. Query tiles pairs are numbered over the batch without
// knowing the lengths: sequence s begins at cu_q[s] / (tokens per pair) + s.
__device__ __forceinline__ bool find_item(const WindowParams &p, uint32_t n, Item &it) {
    const WindowAttnArgs &a = p.a;
    const int lane = threadIdx.x & 31, per = 2 * p.tokens;
    // Head fastest, then the pairs, the last tokens (which see most) first, then the parts:
    // what runs together reads the same keys.
    it.kvh = n % a.nkv;
    n /= a.nkv;
    it.part = n / p.pairs;
    const int g = static_cast<int>(p.pairs - 1 - n % p.pairs);
    auto start = [&](int s) { return min(max(ld_in(a.cu_q + s), 0), a.total_q) / per + s; };
    int lo = 0, hi = a.nseq;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, s = lo + (lane + 1) * step;
        const int below = __popc(__ballot_sync(FULL_MASK, s < hi && start(s) <= g));
        lo += below * step;
        hi = min(hi, lo + step);
    }
    const Sequence x = sequence(a, lo);
    it.q0 = x.q0;
    it.nq = x.nq;
    it.k0 = x.k0;
    it.nk = x.nk;
    const long long t0 = static_cast<long long>(g - (x.q0 / per + lo)) * per;
    it.t0 = static_cast<int>(max(0LL, min(t0, static_cast<long long>(x.nq))));
    it.slot = (g * a.nkv + it.kvh) * p.splits + it.part;
    return t0 >= 0 && t0 < x.nq;
}

// Asks for the index of a CTA of this grid that has not started, which then
// never starts: the 16-byte answer completes on `bar`.
__device__ __forceinline__ void ask_next(uint32_t answer, uint64_t *bar) {
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(answer),
        "r"(smem_u32(bar))
        : "memory");
}
// The answer: false when every CTA has started.
__device__ __forceinline__ bool read_next(uint32_t answer, uint32_t &x) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t.reg .b32 y, z, w;\n\t"
        "ld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, r;\n\t}"
        : "=r"(ok), "=r"(x)
        : "r"(answer)
        : "memory");
    return ok != 0;
}
template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <typename T>
__global__ void __launch_bounds__(WTHREADS, 1) window_kernel(const __grid_constant__ WindowParams p) {
    extern __shared__ unsigned char raw[];
    const WindowAttnArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(FULL_MASK, tid >> 5, 0);   // the same for the warp, as the compiler now knows
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t ring = base + 2 * TILE_BYTES;
    const uint32_t staging = ring + STAGES * TILE_BYTES;
    WindowBarriers *bars = reinterpret_cast<WindowBarriers *>(raw + (staging + 4 * STAGING - smem_u32(raw)));

    Item first_item;
    bool first_found = false;
    if (warp == MMA_WARP) {
        tmem_alloc(&bars->tmem, TMEM_COLS);
        tmem_relinquish();
    } else if (warp == COPY_WARP) {
        if (lane == 0) {
            prefetch_tensor_map(&p.q);
            prefetch_tensor_map(&p.k);
            prefetch_tensor_map(&p.v);
        }
        __syncwarp();
        grid_dependency_wait();
        first_found = find_item(p, blockIdx.x, first_item);
    } else if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->q_full[i], 1);
            mbar_init(&bars->q_empty[i], 1);
            mbar_init(&bars->s_full[i], 1);
            mbar_init(&bars->p_half[i], 4);
            mbar_init(&bars->p_full[i], 4);
            mbar_init(&bars->o_full[i], 1);
            mbar_init(&bars->o_empty[i], 4);
            mbar_init(&bars->sum_full[i], 4);
            mbar_init(&bars->sum_empty[i], 4);
            mbar_init(&bars->item_full[i], 1);
            mbar_init(&bars->item_empty[i], 1 + 8 + 4);
        }
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&bars->kv_full[i], 1);
            mbar_init(&bars->kv_empty[i], 1);
        }
        mbar_init(&bars->next_full, 1);
        mbar_init(&bars->drain, 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = bars->tmem;
    grid_dependency_wait();
    grid_launch_dependents();

    // A wait of the pipeline: the first that runs out sets the error word, and
    // all later ones return at once.
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity)) return true;
        volatile uint32_t *ab = &bars->abort;
        if (*ab == 0u && mbar_wait(bar, parity, p.wait_ns, ab)) return true;
        if (*ab == 0u) {
            *ab = 1u;
            atomicOr(&g_window_error, 1u);
        }
        return false;
    };
    auto wait_warp = [&](uint64_t *bar, uint32_t parity) { return __all_sync(FULL_MASK, wait(bar, parity)); };

    if (warp == COPY_WARP) {
        fewer_registers<FEW_REGISTERS>();
        // ---- items, queries, keys and values in ------------------------------------------
        uint32_t n = blockIdx.x;             // the item's number
        uint32_t asked = 0, kv = 0, nq[2] = {0, 0};
        bool ok = true, more = true, open = false;   // open: an answer is under way
        const uint32_t answer = smem_u32(&bars->next);
        auto ask = [&]() {
            if (lane == 0) {
                fence_proxy_async_smem();    // the last answer has been read
                mbar_arrive_expect_tx(&bars->next_full, 16);
                ask_next(answer, &bars->next_full);
            }
            open = true;
            __syncwarp();
        };
        auto get = [&]() {
            ok = wait_warp(&bars->next_full, asked & 1);
            if (!ok) return;
            open = false;
            ++asked;
            more = read_next(answer, n);
            __syncwarp();
        };
        for (uint32_t k = 0; ok; ++k) {
            Work w;
            bool found = false;
            while (ok && more && !found) {
                Item it = first_item;
                found = asked == 0 ? first_found : find_item(p, n, it);
                w = Work(p, it);
                found = found && it.part < w.parts;
                if (!found) {
                    ask();
                    get();
                }
            }
            if (!ok || !wait_warp(&bars->item_empty[k & 1], ((k >> 1) & 1) ^ 1)) break;
            if (lane == 0) {
                if (!found) w.tokens0 = 0;   // the end
                bars->work[k & 1] = w;
                mbar_arrive(&bars->item_full[k & 1]);
            }
            __syncwarp();
            if (!found) break;
            const Item &it = w.it;
            for (int i = 0; ok && i < (w.tokens1 > 0 ? 2 : 1); ++i, __syncwarp()) {
                ok = wait_warp(&bars->q_empty[i], (nq[i] & 1) ^ 1);
                if (ok && nq[i] > 0) ok = wait_warp(&bars->q_full[i], (nq[i] - 1) & 1);   // landed, needed or not
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&bars->q_full[i], 2u * 128u * p.group * p.tokens);
                    for (int half = 0; half < 2; ++half)
                        tma_load_3d(base + i * TILE_BYTES + half * HALF, &p.q, 64 * half, it.kvh * p.group,
                                    it.q0 + it.t0 + i * p.tokens, &bars->q_full[i]);
                }
                ++nq[i];
            }
            const ItemKeys &keys = w.keys;
            for (int j2 = 2 * w.j0; ok && j2 < 2 * w.j1; ++j2, ++kv) {   // keys, then values of tile j2 / 2
                // The next item is claimed with the last tile's copies: earlier, items would be dealt
                // out by when CTAs start one and not by when they end one.
                if (j2 == 2 * w.j1 - 2 && j2 > 2 * w.j0) ask();
                const int slot = kv % STAGES, i0 = (j2 >> 1) * ROWS;
                ok = wait_warp(&bars->kv_empty[slot], ((kv / STAGES) & 1) ^ 1);
                if (!ok) break;
                if (lane == 0 && !(p.stall != 0 && blockIdx.x == 0 && kv == 0)) {
                    uint64_t *bar = &bars->kv_full[slot];
                    const uint32_t dst = ring + slot * TILE_BYTES;
                    const bool values = j2 & 1;
                    const int head = (values ? p.v_has_heads : p.k_has_heads) ? it.kvh : 0;
                    mbar_arrive_expect_tx(bar, TILE_BYTES);
                    if (i0 < keys.front && i0 + ROWS > keys.front) {
                        for (int r = 0; r < ROWS; r += PIECE) {
                            const int key = i0 + r < keys.front ? i0 + r : i0 + r - keys.front + keys.lo;
                            for (int half = 0; half < 2; ++half)
                                tma_load_3d(dst + half * HALF + r * 128, values ? &p.v_piece : &p.k_piece, 64 * half, head,
                                            it.k0 + key, bar);
                        }
                    } else {
                        const int key = i0 < keys.front ? i0 : i0 - keys.front + keys.lo;
                        for (int half = 0; half < 2; ++half)
                            tma_load_3d(dst + half * HALF, values ? &p.v : &p.k, 64 * half, head, it.k0 + key, bar);
                    }
                }
                __syncwarp();
            }
            if (ok && !open) ask();
            if (ok) get();
        }
        // What was begun here lands before the CTA leaves (at once without an abort).
        if (open) mbar_wait(&bars->next_full, asked & 1, p.wait_ns);
        for (uint32_t d = kv > STAGES ? kv - STAGES : 0; d < kv; ++d)
            mbar_wait(&bars->kv_full[d % STAGES], (d / STAGES) & 1, p.wait_ns);
        for (int i = 0; i < 2; ++i)
            if (nq[i] > 0) mbar_wait(&bars->q_full[i], (nq[i] - 1) & 1, p.wait_ns);
        __syncwarp();
    } else if (warp == MMA_WARP) {
        fewer_registers<FEW_REGISTERS>();
        {
            const bool one = elect_one();   // the warp runs as one, one lane issues
            constexpr uint32_t fmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
            constexpr uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
            constexpr uint32_t idesc_v = idesc | (1u << 16);   // second operand contiguous in N
            // Per query tile, in registers: every index below is a constant.
            struct Tile {
                uint32_t ns = 0, nq = 0;   // products S and query tiles so far
                bool pending, any, free_o;
            } tile0, tile1;
            bool ok = true;
            uint32_t kv = 0;               // copies so far
            for (uint32_t k = 0; ok; ++k) {
                ok = wait_warp(&bars->item_full[k & 1], (k >> 1) & 1);
                if (!ok) break;
                const Work w = bars->work[k & 1];
                __syncwarp();
                if (one) mbar_arrive(&bars->item_empty[k & 1]);
                if (w.tokens0 == 0) break;
                tile0.pending = tile0.any = tile0.free_o = false;
                tile1.pending = tile1.any = tile1.free_o = false;
                // A tile's P V of its last S, then its S of key tile j.
                auto advance = [&](auto which, Tile &t, int j, uint32_t kn) {
                    constexpr int i = decltype(which)::value;
                    const uint32_t s_col = tmem + S_COL + 128 * i, o_col = tmem + O_COL + 128 * i;
                    if (t.pending) {
                        const uint64_t vd = sw128_mnmajor_desc(ring + ((kn - 1) % STAGES) * TILE_BYTES, HALF);
                        if (!t.free_o) ok = t.free_o = wait_warp(&bars->o_empty[i], (k & 1) ^ 1);
                        if (ok) ok = wait_warp(&bars->p_half[i], (t.ns - 1) & 1);
                        if (!ok) return;
                        tc_fence_after_sync();
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            if (one) tc_mma_bf16_ta(o_col, s_col + 8 * kk, vd + 128 * kk, idesc_v, (t.any || kk > 0) ? 1u : 0u);
                        ok = wait_warp(&bars->p_full[i], (t.ns - 1) & 1);
                        if (!ok) return;
                        tc_fence_after_sync();
#pragma unroll
                        for (int kk = 4; kk < 8; ++kk)
                            if (one) tc_mma_bf16_ta(o_col, s_col + 8 * kk, vd + 128 * kk, idesc_v, 1u);
                        t.pending = false;
                        t.any = true;
                    }
                    if (j < w.j1 && w.needed(i, j)) {
                        const uint64_t qd = sw128_kmajor_desc(base + i * TILE_BYTES);
                        const uint64_t kd = sw128_kmajor_desc(ring + (kn % STAGES) * TILE_BYTES);
                        if (!t.any) ok = wait_warp(&bars->q_full[i], t.nq & 1);
                        if (!ok) return;
                        tc_fence_after_sync();
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) {
                            const uint64_t step = (kk >> 2) * (HALF >> 4) + 2 * (kk & 3);
                            if (one) tc_mma_bf16(s_col, qd + step, kd + step, idesc, kk > 0 ? 1u : 0u);
                        }
                        if (one) tc_commit(&bars->s_full[i]);
                        t.pending = true;
                        ++t.ns;
                    }
                };
                for (int j = w.j0; ok && j <= w.j1; ++j) {
                    const uint32_t kn = kv + 2 * (j - w.j0);
                    // Every copy is waited for, also one that no row needs: its slot is reused after this step.
                    if (j < w.j1) ok = wait_warp(&bars->kv_full[kn % STAGES], (kn / STAGES) & 1);
                    if (ok && j > w.j0) ok = wait_warp(&bars->kv_full[(kn - 1) % STAGES], ((kn - 1) / STAGES) & 1);
                    if (ok) advance(std::integral_constant<int, 0>(), tile0, j, kn);
                    if (ok) advance(std::integral_constant<int, 1>(), tile1, j, kn);
                    if (!ok) break;
                    // Tile j's keys and tile j-1's values are free when all of this is done.
                    if (one && j > w.j0) tc_commit(&bars->kv_empty[(kn - 1) % STAGES]);
                    if (one && j < w.j1) tc_commit(&bars->kv_empty[kn % STAGES]);
                    if (j == w.j1 - 1 || w.j0 == w.j1) {
                        if (one) tc_commit(&bars->q_empty[0]);
                        if (one && w.tokens1 > 0) tc_commit(&bars->q_empty[1]);
                    }
                }
                kv += 2 * (w.j1 - w.j0);
                ++tile0.nq;
                if (w.tokens1 > 0) ++tile1.nq;
                // One item ahead of the results at most.
                if (ok && !tile0.free_o) ok = wait_warp(&bars->o_empty[0], (k & 1) ^ 1);
                if (ok && !tile1.free_o) ok = wait_warp(&bars->o_empty[1], (k & 1) ^ 1);
                if (ok) {
                    if (one) tc_commit(&bars->o_full[0]);
                    if (one) tc_commit(&bars->o_full[1]);
                }
            }
            if (one) tc_commit(&bars->drain);
            mbar_wait(&bars->drain, 0, p.wait_ns);
        }
        __syncwarp();
    } else if (warp >= OUT_WARP) {
        fewer_registers<FEW_REGISTERS>();
        // ---- results: rows 32 quarter .. + 31 of both tiles --------------------------------
        const int quarter = warp & 3;
        const uint32_t stage = staging + quarter * STAGING;
        int last_odd = -1;   // of this warp's list of rows to mend
        bool ok = true;
        for (uint32_t k = 0;; ++k) {
            ok = wait_warp(&bars->item_full[k & 1], (k >> 1) & 1);
            if (!ok) break;
            const Work w = bars->work[k & 1];
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->item_empty[k & 1]);
            if (w.tokens0 == 0) break;
            const Item &it = w.it;
            for (int i = 0; i < 2; ++i) {
                ok = wait_warp(&bars->sum_full[i], k & 1) && wait_warp(&bars->o_full[i], k & 1);
                if (!ok) break;
                tc_fence_after_sync();
                const int row = 32 * quarter + lane, tok = row / p.group, head = row - tok * p.group;
                const int ntok = i == 0 ? w.tokens0 : w.tokens1;
                const bool valid = tok < ntok;
                if (ntok == 0) {   // the second tile of a short item
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&bars->o_empty[i]);
                        mbar_arrive(&bars->sum_empty[i]);
                    }
                    continue;
                }
                const float2 sum = bars->sum[i][row];
                const bool any = bars->any[i] != 0u, split = w.parts > 1;
                const int q_row = it.q0 + it.t0 + i * p.tokens + tok, h = it.kvh * p.group + head;
                const long long out_row = static_cast<long long>(q_row) * a.nheads + h;
                const uint32_t rows = __ballot_sync(FULL_MASK, valid);
                // Where this lane's row goes: 4 pieces of 128 bytes of partial sums, or 2 of results.
                char *to = split ? reinterpret_cast<char *>(p.slots + (static_cast<size_t>(it.slot) * 2 * ROWS + i * ROWS + row) * SLOT_ROW)
                                 : reinterpret_cast<char *>(static_cast<T *>(a.out) + out_row * 128);
                const float inv = sum.y == 0.0f ? 0.0f : 1.0f / sum.y;
                float odds[4] = {0.0f, 0.0f, 0.0f, 0.0f};   // stay 0 while everything is finite
                const uint32_t o_at = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + O_COL + 128 * i;
                // A piece is staged with its 16-byte chunks at chunk ^ (row % 8) and leaves as whole
                // 128-byte rows: this lane stores chunk lane % 8 of rows lane / 8 + 0, 4, .. 28.
                char *row_to[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    row_to[e] = reinterpret_cast<char *>(__shfl_sync(FULL_MASK, reinterpret_cast<unsigned long long>(to), 4 * e + (lane >> 3))) +
                                16 * (lane & 7);
                auto leave = [&](int piece) {
                    __syncwarp();
                    uint4 v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int r = 4 * e + (lane >> 3);
                        v[e] = ld_shared_v4(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if ((rows >> (4 * e + (lane >> 3))) & 1u) *reinterpret_cast<uint4 *>(row_to[e] + 128 * piece) = v[e];
                    __syncwarp();
                };
                auto put = [&](int chunk, uint32_t x, uint32_t y, uint32_t z, uint32_t u) {
                    st_shared_v4(stage + lane * 128 + ((chunk ^ (lane & 7)) << 4), x, y, z, u);
                };
#pragma unroll 1
                for (int g = 0; g < 4; ++g) {
                    uint32_t o[32];
                    __syncwarp();
                    if (any) {
                        tmem_ld32(o_at + 32 * g, o);
                        tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0u;
                    }
                    if (g == 3) {
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&bars->o_empty[i]);
                            mbar_arrive(&bars->sum_empty[i]);
                        }
                    }
                    if (split) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) put(e, o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                        leave(g);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) odds[e & 3] = fmaf(__uint_as_float(o[e]), 0.0f, odds[e & 3]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t y[4];
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                y[q] = pack2_rn<T>(__uint_as_float(o[8 * e + 2 * q]) * inv, __uint_as_float(o[8 * e + 2 * q + 1]) * inv);
                            put(4 * (g & 1) + e, y[0], y[1], y[2], y[3]);
                        }
                        if (g & 1) leave(g >> 1);
                    }
                }
                if (split) {
                    if (valid) *reinterpret_cast<float2 *>(to + 512) = sum;
                    continue;
                }
                if (valid && a.lse != nullptr) a.lse[out_row] = sum.y == 0.0f ? -INFINITY : (sum.x + log2f(sum.y)) * LN2;
                // Where the weights' sum is not finite, a visible key did it and all of the row is NaN already.
                const float odd = (odds[0] + odds[1]) + (odds[2] + odds[3]);
                const uint32_t odd_rows = __ballot_sync(FULL_MASK, valid && !(odd == 0.0f) && sum.y - sum.y == 0.0f);
                if (odd_rows == 0u) continue;
                Odd *to_odd = p.odd + 4 * static_cast<size_t>(it.slot) + quarter;
                if (last_odd != it.slot && lane == 0) *to_odd = {last_odd, {0u, 0u}};
                if (lane == 0) to_odd->rows[i] = odd_rows;
                last_odd = it.slot;
            }
            if (!ok) break;
        }
        // Rows are mended when all items are done, as that may take longer than a wait of the pipeline may.
        while (ok && last_odd >= 0) {
            __syncwarp();
            const Odd *odd = p.odd + 4 * static_cast<size_t>(last_odd) + quarter;
            const int at = last_odd / p.splits, g = at / a.nkv;
            Item it;
            find_item(p, static_cast<uint32_t>((p.pairs - 1 - g) * a.nkv + at - g * a.nkv), it);
            const Work w(p, it);
            last_odd = __ldcg(&odd->before);
#pragma unroll 1
            for (int i = 0; i < 2; ++i)
#pragma unroll 1
                for (uint32_t rows = __ldcg(odd->rows + i); rows != 0u; rows &= rows - 1) {
                    const int row = 32 * quarter + __ffs(rows) - 1, tok = row / p.group;
                    mend_row<T, 4, 2>(a, it.q0 + it.t0 + i * p.tokens + tok, it.kvh * p.group + row - tok * p.group, it.k0, it.nk,
                                (i == 0 ? w.pos0 : w.pos1) + tok);
                }
        }
    } else if (warp > COPY_WARP) {
        fewer_registers<FEW_REGISTERS>();   // completes the group of four whose registers the softmax takes
    } else {
        more_registers<MORE_REGISTERS>();
        // ---- softmax of one query tile, one row per thread -----------------------------
        const int i = warp >> 2, row = 32 * (warp & 3) + lane;
        const int tok = row / p.group;
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t s_at = tmem + lanes + S_COL + 128 * i, o_at = tmem + lanes + O_COL + 128 * i;
        const float c = a.scale * LOG2E;
        uint32_t ns = 0;
        for (uint32_t k = 0;; ++k) {
            if (!wait_warp(&bars->item_full[k & 1], (k >> 1) & 1)) break;
            const Work w = bars->work[k & 1];
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->item_empty[k & 1]);
            if (w.tokens0 == 0) break;
            const int ntok = i == 0 ? w.tokens0 : w.tokens1;
            const int pos = (i == 0 ? w.pos0 : w.pos1) + min(tok, max(ntok - 1, 0));
            const int last = w.keys.last(pos), first = w.keys.first(pos), sink_end = w.keys.sink_end, j1 = w.j1;
            const int tile_last = i == 0 ? w.last0 : w.last1, tile_first = i == 0 ? w.first0 : w.first1;
            // The warp's rows stand in order, so lane 0 sees the least far and lane 31 begins last.
            const int last_min = __shfl_sync(FULL_MASK, last, 0), first_max = __shfl_sync(FULL_MASK, first, 31);
            float m = -INFINITY, l = 0.0f;   // m: of the products, before c
            bool any = false, ok = true;
            for (int i0 = w.j0 * ROWS; i0 < j1 * ROWS; i0 += ROWS) {
                if (!(i0 <= tile_last && (i0 < sink_end || i0 + ROWS - 1 >= tile_first))) continue;
                ok = wait_warp(&bars->s_full[i], ns & 1);
                if (!ok) break;
                ++ns;
                tc_fence_after_sync();
                uint32_t sr[4][32];
#pragma unroll
                for (int g = 0; g < 4; ++g) tmem_ld32(s_at + 32 * g, sr[g]);
                tmem_ld_wait();
                if (i0 + ROWS - 1 > last_min || (i0 < first_max && i0 + ROWS > sink_end)) {
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        // Numbers n0 .. n0 + 31: mostly all of them are visible to the warp's rows, or none.
                        const int n0 = i0 + 32 * g;
                        if (n0 + 31 <= last_min && (n0 >= first_max || n0 + 32 <= sink_end)) continue;
                        auto below = [&](int limit) {   // bits of the numbers below the limit
                            const int k = limit - n0;
                            return k <= 0 ? 0u : k >= 32 ? 0xFFFFFFFFu : (1u << k) - 1u;
                        };
                        const uint32_t bits = below(last + 1) & (below(sink_end) | ~below(first));
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!((bits >> e) & 1u)) sr[g][e] = 0xFF800000u;
                    }
                }
                // Weights of 32 columns against the reference as it stands, so that they need not
                // wait for the maximum of this tile, which rarely moves it.
                uint64_t sums[2];
                uint32_t pw[16];
                auto weights = [&](int g) {
                    const float mc = m == -INFINITY ? 0.0f : m * c;
                    const uint64_t c2 = pair(c, c), mc2 = pair(-mc, -mc);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float x0, x1;
                        unpair(fma_pair(pair(__uint_as_float(sr[g][2 * e]), __uint_as_float(sr[g][2 * e + 1])), c2, mc2), x0, x1);
                        x0 = exp2_approx(x0);
                        x1 = exp2_approx(x1);
                        sums[e & 1] = g == 0 && e < 2 ? pair(x0, x1) : add_pair(sums[e & 1], pair(x0, x1));
                        pw[e] = pack2_rn<T>(x0, x1);
                    }
                };
                if (any) weights(0);
                // 8 chains, so that the maximum of 128 is not a chain of 128.
                float tops[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) tops[e] = __uint_as_float(sr[0][e]);
#pragma unroll
                for (int e = 8; e < 128; e += 16)
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float y = __uint_as_float(sr[e >> 5][(e & 31) + k]);
                        tops[k] = e + 8 < 128 ? fmaxf(fmaxf(tops[k], y), __uint_as_float(sr[(e + 8) >> 5][((e + 8) & 31) + k]))
                                              : fmaxf(tops[k], y);
                    }
                const float top = fmaxf(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])),
                                        fmaxf(fmaxf(tops[4], tops[5]), fmaxf(tops[6], tops[7])));
                const bool move = (top - m) * c > LAZY;   // also true from -infinity to a finite maximum
                if (__any_sync(FULL_MASK, move) || !any) {
                    const float f = move ? exp2_approx((m - top) * c) : 1.0f;
                    if (move) m = top;
                    l *= f;
                    if (any) {
#pragma unroll 1
                        for (int g = 0; g < 8; ++g) {
                            uint32_t o[16];
                            tmem_ld16(o_at + 16 * g, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st16(o_at + 16 * g, o);
                        }
                    }
                    weights(0);
                }
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    if (g > 0) weights(g);
                    tmem_st16(s_at + 16 * g, pw);
                    if (g & 1) {   // the products with half of the values can begin
                        tmem_st_wait();
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(g == 1 ? &bars->p_half[i] : &bars->p_full[i]);
                    }
                }
                {
                    float y0, y1;
                    unpair(add_pair(sums[0], sums[1]), y0, y1);
                    l += y0 + y1;
                }
                any = true;
            }
            // The output warps take over; they are done with the last item's sums long since.
            if (!ok || !wait_warp(&bars->sum_empty[i], (k & 1) ^ 1)) break;
            bars->sum[i][row] = make_float2(m == -INFINITY ? -INFINITY : m * c, l);
            if (row == 0) bars->any[i] = any;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->sum_full[i]);
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == MMA_WARP) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// Adds the parts of an item that was split over its keys, in their order: a
// warp takes kRows rows at once and kParts parts of each, whose loads are under way
// together. What the item is it works out itself: a CTA of window_kernel that gave up on a
// wait may have claimed items that it never reached, so nothing but numbers is taken from scratch.
constexpr int JOIN_WARPS = 8;
constexpr int join_blocks(int rows) { return 2 * ROWS / (JOIN_WARPS * rows); }
template <typename T, int kRows, int kParts>
__global__ void __launch_bounds__(32 * JOIN_WARPS) window_join_kernel(const __grid_constant__ WindowParams p) {
    const WindowAttnArgs &a = p.a;
    const int lane = threadIdx.x & 31;
    __shared__ Work w;
    // Before the wait: window_kernel let this grid start only after it had waited for its own
    // predecessors, so the sequences' starts are final (2 us of 216 for the chunks above).
    if (threadIdx.x < 32) {
        Item it;
        const bool found = find_item(p, blockIdx.x, it);   // its first part
        Work mine(p, it);
        if (!found) mine.parts = 0;
        if (lane == 0) w = mine;
    }
    grid_dependency_wait();
    grid_launch_dependents();
    __syncthreads();
    if (w.parts < 2) return;
    constexpr size_t NEXT = static_cast<size_t>(2 * ROWS) * SLOT_ROW;
    const int first = (blockIdx.y * JOIN_WARPS + (threadIdx.x >> 5)) * kRows;   // of the 256 rows of both tiles
    const float *slot = p.slots + (static_cast<size_t>(w.it.slot) * 2 * ROWS + first) * SLOT_ROW;
    float ref[kRows], l[kRows];
    float4 y[kRows];
    bool valid[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int i = (first + r) / ROWS;
        valid[r] = (first + r) % ROWS / p.group < (i == 0 ? w.tokens0 : w.tokens1);
        ref[r] = -INFINITY;
        l[r] = 0.0f;
        y[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int z0 = 0; z0 < w.parts; z0 += kParts) {
        float2 m[kParts][kRows];
        float4 v[kParts][kRows];
#pragma unroll
        for (int z = 0; z < kParts; ++z)
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const float *sp = slot + (z0 + z) * NEXT + r * SLOT_ROW;
                const bool have = valid[r] && z0 + z < w.parts;
                m[z][r] = have ? __ldcg(reinterpret_cast<const float2 *>(sp + 128)) : make_float2(-INFINITY, 0.0f);
                v[z][r] = have ? ld_in(reinterpret_cast<const float4 *>(sp) + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
        for (int z = 0; z < kParts; ++z)
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const float top = fmaxf(ref[r], m[z][r].x), base = top == -INFINITY ? 0.0f : top;
                const float e = exp2_approx(ref[r] - base), f = exp2_approx(m[z][r].x - base);
                ref[r] = top;
                l[r] = fmaf(m[z][r].y, f, l[r] * e);
                y[r].x = fmaf(v[z][r].x, f, y[r].x * e);
                y[r].y = fmaf(v[z][r].y, f, y[r].y * e);
                y[r].z = fmaf(v[z][r].z, f, y[r].z * e);
                y[r].w = fmaf(v[z][r].w, f, y[r].w * e);
            }
    }
    uint32_t again = 0;   // rows to mend
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        if (!valid[r]) continue;
        const int i = (first + r) / ROWS, row = (first + r) % ROWS, tok = row / p.group;
        const int h = w.it.kvh * p.group + row - tok * p.group, q_row = w.it.q0 + w.it.t0 + i * p.tokens + tok;
        const size_t out_row = static_cast<size_t>(q_row) * a.nheads + h;
        const float inv = l[r] == 0.0f ? 0.0f : 1.0f / l[r];
        store4(static_cast<T *>(a.out) + out_row * 128 + 4 * lane,
               make_float4(y[r].x * inv, y[r].y * inv, y[r].z * inv, y[r].w * inv));
        if (a.lse != nullptr && lane == 0) a.lse[out_row] = l[r] == 0.0f ? -INFINITY : (ref[r] + log2f(l[r])) * LN2;
        const float odd = (y[r].x * 0.0f + y[r].y * 0.0f) + (y[r].z * 0.0f + y[r].w * 0.0f);
        if (l[r] - l[r] == 0.0f && __any_sync(FULL_MASK, !(odd == 0.0f))) again |= 1u << r;
    }
#pragma unroll 1
    for (; again != 0u; again &= again - 1) {
        const int at = first + __ffs(again) - 1, i = at / ROWS, row = at % ROWS, tok = row / p.group;
        mend_row<T, 8, 4>(a, w.it.q0 + w.it.t0 + i * p.tokens + tok, w.it.kvh * p.group + row - tok * p.group, w.it.k0, w.it.nk,
                    (i == 0 ? w.pos0 : w.pos1) + tok);
    }
}

// [tokens][heads][128] 16-bit elements as boxes of 64 x heads x tokens, 128-byte swizzle.
bool encode_map(CUtensorMap *map, bool bf16, const void *p, int64_t heads, int64_t tokens, int64_t head_stride,
                int64_t token_stride, int box_heads, int box_tokens) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (enc == nullptr) return false;
    const cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
    // The stride of a dimension of one element is never used.
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(heads > 1 ? head_stride : 128) * 2u,
                                   static_cast<cuuint64_t>(tokens > 1 ? token_stride : 128) * 2u};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_tokens)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(p),
               dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A stride a tensor map takes (a multiple of 16 bytes below 2^40, not 0).
bool map_stride(int64_t n, int64_t elements) { return n <= 1 || (elements > 0 && elements < (1LL << 38)); }

// How the batch is cut, from what the host knows. Items are split over their
// keys when there are fewer than two per SM. Items that fill less than a quarter
// of the SMs: into equal parts of 4 key tiles at least, no more than run at once
// however the lengths fall. More items: into about two parts per SM that fall in
// size, the longer the more items there are, as what a split saves falls and the
// partial sums it moves grow with the items. Measured: 8 items of 123 tiles 32.0 us in
// parts for one per SM, 41.7 for two or three; 200 items of 55 to 128 tiles 216 us, in
// equal parts 234, whole 226; 250 items of 5 tiles 26 us whole and 50 in two parts; 28
// items of 12 tiles 20 us in equal parts of 4 tiles and 23 in falling ones of 6.
struct Split {
    int pairs, splits, part_tiles;
    bool falling;
};
Split split(int nseq, int total_q, int nheads, int nkv) {
    const int per = 2 * (ROWS / (nheads / nkv)), sms = device_sm_count();
    const int pairs = total_q / per + nseq;
    const long long least = static_cast<long long>(std::max(total_q / per, std::min(nseq, total_q))) * nkv;
    // The partial results are laid out for empty sequences too: no more than 8 parts per SM in all.
    const long long room = std::max(1LL, 8LL * sms / (static_cast<long long>(pairs) * nkv));
    const bool falling = 4 * least >= sms;
    const long long wanted = falling ? (2LL * sms + least - 1) / least
                                     : std::max(1LL, sms / (static_cast<long long>(pairs) * nkv));
    const int part_tiles = falling ? 4 + static_cast<int>(std::min(28LL, 16 * least / sms)) : 4;
    return {pairs, static_cast<int>(least >= 2LL * sms ? 1LL : std::min(std::min(wanted, room), 64LL)), part_tiles, falling};
}
size_t odd_bytes(int pairs, int nkv, int splits) { return (4 * sizeof(Odd) * pairs * nkv * splits + 15) / 16 * 16; }
// Parts of at least part_tiles tiles that a long item has.
int most_parts(const WindowAttnArgs &a, int tokens, int part_tiles) {
    // Lengths are not known here: twice the mean stands for the longest (a part may then be longer).
    long long keys = std::min<long long>(a.total_k, 2LL * ((static_cast<long long>(a.total_k) + a.nseq - 1) / a.nseq));
    if (a.window >= 0) keys = std::min(keys, static_cast<long long>(a.window) + std::min(a.sinks, a.total_k) + PIECE + 2 * tokens);
    const long long tiles = (keys + ROWS - 1) / ROWS;
    return static_cast<int>(std::max(1LL, std::min(64LL, (tiles + part_tiles - 1) / part_tiles)));
}

template <typename T>
cudaError_t launch(const WindowAttnArgs &a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const bool bf16 = a.dtype == QSA_BF16;
    const bool k_heads = a.nkv > 1 && a.k_head != 0, v_heads = a.nkv > 1 && a.v_head != 0;
    const bool maps = a.total_k > 0 && map_stride(a.nheads, a.q_head) && map_stride(a.total_q, a.q_tok) &&
                      map_stride(a.total_k, a.k_tok) && map_stride(a.total_k, a.v_tok) &&
                      map_stride(k_heads ? a.nkv : 1, a.k_head) && map_stride(v_heads ? a.nkv : 1, a.v_head);
    if (!maps) {
        cfg.gridDim = dim3((a.max_q + 7) / 8, a.nheads, a.nseq);
        cfg.blockDim = dim3(256);
        return cudaLaunchKernelEx(&cfg, window_rows_kernel<T>, a);
    }
    static thread_local int configured_device = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (configured_device != dev) {
        e = cudaFuncSetAttribute(window_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(WINDOW_SMEM));
        if (e != cudaSuccess) return e;
        configured_device = dev;
    }
    WindowParams p;
    memset(&p, 0, sizeof(p));
    p.a = a;
    p.group = a.nheads / a.nkv;
    p.tokens = ROWS / p.group;
    p.k_has_heads = k_heads;
    p.v_has_heads = v_heads;
    // The output warps wait for a whole item, 2 to 3.5 us a key tile: the limit is beside the work.
    p.wait_ns = wait_limit_ns() + 8192ull * ((a.total_k + static_cast<uint64_t>(ROWS) - 1) / ROWS);
    p.stall = (debug_inject() & 8u) != 0u;
    if (!encode_map(&p.q, bf16, a.q, a.nheads, a.total_q, a.q_head, a.q_tok, p.group, p.tokens) ||
        !encode_map(&p.k, bf16, a.k, k_heads ? a.nkv : 1, a.total_k, a.k_head, a.k_tok, 1, ROWS) ||
        !encode_map(&p.v, bf16, a.v, v_heads ? a.nkv : 1, a.total_k, a.v_head, a.v_tok, 1, ROWS))
        return cudaErrorNotSupported;
    if (a.sinks > 0 && (!encode_map(&p.k_piece, bf16, a.k, k_heads ? a.nkv : 1, a.total_k, a.k_head, a.k_tok, 1, PIECE) ||
                        !encode_map(&p.v_piece, bf16, a.v, v_heads ? a.nkv : 1, a.total_k, a.v_head, a.v_tok, 1, PIECE)))
        return cudaErrorNotSupported;
    const Split x = split(a.nseq, a.total_q, a.nheads, a.nkv);
    p.pairs = x.pairs;
    p.part_tiles = x.part_tiles;
    p.falling = x.falling;
    p.splits = std::min(x.splits, most_parts(a, p.tokens, x.part_tiles));
    p.per_split = make_divider(p.splits);
    p.per_part = make_divider(p.part_tiles);
    p.odd = static_cast<Odd *>(a.scratch);
    p.slots = reinterpret_cast<float *>(static_cast<char *>(a.scratch) + odd_bytes(p.pairs, a.nkv, p.splits));
    const long long items = static_cast<long long>(p.pairs) * a.nkv * p.splits;
    if (items > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    cfg.gridDim = dim3(static_cast<unsigned>(items));
    cfg.blockDim = dim3(WTHREADS);
    cfg.dynamicSmemBytes = WINDOW_SMEM;
    e = cudaLaunchKernelEx(&cfg, window_kernel<T>, p);
    if (e != cudaSuccess || p.splits == 1) return e;
    // Many parts are a long chain for a row, so a warp takes fewer rows and more parts of each at once
    // (38 parts an item 23.2 us against 34.8, 19 parts 32.6 against 40.3); few parts are many rows
    // (2 to 8 parts of 200 to 250 items 216 us against 220, 68.6 against 71.4; 3 parts 25.6 against 26.4).
    const bool many = p.splits > 8;
    cfg.gridDim = dim3(static_cast<unsigned>(p.pairs * a.nkv), many ? join_blocks(2) : join_blocks(4));
    cfg.blockDim = dim3(32 * JOIN_WARPS);
    cfg.dynamicSmemBytes = 0;
    return many ? cudaLaunchKernelEx(&cfg, window_join_kernel<T, 2, 4>, p) : cudaLaunchKernelEx(&cfg, window_join_kernel<T, 4, 2>, p);
}

}  // namespace

size_t window_attn_scratch_bytes(int nseq, int total_q, int nheads, int nkv) {
    if (nheads / nkv > ROWS) return 0;
    const Split x = split(nseq, total_q, nheads, nkv);
    return odd_bytes(x.pairs, nkv, x.splits) + (x.splits > 1 ? sizeof(float) * x.pairs * nkv * x.splits * 2 * ROWS * SLOT_ROW : 0);
}

cudaError_t launch_window_attn(const WindowAttnArgs &a, cudaStream_t stream) {
    return a.dtype == QSA_BF16 ? launch<__nv_bfloat16>(a, stream) : launch<__half>(a, stream);
}

cudaError_t window_error_read_clear(uint32_t *word, cudaStream_t stream) {
    cudaError_t e = cudaMemcpyFromSymbolAsync(word, g_window_error, sizeof(uint32_t), 0, cudaMemcpyDeviceToHost, stream);
    if (e != cudaSuccess) return e;
    e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return e;
    const uint32_t zero = 0u;
    e = cudaMemcpyToSymbolAsync(g_window_error, &zero, sizeof(uint32_t), 0, cudaMemcpyHostToDevice, stream);
    if (e != cudaSuccess) return e;
    return cudaStreamSynchronize(stream);
}

}  // namespace qsa
