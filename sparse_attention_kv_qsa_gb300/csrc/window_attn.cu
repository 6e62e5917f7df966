// Prompt attention over ragged sequences: causal, within a sliding window,
// with the first tokens (sinks) always visible.
//
//   visible(i, j): j <= pos_i and (window < 0 or j > pos_i - window or j < sinks),  pos_i = nk - nq + i
//   s_ij = scale q_i . k_j;  lse_i = log sum_j exp(s_ij);  out_i = sum_j exp(s_ij - lse_i) v_j
//
// window_kernel, tensor cores (tcgen05). A work item is one KV head and two
// query tiles of 128 rows of one sequence; a tile's rows are consecutive
// tokens times the query heads that share the KV head, so heads of a group
// share every key tile and a narrow window wastes little. 10 warps: 4 softmax
// warps per query tile (a thread owns a row), one that issues the MMAs, one
// that issues the tensor copies.
//
//   S = Q K^T   both from shared memory (128-byte swizzle), into TMEM
//   P           2^(c S - c m), c = scale log2(e): registers, rounded once to the
//               inputs' type, back to TMEM over S
//   O += P V    P from TMEM, V from shared memory as stored (keys by d, the
//               d-contiguous operand form), into TMEM
//
// The two query tiles alternate: while one tile's softmax runs, the tensor
// cores run the other's P V and the next S. The running maximum m is a lazy
// reference: O is rescaled only when a row's maximum grew by more than 2^8
// (weights then reach 2^8, whose relative rounding is the same).
//
// The keys that an item's rows see are the sinks and one contiguous range.
// They are numbered without a gap (sinks rounded up to 16 rows, the extra rows
// masked), so a few sinks do not cost a tile of their own: the tile that
// holds both parts is copied in pieces of 16 rows.
//
// Rows that are not visible get weight 0, but 0 times an infinity or NaN in
// such a row's values would reach the sums. A row whose sums are not finite
// is therefore computed again from its visible keys alone (attend_row, also
// the whole path for strides that a tensor map cannot express).
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
constexpr int STAGES = 5;                   // key and value tiles in flight
constexpr int PIECE = 16;                   // rows of a copy in the tile where sinks and window meet
constexpr int MMA_WARP = 8, COPY_WARP = 9, WTHREADS = 320;
constexpr float LAZY = 8.0f;
constexpr uint32_t S_COL = 0, O_COL = 256, TMEM_COLS = 512;

struct WindowParams {
    CUtensorMap q, k, v, k_piece, v_piece;
    WindowAttnArgs a;
    int group, tokens;      // query heads per KV head; tokens of a query tile
    int k_has_heads, v_has_heads;   // 0: all KV heads at one address
    uint64_t wait_ns;
};

struct WindowBarriers {
    uint64_t q_full[2], kv_full[STAGES], kv_empty[STAGES], s_full[2], p_full[2], o_full[2], drain;
    uint32_t tmem, abort;
};
constexpr size_t WINDOW_SMEM = 1024 + (2 + STAGES) * static_cast<size_t>(TILE_BYTES) + sizeof(WindowBarriers);
static_assert(WINDOW_SMEM <= 232448, "shared memory per CTA");

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

// One row by one warp in fp32.
template <typename T>
__device__ void attend_row(const WindowAttnArgs &a, int q_row, int h, int k0, int nk, int pos) {
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
    store4(static_cast<T *>(a.out) + row * 128 + 4 * lane, r.result());
    if (a.lse != nullptr && lane == 0) a.lse[row] = (r.m + log2f(r.l)) * LN2;
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
    if (i < x.nq) attend_row<T>(a, x.q0 + i, blockIdx.y, x.k0, x.nk, x.nk - x.nq + i);
}

// An item's keys, numbered without gaps: numbers below `front` are keys
// 0 .. front-1 (front = the sinks rounded up to whole pieces), number i from
// there on is key i - front + lo. Row limits are in these numbers.
struct ItemKeys {
    int front, lo, count;
    int sink_end;            // numbers below it are sinks of every row
    int window, nk;
    __device__ __forceinline__ ItemKeys(const WindowAttnArgs &a, int nk_, int pos_first, int pos_last) {
        nk = nk_;
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
    // Does any row between these places see a key of tile j?
    __device__ __forceinline__ bool needed(int j, int pos_a, int pos_b) const {
        const int i = j * ROWS;
        return i <= last(pos_b) && (i < sink_end || i + ROWS - 1 >= first(pos_a));
    }
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

template <typename T>
__global__ void __launch_bounds__(WTHREADS, 1) window_kernel(const __grid_constant__ WindowParams p) {
    extern __shared__ unsigned char raw[];
    const WindowAttnArgs &a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t ring = base + 2 * TILE_BYTES;
    WindowBarriers *bars = reinterpret_cast<WindowBarriers *>(raw + (base - smem_u32(raw)) + (2 + STAGES) * TILE_BYTES);

    grid_dependency_wait();
    grid_launch_dependents();

    const int kvh = blockIdx.x % a.nkv, h0 = kvh * p.group;
    const Sequence x = sequence(a, blockIdx.y);
    const int t0 = static_cast<int>((gridDim.x - 1 - blockIdx.x) / a.nkv) * 2 * p.tokens;   // longest rows first
    if (t0 >= x.nq) return;
    const int shift = x.nk - x.nq;                                // pos = shift + token
    const int tokens0 = min(p.tokens, x.nq - t0), tokens1 = min(p.tokens, max(0, x.nq - t0 - p.tokens));
    const int pos0 = shift + t0, pos1 = pos0 + p.tokens;          // first rows of the two tiles
    const ItemKeys keys(a, x.nk, pos0, pos0 + tokens0 + tokens1 - 1);
    const int ntiles = keys.tiles();
    auto needed = [&](int i, int j) {
        return i == 0 ? keys.needed(j, pos0, pos0 + tokens0 - 1)
                      : tokens1 > 0 && keys.needed(j, pos1, pos1 + tokens1 - 1);
    };

    if (warp == MMA_WARP) {
        tmem_alloc(&bars->tmem, TMEM_COLS);
        tmem_relinquish();
    } else if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->q_full[i], 1);
            mbar_init(&bars->s_full[i], 1);
            mbar_init(&bars->p_full[i], 4);
            mbar_init(&bars->o_full[i], 1);
        }
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&bars->kv_full[i], 1);
            mbar_init(&bars->kv_empty[i], 1);
        }
        mbar_init(&bars->drain, 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = bars->tmem;

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

    if (warp == COPY_WARP) {
        if (lane == 0) {
            const uint32_t q_bytes = 2u * 128u * p.group * p.tokens;
            for (int i = 0; i < (tokens1 > 0 ? 2 : 1); ++i) {
                mbar_arrive_expect_tx(&bars->q_full[i], q_bytes);
                for (int half = 0; half < 2; ++half)
                    tma_load_3d(base + i * TILE_BYTES + half * HALF, &p.q, 64 * half, h0, x.q0 + t0 + i * p.tokens,
                                &bars->q_full[i]);
            }
            int n = 0;   // copies begun: tile n / 2, keys then values
            for (; n < 2 * ntiles; ++n) {
                const int slot = n % STAGES, j = n >> 1, i0 = j * ROWS;
                if (!wait(&bars->kv_empty[slot], ((n / STAGES) & 1) ^ 1)) break;
                uint64_t *bar = &bars->kv_full[slot];
                const uint32_t dst = ring + slot * TILE_BYTES;
                const int head = (n & 1) ? (p.v_has_heads ? kvh : 0) : (p.k_has_heads ? kvh : 0);
                mbar_arrive_expect_tx(bar, TILE_BYTES);
                if (i0 < keys.front && i0 + ROWS > keys.front) {
                    const CUtensorMap *map = (n & 1) ? &p.v_piece : &p.k_piece;
                    for (int r = 0; r < ROWS; r += PIECE) {
                        const int key = i0 + r < keys.front ? i0 + r : i0 + r - keys.front + keys.lo;
                        for (int half = 0; half < 2; ++half)
                            tma_load_3d(dst + half * HALF + r * 128, map, 64 * half, head, x.k0 + key, bar);
                    }
                } else {
                    const CUtensorMap *map = (n & 1) ? &p.v : &p.k;
                    const int key = i0 < keys.front ? i0 : i0 - keys.front + keys.lo;
                    for (int half = 0; half < 2; ++half)
                        tma_load_3d(dst + half * HALF, map, 64 * half, head, x.k0 + key, bar);
                }
            }
            // Copies begun here land before the CTA leaves (at once without an abort).
            for (int d = max(0, n - STAGES); d < n; ++d) mbar_wait(&bars->kv_full[d % STAGES], (d / STAGES) & 1, p.wait_ns);
            for (int i = 0; i < (tokens1 > 0 ? 2 : 1); ++i) mbar_wait(&bars->q_full[i], 0, p.wait_ns);
        }
        __syncwarp();
    } else if (warp == MMA_WARP) {
        if (lane == 0) {
            constexpr uint32_t fmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
            constexpr uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
            constexpr uint32_t idesc_v = idesc | (1u << 16);   // second operand contiguous in N
            bool ok = true;
            bool pending[2] = {false, false};
            int np[2] = {0, 0};
            // Step j: each tile's P V of its last S, then its S of key tile j.
            for (int j = 0; ok && j <= ntiles; ++j) {
                const int kn = 2 * j;
                // Every copy is waited for, also one that no row needs: its slot is reused after this step.
                if (j < ntiles) ok = wait(&bars->kv_full[kn % STAGES], (kn / STAGES) & 1);
                if (ok && j > 0) ok = wait(&bars->kv_full[(kn - 1) % STAGES], ((kn - 1) / STAGES) & 1);
                for (int i = 0; ok && i < 2; ++i) {
                    const uint32_t s_col = tmem + S_COL + 128 * i, o_col = tmem + O_COL + 128 * i;
                    if (pending[i]) {
                        const int vn = kn - 1;
                        ok = wait(&bars->p_full[i], (np[i] - 1) & 1);
                        if (!ok) break;
                        tc_fence_after_sync();
                        const uint64_t vd = sw128_mnmajor_desc(ring + (vn % STAGES) * TILE_BYTES, HALF);
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            tc_mma_bf16_ta(o_col, s_col + 8 * kk, vd + 128 * kk, idesc_v, (np[i] > 1 || kk > 0) ? 1u : 0u);
                        pending[i] = false;
                    }
                    if (j < ntiles && needed(i, j)) {
                        if (np[i] == 0) ok = wait(&bars->q_full[i], 0);
                        if (!ok) break;
                        tc_fence_after_sync();
                        const uint64_t qd = sw128_kmajor_desc(base + i * TILE_BYTES);
                        const uint64_t kd = sw128_kmajor_desc(ring + (kn % STAGES) * TILE_BYTES);
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) {
                            const uint64_t step = (kk >> 2) * (HALF >> 4) + 2 * (kk & 3);
                            tc_mma_bf16(s_col, qd + step, kd + step, idesc, kk > 0 ? 1u : 0u);
                        }
                        tc_commit(&bars->s_full[i]);
                        pending[i] = true;
                        ++np[i];
                    }
                }
                if (!ok) break;
                // Tile j's keys and tile j-1's values are free when all of this is done.
                if (j > 0) tc_commit(&bars->kv_empty[(kn - 1) % STAGES]);
                if (j < ntiles) tc_commit(&bars->kv_empty[kn % STAGES]);
            }
            if (ok)
                for (int i = 0; i < 2; ++i) tc_commit(&bars->o_full[i]);
            tc_commit(&bars->drain);
            mbar_wait(&bars->drain, 0, p.wait_ns);
        }
        __syncwarp();
    } else {
        // ---- softmax of one query tile, one row per thread -----------------------------
        const int i = warp >> 2, row = 32 * (warp & 3) + lane;
        const int tok = row / p.group, head = row - tok * p.group;
        const int ntok = i == 0 ? tokens0 : tokens1;
        const bool valid = tok < ntok;
        const int pos = (i == 0 ? pos0 : pos1) + min(tok, max(ntok - 1, 0));
        const int last = keys.last(pos), first = keys.first(pos);
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t s_at = tmem + lanes + S_COL + 128 * i, o_at = tmem + lanes + O_COL + 128 * i;
        const float c = a.scale * LOG2E;
        float m = -INFINITY, l = 0.0f;   // m: of the products, before c
        int n = 0;
        bool ok = true;
        for (int j = 0; j < ntiles; ++j) {
            if (!needed(i, j)) continue;
            ok = __all_sync(FULL_MASK, wait(&bars->s_full[i], n & 1));
            if (!ok) break;
            tc_fence_after_sync();
            uint32_t sr[4][32];
#pragma unroll
            for (int g = 0; g < 4; ++g) tmem_ld32(s_at + 32 * g, sr[g]);
            tmem_ld_wait();
            const int i0 = j * ROWS;
            const bool open = i0 + ROWS - 1 <= last && (i0 >= first || i0 + ROWS <= keys.sink_end);
            if (!__all_sync(FULL_MASK, open)) {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    auto below = [&](int limit) {   // bits of the numbers i0 + 32 g + bit < limit
                        const int k = limit - (i0 + 32 * g);
                        return k <= 0 ? 0u : k >= 32 ? 0xFFFFFFFFu : (1u << k) - 1u;
                    };
                    const uint32_t bits = below(last + 1) & (below(keys.sink_end) | ~below(first));
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!((bits >> e) & 1u)) sr[g][e] = 0xFF800000u;
                }
            }
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
            if (__any_sync(FULL_MASK, move)) {
                const float f = move ? exp2_approx((m - top) * c) : 1.0f;
                if (move) m = top;
                l *= f;
                if (n > 0) {
#pragma unroll 1
                    for (int g = 0; g < 4; ++g) {
                        uint32_t o[32];
                        tmem_ld32(o_at + 32 * g, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st32(o_at + 32 * g, o);
                    }
                }
            }
            const float mc = m == -INFINITY ? 0.0f : m * c;
            const uint64_t c2 = pair(c, c), mc2 = pair(-mc, -mc);
            uint64_t sums[4] = {0, 0, 0, 0};
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                uint32_t pw[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    float x0, x1;
                    unpair(fma_pair(pair(__uint_as_float(sr[2 * g + (e >> 4)][(2 * e) & 31]),
                                         __uint_as_float(sr[2 * g + (e >> 4)][(2 * e + 1) & 31])), c2, mc2), x0, x1);
                    x0 = exp2_approx(x0);
                    x1 = exp2_approx(x1);
                    sums[e & 3] = add_pair(sums[e & 3], pair(x0, x1));
                    pw[e] = pack2_rn<T>(x0, x1);
                }
                tmem_st32(s_at + 32 * g, pw);
            }
            {
                float y0, y1;
                unpair(add_pair(add_pair(sums[0], sums[1]), add_pair(sums[2], sums[3])), y0, y1);
                l += y0 + y1;
            }
            tmem_st_wait();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->p_full[i]);
            ++n;
        }
        // ---- results -------------------------------------------------------------------
        if (ok) ok = __all_sync(FULL_MASK, wait(&bars->o_full[i], 0));
        if (ok && ntok > 0) {
            tc_fence_after_sync();
            const int q_row = x.q0 + t0 + i * p.tokens + tok, h = h0 + head;
            const size_t out_row = static_cast<size_t>(q_row) * a.nheads + h;
            uint4 *out = reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + out_row * 128);
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            float odd = 0.0f;   // stays 0 while everything is finite
#pragma unroll 1
            for (int g = 0; g < 4; ++g) {
                uint32_t o[32];
                if (n > 0) {
                    tmem_ld32(o_at + 32 * g, o);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0u;
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) odd = fmaf(__uint_as_float(o[e]), 0.0f, odd);
                if (valid) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            w[k] = pack2_rn<T>(__uint_as_float(o[8 * e + 2 * k]) * inv, __uint_as_float(o[8 * e + 2 * k + 1]) * inv);
                        out[4 * g + e] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            if (valid && a.lse != nullptr) a.lse[out_row] = l == 0.0f ? -INFINITY : (m * c + log2f(l)) * LN2;
            uint32_t again = __ballot_sync(FULL_MASK, valid && !(odd * l == 0.0f));
            while (again != 0u) {   // the row's visible keys alone
                const int from = __ffs(again) - 1;
                again &= again - 1;
                __syncwarp();
                attend_row<T>(a, __shfl_sync(FULL_MASK, q_row, from), __shfl_sync(FULL_MASK, h, from), x.k0, x.nk,
                              __shfl_sync(FULL_MASK, pos, from));
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == MMA_WARP) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, TMEM_COLS);
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
    p.wait_ns = wait_limit_ns();
    if (!encode_map(&p.q, bf16, a.q, a.nheads, a.total_q, a.q_head, a.q_tok, p.group, p.tokens) ||
        !encode_map(&p.k, bf16, a.k, k_heads ? a.nkv : 1, a.total_k, a.k_head, a.k_tok, 1, ROWS) ||
        !encode_map(&p.v, bf16, a.v, v_heads ? a.nkv : 1, a.total_k, a.v_head, a.v_tok, 1, ROWS))
        return cudaErrorNotSupported;
    if (a.sinks > 0 && (!encode_map(&p.k_piece, bf16, a.k, k_heads ? a.nkv : 1, a.total_k, a.k_head, a.k_tok, 1, PIECE) ||
                        !encode_map(&p.v_piece, bf16, a.v, v_heads ? a.nkv : 1, a.total_k, a.v_head, a.v_tok, 1, PIECE)))
        return cudaErrorNotSupported;
    const long long items = (static_cast<long long>(a.max_q) + 2 * p.tokens - 1) / (2 * p.tokens) * a.nkv;
    if (items > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    cfg.gridDim = dim3(static_cast<unsigned>(items), a.nseq);
    cfg.blockDim = dim3(WTHREADS);
    cfg.dynamicSmemBytes = WINDOW_SMEM;
    return cudaLaunchKernelEx(&cfg, window_kernel<T>, p);
}

}  // namespace

size_t window_attn_scratch_bytes(int, int, int, int, int) { return 0; }

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
