// Attention of one new token per sequence over its paged cache, with a
// sliding window, always-visible first cells, and the weight each cell
// received added to a running mass.
//
//   x_hj = log2(e) scale q_h . k_j;  lse_h = ln 2 log2 sum_j 2^x_hj
//   out_h = sum_j 2^(x_hj - log2 sum) v_j;  mass_out_j = mass_j + sum_h 2^(x_hj - log2 sum)
//
// What bounds it: every visible cell of every KV head is read once and used
// by the few query heads that share it, so HBM.
//
// Work. The visible cells of a sequence, sinks first, are numbered without
// gaps and cut into tiles of 64 (int8: 128); (sequence, KV head, up to 8 or 16
// query heads) is a unit, and all tiles of all units in order are cut into one
// equal range per CTA, two CTAs per SM. Lengths live on the device only: every
// CTA sums the tile counts of all sequences itself, so ragged batches are
// balanced, a captured graph follows the lengths, and a single long sequence
// fills the GPU. A unit that falls into several ranges leaves partial results
// (outputs, maximum, sum per head) in scratch, which join_kernel adds in range
// order; the result does not depend on scheduling.
//
// A tile. Each of the 4 warps takes a quarter of the cells (8 KiB) and runs
// alone: its rows arrive in a ring of its own by 16-byte asynchronous copies
// (rows that do not exist are filled with zeros), two steps ahead and on over
// the units' boundaries; the page numbers are fetched one step before that.
// Both products run on mma.sync m16n8k16 with the heads as rows: x = Q K^T with
// rows 0-7 the heads and rows 8-15 the remainder of q where it has one, then
// P V with rows 0-7 the weights rounded to the operand type and rows 8-15 what
// that rounding left, so the weights carry 17 (bfloat16) or 22 (binary16) bits.
// The fragments of x are the fragments of P. tcgen05 would need 64 rows at
// least for the 1 to 16 heads that share a cell.
//
// int8 cells become binary16 exactly (a byte in the low bits of 1024 + u), q
// is scaled by a power of two per head into binary16's range, and the key
// scale multiplies x. The value scale vs_j joins the weight, and the running
// reference M of the exponent follows x_j + log2 vs_j, so that p_j vs_j =
// 2^(x_j - M) vs_j stays within binary16 whatever the scales' range.
// M moves only when it would have to grow by more than 2^8: the sums are
// scaled by whatever M they started from, and rescaling is rare.
//
// Measured (GB300): 64 ragged sequences of up to 8,192 bfloat16 cells, 8 KV heads
// of 4, 208 us, 6.1 TB/s (0.90 of the measured copy rate); 48 sequences of which
// 1,028 binary16 cells are visible, 46 us, 4.4 TB/s (the first 5 us bring the
// first cells, the ranges end within 4 us of one another, the join takes 2); 4
// sequences of up to 131,072 int8 cells, 2 KV heads, 52 us, 3.7 TB/s: about 850
// instructions per warp and 32 cells, the conversions to binary16 360 of them, at 43
// % of the issue slots with the 8 warps per SM that 245 registers leave (an earlier
// form with 12 warps of 168 registers was 4 % slower than its own with 8). One
// sequence of 700 cells 7.3 us on the device, launches and latencies: 0.7 us to find the
// range, 1.5 for the page and the cells, 1 for the products and the merge, the join.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "attn_row.cuh"
#include "cache_internal.cuh"
#include "qsa_internal.cuh"

namespace qsa {
namespace {

constexpr int WARPS = 4, THREADS = 32 * WARPS;
constexpr int TILE_16BIT = 64, TILE_INT8 = 128;   // cells of a tile
constexpr int CTAS_PER_SM = 2;
constexpr float LAZY = 8.0f;           // log2 of how far the sums may run above their reference
constexpr int SLOT_ROW = 132;          // 128 outputs, maximum, sum, padding

struct Params {
    PagedAttnArgs a;
    Divider page;
    int group;        // query heads per KV head
    int parts;        // units per KV head
    int units;        // units per sequence
    int capacity, stride;   // cells of a table row; columns of a row of kept logits
    float *slots;     // [2 grid][heads of a unit][SLOT_ROW]
    int by_unit;      // no more units than ranges: a place in meta is a unit, else a range
    int4 *meta;       // sequence, unit, first range, last range of the unit to join there, or -1
    float *lse2;      // [nseq][nheads], or null
    float *logits;    // [nseq][nheads][stride], or null
};

// The visible cells of a sequence, numbered without gaps.
struct Span {
    int n, sinks, shift;
    __device__ __forceinline__ int cell(int i) const { return i < sinks ? i : i + shift; }
};
__device__ __forceinline__ Span visible(const Params &p, int s) {
    const int len = min(max(ld_in(p.a.lens + s), 0), p.capacity);
    const int lo = p.a.window < 0 ? 0 : max(0, len - p.a.window);
    const int k = min(p.a.sinks, lo);
    return {k + len - lo, k, lo - k};
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(__cvta_generic_to_global(src)),
                 "r"(ok ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

// Operand type: bfloat16 for bfloat16 cells, binary16 for the others.
template <bool kBf16>
struct Op {
    static constexpr float LO = kBf16 ? 1.0f : 2048.0f;   // what remainders are multiplied by
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        if constexpr (kBf16) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
            return *reinterpret_cast<const uint32_t *>(&v);
        } else {
            const __half2 v = __floats2half2_rn(a, b);
            return *reinterpret_cast<const uint32_t *>(&v);
        }
    }
    static __device__ __forceinline__ float2 unpack(uint32_t w) {
        if constexpr (kBf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    }
    // a, b rounded to the type, and the (scaled) remainders of that.
    static __device__ __forceinline__ void split(float a, float b, uint32_t &hi, uint32_t &lo) {
        hi = pack(a, b);
        const float2 h = unpack(hi);
        lo = pack((a - h.x) * LO, (b - h.y) * LO);
    }
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        if constexpr (kBf16)
            asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                "{%0, %1, %2, %3};"
                : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
        else
            asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                "{%0, %1, %2, %3};"
                : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

// Bytes kSel picks from {lo word, hi word} (0x64 bytes come from the second operand), minus 1152: int8 -> binary16.
__device__ __forceinline__ uint32_t biased_to_half2(uint32_t w, uint32_t sel) {
    const uint32_t x = __byte_perm(w, 0x64646464u, sel);
    const __half2 v = __hsub2(*reinterpret_cast<const __half2 *>(&x), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t *>(&v);
}

template <int kKv>   // QSA_BF16, QSA_F16 or QSA_I8
struct Form {
    static constexpr bool kInt8 = kKv == QSA_I8;
    using O = Op<kKv == QSA_BF16>;
    static constexpr int STEP = kInt8 ? 32 : 16;           // cells of one warp's step: 8 KiB of keys and values
    static constexpr int TILE = STEP * WARPS;
    static_assert(TILE == (kInt8 ? TILE_INT8 : TILE_16BIT), "tile sizes");
    static constexpr int ROW = kInt8 ? 128 : 256;          // bytes of a cell's row
    // Rows 16 bytes apart from a multiple of 128: the fragment loads of both
    // products (ldmatrix, or 16-byte loads for int8) meet no bank twice.
    static constexpr int PITCH = ROW + 16;
    static constexpr int STAGES = 3;
    static constexpr int STAGE = 2 * STEP * PITCH;
    static constexpr int RING = STAGES * STAGE;            // one warp's ring
    static constexpr int SIDE = 8 * STEP + 16;             // a stage's scales (float ks, vs per cell) and cell mask
    static_assert(STAGE >= 16 * 128 * 4, "a stage holds a warp's outputs");
};

template <int kKv, int kMT>
constexpr int smem_bytes() {
    using F = Form<kKv>;
    return WARPS * F::RING + WARPS * F::STAGES * F::SIDE + 2 * WARPS * 8 * kMT * 4;
}

template <int kTile>
__device__ __forceinline__ int tiles_of(const Span &v) {
    return (v.n + kTile - 1) / kTile;
}

// A place in the CTA's range of tiles: tile t of unit u of sequence s.
template <int kTile>
struct Cursor {
    int s, u, t, nt;
    Span v;
    __device__ __forceinline__ void enter(const Params &p, int seq) {
        s = seq;
        v = visible(p, s);
        nt = tiles_of<kTile>(v);
    }
    // The next tile, which exists.
    __device__ __forceinline__ void next(const Params &p) {
        if (++t < nt) return;
        t = 0;
        if (++u < p.units) return;
        u = 0;
        do enter(p, s + 1);
        while (nt == 0);
    }
};

template <int kKv, typename QT, int kMT>
__global__ void __launch_bounds__(THREADS, CTAS_PER_SM) paged_kernel(const __grid_constant__ Params p) {
    using F = Form<kKv>;
    using O = typename F::O;
    constexpr bool kInt8 = F::kInt8;
    constexpr int STEP = F::STEP, TILE = F::TILE, STAGES = F::STAGES, ELEM = kInt8 ? 1 : 2;
    constexpr int HEADS_PER_UNIT = 8 * kMT;
    constexpr int GROUPS = STEP / 16;              // of 16 cells, whose weights are found together
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ long long sh_scan[WARPS];
    __shared__ int sh_seq, sh_unit, sh_tile;
    __shared__ Span sh_span;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = lane >> 2, t = lane & 3;
    const PagedAttnArgs &a = p.a;

    grid_dependency_wait();
    grid_launch_dependents();

    // ---- this CTA's range of tiles -------------------------------------------------
    const int each = (a.nseq + THREADS - 1) / THREADS;
    const int s0 = min(tid * each, a.nseq), s1 = min(s0 + each, a.nseq);
    long long mine = 0;
    Span first_span = {0, 0, 0};   // of s0: its length is read once
    for (int s = s0; s < s1; ++s) {
        const Span v = visible(p, s);
        if (s == s0) first_span = v;
        mine += tiles_of<TILE>(v);
    }
    const int own_n = blockIdx.x < a.nseq ? visible(p, blockIdx.x).n : 1;   // for the rows without a cell, below
    long long before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(FULL_MASK, before, o);
        if (lane >= o) before += y;
    }
    if (lane == 31) sh_scan[warp] = before;
    if (tid == 0) {
        sh_seq = -1;
        if (!p.by_unit) p.meta[blockIdx.x] = make_int4(-1, 0, 0, 0);
    }
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += sh_scan[w];
        total += sh_scan[w];
    }
    before -= mine;
    // Below 2^63: at most 65,535 sequences of 2^24 tiles times 65,535 units.
    const long long all = total * p.units;
    const long long per = (all + gridDim.x - 1) / gridDim.x;
    const long long x0 = per * blockIdx.x, x1 = min(x0 + per, all);
    // The tile that x0 is.
    if (x0 < x1 && x0 >= before * p.units && x0 < (before + mine) * p.units) {
        int s = s0;
        long long b = before;
        Span v = first_span;
        int n = tiles_of<TILE>(v);
        while (x0 >= (b + n) * p.units) {
            b += n;
            v = visible(p, ++s);
            n = tiles_of<TILE>(v);
        }
        const long long in_seq = x0 - b * p.units;
        sh_seq = s;
        sh_span = v;
        sh_unit = static_cast<int>(in_seq / n);
        sh_tile = static_cast<int>(in_seq % n);
    }
    // Sequences without a visible cell have no tile: their rows are written here.
    for (int s = blockIdx.x; s < a.nseq; s += gridDim.x) {
        if ((s == blockIdx.x ? own_n : visible(p, s).n) > 0) continue;
        for (int e = tid; e < a.nheads * 32; e += THREADS)
            store4(static_cast<QT *>(a.out) + static_cast<size_t>(s) * a.nheads * 128 + 4 * e, make_float4(0.f, 0.f, 0.f, 0.f));
        for (int h = tid; h < a.nheads; h += THREADS) {
            if (a.lse != nullptr) a.lse[static_cast<size_t>(s) * a.nheads + h] = -INFINITY;
            if (p.lse2 != nullptr) p.lse2[static_cast<size_t>(s) * a.nheads + h] = -INFINITY;
        }
        if (p.by_unit)
            for (int u = tid; u < p.units; u += THREADS) p.meta[s * p.units + u] = make_int4(-1, 0, 0, 0);
    }
    __syncthreads();
    if (sh_seq < 0) return;

    unsigned char *side_base = smem + WARPS * F::RING;
    float *merge_m = reinterpret_cast<float *>(side_base + WARPS * F::STAGES * F::SIDE);
    float *merge_l = merge_m + WARPS * HEADS_PER_UNIT;
    const uint32_t ring = smem_u32(smem + warp * F::RING);
    unsigned char *side = side_base + warp * F::STAGES * F::SIDE;
    const float c = a.scale * LOG2E;
    const int steps = static_cast<int>(x1 - x0);   // of every warp: 16 or 32 cells of each tile

    // ---- copies, which run ahead over the units without a stop ----------------------
    const int row = lane & (STEP - 1);             // the row whose address this lane finds
    Cursor<TILE> at;                               // the step whose page is fetched next
    at.s = sh_seq;
    at.v = sh_span;
    at.nt = tiles_of<TILE>(at.v);
    at.u = sh_unit;
    at.t = sh_tile;
    Cursor<TILE> here = at;                        // the step that is computed
    struct Place {                                 // of this lane's row: the page, and the rest of its address
        int page;
        long long rest, scale_rest;
    } place = {-1, 0, 0};                          // for the step to copy next
    auto fetch = [&](int step) {
        if (step >= steps) return;
        if (step > 0) at.next(p);
        const int i = at.t * TILE + warp * STEP + row;
        place.page = -1;
        if (i < at.v.n) {
            const int j = at.v.cell(i), pg = static_cast<int>(divide(p.page, j)), in_page = j - pg * a.kv.page_size;
            place.page = ld_in(a.table + at.s * a.table_stride + pg);
            const int kvh = p.parts == 1 ? at.u : at.u / p.parts;
            place.rest = in_page * a.kv.cell_stride + kvh * a.kv.head_stride;
            if constexpr (kInt8) place.scale_rest = in_page * a.kv.scale_cell_stride + kvh * a.kv.scale_head_stride;
        }
    };
    uint16_t key_scale = 0, value_scale = 0;       // this lane's row's of the newest step
    auto issue = [&](int step) {
        if (step < steps) {
            const int slot_at = step % STAGES;
            const int page = place.page;
            const bool ok = page >= 0 && page < a.kv.npages;
            const long long off = ok ? (page * a.kv.page_stride + place.rest) * ELEM : 0;
            const uint32_t mask = __ballot_sync(FULL_MASK, ok);
            if (lane == 0) *reinterpret_cast<uint32_t *>(side + slot_at * F::SIDE + 8 * STEP) = mask;
            if constexpr (kInt8) {
                const long long so = ok ? page * a.kv.scale_page_stride + place.scale_rest : 0;
                key_scale = ok ? ld_in_u16(a.kv.k_scale_f16 + so) : 0;
                value_scale = ok ? ld_in_u16(a.kv.v_scale_f16 + so) : 0;
            }
            constexpr int LANES = F::ROW / 16, ROWS = 32 / LANES;
            const int chunk = 16 * (lane % LANES), first = lane / LANES;
            const uint32_t dst = ring + slot_at * F::STAGE + first * F::PITCH + chunk;
            const char *k = static_cast<const char *>(a.kv.k) + chunk, *v = static_cast<const char *>(a.kv.v) + chunk;
#pragma unroll
            for (int b = 0; b < STEP / ROWS; ++b) {
                const long long ro = __shfl_sync(FULL_MASK, off, b * ROWS + first);
                const bool rok = (mask >> (b * ROWS + first)) & 1u;
                cp_async_16_or_zero(dst + b * ROWS * F::PITCH, k + ro, rok);
                cp_async_16_or_zero(dst + (STEP + b * ROWS) * F::PITCH, v + ro, rok);
            }
        }
        cp_async_commit();
    };
    auto put_scale = [&](int step) {
        if constexpr (kInt8)
            if (step < steps)
                *reinterpret_cast<float2 *>(side + (step % STAGES) * F::SIDE + 8 * row) =
                    make_float2(__half2float(__ushort_as_half(key_scale)), __half2float(__ushort_as_half(value_scale)));
    };
    {   // Both pages, both steps' cells and scales: no load waits for the other step's.
        static_assert(STAGES == 3, "two steps ahead");
        fetch(0);
        const Place first = place;
        fetch(1);
        const Place second = place;
        place = first;
        issue(0);
        const uint16_t first_key_scale = key_scale, first_value_scale = value_scale;
        place = second;
        issue(1);
        fetch(2);
        const uint16_t second_key_scale = key_scale, second_value_scale = value_scale;
        key_scale = first_key_scale;
        value_scale = first_value_scale;
        put_scale(0);
        key_scale = second_key_scale;
        value_scale = second_value_scale;
    }

    // ---- units ------------------------------------------------------------------------
    // The queries of unit `here`, as they lie: d = 32 t + 4 k + {0, 1, 2, 3} of step k for int8
    // cells, else d = 16 k + 2 t + {0, 1} and + 8.
    using Raw = typename std::conditional<kInt8, float4, uint2>::type;
    Raw raw_q[kMT][8];
    auto load_q = [&]() {
        const int kvh = here.u / p.parts, h0 = kvh * p.group + (here.u % p.parts) * HEADS_PER_UNIT;
        const int nh = (kvh + 1) * p.group - h0;
#pragma unroll
        for (int m = 0; m < kMT; ++m) {
            const bool have = 8 * m + r < nh;
            const QT *qp = static_cast<const QT *>(a.q) + here.s * a.q_seq_stride + (h0 + (have ? 8 * m + r : 0)) * a.q_head_stride;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if constexpr (kInt8) {
                    raw_q[m][k] = have ? load4(qp + 32 * t + 4 * k) : make_float4(0.f, 0.f, 0.f, 0.f);
                } else {
                    raw_q[m][k].x = have ? ld_in(reinterpret_cast<const uint32_t *>(qp + 16 * k + 2 * t)) : 0u;
                    raw_q[m][k].y = have ? ld_in(reinterpret_cast<const uint32_t *>(qp + 16 * k + 2 * t + 8)) : 0u;
                }
            }
        }
    };
    constexpr bool AHEAD = kMT == 1;   // the registers for 16 heads' queries are not there
    if (AHEAD) load_q();
    for (int step = 0; step < steps;) {
        if (!AHEAD) load_q();
        const int s = here.s, u = here.u, t0 = here.t, t1 = min(here.nt, t0 + steps - step), nt = here.nt;
        const int kvh = u / p.parts, h0 = kvh * p.group + (u % p.parts) * HEADS_PER_UNIT;
        const int nh = min(HEADS_PER_UNIT, (kvh + 1) * p.group - h0);
        const bool begins = step == 0;

        // Query fragments: head r of each 8 in rows 0-7, remainders in rows 8-15.
        uint32_t qa[kMT][8][kInt8 ? 4 : 2];
        float qc[kMT];   // what a product is multiplied by to become x
#pragma unroll
        for (int m = 0; m < kMT; ++m) {
            qc[m] = c;
            if constexpr (kInt8) {
                float top = 0.0f;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    top = fmaxf(top, fmaxf(fmaxf(fabsf(raw_q[m][k].x), fabsf(raw_q[m][k].y)),
                                           fmaxf(fabsf(raw_q[m][k].z), fabsf(raw_q[m][k].w))));
                top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, 1));
                top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, 2));
                int ex = 0;
                if (top > 0.0f && top < INFINITY) frexpf(top, &ex);
                ex = max(-126, min(127, ex));   // both powers are fp32 numbers
                const float down = ldexpf(1.0f, -ex);
                qc[m] = c * ldexpf(1.0f, ex);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    O::split(raw_q[m][k].x * down, raw_q[m][k].y * down, qa[m][k][0], qa[m][k][1]);
                    O::split(raw_q[m][k].z * down, raw_q[m][k].w * down, qa[m][k][2], qa[m][k][3]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    qa[m][k][0] = raw_q[m][k].x;
                    qa[m][k][1] = raw_q[m][k].y;
                }
            }
        }

        float o[kMT][16][4];
        float ref[kMT], sum[kMT];
#pragma unroll
        for (int m = 0; m < kMT; ++m) {
            ref[m] = -INFINITY;
            sum[m] = 0.0f;
#pragma unroll
            for (int n = 0; n < 16; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[m][n][e] = 0.0f;
        }

#pragma unroll 1
        for (int tile = t0; tile < t1; ++tile, ++step) {
            put_scale(step + STAGES - 2);
            cp_async_wait<STAGES - 2>();
            __syncwarp();
            issue(step + STAGES - 1);
            fetch(step + STAGES);
            const unsigned char *sd = side + (step % STAGES) * F::SIDE;
            const uint32_t mask = *reinterpret_cast<const uint32_t *>(sd + 8 * STEP);
            if (mask == 0u && p.logits == nullptr) continue;
            const uint32_t kb = ring + (step % STAGES) * F::STAGE, vb = kb + STEP * F::PITCH;
            // x of heads (row r) by cells 16 g + 2 t, + 1, + 8, + 9
            float sc[kMT][2 * GROUPS][4];
#pragma unroll
            for (int m = 0; m < kMT; ++m)
#pragma unroll
                for (int n = 0; n < 2 * GROUPS; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[m][n][e] = 0.0f;
            float ks[4 * GROUPS], vs[4 * GROUPS];
            if constexpr (kInt8) {
#pragma unroll
                for (int n = 0; n < 2 * GROUPS; ++n) {
                    const float4 f = *reinterpret_cast<const float4 *>(sd + 8 * (8 * n + 2 * t));
                    ks[2 * n] = f.x;
                    vs[2 * n] = f.y;
                    ks[2 * n + 1] = f.z;
                    vs[2 * n + 1] = f.w;
                }
#pragma unroll
                for (int n = 0; n < 2 * GROUPS; ++n) {
                    const uint32_t at_k = kb + (8 * n + r) * F::PITCH + 32 * t;
                    const uint4 w0 = ld_shared_v4(at_k), w1 = ld_shared_v4(at_k + 16);
                    const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t z = w[k] ^ 0x80808080u;
                        const uint32_t b0 = biased_to_half2(z, 0x4140), b1 = biased_to_half2(z, 0x4342);
#pragma unroll
                        for (int m = 0; m < kMT; ++m) O::mma(sc[m][n], qa[m][k], b0, b1);
                    }
                }
            } else {
                // matrices: cells 0-7 and 8-15 by d 0-7 and 8-15 of step k
                const uint32_t at_k = kb + ((lane & 7) + 8 * (lane >> 4)) * F::PITCH + 16 * ((lane >> 3) & 1);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    uint32_t b[4];
                    ldmatrix4(b, at_k + 32 * k);
#pragma unroll
                    for (int m = 0; m < kMT; ++m) {
                        const uint32_t qf[4] = {qa[m][k][0], 0u, qa[m][k][1], 0u};
                        O::mma(sc[m][0], qf, b[0], b[1]);
                        O::mma(sc[m][1], qf, b[2], b[3]);
                    }
                }
            }
            uint32_t pa[kMT][GROUPS][4];
#pragma unroll
            for (int m = 0; m < kMT; ++m) {
                float xx[4 * GROUPS], top = -INFINITY;
#pragma unroll
                for (int n = 0; n < 2 * GROUPS; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float y = sc[m][n][e];
                        if constexpr (kInt8) y = fmaf(sc[m][n][2 + e], 1.0f / O::LO, y) * ks[2 * n + e];
                        y *= qc[m];
                        if (!((mask >> (8 * n + 2 * t + e)) & 1u)) y = -INFINITY;
                        xx[2 * n + e] = y;
                        float z = y;
                        if constexpr (kInt8) z += __log2f(fmaxf(fabsf(vs[2 * n + e]), 5.9604645e-8f));
                        top = fmaxf(top, z);
                    }
                if (p.logits != nullptr && 8 * m + r < nh) {
                    float *lp = p.logits + (static_cast<size_t>(s) * a.nheads + h0 + 8 * m + r) * p.stride +
                                tile * TILE + warp * STEP + 2 * t;
#pragma unroll
                    for (int n = 0; n < 2 * GROUPS; ++n)
                        *reinterpret_cast<float2 *>(lp + 8 * n) = make_float2(xx[2 * n], xx[2 * n + 1]);
                }
                top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, 1));
                top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, 2));
                bool move = top > ref[m] + LAZY || (ref[m] == -INFINITY && top > -INFINITY);
                if (__any_sync(FULL_MASK, move)) {
                    if constexpr (kInt8)
                        // An infinite value scale must not become the reference, which the sum of weights needs finite:
                        // it counts as binary16's largest number.
                        if (__any_sync(FULL_MASK, top == INFINITY)) {
                            top = -INFINITY;
#pragma unroll
                            for (int n = 0; n < 4 * GROUPS; ++n)
                                top = fmaxf(top, xx[n] + __log2f(fminf(fmaxf(fabsf(vs[n]), 5.9604645e-8f), 65504.0f)));
                            top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, 1));
                            top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, 2));
                            move = top > ref[m] + LAZY || (ref[m] == -INFINITY && top > -INFINITY);
                        }
                    const float f = move ? ex2(ref[m] - top) : 1.0f;
                    if (move) ref[m] = top;
                    sum[m] *= f;
#pragma unroll
                    for (int n = 0; n < 16; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[m][n][e] *= f;
                }
                const float base = ref[m] == -INFINITY ? 0.0f : ref[m];
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) {
                    float w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        w[e] = ex2(xx[4 * g + e] - base);
                        sum[m] += w[e];
                        if constexpr (kInt8) w[e] *= vs[4 * g + e];
                    }
                    O::split(w[0], w[1], pa[m][g][0], pa[m][g][1]);
                    O::split(w[2], w[3], pa[m][g][2], pa[m][g][3]);
                }
            }
#pragma unroll
            for (int gg = 0; gg < GROUPS; ++gg) {
                const uint32_t vg = vb + 16 * gg * F::PITCH;
                if constexpr (kInt8) {
                    // This thread's cells 2 t, 2 t + 1, 2 t + 8, 2 t + 9; column r of product n is d = 16 r + n.
                    uint4 cw[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) cw[e] = ld_shared_v4(vg + (2 * t + (e & 1) + 8 * (e >> 1)) * F::PITCH + 16 * r);
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        uint32_t lo[2], hi[2];   // cells (2t, 2t+1) and (2t+8, 2t+9): d 0, 1 and d 2, 3 of the word
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t w0 = reinterpret_cast<const uint32_t *>(&cw[2 * e])[g] ^ 0x80808080u;
                            const uint32_t w1 = reinterpret_cast<const uint32_t *>(&cw[2 * e + 1])[g] ^ 0x80808080u;
                            lo[e] = __byte_perm(w0, w1, 0x5140);
                            hi[e] = __byte_perm(w0, w1, 0x7362);
                        }
#pragma unroll
                        for (int d = 0; d < 4; ++d) {
                            const uint32_t sel = (d & 1) ? 0x4342 : 0x4140;
                            const uint32_t b0 = biased_to_half2(d < 2 ? lo[0] : hi[0], sel);
                            const uint32_t b1 = biased_to_half2(d < 2 ? lo[1] : hi[1], sel);
#pragma unroll
                            for (int m = 0; m < kMT; ++m) O::mma(o[m][4 * g + d], pa[m][gg], b0, b1);
                        }
                    }
                } else {
                    // matrices: cells 0-7, 8-15 by d 16 n .. + 7, then d 16 n + 8 .. + 15
                    const uint32_t at_v = vg + (lane & 15) * F::PITCH + 16 * (lane >> 4);
#pragma unroll
                    for (int n = 0; n < 8; ++n) {
                        uint32_t b[4];
                        ldmatrix4_t(b, at_v + 32 * n);
#pragma unroll
                        for (int m = 0; m < kMT; ++m) {
                            O::mma(o[m][2 * n], pa[m][gg], b[0], b[1]);
                            O::mma(o[m][2 * n + 1], pa[m][gg], b[2], b[3]);
                        }
                    }
                }
            }
        }

        // ---- join the warps, in warp order, through the stage each has just used ----------
        __syncwarp();
        const int used = (step - 1) % STAGES;
#pragma unroll
        for (int m = 0; m < kMT; ++m) {
            sum[m] += __shfl_xor_sync(FULL_MASK, sum[m], 1);
            sum[m] += __shfl_xor_sync(FULL_MASK, sum[m], 2);
            if (t == 0) {
                merge_m[warp * HEADS_PER_UNIT + 8 * m + r] = ref[m];
                merge_l[warp * HEADS_PER_UNIT + 8 * m + r] = sum[m];
            }
            float *mo = reinterpret_cast<float *>(smem + warp * F::RING + used * F::STAGE) + (8 * m + r) * 128;
#pragma unroll
            for (int n = 0; n < 16; ++n) {
                const float y0 = fmaf(o[m][n][2], 1.0f / O::LO, o[m][n][0]), y1 = fmaf(o[m][n][3], 1.0f / O::LO, o[m][n][1]);
                if constexpr (kInt8) {
                    mo[32 * t + n] = y0;
                    mo[32 * t + 16 + n] = y1;
                } else {
                    *reinterpret_cast<float2 *>(mo + 8 * n + 2 * t) = make_float2(y0, y1);
                }
            }
        }
        if (step < steps) {   // the next unit's queries come while this one's results leave
            here.t = here.nt - 1;
            here.next(p);
            if (AHEAD) load_q();
        }
        __syncthreads();
        const bool whole = t0 == 0 && t1 == nt;
        const int slot = 2 * blockIdx.x + (begins ? 0 : 1);
        for (int h = warp; h < nh; h += WARPS) {
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) top = fmaxf(top, merge_m[w * HEADS_PER_UNIT + h]);
            const float base = top == -INFINITY ? 0.0f : top;
            float l = 0.0f;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const int hw = w * HEADS_PER_UNIT + h;
                const float f = ex2(merge_m[hw] - base);
                l = fmaf(merge_l[hw], f, l);
                const float4 z = *reinterpret_cast<const float4 *>(smem + w * F::RING + used * F::STAGE + (h * 128 + 4 * lane) * 4);
                y.x = fmaf(z.x, f, y.x);
                y.y = fmaf(z.y, f, y.y);
                y.z = fmaf(z.z, f, y.z);
                y.w = fmaf(z.w, f, y.w);
            }
            if (whole) {
                const size_t out_row = static_cast<size_t>(s) * a.nheads + h0 + h;
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                store4(static_cast<QT *>(a.out) + out_row * 128 + 4 * lane, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
                if (lane == 0) {
                    const float e = l == 0.0f ? -INFINITY : top + log2f(l);
                    if (a.lse != nullptr) a.lse[out_row] = e * LN2;
                    if (p.lse2 != nullptr) p.lse2[out_row] = e;
                }
            } else {
                float *sp = p.slots + (static_cast<size_t>(slot) * HEADS_PER_UNIT + h) * SLOT_ROW;
                *reinterpret_cast<float4 *>(sp + 4 * lane) = y;
                if (lane == 0) {
                    sp[128] = top;
                    sp[129] = l;
                }
            }
        }
        // A unit of several ranges is written down for the join by the second of them (by_unit: the
        // place is the unit's own, and every unit has one writer).
        if (tid == 0) {
            int4 *at_unit = p.meta + (p.by_unit ? s * p.units + u : blockIdx.x);
            const long long unit0 = x0 - t0;
            if (whole) {
                if (p.by_unit) *at_unit = make_int4(-1, 0, 0, 0);
            } else if (begins && t0 > 0 && unit0 / per == blockIdx.x - 1) {
                *at_unit = make_int4(s, u, static_cast<int>(unit0 / per) * 2 + (unit0 % per == 0 ? 0 : 1),
                                     static_cast<int>((unit0 + nt - 1) / per));
            }
        }
        __syncthreads();   // the stages are free again
    }
}

// Adds the partial results of one unit's ranges for one head: of W warps, warp w
// takes every W-th range from w on, then the warps are added in order. W is 1
// where a unit has about as many ranges as a warp loads at once, 4 up to 16
// ranges, else 16 (measured, whole call: 2 ranges a unit 45.9 us with 1 warp, 49.8 with
// 4; 11 ranges 7.6 and 7.25; 39 ranges 54.1 with 4, 51.4 with 16; about 300 ranges 15.9
// and 14.0). The ranges are taken from the grid, which goes by the table's width: lengths
// are on the device alone. Short caches on a wide table have fewer ranges than it says.
constexpr int JOIN_WARPS = 16, JOIN_BATCH = 8;
template <typename QT>
__global__ void __launch_bounds__(32 * JOIN_WARPS) join_kernel(const __grid_constant__ Params p, int heads_per_unit) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int4 w = __ldcg(p.meta + blockIdx.x);
    if (w.x < 0) return;
    const PagedAttnArgs &a = p.a;
    const int s = w.x, kvh = w.y / p.parts, h0 = kvh * p.group + (w.y % p.parts) * heads_per_unit;
    const int h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    if (h0 + h >= (kvh + 1) * p.group) return;
    const int c0 = w.z >> 1, n = w.w - c0 + 1;
    auto slot = [&](int i) {   // the unit's first range may be its CTA's second segment
        return p.slots + (static_cast<size_t>(i == 0 ? w.z : 2 * (c0 + i)) * heads_per_unit + h) * SLOT_ROW;
    };
    __shared__ float4 sum[JOIN_WARPS][32];
    __shared__ float weight[JOIN_WARPS];
    // The warp's first ranges come along with all ranges' maxima.
    float2 ml[JOIN_BATCH];
    float4 v[JOIN_BATCH];
    auto load = [&](int i0) {
#pragma unroll
        for (int b = 0; b < JOIN_BATCH; ++b) {
            const int i = i0 + warps * b;
            ml[b] = make_float2(-INFINITY, 0.0f);
            v[b] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < n) {
                ml[b] = __ldcg(reinterpret_cast<const float2 *>(slot(i) + 128));
                v[b] = ld_in(reinterpret_cast<const float4 *>(slot(i)) + lane);
            }
        }
    };
    load(warp);
    float top = -INFINITY;
    for (int i = threadIdx.x; i < n; i += blockDim.x) top = fmaxf(top, __ldcg(slot(i) + 128));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, o));
    if (warps > 1) {
        if (lane == 0) weight[warp] = top;
        __syncthreads();
        top = lane < warps ? weight[lane] : -INFINITY;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, o));
        __syncthreads();   // the place takes the warps' sums next
    }
    const float base = top == -INFINITY ? 0.0f : top;
    float l = 0.0f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = warp; i0 < n; i0 += warps * JOIN_BATCH) {
        if (i0 != warp) load(i0);
#pragma unroll
        for (int b = 0; b < JOIN_BATCH; ++b) {
            const float f = ex2(ml[b].x - base);
            l = fmaf(ml[b].y, f, l);
            y.x = fmaf(v[b].x, f, y.x);
            y.y = fmaf(v[b].y, f, y.y);
            y.z = fmaf(v[b].z, f, y.z);
            y.w = fmaf(v[b].w, f, y.w);
        }
    }
    sum[warp][lane] = y;
    if (lane == 0) weight[warp] = l;
    __syncthreads();
    if (warp > 0) return;
    for (int o = 1; o < warps; ++o) {
        const float4 z = sum[o][lane];
        y.x += z.x;
        y.y += z.y;
        y.z += z.z;
        y.w += z.w;
        l += weight[o];
    }
    const size_t row = static_cast<size_t>(s) * a.nheads + h0 + h;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    store4(static_cast<QT *>(a.out) + row * 128 + 4 * lane, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
    if (lane == 0) {
        const float e = l == 0.0f ? -INFINITY : top + log2f(l);
        if (a.lse != nullptr) a.lse[row] = e * LN2;
        if (p.lse2 != nullptr) p.lse2[row] = e;
    }
}

// mass_out = mass + sum over the heads of the weights of the kept logits. A
// block takes 256 cells, 4 per thread, and 4 groups of threads every fourth
// head each, added in order. Cells that are not visible keep their mass.
constexpr int MASS_CELLS = 256, MASS_GROUPS = 4;
__global__ void __launch_bounds__(MASS_CELLS) mass_kernel(const __grid_constant__ Params p) {
    grid_dependency_wait();
    grid_launch_dependents();
    __shared__ float4 part[MASS_GROUPS - 1][MASS_CELLS / 4];
    const PagedAttnArgs &a = p.a;
    const int s = blockIdx.y, quad = threadIdx.x % (MASS_CELLS / 4), group = threadIdx.x / (MASS_CELLS / 4);
    const Span v = visible(p, s);
    const float *mass = a.mass + s * a.mass_stride;
    float *out = a.mass_out + s * a.mass_stride;
    const float *lse = p.lse2 + static_cast<size_t>(s) * a.nheads;
    for (int i0 = blockIdx.x * MASS_CELLS; i0 < v.n; i0 += gridDim.x * MASS_CELLS) {
        const int i = i0 + 4 * quad;
        float4 got = make_float4(0.f, 0.f, 0.f, 0.f);
        float old[4];   // on its way with the logits
        if (group == 0)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i + k < v.n) old[k] = __ldcg(mass + v.cell(i + k));
        if (i < v.n) {
            const float *lp = p.logits + static_cast<size_t>(s) * a.nheads * p.stride + i;
#pragma unroll 8
            for (int h = group; h < a.nheads; h += MASS_GROUPS) {
                const float e = __ldcg(lse + h);
                const float4 x = ld_in(reinterpret_cast<const float4 *>(lp + static_cast<size_t>(h) * p.stride));
                const float base = e == -INFINITY ? INFINITY : e;   // no visible cell: weight 0
                got.x += ex2(x.x - base);
                got.y += ex2(x.y - base);
                got.z += ex2(x.z - base);
                got.w += ex2(x.w - base);
            }
        }
        if (group > 0) part[group - 1][quad] = got;
        __syncthreads();
        if (group == 0 && i < v.n) {
#pragma unroll
            for (int g = 0; g < MASS_GROUPS - 1; ++g) {
                const float4 z = part[g][quad];
                got.x += z.x;
                got.y += z.y;
                got.z += z.z;
                got.w += z.w;
            }
            const float add[4] = {got.x, got.y, got.z, got.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i + k < v.n) out[v.cell(i + k)] = old[k] + add[k];
        }
        __syncthreads();
    }
    if (out != mass)
        for (int j = v.sinks + blockIdx.x * MASS_CELLS + threadIdx.x; j < v.sinks + v.shift; j += gridDim.x * MASS_CELLS)
            out[j] = __ldcg(mass + j);
}

struct Layout {
    size_t meta, slots, lse2, logits, bytes;
    int heads_per_unit, grid, stride;
};
// A unit of 16 heads reads its cells once where two of 8 read them twice, but its
// steps are slower (255 registers, 116 bytes of them spilled to local memory; no queries ahead,
// and the 16 outputs' merges). It pays for 16-bit cells that do not stay in L2 for the second
// reading: 16 heads on a KV head, bfloat16, 8 x 16,384 cells of 8 KV heads 122 us against 174,
// 64 x 8,192 cells of one 73 against 94, but 16 x 8,192 cells of one 32.8 against 28.5. The rule has only
// the table's width to go by: where the sequences fill less of it, it can choose 16 for
// cells that would stay (87 of 100 to 800 cells, 4 KV heads of 12: 45 us against 40). There is no
// unit of 16 for int8 cells, whose 8 heads' registers leave no room (one that was tried lost a quarter).
constexpr long long L2_BYTES = 128LL << 20;
int heads_per_unit(int nseq, int group, int nkv, int capacity, bool int8) {
    return group > 8 && !int8 && 512LL * nseq * capacity * nkv > L2_BYTES ? 16 : 8;
}
// The scratch is laid out for 16 heads whenever there are as many, whatever the cells' type.
Layout layout(int nseq, int nheads, int nkv, int capacity, bool with_mass) {
    Layout y;
    const int group = nheads / nkv;
    y.heads_per_unit = group <= 8 ? 8 : 16;
    const long long parts = (group + 7) / 8;
    const long long tiles = (static_cast<long long>(capacity) + TILE_16BIT - 1) / TILE_16BIT * nkv * parts * nseq;
    y.grid = static_cast<int>(std::max(1LL, std::min<long long>(static_cast<long long>(CTAS_PER_SM) * device_sm_count(), tiles)));
    y.stride = (capacity + TILE_INT8 - 1) / TILE_INT8 * TILE_INT8;
    size_t at = 0;
    y.meta = at;
    at += sizeof(int4) * y.grid;
    y.slots = at;
    at += sizeof(float) * 2 * y.grid * y.heads_per_unit * SLOT_ROW;
    y.lse2 = at;
    if (with_mass) at += (sizeof(float) * nseq * static_cast<size_t>(nheads) + 15) / 16 * 16;
    y.logits = at;
    if (with_mass) at += sizeof(float) * nseq * static_cast<size_t>(nheads) * y.stride;
    y.bytes = at;
    return y;
}

// Launches as a programmatic dependent of the previous grid on the stream.
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int kKv, typename QT, int kMT>
cudaError_t run(const Params &p, int grid, cudaStream_t stream) {
    constexpr int smem = smem_bytes<kKv, kMT>();
    auto kernel = paged_kernel<kKv, QT, kMT>;
    static thread_local int configured_device = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && configured_device != dev) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess) configured_device = dev;
    }
    if (e == cudaSuccess) e = launch(kernel, dim3(grid), THREADS, smem, stream, p);
    const int ranges = static_cast<int>(grid / (static_cast<long long>(p.a.nseq) * p.units)) + 1;   // of a unit, on average
    const int join_threads = 32 * (ranges <= 4 ? 1 : ranges <= 16 ? 4 : JOIN_WARPS);
    const int places = p.by_unit ? p.a.nseq * p.units : grid;
    if (e == cudaSuccess) e = launch(join_kernel<QT>, dim3(places, std::min(p.group, 8 * kMT)), join_threads, 0, stream, p, 8 * kMT);
    if (e == cudaSuccess && p.logits != nullptr)
        e = launch(mass_kernel, dim3(std::min((p.stride + MASS_CELLS - 1) / MASS_CELLS, 512), p.a.nseq), MASS_CELLS, 0, stream, p);
    return e;
}

}  // namespace

size_t paged_attn_scratch_bytes(int nseq, int nheads, int nkv, int capacity, bool with_mass) {
    return layout(nseq, nheads, nkv, capacity, with_mass).bytes;
}

cudaError_t launch_paged_attn(const PagedAttnArgs &a, cudaStream_t stream) {
    Params p;
    p.a = a;
    p.capacity = a.table_cols * a.kv.page_size;
    const Layout y = layout(a.nseq, a.nheads, a.kv.nkv, p.capacity, a.mass != nullptr);
    p.page = make_divider(a.kv.page_size);
    p.group = a.nheads / a.kv.nkv;
    const bool int8 = a.kv.dtype == QSA_I8;
    const int heads = heads_per_unit(a.nseq, p.group, a.kv.nkv, p.capacity, int8);
    p.parts = (p.group + heads - 1) / heads;
    p.units = a.kv.nkv * p.parts;
    p.stride = y.stride;
    p.by_unit = static_cast<long long>(a.nseq) * p.units <= y.grid;
    char *b = static_cast<char *>(a.scratch);
    p.meta = reinterpret_cast<int4 *>(b + y.meta);
    p.slots = reinterpret_cast<float *>(b + y.slots);
    p.lse2 = a.mass != nullptr ? reinterpret_cast<float *>(b + y.lse2) : nullptr;
    p.logits = a.mass != nullptr && p.capacity > 0 ? reinterpret_cast<float *>(b + y.logits) : nullptr;
    if (a.kv.dtype == QSA_BF16)
        return heads == 8 ? run<QSA_BF16, __nv_bfloat16, 1>(p, y.grid, stream) : run<QSA_BF16, __nv_bfloat16, 2>(p, y.grid, stream);
    if (a.kv.dtype == QSA_F16) return heads == 8 ? run<QSA_F16, __half, 1>(p, y.grid, stream) : run<QSA_F16, __half, 2>(p, y.grid, stream);
    if (a.q_dtype == QSA_F32) return run<QSA_I8, float, 1>(p, y.grid, stream);
    if (a.q_dtype == QSA_F16) return run<QSA_I8, __half, 1>(p, y.grid, stream);
    return run<QSA_I8, __nv_bfloat16, 1>(p, y.grid, stream);
}

}  // namespace qsa
