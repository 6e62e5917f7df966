// Attention of one new token per sequence where groups of sequences share a
// long prefix: the prefix's pages are read once for all of a group.
//
//   x_hj = log2(e) scale q_h . k_j  over the group's prefix cells, then the sequence's own cells
//   lse_h = ln 2 log2 sum_j 2^x_hj;  out_h = sum_j 2^(x_hj - log2 sum) v_j
//
// What bounds it: the prefix's cells are read once per block of rows, from HBM
// or L2 (512 bytes a 16-bit cell and KV head), and cost 4 x 128 flops for
// every row, a row being a sequence times a query head of the KV head. Below some 290
// rows that is HBM, above it the tensor cores.
//
// Three launches: prefix_kernel (this file) leaves each row's partial sums over the
// prefix, paged attention's kernel those over its own cells (it starts
// as the first one's CTAs end), and prefix_join_kernel adds them.
//
// prefix_kernel (tcgen05). A block is up to two tiles of 128 rows of one group and KV
// head; block by block, the tiles of 128 prefix cells are numbered over the batch
// and cut into one equal range per CTA, one CTA per SM, so that any lengths and
// group sizes fill the GPU. Lengths live on the device: every CTA finds its range
// itself. 16 warps:
//
//   8 softmax warps   two streams of four, a thread owns a row
//   1 MMA warp        all tcgen05.mma
//   1 warp            walks the range and publishes its segments (a block's part in this CTA)
//   4 copy warps      cells by 16-byte asynchronous copies, each row from its own page (any page
//                     size), into 128-byte-swizzled tiles; int8 cells become binary16 on the way (and
//                     the queries beside them, by the softmax warps)
//
// Two streams of softmax keep the tensor cores fed: with more than 128 rows
// each takes a tile of rows, and both use every tile of cells; with fewer, both have the
// same rows and take the tiles of cells in turn, and are added at the segment's end.
// All rows of a block see the same cells, so there are no masks but the last
// tile's end and pages that are none; those rows arrive as zeros.
//
// fp32 queries (int8 cells): a row's query is scaled by a power of two and held as a
// binary16 number and what that left of it, another; so are its weights. Both
// halves' products go to the same sums, the second halves being within binary16's
// range as they are: the queries' largest is 2^13 at least, the weights' 2^7, and what
// falls below its smallest number is 2^-32 of that or less. A block is one row tile then, its
// two query tiles the halves.
//
// Measured (GB300, in a CUDA graph, all three launches): 32 sequences of 32 heads on 8 KV heads behind 65,536 bfloat16
// cells 65.5 us, 46 of them streaming at 5.8 TB/s; 64 behind 4,096, up to 1,024 cells of their own, 46.2 us (floor 24.5,
// mostly own cells); 512 of 16 heads on 2 behind 8,192 binary16 cells 59.0 us: a tile of cells for two row tiles takes
// 1.95 us, the tensor cores 1.1 of that, because a tile's weights (1.4 us), its products and the next scores
// follow one another. 40 fp32 sequences of 8 heads on 2 behind 3 texts of up to 65,536 int8 cells 62 us, 2 us a
// tile and 7 for sums put aside. 4 behind 600 cells 13.3 us: launches, and code that comes for the first time.
#include <algorithm>
#include <cfloat>
#include <cstring>
#include <type_traits>

#include "attn_row.cuh"
#include "cache_internal.cuh"
#include "prefix_share.cuh"
#include "qsa_internal.cuh"

namespace qsa {
namespace {

__device__ uint32_t g_prefix_error;

constexpr int ROWS = 128;                   // rows of a row tile, cells of a cell tile
constexpr int HALF = ROWS * 128;            // bytes of 128 rows x 64 elements
constexpr int TILE_BYTES = 2 * HALF;
constexpr int MMA_WARP = 8, WALK_WARP = 9, COPY_WARP = 12, COPY_WARPS = 4, PTHREADS = 512;
// 128 registers a thread at launch: 8 softmax warps x 168 + 8 x 88 = 16 x 128.
constexpr int MORE_REGISTERS = 168, FEW_REGISTERS = 88;
constexpr int BLOCK = 2 * ROWS;             // rows of a block at most
constexpr int OWN_ROW = 132;                // paged attention's partial results: 128 sums, reference, weights' sum, padding
constexpr float LAZY = 8.0f;                // log2 of how far the sums may run above their reference
constexpr int SEGS = 4, SIDES = 4;
constexpr uint32_t S_COL = 0, O_COL = 256, TMEM_COLS = 512;

template <int kKv, typename QT>
struct Form {
    static constexpr bool kInt8 = kKv == QSA_I8;
    static constexpr bool kSplit = std::is_same<QT, float>::value;
    using T = typename std::conditional<kKv == QSA_BF16, __nv_bfloat16, __half>::type;   // operands
    static constexpr int TILES = kSplit ? 1 : 2;         // row tiles of a block at most
    static constexpr int STAGES = kInt8 ? 3 : 5;         // tiles of keys or values
    static constexpr int RAW = kInt8 ? 3 : 0;            // int8 tiles on their way
    // Arrivals that make a tile complete: of every copying thread's copies, or of the warps that converted it.
    static constexpr int COPIES = kInt8 ? COPY_WARPS : 32 * COPY_WARPS;
    // Weights are kept 2^7 above their reference where the operand is binary16, whose smallest
    // numbers they would otherwise reach sooner: 2^(8 + 7) is within its range.
    static constexpr float LIFT = kKv == QSA_BF16 ? 0.0f : 7.0f;
    // Tiles that one sum in tensor memory takes: the tensor cores cut a sum off at every step of 16 cells, always towards
    // zero, so that its error grows with its length. Then it is put aside in scratch, and added there as rounded fp32 numbers.
    // 16 bits: 262,144 cells around 1 in one sum were 6e-4 too small, in sums of 32,768 8e-5, a fraction of the result's
    // rounding. fp32 queries (two halves, 16 steps a tile; relative error against 64 bits, the plain form's in 32 bits in
    // brackets): 512 sequences of 64 heads on 8 behind 4,096 cells 4.3e-6 in sums of 16 tiles, 1.6e-6 of 4, 1.3e-6 of 3,
    // 1.1e-6 of 2 (1.5e-6); 500 behind 1,000 1.3e-6 of 4, 1.1e-6 of 3, 0.92e-6 of 2 (0.95e-6); 2 of 20 heads on 4 behind 26,317
    // 1.36e-6 of 3, 1.12e-6 of 2 (0.94e-6). 40 sequences behind 3 texts took 54.8 us with sums of 16 tiles, 59.8 with 4, 60.2 with 3
    // and 62 with 2; 60 of 64 heads behind 30,000 148.6, 158.6, 163.9 and 172.6.
    static constexpr int CHAIN = kSplit ? 2 : 256;
};

struct Params {
    PrefixAttnArgs a;
    Divider page;
    PrefixShare share;
    int group, seqs, block;   // query heads per KV head; sequences of a row tile, and of a block
    int own_tile;             // cells of paged attention's tile
    // Partial results: sums as sums_at() says, and reference and weights' sum of each row.
    float4 *slots, *whole;    // [2 grid][BLOCK x 32]: a segment at a CTA's begin, and its last; [nkv][whole_rows x 32]
    float2 *slot_refs, *whole_refs;
    int whole_rows;           // of blocks that fall into one CTA, at whole_row()
    int2 *meta;               // [blocks][nkv]: first slot, last CTA; -1 where whole
    int2 *places;             // [nseq]: a sequence's block and its first sequence; -1 without a prefix
    uint64_t wait_ns;
    int stall;                // diagnostics only: CTA 0 never signals its first key tile
};

using Group = PrefixGroup;
__device__ __forceinline__ Group group_of(const Params &p, int g) { return prefix_group(p.share, g); }
// Block b of group g, among all.
__device__ __forceinline__ int block_number(const Params &p, const Group &x, int g, int b) { return x.first / p.block + g + b; }
// First row of a whole block's partial results (of a KV head): a multiple of 8, and behind the rows of the blocks before it.
__device__ __forceinline__ int whole_row(const Params &p, int block, int first) { return ((first * p.group + 7) / 8 + block) * 8; }
// Columns 4 chunk .. + 3 of a row, in 16-byte pieces: 8 rows' pieces are a line, so that a warp whose lanes
// have a row each and one that takes 8 rows by 4 pieces both move whole lines.
__device__ __forceinline__ size_t sums_at(int row, int chunk) { return static_cast<size_t>(row >> 3) * 256 + chunk * 8 + (row & 7); }

// A block's part in this CTA.
struct Segment {
    int g, kvh, first, count;   // count: sequences of the block, 0 at the range's end
    int len, t0, t1;            // cells of the prefix; tiles of cells
    int slot;                   // of the partial results, -1: whole
    int row;                    // of them, where whole
};

struct alignas(16) Bars {
    uint4 mask[SIDES];          // cells of a tile that are there
    Segment seg[SEGS];
    uint64_t seg_full[SEGS], seg_empty[SEGS], q_full, q_empty, kv_full[5], kv_empty[5], s_full[2], p_half[2], p_full[2];
    uint64_t o_full[2], side_full[SIDES], side_empty[SIDES], pair[4], drain;
    uint32_t tmem, abort;
};
struct alignas(16) Scales {                 // of int8 cells
    float key[SIDES][ROWS], value[SIDES][ROWS], log_value[SIDES][ROWS];
    float row[2 * ROWS];        // what a row's products are multiplied by
};
template <int kKv, typename QT>
constexpr size_t smem_bytes() {
    using F = Form<kKv, QT>;
    return 1024 + (2 + F::STAGES) * static_cast<size_t>(TILE_BYTES) + F::RAW * (TILE_BYTES / 2) + sizeof(Bars) +
           (F::kInt8 ? sizeof(Scales) : 0);
}
static_assert(smem_bytes<QSA_BF16, __nv_bfloat16>() <= 232448 && smem_bytes<QSA_I8, float>() <= 232448, "shared memory per CTA");

__device__ __forceinline__ float ex2(float x) {
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
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
template <typename T>
__device__ __forceinline__ uint32_t pack(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack<__half>(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
// a, b as binary16 numbers, and what that left of them.
__device__ __forceinline__ void split(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = pack<__half>(a, b);
    const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    lo = pack<__half>(a - h.x, b - h.y);
}
// Bytes `sel` picks of a word of int8 codes xored with 0x80, as binary16: 0x64 above a byte u is 1024 + u.
__device__ __forceinline__ uint32_t codes_to_half2(uint32_t w, uint32_t sel) {
    const uint32_t x = __byte_perm(w, 0x64646464u, sel);
    const __half2 v = __hsub2(*reinterpret_cast<const __half2 *>(&x), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(__cvta_generic_to_global(src)),
                 "r"(ok ? 16 : 0)
                 : "memory");
}
// Arrives once on `bar`, which counts this thread already, when its copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Waits until at most n (0 to 2) of this thread's most recent groups are pending.
__device__ __forceinline__ void cp_async_wait_at_most(int n) {
    if (n <= 0) cp_async_wait<0>();
    else if (n == 1) cp_async_wait<1>();
    else cp_async_wait<2>();
}
__device__ __forceinline__ void arrive(uint64_t *bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}
__device__ __forceinline__ long long quotient(long long a, long long b) {   // neither is negative
    return ((a | b) >> 32) == 0 ? static_cast<long long>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}
__device__ __forceinline__ long long sum_of_warp(long long x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(FULL_MASK, x, o);
    return x;
}
template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// 32 consecutive fp32 columns of this thread's TMEM lane, there when it returns: load and wait are one
// statement, because registers that a load is still to write may be copied between two.
__device__ __forceinline__ void tmem_read32(uint32_t taddr, uint32_t (&r)[32]) {
    __syncwarp();
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
// 16-byte chunk c (of 16) of row r of a tile: two halves of 64 elements, 128-byte rows, chunks swizzled.
__device__ __forceinline__ uint32_t tile_at(int r, int c) { return (c >> 3) * HALF + r * 128 + (((c & 7) ^ (r & 7)) << 4); }

// Which of a segment's 2 n copies tile j's keys and values are: in the order in which the products use them.
// int8 tiles and segments of two row tiles: keys and values in turn; else keys 0, keys 1, values 0, keys 2, values 1, ..
__device__ __forceinline__ int key_item(bool turn, int j) { return turn ? 2 * j : max(0, 2 * j - 1); }
__device__ __forceinline__ int value_item(bool turn, int j, int n) { return turn ? 2 * j + 1 : min(2 * j + 2, 2 * n - 1); }

template <int kKv, typename QT>
__global__ void __launch_bounds__(PTHREADS, 1) prefix_kernel(const __grid_constant__ Params p) {
    using F = Form<kKv, QT>;
    using T = typename F::T;
    constexpr bool kInt8 = F::kInt8, kSplit = F::kSplit;
    constexpr int STAGES = F::STAGES;
    extern __shared__ unsigned char raw_smem[];
    __shared__ long long sh_scan[PTHREADS / 32 - MMA_WARP], sh_work[PTHREADS / 32 - MMA_WARP], sh_own[PTHREADS / 32 - MMA_WARP];
    __shared__ Group sh_at;                     // the group that the range begins in
    __shared__ int sh_group, sh_kvh, sh_block, sh_tile;
    const PrefixAttnArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(FULL_MASK, tid >> 5, 0);   // the same for the warp, as the compiler now knows
    const uint32_t base = (smem_u32(raw_smem) + 1023u) & ~1023u;
    const uint32_t ring = base + 2 * TILE_BYTES, raws = ring + STAGES * TILE_BYTES;
    Bars *bars = reinterpret_cast<Bars *>(raw_smem + (raws + F::RAW * (TILE_BYTES / 2) - smem_u32(raw_smem)));
    Scales *scales = reinterpret_cast<Scales *>(bars + 1);   // int8 cells only

    if (warp == MMA_WARP) {
        tmem_alloc(&bars->tmem, TMEM_COLS);
        tmem_relinquish();
    } else if (tid == 0) {
        for (int i = 0; i < SEGS; ++i) {
            mbar_init(&bars->seg_full[i], 1);
            mbar_init(&bars->seg_empty[i], 1 + 8 + COPY_WARPS);
        }
        mbar_init(&bars->q_full, kInt8 ? 8 : F::COPIES);
        mbar_init(&bars->q_empty, 8);
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&bars->kv_full[i], F::COPIES);
            mbar_init(&bars->kv_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->s_full[i], 1);
            mbar_init(&bars->p_half[i], 4);
            mbar_init(&bars->p_full[i], 4);
            mbar_init(&bars->o_full[i], 1);
        }
        for (int i = 0; i < SIDES; ++i) {
            mbar_init(&bars->side_full[i], COPY_WARPS);
            mbar_init(&bars->side_empty[i], 8);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&bars->pair[i], 2);
        mbar_init(&bars->drain, 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = bars->tmem;
    long long per = 0, x1 = 0, range = 0;           // tiles of a CTA, the range's end and length (not in softmax warps)
    grid_dependency_wait();
    grid_launch_dependents();
    if (warp >= MMA_WARP) {
        // ---- this CTA's range of tiles -------------------------------------------------
        constexpr int FINDERS = PTHREADS - 32 * MMA_WARP;
        const int me = tid - 32 * MMA_WARP, each = (a.ngroups + FINDERS - 1) / FINDERS;
        const int g0 = min(me * each, a.ngroups), g1 = min(g0 + each, a.ngroups);
        long long mine = 0, work = 0, own = 0;
        Group own_group = {};                       // the last of this thread's, read once where it is the only one
        for (int g = g0; g < g1; ++g) {
            own_group = group_of(p, g);
            mine += prefix_tiles(p.share, own_group);
            work += prefix_work(p.share, own_group);
        }
        const int capacity = a.table_cols * a.kv.page_size;
        for (int s = me; s < a.nseq && !p.share.whole; s += FINDERS) own += (min(max(ld_in(a.lens + s), 0), capacity) + p.own_tile - 1) / p.own_tile;
        long long before = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(FULL_MASK, before, o);
            if (lane >= o) before += y;
        }
        work = sum_of_warp(work);
        own = sum_of_warp(own);
        if (lane == 31) {
            sh_scan[warp - MMA_WARP] = before;
            sh_work[warp - MMA_WARP] = work;
            sh_own[warp - MMA_WARP] = own;
        }
        named_bar_sync(1, FINDERS);
        long long all = 0;
        work = own = 0;
#pragma unroll
        for (int w = 0; w < FINDERS / 32; ++w) {
            if (w < warp - MMA_WARP) before += sh_scan[w];
            all += sh_scan[w];
            work += sh_work[w];
            own += sh_own[w];
        }
        before -= mine;
        int ctas = gridDim.x;
        if (!p.share.whole) ctas = max(1, min(ctas, prefix_ctas(p.share, all, work, own * (p.share.own_units / a.nseq))));
        per = quotient(all + ctas - 1, ctas);
        const long long x0 = per * blockIdx.x;
        x1 = min(x0 + per, all);
        range = max(0LL, x1 - x0);
        if (range > 0 && x0 >= before && x0 < before + mine) {
            long long b = before;
            int g = g0;
            Group x = own_group;
            if (g1 - g0 > 1) {
                x = group_of(p, g);
                for (long long n = prefix_tiles(p.share, x); x0 >= b + n; n = prefix_tiles(p.share, x)) {
                    b += n;
                    x = group_of(p, ++g);
                }
            }
            const long long unit = quotient(x0 - b, x.tiles), kvh = quotient(unit, x.blocks);
            sh_at = x;
            sh_group = g;
            sh_kvh = static_cast<int>(kvh);
            sh_block = static_cast<int>(unit - kvh * x.blocks);
            sh_tile = static_cast<int>(x0 - b - unit * x.tiles);
        }
        named_bar_sync(1, FINDERS);
    }

    // A wait of the pipeline: the first that runs out sets the error word, and
    // all later ones return at once.
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity)) return true;
        volatile uint32_t *ab = &bars->abort;
        if (*ab == 0u && mbar_wait(bar, parity, p.wait_ns, ab)) return true;
        if (*ab == 0u) {
            *ab = 1u;
            atomicOr(&g_prefix_error, 1u);
        }
        return false;
    };
    auto wait_warp = [&](uint64_t *bar, uint32_t parity) { return __all_sync(FULL_MASK, wait(bar, parity)); };
    auto ready_warp = [&](uint64_t *bar, uint32_t parity) { return __all_sync(FULL_MASK, mbar_try_wait(bar, parity)); };

    if (warp == WALK_WARP) {
        fewer_registers<FEW_REGISTERS>();
        // ---- the segments of the range ----------------------------------------------------
        long long left = range;
        int g = sh_group, kvh = sh_kvh, b = sh_block, t = sh_tile;   // unused without a group
        Group x = sh_at;
        for (uint32_t k = 0;; ++k) {
            Segment s = {};
            if (left > 0) {
                const int n = static_cast<int>(min(static_cast<long long>(x.tiles - t), left));
                s.g = g;
                s.kvh = kvh;
                s.first = x.first + b * p.block;
                s.count = min(p.block, x.first + x.count - s.first);
                s.len = x.len;
                s.t0 = t;
                s.t1 = t + n;
                const bool whole = n == x.tiles;
                s.slot = whole ? -1 : 2 * static_cast<int>(blockIdx.x) + (k == 0 ? 0 : 1);
                const int block = block_number(p, x, g, b);
                s.row = whole_row(p, block, s.first);
                if (t == 0 && lane == 0) {
                    // Where the join finds the block: its first tile is tile `at` of the batch.
                    const long long at = x1 - left;
                    p.meta[static_cast<size_t>(block) * a.kv.nkv + kvh] =
                        whole ? make_int2(-1, 0) : make_int2(s.slot, static_cast<int>(quotient(at + x.tiles - 1, per)));
                }
                left -= n;
                t = 0;
                if (++b == x.blocks) {
                    b = 0;
                    if (++kvh == a.kv.nkv) {
                        kvh = 0;
                        // The next group that has tiles: 32 at a time.
                        for (int from = g + 1; left > 0; from += 32) {
                            const bool have = from + lane < a.ngroups && prefix_tiles(p.share, group_of(p, from + lane)) > 0;
                            const uint32_t found = __ballot_sync(FULL_MASK, have);
                            if (found != 0u) {
                                g = from + __ffs(found) - 1;
                                x = group_of(p, g);
                                break;
                            }
                            if (from >= a.ngroups) left = 0;   // not reached: what is left lies in some group
                        }
                    }
                }
            }
            if (!wait_warp(&bars->seg_empty[k % SEGS], ((k / SEGS) & 1) ^ 1)) break;
            if (lane == 0) {
                bars->seg[k % SEGS] = s;
                mbar_arrive(&bars->seg_full[k % SEGS]);
            }
            __syncwarp();
            if (s.count == 0) break;
        }
    } else if (warp >= COPY_WARP) {
        fewer_registers<FEW_REGISTERS>();
        // ---- cells and queries in: rows 32 quarter .. + 31 of every tile ---------------------
        // No fence here: one that orders these writes before the tensor cores' reads would wait for all
        // copies under way. The MMA warp has it, behind its wait.
        const int quarter = warp - COPY_WARP;
        bool ok = true;
        long long off = 0;                          // of this lane's row, in bytes
        uint32_t row_mask = 0;                      // rows of the quarter that are there
        uint16_t key_scale = 0, value_scale = 0;    // of this lane's row
        auto page_of = [&](const Segment &s, int cell) {
            return cell < s.len ? ld_in(a.prefix_table + s.g * a.prefix_stride + divide(p.page, cell)) : -1;
        };
        // This lane's row of a tile is `cell`, in page `page`.
        auto find_row = [&](const Segment &s, int cell, int page) {
            const bool good = page >= 0 && page < a.kv.npages;
            const int slot = cell - divide(p.page, cell) * a.kv.page_size;
            off = good ? (page * a.kv.page_stride + slot * a.kv.cell_stride + s.kvh * a.kv.head_stride) * (kInt8 ? 1 : 2) : 0;
            row_mask = __ballot_sync(FULL_MASK, good);
            if constexpr (kInt8) {
                key_scale = value_scale = 0;
                if (good) {
                    const long long so = page * a.kv.scale_page_stride + slot * a.kv.scale_cell_stride + s.kvh * a.kv.scale_head_stride;
                    key_scale = ld_in_u16(a.kv.k_scale_f16 + so);
                    value_scale = ld_in_u16(a.kv.v_scale_f16 + so);
                }
            }
        };
        if constexpr (!kInt8) {
            // The queries of a segment: 16-byte pieces, zeros where there is no sequence.
            auto queries = [&](const Segment &s) {
                const int n0 = min(p.seqs, s.count), tiles = s.count > p.seqs ? 2 : 1, c = lane & 15;
                for (int i = 0; i < tiles; ++i) {
                    const int rows = (i == 0 ? n0 : s.count - n0) * p.group, row = 32 * quarter + lane, seq = row / p.group;
                    const long long at = row >= rows ? -1 : 2 * ((s.first + i * p.seqs + seq) * a.q_seq_stride +
                                                                 (s.kvh * p.group + row - seq * p.group) * a.q_head_stride);
#pragma unroll 4
                    for (int e = 0; e < 16; ++e) {
                        const int r = 2 * e + (lane >> 4);
                        const long long ro = __shfl_sync(FULL_MASK, at, r);
                        cp_async_16_or_zero(base + i * TILE_BYTES + tile_at(32 * quarter + r, c),
                                            static_cast<const char *>(a.q) + (ro < 0 ? 0 : ro) + 16 * c, ro >= 0);
                    }
                }
                cp_async_arrive(&bars->q_full);
            };
            uint32_t kv = 0, tile = 0;              // tiles of keys or values, of cells, so far
            for (uint32_t k = 0; ok; ++k) {
                ok = wait_warp(&bars->seg_full[k % SEGS], (k / SEGS) & 1);
                if (!ok) break;
                const Segment s = bars->seg[k % SEGS];
                __syncwarp();
                if (s.count == 0) break;
                const bool two = s.count > p.seqs;
                const int n = s.t1 - s.t0;
                int page = page_of(s, s.t0 * ROWS + 32 * quarter + lane);
                bool asked = ready_warp(&bars->q_empty, (k & 1) ^ 1);
                if (asked) queries(s);
                auto copy = [&](const void *what, long long row_off, uint32_t rows) {
                    const uint32_t slot = kv % STAGES;
                    if (!wait_warp(&bars->kv_empty[slot], ((kv / STAGES) & 1) ^ 1)) return false;
                    const char *from = static_cast<const char *>(what) + 16 * (lane & 15);
                    const uint32_t to = ring + slot * TILE_BYTES;
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int r = 2 * e + (lane >> 4);
                        const long long ro = __shfl_sync(FULL_MASK, row_off, r);
                        cp_async_16_or_zero(to + tile_at(32 * quarter + r, lane & 15), from + ro, (rows >> r) & 1u);
                    }
                    if (!(p.stall != 0 && blockIdx.x == 0 && kv == 0)) cp_async_arrive(&bars->kv_full[slot]);
                    ++kv;
                    return true;
                };
                long long last_off = 0;
                uint32_t last_mask = 0;
                for (int j = 0; ok && j <= n; ++j) {
                    // In the order of use (see key_item): with one row tile, keys of tile j go before the values of tile j - 1.
                    if (j < n) {
                        if (!two) {
                            last_off = off;
                            last_mask = row_mask;
                        }
                        const int cell = (s.t0 + j) * ROWS + 32 * quarter + lane;
                        find_row(s, cell, page);
                        page = j + 1 < n ? page_of(s, cell + ROWS) : -1;
                        const uint32_t side = tile % SIDES;
                        ok = wait_warp(&bars->side_empty[side], (tile / SIDES & 1) ^ 1);
                        if (!ok) break;
                        if (lane == 0) {
                            reinterpret_cast<uint32_t *>(&bars->mask[side])[quarter] = row_mask;
                            mbar_arrive(&bars->side_full[side]);
                        }
                        ++tile;
                        ok = copy(a.kv.k, off, row_mask);
                    } else if (!two) {
                        last_off = off;
                        last_mask = row_mask;
                    }
                    if (ok && (two ? j < n : j > 0)) ok = copy(a.kv.v, two ? off : last_off, two ? row_mask : last_mask);
                    if (ok && !asked) {
                        ok = wait_warp(&bars->q_empty, (k & 1) ^ 1);
                        if (ok) queries(s);
                        asked = true;
                    }
                }
                if (ok && lane == 0) mbar_arrive(&bars->seg_empty[k % SEGS]);
            }
        } else {
            // Copies of int8 tiles run ahead of their conversion: keys and values of one tile and the next
            // one's keys are under way. Every thread converts what it copied.
            uint32_t kv = 0, tile = 0;              // tiles of keys or values converted, of cells
            uint32_t sent = 0;                      // of keys or values copied
            auto send = [&](const void *what) {
                const char *from = static_cast<const char *>(what) + 16 * (lane & 7);
                const uint32_t to = raws + (sent % F::RAW) * (TILE_BYTES / 2) + 16 * (32 * quarter * 8 + lane);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int r = 4 * e + (lane >> 3);
                    const long long ro = __shfl_sync(FULL_MASK, off, r);
                    cp_async_16_or_zero(to + 512 * e, from + ro, (row_mask >> r) & 1u);
                }
                cp_async_commit();
                ++sent;
            };
            // The oldest tile on its way, as binary16 operands. `under_way`: copies behind it.
            auto convert = [&](int under_way) {
                if (!wait_warp(&bars->kv_empty[kv % STAGES], ((kv / STAGES) & 1) ^ 1)) return false;
                cp_async_wait_at_most(under_way);
                const uint32_t from = raws + (kv % F::RAW) * (TILE_BYTES / 2) + 16 * (32 * quarter * 8 + lane);
                const uint32_t to = ring + (kv % STAGES) * TILE_BYTES;
                const int c = lane & 7;
                uint4 got[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) got[e] = ld_shared_v4(from + 512 * e);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int r = 32 * quarter + 4 * e + (lane >> 3);
                    const uint32_t w[4] = {got[e].x ^ 0x80808080u, got[e].y ^ 0x80808080u, got[e].z ^ 0x80808080u, got[e].w ^ 0x80808080u};
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        st_shared_v4(to + tile_at(r, 2 * c + h), codes_to_half2(w[2 * h], 0x4140), codes_to_half2(w[2 * h], 0x4342),
                                     codes_to_half2(w[2 * h + 1], 0x4140), codes_to_half2(w[2 * h + 1], 0x4342));
                }
                __syncwarp();
                if (lane == 0 && !(p.stall != 0 && blockIdx.x == 0 && kv == 0)) mbar_arrive(&bars->kv_full[kv % STAGES]);
                ++kv;
                return true;
            };
            Segment s = {}, next = {};              // of the tile that is converted, of the one that is copied
            uint32_t k = 0;                         // segments begun with copies
            int t = 0, t_next = 0, page = -1;       // page: of this lane's row of the tile to copy next
            auto enter = [&]() {                    // the next segment's first tile is to be copied next
                if (!wait_warp(&bars->seg_full[k % SEGS], (k / SEGS) & 1)) return false;
                next = bars->seg[k % SEGS];
                __syncwarp();
                ++k;
                t_next = next.t0;
                page = page_of(next, t_next * ROWS + 32 * quarter + lane);
                return true;
            };
            uint32_t mask = 0;                      // of the tile that is converted, as its scales
            uint16_t scale_k = 0, scale_v = 0;
            auto row = [&]() {                      // the row of the tile to copy, and the page of the one behind it
                const int cell = t_next * ROWS + 32 * quarter + lane;
                find_row(next, cell, page);
                page = t_next + 1 < next.t1 ? page_of(next, cell + ROWS) : -1;
            };
            ok = enter();
            if (ok && next.count > 0) {
                row();
                send(a.kv.k);
                send(a.kv.v);
            }
            while (ok && next.count > 0) {
                s = next;
                t = t_next;
                mask = row_mask;
                scale_k = key_scale;
                scale_v = value_scale;
                const uint32_t seg = k - 1;
                bool more = ++t_next < next.t1;
                if (!more) {
                    ok = enter();
                    if (!ok) break;
                    more = next.count > 0;
                }
                if (more) {
                    row();
                    send(a.kv.k);
                }
                const uint32_t side = tile % SIDES;
                ok = wait_warp(&bars->side_empty[side], ((tile / SIDES) & 1) ^ 1);
                if (!ok) break;
                if (lane == 0) reinterpret_cast<uint32_t *>(&bars->mask[side])[quarter] = mask;
                const float vs = __half2float(__ushort_as_half(scale_v));
                scales->key[side][32 * quarter + lane] = __half2float(__ushort_as_half(scale_k));
                scales->value[side][32 * quarter + lane] = vs;
                // The sums' reference has to be finite, whatever the scale: within binary16's numbers.
                scales->log_value[side][32 * quarter + lane] = __log2f(fminf(fmaxf(fabsf(vs), 5.9604645e-8f), 65504.0f));
                ++tile;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->side_full[side]);
                ok = convert(more ? 2 : 1);
                if (!ok) break;
                if (more) send(a.kv.v);
                ok = convert(more ? 2 : 0);
                if (ok && t + 1 == s.t1 && lane == 0) mbar_arrive(&bars->seg_empty[seg % SEGS]);
            }
        }
        cp_async_wait<0>();
        __syncwarp();
    } else if (warp == MMA_WARP) {
        fewer_registers<FEW_REGISTERS>();
        const bool one = elect_one();   // the warp runs as one, one lane issues
        constexpr uint32_t fmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
        constexpr uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
        constexpr uint32_t idesc_v = idesc | (1u << 16);   // second operand contiguous in N
        bool ok = true;
        uint32_t kv = 0;                   // tiles of keys or values so far
        uint32_t odd = 0;                  // bit i: stream i has had an odd number of products S
        for (uint32_t k = 0; ok; ++k) {
            if (!wait_warp(&bars->seg_full[k % SEGS], (k / SEGS) & 1)) break;
            const Segment s = bars->seg[k % SEGS];
            __syncwarp();
            if (one) mbar_arrive(&bars->seg_empty[k % SEGS]);
            if (s.count == 0) break;
            const bool two = s.count > p.seqs;
            const int n = s.t1 - s.t0;
            if (!wait_warp(&bars->q_full, k & 1)) break;
            // Orders what the copy warps wrote (and waits have shown) before the tensor cores' reads.
            auto landed = [&](uint32_t slot, uint32_t n) {
                if (!wait_warp(&bars->kv_full[slot], n & 1)) return false;
                fence_proxy_async_smem();
                return true;
            };
            // Stream i's S of the keys in a slot with the queries at q_at (and the halves behind them).
            auto scores = [&](int i, uint32_t q_at, uint32_t slot) {
                const uint64_t qd = sw128_kmajor_desc(q_at), kd = sw128_kmajor_desc(ring + slot * TILE_BYTES);
                tc_fence_after_sync();
#pragma unroll
                for (int kk = 0; kk < (kSplit ? 16 : 8); ++kk) {
                    const uint64_t step = ((kk >> 2) & 1) * (HALF >> 4) + 2 * (kk & 3);
                    // The second halves first: the tensor cores cut sums off, less while these are small.
                    const uint64_t half = kSplit && kk < 8 ? TILE_BYTES >> 4 : 0;
                    if (one) tc_mma_bf16(tmem + S_COL + 128 * i, qd + step + half, kd + step, idesc, kk > 0 ? 1u : 0u);
                }
                if (one) tc_commit(&bars->s_full[i]);
                odd ^= 1u << i;
            };
            // Stream i's last weights times the values in a slot; `first`: the sums begin with them.
            auto outputs = [&](int i, uint32_t slot, bool first) {
                const uint32_t p_col = tmem + S_COL + 128 * i, o_col = tmem + O_COL + 128 * i, parity = ~(odd >> i) & 1u;
                const uint64_t vd = sw128_mnmajor_desc(ring + slot * TILE_BYTES, HALF);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (!wait_warp(half == 0 ? &bars->p_half[i] : &bars->p_full[i], parity)) return false;
                    tc_fence_after_sync();
#pragma unroll
                    for (int kk = 4 * half; kk < 4 * half + 4; ++kk) {
                        // 16 cells' weights are 8 columns; with their remainders, 32 cells' are 16 and 16.
                        const uint32_t at = p_col + (kSplit ? 32 * (kk >> 1) + 8 * (kk & 1) : 8 * kk);
                        if (one) tc_mma_bf16_ta(o_col, at, vd + 128 * kk, idesc_v, !first || kk > 0 ? 1u : 0u);
                        if (kSplit && one) tc_mma_bf16_ta(o_col, at + 16, vd + 128 * kk, idesc_v, 1u);
                    }
                }
                return true;
            };
#pragma unroll 1
            for (int j = 0; ok && j <= n; ++j) {
                // keys of tile j, values of tile j - 1
                const uint32_t kn = kv + key_item(two || kInt8, j), vn = kv + value_item(two || kInt8, j - 1, n);
                const uint32_t ks = kn % STAGES, vs = vn % STAGES;
                if (two) {
                    // Both copies are waited for before the weights, so that nothing stands between the products.
                    if (j > 0) ok = landed(vs, vn / STAGES);
                    if (ok && j < n) ok = landed(ks, kn / STAGES);
#pragma unroll 1
                    for (int i = 0; ok && i < 2; ++i) {
                        if (j > 0) ok = outputs(i, vs, (j - 1) % F::CHAIN == 0);
                        if (ok && i == 1 && j > 0 && one) tc_commit(&bars->kv_empty[vs]);
                        if (ok && j < n) scores(i, base + i * TILE_BYTES, ks);
                    }
                    if (ok && j < n && one) tc_commit(&bars->kv_empty[ks]);
                } else {
                    // Tile j goes to stream j % 2; the other's last weights are worked out meanwhile.
                    if (j < n) {
                        ok = landed(ks, kn / STAGES);
                        if (!ok) break;
                        scores(j & 1, base, ks);
                        if (one) tc_commit(&bars->kv_empty[ks]);
                    }
                    if (j > 0) {
                        ok = landed(vs, vn / STAGES) && outputs((j - 1) & 1, vs, ((j - 1) >> 1) % F::CHAIN == 0);
                        if (ok && one) tc_commit(&bars->kv_empty[vs]);
                    }
                }
            }
            kv += 2 * n;
            if (ok && one) {
                tc_commit(&bars->o_full[0]);
                tc_commit(&bars->o_full[1]);
            }
        }
        if (one) tc_commit(&bars->drain);
        mbar_wait(&bars->drain, 0, p.wait_ns);
        __syncwarp();
    } else if (warp > WALK_WARP) {
        fewer_registers<FEW_REGISTERS>();
        // ---- two warps: where the join finds each sequence's block ------------------------------
        const int step = 2 * gridDim.x, at = 2 * blockIdx.x + (warp - WALK_WARP - 1);
        for (int g = at; g < a.ngroups; g += step) {
            const Group x = group_of(p, g);
            for (int i = lane; i < x.count; i += 32) {
                const int b = i / p.block;
                p.places[x.first + i] = x.tiles > 0 ? make_int2(block_number(p, x, g, b), x.first + b * p.block) : make_int2(-1, 0);
            }
        }
        // Sequences of no group.
        const int begin = min(max(ld_in(a.cu), 0), a.nseq), end = min(max(ld_in(a.cu + a.ngroups), 0), a.nseq);
        for (int s = 32 * at + lane; s < a.nseq; s += 32 * step)
            if (s < begin || s >= end) p.places[s] = make_int2(-1, 0);
    } else {
        more_registers<MORE_REGISTERS>();
        // ---- softmax of one stream, one row per thread --------------------------------------
        const int i = warp >> 2, quarter = warp & 3, row = 32 * quarter + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
        const uint32_t s_at = tmem + lanes + S_COL + 128 * i;
        uint32_t ns = 0, tiles = 0;
        // Once through the code as soon as there is a segment, while its first cells come: its instructions are
        // then there (the first tile took 3 to 5 us without it). It waits for nothing, signals nothing and
        // writes nothing.
        bool dry = !kInt8;   // their loops are longer than the wait for the first cells
        for (uint32_t k = 0;; k += dry ? 0 : 1, dry = false) {
            if (!wait_warp(&bars->seg_full[k % SEGS], (k / SEGS) & 1)) break;
            const Segment s = bars->seg[k % SEGS];
            __syncwarp();
            if (lane == 0 && !dry) mbar_arrive(&bars->seg_empty[k % SEGS]);
            if (s.count == 0) break;
            if constexpr (kInt8) {
                // The segment's queries: 16 lanes a row of 128 elements, 8 each, times a power of two that brings
                // the largest to 2^13 at least, as binary16 numbers (and the rest, into the second tile).
                if (!wait_warp(&bars->q_empty, (k & 1) ^ 1)) break;
                const int l8 = lane & 15;
                const float to_log2 = a.scale * LOG2E;
#pragma unroll 1
                for (int tile = 0; tile < (s.count > p.seqs ? 2 : 1); ++tile) {
                    const int seqs = min(p.seqs, s.count - tile * p.seqs), r0 = 16 * warp + (lane >> 4);
                    float4 u[8], v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int r = r0 + 2 * e, seq = r / p.group;
                        const QT *from = static_cast<const QT *>(a.q) + (s.first + tile * p.seqs + seq) * a.q_seq_stride +
                                         (s.kvh * p.group + r - seq * p.group) * a.q_head_stride + 8 * l8;
                        const bool have = seq < seqs;
                        u[e] = have ? load4(from) : make_float4(0.f, 0.f, 0.f, 0.f);
                        v[e] = have ? load4(from + 4) : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int r = r0 + 2 * e;
                        float top = fmaxf(fmaxf(fmaxf(fabsf(u[e].x), fabsf(u[e].y)), fmaxf(fabsf(u[e].z), fabsf(u[e].w))),
                                          fmaxf(fmaxf(fabsf(v[e].x), fabsf(v[e].y)), fmaxf(fabsf(v[e].z), fabsf(v[e].w))));
#pragma unroll
                        for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, o));
                        int ex = 0;
                        if (top > 0.0f && top < INFINITY) frexpf(top, &ex);
                        ex = max(-113, ex);   // 2^(14 - ex) and 2^(ex - 14) are fp32 numbers
                        const float up = ldexpf(1.0f, 14 - ex);
                        uint32_t hi[4], lo[4];
                        split(u[e].x * up, u[e].y * up, hi[0], lo[0]);
                        split(u[e].z * up, u[e].w * up, hi[1], lo[1]);
                        split(v[e].x * up, v[e].y * up, hi[2], lo[2]);
                        split(v[e].z * up, v[e].w * up, hi[3], lo[3]);
                        st_shared_v4(base + tile * TILE_BYTES + tile_at(r, l8), hi[0], hi[1], hi[2], hi[3]);
                        if (kSplit) st_shared_v4(base + TILE_BYTES + tile_at(r, l8), lo[0], lo[1], lo[2], lo[3]);
                        // Not 0, which an absent cell's -infinity would make NaN: a smaller factor's logits (sums are below 2^44)
                        // and this one's are 0 beside 1 all the same.
                        if (l8 == 0) scales->row[tile * ROWS + r] = fmaxf(to_log2 * ldexpf(1.0f, ex - 14), FLT_MIN);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->q_full);
            }
            const bool two = s.count > p.seqs || dry;
            const int n = dry ? 1 : s.t1 - s.t0;
            const int count = !two ? s.count : i == 0 ? p.seqs : s.count - p.seqs;   // sequences of this stream's rows
            const int rows = count * p.group;
            const bool idle = 32 * quarter >= rows && !dry;                          // a warp without rows
            float c = a.scale * LOG2E;
            if constexpr (kInt8) {
                if (!dry && !wait_warp(&bars->q_full, k & 1)) break;
                c = scales->row[(two ? i : 0) * ROWS + row];
            }
            float m = -INFINITY, l = 0.0f;   // m in base 2, LIFT not counted
            bool any = false, ok = true;
            // Sums that have had CHAIN tiles are put aside in the place of the CTA's last segment, which no other has, and which has its
            // own results there from its end on: those of two row tiles in their places there, those of two streams in a half each.
            float m_aside = -INFINITY;
            int summed = 0;                  // tiles in the sums in tensor memory
            bool put = false;                // sums lie aside
            const uint32_t o_mine = tmem + lanes + O_COL + 128 * i;
            // The sums in tensor memory and those put aside, added: put aside, or `back` into tensor memory.
            auto add_aside = [&](bool back) {
                float4 *aside = p.slots + static_cast<size_t>(2 * blockIdx.x + 1) * (BLOCK * 32);
                const int at = (two ? i * p.seqs * p.group : i * ROWS) + row;
                const float f = ex2(m_aside - (m == -INFINITY ? 0.0f : m));
                const bool add = put && row < rows;
#pragma unroll 1
                for (int piece = 0; piece < 4; ++piece) {
                    float4 was[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        was[e] = add ? ld_in(aside + sums_at(at, 8 * piece + e)) : make_float4(0.f, 0.f, 0.f, 0.f);
                    uint32_t o[32];
                    tmem_read32(o_mine + 32 * piece, o);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float y[4] = {was[e].x, was[e].y, was[e].z, was[e].w};
#pragma unroll
                        for (int q = 0; q < 4; ++q) o[4 * e + q] = __float_as_uint(fmaf(y[q], f, __uint_as_float(o[4 * e + q])));
                    }
                    if (back) {
                        tmem_st32(o_mine + 32 * piece, o);
                    } else if (row < rows) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            aside[sums_at(at, 8 * piece + e)] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                                            __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
                    }
                }
                if (back) {
                    tmem_st_wait();
                    tc_fence_before_sync();   // the other stream reads them
                }
                m_aside = m;
                put = true;
            };
            for (int j = 0; j < n; ++j) {
                if (!two && (j & 1) != i) continue;
                const uint32_t side = (tiles + j) % SIDES;
                if (!dry) {
                    ok = wait_warp(&bars->s_full[i], ns & 1);
                    if (!ok) break;
                    ++ns;
                }
                if (idle) {
                    if (lane == 0) {
                        arrive(&bars->side_empty[side], two ? 1u : 2u);
                        mbar_arrive(&bars->p_half[i]);
                        mbar_arrive(&bars->p_full[i]);
                    }
                    continue;
                }
                if (!dry) ok = wait_warp(&bars->side_full[side], ((tiles + j) / SIDES) & 1);
                if (!ok) break;
                tc_fence_after_sync();
                if (__builtin_expect(summed == F::CHAIN, 0)) {
                    add_aside(false);
                    any = false;             // the sums in tensor memory begin again
                    summed = 0;
                }
                // 32 cells at a time, twice: for the largest, and for the weights. The loops stay rolled and read TMEM
                // twice: straight through, the code of a tile did not stay in the instruction cache (fp32
                // queries 4.2 us a tile, rolled 2.1; 16-bit cells, held in registers, were no faster).
                auto products = [&](int g, uint64_t (&x)[16]) {
                    uint32_t r[32];
                    const uint32_t there = reinterpret_cast<const uint32_t *>(&bars->mask[side])[g];
                    tmem_read32(s_at + 32 * g, r);
                    if constexpr (kInt8) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 ks = *reinterpret_cast<const float4 *>(scales->key[side] + 32 * g + e);
                            float y[4];
                            unpair(mul_pair(pair(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), pair(ks.x, ks.y)), y[0], y[1]);
                            unpair(mul_pair(pair(__uint_as_float(r[e + 2]), __uint_as_float(r[e + 3])), pair(ks.z, ks.w)), y[2], y[3]);
#pragma unroll
                            for (int q = 0; q < 4; ++q) r[e + q] = __float_as_uint(y[q]);
                        }
                    }
                    if (there != 0xFFFFFFFFu) {   // behind the scales: an absent cell's is 0
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!((there >> e) & 1u)) r[e] = 0xFF800000u;
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] = pair(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
                };
                float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                for (int g = dry ? 3 : 0; g < 4; ++g) {
                    uint64_t x[16];
                    products(g, x);
                    if constexpr (kInt8) {
                        const uint64_t c2 = pair(c, c);
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const float4 lv = *reinterpret_cast<const float4 *>(scales->log_value[side] + 32 * g + 2 * e);
                            float y[4];
                            unpair(fma_pair(x[e], c2, pair(lv.x, lv.y)), y[0], y[1]);
                            unpair(fma_pair(x[e + 1], c2, pair(lv.z, lv.w)), y[2], y[3]);
#pragma unroll
                            for (int q = 0; q < 4; ++q) tops[q] = fmaxf(tops[q], y[q]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            float y[8];
#pragma unroll
                            for (int q = 0; q < 4; ++q) unpair(x[e + q], y[2 * q], y[2 * q + 1]);
#pragma unroll
                            for (int q = 0; q < 4; ++q) tops[q] = fmaxf(fmaxf(tops[q], y[2 * q]), y[2 * q + 1]);
                        }
                    }
                }
                float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                if constexpr (!kInt8) top *= c;
                const bool move = top - m > LAZY;   // also true from -infinity to a finite maximum
                if (__any_sync(FULL_MASK, move)) {
                    const float f = move ? ex2(m - top) : 1.0f;
                    if (move) m = top;
                    l *= f;
                    if (any) {
#pragma unroll 1
                        for (int g = 0; g < 4; ++g) {
                            uint32_t o[32];
                            tmem_read32(o_mine + 32 * g, o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st32(o_mine + 32 * g, o);
                        }
                    }
                }
                const float mc = m == -INFINITY ? 0.0f : m - F::LIFT;
                const uint64_t c2 = pair(c, c), mc2 = pair(-mc, -mc);
                uint64_t sums[2] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f)};
#pragma unroll 1
                for (int g = dry ? 3 : 0; g < 4; ++g) {
                    uint64_t x[16];
                    products(g, x);
                    uint32_t pw[16], pl[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float x0, x1;
                        unpair(fma_pair(x[e], c2, mc2), x0, x1);
                        x0 = ex2(x0);
                        x1 = ex2(x1);
                        sums[e & 1] = add_pair(sums[e & 1], pair(x0, x1));
                        if constexpr (kInt8) {
                            const float2 vs = *reinterpret_cast<const float2 *>(scales->value[side] + 32 * g + 2 * e);
                            x0 *= vs.x;
                            x1 *= vs.y;
                        }
                        if constexpr (kSplit) split(x0, x1, pw[e], pl[e]);
                        else pw[e] = pack<T>(x0, x1);
                    }
                    // Weights of 32 cells over products that have been read.
                    if (!dry) {
                        tmem_st16(s_at + (kSplit ? 32 : 16) * g, pw);
                        if (kSplit) tmem_st16(s_at + 32 * g + 16, pl);
                    }
                    if (g & 1) {   // the products with half of the values can begin
                        tmem_st_wait();
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0 && !dry) {
                            mbar_arrive(g == 1 ? &bars->p_half[i] : &bars->p_full[i]);
                            if (g == 3) arrive(&bars->side_empty[side], two ? 1u : 2u);
                        }
                    }
                }
                {
                    float y0, y1;
                    unpair(add_pair(sums[0], sums[1]), y0, y1);
                    l += y0 + y1;
                }
                any = true;
                ++summed;
            }
            if (!ok) break;
            if (!dry) tiles += n;
            // ---- the segment's results ---------------------------------------------------------
            float2 sum = make_float2(m == -INFINITY ? -INFINITY : m - F::LIFT, l);
            float f0 = 1.0f, f1 = 1.0f;
            bool any0 = any, any1 = any;
            if (!dry && !(wait_warp(&bars->o_full[0], k & 1) && wait_warp(&bars->o_full[1], k & 1))) break;
            if (__builtin_expect(put, 0)) {
                tc_fence_after_sync();
                add_aside(true);
            }
            if (!two) {
                // Both streams have the same rows: their sums through the second query tile, which nothing reads any more.
                float4 *shared = reinterpret_cast<float4 *>(raw_smem + (base + TILE_BYTES - smem_u32(raw_smem)));
                shared[i * ROWS + row] = make_float4(sum.x, sum.y, any ? 1.0f : 0.0f, 0.0f);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->pair[quarter]);
                if (!wait_warp(&bars->pair[quarter], k & 1)) break;
                const float4 o0 = shared[row], o1 = shared[ROWS + row];
                const float top = fmaxf(o0.x, o1.x), ref = top == -INFINITY ? 0.0f : top;
                f0 = ex2(o0.x - ref);
                f1 = ex2(o1.x - ref);
                any0 = o0.z != 0.0f;
                any1 = o1.z != 0.0f;
                sum = make_float2(top, fmaf(o0.y, f0, o1.y * f1));
            } else if (lane == 0 && !dry) {
                mbar_arrive(&bars->pair[quarter]);   // a phase of each segment
            }
            tc_fence_after_sync();
            if (!idle) {
                const bool valid = row < rows && !dry;
                const int block_row = (two ? i * p.seqs * p.group : 0) + row;
                const int at = s.slot < 0 ? s.row + block_row : block_row;
                const size_t from = s.slot < 0 ? static_cast<size_t>(s.kvh) * p.whole_rows : static_cast<size_t>(s.slot) * BLOCK;
                float4 *to = (s.slot < 0 ? p.whole : p.slots) + from * 32;
                const int piece0 = two ? 0 : 2 * i, piece1 = two ? 4 : 2 * i + 2;   // with the same rows, half of the columns each
#pragma unroll 1
                for (int piece = dry ? 3 : piece0; piece < piece1; ++piece) {
                    uint32_t o[32];
                    tmem_read32(tmem + lanes + O_COL + (two ? 128 * i : 0) + 32 * piece, o);
                    if (!two) {
                        uint32_t u[32];
                        tmem_read32(tmem + lanes + O_COL + 128 + 32 * piece, u);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __float_as_uint((any0 ? __uint_as_float(o[e]) * f0 : 0.0f) + (any1 ? __uint_as_float(u[e]) * f1 : 0.0f));
                    }
                    if (valid)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            to[sums_at(at, 8 * piece + e)] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                                         __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
                }
                if (valid && (two || i == 0)) ((s.slot < 0 ? p.whole_refs : p.slot_refs) + from)[at] = sum;
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0 && !dry) mbar_arrive(&bars->q_empty);
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == MMA_WARP) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// Adds the rows' partial sums: of the prefix, in the order of the CTAs that hold them, and of the sequences'
// own cells, as paged attention left them. Rows are a KV head's: sequence times query heads. A warp takes 8 rows by 32
// columns, a lane the row lane % 8 and pieces lane / 8 and + 4; `split` warps share them, each every split-th
// range, and are added in order.
constexpr int JOIN_WARPS = 8, JOIN_RANGES = 4;
template <typename QT>
__global__ void __launch_bounds__(32 * JOIN_WARPS) prefix_join_kernel(const __grid_constant__ Params p, const PagedPartial own, int grid, int split,
                                                                      int blocks) {
    const PrefixAttnArgs &a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int set = warp / split, part = warp - set * split;
    const int unit = blockIdx.x * (JOIN_WARPS / split) + set, quarter = unit & 3;
    const int all_rows = a.nseq * p.group, row = 8 * (unit >> 2) + (lane & 7), kvh = blockIdx.y;
    const bool valid = row < all_rows;
    const int s = valid ? row / p.group : 0, head = valid ? row - s * p.group : 0, h = kvh * p.group + head;
    const size_t out_row = static_cast<size_t>(s) * a.nheads + h;
    const int chunk = 8 * quarter + (lane >> 3);
    // Before the wait: prefix_kernel let paged attention's kernel start, and that this grid, only after it
    // had waited for its own predecessors, so lengths are final.
    const bool mine = valid && a.table_cols > 0 && ld_in(a.lens + s) > 0;
    grid_dependency_wait();
    grid_launch_dependents();

    // Where this lane's ranges lie: the first, then every second slot from the next CTA's on.
    const float4 *sums0 = p.whole, *sums1 = p.slots;
    const float2 *refs0 = p.whole_refs, *refs1 = p.slot_refs;
    const float *own0 = own.rows, *own1 = own.slots;
    int n = 0, most = 0;
    const int2 place = valid ? __ldcg(p.places + s) : make_int2(-1, 0);
    const int part_of = head / own.heads_per_unit;
    const int4 w = mine ? __ldcg(own.meta + static_cast<size_t>(s) * own.units + kvh * own.parts + part_of) : make_int4(0, 0, 0, 0);
    if (place.x >= 0) {
        // Nothing but numbers is taken from scratch: a CTA that gave up may have left anything.
        const int block = min(place.x, blocks - 1), first = min(max(place.y, max(0, s - p.block + 1)), s);
        const int2 m = __ldcg(p.meta + static_cast<size_t>(block) * a.kv.nkv + kvh);
        const int at = (s - first) * p.group + head;
        if (m.x < 0) {
            const size_t from = static_cast<size_t>(kvh) * p.whole_rows;
            const int whole = min(whole_row(p, block, first) + at, p.whole_rows - 1);
            sums0 += from * 32 + sums_at(whole, chunk);
            refs0 += from + whole;
            n = 1;
        } else {
            const int slot = min(m.x, 2 * grid - 1), c0 = slot >> 1;
            sums0 = p.slots + static_cast<size_t>(slot) * (BLOCK * 32) + sums_at(at, chunk);
            refs0 = p.slot_refs + slot * BLOCK + at;
            sums1 += static_cast<size_t>(2 * c0) * (BLOCK * 32) + sums_at(at, chunk);
            refs1 += 2 * c0 * BLOCK + at;
            n = max(1, min(m.y, grid - 1) - c0 + 1);
        }
    }
    int all = n;
    if (mine) {
        const size_t in_slot = static_cast<size_t>(head - part_of * own.heads_per_unit) * OWN_ROW + 4 * chunk;
        const size_t own_slot = static_cast<size_t>(own.heads_per_unit) * OWN_ROW;
        if (w.x < 0) {
            own0 += out_row * OWN_ROW + 4 * chunk;
            all += 1;
        } else {
            const int slot = min(max(w.z, 0), 2 * own.grid - 1), c0 = slot >> 1;
            own0 = own.slots + slot * own_slot + in_slot;
            own1 += 2 * c0 * own_slot + in_slot;
            all += max(1, min(w.w, own.grid - 1) - c0 + 1);
        }
    }
    most = __reduce_max_sync(FULL_MASK, all);
    float top = -INFINITY, l = 0.0f;
    float4 y[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    auto add = [&](float2 ml, const float4 (&v)[2]) {
        const float t = fmaxf(top, ml.x), ref = t == -INFINITY ? 0.0f : t;
        const float f = ex2(top - ref), g = ex2(ml.x - ref);
        top = t;
        l = fmaf(ml.y, g, l * f);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            y[e].x = fmaf(v[e].x, g, y[e].x * f);
            y[e].y = fmaf(v[e].y, g, y[e].y * f);
            y[e].z = fmaf(v[e].z, g, y[e].z * f);
            y[e].w = fmaf(v[e].w, g, y[e].w * f);
        }
    };
    for (int i0 = part; i0 < most; i0 += split * JOIN_RANGES) {
        float2 ml[JOIN_RANGES];
        float4 v[JOIN_RANGES][2];
#pragma unroll
        for (int e = 0; e < JOIN_RANGES; ++e) {
            const int i = i0 + split * e, j = i - n;
            ml[e] = make_float2(-INFINITY, 0.0f);
            v[e][0] = v[e][1] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < n) {
                const float4 *at = i == 0 ? sums0 : sums1 + static_cast<size_t>(2 * i) * (BLOCK * 32);
                ml[e] = __ldcg(i == 0 ? refs0 : refs1 + 2 * i * BLOCK);
                v[e][0] = ld_in(at);
                v[e][1] = ld_in(at + 4 * 8);
            } else if (i < all) {
                const float *at = j == 0 ? own0 : own1 + 2 * j * static_cast<size_t>(own.heads_per_unit) * OWN_ROW;
                ml[e] = __ldcg(reinterpret_cast<const float2 *>(at - 4 * chunk + 128));
                v[e][0] = ld_in(reinterpret_cast<const float4 *>(at));
                v[e][1] = ld_in(reinterpret_cast<const float4 *>(at + 16));
            }
        }
#pragma unroll
        for (int e = 0; e < JOIN_RANGES; ++e) add(ml[e], v[e]);
    }
    __shared__ float4 sums[JOIN_WARPS][2][32];
    __shared__ float2 refs[JOIN_WARPS][32];
    if (split > 1) {
        sums[warp][0][lane] = y[0];
        sums[warp][1][lane] = y[1];
        refs[warp][lane] = make_float2(top, l);
        __syncthreads();
        if (part > 0) return;
        for (int o = 1; o < split; ++o) {
            const float4 v[2] = {sums[warp + o][0][lane], sums[warp + o][1][lane]};
            add(refs[warp + o][lane], v);
        }
    }
    if (!valid) return;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    QT *out = static_cast<QT *>(a.out) + out_row * 128 + 4 * chunk;
#pragma unroll
    for (int e = 0; e < 2; ++e) store4(out + 16 * e, make_float4(y[e].x * inv, y[e].y * inv, y[e].z * inv, y[e].w * inv));
    if (chunk == 0 && a.lse != nullptr) a.lse[out_row] = l == 0.0f ? -INFINITY : (top + log2f(l)) * LN2;
}

struct Layout {
    size_t meta, places, whole, whole_refs, slots, slot_refs, own, bytes;
    int grid, blocks, whole_rows;
};
// Blocks of fp32 queries are one row tile: the scratch is laid out for as many blocks, whatever the type.
Layout layout(const PrefixAttnSizes &z) {
    Layout y;
    y.blocks = z.nseq / (ROWS / (z.nheads / z.nkv)) + z.ngroups + 1;
    y.whole_rows = (z.nseq * (z.nheads / z.nkv) + 7) / 8 * 8 + 8 * (y.blocks + 1);
    const long long tiles = (static_cast<long long>(z.prefix_capacity) + ROWS - 1) / ROWS * y.blocks * z.nkv;
    y.grid = static_cast<int>(std::max(1LL, std::min<long long>(device_sm_count(), tiles)));
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    size_t at = 0;
    y.meta = at;
    at += up(sizeof(int2) * y.blocks * z.nkv);
    y.places = at;
    at += up(sizeof(int2) * z.nseq);
    y.whole = at;
    at += up(sizeof(float4) * 32 * z.nkv * y.whole_rows);
    y.whole_refs = at;
    at += up(sizeof(float2) * z.nkv * y.whole_rows);
    y.slots = at;
    at += up(sizeof(float4) * 32 * BLOCK * 2 * y.grid);
    y.slot_refs = at;
    at += up(sizeof(float2) * BLOCK * 2 * y.grid);
    y.own = at;
    at += paged_partial_bytes(z.nseq, z.nheads, z.nkv, z.capacity);
    y.bytes = at;
    return y;
}

template <typename K, typename... A>
cudaError_t launch(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args) {
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

template <int kKv, typename QT>
cudaError_t run(Params &p, const Layout &y, const PagedAttnArgs &own_args, cudaStream_t stream) {
    constexpr size_t smem = smem_bytes<kKv, QT>();
    auto kernel = prefix_kernel<kKv, QT>;
    static thread_local int configured_device = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && configured_device != dev) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e == cudaSuccess) configured_device = dev;
    }
    p.seqs = ROWS / p.group;
    p.block = Form<kKv, QT>::TILES * p.seqs;
    // Measured, ns, side by side: a tile of 128 prefix cells for one row tile, for two; paged attention's tile of
    // 16 cells (32 int8), a quarter of a CTA's time for one, and what a unit costs besides.
    constexpr bool kInt8 = Form<kKv, QT>::kInt8;
    p.share = {p.a.cu, p.a.prefix_lens, p.a.ngroups, p.a.nseq, p.a.prefix_cols * p.a.kv.page_size, p.a.kv.nkv, p.seqs, p.block,
               device_sm_count(), y.grid,
               p.block == p.seqs || p.a.nseq <= p.seqs || y.grid + (paged_ctas(own_args) + 1) / 2 <= device_sm_count(),
               1500, kInt8 ? 3000 : 2300, kInt8 ? 550.0f : 400.0f, 400.0f, paged_units(own_args)};
    p.own_tile = Form<kKv, QT>::kInt8 ? 32 : 16;
    if (e == cudaSuccess) e = launch(kernel, dim3(y.grid), PTHREADS, smem, stream, p);
    PagedPartial own;
    if (e == cudaSuccess) e = launch_paged_partial(own_args, p.share, own, stream);
    if (e != cudaSuccess) return e;
    // Ranges of a block, on average.
    const int ranges = static_cast<int>(y.grid / (static_cast<long long>(p.a.kv.nkv) * std::max(1, std::max(p.a.ngroups, p.a.nseq / p.block)))) + 1;
    // As many warps share rows as there are ranges for and the GPU has room for at once.
    const long long units = static_cast<long long>((p.a.nseq * p.group + 7) / 8) * 4;   // of a KV head
    int split = 1;
    while (split < JOIN_WARPS && 2 * split <= ranges && 2 * split * units * p.a.kv.nkv <= 16LL * device_sm_count()) split *= 2;
    const int per = JOIN_WARPS / split;
    return launch(prefix_join_kernel<QT>, dim3(static_cast<unsigned>((units + per - 1) / per), p.a.kv.nkv), 32 * JOIN_WARPS, 0, stream, p, own,
                  y.grid, split, y.blocks);
}

}  // namespace

size_t prefix_attn_scratch_bytes(const PrefixAttnSizes &z) { return layout(z).bytes; }

cudaError_t launch_prefix_attn(const PrefixAttnArgs &a, cudaStream_t stream) {
    Params p = {};
    p.a = a;
    p.page = make_divider(a.kv.page_size);
    p.group = a.nheads / a.kv.nkv;
    const int capacity = a.prefix_cols * a.kv.page_size;
    const Layout y = layout({a.nseq, a.ngroups, a.nheads, a.kv.nkv, capacity, a.table_cols * a.kv.page_size});
    char *b = static_cast<char *>(a.scratch);
    p.meta = reinterpret_cast<int2 *>(b + y.meta);
    p.places = reinterpret_cast<int2 *>(b + y.places);
    p.whole = reinterpret_cast<float4 *>(b + y.whole);
    p.whole_refs = reinterpret_cast<float2 *>(b + y.whole_refs);
    p.slots = reinterpret_cast<float4 *>(b + y.slots);
    p.slot_refs = reinterpret_cast<float2 *>(b + y.slot_refs);
    p.whole_rows = y.whole_rows;
    // A wait may last as long as a CTA takes for a whole prefix: some 2 to 4 us a tile.
    p.wait_ns = wait_limit_ns() + 8192ull * ((static_cast<uint64_t>(capacity) + ROWS - 1) / ROWS);
    if (a.kv.npages == 0) p.a.kv.k = p.a.kv.v = const_cast<void *>(a.q);   // nothing is read, but addresses are formed
    p.stall = (debug_inject() & 32u) != 0u;
    PagedAttnArgs own = {};
    own.q = a.q;
    own.q_dtype = a.q_dtype;
    own.q_seq_stride = a.q_seq_stride;
    own.q_head_stride = a.q_head_stride;
    own.nseq = a.nseq;
    own.nheads = a.nheads;
    own.kv = a.kv;
    own.table = a.table;
    own.table_cols = a.table_cols;
    own.table_stride = a.table_stride;
    own.lens = a.lens;
    own.window = -1;
    own.scale = a.scale;
    own.scratch = b + y.own;
    if (a.kv.dtype == QSA_BF16) return run<QSA_BF16, __nv_bfloat16>(p, y, own, stream);
    if (a.kv.dtype == QSA_F16) return run<QSA_F16, __half>(p, y, own, stream);
    if (a.q_dtype == QSA_F32) return run<QSA_I8, float>(p, y, own, stream);
    if (a.q_dtype == QSA_F16) return run<QSA_I8, __half>(p, y, own, stream);
    return run<QSA_I8, __nv_bfloat16>(p, y, own, stream);
}

cudaError_t prefix_error_read_clear(uint32_t *word, cudaStream_t stream) {
    cudaError_t e = cudaMemcpyFromSymbolAsync(word, g_prefix_error, sizeof(uint32_t), 0, cudaMemcpyDeviceToHost, stream);
    if (e != cudaSuccess) return e;
    e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return e;
    const uint32_t zero = 0u;
    e = cudaMemcpyToSymbolAsync(g_prefix_error, &zero, sizeof(uint32_t), 0, cudaMemcpyHostToDevice, stream);
    if (e != cudaSuccess) return e;
    return cudaStreamSynchronize(stream);
}

}  // namespace qsa
