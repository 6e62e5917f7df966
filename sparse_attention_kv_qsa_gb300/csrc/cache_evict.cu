// Eviction by accumulated attention weight: per sequence the first `sinks`
// cells, the last `recent` cells and, of the cells between, those of largest
// mass are kept in order and copied to new pages.
//
// select_kernel: a cluster of CTAs per sequence finds the mass of the last
// cell to keep by a radix search on the order-preserving key of
// csrc/qsa_internal.cuh, 11, 11 and 10 bits at a time. Each CTA holds a run of
// the candidates' keys in shared memory, so the masses are read once, and
// counts its digits there. Its counts of 32 coarse digits go into every CTA's
// shared memory; after a cluster barrier each CTA finds the same coarse digit
// and fetches all CTAs' counts of the fine ones within it. The search ends with
// the exact 32-bit key of that cell and how many cells with that very key are
// kept, the lowest first, or earlier where a digit's cells are all kept. The
// cells are then listed in order: warps take consecutive runs, count, scan, and
// write. Latency bounds it: per pass a count, a barrier (1,200 cycles) and a
// fetch of the others' counts (2,000).
//
// copy_cells_kernel, copy_pieces_kernel: bandwidth. 16-byte pieces of keys and
// values, a batch of loads before its stores.
//
// Measured (GB300): 2 sequences of up to 131,072 int8 cells of 8 heads cut to
// 16,384, 41 us: 16 to choose, 24 to copy 136 MB (0.83 of the measured copy rate);
// one sequence of 576 cells cut to 512, 7.1 us, launches and latencies. Masses
// crowd into a few digits of the first pass, yet plain shared-memory atomics beat
// one atomic per different digit of a warp (by a sixth of the choice when both were tried).
#include <algorithm>

#include "cache_internal.cuh"
#include "ptx.cuh"
#include "qsa_internal.cuh"

namespace qsa {
namespace {

constexpr int SEL_THREADS = 1024, SEL_WARPS = SEL_THREADS / 32;
constexpr int MAX_CLUSTER = 16;   // not portable, but within a GB300 GPC
constexpr int BINS = 2048;
constexpr int MAX_KEYS = 40960;   // keys a CTA holds; longer runs are read again in every pass

struct alignas(16) SelectShared {
    int hist[3][BINS];
    int4 own[8];                         // this CTA's coarse counts
    int4 coarse[3][MAX_CLUSTER][8];      // each CTA's, which it puts into every CTA's (adding them there by atomics: 2 us a pass)
    int2 run[MAX_CLUSTER];   // kept for their key, and equal to the last key, of each CTA's run
    int warp_sums[SEL_WARPS], warp_ties[SEL_WARPS];
    int digit, left, same;
};

// Shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ void st_shared_rank4(int4 *p, uint32_t rank, int4 v) {
    asm volatile("st.shared::cluster.v4.s32 [%0], {%1, %2, %3, %4};" ::"r"(map_shared_rank(smem_u32(p), rank)), "r"(v.x),
                 "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ void st_shared_rank2(int2 *p, uint32_t rank, int2 v) {
    asm volatile("st.shared::cluster.v2.s32 [%0], {%1, %2};" ::"r"(map_shared_rank(smem_u32(p), rank)), "r"(v.x), "r"(v.y)
                 : "memory");
}
__device__ __forceinline__ int2 ld_shared_rank2(const int *p, uint32_t rank) {
    int2 v;
    asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];"
                 : "=r"(v.x), "=r"(v.y)
                 : "r"(map_shared_rank(smem_u32(p), rank))
                 : "memory");
    return v;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Inclusive prefix sum over the warp.
__device__ __forceinline__ int warp_scan(int x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(FULL_MASK, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

template <int kCluster>
__global__ void __launch_bounds__(SEL_THREADS) select_kernel(const CacheEvictArgs a, int max_keys) {
    constexpr int cluster = kCluster;
    extern __shared__ __align__(16) uint32_t keys[];
    __shared__ SelectShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int s = blockIdx.x / cluster, rank = blockIdx.x % cluster;
    for (int i = tid; i < 3 * BINS; i += SEL_THREADS) (&sh.hist[0][0])[i] = 0;
    grid_dependency_wait();
    grid_launch_dependents();
    const int n = min(max(ld_in(a.lens + s), 0), a.table_cols * a.kv.page_size), m = min(n, a.budget);
    const float *mass = a.mass + s * a.mass_stride;
    int32_t *kept = a.kept + static_cast<size_t>(s) * a.budget;
    float *nm = a.new_mass + s * a.new_mass_stride;
    if (rank == 0 && tid == 0) a.new_lens[s] = m;
    if (n <= a.budget) {   // the whole cluster leaves here
        const int all_tid = rank * SEL_THREADS + tid, all_threads = cluster * SEL_THREADS;
        for (int i = m + all_tid; i < a.new_mass_cols; i += all_threads) nm[i] = 0.0f;
        for (int i = all_tid; i < a.budget; i += all_threads) {
            kept[i] = i < m ? i : -1;
            if (i < m) nm[i] = ld_in(mass + i);
        }
        return;
    }
    // Sinks and recent cells; the candidates between them are [c0, c1).
    const int c0 = a.sinks, c1 = n - a.recent, recent_at = a.budget - a.recent;
    auto edges = [&](int thread, int threads) {   // of each CTA
        const int first = rank * threads + thread, step = cluster * threads;
        for (int i = first; i < a.sinks; i += step) {
            kept[i] = i;
            nm[i] = ld_in(mass + i);
        }
        for (int i = first; i < a.recent; i += step) {
            kept[recent_at + i] = c1 + i;
            nm[recent_at + i] = ld_in(mass + c1 + i);
        }
        for (int i = m + first; i < a.new_mass_cols; i += step) nm[i] = 0.0f;
    };
    int left = recent_at - a.sinks;   // candidates to keep
    if (left == 0) {
        edges(tid, SEL_THREADS);
        return;
    }
    if (cluster > 1) cluster_arrive();   // all CTAs have begun
    const int per = (c1 - c0 + cluster - 1) / cluster;
    const int j0 = min(c0 + rank * per, c1), count = min(per, c1 - j0);
    const bool held = per <= max_keys;   // a run's last quad fits too: max_keys is a multiple of 4
    // Keys i .. i + 3; 0, which is no cell's key, past the end.
    auto quad_at = [&](int i, uint32_t (&key)[4]) {
        if (held) {
            const uint4 k = *reinterpret_cast<const uint4 *>(keys + i);
            key[0] = k.x;
            key[1] = k.y;
            key[2] = k.z;
            key[3] = k.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) key[e] = i + e < count ? score_key(ld_in(mass + j0 + i + e)) : 0u;
        }
    };
    if (held && tid < 4 && count + tid < max_keys) keys[count + tid] = 0u;

    uint32_t prefix = 0;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass < 2 ? 2048 : 1024;
        int *hist = sh.hist[pass];
        __syncthreads();   // the counts are cleared
        if (pass == 0) {
            constexpr int BATCH = 8;   // masses under way at once
            for (int i0 = warp * 32; i0 < count; i0 += BATCH * SEL_THREADS) {
                float x[BATCH];
#pragma unroll
                for (int b = 0; b < BATCH; ++b) {
                    const int i = i0 + b * SEL_THREADS + lane;
                    if (i < count) x[b] = ld_in(mass + j0 + i);
                }
#pragma unroll
                for (int b = 0; b < BATCH; ++b) {
                    const int i = i0 + b * SEL_THREADS + lane;
                    if (i0 + b * SEL_THREADS >= count) break;
                    if (i < count) {
                        const uint32_t key = score_key(x[b]);
                        if (held) keys[i] = key;
                        atomicAdd(hist + (key >> shift), 1);
                    }
                }
            }
        } else {
            const int known = pass == 1 ? 21 : 10;   // bits above it are those of `prefix`
            for (int i = 4 * tid; i < count; i += 4 * SEL_THREADS) {
                uint32_t key[4];
                quad_at(i, key);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if ((key[e] ^ prefix) >> known == 0) atomicAdd(hist + ((key[e] >> shift) & (bins - 1)), 1);
            }
        }
        __syncthreads();
        const int each = bins / 32;   // of a coarse digit, one a warp
        const int sum = __reduce_add_sync(FULL_MASK, hist[warp * each + lane] + (each > 32 ? hist[warp * each + 32 + lane] : 0));
        if (lane == 0) reinterpret_cast<int *>(sh.own)[warp] = sum;
        __syncthreads();
        if (cluster > 1) {
            if (pass == 0) cluster_wait();
            if (tid < 8 * cluster) st_shared_rank4(&sh.coarse[pass][rank][tid & 7], tid >> 3, sh.own[tid & 7]);
            cluster_sync_all();
        }
        if (warp == 0) {
            // From the highest digit down: the coarse digit that the `left`-th key falls into, then the
            // digit within it, two per lane, for which all CTAs' counts are fetched.
            int mine = 0;
#pragma unroll
            for (int r = 0; r < cluster; ++r)
                mine += reinterpret_cast<const int *>(cluster > 1 ? sh.coarse[pass][r] : sh.own)[31 - lane];
            const int upto = warp_scan(mine);
            const int l = __ffs(__ballot_sync(FULL_MASK, upto >= left)) - 1, c = 31 - l;
            int before = __shfl_sync(FULL_MASK, upto - mine, l);
            const int at = each - 2 - 2 * lane;
            int low = 0, high = 0;
            if (at >= 0) {
                const int *counts = hist + c * each + at;
                int2 x[cluster];
#pragma unroll
                for (int r = 0; r < cluster; ++r) x[r] = cluster > 1 ? ld_shared_rank2(counts, r) : *reinterpret_cast<const int2 *>(counts);
#pragma unroll
                for (int r = 0; r < cluster; ++r) {
                    low += x[r].x;
                    high += x[r].y;
                }
            }
            const int upto2 = warp_scan(low + high);
            const int l2 = __ffs(__ballot_sync(FULL_MASK, before + upto2 >= left)) - 1;
            if (lane == l2) {
                before += upto2 - low - high;
                const bool upper = before + high >= left;
                sh.digit = c * each + at + upper;
                sh.left = left - before - (upper ? 0 : high);
                sh.same = upper ? high : low;
            }
        } else if (pass == 0) {
            edges(tid - 32, SEL_THREADS - 32);   // while the first warp searches
        }
        __syncthreads();
        prefix |= static_cast<uint32_t>(sh.digit) << shift;
        left = sh.left;
        if (left == sh.same) {   // all keys of the digit are kept: those above its lowest less one (not 0: no key is)
            --prefix;
            left = 0;
            break;
        }
    }

    // Keys above `prefix` are kept, and the first `left` that equal it. Each warp
    // takes a run of whole 128s, so that the lists stay in order.
    const int run = (count + 4 * SEL_THREADS - 1) / (4 * SEL_THREADS) * 128;
    const int r0 = min(warp * run, count), r1 = min(r0 + run, count);
    int above = 0, ties = 0;
    for (int i = r0 + 4 * lane; i < r1; i += 128) {
        uint32_t key[4];
        quad_at(i, key);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            above += key[e] > prefix;
            ties += key[e] == prefix;
        }
    }
    above = __reduce_add_sync(FULL_MASK, above);
    ties = __reduce_add_sync(FULL_MASK, ties);
    if (lane == 0) {
        sh.warp_sums[warp] = above;
        sh.warp_ties[warp] = ties;
    }
    __syncthreads();
    const int warp_above = sh.warp_sums[lane], warp_ties = sh.warp_ties[lane];
    int above_before = __reduce_add_sync(FULL_MASK, lane < warp ? warp_above : 0);
    int ties_before = __reduce_add_sync(FULL_MASK, lane < warp ? warp_ties : 0);
    if (cluster > 1) {
        if (warp == 0) {
            const int2 all = make_int2(__reduce_add_sync(FULL_MASK, warp_above), __reduce_add_sync(FULL_MASK, warp_ties));
            if (lane < cluster) st_shared_rank2(&sh.run[rank], lane, all);
        }
        // The last that a CTA does with another's memory is before this barrier: any may leave after it.
        cluster_sync_all();
        const int2 x = lane < rank ? sh.run[lane] : make_int2(0, 0);
        above_before += __reduce_add_sync(FULL_MASK, x.x);
        ties_before += __reduce_add_sync(FULL_MASK, x.y);
    }
    for (int i0 = r0; i0 < r1; i0 += 128) {
        const int i = i0 + 4 * lane;
        uint32_t key[4] = {0u, 0u, 0u, 0u};
        if (i < r1) quad_at(i, key);
        int own = 0;   // kept for the key, and equal keys x 2^16
#pragma unroll
        for (int e = 0; e < 4; ++e) own += key[e] > prefix ? 1 : key[e] == prefix ? 0x10000 : 0;
        const int upto = warp_scan(own), before = upto - own, all = __shfl_sync(FULL_MASK, upto, 31);
        int at = above_before + (before & 0xFFFF), tie = ties_before + (before >> 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool up = key[e] > prefix, eq = key[e] == prefix;
            if (up || (eq && tie < left)) {
                const int to = a.sinks + at + min(tie, left);
                kept[to] = j0 + i + e;
                // The mass is its key backwards, except that the key of -0 is +0's and NaN's is -infinity's.
                const bool lost = key[e] == 0x80000000u || key[e] == 0x007FFFFFu;
                nm[to] = lost ? ld_in(mass + j0 + i + e) : __uint_as_float((key[e] >> 31) ? key[e] ^ 0x80000000u : ~key[e]);
            }
            at += up;
            tie += eq;
        }
        above_before += all & 0xFFFF;
        ties_before += all >> 16;
    }
}

constexpr int COPY_THREADS = 256, COPY_BATCH = 4;

// kVecs: 16-byte pieces of one head's row. A warp moves one cell at a time, its
// addresses found once, up to BATCH pieces of keys and of values per lane.
template <int kVecs>
__global__ void __launch_bounds__(COPY_THREADS) copy_cells_kernel(const CacheEvictArgs a, Divider page) {
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int ELEM = kVecs == 8 ? 1 : 2, BATCH = COPY_BATCH;
    const int lane = threadIdx.x & 31, s = blockIdx.y;
    const int m = ld_in(a.new_lens + s), pieces = a.kv.nkv * kVecs;
    char *k = static_cast<char *>(a.kv.k), *v = static_cast<char *>(a.kv.v);
    const int64_t head_bytes = a.kv.head_stride * ELEM;
    for (int i = blockIdx.x * (COPY_THREADS / 32) + (threadIdx.x >> 5); i < m; i += gridDim.x * (COPY_THREADS / 32)) {
        const int j = ld_in(a.kept + static_cast<size_t>(s) * a.budget + i);
        const int jp = divide(page, j), ip = divide(page, i);
        const int src = ld_in(a.table + s * a.table_stride + jp), dst = ld_in(a.new_table + s * a.new_table_stride + ip);
        if (src < 0 || src >= a.kv.npages || dst < 0 || dst >= a.kv.npages) continue;
        const int js = j - jp * a.kv.page_size, is = i - ip * a.kv.page_size;
        const int64_t from = (src * a.kv.page_stride + js * a.kv.cell_stride) * ELEM;
        const int64_t to = (dst * a.kv.page_stride + is * a.kv.cell_stride) * ELEM;
        for (int c0 = 0; c0 < pieces; c0 += 32 * BATCH) {
            uint4 x[BATCH], y[BATCH];
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const int c = c0 + 32 * b + lane;
                const int64_t off = from + (c / kVecs) * head_bytes + 16 * (c % kVecs);
                if (c < pieces) {
                    x[b] = ld_in(reinterpret_cast<const uint4 *>(k + off));
                    y[b] = ld_in(reinterpret_cast<const uint4 *>(v + off));
                }
            }
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const int c = c0 + 32 * b + lane;
                const int64_t off = to + (c / kVecs) * head_bytes + 16 * (c % kVecs);
                if (c < pieces) {
                    *reinterpret_cast<uint4 *>(k + off) = x[b];
                    *reinterpret_cast<uint4 *>(v + off) = y[b];
                }
            }
        }
        if constexpr (ELEM == 1) {
            const int64_t f = src * a.kv.scale_page_stride + js * a.kv.scale_cell_stride;
            const int64_t g = dst * a.kv.scale_page_stride + is * a.kv.scale_cell_stride;
            for (int h = lane; h < a.kv.nkv; h += 32) {
                const uint16_t x = ld_in_u16(a.kv.k_scale_f16 + f + h * a.kv.scale_head_stride);
                const uint16_t y = ld_in_u16(a.kv.v_scale_f16 + f + h * a.kv.scale_head_stride);
                a.kv.k_scale_f16[g + h * a.kv.scale_head_stride] = x;
                a.kv.v_scale_f16[g + h * a.kv.scale_head_stride] = y;
            }
        }
    }
}

// The same for cells of few pieces: a thread moves COPY_BATCH pieces of keys
// and of values at a time, consecutive threads consecutive pieces of a
// cell and then the next cells, so a warp is full whatever the heads' number.
template <int kVecs>
__global__ void __launch_bounds__(COPY_THREADS) copy_pieces_kernel(const CacheEvictArgs a, Divider page, Divider per_cell) {
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int ELEM = kVecs == 8 ? 1 : 2;
    const int s = blockIdx.y, m = ld_in(a.new_lens + s);
    const char *k = static_cast<const char *>(a.kv.k), *v = static_cast<const char *>(a.kv.v);
    const int32_t *kept = a.kept + static_cast<size_t>(s) * a.budget;
    const int32_t *table = a.table + s * a.table_stride, *new_table = a.new_table + s * a.new_table_stride;
    const long long pieces = static_cast<long long>(m) * per_cell.d, step = static_cast<long long>(gridDim.x) * COPY_THREADS;
    // Cells and pieces in 32 bits: a thread's pieces are told apart by whole cells first.
    for (long long t0 = static_cast<long long>(blockIdx.x) * COPY_THREADS + threadIdx.x; t0 < pieces; t0 += COPY_BATCH * step) {
        int64_t from[COPY_BATCH], to[COPY_BATCH], scale_from[COPY_BATCH], scale_to[COPY_BATCH];
        uint4 x[COPY_BATCH], y[COPY_BATCH];
        int cell[COPY_BATCH], piece[COPY_BATCH], j[COPY_BATCH];
        bool ok[COPY_BATCH];
#pragma unroll
        for (int b = 0; b < COPY_BATCH; ++b) {
            const long long t = t0 + b * step;
            ok[b] = t < pieces;
            cell[b] = ok[b] ? (t < 0x7FFFFFFFLL ? static_cast<int>(divide(per_cell, static_cast<uint32_t>(t))) : static_cast<int>(t / per_cell.d)) : 0;
            piece[b] = ok[b] ? static_cast<int>(t - static_cast<long long>(cell[b]) * per_cell.d) : 0;
            j[b] = ok[b] ? ld_in(kept + cell[b]) : 0;
        }
#pragma unroll
        for (int b = 0; b < COPY_BATCH; ++b) {
            const int jp = divide(page, j[b]), ip = divide(page, cell[b]);
            const int src = ok[b] ? ld_in(table + jp) : -1, dst = ok[b] ? ld_in(new_table + ip) : -1;
            ok[b] = src >= 0 && src < a.kv.npages && dst >= 0 && dst < a.kv.npages;
            const int js = j[b] - jp * a.kv.page_size, is = cell[b] - ip * a.kv.page_size, h = piece[b] / kVecs;
            const int64_t off = h * a.kv.head_stride * ELEM + 16 * (piece[b] % kVecs);
            from[b] = (src * a.kv.page_stride + js * a.kv.cell_stride) * ELEM + off;
            to[b] = (dst * a.kv.page_stride + is * a.kv.cell_stride) * ELEM + off;
            if constexpr (ELEM == 1) {
                scale_from[b] = src * a.kv.scale_page_stride + js * a.kv.scale_cell_stride + h * a.kv.scale_head_stride;
                scale_to[b] = dst * a.kv.scale_page_stride + is * a.kv.scale_cell_stride + h * a.kv.scale_head_stride;
            }
        }
#pragma unroll
        for (int b = 0; b < COPY_BATCH; ++b)
            if (ok[b]) {
                x[b] = ld_in(reinterpret_cast<const uint4 *>(k + from[b]));
                y[b] = ld_in(reinterpret_cast<const uint4 *>(v + from[b]));
            }
        if constexpr (ELEM == 1) {   // the scales with each head's first piece
            uint16_t ks[COPY_BATCH], vs[COPY_BATCH];
#pragma unroll
            for (int b = 0; b < COPY_BATCH; ++b)
                if (ok[b] && piece[b] % kVecs == 0) {
                    ks[b] = ld_in_u16(a.kv.k_scale_f16 + scale_from[b]);
                    vs[b] = ld_in_u16(a.kv.v_scale_f16 + scale_from[b]);
                }
#pragma unroll
            for (int b = 0; b < COPY_BATCH; ++b)
                if (ok[b] && piece[b] % kVecs == 0) {
                    a.kv.k_scale_f16[scale_to[b]] = ks[b];
                    a.kv.v_scale_f16[scale_to[b]] = vs[b];
                }
        }
#pragma unroll
        for (int b = 0; b < COPY_BATCH; ++b)
            if (ok[b]) {
                *reinterpret_cast<uint4 *>(static_cast<char *>(a.kv.k) + to[b]) = x[b];
                *reinterpret_cast<uint4 *>(static_cast<char *>(a.kv.v) + to[b]) = y[b];
            }
    }
}

}  // namespace

// CTAs of a sequence. One searches what a few rounds of its threads cover; the
// longer the cache, the more, as long as all sequences' clusters run at once (the
// GPU holds one of 16 CTAs per GPC, two of 8). Measured, whole call with 16, 8, 4 and 1
// CTAs, a quarter of the cells kept: 9 x 9,607 cells 35.9, 28.2, 28.1 and 29.6 us; 4 x
// 20,000 cells 28.4, 27.7, 29.0 and 33.7; 1 x 30,000 cells 18.5, 18.2, 19.9 and 29.0; 2 x
// 60,000 cells 28.6, 29.4, 33.2 and 64.3; 16 x 13,337 cells of one head 34.8, 25.4, 20.1
// and 22.6; 1 x 2,000 cells 10.2, 9.3, 9.0 and 7.2. The length is the table's width, as the
// sequences' own are on the device alone.
static int cluster_size(int capacity, int nseq) {
    int cluster = capacity <= 4 * SEL_THREADS ? 1 : capacity <= 16 * SEL_THREADS ? 4 : capacity <= 48 * SEL_THREADS ? 8 : MAX_CLUSTER;
    while (cluster > 4 && static_cast<long long>(cluster) * nseq > device_sm_count() && 2LL * capacity <= static_cast<long long>(cluster) * MAX_KEYS)
        cluster /= 2;
    return cluster;
}

template <int kCluster>
static cudaError_t launch_select(const CacheEvictArgs &a, int capacity, cudaLaunchConfig_t cfg) {
    static thread_local int configured_device = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && configured_device != dev) {
        e = cudaFuncSetAttribute(select_kernel<kCluster>, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_KEYS * 4);
        if (e == cudaSuccess && kCluster > 8)
            e = cudaFuncSetAttribute(select_kernel<kCluster>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess) configured_device = dev;
    }
    if (e != cudaSuccess) return e;
    const int max_keys = std::min((capacity + kCluster - 1) / kCluster + 3, MAX_KEYS) & ~3;   // whole quads
    cfg.gridDim = dim3(static_cast<unsigned>(a.nseq * kCluster));
    cfg.blockDim = dim3(SEL_THREADS);
    cfg.dynamicSmemBytes = 4 * max_keys;
    return cudaLaunchKernelEx(&cfg, select_kernel<kCluster>, a, max_keys);
}

cudaError_t launch_cache_evict(const CacheEvictArgs &a, cudaStream_t stream) {
    const int capacity = a.table_cols * a.kv.page_size, cluster = cluster_size(capacity, a.nseq);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = cluster;
    attrs[1].val.clusterDim.y = 1;
    attrs[1].val.clusterDim.z = 1;
    cfg.stream = stream;
    cfg.attrs = attrs;
    cfg.numAttrs = 2;
    const cudaError_t e = cluster == 1   ? launch_select<1>(a, capacity, cfg)
                          : cluster == 4 ? launch_select<4>(a, capacity, cfg)
                          : cluster == 8 ? launch_select<8>(a, capacity, cfg)
                                         : launch_select<MAX_CLUSTER>(a, capacity, cfg);
    if (e != cudaSuccess) return e;
    // Cells of at least two pieces per lane go to whole warps (8 heads of int8, 64 pieces: 26
    // sequences of 527 cells 14.1 us against 14.9 by pieces; 2 x 131,072 cells 40.3 against 47.4);
    // smaller ones by pieces (4 heads, 32 pieces: 8 x 20,000 cells 40.3 us against 42.8; 1 head, 8
    // pieces: 16 x 13,337 cells 22.9 against 47.9).
    const int per_cell = a.kv.nkv * (a.kv.dtype == QSA_I8 ? 8 : 16);
    const bool cells = per_cell >= 64;
    const long long wanted = cells ? (a.budget + COPY_THREADS / 32 - 1) / (COPY_THREADS / 32)
                                   : (static_cast<long long>(a.budget) * per_cell + COPY_THREADS * COPY_BATCH - 1) / (COPY_THREADS * COPY_BATCH);
    // As many CTAs as the GPU holds.
    const long long blocks = std::min(wanted, std::max(1LL, 8LL * device_sm_count() / a.nseq));
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), a.nseq);
    cfg.blockDim = dim3(COPY_THREADS);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    const Divider page = make_divider(a.kv.page_size), cell = make_divider(per_cell);
    const bool int8 = a.kv.dtype == QSA_I8;
    if (cells)
        return int8 ? cudaLaunchKernelEx(&cfg, copy_cells_kernel<8>, a, page) : cudaLaunchKernelEx(&cfg, copy_cells_kernel<16>, a, page);
    return int8 ? cudaLaunchKernelEx(&cfg, copy_pieces_kernel<8>, a, page, cell)
                : cudaLaunchKernelEx(&cfg, copy_pieces_kernel<16>, a, page, cell);
}

}  // namespace qsa
