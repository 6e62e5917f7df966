// Eviction by accumulated attention weight: per sequence the first `sinks`
// cells, the last `recent` cells and, of the cells between, those of largest
// mass are kept in order and copied to new pages.
//
// Two launches. evict_select_kernel: one CTA per sequence finds the mass of
// the last cell to keep by a radix search on the order-preserving key of
// csrc/qsa_internal.cuh, 8 bits per pass over shared-memory histograms (the
// search is exact: it ends with the 32-bit key of that cell and how many of
// the cells with that very key are kept, lowest first), then lists the kept
// cells in order by block scans. evict_copy_kernel: one thread per 16 bytes.
#include "cache_internal.cuh"
#include "ptx.cuh"
#include "qsa_internal.cuh"

namespace qsa {
namespace {

constexpr int SEL_THREADS = 1024;

// Inclusive scan over the CTA of one int per thread; the total in *total.
__device__ __forceinline__ int block_scan(int x, int *warp_sums, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(FULL_MASK, v, o);
        if (lane >= o) v += y;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int w = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(FULL_MASK, w, o);
            if (lane >= o) w += y;
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    *total = warp_sums[31];
    return v + (warp > 0 ? warp_sums[warp - 1] : 0);
}

__global__ void __launch_bounds__(SEL_THREADS) evict_select_kernel(const CacheEvictArgs a) {
    __shared__ int hist[256], warp_sums[32], sh_digit, sh_left;
    const int s = blockIdx.x, tid = threadIdx.x;
    const int n = min(max(a.lens[s], 0), a.table_cols * a.kv.page_size), m = min(n, a.budget);
    const float *mass = a.mass + s * a.mass_stride;
    int32_t *kept = a.kept + static_cast<size_t>(s) * a.budget;
    float *nm = a.new_mass + s * a.new_mass_stride;
    if (tid == 0) a.new_lens[s] = m;
    if (n <= a.budget) {
        for (int i = tid; i < a.budget; i += SEL_THREADS) kept[i] = i < m ? i : -1;
        for (int i = tid; i < a.new_mass_cols; i += SEL_THREADS) nm[i] = i < m ? mass[i] : 0.0f;
        return;
    }
    // Candidates: [c0, c1); `left` of them are kept.
    const int c0 = a.sinks, c1 = n - a.recent;
    int left = a.budget - a.sinks - a.recent;
    uint32_t prefix = 0;
    if (left > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += SEL_THREADS) hist[i] = 0;
            __syncthreads();
            for (int j = c0 + tid; j < c1; j += SEL_THREADS) {
                const uint32_t key = score_key(mass[j]);
                if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(key >> shift) & 255u], 1);
            }
            __syncthreads();
            if (tid == 0) {
                int d = 255, need = left;
                for (; d > 0 && hist[d] < need; --d) need -= hist[d];
                sh_digit = d;
                sh_left = need;
            }
            __syncthreads();
            prefix |= static_cast<uint32_t>(sh_digit) << shift;
            left = sh_left;
            __syncthreads();
        }
    }
    // Keys above `prefix` are kept, and the first `left` equal to it. In order:
    int out = 0, ties = 0;
    const bool none = a.budget == a.sinks + a.recent;
    for (int base = 0; base < n; base += SEL_THREADS) {
        const int j = base + tid;
        const bool mid = j >= c0 && j < c1;
        const uint32_t key = mid ? score_key(mass[j]) : 0u;
        const bool tie = mid && !none && key == prefix;
        int nties, ntaken;
        const int trank = block_scan(tie, warp_sums, &nties) + ties;
        const bool take = j < n && (!mid || (!none && (key > prefix || (tie && trank <= left))));
        const int at = block_scan(take, warp_sums, &ntaken) + out - 1;
        if (take) {
            kept[at] = j;
            nm[at] = mass[j];
        }
        ties += nties;
        out += ntaken;
    }
    for (int i = a.budget + tid; i < a.new_mass_cols; i += SEL_THREADS) nm[i] = 0.0f;
}

// Copies cell i of sequence s, 16 bytes of one head's K and V per thread.
__global__ void __launch_bounds__(256) evict_copy_kernel(const CacheEvictArgs a) {
    const int s = blockIdx.y;
    const int elem = a.kv.dtype == QSA_I8 ? 1 : 2, vecs = 128 * elem / 16, per = a.kv.nkv * vecs;
    const int m = a.new_lens[s];
    for (long long t = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; t < static_cast<long long>(m) * per;
         t += static_cast<long long>(gridDim.x) * 256) {
        const int i = static_cast<int>(t / per), r = static_cast<int>(t % per), h = r / vecs, c = r % vecs;
        const int j = a.kept[static_cast<size_t>(s) * a.budget + i];
        const int src = a.table[s * a.table_stride + j / a.kv.page_size];
        const int dst = a.new_table[s * a.new_table_stride + i / a.kv.page_size];
        if (src < 0 || src >= a.kv.npages || dst < 0 || dst >= a.kv.npages) continue;
        const int js = j % a.kv.page_size, is = i % a.kv.page_size;
        const int64_t from = (src * a.kv.page_stride + js * a.kv.cell_stride + h * a.kv.head_stride) * elem + 16 * c;
        const int64_t to = (dst * a.kv.page_stride + is * a.kv.cell_stride + h * a.kv.head_stride) * elem + 16 * c;
        char *k = static_cast<char *>(a.kv.k), *v = static_cast<char *>(a.kv.v);
        const uint4 x = ld_in(reinterpret_cast<const uint4 *>(k + from)), y = ld_in(reinterpret_cast<const uint4 *>(v + from));
        *reinterpret_cast<uint4 *>(k + to) = x;
        *reinterpret_cast<uint4 *>(v + to) = y;
        if (a.kv.dtype == QSA_I8 && c == 0) {
            const int64_t f = src * a.kv.scale_page_stride + js * a.kv.scale_cell_stride + h * a.kv.scale_head_stride;
            const int64_t g = dst * a.kv.scale_page_stride + is * a.kv.scale_cell_stride + h * a.kv.scale_head_stride;
            a.kv.k_scale_f16[g] = a.kv.k_scale_f16[f];
            a.kv.v_scale_f16[g] = a.kv.v_scale_f16[f];
        }
    }
}

}  // namespace

cudaError_t launch_cache_evict(const CacheEvictArgs &a, cudaStream_t stream) {
    evict_select_kernel<<<a.nseq, SEL_THREADS, 0, stream>>>(a);
    evict_copy_kernel<<<dim3(512, a.nseq), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace qsa
