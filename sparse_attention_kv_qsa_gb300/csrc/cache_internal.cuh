// Internal launch interface of the bounded-cache operators (cache_api.cu and
// the kernels of paged_attn.cu, window_attn.cu, cache_evict.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/qsa.h"

namespace qsa {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

// floor(n / d) for 0 <= n < 2^31, by multiplication.
struct Divider {
    uint32_t d, mul, shift;
};
inline Divider make_divider(uint32_t d) {
    if (d == 1) return {1, 0, 0};
    uint32_t l = 0;
    while ((1ull << l) < d) ++l;
    return {d, static_cast<uint32_t>(((1ull << (31 + l)) + d - 1) / d), l - 1};
}
__device__ __forceinline__ uint32_t divide(Divider v, uint32_t n) { return v.d == 1 ? n : __umulhi(n, v.mul) >> v.shift; }

struct PagedAttnArgs {
    const void *q;
    qsa_dtype q_dtype;
    int64_t q_seq_stride, q_head_stride;
    int nseq, nheads;
    qsa_kv_pages kv;
    const int32_t *table;
    int table_cols;
    int64_t table_stride;
    const int32_t *lens;
    int window, sinks;
    float scale;
    void *out;
    float *lse;
    const float *mass;
    float *mass_out;
    int64_t mass_stride;
    void *scratch;
};

size_t paged_attn_scratch_bytes(int nseq, int nheads, int nkv, int capacity, bool with_mass);
cudaError_t launch_paged_attn(const PagedAttnArgs &a, cudaStream_t stream);

// Paged attention's partial results, for another kernel to add: of unit `kvh * parts + part` of sequence s, whole in
// rows [nseq][nheads][132] where meta[s * units + unit].x < 0, else in ranges of slots as its join reads them
// (128 sums, reference in base 2, weights' sum). Sequences without a cell leave nothing.
struct PagedPartial {
    const float *rows, *slots;
    const int4 *meta;
    int parts, units, heads_per_unit, grid;
};

// What prefix_share.cuh's functions go by.
struct PrefixShare {
    const int32_t *cu, *prefix_lens;
    int ngroups, nseq, capacity, nkv;
    int seqs, block;          // sequences of a row tile, and of a block of rows
    int sms, grid;            // SMs, CTAs of the prefix's kernel
    int whole;                // nothing is divided: no block has two row tiles, or both kernels' grids have room
    int one_tile_ns, two_tiles_ns;
    float own_tile_ns, own_unit_ns;   // paged attention's tile of cells, and unit of a sequence and KV head
    int own_units;
};

size_t paged_partial_bytes(int nseq, int nheads, int nkv, int capacity);
// The units and CTAs of a call, for PrefixShare.
int paged_units(const PagedAttnArgs &a);
int paged_ctas(const PagedAttnArgs &a);
// Launched behind the shared prefix's kernel, with which it shares the GPU.
cudaError_t launch_paged_partial(const PagedAttnArgs &a, const PrefixShare &share, PagedPartial &left, cudaStream_t stream);

struct PrefixAttnArgs {
    const void *q;
    qsa_dtype q_dtype;
    int64_t q_seq_stride, q_head_stride;
    int nseq, nheads;
    qsa_kv_pages kv;
    const int32_t *prefix_table;
    int prefix_cols;
    int64_t prefix_stride;
    const int32_t *prefix_lens, *cu;
    int ngroups;
    const int32_t *table;
    int table_cols;
    int64_t table_stride;
    const int32_t *lens;
    float scale;
    void *out;
    float *lse;
    void *scratch;
};
struct PrefixAttnSizes {
    int nseq, ngroups, nheads, nkv, prefix_capacity, capacity;
};

size_t prefix_attn_scratch_bytes(const PrefixAttnSizes &z);
cudaError_t launch_prefix_attn(const PrefixAttnArgs &a, cudaStream_t stream);

struct WindowAttnArgs {
    const void *q, *k, *v;
    qsa_dtype dtype;
    int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head;
    const int32_t *cu_q, *cu_k;
    int nseq, total_q, total_k, max_q, nheads, nkv, window, sinks;
    float scale;
    void *out;
    float *lse;
    void *scratch;
};

size_t window_attn_scratch_bytes(int nseq, int total_q, int nheads, int nkv);
cudaError_t launch_window_attn(const WindowAttnArgs &a, cudaStream_t stream);

struct CacheEvictArgs {
    qsa_kv_pages kv;
    int nseq;
    const int32_t *table;
    int table_cols;
    int64_t table_stride;
    const int32_t *lens;
    const float *mass;
    int64_t mass_stride;
    const int32_t *new_table;
    int new_cols;
    int64_t new_table_stride;
    int budget, sinks, recent;
    int32_t *kept, *new_lens;
    float *new_mass;
    int64_t new_mass_stride;
    int new_mass_cols;
};

cudaError_t launch_cache_evict(const CacheEvictArgs &a, cudaStream_t stream);

cudaError_t launch_rotate(const void *x, int dtype, const int64_t *strides, int ntok, int nheads, const qsa_rotation &rot,
                          void *out, cudaStream_t stream);

struct CacheAppendArgs {
    const void *k, *v, *q;
    int dtype;
    const int64_t *strides;   // of k, v, q, q_out, k_out per token and head
    int ntok, nheads;
    qsa_kv_pages kv;
    const int32_t *table;
    int table_cols;
    int64_t table_stride;
    const int32_t *lens, *cu;
    int nseq;
    const qsa_rotation *rotation;
    void *q_out, *k_out;
};

cudaError_t launch_cache_append(const CacheAppendArgs &a, cudaStream_t stream);

}  // namespace qsa
