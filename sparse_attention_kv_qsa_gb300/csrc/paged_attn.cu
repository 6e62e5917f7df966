// Attention of one new token per sequence over its paged cache, with a
// sliding window, always-visible first cells, and the weight each cell
// received added to a running mass.
//
//   s_hj = scale q_h . k_j;  lse_h = log sum_j exp(s_hj);  out_h = sum_j exp(s_hj - lse_h) v_j
//   mass_out_j = mass_j + sum_h exp(s_hj - lse_h)
//
// One warp per sequence and head in fp32 on CUDA cores, one cell at a time.
#include "attn_row.cuh"
#include "cache_internal.cuh"

namespace qsa {
namespace {

struct Cell {
    const void *k, *v;
    float ks, vs;
    bool ok;
};

template <typename KT>
__device__ __forceinline__ Cell find_cell(const PagedAttnArgs &a, int s, int j, int head) {
    const int page = __ldcg(a.table + s * a.table_stride + j / a.kv.page_size), slot = j % a.kv.page_size;
    Cell c{nullptr, nullptr, 1.0f, 1.0f, page >= 0 && page < a.kv.npages};
    if (!c.ok) return c;
    const int64_t at = page * a.kv.page_stride + slot * a.kv.cell_stride + head * a.kv.head_stride;
    c.k = static_cast<const KT *>(a.kv.k) + at;
    c.v = static_cast<const KT *>(a.kv.v) + at;
    if constexpr (sizeof(KT) == 1) {
        const int64_t sc = page * a.kv.scale_page_stride + slot * a.kv.scale_cell_stride + head * a.kv.scale_head_stride;
        c.ks = __half2float(__ushort_as_half(ld_in_u16(a.kv.k_scale_f16 + sc)));
        c.vs = __half2float(__ushort_as_half(ld_in_u16(a.kv.v_scale_f16 + sc)));
    }
    return c;
}

template <typename KT, typename QT>
__global__ void __launch_bounds__(128) paged_rows_kernel(const PagedAttnArgs a, float *lse2) {
    const int lane = threadIdx.x & 31;
    const long long w = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (w >= static_cast<long long>(a.nseq) * a.nheads) return;
    const int s = static_cast<int>(w / a.nheads), h = static_cast<int>(w % a.nheads), kvh = h / (a.nheads / a.kv.nkv);
    const int n = min(max(a.lens[s], 0), a.table_cols * a.kv.page_size);
    const int lo = a.window < 0 ? 0 : max(0, n - a.window);
    const float4 q = load4(static_cast<const QT *>(a.q) + s * a.q_seq_stride + h * a.q_head_stride + 4 * lane);
    RowState r;
    auto span = [&](int j0, int j1) {
        for (int j = j0; j < j1; ++j) {
            const Cell c = find_cell<KT>(a, s, j, kvh);
            if (!c.ok) continue;
            const float x = warp_sum(dot4(q, load4(static_cast<const KT *>(c.k) + 4 * lane))) * c.ks * a.scale * LOG2E;
            float4 v = load4(static_cast<const KT *>(c.v) + 4 * lane);
            r.add(x, make_float4(v.x * c.vs, v.y * c.vs, v.z * c.vs, v.w * c.vs));
        }
    };
    span(0, min(a.sinks, lo));
    span(lo, n);
    store4(static_cast<QT *>(a.out) + w * 128 + 4 * lane, r.result());
    if (lane == 0) {
        if (a.lse != nullptr) a.lse[w] = (r.m + log2f(r.l)) * LN2;
        if (lse2 != nullptr) lse2[w] = r.m + log2f(r.l);
    }
}

template <typename KT, typename QT>
__global__ void __launch_bounds__(256) paged_mass_kernel(const PagedAttnArgs a, const float *lse2) {
    const int lane = threadIdx.x & 31, s = blockIdx.y;
    const int n = min(max(a.lens[s], 0), a.table_cols * a.kv.page_size);
    const int lo = a.window < 0 ? 0 : max(0, n - a.window);
    for (int j = blockIdx.x * 8 + (threadIdx.x >> 5); j < n; j += gridDim.x * 8) {
        float got = 0.0f;
        if (j >= lo || j < a.sinks) {
            for (int h = 0; h < a.nheads; ++h) {
                const Cell c = find_cell<KT>(a, s, j, h / (a.nheads / a.kv.nkv));
                if (!c.ok) continue;
                const float4 q = load4(static_cast<const QT *>(a.q) + s * a.q_seq_stride + h * a.q_head_stride + 4 * lane);
                const float x = warp_sum(dot4(q, load4(static_cast<const KT *>(c.k) + 4 * lane))) * c.ks * a.scale * LOG2E;
                got += exp2f(x - lse2[static_cast<size_t>(s) * a.nheads + h]);
            }
        }
        if (lane == 0) a.mass_out[s * a.mass_stride + j] = a.mass[s * a.mass_stride + j] + got;
    }
}

template <typename KT, typename QT>
cudaError_t launch(const PagedAttnArgs &a, cudaStream_t stream) {
    const long long warps = static_cast<long long>(a.nseq) * a.nheads;
    float *lse2 = a.mass != nullptr ? static_cast<float *>(a.scratch) : nullptr;
    paged_rows_kernel<KT, QT><<<static_cast<unsigned>((warps + 3) / 4), 128, 0, stream>>>(a, lse2);
    if (a.mass != nullptr && a.table_cols > 0)
        paged_mass_kernel<KT, QT><<<dim3(256, a.nseq), 256, 0, stream>>>(a, lse2);
    return cudaGetLastError();
}

}  // namespace

size_t paged_attn_scratch_bytes(int nseq, int nheads, int, int, bool) {
    return static_cast<size_t>(nseq) * nheads * sizeof(float);
}

cudaError_t launch_paged_attn(const PagedAttnArgs &a, cudaStream_t stream) {
    if (a.kv.dtype == QSA_BF16) return launch<__nv_bfloat16, __nv_bfloat16>(a, stream);
    if (a.kv.dtype == QSA_F16) return launch<__half, __half>(a, stream);
    if (a.q_dtype == QSA_F32) return launch<int8_t, float>(a, stream);
    if (a.q_dtype == QSA_F16) return launch<int8_t, __half>(a, stream);
    return launch<int8_t, __nv_bfloat16>(a, stream);
}

}  // namespace qsa
