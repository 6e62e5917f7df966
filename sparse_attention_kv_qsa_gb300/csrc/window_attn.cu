// Prompt attention over ragged sequences: causal, within a sliding window,
// with the first tokens (sinks) always visible.
//
//   visible(i, j): j <= pos_i and (window < 0 or j > pos_i - window or j < sinks),  pos_i = nk - nq + i
//   s_ij = scale q_i . k_j;  lse_i = log sum_j exp(s_ij);  out_i = sum_j exp(s_ij - lse_i) v_j
//
// One warp per query row and head in fp32 on CUDA cores, one key at a time.
#include "attn_row.cuh"
#include "cache_internal.cuh"

namespace qsa {
namespace {

template <typename T>
__global__ void __launch_bounds__(256) window_rows_kernel(const WindowAttnArgs a) {
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int s = blockIdx.z, h = blockIdx.y, i = blockIdx.x * 8 + warp;
    const int q0 = min(max(a.cu_q[s], 0), a.total_q), q1 = min(max(a.cu_q[s + 1], q0), a.total_q);
    const int k0 = min(max(a.cu_k[s], 0), a.total_k), k1 = min(max(a.cu_k[s + 1], k0), a.total_k);
    if (i >= q1 - q0) return;
    const int kvh = h / (a.nheads / a.nkv);
    const long long pos = static_cast<long long>(k1 - k0) - (q1 - q0) + i;
    const float4 q = load4(static_cast<const T *>(a.q) + (q0 + i) * a.q_tok + h * a.q_head + 4 * lane);
    const T *kp = static_cast<const T *>(a.k) + kvh * a.k_head + 4 * lane;
    const T *vp = static_cast<const T *>(a.v) + kvh * a.v_head + 4 * lane;
    const float c = a.scale * LOG2E;
    RowState r;
    const long long end = pos + 1;
    const long long lo = a.window < 0 ? 0 : max(0LL, end - a.window);
    auto span = [&](long long j0, long long j1) {
        for (long long j = j0; j < j1; ++j) {
            const float x = c * warp_sum(dot4(q, load4(kp + (k0 + j) * a.k_tok)));
            r.add(x, load4(vp + (k0 + j) * a.v_tok));
        }
    };
    span(0, min(min(static_cast<long long>(a.sinks), lo), end));
    span(lo, end);
    const size_t row = static_cast<size_t>(q0 + i) * a.nheads + h;
    store4(static_cast<T *>(a.out) + row * 128 + 4 * lane, r.result());
    if (a.lse != nullptr && lane == 0) a.lse[row] = (r.m + log2f(r.l)) * LN2;
}

}  // namespace

size_t window_attn_scratch_bytes(int, int, int, int, int) { return 0; }

cudaError_t launch_window_attn(const WindowAttnArgs &a, cudaStream_t stream) {
    const dim3 grid((a.max_q + 7) / 8, a.nheads, a.nseq);
    if (a.dtype == QSA_BF16)
        window_rows_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(a);
    else
        window_rows_kernel<__half><<<grid, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace qsa
