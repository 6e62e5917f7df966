// C ABI of the bounded-cache operators: argument checks, then launches on the
// caller's stream. Declarations and the contract: include/qsa.h.
#include <cmath>
#include <cstdint>

#include "cache_internal.cuh"

namespace {

constexpr long long MAX_SEQS = 65535, MAX_HEADS = 65535, MAX_CELLS = 1LL << 30, MAX_TILES = 1LL << 38;

bool aligned(const void *p, uintptr_t n) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int element_size(int dtype) { return dtype == QSA_F32 ? 4 : dtype == QSA_I8 ? 1 : 2; }

// A stride that 16-byte accesses can use.
bool good_stride(int64_t elements, int dtype) { return elements >= 0 && elements * element_size(dtype) % 16 == 0; }

// The kernels work in base 2, with scale log2(e) in fp32.
bool good_scale(float scale) { return scale > 0.0f && std::isfinite(scale * qsa::LOG2E); }

qsa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? QSA_OK : QSA_ERR_CUDA; }

qsa_status check_pages(const qsa_kv_pages *kv) {
    if (kv == nullptr || (kv->dtype != QSA_BF16 && kv->dtype != QSA_F16 && kv->dtype != QSA_I8)) return QSA_ERR_INVALID;
    if (kv->npages < 0 || kv->page_size < 1 || kv->nkv < 1) return QSA_ERR_INVALID;
    if (!good_stride(kv->page_stride, kv->dtype) || !good_stride(kv->cell_stride, kv->dtype) ||
        !good_stride(kv->head_stride, kv->dtype))
        return QSA_ERR_INVALID;
    if (kv->npages > 0 && (!aligned(kv->k, 16) || !aligned(kv->v, 16))) return QSA_ERR_INVALID;
    if (kv->dtype == QSA_I8) {
        if (kv->npages > 0 && (!aligned(kv->k_scale_f16, 2) || !aligned(kv->v_scale_f16, 2))) return QSA_ERR_INVALID;
        if (kv->scale_page_stride < 0 || kv->scale_cell_stride < 0 || kv->scale_head_stride < 0) return QSA_ERR_INVALID;
    } else if (kv->k_scale_f16 != nullptr || kv->v_scale_f16 != nullptr) {
        return QSA_ERR_INVALID;
    }
    return kv->nkv > MAX_HEADS ? QSA_ERR_UNSUPPORTED : QSA_OK;
}

// A page table of nseq rows (its pointer is checked by the caller's rule for empty work).
qsa_status check_table(int cols, int64_t stride, int page_size) {
    if (cols < 0 || stride < cols) return QSA_ERR_INVALID;
    return static_cast<long long>(cols) * page_size > MAX_CELLS ? QSA_ERR_UNSUPPORTED : QSA_OK;
}

}  // namespace

extern "C" {

size_t qsa_paged_attn_scratch_bytes(int nseq, int nheads, int nkv, int table_cols, int page_size, int with_mass) {
    // A table without columns is a call like any other: every sequence is empty, and the kernels say so in scratch.
    if (nseq < 1 || nheads < 1 || nkv < 1 || nheads % nkv != 0 || table_cols < 0 || page_size < 1 ||
        nseq > MAX_SEQS || nheads > MAX_HEADS || static_cast<long long>(table_cols) * page_size > MAX_CELLS)
        return 0;
    return qsa::paged_attn_scratch_bytes(nseq, nheads, nkv, table_cols * page_size, with_mass != 0);
}

qsa_status qsa_paged_attn(const void *q, qsa_dtype q_dtype, int64_t q_seq_stride, int64_t q_head_stride, int nseq,
                          int nheads, const qsa_kv_pages *kv, const int32_t *page_table, int table_cols,
                          int64_t table_stride, const int32_t *lens, int window, int sinks, float scale, void *out,
                          float *lse, const float *mass, float *mass_out, int64_t mass_stride, void *scratch,
                          size_t scratch_bytes, cudaStream_t stream) {
    qsa_status s = check_pages(kv);
    if (s != QSA_OK) return s;
    if (nseq < 0 || nheads < 1 || nheads % kv->nkv != 0 || sinks < 0 || !good_scale(scale)) return QSA_ERR_INVALID;
    if (kv->dtype == QSA_I8 ? (q_dtype != QSA_F32 && q_dtype != QSA_F16 && q_dtype != QSA_BF16)
                            : static_cast<int>(q_dtype) != kv->dtype)
        return QSA_ERR_INVALID;
    s = check_table(table_cols, table_stride, kv->page_size);
    if (s != QSA_OK) return s;
    if (!good_stride(q_seq_stride, q_dtype) || !good_stride(q_head_stride, q_dtype)) return QSA_ERR_INVALID;
    if ((mass == nullptr) != (mass_out == nullptr)) return QSA_ERR_INVALID;
    const long long capacity = static_cast<long long>(table_cols) * kv->page_size;
    if (mass != nullptr && mass_stride < capacity) return QSA_ERR_INVALID;
    if (nseq == 0) return QSA_OK;
    if (nseq > MAX_SEQS || nheads > MAX_HEADS || static_cast<long long>(nseq) * nheads > MAX_CELLS ||
        static_cast<long long>(nseq) * nheads * ((capacity + 63) / 64) > MAX_TILES)
        return QSA_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lens, 4)) return QSA_ERR_INVALID;
    if (lse != nullptr && !aligned(lse, 4)) return QSA_ERR_INVALID;
    if (table_cols > 0 && !aligned(page_table, 4)) return QSA_ERR_INVALID;
    if (mass != nullptr && (!aligned(mass, 4) || !aligned(mass_out, 4))) return QSA_ERR_INVALID;
    const size_t need = qsa_paged_attn_scratch_bytes(nseq, nheads, kv->nkv, table_cols, kv->page_size, mass != nullptr);
    if (need == 0 || !aligned(scratch, 16) || scratch_bytes < need) return QSA_ERR_INVALID;
    const qsa::PagedAttnArgs a{q,     q_dtype, q_seq_stride, q_head_stride, nseq, nheads, *kv,  page_table,
                               table_cols, table_stride, lens, window, sinks, scale, out, lse, mass, mass_out,
                               mass_stride, scratch};
    return from_cuda(qsa::launch_paged_attn(a, stream));
}

size_t qsa_window_attn_scratch_bytes(int nseq, int total_q, int max_q, int nheads, int nkv) {
    if (nseq < 1 || total_q < 1 || max_q < 1 || nheads < 1 || nkv < 1 || nheads % nkv != 0) return 0;
    return qsa::window_attn_scratch_bytes(nseq, total_q, nheads, nkv);   // the longest sequence does not matter
}

qsa_status qsa_window_attn(const void *q, const void *k, const void *v, qsa_dtype dtype, const int64_t *strides,
                           const int32_t *cu_q, const int32_t *cu_k, int nseq, int total_q, int total_k, int max_q,
                           int nheads, int nkv, int window, int sinks, float scale, void *out, float *lse,
                           void *scratch, size_t scratch_bytes, cudaStream_t stream) {
    if (dtype != QSA_BF16 && dtype != QSA_F16) return QSA_ERR_INVALID;
    if (nseq < 0 || total_q < 0 || total_k < 0 || max_q < 0 || nheads < 1 || nkv < 1 || nheads % nkv != 0 ||
        sinks < 0 || !good_scale(scale) || strides == nullptr)
        return QSA_ERR_INVALID;
    for (int i = 0; i < 6; ++i)
        if (!good_stride(strides[i], dtype)) return QSA_ERR_INVALID;
    if (nseq == 0 || total_q == 0 || max_q == 0) return QSA_OK;
    if (nseq > MAX_SEQS || nheads > MAX_HEADS || nheads / nkv > 128 ||
        static_cast<long long>(total_q) * nheads > 0x7FFFFFFFLL)
        return QSA_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(cu_q, 4) || !aligned(cu_k, 4)) return QSA_ERR_INVALID;
    if (total_k > 0 && (!aligned(k, 16) || !aligned(v, 16))) return QSA_ERR_INVALID;
    if (lse != nullptr && !aligned(lse, 4)) return QSA_ERR_INVALID;
    const size_t need = qsa_window_attn_scratch_bytes(nseq, total_q, max_q, nheads, nkv);
    if (need > 0 && (!aligned(scratch, 16) || scratch_bytes < need)) return QSA_ERR_INVALID;
    const qsa::WindowAttnArgs a{q,    k,       v,       dtype, strides[0], strides[1], strides[2], strides[3],
                                strides[4], strides[5], cu_q, cu_k, nseq, total_q, total_k, max_q,
                                nheads, nkv, window, sinks, scale, out, lse, scratch};
    return from_cuda(qsa::launch_window_attn(a, stream));
}

qsa_status qsa_cache_evict(const qsa_kv_pages *kv, int nseq, const int32_t *page_table, int table_cols,
                           int64_t table_stride, const int32_t *lens, const float *mass, int64_t mass_stride,
                           const int32_t *new_table, int new_cols, int64_t new_table_stride, int budget, int sinks,
                           int recent, int32_t *kept, int32_t *new_lens, float *new_mass, int64_t new_mass_stride,
                           int new_mass_cols, cudaStream_t stream) {
    qsa_status s = check_pages(kv);
    if (s != QSA_OK) return s;
    s = check_table(table_cols, table_stride, kv->page_size);
    if (s != QSA_OK) return s;
    s = check_table(new_cols, new_table_stride, kv->page_size);
    if (s != QSA_OK) return s;
    if (nseq < 0 || budget < 1 || sinks < 0 || recent < 0) return QSA_ERR_INVALID;
    if (static_cast<long long>(sinks) + recent > budget) return QSA_ERR_INVALID;
    if (budget > static_cast<long long>(new_cols) * kv->page_size || budget > new_mass_cols) return QSA_ERR_INVALID;
    if (new_mass_stride < new_mass_cols) return QSA_ERR_INVALID;
    if (mass_stride < static_cast<long long>(table_cols) * kv->page_size) return QSA_ERR_INVALID;
    if (nseq == 0) return QSA_OK;
    if (nseq > MAX_SEQS || new_mass_cols > MAX_CELLS) return QSA_ERR_UNSUPPORTED;
    if (!aligned(lens, 4) || !aligned(new_table, 4) || !aligned(kept, 4) || !aligned(new_lens, 4) ||
        !aligned(new_mass, 4))
        return QSA_ERR_INVALID;
    if (table_cols > 0 && (!aligned(page_table, 4) || !aligned(mass, 4))) return QSA_ERR_INVALID;
    if (new_lens == lens || new_mass == mass) return QSA_ERR_INVALID;   // read while they are written
    const qsa::CacheEvictArgs a{*kv,  nseq,   page_table, table_cols, table_stride, lens, mass, mass_stride,
                                new_table, new_cols, new_table_stride, budget, sinks, recent, kept, new_lens,
                                new_mass, new_mass_stride, new_mass_cols};
    return from_cuda(qsa::launch_cache_evict(a, stream));
}

}  // extern "C"
