// C ABI of the bounded-cache operators: argument checks, then launches on the
// caller's stream. Declarations and the contract: include/qsa.h.
#include <cmath>
#include <cstdint>
#include <utility>

#include "cache_internal.cuh"

namespace {

constexpr long long MAX_SEQS = 65535, MAX_HEADS = 65535, MAX_CELLS = 1LL << 30, MAX_TILES = 1LL << 38;
constexpr long long MAX_TOKENS = (1LL << 31) - 64;   // what a CTA adds to a token's number stays within 32 bits

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

// A rotation; positions may be missing where `own_positions`.
qsa_status check_rotation(const qsa_rotation *r, bool own_positions) {
    if (r->npairs < 8 || r->npairs > 64 || r->npairs % 8 != 0 || r->naxes < 1 || !aligned(r->freqs, 4)) return QSA_ERR_INVALID;
    if (r->axis != nullptr && !aligned(r->axis, 4)) return QSA_ERR_INVALID;
    if (r->positions == nullptr) {
        if (!own_positions || r->naxes != 1) return QSA_ERR_INVALID;
    } else if (!aligned(r->positions, 4) || r->position_stride < 0) {
        return QSA_ERR_INVALID;
    }
    return r->naxes > MAX_HEADS ? QSA_ERR_UNSUPPORTED : QSA_OK;
}

// A dimension of memory that is written: `count` pieces, `stride` elements apart.
struct Dim {
    int64_t stride, count;
};
// The dimensions of more than one piece, the widest stride last; returns how many there are.
int by_stride(Dim *dims, int n) {
    int kept = 0;
    for (int i = 0; i < n; ++i)
        if (dims[i].count > 1) dims[kept++] = dims[i];
    for (int i = 1; i < kept; ++i)
        for (int j = i; j > 0 && dims[j].stride < dims[j - 1].stride; --j) std::swap(dims[j], dims[j - 1]);
    return kept;
}
// Whether no two pieces of `size` elements share any: each dimension steps over all that the narrower ones span.
bool apart(Dim *dims, int n, int64_t size) {
    n = by_stride(dims, n);
    int64_t span = size;
    for (int i = 0; i < n; ++i) {
        if (dims[i].stride < span) return false;
        // Past 2^62 elements there is no memory: nothing wider can be stepped over either way.
        span = dims[i].stride > (int64_t{1} << 62) / dims[i].count ? int64_t{1} << 62 : dims[i].stride * (dims[i].count - 1) + span;
    }
    return true;
}

// Strides per token and head of [ntok][nheads][128] elements, which rows written must not share.
bool good_rows(const int64_t *strides, int dtype, int ntok, int nheads, bool written) {
    if (!good_stride(strides[0], dtype) || !good_stride(strides[1], dtype)) return false;
    Dim dims[2] = {{strides[0], ntok}, {strides[1], nheads}};
    return !written || nheads > MAX_HEADS || apart(dims, 2, QSA_D);   // so many are unsupported, whatever their strides
}

// Whether a piece at a, moved by `by`, meets one of dims' (which are apart, and ordered): of a dimension's steps only the two
// beside `by` can bring it within what the narrower ones span.
bool meets(int64_t by, const Dim *dims, int n, int64_t size) {
    if (n == 0) return by > -size && by < size;
    const int64_t stride = dims[n - 1].stride, count = dims[n - 1].count;
    const int64_t below = by / stride - (by % stride < 0 ? 1 : 0);
    for (int64_t step = below; step <= below + 1; ++step)
        if (step > -count && step < count && meets(by - step * stride, dims, n - 1, size)) return true;
    return false;
}
// Two sets of pieces of the same dimensions, at a and b: whether they share memory. Sizes and strides in elements of `bytes`.
bool overlap(const void *a, const void *b, Dim *dims, int n, int64_t size, int bytes) {
    n = by_stride(dims, n);
    for (int i = 0; i < n; ++i) {
        if (dims[i].stride > (int64_t{1} << 60) / bytes) return false;   // no memory is so wide
        dims[i].stride *= bytes;
    }
    return meets(static_cast<int64_t>(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a)), dims, n, size * bytes);
}

// Whether rows would be read after others are written there: out over in, but for the very same rows. Where the strides
// differ, the same address alone is looked at.
bool entangled(const void *in, const int64_t *in_strides, const void *out, const int64_t *out_strides, int dtype, int ntok, int nheads) {
    if ((ntok > 1 && in_strides[0] != out_strides[0]) || (nheads > 1 && in_strides[1] != out_strides[1])) return in == out;
    Dim dims[2] = {{out_strides[0], ntok}, {out_strides[1], nheads}};
    return in != out && overlap(in, out, dims, 2, QSA_D, element_size(dtype));
}

// The limits of the shared prefix's attention; the sizes are not negative, nkv divides nheads.
bool prefix_fits(long long nseq, long long ngroups, long long nheads, int nkv, long long prefix_cols, long long table_cols, int page_size) {
    const long long prefix = prefix_cols * page_size, capacity = table_cols * page_size;
    return nseq <= MAX_SEQS && ngroups <= MAX_SEQS && nheads <= MAX_HEADS && nkv <= MAX_HEADS && nheads / nkv <= 128 &&
           prefix <= MAX_CELLS && capacity <= MAX_CELLS && nseq * nheads <= MAX_CELLS && nseq * nheads * ((capacity + 63) / 64) <= MAX_TILES &&
           (nseq + ngroups) * nheads * ((prefix + 127) / 128) <= MAX_TILES;
}

bool row_type(int dtype) { return dtype == QSA_F32 || dtype == QSA_F16 || dtype == QSA_BF16; }

}  // namespace

extern "C" {

qsa_status qsa_rotate(const void *x, qsa_dtype dtype, const int64_t *strides, int ntok, int nheads,
                      const qsa_rotation *rotation, void *out, cudaStream_t stream) {
    if (!row_type(dtype) || ntok < 0 || nheads < 1 || strides == nullptr || rotation == nullptr) return QSA_ERR_INVALID;
    const qsa_status s = check_rotation(rotation, ntok == 0);
    if (s != QSA_OK) return s;
    if (!good_rows(strides, dtype, ntok, nheads, false) || !good_rows(strides + 2, dtype, ntok, nheads, true)) return QSA_ERR_INVALID;
    if (ntok == 0) return QSA_OK;
    if (nheads > MAX_HEADS || ntok > MAX_TOKENS) return QSA_ERR_UNSUPPORTED;
    if (!aligned(x, 16) || !aligned(out, 16) || entangled(x, strides, out, strides + 2, dtype, ntok, nheads)) return QSA_ERR_INVALID;
    return from_cuda(qsa::launch_rotate(x, dtype, strides, ntok, nheads, *rotation, out, stream));
}

qsa_status qsa_cache_append(const void *k, const void *v, const void *q, qsa_dtype dtype, const int64_t *strides,
                            int ntok, int nheads, const qsa_kv_pages *kv, const int32_t *page_table, int table_cols,
                            int64_t table_stride, const int32_t *lens, const int32_t *cu, int nseq,
                            const qsa_rotation *rotation, void *q_out, void *k_out, cudaStream_t stream) {
    qsa_status s = check_pages(kv);
    if (s != QSA_OK) return s;
    s = check_table(table_cols, table_stride, kv->page_size);
    if (s != QSA_OK) return s;
    if (!row_type(dtype) || (kv->dtype != QSA_I8 && dtype != QSA_F32 && static_cast<int>(dtype) != kv->dtype)) return QSA_ERR_INVALID;
    if (ntok < 0 || nseq < 0 || nheads < 0 || strides == nullptr || (cu == nullptr && ntok != nseq)) return QSA_ERR_INVALID;
    if (rotation == nullptr ? nheads != 0 || k_out != nullptr : rotation->inverse != 0) return QSA_ERR_INVALID;
    if (rotation != nullptr && (s = check_rotation(rotation, true)) != QSA_OK) return s;
    const int nkv = kv->nkv;
    if (!good_rows(strides, dtype, ntok, nkv, false) || !good_rows(strides + 2, dtype, ntok, nkv, false)) return QSA_ERR_INVALID;
    if (nheads > 0 && (!good_rows(strides + 4, dtype, ntok, nheads, false) || !good_rows(strides + 6, dtype, ntok, nheads, true)))
        return QSA_ERR_INVALID;
    if (k_out != nullptr && !good_rows(strides + 8, dtype, ntok, nkv, true)) return QSA_ERR_INVALID;
    // Cells are written: none may share its memory with another.
    Dim cells[3] = {{kv->page_stride, kv->npages}, {kv->cell_stride, kv->page_size}, {kv->head_stride, nkv}};
    if (!apart(cells, 3, QSA_D)) return QSA_ERR_INVALID;
    if (kv->dtype == QSA_I8) {
        Dim scales[3] = {{kv->scale_page_stride, kv->npages}, {kv->scale_cell_stride, kv->page_size}, {kv->scale_head_stride, nkv}};
        if (!apart(scales, 3, 1)) return QSA_ERR_INVALID;
    }
    if (ntok == 0 || nseq == 0) return QSA_OK;
    if (nseq > MAX_SEQS || nheads > MAX_HEADS || nkv > MAX_HEADS || ntok > MAX_TOKENS) return QSA_ERR_UNSUPPORTED;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(lens, 4)) return QSA_ERR_INVALID;
    if (nheads > 0 && (!aligned(q, 16) || !aligned(q_out, 16) || entangled(q, strides + 4, q_out, strides + 6, dtype, ntok, nheads)))
        return QSA_ERR_INVALID;
    if (k_out != nullptr && (!aligned(k_out, 16) || entangled(k, strides, k_out, strides + 8, dtype, ntok, nkv))) return QSA_ERR_INVALID;
    // One pool for both holds what it is given where keys and values are the same rows.
    const bool one_pool = kv->k == kv->v && kv->k_scale_f16 == kv->v_scale_f16 && k == v && rotation == nullptr &&
                          (ntok == 1 || strides[0] == strides[2]) && (nkv == 1 || strides[1] == strides[3]);
    if (kv->npages > 0 && !one_pool) {
        Dim both[3] = {{kv->page_stride, kv->npages}, {kv->cell_stride, kv->page_size}, {kv->head_stride, nkv}};
        if (overlap(kv->k, kv->v, both, 3, QSA_D, element_size(kv->dtype))) return QSA_ERR_INVALID;
        Dim scales[3] = {{kv->scale_page_stride, kv->npages}, {kv->scale_cell_stride, kv->page_size}, {kv->scale_head_stride, nkv}};
        if (kv->dtype == QSA_I8 && overlap(kv->k_scale_f16, kv->v_scale_f16, scales, 3, 1, 2)) return QSA_ERR_INVALID;
    }
    if (cu != nullptr && !aligned(cu, 4)) return QSA_ERR_INVALID;
    if (table_cols > 0 && !aligned(page_table, 4)) return QSA_ERR_INVALID;
    const qsa::CacheAppendArgs a{k, v, q, dtype, strides, ntok, nheads, *kv, page_table, table_cols, table_stride,
                                 lens, cu, nseq, rotation, q_out, k_out};
    return from_cuda(qsa::launch_cache_append(a, stream));
}

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

size_t qsa_prefix_attn_scratch_bytes(int nseq, int ngroups, int nheads, int nkv, int prefix_cols, int table_cols,
                                     int page_size) {
    if (nseq < 1 || ngroups < 0 || nheads < 1 || nkv < 1 || nheads % nkv != 0 || prefix_cols < 0 || table_cols < 0 ||
        page_size < 1 || !prefix_fits(nseq, ngroups, nheads, nkv, prefix_cols, table_cols, page_size))
        return 0;
    return qsa::prefix_attn_scratch_bytes({nseq, ngroups, nheads, nkv, prefix_cols * page_size, table_cols * page_size});
}

qsa_status qsa_prefix_attn(const void *q, qsa_dtype q_dtype, int64_t q_seq_stride, int64_t q_head_stride, int nseq,
                           int nheads, const qsa_kv_pages *kv, const int32_t *prefix_table, int prefix_cols,
                           int64_t prefix_stride, const int32_t *prefix_lens, const int32_t *cu_seqs, int ngroups,
                           const int32_t *page_table, int table_cols, int64_t table_stride, const int32_t *lens,
                           float scale, void *out, float *lse, void *scratch, size_t scratch_bytes,
                           cudaStream_t stream) {
    qsa_status s = check_pages(kv);
    if (s != QSA_OK) return s;
    if (nseq < 0 || ngroups < 0 || nheads < 1 || nheads % kv->nkv != 0 || !good_scale(scale)) return QSA_ERR_INVALID;
    if (kv->dtype == QSA_I8 ? !row_type(q_dtype) : static_cast<int>(q_dtype) != kv->dtype) return QSA_ERR_INVALID;
    s = check_table(table_cols, table_stride, kv->page_size);
    if (s != QSA_OK) return s;
    s = check_table(prefix_cols, prefix_stride, kv->page_size);
    if (s != QSA_OK) return s;
    if (!good_stride(q_seq_stride, q_dtype) || !good_stride(q_head_stride, q_dtype)) return QSA_ERR_INVALID;
    if (nseq == 0) return QSA_OK;
    if (!prefix_fits(nseq, ngroups, nheads, kv->nkv, prefix_cols, table_cols, kv->page_size)) return QSA_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lens, 4) || !aligned(cu_seqs, 4)) return QSA_ERR_INVALID;
    if (ngroups > 0 && (!aligned(prefix_lens, 4) || (prefix_cols > 0 && !aligned(prefix_table, 4)))) return QSA_ERR_INVALID;
    if (lse != nullptr && !aligned(lse, 4)) return QSA_ERR_INVALID;
    if (table_cols > 0 && !aligned(page_table, 4)) return QSA_ERR_INVALID;
    const size_t need = qsa_prefix_attn_scratch_bytes(nseq, ngroups, nheads, kv->nkv, prefix_cols, table_cols, kv->page_size);
    if (need == 0 || !aligned(scratch, 16) || scratch_bytes < need) return QSA_ERR_INVALID;
    const qsa::PrefixAttnArgs a{q, q_dtype, q_seq_stride, q_head_stride, nseq, nheads, *kv, prefix_table, prefix_cols, prefix_stride,
                                prefix_lens, cu_seqs, ngroups, page_table, table_cols, table_stride, lens, scale, out, lse, scratch};
    return from_cuda(qsa::launch_prefix_attn(a, stream));
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
