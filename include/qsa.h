/*
 * qsa.h -- exact QSA block selection on one GB300 (sm_103a): block scoring
 * and an exact per-query top-k, as a C ABI over caller-owned device memory.
 *
 * What is computed (the "QSA select" step of query-aware sparse attention):
 * each query is 4 query heads of D = 128 fp32 values that share one KV head.
 * The KV cache is cut into 4-cell blocks, each summarised by one key of 128
 * values. A query's score for a block is the sum over its 4 heads of the
 * head's dot product with the block key; only the first `active_blocks`
 * blocks exist for this batch, whatever the cache capacity. The top-k then
 * keeps, per query, the k highest-scoring block ids exactly.
 * Passages: "#3108 optimize exact QSA block scoring and top-k selection on
 * gfx12", Summary items 1, 2 and 4 (4-head block score, radix top-k,
 * bitwise parity of scores and ids); "#337 gfx12 QSA select", What items 1-2
 * (select over the active blocks, not the capacity `max_context/4 + 2`;
 * split-bf16 tensor-core scorer with the hi*hi products in their own
 * accumulator; FP64 gate at 1e-6 of the score scale).
 *
 * Conventions for every call below:
 *  - All pointers are DEVICE pointers owned by the caller; the library keeps
 *    no state between calls beyond a per-device error word (see
 *    qsa_get_device_error), the fixed device arrays of the two
 *    allocation-free calls (qsa_block_select_static, qsa_block_select_small)
 *    and the process-wide wait settings of qsa_debug_inject; it allocates
 *    nothing, never synchronises (except qsa_get_device_error), and enqueues
 *    its kernels on `stream` (0 = the legacy default stream).
 *  - Every pointer that is dereferenced must be 16-byte aligned.
 *  - Arguments are checked before anything is launched; a bad argument
 *    returns QSA_ERR_INVALID and launches nothing. A launch failure returns
 *    QSA_ERR_CUDA. Errors of already-enqueued work surface as CUDA errors of
 *    the stream, as for any kernel.
 *  - Calls with no work (nq == 0, or active_blocks == 0 for the scorers)
 *    return QSA_OK without touching memory; pointers may then be NULL.
 *  - Inputs are expected to be finite. In the top-k a NaN score counts as
 *    -infinity (it ties with -inf, below every finite score); -0.0 and +0.0
 *    are equal (and therefore tie).
 */
#ifndef QSA_H
#define QSA_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    QSA_OK = 0,
    QSA_ERR_INVALID = 1,      /* bad argument; nothing was launched            */
    QSA_ERR_UNSUPPORTED = 2,  /* valid, but beyond this library's size limits  */
    QSA_ERR_CUDA = 3          /* a CUDA runtime call or launch failed          */
} qsa_status;

/* Head dimension and query heads per KV head (fixed). */
#define QSA_D 128
#define QSA_HEADS 4

/* Largest active_blocks the top-k accepts (its per-row bitmaps live in shared memory). */
#define QSA_TOPK_MAX_ACTIVE 393216

/*
 * Block scores, fp32 summary keys.
 *   scores[i][b] = sum_{h<4} sum_{d<128} q[i][h][d] * kblk[b][d],  b < active_blocks
 * q       fp32 [nq][4][128], contiguous.
 * kblk    fp32 [max_blocks][128], block-major; only rows < active_blocks are read.
 * scores  fp32 [nq][active_blocks], written; row stride = active_blocks.
 * max_blocks is the key buffer's capacity (validation only: active_blocks <=
 * max_blocks); the launch is sized from active_blocks alone.
 * Accuracy: |scores - exact| <= 1e-6 * max_b |exact[i][b]| per row for
 * finite inputs; scores are exact when every product and partial sum is an
 * integer below 2^24 in magnitude.
 * Kernels: nq >= 5 runs on the tensor cores (3-way exact bf16 split, hi*hi in
 * its own accumulator); nq <= 4 (decode) on CUDA cores with one fp32 FMA
 * chain per query and key row. Both meet the accuracy bound above.
 * ("#3108 ...", Summary item 4; "#337 ...", What items 1-2.)
 */
qsa_status qsa_block_scores(const float *q, const float *kblk, int nq, int max_blocks,
                            int active_blocks, float *scores, cudaStream_t stream);

/*
 * Block scores, int8 summary keys with one IEEE binary16 scale per block
 * (the engine's `--kv int8` cache form; key element = kblk_q8[b][d] *
 * kscale_f16[b], exact in fp32).
 * kblk_q8    int8   [max_blocks][128]
 * kscale_f16 uint16 [max_blocks] (binary16 bit patterns; 2-byte aligned suffices)
 * Other arguments, layouts and accuracy as qsa_block_scores.
 * ("#3108 ...", End-to-End `--kv int8`; "#337 ...", What: `--kv int8`.)
 */
qsa_status qsa_block_scores_q8(const float *q, const int8_t *kblk_q8, const uint16_t *kscale_f16,
                               int nq, int max_blocks, int active_blocks, float *scores,
                               cudaStream_t stream);

/*
 * Block scores on the CUDA cores (FP32 FMA, head-summed query, natural d
 * order) -- the same contract as qsa_block_scores; kept as the measured
 * alternative to the tensor-core scorer. kblk_q8/kscale_f16 may be given
 * instead of kblk (then kblk must be NULL) for the int8 key form.
 */
qsa_status qsa_block_scores_ffma(const float *q, const float *kblk, const int8_t *kblk_q8,
                                 const uint16_t *kscale_f16, int nq, int max_blocks,
                                 int active_blocks, float *scores, cudaStream_t stream);

/*
 * Exact per-query top-k of packed scores.
 * scores  fp32  [nq][active_blocks] (row stride = active_blocks).
 * ids     int32 [nq][k], written: for each row, the ids of the k highest
 *         scores in ascending id order; among equal scores the lower block
 *         id is taken first. If k > active_blocks the row holds all
 *         active_blocks ids ascending followed by -1 (active_blocks == 0
 *         gives a row of -1).
 * k >= 1 and active_blocks <= QSA_TOPK_MAX_ACTIVE (else QSA_ERR_UNSUPPORTED).
 * ("#3108 ...", Summary item 2: radix-bin top-k; "#337 ...", What item 1:
 * the active block count, not the capacity, bounds the selection.)
 */
qsa_status qsa_block_topk(const float *scores, int nq, int active_blocks, int k, int32_t *ids,
                          cudaStream_t stream);

/* Blocks per group of the group-maximum side output (below). */
#define QSA_GROUP_BLOCKS 32

/*
 * Block scores plus their group maxima, for qsa_block_topk_gmax.
 * group_max  uint32 [nq][ceil(active_blocks / 32)], written: element [i][g]
 *            is key(max of scores[i][32 g .. 32 g + 31]) over the blocks
 *            < active_blocks, where key(x) is the order-preserving radix key
 *            of the top-k (-0 counted as +0 and NaN as -inf, then the bits
 *            of a negative x inverted and the sign bit of a positive x set),
 *            so a larger score has a larger unsigned key.
 * 16-byte aligned. Other arguments, layouts and accuracy as qsa_block_scores
 * (the scores are the same bits); the maxima add 1/32 of the score bytes.
 */
qsa_status qsa_block_scores_gmax(const float *q, const float *kblk, int nq, int max_blocks,
                                 int active_blocks, float *scores, uint32_t *group_max,
                                 cudaStream_t stream);

/* The int8-key form of qsa_block_scores_gmax (arguments as qsa_block_scores_q8). */
qsa_status qsa_block_scores_q8_gmax(const float *q, const int8_t *kblk_q8, const uint16_t *kscale_f16,
                                    int nq, int max_blocks, int active_blocks, float *scores,
                                    uint32_t *group_max, cudaStream_t stream);

/*
 * Group maxima of given packed scores (the group_max of
 * qsa_block_scores_gmax, for scores that come from elsewhere).
 * scores     fp32   [nq][active_blocks]
 * group_max  uint32 [nq][ceil(active_blocks / 32)], written (16-byte aligned).
 */
qsa_status qsa_block_group_max(const float *scores, int nq, int active_blocks, uint32_t *group_max,
                               cudaStream_t stream);

/*
 * qsa_block_topk with the group maxima of the same scores (as written by
 * qsa_block_scores_gmax or qsa_block_scores_q8_gmax; 16-byte aligned). The
 * result is identical to qsa_block_topk's. The maxima fix a threshold that
 * at least k groups, hence at least k scores, reach, so a row reads only the
 * groups at or above it; rows where that does not pay (k above half the
 * group count, a threshold list past capacity) take qsa_block_topk's path.
 * group_max that does not match `scores` gives undefined ids (never an
 * out-of-bounds access).
 */
qsa_status qsa_block_topk_gmax(const float *scores, const uint32_t *group_max, int nq, int active_blocks,
                               int k, int32_t *ids, cudaStream_t stream);

/* Largest nq * ceil(active_blocks / 32) qsa_block_select_static accepts:
 * its scratch is a fixed 1 MiB device array of that many uint32. */
#define QSA_SELECT_STATIC_GROUPS_MAX 262144

/*
 * Scores and exact top-k in one call that allocates nothing: exactly
 * qsa_block_scores_gmax followed by qsa_block_topk_gmax, with the group
 * maxima kept in a file-scope device array of QSA_SELECT_STATIC_GROUPS_MAX
 * uint32 (1 MiB, part of the library image) instead of caller memory.
 * scores  fp32  [nq][active_blocks], written (as qsa_block_scores).
 * ids     int32 [nq][k], written (as qsa_block_topk).
 * nq * ceil(active_blocks / 32) > QSA_SELECT_STATIC_GROUPS_MAX returns
 * QSA_ERR_UNSUPPORTED before anything is launched (e.g. 256 queries up to
 * 32,768 active blocks, 128 up to 65,536). The scratch is one per device:
 * calls on one device must be ordered (one stream, or streams joined by
 * events); overlapping calls on unordered streams give undefined ids.
 * Other arguments, errors and accuracy as the two calls it stands for.
 */
qsa_status qsa_block_select_static(const float *q, const float *kblk, int nq, int max_blocks, int active_blocks,
                                   int k, float *scores, int32_t *ids, cudaStream_t stream);

/*
 * Scores and exact top-k for a few queries (decode: 1 <= nq <= 4) in one
 * cooperative kernel launch: the whole grid scores every active block (and
 * its 32-block group maxima, kept in a fixed device array of the library),
 * then nq of its CTAs each select one query's top k from those maxima. The
 * scores and ids equal qsa_block_scores(_q8) followed by qsa_block_topk.
 * Give kblk (fp32 keys) or kblk_q8 + kscale_f16 (int8 keys), not both; the
 * layouts are those of qsa_block_scores / qsa_block_scores_q8.
 * scores  fp32  [nq][active_blocks], written.
 * ids     int32 [nq][k], written (as qsa_block_topk).
 * nq > 4 or active_blocks > QSA_TOPK_MAX_ACTIVE returns QSA_ERR_UNSUPPORTED.
 * Nothing is allocated. The grid meets at a device-wide counter and a
 * generation word of library state, so calls on one device must be ordered
 * (one stream, or streams joined by events). When k >= active_blocks the call
 * runs the scorer and a fill.
 * Passage: "#3108 optimize exact QSA block scoring and top-k selection on
 * gfx12", Summary item 4 (a row kernel for a handful of queries) and the
 * Microbenchmark & Parity Evidence table (decode scores + top-k per layer).
 */
qsa_status qsa_block_select_small(const float *q, const float *kblk, const int8_t *kblk_q8,
                                  const uint16_t *kscale_f16, int nq, int max_blocks, int active_blocks, int k,
                                  float *scores, int32_t *ids, cudaStream_t stream);

/*
 * Attention over the selected blocks: each query's 4 heads attend the KV
 * cells of the blocks listed in its row of ids (block b holds cells
 * 4b .. 4b+3; cells at or past ncells, negative ids and ids at or past the
 * last block are skipped; a block listed twice counts twice):
 *   logit[h][c] = (sum_d q[i][h][d] * k_cells[c][d]) * k_scale[c] / sqrt(128)
 *   out[i][h][d] = sum_c softmax_c(logit[h][.]) * v_cells[c][d] * v_scale[c]
 * and out = 0 for a query with no attended cell. Accumulation is fp32 in a
 * fixed order (the result does not depend on scheduling). With at most half
 * as many queries as the device has SMs the products are fp32 on CUDA cores;
 * with more, they run on the tensor cores (mma.sync): q (per head) and the softmax
 * weights times v_scale, each scaled by a power of two chosen from the data,
 * enter as binary16 high parts plus remainders (about 22 significant bits),
 * the int8 cells exactly, with fp32 accumulation.
 * q        fp32 [nq][4][128], 16-byte aligned.
 * k_cells, v_cells  int8 [ncells][128], 16-byte aligned; k_scale_f16,
 *          v_scale_f16  IEEE binary16 bit patterns [ncells], 2-byte aligned
 *          (may be NULL when ncells == 0).
 * ids      int32 [nq][k] (e.g. qsa_block_topk's output), 16-byte aligned.
 * out      fp32 [nq][4][128], written, 16-byte aligned.
 * nq < 0, k < 1 or ncells < 0 returns QSA_ERR_INVALID; nq == 0 is a no-op;
 * ncells > INT_MAX - 4 returns QSA_ERR_UNSUPPORTED. Allocates nothing and
 * keeps no state.
 * Passages: "#3224 [Engine] perf(hip): tune RDNA4 QSA prompt WMMA path
 * (STRATA_HIP_WMMA stays opt-in)", Summary and Evidence section 2 (int8-KV
 * QSA attention with binary16 k/v scales, gated against FP64); "#3102
 * perf(hip): enable wave32 QSA decode attention and MMVQ row reuse on
 * gfx12", item D5 (decode attention in chunks merged in sequential order).
 * The softmax temperature 1/sqrt(128), the per-cell scales and the 4 heads
 * sharing the cells are readings: the pages print no formula.
 */
qsa_status qsa_sparse_attn(const float *q, const int8_t *k_cells, const uint16_t *k_scale_f16,
                           const int8_t *v_cells, const uint16_t *v_scale_f16, int ncells, const int32_t *ids,
                           int nq, int k, float *out, cudaStream_t stream);

/*
 * Block summary keys from int8 KV cells, for blocks block_begin ..
 * block_end-1 (after an append: block_begin = old ncells / 4, block_end =
 * ceil(new ncells / 4)):
 *   kblk[b][d]    = (sum over the present cells c = 4b .. 4b+3 (< ncells) of
 *                    k_cells[c][d] * k_scale[c]) / (number of present cells)
 *   kblk_scale[b] = binary16(max_d |kblk[b][d]| / 127), round to nearest even
 *   kblk_q8[b][d] = rint(kblk[b][d] / kblk_scale[b])  (0 when the scale is 0)
 * computed in fp32 in that order (IEEE single operations), so the int8 form
 * is reproducible bit for bit; a block with no present cell gets zeros.
 * k_cells  int8 [ncells][128], 16-byte aligned; k_scale_f16 binary16 [ncells],
 *          2-byte aligned (both may be NULL when ncells == 0).
 * kblk     fp32 [>= block_end][128] (row b written), 16-byte aligned, or NULL.
 * kblk_q8  int8 [>= block_end][128] and kblk_scale_f16 binary16 [>= block_end]
 *          (the qsa_block_scores_q8 key layout), both or neither.
 * ncells < 0, block_begin < 0, block_end < block_begin, or no output returns
 * QSA_ERR_INVALID; an empty range is a no-op; 4 * block_end + 4 > INT_MAX
 * returns QSA_ERR_UNSUPPORTED. Allocates nothing.
 * Passage: "#3108 optimize exact QSA block scoring and top-k selection on
 * gfx12", the Microbenchmark & Parity Evidence table (the decode layer's
 * "append" step). The pages do not define the summary function: the mean of
 * the present cells and the int8 form are readings.
 */
qsa_status qsa_block_summary(const int8_t *k_cells, const uint16_t *k_scale_f16, int ncells, int block_begin,
                             int block_end, float *kblk, int8_t *kblk_q8, uint16_t *kblk_scale_f16,
                             cudaStream_t stream);

/*
 * qsa_block_select: the ids of qsa_block_topk(qsa_block_scores(...)) --
 * exactly the same ids -- without writing the scores in the common case
 * (fp32 keys; q, kblk, ids as qsa_block_scores / qsa_block_topk).
 * Method: per query row, a threshold from a strided sample of 1,024 blocks
 * (CUDA cores), chosen so that about 1.8 k scores reach it; the tensor-core
 * scorer then appends every score at or above its row's threshold, with its
 * block id, to the row's list (at most QSA_SELECT_LIST_CAP entries) instead
 * of storing the scores; a row whose list holds at least k entries (and did
 * not overflow) holds its whole top-k and is selected from the list exactly.
 * The other rows' query groups (128 rows each) are scored into `scores` and
 * their rows selected by qsa_block_topk's kernel. When nq <= 4, active_blocks
 * <= QSA_SELECT_LIST_MIN_ACTIVE or k > QSA_SELECT_LIST_K_MAX, it runs the two
 * plain calls (scores written). k >= active_blocks: ids as qsa_block_topk.
 * scores: [nq][active_blocks] fp32, caller-owned; its contents afterwards are
 * unspecified (written only where the fallback ran).
 * scratch: device memory of at least qsa_block_select_scratch_bytes(nq)
 * bytes, 16-byte aligned, caller-owned (thresholds, list counts, failure
 * flags, lists; no contents need survive between calls). Five launches on
 * `stream`; allocates nothing.
 * Errors: as qsa_block_scores and qsa_block_topk, plus QSA_ERR_INVALID for a
 * missing, misaligned or too small scratch.
 * Passages: "#3108 optimize exact QSA block scoring and top-k selection on
 * gfx12", Microbenchmark & Parity Evidence section 2 (selection inside the
 * decode layer, where the scores are only an intermediate); "#337 gfx12 QSA
 * select", What item 1 (scores, then top-k over the active blocks).
 */
#define QSA_SELECT_LIST_CAP 4096
#define QSA_SELECT_LIST_MIN_ACTIVE 8192
#define QSA_SELECT_LIST_K_MAX 1024
size_t qsa_block_select_scratch_bytes(int nq);
qsa_status qsa_block_select(const float *q, const float *kblk, int nq, int max_blocks, int active_blocks, int k,
                            float *scores, int32_t *ids, void *scratch, size_t scratch_bytes, cudaStream_t stream);

/*
 * Reads and clears the current device's error word: nonzero when a kernel
 * of this library gave up a bounded wait (its outputs are then invalid).
 * Bit 0x100: a wait of the tensor-core scorer's pipeline ran out (the CTA
 * then abandons its remaining waits at once, lets its own copies and MMAs
 * in flight finish, and exits); bit 0x2: the fused decode select's grid
 * barrier ran out; bit 0x10000: a wait of the prompt attention's pipeline ran
 * out; bit 0x20000: one of the shared prefix's attention. Synchronises `stream`. *code receives the word.
 */
qsa_status qsa_get_device_error(uint32_t *code, cudaStream_t stream);

/*
 * Diagnostics for the bounded waits (not for production use; the pages have
 * no counterpart). For the kernels launched after the call: every spin-wait
 * gives up after wait_limit_ns (default 2,000,000,000; in the prompt attention
 * 8 us more for every 128 keys of the call, as items take that long, in the shared
 * prefix's for every 128 cells of the prefix table's width), and
 * `faults` plants a wait that cannot complete so that the time-out path runs:
 *   bit 0: the tensor-core scorer's CTA 0 never loads its first key piece
 *          (qsa_block_scores, _q8, _gmax and _select_static with nq > 4);
 *   bit 1: the fused decode select's grid barrier waits for one arrival
 *          more than its grid has (qsa_block_select_small);
 *   bit 3: the prompt attention's CTA 0 never copies its first key tile
 *          (qsa_window_attn, where the strides suit a tensor map);
 *   bit 5: the shared prefix's attention's CTA 0 never hands over its first
 *          key tile (qsa_prefix_attn).
 * The outputs of such calls are invalid and qsa_get_device_error reports
 * them; the device stays usable. Call qsa_debug_inject(0, 2000000000) to
 * restore normal operation. Process-wide; not thread-safe against
 * concurrent launches. faults with other bits, or wait_limit_ns == 0 or
 * above 60 s, returns QSA_ERR_INVALID.
 */
qsa_status qsa_debug_inject(uint32_t faults, uint64_t wait_limit_ns);

/* ---- A cache kept within a budget: prompt attention, paged decode attention, eviction ---- */

/* Element types of the calls below. */
typedef enum {
    QSA_F32 = 0,
    QSA_F16 = 1,
    QSA_BF16 = 2,
    QSA_I8 = 3
} qsa_dtype;

/*
 * A pool of key and value pages. Cell `slot` of page `p` holds, for each of
 * the nkv KV heads, 128 key and 128 value elements at
 *   k[p * page_stride + slot * cell_stride + head * head_stride + d]
 * (v likewise; the strides are in elements and shared by k and v, so cells
 * outside heads, heads outside cells, and keys and values side by side in one
 * allocation are all pools). dtype: QSA_BF16, QSA_F16, or QSA_I8 with one
 * binary16 scale per cell and KV head (element = code * scale) at
 *   k_scale_f16[p * scale_page_stride + slot * scale_cell_stride + head * scale_head_stride]
 * (v_scale_f16 likewise; both NULL for the 16-bit types).
 * k and v are 16-byte aligned and the strides are multiples of 16 bytes and
 * not negative; scales are 2-byte aligned. npages >= 0, page_size >= 1 (any,
 * not only powers of two), nkv >= 1.
 */
typedef struct {
    void *k, *v;
    uint16_t *k_scale_f16, *v_scale_f16;
    int32_t dtype, npages, page_size, nkv;
    int64_t page_stride, cell_stride, head_stride;
    int64_t scale_page_stride, scale_cell_stride, scale_head_stride;
} qsa_kv_pages;

/*
 * Attention of one new token per sequence over its paged cache.
 * Sequence s has n = lens[s] cells (its newest cell, n - 1, is the query's
 * own token); cell j is slot j % page_size of page page_table[s][j / page_size].
 * Head h attends KV head h / (nheads / nkv). Visible cells: j < n and
 * (window < 0 or j >= n - window or j < sinks).
 *   logit[h][j] = scale * sum_d q[s][h][d] * key[j][d]
 *   lse[s][h]   = log sum_j exp(logit[h][j])
 *   out[s][h]   = sum_j exp(logit[h][j] - lse[s][h]) * value[j]
 * With no visible cell out = 0 and lse = -infinity. Cells that are not
 * visible are never used, whatever they hold; an infinity or NaN in a visible
 * value (or its scale) makes the results that use it infinite or NaN. lens is clamped to
 * [0, table_cols * page_size]; a visible cell whose page id is outside
 * [0, npages) is skipped (as if it were not visible).
 * mass, mass_out (both or neither NULL; may be equal):
 *   mass_out[s][j] = mass[s][j] + sum over all heads of exp(logit[h][j] - lse[s][h])
 * for j < n (the sum is 0 for cells that are not visible); columns >= n are
 * not written. Each element is summed in a fixed order.
 * q         [nseq][nheads][128] of q_dtype, element strides q_seq_stride and
 *           q_head_stride (multiples of 16 bytes, not negative). q_dtype is the
 *           pages' dtype for 16-bit pages; QSA_F32, QSA_F16 or QSA_BF16 for int8.
 * page_table int32, row stride table_stride >= table_cols. lens int32 [nseq].
 * out       [nseq][nheads][128] of q_dtype, contiguous, not over an input. lse fp32
 *           [nseq][nheads] or NULL. mass, mass_out fp32 with row stride
 *           mass_stride >= table_cols * page_size.
 * scale     positive, and finite in fp32 times log2(e) (up to 2.3e38).
 * scratch   at least qsa_paged_attn_scratch_bytes(...) bytes, 16-byte aligned;
 *           no contents need survive. Some is needed for a table of no columns
 *           too (it is 0 for nseq = 0 and for arguments that are refused).
 * Sums and softmax statistics are fp32. q, out and the page pool are 16-byte
 * aligned, the others 4-byte.
 * nseq, nheads or nkv out of range, nheads % nkv != 0, a bad type, scale,
 * pointer or stride returns QSA_ERR_INVALID; nseq or nheads above 65,535,
 * nseq * nheads or table_cols * page_size above 2^30, or nseq * nheads *
 * ceil(table_cols * page_size / 64) above 2^38 returns QSA_ERR_UNSUPPORTED.
 */
size_t qsa_paged_attn_scratch_bytes(int nseq, int nheads, int nkv, int table_cols, int page_size, int with_mass);
qsa_status qsa_paged_attn(const void *q, qsa_dtype q_dtype, int64_t q_seq_stride, int64_t q_head_stride, int nseq,
                          int nheads, const qsa_kv_pages *kv, const int32_t *page_table, int table_cols,
                          int64_t table_stride, const int32_t *lens, int window, int sinks, float scale, void *out,
                          float *lse, const float *mass, float *mass_out, int64_t mass_stride, void *scratch,
                          size_t scratch_bytes, cudaStream_t stream);

/*
 * Attention of ragged sequences of new tokens over their keys: causal,
 * within a sliding window, with the first `sinks` tokens always visible.
 * Sequence s has queries cu_q[s] .. cu_q[s+1]-1 and keys cu_k[s] ..
 * cu_k[s+1]-1; its nq queries are the last of its nk tokens: query i stands
 * at pos = nk - nq + i. Visible keys: 0 <= j <= pos, j < nk and
 * (window < 0 or j > pos - window or j < sinks). logit, lse and out as
 * qsa_paged_attn; a query with no visible key (nq > nk, or window 0 without
 * sinks) gets out = 0 and lse = -infinity.
 * q         [total_q][nheads][128], k, v [total_k][nkv][128], all of dtype
 *           (QSA_F16 or QSA_BF16), 16-byte aligned, element strides per token
 *           and head (multiples of 16 bytes, not negative).
 * cu_q, cu_k int32 [nseq + 1], ascending from 0 (device memory; values are
 *           clamped to [0, total_q] and [0, total_k]).
 * max_q     at least the longest sequence's query count (queries past it may
 *           not be computed). Rows of no sequence are not written.
 * out       [total_q][nheads][128] of dtype, contiguous, 16-byte aligned; lse
 *           fp32 [total_q][nheads] or NULL. They do not overlap the inputs.
 * scratch   at least qsa_window_attn_scratch_bytes(...) bytes, 16-byte aligned
 *           (0 without sequences or queries); no contents need survive.
 * Softmax statistics and sums are fp32; the weights are rounded once to dtype
 * for the product with the values. An infinity in a visible value makes its
 * column that infinity, NaN (or infinities of both signs) NaN. The values of
 * keys that are not visible never reach a result, whatever they hold; but where
 * an infinity or NaN lies among the values of a row's key tiles (128 keys, also
 * past a sequence's end), that row is gone through again by one warp, which is
 * slow (about 0.25 us per key and row): keep memory that is not a token's finite.
 * Errors as qsa_paged_attn; nheads / nkv above 128, nseq above 65,535 or
 * total_q * nheads above 2^31 - 1 returns QSA_ERR_UNSUPPORTED.
 */
size_t qsa_window_attn_scratch_bytes(int nseq, int total_q, int max_q, int nheads, int nkv);
qsa_status qsa_window_attn(const void *q, const void *k, const void *v, qsa_dtype dtype, const int64_t *strides,
                           const int32_t *cu_q, const int32_t *cu_k, int nseq, int total_q, int total_k, int max_q,
                           int nheads, int nkv, int window, int sinks, float scale, void *out, float *lse,
                           void *scratch, size_t scratch_bytes, cudaStream_t stream);

/*
 * Eviction by accumulated attention weight: each sequence of n = lens[s]
 * cells (clamped as in qsa_paged_attn) keeps min(n, budget) of them: all when
 * n <= budget, else the first `sinks`, the last `recent`, and of the cells
 * between them the budget - sinks - recent with the largest mass (equal
 * masses: the lower cell first; NaN counts as -infinity, -0 as +0). The kept
 * cells keep their order: cell i of the new cache is a copy of cell kept[s][i]
 * (keys, values and int8 scales, bit for bit) in slot i % page_size of page
 * new_table[s][i / page_size] of the same pool.
 * kept      int32 [nseq][budget], written, ascending, -1 past the kept cells.
 * new_lens  int32 [nseq], written: min(n, budget).
 * new_mass  fp32, row stride new_mass_stride, new_mass_cols columns written:
 *           the kept cells' masses, then zeros.
 * The outputs overlap neither one another nor the inputs (new_lens == lens or
 * new_mass == mass returns QSA_ERR_INVALID).
 * Pages of new_table must not be pages that any row of page_table uses for a
 * cell below its length, nor appear twice (else the copied cells are
 * undefined). A page id outside [0, npages) on either side skips the copy of
 * that cell. budget >= 1, sinks + recent <= budget <= new_cols * page_size,
 * budget <= new_mass_cols; mass_stride >= table_cols * page_size. Size limits
 * as qsa_paged_attn. Allocates nothing.
 */
qsa_status qsa_cache_evict(const qsa_kv_pages *kv, int nseq, const int32_t *page_table, int table_cols,
                           int64_t table_stride, const int32_t *lens, const float *mass, int64_t mass_stride,
                           const int32_t *new_table, int new_cols, int64_t new_table_stride, int budget, int sinks,
                           int recent, int32_t *kept, int32_t *new_lens, float *new_mass, int64_t new_mass_stride,
                           int new_mass_cols, cudaStream_t stream);

/* ---- New tokens in the paged cache: rotation by position, append, attention over a shared prefix ---- */

/*
 * Rotation by position of the first 2 * npairs elements of a head's 128
 * (the others stay as they are). Pair p is elements (p, p + npairs), or
 * (2 p, 2 p + 1) where `interleaved`; it is turned by
 *   angle = position * freqs[p]:  (a, b) -> (a cos - b sin, b cos + a sin),
 * by -angle where `inverse` (which undoes it, and is its gradient). The
 * position of token t for pair p is positions[axis[p] * position_stride + t]:
 * one axis for text, several (time, height, width) for images and video, an
 * axis for each pair. A pair whose axis is outside [0, naxes) is turned by 0. The
 * formula holds for every angle: an infinity or NaN in a pair can make both NaN.
 * The angle is reduced exactly (fixed point, to 2^-32 turns), whatever the
 * position and the frequency; sine, cosine and products are fp32, the result is rounded once.
 * A frequency that is not finite gives NaN.
 * freqs     fp32 [npairs]; npairs a multiple of 8, 8 .. 64.
 * axis      int32 [npairs], or NULL: axis 0 for every pair.
 * positions int32 [naxes] rows of one element per token, row stride
 *           position_stride (elements, not negative), 4-byte aligned.
 */
typedef struct {
    const float *freqs;
    const int32_t *axis, *positions;
    int64_t position_stride;
    int32_t npairs, naxes, interleaved, inverse;
} qsa_rotation;

/*
 * out[t][h] = x[t][h] rotated by token t's position (see qsa_rotation).
 * x, out    [ntok][nheads][128] of dtype (QSA_F32, QSA_F16 or QSA_BF16),
 *           16-byte aligned; strides: element strides of x per token and head,
 *           then of out, multiples of 16 bytes, not negative; out's rows are
 *           apart: its narrower stride is at least 128, its wider one past the last row of the
 *           narrower dimension (a dimension of one element: any). out is x itself (same
 *           address and strides) or does not overlap it: refused where the strides
 *           are the same, or the address; other overlaps are the caller's to avoid.
 * A missing rotation, frequency or position, a bad type, size, pointer or
 * stride returns QSA_ERR_INVALID; nheads or naxes above 65,535 or ntok above
 * 2^31 - 64 QSA_ERR_UNSUPPORTED.
 */
qsa_status qsa_rotate(const void *x, qsa_dtype dtype, const int64_t *strides, int ntok, int nheads,
                      const qsa_rotation *rotation, void *out, cudaStream_t stream);

/*
 * Appends new tokens to a paged cache. Tokens cu[s] .. cu[s+1]-1 are the new
 * tokens of sequence s, the last of its lens[s] cells (lens counts them
 * already, as the attention calls that follow want it): token t's cell is
 * lens[s] - (cu[s+1] - t), in the pages as qsa_paged_attn reads them.
 *   key cell = rotated k[t], value cell = v[t]; q_out[t] = rotated q[t], k_out[t] = rotated k[t]
 * Without a rotation keys are copied and there is no q. Without positions
 * (naxes 1) a token's position is its cell's number; `inverse` has to be 0.
 * int8 pages: scale = binary16(max_d |x_d| / 127) (to nearest even, 65504 at
 * most), codes rint(x_d / scale), at most 127 in size (0 where the scale is 0),
 * in fp32; a cell with an infinity or NaN gets scale NaN and codes 0.
 * Tokens of no sequence (below cu[0], from cu[nseq] on) are left out: nothing
 * of theirs is written. A cell below 0, at or past table_cols * page_size, or
 * whose page number is outside [0, npages) is not written (q_out and k_out are).
 * Two tokens with the same cell leave it undefined.
 * k, v      [ntok][nkv][128], q [ntok][nheads][128] (or NULL, with nheads 0),
 *           of dtype: QSA_F32, or the pages' type; any of the three 16- and
 *           32-bit types for int8 pages. q_out and k_out (or NULL) of dtype.
 *           q_out with q; k_out only with a rotation.
 * strides   of k, v, q, q_out, k_out per token and head (10 numbers, elements;
 *           rules as qsa_rotate's; those of missing tensors are not read).
 *           q_out may be q itself, k_out k itself; no other overlaps.
 * The pages' cells (and scales) are apart here: each stride of a dimension of
 * more than one element is past all that the narrower ones span,
 * and keys' do not overlap values' (without a rotation they may be the same, for
 * k and v that are the same rows).
 * cu        int32 [nseq + 1], ascending (values are clamped to [0, ntok]), or
 *           NULL: one token per sequence, ntok == nseq.
 * page_table, lens as qsa_paged_attn. Errors and limits as qsa_paged_attn and qsa_rotate.
 */
qsa_status qsa_cache_append(const void *k, const void *v, const void *q, qsa_dtype dtype, const int64_t *strides,
                            int ntok, int nheads, const qsa_kv_pages *kv, const int32_t *page_table, int table_cols,
                            int64_t table_stride, const int32_t *lens, const int32_t *cu, int nseq,
                            const qsa_rotation *rotation, void *q_out, void *k_out, cudaStream_t stream);

/*
 * Attention of one new token per sequence where groups of sequences share a
 * long prefix: the result of qsa_paged_attn (without window and mass) over the
 * prefix's cells and then the sequence's own, with the prefix read once for
 * all sequences of its group, and with weights of fewer bits (below). It
 * pays from some 60,000 to 130,000 prefix cells on, counted for every sequence and KV head
 * (int8: 150,000 to 270,000); under that qsa_paged_attn over both, in one table, is faster.
 * Group g is sequences cu_seqs[g] .. cu_seqs[g+1]-1; its prefix is the first
 * prefix_lens[g] cells of the pages of row g of prefix_table. Sequence s has
 * lens[s] cells of its own in the pages of row s of page_table (its own token
 * among them). A sequence of no group (before cu_seqs[0], from cu_seqs[ngroups] on) has
 * no prefix. logit, lse and out as qsa_paged_attn, over both; without any cell
 * out = 0 and lse = -infinity. Lengths are clamped to their tables' capacity;
 * a cell whose page number is outside [0, npages) is skipped. Cells that are
 * not there are never used, whatever they hold; an infinity or NaN in a cell's value
 * (or its scale) makes results of all sequences that see it infinite or NaN.
 * cu_seqs   int32 [ngroups + 1], ascending (values are clamped to [0, nseq];
 *           where they are not ascending the results are unspecified).
 * prefix_table int32, row stride prefix_stride >= prefix_cols; prefix_lens int32
 *           [ngroups]. The rest as in qsa_paged_attn, q_dtype among it.
 * scratch   at least qsa_prefix_attn_scratch_bytes(...) bytes, 16-byte aligned
 *           (0 for nseq = 0 and for arguments that are refused); no contents
 *           need survive.
 * Sums and softmax statistics are fp32; the tensor cores' sums, which they cut
 * off towards zero at every 16 cells, are over 32,768 cells of a prefix at
 * most (256 for fp32 queries) before they are added to others, rounded. The weights of prefix cells are rounded
 * once to the 16-bit operand type (the pages', binary16 for int8 cells), as in
 * qsa_window_attn, where qsa_paged_attn keeps 17 or 22 bits; for fp32 queries they keep 22 bits.
 * Errors and limits as qsa_paged_attn; nheads / nkv above 128, ngroups above 65,535,
 * prefix_cols * page_size above 2^30 or (nseq + ngroups) * nheads *
 * ceil(prefix_cols * page_size / 128) above 2^38 returns QSA_ERR_UNSUPPORTED.
 */
size_t qsa_prefix_attn_scratch_bytes(int nseq, int ngroups, int nheads, int nkv, int prefix_cols, int table_cols,
                                     int page_size);
qsa_status qsa_prefix_attn(const void *q, qsa_dtype q_dtype, int64_t q_seq_stride, int64_t q_head_stride, int nseq,
                           int nheads, const qsa_kv_pages *kv, const int32_t *prefix_table, int prefix_cols,
                           int64_t prefix_stride, const int32_t *prefix_lens, const int32_t *cu_seqs, int ngroups,
                           const int32_t *page_table, int table_cols, int64_t table_stride, const int32_t *lens,
                           float scale, void *out, float *lse, void *scratch, size_t scratch_bytes,
                           cudaStream_t stream);

/* Static description of a status code. */
const char *qsa_status_string(qsa_status status);

#ifdef __cplusplus
}
#endif

#endif /* QSA_H */
