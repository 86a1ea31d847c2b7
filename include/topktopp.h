/*
 * libtopktopp — per-row top-k / top-p logits filter for AMD Instinct MI355X (gfx950).
 *
 * What is computed. For every row b of a [B, V] logits matrix the filter
 * follows the eight steps of the CANN ops-nn page "ApplyTopKTopPWithSorted 的
 * top-k/top-p 采样过滤原理与 aclnn 调用指南" (cited below as AKP), §2:
 *   1-3. the k-th largest value of the row is the top-k threshold and every
 *        value strictly below it is masked;
 *   4-5. a softmax (fp32 or wider) of the surviving values is accumulated
 *        from the smallest probability upwards;
 *   6-7. every position whose cumulative probability is <= 1 - p[b] is masked,
 *        except the last (largest) position, which always survives;
 *   8.   the result is returned in the original vocabulary order.
 * The order is the stable ascending sort of the row: equal values (and -0.0
 * next to +0.0, which compare equal) keep their original index order, so at
 * a top-p boundary inside a run of equal values the lower indices are masked
 * first. A kept position holds the input bits unchanged; a masked position
 * holds the dtype's -inf (fp32 0xFF800000, fp16 0xFC00, bf16 0xFF80; AKP §6.3).
 *
 * Modes (AKP §4, §5.2). p and k are each optional, but not both. k[b] <= 0 or
 * k[b] >= V disables top-k for that row. p[b] >= 1 disables top-p in effect
 * (nothing with positive probability is masked); p[b] <= 0 keeps only the
 * last sorted position. Values of p are applied as given, without clamping.
 *
 * Numerics. t = 1 - p[b] is formed in fp32 from p widened exactly. The
 * cumulative probabilities are computed on the device in fp32/fixed-point
 * arithmetic whose summation order differs from a sequential sum; only
 * positions whose exact cumulative probability lies within about 1e-5 of t
 * can be decided differently from an exact evaluation. The top-k mask and
 * the kept values are exact. Results are deterministic: the same inputs give
 * the same output bits on every call.
 *
 * Memory and streams. Every data pointer is a device pointer owned by the
 * caller; nothing is retained after the call returns. Work is enqueued on
 * `stream` (a hipStream_t; NULL means the default stream) and the call
 * returns without synchronising. The library allocates no device memory
 * and the entry points never call hipMalloc. `out` must not overlap any input.
 * Rows are dense and row-major: element (b, v) sits at offset b * V + v,
 * except where an entry point takes strides (the _ex and _strided ones).
 *
 * Errors. Arguments are checked on the host before anything is enqueued, in
 * the order of the aclnn checks (AKP §5.3): null pointers first, then dtype,
 * then shape. On an error nothing is enqueued, and topktopp_last_error()
 * describes the problem. Device data (the values of p, k, sortedness) is not
 * validated.
 */
#ifndef TOPKTOPP_H
#define TOPKTOPP_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of logits, sorted values, p and out (AKP §3 and §5.2 tables). */
typedef enum {
  TOPKTOPP_F32 = 0,
  TOPKTOPP_F16 = 1,
  TOPKTOPP_BF16 = 2
} topktopp_dtype;

/* Return codes, mirroring the aclnn ones of AKP §5.3. */
typedef enum {
  TOPKTOPP_OK = 0,
  TOPKTOPP_ERR_NULLPTR = 1, /* logits/sorted input/out is NULL, or p and k are both NULL (aclnn 161001) */
  TOPKTOPP_ERR_INVALID = 2, /* unsupported dtype, negative or too large shape, overlapping out (aclnn 161002) */
  TOPKTOPP_ERR_RUNTIME = 3  /* a HIP launch failed; the message names the HIP error */
} topktopp_status;

/* Largest supported row length, 2^20 (the same bound the companion sampling
 * operator, aclnnTopKTopPSampleV2, states for its vocabulary size). */
#define TOPKTOPP_MAX_V (1 << 20)

/* Largest supported number of rows, 2^31 - 1. Batches of more than 2^21
 * rows are launched in row chunks. */
#define TOPKTOPP_MAX_B 0x7FFFFFFFLL

/* Largest row stride accepted by the _ex entry points, in elements (2^31). */
#define TOPKTOPP_MAX_LD (1LL << 31)

/*
 * apply_top_k_top_p — filter raw logits (the aclnn entry of AKP §5 and §6.1,
 * which sorts internally). No sort is materialised: the threshold pair that
 * the stable sort would produce is found by radix selection.
 *
 *   logits  [B, V] device buffer of `dtype` values.
 *   dtype   one of topktopp_dtype.
 *   B, V    rows and row length; B == 0 or V == 0 is a successful no-op
 *           (every pointer may then be NULL; only dtype is checked);
 *           V == 1 copies logits to out (AKP §6.1); V <= TOPKTOPP_MAX_V,
 *           B <= TOPKTOPP_MAX_B.
 *   p       [B] device buffer of `dtype` values, or NULL for no top-p.
 *   k       [B] device buffer of int32, or NULL for no top-k.
 *   out     [B, V] device buffer of `dtype`, written completely.
 *   stream  hipStream_t to enqueue on, or NULL.
 */
topktopp_status apply_top_k_top_p(const void* logits, topktopp_dtype dtype, int64_t B, int64_t V,
                                  const void* p, const int32_t* k, void* out, void* stream);

/*
 * apply_top_k_top_p_with_sorted — the sorted-input operator
 * ApplyTopKTopPWithSorted (AKP §1 and the §3 parameter table).
 *
 *   sorted_value    [B, V] device buffer, each row ascending.
 *   sorted_indices  [B, V] int32 device buffer, each row the permutation that
 *                   produced sorted_value from the original row. Positions in
 *                   this order decide ties.
 *   dtype, B, V, p, k, out, stream   as for apply_top_k_top_p.
 *   logits          [B, V] original (unsorted) values, or NULL. When given,
 *                   kept outputs are read from it in the original order and
 *                   sorted_value[b][j] must equal logits[b][sorted_indices[b][j]].
 *                   When NULL, out is written by scattering through
 *                   sorted_indices.
 * Sortedness and the permutation are the caller's contract and are not checked.
 */
topktopp_status apply_top_k_top_p_with_sorted(const void* sorted_value, const int32_t* sorted_indices,
                                              topktopp_dtype dtype, int64_t B, int64_t V, const void* p,
                                              const int32_t* k, const void* logits, void* out,
                                              void* stream);

/*
 * apply_top_k_top_p_min_p — apply_top_k_top_p followed by the min-p stage of
 * Ascend's "aclnnTopKTopPSampleV2" page ("minP sampling"; cited as TKS).
 *
 *   min_p   [B] device buffer of `dtype` values (like p), or NULL for no
 *           min-p. Other arguments as for apply_top_k_top_p; p, k and min_p
 *           may each be NULL, but not all three (ERR_NULLPTR).
 *
 * Min-p takes the probabilities left after top-k and top-p (the softmax of
 * the top-k survivors, step 4 above) and masks every position whose
 * probability is strictly below the largest one times min_p[b]; as the
 * ratio of two of those probabilities is exp(x - x_max), a position survives
 * iff exp(x - x_max) >= min_p[b]. min_p[b] <= 0 (or NaN) skips the stage;
 * min_p[b] >= 1 keeps a single position, the maximum with the highest
 * original index (TKS keeps one token with the maximum value; this takes the
 * stable order's last one, as p <= 0 does). Each stage masks a prefix of the
 * stable ascending order, so the survivors are those of all stages at once.
 *
 * Numerics. exp is taken in fp32 on the device; only positions whose exact
 * ratio lies within a relative 1e-5 of min_p[b] can be decided differently
 * from an exact evaluation.
 */
topktopp_status apply_top_k_top_p_min_p(const void* logits, topktopp_dtype dtype, int64_t B, int64_t V,
                                        const void* p, const int32_t* k, const void* min_p, void* out,
                                        void* stream);

/*
 * apply_top_k_top_p_min_p_with_sorted — apply_top_k_top_p_with_sorted
 * followed by the min-p stage described for apply_top_k_top_p_min_p.
 *   min_p   [B] device buffer of `dtype` values, or NULL. Other arguments as
 *           for apply_top_k_top_p_with_sorted; p, k and min_p may each be
 *           NULL, but not all three.
 */
topktopp_status apply_top_k_top_p_min_p_with_sorted(const void* sorted_value, const int32_t* sorted_indices,
                                                    topktopp_dtype dtype, int64_t B, int64_t V, const void* p,
                                                    const int32_t* k, const void* min_p, const void* logits,
                                                    void* out, void* stream);

/*
 * apply_top_k_top_p_ex — apply_top_k_top_p_min_p on row-strided operands: row
 * b of logits starts at element b * ld_logits and row b of out at element
 * b * ld_out (a [B, V] view of a wider buffer, e.g. a vocabulary padded to a
 * multiple of 64; the aclnn entry makes such views contiguous first, AKP
 * §6.1). Elements within a row are contiguous. Each stride must be >= V and
 * <= TOPKTOPP_MAX_LD (else ERR_INVALID); the strided extents of out and the
 * inputs must not overlap. Positions between V and the stride are neither
 * read nor written. Other arguments as for apply_top_k_top_p_min_p.
 */
topktopp_status apply_top_k_top_p_ex(const void* logits, int64_t ld_logits, topktopp_dtype dtype, int64_t B, int64_t V,
                                     const void* p, const int32_t* k, const void* min_p, void* out,
                                     int64_t ld_out, void* stream);

/*
 * apply_top_k_top_p_strided — apply_top_k_top_p_min_p on arbitrary strided
 * views (the aclnn entry accepts non-contiguous tensors and makes them
 * contiguous before filtering, AKP §6.1; this reads and writes the views in
 * place instead). All strides are in elements:
 *   logits  element (b, v) at logits[b * logits_row_stride + v * logits_col_stride];
 *   out     element (b, v) at out[b * out_row_stride + v * out_col_stride];
 *   p, k, min_p   entry b at p[b * p_stride], k[b * k_stride],
 *           min_p[b * min_p_stride] (a stride of 0 shares one value among
 *           all rows; the stride of a NULL operand is ignored).
 * E.g. a [V, B] buffer filtered as its transpose passes row stride 1 and
 * column stride B. Input strides must lie in [0, TOPKTOPP_MAX_LD]; out's in
 * [1, TOPKTOPP_MAX_LD] (ignored along an extent of 1), and out must give
 * every (b, v) its own element: one of its strides must be at least the
 * other times that other dimension's extent (out_row_stride >= V *
 * out_col_stride, or out_col_stride >= B * out_row_stride), else
 * ERR_INVALID. The byte span of out (from its first to its last element)
 * must not overlap the span of any input. Elements of the spans that belong
 * to no (b, v) are neither read nor written. Other arguments, checks and
 * results as for apply_top_k_top_p_min_p (p, k and min_p may each be NULL,
 * but not all three).
 *
 * When rows are contiguous (logits_col_stride == out_col_stride == 1, row
 * strides >= V) and p, k and min_p are dense, this is apply_top_k_top_p_ex.
 * Otherwise every element is accessed on its own by a streamed kernel, which
 * is several times slower than the vector path of contiguous rows.
 */
topktopp_status apply_top_k_top_p_strided(const void* logits, int64_t logits_row_stride, int64_t logits_col_stride,
                                          topktopp_dtype dtype, int64_t B, int64_t V, const void* p, int64_t p_stride,
                                          const int32_t* k, int64_t k_stride, const void* min_p,
                                          int64_t min_p_stride, void* out, int64_t out_row_stride,
                                          int64_t out_col_stride, void* stream);

/*
 * apply_top_k_top_p_with_sorted_ex — apply_top_k_top_p_min_p_with_sorted on
 * row-strided operands, one row stride (in elements) per [B, V] operand, with
 * the rules of apply_top_k_top_p_ex. ld_logits is ignored when logits is NULL.
 */
topktopp_status apply_top_k_top_p_with_sorted_ex(const void* sorted_value, int64_t ld_sorted_value,
                                                 const int32_t* sorted_indices, int64_t ld_sorted_indices,
                                                 topktopp_dtype dtype, int64_t B, int64_t V, const void* p,
                                                 const int32_t* k, const void* min_p, const void* logits,
                                                 int64_t ld_logits, void* out, int64_t ld_out, void* stream);

/*
 * sample_top_k_top_p — the filter (top-k, top-p, min-p as in
 * apply_top_k_top_p_min_p) followed by the sampling stage of TKS
 * ("Subsequent processing"), one index per row. probs are the filtered
 * probabilities in descending order; descending order is the reverse of the
 * stable ascending order, so among equal values the higher original index
 * comes first.
 *
 *   logits, dtype, B, V, p, k, min_p   as for apply_top_k_top_p_min_p, except
 *            that p, k and min_p may all be NULL (sampling from the whole row).
 *   q        [B, V] fp32 device buffer, or NULL.
 *            NULL ("None" mode): selected[b] is the index of the first
 *            maximum of probs, the maximum value with the highest index.
 *            Given ("QSample"): selected[b] is the index of the first maximum
 *            of probs / (q[b][r] + eps), q[b][r] pairing with the survivor of
 *            descending rank r; only the first n_b entries of a row are read,
 *            n_b being the row's survivor count.
 *   eps      added to q; finite and >= 0 (the pages give it no value).
 *   out      [B, V] device buffer for the filtered logits, or NULL to skip
 *            them (then the row is only read, not written).
 *   selected [B] int32 device buffer, written completely, with an index in
 *            [0, V) for every row, whatever its number of survivors.
 * Errors as for apply_top_k_top_p_min_p; selected NULL is ERR_NULLPTR, a
 * negative or non-finite eps ERR_INVALID, and out or selected overlapping
 * another buffer ERR_INVALID.
 */
topktopp_status sample_top_k_top_p(const void* logits, topktopp_dtype dtype, int64_t B, int64_t V, const void* p,
                                   const int32_t* k, const void* min_p, const float* q, float eps, void* out,
                                   int32_t* selected, void* stream);

/*
 * top_k_top_p_sorted_survivors — the filter (as apply_top_k_top_p_min_p)
 * returning the survivors themselves, in descending order, instead of the
 * filtered row: the intermediate output of TKS (logitsSortMasked and
 * logitsIdx, "Intermediate result output"), cut to the survivors. For row b
 * and descending rank r < min(n_b, cap), with n_b the row's survivor count:
 *   probs[b][r]    the survivor's probability of step 4 (the softmax over the
 *                  top-k survivors, fp32), or skipped when probs is NULL;
 *   indices[b][r]  its original index (int32);
 * ranks n_b .. cap-1 hold probability 0 and index -1; counts[b] = n_b (which
 * may exceed cap). Descending order is the reverse of the stable ascending
 * order (equal values: higher index first). p, k and min_p may each be NULL.
 *   cap     entries per output row, 1 <= cap <= 2^20 (else ERR_INVALID).
 *   probs   [B, cap] fp32 device buffer, or NULL.
 *   indices [B, cap] int32 device buffer.
 *   counts  [B] int32 device buffer.
 * Every row lists min(n_b, cap) survivors, whatever n_b is (up to V).
 * Errors as for apply_top_k_top_p_min_p; outputs may not overlap inputs or
 * each other (ERR_INVALID).
 */
topktopp_status top_k_top_p_sorted_survivors(const void* logits, topktopp_dtype dtype, int64_t B, int64_t V, const void* p,
                                             const int32_t* k, const void* min_p, int64_t cap, float* probs,
                                             int32_t* indices, int32_t* counts, void* stream);

/*
 * Beam search. A step of a search over K beams for each of N prompts takes
 * the model's logits of the N * K rows (row i * K + b is beam b of prompt i):
 * beam_search_select picks the continuations, beam_reorder_states makes the
 * model's states follow them, and beam_backtrace reads the sequences out of
 * the steps' tokens and parents at the end. Nothing waits for the host, so a
 * step can be captured in a graph. To search among filtered tokens only, pass
 * logits that apply_top_k_top_p has filtered: -inf is no continuation, and
 * probabilities are those of what is left.
 */
#define TOPKTOPP_MAX_BEAMS 128      /* beams per prompt */
#define TOPKTOPP_MAX_CANDIDATES 256 /* continuations picked per prompt */

/*
 * beam_search_select — the n best continuations over beams and vocabulary.
 *
 *   logits     [N * K, V] device buffer of `dtype`; row r starts at element
 *              r * ld_logits (V <= ld_logits <= TOPKTOPP_MAX_LD).
 *   scores     [N, K] fp32: the beams' accumulated log-probabilities c.
 *   finished   [N, K] bytes, nonzero where a beam is finished, or NULL.
 *   end_token  the token of a finished beam's continuation, >= 0 (not read
 *              when finished is NULL).
 *   weights    [N, K] fp32 > 0, or NULL for 1: what the beam's scores are
 *              multiplied with for the ranking, e.g. a length normalisation.
 *   n          continuations per prompt, 1 <= n <= TOPKTOPP_MAX_CANDIDATES.
 *   out_scores [N, n] fp32, out_parents [N, n] int32 (beam), out_tokens
 *              [N, n] int32, in descending rank, written completely.
 *   workspace  beam_search_select_workspace() bytes of device memory,
 *              16-byte aligned. It holds nothing between calls; calls that
 *              may run at the same time need one each.
 *
 * The continuation of beam b with token v has the score
 *   s = c[b] + logits[b][v] - log(sum_u exp(logits[b][u]))
 * and the rank value s * weights[b]. A finished beam has one continuation:
 * itself, with end_token and the score c[b], whatever its logits hold. Equal
 * rank values are ordered by beam (lower first), then by logit (larger
 * first), then by token (lower first). Tokens with a logit of -inf are no
 * continuations. A beam has none at all if its score is infinite or NaN, its
 * weight is not positive and finite, or its logits hold a NaN or +inf or
 * nothing above -inf. Ranks without a continuation hold score -inf, parent
 * -1 and token -1.
 *
 * Numerics. A sum of exp has a relative error below 3.6e-7, what follows is
 * formed in 64 bits and rounded once, to out_scores. Where two beams'
 * continuations come closer than that error and the roundings of their rank
 * values, or tie, their sums are formed again in 64 bits (or found to be those
 * of rows with the same bits), so the order is that of 64-bit values. Of two
 * that only the roundings of 64 bits tell apart, either may come first.
 * Results are deterministic.
 *
 * Errors: ERR_NULLPTR for logits (unless V is 0), scores, an output or the
 * workspace NULL; ERR_INVALID for a dtype, N < 0, K outside
 * [1, TOPKTOPP_MAX_BEAMS], V outside [0, TOPKTOPP_MAX_V], N * K above
 * TOPKTOPP_MAX_B, n out of range, a stride below V, end_token < 0, a
 * workspace that is too small or not aligned, logits not aligned to their
 * element, or an output or the workspace overlapping anything else. N == 0
 * is a successful no-op.
 */
topktopp_status beam_search_select(const void* logits, int64_t ld_logits, topktopp_dtype dtype, int64_t N, int64_t K,
                                   int64_t V, const float* scores, const uint8_t* finished, int32_t end_token,
                                   const float* weights, int64_t n, float* out_scores, int32_t* out_parents,
                                   int32_t* out_tokens, void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace that beam_search_select needs for these sizes (at least
 * 16), or -1 if it would refuse them. */
int64_t beam_search_select_workspace(topktopp_dtype dtype, int64_t N, int64_t K, int64_t V, int64_t n);

/*
 * A state whose rows follow the beams, e.g. one layer's key cache: byte b of
 * the element at row r, indices i0, i1, i2 and position t lies at
 *   data + r * row_stride + i0 * stride[0] + i1 * stride[1] + i2 * stride[2]
 *        + t * position_stride + b,   0 <= b < run.
 * All strides and the run (an element, or several that lie side by side) are
 * in bytes; sizes are counts, 1 for an axis that is not there.
 */
typedef struct {
  void* data;
  int64_t row_stride;
  int64_t size[3];
  int64_t stride[3];
  int64_t positions;
  int64_t position_stride;
  int64_t run;
} topktopp_beam_state;

/*
 * beam_reorder_states — in every state, row i * K + b becomes what row
 * i * K + parents[i][b] was before the call. Columns of the rows are moved, of
 * 16 bytes where all strides, the data and a row's pieces allow it, else of 4, 2
 * or 1 bytes, which is slower. Positions that follow each other without a gap
 * (position_stride == run) take columns of 2 bytes or 1 where the run is no
 * multiple of 4, so that a length may end anywhere; a state that is moved whole
 * is better described without positions, as longer runs.
 *
 *   states   host array of `count` descriptions (0 <= count), read during the
 *            call. Rows of a state: N * K. A state that shares memory with an
 *            earlier one is moved after it.
 *   parents  [N, K] int32 device buffer; a row whose parent lies outside
 *            [0, K) (e.g. the -1 of a rank without a continuation) stays as
 *            it is.
 *   lengths  [N] int32 device buffer, or NULL: positions t < lengths[i] of
 *            prompt i are moved, those behind are neither read nor written
 *            (reads of a moved row may reach up to 15 bytes further).
 *   N, K     1 <= K <= TOPKTOPP_MAX_BEAMS, N * K <= TOPKTOPP_MAX_B.
 * ERR_NULLPTR for states, a state's data or parents NULL; ERR_INVALID for
 * sizes out of range, negative sizes, elements of one state that share memory
 * (a sufficient condition: in ascending order, each axis's stride reaches
 * past all that the axes below it span), a state of more than 2^31 - 1
 * columns per row (columns have 16 bytes where alignment allows), or parents
 * or lengths inside a state. States with a size of 0 are skipped; nothing is
 * moved if any argument is refused.
 */
topktopp_status beam_reorder_states(const topktopp_beam_state* states, int64_t count, const int32_t* parents,
                                    int64_t N, int64_t K, const int32_t* lengths, void* stream);

/*
 * beam_backtrace — sequences out of a search's history.
 *
 *   tokens, parents  [T, N, K] int32: what was picked in each step; parents
 *            of step t are beams of step t - 1 (those of step 0 are not used).
 *   M        hypotheses per prompt, >= 0.
 *   beams    [N, M] int32, the beam at which hypothesis m ends, or NULL for
 *            beam m (then M <= K).
 *   lengths  [N, M] int32, its number of steps, or NULL for T (values are
 *            clamped to [0, T]).
 *   out      [N, M, T] int32, written completely: out[i][m][t] is the token
 *            of step t for t < lengths[i][m], and `pad` behind. Steps before a
 *            beam or parent outside [0, K) hold `pad`, as that step does for
 *            a beam outside.
 * ERR_NULLPTR for tokens, parents or out NULL; ERR_INVALID for negative
 * sizes, K outside [1, TOPKTOPP_MAX_BEAMS], N * K or T above 2^31 - 1, M above
 * 2^20, M > K without beams, or out overlapping an input. N, T or M of 0 is a
 * successful no-op.
 */
topktopp_status beam_backtrace(const int32_t* tokens, const int32_t* parents, int64_t T, int64_t N, int64_t K,
                               const int32_t* beams, const int32_t* lengths, int64_t M, int32_t pad, int32_t* out,
                               void* stream);

/* ------------------------------------------------- speculative decoding --- */

#define TOPKTOPP_MAX_DRAFTS 255

/*
 * speculative_verify — how many drafted tokens stand, and the token behind them.
 *
 *   logits     [N * (D + 1), V], rows ld_logits elements apart, of any dtype:
 *              row i * (D + 1) follows the last token of sequence i, row
 *              i * (D + 1) + 1 + j its draft j. As they are to be sampled from:
 *              divided by the temperature, filtered tokens at -inf.
 *   D          drafts of a sequence, 0 <= D <= TOPKTOPP_MAX_DRAFTS.
 *   drafts     [N, D] int32 tokens.
 *   uniforms   [N, D + 1] fp32 in [0, 1), or NULL: greedy.
 *   draft_logits  [N * D, V] in the dtype of logits, rows ld_draft elements
 *              apart: row i * D + j is what draft j was drawn from; or NULL for
 *              drafts that were not drawn. Needs uniforms, and no parents.
 *   parents    [N, D] int32: draft j follows draft parents[i][j] < j, or -1 for
 *              the last token, so that the drafts form a tree; or NULL for a
 *              chain, each behind the one before it.
 *   lengths    [N] int32, drafts of a sequence that count (values are clamped
 *              to [0, D]), or NULL for D.
 *   out_tokens [N, D + 1] int32, written completely: the accepted drafts, the
 *              token behind them, and -1.
 *   out_accepted  [N] int32, the number of accepted drafts.
 *   out_path   [N, D] int32, the accepted drafts' numbers and -1, or NULL.
 *   workspace  speculative_verify_workspace() bytes of device memory, 16-byte
 *              aligned. It holds nothing between calls; calls that may run at
 *              the same time need one each.
 *
 * With p_w the softmax of target row w, q_j that of draft row j and u the
 * sequence's uniforms, at the last token (w = 0) or behind accepted draft w - 1:
 *   - with draft logits, draft w is accepted if u[w] q_w(d) < p_w(d), d its
 *     token. If it is not, the token behind is drawn from max(p_w - q_w, 0), or
 *     from p_w if that adds up to no more than 2^-40.
 *   - without, the drafts behind w in the order of their numbers cut [0, 1) into
 *     pieces of p_w(token), and the one whose piece holds u[w] is accepted; a
 *     token that an earlier one of them has counts once. If there is none, the
 *     token is drawn from p_w without these tokens, or from p_w if that adds up
 *     to no more than 2^-40.
 *   - where no draft follows, the token is drawn from p_w.
 *   - greedy, the largest logit (the lowest token of equal ones) accepts the
 *     draft behind w that has it, or else is the token behind.
 * Drawn from weights r: the lowest token v with sum_{t <= v} r(t) > u[D] sum r
 * (for a uniform of 1 or more, the last one of any weight).
 * Drafts whose token lies outside [0, V), or whose parent lies outside
 * [-1, j), count as not there. A target row with a NaN or +inf, or with nothing
 * above -inf, accepts nothing and gives the token -1; in such a draft row q is 0.
 *
 * Numerics. The sums of exp behind an acceptance have a relative error below
 * 1e-6; a decision that this could turn is made again with sums in 64 bits, as
 * are all sums behind a drawn token. Of two outcomes that only the roundings of
 * 64 bits tell apart, either may come. Every logit above -inf has weight, so a
 * uniform of 0 draws the first such token, however far it lies below the others;
 * only beyond what 64 bits hold (650 below the row's largest, or more) may it count
 * as 0. Results are deterministic.
 *
 * Errors: ERR_NULLPTR for logits (unless V is 0), drafts (unless D is 0),
 * out_tokens, out_accepted or the workspace NULL; ERR_INVALID for a dtype, N < 0,
 * D or V out of range, N * (2 D + 1) above TOPKTOPP_MAX_B, a stride below V,
 * draft_logits without uniforms or with parents, a workspace that is too small or
 * not aligned, logits not aligned to their element, or an output or the workspace
 * overlapping anything else. N == 0 is a successful no-op.
 */
topktopp_status speculative_verify(const void* logits, int64_t ld_logits, topktopp_dtype dtype, int64_t N, int64_t D,
                                   int64_t V, const int32_t* drafts, const float* uniforms, const void* draft_logits,
                                   int64_t ld_draft, const int32_t* parents, const int32_t* lengths,
                                   int32_t* out_tokens, int32_t* out_accepted, int32_t* out_path, void* workspace,
                                   int64_t workspace_bytes, void* stream);

/* Bytes of workspace that speculative_verify needs for these sizes (at least
 * 16), with or without draft logits, or -1 if it would refuse them. */
int64_t speculative_verify_workspace(topktopp_dtype dtype, int64_t N, int64_t D, int64_t V, int draft_logits);

/* -------------------------------------------------------- caches in pages --- */

/*
 * A page table. Position t of row r lies in page tables[r * ld_tables +
 * t / page_size] at slot t % page_size; a row holds the pages of its first
 * lengths[r] positions, C at most, and its entries behind them are not used.
 *   tables     [R, C] int32 device buffer, rows ld_tables >= C entries apart.
 *   lengths    [R] int32.
 *   uses       [P] int32, how many held entries name each page. A page with 0
 *              is free.
 *   page_size  slots of a page, >= 1; C * page_size <= 2^31 - 1.
 * The three belong together and are kept so by the calls below: begin with
 * lengths and uses of 0. Entries outside [0, P) name no page.
 *
 * cache_pages_fork — rows follow their beams, in place: row i * K + b becomes
 * what row i * K + parents[i][b] was (its length, its pages), for R = N * K. The
 * pages themselves are not touched: rows that come from one share them.
 *   parents  [N, K] int32; a row whose parent lies outside [0, K) stays as it is.
 * ERR_NULLPTR for tables (unless C is 0), lengths, parents or uses (unless P is
 * 0) NULL; ERR_INVALID for K outside [1, TOPKTOPP_MAX_BEAMS], negative sizes,
 * N * K or P above TOPKTOPP_MAX_B, a page_size or C out of range, ld_tables below
 * C, or buffers that overlap.
 */
topktopp_status cache_pages_fork(int32_t* tables, int64_t ld_tables, int64_t C, int32_t* lengths,
                                 const int32_t* parents, int64_t N, int64_t K, int32_t* uses, int64_t P,
                                 int64_t page_size, void* stream);

/*
 * cache_pages_resize — row r is to hold new_lengths[r] positions. First, rows
 * that become shorter give back the pages behind their new end (their entries
 * become -1). Then rows that grow are served in order of their numbers: each gets
 * the pages that it lacks, free ones from the lowest number on, and where it is
 * going to write into its last page (not full) and other rows use that as well,
 * a page in its place into which its slots are copied. Rows that write into the
 * same page in one call and are all that use it copy it but for the last of them.
 * From the first row on that the free pages do not suffice for, growing rows
 * stay as they are; so do rows whose old or new length is below 0 or above
 * C * page_size. lengths[r] becomes new_lengths[r] for all others.
 *   caches     host array of `count` descriptions as for beam_reorder_states,
 *              read during the call, with P rows (the pages) and page_size
 *              positions (the slots). From the first byte of one to its last no
 *              other begins: views that lie between one another's elements, as
 *              keys and values of one tensor may, go as that tensor. With count 0
 *              nothing can be copied: the first row that would have to and the
 *              growing rows behind it stay as they are.
 *   workspace  cache_pages_resize_workspace(R, P) bytes, 16-byte aligned; calls
 *              that may run at the same time need one each.
 * ERR_NULLPTR for tables (unless C is 0), lengths, new_lengths, uses (unless P
 * is 0), the workspace, caches or a cache's data NULL; ERR_INVALID for sizes out
 * of range as above, a cache with other positions than page_size, one whose
 * elements share memory or of more than 2^31 - 1 columns of a page, a workspace
 * too small or not aligned, or buffers (caches: in the sense above) that
 * overlap. Nothing is changed if any argument is refused. R == 0 is a successful
 * no-op.
 */
topktopp_status cache_pages_resize(int32_t* tables, int64_t ld_tables, int64_t R, int64_t C, int32_t* lengths,
                                   const int32_t* new_lengths, int32_t* uses, int64_t P, int64_t page_size,
                                   const topktopp_beam_state* caches, int64_t count, void* workspace,
                                   int64_t workspace_bytes, void* stream);
int64_t cache_pages_resize_workspace(int64_t R, int64_t P);

/*
 * cache_pages_compact — the entries of an accepted path move behind one
 * another: in every cache, position starts[i] + j of sequence i becomes what
 * position starts[i] + path[i][j] was, for j < counts[i].
 *   path     [N, D] int32, D <= TOPKTOPP_MAX_DRAFTS: ascending numbers >= 0 (as
 *            out_path of speculative_verify). A path ends before the first one
 *            that is not larger than the one before it, or whose position lies
 *            outside the table.
 *   counts   [N] int32 (values are clamped to [0, D]); starts [N] int32.
 * Entries whose page, or whose place's page, lies outside [0, P) stay. The pages
 * written to must be used by one sequence only, as cache_pages_resize leaves
 * those behind the length that it started from.
 * Errors as for cache_pages_resize. N, D or count of 0 is a successful no-op.
 */
topktopp_status cache_pages_compact(const topktopp_beam_state* caches, int64_t count, int64_t P, int64_t page_size,
                                    const int32_t* tables, int64_t ld_tables, int64_t N, int64_t C,
                                    const int32_t* starts, const int32_t* path, int64_t D, const int32_t* counts,
                                    void* stream);

/* Text of the most recent error on the calling thread ("" if none); the
 * counterpart of aclGetRecentErrMsg (AKP §8). Valid until the next call on
 * the same thread. */
const char* topktopp_last_error(void);

/*
 * Launch-plan override, for tests and measurement. policy 0 (default) lets
 * the library choose: the candidate plan, with the row held in registers
 * when it fits; 1 forces the multi-pass plan for every row; 2 forces the
 * candidate plan with the row re-read from global memory. Every policy
 * computes the same filter; top-p decisions may differ only inside the
 * tolerance band described above. Returns the previous policy, or -1 for an
 * unknown value (which is ignored). The setting is process-wide.
 */
int topktopp_set_plan_policy(int policy);

#ifdef __cplusplus
}
#endif

#endif /* TOPKTOPP_H */
