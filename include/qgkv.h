/*
 * qgkv: the state of a decode next to the quantised linear layers of
 * qgemv.h: an 8-bit paged key/value cache, the attention that reads it, the
 * page operations of beam search and serving, and the beam selection
 * (sm_103a).  C ABI of libqgemv.so.  Plain pointers and sizes only.
 *
 * The cache.  K and V are held as 8-bit codes, one fp32 scale for each block
 * of tokens and head; the block is a page: `page_tokens` consecutive tokens
 * of one sequence.  value = code * scale.
 *   k, v              uint8 [layers][pages][heads][page_tokens][head_dim]   (QGKV_HND)
 *                  or uint8 [layers][pages][page_tokens][heads][head_dim]   (QGKV_NHD)
 *                  dense inside a page; pages and layers are page_stride and
 *                  layer_stride bytes apart
 *   k_scale, v_scale  fp32 [layers][pages][heads], dense
 * Formats: QGKV_E4M3 (fp8 with 4 exponent and 3 mantissa bits, scales are
 * powers of two) and QGKV_INT8 (-127..127, scale = amax / 127).  The
 * attention takes any finite scales >= 0.
 *
 * A sequence is a row of a page table, int32 [batch][table_width] page
 * numbers of which the first ceil(len / page_tokens) count, and its length in
 * tokens (int32 lens[batch]).  Rows that belong to a sequence (new tokens,
 * queries) are listed by `starts`, int32 [batch + 1]: sequence b has rows
 * starts[b] .. starts[b+1]-1; a null `starts` gives every sequence one row.
 * refs, int32 [pages], counts the table rows that hold a page; a page is free
 * when its count is 0.
 *
 * Everything but the struct itself is caller-owned device memory; the
 * library allocates nothing per call.  Calls are asynchronous on `stream`.
 * Table, lens and starts are read on the device, so a call can be captured
 * in a graph and replayed with other lengths.
 *
 * Errors: as in qgemv.h.  What only the device can see is latched in the
 * status word that qg_device_status reports: QG_EBOUNDS for a page number
 * outside [0, pages), a length beyond the table or a parent outside the
 * batch (such pages are not read or written, their tokens count as masked),
 * QG_EPAGES when an operation found too few free pages.
 *
 * Workspace: qgkv_workspace_bytes() bytes of device memory, 256-byte aligned,
 * zeroed once before its first use and never written by anyone else; the
 * calls leave it ready for the next.  One workspace serves one stream: calls
 * that may overlap on the GPU need one each.
 */
#ifndef QGKV_H
#define QGKV_H

#include "qgemv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define QG_EPAGES (-8) /* device: too few free pages */

#define QGKV_E4M3 1
#define QGKV_INT8 2

#define QGKV_HND 0
#define QGKV_NHD 1

/* Types of queries, outputs, new tokens and logits. */
#define QGKV_F32 0
#define QGKV_F16 1
#define QGKV_BF16 2

/* Pairs of values that a rotation turns into one another. */
#define QGKV_INTERLEAVED 0 /* (0, 1), (2, 3), ... */
#define QGKV_HALVES 1      /* (0, R/2), (1, R/2 + 1), ... */

#define QGKV_MAX_BATCH 4096       /* sequences of one call */
#define QGKV_MAX_PAGES (1 << 20)  /* pages of one cache */
#define QGKV_MAX_BEAMS 64         /* beams of one request */
#define QGKV_MAX_KEEP 128         /* continuations selected per request */
#define QGKV_MAX_HISTORY ((1 << 20) - 1) /* tokens of a row's history */
#define QGKV_MAX_BIASES 2047      /* biases listed for a row */

typedef struct qgkv_cache {
    uint8_t* k;
    uint8_t* v;
    float* k_scale;
    float* v_scale;
    int64_t layers, pages;
    int64_t layer_stride, page_stride; /* bytes, multiples of 16, of k and of v */
    int heads;                         /* 1..1024 */
    int page_tokens;                   /* 16, 32, 64, 128 or 256 */
    int head_dim;                      /* a multiple of 16 up to 256 */
    int format;                        /* QGKV_E4M3 or QGKV_INT8 */
    int order;                         /* QGKV_HND or QGKV_NHD */
} qgkv_cache;

QG_API int64_t qgkv_workspace_bytes(void);

/* Quantise new tokens into the cache, behind the lens[b] tokens that sequence
 * b holds (lens itself is left to the caller).  k, v: `rows` rows of
 * [heads][head_dim] values of `type`; rows and heads are row_stride and
 * head_stride elements apart (multiples of 16 bytes), a head's values dense.
 * For each block the tokens enter, with a the largest finite magnitude of its
 * new values,
 *   need = the smallest power of two >= a / 448, at least 2^-126   (e4m3)
 *        = fl32(a / 127)                                          (int8)
 *        = 0 where a = 0;
 *   scale = max(need, the block's scale if it already holds tokens).
 * Where that raises the scale, the codes held are rescaled:
 *   code = round(fl32(code * fl32(old / scale))).
 * New codes are round(fl32(x / scale)) (to nearest even; 0 where scale = 0);
 * +-inf is stored as the largest code, NaN as NaN (e4m3) or 0 (int8).
 * The pages the tokens fall on must be held by no other sequence. */
QG_API int qgkv_append(const qgkv_cache* cache, int64_t layer, const void* k, const void* v, int type, int64_t rows,
                       int64_t row_stride, int64_t head_stride, const int32_t* table, int64_t table_width,
                       const int32_t* lens, const int32_t* starts, int batch, cudaStream_t stream);

/* qgkv_append of keys that are first turned to their positions, with the
 * queries of the same tokens.  Row i of sequence b has position p = lens[b] + i;
 * rope, fp32 [positions][turned], holds for each position turned / 2 cosines and
 * then as many sines.  Pair j (a, b) of a head's first `turned` values (a multiple
 * of 16 up to head_dim; `pairs` says which values are a pair) becomes
 *   fl32(fl32(a c) - fl32(b s)),  fl32(fl32(a s) + fl32(b c)),
 * c = rope[p][j], s = rope[p][turned / 2 + j]; the other values stay.  The turned
 * keys are quantised as they are, without a rounding to `type`.  k, v: as for
 * qgkv_append.  q: rows of [q_heads][head_dim] values, q_row and q_head elements
 * apart (multiples of 16 bytes), or null; q_out: [rows][q_heads][head_dim] of the
 * same type, dense, 16-byte aligned; it may be q where q is dense.  Rows that no
 * sequence has are left as they are.  Where p is outside the table (QG_EBOUNDS)
 * the token is not stored and its turned queries are NaN. */
QG_API int qgkv_append_rotary(const qgkv_cache* cache, int64_t layer, const void* q, const void* k, const void* v,
                              int type, int64_t rows, int q_heads, int64_t q_row, int64_t q_head, int64_t kv_row,
                              int64_t kv_head, const float* rope, int64_t positions, int turned, int pairs,
                              void* q_out, const int32_t* table, int64_t table_width, const int32_t* lens,
                              const int32_t* starts, int batch, cudaStream_t stream);

/* Attention of `rows` query rows over the cache.  Sequence b holds lens[b]
 * tokens, its own rows' tokens included; row i of its n rows sees the first
 * lens[b] - n + i + 1 of them (causal at the end of the sequence).  Query
 * head j reads cache head j / (q_heads / heads); rows * (q_heads / heads) is at
 * most 2^31 - 512.
 *   out = softmax(scale * q k^T) v,   lse = log(sum(exp(scale * q k^T)))
 * q: rows of [q_heads][head_dim] values of `type`, row_stride and head_stride
 * elements apart (multiples of 16 bytes).  out: [rows][q_heads][head_dim] of
 * the same type, dense, 16-byte aligned.  lse: fp32 [rows][q_heads] or null.
 * A row that sees nothing gives 0 and -inf.  Tokens a row does not see do not
 * reach it, whatever their codes.
 * Numerics: codes enter the tensor cores exactly (f16).  fp32 q enters as the
 * sum of two f16 parts (about 22 bits), 16-bit q exactly, both to 2^-39 of the
 * row's largest.  Weights (probability * scale of V) enter as two f16 parts, 22
 * bits, for bf16 q as one, 11 bits (below the output's rounding); and to within
 * 2^-34 of the row's largest weight, for bf16 q in calls of many rows a sequence
 * 2^-28: smaller ones are lost.
 * All sums are fp32.  Scores may have any size that fp32 holds; a row with one
 * beyond it is NaN.  Repeated calls give the same bits. */
QG_API int qgkv_attention(const qgkv_cache* cache, int64_t layer, const void* q, void* out, float* lse, int type,
                          int64_t rows, int q_heads, int64_t row_stride, int64_t head_stride, const int32_t* table,
                          int64_t table_width, const int32_t* lens, const int32_t* starts, int batch, float scale,
                          void* workspace, int64_t workspace_bytes, cudaStream_t stream);

/* What sequences have in common, for qgkv_attention_shared.  Sequences
 * groups[g] .. groups[g+1]-1 (int32 [ngroups + 1], rising, within the batch) are
 * group g.  The tokens that a group shares are those of the first columns in
 * which all its sequences hold the same pages, as far as every row of it sees
 * them, in whole pages; 0 where fewer than two of its sequences have rows (those
 * without rows take no part).  table, lens, starts and rows: as for the attention.
 * plan, int32 [4 * ngroups + batch], gets for each group (first row, rows, tokens
 * shared, first sequence) and then for each sequence the tokens that it shares.
 * One plan serves all layers of a step.  Borders that do not rise or leave the
 * batch: nothing is shared (QG_EBOUNDS).
 * A group shares what all its sequences with rows have in common: a short one, or
 * one that has left the prompt, sets it for all.  Sequences that share nothing are
 * best left before the first border or behind the last: as groups of their own, or
 * spread among others, they count against sharing (qgkv_attention_shared). */
QG_API int qgkv_share(int64_t pages, int page_tokens, const int32_t* table, int64_t table_width, const int32_t* lens,
                      const int32_t* starts, int64_t rows, int batch, const int32_t* groups, int ngroups,
                      int32_t* plan, cudaStream_t stream);

/* qgkv_attention of a batch whose groups share tokens: the pages shared are read
 * once for all rows of a group, and the results joined with those of the tokens
 * behind them.  plan: what qgkv_share wrote for the same table, lens and starts.
 * QG_EBOUNDS reports entries out of range, groups that begin among the rows of the
 * one before, and sequences that share tokens without a group of their rows that
 * shares as many; the rows of such groups and sequences are not valid.  That a
 * group's sequences still hold the same pages is not looked at again.  Results are
 * those of qgkv_attention to within its numerics, but for what small weights and scales of V keep among the tokens
 * shared: bf16 q to within 2^-28 of the row's largest weight, other types 2^-39; full
 * precision for scales of V of 2^-80 to 2^90 (qgkv_append writes none outside for
 * values of 2^-70 to 2^97).
 * The sizes of a call alone decide whether it shares; where it does not, each
 * sequence reads all its tokens itself and the plan is not read.  It does not where
 * the columns of all sequences but one come to less than 16 MB of pages, where the
 * batch has fewer than four sequences for each of ngroups (a group of one counts as
 * a group), where sequences have many rows, or where there are more results to join
 * than the workspace holds. */
QG_API int qgkv_attention_shared(const qgkv_cache* cache, int64_t layer, const void* q, void* out, float* lse, int type,
                                 int64_t rows, int q_heads, int64_t row_stride, int64_t head_stride,
                                 const int32_t* table, int64_t table_width, const int32_t* lens,
                                 const int32_t* starts, int batch, const int32_t* plan, int ngroups, float scale,
                                 void* workspace, int64_t workspace_bytes, cudaStream_t stream);

/* Copy pages src[i] to dst[i], 0 <= i < n, codes and scales of every layer.
 * n is *count (device) where count is not null, at most `most` either way.
 * No destination may be a source or another destination. */
QG_API int qgkv_copy_pages(const qgkv_cache* cache, const int32_t* src, const int32_t* dst, const int32_t* count,
                           int64_t most, cudaStream_t stream);

/* Replace the sequences of `table` by children: new sequence i continues old
 * sequence parent[i] (a beam search's reordering).  Whole pages are shared by
 * reference; where several new sequences end in the same partly filled page,
 * or a sequence outside the table holds it too, each but one of them (all, in
 * the second case) gets a copy of its own, on the lowest free pages in the
 * order of the sequences, after the pages that no child keeps are free.
 * table2 [batch2][table_width] (-1 behind the last page), lens2 [batch2] and
 * refs2 [pages] are written and must not overlap the inputs; the page copies
 * are made in the cache.  Where no page is free the entry is -1 (QG_EPAGES). */
QG_API int qgkv_fork(const qgkv_cache* cache, const int32_t* table, int64_t table_width, const int32_t* lens,
                     int batch, const int32_t* parent, int batch2, const int32_t* refs, int32_t* table2,
                     int32_t* lens2, int32_t* refs2, void* workspace, int64_t workspace_bytes, cudaStream_t stream);

/* Free the sequences that `drop` marks (uint8 [batch], null for none) and
 * move the pages still held to the lowest page numbers: with n pages held,
 * the i-th held page from n on goes to the i-th free page below n.  table2,
 * lens2, refs2 as for qgkv_fork; *count gets n. */
QG_API int qgkv_compact(const qgkv_cache* cache, const int32_t* table, int64_t table_width, const int32_t* lens,
                        int batch, const uint8_t* drop, const int32_t* refs, int32_t* table2, int32_t* lens2,
                        int32_t* refs2, int32_t* count, void* workspace, int64_t workspace_bytes,
                        cudaStream_t stream);

/* Give sequence b the pages that lens[b] + add[b] tokens need beyond those of
 * lens[b] (add null: one token each), the lowest free ones in the order of
 * the sequences; table and refs are updated, lens is left to the caller, who
 * raises it once the tokens are stored: until then a second call gives other
 * pages for the same places, and a fork, compaction or free passes these by; the
 * pages of before stay held and no table has them.  A
 * sequence for which too few are left gets none (QG_EPAGES). */
QG_API int qgkv_reserve(int64_t pages, int page_tokens, int32_t* table, int64_t table_width, const int32_t* lens,
                        const int32_t* add, int batch, int32_t* refs, void* workspace, int64_t workspace_bytes,
                        cudaStream_t stream);

/* Free the sequences that `drop` marks (null: all): their pages' counts go
 * down, their table rows become -1 and their lengths 0. */
QG_API int qgkv_free(int64_t pages, int page_tokens, int32_t* table, int64_t table_width, int32_t* lens,
                     const uint8_t* drop, int batch, int32_t* refs, cudaStream_t stream);

/* The `keep` best continuations of each request: over its beams' rows of
 * `logits` ([requests * beams] rows of `vocab` values, row_stride elements
 * apart), score = cum[beam] + logit - log(sum(exp(row))), highest first, of
 * equal scores the lowest (beam, token).  keep <= beams * vocab.  scores
 * fp32, tokens int32 and parents int32 (the row number, request * beams +
 * beam, as qgkv_fork takes it), each [requests][keep].  A row that holds NaN
 * or +inf, or nothing but -inf, or whose cum is NaN or +inf, scores -inf throughout.
 * QG_ESCRATCH where requests * beams * (8 * keep + 16) bytes of partial results
 * exceed the workspace's room for them (42 MB). */
QG_API int qgbeam_select(const void* logits, int type, const float* cum, int requests, int beams, int64_t vocab,
                         int64_t row_stride, int keep, float* scores, int32_t* tokens, int32_t* parents,
                         void* workspace, int64_t workspace_bytes, cudaStream_t stream);

/* Adjust `rows` rows of `vocab` logits (row_stride elements apart) before a
 * selection.  For token t of row r, with its logit x in fp32 and every operation
 * rounded to fp32, in this order and each where its argument is not null:
 *   history   int32 [rows][width], the row's first lens[r] tokens, of which the
 *             first prompt_lens[r] (null: none; below 0 none, beyond lens[r] all)
 *             were given and the others produced:
 *     x = x > 0 ? x / repetition[r] : x * repetition[r]  if t is in it;
 *     x = x - frequency[r] * n;  x = x - presence[r]     if t was produced n > 0 times;
 *   bias      x = x + bias[r][i] for the last i with bias_tokens[r][i] = t
 *             (int32 and fp32 [rows][biases]);
 *   temperature  x = x / temperature[r];
 *   mask      x = -inf if bit t % 32 of word t / 32 of the row's mask is 0.  mask:
 *             `masks` rows of `mask_words` words, at least ceil(vocab / 32);
 *             mask_rows, int32 [rows], names the mask of each row, -1 for none
 *             (null: row r has mask r, and masks is at least rows).
 * Tokens outside [0, vocab) in history and bias_tokens are passed over.  out: of
 * `type` or fp32, rows out_stride elements apart; it may be `logits` itself (of
 * the same type and stride), and then, without a temperature, only the logits that
 * change are touched.  A lens[r] outside [0, width] is cut to it, and a mask
 * number outside [-1, masks) counts as -1 (QG_EBOUNDS). */
QG_API int qglogits_adjust(const void* logits, int type, int64_t rows, int64_t vocab, int64_t row_stride, void* out,
                           int out_type, int64_t out_stride, const int32_t* history, int64_t width,
                           const int32_t* lens, const int32_t* prompt_lens, const float* repetition,
                           const float* presence, const float* frequency, const int32_t* bias_tokens,
                           const float* bias, int biases, const float* temperature, const uint32_t* mask,
                           int64_t mask_words, int masks, const int32_t* mask_rows, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QGKV_H */
