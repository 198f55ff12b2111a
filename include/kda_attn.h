/*
 * kda_attn.h: the softmax-attention side of libkda.so.
 *
 * A model that uses the KDA recurrence in most of its attention blocks keeps
 * softmax attention, and with it a growing cache of keys and values, in the
 * others.  These entry points serve those blocks: attention over packed
 * prompts, an 8-bit paged key/value cache, attention over that cache for
 * single tokens and draft windows (of whole sequences, of batches that share
 * prefixes, or over the pages that a cheap score selects), the eviction of
 * pages that received little attention, and the norm and rotation of queries
 * and keys in front of it all.  They follow the conventions of kda.h (device pointers,
 * 16-byte alignment, asynchronous on `stream`, statuses, *err_flag, no
 * allocation, no atomics on data: the same inputs give the same bits), and
 * like the rest of the library they have no gradients.
 *
 * Grouped heads: Hq = q_heads, Hkv = kv_heads, G = Hq / Hkv; query head h
 * reads kv head h / G.
 *
 * The cache.  Pages of 64 positions, named per sequence by an int32 block
 * table [batch][max_pages]; position i of sequence n lives in page
 * block_table[n][i / 64], at place i % 64.
 *   k_pages  e4m3  [num_pages][Hkv][64][d]   a row per position
 *   v_pages  e4m3  [num_pages][Hkv][d][64]   a row per channel: the product
 *            with the attention weights contracts over positions
 *   k_scale, v_scale  f32 [num_pages][Hkv]   one scale per page and head, a
 *            power of two; a byte b stands for scale * e4m3(b)
 * Table entries past a sequence's last page are never read.
 */
#ifndef KDA_ATTN_H_
#define KDA_ATTN_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_PAGE_TOKENS 64

/* Further bits OR-ed into *err_flag. */
enum {
    KDA_DEVERR_PAGE = 256, /* a block-table entry outside 0..num_pages-1, or a
                              sequence longer than its table row             */
    KDA_DEVERR_SCALE = 512 /* a scale that is not a power of two in
                              2^-126..2^126 (a k_scale that is read: not a
                              positive number)                               */
};

typedef struct kda_attn_dims {
    int32_t q_heads;  /* Hq, a multiple of kv_heads, at most 128 per kv head */
    int32_t kv_heads; /* Hkv >= 1                                            */
    int32_t head_dim; /* d in {32, 64, 128}                                  */
    int32_t dtype;    /* kda_dtype of q, k, v and of the outputs             */
    float scale;      /* score scale; <= 0 selects d^-1/2                    */
} kda_attn_dims;

typedef struct kda_kv_cache {
    void *k_pages;
    void *v_pages;
    float *k_scale;
    float *v_scale;
    int64_t num_pages; /* num_pages * Hkv * max(64, d) at most 2^31 - 1 */
} kda_kv_cache;

/*
 * kda_attn_prefill: causal attention over num_seqs packed prompts.  For token
 * i of a sequence and query head h:
 *   o_i   = sum_{j <= i} p_ij v_j / sum_{j <= i} p_ij,
 *   p_ij  = exp(scale q_i . k_j),     lse_i = log sum_{j <= i} p_ij
 * over the tokens j of the same sequence.  The values, infinities and NaN of
 * other sequences and of later tokens have no influence.
 *
 *   cu_seqlens i32 [num_seqs + 1]; sequence s is tokens cu[s]..cu[s+1]-1 and
 *              may be empty.  Offsets that decrease or leave 0..total_tokens
 *              set KDA_DEVERR_SEQLENS; the outputs of the call are then
 *              unspecified.  Tokens of no sequence are not written.
 *   q          dtype [total_tokens][Hq][d], tokens q_stride elements apart
 *   k, v       dtype [total_tokens][Hkv][d], tokens k_stride, v_stride apart
 *              (a multiple of 16 bytes, at least heads * d: the slices of a
 *              fused projection are read in place)
 *   out        dtype [total_tokens][Hq][d], contiguous
 *   lse        f32   [total_tokens][Hq], natural log; may be NULL
 */
KDA_API int kda_attn_prefill(const kda_attn_dims *dims, int32_t num_seqs, const int32_t *cu_seqlens,
                             int64_t total_tokens, const void *q, int64_t q_stride, const void *k,
                             int64_t k_stride, const void *v, int64_t v_stride, void *out, float *lse,
                             int32_t *err_flag, void *stream);

/*
 * kda_cache_append: quantises packed new tokens into the cache.  Sequence s
 * holds start_pos[s] positions; its tokens cu[s]..cu[s+1]-1 take the next
 * ones.  Per (page written, head), for keys and for values apart:
 *   need = the smallest power of two >= 2^-126 with amax <= 448 need, amax the
 *          largest finite magnitude among the page's new rows
 *   s'   = need if the page held no earlier position, else max(scale, need)
 *   new rows:      e4m3(clamp(x / s', -448, 448)), to nearest even; NaN stays
 *   earlier rows:  when s' > scale, e4m3(value * scale / s'): exact but for
 *                  the smallest (subnormal) values, since both are powers of two
 * Places past the sequence's new end are not written.  A page is written for
 * one sequence only in a call (a page shared between sequences is full).
 *
 *   cu_seqlens  as in kda_attn_prefill; with offsets that set
 *               KDA_DEVERR_SEQLENS some of the call's tokens are written, others not
 *   k, v        dtype [total_tokens][Hkv][d], tokens k_stride, v_stride apart
 *   start_pos   i32 [num_seqs], >= 0 (a negative one skips the sequence)
 *   block_table i32 [num_seqs][max_pages]
 * A page outside the cache, or a row too short for the new end, sets
 * KDA_DEVERR_PAGE and that page's tokens are not written; a scale of earlier
 * positions that is no such power of two sets KDA_DEVERR_SCALE, and that page's
 * keys (or values) of that head are not written.
 */
KDA_API int kda_cache_append(const kda_attn_dims *dims, const kda_kv_cache *cache, int32_t num_seqs,
                             const int32_t *cu_seqlens, int64_t total_tokens, const void *k,
                             int64_t k_stride, const void *v, int64_t v_stride, const int32_t *start_pos,
                             const int32_t *block_table, int32_t max_pages, int32_t *err_flag,
                             void *stream);

/*
 * kda_attn_decode: attention of the last draft_len (1..16) tokens of each
 * sequence over the cache, which holds them already: token t of the window
 * sees positions j < seq_lens[n] - draft_len + 1 + t.  A token that sees
 * nothing gets output 0 and lse -inf (seq_lens[n] <= 0: padding).
 *
 *   q           dtype [batch][draft_len][Hq][d], tokens q_stride apart
 *   seq_lens    i32 [batch], the window included
 *   block_table i32 [batch][max_pages]; an entry outside the cache sets
 *               KDA_DEVERR_PAGE and its positions count as unseen, as do
 *               those of a page and head whose scales set
 *               KDA_DEVERR_SCALE; a sequence longer than its row sets
 *               KDA_DEVERR_PAGE and is taken to end with the row
 *   out         dtype [batch][draft_len][Hq][d]
 *   lse         f32 [batch][draft_len][Hq], natural log; may be NULL
 *   weight_out  f32 [batch][max_pages]; may be NULL.  Written with
 *               weight_in[n][p] (0 where weight_in is NULL) plus the attention
 *               weight that the window's rows of all heads gave to the
 *               positions of page p; may be weight_in itself
 *   workspace   kda_attn_decode_workspace_bytes(...) bytes, 256-byte aligned,
 *               owned by the caller, contents undefined before and after
 * The batch's pages are shared out evenly over the GPU, so where a sequence is
 * cut, and with it the last bits of its results, depends on the whole batch.
 */
KDA_API int kda_attn_decode(const kda_attn_dims *dims, const kda_kv_cache *cache, int32_t batch,
                            int32_t draft_len, const void *q, int64_t q_stride, const int32_t *seq_lens,
                            const int32_t *block_table, int32_t max_pages, void *out, float *lse,
                            const float *weight_in, float *weight_out, void *workspace,
                            size_t workspace_bytes, int32_t *err_flag, void *stream);

/* Workspace of kda_attn_decode (with_weight: weight_out is given); 0 for invalid arguments. */
KDA_API size_t kda_attn_decode_workspace_bytes(const kda_attn_dims *dims, int32_t batch,
                                               int32_t draft_len, int32_t max_pages,
                                               int32_t with_weight);

/*
 * kda_cache_evict: drops the lightest pages of sequences that hold more than
 * `budget` pages.  A sequence of P = ceil(seq_lens / 64) pages keeps its first
 * `sink` and last `recent` (>= 1) pages and, of the others, the heaviest by
 * weight until `budget` (>= sink + recent) are left; of equal weights the
 * lower index stays, and a NaN weighs least.  The rows close up in order; the
 * keys keep the positions they were embedded with.
 *
 *   seq_lens, block_table, weight   i32 [batch], i32 and f32 [batch][max_pages]
 *   seq_lens_out      seq_lens less 64 per dropped page
 *   block_table_out   the kept entries (those past page P too) in order, then
 *   weight_out        -1 and 0 in the places that became free
 *   freed             i32 [batch][max_pages]: the dropped pages in order, then -1
 *   freed_count       i32 [batch]
 * Each *_out may be its input.  A sequence longer than its row sets
 * KDA_DEVERR_PAGE and is copied as it is.
 */
KDA_API int kda_cache_evict(int32_t batch, int32_t max_pages, int32_t budget, int32_t sink, int32_t recent,
                            const int32_t *seq_lens, const int32_t *block_table, const float *weight,
                            int32_t *seq_lens_out, int32_t *block_table_out, float *weight_out,
                            int32_t *freed, int32_t *freed_count, int32_t *err_flag, void *stream);

/*
 * kda_norm_rotate: norm of query and key heads and the rotation by their
 * positions.  Per token and head, x a row of d channels:
 *   y = x / sqrt(sum_c x_c^2 / d + eps) * weight     (y = x where weight is NULL)
 *   (y_a, y_b) -> factor (y_a cos t - y_b sin t, y_a sin t + y_b cos t)
 * for the pairs i < rotary_dim / 2 of the first rotary_dim channels:
 * (a, b) = (i, i + rotary_dim / 2), or (2 i, 2 i + 1) where interleaved; the
 * other channels are y.  t = 2 pi positions[token] turns[i] / 2^64: a table of
 * turns per position in units of 2^-64, modulo one, so that angles are exact to
 * 2^-24 at every position.  fp32 throughout, rounded once (a row whose sum of
 * squares leaves fp32's range gives 0).
 *
 *   q, k         dtype [total_tokens][Hq or Hkv][d], tokens q_stride, k_stride apart
 *   q_out, k_out the same, tokens q_out_stride, k_out_stride apart; each may be
 *                its input (with its stride)
 *   positions    i32 [total_tokens], any value; total_tokens < 2^31 - 2^14
 *   turns        u64 [rotary_dim / 2]
 *   q_weight, k_weight  f32 [d], 16-byte aligned; NULL: no norm
 * dims->scale is not used.  rotary_dim even, 0..d (0: norm alone).
 */
KDA_API int kda_norm_rotate(const kda_attn_dims *dims, int64_t total_tokens, const void *q, int64_t q_stride,
                            const void *k, int64_t k_stride, const int32_t *positions, const uint64_t *turns,
                            int32_t rotary_dim, int32_t interleaved, float factor, const float *q_weight,
                            const float *k_weight, float eps, void *q_out, int64_t q_out_stride, void *k_out,
                            int64_t k_out_stride, void *stream);

/*
 * kda_attn_decode_shared: kda_attn_decode for sequences that share prefixes.
 * The sequences group_start[g]..group_start[g+1]-1 are a group: the first
 * shared_pages[g] entries of their block table rows name the same pages (as far
 * as a sequence goes), which are read once for all of them, from the row of a
 * sequence that goes as far as any of those that are computed together.
 * The results are those of kda_attn_decode (the shared pages are full; a
 * sequence that ends inside them sees them as far as it goes).  In bf16, where
 * many rows meet a page, queries are multiplied as two 8-bit terms, and what
 * these leave is added where it could come to more than 2^-11 of a score (in
 * units of log 2), which is the weights' own rounding.  Sequences of no group
 * share nothing.
 *
 * "Once" is for up to 256 query rows of a kv head (a group's tokens times G); in
 * fp32 and at d = 32 for up to 64.  Where groups have up to 8 rows in the mean
 * (of ceil(batch / num_groups) sequences), it is for 8, which is quicker, and
 * groups of more than 32 rows are read apart where the block table is long; in
 * fp32 and at d = 32 a mean of up to 16 or 32 rows is for as many.  Empty groups,
 * groups of one and sequences of no group count in the mean: that can cost time,
 * never results.
 *
 *   group_start  i32 [num_groups + 1], not decreasing, in 0..batch; offsets
 *                that are not set KDA_DEVERR_SEQLENS, and the outputs of the
 *                call are then unspecified
 *   shared_pages i32 [num_groups]; one outside 0..max_pages sets
 *                KDA_DEVERR_PAGE and is taken as the nearer of these
 *   workspace    kda_attn_decode_shared_workspace_bytes(...) bytes, 256-byte
 *                aligned, contents undefined before and after
 * The rest as in kda_attn_decode; page weights are not offered (a shared page
 * is no sequence's to evict).
 */
KDA_API int kda_attn_decode_shared(const kda_attn_dims *dims, const kda_kv_cache *cache, int32_t batch,
                                   int32_t draft_len, const void *q, int64_t q_stride, const int32_t *seq_lens,
                                   const int32_t *block_table, int32_t max_pages, int32_t num_groups,
                                   const int32_t *group_start, const int32_t *shared_pages, void *out, float *lse,
                                   void *workspace, size_t workspace_bytes, int32_t *err_flag, void *stream);

/*
 * Workspace of kda_attn_decode_shared; 0 for invalid arguments, and for calls of
 * more than 2^31 - 1 query rows, or of nearly 2^32 groups times kv heads.
 */
KDA_API size_t kda_attn_decode_shared_workspace_bytes(const kda_attn_dims *dims, int32_t batch, int32_t draft_len,
                                                      int32_t max_pages, int32_t num_groups);

/*
 * Summaries of the cached keys, for a selection of pages: per page, kv head and
 * channel the largest and the smallest key, in whole numbers of one unit.
 *   bounds  i8  [num_pages][Hkv][2][d]  largest, smallest, in -127..127
 *   unit    f32 [num_pages][Hkv]        a power of two
 */
typedef struct kda_key_summary {
    int8_t *bounds;
    float *unit;
} kda_key_summary;

/*
 * kda_cache_summarise: renews the summaries of the pages that a kda_cache_append
 * with the same arguments wrote, from the positions that they hold now.  Per
 * page and head, over the page's positions before the sequence's new end:
 *   unit     the smallest power of two >= 2^-126 with |key| <= 127 unit
 *   bounds   max and min of the channel's keys / unit, to the nearest whole
 *            number, ties to even; a NaN key is passed over (0 for NaN alone)
 * Errors as in kda_cache_append; a k_scale that is not a power of two, or a unit
 * above 2^126, sets KDA_DEVERR_SCALE and that page and head is left alone.
 */
KDA_API int kda_cache_summarise(const kda_attn_dims *dims, const kda_kv_cache *cache, const kda_key_summary *summary,
                                int32_t num_seqs, const int32_t *cu_seqlens, int64_t total_tokens,
                                const int32_t *start_pos, const int32_t *block_table, int32_t max_pages,
                                int32_t *err_flag, void *stream);

/*
 * kda_cache_select: the pages of each sequence and kv head that promise the
 * most.  A sequence of P = ceil(seq_lens / 64) pages keeps them all where
 * P <= budget; else its first `sink`, its last `recent` and, of the others, the
 * best by score until there are `budget`; of equal scores the lower index.  With
 *   u_r   the smallest power of two >= 2^-126 with |q_r| <= 127 u_r (finite elements)
 *   x_rc  q_rc / u_r to the nearest whole number, ties to even, within
 *         -127..127; 0 for NaN
 *   score(page) = max_r u_r unit sum_c max(x_rc hi_c, x_rc lo_c)
 * over the rows r of the window's tokens and the kv head's query heads (whole
 * numbers times powers of two: the order of the sum does not matter).
 *
 *   q            as in kda_attn_decode
 *   seq_lens, block_table  as in kda_attn_decode; a page outside the cache sets
 *                KDA_DEVERR_PAGE, a unit that is not a power of two in
 *                2^-126..2^126 KDA_DEVERR_SCALE; either scores below all others
 *   budget       >= sink + recent, sink >= 0, recent >= 1 (>= 2 for draft_len
 *                > 1: the pages that the window can lie in)
 *   seq_lens_out     i32 [batch]: seq_lens less 64 per page left out
 *   block_table_out  i32 [batch][Hkv][budget]: the selected entries in order, then -1
 *   index_out        i32 [batch][Hkv][budget]: their places in the row, then -1
 *   workspace    kda_cache_select_workspace_bytes(...) bytes, 256-byte aligned
 */
KDA_API int kda_cache_select(const kda_attn_dims *dims, const kda_key_summary *summary, int64_t num_pages,
                             int32_t batch, int32_t draft_len, const void *q, int64_t q_stride,
                             const int32_t *seq_lens, const int32_t *block_table, int32_t max_pages, int32_t budget,
                             int32_t sink, int32_t recent, int32_t *seq_lens_out, int32_t *block_table_out,
                             int32_t *index_out, void *workspace, size_t workspace_bytes, int32_t *err_flag,
                             void *stream);

/* Workspace of kda_cache_select; 0 for invalid arguments. */
KDA_API size_t kda_cache_select_workspace_bytes(const kda_attn_dims *dims, int32_t batch, int32_t max_pages);

/*
 * kda_attn_decode_selected: kda_attn_decode with a block table of its own for
 * every kv head, i32 [batch][Hkv][max_pages] (as kda_cache_select leaves it; the
 * window's positions are the last ones).  Workspace:
 * kda_attn_decode_workspace_bytes for the same sizes, without weights.
 */
KDA_API int kda_attn_decode_selected(const kda_attn_dims *dims, const kda_kv_cache *cache, int32_t batch,
                                     int32_t draft_len, const void *q, int64_t q_stride, const int32_t *seq_lens,
                                     const int32_t *block_table, int32_t max_pages, void *out, float *lse,
                                     void *workspace, size_t workspace_bytes, int32_t *err_flag, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_ATTN_H_ */
