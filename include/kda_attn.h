/*
 * kda_attn.h: the softmax-attention side of libkda.so.
 *
 * A model that uses the KDA recurrence in most of its attention blocks keeps
 * softmax attention, and with it a growing cache of keys and values, in the
 * others.  These entry points serve those blocks: attention over packed
 * prompts, an 8-bit paged key/value cache, attention over that cache for
 * single tokens and draft windows, and the eviction of pages that received
 * little attention.  They follow the conventions of kda.h (device pointers,
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

#ifdef __cplusplus
}
#endif

#endif /* KDA_ATTN_H_ */
