// C ABI of the attention operators: argument validation and dispatch, in the
// manner of kda_api.cu (a host-detectable error returns a negative status and
// launches nothing; otherwise the kernels are enqueued without synchronising).
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "kda_attn.h"
#include "kda_attn_internal.h"

namespace {

constexpr int64_t kMaxI32 = 0x7fffffff;

bool ok16(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (p == nullptr || (reinterpret_cast<uintptr_t>(p) & 15u) != 0) return false;
    return true;
}

bool ok4(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (p == nullptr || (reinterpret_cast<uintptr_t>(p) & 3u) != 0) return false;
    return true;
}

int check_dims(const kda_attn_dims *d) {
    if (d == nullptr || d->q_heads < 1 || d->kv_heads < 1 || d->q_heads % d->kv_heads != 0)
        return KDA_ERR_INVALID_ARG;
    if (d->dtype != KDA_DT_F32 && d->dtype != KDA_DT_BF16) return KDA_ERR_UNSUPPORTED;
    if (d->head_dim != 32 && d->head_dim != 64 && d->head_dim != 128) return KDA_ERR_UNSUPPORTED;
    if (d->q_heads / d->kv_heads > 128 || d->q_heads > 65535) return KDA_ERR_UNSUPPORTED;
    if (isnan(d->scale) || isinf(d->scale)) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

float resolve_scale(const kda_attn_dims *d) {
    return d->scale > 0.f ? d->scale : 1.0f / sqrtf((float)d->head_dim);
}

// Token strides: rows that do not overlap, each starting on 16 bytes.
bool stride_ok(const kda_attn_dims *d, int64_t stride, int64_t heads) {
    const int64_t esz = d->dtype == KDA_DT_BF16 ? 2 : 4;
    return stride >= heads * d->head_dim && stride <= kMaxI32 && (stride * esz) % 16 == 0;
}

int check_cache(const kda_attn_dims *d, const kda_kv_cache *c) {
    if (c == nullptr || c->num_pages < 0) return KDA_ERR_INVALID_ARG;
    const int64_t rows = d->head_dim > KDA_PAGE_TOKENS ? d->head_dim : KDA_PAGE_TOKENS;
    if (c->num_pages > kMaxI32 / rows / d->kv_heads) return KDA_ERR_INVALID_ARG;
    if (c->num_pages > 0 && (!ok16({c->k_pages, c->v_pages}) || !ok4({c->k_scale, c->v_scale})))
        return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

int from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return KDA_OK;
    if (e == cudaErrorNotSupported) return KDA_ERR_UNSUPPORTED;
    return KDA_ERR_CUDA;
}

}  // namespace

extern "C" {

int kda_attn_prefill(const kda_attn_dims *dims, int32_t num_seqs, const int32_t *cu_seqlens, int64_t total_tokens,
                     const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                     int64_t v_stride, void *out, float *lse, int32_t *err_flag, void *stream) {
    if (const int st = check_dims(dims)) return st;
    if (num_seqs < 0 || total_tokens < 0 || total_tokens > kMaxI32) return KDA_ERR_INVALID_ARG;
    if (num_seqs == 0 || total_tokens == 0) return KDA_OK;
    if (!ok4({cu_seqlens}) || !ok16({q, k, v, out})) return KDA_ERR_INVALID_ARG;
    if (lse != nullptr && !ok4({lse})) return KDA_ERR_INVALID_ARG;
    if (!stride_ok(dims, q_stride, dims->q_heads) || !stride_ok(dims, k_stride, dims->kv_heads) ||
        !stride_ok(dims, v_stride, dims->kv_heads))
        return KDA_ERR_INVALID_ARG;
    kda::AttnPrefillParams p{};
    p.cu_seqlens = cu_seqlens; p.total_tokens = total_tokens;
    p.q = q; p.k = k; p.v = v;
    p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride;
    p.out = out; p.lse = lse; p.err_flag = err_flag;
    p.num_seqs = num_seqs; p.Hq = dims->q_heads; p.Hkv = dims->kv_heads; p.G = dims->q_heads / dims->kv_heads;
    p.scale = resolve_scale(dims);
    return from_cuda(kda::launch_attn_prefill(p, dims->head_dim, dims->dtype, (cudaStream_t)stream));
}

int kda_cache_append(const kda_attn_dims *dims, const kda_kv_cache *cache, int32_t num_seqs,
                     const int32_t *cu_seqlens, int64_t total_tokens, const void *k, int64_t k_stride,
                     const void *v, int64_t v_stride, const int32_t *start_pos, const int32_t *block_table,
                     int32_t max_pages, int32_t *err_flag, void *stream) {
    if (const int st = check_dims(dims)) return st;
    if (const int st = check_cache(dims, cache)) return st;
    if (num_seqs < 0 || total_tokens < 0 || total_tokens > kMaxI32 || max_pages < 0 ||
        max_pages > kMaxI32 / KDA_PAGE_TOKENS || dims->kv_heads > 65535)
        return KDA_ERR_INVALID_ARG;
    if (num_seqs == 0 || total_tokens == 0) return KDA_OK;
    if (!ok4({cu_seqlens, start_pos}) || !ok16({k, v})) return KDA_ERR_INVALID_ARG;
    if (max_pages > 0 && !ok4({block_table})) return KDA_ERR_INVALID_ARG;
    if (!stride_ok(dims, k_stride, dims->kv_heads) || !stride_ok(dims, v_stride, dims->kv_heads))
        return KDA_ERR_INVALID_ARG;
    kda::CacheAppendParams p{};
    p.k_pages = static_cast<unsigned char *>(cache->k_pages);
    p.v_pages = static_cast<unsigned char *>(cache->v_pages);
    p.k_scale = cache->k_scale; p.v_scale = cache->v_scale; p.num_pages = cache->num_pages;
    p.cu_seqlens = cu_seqlens; p.total_tokens = total_tokens;
    p.k = k; p.v = v; p.k_stride = k_stride; p.v_stride = v_stride;
    p.start_pos = start_pos; p.block_table = block_table; p.err_flag = err_flag;
    p.num_seqs = num_seqs; p.Hkv = dims->kv_heads; p.max_pages = max_pages;
    return from_cuda(kda::launch_cache_append(p, dims->head_dim, dims->dtype, (cudaStream_t)stream));
}

size_t kda_attn_decode_workspace_bytes(const kda_attn_dims *dims, int32_t batch, int32_t draft_len,
                                       int32_t max_pages, int32_t with_weight) {
    if (check_dims(dims) != KDA_OK || batch < 0 || draft_len < 1 || draft_len > 16 || max_pages < 0 ||
        max_pages > kMaxI32 / KDA_PAGE_TOKENS)
        return 0;
    return kda::attn_decode_workspace_bytes(dims->q_heads, dims->kv_heads, dims->head_dim, dims->dtype, batch,
                                            draft_len, max_pages, with_weight != 0);
}

int kda_attn_decode(const kda_attn_dims *dims, const kda_kv_cache *cache, int32_t batch, int32_t draft_len,
                    const void *q, int64_t q_stride, const int32_t *seq_lens, const int32_t *block_table,
                    int32_t max_pages, void *out, float *lse, const float *weight_in, float *weight_out,
                    void *workspace, size_t workspace_bytes, int32_t *err_flag, void *stream) {
    if (const int st = check_dims(dims)) return st;
    if (const int st = check_cache(dims, cache)) return st;
    if (batch < 0 || draft_len < 1 || draft_len > 16 || max_pages < 0 || max_pages > kMaxI32 / KDA_PAGE_TOKENS)
        return KDA_ERR_INVALID_ARG;
    if (batch == 0) return KDA_OK;
    if (!ok16({q, out}) || !ok4({seq_lens}) || (max_pages > 0 && !ok4({block_table}))) return KDA_ERR_INVALID_ARG;
    if (!stride_ok(dims, q_stride, dims->q_heads)) return KDA_ERR_INVALID_ARG;
    if ((lse != nullptr && !ok4({lse})) || (weight_in != nullptr && !ok4({weight_in})) ||
        (weight_out != nullptr && !ok4({weight_out})))
        return KDA_ERR_INVALID_ARG;
    if (weight_in != nullptr && weight_out == nullptr) return KDA_ERR_INVALID_ARG;
    const size_t need = kda::attn_decode_workspace_bytes(dims->q_heads, dims->kv_heads, dims->head_dim, dims->dtype,
                                                         batch, draft_len, max_pages, weight_out != nullptr);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need ||
                     (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0))
        return KDA_ERR_WORKSPACE;
    kda::AttnDecodeParams p{};
    p.k_pages = static_cast<const unsigned char *>(cache->k_pages);
    p.v_pages = static_cast<const unsigned char *>(cache->v_pages);
    p.k_scale = cache->k_scale; p.v_scale = cache->v_scale; p.num_pages = cache->num_pages;
    p.q = q; p.q_stride = q_stride; p.seq_lens = seq_lens; p.block_table = block_table;
    p.out = out; p.lse = lse; p.weight_in = weight_in; p.weight_out = weight_out;
    p.workspace = workspace; p.err_flag = err_flag;
    p.batch = batch; p.D = draft_len; p.Hq = dims->q_heads; p.Hkv = dims->kv_heads;
    p.G = dims->q_heads / dims->kv_heads; p.max_pages = max_pages;
    p.scale = resolve_scale(dims);
    return from_cuda(kda::launch_attn_decode(p, dims->head_dim, dims->dtype, (cudaStream_t)stream));
}

int kda_cache_evict(int32_t batch, int32_t max_pages, int32_t budget, int32_t sink, int32_t recent,
                    const int32_t *seq_lens, const int32_t *block_table, const float *weight,
                    int32_t *seq_lens_out, int32_t *block_table_out, float *weight_out, int32_t *freed,
                    int32_t *freed_count, int32_t *err_flag, void *stream) {
    if (batch < 0 || max_pages < 0 || max_pages > kMaxI32 / KDA_PAGE_TOKENS || sink < 0 || recent < 1 ||
        sink > kMaxI32 - recent || budget < sink + recent)
        return KDA_ERR_INVALID_ARG;
    if (batch == 0) return KDA_OK;
    if (!ok4({seq_lens, seq_lens_out, freed_count})) return KDA_ERR_INVALID_ARG;
    if (max_pages > 0 && !ok4({block_table, weight, block_table_out, weight_out, freed})) return KDA_ERR_INVALID_ARG;
    kda::CacheEvictParams p{};
    p.seq_lens = seq_lens; p.block_table = block_table; p.weight = weight;
    p.seq_lens_out = seq_lens_out; p.block_table_out = block_table_out; p.weight_out = weight_out;
    p.freed = freed; p.freed_count = freed_count; p.err_flag = err_flag;
    p.batch = batch; p.max_pages = max_pages; p.budget = budget; p.sink = sink; p.recent = recent;
    return from_cuda(kda::launch_cache_evict(p, (cudaStream_t)stream));
}

}  // extern "C"
