// Launch interface between the attention entry points (kda_attn_api.cu) and
// their kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "kda_attn.h"

namespace kda {

constexpr int kPage = KDA_PAGE_TOKENS;

struct AttnPrefillParams {
    const int32_t *cu_seqlens;
    int64_t total_tokens;
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;  // elements between tokens
    void *out;
    float *lse;
    int32_t *err_flag;
    int32_t num_seqs, Hq, Hkv, G;
    float scale;
};

struct CacheAppendParams {
    unsigned char *k_pages, *v_pages;
    float *k_scale, *v_scale;
    int64_t num_pages;
    const int32_t *cu_seqlens;
    int64_t total_tokens;
    const void *k, *v;
    int64_t k_stride, v_stride;
    const int32_t *start_pos, *block_table;
    int32_t *err_flag;
    int32_t num_seqs, Hkv, max_pages;
};

struct AttnDecodeParams {
    const unsigned char *k_pages, *v_pages;
    const float *k_scale, *v_scale;
    int64_t num_pages;
    const void *q;
    int64_t q_stride;
    const int32_t *seq_lens, *block_table;
    void *out;
    float *lse;
    const float *weight_in;
    float *weight_out;
    void *workspace;
    int32_t *err_flag;
    int32_t batch, D, Hq, Hkv, G, max_pages;
    float scale;
};

struct CacheEvictParams {
    const int32_t *seq_lens, *block_table;
    const float *weight;
    int32_t *seq_lens_out, *block_table_out;
    float *weight_out;
    int32_t *freed, *freed_count, *err_flag;
    int32_t batch, max_pages, budget, sink, recent;
};

// The packed sequence that owns unit u when sequence s gets the units
// [cu[s] / per + s extra, cu[s+1] / per + (s + 1) extra), at least
// ceil(len / per) (extra >= 1) of them: the last s whose first unit is <= u, by
// a 32-way search of a converged warp on cu_seqlens alone (two dependent reads
// for 1024 sequences).  Also gives the unit's index within the sequence.
// Reads cu[0..num_seqs] only, whatever the offsets hold.
// Offsets that fall set KDA_DEVERR_SEQLENS where they are met.  All the units'
// searches together miss none: a search compares the ends of the parts that it
// narrows down, and while those do not fall, every part owns a unit and is
// searched for it, down to the single sequences.
__device__ __forceinline__ int seq_of_unit(const int32_t *cu, int num_seqs, int per, int extra, int64_t u,
                                           int32_t *err, int64_t &local) {
    const int lane = threadIdx.x & 31;
    int a = 0, n = num_seqs, first = 0;  // candidates a..a + n - 1, and the first unit of a
    do {
        const int step = (n + 31) / 32, m = a + lane * step;
        int64_t at = 0;
        if (lane * step < n) {
            const int from = cu[m], to = cu[min(m + step, a + n)];
            at = (int64_t)(from / per) + (int64_t)m * extra;
            if (to < from && err) atomicOr(err, KDA_DEVERR_SEQLENS);
        }
        const unsigned in = __ballot_sync(~0u, lane * step < n && (lane == 0 || at <= u));
        const int k = 31 - __clz(in);
        first = __shfl_sync(~0u, (int)(u - at), k);
        a += k * step;
        n = min(step, n - k * step);
    } while (n > 1);
    local = first;
    return a;
}

// Token range of sequence s; false (and KDA_DEVERR_SEQLENS) when it is not one.
__device__ __forceinline__ bool seq_range(const int32_t *cu, int s, int64_t total, int32_t *err, int &lo, int &hi) {
    lo = cu[s];
    hi = cu[s + 1];
    if (lo >= 0 && lo <= hi && (int64_t)hi <= total) return true;
    if (err) atomicOr(err, KDA_DEVERR_SEQLENS);
    return false;
}

// A scale that the cache's arithmetic by exponents can use: a power of two in
// 2^-126..2^126, whose inverse is one too.
__device__ __forceinline__ bool power_of_two(float s) {
    const uint32_t bits = __float_as_uint(s);
    return (bits & 0x7fffffu) == 0 && bits - 0x800000u < 0x7e800000u;
}

// Raises a kernel's dynamic shared memory limit on the current device, once per
// device (`done`: a static of the caller, one per kernel).
inline cudaError_t allow_smem(const void *kernel, int bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    const cudaError_t g = cudaGetDevice(&dev);
    if (g != cudaSuccess) return g;
    const uint64_t bit = (uint64_t)1 << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

cudaError_t launch_attn_prefill(const AttnPrefillParams &p, int d, int dtype, cudaStream_t s);
// Prompts in bf16, on the tensor cores.
cudaError_t launch_attn_prefill_tc(const AttnPrefillParams &p, int d, cudaStream_t s);
cudaError_t launch_cache_append(const CacheAppendParams &p, int d, int dtype, cudaStream_t s);
size_t attn_decode_workspace_bytes(int Hq, int Hkv, int d, int dtype, int64_t batch, int D, int64_t max_pages,
                                   bool with_weight);
cudaError_t launch_attn_decode(const AttnDecodeParams &p, int d, int dtype, cudaStream_t s);
cudaError_t launch_cache_evict(const CacheEvictParams &p, cudaStream_t s);

}  // namespace kda
