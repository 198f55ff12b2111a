// Launch interface between the attention entry points (kda_attn_api.cu) and
// their kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

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

// Rows that attend a run of pages together, where a sequence is attended in
// parts (its shared prefix, the rest): rows row / G of tokens tok0.., the run
// starts at position `base` of their sequences and has `len` positions.  Rows
// that see none of it (see dec::limit_of) are computed as if they saw all of it
// and passed over afterwards.
struct AttnChunk {
    int64_t table;  // of the run's first page in block_table
    int32_t tok0, rows, base, len;
    int32_t seen;   // positions that all rows see which see any
    int32_t limit;  // positions of the run that the first token sees, each further one a position more; or
    static constexpr int32_t kManySequences = -0x7fffffff;  // as seq_lens tells
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
    const AttnChunk *chunks;  // parts: takes the place of sequences, `batch` of them; results stay apart:
    float2 *part_ml;          // (m, l) per row, `out` fp32 and not divided by l
    int64_t table_seq, table_head;  // entries between the table rows of sequences, and of a sequence's kv heads (0: one for all)
    int32_t batch, D, Hq, Hkv, G, max_pages;
    float scale;
};

struct AttnSharedParams {
    AttnDecodeParams call;  // the whole batch
    const int32_t *group_start, *shared_pages;
    int32_t groups;
};

struct NormRotateParams {
    const void *q, *k;
    void *q_out, *k_out;
    int64_t q_stride, k_stride, q_out_stride, k_out_stride;  // elements between tokens
    const int32_t *positions;
    const uint64_t *turns;  // [rot / 2]
    const float *q_weight, *k_weight;
    int64_t total_tokens;
    int32_t Hq, Hkv, rot, interleaved;
    float eps, factor;
};

struct CacheSummariseParams {
    const unsigned char *k_pages;
    const float *k_scale;
    int64_t num_pages;
    int8_t *bounds;
    float *unit;
    const int32_t *cu_seqlens;
    int64_t total_tokens;
    const int32_t *start_pos, *block_table;
    int32_t *err_flag;
    int32_t num_seqs, Hkv, max_pages;
};

struct CacheSelectParams {
    const int8_t *bounds;
    const float *unit;
    int64_t num_pages;
    const void *q;
    int64_t q_stride;
    const int32_t *seq_lens, *block_table;
    int32_t *seq_lens_out, *block_table_out, *index_out;
    void *workspace;
    int32_t *err_flag;
    int32_t batch, D, Hkv, G, max_pages, budget, sink, recent;
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

// A launch that may begin while the kernel before it on the stream ends (the
// kernel waits for that one's results by itself).
template <typename... Args>
cudaError_t launch_after_smem(void (*kern)(Args...), dim3 grid, int threads, int smem, cudaStream_t st,
                              std::common_type_t<Args>... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <typename... Args>
cudaError_t launch_after(void (*kern)(Args...), dim3 grid, int threads, cudaStream_t st,
                         std::common_type_t<Args>... args) {
    return launch_after_smem(kern, grid, threads, 0, st, args...);
}

cudaError_t launch_attn_prefill(const AttnPrefillParams &p, int d, int dtype, cudaStream_t s);
// Prompts in bf16, on the tensor cores.
cudaError_t launch_attn_prefill_tc(const AttnPrefillParams &p, int d, cudaStream_t s);
cudaError_t launch_cache_append(const CacheAppendParams &p, int d, int dtype, cudaStream_t s);
size_t attn_decode_workspace_bytes(int Hq, int Hkv, int d, int dtype, int64_t batch, int D, int64_t max_pages,
                                   bool with_weight);
cudaError_t launch_attn_decode(const AttnDecodeParams &p, int d, int dtype, cudaStream_t s);
size_t attn_shared_workspace_bytes(int Hq, int Hkv, int d, int dtype, int64_t batch, int D, int64_t max_pages,
                                   int64_t groups);
cudaError_t launch_attn_shared(const AttnSharedParams &p, int d, int dtype, cudaStream_t s);
cudaError_t launch_cache_evict(const CacheEvictParams &p, cudaStream_t s);
cudaError_t launch_norm_rotate(const NormRotateParams &p, int d, int dtype, cudaStream_t s);
cudaError_t launch_cache_summarise(const CacheSummariseParams &p, int d, cudaStream_t s);
size_t cache_select_workspace_bytes(int Hkv, int64_t batch, int64_t max_pages);
cudaError_t launch_cache_select(const CacheSelectParams &p, int d, int dtype, cudaStream_t s);

}  // namespace kda
