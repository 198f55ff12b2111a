// Pages by a cheap score: summaries of the cached keys, and the selection.
//
// A page and kv head's summary is, per channel, the largest and the smallest of
// its keys in whole numbers of one unit, a power of two: hi and lo in -127..127.
// A query row is taken in whole numbers of a unit of its own, x in -127..127, and
//
//   score = unit_q unit_p sum_c max(x_c hi_c, x_c lo_c),
//
// about the most that a key of the page can give the row.  Sums of 128 products
// of whole numbers stay below 2^24, so every order of adding gives the same
// bits, and a selection is a matter of the inputs alone.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "kda_attn_decode.cuh"
#include "kda_attn_internal.h"
#include "kda_cache.cuh"

namespace kda {
namespace {

using dec::e4m3x4_to_f16;

// The exponent of the smallest power of two u with amax <= 127 u (amax > 0, finite).
__device__ __forceinline__ int unit_exponent(float amax) {
    // subnormal amax: the caller's floor of -126 is above it
    const uint32_t b = __float_as_uint(amax);
    return (int)(b >> 23) - 127 - 6 + ((b & 0x7fffffu) > 0x7e0000u ? 1 : 0);
}

__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126..127

// ---------------------------------------------------------------- summaries
//
// A warp takes a page and a kv head: it reads the head's keys once (16 bytes a
// lane), keeps the extremes as fp16 pairs (exact for e4m3; the maximum and
// minimum of fp16 pass over NaN), and joins them across its lanes.
constexpr int kSumWarps = 8;

template <int HD>
__global__ void __launch_bounds__(32 * kSumWarps) summarise_kernel(const CacheSummariseParams p) {
    constexpr int LPR = HD / 16, RPP = 32 / LPR;  // lanes of a row, rows of a pass
    constexpr int STEPS = kPage / RPP;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    PageRows pr;
    if (!page_of_unit(p, blockIdx.x, pr)) return;
    if (pr.page < 0 || pr.page >= p.num_pages) {
        if (p.err_flag && threadIdx.x == 0) atomicOr(p.err_flag, KDA_DEVERR_PAGE);
        return;
    }
    const int fill = pr.off + pr.rows;
    for (int h = warp; h < p.Hkv; h += kSumWarps) {
        const int64_t block = pr.page * p.Hkv + h;
        const float scale = p.k_scale[block];
        const uint4 *src = reinterpret_cast<const uint4 *>(p.k_pages + block * (int64_t)(HD * kPage)) + lane;
        uint4 raw[STEPS];
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            raw[i] = make_uint4(0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);  // NaN: passed over
            if (i * RPP + lane / LPR < fill) raw[i] = src[i * 32];
        }
        __half2 hi[8], lo[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            hi[e] = __half2half2(__ushort_as_half(0xfc00));  // -inf
            lo[e] = __half2half2(__ushort_as_half(0x7c00));
        }
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t a, b;
                e4m3x4_to_f16(w[e], a, b);
                const __half2 x = *reinterpret_cast<const __half2 *>(&a), y = *reinterpret_cast<const __half2 *>(&b);
                hi[2 * e] = __hmax2(hi[2 * e], x); lo[2 * e] = __hmin2(lo[2 * e], x);
                hi[2 * e + 1] = __hmax2(hi[2 * e + 1], y); lo[2 * e + 1] = __hmin2(lo[2 * e + 1], y);
            }
        }
#pragma unroll
        for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                hi[e] = __hmax2(hi[e], __shfl_xor_sync(~0u, hi[e], o));
                lo[e] = __hmin2(lo[e], __shfl_xor_sync(~0u, lo[e], o));
            }
        // lanes of the first row take the largest, those of the second the smallest
        const bool low = (lane / LPR) & 1;
        float x[16], amax = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 y = __half22float2(low ? lo[e] : hi[e]);
            x[2 * e] = fabsf(y.x) <= 448.f ? y.x : 0.f;  // (a channel of NaN alone is still infinite)
            x[2 * e + 1] = fabsf(y.y) <= 448.f ? y.y : 0.f;
            amax = fmaxf(amax, fmaxf(fabsf(x[2 * e]), fabsf(x[2 * e + 1])));
        }
#pragma unroll
        for (int o = 1; o < 2 * LPR; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
        const int ke = (int)(__float_as_uint(scale) >> 23) - 127;
        const int ue = amax > 0.f ? max(ke + unit_exponent(amax), -126) : -126;
        if (!power_of_two(scale) || ue > 126) {
            if (p.err_flag && lane == 0) atomicOr(p.err_flag, KDA_DEVERR_SCALE);
            continue;
        }
        const float f = amax > 0.f ? exp2i(ke - ue) : 0.f;  // (2^9 at most: 448 f <= 127)
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[e] = 0;
#pragma unroll
            for (int b = 0; b < 4; ++b) w[e] |= (uint32_t)(__float2int_rn(x[4 * e + b] * f) & 255) << (8 * b);
        }
        if (lane < 2 * LPR)
            *reinterpret_cast<uint4 *>(p.bounds + (block * 2 + (low ? 1 : 0)) * HD + 16 * (lane % LPR)) =
                make_uint4(w[0], w[1], w[2], w[3]);
        if (lane == 0) p.unit[block] = exp2i(ue);
    }
}

template <int HD>
cudaError_t launch_summarise(const CacheSummariseParams &p, cudaStream_t st) {
    const int64_t units = p.total_tokens / kPage + 2 * (int64_t)p.num_seqs;  // as for the append
    if (units > 0x7fffffff) return cudaErrorInvalidValue;
    summarise_kernel<HD><<<(unsigned)units, 32 * kSumWarps, 0, st>>>(p);
    return cudaGetLastError();
}

// ---------------------------------------------------------------- scores
//
// A thread scores a page for all rows of its kv head: the page's bounds lie in
// its registers (staged through shared memory, so that the reads are whole
// lines), the rows' whole numbers come from shared memory for all threads alike,
// positive and negative ones apart: max(x hi, x lo) = max(x, 0) hi + min(x, 0) lo,
// four channels a dp4a.
constexpr int kScorePages = 128;  // pages (threads) of a block
constexpr int kScoreRows = 16;    // rows in shared memory together

__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);  // -0 as 0
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// Four neighbouring elements.
__device__ __forceinline__ void load4(const float *p, float (&x)[4]) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float (&x)[4]) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xffff0000u);
}

__device__ __forceinline__ int64_t held_pages(const int32_t *seq_lens, int n, int max_pages, int &len) {
    const int64_t cap = (int64_t)max_pages * kPage;
    const int64_t l = seq_lens[n];
    len = (int)(l < 0 ? 0 : l > cap ? cap : l);
    return (len + kPage - 1) / kPage;
}

template <typename T, int HD>
__global__ void __launch_bounds__(kScorePages) score_kernel(const CacheSelectParams p, int chunks) {
    constexpr int W = HD / 4;          // words of a bound, and of a row's part
    constexpr int PITCH = 2 * HD + 16; // bytes of a page in shared memory: eight neighbours' pieces lie in different banks
    __shared__ __align__(16) unsigned char tile[kScorePages * PITCH];
    __shared__ __align__(16) uint32_t xs[kScoreRows][2][W];
    __shared__ float x_unit[kScoreRows];
    __shared__ int ids[kScorePages];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int item = (int)(blockIdx.x / (unsigned)chunks), n = item / p.Hkv, h = item % p.Hkv;
    int len;
    const int P = (int)held_pages(p.seq_lens, n, p.max_pages, len);
    const int page0 = (int)(blockIdx.x % (unsigned)chunks) * kScorePages;
    if (page0 >= P || P <= p.budget) return;

    int id = -1;
    float unit = 0.f;
    int err = 0;
    if (page0 + tid < P) {
        id = p.block_table[(int64_t)n * p.max_pages + page0 + tid];
        if (id < 0 || id >= p.num_pages) {
            id = -1;
            err = KDA_DEVERR_PAGE;
        } else {
            unit = p.unit[(int64_t)id * p.Hkv + h];
            if (!power_of_two(unit)) {
                id = -1;
                err = KDA_DEVERR_SCALE;
            }
        }
    }
    if (err != 0 && p.err_flag) atomicOr(p.err_flag, err);
    ids[tid] = id;
    __syncthreads();
    constexpr int PIECES = 2 * HD / 16;  // of a page
    for (int i = tid; i < kScorePages * PIECES; i += kScorePages) {
        const int pg = i / PIECES, piece = i % PIECES;
        if (ids[pg] < 0) continue;
        const int8_t *src = p.bounds + ((int64_t)ids[pg] * p.Hkv + h) * (2 * HD) + 16 * piece;
        const uint32_t dst = (uint32_t)__cvta_generic_to_shared(tile + pg * PITCH + 16 * piece);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");

    const int rows = p.D * p.G;
    uint32_t b[2][W];
    float best = -INFINITY;
    for (int r0 = 0; r0 < rows; r0 += kScoreRows) {
        const int here = min(kScoreRows, rows - r0);
        if (r0 > 0) __syncthreads();
        // the rows' whole numbers, a warp a row
        for (int r = warp; r < here; r += kScorePages / 32) {
            const int tok = (r0 + r) / p.G, g = (r0 + r) % p.G;
            const T *src = static_cast<const T *>(p.q) + ((int64_t)n * p.D + tok) * p.q_stride + (int64_t)(h * p.G + g) * HD;
            float x[4] = {0.f, 0.f, 0.f, 0.f}, amax = 0.f;
            if (lane < W) {
                load4(src + 4 * lane, x);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (fabsf(x[e]) <= 3.402823466e38f) amax = fmaxf(amax, fabsf(x[e]));
                    else if (!(x[e] == x[e])) x[e] = 0.f;
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
            const int e = amax > 0.f ? max(unit_exponent(amax), -126) : -126;
            uint32_t up = 0, down = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int v = __float2int_rn(fminf(fmaxf(x[j] * exp2i(-e), -127.f), 127.f));
                up |= (uint32_t)(max(v, 0) & 255) << (8 * j);
                down |= (uint32_t)(min(v, 0) & 255) << (8 * j);
            }
            if (lane < W) {
                xs[r][0][lane] = up;
                xs[r][1][lane] = down;
            }
            if (lane == 0) x_unit[r] = exp2i(e);
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        if (r0 == 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < W; j += 4) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(tile + tid * PITCH + i * HD + 4 * j);
                    b[i][j] = u.x; b[i][j + 1] = u.y; b[i][j + 2] = u.z; b[i][j + 3] = u.w;
                }
        }
        for (int r = 0; r < here; ++r) {
            int sum[4] = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < W; j += 4) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(&xs[r][i][j]);
                    sum[0] = __dp4a((int)u.x, (int)b[i][j], sum[0]);
                    sum[1] = __dp4a((int)u.y, (int)b[i][j + 1], sum[1]);
                    sum[2] = __dp4a((int)u.z, (int)b[i][j + 2], sum[2]);
                    sum[3] = __dp4a((int)u.w, (int)b[i][j + 3], sum[3]);
                }
            best = fmaxf(best, (float)((sum[0] + sum[1]) + (sum[2] + sum[3])) * x_unit[r]);
        }
    }
    if (page0 + tid < P)
        static_cast<uint32_t *>(p.workspace)[(int64_t)item * p.max_pages + page0 + tid] =
            ordered(id < 0 ? -INFINITY : best * unit);
}

// ---------------------------------------------------------------- selection
//
// A block per sequence and kv head.  The pages that always stay get the largest
// key; a radix selection over the scores as ordered integers (8 bits a pass, the
// histogram in shared memory) finds the score t of the last page that is taken
// and how many of the pages that score exactly t are; of those the lower indices
// are.  One pass in index order then writes the taken pages.
constexpr int kSelectThreads = 256;

__global__ void __launch_bounds__(kSelectThreads) select_kernel(const CacheSelectParams p) {
    constexpr int W = kSelectThreads / 32;
    __shared__ uint32_t hist[256];
    __shared__ uint32_t s_prefix, s_left;
    __shared__ int warp_a[W], warp_b[W];
    const int item = blockIdx.x, n = item / p.Hkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int len;
    const int P = (int)held_pages(p.seq_lens, n, p.max_pages, len);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (item % p.Hkv == 0 && tid == 0) {
        if (p.err_flag && (int64_t)p.seq_lens[n] > (int64_t)p.max_pages * kPage) atomicOr(p.err_flag, KDA_DEVERR_PAGE);
        p.seq_lens_out[n] = len - (P > p.budget ? (P - p.budget) * kPage : 0);
    }
    const int32_t *table = p.block_table + (int64_t)n * p.max_pages;
    const int64_t to = (int64_t)item * p.budget;
    if (P <= p.budget) {
        for (int i = tid; i < p.budget; i += kSelectThreads) {
            p.block_table_out[to + i] = i < P ? table[i] : -1;
            p.index_out[to + i] = i < P ? i : -1;
        }
        return;
    }
    const uint32_t *keys = static_cast<const uint32_t *>(p.workspace) + (int64_t)item * p.max_pages;
    auto key_of = [&](int i) { return i < p.sink || i >= P - p.recent ? ~0u : keys[i]; };
    uint32_t prefix = 0, left = p.budget;
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kSelectThreads) hist[i] = 0;
        __syncthreads();
        const uint32_t mask = shift == 24 ? 0u : ~0u << (shift + 8);
        for (int i = tid; i < P; i += kSelectThreads) {
            const uint32_t key = key_of(i);
            if ((key & mask) == prefix) atomicAdd(&hist[255u - ((key >> shift) & 255u)], 1u);
        }
        __syncthreads();
        if (warp == 0) {  // the bin, from the largest down, in which the running count reaches `left`
            uint32_t c[8], sum = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += c[j] = hist[lane * 8 + j];
            uint32_t incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t t = __shfl_up_sync(~0u, incl, o);
                if (lane >= o) incl += t;
            }
            uint32_t before = incl - sum;
            if (before < left && incl >= left) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (before < left && before + c[j] >= left) {
                        s_prefix = prefix | ((255u - (uint32_t)(lane * 8 + j)) << shift);
                        s_left = left - before;
                    }
                    before += c[j];
                }
            }
        }
        __syncthreads();
        prefix = s_prefix;
        left = s_left;
    }
    // `left` of the pages that score exactly `prefix` are taken: the first ones
    int taken = 0, equal = 0;  // before this chunk
    for (int base = 0; base < P; base += kSelectThreads) {
        const int i = base + tid;
        const uint32_t key = i < P ? key_of(i) : 0;
        const bool eq = i < P && key == prefix, more = i < P && key > prefix;
        const unsigned me = __ballot_sync(~0u, eq), mm = __ballot_sync(~0u, more);
        __syncthreads();
        if (lane == 0) {
            warp_a[warp] = __popc(me);
            warp_b[warp] = __popc(mm);
        }
        __syncthreads();
        int eq_before = equal, more_before = taken;
        for (int w = 0; w < W; ++w) {
            if (w < warp) {
                eq_before += warp_a[w];
                more_before += warp_b[w];
            }
            equal += warp_a[w];
            taken += warp_b[w];
        }
        const unsigned below = (1u << lane) - 1u;
        eq_before += __popc(me & below);
        more_before += __popc(mm & below);
        if (more || (eq && eq_before < (int)left)) {
            const int at = more_before + min(eq_before, (int)left);
            p.block_table_out[to + at] = table[i];
            p.index_out[to + at] = i;
        }
    }
}

template <typename T, int HD>
cudaError_t launch_select(const CacheSelectParams &p, cudaStream_t st) {
    const int64_t items = (int64_t)p.batch * p.Hkv, chunks = ((int64_t)p.max_pages + kScorePages - 1) / kScorePages;
    if (items > 0x7fffffff) return cudaErrorInvalidValue;
    if (p.max_pages <= p.budget) {  // nothing to choose
        select_kernel<<<(unsigned)items, kSelectThreads, 0, st>>>(p);
        return cudaGetLastError();
    }
    if (items * chunks > 0x7fffffff) return cudaErrorInvalidValue;
    score_kernel<T, HD><<<(unsigned)(items * chunks), kScorePages, 0, st>>>(p, (int)chunks);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_after(select_kernel, dim3((unsigned)items), kSelectThreads, st, p);
}

template <typename T>
cudaError_t launch_select_dim(const CacheSelectParams &p, int d, cudaStream_t st) {
    if (d == 128) return launch_select<T, 128>(p, st);
    if (d == 64) return launch_select<T, 64>(p, st);
    return launch_select<T, 32>(p, st);
}

}  // namespace

cudaError_t launch_cache_summarise(const CacheSummariseParams &p, int d, cudaStream_t st) {
    if (d == 128) return launch_summarise<128>(p, st);
    if (d == 64) return launch_summarise<64>(p, st);
    return launch_summarise<32>(p, st);
}

size_t cache_select_workspace_bytes(int Hkv, int64_t batch, int64_t max_pages) {
    return (size_t)(batch * Hkv * max_pages) * sizeof(uint32_t);  // an ordered score per page
}

cudaError_t launch_cache_select(const CacheSelectParams &p, int d, int dtype, cudaStream_t st) {
    return dtype == KDA_DT_BF16 ? launch_select_dim<__nv_bfloat16>(p, d, st) : launch_select_dim<float>(p, d, st);
}

}  // namespace kda
