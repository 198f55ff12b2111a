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
// bits, and a selection is a matter of the inputs alone: of units of any size too,
// since scores are compared without leaving whole numbers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <limits.h>
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
// minimum of fp16 pass over NaN), and joins them across its lanes.  What bounds it
// is one chain of reads (sequence, table, scale and keys) and, of long prompts,
// HBM: 256 sequences of a token 8.7 us, 32 355 tokens of 8 heads, d = 128, 11 us.
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
        const float f = amax > 0.f ? exp2i(ke - ue) : 0.f;  // (2^15 at most, for an amax of 2^-9: amax f <= 127)
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
// its registers, the rows' whole numbers come from shared memory for all threads
// alike, positive and negative ones apart: max(x hi, x lo) = max(x, 0) hi +
// min(x, 0) lo, four channels a dp4a.  A warp goes over groups of 32 pages by
// itself: bounds come through shared memory, so that the reads are whole lines, and
// the next group's are asked for as soon as this one's are in registers (their
// ids and units one group earlier).  A page's 2 d bytes are scored for every row,
// so with few rows it is bound by HBM, in reads of 256 bytes: 64 sequences of up to
// 102 400 positions, 8 heads of 4 rows, d = 128, about 30 us of 41, 3.6 TB/s.
// Two buffers a warp at 12 warps an SM took 38.
constexpr int kScoreWarps = 4;
// Blocks that a call has at least, where it has the pages: 1, 2, 4, 8 times 152 x 3 take 43.9, 41.9, 41.9, 43.9 us
// for the 64 sequences; one of 102 400 positions 12.6 either way.
constexpr int64_t kScoreBlocks = 4 * 152 * 3;
constexpr int kScoreRows = 64;  // rows in shared memory together; more take further rounds over the pages

template <int HD>
struct ScoreSmem {
    static constexpr int kPitch = 2 * HD + 16;  // of a page: eight neighbours' pieces lie in different banks
    static constexpr int kTile = 32 * kPitch;
    static int bytes(int rows) { return kScoreWarps * kTile + (rows < kScoreRows ? rows : kScoreRows) * 2 * HD; }
};

// Scores as whole numbers of the same order.  A sum of 128 products is below 2^21, so as fp32 it has 20 bits behind
// the first and 3 that are 0; what its row's and its page's units add to the exponent, up to 2^248 and 2^252, would leave
// fp32's range, and is added where those 3 bits make room for it.
constexpr int kScoreBits = 20;  // of a score's fraction
__device__ __forceinline__ int unit_step(int e) { return (e + 126) << kScoreBits; }  // of a unit 2^e, e = -126..126
__device__ __forceinline__ int score_of(int sum, int step) {
    const int mag = (int)(__float_as_uint(fabsf((float)sum)) >> (23 - kScoreBits)) + step;
    return sum > 0 ? mag : sum < 0 ? -mag : 0;
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

// blockIdx.x: item (sequence, kv head) and which of `splits` shares of its page groups.
template <typename T, int HD>
__global__ void __launch_bounds__(32 * kScoreWarps) score_kernel(const CacheSelectParams p, int splits) {
    using S = ScoreSmem<HD>;
    constexpr int W = HD / 4;  // words of a bound, and of a row's part
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ int x_step[kScoreRows];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int item = (int)(blockIdx.x / (unsigned)splits), split = (int)(blockIdx.x % (unsigned)splits);
    const int n = item / p.Hkv, h = item % p.Hkv;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int len;
    const int P = (int)held_pages(p.seq_lens, n, p.max_pages, len);
    const int first = 32 * (split * kScoreWarps + warp), step = 32 * splits * kScoreWarps;  // the warp's pages
    if (32 * split * kScoreWarps >= P || P <= p.budget) return;  // (by whole blocks)
    unsigned char *tile = smem + warp * S::kTile;
    uint32_t *xs = reinterpret_cast<uint32_t *>(smem + kScoreWarps * S::kTile);  // [row][2][W]
    const int32_t *table = p.block_table + (int64_t)n * p.max_pages;
    uint32_t *keys = static_cast<uint32_t *>(p.workspace) + (int64_t)item * p.max_pages;

    // A page's id, -1 where there is none; its unit, 0 where it has none that can be used.  A page that is not in
    // the summary, or whose unit is no power of two, scores below all others.
    auto id_of = [&](int page, bool tell) {
        if (page >= P) return -1;
        const int id = table[page];
        const bool in = id >= 0 && id < p.num_pages;
        if (!in && tell && p.err_flag) atomicOr(p.err_flag, KDA_DEVERR_PAGE);
        return in ? id : -1;
    };
    auto unit_of = [&](int id) { return id < 0 ? 0.f : p.unit[(int64_t)id * p.Hkv + h]; };
    // Copies 32 pages' bounds, by the whole warp: 16 bytes a lane.  (Where a page has none some other's, which
    // does not count.)
    constexpr int PIECES = 2 * HD / 16, AT_ONCE = 32 / PIECES;
    const int8_t *from = p.bounds + (int64_t)h * (2 * HD) + 16 * (lane % PIECES);
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(tile + (lane / PIECES) * S::kPitch + 16 * (lane % PIECES));
    const int64_t page_bytes = (int64_t)p.Hkv * (2 * HD);
    auto copy = [&](int id) {
        if (p.num_pages == 0) return;
        const int safe = max(id, 0);
#pragma unroll
        for (int i = 0; i < 32; i += AT_ONCE) {
            const int pg = __shfl_sync(~0u, safe, i + lane / PIECES);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * S::kPitch), "l"(from + pg * page_bytes) : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    const int rows = p.D * p.G;
    for (int r0 = 0; r0 < rows; r0 += kScoreRows) {
        const int here = min(kScoreRows, rows - r0);
        int now = id_of(first + lane, r0 == 0), next = id_of(first + step + lane, r0 == 0);
        copy(now);
        float unit = unit_of(now);
        if (r0 > 0) __syncthreads();
        // the rows' whole numbers, a warp a row
        for (int r = warp; r < here; r += kScoreWarps) {
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
                xs[r * 2 * W + lane] = up;
                xs[r * 2 * W + W + lane] = down;
            }
            if (lane == 0) x_step[r] = unit_step(e);
        }
        __syncthreads();
        for (int page = first; page < P; page += step) {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncwarp();
            uint32_t b[2][W];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < W; j += 4) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(tile + lane * S::kPitch + i * HD + 4 * j);
                    b[i][j] = u.x; b[i][j + 1] = u.y; b[i][j + 2] = u.z; b[i][j + 3] = u.w;
                }
            __syncwarp();
            if (page + step < P) copy(next);
            const float next_unit = unit_of(next);
            const int after = id_of(page + 2 * step + lane, r0 == 0);
            int best = INT_MIN;
#pragma unroll 1
            for (int r = 0; r < here; ++r) {
                int sum[4] = {0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < W; j += 4) {
                        const uint4 u = *reinterpret_cast<const uint4 *>(xs + r * 2 * W + i * W + j);
                        sum[0] = __dp4a((int)u.x, (int)b[i][j], sum[0]);
                        sum[1] = __dp4a((int)u.y, (int)b[i][j + 1], sum[1]);
                        sum[2] = __dp4a((int)u.z, (int)b[i][j + 2], sum[2]);
                        sum[3] = __dp4a((int)u.w, (int)b[i][j + 3], sum[3]);
                    }
                best = max(best, score_of((sum[0] + sum[1]) + (sum[2] + sum[3]), x_step[r]));
            }
            if (page + lane < P) {
                const bool good = now >= 0 && power_of_two(unit);
                if (now >= 0 && !good && r0 == 0 && p.err_flag) atomicOr(p.err_flag, KDA_DEVERR_SCALE);
                const int step = good ? unit_step((int)(__float_as_uint(unit) >> 23) - 127) : 0;
                uint32_t key = good ? 0x80000000u + (uint32_t)(best + (best > 0 ? step : best < 0 ? -step : 0)) : 0;
                if (r0 > 0) key = max(key, keys[page + lane]);
                keys[page + lane] = key;
            }
            now = next;
            unit = next_unit;
            next = after;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");  // (a warp without pages has copies in flight)
        __syncwarp();
    }
}

// ---------------------------------------------------------------- selection
//
// A block per sequence and kv head.  The pages that always stay get the largest
// key.  The score t of the last page that is taken is found by rounds: the range
// of the scores (as ordered integers, in shared memory) that still can be t, from
// the smallest to the largest at first, is cut into 1024 bins and the scores
// counted; the bin in which the taken ones end is the next range, until bins are
// single values.  Bins of the range itself spread the scores, so that counts
// seldom meet, and three rounds are the rule: 1600 pages 8.5 us cold, against 13.3
// with a histogram round per byte.  Of the pages that score exactly t
// the lower indices are taken.  A thread then writes the taken pages of its run
// of neighbours, behind those of the runs before.
constexpr int kSelectThreads = 512;
constexpr int kSelectCached = 50000;  // pages whose scores fit shared memory; longer rows are read where they are

__global__ void __launch_bounds__(kSelectThreads) select_kernel(const CacheSelectParams p, int cached) {
    constexpr int WARPS = kSelectThreads / 32;
    extern __shared__ __align__(16) uint32_t held[];
    constexpr int BIN_BITS = 10, BINS = 1 << BIN_BITS;
    static_assert(BINS == 2 * kSelectThreads, "two bins a thread");
    __shared__ __align__(8) int bins[BINS];
    __shared__ int2 sums[WARPS];
    __shared__ uint2 ends[WARPS];
    __shared__ int found[2];
    const int item = blockIdx.x, n = item / p.Hkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int len;
    const int P = (int)held_pages(p.seq_lens, n, p.max_pages, len);
    const int32_t *table = p.block_table + (int64_t)n * p.max_pages;
    const int64_t to = (int64_t)item * p.budget;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (item % p.Hkv == 0 && tid == 0) {
        if (p.err_flag && (int64_t)p.seq_lens[n] > (int64_t)p.max_pages * kPage) atomicOr(p.err_flag, KDA_DEVERR_PAGE);
        p.seq_lens_out[n] = len - (P > p.budget ? (P - p.budget) * kPage : 0);
    }
    if (P <= p.budget) {
        for (int i = tid; i < p.budget; i += kSelectThreads) {
            const int id = i < P ? table[i] : -1;
            p.block_table_out[to + i] = id;
            p.index_out[to + i] = i < P ? i : -1;
            if (i < P && p.err_flag) {  // (no scores, but errors as with them)
                if (id < 0 || id >= p.num_pages) atomicOr(p.err_flag, KDA_DEVERR_PAGE);
                else if (!power_of_two(p.unit[(int64_t)id * p.Hkv + item % p.Hkv])) atomicOr(p.err_flag, KDA_DEVERR_SCALE);
            }
        }
        return;
    }
    const uint32_t *scores = static_cast<const uint32_t *>(p.workspace) + (int64_t)item * p.max_pages;
    auto score = [&](int i) { return i < p.sink || i >= P - p.recent ? ~0u : scores[i]; };
    uint32_t lo = ~0u, hi = 0;  // of the pages that need not stay
    for (int i = tid; i < P; i += kSelectThreads) {
        const uint32_t key = score(i);
        if (cached > 0) held[i] = key;
        if (i >= p.sink && i < P - p.recent) {
            lo = min(lo, key);
            hi = max(hi, key);
        }
    }
    lo = __reduce_min_sync(~0u, lo);
    hi = __reduce_max_sync(~0u, hi);
    if (lane == 0) ends[warp] = make_uint2(lo, hi);
    *reinterpret_cast<int2 *>(bins + 2 * tid) = make_int2(0, 0);
    __syncthreads();
    const uint2 e = ends[lane % WARPS];
    lo = __reduce_min_sync(~0u, e.x);
    hi = __reduce_max_sync(~0u, e.y);
    auto key_of = [&](int i) { return cached > 0 ? held[i] : score(i); };

    uint32_t t = ~0u;
    int need = p.budget - p.sink - p.recent;  // of the range, the largest ones
    while (need > 0) {
        const int shift = max(0, 32 - __clz(hi - lo) - BIN_BITS);
        for (int i = p.sink + tid; i < P - p.recent; i += kSelectThreads) {
            const uint32_t key = key_of(i);
            if (key >= lo && key <= hi) atomicAdd(&bins[BINS - 1 - ((key - lo) >> shift)], 1);  // the largest first
        }
        __syncthreads();
        const int2 c = *reinterpret_cast<const int2 *>(bins + 2 * tid);
        int incl = c.x + c.y;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(~0u, incl, o);
            if (lane >= o) incl += x;
        }
        if (lane == 31) sums[warp].x = incl;
        __syncthreads();
        *reinterpret_cast<int2 *>(bins + 2 * tid) = make_int2(0, 0);
        int before = lane < warp ? sums[lane].x : 0;  // (WARPS <= 32)
        before = __reduce_add_sync(~0u, before) + incl - c.x - c.y;
        if (before < need && before + c.x + c.y >= need) {  // the range's end lies in one of the thread's bins
            const bool second = before + c.x < need;
            found[0] = BINS - 1 - (2 * tid + (second ? 1 : 0));
            found[1] = need - before - (second ? c.x : 0);
        }
        __syncthreads();
        need = found[1];
        lo += (uint32_t)found[0] << shift;
        if (shift == 0) {
            t = lo;
            break;
        }
        hi = min(hi, lo + ((1u << shift) - 1u));
    }
    __syncthreads();
    // of the pages that score more all are taken, of those that score t the first
    const int run = (P + kSelectThreads - 1) / kSelectThreads;
    const int i0 = min(tid * run, P), i1 = min(i0 + run, P);
    int equal = 0, more = 0;
    for (int i = i0; i < i1; ++i) {
        const uint32_t key = key_of(i);
        equal += key == t;
        more += key > t;
    }
    int eq_before = equal, more_before = more;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(~0u, eq_before, o), y = __shfl_up_sync(~0u, more_before, o);
        if (lane >= o) {
            eq_before += x;
            more_before += y;
        }
    }
    if (lane == 31) sums[warp] = make_int2(eq_before, more_before);
    __syncthreads();
    eq_before -= equal;
    more_before -= more;
    int all_more = 0;
    for (int w = 0; w < WARPS; ++w) {
        const int2 x = sums[w];
        if (w < warp) {
            eq_before += x.x;
            more_before += x.y;
        }
        all_more += x.y;
    }
    const int take = p.budget - all_more;  // of score t
    for (int i = i0; i < i1; ++i) {
        const uint32_t key = key_of(i);
        if (key > t || (key == t && eq_before < take)) {
            const int at = more_before + min(eq_before, take);
            p.block_table_out[to + at] = table[i];
            p.index_out[to + at] = i;
        }
        eq_before += key == t;
        more_before += key > t;
    }
}

template <typename T, int HD>
cudaError_t launch_select(const CacheSelectParams &p, cudaStream_t st) {
    const int64_t items = (int64_t)p.batch * p.Hkv;
    if (items > 0x7fffffff) return cudaErrorInvalidValue;
    if (p.max_pages <= p.budget) {  // nothing to choose
        select_kernel<<<(unsigned)items, kSelectThreads, 0, st>>>(p, 0);
        return cudaGetLastError();
    }
    // enough shares to fill the GPU, of one group of pages a warp at least
    const int64_t most = ((int64_t)p.max_pages + 32 * kScoreWarps - 1) / (32 * kScoreWarps);
    int64_t splits = (kScoreBlocks + items - 1) / items;
    splits = splits < 1 ? 1 : splits > most ? most : splits;
    if (items * splits > 0x7fffffff) return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0}, done_select{0};
    auto score = score_kernel<T, HD>;
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(score), ScoreSmem<HD>::bytes(kScoreRows), done);
    if (e == cudaSuccess) e = allow_smem(reinterpret_cast<const void *>(select_kernel), kSelectCached * 4, done_select);
    if (e != cudaSuccess) return e;
    score<<<(unsigned)(items * splits), 32 * kScoreWarps, ScoreSmem<HD>::bytes(p.D * p.G), st>>>(p, (int)splits);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int cached = p.max_pages <= kSelectCached ? p.max_pages : 0;
    return launch_after_smem(select_kernel, dim3((unsigned)items), kSelectThreads, cached * 4, st, p, cached);
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
