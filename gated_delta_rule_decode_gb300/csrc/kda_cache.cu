// The 8-bit paged key/value cache: append (quantisation) and page eviction.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "kda_attn_internal.h"
#include "kda_cache.cuh"
#include "kda_check.cuh"

namespace kda {
namespace {

// ---------------------------------------------------------------- append
//
// A page that gets new rows, a head, and keys or values make one task.  The new
// rows' largest finite magnitude gives the scale; a page whose scale grows first
// has its earlier rows rescaled.  The scale is a power of two, so x / s' is
// exact and rescaling re-rounds only what becomes subnormal in e4m3.
//
// Two kernels, by the tokens per sequence of the call (kFewTokens): prompts take
// a CTA per task, which holds the page's rows in registers and turns values into
// rows of positions through shared memory; decode steps take a CTA per page and
// a warp per task, which goes over the one or few rows twice.  Measured: 32 355
// tokens in 8 prompts, 8 heads, d = 128, 41.0 us, 4.8 TB/s, bound by the integer
// pipe beside HBM; a token for each of 256 sequences 8.3 us, a chain of five
// dependent reads (26.6 us with a CTA per task and bisection).
//
// The rule: at 1, 2, 4, 7, 8 and 16 tokens for each of 256 sequences (8 heads,
// d = 128, cold caches) a CTA per task took 23, 23, 25, 27, 27 and 27 us, a warp
// per task 11, 13, 17, 33, 29 and 50; for each of 64 both 11, 11 and 13 up to 4,
// then 13 against 19; for each of 16, 8.9 throughout against 8.8, 8.8, 10.9, 19.
// So 4.  The call knows the mean alone: 255 single tokens and a chunk of 500
// (mean 3) take a warp per task 76 us, a CTA per task 23.
constexpr int kAppendThreads = 128;
constexpr int kStepWarps = 8;
constexpr int64_t kFewTokens = 4;

__device__ __forceinline__ float pow2_need(float amax) {
    // smallest e >= -126 with amax <= 1.75 * 2^8 * 2^e
    const uint32_t b = __float_as_uint(amax);
    const int x = (int)(b >> 23) - 127;
    int e = x - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = e < -126 ? -126 : e;
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// 1 / s for a power of two s in 2^-126..2^126.
__device__ __forceinline__ float pow2_inverse(float s) {
    const uint32_t e = __float_as_uint(s) >> 23;
    return __uint_as_float((254u - e) << 23);
}

__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a <= 3.402823466e38f ? a : 0.f;  // false for infinities and NaN
}

__device__ __forceinline__ uint32_t quant2(float a, float b) {
    // saturates to +-448, keeps NaN, rounds to nearest even
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ unsigned char requant1(unsigned char b, float ratio) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(b, __NV_E4M3);
    return (unsigned char)__nv_cvt_float_to_fp8(__half2float(__half(h)) * ratio, __NV_SATFINITE, __NV_E4M3);
}

template <typename T>
struct Piece;  // 16 bytes of a row as floats
template <>
struct Piece<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void get(const uint4 &u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
    }
};
template <>
struct Piece<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(const uint4 &u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};

// Magnitudes are compared as integers (two bf16 values a word): one and-mask and
// one maximum a word.  `finite` is false where a value of the maximum is an
// infinity or NaN; the caller then takes piece_max over the finite ones.
template <typename T>
struct Magnitude;
template <>
struct Magnitude<float> {
    static __device__ __forceinline__ uint32_t of(uint32_t m, uint32_t w) { return max(m, w & 0x7fffffffu); }
    static __device__ __forceinline__ float value(uint32_t m, bool &finite) {
        finite = m < 0x7f800000u;
        return __uint_as_float(m);
    }
};
template <>
struct Magnitude<__nv_bfloat16> {
    static __device__ __forceinline__ uint32_t of(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }
    static __device__ __forceinline__ float value(uint32_t m, bool &finite) {
        const uint32_t x = max(m & 0xffffu, m >> 16);
        finite = x < 0x7f80u;
        return __uint_as_float(x << 16);
    }
};

template <typename T>
__device__ __forceinline__ uint32_t piece_bits(uint32_t m, const uint4 &u) {
    return Magnitude<T>::of(Magnitude<T>::of(Magnitude<T>::of(Magnitude<T>::of(m, u.x), u.y), u.z), u.w);
}

template <typename T>
__device__ __forceinline__ float piece_max(const uint4 &u) {
    float x[Piece<T>::N], m = 0.f;
    Piece<T>::get(u, x);
#pragma unroll
    for (int j = 0; j < Piece<T>::N; ++j) m = fmaxf(m, finite_abs(x[j]));
    return m;
}

__device__ __forceinline__ bool page_ok(const CacheAppendParams &p, int64_t page) {
    if (page >= 0 && page < p.num_pages) return true;
    if (p.err_flag && (threadIdx.x & 31) == 0) atomicOr(p.err_flag, KDA_DEVERR_PAGE);
    return false;
}

// The scale of a page's earlier positions (0 where it has none).
__device__ __forceinline__ bool scale_ok(const CacheAppendParams &p, int off, float old) {
    if (off == 0 || power_of_two(old)) return true;
    if (p.err_flag && (threadIdx.x & 31) == 0) atomicOr(p.err_flag, KDA_DEVERR_SCALE);
    return false;
}

// Rescales the page's first `off` positions; threads tid of n.
template <int HD>
__device__ __forceinline__ void rescale_rows(unsigned char *dst, bool is_v, int off, float ratio, int tid, int n) {
    for (int i = tid; i < off * HD; i += n) {
        unsigned char *b = is_v ? dst + (i / off) * kPage + i % off : dst + i;
        *b = requant1(*b, ratio);
    }
}

template <typename T, int HD>
__global__ void __launch_bounds__(kAppendThreads, sizeof(T) == 2 ? 8 : 5) append_kernel(const CacheAppendParams p) {
    constexpr int N = Piece<T>::N;                 // elements per 16-byte piece
    constexpr int PR = HD / N;                     // pieces per row
    constexpr int GROUPS = kPage / 4;              // groups of four positions
    constexpr int STEPS = (PR * GROUPS + kAppendThreads - 1) / kAppendThreads;
    __shared__ __align__(16) uint32_t tile[HD][GROUPS + 1];  // values: four positions of a channel
    __shared__ float warp_max[kAppendThreads / 32];
    // neighbouring CTAs take the heads of the same rows, which lie side by side
    const int tid = threadIdx.x, h = (int)(blockIdx.x % (unsigned)p.Hkv);
    const unsigned rest = blockIdx.x / (unsigned)p.Hkv;
    const bool is_v = rest & 1;
    PageRows pr;
    if (!page_of_unit(p, rest >> 1, pr)) return;
    const int off = pr.off, last = pr.off + pr.rows;

    // a thread holds one piece of the rows at four neighbouring places of the page
    const int64_t stride = is_v ? p.v_stride : p.k_stride;
    const T *src = static_cast<const T *>(is_v ? p.v : p.k) + (pr.tok - off) * stride + (int64_t)h * HD;
    uint4 raw[STEPS][4];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int x = tid + i * kAppendThreads, grp = x / PR, piece = x % PR;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int at = 4 * grp + e;
            raw[i][e] = make_uint4(0, 0, 0, 0);
            if (at >= off && at < last) raw[i][e] = __ldcs(reinterpret_cast<const uint4 *>(src + (int64_t)at * stride + piece * N));
        }
    }
    if (!page_ok(p, pr.page)) return;
    float *scale = (is_v ? p.v_scale : p.k_scale) + pr.page * p.Hkv + h;
    const float old = off > 0 ? *scale : 0.f;
    if (!scale_ok(p, off, old)) return;
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) bits = piece_bits<T>(bits, raw[i][e]);
    bool finite;
    float amax = Magnitude<T>::value(bits, finite);
    if (!finite) {
        amax = 0.f;
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) amax = fmaxf(amax, piece_max<T>(raw[i][e]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
    if ((tid & 31) == 0) warp_max[tid >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kAppendThreads / 32; ++w) amax = fmaxf(amax, warp_max[w]);
    const float now = fmaxf(old, pow2_need(amax));
    const float inv = pow2_inverse(now);
    unsigned char *dst = (is_v ? p.v_pages : p.k_pages) + (pr.page * p.Hkv + h) * (int64_t)(HD * kPage);
    if (off > 0 && now > old) rescale_rows<HD>(dst, is_v, off, old * inv, tid, kAppendThreads);

#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int x = tid + i * kAppendThreads, grp = x / PR, piece = x % PR;
        if (STEPS * kAppendThreads > PR * GROUPS && grp >= GROUPS) continue;
        uint32_t w[4][N / 4];  // row e, four channels a word
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float y[N];
            Piece<T>::get(raw[i][e], y);
#pragma unroll
            for (int j = 0; j < N / 4; ++j)
                w[e][j] = quant2(y[4 * j] * inv, y[4 * j + 1] * inv) | (quant2(y[4 * j + 2] * inv, y[4 * j + 3] * inv) << 16);
        }
        if (!is_v) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int at = 4 * grp + e;
                if (at < off || at >= last) continue;
                uint32_t *o = reinterpret_cast<uint32_t *>(dst + at * HD + piece * N);
                if constexpr (N == 8) *reinterpret_cast<uint2 *>(o) = make_uint2(w[e][0], w[e][1]);
                else *o = w[e][0];
            }
        } else {
            // 4 x 4 bytes turned: four positions of a channel a word
#pragma unroll
            for (int j = 0; j < N / 4; ++j) {
                const uint32_t a = __byte_perm(w[0][j], w[1][j], 0x5140), b = __byte_perm(w[2][j], w[3][j], 0x5140);
                const uint32_t c = __byte_perm(w[0][j], w[1][j], 0x7362), d = __byte_perm(w[2][j], w[3][j], 0x7362);
                tile[piece * N + 4 * j][grp] = __byte_perm(a, b, 0x5410);
                tile[piece * N + 4 * j + 1][grp] = __byte_perm(a, b, 0x7632);
                tile[piece * N + 4 * j + 2][grp] = __byte_perm(c, d, 0x5410);
                tile[piece * N + 4 * j + 3][grp] = __byte_perm(c, d, 0x7632);
            }
        }
    }
    if (tid == 0) *scale = now;
    if (!is_v) return;
    __syncthreads();
    // words of four new positions, single bytes at the two ends
    const int w0 = off / 4, nw = (last + 3) / 4 - w0;
    for (int i = tid; i < HD * nw; i += kAppendThreads) {
        const int ch = i / nw, g = w0 + i % nw, pos = 4 * g;
        const uint32_t x = tile[ch][g];
        if (pos >= off && pos + 4 <= last) {
            *reinterpret_cast<uint32_t *>(dst + ch * kPage + pos) = x;
        } else {
            for (int j = 0; j < 4; ++j)
                if (pos + j >= off && pos + j < last) dst[ch * kPage + pos + j] = (unsigned char)(x >> (8 * j));
        }
    }
}

template <typename T, int HD>
__global__ void __launch_bounds__(32 * kStepWarps) append_step_kernel(const CacheAppendParams p) {
    constexpr int N = Piece<T>::N, PR = HD / N;  // pieces per row: 4..32
    constexpr int RW = 32 / PR;                  // rows at a time
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    PageRows pr;
    if (!page_of_unit(p, blockIdx.x, pr) || !page_ok(p, pr.page)) return;
    const int off = pr.off, piece = lane % PR, r0 = lane / PR;
    for (int task = warp; task < 2 * p.Hkv; task += kStepWarps) {
        const int h = task >> 1;
        const bool is_v = task & 1;
        const int64_t stride = is_v ? p.v_stride : p.k_stride;
        const T *src = static_cast<const T *>(is_v ? p.v : p.k) + pr.tok * stride + (int64_t)h * HD + piece * N;
        float *scale = (is_v ? p.v_scale : p.k_scale) + pr.page * p.Hkv + h;
        const float old = off > 0 ? *scale : 0.f;
        if (!scale_ok(p, off, old)) continue;
        float amax = 0.f;
        for (int r = r0; r < pr.rows; r += RW) amax = fmaxf(amax, piece_max<T>(*reinterpret_cast<const uint4 *>(src + r * stride)));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
        const float now = fmaxf(old, pow2_need(amax));
        const float inv = pow2_inverse(now);
        unsigned char *dst = (is_v ? p.v_pages : p.k_pages) + (pr.page * p.Hkv + h) * (int64_t)(HD * kPage);
        if (off > 0 && now > old) rescale_rows<HD>(dst, is_v, off, old * inv, lane, 32);
        for (int r = r0; r < pr.rows; r += RW) {
            float y[N];
            Piece<T>::get(*reinterpret_cast<const uint4 *>(src + r * stride), y);
            uint32_t w[N / 4];
#pragma unroll
            for (int j = 0; j < N / 4; ++j)
                w[j] = quant2(y[4 * j] * inv, y[4 * j + 1] * inv) | (quant2(y[4 * j + 2] * inv, y[4 * j + 3] * inv) << 16);
            if (!is_v) {
                uint32_t *o = reinterpret_cast<uint32_t *>(dst + (off + r) * HD + piece * N);
                if constexpr (N == 8) *reinterpret_cast<uint2 *>(o) = make_uint2(w[0], w[1]);
                else *o = w[0];
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j) dst[(piece * N + j) * kPage + off + r] = (unsigned char)(w[j / 4] >> (8 * (j % 4)));
            }
        }
        if (lane == 0) *scale = now;
    }
}

template <typename T, int HD>
cudaError_t launch_append_dim(const CacheAppendParams &p, cudaStream_t st) {
    // units of seq_of_unit: cu / 64 + 2 s, so every sequence has its pages
    const int64_t units = p.total_tokens / kPage + 2 * (int64_t)p.num_seqs;
    if (units * 2 * p.Hkv > 0x7fffffff) return cudaErrorInvalidValue;
    if (p.total_tokens <= kFewTokens * p.num_seqs)
        append_step_kernel<T, HD><<<(unsigned)units, 32 * kStepWarps, 0, st>>>(p);
    else
        append_kernel<T, HD><<<(unsigned)(units * 2 * p.Hkv), kAppendThreads, 0, st>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_append(const CacheAppendParams &p, int d, cudaStream_t st) {
    if (d == 128) return launch_append_dim<T, 128>(p, st);
    if (d == 64) return launch_append_dim<T, 64>(p, st);
    return launch_append_dim<T, 32>(p, st);
}

// ---------------------------------------------------------------- evict
//
// One CTA per sequence.  The E = P - budget lightest pages of the middle go:
// a radix selection over the weights as ordered integers (8 bits a pass, the
// histogram in shared memory) finds the weight t of the last page to go and
// how many of the pages that weigh exactly t go with the lighter ones; of
// those the higher indices go.  Then one pass in index order closes the rows
// up.  256 rows of 1600 pages take 14.4 us, 4 of 64 take 8.2: latency of the
// passes.  An entry never moves to a higher index, and a chunk is read before
// anything of it is written, so the rows may be updated in place.
constexpr int kEvictThreads = 512;

__device__ __forceinline__ uint32_t weight_key(float w) {
    if (!(w == w)) return 0;  // NaN below everything
    const uint32_t b = __float_as_uint(w == 0.f ? 0.f : w);  // -0 as 0
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const CacheEvictParams p) {
    constexpr int W = kEvictThreads / 32;
    __shared__ uint32_t hist[256];
    __shared__ uint32_t s_prefix, s_left;
    __shared__ int warp_a[W], warp_b[W];
    const int n = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = (int64_t)n * p.max_pages;
    const int32_t *table = p.block_table + row;
    const float *weight = p.weight + row;
    const int len = p.seq_lens[n];
    const int64_t held = len > 0 ? ((int64_t)len + kPage - 1) / kPage : 0;
    const bool bad = held > p.max_pages;
    if (bad && tid == 0 && p.err_flag) atomicOr(p.err_flag, KDA_DEVERR_PAGE);
    const int P = bad ? 0 : (int)held;
    const int E = P > p.budget ? P - p.budget : 0;
    const int lo = p.sink, hi = P - p.recent;  // the pages that may go (E > 0: lo < hi)

    uint32_t prefix = 0, equal_go = 0;
    if (E > 0) {
        uint32_t left = E;
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += kEvictThreads) hist[i] = 0;
            __syncthreads();
            const uint32_t mask = shift == 24 ? 0u : ~0u << (shift + 8);
            for (int i = lo + tid; i < hi; i += kEvictThreads) {
                const uint32_t key = weight_key(weight[i]);
                if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1u);
            }
            __syncthreads();
            if (warp == 0) {  // the bin in which the running count reaches `left`
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
                            s_prefix = prefix | ((uint32_t)(lane * 8 + j) << shift);
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
        equal_go = left;  // pages of weight `prefix` that go: the last ones of them
    }
    // how many pages weigh exactly `prefix`
    int equal = 0;
    if (E > 0) {
        for (int i = lo + tid; i < hi; i += kEvictThreads) equal += weight_key(weight[i]) == prefix;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) equal += __shfl_xor_sync(~0u, equal, o);
        if (lane == 0) warp_a[warp] = equal;
        __syncthreads();
        equal = 0;
        for (int w = 0; w < W; ++w) equal += warp_a[w];
        __syncthreads();
    }
    const int equal_stay = equal - (int)equal_go;

    int gone = 0, seen_equal = 0;  // before this chunk
    for (int base = 0; base < p.max_pages; base += kEvictThreads) {
        const int i = base + tid;
        const bool in = i < p.max_pages;
        const int32_t id = in ? table[i] : -1;
        const float wt = in ? weight[i] : 0.f;
        const bool open = E > 0 && in && i >= lo && i < hi;
        const uint32_t key = weight_key(wt);
        const bool eq = open && key == prefix;
        // rank among the pages of weight `prefix`
        const unsigned me = __ballot_sync(~0u, eq);
        if (lane == 0) warp_a[warp] = __popc(me);
        __syncthreads();
        int before = seen_equal, all = 0;
        for (int w = 0; w < W; ++w) {
            if (w < warp) before += warp_a[w];
            all += warp_a[w];
        }
        before += __popc(me & ((1u << lane) - 1u));
        seen_equal += all;
        const bool go = open && (key < prefix || (eq && before >= equal_stay));
        const unsigned mg = __ballot_sync(~0u, go);
        if (lane == 0) warp_b[warp] = __popc(mg);
        __syncthreads();  // also: every entry of the chunk is read
        int at = gone, total = 0;
        for (int w = 0; w < W; ++w) {
            if (w < warp) at += warp_b[w];
            total += warp_b[w];
        }
        at += __popc(mg & ((1u << lane) - 1u));
        if (in) {
            if (go) {
                p.freed[row + at] = id;
            } else {
                p.block_table_out[row + i - at] = id;
                p.weight_out[row + i - at] = wt;
            }
        }
        gone += total;
    }
    __syncthreads();
    for (int i = tid; i < p.max_pages; i += kEvictThreads) {
        if (i >= p.max_pages - E) {
            p.block_table_out[row + i] = -1;
            p.weight_out[row + i] = 0.f;
        }
        if (i >= E) p.freed[row + i] = -1;
    }
    if (tid == 0) {
        p.seq_lens_out[n] = len - E * kPage;
        p.freed_count[n] = E;
    }
}

}  // namespace

cudaError_t launch_cache_append(const CacheAppendParams &p, int d, int dtype, cudaStream_t st) {
    return dtype == KDA_DT_BF16 ? launch_append<__nv_bfloat16>(p, d, st) : launch_append<float>(p, d, st);
}

cudaError_t launch_cache_evict(const CacheEvictParams &p, cudaStream_t st) {
    evict_kernel<<<(unsigned)p.batch, kEvictThreads, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace kda
