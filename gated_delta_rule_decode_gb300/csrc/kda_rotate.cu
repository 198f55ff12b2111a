// Norm of query and key heads and the rotation by their positions, in one pass.
//
//   y = x / sqrt(mean x^2 + eps) * w,   (a, b) -> factor (a cos t - b sin t, a sin t + b cos t)
//
// for the pairs (a, b) of the first rotary_dim channels, t = position * frequency.
//
// Every element is read and written once, so the bound is HBM.  A block takes a
// token: its warps hold the token's rows (16 bytes a lane) while the block
// computes the token's angles once for all heads.
//
// Angles: positions are whole numbers, so turns modulo one are exact in 64-bit
// fixed point: the table holds frequency / 2 pi in units of 2^-64 turns, one
// integer product gives the turn's fraction to position * 2^-65, and only what
// is left after taking out quarter turns becomes a float (2^-25 of at most an
// eighth of a turn).
#include <cuda_bf16.h>
#include <stdint.h>

#include <algorithm>

#include "kda_attn_internal.h"
#include "kda_attn_math.cuh"

namespace kda {
namespace {

constexpr int kMaxWarps = 8;
constexpr int kRowsHeld = 4;  // rows of a lane that are in flight together

template <typename T>
struct Vec;  // 16 bytes of a row
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void get(const uint4 &u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 put(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(const uint4 &u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 put(const float (&x)[8]) {
        return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    }
};

// cos and sin of position * frequency.
__device__ __forceinline__ float2 turn(int position, uint64_t frequency) {
    const uint64_t t = (uint64_t)(int64_t)position * frequency;   // 2^64 is a turn
    const uint32_t quarter = (uint32_t)((t + ((uint64_t)1 << 61)) >> 62);
    const int64_t rest = (int64_t)(t - ((uint64_t)quarter << 62));  // in -2^61 .. 2^61
    float s, c;
    sincospif((float)rest * 0x1p-63f, &s, &c);
    const float cc = (quarter & 1) ? -s : c, ss = (quarter & 1) ? c : s;
    return (quarter & 2) ? make_float2(-cc, -ss) : make_float2(cc, ss);
}

// How a lane finds the partners of its channels: kPairs: neighbours (2 i, 2 i + 1); kHalves: (i, i + rot / 2)
// where rot / 2 is whole pieces of 16 bytes, so that a lane's partners are another lane's; kLoose: other halves.
enum Way { kPairs, kHalves, kLoose };

template <typename T, int HD, int WAY>
__global__ void __launch_bounds__(32 * kMaxWarps) norm_rotate_kernel(const NormRotateParams p) {
    constexpr int N = Vec<T>::N;
    constexpr int LPR = HD / N, RPW = 32 / LPR;  // lanes of a row, rows of a warp
    __shared__ __align__(16) float cs[HD / 2], sn[HD / 2];
    __shared__ float loose[WAY == kLoose ? kMaxWarps : 1][WAY == kLoose ? RPW * HD : 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int64_t tok = blockIdx.x;
    const int piece = lane % LPR, c0 = piece * N;  // the lane's channels c0 .. c0 + N - 1
    const int half = p.rot / 2;
    const int rows = p.Hq + p.Hkv;
    const T *q = static_cast<const T *>(p.q) + tok * p.q_stride, *k = static_cast<const T *>(p.k) + tok * p.k_stride;
    T *qo = static_cast<T *>(p.q_out) + tok * p.q_out_stride, *ko = static_cast<T *>(p.k_out) + tok * p.k_out_stride;

    float c[N], s[N];  // of the lane's channels (of its pairs, in the first half)
    bool on[N];        // the channel is turned
    bool ready = false;
    for (int r0 = warp * RPW + lane / LPR; r0 - lane / LPR < rows; r0 += kRowsHeld * warps * RPW) {
        uint4 raw[kRowsHeld];
#pragma unroll
        for (int i = 0; i < kRowsHeld; ++i) {
            const int r = r0 + i * warps * RPW;
            raw[i] = make_uint4(0, 0, 0, 0);
            if (r < rows) raw[i] = *reinterpret_cast<const uint4 *>((r < p.Hq ? q + r * HD : k + (r - p.Hq) * HD) + c0);
        }
        if (!ready) {  // (once: every warp comes here in its first pass, while its rows are on their way)
            ready = true;
            for (int i = tid; i < half; i += blockDim.x) {
                const float2 t = turn(p.positions[tok], p.turns[i]);
                cs[i] = t.x * p.factor;
                sn[i] = t.y * p.factor;
            }
            __syncthreads();
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const int ch = c0 + e, i = WAY == kPairs ? ch / 2 : ch < half ? ch : ch - half;
                on[e] = ch < p.rot;
                c[e] = on[e] ? cs[i] : 1.f;
                s[e] = on[e] ? sn[i] : 0.f;
                if ((WAY == kPairs ? (e & 1) == 0 : ch < half)) s[e] = -s[e];
            }
        }
#pragma unroll
        for (int i = 0; i < kRowsHeld; ++i) {
            const int r = r0 + i * warps * RPW;
            if (r - lane / LPR >= rows) break;  // (by whole warps)
            float x[N], y[N];
            Vec<T>::get(raw[i], x);
            const float *w = r < p.Hq ? p.q_weight : p.k_weight;
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < N; ++e) sum = fmaf(x[e], x[e], sum);
#pragma unroll
            for (int o = 1; o < LPR; o <<= 1) sum += __shfl_xor_sync(~0u, sum, o);
            if (w != nullptr) {
                const float f = rsqrtf(sum * (1.f / HD) + p.eps);
#pragma unroll
                for (int e = 0; e < N; e += 4) {
                    const float4 g = *reinterpret_cast<const float4 *>(w + c0 + e);
                    x[e] = x[e] * f * g.x; x[e + 1] = x[e + 1] * f * g.y;
                    x[e + 2] = x[e + 2] * f * g.z; x[e + 3] = x[e + 3] * f * g.w;
                }
            }
            if constexpr (WAY == kLoose) {
                __syncwarp();
#pragma unroll
                for (int e = 0; e < N; ++e) loose[warp][(lane / LPR) * HD + c0 + e] = x[e];
                __syncwarp();
            }
#pragma unroll
            for (int e = 0; e < N; ++e) {
                float other;  // the channel's partner
                if constexpr (WAY == kPairs) other = x[e ^ 1];
                else if constexpr (WAY == kHalves) {
                    const int far = half / N;
                    other = __shfl_sync(~0u, x[e], (lane + (c0 < half ? far : c0 < p.rot ? -far : 0)) & 31);
                } else {
                    const int ch = c0 + e;
                    other = loose[warp][(lane / LPR) * HD + (ch < half ? ch + half : ch < p.rot ? ch - half : ch)];
                }
                y[e] = on[e] ? fmaf(x[e], c[e], other * s[e]) : x[e];
            }
            if (r < rows) *reinterpret_cast<uint4 *>((r < p.Hq ? qo + r * HD : ko + (r - p.Hq) * HD) + c0) = Vec<T>::put(y);
        }
    }
}

template <typename T, int HD>
cudaError_t launch_dim(const NormRotateParams &p, cudaStream_t st) {
    constexpr int N = Vec<T>::N, RPW = 32 / (HD / N);
    const int passes = (p.Hq + p.Hkv + RPW - 1) / RPW;
    const int threads = 32 * std::min(kMaxWarps, (passes + kRowsHeld - 1) / kRowsHeld);
    const unsigned blocks = (unsigned)p.total_tokens;
    if (p.interleaved) norm_rotate_kernel<T, HD, kPairs><<<blocks, threads, 0, st>>>(p);
    else if (p.rot % (2 * N) == 0) norm_rotate_kernel<T, HD, kHalves><<<blocks, threads, 0, st>>>(p);
    else norm_rotate_kernel<T, HD, kLoose><<<blocks, threads, 0, st>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch(const NormRotateParams &p, int d, cudaStream_t st) {
    if (d == 128) return launch_dim<T, 128>(p, st);
    if (d == 64) return launch_dim<T, 64>(p, st);
    return launch_dim<T, 32>(p, st);
}

}  // namespace

cudaError_t launch_norm_rotate(const NormRotateParams &p, int d, int dtype, cudaStream_t s) {
    return dtype == KDA_DT_BF16 ? launch<__nv_bfloat16>(p, d, s) : launch<float>(p, d, s);
}

}  // namespace kda
