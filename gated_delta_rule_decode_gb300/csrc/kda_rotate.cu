// Norm of query and key heads and the rotation by their positions, in one pass.
//
//   y = x / sqrt(mean x^2 + eps) * w,   (a, b) -> factor (a cos t - b sin t, a sin t + b cos t)
//
// for the pairs (a, b) of the first rotary_dim channels, t = position * frequency.
//
// Every element is read and written once, so the bound is HBM.  A block goes from
// token to token: its row warps hold a token's rows (two pieces of 16 bytes a
// lane) and ask for the next one's before they work on them, while one or two
// warps more compute the next token's angles, once for all heads.  The pieces
// are chosen so that both channels of a pair lie in one lane.
//
// Angles: positions are whole numbers, so turns modulo one are exact in 64-bit
// fixed point: the table holds frequency / 2 pi in units of 2^-64 turns, one
// integer product gives the turn's fraction to position * 2^-65, and only what
// is left after taking out quarter turns becomes a float (2^-25 of at most an
// eighth of a turn), whose sine and cosine are the first terms of their series.
//
// Measured: 16 384 tokens of 32 and 8 heads, d = 128, bf16, 60 us, 5.6 TB/s (82 %
// of the copy's rate; the writes' share is half); 256 tokens 6.7 us, the launch
// and one chain of reads.
#include <cuda_bf16.h>
#include <stdint.h>

#include <algorithm>

#include "kda_attn_internal.h"
#include "kda_attn_math.cuh"

namespace kda {
namespace {

// For 16 384 tokens of 40 heads: 1, 2, 4 rows a lane 59.8 (at 10 warps), 60.2, 113 us;
// 16, 24, 32 warps an SM 66, 60, 96 (spills); 1, 2, 4, 8 tokens a barrier 61.6, 61.1,
// 60.2, 62.2.
constexpr int kMaxWarps = 6;     // of a block that hold rows
constexpr int kRowsHeld = 2;     // rows of a lane
constexpr int kWarpsPerSm = 24;  // by registers
constexpr int kTokens = 4;       // tokens whose angles a block computes together

// Pairs of floats, each by itself: as the paired instructions of sm_100 the same
// arithmetic took 91 us instead of 61, since pairs that come apart (a factor for
// both, a partner of the other sign) cost moves and registers.
__device__ __forceinline__ float2 fma_pair(float2 a, float2 b, float2 c) { return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y)); }
__device__ __forceinline__ float2 mul_pair(float2 a, float2 b) { return make_float2(a.x * b.x, a.y * b.y); }

// Pieces of 16 bytes of a row as pairs of floats.
template <typename T>
struct Piece;
template <>
struct Piece<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void get(const uint4 &u, float2 (&x)[2]) {
        x[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
        x[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
    }
    static __device__ __forceinline__ uint4 put(const float2 (&x)[2]) {
        return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x), __float_as_uint(x[1].y));
    }
};
template <>
struct Piece<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(const uint4 &u, float2 (&x)[4]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
    }
    static __device__ __forceinline__ uint4 put(const float2 (&x)[4]) {
        return make_uint4(pack_bf16(x[0].x, x[0].y), pack_bf16(x[1].x, x[1].y), pack_bf16(x[2].x, x[2].y),
                          pack_bf16(x[3].x, x[3].y));
    }
};

// cos and sin of position * frequency.
__device__ __forceinline__ float2 turn(int position, uint64_t frequency) {
    const uint64_t t = (uint64_t)(int64_t)position * frequency;   // 2^64 is a turn
    const uint32_t quarter = (uint32_t)((t + ((uint64_t)1 << 61)) >> 62);
    const int64_t rest = (int64_t)(t - ((uint64_t)quarter << 62));  // in -2^61 .. 2^61
    const float y = (float)(int)(rest >> 30) * (6.283185307179586f * 0x1p-34f), z = y * y;  // |y| <= pi / 4
    // y^11 / 11! and y^12 / 12! are below 2^-28
    float s = fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
    s = fmaf(z, s, 1.f / 120.f);
    s = fmaf(z, s, -1.f / 6.f);
    s = fmaf(z * y, s, y);
    float c = fmaf(z, -1.f / 3628800.f, 1.f / 40320.f);
    c = fmaf(z, c, -1.f / 720.f);
    c = fmaf(z, c, 1.f / 24.f);
    c = fmaf(z, c, -0.5f);
    c = fmaf(z, c, 1.f);
    const float cc = (quarter & 1) ? -s : c, ss = (quarter & 1) ? c : s;
    return (quarter & 2) ? make_float2(-cc, -ss) : make_float2(cc, ss);
}

// How the channels lie in lanes.  A lane holds two pieces of a row:
// kPairs: neighbours, so that the pairs (2 i, 2 i + 1) are its own; kHalves: those
// that hold (i, i + rot / 2), where rot / 2 is whole pieces, and neighbours of
// the channels behind rot; kLoose: neighbours, with the partners in shared memory.
enum Way { kPairs, kHalves, kLoose };

template <typename T, int HD, int WAY>
__global__ void __launch_bounds__(32 * (kMaxWarps + 2), kWarpsPerSm / (kMaxWarps + 2))
norm_rotate_kernel(const NormRotateParams p, int warps, int per) {
    using P = Piece<T>;
    constexpr int N = P::N, F = N / 2;                 // channels and pairs of floats of a piece
    constexpr int LPR = HD / (2 * N), RPW = 32 / LPR;  // lanes of a row, rows of a warp
    __shared__ __align__(16) float cs[2][kTokens][HD / 2], sn[2][kTokens][HD / 2];  // of tokens' pairs, two groups in turn
    __shared__ __align__(16) float weight[2][HD];
    __shared__ __align__(16) float loose[WAY == kLoose ? kMaxWarps : 1][WAY == kLoose ? RPW * HD : 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int half = p.rot / 2, rows = p.Hq + p.Hkv, tokens = (int)p.total_tokens;
    const int tok0 = blockIdx.x * per, step = gridDim.x * per;  // groups of `per` tokens

    if (warp >= warps) {
        // ---------------- angles, a token ahead of the rows
        const int first = tid - 32 * warps, threads = blockDim.x - 32 * warps;
        auto angles = [&](int tok, int buf) {
            const int count = min(per, tokens - tok);
            for (int i = first; i < half; i += threads) {
                const uint64_t f = p.turns[i];
                for (int k = 0; k < count; ++k) {
                    const float2 t = turn(p.positions[tok + k], f);
                    cs[buf][k][i] = t.x * p.factor;
                    sn[buf][k][i] = t.y * p.factor;
                }
            }
        };
        angles(tok0, 0);
        for (int i = first; i < HD; i += threads) {
            weight[0][i] = p.q_weight ? p.q_weight[i] : 1.f;
            weight[1][i] = p.k_weight ? p.k_weight[i] : 1.f;
        }
        int buf = 0;
        for (int tok = tok0; tok < tokens; tok += step) {
            __syncthreads();
            buf ^= 1;
            if (tok + step < tokens) angles(tok + step, buf);
        }
        return;
    }

    // ---------------- rows
    const int piece = lane % LPR, sub = lane / LPR;
    int c0 = 2 * N * piece, c1 = c0 + N;  // first channels of the lane's two pieces
    if (WAY == kHalves && piece < half / N) {
        c0 = N * piece;
        c1 = c0 + half;
    }
    const bool on = WAY != kHalves || piece < half / N;  // (kHalves: the lane's channels are turned)
    // the lane's rows, the same ones of every token: a query's or a key's, and whether there is one
    const T *src[kRowsHeld];
    T *dst[kRowsHeld];
    bool is_q[kRowsHeld], there[kRowsHeld];
#pragma unroll
    for (int i = 0; i < kRowsHeld; ++i) {
        const int r = ((int)blockIdx.y * kRowsHeld * warps + warp + i * warps) * RPW + sub;
        is_q[i] = r < p.Hq;
        there[i] = r < rows;
        src[i] = (is_q[i] ? static_cast<const T *>(p.q) + tok0 * p.q_stride + (int64_t)r * HD
                          : static_cast<const T *>(p.k) + tok0 * p.k_stride + (int64_t)(r - p.Hq) * HD) + c0;
        dst[i] = (is_q[i] ? static_cast<T *>(p.q_out) + tok0 * p.q_out_stride + (int64_t)r * HD
                          : static_cast<T *>(p.k_out) + tok0 * p.k_out_stride + (int64_t)(r - p.Hq) * HD) + c0;
    }
    uint4 raw[kRowsHeld][2];
    auto fetch = [&](int ahead) {
#pragma unroll
        for (int i = 0; i < kRowsHeld; ++i) {
            if (!there[i]) continue;
            const T *at = src[i] + (int64_t)ahead * (is_q[i] ? p.q_stride : p.k_stride);
            raw[i][0] = *reinterpret_cast<const uint4 *>(at);
            raw[i][1] = *reinterpret_cast<const uint4 *>(at + (c1 - c0));
        }
    };
#pragma unroll
    for (int i = 0; i < kRowsHeld; ++i) raw[i][0] = raw[i][1] = make_uint4(0, 0, 0, 0);
    fetch(0);
    int buf = 0, k = 0;  // the group's place, the token within it
    for (int ahead = 0; tok0 + ahead < tokens;) {
        const int next = k + 1 < per ? ahead + 1 : ahead + 1 - per + step;
        float2 x[kRowsHeld][2][F];
#pragma unroll
        for (int i = 0; i < kRowsHeld; ++i) {
            P::get(raw[i][0], x[i][0]);
            P::get(raw[i][1], x[i][1]);
        }
        if (tok0 + next < tokens) fetch(next);
        float f[kRowsHeld];  // 1 / the row's norm
#pragma unroll
        for (int i = 0; i < kRowsHeld; ++i) {
            float2 sq = make_float2(0.f, 0.f);
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < F; ++e) sq = fma_pair(x[i][u][e], x[i][u][e], sq);
            f[i] = sq.x + sq.y;
        }
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1)
#pragma unroll
            for (int i = 0; i < kRowsHeld; ++i) f[i] += __shfl_xor_sync(~0u, f[i], o);
        if (k == 0) __syncthreads();  // the group's angles are there, and the other group's no longer read
#pragma unroll
        for (int i = 0; i < kRowsHeld; ++i) {
            if ((is_q[i] ? p.q_weight : p.k_weight) != nullptr) {
                const float n = rsqrtf(f[i] * (1.f / HD) + p.eps);
                const float *w = weight[is_q[i] ? 0 : 1];
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int e = 0; e < F; e += 2) {
                        const float4 g = *reinterpret_cast<const float4 *>(w + (u == 0 ? c0 : c1) + 2 * e);
                        x[i][u][e] = mul_pair(mul_pair(x[i][u][e], make_float2(n, n)), make_float2(g.x, g.y));
                        x[i][u][e + 1] = mul_pair(mul_pair(x[i][u][e + 1], make_float2(n, n)), make_float2(g.z, g.w));
                    }
            }
        }
        if constexpr (WAY == kHalves) {
            if (on) {
#pragma unroll
                for (int e = 0; e < F; e += 2) {
                    const float4 c = *reinterpret_cast<const float4 *>(cs[buf][k] + c0 + 2 * e);
                    const float4 s = *reinterpret_cast<const float4 *>(sn[buf][k] + c0 + 2 * e);
#pragma unroll
                    for (int i = 0; i < kRowsHeld; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float2 a = x[i][0][e + j], b = x[i][1][e + j];
                            const float2 cc = j == 0 ? make_float2(c.x, c.y) : make_float2(c.z, c.w);
                            const float2 ss = j == 0 ? make_float2(s.x, s.y) : make_float2(s.z, s.w);
                            x[i][0][e + j] = fma_pair(a, cc, mul_pair(b, make_float2(-ss.x, -ss.y)));
                            x[i][1][e + j] = fma_pair(a, ss, mul_pair(b, cc));
                        }
                }
            }
        } else if constexpr (WAY == kPairs) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < F; ++e) {
                    const int at = (u == 0 ? c0 : c1) / 2 + e;
                    if (at >= half) continue;
                    const float c = cs[buf][k][at], s = sn[buf][k][at];
#pragma unroll
                    for (int i = 0; i < kRowsHeld; ++i) {
                        const float2 v = x[i][u][e];
                        x[i][u][e] = fma_pair(make_float2(v.x, v.y), make_float2(c, c), mul_pair(make_float2(v.y, v.x), make_float2(-s, s)));
                    }
                }
        } else {
#pragma unroll
            for (int i = 0; i < kRowsHeld; ++i) {
                float *mine = loose[warp] + sub * HD;
                __syncwarp();
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int e = 0; e < F; ++e) *reinterpret_cast<float2 *>(mine + (u == 0 ? c0 : c1) + 2 * e) = x[i][u][e];
                __syncwarp();
                auto turned = [&](float v, int ch) {
                    if (ch >= p.rot) return v;
                    const int at = ch < half ? ch : ch - half;
                    const float c = cs[buf][k][at], s = sn[buf][k][at];
                    return ch < half ? fmaf(v, c, -mine[ch + half] * s) : fmaf(mine[ch - half], s, v * c);
                };
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int e = 0; e < F; ++e) {
                        const int ch = (u == 0 ? c0 : c1) + 2 * e;
                        x[i][u][e] = make_float2(turned(x[i][u][e].x, ch), turned(x[i][u][e].y, ch + 1));
                    }
            }
        }
#pragma unroll
        for (int i = 0; i < kRowsHeld; ++i) {
            if (!there[i]) continue;
            T *at = dst[i] + (int64_t)ahead * (is_q[i] ? p.q_out_stride : p.k_out_stride);
            *reinterpret_cast<uint4 *>(at) = P::put(x[i][0]);
            *reinterpret_cast<uint4 *>(at + (c1 - c0)) = P::put(x[i][1]);
        }
        ahead = next;
        if (++k == per) {
            k = 0;
            buf ^= 1;
        }
    }
}

template <typename T, int HD>
cudaError_t launch_dim(const NormRotateParams &p, cudaStream_t st) {
    constexpr int N = Piece<T>::N, RPW = 32 / (HD / (2 * N));
    const int passes = (p.Hq + p.Hkv + RPW - 1) / RPW;
    const int warps = std::min(kMaxWarps, (passes + kRowsHeld - 1) / kRowsHeld);
    const int parts = (passes + kRowsHeld * warps - 1) / (kRowsHeld * warps);  // blocks that share a token's rows
    const int threads = 32 * (warps + (p.rot > 64 ? 2 : 1));
    const int64_t most = std::max(1, 152 * (32 * kWarpsPerSm / threads) / parts);
    const int per = (int)std::min<int64_t>(kTokens, (p.total_tokens + most - 1) / most);
    const int64_t blocks = std::min<int64_t>((p.total_tokens + per - 1) / per, most);
    static_assert(kTokens * 152 * kWarpsPerSm / 2 < 1 << 14, "a round's tokens behind the last: what the entry point leaves of 31 bits");
    if (parts > 65535) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks, (unsigned)parts);
    if (p.interleaved) norm_rotate_kernel<T, HD, kPairs><<<grid, threads, 0, st>>>(p, warps, per);
    else if (p.rot % (2 * N) == 0) norm_rotate_kernel<T, HD, kHalves><<<grid, threads, 0, st>>>(p, warps, per);
    else norm_rotate_kernel<T, HD, kLoose><<<grid, threads, 0, st>>>(p, warps, per);
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
