// Causal attention over packed prompts on the CUDA cores, in fp32 throughout.
//
//   o_i = sum_{j <= i} e^{s_ij - m_i} v_j / l_i,  s_ij = scale q_i . k_j,
//   m_i, l_i the running maximum and sum over the key blocks
//
// One CTA takes 64 tokens of one query head and walks the sequence's keys in
// blocks of 64.  Scores and outputs are register tiles (8 x 4 scores and
// 8 x d/8.. outputs a thread), operands come from shared memory in 16-byte
// pieces along the contraction, and pairs of products use the packed fp32
// instructions.  This path serves fp32 inputs, whose products the tensor
// cores would round.  Bound by the fp32 units.
#include <cuda_bf16.h>
#include <stdint.h>

#include "kda_attn_internal.h"
#include "kda_check.cuh"

namespace kda {
namespace {

constexpr int BM = 64, BN = 64, kThreads = 128;

template <typename T>
__device__ __forceinline__ float4 load4(const T *p);
template <>
__device__ __forceinline__ float4 load4<float>(const float *p) { return *reinterpret_cast<const float4 *>(p); }
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16 *p) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float *p, const float4 &x) { *reinterpret_cast<float4 *>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float4 &x) {
    __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
    uint2 u;
    u.x = *reinterpret_cast<uint32_t *>(&a);
    u.y = *reinterpret_cast<uint32_t *>(&b);
    *reinterpret_cast<uint2 *>(p) = u;
}

__device__ __forceinline__ float2 fma2(const float2 &a, const float2 &b, const float2 &c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(*reinterpret_cast<uint64_t *>(&d))
        : "l"(*reinterpret_cast<const uint64_t *>(&a)), "l"(*reinterpret_cast<const uint64_t *>(&b)),
          "l"(*reinterpret_cast<const uint64_t *>(&c)));
    return d;
}

template <int HD>
struct Tiles {
    static constexpr int LD = HD + 4;   // row stride in floats: rows 16 bytes apart modulo the banks
    static constexpr int LP = BN + 4;
    static constexpr int kK = BN * LD > BM * LP ? BN * LD : BM * LP;  // the keys' tile holds the weights later
    static constexpr int kBytes = (BM * LD + kK + BN * HD) * 4;
};

// Rows [first, first + 64) of src (token stride `stride`), zero from `end` on.
template <typename T, int HD, int LD>
__device__ __forceinline__ void load_tile(float *dst, const T *src, int64_t stride, int first, int end, int tid) {
    constexpr int C = HD / 4;
#pragma unroll
    for (int i = tid; i < 64 * C; i += kThreads) {
        const int r = i / C, c = i % C;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (first + r < end) x = load4<T>(src + (int64_t)(first + r) * stride + 4 * c);
        *reinterpret_cast<float4 *>(dst + r * LD + 4 * c) = x;
    }
}

template <typename T, int HD>
__global__ void __launch_bounds__(kThreads) prefill_simt_kernel(const AttnPrefillParams p) {
    using TL = Tiles<HD>;
    constexpr int LD = TL::LD, LP = TL::LP;
    constexpr int OC = HD / 16;  // output columns per thread, as groups of 4 (HD >= 64) or 2
    extern __shared__ __align__(16) float sm[];
    float *sq = sm, *sk = sq + BM * LD, *sv = sk + TL::kK, *sp = sk;
    const int tid = threadIdx.x;
    const int tx = tid & 15, ty = tid >> 4;  // 16 column groups, 8 row groups of 8 rows
    const int head = (int)(blockIdx.x % (unsigned)p.Hq), kvh = head / p.G;

    // the last tiles of a sequence have the most keys: they start first
    const int64_t unit = (int64_t)((gridDim.x - 1 - blockIdx.x) / (unsigned)p.Hq);
    int64_t tile;
    const int s = seq_of_unit(p.cu_seqlens, p.num_seqs, BM, 1, unit, tile);
    int t0, t1;
    if (!seq_range(p.cu_seqlens, s, p.total_tokens, p.err_flag, t0, t1)) return;
    if (tile < 0 || tile * BM >= t1 - t0) return;
    const int m0 = t0 + (int)tile * BM;  // first token of the tile
    const int m1 = min(m0 + BM, t1);
    const T *q = static_cast<const T *>(p.q) + (int64_t)head * HD;
    const T *k = static_cast<const T *>(p.k) + (int64_t)kvh * HD;
    const T *v = static_cast<const T *>(p.v) + (int64_t)kvh * HD;
    load_tile<T, HD, LD>(sq, q, p.q_stride, m0, m1, tid);

    const float sl2 = p.scale * 1.4426950408889634f;
    float o[8][OC], m[8], l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < OC; ++c) o[i][c] = 0.f;
    }
    for (int n0 = t0; n0 < m1; n0 += BN) {
        const bool diag = n0 + BN > m0;
        __syncthreads();  // the previous block's weights and values are read
        load_tile<T, HD, LD>(sk, k, p.k_stride, n0, m1, tid);
        load_tile<T, HD, HD>(sv, v, p.v_stride, n0, m1, tid);
        __syncthreads();
        // scores: rows 8 ty + i, columns tx + 16 j
        float2 acc[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int d = 0; d < HD; d += 4) {
            float4 b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4 *>(sk + (tx + 16 * j) * LD + d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 a = *reinterpret_cast<const float4 *>(sq + (8 * ty + i) * LD + d);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[i][j] = fma2(make_float2(a.x, a.y), make_float2(b[j].x, b[j].y), acc[i][j]);
                    acc[i][j] = fma2(make_float2(a.z, a.w), make_float2(b[j].z, b[j].w), acc[i][j]);
                }
            }
        }
        __syncthreads();  // the keys are read: their tile takes the weights
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = m0 + 8 * ty + i;
            float x[4], mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[j] = (acc[i][j].x + acc[i][j].y) * sl2;
                if (diag && n0 + tx + 16 * j > row) x[j] = -INFINITY;
                mx = fmaxf(mx, x[j]);
            }
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, w));
            const float mn = fmaxf(m[i], mx), use = mn == -INFINITY ? 0.f : mn;
            const float alpha = exp2f(m[i] - use);
            m[i] = mn;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float w = exp2f(x[j] - use);
                sum += w;
                sp[(8 * ty + i) * LP + tx + 16 * j] = w;
            }
            l[i] = fmaf(l[i], alpha, sum);
#pragma unroll
            for (int c = 0; c < OC; ++c) o[i][c] *= alpha;
        }
        __syncwarp();  // rows 8 ty..8 ty + 7 belong to one half of this warp
        // outputs: columns OC tx + c.  A key that some rows of the block do not
        // see must not reach them, whatever its value: in the diagonal block a
        // weight of exactly zero skips the product.
        const int kend = min(BN, m1 - n0);
        if (!diag) {
#pragma unroll 2
            for (int n = 0; n < BN; n += 4) {
                float4 w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = *reinterpret_cast<const float4 *>(sp + (8 * ty + i) * LP + n);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float2 b[OC / 2];
#pragma unroll
                    for (int c = 0; c < OC / 2; ++c)
                        b[c] = *reinterpret_cast<const float2 *>(sv + (n + e) * HD + OC * tx + 2 * c);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float x = e == 0 ? w[i].x : e == 1 ? w[i].y : e == 2 ? w[i].z : w[i].w;
#pragma unroll
                        for (int c = 0; c < OC / 2; ++c) {
                            float2 r = fma2(make_float2(x, x), b[c], make_float2(o[i][2 * c], o[i][2 * c + 1]));
                            o[i][2 * c] = r.x;
                            o[i][2 * c + 1] = r.y;
                        }
                    }
                }
            }
        } else {
            for (int n = 0; n < kend; ++n) {
                float b[OC];
#pragma unroll
                for (int c = 0; c < OC; ++c) b[c] = sv[n * HD + OC * tx + c];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float x = sp[(8 * ty + i) * LP + n];
                    if (n0 + n <= m0 + 8 * ty + i) {
#pragma unroll
                        for (int c = 0; c < OC; ++c) o[i][c] = fmaf(x, b[c], o[i][c]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float sum = l[i];
#pragma unroll
        for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(~0u, sum, w);
        const int row = m0 + 8 * ty + i;
        if (row >= m1) continue;
        const float f = 1.f / sum;
        T *dst = static_cast<T *>(p.out) + ((int64_t)row * p.Hq + head) * HD + OC * tx;
        if constexpr (OC >= 4) {
#pragma unroll
            for (int c = 0; c < OC; c += 4)
                store4(dst + c, make_float4(o[i][c] * f, o[i][c + 1] * f, o[i][c + 2] * f, o[i][c + 3] * f));
        } else {
#pragma unroll
            for (int c = 0; c < OC; ++c) dst[c] = T(o[i][c] * f);
        }
        if (p.lse && tx == 0) p.lse[(int64_t)row * p.Hq + head] = (m[i] + log2f(sum)) * 0.6931471805599453f;
    }
}

template <typename T, int HD>
cudaError_t launch_simt(const AttnPrefillParams &p, cudaStream_t st) {
    auto kern = prefill_simt_kernel<T, HD>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(kern), Tiles<HD>::kBytes, done);
    if (e != cudaSuccess) return e;
    const int64_t blocks = (p.total_tokens / BM + p.num_seqs) * p.Hq;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    kern<<<(unsigned)blocks, kThreads, Tiles<HD>::kBytes, st>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_dim(const AttnPrefillParams &p, int d, cudaStream_t st) {
    if (d == 128) return launch_simt<T, 128>(p, st);
    if (d == 64) return launch_simt<T, 64>(p, st);
    return launch_simt<T, 32>(p, st);
}

}  // namespace

cudaError_t launch_attn_prefill(const AttnPrefillParams &p, int d, int dtype, cudaStream_t st) {
    if (attn_prefill_tc_supported(d, dtype)) return launch_attn_prefill_tc(p, d, st);
    return dtype == KDA_DT_BF16 ? launch_dim<__nv_bfloat16>(p, d, st) : launch_dim<float>(p, d, st);
}

}  // namespace kda
