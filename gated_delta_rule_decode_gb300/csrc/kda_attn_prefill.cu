// Causal attention over packed prompts in fp32, on the CUDA cores.
//
//   o_i = sum_{j <= i} e^{s_ij - m_i} v_j / l_i,  s_ij = scale q_i . k_j,
//   m_i, l_i the running maximum and sum over the key blocks
//
// fp32 inputs keep fp32 products, which the tensor cores would round.  One CTA
// takes 32 tokens of one query head and walks the sequence's keys in blocks of
// 64, the next block's keys and values on their way (cp.async, two buffers)
// while it works on this one.  Scores and outputs are register tiles of 4 rows
// x 4 keys and 4 rows x d / 16 channels; operands come from shared memory in
// 16-byte pieces along the contraction, and pairs of products use the packed
// fp32 instructions.  Tiles of 32 rows rather than 64 because the longest tile
// of a call is its tail (1537 tokens in 3 prompts, 8 heads, d = 64: 68 us, 96
// with 64 rows and no copies ahead).  Bound by the fp32 units (4 d operations a
// score) where tiles are many, here by the longest tile's 18 blocks.
#include <stdint.h>

#include "kda_attn_internal.h"
#include "kda_attn_math.cuh"

namespace kda {
namespace {

constexpr int BM = 32, BN = 64, kThreads = 128;
constexpr int RM = 4;  // rows of a thread

template <int HD>
struct Tiles {
    static constexpr int LD = HD + 4;  // row stride in floats: rows 16 bytes apart modulo the banks
    static constexpr int LP = BN + 4;
    static constexpr int kKv = BN * LD + BN * HD;  // a buffer: keys, then values
    static constexpr int kBytes = (BM * LD + BM * LP + 2 * kKv) * 4;
};

// Starts the copy of rows [first, first + ROWS) of src (token stride `stride`)
// in 16-byte pieces; zero from `end` on.
template <int HD, int LD, int ROWS>
__device__ __forceinline__ void copy_tile(float *dst, const float *src, int64_t stride, int first, int end, int tid) {
    constexpr int C = HD / 4;
#pragma unroll
    for (int i = tid; i < ROWS * C; i += kThreads) {
        const int r = i / C, c = i % C;
        const bool in = first + r < end;
        const float *from = in ? src + (int64_t)(first + r) * stride + 4 * c : src;
        const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst + r * LD + 4 * c));
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(in ? 16 : 0) : "memory");
    }
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int HD>
__global__ void __launch_bounds__(kThreads) prefill_fp32_kernel(const AttnPrefillParams p) {
    using TL = Tiles<HD>;
    constexpr int LD = TL::LD, LP = TL::LP;
    constexpr int OC = HD / 16;  // output columns of a thread
    extern __shared__ __align__(16) float sm[];
    float *sq = sm, *sp = sq + BM * LD, *kv = sp + BM * LP;
    const int tid = threadIdx.x;
    const int tx = tid & 15, ty = tid >> 4;  // 16 column groups, 8 row groups
    const int head = (int)(blockIdx.x % (unsigned)p.Hq), kvh = head / p.G;

    // the last tiles of a sequence have the most keys: they start first
    const int64_t unit = (int64_t)((gridDim.x - 1 - blockIdx.x) / (unsigned)p.Hq);
    int64_t tile;
    const int s = seq_of_unit(p.cu_seqlens, p.num_seqs, BM, 1, unit, p.err_flag, tile);
    int t0, t1;
    if (!seq_range(p.cu_seqlens, s, p.total_tokens, p.err_flag, t0, t1)) return;
    if (tile < 0 || tile * BM >= t1 - t0) return;
    const int m0 = t0 + (int)tile * BM;  // first token of the tile
    const int m1 = min(m0 + BM, t1);
    const float *q = static_cast<const float *>(p.q) + (int64_t)head * HD;
    const float *k = static_cast<const float *>(p.k) + (int64_t)kvh * HD;
    const float *v = static_cast<const float *>(p.v) + (int64_t)kvh * HD;
    auto load_kv = [&](int b, int n0) {
        copy_tile<HD, LD, BN>(kv + b * TL::kKv, k, p.k_stride, n0, m1, tid);
        copy_tile<HD, HD, BN>(kv + b * TL::kKv + BN * LD, v, p.v_stride, n0, m1, tid);
        copies_commit();
    };
    copy_tile<HD, LD, BM>(sq, q, p.q_stride, m0, m1, tid);
    load_kv(0, t0);

    const float sl2 = p.scale * 1.4426950408889634f;
    float o[RM][OC], m[RM], l[RM];
#pragma unroll
    for (int i = 0; i < RM; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < OC; ++c) o[i][c] = 0.f;
    }
    int b = 0;
    for (int n0 = t0; n0 < m1; n0 += BN, b ^= 1) {
        const bool diag = n0 + BN > m0;
        if (n0 + BN < m1) {
            load_kv(b ^ 1, n0 + BN);
            copies_wait<1>();
        } else {
            copies_wait<0>();
        }
        __syncthreads();
        const float *sk = kv + b * TL::kKv, *sv = sk + BN * LD;
        // scores: rows RM ty + i, columns tx + 16 j
        float2 acc[RM][4];
#pragma unroll
        for (int i = 0; i < RM; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int d = 0; d < HD; d += 4) {
            float4 x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = *reinterpret_cast<const float4 *>(sk + (tx + 16 * j) * LD + d);
#pragma unroll
            for (int i = 0; i < RM; ++i) {
                const float4 a = *reinterpret_cast<const float4 *>(sq + (RM * ty + i) * LD + d);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[i][j] = fma2(make_float2(a.x, a.y), make_float2(x[j].x, x[j].y), acc[i][j]);
                    acc[i][j] = fma2(make_float2(a.z, a.w), make_float2(x[j].z, x[j].w), acc[i][j]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < RM; ++i) {
            const int row = m0 + RM * ty + i;
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
                sp[(RM * ty + i) * LP + tx + 16 * j] = w;
            }
            l[i] = fmaf(l[i], alpha, sum);
#pragma unroll
            for (int c = 0; c < OC; ++c) o[i][c] *= alpha;
        }
        __syncwarp();  // rows RM ty.. belong to one half of this warp
        // outputs: columns OC tx + c.  A key that some rows of the block do not
        // see must not reach them, whatever its value: in the diagonal block the
        // rows that do not see it skip the product.
        if (!diag) {
#pragma unroll 2
            for (int n = 0; n < BN; n += 4) {
                float4 w[RM];
#pragma unroll
                for (int i = 0; i < RM; ++i) w[i] = *reinterpret_cast<const float4 *>(sp + (RM * ty + i) * LP + n);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float2 y[OC / 2];
#pragma unroll
                    for (int c = 0; c < OC / 2; ++c)
                        y[c] = *reinterpret_cast<const float2 *>(sv + (n + e) * HD + OC * tx + 2 * c);
#pragma unroll
                    for (int i = 0; i < RM; ++i) {
                        const float x = e == 0 ? w[i].x : e == 1 ? w[i].y : e == 2 ? w[i].z : w[i].w;
#pragma unroll
                        for (int c = 0; c < OC / 2; ++c) {
                            const float2 r = fma2(make_float2(x, x), y[c], make_float2(o[i][2 * c], o[i][2 * c + 1]));
                            o[i][2 * c] = r.x;
                            o[i][2 * c + 1] = r.y;
                        }
                    }
                }
            }
        } else {
            const int kend = min(BN, m1 - n0);
#pragma unroll 2
            for (int n = 0; n < kend; ++n) {
                float y[OC];
#pragma unroll
                for (int c = 0; c < OC; ++c) y[c] = sv[n * HD + OC * tx + c];
#pragma unroll
                for (int i = 0; i < RM; ++i) {
                    const float x = sp[(RM * ty + i) * LP + n];
                    if (n0 + n <= m0 + RM * ty + i) {
#pragma unroll
                        for (int c = 0; c < OC; ++c) o[i][c] = fmaf(x, y[c], o[i][c]);
                    }
                }
            }
        }
        __syncthreads();  // the buffer is read: the block after next may come into it
    }
#pragma unroll
    for (int i = 0; i < RM; ++i) {
        float sum = l[i];
#pragma unroll
        for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(~0u, sum, w);
        const int row = m0 + RM * ty + i;
        if (row >= m1) continue;
        const float f = 1.f / sum;
        float *dst = static_cast<float *>(p.out) + ((int64_t)row * p.Hq + head) * HD + OC * tx;
#pragma unroll
        for (int c = 0; c < OC; c += 2) *reinterpret_cast<float2 *>(dst + c) = make_float2(o[i][c] * f, o[i][c + 1] * f);
        if (p.lse && tx == 0) p.lse[(int64_t)row * p.Hq + head] = (m[i] + log2f(sum)) * 0.6931471805599453f;
    }
}

template <int HD>
cudaError_t launch_fp32(const AttnPrefillParams &p, cudaStream_t st) {
    auto kern = prefill_fp32_kernel<HD>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(kern), Tiles<HD>::kBytes, done);
    if (e != cudaSuccess) return e;
    const int64_t blocks = (p.total_tokens / BM + p.num_seqs) * p.Hq;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    kern<<<(unsigned)blocks, kThreads, Tiles<HD>::kBytes, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_prefill(const AttnPrefillParams &p, int d, int dtype, cudaStream_t st) {
    if (dtype == KDA_DT_BF16) return launch_attn_prefill_tc(p, d, st);
    if (d == 128) return launch_fp32<128>(p, st);
    if (d == 64) return launch_fp32<64>(p, st);
    return launch_fp32<32>(p, st);
}

}  // namespace kda
