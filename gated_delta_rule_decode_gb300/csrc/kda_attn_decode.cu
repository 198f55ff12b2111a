// Attention of a few query tokens per sequence over the 8-bit paged cache.
//
//   s_j = scale q . k_j,  o = sum_j e^{s_j - m} v_j / sum_j e^{s_j - m}
//
// The cache is read once, so the bound is HBM: 2 d bytes per position and kv
// head.  Everything else is arranged around a steady stream of pages:
//
//  * Work is counted in pages: the items (sequence, kv head, block of 8 NB MT
//    query rows) of the batch are laid end to end and cut into equal ranges,
//    one per worker, so ragged batches and single long sequences balance
//    alike.  A worker is a CTA of MT warps; an item that a worker holds
//    entirely is finished by it, one that is cut leaves partial results
//    (o, m, l) that join_kernel adds up in a fixed order.  There is one worker
//    per place on the GPU (see make_layout).
//  * The G query heads of a kv head and the window's tokens are the rows of
//    one tile, so a page is read once for all of them.
//  * Each worker keeps a ring of shared-memory slots filled by bulk copies; a
//    page's keys and values are one contiguous block each.
//  * Products run as m16n8k16 fp16 MMAs with fp32 accumulation, transposed:
//    S^T = K Q^T and O^T = V^T P^T, so that the 16-row operand is the page and
//    the 8-column one the query rows, of which there are few.  e4m3 values are
//    exact in fp16.  A query row is scaled by a power of two into fp16's
//    range, which is exact for bf16 inputs (elements below 2^-28 of the row's
//    largest are rounded); fp32 inputs take a second fp16 term for the rest.
//    The weights go into fp16 times their page's value scale, the row's largest
//    such product in 2^14..2^15 (see kda_attn_decode.cuh), so that fp16 holds
//    them down to 2^-39 of it; fp32 takes a second term here as well.
//  * The contraction orders of both products are permuted so that a thread's
//    operand bytes are contiguous 16-byte pieces: thread t of a quad holds
//    channels 16 t.. of a key row and positions 16 t.. of a value channel,
//    and row r of the score tile i stands for position 16 (r % 8 / 2) + 4 i +
//    2 (r / 8) + r % 2; a transposed 8 x 8 move then makes score fragments the
//    second product's operand.  (The pages' value layout, a row of positions
//    per channel, is there for this.)
//  * Each page's product is accumulated from zero and added to the output in
//    fp32 round-to-nearest, because the tensor cores truncate when they add.
//
// Measured (d = 128, bf16): 64 sequences of up to 32 768 positions, 32 heads
// over 8, 381 us, 5.6 TB/s; one sequence of 102 400, 51 us (the join's share
// about 9), 7 pages a worker.  Above 16 rows a warp's conversions are repeated by
// each of MT warps: bf16 calls go to kda_attn_decode_tc.cu there (see
// make_layout); fp32 and d = 32 stay.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <type_traits>

#include "kda_attn_decode.cuh"
#include "kda_attn_internal.h"
#include "kda_bulk.cuh"

namespace kda {
namespace {

using namespace dec;

// Warps per SM, by registers and by shared memory (the rings).
__host__ __device__ constexpr int warps_per_sm(int NB) { return NB == 1 ? 12 : 8; }
// Short rows of the block table are not cut: a worker per item, no partial
// results and no join.  That needs enough items to fill the GPU; with fewer,
// the cut gives each a share of the SMs.  Cut and whole took, at 8 and at 16
// pages: with 512 items of up to 8 rows 43.6 and 31.4, 58 and 48 us; with 128 of
// them 23.2 and 27.3, 35.5 and 39.6; 64 items of kda_attn_decode_tc.cu 33.5 and
// 21.1, 37.5 and 29.3. At 32 pages whole
// still gains 3 to 16 % with that many items (77 and 74 us; 103 and 87), and its
// longest item sets the time of a ragged batch, so the rule stops before.
constexpr int64_t kWholePages = 16;
constexpr int64_t kWholeItems = 512, kWholeItemsTc = 64;
constexpr float kPScale = 32768.f;  // fp16 scale of the weights

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transpose of an 8 x 8 matrix of 16-bit values (two per thread).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <typename T>
__device__ __forceinline__ float load1(const T *p);
template <>
__device__ __forceinline__ float load1<float>(const float *p) { return *p; }
template <>
__device__ __forceinline__ float load1<__nv_bfloat16>(const __nv_bfloat16 *p) { return __bfloat162float(*p); }

// A bounded wait by all lanes of a warp with one answer.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, int64_t phase) {
    return __all_sync(~0u, mbar_wait(bar, (uint32_t)phase & 1u));
}

// Per-thread share of a contraction step: byte i (0..HD/4-1) of the thread's
// part of a row is channel chan(t, i).
template <int HD>
__device__ __forceinline__ int chan(int t, int i) {
    if constexpr (HD == 128) return i < 16 ? 16 * t + i : 64 + 16 * t + (i - 16);
    else return (HD / 4) * t + i;
}

template <typename T, int HD>
__device__ __forceinline__ void load_row(const T *row, int t, bool valid, float (&x)[HD / 4]) {
#pragma unroll
    for (int j = 0; j < HD / 4; ++j) x[j] = valid ? load1<T>(row + chan<HD>(t, j)) : 0.f;
}

template <int HD, int NB, int MT>
struct Smem {
    static constexpr int kHalf = HD * kPage;  // bytes of a page's keys (or values)
    static constexpr int kSlots = (NB == 1 ? 2 : 3) * MT * (128 / HD);  // 16 or 24 KiB per warp
    static constexpr int kRingBytes = kSlots * kHalf;
    static_assert(kSlots / 2 + 1 < kMeta / 2, "copies run at most a batch ahead of the page metadata in use");
    static constexpr int kBytes = 128 + kRingBytes + 2 * kSlots * 8 + kMeta * (int)sizeof(PageMeta);
};

template <typename T, int HD, int NB, int MT>
__global__ void __launch_bounds__(32 * MT, warps_per_sm(NB) / MT) decode_attn_kernel(const AttnDecodeParams p, const Layout lay) {
    using S = Smem<HD, NB, MT>;
    constexpr int TERMS = sizeof(T) == 4 ? 2 : 1;
    constexpr int KS = HD / 16;    // contraction steps of the score product
    constexpr int DT = HD / 16;    // channel tiles of the output
    constexpr int R = 8 * NB * MT; // rows of an item
    constexpr int SL = S::kSlots;
    constexpr int kThreads = 32 * MT;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *ring = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    uint64_t *full = reinterpret_cast<uint64_t *>(ring + S::kRingBytes), *empty = full + SL;
    PageMeta *meta = reinterpret_cast<PageMeta *>(empty + SL);
    __shared__ int64_t warp_sum[MT];
    __shared__ Cursor start;

    const int tid = threadIdx.x, lane = tid & 31, mt = tid >> 5;  // mt: row tile of the warp
    const int g = lane >> 2, t = lane & 3;
    const int rows_all = p.D * p.G, PR = lay.PR, RB = lay.RB, HR = p.Hkv * RB;
    const int64_t w = blockIdx.x;
    float *ws = static_cast<float *>(p.workspace);

    for (int i = tid; i < SL; i += kThreads) {
        mbar_init(full + i, 1);    // the copy's bytes
        mbar_init(empty + i, MT);  // the warps
    }
    fence_barrier_init();

    int64_t U, W, u0, u1;
    find_range<T, HD, MT>(p, HR, lay.whole, warp_sum, &start, U, W, u0, u1);
    if (u0 >= u1) return;
    const int64_t count = u1 - u0;

    // ---- the copies: number c brings the keys (even) or values (odd) of unit
    // c / 2 into slot c % SL.  The worker's first warp looks up the pages of 32
    // units at a time, one per lane.
    Cursor cur = start, fetch_cur = cur;
    int64_t fetched = 0, issued = 0;
    auto fetch = [&]() {
        Cursor c = fetch_cur;
        if (fetched + lane < count) {
            const Unit un = locate(p, HR, c, u0 + fetched + lane);
            const int h = un.hr / RB;
            const int id = p.block_table[(int64_t)un.n * p.max_pages + un.page];
            meta[(fetched + lane) % kMeta] = page_meta(p, id, h);
        }
        const int from = (int)min((int64_t)31, count - 1 - fetched);
        fetch_cur.n = __shfl_sync(~0u, c.n, from);
        fetch_cur.base = __shfl_sync(~0u, c.base, from);
        fetched += 32;
        __syncwarp();
    };
    auto issue = [&](int64_t c) {  // by the whole first warp; slot c % SL is free
        if (c >= 2 * count) return;
        if ((c >> 1) >= fetched) fetch();
        issued = c + 1;
        if (lane != 0) return;
        const int slot = (int)(c % SL), block = meta[(c >> 1) % kMeta].block;
        uint64_t *bar = full + slot;
        if (block < 0) {
            mbar_arrive(bar);
            return;
        }
        mbar_arrive_expect_tx(bar, S::kHalf);
        bulk_g2s(ring + slot * S::kHalf, ((c & 1) ? p.v_pages : p.k_pages) + (int64_t)block * S::kHalf, S::kHalf, bar);
    };
    if (mt == 0)
        for (int c = 0; c < SL; ++c) issue(c);

    // ---- the range, item by item
    int64_t i = 0;
    bool timeout = false;
    while (i < count && !timeout) {
        const Unit un = locate(p, HR, cur, u0 + i);
        const int h = un.hr / RB, rb = un.hr % RB;
        const int pages_here = (int)min((int64_t)(un.pages - un.page), count - i);
        const int row0 = rb * R + mt * 8 * NB;  // the warp's first row
        // operand: row g of each tile; accumulators: rows 2 t and 2 t + 1
        uint32_t qb[TERMS][NB][KS][2];
        float qs[NB][2];
        int limit[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int r = row0 + 8 * nb + g;
            const bool valid = r < rows_all;
            const int tok = valid ? r / p.G : 0, gi = valid ? r - tok * p.G : 0;
            const T *src = static_cast<const T *>(p.q) + ((int64_t)un.n * p.D + tok) * p.q_stride +
                           (int64_t)(h * p.G + gi) * HD;
            float x[HD / 4], amax = 0.f;
            load_row<T, HD>(src, t, valid, x);
#pragma unroll
            for (int j = 0; j < HD / 4; ++j) amax = fmaxf(amax, fabsf(x[j]));
            amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
            // the row times 2^(14 - ex): its largest element in 2^14..2^15
            int ex = (int)(__float_as_uint(amax) >> 23) - 127;
            ex = ex < -100 ? -100 : ex > 127 ? 127 : ex;  // (above 127: infinities and NaN stay what they are)
            const float mul = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
            const float back = __uint_as_float((uint32_t)(127 - 14 + ex) << 23) * p.scale * kLog2e;
#pragma unroll
            for (int st = 0; st < KS; ++st)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const float x0 = x[4 * st + 2 * b] * mul, x1 = x[4 * st + 2 * b + 1] * mul;
                    qb[0][nb][st][b] = pack_f16(x0, x1);
                    if constexpr (TERMS == 2) {
                        const float2 hi = unpack_f16(qb[0][nb][st][b]);
                        qb[1][nb][st][b] = pack_f16(x0 - hi.x, x1 - hi.y);
                    }
                }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                qs[nb][e] = __shfl_sync(~0u, back, 4 * (2 * t + e));
                const int re = row0 + 8 * nb + 2 * t + e;
                limit[nb][e] = re < rows_all ? un.len - p.D + 1 + re / p.G : 0;
            }
        }
        float o[NB][DT][4];
        float m[NB][2], l[NB][2];
        int unit[NB][2];  // the exponent that o is counted in
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int dt = 0; dt < DT; ++dt)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[nb][dt][c] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[nb][e] = -INFINITY;
                l[nb][e] = 0.f;
                unit[nb][e] = kNoUnit;
            }
        }
        const int window0 = un.len - p.D + 1;  // first position that some row does not see

        for (int pi = 0; pi < pages_here; ++pi, ++i) {
            const int page = un.page + pi;
            const int pos0 = page * kPage;
            // ---- scores
            const int64_t ck = 2 * i, cv = 2 * i + 1;
            const int sk = (int)(ck % SL), sv = (int)(cv % SL);
            if (!warp_wait(full + sk, ck / SL)) { timeout = true; break; }
            const PageMeta pm = meta[i % kMeta];
            const int vexp = exponent_of(pm.vs);
            const bool have = pm.block >= 0;
            const bool tail = pos0 + kPage > window0 || !have;
            float s[NB][4][4];
            {
                const unsigned char *kb = ring + sk * S::kHalf + (16 * (g >> 1) + (g & 1)) * HD;
                // two score tiles at a time, so that several chains of products run side by side
#pragma unroll
                for (int i2 = 0; i2 < 4; i2 += 2) {
                    uint32_t kw[2][2][HD / 16];
#pragma unroll
                    for (int ii = 0; ii < 2; ++ii)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const unsigned char *row = kb + (4 * (i2 + ii) + 2 * hf) * HD;
                            if constexpr (HD >= 64) {
#pragma unroll
                                for (int b = 0; b < HD / 64; ++b) {
                                    const uint4 a = *reinterpret_cast<const uint4 *>(row + 64 * b + 16 * t);
                                    kw[ii][hf][4 * b] = a.x; kw[ii][hf][4 * b + 1] = a.y;
                                    kw[ii][hf][4 * b + 2] = a.z; kw[ii][hf][4 * b + 3] = a.w;
                                }
                            } else {
                                const uint2 a = *reinterpret_cast<const uint2 *>(row + 8 * t);
                                kw[ii][hf][0] = a.x; kw[ii][hf][1] = a.y;
                            }
                        }
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int ii = 0; ii < 2; ++ii)
#pragma unroll
                            for (int c = 0; c < 4; ++c) s[nb][i2 + ii][c] = 0.f;
#pragma unroll
                    for (int st = 0; st < KS; ++st)
#pragma unroll
                        for (int ii = 0; ii < 2; ++ii) {
                            uint32_t a0, a1, a2, a3;
                            e4m3x4_to_f16(kw[ii][0][st], a0, a2);
                            e4m3x4_to_f16(kw[ii][1][st], a1, a3);
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                                for (int tm = 0; tm < TERMS; ++tm)
                                    mma16816(s[nb][i2 + ii], a0, a1, a2, a3, qb[tm][nb][st][0], qb[tm][nb][st][1]);
                        }
                }
            }
            __syncwarp();
            if (MT > 1 && lane == 0) mbar_arrive(empty + sk);
            // the next copy into the slot that is free now
            if (mt == 0 && ck + SL < 2 * count) {
                if (MT > 1 && !warp_wait(empty + sk, ck / SL)) { timeout = true; break; }
                issue(ck + SL);
            }
            // ---- softmax
            if (tail) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int ti = 0; ti < 4; ++ti)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int pos = pos0 + 16 * (g >> 1) + 4 * ti + (c & 2) + (g & 1);
                            if (!have || pos >= limit[nb][c & 1]) s[nb][ti][c] = -INFINITY;
                        }
            }
            uint32_t pb[TERMS][NB][4][2];
            float alpha[NB][2];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                float f[2], use[2], rs[2];
                float before[2];
                int bias[2], to[2];  // of the weights' exponents: 2^15 stands for the largest contribution
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    f[e] = fmaxf(qs[nb][e] * pm.ks, 1e-37f);  // positive, so that -inf stays -inf
                    float mx = -INFINITY;
#pragma unroll
                    for (int ti = 0; ti < 4; ++ti) mx = fmaxf(mx, fmaxf(s[nb][ti][e], s[nb][ti][2 + e]));
                    mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 16)) * f[e];
                    before[e] = m[nb][e];
                    m[nb][e] = fmaxf(m[nb][e], mx);
                    use[e] = m[nb][e] == -INFINITY ? 0.f : m[nb][e];
                    to[e] = max(unit[nb][e] + __float2int_ru(fmaxf(before[e] - use[e], kFarBelow)), contribution(vexp, mx, use[e]));
                    bias[e] = 15 + vexp - to[e];
                    alpha[nb][e] = 1.f;
                }
                if (__any_sync(~0u, before[0] != m[nb][0] || before[1] != m[nb][1] || to[0] != unit[nb][0] || to[1] != unit[nb][1])) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 by = moved(before[e], use[e], unit[nb][e], to[e]);
                        l[nb][e] *= by.x;
                        alpha[nb][e] = by.y;
                        unit[nb][e] = to[e];
                    }
                }
                rs[0] = rs[1] = 0.f;
                const float b0 = (float)bias[0] - use[0], b1 = (float)bias[1] - use[1];
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (bias[e] < kApart) {  // the sum apart: these weights may vanish next to a larger contribution
#pragma unroll
                        for (int ti = 0; ti < 4; ++ti)
                            rs[e] += ex2(fmaf(s[nb][ti][e], f[e], -use[e])) + ex2(fmaf(s[nb][ti][2 + e], f[e], -use[e]));
                    }
#pragma unroll
                for (int ti = 0; ti < 4; ++ti) {
                    float w[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) w[c] = ex2(fmaf(s[nb][ti][c], f[c & 1], (c & 1) ? b1 : b0));
                    if (bias[0] >= kApart) rs[0] += w[0] + w[2];
                    if (bias[1] >= kApart) rs[1] += w[1] + w[3];
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const uint32_t x = pack_f16(w[2 * hf], w[2 * hf + 1]);
                        pb[0][nb][ti][hf] = transpose8x8(x);
                        if constexpr (TERMS == 2) {
                            const float2 hi = unpack_f16(x);
                            pb[1][nb][ti][hf] = transpose8x8(pack_f16(w[2 * hf] - hi.x, w[2 * hf + 1] - hi.y));
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (bias[e] >= kApart) rs[e] *= pow2(-bias[e]);
                    l[nb][e] += rs[e];
                }
                if (p.weight_out != nullptr) {  // the page's share, relative to the maximum so far
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = rs[e];
                        x += __shfl_xor_sync(~0u, x, 4);
                        x += __shfl_xor_sync(~0u, x, 8);
                        x += __shfl_xor_sync(~0u, x, 16);
                        const int r = row0 + 8 * nb + 2 * t + e;
                        if (g == 0 && r < rows_all) {
                            const int64_t qrow = ((int64_t)un.n * p.D + r / p.G) * p.Hq + h * p.G + r % p.G;
                            ws[lay.page_w + qrow * p.max_pages + page] = x > 0.f ? log2f(x) + use[e] : -INFINITY;
                        }
                    }
                }
            }
            // ---- output
            if (!warp_wait(full + sv, cv / SL)) { timeout = true; break; }
            const unsigned char *vb = ring + sv * S::kHalf + g * kPage + 16 * t;
#pragma unroll
            for (int d2 = 0; d2 < DT; d2 += 2) {
                uint32_t vw[2][2][4];
                int nan_at[2][2] = {{kPage, kPage}, {kPage, kPage}};
#pragma unroll
                for (int dd = 0; dd < 2; ++dd)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const uint4 a = *reinterpret_cast<const uint4 *>(vb + (16 * (d2 + dd) + 8 * hf) * kPage);
                        vw[dd][hf][0] = a.x; vw[dd][hf][1] = a.y; vw[dd][hf][2] = a.z; vw[dd][hf][3] = a.w;
                    }
                if (tail) {
                    // bytes past the end (whatever they hold) count as zero, and so do
                    // the window's NaN bytes, which only the rows that see them get
                    const int left = have ? un.len - pos0 : 0;  // positions of the page that exist
                    const int seen = window0 - pos0;            // positions that every row sees
#pragma unroll
                    for (int dd = 0; dd < 2; ++dd)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
                            for (int st = 0; st < 4; ++st)
                                nan_at[dd][hf] = min(nan_at[dd][hf], mask_word(vw[dd][hf][st], 16 * t + 4 * st, left, seen));
                            nan_at[dd][hf] = min(nan_at[dd][hf], __shfl_xor_sync(~0u, nan_at[dd][hf], 1));
                            nan_at[dd][hf] = min(nan_at[dd][hf], __shfl_xor_sync(~0u, nan_at[dd][hf], 2));
                        }
                }
                float c[NB][2][4];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int dd = 0; dd < 2; ++dd)
#pragma unroll
                        for (int k = 0; k < 4; ++k) c[nb][dd][k] = 0.f;
#pragma unroll
                for (int st = 0; st < 4; ++st)
#pragma unroll
                    for (int dd = 0; dd < 2; ++dd) {
                        uint32_t a0, a1, a2, a3;
                        e4m3x4_to_f16(vw[dd][0][st], a0, a2);
                        e4m3x4_to_f16(vw[dd][1][st], a1, a3);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int tm = 0; tm < TERMS; ++tm)
                                mma16816(c[nb][dd], a0, a1, a2, a3, pb[tm][nb][st][0], pb[tm][nb][st][1]);
                    }
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int dd = 0; dd < 2; ++dd)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            float &x = o[nb][d2 + dd][k];
                            x = fmaf(x, alpha[nb][k & 1], c[nb][dd][k]);
                            const int at = nan_at[dd][k >> 1];
                            if (tail && at < kPage && pos0 + at < limit[nb][k & 1]) x = NAN;
                        }
            }
            __syncwarp();
            if (MT > 1 && lane == 0) mbar_arrive(empty + sv);
            if (mt == 0 && cv + SL < 2 * count) {
                if (MT > 1 && !warp_wait(empty + sv, cv / SL)) { timeout = true; break; }
                issue(cv + SL);
            }
        }
        if (timeout) break;
        if (i >= count) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

        // ---- the item's end
        const bool whole = un.page == 0 && pages_here == un.pages;
        const int64_t slot = 2 * w + (un.page == 0 ? 1 : 0);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            float f[2], in[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = l[nb][e];
                x += __shfl_xor_sync(~0u, x, 4);
                x += __shfl_xor_sync(~0u, x, 8);
                x += __shfl_xor_sync(~0u, x, 16);
                const int r = row0 + 8 * nb + 2 * t + e;
                f[e] = x == 0.f ? 0.f : whole ? 1.f / x : 1.f;
                in[e] = pow2(unit[nb][e]) * (1.f / kPScale);
                if (r >= rows_all || g != 0) continue;
                if (whole) {
                    const int64_t qrow = ((int64_t)un.n * p.D + r / p.G) * p.Hq + h * p.G + r % p.G;
                    const float lse2 = x == 0.f ? -INFINITY : m[nb][e] + log2f(x);
                    if (p.lse) p.lse[qrow] = lse2 * kLn2;
                    if (p.weight_out) ws[lay.lse2 + qrow] = lse2;
                } else {
                    ws[lay.part_m + slot * PR + r - rb * R] = m[nb][e];
                    ws[lay.part_l + slot * PR + r - rb * R] = x;
                }
            }
            if (whole && sizeof(T) == 2) {
                // rows g, channel pairs 2 t: four lanes write 16 bytes of a row
                const int r = row0 + 8 * nb + g;
                T *dst = static_cast<T *>(p.out) +
                         (((int64_t)un.n * p.D + r / p.G) * p.Hq + h * p.G + r % p.G) * HD + 2 * t;
#pragma unroll
                for (int dt = 0; dt < DT; ++dt)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const float x0 = f[0] == 0.f ? 0.f : o[nb][dt][2 * hf] * in[0] * f[0];
                        const float x1 = f[1] == 0.f ? 0.f : o[nb][dt][2 * hf + 1] * in[1] * f[1];
                        const uint32_t y = transpose8x8(pack_bf16(x0, x1));
                        if (r < rows_all) *reinterpret_cast<uint32_t *>(dst + 16 * dt + 8 * hf) = y;
                    }
            } else {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = row0 + 8 * nb + 2 * t + e;
                    if (r >= rows_all) continue;
                    float *dst = whole ? static_cast<float *>(p.out) +
                                             (((int64_t)un.n * p.D + r / p.G) * p.Hq + h * p.G + r % p.G) * HD
                                       : ws + lay.part_o + (slot * PR + r - rb * R) * HD;
#pragma unroll
                    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf)
                            dst[16 * dt + 8 * hf + g] = f[e] == 0.f ? 0.f : o[nb][dt][2 * hf + e] * in[e] * f[e];
                }
            }
        }
        if (un.page == 0 && tid == 0 && !lay.whole) write_desc(ws, lay, un, cur, HR, whole, W, U);
    }
    if (timeout && p.err_flag) atomicOr(p.err_flag, KDA_DEVERR_TIMEOUT);
    if (timeout && mt == 0)  // the copies in flight land before the CTA's memory goes
        for (int64_t c = issued > SL ? issued - SL : 0; c < issued; ++c)
            mbar_wait_drain(full + c % SL, (uint32_t)(c / SL) & 1u);
}

// Adds up the parts of the cut items: a block takes an item and a row (or,
// where there are many items, its rows in turn).  Groups of HD / 4 threads take
// every kJoinThreads / (HD / 4)-th part; their sums are added in order.
// Blocks of 512 threads where items have many parts, of 128 where they have few.
constexpr int64_t kJoinBlocks = 16384;

template <typename T, int HD, int kJoinThreads>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const AttnDecodeParams p, const Layout lay) {
    constexpr int TPR = HD / 4, GR = kJoinThreads / TPR;
    __shared__ float wmax[kJoinThreads / 32];
    __shared__ float4 so[GR][TPR];
    __shared__ float sl[GR];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float *ws = static_cast<float *>(p.workspace);
    const int RB = lay.RB, R = lay.R, PR = lay.PR;
    const int HR = p.Hkv * RB, n = blockIdx.x / HR, hr = blockIdx.x % HR;
    if (p.seq_lens[n] <= 0) return;
    const int2 desc = *reinterpret_cast<const int2 *>(ws + lay.desc + 2 * (int64_t)blockIdx.x);
    // (a worker that gave up waiting leaves no or stale entries)
    if (desc.x < 0 || desc.x >= desc.y || desc.y >= lay.workers) return;
    const int64_t w = desc.x;
    const int parts = desc.y - desc.x + 1;
    const int rows_all = p.D * p.G;
    const int h = hr / RB, rb = hr % RB;
    const int tid = threadIdx.x;
    for (int r = blockIdx.y; r < PR && rb * R + r < rows_all; r += gridDim.y) {
        const int row = rb * R + r;
        __syncthreads();
        // part x lies in slot 2 (w + x), the first in slot 2 w + 1
        auto at = [&](int x) { return (2 * (w + x) + (x == 0 ? 1 : 0)) * PR + r; };
        float m = -INFINITY;
        for (int x = tid; x < parts; x += kJoinThreads) m = fmaxf(m, ws[lay.part_m + at(x)]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        if ((tid & 31) == 0) wmax[tid >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kJoinThreads / 32; ++i) m = fmaxf(m, wmax[i]);
        const float use = m == -INFINITY ? 0.f : m;
        const int c4 = tid % TPR, gr = tid / TPR;
        float l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int BATCH = 8;  // parts whose loads are in flight together
        for (int x0 = gr; x0 < parts; x0 += GR * BATCH) {
            float pm[BATCH], pl[BATCH];
            float4 v[BATCH];
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const int64_t k = at(min(x0 + b * GR, parts - 1));  // past the end: the last part, with weight 0
                pm[b] = ws[lay.part_m + k];
                pl[b] = ws[lay.part_l + k];
                v[b] = *reinterpret_cast<const float4 *>(ws + lay.part_o + k * HD + 4 * c4);
            }
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                if (x0 + b * GR >= parts) break;
                const float f = ex2(pm[b] - use);
                l = fmaf(f, pl[b], l);
                o.x = fmaf(f, v[b].x, o.x); o.y = fmaf(f, v[b].y, o.y);
                o.z = fmaf(f, v[b].z, o.z); o.w = fmaf(f, v[b].w, o.w);
            }
        }
        so[gr][c4] = o;
        if (c4 == 0) sl[gr] = l;
        __syncthreads();
        if (gr != 0) continue;
#pragma unroll 4
        for (int i = 1; i < GR; ++i) {
            const float4 v = so[i][c4];
            o.x += v.x; o.y += v.y; o.z += v.z; o.w += v.w;
            l += sl[i];
        }
        const int64_t qrow = ((int64_t)n * p.D + row / p.G) * p.Hq + h * p.G + row % p.G;
        const float f = l == 0.f ? 0.f : 1.f / l;
        T *dst = static_cast<T *>(p.out) + qrow * HD + 4 * c4;
        store2(dst, l == 0.f ? 0.f : o.x * f, l == 0.f ? 0.f : o.y * f);
        store2(dst + 2, l == 0.f ? 0.f : o.z * f, l == 0.f ? 0.f : o.w * f);
        if (c4 == 0) {
            const float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
            if (p.lse) p.lse[qrow] = lse2 * kLn2;
            if (p.weight_out) ws[lay.lse2 + qrow] = lse2;
        }
    }
}

// A launch that may begin while the kernel before it on the stream ends (the
// kernel waits for that one's results by itself).
template <typename... Args>
cudaError_t launch_after(void (*kern)(Args...), dim3 grid, int threads, cudaStream_t st,
                         std::common_type_t<Args>... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// weight_out[n][page] = weight_in + sum over the rows of 2^(page share - lse).
// A block takes 32 pages of a sequence; its 8 groups of threads take every
// eighth row and are added up in order.
__global__ void __launch_bounds__(256) page_weight_kernel(const AttnDecodeParams p, Layout lay) {
    __shared__ float part[8][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float *ws = static_cast<const float *>(p.workspace);
    const int64_t chunks = (p.max_pages + 31) / 32;
    const int n = (int)(blockIdx.x / chunks);
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int page = (int)(blockIdx.x % chunks) * 32 + x;
    int len;
    const int pages = pages_of(p, n, len);
    const int rows = p.D * p.Hq;
    float sum = 0.f;
    if (page < pages) {
        for (int r = y; r < rows; r += 8) {
            const int64_t q = (int64_t)n * rows + r;
            const float lse2 = ws[lay.lse2 + q];
            if (lse2 != -INFINITY) sum += ex2(ws[lay.page_w + q * p.max_pages + page] - lse2);
        }
    }
    part[y][x] = sum;
    __syncthreads();
    if (y == 0 && page < p.max_pages) {
        for (int i = 1; i < 8; ++i) sum += part[i][x];
        const int64_t at = (int64_t)n * p.max_pages + page;
        p.weight_out[at] = (p.weight_in ? p.weight_in[at] : 0.f) + sum;
    }
}

template <typename T, int HD, int NB, int MT>
cudaError_t launch_main(const AttnDecodeParams &p, const Layout &lay, cudaStream_t st) {
    using S = Smem<HD, NB, MT>;
    auto kern = decode_attn_kernel<T, HD, NB, MT>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(kern), S::kBytes, done);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)lay.workers, 32 * MT, S::kBytes, st>>>(p, lay);
    return cudaGetLastError();
}

template <typename T, int HD>
cudaError_t launch(const AttnDecodeParams &p, cudaStream_t st) {
    const Layout lay = make_layout(p.batch, p.D, p.Hq, p.Hkv, HD, sizeof(T) == 2 ? KDA_DT_BF16 : KDA_DT_F32, p.max_pages,
                                   p.weight_out != nullptr);
    if (lay.items > 0x7fffffff || (int64_t)p.max_pages * p.Hkv * lay.RB > 0x7fffffff) return cudaErrorInvalidValue;
    cudaError_t e;
    if (lay.MT == 0) e = launch_tc(p, lay, HD, st);
    else if (lay.NB == 1) e = launch_main<T, HD, 1, 1>(p, lay, st);
    else if (lay.MT == 1) e = launch_main<T, HD, 2, 1>(p, lay, st);
    else if (lay.MT == 2) e = launch_main<T, HD, 2, 2>(p, lay, st);
    else e = launch_main<T, HD, 2, 4>(p, lay, st);
    if (e != cudaSuccess || p.max_pages == 0) return e;
    if (lay.whole) {
        if (p.weight_out == nullptr) return cudaSuccess;
    } else {
        int64_t rows = kJoinBlocks / lay.items;
        rows = rows < 1 ? 1 : rows > lay.PR ? lay.PR : rows;
        const dim3 grid((unsigned)lay.items, (unsigned)rows);
        if (lay.workers > 8 * lay.items) e = launch_after(join_kernel<T, HD, 512>, grid, 512, st, p, lay);
        else e = launch_after(join_kernel<T, HD, 128>, grid, 128, st, p, lay);
    }
    if (e != cudaSuccess || p.weight_out == nullptr) return e;
    const int64_t blocks = (int64_t)p.batch * ((p.max_pages + 31) / 32);
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_after(page_weight_kernel, dim3((unsigned)blocks), 256, st, p, lay);
}

template <typename T>
cudaError_t launch_dim(const AttnDecodeParams &p, int d, cudaStream_t st) {
    if (d == 128) return launch<T, 128>(p, st);
    if (d == 64) return launch<T, 64>(p, st);
    return launch<T, 32>(p, st);
}

}  // namespace

namespace dec {

Layout make_layout(int64_t batch, int D, int Hq, int Hkv, int d, int dtype, int64_t max_pages, bool with_weight) {
    auto align64 = [](int64_t x) { return (x + 63) / 64 * 64; };
    const int rows = D * (Hq / Hkv);
    Layout l{};
    // On tcgen05 and on the warps' products, us at 20, 32, 40 and 64 rows of a kv head
    // (same lengths): d = 128, 32 sequences of up to 8192 positions 99, 115, 105, 134 and
    // 105, 126, 163, 211; 64 of up to 900 68, 68, 68, 64 and 81, 82, 109, 95; 8 of up to
    // 2048 29, 29, 29, 31 and 38, 50, 54, 64.  d = 64: 83, 96, 87, 107 and 70, 86, 107,
    // 146; 60, 60, 58, 56 and 52, 54, 74, 66; 25, 25, 27, 27 and 29, 40, 46, 54: up to
    // 32 rows of 64 channels full batches would gain 10 to 20 %, small ones lose as much.
    if (dtype == KDA_DT_BF16 && d >= 64 && rows > 16) {
        l.R = 128;
    } else {
        l.NB = rows <= 8 ? 1 : 2;
        l.MT = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
        l.R = 8 * l.NB * l.MT;
    }
    l.RB = (rows + l.R - 1) / l.R;
    l.PR = rows < l.R ? rows : l.R;
    l.items = batch * Hkv * l.RB;
    // A worker per place on the GPU.  2 and 4 of them per place never took less and
    // up to 1.6 times as much (same lengths for all): the 64-sequence batch above
    // 378, 385 and 399 us, 48 sequences with windows of 4 tokens 168, 179 and 274.
    const int64_t units = l.items * max_pages, places = l.MT == 0 ? kSms : (int64_t)kSms * warps_per_sm(l.NB) / l.MT;
    l.workers = places < units ? places : units;
    if (l.workers < 1) l.workers = 1;
    l.whole = max_pages > 0 && l.items <= 0x7fffffff &&
              (max_pages == 1 || (max_pages <= kWholePages && l.items >= (l.MT == 0 ? kWholeItemsTc : kWholeItems)));
    l.desc = 0;
    l.part_m = align64(2 * l.items);
    l.part_l = l.part_m + align64(2 * l.workers * l.PR);
    l.part_o = l.part_l + align64(2 * l.workers * l.PR);
    l.lse2 = l.part_o + align64(2 * l.workers * l.PR * d);
    l.page_w = l.lse2 + (with_weight ? align64(batch * D * Hq) : 0);
    if (l.whole) l.workers = l.items;
    l.total = l.page_w + (with_weight ? align64(batch * D * Hq * max_pages) : 0);
    return l;
}

}  // namespace dec

size_t attn_decode_workspace_bytes(int Hq, int Hkv, int d, int dtype, int64_t batch, int D, int64_t max_pages,
                                   bool with_weight) {
    if (batch <= 0) return 0;
    return (size_t)make_layout(batch, D, Hq, Hkv, d, dtype, max_pages, with_weight).total * 4;
}

cudaError_t launch_attn_decode(const AttnDecodeParams &p, int d, int dtype, cudaStream_t st) {
    return dtype == KDA_DT_BF16 ? launch_dim<__nv_bfloat16>(p, d, st) : launch_dim<float>(p, d, st);
}

}  // namespace kda
