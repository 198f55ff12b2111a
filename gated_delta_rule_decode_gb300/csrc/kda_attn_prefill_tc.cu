// Causal attention over packed prompts on tcgen05 (bf16).
//
//   S = Q K^T,  P = e^{scale (S - m)},  O = P V,  m and l = sum P per row
//
// A CTA takes two tiles of 128 query rows of one kv head and walks the
// sequence's keys in blocks of 128.  A tile's rows are tokens x the G query
// heads of the kv head, so a block of keys and values is loaded once for all
// of them.  Roles:
//
//   warps 0-3, 4-7  softmax of tile 0 and 1: a thread owns a row, reads its
//                   128 scores from tensor memory, and writes the weights back
//                   over them as bf16, the operand of the second product
//   warp 8          issues the products
//   warp 9          TMA loads: Q once, then rings of key and value blocks; at
//                   the end looks over the value blocks that some row of the
//                   tiles must not see (below)
//
// While one tile's softmax runs, the tensor cores work on the other tile:
// PV(t, j), then QK(t, j + 1), for t = 0, 1 in turn.  Tensor memory holds S
// (P over it) and O of both tiles: 4 x 128 columns.
//
// The running maximum is only moved when it would grow by more than 8 (in
// powers of two); until then weights may reach 2^8, which costs bf16 nothing,
// and O is not rescaled.  When it moves, the row's warp waits for the last PV
// and rescales O in tensor memory.
//
// P in bf16 is rounded to 8 bits, which averages out over many keys but not
// over few.  Where a weight of the block may exceed 1/4 of its row's sum so
// far, the row's P takes a second bf16 term (in the other half of the score
// columns; zero for the tile's other rows) and the tile a second product: rows
// that one or a few keys dominate keep 16 bits.  A row decides by its own
// weights alone, so later tokens do not change its bits.  Sums of P are taken
// in fp32 before rounding.
//
// Measured: 16 384 tokens, 16 heads over 2, d = 128: 890 us, 1.24 PFLOP/s (of an
// earlier 879, second terms were 82); 6021 tokens in 7 prompts, 32 heads over 8:
// 168 us.  The chain softmax - PV - QK of a tile bounds it: about 2200 cycles of
// softmax and 1040 of products, against 2080 of products in the step of both tiles.
//
// Masked values: a weight of zero times a NaN or an infinity would poison a
// row that must not see it.  Scores are masked by selection, so keys need no
// care.  In value blocks that reach past the tiles' first token, rows past the
// sequence's end are zeroed in shared memory, and a non-finite value is zeroed
// and remembered; if there was one, the epilogue adds those values to exactly
// the rows that see them.
//
// Infinite values that every row sees stay in the products, where the second
// term (zero, or of either sign) would turn them into NaN.  An output that comes
// out not finite although its row's sum is a number is therefore settled by the
// values themselves: a warp that has one looks over the keys that all its rows
// see.
#include <cuda_bf16.h>
#include <stdint.h>

#include <type_traits>

#include "kda_attn_internal.h"
#include "kda_attn_math.cuh"
#include "kda_bulk.cuh"
#include "kda_internal.h"
#include "kda_tc.cuh"

namespace kda {
namespace {

constexpr int kRows = 128, kKeys = 128;
constexpr int kThreads = 384;  // warps 10, 11 only give their registers to the softmax, which holds 128 scores
constexpr uint32_t kTmem = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.f;  // log2 growth of the maximum that is let stand
constexpr float kShare = 4.f;  // weights above 1 / kShare of the row's sum take two terms (at 16: 1122 us for 988)

template <int HD>
struct Cfg {
    static constexpr int kTile = 128 * HD * 2;           // bytes of a Q tile, a key block, a value block
    // A tile's rows are swizzled pieces of 64 columns (32 where d is), one chunk of 128 rows after the other.
    static constexpr int kCols = HD < 64 ? HD : 64, kRowBytes = 2 * kCols, kChunks = HD / kCols;
    static constexpr int kChunk = 128 * kRowBytes;
    static constexpr uint32_t kSwizzle = kRowBytes == 128 ? 2u : 4u;  // descriptor code of the 128- and 64-byte swizzle
    static constexpr int NK = HD == 128 ? 2 : 4, NV = HD == 128 ? 3 : 4;
    static constexpr int kBytes = 1024 + (2 + NK + NV) * kTile + 256;
    static constexpr int kO = 256;                       // tensor memory column of O (tile 0); S at 0 and 128
};

struct Bars {
    uint64_t q_full[2], s_full[2], p_full[2], pv_done[2], k_full[4], k_empty[4], v_full[4], v_empty[4], v_fixed[4], drain;
};

// Instruction descriptor of kind::f16 with bf16 operands and fp32 accumulation;
// b_mn: B is stored with its N extent contiguous.
constexpr uint32_t idesc_bf16(int M, int N, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}

// Shared-memory descriptors of one K = 16 step.  Operands with the contraction
// contiguous (Q and K): step ks is 32 bytes of every row.  Values: 16 rows
// (keys) with the channels contiguous; the chunks of channels lie kChunk apart.
// 8-row groups follow one another in both.
template <int HD>
__device__ __forceinline__ uint64_t desc_of(uint32_t saddr, uint32_t chunk_bytes) {
    using C = Cfg<HD>;
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(chunk_bytes >> 4) << 16) |
           ((uint64_t)(8 * C::kRowBytes >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)C::kSwizzle << 61);
}
template <int HD>
__device__ __forceinline__ uint64_t desc_qk(uint32_t tile, int ks) {
    using C = Cfg<HD>;
    constexpr int kSteps = C::kRowBytes / 32;  // in a chunk
    return desc_of<HD>(tile + (uint32_t)((ks / kSteps) * C::kChunk + (ks % kSteps) * 32), 16);
}
template <int HD>
__device__ __forceinline__ uint64_t desc_v(uint32_t block, int ks) {
    using C = Cfg<HD>;
    return desc_of<HD>(block + (uint32_t)(ks * 16 * C::kRowBytes), C::kChunk);
}

__device__ __forceinline__ void tma_load_3d(void *dst, const void *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

// All lanes of a warp, with one answer.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t phase, volatile int *abort_flag) {
    return __all_sync(~0u, mbar_wait_or_abort(bar, (uint32_t)phase, abort_flag));
}

__device__ __forceinline__ bool nonfinite2(uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// What the values of keys 0..last at 32 channels (v: key 0, the first of them)
// make of the outputs of rows that see them all: +inf, -inf or NaN where some
// are not finite.  By a whole warp; `number`: the row's sum of weights is one.
__device__ __forceinline__ void settle(const __nv_bfloat16 *v, int64_t stride, int last, bool number, float (&o)[32]) {
    const int lane = threadIdx.x & 31;
    uint32_t seen = 0;  // of the lane's 8 channels: bits 0.. +inf, 8.. -inf, 16.. NaN
#pragma unroll 1
    for (int key = lane >> 2; key <= last; key += 8) {
        const uint4 x = *reinterpret_cast<const uint4 *>(v + key * stride + 8 * (lane & 3));
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t h = (w[e >> 1] >> (16 * (e & 1))) & 0xffffu;
            if ((h & 0x7f80u) == 0x7f80u) seen |= 1u << (e + ((h & 0x7fu) ? 16 : h >> 15 ? 8 : 0));
        }
    }
#pragma unroll
    for (int at = 4; at < 32; at <<= 1) seen |= __shfl_xor_sync(~0u, seen, at);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const uint32_t of = __shfl_sync(~0u, seen, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const bool up = (of >> e) & 1u, down = (of >> (8 + e)) & 1u, nan = (of >> (16 + e)) & 1u;
            if (number && (up || down || nan)) o[8 * u + e] = nan || (up && down) ? NAN : up ? INFINITY : -INFINITY;
        }
    }
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
prefill_tc_kernel(const AttnPrefillParams p, const __grid_constant__ CUtensorMap qmap,
                  const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    using C = Cfg<HD>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char *sq = smem, *sk = sq + 2 * C::kTile, *sv = sk + C::NK * C::kTile;
    __shared__ Bars bars;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag, v_bad;
    __shared__ __align__(4) volatile unsigned char two_terms[2][4];  // by tile and warp: its P has a second term
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const int kvh = (int)(blockIdx.x % (unsigned)p.Hkv);
    const int64_t unit = (int64_t)((gridDim.x - 1 - blockIdx.x) / (unsigned)p.Hkv);
    const int TT = kRows / p.G;  // tokens of a tile
    int64_t pair;
    const int s = seq_of_unit(p.cu_seqlens, p.num_seqs, 2 * TT, 1, unit, p.err_flag, pair);
    int t0, t1;
    if (!seq_range(p.cu_seqlens, s, p.total_tokens, p.err_flag, t0, t1)) return;
    const int len = t1 - t0;
    if (pair < 0 || pair * 2 * TT >= len) return;
    const int a0 = (int)pair * 2 * TT;  // first token of tile 0, within the sequence
    int nblk[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int a = a0 + t * TT, b = min(a + TT, len);
        nblk[t] = b > a ? (b + kKeys - 1) / kKeys : 0;
    }
    const int n = max(nblk[0], nblk[1]);
    // the first block with a key that some row must not see; at most three more follow
    const int diag = (a0 + 1) / kKeys;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.q_full[i], 1);
            mbar_init(&bars.s_full[i], 1);
            mbar_init(&bars.p_full[i], 4);
            mbar_init(&bars.pv_done[i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bars.k_full[i], 1);
            mbar_init(&bars.k_empty[i], 1);
            mbar_init(&bars.v_full[i], 1);
            mbar_init(&bars.v_fixed[i], 1);
            mbar_init(&bars.v_empty[i], 1);
        }
        mbar_init(&bars.drain, 1);
        fence_barrier_init();
        abort_flag = 0;
        v_bad = 0;
    }
    if (warp == 8) tc::tmem_alloc(&tmem_base, kTmem);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = tmem_base;

    // 168 registers a thread at launch: 2 x 128 x 208 + 128 x 88 = 384 x 168
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 9) {
            // ---------------- loads
            const int box = TT * p.G * C::kRowBytes;  // bytes of a Q box
            auto load_q = [&](int t) {
                if (lane != 0) return;
                mbar_arrive_expect_tx(&bars.q_full[t], box * C::kChunks);
                for (int c = 0; c < C::kChunks; ++c)
                    tma_load_3d(sq + t * C::kTile + c * C::kChunk, &qmap, C::kCols * c, kvh * p.G, t0 + a0 + t * TT, &bars.q_full[t]);
            };
            auto load_kv = [&](unsigned char *dst, const CUtensorMap *map, int j, uint64_t *bar) {
                if (lane != 0) return;
                mbar_arrive_expect_tx(bar, C::kTile);
                for (int c = 0; c < C::kChunks; ++c) tma_load_3d(dst + c * C::kChunk, map, C::kCols * c, kvh, t0 + j * kKeys, bar);
            };
            int jk = 0, jv = 0;
            bool ok = true;
            load_q(0);
            for (int j = 0; j < n && ok; ++j) {
                ok = j < C::NK || warp_wait(&bars.k_empty[j % C::NK], j / C::NK - 1, &abort_flag);
                if (!ok) break;
                load_kv(sk + (j % C::NK) * C::kTile, &kmap, j, &bars.k_full[j % C::NK]);
                jk = j + 1;
                if (j == 0 && nblk[1] > 0) load_q(1);
                ok = j < C::NV || warp_wait(&bars.v_empty[j % C::NV], j / C::NV - 1, &abort_flag);
                if (!ok) break;
                load_kv(sv + (j % C::NV) * C::kTile, &vmap, j, &bars.v_full[j % C::NV]);
                jv = j + 1;
            }
            // ---------------- values that some row must not see
            for (int j = diag; j < n && ok; ++j) {
                ok = warp_wait(&bars.v_full[j % C::NV], j / C::NV, &abort_flag);
                if (!ok) break;
                unsigned char *blk = sv + (j % C::NV) * C::kTile;
                bool bad = false;
#pragma unroll 4
                for (int i = lane; i < C::kTile / 16; i += 32) {
                    const int key = j * kKeys + ((i / (C::kRowBytes / 16)) & (kKeys - 1));
                    uint4 *u = reinterpret_cast<uint4 *>(blk) + i;
                    uint4 x = *u;
                    const bool odd = nonfinite2(x.x) || nonfinite2(x.y) || nonfinite2(x.z) || nonfinite2(x.w);
                    if (key >= len) {
                        *u = make_uint4(0, 0, 0, 0);
                    } else if (key > a0 && odd) {
                        bad = true;
                        uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if ((w[e] & 0x7f80u) == 0x7f80u) w[e] &= 0xffff0000u;
                            if ((w[e] & 0x7f800000u) == 0x7f800000u) w[e] &= 0x0000ffffu;
                        }
                        *u = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                if (bad) v_bad = 1;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.v_fixed[j - diag]);
            }
            // every load lands before the CTA's memory goes
            mbar_wait_drain(&bars.q_full[0], 0);
            if (nblk[1] > 0) mbar_wait_drain(&bars.q_full[1], 0);
            for (int j = max(0, jk - C::NK); j < jk; ++j) mbar_wait_drain(&bars.k_full[j % C::NK], (j / C::NK) & 1u);
            for (int j = max(0, jv - C::NV); j < jv; ++j) mbar_wait_drain(&bars.v_full[j % C::NV], (j / C::NV) & 1u);
        } else if (warp == 8) {
            // ---------------- products (the whole warp in step: see mma_f16_ss_warp)
            const uint32_t id_qk = idesc_bf16(128, 128, false), id_pv = idesc_bf16(128, HD, true);
            auto qk = [&](int t, int j) {
                const uint32_t qa = tc::smem_u32(sq + t * C::kTile), ka = tc::smem_u32(sk + (j % C::NK) * C::kTile);
#pragma unroll
                for (int ks = 0; ks < HD / 16; ++ks)
                    tc::mma_f16_ss_warp(tm + 128 * t, desc_qk<HD>(qa, ks), desc_qk<HD>(ka, ks), id_qk, ks > 0);
                tc::commit_warp(&bars.s_full[t]);
            };
            auto pv = [&](int t, int j) {
                const uint32_t va = tc::smem_u32(sv + (j % C::NV) * C::kTile);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    tc::mma_f16_ts_warp(tm + C::kO + HD * t, tm + 128 * t + 8 * ks, desc_v<HD>(va, ks), id_pv,
                                   (j > 0 || ks > 0) ? 1u : 0u);
                if (__any_sync(~0u, *reinterpret_cast<volatile const int *>(&two_terms[t][0]) != 0)) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        tc::mma_f16_ts_warp(tm + C::kO + HD * t, tm + 128 * t + 64 + 8 * ks, desc_v<HD>(va, ks),
                                       id_pv, 1u);
                }
                tc::commit_warp(&bars.pv_done[t]);
            };
            bool ok = warp_wait(&bars.k_full[0], 0, &abort_flag);
            for (int t = 0; t < 2 && ok; ++t) {
                if (nblk[t] == 0) continue;
                ok = warp_wait(&bars.q_full[t], 0, &abort_flag);
                if (ok) qk(t, 0);
            }
            if (ok) tc::commit_warp(&bars.k_empty[0]);
            for (int j = 0; j < n && ok; ++j) {
                // (what the loads bring is waited for while the softmax still runs)
                ok = (j < diag ? warp_wait(&bars.v_full[j % C::NV], j / C::NV, &abort_flag)
                               : warp_wait(&bars.v_fixed[j - diag], 0, &abort_flag)) &&
                     (j + 1 >= n || warp_wait(&bars.k_full[(j + 1) % C::NK], (j + 1) / C::NK, &abort_flag));
                for (int t = 0; t < 2 && ok; ++t) {
                    if (j >= nblk[t]) continue;
                    ok = warp_wait(&bars.p_full[t], j, &abort_flag);
                    if (!ok) break;
                    tc::fence_after_sync();
                    pv(t, j);
                    if (j + 1 < nblk[t]) qk(t, j + 1);
                }
                if (!ok) break;
                tc::commit_warp(&bars.v_empty[j % C::NV]);
                if (j + 1 < n) tc::commit_warp(&bars.k_empty[(j + 1) % C::NK]);
            }
            tc::commit_warp(&bars.drain);  // every product is done before the memory goes
            __all_sync(~0u, mbar_wait_drain(&bars.drain, 0));
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        // ---------------- softmax: thread = row
        const int t = warp >> 2, row = tid & 127;
        const int tok = a0 + t * TT + row / p.G, gi = row % p.G;  // token within the sequence
        const bool valid = row < TT * p.G && tok < len;
        const uint32_t s_addr = tc::lane_addr(tm, warp, 128 * t);
        const uint32_t o_addr = tc::lane_addr(tm, warp, C::kO + HD * t);
        const float sl2 = p.scale * kLog2e;
        const int nb = nblk[t];
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int j = 0; j < nb; ++j) {
            // (after a wait gave up the loop runs on, on garbage, to its end)
            if (!warp_wait(&bars.s_full[t], j, &abort_flag)) ok = false;
            tc::fence_after_sync();
            float sc[4][32];
#pragma unroll
            for (int i = 0; i < 4; ++i) tc::ld32(s_addr + 32 * i, sc[i]);
            tc::wait_ld();
            const int vis = tok - j * kKeys + 1;  // keys of this block that the row sees
            if (__any_sync(~0u, vis < kKeys)) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (32 * i + c >= vis) sc[i][c] = -INFINITY;
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 32; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) mx[i] = fmaxf(mx[i], sc[i][c]);
            const float mnew = fmaxf(fmaxf(m, fmaxf(mx[0], mx[1])), fmaxf(mx[2], mx[3]));
            if (j == 0) {
                m = mnew;
            } else {
                const bool grow = (mnew - m) * sl2 > kLazy;
                if (__any_sync(~0u, grow)) {
                    const float f = grow ? ex2((m - mnew) * sl2) : 1.f;
                    if (grow) m = mnew;
                    l *= f;
                    if (!warp_wait(&bars.pv_done[t], j - 1, &abort_flag)) ok = false;
                    tc::fence_after_sync();
#pragma unroll 1
                    for (int c = 0; c < HD; c += 16) {
                        float o[16];
                        tc::ld16(o_addr + c, o);
                        tc::wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] *= f;
                        tc::st16(o_addr + c, o);
                    }
                    tc::wait_st();
                }
            }
            const float use = m == -INFINITY ? 0.f : m;
            // a weight above 1 / kShare of the sum (of which it is a part)?
            const float top = ex2((fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) - use) * sl2);
            const bool mine = top * (kShare - 1.f) > l;
            const uint32_t keep = mine ? ~0u : 0u;
            const bool two = __any_sync(~0u, valid && mine);
            const float2 k2 = make_float2(sl2, sl2), b2 = make_float2(-use * sl2, -use * sl2);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            auto weights = [&](auto with_two) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t pk[16], rest[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        float2 x = fma2(make_float2(sc[i][2 * c], sc[i][2 * c + 1]), k2, b2);
                        x.x = ex2(x.x);
                        x.y = ex2(x.y);
                        sum[c & 1] = add2(sum[c & 1], x);
                        pk[c] = pack_bf16(x.x, x.y);
                        // the second term: what the rounding left, or zero (another row of
                        // the tile may have one, and the product takes all rows)
                        rest[c] = with_two ? pack_bf16(x.x - __uint_as_float(pk[c] << 16),
                                                       x.y - __uint_as_float(pk[c] & 0xffff0000u)) & keep
                                           : 0u;
                    }
                    tc::st16u(s_addr + 16 * i, pk);
                    tc::st16u(s_addr + 64 + 16 * i, rest);
                }
            };
            if (two) weights(std::true_type{});
            else weights(std::false_type{});
            tc::wait_st();
            tc::fence_before_sync();
            if (lane == 0) two_terms[t][warp & 3] = two;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.p_full[t]);
            sum[0] = add2(sum[0], sum[1]);
            l += sum[0].x + sum[0].y;
        }
        // ---------------- epilogue
        if (nb > 0 && ok) ok = warp_wait(&bars.pv_done[t], nb - 1, &abort_flag);
        if (nb > 0 && ok) {
            tc::fence_after_sync();
            const float inv = 1.f / l;
            const int64_t orow = ((int64_t)(t0 + tok) * p.Hq + kvh * p.G + gi);
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + orow * HD;
            const bool bad = *reinterpret_cast<volatile int *>(&v_bad) != 0;
            const bool number = valid && l > 0.f && l <= 3.402823466e38f;
#pragma unroll 1
            for (int c = 0; c < HD; c += 32) {
                __syncwarp();  // (the rows that are not written rejoin for the next load)
                float o[32], zero[4] = {0.f, 0.f, 0.f, 0.f};
                tc::ld32(o_addr + c, o);
                tc::wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    o[e] *= inv;
                    zero[e & 3] = fmaf(o[e], 0.f, zero[e & 3]);  // NaN where one is not finite
                }
                if (__any_sync(~0u, number && (zero[0] + zero[1]) + (zero[2] + zero[3]) != 0.f))
                    settle(static_cast<const __nv_bfloat16 *>(p.v) + (int64_t)t0 * p.v_stride + (int64_t)kvh * HD + c,
                           p.v_stride, a0, number, o);
                if (!valid) continue;
                if (bad) {  // the values that were set aside, for the rows that see them
                    for (int key = a0 + 1; key <= tok; ++key) {
                        const uint4 *src = reinterpret_cast<const uint4 *>(
                            static_cast<const __nv_bfloat16 *>(p.v) + (int64_t)(t0 + key) * p.v_stride + (int64_t)kvh * HD + c);
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const uint4 x = src[u];
                            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if ((w[e] & 0x7f80u) == 0x7f80u) o[8 * u + 2 * e] += __uint_as_float(w[e] << 16);
                                if ((w[e] & 0x7f800000u) == 0x7f800000u)
                                    o[8 * u + 2 * e + 1] += __uint_as_float(w[e] & 0xffff0000u);
                            }
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < 32; e += 8)
                    *reinterpret_cast<uint4 *>(dst + c + e) =
                        make_uint4(pack_bf16(o[e], o[e + 1]), pack_bf16(o[e + 2], o[e + 3]), pack_bf16(o[e + 4], o[e + 5]),
                                   pack_bf16(o[e + 6], o[e + 7]));
            }
            if (valid && p.lse) p.lse[orow] = (m * sl2 + log2f(l)) * kLn2;
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 8) tc::tmem_dealloc(tm, kTmem);
    if (tid == 0 && abort_flag && p.err_flag) atomicOr(p.err_flag, KDA_DEVERR_TIMEOUT);
}

bool make_map(CUtensorMap *map, const void *base, int d, int heads, int64_t tokens, int64_t stride, int box_heads,
              int box_tokens) {
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {(cuuint32_t)(d < 64 ? d : 64), (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
    const cuuint32_t elem[3] = {1, 1, 1};
    return tensor_map_encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
                                  elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                  d < 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HD>
cudaError_t launch_tc(const AttnPrefillParams &p, cudaStream_t st) {
    const int TT = kRows / p.G;
    CUtensorMap qmap, kmap, vmap;
    if (!make_map(&qmap, p.q, HD, p.Hq, p.total_tokens, p.q_stride, p.G, TT) ||
        !make_map(&kmap, p.k, HD, p.Hkv, p.total_tokens, p.k_stride, 1, kKeys) ||
        !make_map(&vmap, p.v, HD, p.Hkv, p.total_tokens, p.v_stride, 1, kKeys))
        return cudaErrorInvalidValue;
    auto kern = prefill_tc_kernel<HD>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(kern), Cfg<HD>::kBytes, done);
    if (e != cudaSuccess) return e;
    const int64_t blocks = (p.total_tokens / (2 * TT) + p.num_seqs) * p.Hkv;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    kern<<<(unsigned)blocks, kThreads, Cfg<HD>::kBytes, st>>>(p, qmap, kmap, vmap);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_prefill_tc(const AttnPrefillParams &p, int d, cudaStream_t st) {
    if (tensor_map_encode_fn() == nullptr) return cudaErrorNotSupported;
    if (d == 128) return launch_tc<128>(p, st);
    if (d == 64) return launch_tc<64>(p, st);
    return launch_tc<32>(p, st);
}

}  // namespace kda
