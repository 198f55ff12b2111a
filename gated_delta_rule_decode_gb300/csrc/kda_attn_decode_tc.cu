// Attention of many query rows per sequence over the 8-bit paged cache, on
// tcgen05: draft windows of grouped heads (more than 16 rows of a kv head).
//
// Up to 128 rows (window tokens x grouped heads) are the 128 lanes of one
// product, so a page is read once for all of them; the work is cut into
// workers' ranges as in kda_attn_decode.cu, one worker per SM.  Tiles are two
// pages (128 positions) of one item:
//
//   S = Q K^T (128 x 128),  P = e^{S - m},  O += P V
//
// A page comes as bytes by bulk copies and is turned into fp16 operands (exact)
// by eight warps: both pages' rows lie as the K-major 128-byte-swizzled operand
// wants them (keys by channel, the value layout by position).  Roles:
//
//   warps 0-7    softmax: thread = row, warps 0-3 the tile's first page, 4-7 the
//                second; scores read from tensor memory, weights written back as
//                fp16, O rescaled when the maximum moves
//   warp 8       issues QK(j + 1), then PV(j)
//   warp 9       looks up pages, issues the copies (a ring of page slots)
//   warps 10-17  conversion; the query rows at an item's start
//
// The query rows are scaled by powers of two into fp16's range (exact for
// bf16).  Value scales are powers of two and go into the exponent of the weights,
// which stand at 2^7 for the row's largest contribution (see kda_attn_decode.cuh);
// maximum and unit are only moved when they grow by more than 2^8, so the weights
// reach 2^15.
//
// Per tile the products take 1040 cycles of an SM and the bytes 1400, but two
// tiles in flight take about 2 x 5000: the chain conversion - QK - softmax - PV
// is what bounds it, and within it instruction fetch (five roles' code), which
// is why loops are rolled where they can be (137 us unrolled, 114 rolled).
// Measured: 7 tokens x 8 heads, 32 sequences of up to 8192, d = 128: 108 to 114 us
// from box to box, 1.2 to 1.3 TB/s.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "kda_attn_decode.cuh"
#include "kda_attn_internal.h"
#include "kda_bulk.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace {

using namespace dec;

constexpr int kWarps = 18, kThreads = kWarps * 32;
constexpr int kMmaWarp = 8, kLoadWarp = 9, kConvWarp = 10, kConvWarps = 8, kConv = kConvWarps * 32;
constexpr int kBatch = 16, kMeta = 2 * kBatch;  // page look-ups at a time, and kept
constexpr uint32_t kTmem = 512;
constexpr float kLazy = 8.f;
constexpr int kBias = 7;  // log2 of the weights' fp16 scale

template <int HD>
struct Cfg {
    static constexpr int kHalf = HD * kPage;          // bytes of a page's keys (or values)
    static constexpr int kSlots = HD == 128 ? 4 : 8;  // pages in the ring
    static constexpr int kOp = 128 * HD * 2;          // an fp16 operand of 128 rows of HD, or HD rows of 128
    static constexpr int kRing = kSlots * 2 * kHalf;
    static constexpr int kBytes = 1024 + kRing + 5 * kOp;  // Q, K and V twice
    static constexpr int kO = 256, kP = 384;           // tensor memory columns of O and of P; S at 0 and 128
    static_assert(kSlots + 4 < kBatch, "copies run less than a batch ahead of the page data in use");
};

struct Bars {
    uint64_t full[8], empty[8];                        // ring
    uint64_t k_ready[2], k_free[2], v_ready[2], v_free[2];
    uint64_t s_full[2], p_full[2], pv_done, o_free, drain;
};

// All lanes of a warp, with one answer.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, int phase, volatile int *abort_flag) {
    return __all_sync(~0u, mbar_wait_or_abort(bar, (uint32_t)phase, abort_flag));
}

// The worker's range as tiles: each role walks them by itself, in the same order.
struct Walk {
    Cursor cur;
    int64_t u0;            // first unit
    int i, count;          // units done, units
    Unit un;               // of the item at hand
    int left;              // its pages that are left in the range
    bool first, last;      // of the item (within the range), for the tile at hand
    int pages;             // of the tile: 1 or 2
    int page0;             // the item's first page in the range
    int item, tile;        // counted from 0 within the range

    __device__ __forceinline__ void begin(const Cursor &c, int64_t u, int n) {
        cur = c; u0 = u; count = n; i = 0; left = 0; item = -1; tile = -1; pages = 0;
    }
    // Moves to the next tile; un.page is its first page.
    __device__ __forceinline__ bool next(const AttnDecodeParams &p, int HR) {
        i += pages;
        if (i >= count) return false;
        if (left == 0) {
            un = locate(p, HR, cur, u0 + i);
            left = min(un.pages - un.page, count - i);
            first = true;
            page0 = un.page;
            ++item;
        } else {
            un.page += pages;
            first = false;
        }
        pages = left >= 2 ? 2 : 1;
        left -= pages;
        last = left == 0;
        ++tile;
        return true;
    }
};

template <int HD>
__global__ void __launch_bounds__(kThreads, 1) decode_attn_tc_kernel(const AttnDecodeParams p, const Layout lay) {
    using C = Cfg<HD>;
    using T = __nv_bfloat16;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sq = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char *sk = sq + C::kOp, *sv = sk + 2 * C::kOp, *ring = sv + 2 * C::kOp;
    __shared__ Bars bars;
    __shared__ PageMeta meta[kMeta];
    __shared__ int8_t q_exp[2][128];  // exponents of the rows' scales, by item
    __shared__ int64_t exchange[128];  // the prologue's sums, then a float per (page, row)
    __shared__ Cursor start;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    __shared__ volatile int v_nan;  // a NaN was set aside in some item's window
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rows_all = p.D * p.G, RB = lay.RB, HR = p.Hkv * RB;
    float *ws = static_cast<float *>(p.workspace);

    if (tid == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], kConvWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.k_ready[i], kConvWarps);
            mbar_init(&bars.v_ready[i], kConvWarps);
            mbar_init(&bars.k_free[i], 1);
            mbar_init(&bars.v_free[i], 1);
            mbar_init(&bars.s_full[i], 1);
            mbar_init(&bars.p_full[i], 8);
        }
        mbar_init(&bars.pv_done, 1);
        mbar_init(&bars.o_free, 8);
        mbar_init(&bars.drain, 1);
        fence_barrier_init();
        abort_flag = 0;
        v_nan = 0;
    }
    int64_t U, W, u0, u1;
    find_range<T, HD, kWarps>(p, HR, lay.whole, exchange, &start, U, W, u0, u1);
    if (u0 >= u1) return;
    if (warp == kMmaWarp) tc::tmem_alloc(&tmem_base, kTmem);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = tmem_base;
    const int count = (int)(u1 - u0);
    Walk wk;
    wk.begin(start, u0, count);

    if (warp == kLoadWarp) {
        // ---------------- page look-up (kBatch units at a time, one per lane) and copies
        Cursor fetch_cur = start;
        int fetched = 0, issued = 0;
        for (int i = 0; i < count; ++i) {
            const int slot = i % C::kSlots;
            if (i >= C::kSlots && !warp_wait(&bars.empty[slot], i / C::kSlots - 1, &abort_flag)) break;
            if (i >= fetched) {
                Cursor c = fetch_cur;
                if (lane < kBatch && fetched + lane < count) {
                    const Unit un = locate(p, HR, c, u0 + fetched + lane);
                    const int h = un.hr / RB;
                    const int id = p.block_table[(int64_t)un.n * p.max_pages + un.page];
                    meta[(fetched + lane) % kMeta] = page_meta(p, id, h);
                }
                const int from = min(kBatch - 1, count - 1 - fetched);
                fetch_cur.n = __shfl_sync(~0u, c.n, from);
                fetch_cur.base = __shfl_sync(~0u, c.base, from);
                fetched += kBatch;
                __syncwarp();
            }
            issued = i + 1;
            if (lane == 0) {
                const int block = meta[i % kMeta].block;
                if (block < 0) {
                    mbar_arrive(&bars.full[slot]);
                } else {
                    unsigned char *dst = ring + slot * 2 * C::kHalf;
                    mbar_arrive_expect_tx(&bars.full[slot], 2 * C::kHalf);
                    bulk_g2s(dst, p.k_pages + (int64_t)block * C::kHalf, C::kHalf, &bars.full[slot]);
                    bulk_g2s(dst + C::kHalf, p.v_pages + (int64_t)block * C::kHalf, C::kHalf, &bars.full[slot]);
                }
            }
        }
        // every copy lands before the CTA's memory goes
        for (int i = max(0, issued - C::kSlots); i < issued; ++i)
            mbar_wait_drain(&bars.full[i % C::kSlots], (uint32_t)(i / C::kSlots) & 1u);
    } else if (warp == kMmaWarp) {
        // ---------------- products (the whole warp in step: see mma_f16_ss_warp)
        const uint32_t id_qk = tc::idesc_f16(128, 128), id_pv = tc::idesc_f16(128, HD);
        const uint32_t qa = tc::smem_u32(sq);
        auto pv = [&](int j, bool first, int item) {
            const int b = j & 1;
            if (!warp_wait(&bars.p_full[b], j >> 1, &abort_flag) ||
                !warp_wait(&bars.v_ready[b], j >> 1, &abort_flag))
                return false;
            if (first && item > 0 && !warp_wait(&bars.o_free, item - 1, &abort_flag)) return false;
            tc::fence_after_sync();
            const uint32_t va = tc::smem_u32(sv + b * C::kOp);
#pragma unroll 1
            for (int ks = 0; ks < 8; ++ks)  // 16 positions each; a page is one 128-byte-wide chunk of HD rows
                tc::mma_f16_ts_warp(tm + C::kO, tm + C::kP + 64 * b + 8 * ks,
                               tc::desc_sw128(va + (uint32_t)((ks >> 2) * HD * 128 + (ks & 3) * 32)), id_pv,
                               (first && ks == 0) ? 0u : 1u);
            tc::commit_warp(&bars.v_free[b]);
            tc::commit_warp(&bars.pv_done);
            return true;
        };
        bool ok = true, pfirst = false;
        int pitem = 0;
        while (ok && wk.next(p, HR)) {
            const int j = wk.tile;
            const int b = j & 1;
            ok = warp_wait(&bars.k_ready[b], j >> 1, &abort_flag);
            if (!ok) break;
            tc::fence_after_sync();
            const uint32_t ka = tc::smem_u32(sk + b * C::kOp);
#pragma unroll 1
            for (int ks = 0; ks < HD / 16; ++ks)
                tc::mma_f16_ss_warp(tm + 128 * b, tc::desc_tf32_kstep(qa, 128, ks), tc::desc_tf32_kstep(ka, 128, ks), id_qk,
                               ks > 0);
            tc::commit_warp(&bars.k_free[b]);
            tc::commit_warp(&bars.s_full[b]);
            if (j > 0) ok = pv(j - 1, pfirst, pitem);
            pfirst = wk.first;
            pitem = wk.item;
        }
        if (ok) pv(wk.tile, pfirst, pitem);
        tc::commit_warp(&bars.drain);  // every product is done before the memory goes
        __all_sync(~0u, mbar_wait_drain(&bars.drain, 0));
    } else if (warp >= kConvWarp) {
        // ---------------- conversion
        const int ct = tid - kConvWarp * 32;  // 0..kConv - 1
        bool ok = true;
        while (ok && wk.next(p, HR)) {
            const int j = wk.tile;
            const int b = j & 1;
            // the buffers' last readers are QK(j - 2) and PV(j - 2); the keys need not wait
            // for the latter, so that QK(j) can be ready while softmax (j - 1) runs
            if (j >= 2) {
                ok = warp_wait(&bars.k_free[b], (j >> 1) - 1, &abort_flag) &&
                     (!wk.first || warp_wait(&bars.v_free[b], (j >> 1) - 1, &abort_flag));
                if (!ok) break;
            }
            if (wk.first) {
                // the query rows: the last product of the item before has read its own
                if (j >= 1) {
                    ok = warp_wait(&bars.k_free[b ^ 1], (j - 1) >> 1, &abort_flag);
                    if (!ok) break;
                }
                const int h = wk.un.hr / RB;
#pragma unroll 1
                for (int x = ct; x < 256; x += kConv) {
                    const int r = x >> 1, half = x & 1;  // two threads per row
                    const int row = (wk.un.hr % RB) * 128 + r;
                    const bool valid = row < rows_all;
                    const int tok = valid ? row / p.G : 0, gi = valid ? row - tok * p.G : 0;
                    const uint4 *src = reinterpret_cast<const uint4 *>(
                        static_cast<const T *>(p.q) + ((int64_t)wk.un.n * p.D + tok) * p.q_stride + (int64_t)(h * p.G + gi) * HD +
                        half * (HD / 2));
                    uint4 raw[HD / 16];
                    float amax = 0.f;
#pragma unroll
                    for (int u = 0; u < HD / 16; ++u) {
                        raw[u] = valid ? src[u] : make_uint4(0, 0, 0, 0);
                        const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xffff0000u))));
                    }
                    amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));  // (256 is whole warps of x)
                    int ex = (int)(__float_as_uint(amax) >> 23) - 127;
                    ex = ex < -100 ? -100 : ex > 126 ? 126 : ex;
                    const float mul = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
                    if (half == 0) q_exp[wk.item & 1][r] = (int8_t)ex;
#pragma unroll
                    for (int u = 0; u < HD / 16; ++u) {
                        const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
                        uint32_t y[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            y[e] = pack_f16(__uint_as_float(w[e] << 16) * mul, __uint_as_float(w[e] & 0xffff0000u) * mul);
                        *reinterpret_cast<uint4 *>(sq + tc::sw128_off16(r, half * (HD / 2) + 8 * u, 128)) =
                            make_uint4(y[0], y[1], y[2], y[3]);
                    }
                }
            }
            // keys: 16 channels of a position at a time
#pragma unroll 1
            for (int pg = 0; pg < wk.pages; ++pg) {
                const int i = wk.i + pg;
                const int slot = i % C::kSlots;
                ok = warp_wait(&bars.full[slot], i / C::kSlots, &abort_flag);
                if (!ok) break;
                const unsigned char *kb = ring + slot * 2 * C::kHalf;
                constexpr int PR = HD / 16;  // pieces per position
#pragma unroll
                for (int x = ct; x < kPage * PR; x += kConv) {
                    const int r = x / PR, u = x % PR;
                    const uint4 a = *reinterpret_cast<const uint4 *>(kb + 16 * x);
                    uint4 y0, y1;
                    e4m3x4_to_f16(a.x, y0.x, y0.y);
                    e4m3x4_to_f16(a.y, y0.z, y0.w);
                    e4m3x4_to_f16(a.z, y1.x, y1.y);
                    e4m3x4_to_f16(a.w, y1.z, y1.w);
                    unsigned char *dst = sk + b * C::kOp;
                    const uint32_t o0 = tc::sw128_off16(64 * pg + r, 16 * u, 128), o1 = tc::sw128_off16(64 * pg + r, 16 * u + 8, 128);
                    // the two halves of a row in either order, so that eight lanes write eight 16-byte banks
                    const bool sw = (u & 4) != 0;
                    *reinterpret_cast<uint4 *>(dst + (sw ? o1 : o0)) = sw ? y1 : y0;
                    *reinterpret_cast<uint4 *>(dst + (sw ? o0 : o1)) = sw ? y0 : y1;
                }
            }
            if (!ok) break;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.k_ready[b]);
            // values: 16 positions of a channel at a time
            if (j >= 2) ok = warp_wait(&bars.v_free[b], (j >> 1) - 1, &abort_flag);
            if (!ok) break;
            const int window0 = wk.un.len - p.D + 1;
#pragma unroll 1
            for (int pg = 0; pg < 2; ++pg) {
                unsigned char *dst = sv + b * C::kOp + pg * HD * 128;
                const int i = wk.i + pg;
                const int slot = i % C::kSlots;
                const bool have = pg < wk.pages && meta[i % kMeta].block >= 0;
                const unsigned char *vb = ring + slot * 2 * C::kHalf + C::kHalf;
                const int pos0 = (wk.un.page + pg) * kPage;
                const bool tail = pos0 + kPage > window0;
#pragma unroll
                for (int x = ct; x < HD * 4; x += kConv) {
                    const int r = x >> 2, u = x & 3;
                    uint4 a = make_uint4(0, 0, 0, 0);
                    if (have) {
                        a = *reinterpret_cast<const uint4 *>(vb + 16 * x);
                        if (tail) {  // bytes past the end, and the window's NaN bytes, count as zero
                            asm volatile("" ::: "memory");  // (a branch, not predicates)
                            const int left = wk.un.len - pos0, seen = window0 - pos0;
                            int at = min(min(mask_word(a.x, 16 * u, left, seen), mask_word(a.y, 16 * u + 4, left, seen)),
                                         min(mask_word(a.z, 16 * u + 8, left, seen), mask_word(a.w, 16 * u + 12, left, seen)));
                            if (at < kPage) v_nan = 1;
                        }
                    }
                    uint4 y0, y1;
                    e4m3x4_to_f16(a.x, y0.x, y0.y);
                    e4m3x4_to_f16(a.y, y0.z, y0.w);
                    e4m3x4_to_f16(a.z, y1.x, y1.y);
                    e4m3x4_to_f16(a.w, y1.z, y1.w);
                    *reinterpret_cast<uint4 *>(dst + tc::sw128_off16(r, 16 * u, HD)) = y0;
                    *reinterpret_cast<uint4 *>(dst + tc::sw128_off16(r, 16 * u + 8, HD)) = y1;
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bars.v_ready[b]);
                for (int pg = 0; pg < wk.pages; ++pg) mbar_arrive(&bars.empty[(wk.i + pg) % C::kSlots]);
            }
        }
    } else {
        // ---------------- softmax: thread = (row, page of the tile)
        // Every warp waits for every PV (of the tile before, before it gives the
        // tile's weights): QK(j) is issued before PV(j - 1), so that a wait by parity
        // for a later one alone could take an older for it.  After a wait gave up the
        // loop runs on, on garbage: the two warps of a row meet at barriers.
        const int pg = warp >> 2, quad = warp & 3, r = tid & 127;
        const uint32_t o_addr = tc::lane_addr(tm, quad, C::kO + pg * (HD / 2));  // its half of the channels
        float *mine = reinterpret_cast<float *>(exchange) + pg * 128 + r;
        const float *other = reinterpret_cast<float *>(exchange) + (pg ^ 1) * 128 + r;
        auto pair_sync = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + quad) : "memory"); };
        float m = -INFINITY, l = 0.f, qs = 0.f;
        int limit = 0, unit = kNoUnit;  // the exponent that O is counted in
        bool valid = false, ok = true;
        int64_t qrow = 0;
        while (wk.next(p, HR)) {
            const int j = wk.tile;
            const int b = j & 1;
            const Unit &un = wk.un;
            const int rb = un.hr % RB, h = un.hr / RB, row = rb * 128 + r;
            const bool active = rb * 128 + quad * 32 < rows_all;  // some row of this warp exists
            if (!warp_wait(&bars.s_full[b], j >> 1, &abort_flag)) ok = false;
            tc::fence_after_sync();
            if (wk.first) {
                valid = row < rows_all;
                limit = valid ? un.len - p.D + 1 + row / p.G : 0;
                qrow = valid ? ((int64_t)un.n * p.D + row / p.G) * p.Hq + h * p.G + row % p.G : 0;
                qs = __uint_as_float((uint32_t)(127 - 14 + q_exp[wk.item & 1][r]) << 23) * p.scale * kLog2e;
                m = -INFINITY;
                l = 0.f;
                unit = kNoUnit;
            }
            float fix = 1.f, use = 0.f, f = 1.f, z = 0.f, unbias = 1.f;
            bool masked = false, apart = false;
            int end = 0;  // columns of its page that the row sees
            const uint32_t s_addr = tc::lane_addr(tm, quad, 128 * b + 64 * pg);
            // (the column loops are rolled: their bodies then stay in the instruction caches)
            auto scores = [&](int i, float(&x)[32]) {
                tc::ld32(s_addr + 32 * i, x);
                tc::wait_ld();
                if (masked) {
                    asm volatile("" ::: "memory");  // (a branch, not predicates)
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (32 * i + c >= end) x[c] = -INFINITY;
                }
            };
            if (active) {
                // factor of the raw scores, and the exponents of both pages' value scales
                int vexp[2];
                bool has[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const PageMeta e = meta[(wk.i + x) % kMeta];
                    has[x] = x < wk.pages && e.block >= 0;
                    vexp[x] = exponent_of(e.vs);
                    if (x == pg) f = has[x] ? fmaxf(qs * e.ks, 1e-37f) : 1.f;
                }
                const bool have = pg == 0 ? has[0] : has[1];
                end = have ? limit - (un.page + pg) * kPage : 0;
                masked = !have || (un.page + pg + 1) * kPage > un.len - p.D + 1;
                // (read twice: the maximum first, then the weights)
                float mx = -INFINITY;
#pragma unroll 1
                for (int i = 0; i < 2; ++i) {
                    float x[32], part[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    scores(i, x);
#pragma unroll
                    for (int c = 0; c < 32; ++c) part[c & 3] = fmaxf(part[c & 3], x[c]);
                    mx = fmaxf(mx, fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3])));
                }
                mx *= f;
                *mine = mx;
                pair_sync();
                const float theirs = *other;
                pair_sync();
                const float mnew = fmaxf(m, fmaxf(mx, theirs)), before = m;
                const bool move = wk.first || mnew - m > kLazy || (m == -INFINITY && mnew > m);
                if (move) m = mnew;
                use = m == -INFINITY ? 0.f : m;
                int most = kNoUnit;  // the tile's largest contribution
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    if (has[x]) most = max(most, contribution(vexp[x], x == pg ? mx : theirs, use));
                int to = unit;
                if (move) to += __float2int_ru(fmaxf(before - use, kFarBelow));
                if (move || most > to + (int)kLazy) to = max(to, most);
                if (!wk.first && (move || to != unit)) {
                    const float2 by = moved(move ? before : use, use, unit, to);
                    l *= by.x;
                    fix = by.y;
                }
                unit = to;
                const int e = have ? kBias + (pg == 0 ? vexp[0] : vexp[1]) - unit : 0;
                apart = e < kApart;
                z = (float)e;
                unbias = pow2(-e);
                z -= use;
            }
            if (j > 0 && !warp_wait(&bars.pv_done, j - 1, &abort_flag)) ok = false;
            if (active) {
                if (__any_sync(~0u, !wk.first && fix != 1.f)) {
                    tc::fence_after_sync();
#pragma unroll 1
                    for (int c = 0; c < HD / 2; c += 16) {
                        float o[16];
                        tc::ld16(o_addr + c, o);
                        tc::wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] *= fix;
                        tc::st16(o_addr + c, o);
                    }
                    tc::wait_st();
                }
                float rs = 0.f;
                const uint32_t p_addr = tc::lane_addr(tm, quad, C::kP + 64 * b + 32 * pg);
#pragma unroll 1
                for (int i = 0; i < 2; ++i) {
                    float x[32];
                    scores(i, x);
                    if (apart) {  // these weights may vanish next to a larger value scale: their sum apart
                        asm volatile("" ::: "memory");
#pragma unroll
                        for (int c = 0; c < 32; ++c) rs += ex2(fmaf(x[c], f, -use));
                    }
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
                    uint32_t pk[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const float x0 = ex2(fmaf(x[2 * c], f, z)), x1 = ex2(fmaf(x[2 * c + 1], f, z));
                        sum[2 * (c & 1)] += x0;
                        sum[2 * (c & 1) + 1] += x1;
                        pk[c] = pack_f16(x0, x1);
                    }
                    tc::st16u(p_addr + 16 * i, pk);
                    if (!apart) rs = fmaf((sum[0] + sum[2]) + (sum[1] + sum[3]), unbias, rs);
                }
                tc::wait_st();
                l += rs;
                if (p.weight_out != nullptr && valid && pg < wk.pages)
                    ws[lay.page_w + qrow * p.max_pages + un.page + pg] = rs > 0.f ? log2f(rs) + use : -INFINITY;
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.p_full[b]);
            if (!wk.last) continue;

            // ---- the item's end
            if (!warp_wait(&bars.pv_done, j, &abort_flag)) ok = false;
            tc::fence_after_sync();
            const bool from_start = wk.page0 == 0;
            const bool whole = from_start && un.page + wk.pages == un.pages;
            if (active) {
                *mine = l;
                pair_sync();
                const float l0 = pg == 0 ? l : *other, l1 = pg == 0 ? *other : l;
                pair_sync();
                const float total = l0 + l1;
                const float in = pow2(unit) * (1.f / (float)(1 << kBias));
                const float fo = total == 0.f ? 0.f : whole ? 1.f / total : 1.f;
                const int64_t slot = 2 * (int64_t)blockIdx.x + (from_start ? 1 : 0);
                T *dst = static_cast<T *>(p.out) + qrow * HD + pg * (HD / 2);
                float *part = ws + lay.part_o + (slot * lay.PR + r) * HD + pg * (HD / 2);
                const bool nan = v_nan != 0;
#pragma unroll 1
                for (int c = 0; c < HD / 2; c += 16) {
                    __syncwarp();  // (the rows that are not written rejoin for the next load)
                    float o[16];
                    tc::ld16(o_addr + c, o);
                    tc::wait_ld();
                    if (!valid || !ok) continue;
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = fo == 0.f ? 0.f : o[e] * in * fo;
                    if (nan) {  // the NaN values that this row sees
                        asm volatile("" ::: "memory");
                        for (int pos = max(un.len - p.D + 1, 0); pos < limit; ++pos) {
                            const int block = page_meta(p, p.block_table[(int64_t)un.n * p.max_pages + pos / kPage], h).block;
                            if (block < 0) continue;
                            const unsigned char *vb = p.v_pages + (int64_t)block * C::kHalf +
                                                      (pg * (HD / 2) + c) * kPage + pos % kPage;
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if ((vb[e * kPage] & 0x7f) == 0x7f) o[e] = NAN;
                        }
                    }
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 16; e += 8)
                            *reinterpret_cast<uint4 *>(dst + c + e) =
                                make_uint4(pack_bf16(o[e], o[e + 1]), pack_bf16(o[e + 2], o[e + 3]),
                                           pack_bf16(o[e + 4], o[e + 5]), pack_bf16(o[e + 6], o[e + 7]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            *reinterpret_cast<float4 *>(part + c + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                }
                if (valid && ok && pg == 0) {
                    if (whole) {
                        const float lse2 = total == 0.f ? -INFINITY : m + log2f(total);
                        if (p.lse) p.lse[qrow] = lse2 * kLn2;
                        if (p.weight_out) ws[lay.lse2 + qrow] = lse2;
                    } else {
                        ws[lay.part_m + slot * lay.PR + r] = m;
                        ws[lay.part_l + slot * lay.PR + r] = total;
                    }
                }
            }
            if (from_start && tid == 0 && ok && !lay.whole) write_desc(ws, lay, un, wk.cur, HR, whole, W, U);
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.o_free);
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) tc::tmem_dealloc(tm, kTmem);
    if (tid == 0 && abort_flag && p.err_flag) atomicOr(p.err_flag, KDA_DEVERR_TIMEOUT);
}

template <int HD>
cudaError_t launch_dim(const AttnDecodeParams &p, const Layout &lay, cudaStream_t st) {
    auto kern = decode_attn_tc_kernel<HD>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(kern), Cfg<HD>::kBytes, done);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)lay.workers, kThreads, Cfg<HD>::kBytes, st>>>(p, lay);
    return cudaGetLastError();
}

}  // namespace

namespace dec {

cudaError_t launch_tc(const AttnDecodeParams &p, const Layout &lay, int d, cudaStream_t st) {
    return d == 128 ? launch_dim<128>(p, lay, st) : launch_dim<64>(p, lay, st);
}

}  // namespace dec
}  // namespace kda
