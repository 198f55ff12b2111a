// Attention of chunks of rows over runs of pages on tcgen05 (bf16, d = 64 or
// 128): prefixes that many sequences share, and what follows them.
//
// The formulas and the counting of outputs are those of kda_attn_decode_tc.cu
// (value scales in the exponents of fp16 weights, values turned into fp16).  Keys
// are multiplied as the bytes that they are, with queries as an e4m3 and an e5m2
// term (and what these leave in fp32, where it counts: see load_queries): they
// need no conversion and half the room, so that four blocks are in flight.  And
// two tiles of 128 rows are.  A chunk of more than 128 rows is two tiles, and a block of 128
// positions is read, turned into fp16 and used for both.  A chunk of up to 128
// rows is both tiles itself: they take its blocks in turn, and their results are
// added up at the end.  Either way the tensor cores work on one tile while the
// other one's softmax runs:
//
//   task k is a block on tile k % 2:   ... PV(k), QK(k + 2), PV(k + 1), QK(k + 3) ...
//
//   warps 0-7, 8-15 softmax of tile 0 and 1: thread = row and page of the block, whose
//                   weights go back over its scores as fp16.  The two threads of a row
//                   tell each other their largest score, and keep the same maximum and
//                   unit; an item's query rows and results
//   warps 16, 17    products of tile 0 and 1
//   warps 18, 19    look up pages, issue the copies of keys, of values (and prefetches
//                   into L2 before them).  Every copy costs its warp 400 to 800 cycles
//                   of waiting and issuing: one warp for both bounded a block (3500)
//   warps 20-27     conversion of values
//
// The chunks are cut into workers' ranges by the plan (kda_attn_shared.cu); a
// worker is one CTA on one SM.  Tensor memory: S of both tiles (P over them) and
// O of both, 4 x 128 columns.  Rows of a tile that do not exist stay garbage in
// lanes of their own.
//
// Weights are one fp16 term (11 bits), as in the kernels of whole sequences in bf16.
// Outputs are added up in tensor memory over a worker's whole share of an item,
// 16 positions at a time, by tensor cores that truncate (the warps' kernel adds
// page by page to nearest): after 102 400 positions the error against 64 bits is
// 0.00169 where fp32 sums have 0.00168, the outputs' own rounding.
//
// What bounds it: the chain scores - softmax - outputs of a tile, about 2 700
// cycles a block, of which the tensor pipe has 1 024; every role's code runs in
// short loops, because code that runs straight through is bound by its own
// fetching (3 to 5 cycles an instruction).  Measured (d = 128): 32 sequences after
// one prefix of 102 400 positions, 128 rows, 75 us cold, 2.8 TB/s of pages, tensor pipe 29 %;
// 40 sequences of 7 tokens, 32 heads over 4, after five prefixes of up to 160 pages
// 54 us, 19 %.  In whole calls the steps were (these two cases): 126 and 109 us with one
// thread a row; 106 and 81 with two threads a row and rolled loops of 32 columns
// (straight-line code 138 and 89; without turns 110 and 80); 107 and 74 with loops
// of 16; the rest is the plan's (kda_attn_shared.cu).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "kda_attn_decode.cuh"
#include "kda_attn_internal.h"
#include "kda_attn_shared.cuh"
#include "kda_bulk.cuh"
#include "kda_internal.h"
#include "kda_tc.cuh"

namespace kda {
namespace {

using namespace dec;

constexpr int kThreads = 896;
constexpr int kSoftWarps = 16;
constexpr int kMmaWarp = 16, kLoadWarp = 18;
constexpr int kConvWarp = 20, kConvWarps = 8;
constexpr int kKeyBlocks = 4;  // in flight
// Page look-ups at a time, and kept: when one group is looked up, the softmax may be six blocks behind.
constexpr int kFetch = 16, kMetaRing = 32;
static_assert(kFetch + 2 * (kKeyBlocks + 2) <= kMetaRing, "no entry is overwritten before it is read");
constexpr uint32_t kTmem = 512;
constexpr float kLazy = 8.f;
constexpr int kSoftRegs = 80, kOtherRegs = 56;
static_assert(32 * kSoftWarps * kSoftRegs + (kThreads - 32 * kSoftWarps) * kOtherRegs <= kThreads * 72, "registers of a launched CTA");
constexpr int kBias = 7;  // log2 of the weights' fp16 scale
// What the queries' two terms may leave out of a score (base 2) before it is added in fp32: as much as a weight is
// rounded by.  It is compared with the sum of what is left times the largest key that a page's scale can hold, so rows
// of normal elements leave less until their scores reach thousands.
constexpr float kLeftOut = 0x1p-11f;
constexpr float kLeastQuery = 0x1p-6f, kMostQuery = 448.f;  // scaled elements between these are held by the two terms

template <int HD>
struct Cfg {
    static constexpr int kHalf = HD * kPage;             // bytes of a page's keys (or values)
    static constexpr int kKeys = 128 * HD;               // bytes of a block's keys, and of a term of a tile's queries
    static constexpr int kSlots = HD == 128 ? 4 : 8;     // of the values' ring: kDepth for the first page of a block, and the second
    static constexpr int kDepth = kSlots / 2;
    static __device__ __forceinline__ int slot_of(int pg, int n) { return pg * kDepth + n % kDepth; }  // of the n-th such page
    static constexpr int kOp = 128 * HD * 2;             // an fp16 operand of 128 rows of HD, or HD rows of 128
    static constexpr int kTiles = 4 * kOp + kKeyBlocks * kKeys + kSlots * kHalf;  // Q and V twice, K, the ring
    static constexpr uint32_t kRow = HD;                 // bytes of a key row: swizzled as a whole
    static constexpr uint64_t kSwizzle = HD == 128 ? 2 : 4;  // descriptor code of the 128- and 64-byte swizzle
};

// Behind the tiles.
struct Small {
    uint64_t full[8], empty[8];  // the values' ring
    uint64_t k_full[kKeyBlocks], k_free[kKeyBlocks], v_ready[2], v_free[2], s_full[2], p_full[2], drain[2];
    uint64_t q_full, o_full, o_free;
    uint32_t tmem_base;
    int abort_flag;
    volatile int v_nan;  // a NaN was set aside among the values that not every row sees
    int8_t q_exp[256];
    float q_left[2][4];  // of items in turn and groups of 64 rows: the sum of |what two terms leave|
    float met[2][2][128];         // by tile, page and row: what the threads of a row tell each other
    PageMeta meta[kMetaRing];     // by the keys' warp
    int8_t v_there[kMetaRing];    // by the values' warp: the page is in the cache
};
static_assert(sizeof(Small) + Cfg<128>::kTiles <= 232448, "shared memory of a CTA");

__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t phase, volatile int *abort_flag) {
    return __all_sync(~0u, mbar_wait_or_abort(bar, phase & 1u, abort_flag));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// A value that is the same in all lanes, told to the compiler: roles are then run
// with uniform branches and descriptors (the products' issue otherwise takes the
// way of one lane of a diverged warp, 165 cycles each instead of 65).
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(~0u, x, 0); }

// The worker's items, in order: every role walks them by itself, in whole warps.
struct Items {
    int c, h, page, c_end, h_end, page_end, Hkv;  // the next item (from its page), and the end of the range
    // the item at hand
    AttnChunk chunk;
    int chunk_no, head, pages, page0, page1;  // of the chunk; the range's share of them
    int item, task0, tasks, unit0;            // items, tasks and pages before it
    bool wide;

    __device__ __forceinline__ void begin(const int4 &from, const int4 &to, int heads) {
        c = uniform(from.x); h = uniform(from.y); page = uniform(from.z);
        c_end = uniform(to.x); h_end = uniform(to.y); page_end = uniform(to.z);
        Hkv = heads;
        item = -1; task0 = tasks = unit0 = 0; page0 = page1 = 0;
    }
    __device__ __forceinline__ bool next(const AttnDecodeParams &p) {
        task0 += tasks;
        unit0 += page1 - page0;
        while (true) {
            if (c > c_end || (c == c_end && (h > h_end || (h == h_end && page >= page_end)))) return false;
            const AttnChunk &x = p.chunks[c];
            chunk.len = uniform(x.len);
            chunk.rows = uniform(x.rows);
            chunk.seen = uniform(x.seen);
            chunk.tok0 = uniform(x.tok0);
            chunk.base = uniform(x.base);
            chunk.limit = uniform(x.limit);
            chunk.table = x.table;
            pages = (chunk.len + kPage - 1) / kPage;
            if (page < pages) break;
            ++c;  // (no pages)
            h = page = 0;
        }
        chunk_no = c; head = h; page0 = page;
        page1 = c == c_end && h == h_end ? min(page_end, pages) : pages;
        wide = chunk.rows > 128;
        tasks = ((page1 - page0 + 1) / 2) << (wide ? 1 : 0);
        ++item;
        page = 0;
        if (++h == Hkv) {
            h = 0;
            ++c;
        }
        return true;
    }
    __device__ __forceinline__ int blocks() const { return (page1 - page0 + 1) / 2; }
    __device__ __forceinline__ int pages_of_block(int b) const { return min(2, page1 - page0 - 2 * b); }
};

__device__ __forceinline__ void st8u(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {  // to nearest even
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// Byte offset of (row, channel) of a tile of e4m3 rows, swizzled as the tensor
// copies leave the keys: 16-byte unit u of a 128-byte row r at u ^ (r % 8), of a
// 64-byte row at u ^ (r / 2 % 4).
template <int HD>
__device__ __forceinline__ uint32_t key_off(int row, int ch) {
    const int u = ch >> 4;
    return (uint32_t)(row * HD + ((HD == 128 ? u ^ (row & 7) : u ^ ((row >> 1) & 3)) << 4) + (ch & 15));
}

// Descriptor of such a tile (8-row groups follow one another), as of 128-byte rows of fp16.
template <int HD>
__device__ __forceinline__ uint64_t desc_keys(uint32_t saddr) {
    using C = Cfg<HD>;
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(8 * C::kRow >> 4) << 32) | ((uint64_t)1 << 46) |
           (C::kSwizzle << 61);
}

__device__ __forceinline__ uint32_t to_e5m2x2(float lo, float hi) {  // to nearest even
    uint16_t d;
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// kind::f8f6f4 with 8-bit operands and fp32 accumulation; a step is 32 channels.
__device__ __forceinline__ void mma_f8_ss_warp(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Pairs of a query's elements, scaled (see load_queries): their first term, of e4m3, their second, of e5m2, and what
// the two leave: all of an element that is too large for e4m3.
struct Terms {
    uint32_t first, second;
    float2 left;
};
__device__ __forceinline__ Terms terms_of(float x0, float x1) {
    Terms t;
    // (an infinite query makes its row NaN, as its scores would)
    const float y0 = fabsf(x0) <= kMostQuery ? x0 : x0 - x0, y1 = fabsf(x1) <= kMostQuery ? x1 : x1 - x1;
    t.first = to_e4m3x2(y0, y1);
    uint32_t u, unused;
    e4m3x4_to_f16(t.first, u, unused);
    const float2 first = unpack_f16(u);
    t.second = to_e5m2x2(y0 - first.x, y1 - first.y);
    const float2 second = unpack_f16((t.second & 0xffu) << 8 | (t.second & 0xff00u) << 16);  // (e5m2 is fp16's upper byte)
    t.left = make_float2((x0 - first.x) - second.x, (x1 - first.y) - second.y);
    return t;
}
__device__ __forceinline__ float row_scale(int ex) { return __uint_as_float((uint32_t)(127 + 7 - ex) << 23); }

// An item's query rows, scaled by powers of two to 2^7..2^8, as an e4m3 and an e5m2 term.  Of an element's 8 bits the
// first holds 4 and leaves at most half of the last of these: 3 bits, which the second holds exactly down to elements
// of 2^-6, 2^-13 of the row's largest.  Of those below it leaves up to 2^-14, 2^-21 of the largest, and the softmax
// adds that in fp32 where it may count (add_left).  A row with a few elements of more than 2^7 times the others is
// scaled by the others, and these few are left whole: it is one or two channels then that the softmax adds, not all
// (64 sequences after 128 pages, every row with a channel of 2^10, 2^14, 2^20 times the others: 137, 120, 116 us instead
// of 265, 916, 1068; without one 63).  All softmax threads, 8 channels each.
template <int HD>
__device__ __forceinline__ void load_queries(const AttnDecodeParams &p, const Items &it, unsigned char *sq, int8_t *exps, float *lefts,
                                             int id) {
    constexpr int PIECES = HD / 8, STEP = 32 * kSoftWarps / PIECES, HELD = 2;  // pieces of a row; rows of a pass; passes together
    const int piece = id % PIECES, rows = it.chunk.rows;
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) + (int64_t)it.chunk.tok0 * p.q_stride + (int64_t)it.head * p.G * HD + 8 * piece;
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += HELD * STEP) {  // (by all threads)
        uint4 raw[HELD];
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int row = r0 + i * STEP + id / PIECES, tok = row / p.G, gi = row - tok * p.G;
            raw[i] = make_uint4(0, 0, 0, 0);
            if (row < rows) raw[i] = *reinterpret_cast<const uint4 *>(q + (int64_t)tok * p.q_stride + gi * HD);
        }
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int row = r0 + i * STEP + id / PIECES;
            const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
            float amax = 0.f, amin = INFINITY;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x0 = fabsf(__uint_as_float(w[e] << 16)), x1 = fabsf(__uint_as_float(w[e] & 0xffff0000u));
                amax = fmaxf(amax, fmaxf(x0, x1));
                amin = fminf(amin, fminf(x0, x1));
            }
            const float mine = amax;
#pragma unroll
            for (int o = 1; o < PIECES; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
            int ex = (int)(__float_as_uint(amax) >> 23) - 127;
            ex = ex < -100 ? -100 : ex > 127 ? 127 : ex;  // (128: infinities and NaN stay what they are)
            float mul = row_scale(ex);
            uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const Terms t = terms_of(__uint_as_float(w[e] << 16) * mul, __uint_as_float(w[e] & 0xffff0000u) * mul);
                hi[e >> 1] |= t.first << (16 * (e & 1));
                lo[e >> 1] |= t.second << (16 * (e & 1));
            }
            if (__any_sync(~0u, row < rows && amin * mul < kLeastQuery)) {  // (one warp in twenty, of normal elements)
                // pieces of the row with large elements: where they are few, the others' largest is the row's scale,
                // but within 2^100 of the row's, which has to stay finite
                const bool large = mine > 0x1p-7f * amax;
                const int pieces = __popc(__ballot_sync(~0u, large) >> ((id & 31) / PIECES * PIECES) & ((1u << PIECES) - 1));
                float most = large ? 0.f : mine;
#pragma unroll
                for (int o = 1; o < PIECES; o <<= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, o));
                if (pieces <= PIECES / 8 && most > 0.f && amax <= 3.402823466e38f)
                    ex = max(max((int)(__float_as_uint(most) >> 23) - 127, ex - 100), -100);
                mul = row_scale(ex);
                uint64_t first = 0, second = 0;
                float left = 0.f;
                uint4 v = raw[i];
#pragma unroll 1
                for (int e = 0; e < 64; e += 16) {
                    const Terms t = terms_of(__uint_as_float(v.x << 16) * mul, __uint_as_float(v.x & 0xffff0000u) * mul);
                    first |= (uint64_t)t.first << e;
                    second |= (uint64_t)t.second << e;
                    left += fabsf(t.left.x) + fabsf(t.left.y);
                    v.x = v.y; v.y = v.z; v.z = v.w;
                }
                hi[0] = (uint32_t)first; hi[1] = (uint32_t)(first >> 32);
                lo[0] = (uint32_t)second; lo[1] = (uint32_t)(second >> 32);
                if (row < rows && left > 0.f) atomicAdd(&lefts[row >> 6], left * __uint_as_float((uint32_t)(127 - 7 + ex) << 23));
            }
            if (row < rows) {
                if (piece == 0) exps[row] = (int8_t)ex;
                // 8 bytes of the row, in its swizzled units of 16
                unsigned char *dst = sq + (row >> 7) * 2 * Cfg<HD>::kKeys + key_off<HD>(row & 127, 8 * piece);
                *reinterpret_cast<uint2 *>(dst) = make_uint2(hi[0], hi[1]);
                *reinterpret_cast<uint2 *>(dst + Cfg<HD>::kKeys) = make_uint2(lo[0], lo[1]);
            }
        }
    }
}

// Adds what the terms of the thread's row (-1: none) leave of its scores to the 64 of a page (if it is in the cache), in
// tensor memory at s_addr.  By whole warps, in those rows alone where it may be more than kLeftOut: a row's result does
// not depend on others.  A call, and little code rather than quick code: the rows that come here are rare, and inlined
// it cost the others 6 us of a document's 104 (as it is, 2: the check).
template <int HD>
__device__ __noinline__ void add_left(const AttnDecodeParams &p, const Items &it, uint32_t s_addr, int row, const PageMeta *at,
                                      const int8_t *exps) {
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q);
    const PageMeta page = *at;
    if (page.block < 0) return;
    float mul = 0.f, bound = 0.f;
    if (row >= 0) {
        q += ((int64_t)it.chunk.tok0 + row / p.G) * p.q_stride + (int64_t)(it.head * p.G + row % p.G) * HD;
        mul = row_scale(exps[row]);
        bound = kLeftOut / (448.f * kLog2e) * mul / page.ks / p.scale;  // (in this order within fp32's range)
    }
    auto left_of = [&](uint32_t w) { return terms_of(__uint_as_float(w << 16) * mul, __uint_as_float(w & 0xffff0000u) * mul).left; };
    // the row's pairs of channels of which something is left, and how much of all
    uint64_t pairs = 0;
    float sum = 0.f;
#pragma unroll 1
    for (int c = 0; row >= 0 && c < HD; c += 8) {
        uint4 v = *reinterpret_cast<const uint4 *>(q + c);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        float amin = INFINITY, amax = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x0 = fabsf(__uint_as_float(w[e] << 16)), x1 = fabsf(__uint_as_float(w[e] & 0xffff0000u));
            amin = fminf(amin, fminf(x0, x1));
            amax = fmaxf(amax, fmaxf(x0, x1));
        }
        if (!(amin * mul < kLeastQuery || amax * mul > kMostQuery)) continue;
#pragma unroll 1
        for (int e = 0; e < 4; ++e) {
            const float2 x = left_of(v.x);
            sum += fabsf(x.x) + fabsf(x.y);
            if (x.x != 0.f || x.y != 0.f) pairs |= (uint64_t)1 << (c / 2 + e);
            v.x = v.y; v.y = v.z; v.z = v.w;
        }
    }
    if (!(sum > bound)) pairs = 0;  // (NaN: its scores are NaN already)
    // each row its own pairs, one at a time: the lanes' bytes are of one key's row
    while (__any_sync(~0u, pairs != 0)) {
        const int c = pairs != 0 ? 2 * (__ffsll(pairs) - 1) : 0;
        float2 x = make_float2(0.f, 0.f);
        if (pairs != 0) x = left_of(*reinterpret_cast<const uint32_t *>(q + c));
        pairs &= pairs - 1;
        __syncwarp();
        const unsigned char *key = p.k_pages + (int64_t)page.block * Cfg<HD>::kHalf + c;
#pragma unroll 1
        for (int i = 0; i < 4; ++i, key += 16 * HD) {
            float s[16];
            tc::ld16(s_addr + 16 * i, s);
            tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                uint32_t u, unused;
                e4m3x4_to_f16(*reinterpret_cast<const uint16_t *>(key + e * HD), u, unused);
                const float2 k = unpack_f16(u);
                s[e] = fmaf(x.x, k.x, fmaf(x.y, k.y, s[e]));
            }
            tc::st16(s_addr + 16 * i, s);
            tc::wait_st();
        }
    }
}

// Four lanes that hold 16 columns of a row each exchange them: lane j then holds
// columns 4 j.. of the four rows, the quad's first row in o[0..3], so that four
// lanes write 64 bytes of a row together.
__device__ __forceinline__ void quad_transpose(float (&o)[16]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int bit = 1; bit <= 2; bit <<= 1) {
        const bool up = (lane & bit) != 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k & bit) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float &lo = o[4 * k + e], &hi = o[4 * (k + bit) + e];
                const float got = __shfl_xor_sync(~0u, up ? lo : hi, bit);
                if (up) lo = got;
                else hi = got;
            }
        }
    }
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1) parts_tc_kernel(const AttnDecodeParams p, const PartsPlan plan,
                                                               const __grid_constant__ CUtensorMap keys) {
    using C = Cfg<HD>;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char *sq = smem, *sk = sq + 4 * C::kKeys, *sv = sk + kKeyBlocks * C::kKeys, *ring = sv + 2 * C::kOp;
    Small &S = *reinterpret_cast<Small *>(smem + C::kTiles);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float *part = plan.part;
    volatile int *abort_flag = &S.abort_flag;

    if (tid == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(&S.full[i], 1);
            mbar_init(&S.empty[i], kConvWarps / 2);
        }
        for (int i = 0; i < kKeyBlocks; ++i) {
            mbar_init(&S.k_full[i], 1);
            mbar_init(&S.k_free[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.v_ready[i], kConvWarps);
            mbar_init(&S.v_free[i], 2);
            mbar_init(&S.s_full[i], 1);
            mbar_init(&S.p_full[i], kSoftWarps / 2);
            mbar_init(&S.drain[i], 1);
        }
        mbar_init(&S.q_full, kSoftWarps);
        mbar_init(&S.o_full, 2);
        mbar_init(&S.o_free, kSoftWarps);
        fence_barrier_init();
        for (int i = 0; i < 8; ++i) S.q_left[i >> 2][i & 3] = 0;
        S.abort_flag = 0;
        S.v_nan = 0;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");  // for the plan
    const int4 from = plan.starts[blockIdx.x], to = plan.starts[blockIdx.x + 1];
    Items it;
    it.begin(from, to, p.Hkv);
    {
        Items probe = it;
        if (!probe.next(p)) return;  // (the whole CTA)
    }
    if (warp == kMmaWarp) tc::tmem_alloc(&S.tmem_base, kTmem);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = S.tmem_base;
    constexpr int kO = 256;  // tensor memory column of tile 0's O; tile 1's 128 behind it; S at 0 and 128

    // (72 registers a thread at launch)
    if (warp >= kSoftWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kLoadWarp || warp == kLoadWarp + 1) {
            // ---------------- page look-ups and copies, of keys (a block at a time, swizzled rows that the products read as
            // they are) or of values (a page at a time, bytes that are converted)
            const bool is_v = warp != kLoadWarp;
            int copies[2] = {0, 0}, block = 0;  // values: first pages of blocks, and second ones; keys: blocks
            bool ok = true;
            while (ok && it.next(p)) {
                const int count = it.page1 - it.page0;
                for (int i0 = 0; ok && i0 < count; i0 += kFetch) {
                    // a lane a page: this group's, and behind them the next group's into L2
                    int mine = -1;
                    const int i = i0 + lane;
                    if (lane < 2 * kFetch && i < count) {
                        const int id = p.block_table[it.chunk.table + it.page0 + i];
                        if (lane < kFetch) {
                            const PageMeta e = page_meta(p, id, it.head);
                            mine = e.block;
                            if (is_v) S.v_there[(it.unit0 + i) % kMetaRing] = mine >= 0;
                            else S.meta[(it.unit0 + i) % kMetaRing] = e;
                        } else if (id >= 0 && id < p.num_pages) {
                            bulk_prefetch_l2((is_v ? p.v_pages : p.k_pages) + ((int64_t)id * p.Hkv + it.head) * C::kHalf, C::kHalf);
                        }
                    }
                    __syncwarp();
                    for (int x0 = 0; ok && x0 < min(kFetch, count - i0); x0 += 2) {
                        const int pages = min(2, count - i0 - x0);
                        int page[2];
#pragma unroll
                        for (int pg = 0; pg < 2; ++pg) page[pg] = __shfl_sync(~0u, mine, x0 + pg);
                        if (pages < 2) page[1] = -1;
                        if (!is_v) {
                            const int slot = block % kKeyBlocks;
                            ok = block < kKeyBlocks || warp_wait(&S.k_free[slot], block / kKeyBlocks - 1, abort_flag);
                            if (!ok) break;
                            ++block;
                            if (lane == 0) {
                                const int bytes = ((page[0] >= 0) + (page[1] >= 0)) * C::kHalf;
                                if (bytes > 0) mbar_arrive_expect_tx(&S.k_full[slot], bytes);
                                else mbar_arrive(&S.k_full[slot]);
#pragma unroll
                                for (int pg = 0; pg < 2; ++pg)
                                    if (page[pg] >= 0)
                                        tma_load_3d(sk + slot * C::kKeys + pg * C::kHalf, &keys, 0, 0, page[pg], &S.k_full[slot]);
                            }
                            __syncwarp();
                            continue;
                        }
#pragma unroll
                        for (int pg = 0; pg < 2; ++pg) {
                            if (pg >= pages) break;
                            const int n = copies[pg], slot = C::slot_of(pg, n);
                            ok = n < C::kDepth || warp_wait(&S.empty[slot], n / C::kDepth - 1, abort_flag);
                            if (!ok) break;
                            ++copies[pg];
                            if (lane == 0) {
                                if (page[pg] < 0) {
                                    mbar_arrive(&S.full[slot]);
                                } else {
                                    mbar_arrive_expect_tx(&S.full[slot], C::kHalf);
                                    bulk_g2s(ring + slot * C::kHalf, p.v_pages + (int64_t)page[pg] * C::kHalf, C::kHalf, &S.full[slot]);
                                }
                            }
                            __syncwarp();
                        }
                    }
                }
            }
            // every copy lands before the CTA's memory goes
            for (int n = max(0, block - kKeyBlocks); n < block; ++n)
                mbar_wait_drain(&S.k_full[n % kKeyBlocks], (uint32_t)(n / kKeyBlocks) & 1u);
#pragma unroll
            for (int pg = 0; pg < 2; ++pg)
                for (int n = max(0, copies[pg] - C::kDepth); n < copies[pg]; ++n)
                    mbar_wait_drain(&S.full[C::slot_of(pg, n)], (uint32_t)(n / C::kDepth) & 1u);
        } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
            // ---------------- products of a tile (the whole warp in step: see mma_f16_ss_warp): of each of its tasks the
            // scores, once the outputs of the task before are asked for.  A wait by parity must not take an older phase for
            // its own: within an item a tile's blocks are all or every other one, so that the one that had this one's buffer
            // was the tile's too, and between items all meet (q_full).  What frees a block counts two: one of a narrow
            // item is freed twice by its tile's warp.
            const uint32_t id_qk = tc::idesc_f16(128, 128), id_pv = tc::idesc_f16(128, HD);  // (e4m3 has fp16's code, 0)
            constexpr uint32_t kE5m2 = 1u << 7;  // of the first operand
            const int t = warp - kMmaWarp;
            const uint32_t to_s = tm + 128 * t, to_o = tm + kO + 128 * t;
            int block0 = 0;  // blocks before the item
            bool ok = true;
            // the task whose outputs are still to come: its block, and of its item: number, whether it is the tile's
            // first or last task, whether it is narrow
            int p_block = -1, p_item = 0, p_task = 0;
            bool p_first = false, p_last = false, p_narrow = false;
            auto pv = [&]() {
                if (p_block < 0) return true;
                if (!warp_wait(&S.v_ready[p_block & 1], p_block >> 1, abort_flag)) return false;
                if (p_first && p_item > 0 && !warp_wait(&S.o_free, p_item - 1, abort_flag)) return false;
                if (!warp_wait(&S.p_full[t], p_task >> 1, abort_flag)) return false;
                tc::fence_after_sync();
                const int vb = p_block & 1;
                const uint64_t va = tc::desc_sw128(tc::smem_u32(sv + vb * C::kOp));
                const uint32_t begun = p_first ? 0u : 1u;
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {  // 16 positions each; a page is one 128-byte-wide chunk of HD rows
                    constexpr uint64_t kChunk = HD * 128 >> 4, kStep = 32 >> 4;
                    tc::mma_f16_ts_warp(to_o, to_s + 64 * (ks >> 2) + 8 * (ks & 3), va + (ks >> 2) * kChunk + (ks & 3) * kStep, id_pv, ks == 0 ? begun : 1u);
                }
                tc::commit_warp(&S.v_free[vb]);
                if (p_narrow) tc::commit_warp(&S.v_free[vb]);
                if (p_last) tc::commit_warp(&S.o_full);
                p_block = -1;
                return true;
            };
            while (ok && it.next(p)) {
                ok = pv() && warp_wait(&S.q_full, it.item, abort_flag);  // (the outputs are of the item before)
                const int first = (it.task0 ^ t) & 1, every = 2;  // of the item's tasks, the tile's
                const int buf = it.wide ? first : 0;               // (a wide item's first task is of its first rows)
                if (ok && first >= it.tasks) {
                    // none (a narrow item of one block): its part of the counts, in the order of the items
                    ok = it.item == 0 || warp_wait(&S.o_free, it.item - 1, abort_flag);
                    if (ok && lane == 0) mbar_arrive(&S.o_full);
                    __syncwarp();
                }
                for (int i = first; ok && i < it.tasks; i += every) {
                    ok = pv();
                    if (!ok) break;
                    const int block = block0 + (it.wide ? i >> 1 : i), kb = block % kKeyBlocks;
                    ok = warp_wait(&S.k_full[kb], block / kKeyBlocks, abort_flag);
                    if (!ok) break;
                    tc::fence_after_sync();
                    const uint64_t qa = desc_keys<HD>(tc::smem_u32(sq + buf * 2 * C::kKeys)), ka = desc_keys<HD>(tc::smem_u32(sk + kb * C::kKeys));
                    // (unrolled, the descriptors base + constant: 32 channels are 32 bytes of a row)
#pragma unroll
                    for (int ks = 0; ks < HD / 16; ++ks) {
                        constexpr int STEPS = HD / 32;  // of a term
                        const uint64_t step = (ks % STEPS) * (32 >> 4);
                        mma_f8_ss_warp(to_s, qa + (ks / STEPS) * (C::kKeys >> 4) + step, ka + step, ks < STEPS ? id_qk : id_qk | kE5m2, ks > 0);
                    }
                    tc::commit_warp(&S.s_full[t]);
                    tc::commit_warp(&S.k_free[kb]);
                    if (!it.wide) tc::commit_warp(&S.k_free[kb]);
                    p_block = block;
                    p_item = it.item;
                    p_task = it.task0 + i;
                    p_first = i == first;
                    p_last = i + every >= it.tasks;
                    p_narrow = !it.wide;
                }
                block0 += it.blocks();
            }
            if (ok) pv();
            tc::commit_warp(&S.drain[t]);  // every product is done before the memory goes
            __all_sync(~0u, mbar_wait_drain(&S.drain[t], 0));
        } else if (warp >= kConvWarp) {
            // ---------------- conversion of values: four warps a page of the block
            const int role = warp - kConvWarp, pg = role >> 2, ct = 32 * (role & 3) + lane;  // 0..127
            int block = 0, taken = 0;  // blocks before this one; the warp's pages before it
            bool ok = true;
            while (ok && it.next(p)) {
                const int window0 = it.chunk.seen;
                for (int b = 0; ok && b < it.blocks(); ++b, ++block) {
                    const bool there = pg < it.pages_of_block(b);
                    const int buf = block & 1, slot = C::slot_of(pg, taken);
                    if (block >= 2) ok = warp_wait(&S.v_free[buf], (block >> 1) - 1, abort_flag);
                    if (ok && there) ok = warp_wait(&S.full[slot], taken / C::kDepth, abort_flag);
                    if (!ok) break;
                    const unsigned char *src = ring + slot * C::kHalf + 16 * ct;
                    {
                        // 16 positions of a channel at a time: thread = channel ct / 4 + i ROWS
                        constexpr int ROWS = 32, kTogether = 2;
                        const int r = ct >> 2, u = ct & 3;
                        unsigned char *dst = sv + buf * C::kOp + pg * HD * 128;
                        const uint32_t o0 = tc::sw128_off16(r, 16 * u, HD), o1 = tc::sw128_off16(r, 16 * u + 8, HD);
                        const bool have = there && S.v_there[(it.unit0 + 2 * b + pg) % kMetaRing] != 0;
                        const int pos0 = (it.page0 + 2 * b + pg) * kPage;
                        const bool tail = have && pos0 + kPage > window0;
#pragma unroll 1
                        for (int i0 = 0; i0 < HD / ROWS; i0 += kTogether) {
                            uint4 a[kTogether];
#pragma unroll
                            for (int i = 0; i < kTogether; ++i)
                                a[i] = have ? *reinterpret_cast<const uint4 *>(src + (i0 + i) * 2048) : make_uint4(0, 0, 0, 0);
                            if (tail) {  // bytes past the end, and NaN bytes that not every row sees, count as zero
                                const int left = it.chunk.len - pos0, seen = window0 - pos0;
#pragma unroll
                                for (int i = 0; i < kTogether; ++i) {
                                    const int at = min(min(mask_word(a[i].x, 16 * u, left, seen), mask_word(a[i].y, 16 * u + 4, left, seen)),
                                                       min(mask_word(a[i].z, 16 * u + 8, left, seen), mask_word(a[i].w, 16 * u + 12, left, seen)));
                                    if (at < kPage) S.v_nan = 1;
                                }
                            }
#pragma unroll
                            for (int i = 0; i < kTogether; ++i) {
                                uint4 y0, y1;
                                e4m3x4_to_f16(a[i].x, y0.x, y0.y);
                                e4m3x4_to_f16(a[i].y, y0.z, y0.w);
                                e4m3x4_to_f16(a[i].z, y1.x, y1.y);
                                e4m3x4_to_f16(a[i].w, y1.z, y1.w);
                                *reinterpret_cast<uint4 *>(dst + o0 + (i0 + i) * ROWS * 128) = y0;
                                *reinterpret_cast<uint4 *>(dst + o1 + (i0 + i) * ROWS * 128) = y1;
                            }
                        }
                    }
                    __syncwarp();
                    if (there && lane == 0) mbar_arrive(&S.empty[slot]);
                    taken += there ? 1 : 0;
                    if (!ok) break;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&S.v_ready[buf]);
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        // ---------------- softmax: thread = row and page of the block
        const int t = warp >> 3, pg = (warp >> 2) & 1, quad = warp & 3, r = 32 * quad + lane;
        const uint32_t s_addr = tc::lane_addr(tm, quad, 128 * t + 64 * pg);  // the page's scores, its weights over them
        const uint32_t o_addr = tc::lane_addr(tm, quad, kO + 128 * t);
        auto pair_sync = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + 4 * t + quad) : "memory"); };  // a row's pages
        auto quad_sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(9 + quad) : "memory"); };         // and tiles
        // The tiles take turns at the exponentials, in the order of the tasks: left to themselves both take them at once,
        // and wait for the products at once.
        auto my_turn = [&](int k) {
            if (k > 0) asm volatile("bar.sync %0, %1;" ::"r"(13 + t), "n"(32 * kSoftWarps) : "memory");
        };
        auto other_turn = [&]() { asm volatile("bar.arrive %0, %1;" ::"r"(14 - t), "n"(32 * kSoftWarps) : "memory"); };
        bool ok = true;
        while (it.next(p)) {
            // (after a wait gave up the loop runs on, on garbage: the warps of a row meet at barriers)
            // the query rows: the products of the item before are done (o_full)
            load_queries<HD>(p, it, sq, S.q_exp, S.q_left[it.item & 1], tid);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.q_full);
            const int half = it.wide ? (t ^ (it.task0 & 1)) : 0;
            const int row = 128 * half + r;
            const bool valid = row < it.chunk.rows;
            const bool active = 128 * half + 32 * quad < it.chunk.rows;  // some row of this warp exists
            const int limit = valid ? limit_of(p, it.chunk, row) : 0;
            const int window0 = it.chunk.seen;
            float m = -INFINITY, l = 0.f, qs = 0.f;  // l: of the thread's pages
            int unit = kNoUnit;  // the exponent that O is counted in
            float left = 0.f;  // twice what the queries' terms may leave of a score, by the page's key scale
            bool first = true;
            for (int k = it.task0 + ((it.task0 ^ t) & 1); k < it.task0 + it.tasks; k += 2) {
                if (!warp_wait(&S.s_full[t], k >> 1, abort_flag)) ok = false;
                tc::fence_after_sync();
                if (active) {
                    const int b = (k - it.task0) >> (it.wide ? 1 : 0), page = it.page0 + 2 * b + pg, pages = it.pages_of_block(b);
                    if (first) {
                        // (the sum of a group of rows, its order left open, so half of the bound: add_left looks at the row's own)
                        if (valid) qs = __uint_as_float((uint32_t)(127 - 7 + S.q_exp[row]) << 23) * p.scale * kLog2e;  // (rows that do not exist: scores of next to nothing)
                        left = S.q_left[it.item & 1][(128 * half + 32 * quad) >> 6] * (2.f * 448.f * kLog2e) * p.scale;
                    }
                    const int meta0 = (it.unit0 + 2 * b + pg) % kMetaRing;
                    // (a page that a wait which gave up has left unknown is not read)
                    if (__any_sync(~0u, S.meta[meta0].ks * left > kLeftOut && pg < pages && ok)) {
                        int mine = row;
                        asm volatile("" : "+r"(mine)::"memory");  // (nothing of the call is kept in registers beside it)
                        add_left<HD>(p, it, s_addr, mine < it.chunk.rows ? mine : -1, &S.meta[meta0], S.q_exp);
                        asm volatile("" ::: "memory");
                    }
                    const PageMeta e0 = S.meta[meta0], e1 = S.meta[(it.unit0 + 2 * b + 1 - pg) % kMetaRing];
                    const bool has = pg < pages && e0.block >= 0, other_has = 1 - pg < pages && e1.block >= 0;
                    const int vexp = exponent_of(e0.vs);
                    const float f = has ? fmaxf(qs * e0.ks, 1e-37f) : 1.f;  // positive, so that -inf stays -inf
                    const int end = has ? limit - page * kPage : 0;
                    const bool masked = !has || (page + 1) * kPage > window0;
                    // (rolled loops: code that runs straight through is bound by its own fetching)
                    float x[16];  // a quarter of the page's scores: read for the maximum, and again for the weights
                    auto scores = [&](int i) {
                        tc::ld16(s_addr + 16 * i, x);
                        tc::wait_ld();
                        if (masked) {
                            asm volatile("" ::: "memory");  // (a branch, not predicates)
#pragma unroll
                            for (int c = 0; c < 16; ++c)
                                if (c >= end - 16 * i) x[c] = -INFINITY;
                        }
                    };
                    float best[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
                    for (int i = 0; i < 4; ++i) {
                        scores(i);
#pragma unroll
                        for (int c = 0; c < 8; ++c) best[c & 1] = max3(best[c & 1], x[2 * c], x[2 * c + 1]);
                    }
                    const float raw = fmaxf(best[0], best[1]);
                    const float mx = __fmul_rn(raw, f);  // (not to be fused with the differences below)
                    // (the other thread has read what this one wrote a task ago: its weights came before these scores)
                    S.met[t][pg][r] = mx;
                    pair_sync();
                    const float other = S.met[t][1 - pg][r];
                    const float mnew = fmaxf(m, fmaxf(mx, other)), before = m;
                    const bool move = first || mnew - m > kLazy || (m == -INFINITY && mnew > m);
                    if (move) m = mnew;
                    const float use = m == -INFINITY ? 0.f : m;
                    int most = kNoUnit;  // the block's largest contribution
                    if (has) most = contribution(vexp, mx, use);
                    if (other_has) most = max(most, contribution(exponent_of(e1.vs), other, use));
                    int to = unit;
                    if (move) to += __float2int_ru(fmaxf(before - use, kFarBelow));
                    if (move || most > to + (int)kLazy) to = max(to, most);
                    float fix = 1.f;
                    if (!first && (move || to != unit)) {
                        const float2 by = moved(move ? before : use, use, unit, to);
                        l *= by.x;
                        fix = by.y;
                    }
                    unit = to;
                    // (the last product of this tile came before these scores); half of the channels each
                    if (__any_sync(~0u, !first && fix != 1.f)) {
#pragma unroll 1
                        for (int c = pg * (HD / 2); c < (pg + 1) * (HD / 2); c += 16) {
                            float o[16];
                            tc::ld16(o_addr + c, o);
                            tc::wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= fix;
                            tc::st16(o_addr + c, o);
                        }
                    }
                    first = false;
                    my_turn(k);
                    const int e = has ? kBias + vexp - unit : 0;
                    const bool apart = e < kApart;  // these weights may vanish next to a larger value scale: their sum apart
                    // scores are taken relative to the page's largest before they are scaled: however large they are,
                    // that one's difference is 0
                    const float top = raw == -INFINITY ? 0.f : -raw, off = mx - use;
                    float own = 0.f;
                    const bool some_apart = __any_sync(~0u, apart);  // (the whole warp: the stores below are the warp's)
                    const float z = off + (float)e;
                    const float2 f2 = make_float2(f, f), z2 = make_float2(z, z), t2 = make_float2(top, top);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
                    for (int i = 0; i < 4; ++i) {
                        scores(i);
                        if (some_apart) {
                            asm volatile("" ::: "memory");
#pragma unroll
                            for (int c = 0; c < 16; ++c) own += ex2(fmaf(x[c] + top, f, off));
                        }
                        __syncwarp();
                        uint32_t pk[8];
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            float2 w = fma2(add2(make_float2(x[2 * c], x[2 * c + 1]), t2), f2, z2);
                            w.x = ex2(w.x);
                            w.y = ex2(w.y);
                            sum[c & 1] = add2(sum[c & 1], w);
                            pk[c] = pack_f16(w.x, w.y);
                        }
                        st8u(s_addr + 8 * i, pk);
                    }
                    other_turn();
                    sum[0] = add2(sum[0], sum[1]);
                    l += apart ? own : (sum[0].x + sum[0].y) * pow2(-e);
                    tc::wait_st();
                } else {
                    my_turn(k);
                    other_turn();
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.p_full[t]);
            }

            // ---------------- the item's end
            if (!warp_wait(&S.o_full, it.item, abort_flag)) ok = false;
            tc::fence_after_sync();
            // (every warp has read them; they are written again for the item after the next, once this warp is in that one)
            if (tid < 4) S.q_left[it.item & 1][tid] = 0;
            const bool whole = it.page0 == 0 && it.page1 == it.pages;
            const int64_t slot = 2 * (int64_t)blockIdx.x + (it.page0 == 0 ? 1 : 0);
            const int64_t qrow = valid ? ((int64_t)it.chunk.tok0 + row / p.G) * p.Hq + it.head * p.G + row % p.G : 0;
            const bool rest = it.chunk_no >= plan.first_rest;
            float *out = whole ? (rest ? plan.rest_o : plan.prefix_o) + qrow * HD : part + plan.part_o + (slot * plan.rows + row) * HD;
            // a row's sums: of both pages' threads, and in a narrow item of both tiles' (S.met once more: every product of
            // the item is done, and so are the reads before them)
            S.met[t][pg][r] = l;
            pair_sync();
            l += S.met[t][1 - pg][r];
            float in[2] = {0.f, 0.f};  // of the tiles' O
            if (it.wide) {
                in[0] = l == 0.f ? 0.f : pow2(unit) * (1.f / (float)(1 << kBias));
            } else {
                quad_sync();
                S.met[t][pg][r] = pg == 0 ? m : l;
                quad_sync();
                const float m0 = S.met[0][0][r], l0 = S.met[0][1][r], m1 = S.met[1][0][r], l1 = S.met[1][1][r];
                quad_sync();
                if (pg == 0) S.met[t][0][r] = __int_as_float(unit);
                quad_sync();
                m = fmaxf(m0, m1);
                const float use = m == -INFINITY ? 0.f : m;
                const float g0 = fmaxf(m0 - use, kFarBelow), g1 = fmaxf(m1 - use, kFarBelow);
                // (2^g in two steps: what it is multiplied with may be large)
                const float w0 = floorf(g0), w1 = floorf(g1), r0 = ex2(g0 - w0), r1 = ex2(g1 - w1);
                in[0] = l0 == 0.f ? 0.f : r0 * pow2((int)w0 + __float_as_int(S.met[0][0][r])) * (1.f / (float)(1 << kBias));
                in[1] = l1 == 0.f ? 0.f : r1 * pow2((int)w1 + __float_as_int(S.met[1][0][r])) * (1.f / (float)(1 << kBias));
                l = l0 * r0 * pow2((int)w0) + l1 * r1 * pow2((int)w1);
            }
            const bool writes = valid && ok && (it.wide || t == 0);
            const bool nan = S.v_nan != 0;
            if (active && (it.wide || t == 0)) {
                float *row_out[4];  // of the quad's rows, this lane's columns
                const unsigned row_writes = __ballot_sync(~0u, writes) >> (lane & 28);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    row_out[k] = reinterpret_cast<float *>(__shfl_sync(~0u, reinterpret_cast<unsigned long long>(out), (lane & 28) + k)) + 4 * (lane & 3);
#pragma unroll 1
                for (int c = pg * (HD / 2); c < (pg + 1) * (HD / 2); c += 16) {  // half of the channels each
                    float o[16];
                    tc::ld16(o_addr + c, o);
                    tc::wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = in[0] == 0.f ? 0.f : o[e] * in[0];
                    if (!it.wide) {
                        float o1[16];
                        tc::ld16(o_addr + 128 + c, o1);
                        tc::wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = in[1] == 0.f ? o[e] : fmaf(o1[e], in[1], o[e]);
                    }
                    if (nan) {  // the NaN values that this row sees and others do not
                        asm volatile("" ::: "memory");
                        for (int pos = max(max(window0, 0), it.page0 * kPage); writes && pos < min(limit, it.page1 * kPage); ++pos) {
                            const int block = page_meta(p, p.block_table[it.chunk.table + pos / kPage], it.head).block;
                            if (block < 0) continue;
                            const unsigned char *vb = p.v_pages + (int64_t)block * C::kHalf + c * kPage + pos % kPage;
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if ((vb[e * kPage] & 0x7f) == 0x7f) o[e] = NAN;
                        }
                        __syncwarp();
                    }
                    quad_transpose(o);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if ((row_writes >> k) & 1u) *reinterpret_cast<float4 *>(row_out[k] + c) = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                }
            }
            if (writes && pg == 0) {
                if (whole) {
                    (rest ? plan.rest_ml : plan.prefix_ml)[qrow] = make_float2(m, l);
                } else {
                    part[plan.part_m + slot * plan.rows + row] = m;
                    part[plan.part_l + slot * plan.rows + row] = l;
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.o_free);
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) tc::tmem_dealloc(tm, kTmem);
    if (tid == 0 && S.abort_flag && p.err_flag) atomicOr(p.err_flag, KDA_DEVERR_TIMEOUT);
}

// The keys: rows of d bytes, 64 of a page and kv head, all of these.
template <int HD>
bool make_map(CUtensorMap *map, const AttnDecodeParams &p) {
    const cuuint64_t dims[3] = {(cuuint64_t)HD, (cuuint64_t)kPage, (cuuint64_t)(p.num_pages * p.Hkv)};
    const cuuint64_t strides[2] = {(cuuint64_t)HD, (cuuint64_t)(HD * kPage)};
    const cuuint32_t box[3] = {(cuuint32_t)HD, (cuuint32_t)kPage, 1}, elem[3] = {1, 1, 1};
    return tensor_map_encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<unsigned char *>(p.k_pages), dims, strides, box, elem,
                                  CU_TENSOR_MAP_INTERLEAVE_NONE, HD == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HD>
cudaError_t launch_dim(const AttnDecodeParams &p, const PartsPlan &plan, int workers, cudaStream_t st) {
    CUtensorMap keys{};
    if (tensor_map_encode_fn() == nullptr) return cudaErrorNotSupported;
    // (an empty cache has no rows to describe, and no page is copied)
    if (p.num_pages > 0 && !make_map<HD>(&keys, p)) return cudaErrorInvalidValue;
    auto kern = parts_tc_kernel<HD>;
    constexpr int bytes = Cfg<HD>::kTiles + (int)sizeof(Small);
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(kern), bytes, done);
    if (e != cudaSuccess) return e;
    return launch_after_smem(kern, dim3((unsigned)workers), kThreads, bytes, st, p, plan, keys);
}

}  // namespace

namespace dec {

cudaError_t launch_parts_tc(const AttnDecodeParams &p, const PartsPlan &plan, int workers, int d, cudaStream_t st) {
    return d == 128 ? launch_dim<128>(p, plan, workers, st) : launch_dim<64>(p, plan, workers, st);
}

}  // namespace dec
}  // namespace kda
