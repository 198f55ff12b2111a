// What the two cache attention kernels (kda_attn_decode_rows.cuh, kda_attn_decode_tc.cu)
// share: how the batch's pages are cut into workers' ranges, the workspace, and
// small conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "kda_attn_internal.h"
#include "kda_attn_math.cuh"
#include "kda_bulk.cuh"

namespace kda {
namespace dec {

constexpr int kSms = 152;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Warps per SM, by registers and by shared memory (the rings).
__host__ __device__ constexpr int warps_per_sm(int NB) { return NB == 1 ? 12 : 8; }

// How a call is run, and its workspace, in floats: for each item (sequence, kv
// head, block of R rows) the workers of its first and last page (desc), the cut
// items' partial results, two per worker (the range's first item, the range's
// last item), then the rows' lse (base 2) and page weights where weights are
// asked for.
struct Layout {
    int64_t desc, part_m, part_l, part_o, lse2, page_w, total;
    int64_t items, workers;
    int32_t R, RB, PR;  // rows of an item, row blocks, rows of a partial result
    int32_t NB, MT;     // tiles of a worker of kda_attn_decode_rows.cuh; MT = 0: kda_attn_decode_tc.cu
    int32_t whole;      // a worker per item: short rows of the block table, no item is cut, no join
};

Layout make_layout(int64_t batch, int D, int Hq, int Hkv, int d, int dtype, int64_t max_pages, bool with_weight);
// The same for `batch` chunks of up to `rows` rows, no more than fit an item.
Layout make_parts_layout(int64_t batch, int rows, int Hkv, int d, int dtype, int64_t max_pages);
// Attention of chunks (p.chunks), their parts left for a join; d and dtype as in the layout.
cudaError_t launch_parts(const AttnDecodeParams &p, const Layout &lay, int d, int dtype, cudaStream_t st);

// 2^e up to 2^127, through fp32's subnormal values down to 0.
__device__ __forceinline__ float pow2(int e) {
    const uint32_t up = (uint32_t)(min(e, 127) + 127) << 23;
    return __uint_as_float(e < -126 ? 0x800000u >> min(-126 - e, 31) : up);
}

// The exponent of a value scale (a power of two).
__device__ __forceinline__ int exponent_of(float s) { return (int)(__float_as_uint(s) >> 23) - 127; }

// How a row's output is counted.  The sum of its weights is taken relative to
// the largest weight, e^m.  Its output is not: what a page gives is its weights
// times its value scale, and the pages' scales may differ by any power of two
// (one outlier sets a page's scale), so the largest weights and the largest
// contributions may lie on different pages.  The output is counted in units of
// e^m 2^unit, `unit` no less than the largest (exponent of the page's value
// scale + log2 of its largest weight) so far; a page's fp16 weights are then
// relative to the largest contribution and what is lost of them does not count.
// Exponents are whole numbers, so the scaling is exact.
constexpr int kNoUnit = -8192;    // nothing seen yet
constexpr float kFarBelow = -4096.f;  // log2 of weights that are nothing
// Below this bias of a page's weights their sum is taken apart: with it, those
// that are 2^-100 of the largest and more still count in full.
constexpr int kApart = -25;

// log2 of the largest contribution of a page to a row, rounded up: its largest
// weight is 2^(top - use).
__device__ __forceinline__ int contribution(int scale_exp, float top, float use) {
    return scale_exp + __float2int_ru(fmaxf(top - use, kFarBelow));
}

// The factors of sum and output when the maximum goes from m to use and the
// unit from `unit` to `to` (no less than unit + the maximum's fall, rounded up).
__device__ __forceinline__ float2 moved(float m, float use, int unit, int to) {
    const float by = fmaxf(m - use, kFarBelow), whole = floorf(by), rest = ex2(by - whole);
    return make_float2(rest * pow2((int)whole), rest * pow2((int)whole + unit - to));
}

// Four e4m3 bytes as two pairs of fp16 (exact).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack_f16(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}

__device__ __forceinline__ void store2(float *p, float a, float b) { *reinterpret_cast<float2 *>(p) = make_float2(a, b); }
__device__ __forceinline__ void store2(__nv_bfloat16 *p, float a, float b) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(a, b);
}

// The length of sequence n as far as its row of the block table goes.
__device__ __forceinline__ int capped_len(const AttnDecodeParams &p, int n) {
    const int cap = p.max_pages * kPage, len = p.seq_lens[n];
    return len < 0 ? 0 : len > cap ? cap : len;
}

// PARTS: the batch's entries are chunks, not whole sequences.
template <bool PARTS = false>
__device__ __forceinline__ int pages_of(const AttnDecodeParams &p, int n, int &len) {
    len = PARTS ? p.chunks[n].len : capped_len(p, n);
    return (len + kPage - 1) / kPage;
}

// What an item of entry n needs to know of it.
struct Entry {
    AttnChunk chunk;  // PARTS
    int n, len;
};
template <bool PARTS>
__device__ __forceinline__ Entry entry_of(const AttnDecodeParams &p, int n, int len) {
    Entry e;
    if constexpr (PARTS) e.chunk = p.chunks[n];
    e.n = n;
    e.len = len;
    return e;
}
template <bool PARTS>
__device__ __forceinline__ int rows_of(const AttnDecodeParams &p, const Entry &e) {
    return PARTS ? e.chunk.rows : p.D * p.G;
}
template <bool PARTS>
__device__ __forceinline__ int64_t first_token(const AttnDecodeParams &p, const Entry &e) {
    return PARTS ? (int64_t)e.chunk.tok0 : (int64_t)e.n * p.D;
}
// Positions that row `row` sees.
__device__ __forceinline__ int limit_of(const AttnDecodeParams &p, const AttnChunk &c, int row) {
    int at = c.limit;
    if (at != AttnChunk::kManySequences) {
        at += row / p.G;
    } else {
        const int tok = c.tok0 + row / p.G;
        at = capped_len(p, tok / p.D) - p.D + 1 + tok % p.D - c.base;
    }
    return at <= 0 ? c.len : min(at, c.len);
}
template <bool PARTS>
__device__ __forceinline__ int limit_of(const AttnDecodeParams &p, const Entry &e, int row) {
    if constexpr (PARTS) return limit_of(p, e.chunk, row);
    else return e.len - p.D + 1 + row / p.G;
}
// Positions that every row sees.
template <bool PARTS>
__device__ __forceinline__ int seen_of(const AttnDecodeParams &p, const Entry &e) {
    return PARTS ? e.chunk.seen : e.len - p.D + 1;
}
template <bool PARTS>
__device__ __forceinline__ int page_id(const AttnDecodeParams &p, int n, int h, int page) {
    return PARTS ? p.block_table[p.chunks[n].table + page] : p.block_table[n * p.table_seq + h * p.table_head + page];
}

// Where a unit (one page of one item) lies: sequence n with its first unit at
// `base`, item hr = kv head * row blocks + row block, page index.
struct Cursor {
    int n;
    int64_t base;
};

// What a worker needs to know of a page: its block in the cache (page * Hkv +
// kv head; -1: none) and the scales.
struct PageMeta {
    int block;
    float ks, vs;
};

// A page that is not in the cache, or whose value scale is not a power of two
// (only its exponent is used) or key scale not a positive number, counts as
// unseen and sets the error flag.
__device__ __forceinline__ PageMeta page_meta(const AttnDecodeParams &p, int id, int h) {
    PageMeta e{-1, 0.f, 0.f};
    int err = 0;
    if (id >= 0 && id < p.num_pages) {
        const int block = id * p.Hkv + h;
        e.ks = p.k_scale[block];
        e.vs = p.v_scale[block];
        if (power_of_two(e.vs) && e.ks > 0.f && e.ks <= 3.402823466e38f) e.block = block;
        else err = KDA_DEVERR_SCALE;
    } else {
        err = KDA_DEVERR_PAGE;
    }
    if (err != 0 && p.err_flag) atomicOr(p.err_flag, err);
    return e;
}
constexpr int kMeta = 64;  // entries per worker: two batches of 32 units

struct Unit {
    int n, hr, page, pages, len;
};

// Moves the cursor to the sequence that holds unit u >= cursor.base.
template <bool PARTS>
__device__ __forceinline__ Unit locate(const AttnDecodeParams &p, int HR, Cursor &c, int64_t u) {
    Unit r;
    while (true) {
        r.pages = pages_of<PARTS>(p, c.n, r.len);
        const int64_t end = c.base + (int64_t)r.pages * HR;
        if (u < end || c.n + 1 >= p.batch) break;
        c.base = end;
        ++c.n;
    }
    const int rem = (int)(u - c.base);  // (a sequence's units fit 32 bits: checked by the launcher)
    r.n = c.n;
    r.hr = r.pages > 0 ? rem / r.pages : 0;
    r.page = r.pages > 0 ? rem - r.hr * r.pages : 0;
    return r;
}

// Clears the bytes of a value word (positions pos..pos + 3 of the page) from
// `left` on, and the NaN bytes from `seen` on; the first of the latter, or kPage.
__device__ __forceinline__ int mask_word(uint32_t &w, int pos, int left, int seen) {
    int at = kPage;
#pragma unroll
    for (int b = 3; b >= 0; --b) {
        const bool nan = ((w >> (8 * b)) & 0x7fu) == 0x7fu;
        if (pos + b >= left) {
            w &= ~(0xffu << (8 * b));
        } else if (nan && pos + b >= seen) {
            w &= ~(0xffu << (8 * b));
            at = pos + b;
        }
    }
    return at;
}

// The rows of a sequence that sees nothing.
template <typename T, int HD>
__device__ __forceinline__ void write_empty(const AttnDecodeParams &p, int n, int tid, int threads) {
    T *o = static_cast<T *>(p.out) + (int64_t)n * p.D * p.Hq * HD;
    for (int64_t i = tid; i < (int64_t)p.D * p.Hq * HD / 2; i += threads) store2(o + 2 * i, 0.f, 0.f);
    if (p.lse)
        for (int i = tid; i < p.D * p.Hq; i += threads) p.lse[(int64_t)n * p.D * p.Hq + i] = -INFINITY;
}

// Finds the range [u0, u1) of worker blockIdx.x among the batch's U units and
// the cursor of its start (in shared memory, after the call's barrier; unset
// for an empty range).  W: the workers with a range, no more than units.  Also
// writes the rows of sequences without pages, which have no unit.
template <typename T, int HD, int WARPS, bool PARTS>
__device__ __forceinline__ void find_range(const AttnDecodeParams &p, int HR, bool whole, int64_t *warp_sum, Cursor *start,
                                           int64_t &U, int64_t &W, int64_t &u0, int64_t &u1) {
    constexpr int kThreads = 32 * WARPS;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t w = blockIdx.x;
    if (whole) {  // units are counted within the sequence
        const int n = (int)(w / HR), hr = (int)(w % HR);
        int len;
        const int pages = pages_of<PARTS>(p, n, len);
        U = W = 1;
        u0 = (int64_t)hr * pages;
        u1 = u0 + pages;
        if (tid == 0) {
            *start = Cursor{n, 0};
            if (!PARTS && hr == 0 && p.err_flag && p.seq_lens[n] > p.max_pages * kPage) atomicOr(p.err_flag, KDA_DEVERR_PAGE);
        }
        if (!PARTS && pages == 0 && hr == 0) write_empty<T, HD>(p, n, tid, kThreads);
        __syncthreads();
        return;
    }
    const int per = (p.batch + kThreads - 1) / kThreads;
    const int nb = min(tid * per, p.batch), ne = min(nb + per, p.batch);
    int64_t mine = 0;
    for (int n = nb; n < ne; ++n) {
        int len;
        mine += (int64_t)pages_of<PARTS>(p, n, len) * HR;
        if (!PARTS && w == 0 && p.err_flag && p.seq_lens[n] > p.max_pages * kPage) atomicOr(p.err_flag, KDA_DEVERR_PAGE);
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(~0u, incl, o);
        if (lane >= o) incl += x;
    }
    U = __shfl_sync(~0u, incl, 31);
    int64_t excl = incl - mine;
    if constexpr (WARPS > 1) {
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        U = 0;
        for (int i = 0; i < WARPS; ++i) {
            if (i < warp) excl += warp_sum[i];
            U += warp_sum[i];
        }
    }
    W = min((int64_t)gridDim.x, max(U, (int64_t)1));
    u0 = w < W ? U * w / W : 0;
    u1 = w < W ? U * (w + 1) / W : 0;
    if (mine > 0 && u0 >= excl && u0 < excl + mine) {
        Cursor c{nb, excl};
        locate<PARTS>(p, HR, c, u0);
        *start = c;
    }
    for (int n = blockIdx.x; !PARTS && n < p.batch; n += gridDim.x) {
        if (p.seq_lens[n] > 0 && p.max_pages > 0) continue;
        write_empty<T, HD>(p, n, tid, kThreads);
    }
    __syncthreads();
}

// The worker's entry for an item whose first page it holds: the join adds up
// the parts of workers w..last.
__device__ __forceinline__ void write_desc(float *ws, const Layout &lay, const Unit &un, const Cursor &c, int HR, bool whole,
                                           int64_t W, int64_t U) {
    const int64_t end = c.base + (int64_t)(un.hr + 1) * un.pages;  // one past the item's last unit
    const int w = (int)blockIdx.x;
    *reinterpret_cast<int2 *>(ws + lay.desc + 2 * ((int64_t)un.n * HR + un.hr)) =
        make_int2(w, whole ? w : (int)((end * W + U - 1) / U - 1));  // the worker of its last unit
}

// Many rows on tcgen05 (bf16, d = 64 or 128).
cudaError_t launch_tc(const AttnDecodeParams &p, const Layout &lay, int d, cudaStream_t st);

}  // namespace dec
}  // namespace kda
