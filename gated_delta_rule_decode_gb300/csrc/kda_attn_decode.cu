// Attention of a few query tokens per sequence over the 8-bit paged cache.
//
//   s_j = scale q . k_j,  o = sum_j e^{s_j - m} v_j / sum_j e^{s_j - m}
//
// The cache is read once, so the bound is HBM: 2 d bytes per position and kv
// head.  Everything else is arranged around a steady stream of pages:
//
//  * Work is counted in pages: the items (sequence, kv head, block of 16 MT
//    query rows) of the batch are laid end to end and cut into equal ranges,
//    one per worker, so ragged batches and single long sequences balance
//    alike.  A worker is MT warps; an item that a worker holds entirely is
//    finished by it, one that is cut leaves partial results (o, m, l) that
//    join_kernel adds up in worker order.
//  * The G query heads of a kv head and the window's tokens are the rows of
//    one tile, so a page is read once for all of them.
//  * Each worker keeps a ring of shared-memory slots filled by bulk copies; a
//    page's keys and values are one contiguous block each.
//  * Products run as m16n8k16 fp16 MMAs with fp32 accumulation.  e4m3 values
//    are exact in fp16.  A query row is scaled by a power of two into fp16's
//    range, which is exact for bf16 inputs (elements below 2^-28 of the row's
//    largest are rounded); fp32 inputs take a second fp16 term for the rest.
//    The weights e^{s - m} are scaled by 2^15, so that fp16 holds them down
//    to 2^-39 of the largest; fp32 takes a second term here as well.
//  * The contraction orders of both products are permuted so that a thread's
//    operand bytes are contiguous 16-byte pieces: thread t of a quad holds
//    channels 16 t.. of a key row and positions 16 t.. of a value channel,
//    and the score tile j, column c stands for position 16 (c / 2) + 2 j +
//    c % 2, which makes the score fragment the second product's operand as
//    it is.  (The pages' value layout, a row of positions per channel, is
//    there for this.)
//  * Each page's product is accumulated from zero and added to the output in
//    fp32 round-to-nearest, because the tensor cores truncate when they add.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "kda_attn_internal.h"
#include "kda_bulk.cuh"
#include "kda_check.cuh"

namespace kda {
namespace {

constexpr int kWarpsPerCta = 8;
constexpr int kThreads = kWarpsPerCta * 32;
constexpr int kMaxCtas = 152;  // one CTA per SM (the ring takes most of its shared memory)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kPScale = 32768.f;  // fp16 scale of the weights
constexpr int kRing = 3;            // page halves in flight per warp of a worker

// Workspace, in floats: the cut items' partial results, two per worker (the
// range's first item, the range's last item), then the rows' lse (base 2) and
// page weights where weights are asked for.
struct Layout {
    int64_t desc, part_m, part_l, part_o, lse2, page_w, total;
};

__host__ __device__ inline int row_tile(int rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }
__host__ __device__ inline int64_t align64(int64_t x) { return (x + 63) / 64 * 64; }

__host__ __device__ inline Layout make_layout(int64_t batch, int D, int Hq, int Hkv, int d, int64_t max_pages,
                                              bool with_weight) {
    const int rows = D * (Hq / Hkv), MT = row_tile(rows);
    const int64_t workers = (int64_t)kMaxCtas * kWarpsPerCta / MT;
    Layout l;
    l.desc = 0;
    l.part_m = align64(4 * workers);
    l.part_l = l.part_m + align64(2 * workers * 16 * MT);
    l.part_o = l.part_l + align64(2 * workers * 16 * MT);
    l.lse2 = l.part_o + 2 * workers * 16 * MT * d;
    l.page_w = l.lse2 + (with_weight ? align64(batch * D * Hq) : 0);
    l.total = l.page_w + (with_weight ? align64(batch * D * Hq * max_pages) : 0);
    return l;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

template <typename T>
__device__ __forceinline__ float load1(const T *p);
template <>
__device__ __forceinline__ float load1<float>(const float *p) { return *p; }
template <>
__device__ __forceinline__ float load1<__nv_bfloat16>(const __nv_bfloat16 *p) { return __bfloat162float(*p); }

__device__ __forceinline__ void store2(float *p, float a, float b) { *reinterpret_cast<float2 *>(p) = make_float2(a, b); }
__device__ __forceinline__ void store2(__nv_bfloat16 *p, float a, float b) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(a, b);
}

__device__ __forceinline__ int pages_of(const AttnDecodeParams &p, int n, int &len) {
    const int cap = p.max_pages * kPage;
    len = p.seq_lens[n];
    len = len < 0 ? 0 : len > cap ? cap : len;
    return (len + kPage - 1) / kPage;
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
constexpr int kMeta = 64;  // entries per worker: two batches of 32 units

struct Unit {
    int n, hr, page, pages, len;
};

// Moves the cursor to the sequence that holds unit u >= cursor.base.
__device__ __forceinline__ Unit locate(const AttnDecodeParams &p, int HR, Cursor &c, int64_t u) {
    Unit r;
    while (true) {
        r.pages = pages_of(p, c.n, r.len);
        const int64_t end = c.base + (int64_t)r.pages * HR;
        if (u < end || c.n + 1 >= p.batch) break;
        c.base = end;
        ++c.n;
    }
    const int64_t rem = u - c.base;
    r.n = c.n;
    r.hr = r.pages > 0 ? (int)(rem / r.pages) : 0;
    r.page = r.pages > 0 ? (int)(rem - (int64_t)r.hr * r.pages) : 0;
    return r;
}

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

template <typename T, int HD, int MT>
struct Smem {
    static constexpr int kHalf = HD * kPage;  // bytes of a page's keys (or values)
    static constexpr int kWorkers = kWarpsPerCta / MT;
    static constexpr int kSlots = kRing * MT * (128 / HD);  // per worker
    static constexpr int kRingBytes = kWorkers * kSlots * kHalf;
    static constexpr int kBars = 2 * kWorkers * kSlots;
    static_assert(kSlots / 2 + 1 < kMeta / 2, "copies run at most a batch ahead of the page metadata in use");
    static constexpr int kBytes = 128 + kRingBytes + kBars * 8 + kWorkers * (16 + kMeta * 12);
};

template <typename T, int HD, int MT>
__global__ void __launch_bounds__(kThreads, 1) decode_attn_kernel(const AttnDecodeParams p) {
    using S = Smem<T, HD, MT>;
    constexpr int TERMS = sizeof(T) == 4 ? 2 : 1;
    constexpr int KS = HD / 16;    // contraction steps of the score product
    constexpr int NT = HD / 8;     // column tiles of the output
    constexpr int R = 16 * MT;     // rows of an item
    constexpr int SL = S::kSlots;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *ring_all = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    uint64_t *bars = reinterpret_cast<uint64_t *>(ring_all + S::kRingBytes);
    Cursor *starts = reinterpret_cast<Cursor *>(bars + S::kBars);
    PageMeta *meta_all = reinterpret_cast<PageMeta *>(starts + S::kWorkers);
    __shared__ int64_t warp_sum[kWarpsPerCta];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int wk = warp / MT, mt = warp % MT;  // worker within the CTA, row tile of the warp
    const int rows_all = p.D * p.G;
    const int RB = (rows_all + R - 1) / R, HR = p.Hkv * RB;
    const int64_t w = (int64_t)wk * gridDim.x + blockIdx.x;  // neighbours in work on different SMs
    float *ws = static_cast<float *>(p.workspace);
    const Layout lay = make_layout(p.batch, p.D, p.Hq, p.Hkv, HD, p.max_pages, p.weight_out != nullptr);

    for (int i = tid; i < S::kBars / 2; i += kThreads) {
        mbar_init(bars + i, 1);                   // full: the copy's bytes
        mbar_init(bars + S::kBars / 2 + i, MT);   // empty: the worker's warps
    }
    fence_barrier_init();

    // ---- the batch's units, and where each worker's range starts
    const int per = (p.batch + kThreads - 1) / kThreads;
    const int nb = min(tid * per, p.batch), ne = min(nb + per, p.batch);
    int64_t mine = 0;
    for (int n = nb; n < ne; ++n) {
        int len;
        const int pg = pages_of(p, n, len);
        mine += (int64_t)pg * HR;
        if (blockIdx.x == 0 && p.err_flag && p.seq_lens[n] > p.max_pages * kPage) atomicOr(p.err_flag, KDA_DEVERR_PAGE);
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(~0u, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int64_t U = 0, excl = incl - mine;
#pragma unroll
    for (int i = 0; i < kWarpsPerCta; ++i) {
        if (i < warp) excl += warp_sum[i];
        U += warp_sum[i];
    }
    // no more workers than units, so that no range is empty
    const int64_t W = min((int64_t)gridDim.x * S::kWorkers, max(U, (int64_t)1));
    for (int i = 0; i < S::kWorkers; ++i) {
        const int64_t u = U * ((int64_t)i * gridDim.x + blockIdx.x) / W;
        if (mine > 0 && u >= excl && u < excl + mine) {
            Cursor c{nb, excl};
            locate(p, HR, c, u);
            starts[i] = c;
        }
    }
    // sequences without pages have no unit: their rows are written here
    for (int n = blockIdx.x; n < p.batch; n += gridDim.x) {
        if (p.seq_lens[n] > 0 && p.max_pages > 0) continue;
        T *o = static_cast<T *>(p.out) + (int64_t)n * p.D * p.Hq * HD;
        for (int64_t i = tid; i < (int64_t)p.D * p.Hq * HD / 2; i += kThreads) store2(o + 2 * i, 0.f, 0.f);
        for (int i = tid; i < p.D * p.Hq; i += kThreads) {
            if (p.lse) p.lse[(int64_t)n * p.D * p.Hq + i] = -INFINITY;
        }
    }
    __syncthreads();

    const int64_t u0 = w < W ? U * w / W : 0, u1 = w < W ? U * (w + 1) / W : 0;
    int *desc = reinterpret_cast<int *>(ws + lay.desc) + 4 * w;
    if (mt == 0 && lane == 0) desc[0] = -1;
    if (u0 >= u1) return;

    unsigned char *ring = ring_all + wk * SL * S::kHalf;
    uint64_t *full = bars + wk * SL, *empty = bars + S::kBars / 2 + wk * SL;
    const int64_t count = u1 - u0;

    // ---- the copies: number c brings the keys (even) or values (odd) of unit
    // c / 2 into slot c % SL.  The worker's first warp looks up the pages of 32
    // units at a time, one per lane.
    Cursor cur = starts[wk], fetch_cur = cur;
    PageMeta *meta = meta_all + wk * kMeta;
    int64_t fetched = 0, issued = 0;
    auto fetch = [&]() {
        Cursor c = fetch_cur;
        if (fetched + lane < count) {
            const Unit un = locate(p, HR, c, u0 + fetched + lane);
            const int h = un.hr / RB;
            const int id = p.block_table[(int64_t)un.n * p.max_pages + un.page];
            PageMeta e{-1, 0.f, 0.f};
            if (id >= 0 && id < p.num_pages) {
                e.block = id * p.Hkv + h;
                e.ks = p.k_scale[e.block];
                e.vs = p.v_scale[e.block];
            } else if (p.err_flag) {
                atomicOr(p.err_flag, KDA_DEVERR_PAGE);
            }
            meta[(fetched + lane) % kMeta] = e;
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
        // rows g and g + 8 of the warp's tile
        int limit[2];
        int64_t qrow[2], qtok[2];
        int qhead[2];
        bool valid[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = rb * R + mt * 16 + g + 8 * e;
            valid[e] = r < rows_all;
            const int tok = valid[e] ? r / p.G : 0, gi = valid[e] ? r % p.G : 0;
            limit[e] = valid[e] ? un.len - p.D + 1 + tok : 0;
            qtok[e] = (int64_t)un.n * p.D + tok;
            qhead[e] = h * p.G + gi;
            qrow[e] = qtok[e] * p.Hq + qhead[e];
        }
        uint32_t qa[TERMS][KS][4];
        float qs[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const T *src = static_cast<const T *>(p.q) + qtok[e] * p.q_stride + (int64_t)qhead[e] * HD;
            float x[HD / 4], amax = 0.f;
#pragma unroll
            for (int j = 0; j < HD / 4; ++j) {
                x[j] = valid[e] ? load1<T>(src + chan<HD>(t, j)) : 0.f;
                amax = fmaxf(amax, fabsf(x[j]));
            }
            amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
            // the row times 2^(14 - ex): its largest element in 2^14..2^15
            int ex = (int)(__float_as_uint(amax) >> 23) - 127;
            ex = ex < -100 ? -100 : ex > 126 ? 126 : ex;
            const float mul = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
            qs[e] = __uint_as_float((uint32_t)(127 - 14 + ex) << 23) * p.scale * kLog2e;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const float x0 = x[4 * s + 2 * b] * mul, x1 = x[4 * s + 2 * b + 1] * mul;
                    qa[0][s][2 * b + e] = pack_f16(x0, x1);
                    if constexpr (TERMS == 2) {
                        const float2 hi = unpack_f16(qa[0][s][2 * b + e]);
                        qa[1][s][2 * b + e] = pack_f16(x0 - hi.x, x1 - hi.y);
                    }
                }
            }
        }
        float o[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[nt][c] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        float vref = 0.f;  // the scale that o is counted in
        const int window0 = un.len - p.D + 1;  // first position that some row does not see

        for (int pi = 0; pi < pages_here; ++pi, ++i) {
            const int page = un.page + pi;
            const int pos0 = page * kPage;
            // ---- scores
            const int64_t ck = 2 * i, cv = 2 * i + 1;
            const int sk = (int)(ck % SL), sv = (int)(cv % SL);
            if (!warp_wait(full + sk, ck / SL)) { timeout = true; break; }
            const PageMeta pm = meta[i % kMeta];
            const float ks = pm.ks, vs = pm.vs;
            const bool have = pm.block >= 0;
            const bool tail = pos0 + kPage > window0 || !have;
            float s[8][4];
            {
                const unsigned char *kb = ring + sk * S::kHalf;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const unsigned char *row = kb + (16 * (g >> 1) + 2 * j + (g & 1)) * HD;
                    uint32_t kw[HD / 16];
                    if constexpr (HD == 128) {
                        const uint4 a = *reinterpret_cast<const uint4 *>(row + 16 * t);
                        const uint4 b = *reinterpret_cast<const uint4 *>(row + 64 + 16 * t);
                        kw[0] = a.x; kw[1] = a.y; kw[2] = a.z; kw[3] = a.w;
                        kw[4] = b.x; kw[5] = b.y; kw[6] = b.z; kw[7] = b.w;
                    } else if constexpr (HD == 64) {
                        const uint4 a = *reinterpret_cast<const uint4 *>(row + 16 * t);
                        kw[0] = a.x; kw[1] = a.y; kw[2] = a.z; kw[3] = a.w;
                    } else {
                        const uint2 a = *reinterpret_cast<const uint2 *>(row + 8 * t);
                        kw[0] = a.x; kw[1] = a.y;
                    }
                    float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
                    for (int st = 0; st < KS; ++st) {
                        uint32_t b0, b1;
                        e4m3x4_to_f16(kw[st], b0, b1);
                        float(&c)[4] = acc[st & 1];
                        mma16816(c, qa[0][st][0], qa[0][st][1], qa[0][st][2], qa[0][st][3], b0, b1);
                        if constexpr (TERMS == 2)
                            mma16816(c, qa[1][st][0], qa[1][st][1], qa[1][st][2], qa[1][st][3], b0, b1);
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[j][c] = acc[0][c] + acc[1][c];
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + sk);
            // the next copy into the slot that is free now
            if (mt == 0 && ck + SL < 2 * count) {
                if (!warp_wait(empty + sk, ck / SL)) { timeout = true; break; }
                issue(ck + SL);
            }
            // ---- softmax
            const float f0 = qs[0] * ks, f1 = qs[1] * ks;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s[j][0] *= f0; s[j][1] *= f0;
                s[j][2] *= f1; s[j][3] *= f1;
            }
            if (tail) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int pos = pos0 + 16 * t + 2 * j + (c & 1);
                        if (!have || pos >= limit[c >> 1]) s[j][c] = -INFINITY;
                    }
            }
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                mx[0] = fmaxf(mx[0], fmaxf(s[j][0], s[j][1]));
                mx[1] = fmaxf(mx[1], fmaxf(s[j][2], s[j][3]));
            }
            float alpha[2], use[2];
            const float vnew = fmaxf(vref, have ? vs : 0.f);
            const float pmul = have ? kPScale * (vs / vnew) : 0.f;
            const float vfix = vref > 0.f ? vref / vnew : 1.f;
            vref = vnew;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mx[e] = fmaxf(mx[e], __shfl_xor_sync(~0u, mx[e], 1));
                mx[e] = fmaxf(mx[e], __shfl_xor_sync(~0u, mx[e], 2));
                const float mn = fmaxf(m[e], mx[e]);
                use[e] = mn == -INFINITY ? 0.f : mn;
                alpha[e] = ex2(m[e] - use[e]);
                m[e] = mn;
                l[e] *= alpha[e];
            }
            uint32_t pa[TERMS][4][4];
            float rs[2] = {0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float p0 = ex2(s[j][2 * e] - use[e]), p1 = ex2(s[j][2 * e + 1] - use[e]);
                    rs[e] += p0 + p1;
                    const float x0 = p0 * pmul, x1 = p1 * pmul;
                    // tile 2 s: registers 0 (row g), 1 (row g + 8); tile 2 s + 1: registers 2, 3
                    uint32_t &d = pa[0][j >> 1][2 * (j & 1) + e];
                    d = pack_f16(x0, x1);
                    if constexpr (TERMS == 2) {
                        const float2 hi = unpack_f16(d);
                        pa[1][j >> 1][2 * (j & 1) + e] = pack_f16(x0 - hi.x, x1 - hi.y);
                    }
                }
            }
            l[0] += rs[0];
            l[1] += rs[1];
            if (p.weight_out != nullptr) {  // the page's share, relative to the maximum so far
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = rs[e];
                    x += __shfl_xor_sync(~0u, x, 1);
                    x += __shfl_xor_sync(~0u, x, 2);
                    if (t == 0 && valid[e])
                        ws[lay.page_w + qrow[e] * p.max_pages + page] = x > 0.f ? log2f(x) + use[e] : -INFINITY;
                }
            }
            alpha[0] *= vfix;
            alpha[1] *= vfix;
            // ---- output
            if (!warp_wait(full + sv, cv / SL)) { timeout = true; break; }
            const unsigned char *vb = ring + sv * S::kHalf;
            if (!tail) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint4 a = *reinterpret_cast<const uint4 *>(vb + (8 * nt + g) * kPage + 16 * t);
                    const uint32_t vw[4] = {a.x, a.y, a.z, a.w};
                    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int st = 0; st < 4; ++st) {
                        uint32_t b0, b1;
                        e4m3x4_to_f16(vw[st], b0, b1);
                        mma16816(c, pa[0][st][0], pa[0][st][1], pa[0][st][2], pa[0][st][3], b0, b1);
                        if constexpr (TERMS == 2)
                            mma16816(c, pa[1][st][0], pa[1][st][1], pa[1][st][2], pa[1][st][3], b0, b1);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[nt][k] = fmaf(o[nt][k], alpha[k >> 1], c[k]);
                }
            } else {
                // bytes past the end (whatever they hold) count as zero, and so do
                // the window's NaN bytes, which only the rows that see them get
                const int left = have ? un.len - pos0 : 0;     // positions of the page that exist
                const int seen = window0 - pos0;               // positions that every row sees
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint4 a = *reinterpret_cast<const uint4 *>(vb + (8 * nt + g) * kPage + 16 * t);
                    uint32_t vw[4] = {a.x, a.y, a.z, a.w};
                    int nan_at = kPage;
#pragma unroll
                    for (int st = 0; st < 4; ++st)
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            const int pos = 16 * t + 4 * st + b;
                            const bool nan = ((vw[st] >> (8 * b)) & 0x7fu) == 0x7fu;
                            if (pos >= left) {
                                vw[st] &= ~(0xffu << (8 * b));
                            } else if (nan && pos >= seen) {
                                vw[st] &= ~(0xffu << (8 * b));
                                nan_at = min(nan_at, pos);
                            }
                        }
                    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int st = 0; st < 4; ++st) {
                        uint32_t b0, b1;
                        e4m3x4_to_f16(vw[st], b0, b1);
                        mma16816(c, pa[0][st][0], pa[0][st][1], pa[0][st][2], pa[0][st][3], b0, b1);
                        if constexpr (TERMS == 2)
                            mma16816(c, pa[1][st][0], pa[1][st][1], pa[1][st][2], pa[1][st][3], b0, b1);
                    }
                    nan_at = min(nan_at, __shfl_xor_sync(~0u, nan_at, 1));
                    nan_at = min(nan_at, __shfl_xor_sync(~0u, nan_at, 2));
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // accumulator column 8 nt + 2 t + k % 2 is the channel of quad 2 t + k % 2
                        const int at = __shfl_sync(~0u, nan_at, 4 * (2 * t + (k & 1)));
                        o[nt][k] = fmaf(o[nt][k], alpha[k >> 1], c[k]);
                        if (at < kPage && pos0 + at < limit[k >> 1]) o[nt][k] = NAN;
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + sv);
            if (mt == 0 && cv + SL < 2 * count) {
                if (!warp_wait(empty + sv, cv / SL)) { timeout = true; break; }
                issue(cv + SL);
            }
        }
        if (timeout) break;

        // ---- the item's end
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(~0u, l[e], 1);
            l[e] += __shfl_xor_sync(~0u, l[e], 2);
        }
        const float unit = vref * (1.f / kPScale);
        const bool whole = un.page == 0 && pages_here == un.pages;
        if (whole) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (!valid[e]) continue;
                const float f = l[e] == 0.f ? 0.f : unit / l[e];
                T *dst = static_cast<T *>(p.out) + qrow[e] * HD;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    store2(dst + 8 * nt + 2 * t, l[e] == 0.f ? 0.f : o[nt][2 * e] * f,
                           l[e] == 0.f ? 0.f : o[nt][2 * e + 1] * f);
                if (t == 0) {
                    const float lse2 = l[e] == 0.f ? -INFINITY : m[e] + log2f(l[e]);
                    if (p.lse) p.lse[qrow[e]] = lse2 * kLn2;
                    if (p.weight_out) ws[lay.lse2 + qrow[e]] = lse2;
                }
            }
        } else {
            const int64_t slot = 2 * w + (un.page == 0 ? 1 : 0);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = mt * 16 + g + 8 * e;
                float *dst = ws + lay.part_o + (slot * R + r) * HD;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) store2(dst + 8 * nt + 2 * t, o[nt][2 * e] * unit, o[nt][2 * e + 1] * unit);
                if (t == 0) {
                    ws[lay.part_m + slot * R + r] = m[e];
                    ws[lay.part_l + slot * R + r] = l[e];
                }
            }
            if (un.page == 0 && mt == 0 && lane == 0) {
                // this worker holds the item's first part: the join starts here
                const int64_t end = cur.base + (int64_t)(un.hr + 1) * un.pages;  // one past the item's last unit
                desc[1] = un.hr;
                desc[2] = (int)((end * W + U - 1) / U - 1);                      // the worker of that last unit
                desc[0] = un.n;
            }
        }
    }
    if (timeout && p.err_flag) atomicOr(p.err_flag, KDA_DEVERR_TIMEOUT);
    if (timeout && mt == 0)  // the copies in flight land before the CTA's memory goes
        for (int64_t c = issued > SL ? issued - SL : 0; c < issued; ++c)
            mbar_wait_drain(full + c % SL, (uint32_t)(c / SL) & 1u);
}

// Adds up the parts of one cut item: block (w, y) takes the item that starts
// in worker w and is continued, rows 8 y..8 y + 7 of it.
template <typename T, int HD, int MT>
__global__ void __launch_bounds__(128) join_kernel(const AttnDecodeParams p) {
    constexpr int R = 16 * MT;
    const float *ws = static_cast<const float *>(p.workspace);
    const Layout lay = make_layout(p.batch, p.D, p.Hq, p.Hkv, HD, p.max_pages, p.weight_out != nullptr);
    const int64_t w = blockIdx.x;
    const int *desc = reinterpret_cast<const int *>(ws + lay.desc) + 4 * w;
    const int n = desc[0];
    if (n < 0) return;
    const int hr = desc[1], last = desc[2];
    const int rows_all = p.D * p.G, RB = (rows_all + R - 1) / R;
    const int h = hr / RB, rb = hr % RB;
    // HD / 4 threads per row
    constexpr int TPR = HD / 4, RPB = 128 / TPR;
    const int c4 = threadIdx.x % TPR;
    const int r = blockIdx.y * RPB + threadIdx.x / TPR;
    const int row = rb * R + r;
    if (r >= R || row >= rows_all) return;
    auto slot_of = [&](int64_t x) { return 2 * x + (x == w ? 1 : 0); };
    float m = -INFINITY;
    for (int64_t x = w; x <= last; ++x) m = fmaxf(m, ws[lay.part_m + slot_of(x) * R + r]);
    const float use = m == -INFINITY ? 0.f : m;
    float l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int64_t x = w; x <= last; ++x) {
        const int64_t sl = slot_of(x) * R + r;
        const float f = ex2(ws[lay.part_m + sl] - use);
        const float4 v = *reinterpret_cast<const float4 *>(ws + lay.part_o + sl * HD + 4 * c4);
        l = fmaf(f, ws[lay.part_l + sl], l);
        o[0] = fmaf(f, v.x, o[0]); o[1] = fmaf(f, v.y, o[1]);
        o[2] = fmaf(f, v.z, o[2]); o[3] = fmaf(f, v.w, o[3]);
    }
    const int64_t qrow = ((int64_t)n * p.D + row / p.G) * p.Hq + h * p.G + row % p.G;
    const float f = l == 0.f ? 0.f : 1.f / l;
    T *dst = static_cast<T *>(p.out) + qrow * HD + 4 * c4;
    store2(dst, l == 0.f ? 0.f : o[0] * f, l == 0.f ? 0.f : o[1] * f);
    store2(dst + 2, l == 0.f ? 0.f : o[2] * f, l == 0.f ? 0.f : o[3] * f);
    if (c4 == 0) {
        const float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
        if (p.lse) p.lse[qrow] = lse2 * kLn2;
        if (p.weight_out) static_cast<float *>(p.workspace)[lay.lse2 + qrow] = lse2;
    }
}

// weight_out[n][page] = weight_in + sum over the rows of 2^(page share - lse).
// A block takes 32 pages of a sequence; its 8 groups of threads take every
// eighth row and are added up in order.
__global__ void __launch_bounds__(256) page_weight_kernel(const AttnDecodeParams p, Layout lay) {
    __shared__ float part[8][33];
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

template <typename T, int HD, int MT>
cudaError_t launch(const AttnDecodeParams &p, cudaStream_t st) {
    using S = Smem<T, HD, MT>;
    auto kern = decode_attn_kernel<T, HD, MT>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(kern), S::kBytes, done);
    if (e != cudaSuccess) return e;
    const int rows = p.D * p.G, RB = (rows + 16 * MT - 1) / (16 * MT);
    // no more workers than pages
    const int64_t units = (int64_t)p.batch * p.Hkv * RB * p.max_pages;
    int64_t ctas = (units + S::kWorkers - 1) / S::kWorkers;
    ctas = ctas < 1 ? 1 : ctas > kMaxCtas ? kMaxCtas : ctas;
    kern<<<(unsigned)ctas, kThreads, S::kBytes, st>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int rpb = 128 / (HD / 4);
    const dim3 grid((unsigned)(ctas * S::kWorkers), (unsigned)((16 * MT + rpb - 1) / rpb));
    join_kernel<T, HD, MT><<<grid, 128, 0, st>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.weight_out == nullptr || p.max_pages == 0) return e;
    const Layout lay = make_layout(p.batch, p.D, p.Hq, p.Hkv, HD, p.max_pages, true);
    const int64_t blocks = (int64_t)p.batch * ((p.max_pages + 31) / 32);
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    page_weight_kernel<<<(unsigned)blocks, 256, 0, st>>>(p, lay);
    return cudaGetLastError();
}

template <typename T, int HD>
cudaError_t launch_rows(const AttnDecodeParams &p, cudaStream_t st) {
    switch (row_tile(p.D * p.G)) {
        case 1: return launch<T, HD, 1>(p, st);
        case 2: return launch<T, HD, 2>(p, st);
        default: return launch<T, HD, 4>(p, st);
    }
}

template <typename T>
cudaError_t launch_dim(const AttnDecodeParams &p, int d, cudaStream_t st) {
    if (d == 128) return launch_rows<T, 128>(p, st);
    if (d == 64) return launch_rows<T, 64>(p, st);
    return launch_rows<T, 32>(p, st);
}

}  // namespace

size_t attn_decode_workspace_bytes(int Hq, int Hkv, int d, int dtype, int64_t batch, int D, int64_t max_pages,
                                   bool with_weight) {
    (void)dtype;
    if (batch <= 0) return 0;
    return (size_t)make_layout(batch, D, Hq, Hkv, d, max_pages, with_weight).total * 4;
}

cudaError_t launch_attn_decode(const AttnDecodeParams &p, int d, int dtype, cudaStream_t st) {
    return dtype == KDA_DT_BF16 ? launch_dim<__nv_bfloat16>(p, d, st) : launch_dim<float>(p, d, st);
}

}  // namespace kda
