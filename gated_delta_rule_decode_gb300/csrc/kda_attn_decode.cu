// Attention over the 8-bit paged cache: how a call is cut into items and workers,
// the kernels of a few rows (kda_attn_decode_rows.cuh), the join of the cut
// items and the page weights.
#include <cuda_bf16.h>
#include <stdint.h>

#include "kda_attn_decode.cuh"
#include "kda_attn_decode_rows.cuh"
#include "kda_attn_internal.h"

namespace kda {
namespace {

using namespace dec;

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

template <typename T, int HD>
cudaError_t launch(const AttnDecodeParams &p, cudaStream_t st) {
    const Layout lay = make_layout(p.batch, p.D, p.Hq, p.Hkv, HD, sizeof(T) == 2 ? KDA_DT_BF16 : KDA_DT_F32, p.max_pages,
                                   p.weight_out != nullptr);
    if (lay.items > 0x7fffffff || (int64_t)p.max_pages * p.Hkv * lay.RB > 0x7fffffff) return cudaErrorInvalidValue;
    cudaError_t e = launch_items<T, HD, false>(p, lay, st);
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

// weight_rows: the batch's query rows where page weights are asked for
static Layout lay_out(int64_t batch, int rows, int Hkv, int d, int dtype, int64_t max_pages, int64_t weight_rows) {
    auto align64 = [](int64_t x) { return (x + 63) / 64 * 64; };
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
    l.page_w = l.lse2 + align64(weight_rows);
    if (l.whole) l.workers = l.items;
    l.total = l.page_w + align64(weight_rows * max_pages);
    return l;
}

Layout make_layout(int64_t batch, int D, int Hq, int Hkv, int d, int dtype, int64_t max_pages, bool with_weight) {
    return lay_out(batch, D * (Hq / Hkv), Hkv, d, dtype, max_pages, with_weight ? batch * D * Hq : 0);
}

Layout make_parts_layout(int64_t batch, int rows, int Hkv, int d, int dtype, int64_t max_pages) {
    return lay_out(batch, rows, Hkv, d, dtype, max_pages, 0);
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
