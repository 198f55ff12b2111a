// Attention of a batch whose sequences share prefixes, over the 8-bit paged
// cache: a prefix's pages are read once for all the sequences that share it.
//
//   o = (sum_prefix e^{s_j} v_j + sum_rest e^{s_j} v_j) / (the same sums of e^{s_j})
//
// Four launches: plan_kernel lays the batch out as chunks (up to R query rows of
// one group and its prefix; a sequence's rows and the rest of it), the chunks of
// the prefixes and those of the rests are attended as items of the cache
// attention kernels, whose results stay apart as (o, m, l), and merge_kernel
// adds up all parts of a row in a fixed order.
#include <cuda_bf16.h>
#include <stdint.h>

#include <algorithm>

#include "kda_attn_decode.cuh"
#include "kda_attn_internal.h"

namespace kda {
namespace {

using namespace dec;

constexpr int kPlanThreads = 1024;

// Where a sequence's parts lie: base: positions of its prefix; first: the first
// chunk of its group's; token: its first token within the group's.
struct SeqPlan {
    int32_t base, first, token, pad;
};

// The workspace, in bytes: the plan, the results of whole items, and a
// workspace of each of the two attention launches.
struct SharedLayout {
    int64_t group_chunk, seqs, prefix_chunks, rest_chunks, prefix_ml, rest_ml, prefix_o, rest_o, prefix_ws, rest_ws, total;
    Layout prefix, rest;
    int64_t prefix_count, rest_count;
    int32_t prefix_tokens, rest_tokens, per_seq;  // tokens of a chunk; chunks of a sequence's rest
};

SharedLayout shared_layout(int Hq, int Hkv, int d, int dtype, int64_t batch, int D, int64_t max_pages, int64_t groups) {
    auto align = [](int64_t x) { return (x + 255) / 256 * 256; };
    const int G = Hq / Hkv;
    SharedLayout l{};
    // a chunk has the whole tokens that fit an item's rows: of a group of mean size, of a sequence
    const int64_t mean = (batch + groups - 1) / std::max<int64_t>(groups, 1) * D * G;
    auto tokens = [&](int64_t rows) {
        return std::max(1, make_parts_layout(1, (int)std::min<int64_t>(rows, 4096), Hkv, d, dtype, max_pages).R / G);
    };
    l.prefix_tokens = tokens(std::max<int64_t>(mean, G));
    l.rest_tokens = std::min(D, tokens((int64_t)D * G));
    l.per_seq = (D + l.rest_tokens - 1) / l.rest_tokens;
    l.prefix_count = groups > 0 ? batch * D / l.prefix_tokens + groups : 0;
    l.rest_count = batch * l.per_seq;
    l.prefix = make_parts_layout(l.prefix_count, l.prefix_tokens * G, Hkv, d, dtype, max_pages);
    l.rest = make_parts_layout(l.rest_count, l.rest_tokens * G, Hkv, d, dtype, max_pages);
    const int64_t q = batch * D * Hq;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += align(bytes);
        return here;
    };
    l.group_chunk = take(groups * 4);
    l.seqs = take(batch * (int64_t)sizeof(SeqPlan));
    l.prefix_chunks = take(l.prefix_count * (int64_t)sizeof(AttnChunk));
    l.rest_chunks = take(l.rest_count * (int64_t)sizeof(AttnChunk));
    l.prefix_ml = take(q * 8);
    l.rest_ml = take(q * 8);
    l.prefix_o = take(q * d * 4);
    l.rest_o = take(q * d * 4);
    l.prefix_ws = take(l.prefix.total * 4);
    l.rest_ws = take(l.rest.total * 4);
    l.total = at;
    return l;
}

// A group's sequences and prefix; none where its offsets are wrong.
struct Group {
    int32_t first, count, pages;
};

__device__ __forceinline__ Group group_of(const AttnSharedParams &p, int g, bool tell) {
    const int a = p.group_start[g], b = p.group_start[g + 1], s = p.shared_pages[g];
    const bool bad = a < 0 || b < a || b > p.call.batch;
    if (tell && p.call.err_flag) {
        if (bad) atomicOr(p.call.err_flag, KDA_DEVERR_SEQLENS);
        if (s < 0 || s > p.call.max_pages) atomicOr(p.call.err_flag, KDA_DEVERR_PAGE);
    }
    return Group{a, bad ? 0 : b - a, s < 0 ? 0 : min(s, p.call.max_pages)};
}

// The last of a[0..n-1] that is <= x, -1 for none.
__device__ __forceinline__ int last_at_most(const int32_t *a, int n, int x) {
    int lo = -1, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const AttnSharedParams p, const SharedLayout lay) {
    __shared__ int warp_sum[kPlanThreads / 32];
    unsigned char *ws = static_cast<unsigned char *>(p.call.workspace);
    int32_t *group_chunk = reinterpret_cast<int32_t *>(ws + lay.group_chunk);
    SeqPlan *seqs = reinterpret_cast<SeqPlan *>(ws + lay.seqs);
    AttnChunk *prefix = reinterpret_cast<AttnChunk *>(ws + lay.prefix_chunks), *rest = reinterpret_cast<AttnChunk *>(ws + lay.rest_chunks);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int D = p.call.D;

    // the groups' first chunks
    int before = 0;
    for (int g0 = 0; g0 < p.groups; g0 += kPlanThreads) {
        int mine = 0;
        if (g0 + tid < p.groups) {
            const Group g = group_of(p, g0 + tid, true);
            if (g.pages > 0) mine = (g.count * D + lay.prefix_tokens - 1) / lay.prefix_tokens;
        }
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(~0u, incl, o);
            if (lane >= o) incl += x;
        }
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        int at = before + incl - mine;
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            if (w < warp) at += warp_sum[w];
            before += warp_sum[w];
        }
        if (g0 + tid < p.groups) group_chunk[g0 + tid] = at;
        __syncthreads();
    }
    const int used = (int)min((int64_t)before, lay.prefix_count);

    // the prefixes' chunks
    for (int c = tid; c < lay.prefix_count; c += kPlanThreads) {
        AttnChunk out{};
        if (c < used) {
            const int gi = last_at_most(group_chunk, p.groups, c);
            const Group g = group_of(p, gi, false);
            const int t0 = (c - group_chunk[gi]) * lay.prefix_tokens, tokens = min(lay.prefix_tokens, g.count * D - t0);
            if (tokens > 0) {
                out.table = (int64_t)g.first * p.call.max_pages;
                out.tok0 = g.first * D + t0;
                out.rows = tokens * p.call.G;
                out.len = out.seen = g.pages * kPage;
                for (int n = out.tok0 / D; n <= (out.tok0 + tokens - 1) / D; ++n) {
                    const int len = capped_len(p.call, n);
                    if (len > 0) out.seen = min(out.seen, max(1, len - D + 1));
                }
            }
        }
        prefix[c] = out;
    }
    // the sequences, and the chunks of what follows their prefixes
    for (int n = tid; n < p.call.batch; n += kPlanThreads) {
        SeqPlan out{};
        const int len = capped_len(p.call, n), gi = last_at_most(p.group_start, p.groups, n);
        if (p.call.err_flag && p.call.seq_lens[n] > p.call.max_pages * kPage) atomicOr(p.call.err_flag, KDA_DEVERR_PAGE);
        if (gi >= 0) {
            const Group g = group_of(p, gi, false);
            if (n >= g.first && n < g.first + g.count) {
                out.base = g.pages * kPage;
                out.first = group_chunk[gi];
                out.token = (n - g.first) * D;
            }
        }
        seqs[n] = out;
        for (int i = 0; i < lay.per_seq; ++i) {
            AttnChunk c{};
            const int t0 = i * lay.rest_tokens;
            c.table = (int64_t)n * p.call.max_pages + out.base / kPage;
            c.tok0 = n * D + t0;
            c.rows = min(lay.rest_tokens, D - t0) * p.call.G;
            c.base = out.base;
            c.len = max(0, len - out.base);
            c.seen = min(c.len, max(1, len - D + 1 + t0 - out.base));
            rest[(int64_t)n * lay.per_seq + i] = c;
        }
    }
}

// A row's parts of one of the two attentions.
struct Parts {
    const float *ws;  // of the attention's launch
    int64_t first;    // worker of the first part; -1: one result, in the rows' arrays
    int count, row;   // row within the item's partial results
};

// Adds up the parts of a row: a block takes a row, its groups of HD / 4 threads
// every GR-th part, in order; the groups' sums are added in order.
constexpr int kMergeThreads = 128;

template <typename T, int HD>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const AttnSharedParams p, const SharedLayout lay) {
    constexpr int TPR = HD / 4, GR = kMergeThreads / TPR;
    __shared__ float wmax[kMergeThreads / 32];
    __shared__ float4 so[GR][TPR];
    __shared__ float sl[GR];
    const AttnDecodeParams &c = p.call;
    const int64_t qrow = blockIdx.x;
    const int hq = (int)(qrow % c.Hq), h = hq / c.G, gi = hq % c.G;
    const int64_t tok = qrow / c.Hq;
    const int n = (int)(tok / c.D), t = (int)(tok % c.D), tid = threadIdx.x;
    const unsigned char *ws = static_cast<const unsigned char *>(c.workspace);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const SeqPlan sp = reinterpret_cast<const SeqPlan *>(ws + lay.seqs)[n];
    const int sees = capped_len(c, n) - c.D + 1 + t;  // positions in all

    // where the two attentions left the row's results
    Parts from[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const Layout &l = s == 0 ? lay.prefix : lay.rest;
        const int tokens = s == 0 ? lay.prefix_tokens : lay.rest_tokens;
        const int local = s == 0 ? sp.token + t : t;
        const int64_t chunk = s == 0 ? (int64_t)sp.first + local / tokens : (int64_t)n * lay.per_seq + local / tokens;
        const int row = (local % tokens) * c.G + gi, rb = row / l.R;
        const int64_t item = (chunk * c.Hkv + h) * l.RB + rb;
        Parts &f = from[s];
        f.ws = reinterpret_cast<const float *>(ws + (s == 0 ? lay.prefix_ws : lay.rest_ws));
        f.row = row - rb * l.R;
        f.first = -1;
        f.count = (s == 0 ? min(sees, sp.base) : sees - sp.base) > 0 && chunk < (s == 0 ? lay.prefix_count : lay.rest_count) ? 1 : 0;
        if (f.count > 0 && !l.whole) {
            const int2 desc = *reinterpret_cast<const int2 *>(f.ws + l.desc + 2 * item);
            // (a worker that gave up waiting leaves no or stale entries)
            if (desc.x < 0 || desc.x > desc.y || desc.y >= l.workers) f.count = 0;
            else if (desc.y > desc.x) {
                f.first = desc.x;
                f.count = desc.y - desc.x + 1;
            }
        }
    }
    const int parts = from[0].count + from[1].count;
    // (m, l) and the output of part x
    auto at = [&](int x, float &m, float &l, const float *&o) {
        const int s = x < from[0].count ? 0 : 1;
        const Parts f = s == 0 ? from[0] : from[1];
        const Layout &y = s == 0 ? lay.prefix : lay.rest;
        if (s == 1) x -= from[0].count;
        if (f.first < 0) {
            const float2 ml = reinterpret_cast<const float2 *>(ws + (s == 0 ? lay.prefix_ml : lay.rest_ml))[qrow];
            m = ml.x;
            l = ml.y;
            o = reinterpret_cast<const float *>(ws + (s == 0 ? lay.prefix_o : lay.rest_o)) + qrow * HD;
        } else {  // part x lies in slot 2 (w + x), the first in slot 2 w + 1
            const int64_t k = (2 * (f.first + x) + (x == 0 ? 1 : 0)) * y.PR + f.row;
            m = f.ws[y.part_m + k];
            l = f.ws[y.part_l + k];
            o = f.ws + y.part_o + k * HD;
        }
    };
    float m = -INFINITY;
    for (int x = tid; x < parts; x += kMergeThreads) {
        float pm, pl;
        const float *o;
        at(x, pm, pl, o);
        m = fmaxf(m, pm);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    if ((tid & 31) == 0) wmax[tid >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMergeThreads / 32; ++i) m = fmaxf(m, wmax[i]);
    const float use = m == -INFINITY ? 0.f : m;
    const int c4 = tid % TPR, gr = tid / TPR;
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x = gr; x < parts; x += GR) {
        float pm, pl;
        const float *po;
        at(x, pm, pl, po);
        if (pl == 0.f) continue;  // (a part whose pages are not in the cache)
        const float4 v = *reinterpret_cast<const float4 *>(po + 4 * c4);
        const float f = ex2(pm - use);
        l = fmaf(f, pl, l);
        o.x = fmaf(f, v.x, o.x); o.y = fmaf(f, v.y, o.y);
        o.z = fmaf(f, v.z, o.z); o.w = fmaf(f, v.w, o.w);
    }
    so[gr][c4] = o;
    if (c4 == 0) sl[gr] = l;
    __syncthreads();
    if (gr != 0) return;
    for (int i = 1; i < GR; ++i) {
        const float4 v = so[i][c4];
        o.x += v.x; o.y += v.y; o.z += v.z; o.w += v.w;
        l += sl[i];
    }
    const float f = l == 0.f ? 0.f : 1.f / l;
    T *dst = static_cast<T *>(c.out) + qrow * HD + 4 * c4;
    store2(dst, l == 0.f ? 0.f : o.x * f, l == 0.f ? 0.f : o.y * f);
    store2(dst + 2, l == 0.f ? 0.f : o.z * f, l == 0.f ? 0.f : o.w * f);
    if (c4 == 0 && c.lse) c.lse[qrow] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <typename T>
cudaError_t launch_merge(const AttnSharedParams &p, const SharedLayout &lay, int d, cudaStream_t st) {
    const dim3 grid((unsigned)((int64_t)p.call.batch * p.call.D * p.call.Hq));
    if (d == 128) return launch_after(merge_kernel<T, 128>, grid, kMergeThreads, st, p, lay);
    if (d == 64) return launch_after(merge_kernel<T, 64>, grid, kMergeThreads, st, p, lay);
    return launch_after(merge_kernel<T, 32>, grid, kMergeThreads, st, p, lay);
}

}  // namespace

size_t attn_shared_workspace_bytes(int Hq, int Hkv, int d, int dtype, int64_t batch, int D, int64_t max_pages,
                                   int64_t groups) {
    return batch <= 0 ? 0 : (size_t)shared_layout(Hq, Hkv, d, dtype, batch, D, max_pages, groups).total;
}

cudaError_t launch_attn_shared(const AttnSharedParams &p, int d, int dtype, cudaStream_t st) {
    const AttnDecodeParams &c = p.call;
    const SharedLayout lay = shared_layout(c.Hq, c.Hkv, d, dtype, c.batch, c.D, c.max_pages, p.groups);
    if ((int64_t)c.batch * c.D * c.Hq > 0x7fffffff || lay.prefix_count > 0x7fffffff) return cudaErrorInvalidValue;
    unsigned char *ws = static_cast<unsigned char *>(c.workspace);
    plan_kernel<<<1, kPlanThreads, 0, st>>>(p, lay);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    for (int s = 0; s < 2; ++s) {
        const bool prefix = s == 0;
        if (c.max_pages == 0 || (prefix ? lay.prefix_count : lay.rest_count) == 0) continue;
        AttnDecodeParams q = c;
        q.chunks = reinterpret_cast<const AttnChunk *>(ws + (prefix ? lay.prefix_chunks : lay.rest_chunks));
        q.part_ml = reinterpret_cast<float2 *>(ws + (prefix ? lay.prefix_ml : lay.rest_ml));
        q.out = ws + (prefix ? lay.prefix_o : lay.rest_o);
        q.lse = nullptr;
        q.workspace = ws + (prefix ? lay.prefix_ws : lay.rest_ws);
        q.batch = (int32_t)(prefix ? lay.prefix_count : lay.rest_count);
        e = launch_parts(q, prefix ? lay.prefix : lay.rest, d, dtype, st);
        if (e != cudaSuccess) return e;
    }
    return dtype == KDA_DT_BF16 ? launch_merge<__nv_bfloat16>(p, lay, d, st) : launch_merge<float>(p, lay, d, st);
}

}  // namespace kda
