// Attention of a batch whose sequences share prefixes, over the 8-bit paged
// cache: a prefix's pages are read once for all the sequences that share it.
//
//   o = (sum_prefix e^{s_j} v_j + sum_rest e^{s_j} v_j) / (the same sums of e^{s_j})
//
// plan_kernel lays the batch out as chunks: up to R query rows of one group and
// its prefix; a sequence's rows and the rest of it.  The chunks are attended as
// items of kernels whose results stay apart as (o, m, l): on tcgen05 (bf16,
// d = 64 and 128; kda_attn_shared_tc.cu) in one launch, whose workers' ranges the
// plan cuts by cost, or by the kernels of kda_attn_decode_rows.cuh, the prefixes'
// chunks and then the others'.  Where groups are small in the mean, their prefixes
// have a launch for few rows, and groups that are large all the same one of their
// own.  merge_kernel adds up all parts of a row in a fixed order.
//
// Measured (bf16, d = 128, 32 heads over 8): 64 sequences of up to 2048 positions
// after a prefix of 8192: 98 us, of which the plan 7, the prefix 26, the rests 55 and
// the sum 11 (each cold and by itself); 32 of up to 512 after 102 400: 106 us (6, 75,
// 17, 10).  The plan and the sum are chains of dependent reads; the rests, a few
// pages a worker, are the start and end of their items.
#include <cuda_bf16.h>
#include <stdint.h>

#include <algorithm>

#include "kda_attn_decode.cuh"
#include "kda_attn_internal.h"
#include "kda_attn_shared.cuh"

namespace kda {
namespace {

using namespace dec;

constexpr int kPlanThreads = 1024;

// Where a sequence's parts lie: base: positions of its prefix; first: the first
// chunk of its group's (few: among those of small groups); token: its first token
// within the group's.
struct SeqPlan {
    int32_t base, first, token, few;
};

// The tcgen05 workers' costs, in half blocks of 64 positions of up to 128 rows: a
// page of a chunk of more rows is two, an item's start and end about kItemCost
// (2, 6, 9, 12, 18: 40 sequences of 7 tokens in five groups, whose rests are short
// items, 110, 70, 64, 64, 66 us; 64 of 8 tokens after one prefix 90, 85, 86, 88, 93).
constexpr int kItemCost = 9;
// On tcgen05 go prefixes of groups of more rows (of mean size, with all tokens
// and heads of a kv head) than kFewShared, and sequences' rests of more rows than
// kFewRows; the warps' kernel is quicker with few.  Prefixes of 32 pages and 64
// sequences in groups of 4, 8, 16 and 32 rows: 149, 104, 81, 69 us there, 110, 85,
// 83, 93 us with the warps' kernel.  Rests of 4 rows (32 sequences after 1600
// pages) 121 us there, 104 with the warps' kernel; of 20 rows 106 and 257.
constexpr int kFewShared = 8, kFewRows = 16;
// Among groups of kFewShared rows in the mean, those of more than kLargeGroup are read apart, once for up to 256 rows
// on tcgen05 and for up to 64 elsewhere instead of once for 8.  That launch costs 4 us where there are none, so it is
// left out where it could not save much: where no more than kLongReads pages of a kv head could be read for chunks of 8
// rows.  One group of 64 sequences among 63 of one (32 heads over 8, d = 128): prefixes of 1600 pages 922 us without
// and 228 with it, of 128 pages 194 and 202; 16, 32 and 64 groups of 64 sequences, 32 pages, 55, 74, 82 and 60, 80, 87.
constexpr int kLargeGroup = 32;
constexpr double kLongReads = 1 << 16;
constexpr int kPlanCached = 2048;  // chunks whose costs fit the plan's shared memory

// Where the parts of one of the attentions are: an item's workers (first,
// last) in desc, two slots a worker of PR rows each, RB items a chunk and kv head
// of R rows.
struct PartsAt {
    int64_t desc, part_m, part_l, part_o, ml, o;  // bytes
    int64_t workers, chunks;
    int32_t R, RB, PR, tokens, per;  // tokens of a chunk; chunks of a sequence's rest
    int32_t whole;                   // no item is cut
};

// The workspace, in bytes: the plan, the results of whole items, and the parts.  total 0: a call that is too large.
struct SharedLayout {
    int64_t group_chunk, seqs, chunks, costs, starts, total;
    PartsAt at[3];  // of the prefixes, of the rests, of the prefixes of small groups; their chunks follow one another
    int64_t ws[3];  // off tcgen05: workspaces of the launches
    Layout lay[3];
    int32_t tc[3], workers;
    int32_t few;  // where groups are small in the mean, the most rows of one that counts as small, else 0
    int32_t on_tc;
};

SharedLayout shared_layout(int Hq, int Hkv, int d, int dtype, int64_t batch, int D, int64_t max_pages, int64_t groups) {
    const int G = Hq / Hkv;
    SharedLayout l{};
    l.tc[0] = dtype == KDA_DT_BF16 && d >= 64;
    l.tc[1] = l.tc[0] && D * G > kFewRows;
    // the rows of a group of mean size
    const int64_t mean = (batch + groups - 1) / std::max<int64_t>(groups, 1) * D * G;
    const double reads = (double)batch * D * G / kFewShared * max_pages * Hkv;
    l.few = groups == 0 || mean > kFewShared ? 0 : reads > kLongReads ? kLargeGroup : 0x7fffffff;
    l.workers = kSms;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    // a chunk has the whole tokens that fit an item's rows
    auto tokens = [&](int s, int64_t rows) {
        if (l.tc[s]) return kPartRows / G;
        return std::max(1, make_parts_layout(1, (int)std::min<int64_t>(rows, 4096), Hkv, d, dtype, max_pages).R / G);
    };
    l.at[0].tokens = tokens(0, l.few > 0 ? kPartRows : std::max<int64_t>(mean, G));
    l.at[1].tokens = std::min(D, tokens(1, (int64_t)D * G));
    l.at[1].per = (D + l.at[1].tokens - 1) / l.at[1].tokens;
    l.at[0].chunks = groups > 0 && batch * D * G > l.few ? batch * D / l.at[0].tokens + groups : 0;
    l.at[1].chunks = batch * l.at[1].per;
    if (l.few > 0) {
        l.at[2].tokens = kFewShared / G;  // (a sequence has no more rows)
        l.at[2].chunks = batch * D / l.at[2].tokens + groups;
    }
    l.on_tc = (l.tc[0] && l.at[0].chunks > 0) || l.tc[1];
    const int64_t count = l.at[0].chunks + l.at[1].chunks + l.at[2].chunks, q = batch * D * Hq;
    if (count * Hkv > 0xfffff000ll || q > 0x7fffffff) return l;  // (the kernels count these in 32 and 31 bits)
    l.group_chunk = take(2 * groups * 4);
    l.seqs = take(batch * (int64_t)sizeof(SeqPlan));
    l.chunks = take(count * (int64_t)sizeof(AttnChunk));
    for (int s = 0; s < 2; ++s) {
        l.at[s].ml = take(q * 8);
        l.at[s].o = take(q * d * 4);
    }
    l.at[2].ml = l.at[0].ml;  // (a row has one prefix)
    l.at[2].o = l.at[0].o;
    if (l.on_tc) {
        l.costs = take(count * 8);
        l.starts = take((l.workers + 1) * (int64_t)sizeof(int4));
        const int64_t rows = 2 * (int64_t)l.workers * kPartRows;
        const int64_t desc = take(count * Hkv * 8), part_m = take(rows * 4), part_l = take(rows * 4), part_o = take(rows * d * 4);
        for (int s = 0; s < 2; ++s) {
            PartsAt &a = l.at[s];
            a.desc = desc + (s == 0 ? 0 : l.at[0].chunks * Hkv * 8);
            a.part_m = part_m; a.part_l = part_l; a.part_o = part_o;
            a.workers = l.workers; a.R = a.PR = kPartRows; a.RB = 1;
        }
    }
    for (int s = 0; s < 3; ++s) {
        if (l.tc[s] || l.at[s].chunks == 0) continue;
        PartsAt &a = l.at[s];
        const Layout y = make_parts_layout(a.chunks, a.tokens * G, Hkv, d, dtype, max_pages);
        const int64_t ws = take(y.total * 4);
        a.desc = ws + 4 * y.desc;
        a.part_m = ws + 4 * y.part_m; a.part_l = ws + 4 * y.part_l; a.part_o = ws + 4 * y.part_o;
        a.workers = y.workers; a.R = y.R; a.RB = y.RB; a.PR = y.PR; a.whole = y.whole;
        l.lay[s] = y;
        l.ws[s] = ws;
    }
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

// How a group's prefix is attended: not at all, among those of small groups, among the others.
enum Sharing { kNone, kFew, kMany };
__device__ __forceinline__ Sharing sharing_of(const AttnSharedParams &p, const SharedLayout &lay, const Group &g) {
    if (g.pages == 0 || g.count == 0) return kNone;
    return (int64_t)g.count * p.call.D * p.call.G <= lay.few ? kFew : kMany;
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

// Sums of counts that may leave 31 bits stay at the most that these hold.
__device__ __forceinline__ int add(int a, int b) { return (int)min((unsigned)a + (unsigned)b, 0x7fffffffu); }
__device__ __forceinline__ int64_t add(int64_t a, int64_t b) { return a + b; }

// What the threads before this one have of `mine` (not negative), and all together; by the whole block of 1024.
template <typename T>
__device__ __forceinline__ T scan(T mine, T *warp_sum, T &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T x = __shfl_up_sync(~0u, incl, o);
        if (lane >= o) incl = add(incl, x);
    }
    if (lane == 31) warp_sum[warp] = incl;
    const T excl = __shfl_up_sync(~0u, incl, 1);
    __syncthreads();
    T sums = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T x = __shfl_up_sync(~0u, sums, o);
        if (lane >= o) sums = add(sums, x);
    }
    __syncthreads();  // (warp_sum is free again)
    total = __shfl_sync(~0u, sums, 31);
    const T before = __shfl_sync(~0u, sums, max(warp - 1, 0));
    return add(warp > 0 ? before : 0, lane > 0 ? excl : 0);
}
static_assert(kPlanThreads == 1024, "a lane a warp");

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const AttnSharedParams p, const SharedLayout lay) {
    __shared__ int warp_sum[kPlanThreads / 32];
    __shared__ int sizes[kPlanCached];  // of the chunks: pages, and whether they are of more than 128 rows
    auto size_of = [](const AttnChunk &c) { return 2 * ((c.len + kPage - 1) / kPage) + (c.rows > 128 ? 1 : 0); };
    unsigned char *ws = static_cast<unsigned char *>(p.call.workspace);
    int32_t *group_chunk = reinterpret_cast<int32_t *>(ws + lay.group_chunk);
    SeqPlan *seqs = reinterpret_cast<SeqPlan *>(ws + lay.seqs);
    AttnChunk *prefix = reinterpret_cast<AttnChunk *>(ws + lay.chunks), *rest = prefix + lay.at[0].chunks;
    AttnChunk *few_prefix = rest + lay.at[1].chunks;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int D = p.call.D;

    // the groups' first chunks, of `cap` in all.  Groups of wrong offsets may overlap, so that there are more than their
    // sequences can have, in all more than 31 bits hold: those that have no place here start at the end, and are no one's.
    const int64_t many = lay.at[0].chunks, few = lay.at[2].chunks;
    auto first_chunks = [&](int32_t *first, Sharing which, int tokens, int64_t cap) {
        int before = 0;
        for (int g0 = 0; g0 < p.groups; g0 += kPlanThreads) {
            int mine = 0;
            if (g0 + tid < p.groups) {
                const Group g = group_of(p, g0 + tid, which == kMany || many == 0);
                if (sharing_of(p, lay, g) == which) mine = add(g.count * D, tokens - 1) / tokens;
            }
            int all;
            const int at = add(before, scan(mine, warp_sum, all));
            before = add(before, all);
            if (g0 + tid < p.groups) first[g0 + tid] = (int32_t)min((int64_t)at, cap);
        }
        return min((int64_t)before, cap);
    };
    int32_t *few_chunk = group_chunk + p.groups;
    const int64_t used = many > 0 ? first_chunks(group_chunk, kMany, lay.at[0].tokens, many) : 0;
    const int64_t few_used = few > 0 ? first_chunks(few_chunk, kFew, lay.at[2].tokens, few) : 0;

    // the prefixes' chunks, a warp each: a lane a sequence.  A chunk goes as far as its longest sequence, whose row of
    // the table names its pages: what lies behind a sequence's last page is not read.
    __syncthreads();
    // (where there are none on tcgen05, no chunk is looked at there)
    for (int64_t c = warp + (used == 0 && lay.tc[0] && !lay.tc[1] ? many : 0); c < many + few; c += kPlanThreads / 32) {
        AttnChunk out{};
        const bool is_few = c >= many;
        const int at = (int)(is_few ? c - many : c);
        if (at < (is_few ? few_used : used)) {
            const int32_t *first = is_few ? few_chunk : group_chunk;
            const int gi = last_at_most(first, p.groups, at), most = lay.at[is_few ? 2 : 0].tokens;
            const Group g = group_of(p, gi, false);
            const int t0 = (at - first[gi]) * most, tokens = min(most, g.count * D - t0);
            if (tokens > 0) {
                out.tok0 = g.first * D + t0;
                out.rows = tokens * p.call.G;
                out.seen = g.pages * kPage;
                out.limit = AttnChunk::kManySequences;
                int longest = out.tok0 / D;
                for (int n = out.tok0 / D + lane; n <= (out.tok0 + tokens - 1) / D; n += 32) {
                    const int len = capped_len(p.call, n);
                    if (len > 0) out.seen = min(out.seen, max(1, len - D + 1));
                    if (len > out.len) {
                        out.len = len;
                        longest = n;
                    }
                }
                const int len = __reduce_max_sync(~0u, out.len);
                longest = __shfl_sync(~0u, longest, __ffs(__ballot_sync(~0u, out.len == len)) - 1);
                out.len = min(len, g.pages * kPage);
                out.seen = min(out.seen, out.len);
                out.table = (int64_t)longest * p.call.max_pages;
            }
        }
        out.seen = __reduce_min_sync(~0u, out.seen);
        if (lane == 0) {
            (is_few ? few_prefix : prefix)[at] = out;
            if (!is_few && at < kPlanCached) sizes[at] = size_of(out);
        }
    }
    // the sequences, and the chunks of what follows their prefixes (from the last warps on: the first have the chunks above)
    for (int n = kPlanThreads - 1 - tid; n < p.call.batch; n += kPlanThreads) {
        SeqPlan out{};
        const int len = capped_len(p.call, n), gi = last_at_most(p.group_start, p.groups, n);
        if (p.call.err_flag && p.call.seq_lens[n] > p.call.max_pages * kPage) atomicOr(p.call.err_flag, KDA_DEVERR_PAGE);
        if (gi >= 0) {
            const Group g = group_of(p, gi, false);
            const Sharing how = sharing_of(p, lay, g);
            if (how != kNone && n >= g.first && n < g.first + g.count) {
                out.base = g.pages * kPage;
                out.few = how == kFew;
                out.first = how == kFew ? few_chunk[gi] : group_chunk[gi];
                out.token = (n - g.first) * D;
            }
        }
        seqs[n] = out;
        for (int i = 0; i < lay.at[1].per; ++i) {
            AttnChunk c{};
            const int t0 = i * lay.at[1].tokens;
            c.table = (int64_t)n * p.call.max_pages + out.base / kPage;
            c.tok0 = n * D + t0;
            c.rows = min(lay.at[1].tokens, D - t0) * p.call.G;
            c.base = out.base;
            c.len = max(0, len - out.base);
            c.limit = len - D + 1 + t0 - out.base;
            c.seen = min(c.len, max(1, c.limit));
            rest[(int64_t)n * lay.at[1].per + i] = c;
            const int64_t at = lay.at[0].chunks + (int64_t)n * lay.at[1].per + i;
            if (at < kPlanCached) sizes[at] = size_of(c);
        }
    }
    if (!lay.on_tc) return;

    // ---- the workers' ranges: the chunks' costs laid end to end, cut evenly
    __shared__ int64_t cached[kPlanCached];
    __shared__ int64_t warp_cost[kPlanThreads / 32];
    __shared__ int4 starts[kSms + 1];
    const int count = (int)(lay.at[0].chunks + (lay.tc[1] ? lay.at[1].chunks : 0)), Hkv = p.call.Hkv;
    int64_t *costs = count <= kPlanCached ? cached : reinterpret_cast<int64_t *>(ws + lay.costs);
    if (used == 0 && !lay.tc[1]) {  // small groups alone
        if (tid <= lay.workers) reinterpret_cast<int4 *>(ws + lay.starts)[tid] = make_int4(count, 0, 0, 0);
        return;
    }
    __syncthreads();  // (the chunks are written)
    auto size = [&](int c) { return c < kPlanCached ? sizes[c] : size_of(prefix[c]); };
    auto weight = [](int size) { return 1 + (size & 1); };
    auto item_cost = [&](int size) { return size > 1 ? kItemCost + (size >> 1) * weight(size) : 0; };
    int64_t sum = 0;
    for (int c0 = 0; c0 < count; c0 += kPlanThreads) {
        const int64_t mine = c0 + tid < count ? (int64_t)item_cost(size(c0 + tid)) * Hkv : 0;
        int64_t all;
        const int64_t at = sum + scan(mine, warp_cost, all);
        sum += all;
        if (c0 + tid < count) costs[c0 + tid] = at;  // before the chunk
    }
    __syncthreads();
    // no more workers than have a block of their own (starts that differ), however the cuts are rounded
    const int W = (int)max((int64_t)1, min((int64_t)lay.workers, sum / (kItemCost + 4)));
    if (tid <= lay.workers) {
        int4 start = make_int4(count, 0, 0, 0);
        if (tid < W && sum > 0) {
            const int64_t target = sum * tid / W;
            int lo = 0, hi = count;  // the last chunk with costs[c] <= target
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (costs[mid] <= target) lo = mid;
                else hi = mid;
            }
            const int c = size(lo);
            const int64_t rem = target - costs[lo];
            const int each = item_cost(c), head = (int)(rem / each), in = (int)(rem % each);
            start = make_int4(lo, head, in <= kItemCost ? 0 : ((in - kItemCost) / weight(c)) & ~1, 0);
        }
        starts[tid] = start;
        reinterpret_cast<int4 *>(ws + lay.starts)[tid] = start;
    }
    __syncthreads();
    // the first and last worker of each item, a thread each
    int *desc = reinterpret_cast<int *>(ws + lay.at[0].desc);  // (the rest's follow the prefixes')
    for (uint32_t i = tid >> 1; i < (uint32_t)count * Hkv; i += kPlanThreads / 2) {  // (shared_layout)
        const int c = (int)(i / Hkv), h = (int)(i % Hkv), pages = size(c) >> 1, page = tid & 1 ? pages - 1 : 0;
        int lo = 0, hi = W;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            const int4 x = starts[mid];
            if (x.x < c || (x.x == c && (x.y < h || (x.y == h && x.z <= page)))) lo = mid;
            else hi = mid;
        }
        desc[2 * (int64_t)i + (tid & 1)] = pages > 0 ? lo : -(tid & 1);
    }
}

// Adds up the parts of the rows, in order: HD / 4 lanes a row, four parts' loads in
// flight together.  A part is (m, l, o) of one of the two attentions, at the row
// where one worker had all of it, else in the workers' slots.
constexpr int kMergeThreads = 128;

template <typename T, int HD>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const AttnSharedParams p, const SharedLayout lay) {
    constexpr int TPR = HD / 4, ROWS = kMergeThreads / TPR;
    const AttnDecodeParams &c = p.call;
    const int64_t qrow = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
    const int c4 = threadIdx.x % TPR;
    if (qrow >= (int64_t)c.batch * c.D * c.Hq) return;
    const int hq = (int)(qrow % c.Hq), h = hq / c.G, gi = hq % c.G;
    const int64_t tok = qrow / c.Hq;
    const int n = (int)(tok / c.D), t = (int)(tok % c.D);
    const unsigned char *ws = static_cast<const unsigned char *>(c.workspace);
    const int sees = capped_len(c, n) - c.D + 1 + t;  // positions in all
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const SeqPlan sp = reinterpret_cast<const SeqPlan *>(ws + lay.seqs)[n];

    // where the two attentions left the row's results: parts (one: at the row), the first part's worker, the row
    // within the item's partial results
    int count[2], first[2], row[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const bool few = s == 0 && sp.few;
        const PartsAt &a = lay.at[few ? 2 : s];
        const int local = s == 0 ? sp.token + t : t;
        const int64_t chunk = (s == 0 ? (int64_t)sp.first : (int64_t)n * a.per) + local / a.tokens;
        const int r = (local % a.tokens) * c.G + gi, rb = r / a.R;
        row[s] = r - rb * a.R;
        first[s] = 0;
        count[s] = (s == 0 ? min(sees, sp.base) : sees - sp.base) > 0 && chunk < a.chunks ? 1 : 0;
        if (count[s] > 0 && !a.whole) {
            const int2 desc = *reinterpret_cast<const int2 *>(ws + a.desc + 8 * ((chunk * c.Hkv + h) * a.RB + rb));
            // (a worker that gave up waiting leaves no or stale entries)
            first[s] = desc.x;
            count[s] = desc.x < 0 || desc.x > desc.y || desc.y >= a.workers ? 0 : desc.y - desc.x + 1;
        }
    }
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const PartsAt &a = lay.at[s == 0 && sp.few ? 2 : s];
        const float *part_m = reinterpret_cast<const float *>(ws + a.part_m), *part_l = reinterpret_cast<const float *>(ws + a.part_l);
        const float *part_o = reinterpret_cast<const float *>(ws + a.part_o);
        constexpr int BATCH = 4;
        for (int x0 = 0; x0 < count[s]; x0 += BATCH) {
            float pm[BATCH], pl[BATCH];
            float4 v[BATCH];
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const int x = min(x0 + b, count[s] - 1);
                if (count[s] == 1) {
                    const float2 ml = reinterpret_cast<const float2 *>(ws + lay.at[s].ml)[qrow];
                    pm[b] = ml.x;
                    pl[b] = ml.y;
                    v[b] = reinterpret_cast<const float4 *>(ws + lay.at[s].o)[qrow * TPR + c4];
                } else {  // part x lies in slot 2 (w + x), the first in slot 2 w + 1
                    const int64_t k = (2 * ((int64_t)first[s] + x) + (x == 0 ? 1 : 0)) * a.PR + row[s];
                    pm[b] = part_m[k];
                    pl[b] = part_l[k];
                    v[b] = reinterpret_cast<const float4 *>(part_o)[k * TPR + c4];
                }
            }
            float most = m;
#pragma unroll
            for (int b = 0; b < BATCH; ++b) most = fmaxf(most, pl[b] == 0.f ? m : pm[b]);
            const float use = most == -INFINITY ? 0.f : most, fix = ex2(m - use);
            l *= fix;
            o.x *= fix; o.y *= fix; o.z *= fix; o.w *= fix;
            m = most;
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                if (x0 + b >= count[s] || pl[b] == 0.f) continue;  // (a part whose pages are not in the cache has l = 0)
                const float f = ex2(pm[b] - use);
                l = fmaf(f, pl[b], l);
                o.x = fmaf(f, v[b].x, o.x); o.y = fmaf(f, v[b].y, o.y);
                o.z = fmaf(f, v[b].z, o.z); o.w = fmaf(f, v[b].w, o.w);
            }
        }
    }
    const float f = l == 0.f ? 0.f : 1.f / l;
    T *dst = static_cast<T *>(c.out) + qrow * HD + 4 * c4;
    store2(dst, l == 0.f ? 0.f : o.x * f, l == 0.f ? 0.f : o.y * f);
    store2(dst + 2, l == 0.f ? 0.f : o.z * f, l == 0.f ? 0.f : o.w * f);
    if (c4 == 0 && c.lse) c.lse[qrow] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <typename T>
cudaError_t launch_merge(const AttnSharedParams &p, const SharedLayout &lay, int d, cudaStream_t st) {
    const int64_t rows = (int64_t)p.call.batch * p.call.D * p.call.Hq, each = kMergeThreads / (d / 4);
    const dim3 grid((unsigned)((rows + each - 1) / each));
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
    if (lay.total == 0) return cudaErrorInvalidValue;
    unsigned char *ws = static_cast<unsigned char *>(c.workspace);
    plan_kernel<<<1, kPlanThreads, 0, st>>>(p, lay);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const AttnChunk *chunks = reinterpret_cast<const AttnChunk *>(ws + lay.chunks);
    auto floats = [&](int64_t at) { return reinterpret_cast<float *>(ws + at); };
    auto attend_tc = [&] {
        AttnDecodeParams q = c;
        q.chunks = chunks;
        PartsPlan plan{};
        plan.starts = reinterpret_cast<const int4 *>(ws + lay.starts);
        plan.part = floats(0);
        plan.part_m = lay.at[0].part_m / 4; plan.part_l = lay.at[0].part_l / 4; plan.part_o = lay.at[0].part_o / 4;
        plan.prefix_o = floats(lay.at[0].o); plan.rest_o = floats(lay.at[1].o);
        plan.prefix_ml = reinterpret_cast<float2 *>(ws + lay.at[0].ml);
        plan.rest_ml = reinterpret_cast<float2 *>(ws + lay.at[1].ml);
        plan.first_rest = (int32_t)lay.at[0].chunks;
        plan.rows = kPartRows;
        return launch_parts_tc(q, plan, lay.workers, d, st);
    };
    auto attend = [&](int s) {
        if (lay.tc[s] || lay.at[s].chunks == 0) return cudaSuccess;
        AttnDecodeParams q = c;
        q.chunks = chunks + (s == 0 ? 0 : lay.at[0].chunks + (s == 1 ? 0 : lay.at[1].chunks));
        q.part_ml = reinterpret_cast<float2 *>(ws + lay.at[s].ml);
        q.out = ws + lay.at[s].o;
        q.lse = nullptr;
        q.workspace = ws + lay.ws[s];
        q.batch = (int32_t)lay.at[s].chunks;
        return launch_parts(q, lay.lay[s], d, dtype, st);
    };
    if (c.max_pages > 0) {
        if (lay.on_tc && (e = attend_tc()) != cudaSuccess) return e;
        for (int s : {0, 2, 1})
            if ((e = attend(s)) != cudaSuccess) return e;
    }
    return dtype == KDA_DT_BF16 ? launch_merge<__nv_bfloat16>(p, lay, d, st) : launch_merge<float>(p, lay, d, st);
}

}  // namespace kda
