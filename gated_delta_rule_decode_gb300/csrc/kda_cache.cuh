// The pages that a call with packed new tokens touches: one unit of seq_of_unit
// each, shared by the append and the key summaries.
#pragma once

#include <stdint.h>

#include "kda_attn_internal.h"

namespace kda {

// The page of a unit: its sequence's rows lo..hi - 1 (positions), the first of
// them token `tok`.  False where the unit has no page.  The page's id is not
// checked here, so that its read and those of the rows overlap.
struct PageRows {
    int64_t page, tok;
    int rows, off;  // new rows, and the place of the first in the page
};

template <typename P>
__device__ __forceinline__ bool page_of_unit(const P &p, int64_t unit, PageRows &r) {
    int64_t c = 0;
    const int s = seq_of_unit(p.cu_seqlens, p.num_seqs, kPage, 2, unit, p.err_flag, c);
    int t0, t1;
    const int64_t start = p.start_pos[s];
    if (!seq_range(p.cu_seqlens, s, p.total_tokens, p.err_flag, t0, t1)) return false;
    if (c < 0 || t1 == t0 || start < 0) return false;
    const int64_t end = start + (t1 - t0), idx = start / kPage + c;
    if (idx * kPage >= end) return false;
    const int64_t lo = idx * kPage > start ? idx * kPage : start;
    const int64_t hi = (idx + 1) * kPage < end ? (idx + 1) * kPage : end;
    r.rows = (int)(hi - lo);
    r.off = (int)(lo - idx * kPage);
    r.tok = (int64_t)t0 + (lo - start);
    r.page = idx < p.max_pages ? p.block_table[(int64_t)s * p.max_pages + idx] : -1;
    return true;
}

}  // namespace kda
