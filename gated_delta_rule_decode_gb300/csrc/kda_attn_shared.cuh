// How a batch that shares prefixes is laid out for its attention: between the
// plan (kda_attn_shared.cu) and the tcgen05 kernel (kda_attn_shared_tc.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_attn_internal.h"

namespace kda {
namespace dec {

constexpr int kPartRows = 256;  // rows of a chunk and of a partial result, on tcgen05

// Ranges of the workers (chunk, kv head, page; starts[workers] is the end) and
// where results go: those of items that one worker has to itself at their rows,
// fp32 and not divided by l, others to the worker's slots: the one that begins
// at its item's first page in slot 2 w + 1, the other in slot 2 w.
struct PartsPlan {
    const int4 *starts;
    float *part;
    int64_t part_m, part_l, part_o;  // in floats
    float *prefix_o, *rest_o;
    float2 *prefix_ml, *rest_ml;
    int32_t first_rest, rows;        // the chunks from here on are no prefixes'; kPartRows
};

cudaError_t launch_parts_tc(const AttnDecodeParams &p, const PartsPlan &plan, int workers, int d, cudaStream_t st);

}  // namespace dec
}  // namespace kda
