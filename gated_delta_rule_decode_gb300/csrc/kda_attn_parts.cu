// The cache attention kernels of chunks of rows whose results stay apart (see
// AttnChunk): built by themselves, beside those of whole sequences.  As quick as
// these: 943 pages of 64 sequences (32 heads over 8, d = 128) 63 us cold, both.
#include "kda_attn_decode.cuh"
#include "kda_attn_decode_rows.cuh"
#include "kda_attn_internal.h"

namespace kda {
namespace dec {

template <typename T>
static cudaError_t launch_parts_dim(const AttnDecodeParams &p, const Layout &lay, int d, cudaStream_t st) {
    if (d == 128) return launch_items<T, 128, true>(p, lay, st);
    if (d == 64) return launch_items<T, 64, true>(p, lay, st);
    return launch_items<T, 32, true>(p, lay, st);
}

cudaError_t launch_parts(const AttnDecodeParams &p, const Layout &lay, int d, int dtype, cudaStream_t st) {
    if (lay.items > 0x7fffffff || (int64_t)p.max_pages * p.Hkv * lay.RB > 0x7fffffff) return cudaErrorInvalidValue;
    return dtype == KDA_DT_BF16 ? launch_parts_dim<__nv_bfloat16>(p, lay, d, st) : launch_parts_dim<float>(p, lay, d, st);
}

}  // namespace dec
}  // namespace kda
