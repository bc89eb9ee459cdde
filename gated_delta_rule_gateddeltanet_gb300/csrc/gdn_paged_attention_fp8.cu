// Paged attention over 8-bit e4m3 caches (see gdn_paged_attention.cuh).
#include "gdn_paged_attention.cuh"

namespace gdn {
template cudaError_t launch_paged_attention<GDN_FP8_E4M3>(const PagedAttnParams &p, cudaStream_t stream);
}
