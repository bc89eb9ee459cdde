// Paged attention over 8-bit integer caches (see gdn_paged_attention.cuh).
#include "gdn_paged_attention.cuh"

namespace gdn {
template cudaError_t launch_paged_attention<GDN_INT8>(const PagedAttnParams &p, cudaStream_t stream);
}
