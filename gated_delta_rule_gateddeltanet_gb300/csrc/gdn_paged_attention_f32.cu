// Paged attention over FP32 caches (see gdn_paged_attention.cuh).
#include "gdn_paged_attention.cuh"

namespace gdn {
template cudaError_t launch_paged_attention<GDN_F32>(const PagedAttnParams &p, cudaStream_t stream);
}
