// Paged attention over BF16 caches (see gdn_paged_attention.cuh).
#include "gdn_paged_attention.cuh"

namespace gdn {
template cudaError_t launch_paged_attention<GDN_BF16>(const PagedAttnParams &p, cudaStream_t stream);
}
