// Paged-cache kernels and launchers for vectors of length d = 256.
#include "kvq_paged_inst.cuh"

namespace kvq {
template cudaError_t launch_norm_rope<256>(int, const NormRopeArgs&, int, cudaStream_t);
template cudaError_t launch_append<256>(int, int, const AppendArgs&, int, cudaStream_t);
template cudaError_t launch_paged_attn<256>(const PagedAttnArgs&, int, int, cudaStream_t);
template cudaError_t read_paged_status<256>(uint32_t*, bool);
}  // namespace kvq
