#include "simt_gated_delta_launch.cuh"

namespace kata {
template cudaError_t simt_gated_delta<__nv_bfloat16>(const GatedDeltaLaunch &, int, int);
template cudaError_t simt_gated_delta_backward<__nv_bfloat16>(const GatedDeltaLaunch &, int, int);
}  // namespace kata
