#include "simt_gated_delta_launch.cuh"

namespace kata {
template cudaError_t simt_gated_delta<float>(const GatedDeltaLaunch &, int, int);
template cudaError_t simt_gated_delta_backward<float>(const GatedDeltaLaunch &, int, int);
}  // namespace kata
