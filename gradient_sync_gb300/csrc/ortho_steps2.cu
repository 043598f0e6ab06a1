// The Newton-Schulz steps with tiles of a pair of CTAs.
#include "ortho_steps.cuh"

namespace ar {

template cudaError_t launch_steps<false, 2>(OrthoTable&, cudaStream_t);
template cudaError_t launch_steps<true, 2>(OrthoTable&, cudaStream_t);

}  // namespace ar
