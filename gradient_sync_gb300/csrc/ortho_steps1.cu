// The Newton-Schulz steps with tiles of one CTA.
#include "ortho_steps.cuh"

namespace ar {

template cudaError_t launch_steps<false, 1>(OrthoTable&, cudaStream_t);
template cudaError_t launch_steps<true, 1>(OrthoTable&, cudaStream_t);

}  // namespace ar
