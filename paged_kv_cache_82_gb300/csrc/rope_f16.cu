// rope_f16.cu -- pa_norm_rope_and_cache over f16 inputs.
#include "rope_kernels.cuh"

namespace pa {

template cudaError_t launch_rope<__half>(const RopeArgs&, int, unsigned*, cudaStream_t);

}  // namespace pa
