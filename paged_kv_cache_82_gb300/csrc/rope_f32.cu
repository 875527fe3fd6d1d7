// rope_f32.cu -- pa_norm_rope_and_cache over fp32 inputs.
#include "rope_kernels.cuh"

namespace pa {

template cudaError_t launch_rope<float>(const RopeArgs&, int, unsigned*, cudaStream_t);

}  // namespace pa
