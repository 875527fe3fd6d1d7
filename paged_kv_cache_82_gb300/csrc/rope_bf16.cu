// rope_bf16.cu -- pa_norm_rope_and_cache: over bf16 inputs, and the choice of type.
#include "rope_kernels.cuh"

namespace pa {

template cudaError_t launch_rope<__nv_bfloat16>(const RopeArgs&, int, unsigned*, cudaStream_t);

cudaError_t launch_norm_rope_and_cache(const RopeArgs& a, int num_sms, unsigned* err,
                                       cudaStream_t stream) {
  switch (a.dtype) {
    case PA_F32: return launch_rope<float>(a, num_sms, err, stream);
    case PA_F16: return launch_rope<__half>(a, num_sms, err, stream);
    case PA_BF16: return launch_rope<__nv_bfloat16>(a, num_sms, err, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pa
