// Norm and rotation by one position a token, and the gradient (norm_rope_kernels.cuh).
#include "norm_rope_kernels.cuh"

namespace mita {

int norm_rope_backward_blocks(int sms) { return 8 * sms; }

template <typename T>
cudaError_t launch_norm_rope(NormRopeArgs<T> a, int d, int sms, cudaStream_t st) {
  return forward_any<T, OnePosition>(a, d, sms, st);
}

template <typename T>
cudaError_t launch_norm_rope_backward(NormRopeBackwardArgs<T> a, int d, float* partial, int sms,
                                      float* dwq, float* dwk, cudaStream_t st) {
  return backward_any<T, OnePosition>(a, d, partial, sms, dwq, dwk, st);
}

template cudaError_t launch_norm_rope<float>(NormRopeArgs<float>, int, int, cudaStream_t);
template cudaError_t launch_norm_rope<bf16>(NormRopeArgs<bf16>, int, int, cudaStream_t);
template cudaError_t launch_norm_rope_backward<float>(NormRopeBackwardArgs<float>, int, float*, int,
                                                      float*, float*, cudaStream_t);
template cudaError_t launch_norm_rope_backward<bf16>(NormRopeBackwardArgs<bf16>, int, float*, int,
                                                     float*, float*, cudaStream_t);

}  // namespace mita
