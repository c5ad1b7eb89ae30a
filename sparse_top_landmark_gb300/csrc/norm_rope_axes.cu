// Norm and rotation by positions of several axes, and the gradient (norm_rope_kernels.cuh).
#include "norm_rope_kernels.cuh"

namespace mita {

template <typename T>
cudaError_t launch_norm_rope_axes(NormRopeArgs<T> a, int d, int sms, cudaStream_t st) {
  return forward_any<T, AxisPositions>(a, d, sms, st);
}

template <typename T>
cudaError_t launch_norm_rope_axes_backward(NormRopeBackwardArgs<T> a, int d, float* partial, int sms,
                                      float* dwq, float* dwk, cudaStream_t st) {
  return backward_any<T, AxisPositions>(a, d, partial, sms, dwq, dwk, st);
}

template cudaError_t launch_norm_rope_axes<float>(NormRopeArgs<float>, int, int, cudaStream_t);
template cudaError_t launch_norm_rope_axes<bf16>(NormRopeArgs<bf16>, int, int, cudaStream_t);
template cudaError_t launch_norm_rope_axes_backward<float>(NormRopeBackwardArgs<float>, int, float*, int,
                                                      float*, float*, cudaStream_t);
template cudaError_t launch_norm_rope_axes_backward<bf16>(NormRopeBackwardArgs<bf16>, int, float*, int,
                                                     float*, float*, cudaStream_t);

}  // namespace mita
