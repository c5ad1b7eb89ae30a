// Norm and rotation by positions of several axes, and the gradient (norm_rope_kernels.cuh).
//
// A lane has four frequencies, so four positions a token instead of one, and no more arithmetic.  Measured (bf16):
// 66,313 tokens of 16 + 4 heads of 128, three axes, in 111 us, 6.1 TB/s (one position:
// 114; fp32 222, gradients 171 and 306, 6.0 and 6.7 TB/s); 16 x 1025 tokens of 12 + 12 heads of 64, two axes,
// in 23 us (20.4; fp32 36), their gradient in 34.5 us (32; fp32 53), 4.4 TB/s, where neither HBM (45 %) nor the
// schedulers (53 %) are full: latency, and 5 us of start, reduction and a second launch.
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
