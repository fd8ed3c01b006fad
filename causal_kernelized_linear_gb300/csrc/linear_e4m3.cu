// The product of e4m3 operands with a scale for each of their rows (see linear_tc.cuh).
#include "linear_tc.cuh"

namespace la {

const char* tc_linear_e4m3_kernel(const LinearArgs& a) { return kernel_name<true>(a); }

cudaError_t tc_linear_e4m3(const LinearE4m3Args& a, cudaStream_t s) {
  return by_activation<true>(a.base, a.x_scale, a.w_scale, s);
}

}  // namespace la
