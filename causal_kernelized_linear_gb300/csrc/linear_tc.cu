// The bf16 product (see linear_tc.cuh).
#include "linear_tc.cuh"

namespace la {

const char* tc_linear_kernel(const LinearArgs& a) { return kernel_name<false>(a); }

cudaError_t tc_linear(const LinearArgs& a, cudaStream_t s) {
  return by_activation<false>(a, nullptr, nullptr, s);
}

}  // namespace la
