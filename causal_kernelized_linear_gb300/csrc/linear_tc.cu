// The bf16 product (see linear_tc.cuh).
#include "linear_tc.cuh"

namespace la {

const char* tc_linear_kernel(const LinearArgs& a) {
  static const char* const names[] = {"few16", "few32", "few64", "few128", "pair128", "pair256"};
  return names[choose(a, kblocks_of<false>(a))];
}

cudaError_t tc_linear(const LinearArgs& a, cudaStream_t s) {
  return by_activation<false>(a, nullptr, nullptr, s);
}

}  // namespace la
