// Instances of the MXFP4 product kernels.
#include "mg_kernel.cuh"
#include "mgp_kernel.cuh"

namespace fn {

template <int TOK>
MGInstance instance() {
  return {mg_kernel<TOK>, TOK, MGShape<TOK>::kSmem, MGShape<TOK>::kPerSm};
}

MGInstance mg_pick(int tok) {
  return tok <= 16 ? instance<16>() : instance<64>();
}

MGInstance mg_pair() { return {mgp_kernel, kMgPairRows, MGPShape::kSmem, 1}; }

MGArrangeKernel mg_arrange() { return mgp_arrange_kernel; }

}  // namespace fn
