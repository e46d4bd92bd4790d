// Instances of the MXFP4 product kernels.
#include "mg_kernel.cuh"
#include "mgp_kernel.cuh"

namespace fn {

template <int TOK, int ID>
MGInstance instance() {
  return {mg_kernel<TOK>, TOK, MGShape<TOK>::kSmem, 2, ID};
}

MGInstance mg_pick(int tok) {
  return tok <= 16 ? instance<16, 0>() : instance<64, 1>();
}

MGInstance mg_pair() { return {mgp_kernel, kMgPairRows, MGPShape::kSmem, 1, 2}; }

MGArrangeKernel mg_arrange() { return mgp_arrange_kernel; }

}  // namespace fn
