// Instances of the MXFP4 product kernel per token-tile size.
#include "mg_kernel.cuh"

namespace fn {

MGInstance mg_pick(int tok) {
  switch (tok) {
    case 16: return {mg_kernel<16, 1>, 16, 1, MGShape<16, 1>::kSmem};
    case 64: return {mg_kernel<64, 1>, 64, 1, MGShape<64, 1>::kSmem};
    case 128: return {mg_kernel<128, 1>, 128, 1, MGShape<128, 1>::kSmem};
    case 256: return {mg_kernel<256, 2>, 256, 2, MGShape<256, 2>::kSmem};
    default: return {nullptr, 0, 0, 0};
  }
}

}  // namespace fn
