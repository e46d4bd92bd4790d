// Instances of the MXFP4 product kernel per token-tile size.
#include "mg_kernel.cuh"

namespace fn {

MGInstance mg_pick(int tok) {
  switch (tok) {
    case 16: return {mg_kernel<16>, 16, MGShape<16>::kSmem};
    case 64: return {mg_kernel<64>, 64, MGShape<64>::kSmem};
    case 128: return {mg_kernel<128>, 128, MGShape<128>::kSmem};
    case 256: return {mg_kernel<256>, 256, MGShape<256>::kSmem};
    default: return {nullptr, 0, 0};
  }
}

}  // namespace fn
