// Instances of the rotary kernels: halves that only 8- or 4-byte vectors fit.
#include "rope.cuh"

namespace adaln {

namespace {
template <int SIZE, int W>
void* narrow(int lanes, int mode) {
  return lanes == 10   ? rope::vec_kernel<SIZE, W, 10, true, false>(mode)
         : lanes == 16 ? rope::vec_kernel<SIZE, W, 16, true, false>(mode)
                       : rope::vec_kernel<SIZE, W, 32, true, false>(mode);
}
}  // namespace

void* rope_narrow_kernel(int es, int width, int lanes, int mode) {
  if (es == 4) return narrow<4, 2>(lanes, mode);
  return width == 2 ? narrow<2, 2>(lanes, mode) : narrow<2, 1>(lanes, mode);
}

}  // namespace adaln
