// Instances of the rotary kernels: sides of few heads, several tokens to a warp.
#include "rope.cuh"

namespace adaln {

void* rope_few_kernel(int es, int lanes, bool half, int mode) {
  if (es == 2)
    return half ? rope::wide_kernel<2, true, true>(lanes, mode)
                : rope::wide_kernel<2, false, true>(lanes, mode);
  return half ? rope::wide_kernel<4, true, true>(lanes, mode)
              : rope::wide_kernel<4, false, true>(lanes, mode);
}

}  // namespace adaln
