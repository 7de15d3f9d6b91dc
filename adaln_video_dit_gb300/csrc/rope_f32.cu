// Instances of the rotary kernels: fp32 heads in 16-byte vectors.
#include "rope.cuh"

namespace adaln {

void* rope_f32_kernel(int lanes, bool half, int mode) {
  return half ? rope::wide_kernel<4, true, false>(lanes, mode)
              : rope::wide_kernel<4, false, false>(lanes, mode);
}

}  // namespace adaln
