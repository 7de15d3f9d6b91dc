// Instances of the rotary kernels: bf16 heads in 16-byte vectors.
#include "rope.cuh"

namespace adaln {

void* rope_bf16_kernel(int lanes, bool half, int mode) {
  return half ? rope::wide_kernel<2, true, false>(lanes, mode)
              : rope::wide_kernel<2, false, false>(lanes, mode);
}

}  // namespace adaln
