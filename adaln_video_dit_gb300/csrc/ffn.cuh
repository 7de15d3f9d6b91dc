// Shared by the two forms of the gated feed-forward block: the activations, the
// format of what a forward saves, and the host's tensor maps and launches.
#pragma once

#include "internal.h"
#include "tc.cuh"

namespace adaln {

// The saved g and u are only ever read by the backward's epilogue, so they lie
// in its order: for each 32 x 32 block twelve rows of 32 lanes x 16 bytes (g:
// four of upper halves, two of the next bytes; then u), each one coalesced
// access of a warp.
constexpr int kSavedVecs = 12, kSavedBlock = kSavedVecs * 512;
// ----- activations --------------------------------------------------------------
// p such that act(g) = g p, and act'(g).  The sigmoid form of the tanh
// approximation (0.5 (1 + tanh z) = 1 / (1 + exp(-2 z))) keeps its relative
// accuracy for negative g.  The fast exponential and division are good to a
// few fp32 units, far below the bf16 rounding that follows.
__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

template <int ACT>
__device__ __forceinline__ void gate(float g, float& p, float& d) {
  if (ACT == ADALN_ACT_SILU) {
    p = sigmoid(g);
    d = p * (1.0f + g * (1.0f - p));
  } else if (ACT == ADALN_ACT_GELU_TANH) {
    const float k = 0.7978845608028654f, c = 0.044715f;
    const float g2 = g * g;
    p = sigmoid(2.0f * k * g * (1.0f + c * g2));
    const float q = p * (1.0f - p);
    d = q > 0.0f ? p + 2.0f * k * g * q * (1.0f + 3.0f * c * g2) : p;
  } else {
    p = 0.5f * erfcf(-0.7071067811865476f * g);
    d = p + g * 0.3989422804014327f * __expf(-0.5f * g * g);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}

// ----- host side ------------------------------------------------------------------

inline int div_up(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

inline size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

inline size_t saved_bytes(int64_t T, int32_t F) {
  return (size_t)div_up(T, 32) * div_up(F, 32) * kSavedBlock;
}

// Tensor map of a row-major bf16 matrix [rows, cols] in boxes of box_cols (64
// or 32: rows of 128 or 64 bytes, swizzled at that width) x box_rows.  What
// lies outside reads as zero and is not written.
cudaError_t make_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int box_cols,
                     int box_rows);

// Launch as a programmatic dependent, in clusters of `cluster` CTAs.
cudaError_t launch_cluster(void* kernel, int grid, int threads, int smem, int cluster, void** params,
                           cudaStream_t st);

// The few-token form (ffn_skinny.cu): whether it serves T tokens, the workspace
// it needs, and its two launches.  `saved` may be NULL.
bool skinny_serves(int64_t T);
size_t skinny_workspace(int64_t T, int32_t F);
cudaError_t skinny_fwd(const void* x, const void* wg, const void* wu, const void* wd, int T, int D,
                       int F, int act, void* y, void* saved, void* workspace, unsigned* status,
                       cudaStream_t st);

}  // namespace adaln
