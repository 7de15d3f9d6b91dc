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
// p such that act(g) = g p, and d = act'(g), for two values at a time.  The
// sigmoid form of the tanh approximation (0.5 (1 + tanh z) = 1 / (1 + exp(-2 z)))
// keeps its relative accuracy for negative g.  The exponential and reciprocal
// are the hardware's, good to a few fp32 units and flushing denormals, far below
// the bf16 rounding that follows; the epilogues that use them are bound by
// instructions, not by their own data.
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;
// 1 / (1 + exp(-z)), z given as z log2(e).
__device__ __forceinline__ float2 sigmoid2(float2 z) {
  return make_float2(rcp_approx(1.0f + ex2_approx(-z.x)), rcp_approx(1.0f + ex2_approx(-z.y)));
}

template <int ACT>
__device__ __forceinline__ void gate(float2 g, float2& p, float2& d) {
  const float2 one = splat2(1.0f);
  if (ACT == ADALN_ACT_SILU) {
    p = sigmoid2(mul2(g, splat2(kLog2e)));
    d = mul2(p, fma2(g, fma2(p, splat2(-1.0f), one), one));
  } else if (ACT == ADALN_ACT_GELU_TANH) {
    const float k = 0.7978845608028654f, c = 0.044715f;
    const float2 g2 = mul2(g, g);
    p = sigmoid2(mul2(g, fma2(g2, splat2(2.0f * k * c * kLog2e), splat2(2.0f * k * kLog2e))));
    const float2 q = mul2(p, fma2(p, splat2(-1.0f), one));
    const float2 t = mul2(mul2(g, q), fma2(g2, splat2(6.0f * k * c), splat2(2.0f * k)));
    // (Where q has vanished g^2 may have overflowed: 0 * inf.)
    d = make_float2(q.x > 0.0f ? p.x + t.x : p.x, q.y > 0.0f ? p.y + t.y : p.y);
  } else {
    p = make_float2(0.5f * erfcf(-0.7071067811865476f * g.x), 0.5f * erfcf(-0.7071067811865476f * g.y));
    const float2 e = mul2(mul2(g, g), splat2(-0.5f * kLog2e));
    const float2 n = mul2(g, splat2(0.3989422804014327f));
    d = make_float2(fmaf(n.x, ex2_approx(e.x), p.x), fmaf(n.y, ex2_approx(e.y), p.y));
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

// The same of `depth` such matrices, one after the other: 3-D, so that a box past
// one's rows reads zeros and not the next one's.
cudaError_t make_map(CUtensorMap* m, const void* p, int64_t depth, int64_t rows, int64_t cols,
                     int box_cols, int box_rows);

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

// CTAs that share the k blocks of each of `blocks` blocks of features in the few-token
// forms: as many as are resident at two an SM, up to a cluster.
int choose_splits(int64_t blocks, int kb, int sms);

// The experts' blocks for few rows an expert (experts_few.cu): whether it serves, the
// forward's two launches and the backward's up to dx.  `saved` may be NULL; h, dg and
// du are [rows, F].
struct Experts {
  const void *xs, *wg, *wu, *wd;
  const int32_t* starts;
  int64_t rows;
  int32_t E, D, F;
  int act;
};
bool experts_few_serve(int64_t rows, int32_t E);
cudaError_t experts_few_fwd(const Experts& x, void* ys, void* saved, void* h, unsigned* status,
                            cudaStream_t st);
cudaError_t experts_few_bwd(const Experts& x, const void* dys, const void* saved, void* h, void* dg, void* du,
                            void* dxs, unsigned* status, cudaStream_t st);

}  // namespace adaln
