// Gated feed-forward block on the tensor cores, forward and backward.
//
//   g = x Wg',  u = x Wu',  h = act(g) * u,  y = h Wd'
//   dh = dy Wd, dg = dh * u * act'(g), du = dh * act(g)
//   dx = dg Wg + du Wu,  dWg = dg' x,  dWu = du' x,  dWd = dy' h
//
// with x, y, dy, dx [T, D]; Wg, Wu [F, D]; Wd [D, F], all bf16 and row-major
// (so an operand is either K-major or MN-major in memory, and the matrix
// instructions take both: nothing is transposed).  Sums are fp32 in tensor
// memory.  The forward needs 6 T D F operations, the backward 12 T D F.
//
// Two kernels make the forward: both projections with the activation and the
// product in their epilogue (g and u meet in one tile: the even CTA of a pair
// stages rows of Wg, the odd one rows of Wu, so an accumulator holds 128
// columns of g and the same 128 of u), then the product with Wd.  The backward
// makes dh with the gate's gradient in its epilogue, then dx and the three
// weight gradients in one launch.
//
// Roundings to bf16: h, dg and du, once each, because the matrix instructions
// take 16-bit operands; and the outputs.  g and u themselves are kept for the
// backward as fp32 cut to 24 bits (2^-15 relative), not as bf16: with 8 bits of
// mantissa their rounding would enter dg, du and h beside those arrays' own.
//
// A kernel is persistent, one CTA pair per two SMs: a 256 x 256 tile a pair
// (narrower ones where that fills the pairs better), k steps of 64 through a
// ring of TMA-filled stages; per CTA one producer warp, one issuing warp (even
// CTA) and eight epilogue warps, two accumulators in tensor memory so that a
// tile's epilogue runs under the next tile's products.
//
// Bound: the tensor cores where there are tiles for every pair, the L2 rate
// where a unit's operands are read for few products, idle pairs where neither
// the tiles nor the splits of k that pay for their join fill them.  Measured (one
// GB300; 1725 TFLOP/s is what the library's bf16 product sustains under the power
// limit, 1947 in a burst; ranges over two runs): T = 32760, D = 5120, F = 13824
// forward 7.7 to 7.8 ms, 1774 to 1815 TFLOP/s; T = 8192 forward and backward 6.2
// to 6.3 ms, 1647 to 1690; T = 8192, D = 1536, F = 4096 forward 168 us, 1840,
// forward and backward 625 to 642 us, 1445 to 1484.  There (k = 1536) the products
// are busy for 96 % of the weight gradients' and dx's launch, 87 % of y's (192 tiles
// are 2.5 rounds of 76 pairs), 73 % of the projections' while saving and 53 % of the
// gate's gradient: the last two move 10 and 14 bytes through L2 per 1000 operations
// where the first moves 7, and all three run at the same 15 TB/s of it.  T = 256,
// D = 5120, F = 13824 forward 98 us: the projections at that rate too, y on 60 of 76
// pairs.  T = 1111, D = 1000, F = 2728 forward and backward 90 us: y on 40 pairs, the
// gate's gradient on 55, 1111 rows computed as 1280.
#include <mutex>

#include "ffn_gemm.cuh"

namespace adaln {
namespace {

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                             const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                             const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

cudaError_t encode_fn(EncodeFn* out) {
  static std::mutex mu;
  static EncodeFn fn = nullptr;
  std::lock_guard<std::mutex> lk(mu);
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                           cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || !p) return cudaErrorNotSupported;
    fn = reinterpret_cast<EncodeFn>(p);
  }
  *out = fn;
  return cudaSuccess;
}

cudaError_t encode(CUtensorMap* m, int rank, const void* p, int64_t depth, int64_t rows, int64_t cols,
                   int box_cols, int box_rows) {
  EncodeFn fn;
  const cudaError_t e = encode_fn(&fn);
  if (e != cudaSuccess) return e;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)depth};
  const cuuint64_t strides[2] = {(cuuint64_t)cols * 2, (cuuint64_t)cols * rows * 2};
  const cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1}, one[3] = {1, 1, 1};
  const CUresult r =
      fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(p), dims, strides, box, one,
         CU_TENSOR_MAP_INTERLEAVE_NONE,
         box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t make_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int box_cols,
                     int box_rows) {
  return encode(m, 2, p, 1, rows, cols, box_cols, box_rows);
}
cudaError_t make_map(CUtensorMap* m, const void* p, int64_t depth, int64_t rows, int64_t cols,
                     int box_cols, int box_rows) {
  return encode(m, 3, p, depth, rows, cols, box_cols, box_rows);
}

cudaError_t launch_cluster(void* kernel, int grid, int threads, int smem, int cluster, void** params,
                           cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelExC(&cfg, kernel, params);
}

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int check(int64_t T, int32_t D, int32_t F, adaln_dtype_t dt, int act) {
  if (dt != ADALN_BF16) return ADALN_ERR_DTYPE;
  if (T < 0 || T > ADALN_FFN_MAX_T) return ADALN_ERR_DIM;
  if (D < 8 || D > ADALN_FFN_MAX_DIM || D % 8 != 0) return ADALN_ERR_DIM;
  if (F < 8 || F > ADALN_FFN_MAX_DIM || F % 8 != 0) return ADALN_ERR_DIM;
  if (act != ADALN_ACT_SILU && act != ADALN_ACT_GELU_TANH && act != ADALN_ACT_GELU)
    return ADALN_ERR_ARG;
  return ADALN_OK;
}

struct FwdPlan {
  Tiling gate, y;
  size_t bytes;
};
FwdPlan fwd_plan(int64_t T, int32_t D, int32_t F, int pairs) {
  FwdPlan p = {};
  if (skinny_serves(T)) {
    p.bytes = skinny_workspace(T, F);
    return p;
  }
  const int tiles = div_up(T, kTM);
  p.gate = choose_tiling(T, tiles, F, div_up(D, kBK), true, false, false, pairs);
  p.y = choose_tiling(T, tiles, D, div_up(F, kBK), false, false, true, pairs);
  p.bytes = round256((size_t)T * F * 2) + round256(p.y.bytes);
  return p;
}

struct BwdPlan {
  Tiling gate, dx, dw;
  int worth;
  size_t bytes;
};
BwdPlan bwd_plan(int64_t T, int32_t D, int32_t F, int pairs) {
  BwdPlan p = {};
  const int tiles_m = div_up(T, kTM);
  p.gate = choose_tiling(T, tiles_m, F, div_up(D, kBK), false, true, false, pairs);
  p.dw = {128, 1, 0};
  const double unit = unit_clocks(div_up(T, kBK), 128);
  const int64_t tiles = 2 * tiles_of(div_up(F, kTM), D, false, 128) + tiles_of(div_up(D, kTM), F, false, 128);
  const int kb = 2 * div_up(F, kBK);
  p.dx = choose_tiling(T, tiles_m, D, kb, false, true, true, pairs, tiles * unit, unit);
  p.worth = (int)(unit_clocks(div_up(kb, p.dx.splits), p.dx.w) / unit);
  p.bytes = 3 * round256((size_t)T * F * 2) + round256(p.dx.bytes);
  return p;
}

}  // namespace
}  // namespace adaln

using namespace adaln;

extern "C" {

int adaln_ffn_saved_size(int64_t T, int32_t D, int32_t F, adaln_dtype_t dtype, size_t* bytes) {
  const int rc = check(T, D, F, dtype, ADALN_ACT_SILU);
  if (rc != ADALN_OK) return rc;
  if (!bytes) return ADALN_ERR_NULL;
  *bytes = saved_bytes(T, F);
  return ADALN_OK;
}

int adaln_ffn_workspace_size(int64_t T, int32_t D, int32_t F, adaln_dtype_t dtype, size_t* fwd_bytes,
                             size_t* bwd_bytes) {
  const int rc = check(T, D, F, dtype, ADALN_ACT_SILU);
  if (rc != ADALN_OK) return rc;
  if (!fwd_bytes && !bwd_bytes) return ADALN_ERR_NULL;
  int pairs = 0;
  const cudaError_t e = pairs_of_device<false>(&pairs);
  if (e != cudaSuccess) return launch_failed(e);
  if (fwd_bytes) *fwd_bytes = fwd_plan(T, D, F, pairs).bytes;
  if (bwd_bytes) *bwd_bytes = bwd_plan(T, D, F, pairs).bytes;
  return ADALN_OK;
}

int adaln_ffn_fwd(const void* x, const void* wg, const void* wu, const void* wd, int64_t T,
                  int32_t D, int32_t F, adaln_dtype_t dtype, adaln_act_t act, void* y, void* saved,
                  void* workspace, size_t workspace_bytes, void* stream) {
  const int rc = check(T, D, F, dtype, act);
  if (rc != ADALN_OK) return rc;
  if (T == 0) return ADALN_OK;
  if (!x || !wg || !wu || !wd || !y || !workspace) return ADALN_ERR_NULL;
  if (!aligned16(x) || !aligned16(wg) || !aligned16(wu) || !aligned16(wd) || !aligned16(y) ||
      !aligned16(saved) || !aligned16(workspace))
    return ADALN_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int pairs = 0;
  cudaError_t e = pairs_of_device<false>(&pairs);
  if (e != cudaSuccess) return launch_failed(e);
  const FwdPlan plan = fwd_plan(T, D, F, pairs);
  if (workspace_bytes < plan.bytes) return ADALN_ERR_WORKSPACE;
  GemmArgs a = {};
  if ((e = status_word(&a.status)) != cudaSuccess) return launch_failed(e);
  if (skinny_serves(T)) {
    e = skinny_fwd(x, wg, wu, wd, (int)T, D, F, act, y, saved, workspace, a.status, st);
    return e == cudaSuccess ? ADALN_OK : launch_failed(e);
  }

  char* ws = static_cast<char*>(workspace);
  a.saved = static_cast<uint4*>(saved);
  e = block_map(&a.h, ws, T, F);
  if (e != cudaSuccess) return launch_failed(e);
  const Operand none = {};
  a.problems = 1;
  e = set_problem(&a.p[0], {{x, T, D, false}, none}, {{wg, F, D, false}, {wu, F, D, false}}, 1, T, F,
                  true, plan.gate, D, 0, nullptr);
  if (e == cudaSuccess) e = launch_gemm<false>(a, saved ? kGateSave : kGate, act, pairs, 0, st);
  if (e != cudaSuccess) return launch_failed(e);

  e = set_problem(&a.p[0], {{ws, T, F, false}, none}, {{wd, D, F, false}, none}, 1, T, D, false, plan.y,
                  F, 0, y);
  a.p[0].partial = reinterpret_cast<float*>(ws + round256((size_t)T * F * 2));
  if (e == cudaSuccess) e = launch_gemm<false>(a, kPlain, act, pairs, 0, st);
  if (e == cudaSuccess && plan.y.splits > 1) e = launch_join(a.p[0], y, nullptr, pairs, st);
  return e == cudaSuccess ? ADALN_OK : launch_failed(e);
}

int adaln_ffn_bwd(const void* dy, const void* x, const void* wg, const void* wu, const void* wd,
                  const void* saved, int64_t T, int32_t D, int32_t F, adaln_dtype_t dtype,
                  adaln_act_t act, void* dx, void* dwg, void* dwu, void* dwd, void* workspace,
                  size_t workspace_bytes, void* stream) {
  const int rc = check(T, D, F, dtype, act);
  if (rc != ADALN_OK) return rc;
  if (!dwg || !dwu || !dwd) return ADALN_ERR_NULL;
  if (T > 0 && (!dy || !x || !wg || !wu || !wd || !saved || !dx || !workspace))
    return ADALN_ERR_NULL;
  if (!aligned16(dwg) || !aligned16(dwu) || !aligned16(dwd)) return ADALN_ERR_ALIGN;
  if (T > 0 && (!aligned16(dy) || !aligned16(x) || !aligned16(wg) || !aligned16(wu) ||
                !aligned16(wd) || !aligned16(saved) || !aligned16(dx) || !aligned16(workspace)))
    return ADALN_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (T == 0) {  // empty sums
    void* const out[3] = {dwg, dwu, dwd};
    for (int i = 0; i < 3 && e == cudaSuccess; ++i)
      e = cudaMemsetAsync(out[i], 0, (size_t)D * F * 2, st);
    return e == cudaSuccess ? ADALN_OK : launch_failed(e);
  }
  int pairs = 0;
  if ((e = pairs_of_device<false>(&pairs)) != cudaSuccess) return launch_failed(e);
  const BwdPlan plan = bwd_plan(T, D, F, pairs);
  if (workspace_bytes < plan.bytes) return ADALN_ERR_WORKSPACE;
  GemmArgs a = {};
  if ((e = status_word(&a.status)) != cudaSuccess) return launch_failed(e);

  const size_t tf = round256((size_t)T * F * 2);
  char* ws = static_cast<char*>(workspace);
  char *h = ws, *dg = ws + tf, *du = ws + 2 * tf;
  a.saved = static_cast<uint4*>(const_cast<void*>(saved));  // read only here
  e = block_map(&a.h, h, T, F);
  if (e == cudaSuccess) e = block_map(&a.dg, dg, T, F);
  if (e == cudaSuccess) e = block_map(&a.du, du, T, F);
  if (e != cudaSuccess) return launch_failed(e);

  const Operand none = {};
  a.problems = 1;
  e = set_problem(&a.p[0], {{dy, T, D, false}, none}, {{wd, D, F, true}, none}, 1, T, F, false,
                  plan.gate, D, 0, nullptr);
  if (e == cudaSuccess) e = launch_gemm<false>(a, kGateBwd, act, pairs, 0, st);
  if (e != cudaSuccess) return launch_failed(e);

  // dx first: its units are the longer ones.
  const Operand dgk = {dg, T, F, false}, duk = {du, T, F, false};
  const Operand dgm = {dg, T, F, true}, dum = {du, T, F, true};
  const Operand xm = {x, T, D, true}, dym = {dy, T, D, true}, hm = {h, T, F, true};
  a.problems = 4;
  e = set_problem(&a.p[0], {dgk, duk}, {{wg, F, D, true}, {wu, F, D, true}}, 2, T, D, false,
                  plan.dx, F, F, dx);
  a.p[0].partial = reinterpret_cast<float*>(ws + 3 * tf);
  if (e == cudaSuccess)
    e = set_problem(&a.p[1], {dgm, none}, {xm, none}, 1, F, D, false, plan.dw, T, 0, dwg);
  if (e == cudaSuccess)
    e = set_problem(&a.p[2], {dum, none}, {xm, none}, 1, F, D, false, plan.dw, T, 0, dwu);
  if (e == cudaSuccess)
    e = set_problem(&a.p[3], {dym, none}, {hm, none}, 1, D, F, false, plan.dw, T, 0, dwd);
  if (e == cudaSuccess) e = launch_gemm<false>(a, kPlain, act, pairs, plan.worth, st);
  if (e == cudaSuccess && plan.dx.splits > 1) e = launch_join(a.p[0], dx, nullptr, pairs, st);
  return e == cudaSuccess ? ADALN_OK : launch_failed(e);
}

}  // extern "C"
