// The gated feed-forward block of each expert of a mixture, on its rows of a sorted
// array (route.cu), forward and backward.
//
//   y = (act(x Wg[e]') * (x Wu[e]')) Wd[e]'     for the rows x of expert e
//
// with xs, ys, dys, dxs [rows, D]; Wg, Wu [E, F, D]; Wd [E, D, F], all bf16; the
// formulas, roundings and kernel are the block's (ffn.cu), whose tiles of rows are
// here each one expert's: a tile starts at an expert's first row or 256 rows on, and
// multiplies with that expert's matrix.  Where the experts' rows start is read on the
// device, so the number of tiles is not known on the host: the kernel counts them
// (fetch_starts), and its CTA pairs walk what there is.
//
// Starts are multiples of 64 rows with zeros between, so that a warp's 32-row block of
// an output and a 64-row step of a weight gradient's sum are each one expert's; the
// weight gradients' sums take the zeros in.  A tile past its expert's rows neither
// reads A there nor stores what comes of it.
//
// Few rows an expert have a form of their own (experts_few.cu), while the arrays hold at
// most one block of 64 rows and a half an expert: filled with 64 rows of each of 16
// experts at 1000 x 2728, 8 at 1536 x 4096, 64 at 2048 x 1024 and 4 at 5120 x 3584 it takes
// 61, 62, 137 and 80 us for the forward where the tiles take 63, 70, 150 and 108; with 128
// rows 95, 74, 164 and 85 against 81, 73, 156 and 105, with 192 rows it loses on all four.
// The rule sees the arrays' rows only, and a route's hold 63 an expert beside its pairs:
// a routed call leaves the form at 33 (many experts) to 40 (eight) pairs an expert on
// average, wherever they go.  On both sides of that, spread evenly, forward and backward
// alone from cold caches: 8 experts of 1536 x 4096 76 and 136 us with 34 pairs, 83 and 134
// with 48; 16 of 1000 x 2728 75 and 153, 74 and 147; 64 of 2048 x 1024 154 and 324 with
// 33, 158 and 313 with 34.  All to one expert, whose weights the form then reads again for
// every 64 rows: 64 of 2048 x 1024 54 and 218 us with 32 pairs an expert, 37 and 250 with
// 34; 256 of 512 x 1024 93 and 300, 38 and 269.
//
// Bound (one GB300): the tensor cores at the power limit with thousands of rows an
// expert (T = 32760, two of 8 experts, D = 5120, F = 13824, forward 15.9 to 16.4 ms, 1700
// to 1750 TFLOP/s; 8192 tokens, two of 8, D = 1536, F = 4096, forward and backward 1333
// to 1395 us, 1330 to 1390, where the gate's two kernels run at the L2 rate as the
// block's do); the L2 rate and what a unit's start and end cost with a few hundred rows
// (2222 rows of 16 experts, D = 1000, F = 2728, both passes 261 to 265 us for 540 MB: a
// weight-gradient tile is two or three k blocks, and reads as much as it writes).
#include "ffn_gemm.cuh"

namespace adaln {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int check(int64_t rows, int32_t E, int32_t D, int32_t F, adaln_dtype_t dt, int act) {
  if (dt != ADALN_BF16) return ADALN_ERR_DTYPE;
  if (rows < 0 || rows > ADALN_FFN_MAX_T || E < 1 || E > ADALN_MAX_EXPERTS) return ADALN_ERR_DIM;
  if (D < 8 || D > ADALN_FFN_MAX_DIM || D % 8 != 0) return ADALN_ERR_DIM;
  if (F < 8 || F > ADALN_FFN_MAX_DIM || F % 8 != 0) return ADALN_ERR_DIM;
  if (act != ADALN_ACT_SILU && act != ADALN_ACT_GELU_TANH && act != ADALN_ACT_GELU) return ADALN_ERR_ARG;
  return ADALN_OK;
}

// Tiles of rows, at most, and as many as are likely: `rows` is a route's, the pairs'
// number and 63 for each expert that they may meet, and an expert's last tile is half
// full on average.
int64_t most_tiles(int64_t rows, int32_t E) {
  const int64_t blocks = rows / kRowAlign, met = blocks < E ? blocks : E;
  return (blocks + 3 * met) / 4;
}
int64_t likely_tiles(int64_t rows, int32_t E) {
  const int64_t blocks = rows / kRowAlign, pairs = rows - (kRowAlign - 1) * (int64_t)E;
  if (blocks <= E) return blocks;
  const int64_t tiles = pairs / kTM + E / 2;
  return tiles > E ? tiles : E;
}

struct FwdPlan {
  bool few;
  Tiling gate, y;
  size_t bytes;
};
FwdPlan fwd_plan(int64_t rows, int32_t E, int32_t D, int32_t F, int pairs) {
  FwdPlan p = {};
  p.few = experts_few_serve(rows, E);
  if (p.few) {
    p.bytes = round256((size_t)rows * F * 2);
    return p;
  }
  const int64_t tiles = likely_tiles(rows, E);
  p.gate = choose_tiling(rows, tiles, F, div_up(D, kBK), true, false, false, pairs);
  p.y = choose_tiling(rows, tiles, D, div_up(F, kBK), false, false, true, pairs);
  p.bytes = round256((size_t)rows * F * 2) + round256(p.y.bytes);
  return p;
}

struct BwdPlan {
  bool few;
  Tiling gate, dx, dw;
  int worth;
  size_t bytes;
};
BwdPlan bwd_plan(int64_t rows, int32_t E, int32_t D, int32_t F, int pairs) {
  BwdPlan p = {};
  const int64_t tiles_m = likely_tiles(rows, E);
  p.gate = choose_tiling(rows, tiles_m, F, div_up(D, kBK), false, true, false, pairs);
  p.dw = {128, 1, 0};
  p.few = experts_few_serve(rows, E);
  if (p.few) {
    p.bytes = 3 * round256((size_t)rows * F * 2);
    return p;
  }
  const double unit = unit_clocks(div_up(rows, (int64_t)E * kBK), 128);
  const int64_t tiles = 2 * tiles_of(div_up(F, kTM), D, false, 128) + tiles_of(div_up(D, kTM), F, false, 128);
  const int kb = 2 * div_up(F, kBK);
  p.dx = choose_tiling(rows, tiles_m, D, kb, false, true, true, pairs, tiles * E * unit, unit);
  p.worth = (int)(unit_clocks(div_up(kb, p.dx.splits), p.dx.w) / unit);
  p.bytes = 3 * round256((size_t)rows * F * 2) + round256(p.dx.bytes);
  return p;
}

// A sorted array [rows, cols] (depth 1), or the experts' matrices [E, rows, cols].
struct Matrix {
  const void* p;
  int64_t depth, rows, cols;
  bool mn;
};
cudaError_t map_of(CUtensorMap* m, const Matrix& o, int box_rows) {
  return make_map(m, o.p, o.depth, o.rows, o.cols, kBK, o.mn ? kBK : box_rows);
}
cudaError_t blocks_of(CUtensorMap* m, const void* p, int64_t depth, int64_t rows, int64_t cols) {
  return make_map(m, p, depth, rows, cols, 32, 32);
}

// out [M, N] (of each expert where by_k) = the sum over up to two segments of a b,
// each over k values (by_k: over the expert's rows).
cudaError_t set_problem(Problem* p, const Matrix (&a)[2], const Matrix (&b)[2], int segs, int64_t M, int N,
                        int64_t tiles_m, bool gate, const Tiling& t, int64_t k, bool by_k, int64_t depth,
                        void* out) {
  cudaError_t e = map_of(&p->a[0], a[0], kRowAlign);
  if (e == cudaSuccess) e = map_of(&p->b[0], b[0], t.w);
  if (e == cudaSuccess && segs > 1) e = map_of(&p->a[1], a[1], kRowAlign);
  if (e == cudaSuccess && b[1].p != nullptr) e = map_of(&p->b[1], b[1], t.w);
  if (e == cudaSuccess && out) e = make_map(&p->out, out, depth, M, N, 64, 32);
  p->partial = nullptr;
  Dims& s = p->s;
  s.M = (int)M;
  s.N = N;
  s.kb0 = by_k ? INT32_MAX : div_up(k, kBK);
  s.kb = by_k ? 0 : segs * s.kb0;
  s.tiles_m = (int)tiles_m;
  s.w = t.w;
  s.tiles_n = div_up(N, cover(gate, t.w));
  s.splits = t.splits;
  s.first = 0;
  s.a_mn = a[0].mn;
  s.b_mn = b[0].mn;
  s.by_k = by_k;
  s.inv_each = 1.0f / (float)((by_k ? s.tiles_m : s.splits) * (int64_t)s.tiles_n);
  s.inv_group = 1.0f / (float)(kGroupM * s.tiles_n);
  return e;
}

GemmArgs args_of(int64_t rows, int32_t E, const int32_t* starts, unsigned* status) {
  GemmArgs a = {};
  a.starts = starts, a.experts = E, a.rows = rows, a.status = status;
  return a;
}

}  // namespace
}  // namespace adaln

using namespace adaln;

extern "C" {

int adaln_experts_ffn_saved_size(int64_t rows, int32_t E, int32_t D, int32_t F, adaln_dtype_t dtype,
                                 size_t* bytes) {
  const int rc = check(rows, E, D, F, dtype, ADALN_ACT_SILU);
  if (rc != ADALN_OK) return rc;
  if (!bytes) return ADALN_ERR_NULL;
  *bytes = saved_bytes(rows, F);
  return ADALN_OK;
}

int adaln_experts_ffn_workspace_size(int64_t rows, int32_t E, int32_t D, int32_t F, adaln_dtype_t dtype,
                                     size_t* fwd_bytes, size_t* bwd_bytes) {
  const int rc = check(rows, E, D, F, dtype, ADALN_ACT_SILU);
  if (rc != ADALN_OK) return rc;
  if (!fwd_bytes && !bwd_bytes) return ADALN_ERR_NULL;
  int pairs = 0;
  const cudaError_t e = pairs_of_device<true>(&pairs);
  if (e != cudaSuccess) return launch_failed(e);
  if (fwd_bytes) *fwd_bytes = fwd_plan(rows, E, D, F, pairs).bytes;
  if (bwd_bytes) *bwd_bytes = bwd_plan(rows, E, D, F, pairs).bytes;
  return ADALN_OK;
}

int adaln_experts_ffn_fwd(const void* xs, const void* wg, const void* wu, const void* wd,
                          const int32_t* starts, int64_t rows, int32_t E, int32_t D, int32_t F,
                          adaln_dtype_t dtype, adaln_act_t act, void* ys, void* saved, void* workspace,
                          size_t workspace_bytes, void* stream) {
  const int rc = check(rows, E, D, F, dtype, act);
  if (rc != ADALN_OK) return rc;
  if (rows < kRowAlign) return ADALN_OK;  // no expert has a row
  if (!xs || !wg || !wu || !wd || !starts || !ys || !workspace) return ADALN_ERR_NULL;
  if (!aligned16(xs) || !aligned16(wg) || !aligned16(wu) || !aligned16(wd) || !aligned16(ys) ||
      !aligned16(saved) || !aligned16(workspace) || (reinterpret_cast<uintptr_t>(starts) & 3) != 0)
    return ADALN_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int pairs = 0;
  cudaError_t e = pairs_of_device<true>(&pairs);
  if (e != cudaSuccess) return launch_failed(e);
  const FwdPlan plan = fwd_plan(rows, E, D, F, pairs);
  if (workspace_bytes < plan.bytes) return ADALN_ERR_WORKSPACE;
  unsigned* status = nullptr;
  if ((e = status_word(&status)) != cudaSuccess) return launch_failed(e);
  GemmArgs a = args_of(rows, E, starts, status);
  char* h = static_cast<char*>(workspace);
  if (plan.few) {
    e = experts_few_fwd({xs, wg, wu, wd, starts, rows, E, D, F, act}, ys, saved, h, status, st);
    return e == cudaSuccess ? ADALN_OK : launch_failed(e);
  }
  const int64_t tiles = most_tiles(rows, E);
  const Matrix none = {}, x = {xs, 1, rows, D, false}, hk = {h, 1, rows, F, false};
  const Matrix g = {wg, E, F, D, false}, u = {wu, E, F, D, false}, d = {wd, E, D, F, false};
  a.saved = static_cast<uint4*>(saved);
  a.problems = 1;
  e = blocks_of(&a.h, h, 1, rows, F);
  if (e == cudaSuccess)
    e = set_problem(&a.p[0], {x, none}, {g, u}, 1, rows, F, tiles, true, plan.gate, D, false, 1, nullptr);
  if (e == cudaSuccess) e = launch_gemm<true>(a, saved ? kGateSave : kGate, act, pairs, 0, st);
  if (e == cudaSuccess)
    e = set_problem(&a.p[0], {hk, none}, {d, none}, 1, rows, D, tiles, false, plan.y, F, false, 1, ys);
  a.p[0].partial = reinterpret_cast<float*>(h + round256((size_t)rows * F * 2));
  if (e == cudaSuccess) e = launch_gemm<true>(a, kPlain, act, pairs, 0, st);
  if (e == cudaSuccess && plan.y.splits > 1) e = launch_join(a.p[0], ys, starts + E, pairs, st);
  return e == cudaSuccess ? ADALN_OK : launch_failed(e);
}

int adaln_experts_ffn_bwd(const void* dys, const void* xs, const void* wg, const void* wu, const void* wd,
                          const int32_t* starts, const void* saved, int64_t rows, int32_t E, int32_t D,
                          int32_t F, adaln_dtype_t dtype, adaln_act_t act, void* dxs, void* dwg, void* dwu,
                          void* dwd, void* workspace, size_t workspace_bytes, void* stream) {
  const int rc = check(rows, E, D, F, dtype, act);
  if (rc != ADALN_OK) return rc;
  const bool any = rows >= kRowAlign;
  if (!dwg || !dwu || !dwd) return ADALN_ERR_NULL;
  if (any && (!dys || !xs || !wg || !wu || !wd || !starts || !saved || !dxs || !workspace))
    return ADALN_ERR_NULL;
  if (!aligned16(dwg) || !aligned16(dwu) || !aligned16(dwd)) return ADALN_ERR_ALIGN;
  if (any && (!aligned16(dys) || !aligned16(xs) || !aligned16(wg) || !aligned16(wu) || !aligned16(wd) ||
              !aligned16(saved) || !aligned16(dxs) || !aligned16(workspace) ||
              (reinterpret_cast<uintptr_t>(starts) & 3) != 0))
    return ADALN_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (!any) {  // empty sums
    void* const out[3] = {dwg, dwu, dwd};
    for (int i = 0; i < 3 && e == cudaSuccess; ++i)
      e = cudaMemsetAsync(out[i], 0, (size_t)E * D * F * 2, st);
    return e == cudaSuccess ? ADALN_OK : launch_failed(e);
  }
  int pairs = 0;
  if ((e = pairs_of_device<true>(&pairs)) != cudaSuccess) return launch_failed(e);
  const BwdPlan plan = bwd_plan(rows, E, D, F, pairs);
  if (workspace_bytes < plan.bytes) return ADALN_ERR_WORKSPACE;
  unsigned* status = nullptr;
  if ((e = status_word(&status)) != cudaSuccess) return launch_failed(e);
  GemmArgs a = args_of(rows, E, starts, status);

  const size_t rf = round256((size_t)rows * F * 2);
  char* ws = static_cast<char*>(workspace);
  char *h = ws, *dg = ws + rf, *du = ws + 2 * rf;
  const Matrix none = {};
  const int64_t tiles = most_tiles(rows, E);
  if (plan.few) {
    e = experts_few_bwd({xs, wg, wu, wd, starts, rows, E, D, F, act}, dys, saved, h, dg, du, dxs, status, st);
  } else {
    a.saved = static_cast<uint4*>(const_cast<void*>(saved));  // read only here
    e = blocks_of(&a.h, h, 1, rows, F);
    if (e == cudaSuccess) e = blocks_of(&a.dg, dg, 1, rows, F);
    if (e == cudaSuccess) e = blocks_of(&a.du, du, 1, rows, F);
    const Matrix dyk = {dys, 1, rows, D, false}, dn = {wd, E, D, F, true};
    a.problems = 1;
    if (e == cudaSuccess)
      e = set_problem(&a.p[0], {dyk, none}, {dn, none}, 1, rows, F, tiles, false, plan.gate, D, false, 1,
                      nullptr);
    if (e == cudaSuccess) e = launch_gemm<true>(a, kGateBwd, act, pairs, 0, st);
  }
  if (e != cudaSuccess) return launch_failed(e);

  // dx first: its units are the longer ones.
  const Matrix dgk = {dg, 1, rows, F, false}, duk = {du, 1, rows, F, false};
  const Matrix gn = {wg, E, F, D, true}, un = {wu, E, F, D, true};
  const Matrix dgm = {dg, 1, rows, F, true}, dum = {du, 1, rows, F, true}, hm = {h, 1, rows, F, true};
  const Matrix xm = {xs, 1, rows, D, true}, dym = {dys, 1, rows, D, true};
  const int64_t tf = div_up(F, kTM), td = div_up(D, kTM);
  Problem* p = a.p;
  if (!plan.few) {
    e = set_problem(p, {dgk, duk}, {gn, un}, 2, rows, D, tiles, false, plan.dx, F, false, 1, dxs);
    p->partial = reinterpret_cast<float*>(ws + 3 * rf);
    ++p;
  }
  if (e == cudaSuccess)
    e = set_problem(p++, {dgm, none}, {xm, none}, 1, F, D, tf, false, plan.dw, 0, true, E, dwg);
  if (e == cudaSuccess)
    e = set_problem(p++, {dum, none}, {xm, none}, 1, F, D, tf, false, plan.dw, 0, true, E, dwu);
  if (e == cudaSuccess)
    e = set_problem(p++, {dym, none}, {hm, none}, 1, D, F, td, false, plan.dw, 0, true, E, dwd);
  a.problems = (int)(p - a.p);
  if (e == cudaSuccess) e = launch_gemm<true>(a, kPlain, act, pairs, plan.few ? 1 : plan.worth, st);
  if (e == cudaSuccess && !plan.few && plan.dx.splits > 1) e = launch_join(a.p[0], dxs, starts + E, pairs, st);
  return e == cudaSuccess ? ADALN_OK : launch_failed(e);
}

}  // extern "C"
