// Rotary positions over several axes for queries and keys, with an optional
// RMS norm of every head in the same pass; forward and backward.
//
// For one head x[0..dh) of token t, with R = 2P rotated elements, pair p made
// of elements (2p, 2p+1) (interleaved) or (p, p+P) (halves), pair p on axis
// a(p), and (c, s) = table[pos[t, a(p)], p] (or (1, 0) at position -1):
//
//   n  = x * r * w,  r = 1 / sqrt(mean(x^2) + eps)      (n = x without norm)
//   y1 = n1 c - n2 s,  y2 = n2 c + n1 s                 (elements >= R: y = n)
//
// and backward, from dy (R' is the rotation by the opposite angle):
//
//   g  = R' dy,  dw = sum over tokens and heads of g x r,  h = g w,
//   dx = r h - x (r^3 mean(h x))                        (dx = g without norm)
//
// Bound: HBM.  Forward and plain rotation read and write every element once;
// the norm's backward reads x and dy and writes dx.  Nothing is saved by the
// forward: r is recomputed from the x that the backward has to read anyway.
//
// Measured (one GB300, share of the rate of a plain copy): rotation backward of
// T = 36864 x 48 heads x 128, bf16, 135.8 us, 98 %; norm and rotation of T = 32760
// x 80 heads x 128 read out of a packed projection 203.3 us, 97 %; norm, forward
// and backward, of T = 16384 x 48 heads: 128 wide 84 % (bf16) and 92 % (fp32), 80
// wide 70 and 92 %, 64 wide 71 and 94 %.  Bf16, T = 16384 x 48 heads: halves in
// 8-byte vectors (72 wide) rotation 64, norm 58, its backward 55 %; in 4-byte ones
// (68 wide: 17 of 32 lanes at work) 35, 33 and 23 %; the scalar path (100 wide,
// interleaved) 22, 18 and 22 %.  These are bound by their instructions and by what
// they have in flight: a lane's loads are 2 to 8 times as narrow, so the issue
// slots are 51 to 62 % busy (scalar 28 to 34 %) where the memory is half idle.
// A call on one token takes 2.6 us of the GPU.
//
// Layout of the work: P lanes share a head, each holding two 16-byte vectors
// of it that contain whole pairs (interleaved: vectors j and j + half, halves:
// a vector and its partner; 8- or 4-byte vectors where the halves need it), so a
// rotation never leaves its lane and a norm
// takes about log2(P) shuffles (P need not be a power of two: heads of 80 bf16
// elements take 5 lanes, six heads to a warp).  A warp walks tokens, and of each
// token the heads of its chunk, U groups of 32 / P heads at a time with the next
// ones on their way; where a side has no more heads than one group (grouped
// keys), it takes as many tokens at a time instead as fill U groups.  The
// cosines and sines of its tokens and the weights are read from shared memory,
// where the lanes of different heads read the same words: in registers they
// would cost half of what a thread has, and with it the loads in flight.
#include <cmath>

#include "rope.cuh"

namespace adaln {
namespace {

using namespace rope;

template <class E>
__device__ __forceinline__ float load1(const char* p);
template <>
__device__ __forceinline__ float load1<BF16>(const char* p) {
  return __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(p));
}
template <>
__device__ __forceinline__ float load1<F32>(const char* p) {
  return *reinterpret_cast<const float*>(p);
}
__device__ __forceinline__ void store1(char* p, float v, BF16) {
  *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(v);
}
__device__ __forceinline__ void store1(char* p, float v, F32) { *reinterpret_cast<float*>(p) = v; }

// Scalar path: any head width up to 64 kScalarPairs, any strides, element
// alignment.  A warp holds one head, lane l the pairs l, l + 32, ...; pairs from P on are
// the unrotated elements, two by two.
template <class E, int MODE, int kScalarPairs>
__global__ void __launch_bounds__(kThreads) rope_scalar_kernel(const __grid_constant__ RopeArgs a,
                                                               int interleaved) {
  constexpr bool kNorm = MODE == kNormFwd || MODE == kNormBwd;
  extern __shared__ float red[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool is_k = (int)blockIdx.x >= a.side[0].chunks * a.side[0].ctas;
  const Side& sd = a.side[is_k];
  const int cta = blockIdx.x - (is_k ? a.side[0].chunks * a.side[0].ctas : 0);
  const int chunk = cta / sd.ctas;
  const int h_end = min(sd.heads, (chunk + 1) * sd.per_chunk);

  int da[kScalarPairs], db[kScalarPairs];  // elements of the pair, -1: none
#pragma unroll
  for (int i = 0; i < kScalarPairs; ++i) {
    const int p = lane + 32 * i;
    da[i] = p >= a.P ? 2 * p : interleaved ? 2 * p : p;
    db[i] = p >= a.P ? 2 * p + 1 : interleaved ? 2 * p + 1 : p + a.P;
    if (da[i] >= a.dh) da[i] = -1;
    if (db[i] >= a.dh) db[i] = -1;
  }

  grid_wait();
  grid_launch_dependents();

  float wa[kScalarPairs], wb[kScalarPairs], dwa[kScalarPairs], dwb[kScalarPairs];
#pragma unroll
  for (int i = 0; i < kScalarPairs; ++i) {
    const char* wp = static_cast<const char*>(sd.w);
    wa[i] = kNorm && wp && da[i] >= 0 ? load1<E>(wp + da[i] * E::SIZE) : 1.0f;
    wb[i] = kNorm && wp && db[i] >= 0 ? load1<E>(wp + db[i] * E::SIZE) : 1.0f;
    dwa[i] = dwb[i] = 0.0f;
  }

  const int64_t step = (int64_t)sd.ctas * kWarps;
  for (int64_t t = (int64_t)(cta - chunk * sd.ctas) * kWarps + warp; t < a.T; t += step) {
    Rows rows;
    rows.load(a, t, lane == 0);
    float2 cs[kScalarPairs];
#pragma unroll
    for (int i = 0; i < kScalarPairs; ++i)
      cs[i] = rows.at(a, axis_of(a, lane + 32 * i), lane + 32 * i);
    for (int h = chunk * sd.per_chunk; h < h_end; ++h) {
      const char* x = sd.x.p + t * sd.x.ts + h * sd.x.hs;
      float fa[kScalarPairs], fb[kScalarPairs], sx = 0.0f;
#pragma unroll
      for (int i = 0; i < kScalarPairs; ++i) {
        fa[i] = da[i] >= 0 ? load1<E>(x + da[i] * E::SIZE) : 0.0f;
        fb[i] = db[i] >= 0 ? load1<E>(x + db[i] * E::SIZE) : 0.0f;
        sx = fmaf(fa[i], fa[i], fmaf(fb[i], fb[i], sx));
      }
      float r = 1.0f;
      if (kNorm) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sx += __shfl_xor_sync(~0u, sx, o);
        r = rsqrtf(fmaf(sx, a.inv_dh, a.eps));
      }
      if (MODE != kNormBwd) {
#pragma unroll
        for (int i = 0; i < kScalarPairs; ++i) {
          if (MODE == kNormFwd) {
            fa[i] = fa[i] * r * wa[i];
            fb[i] = fb[i] * r * wb[i];
          }
          turn<MODE == kRotateBack>(fa[i], fb[i], cs[i].x, cs[i].y);
        }
      } else {
        const char* y = sd.dy.p + t * sd.dy.ts + h * sd.dy.hs;
        float ga[kScalarPairs], gb[kScalarPairs], sh = 0.0f;
#pragma unroll
        for (int i = 0; i < kScalarPairs; ++i) {
          ga[i] = da[i] >= 0 ? load1<E>(y + da[i] * E::SIZE) : 0.0f;
          gb[i] = db[i] >= 0 ? load1<E>(y + db[i] * E::SIZE) : 0.0f;
          turn<true>(ga[i], gb[i], cs[i].x, cs[i].y);
          sh = fmaf(ga[i] * wa[i], fa[i], fmaf(gb[i] * wb[i], fb[i], sh));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sh += __shfl_xor_sync(~0u, sh, o);
        const float k = -(sh * a.inv_dh * r) * r * r;  // (r^3 alone may overflow)
#pragma unroll
        for (int i = 0; i < kScalarPairs; ++i) {
          if (da[i] >= 0) dwa[i] = fmaf(ga[i], fa[i] * r, dwa[i]);
          if (db[i] >= 0) dwb[i] = fmaf(gb[i], fb[i] * r, dwb[i]);
          fa[i] = fmaf(fa[i], k, ga[i] * wa[i] * r);
          fb[i] = fmaf(fb[i], k, gb[i] * wb[i] * r);
        }
      }
      // A lane writes the elements it read: in place works.
      char* o = sd.out + t * sd.out_ts + h * sd.out_hs;
#pragma unroll
      for (int i = 0; i < kScalarPairs; ++i) {
        if (da[i] >= 0) store1(o + da[i] * E::SIZE, fa[i], E());
        if (db[i] >= 0) store1(o + db[i] * E::SIZE, fb[i], E());
      }
    }
  }

  if (MODE == kNormBwd && sd.partial != nullptr) {
#pragma unroll
    for (int i = 0; i < kScalarPairs; ++i) {
      if (da[i] >= 0) red[warp * a.dh + da[i]] = dwa[i];
      if (db[i] >= 0) red[warp * a.dh + db[i]] = dwb[i];
    }
    store_partial(red, sd.partial + (int64_t)cta * a.dh, a.dh);
  }
}

// dw[d] = sum of the partial slots of a side, in a fixed order: 32 columns a
// CTA, warp w the slots w, w + 32, ... in order, then the 32 warps in order.
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* pq, int nq, float* dwq,
                                                       const float* pk, int nk, float* dwk,
                                                       int dh) {
  __shared__ float red[32][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int d = blockIdx.x * 32 + lane;
  const float* p = blockIdx.y == 0 ? pq : pk;
  const int n = blockIdx.y == 0 ? nq : nk;
  float* dw = blockIdx.y == 0 ? dwq : dwk;
  grid_wait();
  if (dw == nullptr) return;
  float s = 0.0f;
  if (d < dh) {
#pragma unroll 4
    for (int i = warp; i < n; i += 32) s += p[(int64_t)i * dh + d];
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && d < dh) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < 32; ++w) t += red[w][lane];
    dw[d] = t;
  }
}

// ----- host side ---------------------------------------------------------------

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

cudaError_t launch(void* kernel, dim3 grid, int threads, size_t smem, void** params,
                   cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, kernel, params);
}

// Lanes of a head of which `want` hold data: each count that puts one more head
// into a warp than the next (the narrower vectors: the widths they are for).
int lanes_of(int want, int width) {
  if (width == 4 && want <= 8) return want <= 4 ? 4 : want <= 6 ? want : 8;
  return want <= 10 ? 10 : want <= 16 ? 16 : 32;
}

void* pick_kernel(int es, int width, int lanes, bool half, bool few, int mode) {
  if (width < 4) return rope_narrow_kernel(es, width, lanes, mode);
  if (few) return rope_few_kernel(es, lanes, half, mode);
  return es == 2 ? rope_bf16_kernel(lanes, half, mode) : rope_f32_kernel(lanes, half, mode);
}

template <class E, int PAIRS>
void* scalar_kernel(int mode) {
  return mode == kRotate       ? (void*)rope_scalar_kernel<E, kRotate, PAIRS>
         : mode == kRotateBack ? (void*)rope_scalar_kernel<E, kRotateBack, PAIRS>
         : mode == kNormFwd    ? (void*)rope_scalar_kernel<E, kNormFwd, PAIRS>
                               : (void*)rope_scalar_kernel<E, kNormBwd, PAIRS>;
}

// The most shared memory that a plan of the vector path can need: per warp two
// sets of three groups' tokens' tables, and the weights' table.  Tokens side by
// side in a warp times entries of a token's table are at most M x 32 (M = 4 with
// 16-byte vectors of bf16).
constexpr int kMostShared = 4 * 32 * (int)sizeof(float4) * (2 * kWarps * 3 + 1);

struct Plan {
  int width;      // words of a vector, 0: scalar path
  int lanes;      // lanes of a head (vector path)
  int chunks[2];  // per side
  int per_chunk[2];
  int ctas[2];    // per chunk
  int tpw[2];     // few heads: tokens side by side in a warp, else 0
  bool few;       // some tpw is not 0
  int batch;      // tokens whose angles a warp's table holds
};

// Split of a call: the warps of a CTA walk tokens of one chunk of heads, with
// two CTAs an SM in all.  A side is one chunk, so that a token's angles are
// fetched once a side; with few tokens its heads are split until about every
// warp has work.  A side of no more heads than a warp holds (and plenty of
// tokens) takes several tokens at a time: T = 65536 with 8 + 1 heads of 64 took
// 81.0 us a token at a time and 51.6 us so.  The CTAs go to the chunks by
// their cost: a group of heads, and 0.8 of one for a token's angles.
cudaError_t make_plan(int64_t T, const int (&heads)[2], int dh, int mode, int width, int es,
                      Plan* p) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = sm_count(dev, &sms);
  if (e != cudaSuccess) return e;
  *p = Plan{};
  p->width = width;
  p->lanes = 32;
  p->batch = 1;
  int unit = 1;
  if (width) {
    p->lanes = lanes_of((dh * es / (4 * width) + 1) / 2, width);
    unit = 32 / p->lanes;
  }
  const int64_t total = (int64_t)kCtasPerSm * sms, warps = total * kWarps;
  const int64_t split = T > 0 ? (warps + T - 1) / T : 1;  // chunks that give every warp a token
  int64_t small = (heads[0] + heads[1] + split - 1) / split;
  small = (small + unit - 1) / unit * unit;
  double cost[2], all = 0;
  int tokens[2];
  for (int s = 0; s < 2; ++s) {
    int64_t per = heads[s] < small ? heads[s] : small;
    if (per < 1) per = 1;
    const bool few = width == 4 && heads[s] == per && per <= unit && T >= 2 * warps;
    p->per_chunk[s] = (int)per;
    p->chunks[s] = (int)((heads[s] + per - 1) / per);
    p->tpw[s] = few ? unit / (int)per : 0;
    p->few |= few;
    cost[s] = (few ? 1.0 / p->tpw[s] : (double)((per + unit - 1) / unit)) + 0.8;
    all += p->chunks[s] * cost[s];
  }
  const int groups = groups_in_flight(mode, es, p->few);
  for (int s = 0; s < 2; ++s) {
    tokens[s] = p->tpw[s] ? groups * p->tpw[s] : 1;
    if (tokens[s] > p->batch) p->batch = tokens[s];
    int64_t n = (int64_t)(total * cost[s] / all);  // rounded down: one wave, not a CTA more
    const int64_t most = (T + kWarps * tokens[s] - 1) / (kWarps * tokens[s]);
    if (n > most) n = most;
    p->ctas[s] = (int)(n < 1 ? 1 : n);
  }
  return cudaSuccess;
}

int64_t slots_of(const Plan& p, int side) { return (int64_t)p.chunks[side] * p.ctas[side]; }
size_t dw_bytes(const Plan& p, int dh) {
  return (size_t)(slots_of(p, 0) + slots_of(p, 1)) * dh * sizeof(float);
}

int check_common(int64_t T, int32_t hq, int32_t hk, int32_t dh, adaln_dtype_t dt) {
  if (dt != ADALN_F32 && dt != ADALN_BF16) return ADALN_ERR_DTYPE;
  if (T < 0 || T > (int64_t)INT32_MAX) return ADALN_ERR_DIM;
  if (hq < 0 || hk < 0 || hq + (int64_t)hk < 1 || hq > ADALN_MAX_HEADS || hk > ADALN_MAX_HEADS)
    return ADALN_ERR_DIM;
  if (dh < 1 || dh > ADALN_MAX_HEAD_DIM) return ADALN_ERR_DIM;
  return ADALN_OK;
}

int check_rope(const adaln_rope_t* r, int32_t dh, int64_t T) {
  if (!r) return ADALN_ERR_NULL;
  if (r->axes < 1 || r->axes > ADALN_MAX_ROPE_AXES || r->rows < 1) return ADALN_ERR_DIM;
  int64_t pairs = 0;
  for (int i = 0; i < r->axes; ++i) {
    if (r->pairs[i] < 0) return ADALN_ERR_DIM;
    pairs += r->pairs[i];
  }
  if (pairs < 1 || 2 * pairs > dh) return ADALN_ERR_DIM;
  if (T > 0 && (!r->table || !r->pos)) return ADALN_ERR_NULL;
  if (!aligned_to(r->table, 8) || !aligned_to(r->pos, 4)) return ADALN_ERR_ALIGN;
  return ADALN_OK;
}

// A tensor's pointer and strides, and whether vectors of *width words fit them
// (else *width = 0).
int check_heads(const adaln_heads_t* h, int heads, int64_t T, int es, int* width) {
  if (heads == 0) return ADALN_OK;
  if (!h) return ADALN_ERR_NULL;
  if (T > 0 && !h->ptr) return ADALN_ERR_NULL;
  if (h->token_stride < 0 || h->head_stride < 0) return ADALN_ERR_DIM;
  if (!aligned_to(h->ptr, es)) return ADALN_ERR_ALIGN;
  const int bytes = 4 * *width;
  if (bytes && (!aligned_to(h->ptr, bytes) || h->token_stride * es % bytes != 0 ||
                h->head_stride * es % bytes != 0))
    *width = 0;
  return ADALN_OK;
}

// Whether no two of [T, heads] rows of dh elements meet: neither neighbours along
// one axis nor, where one axis's rows do not lie wholly between two of the other's,
// any (t, h) and (t', h').  Those meet if t' - t and h - h' of the same sign bring
// the two offsets within dh of each other, so for each distance in heads the
// tokens on either side of it are looked at.
bool rows_apart(int64_t T, int64_t ts, int heads, int64_t hs, int dh) {
  if (T > 1 && ts < dh) return false;
  if (heads > 1 && hs < dh) return false;
  if (T <= 1 || heads <= 1) return true;
  typedef __int128 wide;  // strides are the caller's: their products may pass 64 bits
  if (ts >= (wide)(heads - 1) * hs + dh || hs >= (wide)(T - 1) * ts + dh) return true;
  for (int j = 1; j < heads; ++j) {
    const wide far = (wide)j * hs, i = far / ts;
    if (i < T && far - i * ts < dh) return false;
    if (i + 1 < T && (i + 1) * ts - far < dh) return false;
  }
  return true;
}

// An output's: its rows may not overlap each other.
int check_out(const adaln_heads_t* h, int heads, int64_t T, int dh, int es, int* width) {
  const int rc = check_heads(h, heads, T, es, width);
  if (rc != ADALN_OK || heads == 0 || T == 0) return rc;
  return rows_apart(T, h->token_stride, heads, h->head_stride, dh) ? ADALN_OK : ADALN_ERR_DIM;
}

Tensor tensor_of(const adaln_heads_t* h, int es) {
  if (!h) return Tensor{nullptr, 0, 0};
  return Tensor{static_cast<const char*>(h->ptr), h->token_stride * es, h->head_stride * es};
}

// Words of the vectors that suit the head's layout (its pointers aside), 0 for
// the scalar path: 16 bytes, or for halves of a number of elements that is no
// multiple of theirs 8 or 4.
int width_of(int dh, int es, int pairs, bool half) {
  for (int w = 4; w >= (es == 2 ? 1 : 2); w /= 2) {
    const int bytes = 4 * w;
    if (dh * es % bytes == 0 && dh * es / bytes <= 64 && (!half || pairs * es % bytes == 0)) return w;
    if (!half) break;
  }
  return 0;
}

int run(int mode, const adaln_heads_t* const (&x)[2], const adaln_heads_t* const (&dy)[2],
        const adaln_heads_t* const (&out)[2], int64_t T, const int (&heads)[2], int32_t dh,
        adaln_dtype_t dtype, const adaln_rope_t* rope, const void* const (&w)[2], float eps,
        float* const (&dw)[2], void* workspace, size_t workspace_bytes, int width,
        cudaStream_t st) {
  const int es = dtype == ADALN_BF16 ? 2 : 4;
  RopeArgs a = {};
  for (int i = 0, at = 0; i < 4; ++i) {
    if (i < rope->axes) at += rope->pairs[i];
    a.axis_end[i] = at;
    a.P = at;
  }
  Plan p;
  cudaError_t e = make_plan(T, heads, dh, mode, width, es, &p);
  unsigned* status = nullptr;
  if (e == cudaSuccess) e = status_word(&status);
  if (e != cudaSuccess) return launch_failed(e);
  const bool want_dw = mode == kNormBwd && (dw[0] || dw[1]);
  if (want_dw && workspace_bytes < dw_bytes(p, dh)) return ADALN_ERR_WORKSPACE;

  float* partial = want_dw ? static_cast<float*>(workspace) : nullptr;
  for (int s = 0; s < 2; ++s) {
    Side& sd = a.side[s];
    sd.x = tensor_of(x[s], es);
    sd.dy = tensor_of(dy[s], es);
    const Tensor o = tensor_of(out[s], es);
    sd.out = const_cast<char*>(o.p);
    sd.out_ts = o.ts;
    sd.out_hs = o.hs;
    sd.w = w[s];
    sd.heads = heads[s];
    sd.chunks = p.chunks[s];
    sd.per_chunk = p.per_chunk[s];
    sd.ctas = p.ctas[s];
    sd.tpw = p.tpw[s];
    sd.partial = partial && dw[s] ? partial + (s ? slots_of(p, 0) : 0) * dh : nullptr;
  }
  a.table = reinterpret_cast<const float2*>(rope->table);
  a.pos = rope->pos;
  a.T = T;
  a.rows = rope->rows;
  a.axes = rope->axes;
  a.dh = dh;
  a.nvec = p.width ? dh * es / (4 * p.width) : 0;
  a.batch = p.batch;
  a.eps = eps;
  a.inv_dh = 1.0f / (float)dh;
  a.status = status;

  const bool half = !rope->interleaved;
  int interleaved = rope->interleaved != 0;
  void* kernel;
  size_t smem = mode == kNormBwd ? (size_t)kWarps * dh * sizeof(float) : 0;
  if (p.width) {
    kernel = pick_kernel(es, p.width, p.lanes, half, p.few, mode);
    const size_t table = (size_t)(4 * p.width / es / 2) * ((a.nvec + 1) / 2) * sizeof(float4);
    const size_t tables =
        table * (2 * kWarps * p.batch + (mode == kNormFwd || mode == kNormBwd ? 1 : 0));
    smem = tables > smem ? tables : smem;
    if (smem > 48 * 1024) {
      // The same value by every call: calls of other sizes that share the kernel
      // may set it between this line and the launch (another thread's).
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared);
      if (e != cudaSuccess) return launch_failed(e);
    }
  } else if (dh <= 128) {
    kernel = dtype == ADALN_BF16 ? scalar_kernel<BF16, 2>(mode) : scalar_kernel<F32, 2>(mode);
  } else {
    kernel = dtype == ADALN_BF16 ? scalar_kernel<BF16, 8>(mode) : scalar_kernel<F32, 8>(mode);
  }
  void* params[2] = {&a, &interleaved};
  const dim3 grid((unsigned)(slots_of(p, 0) + slots_of(p, 1)));
  if (T > 0) {
    e = traced_launch(ADALN_KERNEL_QK_ROPE, st,
                      [&] { return launch(kernel, grid, kThreads, smem, params, st); });
    if (e != cudaSuccess) return launch_failed(e);
  }
  if (want_dw) {
    const float* pq = a.side[0].partial;
    const float* pk = a.side[1].partial;
    // No tokens (or no heads): the sums are empty.
    int nq = T > 0 ? (int)slots_of(p, 0) : 0, nk = T > 0 ? (int)slots_of(p, 1) : 0;
    float *dwq = dw[0], *dwk = dw[1];
    int d = dh;
    void* params2[7] = {&pq, &nq, &dwq, &pk, &nk, &dwk, &d};
    e = traced_launch(ADALN_KERNEL_QK_ROPE, st, [&] {
      return launch((void*)rope_dw_kernel, dim3((unsigned)(dh + 31) / 32, 2), 1024, 0, params2,
                    st);
    });
    if (e != cudaSuccess) return launch_failed(e);
  }
  return ADALN_OK;
}

}  // namespace
}  // namespace adaln

using namespace adaln;

extern "C" {

int adaln_qk_rope_fwd(const adaln_heads_t* q, const adaln_heads_t* k, int64_t T, int32_t hq,
                      int32_t hk, int32_t dh, adaln_dtype_t dtype, const adaln_rope_t* rope,
                      int32_t norm, const void* wq, const void* wk, float eps,
                      const adaln_heads_t* q_out, const adaln_heads_t* k_out, void* stream) {
  int rc = check_common(T, hq, hk, dh, dtype);
  if (rc == ADALN_OK) rc = check_rope(rope, dh, T);
  if (rc != ADALN_OK) return rc;
  const int es = dtype == ADALN_BF16 ? 2 : 4;
  int pairs = 0;
  for (int i = 0; i < rope->axes; ++i) pairs += rope->pairs[i];
  int width = width_of(dh, es, pairs, !rope->interleaved);
  if ((rc = check_heads(q, hq, T, es, &width)) || (rc = check_heads(k, hk, T, es, &width)) ||
      (rc = check_out(q_out, hq, T, dh, es, &width)) || (rc = check_out(k_out, hk, T, dh, es, &width)))
    return rc;
  if (norm) {
    if (!std::isfinite(eps) || eps < 0.0f) return ADALN_ERR_ARG;
    if (!aligned_to(wq, es) || !aligned_to(wk, es)) return ADALN_ERR_ALIGN;
  }
  if (T == 0) return ADALN_OK;
  return run(norm ? kNormFwd : kRotate, {q, k}, {nullptr, nullptr}, {q_out, k_out}, T, {hq, hk},
             dh, dtype, rope, {wq, wk}, eps, {nullptr, nullptr}, nullptr, 0, width,
             static_cast<cudaStream_t>(stream));
}

int adaln_qk_rope_bwd_workspace_size(int64_t T, int32_t hq, int32_t hk, int32_t dh,
                                     adaln_dtype_t dtype, size_t* bytes) {
  const int rc = check_common(T, hq, hk, dh, dtype);
  if (rc != ADALN_OK) return rc;
  if (!bytes) return ADALN_ERR_NULL;
  // The largest need of the paths that may run (which one depends on the pairs
  // and on alignment).
  const int es = dtype == ADALN_BF16 ? 2 : 4;
  size_t most = 0;
  for (int width = 0; width <= 4; width = width ? 2 * width : 1) {
    if (width && (dh * es % (4 * width) != 0 || dh * es / (4 * width) > 64)) continue;
    Plan p;
    const cudaError_t e = make_plan(T, {hq, hk}, dh, kNormBwd, width, es, &p);
    if (e != cudaSuccess) return launch_failed(e);
    const size_t need = (dw_bytes(p, dh) + 255) & ~(size_t)255;
    most = need > most ? need : most;
  }
  *bytes = most;
  return ADALN_OK;
}

int adaln_qk_rope_bwd(const adaln_heads_t* dq_out, const adaln_heads_t* dk_out,
                      const adaln_heads_t* q, const adaln_heads_t* k, int64_t T, int32_t hq,
                      int32_t hk, int32_t dh, adaln_dtype_t dtype, const adaln_rope_t* rope,
                      int32_t norm, const void* wq, const void* wk, float eps,
                      const adaln_heads_t* dq, const adaln_heads_t* dk, float* dwq, float* dwk,
                      void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_common(T, hq, hk, dh, dtype);
  if (rc == ADALN_OK) rc = check_rope(rope, dh, T);
  if (rc != ADALN_OK) return rc;
  const int es = dtype == ADALN_BF16 ? 2 : 4;
  int pairs = 0;
  for (int i = 0; i < rope->axes; ++i) pairs += rope->pairs[i];
  int width = width_of(dh, es, pairs, !rope->interleaved);
  if ((rc = check_heads(dq_out, hq, T, es, &width)) || (rc = check_heads(dk_out, hk, T, es, &width)) ||
      (rc = check_out(dq, hq, T, dh, es, &width)) || (rc = check_out(dk, hk, T, dh, es, &width)))
    return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!norm) {
    // The rotation's transpose is the rotation by the opposite angle.
    if (dwq || dwk) return ADALN_ERR_ARG;
    if (T == 0) return ADALN_OK;
    return run(kRotateBack, {dq_out, dk_out}, {nullptr, nullptr}, {dq, dk}, T, {hq, hk}, dh,
               dtype, rope, {nullptr, nullptr}, 0.0f, {nullptr, nullptr}, nullptr, 0, width, st);
  }
  if ((rc = check_heads(q, hq, T, es, &width)) || (rc = check_heads(k, hk, T, es, &width))) return rc;
  if (!std::isfinite(eps) || eps < 0.0f) return ADALN_ERR_ARG;
  if (!aligned_to(wq, es) || !aligned_to(wk, es) || !aligned_to(dwq, 4) || !aligned_to(dwk, 4))
    return ADALN_ERR_ALIGN;
  if ((dwq || dwk) && !workspace) return ADALN_ERR_NULL;
  if (!aligned_to(workspace, 16)) return ADALN_ERR_ALIGN;
  if (T == 0 && !dwq && !dwk) return ADALN_OK;
  return run(kNormBwd, {q, k}, {dq_out, dk_out}, {dq, dk}, T, {hq, hk}, dh, dtype, rope, {wq, wk},
             eps, {dwq, dwk}, workspace, workspace_bytes, width, st);
}

}  // extern "C"
