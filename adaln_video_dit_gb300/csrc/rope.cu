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
// T = 36864 x 48 heads x 128, bf16, 135.1 us, 99 %; norm and rotation of T = 32760
// x 80 heads x 128 read out of a packed projection 207.9 us, 95 %; forward and
// backward of T = 16384 x 48 heads, 128 wide bf16 172.7 us, 86 %, 80 wide 70 %
// (bf16) and 92 % (fp32).  A call on one token takes 2.6 us of the GPU.
//
// Layout of the work: P lanes share a head, each holding two 16-byte vectors
// of it that contain whole pairs (interleaved: vectors j and j + half, halves:
// a vector and its partner), so a rotation never leaves its lane and a norm
// takes about log2(P) shuffles (P need not be a power of two: heads of 80 bf16
// elements take 5 lanes, six heads to a warp).  A warp walks tokens, and of each token the heads of
// its chunk, U groups of 32 / P heads at a time with the next ones on their
// way.  A token's cosines and sines and the weights are read from shared
// memory, where the lanes of different heads read the same words: in registers
// they would cost half of what a thread has, and with it the loads in flight.
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace adaln {
namespace {

constexpr int kWarps = 8;  // warps of a CTA
constexpr int kThreads = kWarps * 32;
constexpr int kCtasPerSm = 2;
// Elements of a head that the scalar path's 32 lanes hold (8 pairs a lane).
constexpr int kScalarPairs = 8;

enum { kRotate = 0, kRotateBack = 1, kNormFwd = 2, kNormBwd = 3 };

struct Tensor {
  const char* p;
  int64_t ts, hs;  // bytes from token to token, head to head
};

struct Side {  // queries or keys
  Tensor x;    // forward input (kRotate, kRotateBack: what is turned)
  Tensor dy;   // kNormBwd only
  char* out;
  int64_t out_ts, out_hs;
  const void* w;   // [dh] norm weight, or nullptr: ones
  float* partial;  // kNormBwd: [chunks * gridDim.x][dh], or nullptr: no dw
  int heads;
  int chunks;      // the heads are split into this many chunks
  int per_chunk;   // heads of a chunk
};

struct RopeArgs {
  Side side[2];
  const float2* table;  // [rows][P]
  const int32_t* pos;   // [T][axes]
  int64_t T;
  int rows, axes, P, dh, nvec;
  int axis_end[4];  // pairs [axis_end[a-1], axis_end[a]) belong to axis a
  float eps, inv_dh;
  unsigned* status;
};

// Axis of pair p, or 4 for an unrotated one.
__device__ __forceinline__ int axis_of(const RopeArgs& a, int p) {
  return (p >= a.axis_end[0]) + (p >= a.axis_end[1]) + (p >= a.axis_end[2]) + (p >= a.axis_end[3]);
}

// Table rows of a token's axes, -1 where the axis does not turn the token.
// A position outside [-1, rows) is recorded and does not turn it either.
struct Rows {
  int r[4];
  __device__ __forceinline__ void load(const RopeArgs& a, int64_t t, int lane) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r[i] = -1;
      if (i < a.axes) {
        const int p = a.pos[t * a.axes + i];
        if (p >= 0 && p < a.rows) r[i] = p;
        bad |= p < -1 || p >= a.rows;
      }
    }
    if (bad && lane == 0) atomicOr(a.status, ADALN_DEV_POS_RANGE);
  }
  __device__ __forceinline__ float2 at(const RopeArgs& a, int axis, int p) const {
    const int row = axis == 0 ? r[0] : axis == 1 ? r[1] : axis == 2 ? r[2] : axis == 3 ? r[3] : -1;
    if (row < 0) return make_float2(1.0f, 0.0f);
    return __ldg(a.table + (int64_t)row * a.P + p);
  }
};

// (u, v) turned by (c, s), or back.  A pair with a zero sine takes nothing from
// its partner, so an unrotated element passes exactly, whatever the other holds.
template <bool BACK>
__device__ __forceinline__ void turn(float& u, float& v, float c, float s) {
  const float a = u, b = v;
  const float bs = s == 0.0f ? 0.0f : b * s, as = s == 0.0f ? 0.0f : a * s;
  u = fmaf(a, c, BACK ? bs : -bs);
  v = fmaf(b, c, BACK ? -as : as);
}

// Sum over the CTA's warps of red[warp][0..dh), in warp order, into slot.
__device__ __forceinline__ void store_partial(const float* red, float* slot, int dh) {
  __syncthreads();
  for (int d = threadIdx.x; d < dh; d += kThreads) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += red[w * dh + d];
    slot[d] = s;
  }
}

// (volatile: read where it is used, not kept in registers meanwhile)
__device__ __forceinline__ float4 ld_shared_f4(const float4* p) {
  const uint4 v = ld_shared_v4(smem_addr(p));
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                     __uint_as_float(v.w));
}
__device__ __forceinline__ void cp_async4(float* dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// A lane's two vectors as N pairs, split: the first elements of pairs 2 i and
// 2 i + 1 in A[i], the second ones in B[i], so that two pairs turn in packed
// arithmetic.  Interleaved pairs are neighbours in a vector (vector a's, then
// b's); those of the halves layout are the same element of a and of b.
template <bool HALF>
__device__ __forceinline__ void split(const uint4& a, const uint4& b, float2 (&A)[4], float2 (&B)[4],
                                      BF16) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  auto lo = [&](int i) { return __uint_as_float(w[i] << 16); };
  auto hi = [&](int i) { return __uint_as_float(w[i] & 0xffff0000u); };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    A[i] = HALF ? make_float2(lo(i), hi(i)) : make_float2(lo(2 * i), lo(2 * i + 1));
    B[i] = HALF ? make_float2(lo(4 + i), hi(4 + i)) : make_float2(hi(2 * i), hi(2 * i + 1));
  }
}
template <bool HALF>
__device__ __forceinline__ void split(const uint4& a, const uint4& b, float2 (&A)[2], float2 (&B)[2],
                                      F32) {
  const float f[8] = {__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z),
                      __uint_as_float(a.w), __uint_as_float(b.x), __uint_as_float(b.y),
                      __uint_as_float(b.z), __uint_as_float(b.w)};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    A[i] = HALF ? make_float2(f[2 * i], f[2 * i + 1]) : make_float2(f[4 * i], f[4 * i + 2]);
    B[i] = HALF ? make_float2(f[4 + 2 * i], f[5 + 2 * i]) : make_float2(f[4 * i + 1], f[4 * i + 3]);
  }
}
// And back, rounded to the element type.
template <bool HALF>
__device__ __forceinline__ void join(const float2 (&A)[4], const float2 (&B)[4], uint4& a, uint4& b,
                                     BF16) {
  float2 f[4], g[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = HALF ? A[i] : i % 2 ? make_float2(A[i / 2].y, B[i / 2].y) : make_float2(A[i / 2].x, B[i / 2].x);
    g[i] = HALF    ? B[i]
           : i % 2 ? make_float2(A[2 + i / 2].y, B[2 + i / 2].y)
                   : make_float2(A[2 + i / 2].x, B[2 + i / 2].x);
  }
  a = BF16::pack2(f);
  b = BF16::pack2(g);
}
template <bool HALF>
__device__ __forceinline__ void join(const float2 (&A)[2], const float2 (&B)[2], uint4& a, uint4& b,
                                     F32) {
  float2 f[2], g[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[i] = HALF ? A[i] : i ? make_float2(A[0].y, B[0].y) : make_float2(A[0].x, B[0].x);
    g[i] = HALF ? B[i] : i ? make_float2(A[1].y, B[1].y) : make_float2(A[1].x, B[1].x);
  }
  a = F32::pack2(f);
  b = F32::pack2(g);
}

// Sum over the P lanes of a head, in each of them.
template <int P>
__device__ __forceinline__ float head_sum(float v, int lane, int j) {
  if constexpr ((P & (P - 1)) == 0) {
#pragma unroll
    for (int o = P / 2; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
  } else {  // pairwise towards the head's first lane, and back from it
#pragma unroll
    for (int o = P > 8 ? 8 : 4; o > 0; o >>= 1) {
      const float w = __shfl_sync(~0u, v, (lane + o) & 31);
      if (j + o < P) v += w;
    }
    return __shfl_sync(~0u, v, lane - j);
  }
}

// Vector path: head rows of whole, aligned 16-byte vectors, at most 64.
// P lanes a head, U groups of 32 / P heads in flight.
template <class E, int P, bool HALF, int MODE, int U>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    rope_vec_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int N = E::EPV;    // elements of a vector, pairs of a lane
  constexpr int M = N / 2;     // packed pairs of pairs of a lane
  constexpr int HPW = 32 / P;  // heads side by side in a warp
  constexpr bool kNorm = MODE == kNormFwd || MODE == kNormBwd;
  constexpr bool kGrad = MODE == kNormBwd;
  constexpr bool kBack = MODE == kRotateBack || MODE == kNormBwd;
  // Tables of [M][half] float4: lane j's i-th entry holds, for its pairs 2 i
  // and 2 i + 1, two cosines and two sines, or the two weights of A and of B;
  // neighbouring lanes' entries are neighbours, so a read has no bank conflict.
  // The weights' table, then two of angles (this token's, the next's) per warp.
  // After the walk the norm's backward puts [kWarps][dh] weight sums there.
  extern __shared__ __align__(16) float4 shared[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = (a.nvec + 1) >> 1, entries = M * half;
  float4* const weights = shared;
  float4* const angles = shared + (kNorm ? entries : 0) + warp * 2 * entries;
  const int j = lane % P, sub = lane / P;  // (sub = HPW: lanes left over)
  const bool is_k = (int)blockIdx.y >= a.side[0].chunks;
  const Side& sd = a.side[is_k];
  const int chunk = is_k ? blockIdx.y - a.side[0].chunks : blockIdx.y;
  const int h_begin = chunk * sd.per_chunk, h_end = min(sd.heads, h_begin + sd.per_chunk);

  // This lane's two vectors (-1: none).
  const int nr = a.P / N;  // halves: vectors of the first half
  int va = HALF && j >= nr ? 2 * nr + 2 * (j - nr) : j;
  int vb = HALF ? (j < nr ? j + nr : va + 1) : j + half;
  if (va >= a.nvec || j >= half || sub >= HPW) va = -1;
  if (vb >= a.nvec || j >= half || sub >= HPW) vb = -1;
  const int jj = min(j, half - 1);
  // Lane and pair of the lane that pair p of the head is, as a float's index
  // into a table (its partner word two further on).
  auto entry = [&](int jl, int e) { return ((e >> 1) * half + jl) * 4 + (e & 1); };
  auto entry_of_pair = [&](int p) {
    if (HALF) return entry(p / N, p % N);
    const int v = p / M, q = p % M;
    return v < half ? entry(v, q) : entry(v - half, q + M);
  };

  grid_wait();
  grid_launch_dependents();

  // The angles of a token into table b, from its rows.
  auto fetch_angles = [&](const Rows& rows, int b) {
    float* const to = reinterpret_cast<float*>(angles + b * entries);
    for (int p = lane; p < a.P; p += 32) {
      const int axis = axis_of(a, p);
      const int row = axis == 0 ? rows.r[0] : axis == 1 ? rows.r[1] : axis == 2 ? rows.r[2] : rows.r[3];
      float* const at = to + entry_of_pair(p);
      if (row >= 0) {
        const float* from = reinterpret_cast<const float*>(a.table + (int64_t)row * a.P + p);
        cp_async4(at, from);
        cp_async4(at + 2, from + 1);
      } else {
        at[0] = 1.0f;
        at[2] = 0.0f;
      }
    }
  };
  // Whether some pair of the token has a zero sine: only then is each looked
  // at (turn() below), else two pairs turn in four packed operations.
  const bool partial = 2 * a.P < a.dh;
  auto any_still = [&](int b) {
    const float* const from = reinterpret_cast<const float*>(angles + b * entries);
    bool z = partial;
    for (int p = lane; p < a.P; p += 32) z |= from[entry_of_pair(p) + 2] == 0.0f;
    return (bool)__any_sync(~0u, z);
  };

  struct Group {
    uint4 xa[U], xb[U], ya[kGrad ? U : 1], yb[kGrad ? U : 1];
  };
  auto load = [&](Group& g, int64_t t, int h0) {
    const char* x = sd.x.p + t * sd.x.ts + (h0 + sub) * sd.x.hs;
    const char* y = kGrad ? sd.dy.p + t * sd.dy.ts + (h0 + sub) * sd.dy.hs : nullptr;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool on = h0 + u * HPW + sub < h_end && t < a.T;
      g.xa[u] = on && va >= 0 ? ld_global_v4(x + va * 16) : make_uint4(0, 0, 0, 0);
      g.xb[u] = on && vb >= 0 ? ld_global_v4(x + vb * 16) : make_uint4(0, 0, 0, 0);
      x += HPW * sd.x.hs;
      if (kGrad) {
        g.ya[u] = on && va >= 0 ? ld_global_v4(y + va * 16) : make_uint4(0, 0, 0, 0);
        g.yb[u] = on && vb >= 0 ? ld_global_v4(y + vb * 16) : make_uint4(0, 0, 0, 0);
        y += HPW * sd.dy.hs;
      }
    }
  };
  auto rotate = [&](float2(&A)[M], float2(&B)[M], const float4* cs, bool still) {
#pragma unroll
    for (int i = 0; i < M; ++i) {
      const float4 t = ld_shared_f4(cs + i * half + jj);
      if (still) {
        turn<kBack>(A[i].x, B[i].x, t.x, t.z);
        turn<kBack>(A[i].y, B[i].y, t.y, t.w);
      } else {
        const float2 c = make_float2(t.x, t.y);
        const float2 s = kBack ? make_float2(-t.z, -t.w) : make_float2(t.z, t.w);
        const float2 bs = mul2(B[i], make_float2(-s.x, -s.y)), as = mul2(A[i], s);
        A[i] = fma2(A[i], c, bs);
        B[i] = fma2(B[i], c, as);
      }
    }
  };

  float2 dwa[kGrad ? M : 1], dwb[kGrad ? M : 1];
  if (kGrad) {
#pragma unroll
    for (int i = 0; i < M; ++i) dwa[i] = dwb[i] = make_float2(0.0f, 0.0f);
  }

  const int64_t step = (int64_t)gridDim.x * kWarps;
  int64_t t = (int64_t)blockIdx.x * kWarps + warp;
  Group cur;
  load(cur, t, h_begin);
  Rows rows;  // of the token after the one whose angles are on their way
  if (t < a.T) rows.load(a, t, lane);
  if (kNorm) {
    for (int i = threadIdx.x; i < entries; i += kThreads)
      weights[i] = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    if (sd.w != nullptr) {
      __syncthreads();
      for (int d = threadIdx.x; d < a.dh; d += kThreads) {
        int at;
        if (!HALF)
          at = entry_of_pair(d >> 1) + 2 * (d & 1);
        else if (d < 2 * a.P)
          at = entry_of_pair(d < a.P ? d : d - a.P) + (d < a.P ? 0 : 2);
        else
          at = entry(nr + (d / N - 2 * nr) / 2, d % N) + (d / N - 2 * nr) % 2 * 2;
        reinterpret_cast<float*>(weights)[at] =
            E::SIZE == 2 ? __bfloat162float(static_cast<const __nv_bfloat16*>(sd.w)[d])
                         : static_cast<const float*>(sd.w)[d];
      }
    }
  }
  for (int i = lane; i < 2 * entries; i += 32) angles[i] = make_float4(1.0f, 1.0f, 0.0f, 0.0f);
  __syncthreads();
  if (t < a.T) {
    fetch_angles(rows, 0);
    if (t + step < a.T) rows.load(a, t + step, lane);
  }
  for (int slot = 0; t < a.T; t += step, slot ^= 1) {
    cp_async_wait();
    __syncwarp();
    const bool still = any_still(slot);
    if (t + step < a.T) {
      fetch_angles(rows, slot ^ 1);
      if (t + 2 * step < a.T) rows.load(a, t + 2 * step, lane);
    }
    const float4* cs = angles + slot * entries;

    for (int h0 = h_begin; h0 < h_end; h0 += U * HPW) {
      Group next;
      const bool more = h0 + U * HPW < h_end;
      load(next, more ? t : t + step, more ? h0 + U * HPW : h_begin);
      char* out = sd.out + t * sd.out_ts + (h0 + sub) * sd.out_hs;
#pragma unroll
      for (int u = 0; u < U; ++u, out += HPW * sd.out_hs) {
        if (h0 + u * HPW >= h_end) break;
        const bool on = h0 + u * HPW + sub < h_end;
        float2 A[M], B[M];
        split<HALF>(cur.xa[u], cur.xb[u], A, B, E());
        if (!kNorm) {
          rotate(A, B, cs, still);
        } else {
          float2 ss = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int i = 0; i < M; ++i) ss = fma2(A[i], A[i], fma2(B[i], B[i], ss));
          float sx = ss.x + ss.y;
          if (!kGrad) {
            // The rotation is linear: the weights before it, r after it, so
            // that it does not wait for the sum.
#pragma unroll
            for (int i = 0; i < M; ++i) {
              const float4 w = ld_shared_f4(weights + i * half + jj);
              A[i] = mul2(A[i], make_float2(w.x, w.y));
              B[i] = mul2(B[i], make_float2(w.z, w.w));
            }
            rotate(A, B, cs, still);
            sx = head_sum<P>(sx, lane, j);
            const float2 r = splat2(rsqrtf(fmaf(sx, a.inv_dh, a.eps)));
#pragma unroll
            for (int i = 0; i < M; ++i) {
              A[i] = mul2(A[i], r);
              B[i] = mul2(B[i], r);
            }
          } else {
            float2 GA[M], GB[M];
            split<HALF>(cur.ya[u], cur.yb[u], GA, GB, E());
            rotate(GA, GB, cs, still);
            float2 hs = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < M; ++i) {
              const float4 w = ld_shared_f4(weights + i * half + jj);
              hs = fma2(mul2(GA[i], make_float2(w.x, w.y)), A[i], hs);
              hs = fma2(mul2(GB[i], make_float2(w.z, w.w)), B[i], hs);
            }
            float sh = hs.x + hs.y;
            sx = head_sum<P>(sx, lane, j);
            sh = head_sum<P>(sh, lane, j);
            const float r = rsqrtf(fmaf(sx, a.inv_dh, a.eps));
            const float2 k = splat2(-r * r * r * (sh * a.inv_dh)), r2 = splat2(r);
            // Lanes past the last head hold zeros, so they add nothing to dw
            // (g = 0) as long as r is finite; eps = 0 would make it 0 * inf.
            const float2 rd = splat2(on ? r : 0.0f);
#pragma unroll
            for (int i = 0; i < M; ++i) {
              const float4 w = ld_shared_f4(weights + i * half + jj);
              dwa[i] = fma2(GA[i], mul2(A[i], rd), dwa[i]);
              dwb[i] = fma2(GB[i], mul2(B[i], rd), dwb[i]);
              A[i] = fma2(A[i], k, mul2(mul2(GA[i], make_float2(w.x, w.y)), r2));
              B[i] = fma2(B[i], k, mul2(mul2(GB[i], make_float2(w.z, w.w)), r2));
            }
          }
        }
        if (on) {
          uint4 oa, ob;
          join<HALF>(A, B, oa, ob, E());
          if (va >= 0) *reinterpret_cast<uint4*>(out + va * 16) = oa;
          if (vb >= 0) *reinterpret_cast<uint4*>(out + vb * 16) = ob;
        }
      }
      cur = next;
    }
  }

  if (kGrad && sd.partial != nullptr) {
    __syncthreads();  // the tables' place is reused
    float* const red = reinterpret_cast<float*>(shared);
    // Lanes of the same j hold the same columns: their sums, in order, in sub 0.
    auto over_heads = [&](float v) {
      float t = v;
#pragma unroll
      for (int k = 1; k < HPW; ++k) t += __shfl_sync(~0u, v, (j + k * P) & 31);
      return t;
    };
#pragma unroll
    for (int i = 0; i < M; ++i) {
      dwa[i] = make_float2(over_heads(dwa[i].x), over_heads(dwa[i].y));
      dwb[i] = make_float2(over_heads(dwb[i].x), over_heads(dwb[i].y));
      if (sub == 0) {
        float* const to = red + warp * a.dh;
        if (HALF) {
          if (va >= 0) to[va * N + 2 * i] = dwa[i].x, to[va * N + 2 * i + 1] = dwa[i].y;
          if (vb >= 0) to[vb * N + 2 * i] = dwb[i].x, to[vb * N + 2 * i + 1] = dwb[i].y;
        } else {
          const int v = i < M / 2 ? va : vb, e = 4 * (i < M / 2 ? i : i - M / 2);
          if (v >= 0) {
            to[v * N + e] = dwa[i].x, to[v * N + e + 1] = dwb[i].x;
            to[v * N + e + 2] = dwa[i].y, to[v * N + e + 3] = dwb[i].y;
          }
        }
      }
    }
    store_partial(red, sd.partial + ((int64_t)chunk * gridDim.x + blockIdx.x) * a.dh, a.dh);
  }
}

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

// Scalar path: any head width up to 512, any strides, element alignment.  A
// warp holds one head, lane l the pairs l, l + 32, ...; pairs from P on are
// the unrotated elements, two by two.
template <class E, int MODE>
__global__ void __launch_bounds__(kThreads) rope_scalar_kernel(const __grid_constant__ RopeArgs a,
                                                               int interleaved) {
  constexpr bool kNorm = MODE == kNormFwd || MODE == kNormBwd;
  extern __shared__ float red[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool is_k = (int)blockIdx.y >= a.side[0].chunks;
  const Side& sd = a.side[is_k];
  const int chunk = is_k ? blockIdx.y - a.side[0].chunks : blockIdx.y;
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

  const int64_t step = (int64_t)gridDim.x * kWarps;
  for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < a.T; t += step) {
    Rows rows;
    rows.load(a, t, lane);
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
        const float k = -r * r * r * (sh * a.inv_dh);
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
    store_partial(red, sd.partial + ((int64_t)chunk * gridDim.x + blockIdx.x) * a.dh, a.dh);
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

// Head groups in flight: what fits 128 registers a thread.  Forward and plain
// rotation, T = 32760 x 80 heads x 128: three groups 205.9 us, four (spilling
// with the norm) 226.5, two 206.9 (T = 36864 x 48 heads, rotation alone: 134.9,
// 135.2 and 144.4).  The norm's backward holds twice the tensors and its weight
// sums: with two groups of bf16 heads it spilled, and 8192 tokens x 24 heads x
// 128 took 41.0 instead of 30.6 us.
constexpr int groups_in_flight(int mode, int es) { return mode != kNormBwd ? 3 : es == 2 ? 1 : 2; }

template <class E, int P, bool HALF>
void* vec_kernel(int mode) {
  switch (mode) {
    case kRotate: return (void*)rope_vec_kernel<E, P, HALF, kRotate, groups_in_flight(kRotate, E::SIZE)>;
    case kRotateBack: return (void*)rope_vec_kernel<E, P, HALF, kRotateBack, groups_in_flight(kRotateBack, E::SIZE)>;
    case kNormFwd: return (void*)rope_vec_kernel<E, P, HALF, kNormFwd, groups_in_flight(kNormFwd, E::SIZE)>;
    default: return (void*)rope_vec_kernel<E, P, HALF, kNormBwd, groups_in_flight(kNormBwd, E::SIZE)>;
  }
}

template <class E, bool HALF>
void* pick_kernel(int lanes, int mode) {
  switch (lanes) {
    case 4: return vec_kernel<E, 4, HALF>(mode);
    case 5: return vec_kernel<E, 5, HALF>(mode);
    case 6: return vec_kernel<E, 6, HALF>(mode);
    case 8: return vec_kernel<E, 8, HALF>(mode);
    case 10: return vec_kernel<E, 10, HALF>(mode);
    case 16: return vec_kernel<E, 16, HALF>(mode);
    default: return vec_kernel<E, 32, HALF>(mode);
  }
}
// Lanes of a head of which `want` hold data: each count that puts one more head
// into a warp than the next.
int lanes_of(int want) {
  return want <= 4    ? 4
         : want <= 6  ? want
         : want <= 8  ? 8
         : want <= 10 ? 10
         : want <= 16 ? 16
                      : 32;
}

template <class E>
void* scalar_kernel(int mode) {
  return mode == kRotate       ? (void*)rope_scalar_kernel<E, kRotate>
         : mode == kRotateBack ? (void*)rope_scalar_kernel<E, kRotateBack>
         : mode == kNormFwd    ? (void*)rope_scalar_kernel<E, kNormFwd>
                               : (void*)rope_scalar_kernel<E, kNormBwd>;
}

struct Plan {
  bool vec;
  int lanes;      // lanes of a head (vector path)
  int chunks[2];  // per side
  int per_chunk[2];
  int grid_x;
};

// Split of a call: the warps of a CTA walk tokens of one chunk of heads, with
// two CTAs an SM in all.  A chunk is at least as many heads as the smaller side
// has, so that chunks take about as long (grouped keys) and a token's angles
// are fetched once a chunk; with few tokens the heads are split until about
// every warp has work.
cudaError_t make_plan(int64_t T, const int (&heads)[2], int dh, int mode, bool vec, int es,
                      Plan* p) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = sm_count(dev, &sms);
  if (e != cudaSuccess) return e;
  p->vec = vec;
  p->lanes = 32;
  int unit = 1;
  if (vec) {
    p->lanes = lanes_of((dh * es / 16 + 1) / 2);
    unit = 32 / p->lanes;
  }
  const int64_t warps = (int64_t)sms * kCtasPerSm * kWarps;
  const int fewer = heads[0] == 0   ? heads[1]
                    : heads[1] == 0 ? heads[0]
                                    : (heads[0] < heads[1] ? heads[0] : heads[1]);
  const int most = unit * (vec ? groups_in_flight(mode, es) : 4);
  int64_t per = fewer > most ? fewer : most;
  const int64_t split = T > 0 ? (warps + T - 1) / T : 1;  // chunks that give every warp a token
  const int64_t small = (heads[0] + heads[1] + split - 1) / split;
  if (small < per) per = small;
  per = (per + unit - 1) / unit * unit;
  for (int s = 0; s < 2; ++s) {
    p->per_chunk[s] = (int)per;
    p->chunks[s] = (int)((heads[s] + per - 1) / per);
  }
  const int chunks = p->chunks[0] + p->chunks[1];
  int64_t gx = (T + kWarps - 1) / kWarps;
  const int64_t all = (int64_t)kCtasPerSm * sms / chunks;  // one wave, not a CTA more
  if (gx > all) gx = all;
  p->grid_x = (int)(gx < 1 ? 1 : gx);
  return cudaSuccess;
}

size_t dw_bytes(const Plan& p, int dh) {
  return (size_t)(p.chunks[0] + p.chunks[1]) * p.grid_x * dh * sizeof(float);
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

// A tensor's pointer, and whether vectors fit it.
int check_heads(const adaln_heads_t* h, int heads, int64_t T, int es, bool* vec) {
  if (heads == 0) return ADALN_OK;
  if (!h) return ADALN_ERR_NULL;
  if (T > 0 && !h->ptr) return ADALN_ERR_NULL;
  if (h->token_stride < 0 || h->head_stride < 0) return ADALN_ERR_DIM;
  if (!aligned_to(h->ptr, es)) return ADALN_ERR_ALIGN;
  if (!aligned_to(h->ptr, 16) || h->token_stride * es % 16 != 0 || h->head_stride * es % 16 != 0)
    *vec = false;
  return ADALN_OK;
}

Tensor tensor_of(const adaln_heads_t* h, int es) {
  if (!h) return Tensor{nullptr, 0, 0};
  return Tensor{static_cast<const char*>(h->ptr), h->token_stride * es, h->head_stride * es};
}

// Whether the head's layout suits the vector path (its pointers aside).
bool vec_layout(int dh, int es, int pairs, bool half) {
  return dh * es % 16 == 0 && dh * es / 16 <= 64 && (!half || pairs * es % 16 == 0);
}

int run(int mode, const adaln_heads_t* const (&x)[2], const adaln_heads_t* const (&dy)[2],
        const adaln_heads_t* const (&out)[2], int64_t T, const int (&heads)[2], int32_t dh,
        adaln_dtype_t dtype, const adaln_rope_t* rope, const void* const (&w)[2], float eps,
        float* const (&dw)[2], void* workspace, size_t workspace_bytes, bool vec,
        cudaStream_t st) {
  const int es = dtype == ADALN_BF16 ? 2 : 4;
  RopeArgs a = {};
  for (int i = 0, at = 0; i < 4; ++i) {
    if (i < rope->axes) at += rope->pairs[i];
    a.axis_end[i] = at;
    a.P = at;
  }
  Plan p;
  cudaError_t e = make_plan(T, heads, dh, mode, vec, es, &p);
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
    sd.partial = partial && dw[s] ? partial + (size_t)(s ? p.chunks[0] : 0) * p.grid_x * dh
                                  : nullptr;
  }
  a.table = reinterpret_cast<const float2*>(rope->table);
  a.pos = rope->pos;
  a.T = T;
  a.rows = rope->rows;
  a.axes = rope->axes;
  a.dh = dh;
  a.nvec = dh * es / 16;
  a.eps = eps;
  a.inv_dh = 1.0f / (float)dh;
  a.status = status;

  const bool half = !rope->interleaved;
  int interleaved = rope->interleaved != 0;
  void* kernel;
  size_t smem = mode == kNormBwd ? (size_t)kWarps * dh * sizeof(float) : 0;
  if (p.vec) {
    if (dtype == ADALN_BF16)
      kernel = half ? pick_kernel<BF16, true>(p.lanes, mode) : pick_kernel<BF16, false>(p.lanes, mode);
    else
      kernel = half ? pick_kernel<F32, true>(p.lanes, mode) : pick_kernel<F32, false>(p.lanes, mode);
    const size_t table = (size_t)(16 / es / 2) * ((a.nvec + 1) / 2) * sizeof(float4);
    const size_t tables = table * (2 * kWarps + (mode == kNormFwd || mode == kNormBwd ? 1 : 0));
    smem = tables > smem ? tables : smem;
  } else {
    kernel = dtype == ADALN_BF16 ? scalar_kernel<BF16>(mode) : scalar_kernel<F32>(mode);
  }
  void* params[2] = {&a, &interleaved};
  const dim3 grid((unsigned)p.grid_x, (unsigned)(p.chunks[0] + p.chunks[1]));
  if (T > 0) {
    e = traced_launch(ADALN_KERNEL_QK_ROPE, st,
                      [&] { return launch(kernel, grid, kThreads, smem, params, st); });
    if (e != cudaSuccess) return launch_failed(e);
  }
  if (want_dw) {
    const float* pq = a.side[0].partial;
    const float* pk = a.side[1].partial;
    // No tokens (or no heads): the sums are empty.
    int nq = T > 0 ? p.chunks[0] * p.grid_x : 0, nk = T > 0 ? p.chunks[1] * p.grid_x : 0;
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
  bool vec = vec_layout(dh, es, pairs, !rope->interleaved);
  if ((rc = check_heads(q, hq, T, es, &vec)) || (rc = check_heads(k, hk, T, es, &vec)) ||
      (rc = check_heads(q_out, hq, T, es, &vec)) || (rc = check_heads(k_out, hk, T, es, &vec)))
    return rc;
  if (norm) {
    if (!std::isfinite(eps) || eps < 0.0f) return ADALN_ERR_ARG;
    if (!aligned_to(wq, es) || !aligned_to(wk, es)) return ADALN_ERR_ALIGN;
    if (!aligned_to(wq, 16) || !aligned_to(wk, 16)) vec = false;
  }
  if (T == 0) return ADALN_OK;
  return run(norm ? kNormFwd : kRotate, {q, k}, {nullptr, nullptr}, {q_out, k_out}, T, {hq, hk},
             dh, dtype, rope, {wq, wk}, eps, {nullptr, nullptr}, nullptr, 0, vec,
             static_cast<cudaStream_t>(stream));
}

int adaln_qk_rope_bwd_workspace_size(int64_t T, int32_t hq, int32_t hk, int32_t dh,
                                     adaln_dtype_t dtype, size_t* bytes) {
  const int rc = check_common(T, hq, hk, dh, dtype);
  if (rc != ADALN_OK) return rc;
  if (!bytes) return ADALN_ERR_NULL;
  // The larger of the two paths' needs (which one runs depends on alignment).
  const int es = dtype == ADALN_BF16 ? 2 : 4;
  size_t most = 0;
  for (int vec = 0; vec < 2; ++vec) {
    if (vec && !vec_layout(dh, es, 0, false)) continue;
    Plan p;
    const cudaError_t e = make_plan(T, {hq, hk}, dh, kNormBwd, vec != 0, es, &p);
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
  bool vec = vec_layout(dh, es, pairs, !rope->interleaved);
  if ((rc = check_heads(dq_out, hq, T, es, &vec)) || (rc = check_heads(dk_out, hk, T, es, &vec)) ||
      (rc = check_heads(dq, hq, T, es, &vec)) || (rc = check_heads(dk, hk, T, es, &vec)))
    return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!norm) {
    // The rotation's transpose is the rotation by the opposite angle.
    if (dwq || dwk) return ADALN_ERR_ARG;
    if (T == 0) return ADALN_OK;
    return run(kRotateBack, {dq_out, dk_out}, {nullptr, nullptr}, {dq, dk}, T, {hq, hk}, dh,
               dtype, rope, {nullptr, nullptr}, 0.0f, {nullptr, nullptr}, nullptr, 0, vec, st);
  }
  if ((rc = check_heads(q, hq, T, es, &vec)) || (rc = check_heads(k, hk, T, es, &vec))) return rc;
  if (!std::isfinite(eps) || eps < 0.0f) return ADALN_ERR_ARG;
  if (!aligned_to(wq, es) || !aligned_to(wk, es) || !aligned_to(dwq, 4) || !aligned_to(dwk, 4))
    return ADALN_ERR_ALIGN;
  if (!aligned_to(wq, 16) || !aligned_to(wk, 16)) vec = false;
  if ((dwq || dwk) && !workspace) return ADALN_ERR_NULL;
  if (!aligned_to(workspace, 16)) return ADALN_ERR_ALIGN;
  if (T == 0 && !dwq && !dwk) return ADALN_OK;
  return run(kNormBwd, {q, k}, {dq_out, dk_out}, {dq, dk}, T, {hq, hk}, dh, dtype, rope, {wq, wk},
             eps, {dwq, dwk}, workspace, workspace_bytes, vec, st);
}

}  // extern "C"
