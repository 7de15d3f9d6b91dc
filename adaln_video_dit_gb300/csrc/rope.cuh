// The vector kernels of the rotary operator (rope.cu), a template that several
// files instantiate.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace adaln {
namespace rope {

constexpr int kWarps = 8;  // warps of a CTA
constexpr int kThreads = kWarps * 32;
constexpr int kCtasPerSm = 2;
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
  float* partial;  // kNormBwd: [chunks * ctas][dh], or nullptr: no dw
  int heads;
  int chunks;      // the heads are split into this many chunks
  int per_chunk;   // heads of a chunk
  int ctas;        // CTAs of a chunk
  int tpw;         // few heads: tokens side by side in a warp; 0: heads only
};

struct RopeArgs {
  Side side[2];
  const float2* table;  // [rows][P]
  const int32_t* pos;   // [T][axes]
  int64_t T;
  int rows, axes, P, dh, nvec;
  int axis_end[4];  // pairs [axis_end[a-1], axis_end[a]) belong to axis a
  int batch;        // tokens whose angles a table in shared memory holds
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
  __device__ __forceinline__ void load(const RopeArgs& a, int64_t t, bool report) {
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
    if (bad && report) atomicOr(a.status, ADALN_DEV_POS_RANGE);
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

// A vector of W 32-bit words, in memory at W * 4 byte alignment.
template <int W>
struct Words {
  uint32_t w[W];
};
template <int W>
__device__ __forceinline__ Words<W> ld_words(const char* p) {
  Words<W> r;
  if constexpr (W == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
  } else if constexpr (W == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r.w[0] = v.x, r.w[1] = v.y;
  } else {
    r.w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
  return r;
}
template <int W>
__device__ __forceinline__ void st_words(char* p, const Words<W>& r) {
  if constexpr (W == 4)
    *reinterpret_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
  else if constexpr (W == 2)
    *reinterpret_cast<uint2*>(p) = make_uint2(r.w[0], r.w[1]);
  else
    *reinterpret_cast<uint32_t*>(p) = r.w[0];
}
__device__ __forceinline__ uint32_t pack_pair(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A lane's two vectors (SIZE bytes an element) as pairs, split: the first
// elements of pairs 2 i and 2 i + 1 in A[i], the second ones in B[i], so that two
// pairs turn in packed arithmetic.  Interleaved pairs are neighbours in a vector
// (vector a's, then b's); those of the halves layout are the same element of a
// and of b.
template <int SIZE, int W, bool HALF, int M>
__device__ __forceinline__ void split(const Words<W>& a, const Words<W>& b, float2 (&A)[M],
                                      float2 (&B)[M]) {
  auto word = [&](int i) { return i < W ? a.w[i] : b.w[i - W]; };
  auto lo = [&](int i) { return __uint_as_float(word(i) << 16); };
  auto hi = [&](int i) { return __uint_as_float(word(i) & 0xffff0000u); };
  auto f = [&](int i) { return __uint_as_float(word(i)); };
#pragma unroll
  for (int i = 0; i < M; ++i) {
    if (SIZE == 2) {
      A[i] = HALF ? make_float2(lo(i), hi(i)) : make_float2(lo(2 * i), lo(2 * i + 1));
      B[i] = HALF ? make_float2(lo(W + i), hi(W + i)) : make_float2(hi(2 * i), hi(2 * i + 1));
    } else {
      A[i] = HALF ? make_float2(f(2 * i), f(2 * i + 1)) : make_float2(f(4 * i), f(4 * i + 2));
      B[i] = HALF ? make_float2(f(W + 2 * i), f(W + 2 * i + 1))
                  : make_float2(f(4 * i + 1), f(4 * i + 3));
    }
  }
}
// And back, rounded to the element type.
template <int SIZE, int W, bool HALF, int M>
__device__ __forceinline__ void join(const float2 (&A)[M], const float2 (&B)[M], Words<W>& a,
                                     Words<W>& b) {
  auto put = [&](int i, uint32_t v) { (i < W ? a.w[i] : b.w[i - W]) = v; };
#pragma unroll
  for (int i = 0; i < M; ++i) {
    if (SIZE == 2 && HALF) {
      put(i, pack_pair(A[i].x, A[i].y));
      put(W + i, pack_pair(B[i].x, B[i].y));
    } else if (SIZE == 2) {
      put(2 * i, pack_pair(A[i].x, B[i].x));
      put(2 * i + 1, pack_pair(A[i].y, B[i].y));
    } else {
      put(HALF ? 2 * i : 4 * i, __float_as_uint(A[i].x));
      put(HALF ? 2 * i + 1 : 4 * i + 2, __float_as_uint(A[i].y));
      put(HALF ? W + 2 * i : 4 * i + 1, __float_as_uint(B[i].x));
      put(HALF ? W + 2 * i + 1 : 4 * i + 3, __float_as_uint(B[i].y));
    }
  }
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

// Vector path: heads of whole, aligned vectors of W words, at most 64 of them.
// P lanes a head, U groups of 32 / P heads in flight.
// FEW: a side may have at most 32 / P heads and take several tokens at a time.
template <int SIZE, int W, int P, bool HALF, bool FEW, int MODE, int U>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    rope_vec_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int VB = 4 * W;      // bytes of a vector
  constexpr int N = VB / SIZE;   // its elements, and the pairs of a lane
  constexpr int M = N / 2;       // packed pairs of pairs of a lane
  constexpr int HPW = 32 / P;    // heads side by side in a warp
  constexpr bool kNorm = MODE == kNormFwd || MODE == kNormBwd;
  constexpr bool kGrad = MODE == kNormBwd;
  constexpr bool kBack = MODE == kRotateBack || MODE == kNormBwd;
  // Tables of [M][half] float4: lane j's i-th entry holds, for its pairs 2 i
  // and 2 i + 1, two cosines and two sines, or the two weights of A and of B;
  // neighbouring lanes' entries are neighbours, so a read has no bank conflict.
  // The weights' table, then per warp two sets of `batch` tables of angles (the
  // tokens at work, the next ones).  After the walk the norm's backward puts
  // [kWarps][dh] weight sums there.
  extern __shared__ __align__(16) float4 shared[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = (a.nvec + 1) >> 1, entries = M * half;
  float4* const weights = shared;
  const int j = lane % P, sub = lane / P;  // (sub = HPW: lanes left over)
  const bool is_k = (int)blockIdx.x >= a.side[0].chunks * a.side[0].ctas;
  const Side& sd = a.side[is_k];
  const int cta = blockIdx.x - (is_k ? a.side[0].chunks * a.side[0].ctas : 0);
  const int chunk = cta / sd.ctas;
  const int h_begin = chunk * sd.per_chunk, h_end = min(sd.heads, h_begin + sd.per_chunk);
  // A batch is one token (group u of heads is HPW further on), or with few heads
  // U tpw tokens (group u is tpw tokens further on).
  const bool few = FEW && sd.tpw > 0;
  const int tpw = few ? sd.tpw : 1;
  const int tsub = few ? sub / sd.per_chunk : 0, hsub = few ? sub - tsub * sd.per_chunk : sub;
  const int tokens = few ? U * tpw : 1, batch = FEW ? a.batch : 1;
  float4* const angles = shared + (kNorm ? entries : 0) + warp * 2 * batch * entries;

  // This lane's two vectors (-1: none).
  const int nr = a.P / N;  // halves: vectors of the first half
  int va = HALF && j >= nr ? 2 * nr + 2 * (j - nr) : j;
  int vb = HALF ? (j < nr ? j + nr : va + 1) : j + half;
  const bool idle = j >= half || sub >= HPW || (few && tsub >= tpw);
  if (va >= a.nvec || idle) va = -1;
  if (vb >= a.nvec || idle) vb = -1;
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

  // This lane's share of a token's pairs, p = lane, lane + 32, ...: f(p, its index
  // into a table, its axis).  The norm's backward, which is the furthest from the
  // memory's rate, keeps those of the first two (heads of up to 128 elements have no
  // more): 16384 tokens of 24 + 24 heads x 64 bf16, both passes, 102.4 -> 101.1 us.
  // The other kernels work them out anew: with more registers held the rotation of
  // the joint stream went from 135.8 to 138.0 us, the long video's norm from 203 to 208.
  const int at0 = entry_of_pair(min(lane, a.P - 1)), at1 = entry_of_pair(min(lane + 32, a.P - 1));
  const int axis0 = axis_of(a, lane), axis1 = axis_of(a, lane + 32);
  auto each_pair = [&](auto f) {
    if constexpr (kGrad) {
      if (lane < a.P) f(lane, at0, axis0);
      if (lane + 32 < a.P) f(lane + 32, at1, axis1);
    }
    for (int p = lane + (kGrad ? 64 : 0); p < a.P; p += 32) f(p, entry_of_pair(p), axis_of(a, p));
  };
  // Angles of pair p from table row `row` (-1: unrotated) into a table at `index`.
  auto put_angle = [&](float4* table, int index, int p, int row) {
    float* const at = reinterpret_cast<float*>(table) + index;
    if (row >= 0) {
      const float* from = reinterpret_cast<const float*>(a.table + (int64_t)row * a.P + p);
      cp_async4(at, from);
      cp_async4(at + 2, from + 1);
    } else {
      at[0] = 1.0f;
      at[2] = 0.0f;
    }
  };
  auto pick = [](int axis, int r0, int r1, int r2, int r3) {
    return axis == 0 ? r0 : axis == 1 ? r1 : axis == 2 ? r2 : r3;
  };
  // The angles of a batch into set b.  `rows`: the token's, in every lane; with
  // few heads, lane n's are those of the batch's n-th token.
  auto fetch_angles = [&](const Rows& rows, int b) {
    float4* const set = angles + b * batch * entries;
    if (!few) {
      each_pair([&](int p, int at, int axis) {
        put_angle(set, at, p, pick(axis, rows.r[0], rows.r[1], rows.r[2], rows.r[3]));
      });
      return;
    }
    int n = 0, p = lane;
    for (int i = 0; i < tokens * a.P; i += 32) {  // (all lanes: the shuffles)
      while (p >= a.P) p -= a.P, ++n;
      int r[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) r[k] = k < a.axes ? __shfl_sync(~0u, rows.r[k], n & 31) : -1;
      if (n < tokens)
        put_angle(set + n * entries, entry_of_pair(p), p, pick(axis_of(a, p), r[0], r[1], r[2], r[3]));
      p += 32;
    }
  };
  auto load_rows = [&](Rows& rows, int64_t t) {
    if (few) {
      rows = Rows{{-1, -1, -1, -1}};
      if (lane < tokens && t + lane < a.T) rows.load(a, t + lane, true);
    } else if (t < a.T) {
      rows.load(a, t, lane == 0);
    }
  };
  // Whether some pair of the token has a zero sine: only then is each looked
  // at (turn() below), else two pairs turn in four packed operations.
  const bool always = few || 2 * a.P < a.dh;
  auto any_still = [&](int b) {
    if (always) return true;
    const float* const from = reinterpret_cast<const float*>(angles + b * batch * entries);
    bool z = false;
    each_pair([&](int, int at, int) { z |= from[at + 2] == 0.0f; });
    return (bool)__any_sync(~0u, z);
  };

  struct Group {
    Words<W> xa[U], xb[U], ya[kGrad ? U : 1], yb[kGrad ? U : 1];
  };
  // Whether this lane has a head in group u of the batch at (t, h0).
  auto on = [&](int64_t t, int h0, int u) {
    return few ? tsub < tpw && t + u * tpw + tsub < a.T
               : t < a.T && h0 + u * HPW + sub < h_end;
  };
  auto load = [&](Group& g, int64_t t, int h0) {
    const char* x = sd.x.p + (t + tsub) * sd.x.ts + (h0 + hsub) * sd.x.hs;
    const char* y = kGrad ? sd.dy.p + (t + tsub) * sd.dy.ts + (h0 + hsub) * sd.dy.hs : nullptr;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = on(t, h0, u);
      g.xa[u] = in && va >= 0 ? ld_words<W>(x + va * VB) : Words<W>{};
      g.xb[u] = in && vb >= 0 ? ld_words<W>(x + vb * VB) : Words<W>{};
      x += few ? tpw * sd.x.ts : HPW * sd.x.hs;
      if (kGrad) {
        g.ya[u] = in && va >= 0 ? ld_words<W>(y + va * VB) : Words<W>{};
        g.yb[u] = in && vb >= 0 ? ld_words<W>(y + vb * VB) : Words<W>{};
        y += few ? tpw * sd.dy.ts : HPW * sd.dy.hs;
      }
    }
  };
  auto rotate = [&](float2(&A)[M], float2(&B)[M], const float4* cs, bool still) {
#pragma unroll
    for (int i = 0; i < M; ++i) {
      const float4 t = ld_shared_f4(cs + i * half);
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

  const int64_t step = (int64_t)sd.ctas * kWarps * tokens;
  int64_t t = ((int64_t)(cta - chunk * sd.ctas) * kWarps + warp) * tokens;
  Group cur;
  load(cur, t, h_begin);
  Rows rows;  // of the batch after the one whose angles are on their way
  load_rows(rows, t);
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
            SIZE == 2 ? __bfloat162float(static_cast<const __nv_bfloat16*>(sd.w)[d])
                      : static_cast<const float*>(sd.w)[d];
      }
    }
  }
  for (int i = lane; i < 2 * batch * entries; i += 32)
    angles[i] = make_float4(1.0f, 1.0f, 0.0f, 0.0f);
  __syncthreads();
  if (t < a.T) {
    fetch_angles(rows, 0);
    load_rows(rows, t + step);
  }
  for (int slot = 0; t < a.T; t += step, slot ^= 1) {
    cp_async_wait();
    __syncwarp();
    const bool still = any_still(slot);
    if (t + step < a.T) {
      fetch_angles(rows, slot ^ 1);
      load_rows(rows, t + 2 * step);
    }
    const float4* cs0 = angles + (slot * batch + (few ? min(tsub, tpw - 1) : 0)) * entries + jj;

    for (int h0 = h_begin; h0 < h_end; h0 += few ? sd.per_chunk : U * HPW) {
      Group next;
      const bool more = !few && h0 + U * HPW < h_end;
      load(next, more ? t : t + step, more ? h0 + U * HPW : h_begin);
      char* out = sd.out + (t + tsub) * sd.out_ts + (h0 + hsub) * sd.out_hs;
#pragma unroll
      for (int u = 0; u < U; ++u, out += few ? tpw * sd.out_ts : HPW * sd.out_hs) {
        if (few ? t + u * tpw >= a.T : h0 + u * HPW >= h_end) break;
        const bool in = on(t, h0, u);
        const float4* cs = cs0 + (few ? u * tpw * entries : 0);
        float2 A[M], B[M];
        split<SIZE, W, HALF, M>(cur.xa[u], cur.xb[u], A, B);
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
            split<SIZE, W, HALF, M>(cur.ya[u], cur.yb[u], GA, GB);
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
            // (In this order: r^3 alone may overflow.)
            const float2 k = splat2(-(sh * a.inv_dh * r) * r * r), r2 = splat2(r);
            // Lanes without a head hold zeros, so they add nothing to dw (g = 0)
            // as long as r is finite; eps = 0 would make it 0 * inf.
            const float2 rd = splat2(in ? r : 0.0f);
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
        if (in) {
          Words<W> oa, ob;
          join<SIZE, W, HALF, M>(A, B, oa, ob);
          if (va >= 0) st_words<W>(out + va * VB, oa);
          if (vb >= 0) st_words<W>(out + vb * VB, ob);
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
    store_partial(red, sd.partial + (int64_t)cta * a.dh, a.dh);
  }
}

// ----- instantiation -------------------------------------------------------------

// Head groups in flight: what fits 128 registers a thread.  Forward and plain
// rotation, T = 32760 x 80 heads x 128: three groups 205.9 us, four (spilling
// with the norm) 226.5, two 206.9 (T = 36864 x 48 heads, rotation alone: 134.9,
// 135.2 and 144.4).  The norm's backward holds twice the tensors and its weight
// sums: with two groups of bf16 heads it spilled, and 8192 tokens x 24 heads x
// 128 took 41.0 instead of 30.6 us.
ADALN_HD constexpr int groups_in_flight(int mode, int es, bool few) {
  return mode != kNormBwd ? 3 : es == 2 || few ? 1 : 2;
}

template <int SIZE, int W, int P, bool HALF, bool FEW, int MODE>
void* vec_kernel_of() {
  return (void*)rope_vec_kernel<SIZE, W, P, HALF, FEW, MODE, groups_in_flight(MODE, SIZE, FEW)>;
}
template <int SIZE, int W, int P, bool HALF, bool FEW>
void* vec_kernel(int mode) {
  return mode == kRotate       ? vec_kernel_of<SIZE, W, P, HALF, FEW, kRotate>()
         : mode == kRotateBack ? vec_kernel_of<SIZE, W, P, HALF, FEW, kRotateBack>()
         : mode == kNormFwd    ? vec_kernel_of<SIZE, W, P, HALF, FEW, kNormFwd>()
                               : vec_kernel_of<SIZE, W, P, HALF, FEW, kNormBwd>();
}
template <int SIZE, bool HALF, bool FEW>
void* wide_kernel(int lanes, int mode) {
  switch (lanes) {
    case 4: return vec_kernel<SIZE, 4, 4, HALF, FEW>(mode);
    case 5: return vec_kernel<SIZE, 4, 5, HALF, FEW>(mode);
    case 6: return vec_kernel<SIZE, 4, 6, HALF, FEW>(mode);
    case 8: return vec_kernel<SIZE, 4, 8, HALF, FEW>(mode);
    case 10: return vec_kernel<SIZE, 4, 10, HALF, FEW>(mode);
    case 16: return vec_kernel<SIZE, 4, 16, HALF, FEW>(mode);
    default: return vec_kernel<SIZE, 4, 32, HALF, FEW>(mode);
  }
}

}  // namespace rope

// The kernel for heads of `lanes` lanes (lanes_of) and a mode, by file.
void* rope_bf16_kernel(int lanes, bool half, int mode);
void* rope_f32_kernel(int lanes, bool half, int mode);
void* rope_few_kernel(int es, int lanes, bool half, int mode);
void* rope_narrow_kernel(int es, int width, int lanes, int mode);

}  // namespace adaln
