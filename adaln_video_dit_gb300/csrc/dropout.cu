// Dropout from a counter-based generator, with the gate and the residual that
// stand around it in an adaLN-Zero block; the mask is never stored.
//
//   y  = [x +] [gate[b] *] m s h           b = seg_id[t], m = 0 or 1, s = 1 / P(m = 1)
//   dh = [gate[b] *] m s dy,   dgate[b] = sum over the segment's tokens of m s dy h
//
// m is a function of (seed, offset, place) alone, so the backward makes it again:
// Philox-4x32 with ten rounds (Salmon, Moraes, Dror, Shaw: "Parallel random
// numbers: as easy as 1, 2, 3", 2011) at key = seed and counter = (t ceil(D / 8) +
// c, offset) gives the eight 16-bit parts that elements 8 c .. 8 c + 7 of token t
// are compared with.  16 bits an element, not 32: one generator call of about 40
// instructions serves eight elements, which leaves the kernels bound by their
// bytes; the probability is a multiple of 2^-16, and s is that multiple's, so the
// expectation is kept exactly.  Arithmetic is fp32, each output rounded once.
//
// A thread owns the eight elements of a generator call ("group"): one 16-byte
// vector of bf16, two of fp32.  The forward gives it kRows rows of its column
// group, all loads ahead of the arithmetic; the generator's key schedule is then
// shared by the rows (with one row a thread it, not memory, set the time: 180 us
// where four take 153).  The backward with a gate gives it a range of rows, over
// which it sums dgate in registers, one fp32 partial for each (range, segment) it
// meets; a second launch adds the partials in a fixed order (no atomics: bitwise
// reproducible).  The (range, segment) pairs met along the rows form a monotone
// path, so slot = range + segment is unique for each.
//
// Bound: memory.  Measured (one GB300, T = 32760, D = 5120, bf16, p = 0.1, one
// segment; 1007 MB each way): forward 146 us, 6.9 TB/s; backward with dgate 166 us
// (its rows 155, its sums the rest; with p = 0 about 10 us less: the generator keeps
// the issue slots busy).  T = 5003, D = 1000, fp32, 37 segments, 60 MB: 12 and 21 us,
// of which the start and end of two and three launches are a third.  T = 262144, D =
// 1024, 300 segments: backward 260 us, but 525 where one of them has nearly all tokens:
// the sums' lanes go by the average segment, and one lane then adds its 900 partials.
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace adaln {
namespace {

template <class E>
constexpr int kRows = E::EPV == 8 ? 4 : 2;  // rows of a thread, all in flight
constexpr int kThreads = 256;
// The backward's threads a block, and threads an SM: rings of 32 KB, three or six of them.
template <class E>
constexpr int kBwdThreads = E::EPV == 8 ? 256 : 128;
constexpr int kBwdResident = 768;
constexpr int kBwdRows = 8;    // its least rows a thread

// What is dropped: nothing (the generator is not run), by chance, everything.
enum { kNone = 0, kSome = 1, kAll = 2 };

struct Rng {
  uint64_t seed, offset;
  const int64_t* state;  // device (seed, offset) instead of the two, or NULL
};

struct DropArgs {
  const void* h;       // dy in the backward
  const void* x;       // residual (forward) or NULL
  const void* saved;   // the forward's h (backward with dgate)
  const void* gate;
  const int32_t* seg;
  void* y;             // dh in the backward
  float* partials;     // [ranges + nseg - 1][D]
  int32_t* seg_start;  // [nseg + 1]
  int64_t T;
  int32_t D, nseg;
  int32_t groups;      // ceil(D / 8)
  int32_t ranges;      // of rows (backward)
  uint32_t limit;      // an element is dropped where its part << 16 is below this
  float factor;        // s
  Rng rng;
  unsigned* status;
};

struct Philox {
  uint32_t k0, k1, o0, o1;
  __device__ __forceinline__ explicit Philox(const Rng& r) {
    uint64_t seed = r.seed, offset = r.offset;
    if (r.state != nullptr) {
      seed = (uint64_t)r.state[0];
      offset = (uint64_t)r.state[1];
    }
    k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
    o0 = (uint32_t)offset, o1 = (uint32_t)(offset >> 32);
  }
  __device__ __forceinline__ void operator()(uint64_t at, uint32_t (&w)[4]) const {
    uint32_t c0 = (uint32_t)at, c1 = (uint32_t)(at >> 32), c2 = o0, c3 = o1, a = k0, b = k1;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
      const uint64_t p = (uint64_t)0xD2511F53u * c0, q = (uint64_t)0xCD9E8D57u * c2;
      c0 = (uint32_t)(q >> 32) ^ c1 ^ a;
      c2 = (uint32_t)(p >> 32) ^ c3 ^ b;
      c1 = (uint32_t)q;
      c3 = (uint32_t)p;
      a += 0x9E3779B9u;
      b += 0xBB67AE85u;
    }
    w[0] = c0, w[1] = c1, w[2] = c2, w[3] = c3;
  }
};

// The eight values of a group, as loaded and as fp32.
template <class E>
struct Raw {
  static constexpr int V = 8 / E::EPV;  // vectors
  uint4 v[V];
  __device__ __forceinline__ void load(const void* row, int g, int D) {
    const uint4* p = static_cast<const uint4*>(row) + (int64_t)g * V;
    v[0] = p[0];
    if (V > 1) v[V - 1] = 8 * g + 4 < D ? p[V - 1] : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void store(void* row, int g, int D) const {
    uint4* p = static_cast<uint4*>(row) + (int64_t)g * V;
    st_global_cs_v4(p, v[0]);
    if (V > 1 && 8 * g + 4 < D) st_global_cs_v4(p + V - 1, v[V - 1]);
  }
  __device__ __forceinline__ void get(float2 (&f)[4]) const {
    if constexpr (V == 1) {
      E::unpack2(v[0], f);
    } else {
      f[0] = make_float2(__uint_as_float(v[0].x), __uint_as_float(v[0].y));
      f[1] = make_float2(__uint_as_float(v[0].z), __uint_as_float(v[0].w));
      f[2] = make_float2(__uint_as_float(v[V - 1].x), __uint_as_float(v[V - 1].y));
      f[3] = make_float2(__uint_as_float(v[V - 1].z), __uint_as_float(v[V - 1].w));
    }
  }
  __device__ __forceinline__ void set(const float2 (&f)[4]) {
    if constexpr (V == 1) {
      v[0] = E::pack2(f);
    } else {
      const float2 lo[2] = {f[0], f[1]}, hi[2] = {f[2], f[3]};
      v[0] = F32::pack2(lo);
      v[V - 1] = F32::pack2(hi);
    }
  }
};

// Which of a group's elements are kept.
template <int DROP>
struct Kept {
  uint32_t w[4], limit;
  __device__ __forceinline__ Kept(const Philox& gen, uint64_t at, uint32_t limit) : limit(limit) {
    if (DROP == kSome) gen(at, w);
  }
  __device__ __forceinline__ bool first(int i) const {  // element 2 i
    return DROP == kNone || (DROP == kSome && w[i] << 16 >= limit);
  }
  __device__ __forceinline__ bool second(int i) const {  // element 2 i + 1
    return DROP == kNone || (DROP == kSome && w[i] >= limit);  // (limit's lower half is zero)
  }
  // f where kept and zero where not: chosen, not multiplied by zero, so nothing of a
  // dropped element, an infinity say, comes through.
  __device__ __forceinline__ float2 pick(int i, float2 f) const {
    return make_float2(first(i) ? f.x : 0.0f, second(i) ? f.y : 0.0f);
  }
};

template <class E>
__device__ __forceinline__ const unsigned char* row_of(const void* p, int64_t t, int D) {
  return static_cast<const unsigned char*>(p) + t * D * E::SIZE;
}
template <class E>
__device__ __forceinline__ unsigned char* row_of(void* p, int64_t t, int D) {
  return static_cast<unsigned char*>(p) + t * D * E::SIZE;
}

// Bits of what is wrong with segment b after segment `before` (raw values).
__device__ __forceinline__ unsigned wrong(int b, int before, int nseg) {
  return ((unsigned)b >= (unsigned)nseg ? ADALN_DEV_SEG_RANGE : 0u) |
         (before > b ? ADALN_DEV_SEG_ORDER : 0u);
}
__device__ __forceinline__ int clamped(int b, int nseg) { return min(max(b, 0), nseg - 1); }

// One pass without sums: the forward, and the backward without dgate.
template <class E, int DROP, bool GATE, bool ADD>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const __grid_constant__ DropArgs a) {
  grid_wait();
  grid_launch_dependents();
  const int D = a.D, groups = a.groups;
  const uint32_t at = blockIdx.x * (uint32_t)kThreads + threadIdx.x;  // (the host checks that it fits)
  const uint32_t rows = at / (uint32_t)groups;
  const int g = (int)(at - rows * (uint32_t)groups);
  const int64_t t0 = (int64_t)rows * kRows<E>;
  if (t0 >= a.T) return;
  Raw<E> h[kRows<E>], x[kRows<E>];
#pragma unroll
  for (int i = 0; i < kRows<E>; ++i)
    if (t0 + i < a.T) {
      if (DROP != kAll) h[i].load(row_of<E>(a.h, t0 + i, D), g, D);
      if (ADD) x[i].load(row_of<E>(a.x, t0 + i, D), g, D);
    }
  const Philox gen(a.rng);
  const float2 factor = splat2(a.factor), zero = splat2(0.0f);
  Raw<E> gate;
  int held = -1;
#pragma unroll
  for (int i = 0; i < kRows<E>; ++i) {
    const int64_t t = t0 + i;
    if (t >= a.T) break;
    if (GATE) {
      const int raw = a.seg[t], b = clamped(raw, a.nseg);
      if (g == 0) {  // one thread of a row checks it
        const unsigned bad = wrong(raw, t > 0 ? a.seg[t - 1] : raw, a.nseg);
        if (bad) atomicOr(a.status, bad);
      }
      if (b != held) gate.load(row_of<E>(a.gate, b, D), g, D);
      held = b;
    }
    float2 f[4], k[4], v[4];
    if (DROP != kAll) h[i].get(f);
    if (GATE) gate.get(k);
    if (ADD) x[i].get(v);
    const Kept<DROP> kept(gen, (uint64_t)t * groups + g, a.limit);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float2 q = zero;
      if (DROP != kAll) {
        q = DROP == kSome ? mul2(f[j], factor) : f[j];
        if (GATE) q = mul2(q, k[j]);
        q = kept.pick(j, q);
      }
      f[j] = ADD ? add2(q, v[j]) : q;
    }
    Raw<E> y;
    y.set(f);
    y.store(row_of<E>(a.y, t, D), g, D);
  }
}

// 16 bytes from global to shared memory, in groups of this thread's own.
__device__ __forceinline__ void copy_async(uint32_t to, const uint4* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The backward with dgate: thread (range, group) walks the range's rows.  The rows
// ahead are on their way into shared memory, each thread's own vectors into its own
// places (so nothing waits for another thread): the sums, the gate and the generator
// leave no registers for them.
template <class E, int DROP>
__global__ void __launch_bounds__(kBwdThreads<E>, kBwdResident / kBwdThreads<E>)
    dropout_bwd_kernel(const __grid_constant__ DropArgs a) {
  constexpr int V = Raw<E>::V, S = 4, N = kBwdThreads<E>;  // S stages of a vector or two a thread
  __shared__ uint4 ring[S][2 * V][N];
  grid_wait();
  grid_launch_dependents();
  const int D = a.D, groups = a.groups;
  const uint32_t at = blockIdx.x * (uint32_t)N + threadIdx.x;  // (the host checks that it fits)
  const uint32_t r = at / (uint32_t)groups;
  if (r >= (uint32_t)a.ranges) return;
  const int g = (int)(at - r * (uint32_t)groups);
  const int64_t begin = part_begin(r, a.T, a.ranges);
  const int rows = (int)(part_begin(r + 1, a.T, a.ranges) - begin);
  const int64_t pitch = (int64_t)D * E::SIZE / 16;  // vectors of a row
  const bool whole = 8 * g + 4 < D;                 // the group has both its vectors
  const uint4* dys = reinterpret_cast<const uint4*>(row_of<E>(a.h, begin, D)) + g * V;
  const uint4* hs = reinterpret_cast<const uint4*>(row_of<E>(a.saved, begin, D)) + g * V;
  unsigned char* out = row_of<E>(a.y, begin, D);
  const int32_t* const seg = a.seg + begin;
  const uint32_t mine = smem_addr(&ring[0][0][threadIdx.x]);
  auto fetch = [&](int t, int s) {
    if (DROP != kAll && t < rows) {
      const uint32_t to = mine + s * (2 * V * N * 16);
      copy_async(to, dys);
      copy_async(to + V * N * 16, hs);
      if (V > 1 && whole) {
        copy_async(to + N * 16, dys + 1);
        copy_async(to + (V + 1) * N * 16, hs + 1);
      }
      dys += pitch;
      hs += pitch;
    }
    copy_commit();
  };
  for (int t = 0; t < S - 1; ++t) fetch(t, t);
  const Philox gen(a.rng);
  const float2 factor = splat2(a.factor), zero = splat2(0.0f);
  float2 gate[4];  // times the factor
  int held = -1;
  float2 sum[4] = {};  // without it
  auto flush = [&] {
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[j] = mul2(sum[j], factor);
    float4* p = reinterpret_cast<float4*>(a.partials + ((int64_t)r + held) * D + 8 * g);
    p[0] = make_float4(sum[0].x, sum[0].y, sum[1].x, sum[1].y);
    if (whole) p[1] = make_float4(sum[2].x, sum[2].y, sum[3].x, sum[3].y);
  };
  // One thread of a row checks its segment and notes where segments start.
  int before = begin > 0 ? seg[-1] : -1, noted = begin > 0 ? clamped(before, a.nseg) : -1;
  uint64_t place = (uint64_t)begin * groups + g;
  int s = 0, next = seg[0];
  for (int t = 0; t < rows; ++t) {
    fetch(t + S - 1, s == 0 ? S - 1 : s - 1);
    const int raw = next, b = clamped(raw, a.nseg);
    if (t + 1 < rows) next = seg[t + 1];
    if (g == 0) {
      const unsigned bad = wrong(raw, before, a.nseg);
      if (bad) atomicOr(a.status, bad);
      before = raw;
      for (; noted < b; ++noted) a.seg_start[noted + 1] = (int32_t)(begin + t);
    }
    if (b != held) {
      if (held >= 0) flush();
      Raw<E> x;
      x.load(row_of<E>(a.gate, b, D), g, D);
      x.get(gate);
      held = b;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        gate[j] = mul2(gate[j], factor);
        sum[j] = zero;
      }
    }
    const Kept<DROP> kept(gen, place, a.limit);
    place += groups;
    copy_wait<S - 1>();
    float2 f[4], v[4];
    if (DROP != kAll) {
      Raw<E> x;
#pragma unroll
      for (int n = 0; n < V; ++n) x.v[n] = ring[s][n][threadIdx.x];
      x.get(f);
#pragma unroll
      for (int n = 0; n < V; ++n) x.v[n] = ring[s][V + n][threadIdx.x];
      x.get(v);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (DROP == kAll) {
        f[j] = zero;
      } else if (DROP == kNone) {
        sum[j] = fma2(f[j], v[j], sum[j]);
        f[j] = mul2(f[j], gate[j]);
      } else {
        if (kept.first(j)) sum[j].x = fmaf(f[j].x, v[j].x, sum[j].x);
        if (kept.second(j)) sum[j].y = fmaf(f[j].y, v[j].y, sum[j].y);
        f[j] = kept.pick(j, mul2(f[j], gate[j]));
      }
    }
    Raw<E> y;
    y.set(f);
    y.store(out, g, D);
    out += pitch * 16;
    if (++s == S) s = 0;
  }
  if (g == 0 && begin + rows == a.T)
    for (; noted < a.nseg; ++noted) a.seg_start[noted + 1] = (int32_t)a.T;
  if (held >= 0) flush();
}

// dgate[b] = the sum of the segment's partials in slot order: `lanes` groups of
// them, each summed in order, joined in lane order.  A block takes `lanes` groups
// of slots x (kThreads / lanes) vectors of four columns.
__global__ void __launch_bounds__(kThreads) dropout_gate_kernel(const float* partials,
                                                                const int32_t* seg_start, int64_t T,
                                                                int D, int nseg, int ranges, int lanes,
                                                                float* dgate) {
  __shared__ float4 part[kThreads];
  grid_wait();
  grid_launch_dependents();
  const int cols = kThreads / lanes, vecs = D / 4, chunks = (vecs + cols - 1) / cols;
  const int lane = threadIdx.x / cols, col = threadIdx.x - lane * cols;
  for (int64_t u = blockIdx.x; u < (int64_t)nseg * chunks; u += gridDim.x) {
    const int b = (int)(u / chunks), c = (int)(u - (int64_t)b * chunks) * cols + col;
    const int64_t s = seg_start[b], e = seg_start[b + 1];
    float4 sum = make_float4(0, 0, 0, 0);
    if (s < e && c < vecs) {
      const int first = (int)part_owner(s, T, ranges), last = (int)part_owner(e - 1, T, ranges);
      const int n = last - first + 1;
      const int lo = first + (int)((int64_t)n * lane / lanes);
      const int hi = first + (int)((int64_t)n * (lane + 1) / lanes);
      const float4* p = reinterpret_cast<const float4*>(partials) + c;
#pragma unroll 8
      for (int r = lo; r < hi; ++r) {
        const float4 v = p[((int64_t)r + b) * vecs];
        sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
      }
    }
    if (lanes > 1) {
      part[threadIdx.x] = sum;
      __syncthreads();
      if (lane == 0)
        for (int i = 1; i < lanes; ++i) {
          const float4 v = part[i * cols + col];
          sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
        }
      __syncthreads();
    }
    if (lane == 0 && c < vecs) reinterpret_cast<float4*>(dgate + (int64_t)b * D)[c] = sum;
  }
}

// ----- host side ------------------------------------------------------------------

cudaError_t launch(void* kernel, int64_t grid, int threads, void** params, cudaStream_t st) {
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  Shape s = {};
  s.grid = (int)grid;
  s.threads = threads;
  return traced_launch(ADALN_KERNEL_DROPOUT, st,
                       [&] { return launch_dependent(kernel, s, params, st); });
}

template <class E, int DROP>
void* pass_kernel(bool gate, bool add) {
  return gate ? add ? (void*)dropout_kernel<E, DROP, true, true> : (void*)dropout_kernel<E, DROP, true, false>
         : add ? (void*)dropout_kernel<E, DROP, false, true>
               : (void*)dropout_kernel<E, DROP, false, false>;
}
template <class E>
void* pass_kernel(int drop, bool gate, bool add) {
  return drop == kNone   ? pass_kernel<E, kNone>(gate, add)
         : drop == kSome ? pass_kernel<E, kSome>(gate, add)
                         : pass_kernel<E, kAll>(gate, add);
}
template <class E>
void* bwd_kernel(int drop) {
  return drop == kNone   ? (void*)dropout_bwd_kernel<E, kNone>
         : drop == kSome ? (void*)dropout_bwd_kernel<E, kSome>
                         : (void*)dropout_bwd_kernel<E, kAll>;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check(int64_t T, int32_t D, int32_t nseg, adaln_dtype_t dt, bool gate) {
  if (dt != ADALN_F32 && dt != ADALN_BF16) return ADALN_ERR_DTYPE;
  if (T < 0 || T > (int64_t)INT32_MAX) return ADALN_ERR_DIM;
  if (D < 1 || D > ADALN_DROPOUT_MAX_D || D * (dt == ADALN_BF16 ? 2 : 4) % 16 != 0) return ADALN_ERR_DIM;
  if (T * ((D + 7) / 8) > ((int64_t)UINT32_MAX - kThreads)) return ADALN_ERR_DIM;
  if (gate && (nseg < 1 || nseg > ADALN_MAX_NSEG)) return ADALN_ERR_DIM;
  return ADALN_OK;
}

// How often an element is dropped, in 2^-16; -1 for a bad p.
int dropped_of(double p) {
  return p >= 0.0 && p <= 1.0 ? (int)std::floor(65536.0 * p + 0.5) : -1;
}
int kind_of(int dropped) { return dropped == 0 ? kNone : dropped < 65536 ? kSome : kAll; }

// Ranges of rows of the backward: threads for one wave of blocks, with at least
// kBwdRows rows each (a range costs a partial).
int ranges_of(int64_t T, int32_t D, int sms) {
  const int64_t groups = (D + 7) / 8;
  const int64_t wave = (int64_t)sms * kBwdResident / groups;
  const int64_t most = (T + kBwdRows - 1) / kBwdRows;
  const int64_t n = wave < most ? wave : most;
  return (int)(n < 1 ? 1 : n);
}
size_t partial_bytes(int32_t D, int32_t nseg, int ranges) {
  return ((size_t)ranges + nseg - 1) * (size_t)D * sizeof(float);
}
size_t workspace_bytes_of(int32_t D, int32_t nseg, int ranges) {
  return (partial_bytes(D, nseg, ranges) + ((size_t)nseg + 1) * 4 + 255) & ~(size_t)255;
}

cudaError_t device_sms(int* sms) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e == cudaSuccess ? sm_count(dev, sms) : e;
}

DropArgs args_of(int64_t T, int32_t D, int32_t nseg, int dropped, const adaln_rng_t* rng) {
  DropArgs a = {};
  a.T = T;
  a.D = D;
  a.nseg = nseg;
  a.groups = (D + 7) / 8;
  a.limit = dropped < 65536 ? (uint32_t)dropped << 16 : 0u;
  a.factor = dropped < 65536 ? (float)(65536.0 / (65536 - dropped)) : 0.0f;
  if (rng) a.rng = Rng{rng->seed, rng->offset, rng->state};
  return a;
}

int run_pass(DropArgs& a, int drop, adaln_dtype_t dt, cudaStream_t st) {
  cudaError_t e = status_word(&a.status);
  if (e != cudaSuccess) return launch_failed(e);
  void* params[1] = {&a};
  const int rows = dt == ADALN_BF16 ? kRows<BF16> : kRows<F32>;
  const int64_t threads = (a.T + rows - 1) / rows * a.groups;
  void* k = dt == ADALN_BF16 ? pass_kernel<BF16>(drop, a.gate != nullptr, a.x != nullptr)
                             : pass_kernel<F32>(drop, a.gate != nullptr, a.x != nullptr);
  e = launch(k, (threads + kThreads - 1) / kThreads, kThreads, params, st);
  return e == cudaSuccess ? ADALN_OK : launch_failed(e);
}

}  // namespace
}  // namespace adaln

using namespace adaln;

extern "C" {

int adaln_dropout_fwd(const void* h, const void* x, const void* gate, const int32_t* seg_id, int64_t T,
                      int32_t D, int32_t nseg, adaln_dtype_t dtype, double p, const adaln_rng_t* rng,
                      void* y, void* stream) {
  const int rc = check(T, D, nseg, dtype, gate != nullptr);
  if (rc != ADALN_OK) return rc;
  const int dropped = dropped_of(p);
  if (dropped < 0) return ADALN_ERR_ARG;
  const int drop = kind_of(dropped);
  if (drop == kSome && !rng) return ADALN_ERR_NULL;
  if (drop == kSome && !aligned(rng->state, 8)) return ADALN_ERR_ALIGN;
  if (T == 0) return ADALN_OK;
  if (!h || !y || (gate && !seg_id)) return ADALN_ERR_NULL;
  if (!aligned(h, 16) || !aligned(x, 16) || !aligned(gate, 16) || !aligned(y, 16) ||
      (gate && !aligned(seg_id, 4)))
    return ADALN_ERR_ALIGN;
  DropArgs a = args_of(T, D, nseg, dropped, drop == kSome ? rng : nullptr);
  a.h = h, a.x = x, a.gate = gate, a.seg = seg_id, a.y = y;
  return run_pass(a, drop, dtype, static_cast<cudaStream_t>(stream));
}

int adaln_dropout_bwd_workspace_size(int64_t T, int32_t D, int32_t nseg, adaln_dtype_t dtype,
                                     size_t* bytes) {
  const int rc = check(T, D, nseg, dtype, true);
  if (rc != ADALN_OK) return rc;
  if (!bytes) return ADALN_ERR_NULL;
  int sms = 0;
  const cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return launch_failed(e);
  *bytes = workspace_bytes_of(D, nseg, ranges_of(T, D, sms));
  return ADALN_OK;
}

int adaln_dropout_bwd(const void* dy, const void* h, const void* gate, const int32_t* seg_id, int64_t T,
                      int32_t D, int32_t nseg, adaln_dtype_t dtype, double p, const adaln_rng_t* rng,
                      void* dh, float* dgate, void* workspace, size_t workspace_bytes, void* stream) {
  const int rc = check(T, D, nseg, dtype, gate || dgate);
  if (rc != ADALN_OK) return rc;
  const int dropped = dropped_of(p);
  if (dropped < 0) return ADALN_ERR_ARG;
  const int drop = kind_of(dropped);
  if (drop == kSome && !rng) return ADALN_ERR_NULL;
  if (drop == kSome && !aligned(rng->state, 8)) return ADALN_ERR_ALIGN;
  if (dgate && !aligned(dgate, 16)) return ADALN_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) {  // empty sums
    if (!dgate) return ADALN_OK;
    const cudaError_t e = cudaMemsetAsync(dgate, 0, (size_t)nseg * D * sizeof(float), st);
    return e == cudaSuccess ? ADALN_OK : launch_failed(e);
  }
  if (!dy || !dh || (gate && !seg_id) || (dgate && (!gate || !h || !workspace))) return ADALN_ERR_NULL;
  if (!aligned(dy, 16) || !aligned(gate, 16) || !aligned(dh, 16) || (gate && !aligned(seg_id, 4)) ||
      (dgate && (!aligned(h, 16) || !aligned(workspace, 16))))
    return ADALN_ERR_ALIGN;
  DropArgs a = args_of(T, D, nseg, dropped, drop == kSome ? rng : nullptr);
  a.h = dy, a.gate = gate, a.seg = seg_id, a.y = dh;
  if (!dgate) return run_pass(a, drop, dtype, st);

  int sms = 0;
  cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return launch_failed(e);
  a.ranges = ranges_of(T, D, sms);
  if (workspace_bytes < workspace_bytes_of(D, nseg, a.ranges)) return ADALN_ERR_WORKSPACE;
  a.saved = h;
  a.partials = static_cast<float*>(workspace);
  a.seg_start = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + partial_bytes(D, nseg, a.ranges));
  if ((e = status_word(&a.status)) != cudaSuccess) return launch_failed(e);
  void* params[1] = {&a};
  const int64_t threads = (int64_t)a.ranges * a.groups;
  const int block = dtype == ADALN_BF16 ? kBwdThreads<BF16> : kBwdThreads<F32>;
  e = launch(dtype == ADALN_BF16 ? bwd_kernel<BF16>(drop) : bwd_kernel<F32>(drop),
             (threads + block - 1) / block, block, params, st);
  if (e != cudaSuccess) return launch_failed(e);

  const int64_t each = a.ranges / nseg + 1;  // partials of a segment, about
  int lanes = each > 64 ? 32 : each > 4 ? 8 : 1;
  const int cols = kThreads / lanes, chunks = (D / 4 + cols - 1) / cols;
  const int64_t units = (int64_t)nseg * chunks, most = (int64_t)sms * 8;
  void* join[8] = {&a.partials, &a.seg_start, &a.T, &a.D, &a.nseg, &a.ranges, &lanes, &dgate};
  e = launch((void*)dropout_gate_kernel, units < most ? units : most, kThreads, join, st);
  return e == cudaSuccess ? ADALN_OK : launch_failed(e);
}

}  // extern "C"
