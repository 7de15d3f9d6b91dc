// Tokens sorted by expert and back, for feed-forward blocks that are mixtures of
// experts.
//
//   row[t, j]  = start[e] + rank of (t, j) among the pairs with e = expert[t, j]
//   sort:    xs[row[t, j]] = x[t]               back: dx[t] = sum_j dxs[row[t, j]]
//   combine: y[t] = sum_j w[t, j] ys[row[t, j]]
//            back: dys[row[t, j]] = w[t, j] dy[t],  dw[t, j] = <dy[t], ys[row[t, j]]>
//
// The route is a stable counting sort of the (token, choice) pairs, so it and all
// that follows are reproducible: a warp ranks its pairs among their expert's 32 at a
// time (lanes with the same expert find each other by votes), and the warps' and
// blocks' counts are summed in order.  Up to kOneLaunch pairs the blocks are one
// cluster, which exchanges its counts through shared memory; more take a counting
// launch over blocks of pairs before it.
//
// The copies are bound by memory, and go by token, not by sorted row: sorting
// reads a token once and writes it k times, the way back reads k rows a token
// and writes one.  A warp takes a token's (or a part of a token's) 16-byte vectors,
// several loads in flight.  Sums are fp32, over j in order, outputs rounded once.
//
// Measured (one GB300, T = 32760, D = 5120, bf16, two of 8 experts): the route 7 us,
// sorting 143 us and back 147, combining 141 us and back 239 (1007 and 1678 MB: 102 to
// 107 % of the copy rate, the last writes still in L2).  The route of 6666 pairs, 64 experts, 5.6 us
// (with the instruction that finds equal lanes in place of the votes, and the pairs
// walked twice, 9.0), of 524288, 256 experts, 12 us (28).
#include "ffn.cuh"

namespace adaln {
namespace {

constexpr int kMaxE = ADALN_MAX_EXPERTS;
constexpr int kRouteThreads = 1024, kRouteWarps = kRouteThreads / 32;
constexpr int kAhead = 16;          // rounds of a warp's pairs loaded together
constexpr int kClusterPairs = 4096; // pairs of a block in a cluster, while it may grow
constexpr int kMaxCluster = 8, kOneLaunch = kMaxCluster * kAhead * kRouteThreads;
constexpr int kBlockPairs = 8192, kMaxBlocks = 512;
static_assert(kOneLaunch == 131072, "the documented limit");
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kVecs = 4;          // vectors of a lane in a part of a row (copies)
constexpr int kPart = 32 * kVecs;

struct RouteArgs {
  const int32_t* expert;
  int32_t *row, *starts, *counts;
  int32_t* hist;  // [blocks][E], or NULL: the blocks are one cluster
  int64_t pairs, block_pairs;
  int32_t E, align, blocks;
  unsigned* status;
};

// The pairs of a warp of a block: [lo, hi).
struct Range {
  int64_t lo, hi;
};
__device__ __forceinline__ Range warp_range(const RouteArgs& a, int block, int warp) {
  const int64_t begin = block * a.block_pairs, end = min(begin + a.block_pairs, a.pairs);
  const int64_t each = ((end - begin + kRouteThreads - 1) / kRouteThreads) * 32;
  const int64_t lo = min(begin + warp * each, end);
  return {lo, min(lo + each, end)};
}

// f(n, place, expert) for a warp's pairs in order, 32 at a time (the n-th 32), kAhead of
// those loaded together; expert E for none.  What is neither an expert nor -1 is
// recorded, if `check`.
template <class F>
__device__ __forceinline__ void for_pairs(const RouteArgs& a, Range r, int lane, bool check, F f) {
  for (int64_t i0 = r.lo; i0 < r.hi; i0 += 32 * kAhead) {
    int e[kAhead];
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      const int64_t i = i0 + 32 * n + lane;
      e[n] = i < r.hi ? a.expert[i] : -1;
    }
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      if (i0 + 32 * n >= r.hi) break;
      if ((unsigned)e[n] >= (unsigned)a.E) {
        if (check && e[n] != -1) atomicOr(a.status, ADALN_DEV_EXPERT_RANGE);
        e[n] = a.E;
      }
      f(n, i0 + 32 * n + lane, e[n]);
    }
  }
}

__device__ __forceinline__ void clear_counts(const RouteArgs& a, int* count, int lane) {
  for (int e = lane; e < a.E; e += 32) count[e] = 0;
  __syncwarp();
}
// count[e] of this warp: its pairs by expert.
__device__ __forceinline__ void count_pairs(const RouteArgs& a, Range r, int* count, int lane,
                                            bool check) {
  clear_counts(a, count, lane);
  for_pairs(a, r, lane, check, [&](int, int64_t, int e) {
    if (e < a.E) atomicAdd(&count[e], 1);
  });
}

// Which lanes hold the same expert (`bits` of it): a vote for each bit.
__device__ __forceinline__ unsigned same_expert(int e, int bits) {
  unsigned same = ~0u;
  for (int b = 0; b < bits; ++b) {
    const unsigned ones = __ballot_sync(~0u, e >> b & 1);
    same &= e >> b & 1 ? ones : ~ones;
  }
  return same;
}
// The rank of this lane's pair among its expert's, next[e] the first one's of these 32.
__device__ __forceinline__ int take_rank(const RouteArgs& a, int* next, int e, int lane, int bits) {
  const unsigned same = same_expert(e, bits);
  const int rank = e < a.E ? next[e] : 0;
  __syncwarp();
  if (e < a.E && lane == __ffs(same) - 1) next[e] = rank + __popc(same);
  __syncwarp();
  return rank + __popc(same & ((1u << lane) - 1));
}

__global__ void __launch_bounds__(kRouteThreads) route_count_kernel(const __grid_constant__ RouteArgs a) {
  __shared__ int count[kRouteWarps][kMaxE];
  grid_wait();
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  count_pairs(a, warp_range(a, blockIdx.x, warp), count[warp], lane, true);
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kRouteThreads) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < kRouteWarps; ++w) n += count[w][e];
    a.hist[(int64_t)blockIdx.x * a.E + e] = n;
  }
}

__device__ __forceinline__ int ld_cluster(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

template <bool CLUSTER>
__global__ void __launch_bounds__(kRouteThreads) route_place_kernel(const __grid_constant__ RouteArgs a) {
  __shared__ int count[kRouteWarps][kMaxE];
  __shared__ int first[kMaxE], block_sum[kMaxE], sums[kMaxE / 32];
  grid_wait();
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, block = blockIdx.x;
  const Range range = warp_range(a, block, warp);
  int before = 0, total = 0;  // expert threadIdx.x's pairs in the blocks before, in all
  if (!CLUSTER) {             // from the counting launch, by several threads an expert
    constexpr int kShares = kRouteThreads / kMaxE;
    const int e = threadIdx.x % kMaxE, share = threadIdx.x / kMaxE;
    int n = 0, all = 0;
    if (e < a.E)
#pragma unroll 8
      for (int b = share; b < a.blocks; b += kShares) {
        const int v = a.hist[(int64_t)b * a.E + e];
        all += v;
        n += b < block ? v : 0;
      }
    count[share][e] = n;
    count[kShares + share][e] = all;
    __syncthreads();
    if (threadIdx.x < kMaxE)
      for (int s = 0; s < kShares; ++s) {
        before += count[s][e];
        total += count[kShares + s][e];
      }
    __syncthreads();
  }
  const int bits = 32 - __clz(a.E);
  int ranks[kAhead];  // CLUSTER: a warp's pairs are kAhead rounds at most, kept with their
                      // experts from the one walk over them
  if (CLUSTER) {
    clear_counts(a, count[warp], lane);
    for_pairs(a, range, lane, true, [&](int n, int64_t, int e) {
      ranks[n] = e << 16 | take_rank(a, count[warp], e, lane, bits);
    });
  } else {
    count_pairs(a, range, count[warp], lane, false);
  }
  __syncthreads();
  if (CLUSTER) {
    const int e = threadIdx.x;
    if (e < kMaxE) {
      int n = 0;
      if (e < a.E)
#pragma unroll
        for (int w = 0; w < kRouteWarps; ++w) n += count[w][e];
      block_sum[e] = total = n;
    }
    if (a.blocks > 1) {
      cluster_sync();
      if (e < a.E) {
        total = 0;
        const uint32_t mine = smem_addr(&block_sum[e]);
        for (int b = 0; b < a.blocks; ++b) {
          const int n = ld_cluster(map_rank(mine, b));
          before += b < block ? n : 0;
          total += n;
        }
      }
    }
  }

  // Every expert's start: a scan of the rounded-up totals.
  int padded = 0, start = 0;
  if (threadIdx.x < kMaxE) {
    const int e = threadIdx.x;
    if (e < a.E) {
      int sum = before;
#pragma unroll
      for (int w = 0; w < kRouteWarps; ++w) {  // each warp's first rank
        const int c = count[w][e];
        count[w][e] = sum;
        sum += c;
      }
    }
    padded = e < a.E ? (int)(((int64_t)total + a.align - 1) / a.align * a.align) : 0;
    start = padded;
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(~0u, start, d);
      if (lane >= d) start += v;
    }
    if (lane == 31) sums[warp] = start;
  }
  __syncthreads();
  if (threadIdx.x < kMaxE) {
    const int e = threadIdx.x;
    for (int w = 0; w < warp; ++w) start += sums[w];
    first[e] = start - padded;
    if (block == 0 && e < a.E) {
      if (e == 0) a.starts[0] = 0;
      a.starts[e + 1] = start;
      a.counts[e] = total;
    }
  }
  __syncthreads();

  if (CLUSTER) {
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      const int64_t i = range.lo + 32 * n + lane;
      if (i >= range.hi) break;
      const int e = ranks[n] >> 16;
      a.row[i] = e == a.E ? -1 : first[e] + count[warp][e] + (ranks[n] & 0xffff);
    }
  } else {
    for_pairs(a, range, lane, false, [&](int, int64_t i, int e) {
      const int rank = take_rank(a, count[warp], e, lane, bits);
      if (i < range.hi) a.row[i] = e == a.E ? -1 : first[e] + rank;
    });
  }
  if (CLUSTER && a.blocks > 1) cluster_sync();  // the others have read this block's sums
}

// ----- copies ----------------------------------------------------------------------

struct CopyArgs {
  const void* x;        // by token: x, dy
  const void* sorted;   // by sorted row: ys, dxs
  const float* weight;  // [T, k] or NULL (ones)
  const int32_t *row, *starts, *counts;
  void* to;             // xs, dys or y, dx
  float* dweight;
  int64_t T, rows;
  int32_t k, E, align, nvec;
  int32_t share, shares; // combine_bwd: choices of a token that a warp takes, warps of a token
  int32_t pad_blocks;   // blocks that write the zeros between the experts
  unsigned* status;
};

__device__ __forceinline__ const uint4* vecs_of(const void* p, int64_t row, int nvec) {
  return static_cast<const uint4*>(p) + row * nvec;
}
__device__ __forceinline__ uint4* vecs_of(void* p, int64_t row, int nvec) {
  return static_cast<uint4*>(p) + row * nvec;
}

// The sorted row of this lane's choice of token t (lanes k and up: -1), and its
// weight (one where there are none: a product with it is exact).
__device__ __forceinline__ int row_of(const CopyArgs& a, int64_t t, int lane, float* w) {
  *w = 1.0f;
  if (lane >= a.k) return -1;
  const int r = a.row[t * a.k + lane];
  if (a.weight != nullptr) *w = a.weight[t * a.k + lane];
  if (r >= 0 && r < a.rows) return r;
  if (r != -1) atomicOr(a.status, ADALN_DEV_EXPERT_RANGE);
  return -1;
}

// Zeros in the rows between an expert's last and the next one's start, which lie side
// by side.  The grid's first pad_blocks blocks do that, a few for each expert, and
// return true.  (A warp for each row that might be one cost 7 us with 64 experts.)
__device__ __forceinline__ bool clear_pads(const CopyArgs& a) {
  if ((int)blockIdx.x >= a.pad_blocks) return false;
  const int each = a.pad_blocks / a.E, e = blockIdx.x / each, share = blockIdx.x - e * each;
  const int64_t start = a.starts[e], end = min((int64_t)a.starts[e + 1], a.rows);
  const int64_t at = start + a.counts[e];
  if (start < 0 || at < start || at >= end) return true;
  const int64_t vecs = min(end - at, (int64_t)a.align - 1) * a.nvec;
  uint4* to = vecs_of(a.to, at, a.nvec);
  for (int64_t v = (int64_t)share * kThreads + threadIdx.x; v < vecs; v += (int64_t)each * kThreads)
    to[v] = make_uint4(0, 0, 0, 0);
  return true;
}

// xs[row[t, j]] = x[t]: a warp takes a part of a token's row.
__global__ void __launch_bounds__(kThreads) sort_kernel(const __grid_constant__ CopyArgs a) {
  grid_wait();
  grid_launch_dependents();
  if (clear_pads(a)) return;
  const int lane = threadIdx.x & 31, nvec = a.nvec, parts = (nvec + kPart - 1) / kPart;
  const int64_t i = (int64_t)(blockIdx.x - a.pad_blocks) * kWarps + (threadIdx.x >> 5);
  if (i >= a.T * parts) return;
  const int64_t t = i / parts;
  const int v0 = (int)(i - t * parts) * kPart + lane;
  const uint4* from = vecs_of(a.x, t, nvec);
  uint4 v[kVecs];
#pragma unroll
  for (int n = 0; n < kVecs; ++n)
    if (v0 + 32 * n < nvec) v[n] = from[v0 + 32 * n];
  float w;
  const int row = row_of(a, t, lane, &w);
  for (int j = 0; j < a.k; ++j) {
    const int r = __shfl_sync(~0u, row, j);
    if (r < 0) continue;
    uint4* to = vecs_of(a.to, r, nvec);
#pragma unroll
    for (int n = 0; n < kVecs; ++n)
      if (v0 + 32 * n < nvec) to[v0 + 32 * n] = v[n];
  }
}

// y[t] = sum_j w[t, j] ys[row[t, j]].  A warp takes parts of tokens' rows, as many
// warps as are resident, the next one's indices on their way with this one's rows: the
// same part of TOK tokens, so that few choices keep as many vectors in flight as many
// (TOK 2 with one or two choices, or 4 with one vector a lane: k <= 2).
template <class E, int V, int TOK>
__global__ void __launch_bounds__(kThreads) combine_kernel(const __grid_constant__ CopyArgs a) {
  constexpr int kIn = V == 1 ? 8 : 4, kEach = kIn / TOK;  // choices in flight, of a token
  constexpr int kLanes = 32 / TOK;                        // that hold a token's indices
  grid_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, nvec = a.nvec, parts = (nvec + 32 * V - 1) / (32 * V);
  const int64_t items = (a.T + TOK - 1) / TOK * parts, step = (int64_t)gridDim.x * kWarps;
  int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (i >= items) return;
  auto group = [&](int64_t item) -> int64_t {  // of TOK tokens
    return items <= UINT32_MAX ? (int64_t)((uint32_t)item / (uint32_t)parts) : item / parts;
  };
  auto indices = [&](int64_t g, float* w) {
    const int64_t t = g * TOK + lane / kLanes;
    if (TOK > 1 && t >= a.T) {
      *w = 1.0f;
      return -1;
    }
    return row_of(a, t, lane % kLanes, w);
  };
  float w_next;
  int64_t g_next = group(i);
  int row_next = indices(g_next, &w_next);
  for (; i < items; i += step) {
    const int64_t g = g_next;
    const int v0 = (int)(i - g * parts) * 32 * V + lane;
    const float w = w_next;
    const int row = row_next;
    if (i + step < items) {
      g_next = group(i + step);
      row_next = indices(g_next, &w_next);
    }
    float2 sum[V][E::EPV / 2] = {};
    for (int j0 = 0; j0 < a.k; j0 += kEach) {  // (once where TOK > 1)
      uint4 in[kIn][V];
      int r[kIn];
#pragma unroll
      for (int n = 0; n < kIn; ++n) {
        const int j = j0 + n % kEach;
        r[n] = __shfl_sync(~0u, row, n / kEach * kLanes + min(j, kLanes - 1));
        if (j >= a.k) r[n] = -1;
        if (r[n] < 0) continue;
        const uint4* from = vecs_of(a.sorted, r[n], nvec);
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (v0 + 32 * v < nvec) in[n][v] = from[v0 + 32 * v];
      }
#pragma unroll
      for (int n = 0; n < kIn; ++n) {
        const float wj = __shfl_sync(~0u, w, n / kEach * kLanes + min(j0 + n % kEach, kLanes - 1));
        if (r[n] >= 0) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            if (v0 + 32 * v >= nvec) continue;
            float2 f[E::EPV / 2];
            E::unpack2(in[n][v], f);
#pragma unroll
            for (int q = 0; q < E::EPV / 2; ++q)
              sum[v][q] = fma2(f[q], splat2(wj), sum[v][q]);
          }
        }
        if (n % kEach + 1 < kEach || (TOK == 1 && j0 + kEach < a.k)) continue;  // more of this token
        const int64_t t = g * TOK + n / kEach;
        if (TOK > 1 && t >= a.T) break;
        uint4* to = vecs_of(a.to, t, nvec);
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (v0 + 32 * v < nvec) {
            st_global_cs_v4(to + v0 + 32 * v, E::pack2(sum[v]));
#pragma unroll
            for (int q = 0; q < E::EPV / 2; ++q) sum[v][q] = splat2(0.0f);
          }
      }
    }
  }
}

// dys[row[t, j]] = w[t, j] dy[t] and dw[t, j] = <dy[t], ys[row[t, j]]>: a warp takes
// a.share of a token's choices, kDots at a time over the parts of its row, eight of their
// vectors in flight.
template <class E, int V>
__global__ void __launch_bounds__(kThreads) combine_bwd_kernel(const __grid_constant__ CopyArgs a) {
  constexpr int kDots = 8, kIn = 8 / V;
  grid_wait();
  grid_launch_dependents();
  if (clear_pads(a)) return;
  const int lane = threadIdx.x & 31, nvec = a.nvec, parts = (nvec + 32 * V - 1) / (32 * V);
  const int64_t i = (int64_t)(blockIdx.x - a.pad_blocks) * kWarps + (threadIdx.x >> 5);
  const int64_t t = a.shares == 1 ? i : (uint32_t)i / (uint32_t)a.shares;  // (few warps, then)
  if (t >= a.T) return;
  const int first = a.shares == 1 ? 0 : (int)(i - t * a.shares) * a.share;
  const int end = min(first + a.share, a.k);
  float w;
  const int row = row_of(a, t, lane, &w);
  const uint4* dy = vecs_of(a.x, t, nvec);
  float dw = 0.0f;
  for (int j0 = first; j0 < end; j0 += kDots) {
    float2 dot[kDots] = {};
    for (int part = 0; part < parts; ++part) {  // (the whole warp: rows and weights come from its lanes)
      const int v0 = part * 32 * V + lane;
      uint4 d[V];
#pragma unroll
      for (int n = 0; n < V; ++n)
        if (v0 + 32 * n < nvec) d[n] = dy[v0 + 32 * n];
#pragma unroll
      for (int j1 = 0; j1 < kDots; j1 += kIn) {
        if (j0 + j1 >= end) break;
        uint4 s[kIn][V];
        int r[kIn];
#pragma unroll
        for (int j = 0; j < kIn; ++j) {
          const int c = j0 + j1 + j;
          r[j] = __shfl_sync(~0u, row, min(c, 31));
          if (c >= end) r[j] = -1;
          if (r[j] < 0) continue;
          const uint4* ys = vecs_of(a.sorted, r[j], nvec);
#pragma unroll
          for (int n = 0; n < V; ++n)
            if (v0 + 32 * n < nvec) s[j][n] = ys[v0 + 32 * n];
        }
#pragma unroll
        for (int j = 0; j < kIn; ++j) {
          const float wj = __shfl_sync(~0u, w, min(j0 + j1 + j, 31));
          if (r[j] < 0) continue;
          uint4* to = vecs_of(a.to, r[j], nvec);
#pragma unroll
          for (int n = 0; n < V; ++n) {
            if (v0 + 32 * n >= nvec) continue;
            float2 f[E::EPV / 2], g[E::EPV / 2];
            E::unpack2(d[n], f);
            E::unpack2(s[j][n], g);
#pragma unroll
            for (int q = 0; q < E::EPV / 2; ++q) {
              dot[j1 + j] = fma2(f[q], g[q], dot[j1 + j]);
              f[q] = mul2(f[q], splat2(wj));
            }
            to[v0 + 32 * n] = E::pack2(f);
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kDots; ++j) {
      if (j0 + j >= end) break;
      float sum = dot[j].x + dot[j].y;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
      if (lane == j0 + j) dw = sum;
    }
  }
  if (lane >= first && lane < end) a.dweight[t * a.k + lane] = dw;
}

// ----- host side ------------------------------------------------------------------

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

cudaError_t launch(void* kernel, int64_t grid, int threads, void* args, cudaStream_t st) {
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  Shape s = {};
  s.grid = (int)grid;
  s.threads = threads;
  void* params[1] = {args};
  return traced_launch(ADALN_KERNEL_EXPERTS, st,
                       [&] { return launch_dependent(kernel, s, params, st); });
}

cudaError_t device_sms(int* sms) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e == cudaSuccess ? sm_count(dev, sms) : e;
}

int64_t rows_of(int64_t T, int32_t k, int32_t E, int32_t align) {
  const int64_t pairs = T * k, met = pairs < E ? pairs : E;
  return (pairs + met * (align - 1)) / align * align;
}

int check_route(int64_t T, int32_t k, int32_t E, int32_t align) {
  if (T < 0 || T > INT32_MAX || k < 1 || k > ADALN_MAX_TOPK || E < 1 || E > ADALN_MAX_EXPERTS ||
      align < 1 || align > ADALN_MAX_ROUTE_ALIGN)
    return ADALN_ERR_DIM;
  return rows_of(T, k, E, align) > INT32_MAX ? ADALN_ERR_DIM : ADALN_OK;
}

int64_t block_pairs_of(int64_t pairs) {
  const int64_t least = (pairs + kMaxBlocks - 1) / kMaxBlocks;
  const int64_t n = least > kBlockPairs ? least : kBlockPairs;
  return (n + kRouteThreads - 1) / kRouteThreads * kRouteThreads;
}
int blocks_of(int64_t pairs) { return (int)((pairs + block_pairs_of(pairs) - 1) / block_pairs_of(pairs)); }
size_t route_bytes(int64_t pairs, int32_t E) {
  return pairs <= kOneLaunch ? 0 : ((size_t)blocks_of(pairs) * E * 4 + 255) & ~(size_t)255;
}

int check_copy(int64_t T, int32_t k, int32_t D, adaln_dtype_t dt, int64_t rows) {
  if (dt != ADALN_F32 && dt != ADALN_BF16) return ADALN_ERR_DTYPE;
  if (T < 0 || T > INT32_MAX || k < 1 || k > ADALN_MAX_TOPK || rows < 0 || rows > INT32_MAX)
    return ADALN_ERR_DIM;
  if (D < 1 || D > ADALN_DROPOUT_MAX_D || D * (dt == ADALN_BF16 ? 2 : 4) % 16 != 0) return ADALN_ERR_DIM;
  return ADALN_OK;
}
int check_pads(int32_t E, int32_t align) {
  return E < 1 || E > ADALN_MAX_EXPERTS || align < 1 || align > ADALN_MAX_ROUTE_ALIGN ? ADALN_ERR_DIM
                                                                                      : ADALN_OK;
}
int64_t blocks_for(int64_t warps) { return (warps + kWarps - 1) / kWarps; }
int64_t parts_of(int nvec, int part) { return (nvec + part - 1) / part; }

// Blocks for an expert's rows of zeros: one for each 32 KB that they might take, at
// most eight.
int pad_blocks_of(int32_t E, int32_t align, int nvec) {
  const int64_t each = ((int64_t)(align - 1) * nvec * 16 + 32767) / 32768;
  return E * (int)(each < 8 ? each : 8);
}

CopyArgs copy_args(int64_t T, int32_t k, int32_t D, adaln_dtype_t dt, int64_t rows, const int32_t* row) {
  CopyArgs a = {};
  a.T = T, a.k = k, a.rows = rows, a.row = row;
  a.nvec = D * (dt == ADALN_BF16 ? 2 : 4) / 16;
  return a;
}

int run_copy(CopyArgs& a, void* kernel, int64_t grid, cudaStream_t st) {
  cudaError_t e = status_word(&a.status);
  if (e == cudaSuccess) e = launch(kernel, grid, kThreads, &a, st);
  return e == cudaSuccess ? ADALN_OK : launch_failed(e);
}

// 16-byte vectors of a row that a lane takes at a time: four, unless a row of so few
// would leave more than a quarter of the lanes' places empty.
int vecs_a_lane(int nvec) {
  for (int v = 4; v > 1; v /= 2)
    if (3 * parts_of(nvec, 32 * v) * 32 * v <= 4 * nvec) return v;
  return 1;
}
template <class E>
void* combine_of(int v, int tokens) {
  return v == 4   ? tokens > 1 ? (void*)combine_kernel<E, 4, 2> : (void*)combine_kernel<E, 4, 1>
         : v == 2 ? tokens > 1 ? (void*)combine_kernel<E, 2, 2> : (void*)combine_kernel<E, 2, 1>
         : tokens > 1 ? (void*)combine_kernel<E, 1, 4> : (void*)combine_kernel<E, 1, 1>;
}
template <class E>
void* combine_bwd_of(int v) {
  return v == 4   ? (void*)combine_bwd_kernel<E, 4>
         : v == 2 ? (void*)combine_bwd_kernel<E, 2>
                  : (void*)combine_bwd_kernel<E, 1>;
}

// y = the weighted (or plain) sum of each token's sorted rows.
int run_combine(const void* sorted, const float* weight, const int32_t* row, int64_t T, int32_t k,
                int32_t D, adaln_dtype_t dtype, int64_t rows, void* to, void* stream) {
  CopyArgs a = copy_args(T, k, D, dtype, rows, row);
  a.sorted = sorted, a.weight = weight, a.to = to;
  const int v = vecs_a_lane(a.nvec);
  const int64_t parts = parts_of(a.nvec, 32 * v);
  int sms = 0;
  const cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return launch_failed(e);
  const int64_t most = (int64_t)sms * (v == 4 ? 2 : 3);  // resident
  // (Several tokens to a warp only where all warps find some.)
  const int several = v == 1 ? 4 : 2;
  const int tokens = k <= 2 && T * parts >= several * most * kWarps ? several : 1;
  void* kernel = dtype == ADALN_BF16 ? combine_of<BF16>(v, tokens) : combine_of<F32>(v, tokens);
  const int64_t blocks = blocks_for((T + tokens - 1) / tokens * parts);
  return run_copy(a, kernel, blocks < most ? blocks : most, static_cast<cudaStream_t>(stream));
}

}  // namespace
}  // namespace adaln

using namespace adaln;

extern "C" {

int adaln_route_rows(int64_t T, int32_t k, int32_t E, int32_t align, int64_t* rows) {
  const int rc = check_route(T, k, E, align);
  if (rc != ADALN_OK) return rc;
  if (!rows) return ADALN_ERR_NULL;
  *rows = rows_of(T, k, E, align);
  return ADALN_OK;
}

int adaln_route_workspace_size(int64_t T, int32_t k, int32_t E, size_t* bytes) {
  const int rc = check_route(T, k, E, 1);
  if (rc != ADALN_OK) return rc;
  if (!bytes) return ADALN_ERR_NULL;
  *bytes = route_bytes(T * k, E);
  return ADALN_OK;
}

int adaln_route(const int32_t* expert, int64_t T, int32_t k, int32_t E, int32_t align, int32_t* row,
                int32_t* starts, int32_t* counts, void* workspace, size_t workspace_bytes, void* stream) {
  const int rc = check_route(T, k, E, align);
  if (rc != ADALN_OK) return rc;
  const int64_t pairs = T * k;
  const size_t need = route_bytes(pairs, E);
  if (!starts || !counts || (T > 0 && (!expert || !row)) || (need > 0 && !workspace)) return ADALN_ERR_NULL;
  if (!aligned(starts, 4) || !aligned(counts, 4) || !aligned(expert, 4) || !aligned(row, 4) ||
      (need > 0 && !aligned(workspace, 16)))
    return ADALN_ERR_ALIGN;
  if (workspace_bytes < need) return ADALN_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  RouteArgs a = {};
  a.expert = expert, a.row = row, a.starts = starts, a.counts = counts;
  a.pairs = pairs, a.E = E, a.align = align;
  cudaError_t e = status_word(&a.status);
  if (need > 0) {
    a.blocks = blocks_of(pairs);
    a.block_pairs = block_pairs_of(pairs);
    a.hist = static_cast<int32_t*>(workspace);
    if (e == cudaSuccess) e = launch((void*)route_count_kernel, a.blocks, kRouteThreads, &a, st);
    if (e == cudaSuccess) e = launch((void*)route_place_kernel<false>, a.blocks, kRouteThreads, &a, st);
  } else {
    const int64_t blocks = (pairs + kClusterPairs - 1) / kClusterPairs;
    a.blocks = (int)(blocks < 1 ? 1 : blocks < kMaxCluster ? blocks : kMaxCluster);
    a.block_pairs = (pairs + a.blocks - 1) / a.blocks;
    void* params[1] = {&a};
    if (e == cudaSuccess)
      e = traced_launch(ADALN_KERNEL_EXPERTS, st, [&] {
        return launch_cluster((void*)route_place_kernel<true>, a.blocks, kRouteThreads, 0, a.blocks, params, st);
      });
  }
  return e == cudaSuccess ? ADALN_OK : launch_failed(e);
}

int adaln_expert_sort_fwd(const void* x, const int32_t* row, const int32_t* starts, const int32_t* counts,
                          int64_t T, int32_t k, int32_t E, int32_t align, int32_t D, adaln_dtype_t dtype,
                          int64_t rows, void* xs, void* stream) {
  int rc = check_copy(T, k, D, dtype, rows);
  if (rc == ADALN_OK) rc = check_pads(E, align);
  if (rc != ADALN_OK) return rc;
  if (T == 0) return ADALN_OK;
  if (!x || !row || !starts || !counts || !xs) return ADALN_ERR_NULL;
  if (!aligned(x, 16) || !aligned(xs, 16) || !aligned(row, 4) || !aligned(starts, 4) || !aligned(counts, 4))
    return ADALN_ERR_ALIGN;
  CopyArgs a = copy_args(T, k, D, dtype, rows, row);
  a.x = x, a.starts = starts, a.counts = counts, a.E = E, a.align = align, a.to = xs;
  a.pad_blocks = pad_blocks_of(E, align, a.nvec);
  return run_copy(a, (void*)sort_kernel, a.pad_blocks + blocks_for(T * parts_of(a.nvec, kPart)),
                  static_cast<cudaStream_t>(stream));
}

int adaln_expert_sort_bwd(const void* dxs, const int32_t* row, int64_t T, int32_t k, int32_t D,
                          adaln_dtype_t dtype, int64_t rows, void* dx, void* stream) {
  const int rc = check_copy(T, k, D, dtype, rows);
  if (rc != ADALN_OK) return rc;
  if (T == 0) return ADALN_OK;
  if (!dxs || !row || !dx) return ADALN_ERR_NULL;
  if (!aligned(dxs, 16) || !aligned(dx, 16) || !aligned(row, 4)) return ADALN_ERR_ALIGN;
  return run_combine(dxs, nullptr, row, T, k, D, dtype, rows, dx, stream);
}

int adaln_expert_combine_fwd(const void* ys, const float* weight, const int32_t* row, int64_t T, int32_t k,
                             int32_t D, adaln_dtype_t dtype, int64_t rows, void* y, void* stream) {
  const int rc = check_copy(T, k, D, dtype, rows);
  if (rc != ADALN_OK) return rc;
  if (T == 0) return ADALN_OK;
  if (!ys || !weight || !row || !y) return ADALN_ERR_NULL;
  if (!aligned(ys, 16) || !aligned(y, 16) || !aligned(weight, 4) || !aligned(row, 4)) return ADALN_ERR_ALIGN;
  return run_combine(ys, weight, row, T, k, D, dtype, rows, y, stream);
}

int adaln_expert_combine_bwd(const void* dy, const void* ys, const float* weight, const int32_t* row,
                             const int32_t* starts, const int32_t* counts, int64_t T, int32_t k, int32_t E,
                             int32_t align, int32_t D, adaln_dtype_t dtype, int64_t rows, void* dys,
                             float* dweight, void* stream) {
  int rc = check_copy(T, k, D, dtype, rows);
  if (rc == ADALN_OK) rc = check_pads(E, align);
  if (rc != ADALN_OK) return rc;
  if (T == 0) return ADALN_OK;
  if (!dy || !ys || !weight || !row || !starts || !counts || !dys || !dweight) return ADALN_ERR_NULL;
  if (!aligned(dy, 16) || !aligned(ys, 16) || !aligned(dys, 16) || !aligned(weight, 4) || !aligned(row, 4) ||
      !aligned(starts, 4) || !aligned(counts, 4) || !aligned(dweight, 4))
    return ADALN_ERR_ALIGN;
  CopyArgs a = copy_args(T, k, D, dtype, rows, row);
  a.x = dy, a.sorted = ys, a.weight = weight, a.starts = starts, a.counts = counts;
  a.E = E, a.align = align, a.to = dys, a.dweight = dweight;
  a.pad_blocks = pad_blocks_of(E, align, a.nvec);
  const int v = vecs_a_lane(a.nvec);
  void* kernel = dtype == ADALN_BF16 ? combine_bwd_of<BF16>(v) : combine_bwd_of<F32>(v);
  // All of a token's choices to a warp, so that dy is read once, unless that leaves an SM
  // with fewer than 16 warps.
  int sms = 0;
  const cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return launch_failed(e);
  a.share = k;
  while (a.share > 1 && T * ((k + a.share - 1) / a.share) < (int64_t)sms * 16) a.share = (a.share + 1) / 2;
  a.shares = (k + a.share - 1) / a.share;
  return run_copy(a, kernel, a.pad_blocks + blocks_for(T * a.shares), static_cast<cudaStream_t>(stream));
}

}  // extern "C"
