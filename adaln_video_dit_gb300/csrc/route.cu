// Tokens sorted by expert and back, for feed-forward blocks that are mixtures of
// experts.
//
//   row[t, j]  = start[e] + rank of (t, j) among the pairs with e = expert[t, j]
//   sort:    xs[row[t, j]] = x[t]               back: dx[t] = sum_j dxs[row[t, j]]
//   combine: y[t] = sum_j w[t, j] ys[row[t, j]]
//            back: dys[row[t, j]] = w[t, j] dy[t],  dw[t, j] = <dy[t], ys[row[t, j]]>
//
// The route is a stable counting sort of the (token, choice) pairs, so it and all
// that follows are reproducible: a warp counts its pairs by expert 32 at a time
// (lanes with the same expert find each other, the lowest adds their number), the
// warps' and blocks' counts are summed in order, and a second walk over the same
// pairs gives each its place.  Up to kOneBlock pairs one block does it in one
// launch; more take a counting launch over blocks of pairs before it.
//
// The copies are bound by memory, and go by token, not by sorted row: sorting
// reads a token once and writes it k times, the way back reads k rows a token
// and writes one.  A warp takes a token's (or a part of a token's) 16-byte vectors,
// several loads in flight.  Sums are fp32, over j in order, outputs rounded once.
#include "common.cuh"
#include "internal.h"

namespace adaln {
namespace {

constexpr int kMaxE = ADALN_MAX_EXPERTS;
constexpr int kRouteThreads = 1024, kRouteWarps = kRouteThreads / 32;
constexpr int kOneBlock = 16384;  // pairs that one block routes by itself
constexpr int kBlockPairs = 8192, kMaxBlocks = 256;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kVecs = 4;          // vectors of a lane in a part of a row (copies)
constexpr int kPart = 32 * kVecs;

struct RouteArgs {
  const int32_t* expert;
  int32_t *row, *starts, *counts;
  int32_t* hist;  // [blocks][E], or NULL with one block
  int64_t pairs, block_pairs;
  int32_t E, align, blocks;
  unsigned* status;
};

// A pair's expert, or -1; what is neither is recorded.
__device__ __forceinline__ int expert_of(const RouteArgs& a, int64_t i, int64_t end, bool check) {
  if (i >= end) return -1;
  const int e = a.expert[i];
  if ((unsigned)e < (unsigned)a.E) return e;
  if (check && e != -1) atomicOr(a.status, ADALN_DEV_EXPERT_RANGE);
  return -1;
}

// The pairs of warp w of a block: [lo, hi).
struct Range {
  int64_t lo, hi;
};
__device__ __forceinline__ Range warp_range(const RouteArgs& a, int block, int warp) {
  const int64_t begin = block * a.block_pairs, end = min(begin + a.block_pairs, a.pairs);
  const int64_t each = ((end - begin + kRouteThreads - 1) / kRouteThreads) * 32;
  const int64_t lo = min(begin + warp * each, end);
  return {lo, min(lo + each, end)};
}

// count[e] of this warp: its pairs by expert.
__device__ __forceinline__ void count_pairs(const RouteArgs& a, Range r, int* count, int lane,
                                            bool check) {
  for (int e = lane; e < a.E; e += 32) count[e] = 0;
  __syncwarp();
  for (int64_t i = r.lo; i < r.hi; i += 32) {
    const int e = expert_of(a, i + lane, r.hi, check);
    const unsigned same = __match_any_sync(~0u, e);
    if (e >= 0 && lane == __ffs(same) - 1) count[e] += __popc(same);
    __syncwarp();
  }
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
    for (int w = 0; w < kRouteWarps; ++w) n += count[w][e];
    a.hist[(int64_t)blockIdx.x * a.E + e] = n;
  }
}

__global__ void __launch_bounds__(kRouteThreads) route_place_kernel(const __grid_constant__ RouteArgs a) {
  __shared__ int count[kRouteWarps][kMaxE];
  __shared__ int before[kMaxE], total[kMaxE], sums[kMaxE / 32];
  grid_wait();
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, block = blockIdx.x;
  const Range range = warp_range(a, block, warp);
  if (a.hist != nullptr) {  // all blocks' counts, by kRouteThreads / kMaxE threads an expert
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
    if (threadIdx.x < kMaxE) {
      n = all = 0;
      for (int s = 0; s < kShares; ++s) {
        n += count[s][e];
        all += count[kShares + s][e];
      }
      before[e] = n;
      total[e] = all;
    }
    __syncthreads();
  }
  count_pairs(a, range, count[warp], lane, a.hist == nullptr);
  __syncthreads();

  // Every expert's start: a scan of the rounded-up totals.
  int n = 0, padded = 0, start = 0;
  if (threadIdx.x < kMaxE) {
    const int e = threadIdx.x;
    int sum = a.hist != nullptr ? before[e] : 0;
    if (e < a.E)
      for (int w = 0; w < kRouteWarps; ++w) {  // each warp's first rank
        const int c = count[w][e];
        count[w][e] = sum;
        sum += c;
      }
    n = e >= a.E ? 0 : a.hist != nullptr ? total[e] : sum;
    padded = (int)((int64_t)(n + a.align - 1) / a.align * a.align);
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
    before[e] = start - padded;
    if (block == 0 && e < a.E) {
      if (e == 0) a.starts[0] = 0;
      a.starts[e + 1] = start;
      a.counts[e] = n;
    }
  }
  __syncthreads();

  int* next = count[warp];
  for (int64_t i = range.lo; i < range.hi; i += 32) {
    const int e = expert_of(a, i + lane, range.hi, false);
    const unsigned same = __match_any_sync(~0u, e);
    const int first = e >= 0 ? next[e] : 0;
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) next[e] = first + __popc(same);
    __syncwarp();
    if (i + lane < range.hi)
      a.row[i + lane] = e < 0 ? -1 : before[e] + first + __popc(same & ((1u << lane) - 1));
  }
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
  unsigned* status;
};

__device__ __forceinline__ const uint4* vecs_of(const void* p, int64_t row, int nvec) {
  return static_cast<const uint4*>(p) + row * nvec;
}
__device__ __forceinline__ uint4* vecs_of(void* p, int64_t row, int nvec) {
  return static_cast<uint4*>(p) + row * nvec;
}

// The sorted row of this lane's choice of token t (lanes k and up: -1), and its
// weight.
__device__ __forceinline__ int row_of(const CopyArgs& a, int64_t t, int lane, float* w) {
  *w = 0.0f;
  if (lane >= a.k) return -1;
  const int r = a.row[t * a.k + lane];
  if (a.weight != nullptr) *w = a.weight[t * a.k + lane];
  if (r >= 0 && r < a.rows) return r;
  if (r != -1) atomicOr(a.status, ADALN_DEV_EXPERT_RANGE);
  return -1;
}

// Zeros in the rows between an expert's last and the next one's start: `i` counts
// (expert, row past its last, part of the row).
__device__ __forceinline__ void clear_pad(const CopyArgs& a, int64_t i, int parts, int lane) {
  const int64_t r = i / parts;
  const int part = (int)(i - r * parts);
  const int e = (int)(r / a.align);
  if (e >= a.E) return;
  const int64_t at = (int64_t)a.starts[e] + a.counts[e] + (r - (int64_t)e * a.align);
  if (at < 0 || at >= a.starts[e + 1] || at >= a.rows) return;
  uint4* to = vecs_of(a.to, at, a.nvec);
  for (int v = part * kPart + lane; v < min((part + 1) * kPart, a.nvec); v += 32)
    to[v] = make_uint4(0, 0, 0, 0);
}

// xs[row[t, j]] = x[t]: a warp takes a part of a token's row.
__global__ void __launch_bounds__(kThreads) sort_kernel(const __grid_constant__ CopyArgs a) {
  grid_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, nvec = a.nvec, parts = (nvec + kPart - 1) / kPart;
  const int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (i >= a.T * parts) {
    clear_pad(a, i - a.T * parts, parts, lane);
    return;
  }
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

// y[t] = sum_j w[t, j] ys[row[t, j]].
template <class E, bool WEIGHT>
__global__ void __launch_bounds__(kThreads) combine_kernel(const __grid_constant__ CopyArgs a) {
  constexpr int V = 2, kIn = 4;  // vectors a lane, choices in flight
  grid_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, nvec = a.nvec, parts = (nvec + 32 * V - 1) / (32 * V);
  const int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (i >= a.T * parts) return;
  const int64_t t = i / parts;
  const int v0 = (int)(i - t * parts) * 32 * V + lane;
  float w;
  const int row = row_of(a, t, lane, &w);
  float2 sum[V][E::EPV / 2] = {};
  for (int j0 = 0; j0 < a.k; j0 += kIn) {
    uint4 in[kIn][V];
    int r[kIn];
#pragma unroll
    for (int j = 0; j < kIn; ++j) {
      r[j] = __shfl_sync(~0u, row, min(j0 + j, 31));
      if (j0 + j >= a.k) r[j] = -1;
      if (r[j] < 0) continue;
      const uint4* from = vecs_of(a.sorted, r[j], nvec);
#pragma unroll
      for (int n = 0; n < V; ++n)
        if (v0 + 32 * n < nvec) in[j][n] = from[v0 + 32 * n];
    }
#pragma unroll
    for (int j = 0; j < kIn; ++j) {
      const float wj = __shfl_sync(~0u, w, min(j0 + j, 31));
      if (r[j] < 0) continue;
#pragma unroll
      for (int n = 0; n < V; ++n) {
        if (v0 + 32 * n >= nvec) continue;
        float2 f[E::EPV / 2];
        E::unpack2(in[j][n], f);
#pragma unroll
        for (int q = 0; q < E::EPV / 2; ++q)
          sum[n][q] = WEIGHT ? fma2(f[q], splat2(wj), sum[n][q]) : add2(f[q], sum[n][q]);
      }
    }
  }
  uint4* to = vecs_of(a.to, t, nvec);
#pragma unroll
  for (int n = 0; n < V; ++n)
    if (v0 + 32 * n < nvec) st_global_cs_v4(to + v0 + 32 * n, E::pack2(sum[n]));
}

// dys[row[t, j]] = w[t, j] dy[t] and dw[t, j] = <dy[t], ys[row[t, j]]>: a warp a token.
template <class E>
__global__ void __launch_bounds__(kThreads) combine_bwd_kernel(const __grid_constant__ CopyArgs a) {
  grid_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, nvec = a.nvec, parts = (nvec + kPart - 1) / kPart;
  const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= a.T) {
    clear_pad(a, t - a.T, parts, lane);
    return;
  }
  float w;
  const int row = row_of(a, t, lane, &w);
  const uint4* dy = vecs_of(a.x, t, nvec);
  float dw = 0.0f;
  for (int j = 0; j < a.k; ++j) {
    const int r = __shfl_sync(~0u, row, j);
    const float wj = __shfl_sync(~0u, w, j);
    if (r < 0) continue;
    const uint4* ys = vecs_of(a.sorted, r, nvec);
    uint4* to = vecs_of(a.to, r, nvec);
    float2 dot = splat2(0.0f);
    for (int v0 = lane; v0 < nvec; v0 += kPart) {
      uint4 d[kVecs], s[kVecs];
#pragma unroll
      for (int n = 0; n < kVecs; ++n)
        if (v0 + 32 * n < nvec) {
          s[n] = ys[v0 + 32 * n];
          d[n] = dy[v0 + 32 * n];
        }
#pragma unroll
      for (int n = 0; n < kVecs; ++n) {
        if (v0 + 32 * n >= nvec) continue;
        float2 f[E::EPV / 2], g[E::EPV / 2];
        E::unpack2(d[n], f);
        E::unpack2(s[n], g);
#pragma unroll
        for (int q = 0; q < E::EPV / 2; ++q) {
          dot = fma2(f[q], g[q], dot);
          f[q] = mul2(f[q], splat2(wj));
        }
        to[v0 + 32 * n] = E::pack2(f);
      }
    }
    float sum = dot.x + dot.y;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
    if (lane == j) dw = sum;
  }
  if (lane < a.k) a.dweight[t * a.k + lane] = dw;
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
int blocks_of(int64_t pairs) {
  return pairs <= kOneBlock ? 1 : (int)((pairs + block_pairs_of(pairs) - 1) / block_pairs_of(pairs));
}
size_t route_bytes(int64_t pairs, int32_t E) {
  return pairs <= kOneBlock ? 0 : ((size_t)blocks_of(pairs) * E * 4 + 255) & ~(size_t)255;
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

// y = the weighted (or plain) sum of each token's sorted rows.
int run_combine(const void* sorted, const float* weight, const int32_t* row, int64_t T, int32_t k,
                int32_t D, adaln_dtype_t dtype, int64_t rows, void* to, void* stream) {
  CopyArgs a = copy_args(T, k, D, dtype, rows, row);
  a.sorted = sorted, a.weight = weight, a.to = to;
  void* kernel = dtype == ADALN_BF16
                     ? weight ? (void*)combine_kernel<BF16, true> : (void*)combine_kernel<BF16, false>
                     : weight ? (void*)combine_kernel<F32, true> : (void*)combine_kernel<F32, false>;
  return run_copy(a, kernel, blocks_for(T * parts_of(a.nvec, 64)), static_cast<cudaStream_t>(stream));
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
  a.blocks = blocks_of(pairs);
  a.block_pairs = a.blocks == 1 ? kOneBlock : block_pairs_of(pairs);
  a.hist = need > 0 ? static_cast<int32_t*>(workspace) : nullptr;
  cudaError_t e = status_word(&a.status);
  if (e == cudaSuccess && need > 0)
    e = launch((void*)route_count_kernel, a.blocks, kRouteThreads, &a, st);
  if (e == cudaSuccess) e = launch((void*)route_place_kernel, a.blocks, kRouteThreads, &a, st);
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
  const int64_t pads = (int64_t)E * (align - 1) > 0 ? (int64_t)E * align : 0;
  return run_copy(a, (void*)sort_kernel, blocks_for((T + pads) * parts_of(a.nvec, kPart)),
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
  const int64_t pads = (int64_t)E * (align - 1) > 0 ? (int64_t)E * align : 0;
  void* kernel = dtype == ADALN_BF16 ? (void*)combine_bwd_kernel<BF16> : (void*)combine_bwd_kernel<F32>;
  return run_copy(a, kernel, blocks_for(T + pads * parts_of(a.nvec, kPart)),
                  static_cast<cudaStream_t>(stream));
}

}  // extern "C"
