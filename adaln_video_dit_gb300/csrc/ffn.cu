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
#include <cmath>
#include <mutex>

#include "ffn.cuh"

namespace adaln {
namespace {

// Epilogues: the product alone; the gate; the gate, saving g and u; the
// gate's gradient.
enum { kPlain = 0, kGate = 1, kGateSave = 2, kGateBwd = 3, kKinds = 4 };

constexpr int kBK = 64;                    // k values of a stage
constexpr int kTileBytes = 128 * kBK * 2;  // one CTA's share of an operand stage
constexpr int kStageBytes = 2 * kTileBytes;
// Tile of a CTA pair: 256 rows x 2 w columns, w the rows of B that each CTA
// stages (128, 96 or 64: choose_tiling); kGate: w columns of g and w of u.
constexpr int kTM = 256, kAccCols = 256;
constexpr int kEpiWarps = 8;
constexpr int kThreads = (2 + kEpiWarps) * 32;
// Outputs leave through blocks of 32 rows x 32 columns in shared memory, copied
// by TMA: a lane holds a row of its accumulator, and 32 lanes writing 16 bytes
// each to 32 rows of global memory cost a cache-line lookup per lane (the stores
// of g, u and h alone took half as long again as the products at D = 1536).
constexpr int kBlock = 32 * 32 * 2;
// A warp's shared memory: dg, du and h for kGateBwd, two blocks in turn for the
// others; and the ring stages that fit beside it.
ADALN_HD constexpr int staging_bytes(int kind) { return (kind == kGateBwd ? 3 : 2) * kBlock; }
ADALN_HD constexpr int stages_of(int kind) { return kind == kGateBwd ? 5 : 6; }
constexpr int smem_of(int kind) {
  return 1024 + stages_of(kind) * kStageBytes + kEpiWarps * staging_bytes(kind) + 256;
}
constexpr int kGroupM = 8;                 // tile rows walked together (L2 reuse)
constexpr int kMaxProblems = 4;

// C[M, N] = sum over its K segments of A B.
struct Dims {        // what the roles of a CTA read of a problem
  int M, N;
  int kb0, kb;         // k blocks of segment 0, of both
  int w;               // rows of B a CTA stages
  int tiles_m, tiles_n, splits;
  int first;           // first unit of the problem
  int a_mn, b_mn;      // operand layouts
};
struct Problem {
  CUtensorMap a[2], b[2];
  CUtensorMap out;     // bf16 [M, N]
  float* partial;      // fp32 [splits][M][N] when splits > 1
  Dims s;
};

struct GemmArgs {
  Problem p[kMaxProblems];
  int problems, units;
  // Order of the units (unit_index): the first `lead` are long ones, each worth
  // `worth` of the others.
  int lead, worth;
  // Gate epilogues ([T, F] each).
  CUtensorMap h, dg, du;
  uint4* saved;
  unsigned* status;
};

struct Unit {
  int i;           // problem
  int m, n;        // tile
  int k0, k1;      // k blocks
  int split;
};

// Unit i of CTA pair c out of n, or one past the last unit.  All pairs walk the
// long units round-robin; those that a last, partial round of them leaves free
// take `worth` shorter ones each meanwhile; then all walk the rest.  (Unit costs
// are known, so this is the order in which a queue would hand them out.)
__device__ __forceinline__ int unit_index(int c, int i, int n, int lead, int worth) {
  const int extra = lead % n, first = lead / n + (c < extra);
  if (i < first) return i * n + c;
  i -= first;
  const int free = n - extra, rest = lead + worth * free;
  if (c < extra) return rest + i * n + free + c;
  return i < worth ? lead + i * free + c - extra : rest + (i - worth) * n + c - extra;
}

// `shapes` is the problems' copy in shared memory (reads of the kernel's
// parameters with an index cost several hundred cycles each).
__device__ __forceinline__ Unit unit_of(const Dims* shapes, int problems, int u) {
  Unit r;
  r.i = 0;
  while (r.i + 1 < problems && u >= shapes[r.i + 1].first) ++r.i;
  const Dims& s = shapes[r.i];
  u -= s.first;
  r.split = 0;
  int tile = u;
  r.k0 = 0;
  r.k1 = s.kb;
  if (s.splits > 1) {
    tile = u / s.splits;
    r.split = u - tile * s.splits;
    r.k0 = (int)((int64_t)s.kb * r.split / s.splits);
    r.k1 = (int)((int64_t)s.kb * (r.split + 1) / s.splits);
  }
  const int per_group = kGroupM * s.tiles_n;
  const int group = tile / per_group, in = tile - group * per_group;
  const int rows = min(kGroupM, s.tiles_m - group * kGroupM);
  r.n = in / rows;
  r.m = group * kGroupM + in - r.n * rows;
  return r;
}

// This lane's row of 32 values, as 16 words of bf16 pairs, into a block (rows
// of 64 bytes, swizzled as a tensor map of that width has them).
__device__ __forceinline__ void put_row(uint32_t block, int lane, const uint32_t (&w)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    st_shared_v4(block + lane * 64 + ((i ^ (lane >> 1 & 3)) << 4), w[4 * i], w[4 * i + 1],
                 w[4 * i + 2], w[4 * i + 3]);
}

// Where block (row0 / 32, col / 32) of the saved g and u starts, for this lane.
__device__ __forceinline__ uint4* saved_at(uint4* saved, int row0, int col, int N, int lane) {
  return saved + ((int64_t)(row0 >> 5) * ((N + 31) >> 5) + (col >> 5)) * (kSavedBlock / 16) + lane;
}

// 32 fp32 values of a row as their upper 16 bits and their next 8.
__device__ __forceinline__ void save_row(uint4* to, const uint32_t (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    st_global_cs_v4(to + 32 * i, make_uint4(__byte_perm(v[8 * i], v[8 * i + 1], 0x7632),
                                            __byte_perm(v[8 * i + 2], v[8 * i + 3], 0x7632),
                                            __byte_perm(v[8 * i + 4], v[8 * i + 5], 0x7632),
                                            __byte_perm(v[8 * i + 6], v[8 * i + 7], 0x7632)));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t* x = &v[16 * i + 4 * j];
      b[j] = __byte_perm(__byte_perm(x[0], x[1], 0x51), __byte_perm(x[2], x[3], 0x51), 0x5410);
    }
    st_global_cs_v4(to + 32 * (4 + i), make_uint4(b[0], b[1], b[2], b[3]));
  }
}
// And back: values 2 i and 2 i + 1 (i = 0..3) from their word of upper halves and
// from the four next bytes that they are the lower (i even) or upper two of.
// (The lowest byte, which was not kept, repeats the one before it: one
// instruction a value.)
__device__ __forceinline__ float2 saved_pair(uint32_t w, uint32_t b, int i) {
  return i % 2 ? make_float2(__uint_as_float(__byte_perm(w, b, 0x1066)),
                             __uint_as_float(__byte_perm(w, b, 0x3277)))
               : make_float2(__uint_as_float(__byte_perm(w, b, 0x1044)),
                             __uint_as_float(__byte_perm(w, b, 0x3255)));
}

// ----- epilogues: one warp's 32 rows x every other 32 of the tile's columns -----------------
// `row0` is the warp's first row of the output, `half` which ones, `acc`
// its lanes of the accumulator, `buf` its staging memory.

__device__ __forceinline__ void epilogue_plain(const Problem& p, const Dims& s, const Unit& u,
                                               uint32_t acc, int row0, int half, uint32_t buf,
                                               int lane, int& turn) {
  const int M = s.M, N = s.N, splits = s.splits, chunks = s.w / 16;
#pragma unroll 1
  for (int c = half; c < chunks; c += 2) {
    const int col = u.n * 2 * s.w + c * 32;
    if (col >= N) break;
    __syncwarp();
    uint32_t r[32];
    tmem_ld32(acc + c * 32, r);
    tc_wait_ld();
    if (splits > 1) {
      const int left = row0 + lane < M ? N - col : 0;  // columns of this row to write
      float4* o = reinterpret_cast<float4*>(p.partial +
                                            ((int64_t)u.split * M + row0 + lane) * N + col);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (4 * i < left)
          o[i] = make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]),
                             __uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3]));
    } else {
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i)
        w[i] = pack_bf16(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
      const uint32_t block = buf + turn * kBlock;
      turn ^= 1;
      bulk_wait_read<1>();  // the copy before the last one used this block
      __syncwarp();
      put_row(block, lane, w);
      fence_async_shared();
      __syncwarp();
      if (elect_one()) {
        if (row0 < M) tma_store(&p.out, col, row0, block);
        bulk_commit();
      }
    }
  }
}

template <int ACT, bool SAVE>
__device__ __forceinline__ void epilogue_gate(const GemmArgs& a, const Dims& s, const Unit& u,
                                              uint32_t acc, int row0, int half, uint32_t buf,
                                              int lane, int& turn) {
  const int M = s.M, N = s.N, w_cols = s.w;
#pragma unroll 1
  for (int c = half; c < w_cols / 32; c += 2) {
    const int col = u.n * w_cols + c * 32;
    if (col >= N) break;
    __syncwarp();
    uint32_t g[32], v[32];
    tmem_ld32(acc + c * 32, g);
    tmem_ld32(acc + w_cols + c * 32, v);
    tc_wait_ld();
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 x = make_float2(__uint_as_float(g[2 * i]), __uint_as_float(g[2 * i + 1]));
      float2 p, d;
      gate<ACT>(x, p, d);
      const float2 h = mul2(mul2(x, p), make_float2(__uint_as_float(v[2 * i]),
                                                    __uint_as_float(v[2 * i + 1])));
      w[i] = pack_bf16(h.x, h.y);
    }
    const uint32_t block = buf + turn * kBlock;
    turn ^= 1;
    bulk_wait_read<1>();  // the copy before the last one used this block
    __syncwarp();
    put_row(block, lane, w);
    fence_async_shared();
    __syncwarp();
    if (elect_one()) {
      if (row0 < M) tma_store(&a.h, col, row0, block);
      bulk_commit();
    }
    if (SAVE && row0 < M) {
      uint4* to = saved_at(a.saved, row0, col, N, lane);
      save_row(to, g);
      save_row(to + 32 * (kSavedVecs / 2), v);
    }
  }
}

// The saved values of one chunk, a lane's twelve vectors.
struct SavedRow {
  uint4 v[kSavedVecs];
  __device__ __forceinline__ void load(const uint4* p, int i) {
    if (p != nullptr) v[i] = __ldcs(p + 32 * i);
  }
};

// One chunk of the gate's gradient: dh from the accumulator with g and u from
// `in`, which takes the next chunk's values (at `next`, or none) as soon as
// its own are used.
template <int ACT>
__device__ __forceinline__ void chunk_gate_bwd(const GemmArgs& a, uint32_t acc, int col, int row0,
                                               int M, uint32_t buf, int lane, SavedRow& in,
                                               const uint4* next) {
  uint32_t r[32], wg[16], wu[16], wh[16];
  __syncwarp();
  tmem_ld32(acc, r);
  tc_wait_ld();
#pragma unroll
  for (int j = 0; j < 4; ++j) {  // 8 columns
    const uint4 gb = in.v[4 + j / 2], ub = in.v[10 + j / 2];
    const uint32_t g0 = j % 2 ? gb.z : gb.x, g1 = j % 2 ? gb.w : gb.y;
    const uint32_t u0 = j % 2 ? ub.z : ub.x, u1 = j % 2 ? ub.w : ub.y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 &gw = in.v[j], &uw = in.v[6 + j];
      const float2 x = saved_pair(i == 0 ? gw.x : i == 1 ? gw.y : i == 2 ? gw.z : gw.w, i < 2 ? g0 : g1, i);
      const float2 w = saved_pair(i == 0 ? uw.x : i == 1 ? uw.y : i == 2 ? uw.z : uw.w, i < 2 ? u0 : u1, i);
      const float2 dh = make_float2(__uint_as_float(r[8 * j + 2 * i]),
                                    __uint_as_float(r[8 * j + 2 * i + 1]));
      float2 p, d;
      gate<ACT>(x, p, d);
      const float2 act = mul2(x, p);
      const float2 dg = mul2(mul2(dh, w), d), du = mul2(dh, act), h = mul2(act, w);
      wg[4 * j + i] = pack_bf16(dg.x, dg.y);
      wu[4 * j + i] = pack_bf16(du.x, du.y);
      wh[4 * j + i] = pack_bf16(h.x, h.y);
    }
    in.load(next, j);
    in.load(next, 6 + j);
    if (j % 2) {
      in.load(next, 4 + j / 2);
      in.load(next, 10 + j / 2);
    }
  }
  bulk_wait_read<0>();  // the previous chunk's copies used these blocks
  __syncwarp();
  put_row(buf, lane, wg);
  put_row(buf + kBlock, lane, wu);
  put_row(buf + 2 * kBlock, lane, wh);
  fence_async_shared();
  __syncwarp();
  if (elect_one()) {
    if (row0 < M) {
      tma_store(&a.dg, col, row0, buf);
      tma_store(&a.du, col, row0, buf + kBlock);
      tma_store(&a.h, col, row0, buf + 2 * kBlock);
    }
    bulk_commit();
  }
}

template <int KIND, int ACT>
__global__ void __launch_bounds__(kThreads, 1)
    ffn_gemm_kernel(const __grid_constant__ GemmArgs a) {
  constexpr int kStages = stages_of(KIND);
  constexpr bool kIsGate = KIND == kGate || KIND == kGateSave;
  extern __shared__ unsigned char smem_raw[];
  __shared__ Dims shapes[kMaxProblems];
  const uint32_t ring = (smem_addr(smem_raw) + 1023) & ~1023u;
  const uint32_t staging = ring + kStages * kStageBytes;
  const uint32_t bars = staging + kEpiWarps * staging_bytes(KIND);
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (kStages + s); };
  auto acc_full = [&](int i) { return bars + 8 * (2 * kStages + i); };
  auto acc_empty = [&](int i) { return bars + 8 * (2 * kStages + 2 + i); };
  const uint32_t drain = bars + 8 * (2 * kStages + 4);
  const uint32_t tmem_ptr = bars + 8 * (2 * kStages + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(
      smem_raw + (bars - smem_addr(smem_raw)) + 8 * (2 * kStages + 6));

  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = blockIdx.x & 1;  // within the pair
  const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full(i), 1);
      mbar_init(acc_empty(i), 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  // (Constant while the previous kernel runs: fetched before the wait for it.)
  if (threadIdx.x >= 64 && threadIdx.x < 64 + a.problems) {
    const Problem& p = a.p[threadIdx.x - 64];
    prefetch_map(&p.a[0]);
    prefetch_map(&p.b[kIsGate ? (int)rank : 0]);
  }
  if (threadIdx.x >= 32 && threadIdx.x < 32 + kMaxProblems)
    shapes[threadIdx.x - 32] = a.p[threadIdx.x - 32].s;
  if (warp == 2) tmem_alloc<2>(tmem_ptr, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tmem_ptr) : "memory");

  grid_wait();
  grid_launch_dependents();

  const int units = a.units, problems = a.problems;
  const int lead = a.lead, worth = a.worth;
  auto index = [&](int i) { return unit_index(cluster, i, clusters, lead, worth); };
  auto unit = [&](int ui) { return unit_of(shapes, problems, min(ui, units - 1)); };
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (mbar_wait_spin(bar, parity, abort_flag)) return true;
    *abort_flag = 1;
    atomicOr(a.status, ADALN_DEV_TIMEOUT);
    return false;
  };

  if (warp == 0) {
    // Producer: this CTA's 128 rows of A and of B, a stage at a time.
    int s = 0;
    uint32_t parity = 0;
    bool ok = true;
    int ui = index(0);
    Unit next = unit(ui);
    for (int i = 1; ok && ui < units; ++i) {
      const Unit u = next;
      // In registers before the loop: after each asm with a memory clobber
      // they would be read again.
      const Problem& p = a.p[u.i];
      const Dims& sh = shapes[u.i];
      const int m = u.m * kTM + (int)rank * 128;
      const int w = sh.w;
      const int n = kIsGate ? u.n * w : u.n * 2 * w + (int)rank * w;
      const int kb0 = sh.kb0;
      const bool a_mn = sh.a_mn, b_mn = sh.b_mn;
      const CUtensorMap* const maps_a = p.a;
      const CUtensorMap* const maps_b = p.b + (kIsGate ? (int)rank : 0);
      for (int kb = u.k0; kb < u.k1; ++kb) {
        if (!__all_sync(~0u, wait(empty(s), parity ^ 1))) {
          ok = false;
          break;
        }
        const int seg = kb >= kb0;
        const int k = (kb - (seg ? kb0 : 0)) * kBK;
        const CUtensorMap* ma = maps_a + seg;
        const CUtensorMap* mb = maps_b + seg;
        const uint32_t da = ring + s * kStageBytes, db = da + kTileBytes;
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(full(s), 2 * (kTileBytes + w * kBK * 2));
          if (a_mn) {
            tma_load_pair(da, ma, m, k, full(s));
            tma_load_pair(da + kTileBytes / 2, ma, m + 64, k, full(s));
          } else {
            tma_load_pair(da, ma, k, m, full(s));
          }
          if (b_mn) {
            tma_load_pair(db, mb, n, k, full(s));
            if (w > 64) tma_load_pair(db + kTileBytes / 2, mb, n + 64, k, full(s));
          } else {
            tma_load_pair(db, mb, k, n, full(s));
          }
        }
        if (kb == u.k0) {  // decoded under the copies
          ui = index(i);
          next = unit(ui);
        }
        if (++s == kStages) {
          s = 0;
          parity ^= 1;
        }
      }
    }
    if (!ok) {
      // Copies may be in flight into this CTA: let them land before it can
      // exit.  The last phase armed of each stage, waited for with a limit.
      for (int i = 0; i < kStages; ++i)
        mbar_wait_bounded(full(i), i < s ? parity : parity ^ 1, nullptr, kDrainLimitNs);
    }
  } else if (warp == 1 && rank == 0) {
    // Issuer of the pair's matrix instructions.
    int s = 0, acc = 0;
    uint32_t parity = 0, acc_parity = 0;
    bool ok = true;
    int ui = index(0);
    Unit next = unit(ui);
    for (int i = 1; ok && ui < units; ++i) {
      const Unit u = next;
      const bool a_mn = shapes[u.i].a_mn, b_mn = shapes[u.i].b_mn;
      const uint32_t idesc = instr_desc(kTM, 2 * shapes[u.i].w, a_mn, b_mn);
      const uint32_t step_a = k_step_bytes(a_mn) >> 4, step_b = k_step_bytes(b_mn) >> 4;
      if (!(ok = __all_sync(~0u, wait(acc_empty(acc), acc_parity ^ 1)))) break;
      tc_fence_after();
      const uint32_t d = tmem + acc * kAccCols;
      for (int kb = u.k0; kb < u.k1; ++kb) {
        if (!(ok = __all_sync(~0u, wait(full(s), parity)))) break;
        tc_fence_after();
        const uint64_t da = smem_desc(ring + s * kStageBytes, a_mn, kTileBytes / 2);
        const uint64_t db = smem_desc(ring + s * kStageBytes + kTileBytes, b_mn, kTileBytes / 2);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k)
            tc_mma<2>(d, da + k * step_a, db + k * step_b, idesc, kb > u.k0 || k > 0);
          tc_commit<2>(empty(s));
          if (kb + 1 == u.k1) tc_commit<2>(acc_full(acc));
        }
        if (kb == u.k0) {  // decoded under the products
          ui = index(i);
          next = unit(ui);
        }
        if (++s == kStages) {
          s = 0;
          parity ^= 1;
        }
      }
      acc ^= 1;
      if (acc == 0) acc_parity ^= 1;
    }
    if (!ok) {  // matrix instructions may be in flight: wait for them, with a limit
      if (elect_one()) tc_commit<2>(drain);
      mbar_wait_bounded(drain, 0, nullptr, kDrainLimitNs);
    }
  } else if (warp >= 2) {
    // Epilogue.  A warp reads the 32 lanes of tensor memory of its quarter.
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t buf = staging + (warp - 2) * staging_bytes(KIND);
    const int row_in = (int)rank * 128 + quarter * 32, lanes = quarter * 32;
    int acc = 0, turn = 0;
    uint32_t acc_parity = 0;
    bool ok = true;
    // kGateBwd: this warp's chunks are every other 32 columns of a unit; its
    // chunk c exists if it starts before the last column.  The saved values are
    // read one chunk ahead, into the next unit that has one.
    auto col_of = [&](const Unit& u, int c) { return u.n * 2 * shapes[u.i].w + (2 * c + half) * 32; };
    auto saved_of = [&](const Unit& u) -> const uint4* {  // of the unit's first chunk
      const Dims& s = shapes[u.i];
      const int row0 = u.m * kTM + row_in;
      return row0 < s.M ? saved_at(a.saved, row0, col_of(u, 0), s.N, lane) : nullptr;
    };
    // The first unit from the pair's i-th on with a chunk for this warp.
    auto seek = [&](int i) -> const uint4* {
      for (int ui; (ui = index(i)) < units; ++i) {
        const Unit u = unit(ui);
        if (col_of(u, 0) < shapes[u.i].N) return saved_of(u);
      }
      return nullptr;
    };
    SavedRow in = {};
    const uint4* at_saved = nullptr;  // of the next unit's first chunk
    if (KIND == kGateBwd) {
      at_saved = seek(0);
#pragma unroll
      for (int i = 0; i < kSavedVecs; ++i) in.load(at_saved, i);
    }
    int ui = index(0);
    Unit next = unit(ui);
    for (int i = 1; ok && ui < units; ++i) {
      const Unit u = next;
      ui = index(i);
      next = unit(ui);
      const Dims& sh = shapes[u.i];
      const uint4* here = at_saved;
      if (KIND == kGateBwd && col_of(u, 0) < sh.N) at_saved = seek(i);
      if (!(ok = __all_sync(~0u, wait(acc_full(acc), acc_parity)))) break;
      tc_fence_after();
      const int row0 = u.m * kTM + row_in;
      const uint32_t at = tmem + acc * kAccCols + ((uint32_t)lanes << 16);
      if constexpr (KIND == kPlain) {
        epilogue_plain(a.p[u.i], sh, u, at, row0, half, buf, lane, turn);
      } else if constexpr (kIsGate) {
        epilogue_gate<ACT, KIND == kGateSave>(a, sh, u, at, row0, half, buf, lane, turn);
      } else {
        const int M = sh.M, N = sh.N, chunks = sh.w / 32;
#pragma unroll 1
        for (int c = 0; c < chunks && col_of(u, c) < N; ++c) {
          const bool last = c + 1 == chunks || col_of(u, c + 1) >= N;
          if (here != nullptr) here += 2 * kSavedBlock / 16;
          chunk_gate_bwd<ACT>(a, at + (2 * c + half) * 32, col_of(u, c), row0, M, buf, lane, in,
                              last ? at_saved : here);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_rank(acc_empty(acc), 0));
      acc ^= 1;
      if (acc == 0) acc_parity ^= 1;
    }
    bulk_wait();
  }
  __syncwarp();
  tc_fence_before();
  // The pair's copies, commits and arrivals reach both CTAs: neither leaves
  // before the other is done.
  __syncthreads();
  cluster_sync();
  if (warp == 2) tmem_free<2>(tmem, 512);
}

// out = the sum of the split partials, in split order, rounded to bf16.
__global__ void __launch_bounds__(256) ffn_join_kernel(const float* partial, int splits,
                                                       int64_t vecs, __nv_bfloat16* out) {
  grid_wait();
  grid_launch_dependents();
  const float4* p = reinterpret_cast<const float4*>(partial);
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < vecs; i += gridDim.x * 256ll) {
    float4 s = p[i];
    for (int k = 1; k < splits; ++k) {
      const float4 v = p[i + k * vecs];
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    reinterpret_cast<uint2*>(out)[i] = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
  }
}

// ----- host side ------------------------------------------------------------------

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

}  // namespace

cudaError_t make_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int box_cols,
                     int box_rows) {
  EncodeFn fn;
  const cudaError_t e = encode_fn(&fn);
  if (e != cudaSuccess) return e;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)cols * 2};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows}, one[2] = {1, 1};
  const CUresult r =
      fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, one,
         CU_TENSOR_MAP_INTERLEAVE_NONE,
         box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
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

// Operand of a product: a row-major matrix whose rows run along k (K-major)
// or along m or n (MN-major).
struct Operand {
  const void* p;
  int64_t rows, cols;
  bool mn;
};
cudaError_t operand_map(CUtensorMap* m, const Operand& o, int rows) {
  return make_map(m, o.p, o.rows, o.cols, 64, o.mn ? kBK : rows);
}
// Blocks of 32 x 32 of an epilogue.
cudaError_t block_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols) {
  return make_map(m, p, rows, cols, 32, 32);
}

template <int KIND>
void* gemm_kernel(int act) {
  if constexpr (KIND == kPlain) return (void*)ffn_gemm_kernel<kPlain, 0>;
  else switch (act) {
    case ADALN_ACT_SILU: return (void*)ffn_gemm_kernel<KIND, ADALN_ACT_SILU>;
    case ADALN_ACT_GELU_TANH: return (void*)ffn_gemm_kernel<KIND, ADALN_ACT_GELU_TANH>;
    default: return (void*)ffn_gemm_kernel<KIND, ADALN_ACT_GELU>;
  }
}
void* kernel_of(int kind, int act) {
  return kind == kPlain      ? gemm_kernel<kPlain>(act)
         : kind == kGate     ? gemm_kernel<kGate>(act)
         : kind == kGateSave ? gemm_kernel<kGateSave>(act)
                             : gemm_kernel<kGateBwd>(act);
}

// CTA pairs that the device holds at once (one CTA an SM), after allowing the
// kernels their shared memory on it.  Asked once per device.
constexpr int kMaxDev = 64;
cudaError_t pairs_of_device(int* pairs) {
  static std::mutex mu;
  static int known[kMaxDev] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(mu);
  if (!known[dev]) {
    for (int kind = 0; kind < kKinds; ++kind)
      for (int act = 0; act < 3; ++act) {
        e = cudaFuncSetAttribute(kernel_of(kind, act), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 smem_of(kind));
        if (e != cudaSuccess) return e;
      }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_of(kPlain);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, kernel_of(kPlain, 0), &cfg);
    if (e != cudaSuccess) return e;
    known[dev] = n > 0 ? n : 1;
  }
  *pairs = known[dev];
  return cudaSuccess;
}

// How a product [M, N] over kb k blocks is cut into units for the CTA pairs: the
// width w of a tile and the splits of k.
struct Tiling {
  int w, splits;
  size_t bytes;  // of the fp32 partials
};
// Clocks of a unit: a k block takes its products' time (4 w) or that of the
// copies that feed them (about 62 bytes a clock and SM, from L2), and a unit's
// start and end cost about 3000.
double unit_clocks(int kb, int w) {
  const double copies = (128 + w) * 128 / 62.0;
  return kb * (copies > 4.0 * w ? copies : 4.0 * w) + 3000;
}
int cover(bool gate, int w) { return gate ? w : 2 * w; }
int tiles_of(int64_t M, int N, bool gate, int w) { return div_up(M, kTM) * div_up(N, cover(gate, w)); }

// The cheapest tiling.  256-column tiles (w = 128) feed the products best; w =
// 96 and 64 (an MN-major B: 64 only) fill the pairs better where there are few
// tiles: with 256 tokens, D = 5120, F = 13824 the 108 tiles of the projections
// take two rounds of 76 pairs, the 144 of w = 96 two shorter ones.  A split of k
// costs the joining launch and its partials, written and read again.  `other`:
// clocks of shorter units beside it in the launch, of `other_unit` each.
Tiling choose_tiling(int64_t M, int N, int kb, bool gate, bool b_mn, bool may_split, int pairs,
                     double other = 0, double other_unit = 0) {
  Tiling best = {};
  double least = 0;
  for (int w = 128; w >= 64; w -= b_mn ? 64 : 32) {
    const int64_t tiles = tiles_of(M, N, gate, w);
    // (Twice as many units as pairs are as many as a split can be good for.)
    for (int s = 1; s == 1 || (may_split && tiles * (s - 1) < 2 * pairs && kb / s >= 8); ++s) {
      const double unit = unit_clocks(div_up(kb, s), w);
      const double rounds = (double)div_up(tiles * s, pairs);
      double cost = rounds * unit;
      if (other > 0) {
        const double even = (tiles * s * unit + other) / pairs + other_unit / 2;
        if (even > cost) cost = even;
      }
      if (s > 1) cost += 7000 + 3e-3 * s * (double)M * N;
      if (best.w == 0 || cost < least) {
        least = cost;
        best = {w, s, s > 1 ? (size_t)s * M * N * 4 : 0};
      }
    }
  }
  return best;
}

cudaError_t set_problem(Problem* p, const Operand (&a)[2], const Operand (&b)[2], int segs, int64_t M,
                        int N, bool gate, const Tiling& t, int64_t k0, int64_t k1, void* out) {
  cudaError_t e = operand_map(&p->a[0], a[0], 128);
  if (e == cudaSuccess) e = operand_map(&p->b[0], b[0], t.w);
  if (e == cudaSuccess && segs > 1) e = operand_map(&p->a[1], a[1], 128);
  if (e == cudaSuccess && b[1].p != nullptr) e = operand_map(&p->b[1], b[1], t.w);
  if (e == cudaSuccess && out) e = block_map(&p->out, out, M, N);
  p->partial = nullptr;
  Dims& s = p->s;
  s.M = (int)M;
  s.N = N;
  s.kb0 = div_up(k0, kBK);
  s.kb = s.kb0 + (segs > 1 ? div_up(k1, kBK) : 0);
  s.tiles_m = div_up(M, kTM);
  s.w = t.w;
  s.tiles_n = div_up(N, cover(gate, t.w));
  s.splits = t.splits;
  s.first = 0;
  s.a_mn = a[0].mn;
  s.b_mn = b[0].mn;
  return e;
}

// `worth`: with several problems, how many units of the others one of the first
// takes the time of.
cudaError_t launch_gemm(GemmArgs& a, int kind, int act, int pairs, int worth, cudaStream_t st) {
  int at = 0;
  for (int i = 0; i < a.problems; ++i) {
    Dims& s = a.p[i].s;
    s.first = at;
    at += s.tiles_m * s.tiles_n * s.splits;
  }
  a.units = at;
  a.lead = a.problems > 1 ? a.p[1].s.first : 0;
  a.worth = worth;
  const int grid = 2 * (at < pairs ? at : pairs);
  void* params[1] = {&a};
  return traced_launch(ADALN_KERNEL_FFN, st, [&] {
    return launch_cluster(kernel_of(kind, act), grid, kThreads, smem_of(kind), 2, params, st);
  });
}

cudaError_t launch_join(const Problem& p, void* to, int pairs, cudaStream_t st) {
  const float* partial = p.partial;
  int splits = p.s.splits;
  int64_t vecs = (int64_t)p.s.M * p.s.N / 4;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(to);
  void* params[4] = {&partial, &splits, &vecs, &out};
  const int64_t blocks = (vecs + 255) / 256;
  const int most = 2 * pairs * 8;  // resident at 256 threads: eight an SM
  const int grid = (int)(blocks < most ? blocks : most);
  return traced_launch(ADALN_KERNEL_FFN, st, [&] {
    return launch_cluster((void*)ffn_join_kernel, grid, 256, 0, 1, params, st);
  });
}

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
  p.gate = choose_tiling(T, F, div_up(D, kBK), true, false, false, pairs);
  p.y = choose_tiling(T, D, div_up(F, kBK), false, false, true, pairs);
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
  p.gate = choose_tiling(T, F, div_up(D, kBK), false, true, false, pairs);
  p.dw = {128, 1, 0};
  const double unit = unit_clocks(div_up(T, kBK), 128);
  const int64_t tiles = 2 * (int64_t)tiles_of(F, D, false, 128) + tiles_of(D, F, false, 128);
  const int kb = 2 * div_up(F, kBK);
  p.dx = choose_tiling(T, D, kb, false, true, true, pairs, tiles * unit, unit);
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
  const cudaError_t e = pairs_of_device(&pairs);
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
  cudaError_t e = pairs_of_device(&pairs);
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
  if (e == cudaSuccess) e = launch_gemm(a, saved ? kGateSave : kGate, act, pairs, 0, st);
  if (e != cudaSuccess) return launch_failed(e);

  e = set_problem(&a.p[0], {{ws, T, F, false}, none}, {{wd, D, F, false}, none}, 1, T, D, false, plan.y,
                  F, 0, y);
  a.p[0].partial = reinterpret_cast<float*>(ws + round256((size_t)T * F * 2));
  if (e == cudaSuccess) e = launch_gemm(a, kPlain, act, pairs, 0, st);
  if (e == cudaSuccess && plan.y.splits > 1) e = launch_join(a.p[0], y, pairs, st);
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
  if ((e = pairs_of_device(&pairs)) != cudaSuccess) return launch_failed(e);
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
  if (e == cudaSuccess) e = launch_gemm(a, kGateBwd, act, pairs, 0, st);
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
  if (e == cudaSuccess) e = launch_gemm(a, kPlain, act, pairs, plan.worth, st);
  if (e == cudaSuccess && plan.dx.splits > 1) e = launch_join(a.p[0], dx, pairs, st);
  return e == cudaSuccess ? ADALN_OK : launch_failed(e);
}

}  // extern "C"
