// The products of the gated feed-forward blocks on the tensor cores: the kernel, its
// epilogues, and the host's choice of tiles.  ffn.cu has the block itself, experts.cu
// the block of each expert on its rows of a sorted array; each compiles its own
// instances (GROUPED false and true).
#pragma once

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

// GROUPED: the rows of a sorted array are those of `experts` experts, each on its own
// weights: starts[e] is expert e's first row, a multiple of kRowAlign.  A problem
// either has those rows as the output's (B is expert e's matrix) or, `by_k`, sums over
// them (the weight gradients: a matrix for each expert; zeros for one without rows).
constexpr int kRowAlign = 64;
constexpr int kMaxExperts = ADALN_MAX_EXPERTS;
static_assert(kMaxExperts < kThreads && kThreads / 32 <= kMaxExperts, "a thread for each start");

// C[M, N] = sum over its K segments of A B.
struct Dims {        // what the roles of a CTA read of a problem
  int M, N;
  int kb0, kb;         // k blocks of segment 0, of both
  int w;               // rows of B a CTA stages
  int tiles_m, tiles_n, splits;
  int first;           // first unit of the problem
  int a_mn, b_mn;      // operand layouts
  int by_k;            // GROUPED
  float inv_each, inv_group;  // GROUPED: 1 / the units of an expert (by_k) or of a tile of
                              // rows, 1 / (kGroupM tiles_n)
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
  // GROUPED.
  const int32_t* starts;  // [experts + 1]
  int experts;
  int64_t rows;           // of the sorted arrays
};

struct Unit {
  int i;           // problem
  int row, end;    // the tile's first row of the output, the end of the output's rows
  int n;           // tile of columns
  int k0, k1;      // k blocks
  int split;
  int e, k_row;    // GROUPED: expert, and (by_k) its first row
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

// Where the experts' rows and tiles of rows start, an entry an expert and one for
// the end: its first row in kRowAlign, over its tiles' first, which is that of four
// kRowAlign a tile with what the experts before it fell short of whole tiles (at
// most 3 each): 18 and 10 bits.
struct Starts {
  const int* v;
  __device__ __forceinline__ static int pack(int rows, int rest) { return rows << 10 | rest; }
  __device__ __forceinline__ int rows(int e) const { return v[e] >> 10; }
  __device__ __forceinline__ int tiles(int e) const { return ((v[e] >> 10) + (v[e] & 1023)) >> 2; }
};
static_assert(kTM == 4 * kRowAlign && 3 * kMaxExperts < 1024 &&
                  ADALN_FFN_MAX_T / kRowAlign <= 1 << 18, "packed starts");

// Fills `to` from a.starts, with the whole CTA; what is not a list of starts (from 0, not
// decreasing, in whole kRowAlign, within the rows) is recorded and taken for one without
// rows.
__device__ __forceinline__ void fetch_starts(const GemmArgs& a, int* to, int* bad) {
  const int e = threadIdx.x;
  if (e == 0) *bad = 0;
  int s = 0;
  if (e <= a.experts) {
    s = a.starts[e];
    to[e] = s;
  }
  __syncthreads();
  if (e <= a.experts && (s > a.rows || s % kRowAlign != 0 || (e > 0 ? to[e - 1] > s : s != 0))) *bad = 1;
  __syncthreads();
  if (*bad) {
    s = 0;
    if (e == 0) atomicOr(a.status, ADALN_DEV_EXPERT_RANGE);
  }
  // What the expert before e fell short of whole tiles, summed up to e.
  s /= kRowAlign;
  int rest = e > 0 && e <= a.experts && !*bad ? -(s - to[e - 1] / kRowAlign) & 3 : 0;
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(~0u, rest, d);
    if ((e & 31) >= d) rest += v;
  }
  __syncthreads();
  if ((e & 31) == 31) to[e >> 5] = rest;  // (a warp's sum)
  __syncthreads();
  for (int w = 0; w < e >> 5; ++w) rest += to[w];
  __syncthreads();
  if (e <= a.experts) to[e] = Starts::pack(s, rest);
  __syncthreads();
}

// The expert of tile v of rows: the last one that starts at or before it.  (The
// whole warp: two rounds of comparisons.)
__device__ __forceinline__ int expert_of_tile(Starts starts, int experts, int v) {
  const int lane = threadIdx.x & 31, stride = (experts + 31) / 32;
  int at = lane * stride;
  unsigned hit = __ballot_sync(~0u, at < experts && starts.tiles(min(at, experts)) <= v);
  const int base = (31 - __clz(hit)) * stride;
  at = base + lane;
  hit = __ballot_sync(~0u, lane < stride && at < experts && starts.tiles(min(at, experts)) <= v);
  return base + 31 - __clz(hit);
}

// u / d for 0 <= u < 2^24 (kMaxUnits) and d >= 1, by a rounded 1 / d and two corrections
// by one (the product is off by at most two): units of few k blocks are over before a
// chain of integer divisions is.
constexpr int kMaxUnits = 1 << 24;
__device__ __forceinline__ int quotient(int u, int d, float inv) {
  int q = (int)((float)u * inv), r = u - q * d;
  int fix = (r >= d) - (r < 0);
  q += fix;
  r -= fix * d;
  return q + (r >= d) - (r < 0);
}

// `shapes` is the problems' copy in shared memory (reads of the kernel's
// parameters with an index cost several hundred cycles each).
template <bool GROUPED>
__device__ __forceinline__ Unit unit_of(const Dims* shapes, int problems, int u, Starts starts,
                                        int experts) {
  Unit r;
  r.i = 0;
  while (r.i + 1 < problems && u >= shapes[r.i + 1].first) ++r.i;
  const Dims& s = shapes[r.i];
  u -= s.first;
  r.split = r.e = r.k_row = 0;
  int base = 0, tiles_m = s.tiles_m, kb = s.kb;
  r.end = s.M;
  if (GROUPED) {
    if (s.by_k) {
      const int each = tiles_m * s.tiles_n;
      r.e = quotient(u, each, s.inv_each);
      u -= r.e * each;
      r.k_row = starts.rows(r.e) * kRowAlign;
      kb = starts.rows(r.e + 1) - starts.rows(r.e);
    } else {
      const int each = s.tiles_n * s.splits;
      r.e = expert_of_tile(starts, experts, quotient(u, each, s.inv_each));
      u -= starts.tiles(r.e) * each;
      tiles_m = starts.tiles(r.e + 1) - starts.tiles(r.e);
      base = starts.rows(r.e) * kRowAlign;
      r.end = starts.rows(r.e + 1) * kRowAlign;
    }
  }
  int tile = u;
  r.k0 = 0;
  r.k1 = kb;
  if (s.splits > 1) {
    tile = u / s.splits;
    r.split = u - tile * s.splits;
    r.k0 = (int)((int64_t)kb * r.split / s.splits);
    r.k1 = (int)((int64_t)kb * (r.split + 1) / s.splits);
  }
  const int per_group = kGroupM * s.tiles_n;
  const int group = GROUPED ? quotient(tile, per_group, s.inv_group) : tile / per_group;
  const int in = tile - group * per_group;
  const int rows = max(min(kGroupM, tiles_m - group * kGroupM), 1);  // (no tiles: no unit is used)
  r.n = GROUPED ? quotient(in, rows, __fdividef(1.0f, (float)rows)) : in / rows;
  r.row = base + (group * kGroupM + in - r.n * rows) * kTM;
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

// Where the rows of a unit's output end.
template <bool GROUPED>
__device__ __forceinline__ int end_of(const Dims& s, const Unit& u) {
  return GROUPED ? u.end : s.M;
}

template <bool GROUPED>
__device__ __forceinline__ void store_block(const CUtensorMap* m, int col, int row, uint32_t block) {
  if constexpr (GROUPED)
    tma_store(m, col, row, 0, block);
  else
    tma_store(m, col, row, block);
}

// GROUPED, plain: outputs leave in blocks of 64 columns, half as many copies as blocks of
// 32: with few rows an expert a weight gradient's tile is a few k blocks of products,
// and its copies out are what takes the time.
__device__ __forceinline__ void put_wide_row(uint32_t block, int lane, const uint32_t (&w)[32]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    st_shared_v4(block + lane * 128 + ((i ^ (lane & 7)) << 4), w[4 * i], w[4 * i + 1], w[4 * i + 2],
                 w[4 * i + 3]);
}
__device__ __forceinline__ void epilogue_wide(const Problem& p, const Dims& s, const Unit& u, uint32_t acc,
                                              int row0, int half, uint32_t buf, int lane) {
  const int N = s.N, chunks = s.w / 32, z = s.by_k ? u.e : 0;
  const bool none = u.k0 == u.k1;  // an empty sum
#pragma unroll 1
  for (int c = half; c < chunks; c += 2) {
    const int col = u.n * 2 * s.w + c * 64;
    if (col >= N) break;
    __syncwarp();
    uint32_t w[32];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t r[32];
      tmem_ld32(acc + c * 64 + j * 32, r);
      tc_wait_ld();
#pragma unroll
      for (int i = 0; i < 16; ++i)
        w[16 * j + i] = none ? 0 : pack_bf16(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
    }
    bulk_wait_read<0>();  // the copy before used this block
    __syncwarp();
    put_wide_row(buf, lane, w);
    fence_async_shared();
    __syncwarp();
    if (elect_one()) {
      tma_store(&p.out, col, row0, z, buf);
      bulk_commit();
    }
  }
}

template <bool GROUPED>
__device__ __forceinline__ void epilogue_plain(const Problem& p, const Dims& s, const Unit& u,
                                               uint32_t acc, int row0, int half, uint32_t buf,
                                               int lane, int& turn) {
  const int M = s.M, N = s.N, splits = s.splits, chunks = s.w / 16, end = end_of<GROUPED>(s, u);
#pragma unroll 1
  for (int c = half; c < chunks; c += 2) {
    const int col = u.n * 2 * s.w + c * 32;
    if (col >= N) break;
    __syncwarp();
    uint32_t r[32];
    tmem_ld32(acc + c * 32, r);
    tc_wait_ld();
    if (GROUPED || splits > 1) {  // (GROUPED: partial sums only)
      const int left = row0 + lane < end ? N - col : 0;  // columns of this row to write
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
        if (row0 < end) tma_store(&p.out, col, row0, block);
        bulk_commit();
      }
    }
  }
}

template <int ACT, bool SAVE, bool GROUPED>
__device__ __forceinline__ void epilogue_gate(const GemmArgs& a, const Dims& s, const Unit& u,
                                              uint32_t acc, int row0, int half, uint32_t buf,
                                              int lane, int& turn) {
  const int end = end_of<GROUPED>(s, u), N = s.N, w_cols = s.w;
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
      if (row0 < end) store_block<GROUPED>(&a.h, col, row0, block);
      bulk_commit();
    }
    if (SAVE && row0 < end) {
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
template <int ACT, bool GROUPED>
__device__ __forceinline__ void chunk_gate_bwd(const GemmArgs& a, uint32_t acc, int col, int row0,
                                               int end, uint32_t buf, int lane, SavedRow& in,
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
    if (row0 < end) {
      store_block<GROUPED>(&a.dg, col, row0, buf);
      store_block<GROUPED>(&a.du, col, row0, buf + kBlock);
      store_block<GROUPED>(&a.h, col, row0, buf + 2 * kBlock);
    }
    bulk_commit();
  }
}

template <int KIND, int ACT, bool GROUPED>
__global__ void __launch_bounds__(kThreads, 1)
    ffn_gemm_kernel(const __grid_constant__ GemmArgs a) {
  constexpr int kStages = stages_of(KIND);
  constexpr bool kIsGate = KIND == kGate || KIND == kGateSave;
  extern __shared__ unsigned char smem_raw[];
  __shared__ Dims shapes[kMaxProblems];
  __shared__ int starts_of[GROUPED ? kMaxExperts + 1 : 1];
  __shared__ int found[2];  // GROUPED: whether the starts are bad, the number of units
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

  const int problems = a.problems, experts = a.experts, worth = a.worth;
  const Starts starts = {starts_of};
  int units = a.units, lead = a.lead;
  if constexpr (GROUPED) {  // known here only
    fetch_starts(a, starts_of, &found[0]);
    if (threadIdx.x == 0) {
      int at = 0;
      for (int i = 0; i < problems; ++i) {
        Dims& s = shapes[i];
        s.first = at;
        at += s.by_k ? experts * s.tiles_m * s.tiles_n : starts.tiles(experts) * s.tiles_n * s.splits;
      }
      found[1] = at;
    }
    __syncthreads();
    units = found[1];
    lead = problems > 1 ? shapes[1].first : 0;
  }
  auto index = [&](int i) { return unit_index(cluster, i, clusters, lead, worth); };
  auto unit = [&](int ui) {
    return unit_of<GROUPED>(shapes, problems, max(min(ui, units - 1), 0), starts, experts);
  };
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
      const int m = u.row + (int)rank * 128;
      const int w = sh.w;
      const int n = kIsGate ? u.n * w : u.n * 2 * w + (int)rank * w;
      const int kb0 = sh.kb0;
      const bool a_mn = sh.a_mn, b_mn = sh.b_mn;
      const int zb = GROUPED && !sh.by_k ? u.e : 0, k_row = GROUPED ? u.k_row : 0;
      // GROUPED: blocks of kRowAlign rows of A that this CTA stages, and the bytes that the
      // pair does.  Those past the expert's rows are left out: they are read for nothing
      // (2222 rows of 16 experts fill a tile to a half), and what the products make of the
      // stage's old contents there goes into rows that nothing stores.
      const int left = u.end - m, blocks = min(max(left, 0) / kRowAlign, 2);
      const int pair_blocks = min((u.end - u.row) / kRowAlign, 4);
      const uint32_t pair_bytes = GROUPED && !a_mn ? pair_blocks * (kTileBytes / 2) + 2 * w * kBK * 2
                                                   : 2 * (kTileBytes + w * kBK * 2);
      auto load = [&](uint32_t to, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
        if constexpr (GROUPED)
          tma_load_pair(to, map, x, y, z, bar);
        else
          tma_load_pair(to, map, x, y, bar);
      };
      if (GROUPED && u.k0 == u.k1) {
        ui = index(i);
        next = unit(ui);
      }
      const CUtensorMap* const maps_a = p.a;
      const CUtensorMap* const maps_b = p.b + (kIsGate ? (int)rank : 0);
      for (int kb = u.k0; kb < u.k1; ++kb) {
        if (!__all_sync(~0u, wait(empty(s), parity ^ 1))) {
          ok = false;
          break;
        }
        const int seg = kb >= kb0;
        const int k = k_row + (kb - (seg ? kb0 : 0)) * kBK;
        const CUtensorMap* ma = maps_a + seg;
        const CUtensorMap* mb = maps_b + seg;
        const uint32_t da = ring + s * kStageBytes, db = da + kTileBytes;
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(full(s), pair_bytes);
          if (a_mn) {
            load(da, ma, m, k, 0, full(s));
            load(da + kTileBytes / 2, ma, m + 64, k, 0, full(s));
          } else if (GROUPED) {
            if (blocks > 0) load(da, ma, k, m, 0, full(s));
            if (blocks > 1) load(da + kTileBytes / 2, ma, k, m + kRowAlign, 0, full(s));
          } else {
            load(da, ma, k, m, 0, full(s));
          }
          if (b_mn) {
            load(db, mb, n, k, zb, full(s));
            if (w > 64) load(db + kTileBytes / 2, mb, n + 64, k, zb, full(s));
          } else {
            load(db, mb, k, n, zb, full(s));
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
      if (GROUPED && u.k0 == u.k1) {  // nothing to sum: the epilogue writes zeros
        if (elect_one()) tc_commit<2>(acc_full(acc));
        ui = index(i);
        next = unit(ui);
      }
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
      const int row0 = u.row + row_in;
      return row0 < end_of<GROUPED>(s, u) ? saved_at(a.saved, row0, col_of(u, 0), s.N, lane) : nullptr;
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
      const int row0 = u.row + row_in;
      const uint32_t at = tmem + acc * kAccCols + ((uint32_t)lanes << 16);
      if (GROUPED && row0 >= u.end) {  // none of this warp's rows are the expert's
        if (KIND == kGateBwd && col_of(u, 0) < sh.N) {
#pragma unroll
          for (int i = 0; i < kSavedVecs; ++i) in.load(at_saved, i);
        }
      } else if constexpr (KIND == kPlain) {
        if (GROUPED && sh.splits == 1)
          epilogue_wide(a.p[u.i], sh, u, at, row0, half, buf, lane);
        else
          epilogue_plain<GROUPED>(a.p[u.i], sh, u, at, row0, half, buf, lane, turn);
      } else if constexpr (kIsGate) {
        epilogue_gate<ACT, KIND == kGateSave, GROUPED>(a, sh, u, at, row0, half, buf, lane, turn);
      } else {
        const int N = sh.N, end = end_of<GROUPED>(sh, u), chunks = sh.w / 32;
#pragma unroll 1
        for (int c = 0; c < chunks && col_of(u, c) < N; ++c) {
          const bool last = c + 1 == chunks || col_of(u, c + 1) >= N;
          if (here != nullptr) here += 2 * kSavedBlock / 16;
          chunk_gate_bwd<ACT, GROUPED>(a, at + (2 * c + half) * 32, col_of(u, c), row0, end, buf, lane, in,
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

// out = the sum of the split partials, in split order, rounded to bf16; up to row
// *end of rows of `row_vecs` where `end` is given.
__global__ void __launch_bounds__(256) ffn_join_kernel(const float* partial, int splits,
                                                       int64_t vecs, __nv_bfloat16* out,
                                                       const int32_t* end, int row_vecs) {
  grid_wait();
  grid_launch_dependents();
  const int64_t all = vecs;  // of a split
  if (end != nullptr) vecs = min(vecs, (int64_t)max(*end, 0) * row_vecs);
  const float4* p = reinterpret_cast<const float4*>(partial);
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < vecs; i += gridDim.x * 256ll) {
    float4 s = p[i];
    for (int k = 1; k < splits; ++k) {
      const float4 v = p[i + k * all];
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    reinterpret_cast<uint2*>(out)[i] = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
  }
}

// ----- host side ------------------------------------------------------------------

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

template <int KIND, bool GROUPED>
void* gemm_kernel(int act) {
  if constexpr (KIND == kPlain) return (void*)ffn_gemm_kernel<kPlain, 0, GROUPED>;
  else switch (act) {
    case ADALN_ACT_SILU: return (void*)ffn_gemm_kernel<KIND, ADALN_ACT_SILU, GROUPED>;
    case ADALN_ACT_GELU_TANH: return (void*)ffn_gemm_kernel<KIND, ADALN_ACT_GELU_TANH, GROUPED>;
    default: return (void*)ffn_gemm_kernel<KIND, ADALN_ACT_GELU, GROUPED>;
  }
}
template <bool GROUPED>
void* kernel_of(int kind, int act) {
  return kind == kPlain      ? gemm_kernel<kPlain, GROUPED>(act)
         : kind == kGate     ? gemm_kernel<kGate, GROUPED>(act)
         : kind == kGateSave ? gemm_kernel<kGateSave, GROUPED>(act)
                             : gemm_kernel<kGateBwd, GROUPED>(act);
}

// CTA pairs that the device holds at once (one CTA an SM), after allowing the
// kernels their shared memory on it.  Asked once per device.
constexpr int kMaxDev = 64;
template <bool GROUPED>
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
        e = cudaFuncSetAttribute(kernel_of<GROUPED>(kind, act), cudaFuncAttributeMaxDynamicSharedMemorySize,
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
    e = cudaOccupancyMaxActiveClusters(&n, kernel_of<GROUPED>(kPlain, 0), &cfg);
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
int64_t tiles_of(int64_t tiles_m, int N, bool gate, int w) { return tiles_m * div_up(N, cover(gate, w)); }

// The cheapest tiling of a product of M rows in tiles_m tiles.  256-column tiles (w = 128) feed the products best; w =
// 96 and 64 (an MN-major B: 64 only) fill the pairs better where there are few
// tiles: with 256 tokens, D = 5120, F = 13824 the 108 tiles of the projections
// take two rounds of 76 pairs, the 144 of w = 96 two shorter ones.  A split of k
// costs the joining launch and its partials, written and read again.  `other`:
// clocks of shorter units beside it in the launch, of `other_unit` each.
Tiling choose_tiling(int64_t M, int64_t tiles_m, int N, int kb, bool gate, bool b_mn, bool may_split, int pairs,
                     double other = 0, double other_unit = 0) {
  Tiling best = {};
  double least = 0;
  for (int w = 128; w >= 64; w -= b_mn ? 64 : 32) {
    const int64_t tiles = tiles_of(tiles_m, N, gate, w);
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
  s.by_k = 0;
  s.inv_each = s.inv_group = 0;
  return e;
}

// `worth`: with several problems, how many units of the others one of the first
// takes the time of.
template <bool GROUPED>
cudaError_t launch_gemm(GemmArgs& a, int kind, int act, int pairs, int worth, cudaStream_t st) {
  int64_t at = 0;
  for (int i = 0; i < a.problems; ++i) {
    Dims& s = a.p[i].s;
    s.first = (int)at;  // (GROUPED: an upper bound, the kernel counts them)
    at += (int64_t)s.tiles_m * s.tiles_n * s.splits * (s.by_k ? a.experts : 1);
  }
  if (GROUPED && at >= kMaxUnits) return cudaErrorInvalidConfiguration;
  a.units = (int)at;
  a.lead = a.problems > 1 ? a.p[1].s.first : 0;
  a.worth = worth;
  const int grid = 2 * (int)(at < pairs ? at : pairs);
  void* params[1] = {&a};
  return traced_launch(GROUPED ? ADALN_KERNEL_EXPERTS : ADALN_KERNEL_FFN, st, [&] {
    return launch_cluster(kernel_of<GROUPED>(kind, act), grid, kThreads, smem_of(kind), 2, params, st);
  });
}

// `end`: the row on the device that the sorted rows end at, or NULL.
cudaError_t launch_join(const Problem& p, void* to, const int32_t* end, int pairs, cudaStream_t st) {
  const float* partial = p.partial;
  int splits = p.s.splits;
  int64_t vecs = (int64_t)p.s.M * p.s.N / 4;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(to);
  int row_vecs = p.s.N / 4;
  void* params[6] = {&partial, &splits, &vecs, &out, &end, &row_vecs};
  const int64_t blocks = (vecs + 255) / 256;
  const int most = 2 * pairs * 8;  // resident at 256 threads: eight an SM
  const int grid = (int)(blocks < most ? blocks : most);
  return traced_launch(end ? ADALN_KERNEL_EXPERTS : ADALN_KERNEL_FFN, st, [&] {
    return launch_cluster((void*)ffn_join_kernel, grid, 256, 0, 1, params, st);
  });
}

}  // namespace
}  // namespace adaln
