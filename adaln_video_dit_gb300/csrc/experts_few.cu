// The experts' feed-forward for few rows an expert, forward and backward (but for the
// weight gradients, whose sums run over rows: experts.cu).
//
// With few rows the experts' weights are what a call costs, each read once for 64
// rows, so they are the matrix instructions' wide operand: a CTA owns a block of 64
// sorted rows (one expert's: starts are multiples of 64) and 128 rows of that
// expert's weights (64 of Wg and the same of Wu for the projections), streams the
// weights through a TMA ring, and multiplies them with the 64 rows at a time (an
// accumulator holds 128 features x 64 rows).  The other form's tiles of 256 rows are
// bound here by what they copy and multiply for empty rows, and by one tile's k loop
// where few experts are met.  Measured (one GB300, forward, calls in a row on arrays
// without spare rows; floor from the weights at the copy rate): D = 1536, F = 4096, eight
// experts met 62 us (45; tiles 70), two 26 us (11), one 16.5 us (5.6; tiles 31.8); D = 5120,
// F = 13824, two experts 137 us (127); 64 experts of 2048 x 1024 139 us (120).  What is left
// is each CTA's start and end, some 5 us a launch.  16 pairs in a route's array for eight
// experts (512 rows, which the splits of k are chosen by): seven met 50 us, six 46, two 25,
// one 22.  Their backward, whose weight gradients are written for all eight: 132 us with
// eight met (90 for the bytes), 118 with six, 87 with one (51).
//
// Four products, alike but for their maps and epilogues:
//   projections  [g; u] = [Wg; Wu] x'       h = act(g) u, g and u saved
//   y            y' = Wd h'
//   gate         dh' = Wd' dy'              dg, du, h from the saved g and u
//   dx           dx' = Wg' dg' + Wu' du'
// In the first two a row of the weights runs along k, in the others along the
// features (MN-major): the boxes of 64 x 64 that fill a stage are the same.
//
// The sum over k is split over a cluster of up to 8 CTAs, as many as keep all CTAs
// resident at two an SM; the partial sums meet in shared memory of the cluster, in rank
// order.  (More splits than that cost more at their joins than they fill: eight experts
// met 62 us, 71 with at most 16 k blocks a CTA, 94 with 8.)  Three CTAs an SM of three
// stages keep 144 KB of weights an SM in flight (two of four stages 66 us).  A call's
// second product starts to fetch its weights while the first one still runs.
#include <mutex>

#include "ffn.cuh"

namespace adaln {
namespace {

constexpr int kBK = 64, kRows = 64, kFeatures = 128;
constexpr int kHalf = 64 * kBK * 2;            // a box of 64 x 64
constexpr int kStage = 3 * kHalf;              // two of weights, one of rows
constexpr int kStages = 3;                     // three CTAs an SM
constexpr int kThreads = 128;
constexpr int kSmem = 1024 + kStages * kStage + 256;
constexpr int kCols = kRows;                   // of tensor memory

enum { kProject = 0, kOut = 1, kGradGate = 2, kGradIn = 3 };

struct FewArgs {
  CUtensorMap w[2], b[2];  // the halves' weights (kGradIn: the segments'), the rows
  const int32_t* starts;   // [E + 1]
  int64_t rows;
  int E;
  int blocks;              // of the weights' features
  int features;            // of the output
  int kb0, kb;             // k blocks of segment 0, of both
  __nv_bfloat16* out;      // h, y, h, dx
  __nv_bfloat16 *dg, *du;
  unsigned char* saved;    // or nullptr (kProject)
  unsigned* status;
};

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* m, int x, int y, int z,
                                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(m), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// The expert of sorted row `row`, or -1 where there is none (or the starts are bad,
// which is recorded).  The whole warp.
__device__ __forceinline__ int expert_of_row(const FewArgs& a, int64_t row) {
  const int lane = threadIdx.x & 31;
  int reached = 0;
  bool bad = false;
  for (int e = lane; e <= a.E; e += 32) {
    const int s = a.starts[e];
    bad |= s > a.rows || s % kRows != 0 || (e > 0 ? a.starts[e - 1] > s : s != 0);
    reached += s <= row;
  }
  if (__any_sync(~0u, bad)) {
    if (lane == 0) atomicOr(a.status, ADALN_DEV_EXPERT_RANGE);
    return -1;
  }
  reached = __reduce_add_sync(~0u, reached);
  return reached > a.E ? -1 : reached - 1;
}

struct Values {
  float2 v[4];
};
// Eight neighbouring features of a row: the sums of the cluster's parts.
__device__ __forceinline__ Values sum_of(uint32_t at, uint32_t splits) {
  Values s = {};
  for (uint32_t k = 0; k < splits; ++k) {
    const uint32_t from = map_rank(at, k);
    const float4 x = ld_cluster_f32x4(from), y = ld_cluster_f32x4(from + 16);
    s.v[0] = add2(s.v[0], make_float2(x.x, x.y));
    s.v[1] = add2(s.v[1], make_float2(x.z, x.w));
    s.v[2] = add2(s.v[2], make_float2(y.x, y.y));
    s.v[3] = add2(s.v[3], make_float2(y.z, y.w));
  }
  return s;
}
__device__ __forceinline__ void store(__nv_bfloat16* to, const Values& s) {
  *reinterpret_cast<uint4*>(to) = BF16::pack2(s.v);
}

// Eight saved values (kSavedVecs): the upper halves of features c .. c + 7 of a block's
// row `lane`, and their next bytes.
__device__ __forceinline__ void save(unsigned char* block, int lane, int c, const Values& s) {
  uint32_t x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __float_as_uint(s.v[i].x);
    x[2 * i + 1] = __float_as_uint(s.v[i].y);
  }
  *reinterpret_cast<uint4*>(block + (c / 8 * 32 + lane) * 16) =
      make_uint4(__byte_perm(x[0], x[1], 0x7632), __byte_perm(x[2], x[3], 0x7632),
                 __byte_perm(x[4], x[5], 0x7632), __byte_perm(x[6], x[7], 0x7632));
  *reinterpret_cast<uint2*>(block + ((4 + c / 16) * 32 + lane) * 16 + c % 16) =
      make_uint2(__byte_perm(__byte_perm(x[0], x[1], 0x51), __byte_perm(x[2], x[3], 0x51), 0x5410),
                 __byte_perm(__byte_perm(x[4], x[5], 0x51), __byte_perm(x[6], x[7], 0x51), 0x5410));
}
// And back (the lowest byte, which was not kept, repeats the one before it).
__device__ __forceinline__ Values saved_values(const unsigned char* block, int lane, int c) {
  const uint4 w = *reinterpret_cast<const uint4*>(block + (c / 8 * 32 + lane) * 16);
  const uint2 b = *reinterpret_cast<const uint2*>(block + ((4 + c / 16) * 32 + lane) * 16 + c % 16);
  const uint32_t up[4] = {w.x, w.y, w.z, w.w}, low[2] = {b.x, b.y};
  Values s;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    s.v[i] = i % 2 ? make_float2(__uint_as_float(__byte_perm(up[i], low[i / 2], 0x1066)),
                                 __uint_as_float(__byte_perm(up[i], low[i / 2], 0x3277)))
                   : make_float2(__uint_as_float(__byte_perm(up[i], low[i / 2], 0x1044)),
                                 __uint_as_float(__byte_perm(up[i], low[i / 2], 0x3255)));
  return s;
}

template <int MODE, int ACT>
__global__ void __launch_bounds__(kThreads) experts_few_kernel(const __grid_constant__ FewArgs a) {
  constexpr bool kMn = MODE == kGradGate || MODE == kGradIn;    // the weights' layout
  constexpr bool kSecond = MODE == kOut || MODE == kGradIn;     // a call's second product
  extern __shared__ unsigned char smem_raw[];
  const uint32_t ring = (smem_addr(smem_raw) + 1023) & ~1023u;
  const uint32_t bars = ring + kStages * kStage;
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (kStages + s); };
  const uint32_t done = bars + 16 * kStages, tmem_ptr = done + 8;
  volatile int* abort_flag =
      reinterpret_cast<volatile int*>(smem_raw + (done + 16 - smem_addr(smem_raw)));
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  uint32_t rank, splits;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(splits));
  const int cluster = blockIdx.x / splits, block = cluster % a.blocks;
  const int64_t row0 = (int64_t)(cluster / a.blocks) * kRows;
  const int k0 = (int)((int64_t)a.kb * rank / splits);
  const int n = (int)((int64_t)a.kb * (rank + 1) / splits) - k0;  // >= 1

  // The first product waits for what is before it; the second's starts and weights were
  // complete before the first one began (it waited, and only then let this one be
  // scheduled): only its rows are the first one's.
  if (!kSecond) {
    grid_wait();
    grid_launch_dependents();
  }
  const int e = expert_of_row(a, row0);
  if (e < 0) {  // (the whole cluster)
    if (kSecond) {
      grid_wait();
      grid_launch_dependents();
    }
    return;
  }

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc<1>(tmem_ptr, kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tmem_ptr) : "memory");

  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (mbar_wait_spin(bar, parity, abort_flag)) return true;
    *abort_flag = 1;
    atomicOr(a.status, ADALN_DEV_TIMEOUT);
    return false;
  };
  auto load_weights = [&](int i, int s) {
    const uint32_t at = ring + s * kStage;
    const int kb = k0 + i, seg = MODE == kGradIn && kb >= a.kb0;
    const int k = (kb - (seg ? a.kb0 : 0)) * kBK;
    mbar_arrive_expect_tx(full(s), kStage);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const CUtensorMap* m = &a.w[MODE == kProject ? half : seg];
      const int f = MODE == kProject ? block * 64 : block * kFeatures + half * 64;
      tma_load(at + half * kHalf, m, kMn ? f : k, kMn ? k : f, e, full(s));
    }
  };
  auto load_rows = [&](int i, int s) {
    const int kb = k0 + i, seg = MODE == kGradIn && kb >= a.kb0;
    tma_load(ring + s * kStage + 2 * kHalf, &a.b[seg], (kb - (seg ? a.kb0 : 0)) * kBK, (int)row0, 0, full(s));
  };

  if (kSecond && warp != 0) {
    grid_wait();
    grid_launch_dependents();
  }
  if (MODE == kGradGate && warp >= 2) {  // on their way into L2 under the products
    const int across = (a.features + 31) >> 5, left = min(kFeatures / 32, across - block * (kFeatures / 32));
    for (int r = 0; r < kRows / 32; ++r) {
      const unsigned char* from =
          a.saved + (((row0 >> 5) + r) * across + block * (kFeatures / 32)) * (int64_t)kSavedBlock;
      for (int i = (threadIdx.x - 64) * 128; i < left * kSavedBlock; i += 64 * 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(from + i));
    }
  }
  bool ok = true;
  if (warp == 0) {
    int s = 0;
    uint32_t parity = 0;
    const int early = kSecond ? min(n, kStages) : 0;
    if (kSecond) {
      if (elect_one())
        for (int i = 0; i < early; ++i) load_weights(i, i);
      __syncwarp();
      grid_wait();
      if (elect_one())
        for (int i = 0; i < early; ++i) load_rows(i, i);
      s = early == kStages ? 0 : early;
      parity = early == kStages;
    }
    int issued = early;
    for (int i = early; i < n; ++i, ++issued) {
      if (!(ok = __all_sync(~0u, wait(empty(s), parity ^ 1)))) break;
      if (elect_one()) {
        load_weights(i, s);
        load_rows(i, s);
      }
      if (++s == kStages) {
        s = 0;
        parity ^= 1;
      }
    }
    if (!ok)  // copies may be in flight: wait for the last of each stage, with a limit
      for (int i = max(0, issued - kStages); i < issued; ++i)
        mbar_wait_bounded(full(i % kStages), i / kStages & 1, nullptr, kDrainLimitNs);
  } else if (warp == 1) {
    constexpr uint32_t idesc = instr_desc(kFeatures, kRows, kMn, false);
    const uint32_t step = k_step_bytes(kMn) >> 4;
    int s = 0;
    uint32_t parity = 0;
    for (int i = 0; i < n; ++i) {
      if (!(ok = __all_sync(~0u, wait(full(s), parity)))) break;
      tc_fence_after();
      const uint32_t at = ring + s * kStage;
      const uint64_t w = smem_desc(at, kMn, kHalf), b = smem_desc(at + 2 * kHalf, false, 0);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kBK / 16; ++k) tc_mma<1>(tmem, w + k * step, b + 2 * k, idesc, i > 0 || k > 0);
        tc_commit<1>(empty(s));
        if (i + 1 == n) tc_commit<1>(done);
      }
      if (++s == kStages) {
        s = 0;
        parity ^= 1;
      }
    }
    if (!ok && elect_one()) tc_commit<1>(done);
  }
  __syncwarp();
  // (Once a wait has given up, this waits for the products in flight, with a limit; the
  // sums below are then of no use, but in bounds.)
  if (!wait(done, 0)) mbar_wait_bounded(done, 0, nullptr, kDrainLimitNs);
  __syncwarp();
  tc_fence_after();

  // The sums over the cluster.  red: [rows][128] fp32 over the ring, which nothing is
  // copied into any more.
  const uint32_t red = ring;
  {
    uint32_t r[32];
    const uint32_t at = tmem + ((uint32_t)(warp * 32) << 16), to = red + (warp * 32 + lane) * 4;
#pragma unroll
    for (int c = 0; c < kCols; c += 32) {
      tmem_ld32(at + c, r);
      tc_wait_ld();
#pragma unroll
      for (int i = 0; i < 32; ++i)
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + (c + i) * 512), "r"(r[i]) : "memory");
    }
  }
  __syncwarp();
  cluster_sync();
  constexpr int kWide = MODE == kProject ? 8 : 16;  // groups of eight features of a row
  constexpr int kItems = kRows * kWide;
  const int end = (int)(kItems * (rank + 1) / splits);
  const int N = a.features;
  for (int i = (int)(kItems * rank / splits) + threadIdx.x; i < end; i += kThreads) {
    const int t = i / kWide, c = i % kWide;
    const uint32_t at = red + t * 512 + c * 32;
    const int f = block * 8 * kWide + c * 8;
    if (f >= N) continue;
    const int64_t row = row0 + t, o = row * N + f;
    Values s = sum_of(at, splits);
    if constexpr (MODE == kProject) {
      const Values u = sum_of(at + 256, splits);
      Values h;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float2 p, d;
        gate<ACT>(s.v[q], p, d);
        h.v[q] = mul2(mul2(s.v[q], p), u.v[q]);
      }
      store(a.out + o, h);
      if (a.saved != nullptr) {
        unsigned char* to = a.saved + ((row >> 5) * ((N + 31) >> 5) + (f >> 5)) * kSavedBlock;
        save(to, row & 31, f & 31, s);
        save(to + kSavedBlock / 2, row & 31, f & 31, u);
      }
    } else if constexpr (MODE == kGradGate) {
      const unsigned char* from = a.saved + ((row >> 5) * ((N + 31) >> 5) + (f >> 5)) * kSavedBlock;
      const Values g = saved_values(from, row & 31, f & 31);
      const Values u = saved_values(from + kSavedBlock / 2, row & 31, f & 31);
      Values dg, du, h;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float2 p, d;
        gate<ACT>(g.v[q], p, d);
        const float2 act = mul2(g.v[q], p);
        dg.v[q] = mul2(mul2(s.v[q], u.v[q]), d);
        du.v[q] = mul2(s.v[q], act);
        h.v[q] = mul2(act, u.v[q]);
      }
      store(a.dg + o, dg);
      store(a.du + o, du);
      store(a.out + o, h);
    } else {
      store(a.out + o, s);
    }
  }
  __syncwarp();
  cluster_sync();  // before an owner of sums leaves
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_free<1>(tmem, kCols);
}

template <int MODE>
void* kernel_act(int act) {
  return act == ADALN_ACT_SILU        ? (void*)experts_few_kernel<MODE, ADALN_ACT_SILU>
         : act == ADALN_ACT_GELU_TANH ? (void*)experts_few_kernel<MODE, ADALN_ACT_GELU_TANH>
                                      : (void*)experts_few_kernel<MODE, ADALN_ACT_GELU>;
}
void* kernel_of(int mode, int act) {
  return mode == kProject    ? kernel_act<kProject>(act)
         : mode == kGradGate ? kernel_act<kGradGate>(act)
         : mode == kOut      ? (void*)experts_few_kernel<kOut, 0>
                             : (void*)experts_few_kernel<kGradIn, 0>;
}

// Allow the kernels their shared memory on the current device (once), and its SM
// count.
cudaError_t prepare(int* sms) {
  constexpr int kMaxDev = 64;
  static std::mutex mu;
  static int known[kMaxDev] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(mu);
  if (!known[dev]) {
    for (int mode = kProject; mode <= kGradIn && e == cudaSuccess; ++mode)
      for (int act = 0; act < 3 && e == cudaSuccess; ++act)
        e = cudaFuncSetAttribute(kernel_of(mode, act), cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    int n = 0;
    if (e == cudaSuccess) e = sm_count(dev, &n);
    if (e != cudaSuccess) return e;
    known[dev] = n;
  }
  *sms = known[dev];
  return cudaSuccess;
}

cudaError_t launch(FewArgs& a, int mode, int act, int sms, cudaStream_t st) {
  const int row_blocks = (int)(a.rows / kRows);
  const int splits = choose_splits((int64_t)row_blocks * a.blocks, a.kb, sms);
  const int64_t grid = (int64_t)row_blocks * a.blocks * splits;
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  void* params[1] = {&a};
  return traced_launch(ADALN_KERNEL_EXPERTS, st, [&] {
    return launch_cluster(kernel_of(mode, act), (int)grid, kThreads, kSmem, splits, params, st);
  });
}

// Boxes of 64 x 64 of the experts' matrices [E, rows, cols], or of sorted rows.
cudaError_t box_map(CUtensorMap* m, const void* p, int64_t depth, int64_t rows, int64_t cols) {
  return make_map(m, p, depth, rows, cols, 64, 64);
}

FewArgs args_of(const Experts& x, unsigned* status) {
  FewArgs a = {};
  a.starts = x.starts, a.rows = x.rows, a.E = x.E, a.status = status;
  return a;
}

}  // namespace

// Arrays of at most a block and a half of 64 rows an expert: a route's up to 33 to 40 pairs
// an expert on average (they hold 63 rows an expert beside the pairs); both sides measured
// in experts.cu.
bool experts_few_serve(int64_t rows, int32_t E) { return 2 * (rows / kRows) <= 3 * (int64_t)E; }

cudaError_t experts_few_fwd(const Experts& x, void* ys, void* saved, void* h, unsigned* status,
                            cudaStream_t st) {
  int sms = 0;
  cudaError_t e = prepare(&sms);
  FewArgs a = args_of(x, status);
  a.blocks = div_up(x.F, 64);
  a.features = x.F;
  a.kb0 = a.kb = div_up(x.D, kBK);
  a.out = static_cast<__nv_bfloat16*>(h);
  a.saved = static_cast<unsigned char*>(saved);
  if (e == cudaSuccess) e = box_map(&a.w[0], x.wg, x.E, x.F, x.D);
  if (e == cudaSuccess) e = box_map(&a.w[1], x.wu, x.E, x.F, x.D);
  if (e == cudaSuccess) e = box_map(&a.b[0], x.xs, 1, x.rows, x.D);
  if (e == cudaSuccess) e = launch(a, kProject, x.act, sms, st);
  a.blocks = div_up(x.D, kFeatures);
  a.features = x.D;
  a.kb0 = a.kb = div_up(x.F, kBK);
  a.out = static_cast<__nv_bfloat16*>(ys);
  a.saved = nullptr;
  if (e == cudaSuccess) e = box_map(&a.w[0], x.wd, x.E, x.D, x.F);
  if (e == cudaSuccess) e = box_map(&a.b[0], h, 1, x.rows, x.F);
  return e == cudaSuccess ? launch(a, kOut, x.act, sms, st) : e;
}

cudaError_t experts_few_bwd(const Experts& x, const void* dys, const void* saved, void* h, void* dg, void* du,
                            void* dxs, unsigned* status, cudaStream_t st) {
  int sms = 0;
  cudaError_t e = prepare(&sms);
  FewArgs a = args_of(x, status);
  a.blocks = div_up(x.F, kFeatures);
  a.features = x.F;
  a.kb0 = a.kb = div_up(x.D, kBK);
  a.out = static_cast<__nv_bfloat16*>(h);
  a.dg = static_cast<__nv_bfloat16*>(dg);
  a.du = static_cast<__nv_bfloat16*>(du);
  a.saved = static_cast<unsigned char*>(const_cast<void*>(saved));  // read only here
  if (e == cudaSuccess) e = box_map(&a.w[0], x.wd, x.E, x.D, x.F);
  if (e == cudaSuccess) e = box_map(&a.b[0], dys, 1, x.rows, x.D);
  if (e == cudaSuccess) e = launch(a, kGradGate, x.act, sms, st);
  a.blocks = div_up(x.D, kFeatures);
  a.features = x.D;
  a.kb0 = div_up(x.F, kBK);
  a.kb = 2 * a.kb0;
  a.out = static_cast<__nv_bfloat16*>(dxs);
  if (e == cudaSuccess) e = box_map(&a.w[0], x.wg, x.E, x.F, x.D);
  if (e == cudaSuccess) e = box_map(&a.w[1], x.wu, x.E, x.F, x.D);
  if (e == cudaSuccess) e = box_map(&a.b[0], dg, 1, x.rows, x.F);
  if (e == cudaSuccess) e = box_map(&a.b[1], du, 1, x.rows, x.F);
  return e == cudaSuccess ? launch(a, kGradIn, x.act, sms, st) : e;
}

}  // namespace adaln
