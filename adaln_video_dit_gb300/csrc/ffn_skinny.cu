// The gated feed-forward block's forward for few tokens (up to 32).
//
// With few tokens the weights' 6 D F bytes are what the call costs, so they
// are the matrix instructions' wide operand: a CTA owns 128 rows of Wg and the
// same rows of Wu (or 128 of Wd), streams them once through a TMA ring, and
// multiplies them with all tokens at a time (an accumulator holds 128 features
// x 16 or 32 tokens).  Two CTAs an SM keep about 200 KB an SM in flight.
// One token, D = 5120, F = 13824: 68.5 us, 91 % of the measured copy rate (the
// other form, which pads to 256 tokens, 117 us); 32 tokens 78 and 90 us.  With
// 64 tokens, and so two stages in the ring, 92 and 94 us (D = 1536, F = 4096:
// 30 and 28 us), so there the other form takes over.
//
// There are few such row blocks (32 for F = 4096), so the sum over k is split
// over a cluster of up to 8 CTAs, as many as keep all CTAs resident; the
// partial sums meet in shared memory of the cluster, in rank order.
//
// h goes to the second product as two bf16 tensors, its rounding and what the
// rounding left: both multiply the same weights into one accumulator, at no
// cost in bytes, and y is then as exact as from an fp32 h.  The second
// product's CTAs start to fetch Wd while the first ones still run.
#include <mutex>

#include "ffn.cuh"

namespace adaln {
namespace {

constexpr int kBK = 64, kRows = 128;
constexpr int kWBytes = kRows * kBK * 2;
constexpr int kThreads = 128;
constexpr int kRingBytes = 108 * 1024;  // two CTAs an SM
constexpr int kMaxSplits = 8;           // portable cluster size
constexpr int kMaxTokens = 32;

ADALN_HD constexpr int stage_bytes(bool gate, int nt) {
  return gate ? 2 * kWBytes + nt * 128 : kWBytes + 2 * nt * 128;
}
ADALN_HD constexpr int stages_of(bool gate, int nt) { return kRingBytes / stage_bytes(gate, nt); }
constexpr int smem_of(bool gate, int nt) {
  return 1024 + stages_of(gate, nt) * stage_bytes(gate, nt) + 256;
}

struct SkinnyArgs {
  CUtensorMap w[2], b[2];  // Wg, Wu and x; or Wd and h's two parts
  int T, rows, kb;         // rows of the weights (features), k blocks
  __nv_bfloat16* out[2];   // h's two parts [T, rows]; or y [T, rows]
  unsigned char* saved;    // or nullptr
  unsigned* status;
};

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// One value of the saved format (kSavedVecs): its upper 16 bits and next 8.
__device__ __forceinline__ void save_value(unsigned char* block, int lane, int c, float v) {
  const uint32_t x = __float_as_uint(v);
  *reinterpret_cast<uint16_t*>(block + (c / 8 * 32 + lane) * 16 + c % 8 * 2) = (uint16_t)(x >> 16);
  block[((4 + c / 16) * 32 + lane) * 16 + c % 16] = (unsigned char)(x >> 8);
}

template <bool GATE, int ACT, int NT>
__global__ void __launch_bounds__(kThreads) ffn_skinny_kernel(const __grid_constant__ SkinnyArgs a) {
  constexpr int kStages = stages_of(GATE, NT), kStage = stage_bytes(GATE, NT);
  constexpr int kCols = GATE ? 2 * NT : 32;  // of tensor memory
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
  const int row0 = blockIdx.x / splits * kRows;
  const int k0 = (int)((int64_t)a.kb * rank / splits);
  const int n = (int)((int64_t)a.kb * (rank + 1) / splits) - k0;  // >= 1

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
    mbar_arrive_expect_tx(full(s), kStage);
    tma_load(at, &a.w[0], (k0 + i) * kBK, row0, full(s));
    if (GATE) tma_load(at + kWBytes, &a.w[1], (k0 + i) * kBK, row0, full(s));
  };
  auto load_tokens = [&](int i, int s) {
    const uint32_t at = ring + s * kStage + (GATE ? 2 : 1) * kWBytes;
    tma_load(at, &a.b[0], (k0 + i) * kBK, 0, full(s));
    if (!GATE) tma_load(at + NT * 128, &a.b[1], (k0 + i) * kBK, 0, full(s));
  };

  if (GATE || warp != 0) {
    grid_wait();
    grid_launch_dependents();
  }
  bool ok = true;
  if (warp == 0) {
    int s = 0;
    uint32_t parity = 0;
    const int early = GATE ? 0 : min(n, kStages);
    if (!GATE) {
      // The first weights before the wait: they were complete before the first
      // product's kernel began (it waited for what was before it, and only then
      // let this one be scheduled), only h is that kernel's.
      if (elect_one())
        for (int i = 0; i < early; ++i) load_weights(i, i);
      __syncwarp();
      grid_wait();
      if (elect_one())
        for (int i = 0; i < early; ++i) load_tokens(i, i);
      s = early == kStages ? 0 : early;
      parity = early == kStages;
    }
    int issued = early;
    for (int i = early; i < n; ++i, ++issued) {
      if (!(ok = __all_sync(~0u, wait(empty(s), parity ^ 1)))) break;
      if (elect_one()) {
        load_weights(i, s);
        load_tokens(i, s);
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
    constexpr uint32_t idesc = instr_desc(kRows, NT, false, false);
    int s = 0;
    uint32_t parity = 0;
    for (int i = 0; i < n; ++i) {
      if (!(ok = __all_sync(~0u, wait(full(s), parity)))) break;
      tc_fence_after();
      const uint32_t at = ring + s * kStage;
      const uint64_t w0 = smem_desc(at, false, 0), w1 = smem_desc(at + kWBytes, false, 0);
      const uint64_t b0 = smem_desc(at + (GATE ? 2 : 1) * kWBytes, false, 0);
      const uint64_t b1 = smem_desc(at + kWBytes + NT * 128, false, 0);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kBK / 16; ++k) {
          tc_mma<1>(tmem, w0 + 2 * k, b0 + 2 * k, idesc, i > 0 || k > 0);
          if (GATE)
            tc_mma<1>(tmem + NT, w1 + 2 * k, b0 + 2 * k, idesc, i > 0 || k > 0);
          else
            tc_mma<1>(tmem, w0 + 2 * k, b1 + 2 * k, idesc, true);
        }
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
  // (Once a wait has given up, this waits for the products in flight, with a
  // limit; the sums below are then of no use, but in bounds.)
  if (!wait(done, 0)) mbar_wait_bounded(done, 0, nullptr, kDrainLimitNs);
  __syncwarp();
  tc_fence_after();

  // Sums over the cluster.  red: [columns][128] fp32 over the ring, which
  // nothing is copied into any more.
  const uint32_t red = ring;
  {
    uint32_t r[32];
    const uint32_t at = tmem + ((uint32_t)(warp * 32) << 16);
    const uint32_t to = red + (warp * 32 + lane) * 4;
#pragma unroll
    for (int c = 0; c < kCols; c += 32) {  // (NT = 16: g and u, or 16 columns of no use)
      tmem_ld32(at + c, r);
      tc_wait_ld();
#pragma unroll
      for (int i = 0; i < 32; ++i)
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + (c + i) * 512), "r"(r[i]) : "memory");
    }
  }
  __syncwarp();
  cluster_sync();
  const int items = a.T * kRows;
  const int end = (int)((int64_t)items * (rank + 1) / splits);
  for (int i = (int)((int64_t)items * rank / splits) + threadIdx.x; i < end; i += kThreads) {
    const int t = i / kRows, f = row0 + i % kRows;
    float g = 0.0f, u = 0.0f;
    for (uint32_t k = 0; k < splits; ++k) {
      const uint32_t from = map_rank(red, k) + i * 4;
      g += ld_cluster_f32(from);
      if (GATE) u += ld_cluster_f32(from + NT * 512);
    }
    if (f >= a.rows) continue;
    const int64_t o = (int64_t)t * a.rows + f;
    if (GATE) {
      float2 p, d;
      gate<ACT>(splat2(g), p, d);
      const float h = g * p.x * u;
      const __nv_bfloat16 hi = __float2bfloat16_rn(h);
      a.out[0][o] = hi;
      // (An infinite h has no rest: inf - inf would make y NaN.)
      const float rest = h - __bfloat162float(hi);
      a.out[1][o] = __float2bfloat16_rn(isfinite(rest) ? rest : 0.0f);
      if (a.saved != nullptr) {
        unsigned char* block =
            a.saved + ((int64_t)(t >> 5) * ((a.rows + 31) >> 5) + (f >> 5)) * kSavedBlock;
        save_value(block, t & 31, f & 31, g);
        save_value(block + kSavedBlock / 2, t & 31, f & 31, u);
      }
    } else {
      a.out[0][o] = __float2bfloat16_rn(g);
    }
  }
  __syncwarp();
  cluster_sync();  // before an owner of sums leaves
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_free<1>(tmem, kCols);
}

template <bool GATE, int NT>
void* kernel_nt(int act) {
  if constexpr (!GATE)
    return (void*)ffn_skinny_kernel<false, 0, NT>;
  else
    return act == ADALN_ACT_SILU        ? (void*)ffn_skinny_kernel<true, ADALN_ACT_SILU, NT>
           : act == ADALN_ACT_GELU_TANH ? (void*)ffn_skinny_kernel<true, ADALN_ACT_GELU_TANH, NT>
                                        : (void*)ffn_skinny_kernel<true, ADALN_ACT_GELU, NT>;
}
template <bool GATE>
void* kernel_of(int nt, int act) {
  return nt == 16 ? kernel_nt<GATE, 16>(act) : kernel_nt<GATE, 32>(act);
}

// Allow the kernels their shared memory on the current device (once), and its
// SM count.
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
    for (int nt = 16; nt <= kMaxTokens && e == cudaSuccess; nt *= 2) {
      for (int act = 0; act < 3 && e == cudaSuccess; ++act)
        e = cudaFuncSetAttribute(kernel_of<true>(nt, act),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, smem_of(true, nt));
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel_of<false>(nt, 0),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, smem_of(false, nt));
    }
    int n = 0;
    if (e == cudaSuccess) e = sm_count(dev, &n);
    if (e != cudaSuccess) return e;
    known[dev] = n;
  }
  *sms = known[dev];
  return cudaSuccess;
}

int tokens_of(int64_t T) { return T <= 16 ? 16 : 32; }

}  // namespace

// Clusters of 7 or 8 only where one CTA an SM holds them all: two an SM, fewer of
// them find room in the SMs' groups (one token, D = 5120, F = 13824: 77.5 and
// 74.7 us with 7 and 8 for the second product, 68.5 us with 6).
int choose_splits(int64_t blocks, int kb, int sms) {
  int64_t s = 2 * sms / blocks;
  if (s > kMaxSplits) s = kMaxSplits;
  if (s > 6 && blocks * s > sms) s = 6;
  if (s > kb) s = kb;
  return s < 1 ? 1 : (int)s;
}

bool skinny_serves(int64_t T) { return T <= kMaxTokens; }

size_t skinny_workspace(int64_t T, int32_t F) { return 2 * round256((size_t)T * F * 2); }

cudaError_t skinny_fwd(const void* x, const void* wg, const void* wu, const void* wd, int T, int D,
                       int F, int act, void* y, void* saved, void* workspace, unsigned* status,
                       cudaStream_t st) {
  int sms = 0;
  cudaError_t e = prepare(&sms);
  if (e != cudaSuccess) return e;
  const int nt = tokens_of(T);
  char* hi = static_cast<char*>(workspace);
  char* lo = hi + round256((size_t)T * F * 2);

  SkinnyArgs a = {};
  a.T = T;
  a.status = status;
  a.rows = F;
  a.kb = div_up(D, kBK);
  a.out[0] = reinterpret_cast<__nv_bfloat16*>(hi);
  a.out[1] = reinterpret_cast<__nv_bfloat16*>(lo);
  a.saved = static_cast<unsigned char*>(saved);
  e = make_map(&a.w[0], wg, F, D, kBK, kRows);
  if (e == cudaSuccess) e = make_map(&a.w[1], wu, F, D, kBK, kRows);
  if (e == cudaSuccess) e = make_map(&a.b[0], x, T, D, kBK, nt);
  a.b[1] = a.b[0];
  if (e != cudaSuccess) return e;
  void* params[1] = {&a};
  int blocks = div_up(F, kRows), splits = choose_splits(blocks, a.kb, sms);
  e = traced_launch(ADALN_KERNEL_FFN, st, [&] {
    return launch_cluster(kernel_of<true>(nt, act), blocks * splits, kThreads, smem_of(true, nt),
                          splits, params, st);
  });
  if (e != cudaSuccess) return e;

  a.rows = D;
  a.kb = div_up(F, kBK);
  a.out[0] = static_cast<__nv_bfloat16*>(y);
  a.out[1] = nullptr;
  a.saved = nullptr;
  e = make_map(&a.w[0], wd, D, F, kBK, kRows);
  a.w[1] = a.w[0];
  if (e == cudaSuccess) e = make_map(&a.b[0], hi, T, F, kBK, nt);
  if (e == cudaSuccess) e = make_map(&a.b[1], lo, T, F, kBK, nt);
  if (e != cudaSuccess) return e;
  blocks = div_up(D, kRows);
  splits = choose_splits(blocks, a.kb, sms);
  return traced_launch(ADALN_KERNEL_FFN, st, [&] {
    return launch_cluster(kernel_of<false>(nt, act), blocks * splits, kThreads, smem_of(false, nt),
                          splits, params, st);
  });
}

}  // namespace adaln
