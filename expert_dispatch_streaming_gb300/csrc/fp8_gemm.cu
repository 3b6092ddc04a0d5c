// Grouped matrix product of E4M3 token rows with E4M3 expert weights on the 5th-generation
// tensor cores (tcgen05 + TMEM), one fp32 scale per row and 128 columns of the activations and
// per 128 x 128 block of the weights:
//
//   acc[row][n] = sum_b xs[row][b] ws[n / 128][b] sum_{k in block b} xq[row][k] w[n][k]
//
// Each block's inner sum is formed by the tensor cores from zero and scaled into an fp32
// accumulator in registers, so arbitrary fp32 scales are exact to one rounding per block and the
// tensor cores' own accumulation never runs over more than 128 products.
//
// Tile: 128 token rows (the MMA's M, one TMEM lane each) x 256 weight rows (N: a gate tile and
// its up tile when fused, else two neighbouring tiles), one block of 128 k per step.  With tokens
// on the lanes a thread owns one token: its scale is one value per step, a weight block is one
// value per 128 columns, and the row's largest |h| (fused: h is requantised here) is a maximum
// over the thread's own registers.  (Weights on the lanes would need every token's scale in
// every thread, 128 shared-memory reads a step.)
//
// Persistent kernel, one CTA per SM, 384 threads:
//   warp 0     producer: per step 16 KB of token rows by 2-D TMA (128-byte swizzle; a tile that is
//              not full in boxes of 32 rows) and 32 KB of weights: two bundle tiles by bulk copy
//              (each is stored as its swizzled shared-memory image), or two TMA boxes of a
//              row-major weight; four stages;
//   warp 1     MMA issuer: four tcgen05.mma (K = 32 each) per step into one of two 256-column
//              TMEM buffers;
//   warps 4-11 two warps per TMEM lane quarter, 64 columns of each weight tile per thread: per
//              step, tcgen05.ld and a packed fp32 multiply-add by xs * ws into 128 accumulators
//              (they take the registers warps 0-3 give up).
//
// Work: tiles (expert, weight tile pair, token tile), token tile fastest so that CTAs running
// together share weights through L2.  With few tiles the steps of all tiles, in order, are cut
// into one equal range per CTA: a tile cut by range ends is finished by the last of its CTAs to
// arrive (a counter per lane quarter), which adds the pieces' fp32 sums in range order, so the
// result does not depend on the arrival order.
//
// Every wait is bounded (2 s; then an error word and the kernel ends).
#include <cuda.h>
#include <cudaTypedefs.h>

#include "fp8.cuh"

namespace moe {
namespace {

constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kStages = 4;
constexpr int kABytes = kFp8TileBytes, kBBytes = 2 * kFp8TileBytes;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kThreads = 384;
// Registers per thread after the split: warps 0-3 and warps 4-11 (128 * 40 + 256 * 232 = the
// 384 * 168 the block is launched with).
constexpr int kRegsLow = 40, kRegsHigh = 232;
static_assert(128 * kRegsLow + 256 * kRegsHigh <= kThreads * 168, "within the launch's registers");
constexpr int kAccCols = 256, kTmemCols = 512;
// Tiles below this many per CTA are cut into equal ranges of steps.
constexpr int kRangeTiles = 4;

struct alignas(16) Ctl {
  uint64_t full[kStages], empty[kStages], tfull[2], tempty[2], pair[4];
  uint32_t tmem;
  int last[4];
  int pref[kMaxExperts + 1];
  float amax[2][2][128];
};
constexpr int kSmem = kStages * kStageBytes + 1024 + (int)sizeof(Ctl);
static_assert(kSmem <= 232448, "over the 227 KB shared-memory limit of a CTA");

struct Fp8Params {
  CUtensorMap tm_x, tm_x32;     // token rows [max_rows][K], boxes of 128 / 32 rows x 128 bytes
  CUtensorMap tm_w;             // row-major weights [E * N][K], boxes of 128 x 128 bytes
  const float* xs;
  const int32_t* offsets;
  int E, N, K, KB, NT, max_rows, RP;
  BundleTable tab;
  const void* const* dev_tab;
  size_t w_off, s_off;
  const float* ws;              // row-major weights: their scales (else the bundles')
  const int32_t* active;
  const int32_t* n_active;
  int host_n;
  int16_t host_ids[kMaxExperts];
  uint8_t* hq;
  float* hs;
  void* y;
  int y_f32;
  float* part;                  // [CTAs][2][RP][256]
  int32_t* counters;            // [tiles][4], used when tiles are cut
  int32_t* err;
};
static_assert(sizeof(Fp8Params) <= 4096, "kernel parameters stay within 4 KB");

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ uint64_t globaltimer() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count));
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait of a converged warp (every lane polls, votes decide: the warp never diverges).
__device__ __forceinline__ bool warp_wait(uint64_t* b, uint32_t parity, int32_t* err, int code) {
  const uint32_t bar = smem_u32(b);
  if (__all_sync(0xffffffffu, mbar_try(bar, parity))) return true;
  const uint64_t t0 = globaltimer();
  for (uint32_t i = 1;; ++i) {
    if (__all_sync(0xffffffffu, mbar_try(bar, parity))) return true;
    if ((i & 255) == 0 && __any_sync(0xffffffffu, globaltimer() - t0 > kWaitNs)) {
      if ((threadIdx.x & 31) == 0) atomicExch(err, code);
      return false;
    }
  }
}
__device__ __forceinline__ void bulk_g2s(uint32_t dst, const void* src, uint32_t bytes,
                                         uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      ::"r"(dst), "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                       uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t pred = 0;
  asm volatile(
      "{\n.reg .pred p;\n.reg .b32 r;\nelect.sync r|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(pred));
  return pred != 0;
}
// Shared-memory matrix descriptor: K-major, 128-byte swizzle, 8-row groups 1024 B apart.
__device__ __forceinline__ uint64_t sdesc_sw128(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)1 << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
// Instruction descriptor of kind::f8f6f4: E4M3 A and B (type 0), fp32 D, both K-major, M x N.
__device__ __forceinline__ uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_fp8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// 32 columns of the warp's 32 lanes, without and with the wait.
__device__ __forceinline__ void tmem_ld32_nw(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr));
}
// Waits for this thread's TMEM loads; the registers are tied to the wait so that no use of them
// is scheduled above it.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
        "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
        "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]),
        "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
        "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]),
        "+r"(r[31])
      :
      : "memory");
}
// acc[2i], acc[2i+1] += v[2i], v[2i+1] times f, as packed fp32 pairs
__device__ __forceinline__ void fma32(uint64_t* acc, const uint32_t (&v)[32], uint64_t f) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    uint64_t p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "r"(v[2 * i]), "r"(v[2 * i + 1]));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc[i]) : "l"(p), "l"(f));
  }
}
__device__ __forceinline__ float2 unpack(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t pack(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}

// silu(g) * u with the hardware exponential and reciprocal (relative error ~1e-6, far below
// E4M3's step); for g below about -88 e^-g is infinite and the quotient -0, the limit of silu.
__device__ __forceinline__ float silu_mul(float g, float u) {
  return __fdividef(g, 1.f + __expf(-g)) * u;
}

__device__ __forceinline__ int expert_of(const Fp8Params& p, int a) {
  return p.host_n >= 0 ? p.host_ids[a] : p.active ? p.active[a] : a;
}
// Rows [r0, r1) of expert e clipped to [0, max_rows); true when the clip changed anything.
__device__ __forceinline__ bool expert_rows(const Fp8Params& p, int e, int& r0, int& r1) {
  const int a = p.offsets ? p.offsets[e] : 0, b = p.offsets ? p.offsets[e + 1] : p.max_rows;
  r0 = min(max(a, 0), p.max_rows);
  r1 = min(max(b, r0), p.max_rows);
  return r0 != a || r1 != b;
}

// The CTA's share of the steps: whole tiles CTA, CTA + G, ... or one range of all tiles' steps.
struct Walk {
  int KB, U, G, u, lo, hi;
  long long pos, end;
  bool cut;
  __device__ __forceinline__ Walk(int U_, int KB_) : KB(KB_), U(U_), G(gridDim.x) {
    cut = U < kRangeTiles * G;
    const long long W = (long long)U * KB;
    if (cut && W < G) G = (int)W;               // no empty ranges
    if ((int)blockIdx.x >= G) {
      pos = end = 0;
      return;
    }
    pos = cut ? (long long)blockIdx.x * W / G : (long long)blockIdx.x * KB;
    end = cut ? (long long)(blockIdx.x + 1) * W / G : W;
  }
  __device__ __forceinline__ bool next() {
    if (pos >= end) return false;
    u = (int)(pos / KB);
    lo = (int)(pos - (long long)u * KB);
    hi = cut ? (int)min((long long)KB, lo + (end - pos)) : KB;
    pos += cut ? hi - lo : (long long)G * KB;
    return true;
  }
};

struct Tile {
  int e, nt, r0, rows;
};
__device__ __forceinline__ Tile tile_of(const Fp8Params& p, const int* pref, int n_act, int u) {
  int lo = 0, hi = n_act - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pref[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  Tile t;
  t.e = expert_of(p, lo);
  int r0, r1;
  expert_rows(p, t.e, r0, r1);
  const int mts = (r1 - r0 + 127) >> 7, rem = u - pref[lo];
  t.nt = rem / mts;
  t.r0 = r0 + (rem - t.nt * mts) * 128;
  t.rows = min(128, r1 - t.r0);
  return t;
}

// FUSED: N = columns of h (gate rows 0..N-1, up rows N..2N-1).  PLAIN: row-major weights by TMA.
template <bool FUSED, bool PLAIN>
__global__ void __launch_bounds__(kThreads, 1) fp8_gemm_kernel(const __grid_constant__ Fp8Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  Ctl& c = *reinterpret_cast<Ctl*>(smem + kStages * kStageBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&c.full[s], 1);
      mbar_init(&c.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&c.tfull[b], 1);
      mbar_init(&c.tempty[b], 8);
    }
    for (int q = 0; q < 4; ++q) mbar_init(&c.pair[q], 2);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&c.tmem)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pdl_wait();
  const int n_act = p.host_n >= 0 ? p.host_n : p.active ? *p.n_active : p.E;
  if (warp == 2) {
    // prefix of the experts' tile counts
    int carry = 0;
    for (int base = 0; base < n_act; base += 32) {
      const int a = base + lane;
      int cnt = 0;
      if (a < n_act) {
        int r0, r1;
        if (expert_rows(p, expert_of(p, a), r0, r1)) atomicExch(p.err, 8);
        cnt = p.NT * ((r1 - r0 + 127) >> 7);
      }
      int incl = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (a < n_act) c.pref[a] = carry + incl - cnt;
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) c.pref[n_act] = carry;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;
  const int U = c.pref[n_act], KB = p.KB;
  Walk wk(U, KB);

  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    while (ok && wk.next()) {
      const Tile t = tile_of(p, c.pref, n_act, wk.u);
      const int nsub = t.rows > 96 ? 0 : (t.rows + 31) >> 5;
      const int n0 = t.nt * (FUSED ? 128 : 256);
      const bool two = FUSED || n0 + 128 < p.N;
      const char *w0 = nullptr, *w1 = nullptr;
      if (!PLAIN) {
        const char* b = static_cast<const char*>(p.dev_tab ? p.dev_tab[t.e] : p.tab.p[t.e]);
        w0 = b + p.w_off + (size_t)(n0 >> 7) * KB * kFp8TileBytes;
        w1 = w0 + (size_t)(FUSED ? p.N >> 7 : 1) * KB * kFp8TileBytes;
      }
      for (int kb = wk.lo; kb < wk.hi; ++kb) {
        if (!(ok = warp_wait(&c.empty[stage], phase ^ 1, p.err, 1))) break;
        uint64_t* fb = &c.full[stage];
        const uint32_t sa = smem_u32(smem + stage * kStageBytes), sb = sa + kABytes;
        if (elect_one()) {
          mbar_expect_tx(fb, (nsub ? nsub * 4096 : kABytes) + (two ? kBBytes : kFp8TileBytes));
          if (PLAIN) {
            tma_2d(sb, &p.tm_w, kb * 128, t.e * p.N + n0, fb);
            if (two) tma_2d(sb + kFp8TileBytes, &p.tm_w, kb * 128, t.e * p.N + n0 + 128, fb);
          } else {
            bulk_g2s(sb, w0 + (size_t)kb * kFp8TileBytes, kFp8TileBytes, fb);
            if (two)
              bulk_g2s(sb + kFp8TileBytes, w1 + (size_t)kb * kFp8TileBytes, kFp8TileBytes, fb);
          }
          if (nsub) {
            // 32-row boxes stacked at 4 KB: the same swizzled layout as one box of all rows
            for (int s = 0; s < nsub; ++s)
              tma_2d(sa + 4096 * s, &p.tm_x32, kb * 128, t.r0 + 32 * s, fb);
          } else {
            tma_2d(sa, &p.tm_x, kb * 128, t.r0, fb);
          }
        }
        __syncwarp();
        if (++stage == kStages) { stage = 0; phase ^= 1; }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    int stage = 0, buf = 0;
    uint32_t phase = 0, tphase = 0;
    bool ok = true;
    while (ok && wk.next()) {
      const Tile t = tile_of(p, c.pref, n_act, wk.u);
      const int left = FUSED ? 256 : p.N - t.nt * 256;
      const uint32_t idesc = idesc_e4m3(128, min(256, (left + 15) & ~15));
      for (int kb = wk.lo; kb < wk.hi; ++kb) {
        if (!(ok = warp_wait(&c.tempty[buf], tphase ^ 1, p.err, 2))) break;
        if (!(ok = warp_wait(&c.full[stage], phase, p.err, 3))) break;
        const uint32_t sa = smem_u32(smem + stage * kStageBytes);
        const uint64_t da = sdesc_sw128(sa), db = sdesc_sw128(sa + kABytes);
        if (elect_one()) {
          tc_fence_after();
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_fp8(tmem + buf * kAccCols, da + 2 * j, db + 2 * j, idesc, j > 0);
          mma_commit(&c.empty[stage]);
          mma_commit(&c.tfull[buf]);
        }
        __syncwarp();
        if (++stage == kStages) { stage = 0; phase ^= 1; }
        buf ^= 1;
        if (buf == 0) tphase ^= 1;
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ scaling and epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsHigh));
    const int q = warp & 3, half = (warp - 4) >> 2, r = q * 32 + lane;
    int buf = 0, flip = 0;
    uint32_t tphase = 0, pphase = 0;
    bool ok = true;
    // the two warps of a lane quarter meet (bounded, as every wait)
    auto meet = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.pair[q]);
      const bool w = warp_wait(&c.pair[q], pphase, p.err, 5);
      pphase ^= 1;
      return w;
    };
    while (ok && wk.next()) {
      const Tile t = tile_of(p, c.pref, n_act, wk.u);
      const int n0 = t.nt * (FUSED ? 128 : 256);
      const bool two = FUSED || n0 + 128 < p.N, here = q * 32 < t.rows, mine = r < t.rows;
      const int NB = (p.N + 127) >> 7;
      const float* sw0;
      if (PLAIN) {
        sw0 = p.ws + ((size_t)t.e * NB + (n0 >> 7)) * KB;
      } else {
        const char* b = static_cast<const char*>(p.dev_tab ? p.dev_tab[t.e] : p.tab.p[t.e]);
        sw0 = reinterpret_cast<const float*>(b + p.s_off) + (size_t)(n0 >> 7) * KB;
      }
      const float* sw1 = two ? sw0 + (size_t)(FUSED ? NB : 1) * KB : sw0;
      const float* sx = p.xs + (size_t)(t.r0 + (mine ? r : 0)) * KB;
      uint64_t acc[64];   // pairs of columns: 32 of the first weight tile, 32 of the second
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0;
      float x = __ldg(sx + wk.lo), a = __ldg(sw0 + wk.lo), b = __ldg(sw1 + wk.lo);
      for (int kb = wk.lo; kb < wk.hi; ++kb) {
        const float f0 = x * a, f1 = x * b;
        if (kb + 1 < wk.hi) {
          x = __ldg(sx + kb + 1);
          a = __ldg(sw0 + kb + 1);
          b = __ldg(sw1 + kb + 1);
        }
        if (!(ok = warp_wait(&c.tfull[buf], tphase, p.err, 4))) break;
        if (here) {
          tc_fence_after();
          const uint32_t ta = tmem + ((uint32_t)(q * 32) << 16) + buf * kAccCols + half * 64;
          uint32_t v[32], v2[32];
          tmem_ld32_nw(ta, v);
          tmem_wait_ld(v);
          tmem_ld32_nw(ta + 32, v2);
          const uint64_t p0 = pack(f0, f0), p1 = pack(f1, f1);
          fma32(acc, v, p0);
          tmem_wait_ld(v2);
          if (two) tmem_ld32_nw(ta + 128, v);
          fma32(acc + 16, v2, p0);
          if (two) {
            tmem_wait_ld(v);
            tmem_ld32_nw(ta + 160, v2);
            fma32(acc + 32, v, p1);
            tmem_wait_ld(v2);
            fma32(acc + 48, v2, p1);
          }
          tc_fence_before();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(&c.tempty[buf]);
        buf ^= 1;
        if (buf == 0) tphase ^= 1;
      }
      if (!ok) break;
      if (!here) continue;
      if (wk.lo > 0 || wk.hi < KB) {
        // a piece of the tile: its sums to this CTA's slot (0: begins inside the tile, 1: ends
        // inside it); the last piece's CTA adds them all in range order
        const size_t slot = (size_t)p.RP * 256;
        float* mp = p.part + ((size_t)blockIdx.x * 2 + (wk.lo > 0 ? 0 : 1)) * slot +
                    (size_t)r * 256 + half * 128;
        if (mine) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float2 u0 = unpack(acc[2 * i]), u1 = unpack(acc[2 * i + 1]);
            __stcg(reinterpret_cast<float4*>(mp) + i, make_float4(u0.x, u0.y, u1.x, u1.y));
          }
        }
        const long long W = (long long)U * KB, first = (long long)wk.u * KB;
        const int c_lo = (int)(((first + 1) * wk.G - 1) / W);
        const int c_hi = (int)(((first + KB) * wk.G - 1) / W);
        __threadfence();
        if (!(ok = meet())) break;
        if (half == 0 && lane == 0) {
          int32_t* ctr = p.counters + (size_t)wk.u * 4 + q;
          const int l = atomicAdd(ctr, 1) == c_hi - c_lo;
          if (l) *ctr = 0;
          c.last[q] = l;
          __threadfence();
        }
        if (!(ok = meet())) break;
        if (!c.last[q]) continue;
        __threadfence();
#pragma unroll
        for (int i = 0; i < 64; ++i) acc[i] = 0;
        if (mine) {
          for (int cc = c_lo; cc <= c_hi; ++cc) {
            const bool inside = (long long)cc * W / wk.G > first;
            const float4* op = reinterpret_cast<const float4*>(
                p.part + ((size_t)cc * 2 + (inside ? 0 : 1)) * slot + (size_t)r * 256 + half * 128);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float4 o = __ldcg(op + i);
              const float2 u0 = unpack(acc[2 * i]), u1 = unpack(acc[2 * i + 1]);
              acc[2 * i] = pack(u0.x + o.x, u0.y + o.y);
              acc[2 * i + 1] = pack(u1.x + o.z, u1.y + o.w);
            }
          }
        }
      }
      const size_t row = (size_t)t.r0 + r;
      if (FUSED) {
        // h over the gate pairs; the row's largest |h| over both warps' 64 columns
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float2 g = unpack(acc[i]), u = unpack(acc[32 + i]);
          const float h0 = silu_mul(g.x, u.x), h1 = silu_mul(g.y, u.y);
          m = fmaxf(m, fmaxf(fabsf(h0), fabsf(h1)));
          acc[i] = pack(h0, h1);
        }
        c.amax[flip][half][r] = m;
        if (!(ok = meet())) break;
        m = fmaxf(fmaxf(m, c.amax[flip][half ^ 1][r]), kFp8MinAmax);
        flip ^= 1;
        if (mine) {
          const float inv = __fdiv_rn(kFp8Max, m);
          uint4* dst = reinterpret_cast<uint4*>(p.hq + row * p.N + n0 + half * 64);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 u0 = unpack(acc[8 * i + 2 * j]), u1 = unpack(acc[8 * i + 2 * j + 1]);
              o[j] = fp8_pack4(u0.x, u0.y, u1.x, u1.y, inv);
            }
            dst[i] = make_uint4(o[0], o[1], o[2], o[3]);
          }
          if (half == 0) p.hs[row * NB + (n0 >> 7)] = __fdiv_rn(m, kFp8Max);
        }
      } else if (mine) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int col = n0 + 128 * w + 64 * half;
          const int left = p.N - col;             // columns from `col` on
          const size_t at = row * p.N + col;
          if (p.y_f32) {
            float* y = static_cast<float*>(p.y) + at;
            const bool vec = (p.N & 3) == 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 u0 = unpack(acc[32 * w + 2 * i]), u1 = unpack(acc[32 * w + 2 * i + 1]);
              if (vec) {
                if (4 * i < left)
                  reinterpret_cast<float4*>(y)[i] = make_float4(u0.x, u0.y, u1.x, u1.y);
              } else {
                if (4 * i < left) y[4 * i] = u0.x;
                if (4 * i + 1 < left) y[4 * i + 1] = u0.y;
                if (4 * i + 2 < left) y[4 * i + 2] = u1.x;
                if (4 * i + 3 < left) y[4 * i + 3] = u1.y;
              }
            }
          } else {
            uint16_t* y = static_cast<uint16_t*>(p.y) + at;
            const bool vec = (p.N & 7) == 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              uint32_t o[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 u = unpack(acc[32 * w + 4 * i + j]);
                o[j] = float2_to_bf16x2(u.x, u.y);
              }
              if (vec) {
                if (8 * i < left) reinterpret_cast<uint4*>(y)[i] = make_uint4(o[0], o[1], o[2], o[3]);
              } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  if (8 * i + j < left) y[8 * i + j] = (uint16_t)(o[j >> 1] >> (16 * (j & 1)));
              }
            }
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols));
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }
  return fn;
}

// Map of byte rows [rows][K] with boxes of box_rows x 128 bytes, 128-byte swizzle; reads past K
// or the last row give zeros.
bool encode_rows(CUtensorMap* m, const uint8_t* base, int K, size_t rows, int box_rows) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)K};
  cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

template <bool FUSED, bool PLAIN>
int launch_variant(const Fp8Params& p, cudaStream_t st) {
  static bool attr = false;
  if (!attr) {
    MOE_CUDA_TRY(cudaFuncSetAttribute(fp8_gemm_kernel<FUSED, PLAIN>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem));
    attr = true;
  }
  MOE_LAUNCH_PDL((fp8_gemm_kernel<FUSED, PLAIN>), dim3(sm_count()), dim3(kThreads), kSmem, st, p);
  MOE_COUNT_LAUNCH();
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace

Fp8Plan plan_fp8(const Fp8Args& a) {
  Fp8Plan pl{};
  const int G = sm_count();
  pl.part_elems = (size_t)G * 2 * std::min(std::max(a.max_rows, 1), 128) * 256;
  pl.counter_elems = (size_t)4 * kRangeTiles * G;
  return pl;
}

int launch_fp8(const Fp8Args& a, const Fp8Plan&, float* part, int32_t* counters, int32_t* err,
               cudaStream_t st) {
  if (a.max_rows <= 0 || a.host_n == 0) return MOE_OK;
  if (!encode_fn()) return MOE_ERR_UNSUPPORTED;
  Fp8Params p{};
  if (!encode_rows(&p.tm_x, a.xq, a.K, a.max_rows, 128) ||
      !encode_rows(&p.tm_x32, a.xq, a.K, a.max_rows, 32) ||
      (a.w && !encode_rows(&p.tm_w, a.w, a.K, (size_t)a.E * a.N, 128)))
    return MOE_ERR_INVALID_ARG;
  p.xs = a.xs; p.offsets = a.offsets; p.E = a.E; p.N = a.N; p.K = a.K;
  p.KB = ceil_div(a.K, 128); p.NT = a.fused ? a.N / 128 : ceil_div(a.N, 256);
  p.max_rows = a.max_rows; p.RP = std::min(a.max_rows, 128);
  if (a.tab) p.tab = *a.tab;
  p.dev_tab = a.dev_tab; p.w_off = a.w_off; p.s_off = a.s_off; p.ws = a.ws;
  p.active = a.active; p.n_active = a.n_active; p.host_n = a.host_n;
  for (int i = 0; i < (a.host_n > 0 ? a.host_n : 0); ++i) p.host_ids[i] = (int16_t)a.host_ids[i];
  p.hq = a.hq; p.hs = a.hs; p.y = a.y; p.y_f32 = a.y_f32;
  p.part = part; p.counters = counters; p.err = err;
  if (a.fused) return launch_variant<true, false>(p, st);
  return a.w ? launch_variant<false, true>(p, st) : launch_variant<false, false>(p, st);
}

}  // namespace moe
