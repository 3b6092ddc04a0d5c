// Router product of a large group-limited batch on the tensor cores (tcgen05 + TMEM): the fp32
// router is three bf16 pieces hi + mid + lo (router_prep_kernel's image), and
//
//   logit[t][e] = sum over blocks of 64 h of  x[t] . (hi + mid + lo)[e]   of that block,
//
// each block's 192 products a column summed by the tensor cores from zero and added in fp32
// registers.  (One sum over all 3 H products inside the tensor cores is cut off, not rounded, at
// every addition: the weights are off by 2.6e-6 at H = 7168 that way, by 7e-8 this way.)
//
// Tile: 128 tokens (M, a TMEM lane each) x up to 256 router columns (N), split over H so that the
// tiles fill the GPU; a CTA runs one part of one tile, 384 threads:
//   warp 0      producer: per block one 2-D TMA box of the tokens' rows (16 KB, 128-byte swizzle)
//               and per piece one or two 16 KB image tiles by bulk copy, in rings of their own;
//   warp 1      MMA issuer: per block 12 tcgen05.mma (K = 16) into one of two TMEM buffers;
//   warps 4-11  two per TMEM lane quarter: tcgen05.ld and an fp32 add, 128 accumulators a thread;
//               at the end the sums leave through shared memory by rows.
//
// Bound by shared memory and its filling: a block reads 12 x 12 KB of operands and takes in 112 KB
// for 1536 clocks of tensor work.  8192 tokens x 7168 x 256 columns (two parts, 128 CTAs): 68 us,
// 1.3 PFLOP/s of the three pieces' products, tensor pipe 70% busy on the SMs in use (ungrouped
// routing's kernel, weights as M: 94 us).
// Every wait is bounded (2 s; then an error word and the end).
#include "route.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int kA = 3, kB = 5;                   // ring slots
constexpr int kABytes = 16384, kBBytes = 32768;
constexpr int kThreads = 384;
constexpr int kRegsLow = 56, kRegsHigh = 224;   // 128 * 56 + 256 * 224 = 384 * 168
static_assert(128 * kRegsLow + 256 * kRegsHigh <= kThreads * 168, "within the launch's registers");
constexpr int kAccCols = 256, kTmemCols = 512;

struct TcParams {
  CUtensorMap tm_x;       // x [T][H] bf16, boxes of 128 rows x 64 columns
  const uint16_t* img;    // [Mpad / 128][3][KT] tiles of 128 columns x 64 h
  float* part;            // [S][T][Mpad]
  int32_t* err;
  int T, Mpad, KT, per;   // KT = H / 64 blocks, `per` of them a part
};

struct alignas(16) Ctl {
  uint64_t afull[kA], aempty[kA], bfull[kB], bempty[kB], tfull[2], tempty[2], drain;
  uint32_t tmem;
};
constexpr int kRing = kA * kABytes + kB * kBBytes;
constexpr int kSmem = kRing + 1024 + (int)sizeof(Ctl);
static_assert(kSmem <= 232448, "over the 227 KB shared-memory limit of a CTA");
static_assert(8 * 32 * 128 * 4 <= kRing, "the sums leave through the rings");

__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
// 32 columns of the warp's 32 lanes, without the wait.
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
// acc[i] += v[i]; volatile, as the load and its wait are, so that no use of v moves above the wait.
__device__ __forceinline__ void add32(float* acc, const uint32_t (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 16; ++i)
    asm volatile(
        "{\n.reg .b64 t, a;\nmov.b64 t, {%2, %3};\nmov.b64 a, {%0, %1};\n"
        "add.rn.f32x2 a, a, t;\nmov.b64 {%0, %1}, a;\n}\n"
        : "+f"(acc[2 * i]), "+f"(acc[2 * i + 1])
        : "r"(v[2 * i]), "r"(v[2 * i + 1]));
}

// blockIdx: tile of 128 tokens, columns 256 y.., part of H.
__global__ void __launch_bounds__(kThreads, 1)
router_tc_kernel(const __grid_constant__ TcParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* const ring_b = smem + kA * kABytes;
  Ctl& c = *reinterpret_cast<Ctl*>(smem + kRing);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = blockIdx.x * 128, mt0 = blockIdx.y * 2;
  const int lo = blockIdx.z * p.per, hi = min(p.KT, lo + p.per);
  const bool two = (mt0 + 1) * 128 < p.Mpad;    // a second tile of 128 columns
  if (threadIdx.x == 0) {
    for (int s = 0; s < kA; ++s) {
      mbar_init(&c.afull[s], 1);
      mbar_init(&c.aempty[s], 1);
    }
    for (int s = 0; s < kB; ++s) {
      mbar_init(&c.bfull[s], 1);
      mbar_init(&c.bempty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&c.tfull[b], 1);
      mbar_init(&c.tempty[b], 8);
    }
    mbar_init(&c.drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (threadIdx.x == 32) prefetch_map(&p.tm_x);
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&c.tmem)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;
  pdl_wait();
  pdl_trigger();
  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const int who = !elect_one();               // 0: the lane that waits and issues
    int as = 0, bs = 0, na = 0, nb = 0;
    uint32_t ap = 0, bp = 0;
    bool ok = true;
    for (int kt = lo; ok && kt < hi; ++kt) {
      if (!(ok = lead_wait(&c.aempty[as], ap ^ 1, p.err, 1, who))) break;
      if (elect_one()) {
        mbar_expect_tx(&c.afull[as], kABytes);
        tma_2d(smem_u32(smem + as * kABytes), &p.tm_x, kt * 64, t0, &c.afull[as]);
      }
      __syncwarp();
      ++na;
      if (++as == kA) { as = 0; ap ^= 1; }
      for (int q = 0; q < 3; ++q) {
        if (!(ok = lead_wait(&c.bempty[bs], bp ^ 1, p.err, 2, who))) break;
        if (elect_one()) {
          mbar_expect_tx(&c.bfull[bs], two ? kBBytes : kBBytes / 2);
          for (int i = 0; i < 1 + (int)two; ++i)
            bulk_g2s(smem_u32(ring_b + bs * kBBytes + i * (kBBytes / 2)),
                     p.img + ((size_t)(mt0 + i) * (3 * p.KT) + q * p.KT + kt) * 8192, kBBytes / 2,
                     &c.bfull[bs]);
        }
        __syncwarp();
        ++nb;
        if (++bs == kB) { bs = 0; bp ^= 1; }
      }
    }
    // after a failed wait, copies may still be on their way: wait (bounded) for the last of each
    // slot
    for (int i = 0; !ok && i < min(na, kA); ++i) {
      if (--as < 0) { as = kA - 1; ap ^= 1; }
      lead_wait(&c.afull[as], ap, p.err, 1, who);
    }
    for (int i = 0; !ok && i < min(nb, kB); ++i) {
      if (--bs < 0) { bs = kB - 1; bp ^= 1; }
      lead_wait(&c.bfull[bs], bp, p.err, 2, who);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // (bf16 A and B, fp32 D, 128 x 256; without a second tile its columns take what the slot held
    // and are not stored)
    const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((256u >> 3) << 17) |
                           ((128u >> 4) << 24);
    const int who = !elect_one();
    int as = 0, bs = 0, buf = 0;
    uint32_t ap = 0, bp = 0, tp = 0;
    bool ok = true;
    for (int kt = lo; ok && kt < hi; ++kt) {
      if (!(ok = lead_wait(&c.tempty[buf], tp ^ 1, p.err, 3, who))) break;
      if (!(ok = lead_wait(&c.afull[as], ap, p.err, 4, who))) break;
      const uint64_t da = sdesc_sw128(smem_u32(smem + as * kABytes));
      const uint32_t d = tmem + buf * kAccCols;
      for (int q = 0; q < 3; ++q) {
        if (!(ok = lead_wait(&c.bfull[bs], bp, p.err, 4, who))) break;
        const uint64_t db = sdesc_sw128(smem_u32(ring_b + bs * kBBytes));
        if (elect_one()) {
          tc_fence_after();
#pragma unroll
          for (int j = 0; j < 4; ++j) mma_bf16(d, da + 2 * j, db + 2 * j, idesc, q + j > 0);
          mma_commit(&c.bempty[bs]);
          if (q == 2) {
            mma_commit(&c.aempty[as]);
            mma_commit(&c.tfull[buf]);
          }
        }
        __syncwarp();
        if (++bs == kB) { bs = 0; bp ^= 1; }
      }
      if (++as == kA) { as = 0; ap ^= 1; }
      buf ^= 1;
      if (buf == 0) tp ^= 1;
    }
    if (!ok) {   // after a failed wait: the products still running write TMEM until they end
      if (elect_one()) mma_commit(&c.drain);
      __syncwarp();
      lead_wait(&c.drain, 0, p.err, 7, who);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ sums
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsHigh));
    const int q = warp & 3, half = (warp - 4) >> 2;   // lanes 32 q.., columns 128 half..
    float acc[128];
#pragma unroll
    for (int i = 0; i < 128; ++i) acc[i] = 0.f;
    int buf = 0;
    uint32_t tp = 0;
    bool ok = true;
    for (int kt = lo; kt < hi; ++kt) {
      if (!(ok = warp_wait(&c.tfull[buf], tp, p.err, 5))) break;
      tc_fence_after();
      const uint32_t ta = tmem + ((uint32_t)(q * 32) << 16) + buf * kAccCols + half * 128;
      uint32_t v[32], w[32];
      tmem_ld32_nw(ta, v);
      tmem_wait_ld();
      tmem_ld32_nw(ta + 32, w);
      add32(acc, v);
      tmem_wait_ld();
      tmem_ld32_nw(ta + 64, v);
      add32(acc + 32, w);
      tmem_wait_ld();
      tmem_ld32_nw(ta + 96, w);
      add32(acc + 64, v);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      warp_arrive(&c.tempty[buf], lane);
      add32(acc + 96, w);
      buf ^= 1;
      if (buf == 0) tp ^= 1;
    }
    // The last products are done, so the rings are free: the warp's 32 rows of 128 columns leave
    // through 16 KB of them, a row at a time (16-byte piece i of row l at i ^ l).
    if (ok && (half == 0 || two)) {
      float4* box = reinterpret_cast<float4*>(smem + (warp - 4) * 16384);
#pragma unroll
      for (int i = 0; i < 32; ++i)
        box[lane * 32 + (i ^ lane)] =
            make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
      __syncwarp();
      const int row = t0 + q * 32, have = min(32, p.T - row);
      float* out = p.part + ((size_t)blockIdx.z * p.T + row) * p.Mpad + (mt0 + half) * 128;
#pragma unroll 4
      for (int l = 0; l < have; ++l)
        reinterpret_cast<float4*>(out + (size_t)l * p.Mpad)[lane] = box[l * 32 + (lane ^ l)];
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols));
}

}  // namespace

// Parts of H: as many as leave each at least four blocks and fill the GPU once, at most 16 (the
// gating kernel sums them).
int route_tc_parts(int T, int H, int Mpad) {
  const int tiles = ceil_div(T, 128) * ceil_div(Mpad, 256), KT = H / 64;
  const int S = std::max(1, std::min({16, sm_count() / tiles, KT / 4}));
  return ceil_div(KT, ceil_div(KT, S));
}

int launch_route_tc(const uint16_t* x, int T, int H, const uint16_t* img, int Mpad, int S,
                    float* part, int32_t* err, cudaStream_t st) {
  auto enc = encode_fn();
  if (!enc) return MOE_ERR_UNSUPPORTED;
  TcParams p{};
  cuuint64_t dims[2] = {(cuuint64_t)H, (cuuint64_t)T};
  cuuint64_t strides[1] = {(cuuint64_t)H * 2};
  cuuint32_t box[2] = {64, 128}, estr[2] = {1, 1};
  if (enc(&p.tm_x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(x), dims, strides,
          box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return MOE_ERR_INVALID_ARG;
  p.img = img; p.part = part; p.err = err; p.T = T; p.Mpad = Mpad; p.KT = H / 64;
  p.per = ceil_div(p.KT, S);
  static bool attr = false;
  if (!attr) {
    MOE_CUDA_TRY(cudaFuncSetAttribute(router_tc_kernel,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem));
    attr = true;
  }
  MOE_LAUNCH_NEXT(true, router_tc_kernel, dim3(ceil_div(T, 128), ceil_div(Mpad, 256), S),
                  dim3(kThreads), kSmem, st, p);
  MOE_COUNT_LAUNCH();
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace moe
