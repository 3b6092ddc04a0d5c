// Products of few rows with 4-bit weights: what the kernel for up to eight token rows and the one for
// more share (internal to libmoe).  See gemv_int4.cu for the mathematics.
#pragma once
#include "common.cuh"
#include "route.cuh"
#include "tc_ptx.cuh"

namespace moe {

constexpr int kGvWarps = 8, kGvThreads = kGvWarps * 32;
constexpr int kGvStep = 256;             // codes of K of a box (128 bytes a row)
constexpr int kGvErrWait = 6;            // error word: a bounded wait ran out of time

struct GemvArgs {
  const uint16_t* x;
  const uint16_t* s;
  const uint8_t* z;
  const int32_t* offsets;
  int E, N, K, ng, max_rows;
  bool f32, wide;                              // wide: a step's scales of a row are one aligned load
  void* y;
  int32_t* err;
};

static __device__ __forceinline__ void mma_bf16(float* d, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The four pairs of a code word as (q - z) 2^-6; nz: -z 2^-6 in both halves.
static __device__ __forceinline__ void code_pairs(uint32_t w, uint32_t nz, uint32_t (&p)[4]) {
  const uint32_t h = w >> 8;
  const uint32_t v[4] = {w & 0x000F000Fu, w & 0x00F000F0u, h & 0x000F000Fu, h & 0x00F000F0u};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("fma.rn.bf16x2 %0, %1, %2, %3;"
        : "=r"(p[i])
        : "r"(v[i]), "r"(i & 1 ? 0x7D007D00u : 0x7F007F00u), "r"(nz));
}
// -z 2^-6 in both halves, z = byte I of `zeros`, 0..127: 128 + z by its bits, then an exact fma.
template <int I>
static __device__ __forceinline__ uint32_t zero_pair(uint32_t zeros) {
  const uint32_t v = __byte_perm(zeros, 0x43434343u, 0x4040 | (I << 8) | I);
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(v), "r"(0xBC80BC80u), "r"(0x40004000u));
  return d;
}

struct GemvExperts {
  int lo[kMaxExperts], hi[kMaxExperts];        // token rows of the experts that have some
  int passes[kMaxExperts + 1];                 // passes over the weights of the experts before
  int eights[kMaxExperts + 1];                 // eights of token rows of the experts before
  int16_t act[kMaxExperts];
  int wsum[3][kMaxExperts / 32];
};

// The experts with rows, ascending, with their ranges; a pass takes `per` eights of token rows.
// Returns how many there are; their passes and eights stand behind the last one's.  `record`: CTA 0
// writes to the error word whether a range was clipped.  By every thread of the CTA.
static __device__ int active_experts(const GemvArgs& a, GemvExperts& sm, int per, bool record) {
  const int e = threadIdx.x, lane = e & 31, warp = e >> 5;
  int b = 0, n = 0;
  bool clipped = false;
  if (e < a.E) {
    b = a.offsets ? __ldg(a.offsets + e) : 0;
    const int end = a.offsets ? __ldg(a.offsets + e + 1) : a.max_rows;
    const int cb = min(max(b, 0), a.max_rows), ce = min(max(end, 0), a.max_rows);
    clipped = end > b && (cb != b || ce != end);
    b = cb;
    n = max(ce - cb, 0);
  }
  const int eights = (n + 7) / 8, passes = (eights + per - 1) / per;
  int be = eights, bp = passes;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, be, o), w = __shfl_up_sync(0xffffffffu, bp, o);
    if (lane >= o) {
      be += v;
      bp += w;
    }
  }
  const unsigned m = __ballot_sync(0xffffffffu, n > 0);
  if (lane == 31 && warp < kMaxExperts / 32) {
    sm.wsum[0][warp] = __popc(m);
    sm.wsum[1][warp] = be;
    sm.wsum[2][warp] = bp;
  }
  be -= eights;
  bp -= passes;
  const int any = __syncthreads_or(clipped);
  if (record && blockIdx.x == 0 && threadIdx.x == 0) *a.err = any ? 8 : 0;
  int at = __popc(m & ((1u << lane) - 1u)), total = 0, all_e = 0, all_p = 0;
#pragma unroll
  for (int i = 0; i < kMaxExperts / 32; ++i) {
    at += i < warp ? sm.wsum[0][i] : 0;
    be += i < warp ? sm.wsum[1][i] : 0;
    bp += i < warp ? sm.wsum[2][i] : 0;
    total += sm.wsum[0][i];
    all_e += sm.wsum[1][i];
    all_p += sm.wsum[2][i];
  }
  if (n > 0) {
    sm.act[at] = (int16_t)e;
    sm.lo[at] = b;
    sm.hi[at] = b + n;
    sm.passes[at] = bp;
    sm.eights[at] = be;
  }
  if (threadIdx.x == 0) {
    sm.passes[total] = all_p;
    sm.eights[total] = all_e;
  }
  __syncthreads();
  return total;
}
// The last of n_act experts whose count `before` starts at or before i.
static __device__ __forceinline__ int find_expert(const int* before, int n_act, int i) {
  int a = 0, b = n_act;
  while (b - a > 1) {
    const int c = (a + b) >> 1;
    if (before[c] <= i) a = c;
    else b = c;
  }
  return a;
}

static __device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2,
                                       uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}


// The words of four 8 x 16-byte blocks: a lane gets word t of row gr of each.
static __device__ __forceinline__ void load_words(uint32_t (&w)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(addr)
               : "memory");
}
static __device__ __forceinline__ uint4 load_shared(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
// A token row's eight values in the order of a word's pairs: (0, 4), (1, 5), (2, 6), (3, 7).
static __device__ __forceinline__ uint4 pair_order(const uint4& v) {
  return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                    __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
}

// A TMA map of the codes [E][N][K / 2] with boxes of `rows` weight rows x 256 codes, swizzled.
inline bool encode_weights(CUtensorMap* m, const uint8_t* w, int E, int N, int K, int rows) {
  const cuuint64_t row = (cuuint64_t)K / 2;
  const cuuint64_t dims[3] = {row, (cuuint64_t)N, (cuuint64_t)E};
  const cuuint64_t strides[2] = {row, row * N};
  const cuuint32_t box[3] = {kGvStep / 2, (cuuint32_t)rows, 1}, step[3] = {1, 1, 1};
  auto enc = encode_fn();
  return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(w), dims, strides, box,
                    step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// moe_grouped_gemv_int4 for more than eight token rows an expert (gemv_int4_rows.cu); packed: scratch of
// gemv_packed_bytes.
size_t gemv_packed_bytes(int max_rows, int E, int K);
int launch_gemv_rows(const GemvArgs& a, const uint8_t* w, int group, void* packed, cudaStream_t st);

}  // namespace moe
