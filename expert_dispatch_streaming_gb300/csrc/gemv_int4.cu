// moe_grouped_gemv_int4: products of few rows with 4-bit weights.
//
//   y[r][n] = sum_g s[e][n][g] * sum_{k in group g} (q[e][n][k] - z[e][n][g]) x[r][k]
//
// for the rows r of expert e; q a 4-bit code, s a bf16 scale and z a zero point of `G` codes along
// K.  A weight is read once and used for at most a few rows, so reading the codes bounds it.
//
// m16n8k16 products of bf16 values: 16 weight rows against eight token rows.  q - z is exact in
// bf16: 0x4300 | q is 128 + q, and (128 + q) - (128 + z) loses nothing.  One group's products are
// added in fp32 before its scale is applied, in fp32, as moe_grouped_gemm_fp8 does.
//
// The order of K inside a product is free as long as both operands agree.  A lane's codes for
// weight row n are the 8 of one 32-bit word, words of the four lanes of a row next to each other:
// nibble pairs (i, i + 4) come out of one shift and one mask, and the token row's eight values from
// one 16-byte load.  With 128-code groups a lane loads 16 bytes (four words of one group), with
// 64-code groups twice 8, with 32-code groups four times 4, so that the four lanes of a row hold
// the same group in every product.
//
// A CTA takes 16 weight rows of one expert, its eight warps 128-code steps of K in turn; the warps'
// sums are added in warp order in shared memory.
#include "common.cuh"
#include "route.cuh"

#include <type_traits>

namespace moe {
namespace {

constexpr int kGvWarps = 8, kGvThreads = kGvWarps * 32, kGvRows = 16, kGvStep = 128;

struct GemvArgs {
  const uint16_t* x;
  const uint8_t* w;
  const uint16_t* s;
  const uint8_t* z;
  const int32_t* offsets;
  int E, N, K, ng, max_rows;
  void* y;
  int32_t* err;
};

__device__ __forceinline__ void mma_bf16(float* d, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Codes I and I + 4 of a word as the bf16 pair q - z; zp: 128 + z in both halves.
template <int I>
__device__ __forceinline__ uint32_t code_pair(uint32_t word, uint32_t zp) {
  const uint32_t v = ((word >> (4 * I)) & 0x000F000Fu) | 0x43004300u;
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(zp));
  return d;
}

// The experts with rows, ascending, in `act`, their row ranges in lo / hi; returns their number.
// CTA 0 records in the error word whether a range was clipped.
__device__ int active_experts(const GemvArgs& a, int16_t* act, int* lo, int* hi, int* wsum) {
  const int e = threadIdx.x, lane = e & 31, warp = e >> 5;
  int b = 0, n = 0;
  bool clipped = false;
  if (e < a.E) {
    int end = a.max_rows;
    if (a.offsets) {
      b = __ldg(a.offsets + e);
      end = __ldg(a.offsets + e + 1);
    }
    const int cb = min(max(b, 0), a.max_rows), ce = min(max(end, 0), a.max_rows);
    clipped = end > b && (cb != b || ce != end);
    b = cb;
    n = max(ce - cb, 0);
  }
  const unsigned m = __ballot_sync(0xffffffffu, n > 0);
  if (lane == 0) wsum[warp] = __popc(m);
  const int any = __syncthreads_or(clipped);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = any ? 8 : 0;
  int at = __popc(m & ((1u << lane) - 1u)), total = 0;
#pragma unroll
  for (int i = 0; i < kGvWarps; ++i) {
    at += i < warp ? wsum[i] : 0;
    total += wsum[i];
  }
  if (n > 0) {
    act[at] = (int16_t)e;
    lo[at] = b;
    hi[at] = b + n;
  }
  __syncthreads();
  return total;
}

// G: codes a scale covers; RT: groups of eight token rows that pass through the weights together.
template <int G, bool ZERO, bool F32, int RT>
__global__ void __launch_bounds__(kGvThreads)
gemv_int4_kernel(const GemvArgs a) {
  constexpr int NG = kGvStep / G;          // groups of a step
  constexpr int WPL = G / 32;              // words of a lane in one group
  static_assert(kMaxExperts <= kGvThreads, "one thread per expert");
  __shared__ int16_t act[kMaxExperts];
  __shared__ int e_lo[kMaxExperts], e_hi[kMaxExperts], wsum[kGvWarps];
  __shared__ float red[kGvWarps][8 * RT][kGvRows + 1];
  pdl_trigger();
  pdl_wait();
  const int n_act = active_experts(a, act, e_lo, e_hi, wsum);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gr = lane >> 2, t = lane & 3;
  const int ntile = (a.N + kGvRows - 1) / kGvRows;
  const int steps = (a.K + kGvStep - 1) / kGvStep;
  const size_t row_bytes = (size_t)a.K / 2;
  const long long items = (long long)n_act * ntile;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int ai = (int)(it / ntile), n0 = (int)(it % ntile) * kGvRows;
    const int e = act[ai], hi = e_hi[ai];
    // the lane's two weight rows (those past the end read the last one; not stored)
    const size_t r0 = (size_t)e * a.N + min(n0 + gr, a.N - 1);
    const size_t r1 = (size_t)e * a.N + min(n0 + gr + 8, a.N - 1);
    const uint8_t* w0 = a.w + r0 * row_bytes;
    const uint8_t* w1 = a.w + r1 * row_bytes;
    const uint16_t *s0 = a.s + r0 * a.ng, *s1 = a.s + r1 * a.ng;
    const uint8_t *z0 = ZERO ? a.z + r0 * a.ng : nullptr, *z1 = ZERO ? a.z + r1 * a.ng : nullptr;
    for (int rb = e_lo[ai]; rb < hi; rb += 8 * RT) {
      float acc[RT][4];
#pragma unroll
      for (int i = 0; i < RT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
      for (int st = warp; st < steps; st += kGvWarps) {
        const int k0 = st * kGvStep;
        uint32_t q0[4], q1[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q0[i] = q1[i] = 0u;
#pragma unroll
        for (int j = 0; j < NG; ++j) {
          const int k = k0 + j * G + t * 8 * WPL;
          if (k < a.K) {
            const uint8_t *p0 = w0 + k / 2, *p1 = w1 + k / 2;
            if (WPL == 4) {
              const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p0));
              const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p1));
              q0[0] = u.x; q0[1] = u.y; q0[2] = u.z; q0[3] = u.w;
              q1[0] = v.x; q1[1] = v.y; q1[2] = v.z; q1[3] = v.w;
            } else if (WPL == 2) {
              const uint2 u = __ldg(reinterpret_cast<const uint2*>(p0));
              const uint2 v = __ldg(reinterpret_cast<const uint2*>(p1));
              q0[2 * j] = u.x; q0[2 * j + 1] = u.y;
              q1[2 * j] = v.x; q1[2 * j + 1] = v.y;
            } else {
              q0[j] = __ldg(reinterpret_cast<const uint32_t*>(p0));
              q1[j] = __ldg(reinterpret_cast<const uint32_t*>(p1));
            }
          }
        }
        // lane t of a row reads the scale of the step's group t (mod NG)
        const int gi = st * NG + (t & (NG - 1));
        float f0 = 0.f, f1 = 0.f;
        uint32_t y0 = 8, y1 = 8;
        if (gi < a.ng) {
          f0 = bf16_bits_to_float(__ldg(s0 + gi));
          f1 = bf16_bits_to_float(__ldg(s1 + gi));
          if (ZERO) {
            y0 = __ldg(z0 + gi);
            y1 = __ldg(z1 + gi);
          }
        }
#pragma unroll
        for (int j = 0; j < NG; ++j) {
          const int from = (lane & 28) | j;
          const float sc0 = NG == 1 ? f0 : __shfl_sync(0xffffffffu, f0, from);
          const float sc1 = NG == 1 ? f1 : __shfl_sync(0xffffffffu, f1, from);
          uint32_t zp0 = 0x43084308u, zp1 = 0x43084308u;
          if (ZERO) {
            zp0 = 0x43004300u | (NG == 1 ? y0 : __shfl_sync(0xffffffffu, y0, from)) * 0x10001u;
            zp1 = 0x43004300u | (NG == 1 ? y1 : __shfl_sync(0xffffffffu, y1, from)) * 0x10001u;
          }
          float d[RT][4];
#pragma unroll
          for (int i = 0; i < RT; ++i) d[i][0] = d[i][1] = d[i][2] = d[i][3] = 0.f;
#pragma unroll
          for (int wd = 0; wd < WPL; ++wd) {
            const uint32_t u = q0[j * WPL + wd], v = q1[j * WPL + wd];
            const int k = k0 + j * G + t * 8 * WPL + 8 * wd;
            const uint32_t a00 = code_pair<0>(u, zp0), a01 = code_pair<0>(v, zp1);
            const uint32_t a10 = code_pair<1>(u, zp0), a11 = code_pair<1>(v, zp1);
            const uint32_t a20 = code_pair<2>(u, zp0), a21 = code_pair<2>(v, zp1);
            const uint32_t a30 = code_pair<3>(u, zp0), a31 = code_pair<3>(v, zp1);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
              const int r = rb + 8 * i + gr;
              uint4 xv = make_uint4(0u, 0u, 0u, 0u);
              if (r < hi && k < a.K)
                xv = __ldg(reinterpret_cast<const uint4*>(a.x + (size_t)r * a.K + k));
              mma_bf16(d[i], a00, a01, a10, a11, __byte_perm(xv.x, xv.z, 0x5410),
                       __byte_perm(xv.x, xv.z, 0x7632));
              mma_bf16(d[i], a20, a21, a30, a31, __byte_perm(xv.y, xv.w, 0x5410),
                       __byte_perm(xv.y, xv.w, 0x7632));
            }
          }
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            acc[i][0] = fmaf(sc0, d[i][0], acc[i][0]);
            acc[i][1] = fmaf(sc0, d[i][1], acc[i][1]);
            acc[i][2] = fmaf(sc1, d[i][2], acc[i][2]);
            acc[i][3] = fmaf(sc1, d[i][3], acc[i][3]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        red[warp][8 * i + 2 * t][gr] = acc[i][0];
        red[warp][8 * i + 2 * t + 1][gr] = acc[i][1];
        red[warp][8 * i + 2 * t][gr + 8] = acc[i][2];
        red[warp][8 * i + 2 * t + 1][gr + 8] = acc[i][3];
      }
      __syncthreads();
      for (int i = threadIdx.x; i < 8 * RT * kGvRows; i += kGvThreads) {
        const int n = i % kGvRows, r = i / kGvRows;
        float v = red[0][r][n];
#pragma unroll
        for (int q = 1; q < kGvWarps; ++q) v += red[q][r][n];
        if (n0 + n < a.N && rb + r < hi) {
          const size_t o = (size_t)(rb + r) * a.N + n0 + n;
          if (F32) static_cast<float*>(a.y)[o] = v;
          else static_cast<uint16_t*>(a.y)[o] = float_to_bf16_bits(v);
        }
      }
      __syncthreads();
    }
  }
}

bool valid_gemv_shape(int E, int N, int K, int max_rows) {
  return E > 0 && E <= kMaxExperts && N > 0 && K > 0 && K % 32 == 0 && max_rows >= 0 &&
         N <= (1 << 24) && K <= (1 << 24) && (long long)E * N < (1LL << 31);
}

template <int G, bool ZERO, bool F32, int RT>
int launch_gemv(const GemvArgs& a, cudaStream_t st) {
  const long long most = (long long)std::min(a.E, a.max_rows) * ceil_div(a.N, kGvRows);
  const int grid = (int)std::min<long long>(most, 4LL * sm_count());
  MOE_LAUNCH_PDL((gemv_int4_kernel<G, ZERO, F32, RT>), dim3(grid), dim3(kGvThreads), 0, st, a);
  MOE_COUNT_LAUNCH();
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

template <int G, bool ZERO, bool F32>
int launch_gemv_rows(const GemvArgs& a, cudaStream_t st) {
  const int rows = ceil_div(a.max_rows, a.E);
  if (rows <= 8) return launch_gemv<G, ZERO, F32, 1>(a, st);
  if (rows <= 16) return launch_gemv<G, ZERO, F32, 2>(a, st);
  return launch_gemv<G, ZERO, F32, 4>(a, st);
}

template <int G>
int launch_gemv_types(const GemvArgs& a, bool f32, cudaStream_t st) {
  if (a.z) return f32 ? launch_gemv_rows<G, true, true>(a, st)
                      : launch_gemv_rows<G, true, false>(a, st);
  return f32 ? launch_gemv_rows<G, false, true>(a, st) : launch_gemv_rows<G, false, false>(a, st);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_grouped_gemv_int4_workspace_size(int max_rows, int E, int N, int K) {
  return valid_gemv_shape(E, N, K, max_rows) ? 256 : 0;
}

int moe_grouped_gemv_int4(const uint16_t* x, const uint8_t* w, const uint16_t* w_scale,
                          const uint8_t* w_zero, const int32_t* offsets, int E, int N, int K,
                          int group, int max_rows, int out_f32, void* y, void* ws,
                          size_t ws_bytes, void* stream) {
  MOE_REQUIRE(valid_gemv_shape(E, N, K, max_rows) && (offsets || E == 1) &&
              (out_f32 == 0 || out_f32 == 1));
  MOE_REQUIRE(group == 32 || group == 64 || group == 128);
  if (max_rows == 0) return MOE_OK;
  MOE_REQUIRE(x && w && w_scale && y && ws);
  MOE_REQUIRE(aligned16(x) && aligned16(w) && aligned4(w_scale) && aligned16(y) &&
              aligned4(offsets) && aligned256(ws));
  MOE_REQUIRE(ws_bytes >= moe_grouped_gemv_int4_workspace_size(max_rows, E, N, K));
  GemvArgs a{x, w, w_scale, w_zero, offsets, E, N, K, ceil_div(K, group), max_rows, y,
             static_cast<int32_t*>(ws)};
  cudaStream_t st = (cudaStream_t)stream;
  if (group == 32) return launch_gemv_types<32>(a, out_f32 != 0, st);
  if (group == 64) return launch_gemv_types<64>(a, out_f32 != 0, st);
  return launch_gemv_types<128>(a, out_f32 != 0, st);
}

}  // extern "C"
