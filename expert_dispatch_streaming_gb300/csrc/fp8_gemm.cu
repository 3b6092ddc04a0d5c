// Grouped matrix product of E4M3 token rows with E4M3 expert weights, one fp32 scale per row
// and 128 columns of the activations and per 128 x 128 block of the weights.
//
//   acc[row][n] = sum_b xs[row][b] ws[n / 128][b] sum_{k in block b} xq[row][k] w[n][k]
//
// Each block's inner sum is formed first and then scaled into an fp32 accumulator, so a block's
// scales never mix with another's.
//
// CUDA-core form: a CTA takes 128 output columns (fused: of the gate and of the up rows) of 16
// token rows; per block of 128 k the weights' bytes and the rows' values sit in shared memory,
// a thread holds one column of eight rows.
#include "fp8.cuh"

namespace moe {
namespace {

struct Fp8Params {
  const uint8_t* xq;
  const float* xs;
  const int32_t* offsets;
  int E, N, K, KB, max_rows;
  BundleTable tab;
  const void* const* dev_tab;
  size_t w_off, s_off;
  const uint8_t* w;
  const float* ws;
  const int32_t* active;
  const int32_t* n_active;
  int host_n;
  int16_t host_ids[kMaxExperts];
  uint8_t* hq;
  float* hs;
  void* y;
  int y_f32;
  int32_t* err;
};

__device__ __forceinline__ float silu_mul(float g, float u) {
  return __fdividef(g, 1.f + __expf(-g)) * u;
}
__device__ __forceinline__ float e4m3_value(uint8_t b) {
  __nv_fp8_e4m3 v;
  v.__x = b;
  return static_cast<float>(v);
}

constexpr int kRows = 16;

template <bool FUSED>
__global__ void __launch_bounds__(256) fp8_simple_kernel(const __grid_constant__ Fp8Params p) {
  pdl_trigger();
  pdl_wait();
  constexpr int NA = FUSED ? 2 : 1;
  __shared__ uint8_t ws[NA][128][132];
  __shared__ float xv[kRows][128];
  __shared__ float red[2][8][4];
  const int tid = threadIdx.x, col = tid & 127, grp = tid >> 7, n0 = blockIdx.x * 128;
  int a = blockIdx.y;
  const int n_act = p.host_n >= 0 ? p.host_n : p.active ? *p.n_active : p.E;
  if (a >= n_act) return;
  const int e = p.host_n >= 0 ? p.host_ids[a] : p.active ? p.active[a] : a;
  int r0 = p.offsets ? p.offsets[e] : 0, r1 = p.offsets ? p.offsets[e + 1] : p.max_rows;
  const int c0 = min(max(r0, 0), p.max_rows), c1 = min(max(r1, c0), p.max_rows);
  if ((c0 != r0 || c1 != r1) && tid == 0) atomicExch(p.err, 8);
  r0 = c0;
  r1 = c1;
  if (r0 >= r1) return;
  const uint8_t* wb;
  const float* sb;
  const int NB = (p.N + 127) / 128;
  if (p.w) {
    wb = p.w + (size_t)e * p.N * p.K;
    sb = p.ws + (size_t)e * NB * p.KB;
  } else {
    const uint8_t* b = static_cast<const uint8_t*>(p.dev_tab ? p.dev_tab[e] : p.tab.p[e]);
    wb = b + p.w_off;
    sb = reinterpret_cast<const float*>(b + p.s_off);
  }
  for (int rb = r0 + blockIdx.z * kRows; rb < r1; rb += gridDim.z * kRows) {
    float acc[NA][8] = {};
    for (int kb = 0; kb < p.KB; ++kb) {
      __syncthreads();
      for (int i = tid; i < NA * 128 * 128; i += 256) {
        const int w = i >> 14, r = (i >> 7) & 127, kk = i & 127, k = kb * 128 + kk, n = n0 + r;
        uint8_t v = 0;
        if (k < p.K && n < p.N) {
          if (p.w) {
            v = wb[(size_t)n * p.K + k];
          } else {
            const int mt = (n0 >> 7) + w * NB;
            v = wb[((size_t)mt * p.KB + kb) * kFp8TileBytes + r * 128 +
                   (((kk >> 4) ^ (r & 7)) << 4) + (kk & 15)];
          }
        }
        ws[w][r][kk] = v;
      }
      for (int i = tid; i < kRows * 128; i += 256) {
        const int r = i >> 7, kk = i & 127, k = kb * 128 + kk;
        xv[r][kk] = (rb + r < r1 && k < p.K) ? e4m3_value(p.xq[(size_t)(rb + r) * p.K + k]) : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int w = 0; w < NA; ++w) {
        float s[8] = {};
        for (int kk = 0; kk < 128; ++kk) {
          const float wv = e4m3_value(ws[w][col][kk]);
#pragma unroll
          for (int j = 0; j < 8; ++j) s[j] = fmaf(wv, xv[grp * 8 + j][kk], s[j]);
        }
        const float sw = sb[(size_t)((n0 >> 7) + w * NB) * p.KB + kb];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int row = rb + grp * 8 + j;
          const float f = row < r1 ? p.xs[(size_t)row * p.KB + kb] * sw : 0.f;
          acc[w][j] = fmaf(s[j], f, acc[w][j]);
        }
      }
    }
    if (FUSED) {
      float h[8];
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[j] = silu_mul(acc[0][j], acc[NA - 1][j]);
        float m = fabsf(h[j]);
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if ((tid & 31) == 0) red[grp][j][(tid >> 5) & 3] = m;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float* m4 = red[grp][j];
        const float m = fmaxf(fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])), kFp8MinAmax);
        const int row = rb + grp * 8 + j;
        if (row < r1) {
          p.hq[(size_t)row * p.N + n0 + col] =
              (uint8_t)fp8_pack4(h[j], 0.f, 0.f, 0.f, __fdiv_rn(kFp8Max, m));
          if (col == 0) p.hs[(size_t)row * NB + (n0 >> 7)] = __fdiv_rn(m, kFp8Max);
        }
      }
    } else if (n0 + col < p.N) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int row = rb + grp * 8 + j;
        if (row >= r1) continue;
        const size_t at = (size_t)row * p.N + n0 + col;
        if (p.y_f32) static_cast<float*>(p.y)[at] = acc[0][j];
        else static_cast<uint16_t*>(p.y)[at] = float_to_bf16_bits(acc[0][j]);
      }
    }
  }
}

}  // namespace

Fp8Plan plan_fp8(const Fp8Args&) { return Fp8Plan{1, 1}; }

int launch_fp8(const Fp8Args& a, const Fp8Plan&, float*, int32_t*, int32_t* err,
               cudaStream_t st) {
  if (a.max_rows <= 0 || a.host_n == 0) return MOE_OK;
  Fp8Params p{};
  p.xq = a.xq; p.xs = a.xs; p.offsets = a.offsets; p.E = a.E; p.N = a.N; p.K = a.K;
  p.KB = ceil_div(a.K, 128); p.max_rows = a.max_rows;
  if (a.tab) p.tab = *a.tab;
  p.dev_tab = a.dev_tab; p.w_off = a.w_off; p.s_off = a.s_off; p.w = a.w; p.ws = a.ws;
  p.active = a.active; p.n_active = a.n_active; p.host_n = a.host_n;
  for (int i = 0; i < (a.host_n > 0 ? a.host_n : 0); ++i) p.host_ids[i] = (int16_t)a.host_ids[i];
  p.hq = a.hq; p.hs = a.hs; p.y = a.y; p.y_f32 = a.y_f32; p.err = err;
  const dim3 grid(ceil_div(a.N, 128), a.host_n > 0 ? a.host_n : a.E,
                  std::min(ceil_div(a.max_rows, kRows), 16));
  if (a.fused) MOE_LAUNCH_PDL(fp8_simple_kernel<true>, grid, dim3(256), 0, st, p);
  else MOE_LAUNCH_PDL(fp8_simple_kernel<false>, grid, dim3(256), 0, st, p);
  MOE_COUNT_LAUNCH();
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace moe
