// Quantisation of bf16 rows to E4M3 with one fp32 scale per row and 128 columns, optionally
// gathered into expert order on the way, and the device-side packer of FP8 bundles.
#include "fp8.cuh"

namespace moe {
namespace {

// One warp per row and 128-column block: a lane holds four columns.
__global__ void __launch_bounds__(256)
quantize_fp8_kernel(const uint16_t* __restrict__ x, const int32_t* __restrict__ src, int rows,
                    int k, int T, int H, int nb, uint8_t* __restrict__ q,
                    float* __restrict__ scale) {
  pdl_trigger();
  pdl_wait();
  const long long item = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (item >= (long long)rows * nb) return;
  const int row = (int)(item / nb), b = (int)(item % nb), col = b * kFp8Block + 4 * lane;
  int from = row;
  if (src) {
    const int s = src[row];
    from = s >= 0 && s < T * k ? s / k : -1;   // outside [0, T k): a row of zeros
  }
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  if (from >= 0 && col < H) {
    const uint2 w = *reinterpret_cast<const uint2*>(x + (size_t)from * H + col);
    const float2 a = bf16x2_to_float2(w.x), c = bf16x2_to_float2(w.y);
    v[0] = a.x; v[1] = a.y; v[2] = c.x; v[3] = c.y;
  }
  float m = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  m = fmaxf(m, kFp8MinAmax);
  const float inv = __fdiv_rn(kFp8Max, m);
  if (col < H)
    *reinterpret_cast<uint32_t*>(q + (size_t)row * H + col) =
        fp8_pack4(v[0], v[1], v[2], v[3], inv);
  if (lane == 0) scale[(size_t)row * nb + b] = __fdiv_rn(m, kFp8Max);
}

// Row-major codes [rows][K] -> the section's 128 x 128 tiles: row r's 16-byte chunk c of tile
// (mt, kt) at r * 128 + ((c ^ (r % 8)) * 16).  One thread per 16-byte chunk, writes in order.
__global__ void __launch_bounds__(256)
pack_fp8_kernel(const uint8_t* __restrict__ w, int rows, int K, uint8_t* __restrict__ dst) {
  const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (size_t)rows * K / 16) return;
  const int c = (int)(i & 7), r = (int)((i >> 3) & 127);
  const size_t tile = i >> 10, kt = tile % (K / 128), mt = tile / (K / 128);
  const uint4 v = *reinterpret_cast<const uint4*>(w + (mt * 128 + r) * (size_t)K + kt * 128 +
                                                  ((c ^ (r & 7)) << 4));
  *reinterpret_cast<uint4*>(dst + 16 * i) = v;
}

}  // namespace

int launch_quantize_fp8(const uint16_t* x, const int32_t* src, int rows, int k, int T, int H,
                        uint8_t* q, float* scale, cudaStream_t st) {
  if (rows <= 0) return MOE_OK;
  const int nb = ceil_div(H, kFp8Block);
  const long long items = (long long)rows * nb;
  MOE_LAUNCH_PDL(quantize_fp8_kernel, dim3((unsigned)((items + 7) / 8)), dim3(256), 0, st, x, src,
                 rows, k, T, H, nb, q, scale);
  MOE_COUNT_LAUNCH();
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" {

int moe_quantize_fp8(const uint16_t* x, const int32_t* src, int T, int k, int H, uint8_t* q,
                     float* scale, void* stream) {
  MOE_REQUIRE(T >= 0 && H > 0 && H % 16 == 0);
  MOE_REQUIRE(!src || (k >= 1 && (long long)T * k <= 0x7fffffffLL));
  if (T == 0) return MOE_OK;
  MOE_REQUIRE(x && q && scale && aligned16(x) && aligned16(q) && aligned4(scale) &&
              aligned4(src));
  return launch_quantize_fp8(x, src, src ? T * k : T, k, T, H, q, scale, (cudaStream_t)stream);
}

int moe_pack_bundle_fp8_device(int H, int I, const uint8_t* w_gate_up, const float* s_gate_up,
                               const uint8_t* w_down, const float* s_down, void* dst,
                               void* stream) {
  moe_bundle_layout lay;
  MOE_REQUIRE(moe_bundle_layout_of(H, I, MOE_W_FP8_B128, &lay) == MOE_OK);
  MOE_REQUIRE(w_gate_up && s_gate_up && w_down && s_down && dst && aligned16(w_gate_up) &&
              aligned16(w_down) && aligned16(dst));
  cudaStream_t st = (cudaStream_t)stream;
  uint8_t* b = static_cast<uint8_t*>(dst);
  const size_t gu = (size_t)2 * I * H, dn = (size_t)I * H;
  pack_fp8_kernel<<<(unsigned)((gu / 16 + 255) / 256), 256, 0, st>>>(w_gate_up, 2 * I, H,
                                                                     b + lay.gate_up_offset);
  MOE_COUNT_LAUNCH();
  MOE_LAUNCH_CHECK();
  pack_fp8_kernel<<<(unsigned)((dn / 16 + 255) / 256), 256, 0, st>>>(w_down, H, I,
                                                                     b + lay.down_offset);
  MOE_COUNT_LAUNCH();
  MOE_LAUNCH_CHECK();
  MOE_CUDA_TRY(cudaMemcpyAsync(b + lay.gate_up_scale_offset, s_gate_up, gu / 16384 * sizeof(float),
                               cudaMemcpyDeviceToDevice, st));
  MOE_CUDA_TRY(cudaMemcpyAsync(b + lay.down_scale_offset, s_down, dn / 16384 * sizeof(float),
                               cudaMemcpyDeviceToDevice, st));
  return MOE_OK;
}

}  // extern "C"
