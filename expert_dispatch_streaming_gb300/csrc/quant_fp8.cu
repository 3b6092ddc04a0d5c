// Quantisation of bf16 rows to E4M3 with one fp32 scale per row and 128 columns, optionally
// gathered into expert order on the way, and the device-side packer of FP8 bundles.
#include "fp8.cuh"

namespace moe {
namespace {

// A lane holds 16 consecutive columns (two 16-byte loads, one 16-byte store), eight lanes a block,
// a warp 512 columns at a time; a warp takes one row's kCols columns, both halves' loads in
// flight together.  It needs 2 bytes in (gathered rows mostly from L2: the codes are stored with a
// streaming hint so that they do not push x out of it) and 1 byte out per value; 8192 x 7168 rows
// gathered eightfold take 136 us, 66% of the copy bandwidth, with the issue slots 75% busy:
// converting each value (unpack, multiply, convert, pack, its part of the maximum) bounds it.
// The largest magnitude of bf16 values is taken in bf16, which is exact and skips NaNs.
constexpr int kCols = 1024;

// The larger magnitudes of two pairs, in one instruction; the signs are of no meaning.
__device__ __forceinline__ uint32_t abs_max2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__global__ void __launch_bounds__(256)
quantize_fp8_kernel(const uint16_t* __restrict__ x, const int32_t* __restrict__ src, int rows,
                    int k, int T, int H, int nb, uint8_t* __restrict__ q,
                    float* __restrict__ scale) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, row = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;
  // (grid x first: all rows' first columns, then the next.  A gathered x row is read k times, and
  // 2 KB of every row at a time stay in L2 where whole rows, 117 MB at 8192 x 7168, would not)
  const int c0 = blockIdx.y * kCols + 16 * lane;
  int from = row;
  if (src) {
    const int s = __ldg(src + row);
    from = s >= 0 && s < T * k ? s / k : -1;   // outside [0, T k): a row of zeros
  }
  uint4 v[2][2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int col = c0 + 512 * h;
    v[h][0] = v[h][1] = make_uint4(0u, 0u, 0u, 0u);
    if (from >= 0 && col < H) {
      const uint4* p = reinterpret_cast<const uint4*>(x + (size_t)from * H + col);
      v[h][0] = __ldg(p);
      v[h][1] = __ldg(p + 1);
    }
  }
  // the blocks' largest magnitudes, both halves' pairs reduced side by side
  uint32_t m2[2] = {0u, 0u};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t w[8] = {v[h][0].x, v[h][0].y, v[h][0].z, v[h][0].w,
                           v[h][1].x, v[h][1].y, v[h][1].z, v[h][1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) m2[h] = abs_max2(m2[h], w[i]);
  }
  // each as one bf16: this half's in the low half-word, the other's in the high one
  uint32_t mm = abs_max2(__byte_perm(m2[0], m2[1], 0x5410), __byte_perm(m2[0], m2[1], 0x7632));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) mm = abs_max2(mm, __shfl_xor_sync(0xffffffffu, mm, o));
  const float2 mf = bf16x2_to_float2(mm);
  // one division a lane: of a block's eight lanes, the first four take 448 / amax and amax / 448
  // of the two halves
  const int kind = lane & 3;
  const float m = fmaxf(fabsf(kind < 2 ? mf.x : mf.y), kFp8MinAmax);
  const float d = __fdiv_rn(kind & 1 ? m : kFp8Max, kind & 1 ? kFp8Max : m);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int col = c0 + 512 * h;
    const float inv = __shfl_sync(0xffffffffu, d, (lane & 24) + 2 * h);
    const uint32_t w[8] = {v[h][0].x, v[h][0].y, v[h][0].z, v[h][0].w,
                           v[h][1].x, v[h][1].y, v[h][1].z, v[h][1].w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = bf16x2_to_float2(w[2 * i]), b = bf16x2_to_float2(w[2 * i + 1]);
      o[i] = fp8_pack4(a.x, a.y, b.x, b.y, inv);
    }
    if (col < H)
      __stcs(reinterpret_cast<uint4*>(q + (size_t)row * H + col),
             make_uint4(o[0], o[1], o[2], o[3]));
    if ((lane & 7) == 2 * h + 1 && col - 16 * (lane & 7) < H)
      scale[(size_t)row * nb + (col >> 7)] = d;
  }
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
  MOE_LAUNCH_PDL(quantize_fp8_kernel, dim3(ceil_div(rows, 8), ceil_div(H, kCols)), dim3(256), 0,
                 st, x, src, rows, k, T, H, ceil_div(H, kFp8Block), q, scale);
  MOE_COUNT_LAUNCH();
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" {

int moe_quantize_fp8(const uint16_t* x, const int32_t* src, int T, int k, int H, uint8_t* q,
                     float* scale, void* stream) {
  MOE_REQUIRE(T >= 0 && H > 0 && H % 16 == 0 && H <= (1 << 24));
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
  // the scales, and zeros in what rounding their sections up to 256 bytes leaves (as on the host: a
  // bundle's checksum covers it)
  const size_t sg = gu / 16384 * sizeof(float), sd = dn / 16384 * sizeof(float);
  const size_t end_g = lay.gate_up_scale_offset + sg, end_d = lay.down_scale_offset + sd;
  MOE_CUDA_TRY(cudaMemcpyAsync(b + lay.gate_up_scale_offset, s_gate_up, sg,
                               cudaMemcpyDeviceToDevice, st));
  MOE_CUDA_TRY(cudaMemcpyAsync(b + lay.down_scale_offset, s_down, sd, cudaMemcpyDeviceToDevice,
                               st));
  if (end_g < lay.down_scale_offset)
    MOE_CUDA_TRY(cudaMemsetAsync(b + end_g, 0, lay.down_scale_offset - end_g, st));
  if (end_d < lay.total_bytes)
    MOE_CUDA_TRY(cudaMemsetAsync(b + end_d, 0, lay.total_bytes - end_d, st));
  return MOE_OK;
}

}  // extern "C"
