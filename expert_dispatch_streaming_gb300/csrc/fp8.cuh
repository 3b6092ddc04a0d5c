// FP8 (E4M3) expert path: host interface and shared device helpers (internal to libmoe).
//
// A quantised block of up to 128 values x holds codes q = e4m3(x * (448 / amax)) and the fp32
// scale s = amax / 448, amax = max(largest |x| of the block, 2^-96): E4M3's largest value is 448,
// so the block's largest element lands on it, and the floor keeps s a normal number (a block of
// zeros has zero codes).  A NaN stays a NaN code and does not move its block's scale; an
// infinity makes s infinite, so its block reads NaN.
#pragma once
#include "expert_ffn.cuh"

namespace moe {

constexpr int kFp8Block = 128;          // elements per scale
constexpr float kFp8Max = 448.f;
constexpr float kFp8MinAmax = 0x1p-96f;
constexpr int kFp8TileBytes = 16384;    // 128 rows x 128 k

// Four floats times inv -> four E4M3 codes (round to nearest even, saturating), the first in the
// low byte.  (The instruction takes its second operand as the low half; written out, the two
// conversions merge into one register without extracting and shifting 16-bit values.)
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d, float inv) {
  uint32_t r;
  asm("{\n.reg .b64 p, q, s;\n.reg .f32 e, f, g, i;\n.reg .b16 l, h;\n"
      "mov.b64 p, {%1, %2};\nmov.b64 q, {%3, %4};\nmov.b64 s, {%5, %5};\n"
      "mul.rn.f32x2 p, p, s;\nmul.rn.f32x2 q, q, s;\n"
      "mov.b64 {e, f}, p;\nmov.b64 {g, i}, q;\n"
      "cvt.rn.satfinite.e4m3x2.f32 l, f, e;\ncvt.rn.satfinite.e4m3x2.f32 h, i, g;\n"
      "mov.b32 %0, {l, h};\n}\n"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d), "f"(inv));
  return r;
}

// One grouped product over FP8 operands:
//   acc[row][n] = sum_b xs[row][b] ws_e[n / 128][b] sum_{k in block b} xq[row][k] w_e[n][k]
// fused: w_e = gate rows 0..N-1 and up rows N..2N-1; h = silu(gate) * up is quantised per row
//        and 128 columns into hq / hs;  else y = acc rounded to bf16, or kept in fp32.
// What the kernel before a product on the stream writes: anything, so that the product starts when
// it has ended; or, so that the product may start earlier and waits where it needs that, only the
// product's token rows and scales (the product before it) or only its counters and error word
// (launch_clear).
enum Fp8After { kAfterAny = 0, kAfterRows = 1, kAfterClear = 2 };
struct Fp8Args {
  const uint8_t* xq;          // [max_rows][K] E4M3
  const float* xs;            // [max_rows][ceil(K / 128)]
  const int32_t* offsets;     // device [E+1], or NULL: one group of max_rows rows
  int E, N, K, max_rows;
  bool fused, y_f32;
  int after;                  // Fp8After: what the kernel before it on the stream does
  // weights: bundles (host table or device table) with the section's codes at w_off and its
  // scales at s_off, or plain row-major w [E][N][K] with ws [E][ceil(N/128)][ceil(K/128)]
  const BundleTable* tab;
  const void* const* dev_tab;
  size_t w_off, s_off;
  const uint8_t* w;
  const float* ws;
  // the experts to run: a device list, a host list (host_n >= 0), or all of them
  const int32_t* active;
  const int32_t* n_active;
  int host_n;
  const int32_t* host_ids;
  uint8_t* hq;                // [max_rows][N]
  float* hs;                  // [max_rows][N / 128]
  void* y;                    // [max_rows][N] bf16 or fp32
};

struct Fp8Plan {
  size_t part_elems, counter_elems;
};

// counters must be zero on entry and are zero again when the launch has finished
Fp8Plan plan_fp8(const Fp8Args& a);
int launch_fp8(const Fp8Args& a, float* part, int32_t* counters, int32_t* err, cudaStream_t st);

// zeroes the control words of a workspace (bytes: a multiple of 16)
int launch_clear(void* words, size_t bytes, cudaStream_t st);

int launch_quantize_fp8(const uint16_t* x, const int32_t* src, int rows, int k, int T, int H,
                        uint8_t* q, float* scale, cudaStream_t st);

}  // namespace moe
