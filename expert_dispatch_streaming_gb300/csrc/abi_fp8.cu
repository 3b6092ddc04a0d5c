// C-ABI entry points of the FP8 expert path: the grouped FP8 product and the SwiGLU expert FFN
// on FP8 bundles (the quantiser and the packers are in quant_fp8.cu and bundle.cpp).
//
// Only the experts a batch selected are touched ("NovaLLM: Running Massive MoE Models Fully
// In-Memory", "3. Optimization #1 -- Expert-Level Streaming"); the FP8 codes travel with their
// scales in one bundle ("Running 35B MoE Models on 8GB GPUs ...", "Technical Insight", which
// names FP8 among the checkpoint formats without defining one).
#include <cstring>

#include "fp8.cuh"

using namespace moe;

namespace {

bool fp8_shape(int E, int N, int K, int max_rows) {
  return E > 0 && E <= kMaxExperts && N > 0 && K > 0 && K % 16 == 0 && max_rows >= 0 &&
         N <= (1 << 24) && K <= (1 << 24) && (long long)E * N < (1LL << 31);
}

Fp8Args gemm_args_fp8(int E, int N, int K, int max_rows) {
  Fp8Args a{};
  a.E = E; a.N = N; a.K = K; a.max_rows = max_rows; a.host_n = -1;
  return a;
}

}  // namespace

extern "C" {

size_t moe_grouped_gemm_fp8_workspace_size(int max_rows, int E, int N, int K) {
  if (!fp8_shape(E, N, K, max_rows)) return 0;
  const Fp8Plan pl = plan_fp8(gemm_args_fp8(E, N, K, max_rows));
  WsCursor c(nullptr, 0);
  c.take<int32_t>(64);
  c.take<int32_t>(pl.counter_elems);
  c.take<float>(pl.part_elems);
  return c.used;
}

int moe_grouped_gemm_fp8(const uint8_t* xq, const float* x_scale, const uint8_t* w,
                         const float* w_scale, const int32_t* offsets, int E, int N, int K,
                         int max_rows, int out_f32, void* y, void* ws, size_t ws_bytes,
                         void* stream) {
  MOE_REQUIRE(fp8_shape(E, N, K, max_rows) && (offsets || E == 1) &&
              (out_f32 == 0 || out_f32 == 1));
  if (max_rows == 0) return MOE_OK;
  MOE_REQUIRE(xq && x_scale && w && w_scale && y && ws);
  MOE_REQUIRE(aligned16(xq) && aligned16(w) && aligned16(y) && aligned4(x_scale) &&
              aligned4(w_scale) && aligned4(offsets) && aligned256(ws));
  cudaStream_t st = (cudaStream_t)stream;
  Fp8Args a = gemm_args_fp8(E, N, K, max_rows);
  a.xq = xq; a.xs = x_scale; a.w = w; a.ws = w_scale; a.offsets = offsets; a.y = y;
  a.y_f32 = out_f32 != 0;
  const Fp8Plan pl = plan_fp8(a);
  WsCursor c(ws, ws_bytes);
  int32_t* err = c.take<int32_t>(64);
  int32_t* ctr = c.take<int32_t>(pl.counter_elems);
  const size_t ctl = c.used;
  float* part = c.take<float>(pl.part_elems);
  MOE_REQUIRE(c.ok());
  const int r = launch_clear(err, ctl, st);
  if (r != MOE_OK) return r;
  a.after = kAfterClear;
  return launch_fp8(a, part, ctr, err, st);
}

size_t moe_grouped_swiglu_fp8_workspace_size(int max_rows, int E, int H, int I) {
  moe_bundle_layout lay;
  if (max_rows < 0 || E <= 0 || E > kMaxExperts ||
      moe_bundle_layout_of(H, I, MOE_W_FP8_B128, &lay) != MOE_OK)
    return 0;
  Fp8Args gu = gemm_args_fp8(E, I, H, max_rows), dn = gemm_args_fp8(E, H, I, max_rows);
  gu.fused = true;
  const Fp8Plan a = plan_fp8(gu), b = plan_fp8(dn);
  WsCursor c(nullptr, 0);
  c.take<int32_t>(64);
  c.take<int32_t>(std::max(a.counter_elems, b.counter_elems));
  c.take<uint8_t>((size_t)max_rows * I);
  c.take<float>((size_t)max_rows * (I / 128));
  c.take<float>(std::max(a.part_elems, b.part_elems));
  return c.used;
}

int moe_grouped_swiglu_fp8(const uint8_t* xq, const float* x_scale, const int32_t* offsets,
                           const void* const* bundles, int E, int H, int I, int max_rows,
                           uint16_t* y_perm, void* ws, size_t ws_bytes, void* stream) {
  moe_bundle_layout lay;
  MOE_REQUIRE(E > 0 && E <= kMaxExperts && max_rows >= 0);
  MOE_REQUIRE(moe_bundle_layout_of(H, I, MOE_W_FP8_B128, &lay) == MOE_OK);
  if (max_rows == 0) return MOE_OK;
  MOE_REQUIRE(xq && x_scale && offsets && bundles && y_perm && ws);
  MOE_REQUIRE(aligned16(xq) && aligned16(y_perm) && aligned4(x_scale) && aligned4(offsets) &&
              aligned256(ws));
  cudaStream_t st = (cudaStream_t)stream;
  BundleTable tab{};
  for (int e = 0; e < E; ++e) {
    MOE_REQUIRE(aligned16(bundles[e]));
    tab.p[e] = bundles[e];
  }
  Fp8Args gu = gemm_args_fp8(E, I, H, max_rows), dn = gemm_args_fp8(E, H, I, max_rows);
  gu.fused = true;
  const Fp8Plan pg = plan_fp8(gu), pd = plan_fp8(dn);
  WsCursor c(ws, ws_bytes);
  int32_t* err = c.take<int32_t>(64);
  int32_t* ctr = c.take<int32_t>(std::max(pg.counter_elems, pd.counter_elems));
  const size_t ctl = c.used;
  uint8_t* hq = c.take<uint8_t>((size_t)max_rows * I);
  float* hs = c.take<float>((size_t)max_rows * (I / 128));
  float* part = c.take<float>(std::max(pg.part_elems, pd.part_elems));
  MOE_REQUIRE(c.ok());
  int r = launch_clear(err, ctl, st);
  if (r != MOE_OK) return r;
  gu.after = kAfterClear;
  gu.xq = xq; gu.xs = x_scale; gu.offsets = offsets; gu.tab = &tab;
  gu.w_off = lay.gate_up_offset; gu.s_off = lay.gate_up_scale_offset; gu.hq = hq; gu.hs = hs;
  r = launch_fp8(gu, part, ctr, err, st);
  if (r != MOE_OK) return r;
  dn.after = kAfterRows;
  dn.xq = hq; dn.xs = hs; dn.offsets = offsets; dn.tab = &tab;
  dn.w_off = lay.down_offset; dn.s_off = lay.down_scale_offset; dn.y = y_perm;
  return launch_fp8(dn, part, ctr, err, st);
}

}  // extern "C"
