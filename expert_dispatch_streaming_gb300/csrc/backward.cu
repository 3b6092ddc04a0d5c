// Gradients of the way into expert order, of the gate-weighted way back, and of the gating.
#include "common.cuh"
#include "route.cuh"

#include <math_constants.h>
#include <type_traits>

namespace moe {
namespace {

constexpr int kBackThreads = 128;   // one 16-byte vector (8 bf16) a thread

__device__ __forceinline__ void unpack8(const uint4& q, float* f) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = bf16x2_to_float2(w[i]);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(float2_to_bf16x2(f[0], f[1]), float2_to_bf16x2(f[2], f[3]),
                    float2_to_bf16x2(f[4], f[5]), float2_to_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ float reduce_warp(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ------------------------------------------------------------------------------ permute
// The rows x_perm[pos[t][j]] are copies of x[t], so
//   dx[t] = sum_{j<k} dx_perm[pos[t][j]]  (+ add[t])
// in fp32, j in order, rounded once.  Block (c, t): elements [1024 c, 1024 c + 1024) of token t, one
// 16-byte piece of each of the k rows a thread.  Reading the rows bounds it: 8192 tokens of eight rows
// of 7168 take 156 us, the 1057 MB it needs at the copy bandwidth.
template <int K, bool F32>
__global__ void __launch_bounds__(kBackThreads)
permute_backward_kernel(const uint16_t* __restrict__ dxp, const int32_t* __restrict__ pos,
                        const uint16_t* add, int T, int H, void* dx) {   // (dx may be add)
  pdl_trigger();
  pdl_wait();
  const int v = blockIdx.x * kBackThreads + threadIdx.x;
  if (v >= H / 8) return;
  const unsigned rows = (unsigned)T * K;
  for (unsigned t = blockIdx.y; t < (unsigned)T; t += gridDim.y) {   // (the last step passes 2^31)
    uint4 q[K], a = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const int p = __ldg(pos + (size_t)t * K + j);
      q[j] = make_uint4(0u, 0u, 0u, 0u);
      if ((unsigned)p < rows) q[j] = __ldg(reinterpret_cast<const uint4*>(dxp + (size_t)p * H) + v);
    }
    if (add) a = reinterpret_cast<const uint4*>(add + (size_t)t * H)[v];
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, f[8];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      unpack8(q[j], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += f[i];
    }
    if (add) {
      unpack8(a, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += f[i];
    }
    if (F32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(dx) + (size_t)t * H) + 2 * v;
      o[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      o[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    } else {
      reinterpret_cast<uint4*>(static_cast<uint16_t*>(dx) + (size_t)t * H)[v] = pack8(acc);
    }
  }
}

// ------------------------------------------------------------------------------ combine
// Of out[t] = sum_j w[t][j] y_perm[pos[t][j]] + g_t shared[t]:
//   dy_perm[pos[t][j]] = w[t][j] dout[t],   dw[t][j] = <dout[t], y_perm[pos[t][j]]>,
//   dshared[t] = g_t dout[t],               dg_t = <dout[t], shared[t]>
// A CTA takes one token: a thread reads a 16-byte vector of dout[t] and of the k rows, writes the
// k scaled vectors and keeps k + 1 partial dot products, which the CTA adds in a fixed order: one
// pass over y_perm and dy_perm, which bound it.  8192 tokens of eight rows of 7168 and a shared expert
// take 311 us, the 2115 MB it needs at the copy bandwidth.
constexpr int kCombineBackThreads = 256;

template <int K>
__global__ void __launch_bounds__(kCombineBackThreads)
combine_backward_kernel(const uint16_t* __restrict__ dout, const uint16_t* __restrict__ y,
                        const int32_t* __restrict__ pos, const float* __restrict__ w, int T, int H,
                        const uint16_t* __restrict__ shared, const float* __restrict__ shared_gate,
                        uint16_t* __restrict__ dy, float* __restrict__ dw,
                        uint16_t* __restrict__ dshared, float* __restrict__ dgate) {
  pdl_trigger();
  pdl_wait();
  __shared__ float red[kCombineBackThreads / 32][K + 1];
  const unsigned rows = (unsigned)T * K;
  const int nv = H / 8, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = blockIdx.x;
  int p[K];
  float wj[K], dot[K + 1];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    p[j] = __ldg(pos + (size_t)t * K + j);
    wj[j] = __ldg(w + (size_t)t * K + j);
  }
#pragma unroll
  for (int j = 0; j <= K; ++j) dot[j] = 0.f;
  const float gs = shared_gate ? __ldg(shared_gate + t) : 1.f;
  for (int v = threadIdx.x; v < nv; v += blockDim.x) {
    const uint4 dq = __ldg(reinterpret_cast<const uint4*>(dout + (size_t)t * H) + v);
    uint4 q[K], sq = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      q[j] = make_uint4(0u, 0u, 0u, 0u);
      if (dw && (unsigned)p[j] < rows)
        q[j] = __ldg(reinterpret_cast<const uint4*>(y + (size_t)p[j] * H) + v);
    }
    if (dgate) sq = __ldg(reinterpret_cast<const uint4*>(shared + (size_t)t * H) + v);
    float d[8], f[8];
    unpack8(dq, d);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      unpack8(q[j], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) dot[j] = fmaf(d[i], f[i], dot[j]);
      if (dy && (unsigned)p[j] < rows) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = wj[j] * d[i];
        reinterpret_cast<uint4*>(dy + (size_t)p[j] * H)[v] = pack8(f);
      }
    }
    if (dgate) {
      unpack8(sq, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) dot[K] = fmaf(d[i], f[i], dot[K]);
    }
    if (dshared) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = gs * d[i];
      reinterpret_cast<uint4*>(dshared + (size_t)t * H)[v] = pack8(f);
    }
  }
#pragma unroll
  for (int j = 0; j <= K; ++j) {
    const float s = reduce_warp(dot[j]);
    if (lane == 0) red[warp][j] = s;
  }
  __syncthreads();
  if (threadIdx.x <= K) {
    float s = 0.f;
    for (int i = 0; i < (int)blockDim.x / 32; ++i) s += red[i][threadIdx.x];
    if (threadIdx.x == K) {
      if (dgate) dgate[t] = s;
    } else if (dw) {
      // (a slot without a row has no term in out[t], whatever dout[t] holds)
      const int pj = __ldg(pos + (size_t)t * K + threadIdx.x);
      dw[(size_t)t * K + threadIdx.x] = (unsigned)pj < rows ? s : 0.f;
    }
  }
}

// ------------------------------------------------------------------------------ gating
// With v_j the unnormalised weights of a token's chosen experts, r_j = v_j / sum v and
// w_j = scale r_j:  D = sum_j r_j dw_j and
//   softmax_renorm:       dl_j = scale r_j (dw_j - D)
//   sigmoid_bias_renorm:  dl_j = scale r_j (dw_j - D) (1 - sigmoid(l_j))
//   softmax (over all E): dl_e = scale p_e ([e chosen] dw_e - D),  D = sum_j p_j dw_j
// where the ids are those that w was normalised over.  SOFTMAX_RENORM and SIGMOID_BIAS_RENORM read the chosen
// logits only: a warp takes four tokens, eight lanes each for the chosen experts.  It stores zeros to the four
// rows, which lie next to each other, while the chosen logits are on their way, and then the chosen
// experts' values over them.  The chain of ids, gathered logits, exponentials and stores bounds it, each
// warp once: 32768 tokens of 256 experts, eight chosen, take 10.9 us in graphs of calls whose inputs change
// (5.4 at the copy bandwidth, 8.5 with the 64 bytes fetched for a gathered logit) and 7.7 on the same
// inputs again, where putting the rows together in shared memory first cost 1 us more.  SOFTMAX: a warp a
// token, 16.7 us (10.2) and 12.8.
constexpr int kGateBackWarps = 8;

// g of an expert that stands more than once in the lane's eight: the sum, in lane order, on the first
// of its lanes; the others' id becomes -1.
__device__ __forceinline__ void merge_chosen(int& id, float& g, int lane) {
  const unsigned same = __match_any_sync(0xffffffffu, id < 0 ? -1 - lane : id + kMaxExperts * (lane >> 3));
  if (!__any_sync(0xffffffffu, __popc(same) > 1)) return;
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < kMaxK; ++j) {
    const float o = __shfl_sync(0xffffffffu, g, (lane & 24) | j);
    sum += (same >> ((lane & 24) | j)) & 1u ? o : 0.f;
  }
  if (__popc(same) > 1) {
    g = sum;
    if (lane != __ffs(same) - 1) id = -1;
  }
}
__device__ __forceinline__ float sum8(float v) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float max8(float v) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

template <bool SIGMOID>
__global__ void __launch_bounds__(kGateBackWarps * 32)
gate_backward_chosen_kernel(const float* __restrict__ logits, const int32_t* __restrict__ ids,
                            const float* __restrict__ dw, int T, int E, int k, float scale,
                            float* __restrict__ dl) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = lane & 7;
  const unsigned t0 = (blockIdx.x * kGateBackWarps + warp) * 4, t = t0 + (lane >> 3), end = T;
  if (t0 >= end) return;
  int id = -1;
  float up = 0.f, l = -CUDART_INF_F;
  if (t < end && j < k) {
    id = __ldg(ids + (size_t)t * k + j);
    const float d = __ldg(dw + (size_t)t * k + j);
    if ((unsigned)id < (unsigned)E) {
      up = d;
      l = __ldg(logits + (size_t)t * E + id);
    } else {
      id = -1;
    }
  }
  // four rows of E floats start on a 16-byte boundary
  float* rows = dl + (size_t)t0 * E;
  const int n = (int)min(4u, end - t0) * E;
  for (int i = lane; i < n / 4; i += 32)
    reinterpret_cast<float4*>(rows)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (lane < (n & 3)) rows[(n & ~3) + lane] = 0.f;
  float v, total;
  if (!SIGMOID) {
    const float top = max8(l);
    // (zero by the logit, not by the largest: fmaxf drops NaNs, and those of a row with nothing else would
    // be lost; so they make every weight of the token NaN, as they do in routing)
    v = id >= 0 && l != -CUDART_INF_F ? expf(l - top) : 0.f;
    total = sum8(v);
  } else {
    v = id >= 0 ? 1.f / (1.f + expf(-l)) : 0.f;
    total = sum8(v);
    const bool tiny = total < 0x1p-64f;
    if (__any_sync(0xffffffffu, tiny)) {
      // sigmoids that fp32 is about to lose: e^l is their ratio to 2^-64, as far as 64 bits hold them
      // (group-limited routing's rule for the weights); beyond, weights and gradients are zero
      const float top = max8(l);
      if (tiny) v = id >= 0 && top > -709.f ? expf(l - top) : 0.f;
      const float again = sum8(v);
      if (tiny) total = again;
    }
  }
  const float r = total == 0.f ? 0.f : v / total;
  const bool live = r != 0.f;                  // (a slot of weight zero is in no sum, whatever its dw)
  const float D = sum8(live ? r * up : 0.f);
  float g = live ? scale * (r * (up - D)) : 0.f;
  if (SIGMOID) g *= 1.f / (1.f + expf(l));
  merge_chosen(id, g, lane);
  __syncwarp();                                // (the zeros come first)
  if (id >= 0) dl[(size_t)t * E + id] = g;
}

__global__ void __launch_bounds__(kGateBackWarps * 32)
gate_backward_softmax_kernel(const float* __restrict__ logits, const int32_t* __restrict__ ids,
                             const float* __restrict__ dw, int T, int E, int k, float scale,
                             float* __restrict__ dl) {
  pdl_trigger();
  __shared__ float row_s[kGateBackWarps][kMaxExperts];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* row = row_s[warp];
  const unsigned t = blockIdx.x * kGateBackWarps + warp;
  pdl_wait();
  if (t >= (unsigned)T) return;
  const float* lr = logits + (size_t)t * E;
  float z[kMaxExperts / 32], top = -CUDART_INF_F;
#pragma unroll
  for (int c = 0; c < kMaxExperts / 32; ++c)
    z[c] = lane + 32 * c < E ? __ldg(lr + lane + 32 * c) : -CUDART_INF_F;
  int id = -1;
  float up = 0.f;
  if (lane < k) {
    id = __ldg(ids + (size_t)t * k + lane);
    up = __ldg(dw + (size_t)t * k + lane);
    if ((unsigned)id >= (unsigned)E) id = -1;
  }
#pragma unroll
  for (int c = 0; c < kMaxExperts / 32; ++c) top = fmaxf(top, z[c]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float total = 0.f;
#pragma unroll
  for (int c = 0; c < kMaxExperts / 32; ++c) {
    z[c] = z[c] != -CUDART_INF_F ? expf(z[c] - top) : 0.f;   // (a NaN stays one; past E: -infinity)
    total += z[c];
    row[lane + 32 * c] = z[c];
  }
  total = reduce_warp(total);
  const float inv = total == 0.f ? 0.f : 1.f / total;
  __syncwarp();
  const float p = id >= 0 ? row[id] * inv : 0.f;
  float g = p != 0.f ? p * up : 0.f;           // (a slot of weight zero is in no sum, whatever its dw)
  const float D = reduce_warp(g);
  merge_chosen(id, g, lane);
  // (a token without an expert is in no loss: zeros, whatever its logits hold)
  const bool some = __any_sync(0xffffffffu, id >= 0);
  __syncwarp();
#pragma unroll
  for (int c = 0; c < kMaxExperts / 32; ++c) row[lane + 32 * c] = some ? -scale * (z[c] * inv * D) : 0.f;
  __syncwarp();
  if (id >= 0) row[id] += scale * g;
  __syncwarp();
#pragma unroll
  for (int c = 0; c < kMaxExperts / 32; ++c)
    if (lane + 32 * c < E) dl[(size_t)t * E + lane + 32 * c] = row[lane + 32 * c];
}

template <class F>
int by_k(int k, F go) {
  switch (k) {
    case 1: return go(std::integral_constant<int, 1>{});
    case 2: return go(std::integral_constant<int, 2>{});
    case 3: return go(std::integral_constant<int, 3>{});
    case 4: return go(std::integral_constant<int, 4>{});
    case 5: return go(std::integral_constant<int, 5>{});
    case 6: return go(std::integral_constant<int, 6>{});
    case 7: return go(std::integral_constant<int, 7>{});
    case 8: return go(std::integral_constant<int, 8>{});
    default: return MOE_ERR_INVALID_ARG;
  }
}

bool valid_rows(int T, int k, int H) {
  return T >= 0 && k >= 1 && k <= kMaxK && H > 0 && H % 8 == 0 && H <= (1 << 24) &&
         (long long)T * k <= 0x7fffffffLL;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_permute_backward(const uint16_t* dx_perm, const int32_t* pos, const uint16_t* add, int T,
                         int k, int H, int out_f32, void* dx, void* stream) {
  MOE_REQUIRE(valid_rows(T, k, H) && (out_f32 == 0 || out_f32 == 1));
  if (T == 0) return MOE_OK;
  MOE_REQUIRE(dx_perm && pos && dx && aligned16(dx_perm) && aligned16(dx) && aligned4(pos) &&
              aligned16(add));
  const dim3 grid(ceil_div(H / 8, kBackThreads), std::min(T, 65535)), block(kBackThreads);
  return by_k(k, [&](auto kc) -> int {
    constexpr int K = decltype(kc)::value;
    if (out_f32)
      MOE_LAUNCH_NEXT(true, (permute_backward_kernel<K, true>), grid, block, 0, (cudaStream_t)stream,
                     dx_perm, pos, add, T, H, dx);
    else
      MOE_LAUNCH_NEXT(true, (permute_backward_kernel<K, false>), grid, block, 0, (cudaStream_t)stream,
                     dx_perm, pos, add, T, H, dx);
    MOE_COUNT_LAUNCH();
    MOE_LAUNCH_CHECK();
    return MOE_OK;
  });
}

int moe_combine_backward(const uint16_t* dout, const uint16_t* y_perm, const int32_t* pos,
                         const float* w, int T, int k, int H, const uint16_t* shared,
                         const float* shared_gate, uint16_t* dy_perm, float* dw,
                         uint16_t* dshared, float* dshared_gate, void* stream) {
  MOE_REQUIRE(valid_rows(T, k, H));
  if (T == 0) return MOE_OK;
  MOE_REQUIRE(dout && pos && w && (dy_perm || dw || dshared || dshared_gate));
  MOE_REQUIRE(!dw || y_perm);
  MOE_REQUIRE(!dshared_gate || (shared && shared_gate));
  MOE_REQUIRE(aligned16(dout) && aligned16(y_perm) && aligned16(shared) && aligned16(dy_perm) &&
              aligned16(dshared) && aligned4(pos) && aligned4(w) && aligned4(dw) &&
              aligned4(shared_gate) && aligned4(dshared_gate));
  const int threads = std::min(kCombineBackThreads, (int)round_up((size_t)H / 8, 32));
  return by_k(k, [&](auto kc) -> int {
    constexpr int K = decltype(kc)::value;
    MOE_LAUNCH_NEXT(true, combine_backward_kernel<K>, dim3(T), dim3(threads), 0, (cudaStream_t)stream,
                   dout, y_perm, pos, w, T, H, shared, shared_gate, dy_perm, dw, dshared,
                   dshared_gate);
    MOE_COUNT_LAUNCH();
    MOE_LAUNCH_CHECK();
    return MOE_OK;
  });
}

int moe_gate_backward(const float* logits, const int32_t* ids, const float* dw, int T, int E,
                      int k, int gating, float scale, float* dlogits, void* stream) {
  MOE_REQUIRE(T >= 0 && E >= 1 && E <= kMaxExperts && k >= 1 && k <= kMaxK && k <= E);
  MOE_REQUIRE(gating >= MOE_GATING_SOFTMAX_RENORM && gating <= MOE_GATING_SIGMOID_BIAS_RENORM);
  if (T == 0) return MOE_OK;
  MOE_REQUIRE(logits && ids && dw && dlogits && aligned4(logits) && aligned4(ids) &&
              aligned4(dw) && aligned16(dlogits));
  cudaStream_t st = (cudaStream_t)stream;
  const dim3 block(kGateBackWarps * 32);
  const dim3 four(ceil_div(T, 4 * kGateBackWarps));
  if (gating == MOE_GATING_SOFTMAX)
    MOE_LAUNCH_NEXT(true, gate_backward_softmax_kernel, dim3(ceil_div(T, kGateBackWarps)), block, 0, st,
                   logits, ids, dw, T, E, k, scale, dlogits);
  else if (gating == MOE_GATING_SOFTMAX_RENORM)
    MOE_LAUNCH_NEXT(true, gate_backward_chosen_kernel<false>, four, block, 0, st, logits, ids, dw, T, E, k,
                   scale, dlogits);
  else
    MOE_LAUNCH_NEXT(true, gate_backward_chosen_kernel<true>, four, block, 0, st, logits, ids, dw, T, E, k,
                   scale, dlogits);
  MOE_COUNT_LAUNCH();
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // extern "C"
