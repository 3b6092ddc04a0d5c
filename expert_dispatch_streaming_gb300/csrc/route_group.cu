// Group-limited top-k gating: the experts form n_group groups of consecutive experts, a token
// first takes its `take` best groups and then its k best experts inside them.
//
// The router picks a handful of experts per token ("NovaLLM: Running Massive MoE Models Fully
// In-Memory", section "2. Why MoE Is a Natural Breakthrough Point"); the pages know no groups.
// With c_e the selection score of expert e (sigmoid(l_e) + bias_e, or the logit l_e):
//   group score  G_g = the sum of the two largest c_e of group g (sigmoid), or the largest
//                      (softmax modes); a group of one expert has its score;
//   taken        = the `take` groups of largest G_g, ties to the lower group;
//   chosen       = the k largest c_e inside the taken groups, ties to the lower expert;
//   weights      = those of the ungrouped gating at the chosen experts (gate_finish).
// A NaN score counts as -infinity.
//
// Both selections are exact in the sense of gate.cuh: fp32 scores decide unless the k-th and
// the next lie within the fp32 error margin; then the experts near the boundary (for a group:
// the candidates for its two largest) are re-scored with exact_score and compared in fp64.
//
// One warp gates one token.  Expert e's score sits in slot e / 32 of lane e % 32; a copy in
// shared memory lets the 32 / n_group lanes of a group (rounded down to a power of two) scan
// its experts, each keeping the two largest it saw, merged by shuffles.
#include "gate.cuh"
#include "route.cuh"

namespace moe {
namespace {

struct GroupSmem {
  float lrow[kMaxExperts];      // logits
  float srow[kMaxExperts];      // selection scores (NaN replaced)
  double exact_s[kMaxExperts];  // re-scored experts (NaN: not re-scored)
  double gx[32];                // re-scored groups
};

// Order-preserving map of a non-NaN float to an unsigned integer (0 is below every score).
__device__ __forceinline__ uint32_t score_key(float s) {
  const uint32_t u = __float_as_uint(s + 0.f);   // -0 becomes +0
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_score(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// Re-scores expert b once (exact_s[b] keeps it); every lane returns the same value.
__device__ __noinline__ double rescored(const GateParams& p, int t, int b, int lane,
                                        GroupSmem& sm) {
  double s = sm.exact_s[b];
  __syncwarp();
  if (s == s) return s;
  s = exact_score(p, t, b, lane);
  if (s != s) s = -CUDART_INF;
  s = __shfl_sync(0xffffffffu, s, 0);
  if (lane == 0) sm.exact_s[b] = s;
  __syncwarp();
  return s;
}

// Gating of token t by one warp (see the top of the file).  raw: the token's C summed router
// outputs, or NULL: sum the S slices of p.part.
template <int NC>
__device__ __forceinline__ void gate_token_grouped(const GateParams& p, int n_group, int take,
                                                   int t, const float* raw, GroupSmem& sm) {
  const int lane = threadIdx.x & 31, E = p.E, k = p.k, gs = E / n_group;
  const bool sig = p.mode == MOE_GATING_SIGMOID_BIAS_RENORM;
  float l[NC], sc[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int e = lane + 32 * c;
    float v = -CUDART_INF_F, s = -CUDART_INF_F;
    if (e < E) {
      v = raw ? raw[e] : sum_slices(p.part + (size_t)t * p.ldp + e, p.S, (size_t)p.T * p.ldp);
      if (p.logit_bias) v += p.logit_bias[e];
      s = v;
      if (sig) {
        s = 1.f / (1.f + expf(-v));
        if (p.sel_bias) s += p.sel_bias[e];
      }
      if (s != s) s = -CUDART_INF_F;
      sm.lrow[e] = v;
      sm.srow[e] = s;
      sm.exact_s[e] = CUDART_NAN;
      if (p.logits) p.logits[(size_t)t * E + e] = v;
    }
    l[c] = v;
    sc[c] = s;
  }
  if (lane == 0 && p.shared_gate && p.C > E) {
    const float z =
        raw ? raw[E] : sum_slices(p.part + (size_t)t * p.ldp + E, p.S, (size_t)p.T * p.ldp);
    p.shared_gate[t] = 1.f / (1.f + expf(-z));
  }
  __syncwarp();

  // ---- group scores: P lanes per group, lane (g, part) scans experts part, part + P, ...
  int P = 1;
  while (2 * P * n_group <= 32) P *= 2;
  const int g = lane / P, part = lane % P;
  float m1 = -CUDART_INF_F, m2 = -CUDART_INF_F;
  if (g < n_group)
    for (int i = part; i < gs; i += P) {
      const float s = sm.srow[g * gs + i];
      m2 = fmaxf(m2, fminf(m1, s));
      m1 = fmaxf(m1, s);
    }
  for (int o = 1; o < P; o <<= 1) {
    const float a1 = __shfl_xor_sync(0xffffffffu, m1, o), a2 = __shfl_xor_sync(0xffffffffu, m2, o);
    m2 = fmaxf(fmaxf(m2, a2), fminf(m1, a1));
    m1 = fmaxf(m1, a1);
  }
  float gsc = sig && gs > 1 ? m1 + m2 : m1;
  if (gsc != gsc) gsc = -CUDART_INF_F;
  // ---- the `take` best groups
  int rank = 0;
  for (int q = 0; q < n_group; ++q) {
    const float so = __shfl_sync(0xffffffffu, gsc, q * P);
    rank += better(so, q, gsc, g);
  }
  const bool lead = part == 0 && g < n_group;
  bool kept = lead && rank < take;
  int flag = 0;
  if (take < n_group) {
    const unsigned bk = __ballot_sync(0xffffffffu, lead && rank == take - 1);
    const unsigned bn = __ballot_sync(0xffffffffu, lead && rank == take);
    const float kth = __shfl_sync(0xffffffffu, gsc, __ffs(bk) - 1);
    const float nxt = __shfl_sync(0xffffffffu, gsc, __ffs(bn) - 1);
    const float tau = sig && gs > 1 ? 2.f * kTau : kTau;
    if (kth - nxt <= tau) {
      flag = 1;
      const bool def = kept && gsc - nxt > tau;
      const bool band = lead && !def && gsc >= kth - tau;
      unsigned bm = __ballot_sync(0xffffffffu, band);
      const int need = take - __popc(__ballot_sync(0xffffffffu, def));
      for (unsigned m = bm; m; m &= m - 1) {
        const int ll = __ffs(m) - 1, q = ll / P;
        // the experts that can be among the group's two largest (its largest, one-expert sums)
        const float lo = __shfl_sync(0xffffffffu, sig && gs > 1 ? m2 : m1, ll) - kTau;
        double x1 = -CUDART_INF, x2 = -CUDART_INF;
        for (int i = 0; i < gs; ++i) {
          if (!(sm.srow[q * gs + i] >= lo)) continue;
          const double s = rescored(p, t, q * gs + i, lane, sm);
          x2 = fmax(x2, fmin(x1, s));
          x1 = fmax(x1, s);
        }
        if (lane == 0) sm.gx[q] = sig && gs > 1 ? x1 + x2 : x1;
      }
      __syncwarp();
      const double mine = band ? sm.gx[g] : -CUDART_INF;
      int r = 0;
      double last = CUDART_INF, first = -CUDART_INF;   // worst taken, best left
      for (unsigned m = bm; m; m &= m - 1) {
        const int q = (__ffs(m) - 1) / P;
        r += better_d(sm.gx[q], q, mine, g);
      }
      kept = def || (band && r < need);
      const unsigned tk = __ballot_sync(0xffffffffu, band && r < need);
      for (unsigned m = bm; m; m &= m - 1) {
        const int ll = __ffs(m) - 1;
        const double s = sm.gx[ll / P];
        if ((tk >> ll) & 1) last = fmin(last, s);
        else first = fmax(first, s);
      }
      if (last - first < kNearTie) flag = 2;
    }
  }
  const unsigned gm = __ballot_sync(0xffffffffu, kept);   // leader lane of group q: q * P

  // ---- the k + 1 best experts inside the taken groups
  uint32_t key[NC];
  bool open[NC], chosen[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int e = lane + 32 * c;
    open[c] = e < E && ((gm >> ((e / gs) * P)) & 1);
    key[c] = open[c] ? score_key(sc[c]) : 0u;
    chosen[c] = false;
  }
  const int pool = take * gs;
  float kth = 0.f, nxt = -CUDART_INF_F;
#pragma unroll 1
  for (int r = 0; r < min(k + 1, pool); ++r) {
    uint32_t best = 0;
    int id = 0x7fffffff;
#pragma unroll
    for (int c = NC - 1; c >= 0; --c)
      if (key[c] >= best) { best = key[c]; id = lane + 32 * c; }
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    id = (int)__reduce_min_sync(0xffffffffu, best == top ? (unsigned)id : 0x7fffffffu);
    if (r == k - 1) kth = key_score(top);
    if (r == k) nxt = key_score(top);
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (lane + 32 * c == id) {
        key[c] = 0u;
        if (r < k) chosen[c] = true;
      }
  }
  if (k < pool && kth - nxt <= kTau) {
    // experts within the margin of the boundary are re-scored; the ones clear of it stay
    if (flag == 0) flag = 1;
    bool band[NC];
    int n_def = 0;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const bool d = chosen[c] && sc[c] - nxt > kTau;
      band[c] = open[c] && !d && sc[c] >= kth - kTau;
      chosen[c] = d;
      n_def += __popc(__ballot_sync(0xffffffffu, d));
    }
#pragma unroll 1
    for (int c = 0; c < NC; ++c) {
      unsigned m = 0;
#pragma unroll
      for (int c2 = 0; c2 < NC; ++c2) {
        const unsigned b = __ballot_sync(0xffffffffu, band[c2]);
        m = c2 == c ? b : m;
      }
      for (; m; m &= m - 1) rescored(p, t, 32 * c + __ffs(m) - 1, lane, sm);
    }
    double last = CUDART_INF;
    for (int r = n_def; r <= k; ++r) {   // the last round finds the best one left out
      double bs = -CUDART_INF;
      int bi = 0x7fffffff;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int e = lane + 32 * c;
        if (band[c] && !chosen[c] && better_d(sm.exact_s[e], e, bs, bi)) {
          bs = sm.exact_s[e];
          bi = e;
        }
      }
      warp_argmax_d(bs, bi);
      if (r == k) {
        if (bi != 0x7fffffff && last - bs < kNearTie) flag = 2;
        break;
      }
      last = bs;
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (lane + 32 * c == bi) chosen[c] = true;
    }
  }
  __syncwarp();
  gate_finish<NC>(p, t, l, chosen, sm.lrow, flag);
  // a token whose chosen scores are all zero (every expert left to it is masked) would get
  // 0 / 0: its weights are zero instead
  __syncwarp();
  float left = 0.f;
  if (lane < k) {
    const float lj = sm.lrow[p.ids[(size_t)t * k + lane]];
    left = sig ? 1.f / (1.f + expf(-lj)) : (lj == -CUDART_INF_F ? 0.f : 1.f);
  }
  if (__all_sync(0xffffffffu, left == 0.f) && lane < k) p.w[(size_t)t * k + lane] = 0.f;
}

template <int NC>
__global__ void __launch_bounds__(G_WARPS * 32)
gate_group_kernel(GateParams p, int n_group, int take) {
  pdl_trigger();
  pdl_wait();
  __shared__ GroupSmem sm[G_WARPS];
  const int warp = threadIdx.x >> 5;
  for (int it = 0; it < p.tok_per_warp; ++it) {
    const int t = (blockIdx.x * G_WARPS + warp) * p.tok_per_warp + it;
    if (t >= p.T) break;
    gate_token_grouped<NC>(p, n_group, take, t, nullptr, sm[warp]);
    __syncwarp();
  }
}

// Everything after the router product for a batch of at most kSmallT tokens in one CTA, as
// route_tail_kernel: the slices of every logit summed (G lanes a logit, fixed order), one warp a
// token gating, then the histogram, scan, ranks and tables (route_dispatch_block).
constexpr int kTailWarps = 32;
struct GroupTailSmem {
  TailSmem tail;                 // (lrow / exact_s unused)
  GroupSmem g[kSmallT];
};
__global__ void __launch_bounds__(kTailWarps * 32)
route_group_tail_kernel(GateParams p, int n_group, int take, int32_t* __restrict__ counts,
                        int32_t* __restrict__ offsets, int32_t* __restrict__ pos,
                        int32_t* __restrict__ src, int32_t* __restrict__ active,
                        int32_t* __restrict__ n_active, int32_t* __restrict__ shared_meta,
                        uint16_t* __restrict__ x_perm) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ __align__(16) uint8_t raw_smem[];
  GroupTailSmem& sm = *reinterpret_cast<GroupTailSmem*>(raw_smem);
  constexpr int NT = kTailWarps * 32;
  const int tid = threadIdx.x, warp = tid >> 5, T = p.T, C = p.C, E = p.E, S = p.S, n = T * C;
  const size_t stride = (size_t)T * C;
  int G = 32;
  while (G > 1 && n * G > NT) G >>= 1;
  const int per = NT / G, g = tid % G;
  for (int li = tid / G; li < ((n + per - 1) / per) * per; li += per) {
    float a[4] = {0.f, 0.f, 0.f, 0.f};
    if (li < n) {
      int sp = g, i = 0;
#pragma unroll 4
      for (; sp < S; sp += G, ++i) a[i & 3] += __ldcg(p.part + (size_t)sp * stride + li);
    }
    float v = (a[0] + a[1]) + (a[2] + a[3]);
    for (int o = G >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (g == 0 && li < n) sm.tail.lg[li] = v;
  }
  for (int e = tid; e < kMaxExperts; e += NT) sm.tail.hist[e] = 0;
  __syncthreads();
  if (warp < T) {
    GateParams q = p;
    q.hist = sm.tail.hist;
    const float* raw = sm.tail.lg + (size_t)warp * C;
    if (E <= 64) gate_token_grouped<2>(q, n_group, take, warp, raw, sm.g[warp]);
    else gate_token_grouped<EC>(q, n_group, take, warp, raw, sm.g[warp]);
  }
  __syncthreads();
  route_dispatch_block<NT>(p.ids, T, p.k, E, counts, offsets, pos, src, active, n_active,
                           shared_meta, x_perm, p.x, p.H, sm.tail);
}

}  // namespace

int launch_route_group_tail(const GateParams& p, int n_group, int take, int32_t* counts,
                            int32_t* offsets, int32_t* pos, int32_t* src, int32_t* active,
                            int32_t* n_active, int32_t* shared_meta, uint16_t* x_perm,
                            cudaStream_t st) {
  static bool attr = false;
  if (!attr) {
    MOE_CUDA_TRY(cudaFuncSetAttribute(route_group_tail_kernel,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      (int)sizeof(GroupTailSmem)));
    attr = true;
  }
  MOE_LAUNCH_PDL(route_group_tail_kernel, dim3(1), dim3(kTailWarps * 32), sizeof(GroupTailSmem),
                 st, p, n_group, take, counts, offsets, pos, src, active, n_active, shared_meta,
                 x_perm);
  MOE_COUNT_LAUNCH();
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

int launch_gate_group(const GateParams& p, int n_group, int take, cudaStream_t st) {
  GateParams q = p;
  q.tok_per_warp = 1;
  const dim3 grid(ceil_div(q.T, G_WARPS * q.tok_per_warp)), block(G_WARPS * 32);
  if (q.E <= 32) MOE_LAUNCH_PDL(gate_group_kernel<1>, grid, block, 0, st, q, n_group, take);
  else if (q.E <= 64) MOE_LAUNCH_PDL(gate_group_kernel<2>, grid, block, 0, st, q, n_group, take);
  else if (q.E <= 128) MOE_LAUNCH_PDL(gate_group_kernel<4>, grid, block, 0, st, q, n_group, take);
  else MOE_LAUNCH_PDL(gate_group_kernel<EC>, grid, block, 0, st, q, n_group, take);
  MOE_COUNT_LAUNCH();
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace moe
