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
//   weights      = those of the ungrouped gating at the chosen experts.
// A NaN score counts as -infinity.
//
// Both selections are exact in the sense of gate.cuh: fp32 scores decide unless the k-th and
// the next lie within the fp32 error margin; then the experts near the boundary (for a group:
// the candidates for its two largest) are re-scored and compared in fp64.
//
// One warp gates one token, its scores in shared memory: expert e's is handled by lane e % 32;
// 32 / n_group lanes (rounded down to a power of two) scan a group, each keeping the two largest
// it saw.  What costs here is latency: a lane's loads go out together, a token takes 5,600 clocks
// (scores 1,950, groups 930, experts 1,420, weights and tables 1,300), and the few tokens that need
// re-scoring, 12 us each by device clock stamps, are shared by their whole CTA.
#include "gate.cuh"
#include "route.cuh"

namespace moe {
namespace {

struct GroupSmem {
  float lrow[kMaxExperts];      // logits
  float srow[kMaxExperts];      // selection scores (NaN replaced)
  double exact_s[kMaxExperts];  // re-scored experts (NaN: not re-scored)
  int ids[kMaxK];               // the chosen, ascending
};

// The groups' layout over a warp's lanes.
struct Groups {
  int n, take, gs, P;           // groups, groups taken, experts per group, lanes per group
  unsigned mul;                 // e / gs = e * mul >> 16 for e < 256
  bool pairs;                   // a group's score is the sum of its two largest
  __device__ __forceinline__ Groups(int n_, int take_, int E, bool sig) : n(n_), take(take_) {
    gs = E / n;
    P = 1;
    while (2 * P * n <= 32) P *= 2;
    mul = (65536u + gs - 1) / gs;
    pairs = sig && gs > 1;
  }
  __device__ __forceinline__ int of(int e) const { return (int)(e * mul >> 16); }
  // the lane that holds group g's score
  __device__ __forceinline__ int lane_of(int g) const { return g * P; }
};

// Order-preserving map of a non-NaN float to an unsigned integer (0 is below every score).
__device__ __forceinline__ uint32_t score_key(float s) {
  const uint32_t u = __float_as_uint(s + 0.f);   // -0 becomes +0
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_score(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// Logits and selection scores of token t into sm, all of a lane's loads in flight together.  raw:
// the token's C summed router outputs, or NULL: sum the S slices of p.part.
template <int NC>
__device__ __forceinline__ void score_token(const GateParams& p, int t, const float* raw,
                                            GroupSmem& sm) {
  const int lane = threadIdx.x & 31, E = p.E;
  const bool sig = p.mode == MOE_GATING_SIGMOID_BIAS_RENORM;
  const size_t stride = (size_t)p.T * p.ldp;
  const float* part = raw ? raw : p.part + (size_t)t * p.ldp;
  const int S = raw ? 1 : p.S;
  float v[NC], lb[NC], sb[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int e = min(lane + 32 * c, E - 1);
    v[c] = part[e];
    lb[c] = p.logit_bias ? __ldg(p.logit_bias + e) : 0.f;
    sb[c] = sig && p.sel_bias ? __ldg(p.sel_bias + e) : 0.f;
  }
  if (S > 1)
#pragma unroll
    for (int c = 0; c < NC; ++c) v[c] = sum_slices(part + min(lane + 32 * c, E - 1), S, stride);
  if (lane == 0 && p.shared_gate && p.C > E)
    p.shared_gate[t] = 1.f / (1.f + expf(-(S == 1 ? part[E] : sum_slices(part + E, S, stride))));
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int e = lane + 32 * c;
    const float l = v[c] + lb[c];
    // (hardware exponential and reciprocal: off by less than 1e-6, far inside kTau)
    const float s = sig ? __fdividef(1.f, 1.f + __expf(-l)) + sb[c] : l;
    if (e < E) {
      sm.lrow[e] = l;
      sm.srow[e] = s != s ? -CUDART_INF_F : s;
      if (p.logits) p.logits[(size_t)t * E + e] = l;
    }
  }
  __syncwarp();
}

// Scores of the groups and the `take` best: of this lane's group (lane / P) its score, the score an
// expert needs to be among its deciding ones, and its rank; kth / nxt: the take-th score and the
// next (nxt = -infinity when every group is taken).  A sum of two scores is held as half of it:
// halves are exact, and two of the lowest finite value (a mask) do not add up to -infinity.
struct GroupRank {
  float score, least, kth, nxt;
  int rank;
};
__device__ __forceinline__ GroupRank rank_groups(const Groups& G, const GroupSmem& sm) {
  const int lane = threadIdx.x & 31, g = lane / G.P, part = lane % G.P;
  float m1 = -CUDART_INF_F, m2 = -CUDART_INF_F;
  if (g < G.n) {
    // eight scores at a time, their loads in flight together
    const float* s = sm.srow + g * G.gs;
#pragma unroll 1
    for (int i0 = part; i0 < G.gs; i0 += 8 * G.P) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = i0 + j * G.P < G.gs ? s[i0 + j * G.P] : -CUDART_INF_F;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        m2 = fmaxf(m2, fminf(m1, v[j]));
        m1 = fmaxf(m1, v[j]);
      }
    }
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    if (o >= G.P) break;
    const float a1 = __shfl_xor_sync(0xffffffffu, m1, o), a2 = __shfl_xor_sync(0xffffffffu, m2, o);
    m2 = fmaxf(fmaxf(m2, a2), fminf(m1, a1));
    m1 = fmaxf(m1, a1);
  }
  GroupRank r;
  r.score = G.pairs ? 0.5f * m1 + 0.5f * m2 : m1;
  if (r.score != r.score) r.score = -CUDART_INF_F;
  r.least = (G.pairs ? m2 : m1) - kTau;
  r.rank = 0;
  r.kth = 0.f;
  r.nxt = -CUDART_INF_F;
#pragma unroll 1
  for (int q0 = 0; q0 < G.n; q0 += 8) {
    float o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)     // (past the last group: a lane of no group, not counted)
      o[j] = __shfl_sync(0xffffffffu, r.score, G.lane_of(q0 + j) & 31);
#pragma unroll
    for (int j = 0; j < 8; ++j) r.rank += q0 + j < G.n && better(o[j], q0 + j, r.score, g);
  }
  if (g >= G.n) r.rank = 32;
  const unsigned bk = __ballot_sync(0xffffffffu, r.rank == G.take - 1);
  const unsigned bn = __ballot_sync(0xffffffffu, r.rank == G.take);
  r.kth = __shfl_sync(0xffffffffu, r.score, __ffs(bk) - 1);
  if (bn) r.nxt = __shfl_sync(0xffffffffu, r.score, __ffs(bn) - 1);
  return r;
}

// The k + 1 best experts of the groups in gm (bit lane_of(g)): chosen: bit c = the lane's expert
// lane + 32 c is among the k; kth / nxt the k-th score and the next.
struct Top {
  unsigned chosen;
  float kth, nxt;
};
template <int NC>
__device__ __noinline__ Top top_experts(const Groups& G, const GroupSmem& sm, unsigned gm, int E,
                                        int k) {
  const int lane = threadIdx.x & 31;
  uint32_t key[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int e = lane + 32 * c;
    const bool open = e < E && ((gm >> G.lane_of(G.of(e))) & 1);
    key[c] = open ? score_key(sm.srow[e]) : 0u;
  }
  Top r{0u, 0.f, -CUDART_INF_F};
#pragma unroll 1
  for (int i = 0; i < min(k + 1, G.take * G.gs); ++i) {
    uint32_t best = 0;
    int id = 0x7fffffff;
#pragma unroll
    for (int c = 0; c < NC; ++c) best = max(best, key[c]);
#pragma unroll
    for (int c = NC - 1; c >= 0; --c)
      if (key[c] == best) id = lane + 32 * c;
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    const unsigned ties = __ballot_sync(0xffffffffu, best == top);
    if ((ties & (ties - 1)) == 0)
      id = __shfl_sync(0xffffffffu, id, __ffs(ties) - 1);
    else
      id = (int)__reduce_min_sync(0xffffffffu, best == top ? (unsigned)id : 0x7fffffffu);
    if (i == k - 1) r.kth = key_score(top);
    if (i == k) r.nxt = key_score(top);
    const bool won = (id & 31) == lane;
    if (won && i < k) r.chosen |= 1u << (id >> 5);
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (won && (id >> 5) == c) key[c] = 0u;
  }
  return r;
}

// The same where no boundary is near: the k are taken by the upper 24 bits of their keys, ties to
// the lower expert (one warp reduction a round, where the exact order takes three dependent ones),
// then kth and nxt are the exact worst taken and best left.  A wrong choice shows as kth < nxt.
template <int NC>
__device__ __forceinline__ Top top_quick(const Groups& G, const GroupSmem& sm, unsigned gm, int E,
                                         int k) {
  const int lane = threadIdx.x & 31;
  uint32_t key[NC], cut[NC];
  unsigned open = 0, left = 0;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int e = lane + 32 * c;
    const bool in = e < E && ((gm >> G.lane_of(G.of(e))) & 1);
    key[c] = score_key(sm.srow[min(e, E - 1)]);
    cut[c] = in ? (key[c] & ~255u) | (255u - e) : 0u;
    open |= (unsigned)in << c;
  }
#pragma unroll 1
  for (int i = 0; i < k; ++i) {
    uint32_t best = 0;
#pragma unroll
    for (int c = 0; c < NC; ++c) best = max(best, cut[c]);
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
#pragma unroll
    for (int c = 0; c < NC; ++c) cut[c] = cut[c] == top ? 0u : cut[c];
  }
  uint32_t worst = 0xffffffffu, next = 0u;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    left |= (unsigned)(cut[c] != 0u) << c;
    if (cut[c]) next = max(next, key[c]);
    else if ((open >> c) & 1) worst = min(worst, key[c]);
  }
  Top r;
  r.chosen = open & ~left;
  r.kth = key_score(__reduce_min_sync(0xffffffffu, worst));
  next = __reduce_max_sync(0xffffffffu, next);
  r.nxt = next ? key_score(next) : -CUDART_INF_F;
  return r;
}

// The chosen in ascending id order, lane j the j-th, and their weights (those of gate_finish,
// which has one lane do it, summed in the same order).
template <int NC>
__device__ __forceinline__ void finish_token(const GateParams& p, int t, GroupSmem& sm,
                                             unsigned chosen, int flag) {
  const int lane = threadIdx.x & 31, E = p.E, k = p.k;
  const bool sig = p.mode == MOE_GATING_SIGMOID_BIAS_RENORM;
  unsigned m[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) m[c] = __ballot_sync(0xffffffffu, (chosen >> c) & 1);
  int base = 0;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    if ((chosen >> c) & 1) sm.ids[base + __popc(m[c] & ((1u << lane) - 1u))] = lane + 32 * c;
    base += __popc(m[c]);
  }
  __syncwarp();
  const int id = lane < k ? sm.ids[lane] : 0;
  const float lj = lane < k ? sm.lrow[id] : -CUDART_INF_F;
  const bool all = p.mode == MOE_GATING_SOFTMAX;
  float v, denom = 0.f;
  if (sig) {
    v = 1.f / (1.f + expf(-lj));
  } else {
    float top = lj;
    if (all)
#pragma unroll 1
      for (int e = lane; e < E; e += 32) top = fmaxf(top, sm.lrow[e]);
    top = warp_max(top);
    v = expf(lj - top);
    if (all) {
#pragma unroll 1
      for (int e = lane; e < E; e += 32) denom += expf(sm.lrow[e] - top);
      denom = warp_sum(denom);
    }
  }
  auto sum = [&] {   // of the chosen's v, in order
    float o[kMaxK], s = 0.f;
#pragma unroll
    for (int j = 0; j < kMaxK; ++j) o[j] = __shfl_sync(0xffffffffu, v, j);
#pragma unroll
    for (int j = 0; j < kMaxK; ++j) s += j < k ? o[j] : 0.f;
    return s;
  };
  if (!all) denom = sum();
  if (sig && denom < 0x1p-64f) {
    // sigmoids that fp32 is about to lose (logits below -44): e^l is their ratio to 2^-64, as far
    // as 64 bits hold them; beyond, they are zero
    const float top = warp_max(lj);
    v = top > -709.f ? expf(lj - top) : 0.f;
    denom = sum();
  }
  // a token whose chosen scores are all zero (every expert left to it is masked) would get
  // 0 / 0: its weights are zero instead
  const float has = lane >= k ? 0.f : sig ? v : (lj == -CUDART_INF_F ? 0.f : 1.f);
  const bool none = __all_sync(0xffffffffu, has == 0.f);
  if (lane < k) {
    p.ids[(size_t)t * k + lane] = id;
    p.w[(size_t)t * k + lane] = none ? 0.f : v * (p.scale / denom);
    atomicAdd(&p.hist[(t / kTileT) * E + id], 1);
  }
  if (lane == 0 && p.tie_flags) p.tie_flags[t] = flag;
  __syncwarp();
}

// Gating of token t by one warp when no boundary is near; returns false, with the scores in sm
// and nothing chosen, when one is.
template <int NC>
__device__ __forceinline__ bool gate_quick(const GateParams& p, const Groups& G, int t,
                                           const float* raw, GroupSmem& sm) {
  score_token<NC>(p, t, raw, sm);
  const GroupRank r = rank_groups(G, sm);
  if (r.kth - r.nxt <= kTau) return false;
  const unsigned lead = __ballot_sync(0xffffffffu, r.rank < G.take);
  const Top top = top_quick<NC>(G, sm, lead, p.E, p.k);
  if (top.kth - top.nxt <= kTau) return false;
  finish_token<NC>(p, t, sm, top.chosen, 0);
  return true;
}

// Re-scoring of near-boundary experts by the whole CTA.  The token's warp lists the experts it
// needs; all threads share each dot product (their loads in flight together: one memory latency
// an expert where a warp by itself would wait for dozens); then the token's warp turns them into
// fp64 scores, an expert per lane (fp64 functions are slow here, once for all lanes).  One token
// in a hundred needs it, and one that is slow sets the time of the kernel.
constexpr int kBatch = 16;
struct Service {
  int n, token;                // n = 0: nothing more
  int list[kMaxExperts];
  float2 part[kBatch][32];     // per expert of a batch and warp: (hi, lo) of its share
};

// All the CTA's threads: their shares of x[token] . W_r[:, list[i0 + i]] in compensated fp32 (as
// exact_score's), thread i the 8-element chunks i, i + threads, ...
__device__ __noinline__ void dots(const GateParams& p, Service& sv, int i0) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
  const uint16_t* xr = p.x + (size_t)sv.token * p.H;
  const int n = min(sv.n - i0, kBatch), nch = p.H / 8;
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const int b = sv.list[i0 + i];
    float hi = 0.f, lo = 0.f;
#pragma unroll 1
    for (int c0 = tid; c0 < nch; c0 += 4 * nt) {
      uint4 xq[4];
      float4 wa[4], wb[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = c0 + j * nt;
        xq[j] = make_uint4(0u, 0u, 0u, 0u);
        wa[j] = wb[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c >= nch) continue;
        xq[j] = __ldg(reinterpret_cast<const uint4*>(xr + 8 * c));
        if (p.w_rT) {
          const float4* w = reinterpret_cast<const float4*>(p.w_rT + (size_t)b * p.H + 8 * c);
          wa[j] = w[0];
          wb[j] = w[1];
        } else {
          const float* w = p.w_r + (size_t)8 * c * p.E + b;
          const size_t E = p.E;
          wa[j] = make_float4(w[0], w[E], w[2 * E], w[3 * E]);
          wb[j] = make_float4(w[4 * E], w[5 * E], w[6 * E], w[7 * E]);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 x01 = bf16x2_to_float2(xq[j].x), x23 = bf16x2_to_float2(xq[j].y);
        const float2 x45 = bf16x2_to_float2(xq[j].z), x67 = bf16x2_to_float2(xq[j].w);
        dot_term(hi, lo, x01.x, wa[j].x);
        dot_term(hi, lo, x01.y, wa[j].y);
        dot_term(hi, lo, x23.x, wa[j].z);
        dot_term(hi, lo, x23.y, wa[j].w);
        dot_term(hi, lo, x45.x, wb[j].x);
        dot_term(hi, lo, x45.y, wb[j].y);
        dot_term(hi, lo, x67.x, wb[j].z);
        dot_term(hi, lo, x67.y, wb[j].w);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float h2 = __shfl_xor_sync(0xffffffffu, hi, o);
      const float l2 = __shfl_xor_sync(0xffffffffu, lo, o);
      df_add(hi, lo, h2, l2);
    }
    if (lane == 0) sv.part[i][warp] = make_float2(hi, lo);
  }
  __syncthreads();
}
// The asking warp: exact scores of the experts e of token t with srow[e] >= lo(e) that are
// open(e) and have none yet.
template <class Want>
__device__ __forceinline__ void rescore(const GateParams& p, int t, GroupSmem& sm, Service& sv,
                                        Want want) {
  const int lane = threadIdx.x & 31;
  int n = 0;
#pragma unroll 1
  for (int c = 0; 32 * c < p.E; ++c) {
    const int e = lane + 32 * c;
    const bool asked = want(min(e, p.E - 1));       // (all lanes call it: it may shuffle)
    const bool w = e < p.E && asked && sm.exact_s[e] != sm.exact_s[e];
    const unsigned m = __ballot_sync(0xffffffffu, w);
    if (w) sv.list[n + __popc(m & ((1u << lane) - 1u))] = e;
    n += __popc(m);
  }
  if (n == 0) return;
  if (lane == 0) {
    sv.n = n;
    sv.token = t;
  }
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += kBatch) {
    __syncthreads();
    dots(p, sv, i0);
    if (lane < min(n - i0, kBatch)) {
      const int e = sv.list[i0 + lane];
      float hi = 0.f, lo = 0.f;
#pragma unroll 1
      for (int w = 0; w < (int)(blockDim.x >> 5); ++w)
        df_add(hi, lo, sv.part[lane][w].x, sv.part[lane][w].y);
      double d = (double)hi + (double)lo;
      if (p.logit_bias) d += (double)p.logit_bias[e];
      if (p.mode == MOE_GATING_SIGMOID_BIAS_RENORM) {
        d = 1.0 / (1.0 + exp(-d));
        if (p.sel_bias) d += (double)p.sel_bias[e];
      }
      sm.exact_s[e] = d != d ? -CUDART_INF : d;
    }
    __syncwarp();
  }
}

// Gating of token t (scores in sm) with the boundaries that are near decided by exact scores.
template <int NC>
__device__ __noinline__ void gate_slow(const GateParams& p, const Groups& G, int t, GroupSmem& sm,
                                       Service& sv) {
  const int lane = threadIdx.x & 31, E = p.E, k = p.k, g = lane / G.P;
#pragma unroll 1
  for (int e = lane; e < E; e += 32) sm.exact_s[e] = CUDART_NAN;
  __syncwarp();
  int flag = 0;
  const GroupRank r = rank_groups(G, sm);
  bool kept = r.rank < G.take;
  if (r.kth - r.nxt <= kTau) {
    flag = 1;
    // groups clear of the boundary stay; the band is decided by its exact scores
    const bool in = g < G.n, def = kept && r.score - r.nxt > kTau;
    const bool band = in && !def && r.score >= r.kth - kTau;
    const unsigned bm = __ballot_sync(0xffffffffu, band);
    rescore(p, t, sm, sv, [&](int e) {
      const int ll = G.lane_of(G.of(e));
      const float lo = __shfl_sync(0xffffffffu, r.least, ll);
      return ((bm >> ll) & 1) && sm.srow[e] >= lo;
    });
    double x1 = -CUDART_INF, x2 = -CUDART_INF;
    if (band)
#pragma unroll 1
      for (int i = 0; i < G.gs; ++i) {
        const int e = g * G.gs + i;
        if (!(sm.srow[e] >= r.least)) continue;
        const double s = sm.exact_s[e];
        if (s > x1) { x2 = x1; x1 = s; }
        else if (s > x2) x2 = s;
      }
    const double gx = G.pairs ? x1 + x2 : x1;
    int clear = 0, rank = 0;
    double last = CUDART_INF, first = -CUDART_INF;   // the band's worst taken, best left
#pragma unroll 1
    for (int q = 0; q < G.n; ++q) {
      clear += (int)__shfl_sync(0xffffffffu, (int)def, G.lane_of(q));
      const double o = __shfl_sync(0xffffffffu, gx, G.lane_of(q));
      rank += ((bm >> G.lane_of(q)) & 1) && better_d(o, q, gx, g);
    }
    kept = def || (band && rank < G.take - clear);
#pragma unroll 1
    for (int q = 0; q < G.n; ++q) {
      const double o = __shfl_sync(0xffffffffu, gx, G.lane_of(q));
      const int tk = __shfl_sync(0xffffffffu, (int)kept, G.lane_of(q));
      if (!((bm >> G.lane_of(q)) & 1)) continue;
      if (tk) last = o < last ? o : last;
      else first = o > first ? o : first;
    }
    if (last - first < kNearTie) flag = 2;
  }
  const unsigned gm = __ballot_sync(0xffffffffu, kept);
  Top top = top_experts<NC>(G, sm, gm, E, k);
  if (top.kth - top.nxt <= kTau) {
    if (flag == 0) flag = 1;
    // experts clear of the boundary stay; the band is decided by its exact scores
    const float lo = top.kth - kTau;
    auto in_band = [&](int e) {
      const float s = sm.srow[e];
      return ((gm >> G.lane_of(G.of(e))) & 1) && !(s - top.nxt > kTau) && s >= lo;
    };
    rescore(p, t, sm, sv, in_band);
    unsigned chosen = 0, band = 0;
    int clear = 0;
#pragma unroll 1
    for (int c = 0; 32 * c < E; ++c) {
      const int e = lane + 32 * c;
      const bool b = e < E && in_band(e), d = ((top.chosen >> c) & 1) && !b;
      band |= (unsigned)b << c;
      chosen |= (unsigned)d << c;
      clear += __popc(__ballot_sync(0xffffffffu, d));
    }
    double last = CUDART_INF;
#pragma unroll 1
    for (int i = clear; i <= k; ++i) {   // the last round finds the best one left out
      double bs = -CUDART_INF;
      int bi = 0x7fffffff;
#pragma unroll 1
      for (unsigned m = band & ~chosen; m; m &= m - 1) {
        const int e = lane + 32 * (__ffs(m) - 1);
        if (better_d(sm.exact_s[e], e, bs, bi)) {
          bs = sm.exact_s[e];
          bi = e;
        }
      }
#pragma unroll 1
      for (int o = 16; o > 0; o >>= 1) {
        const double so = __shfl_xor_sync(0xffffffffu, bs, o);
        const int io = __shfl_xor_sync(0xffffffffu, bi, o);
        if (better_d(so, io, bs, bi)) {
          bs = so;
          bi = io;
        }
      }
      if (i == k) {
        if (bi != 0x7fffffff && last - bs < kNearTie) flag = 2;
        break;
      }
      last = bs;
      if ((bi & 31) == lane && bi != 0x7fffffff) chosen |= 1u << (bi >> 5);
    }
    top.chosen = chosen;
  }
  finish_token<NC>(p, t, sm, top.chosen, flag);
}

// The tokens of the CTA's warps that need re-scoring (bit w of `slow`: warp w's, t0 + w), one after
// another, each by its own warp with the others serving.  All threads call it.
template <int NC>
__device__ __forceinline__ void gate_slow_all(const GateParams& p, const Groups& G, int t0,
                                              unsigned slow, GroupSmem* sm, Service& sv) {
  const int warp = threadIdx.x >> 5;
#pragma unroll 1
  for (; slow; slow &= slow - 1) {
    const int w = __ffs(slow) - 1;
    if (warp == w) {
      gate_slow<NC>(p, G, t0 + w, sm[w], sv);
      if ((threadIdx.x & 31) == 0) sv.n = 0;
      __syncthreads();
    } else {
      // (sv.n is read between a batch's two barriers only: once the second has passed, the asking
      // warp may write the next request)
      for (int i0 = 0;;) {
        __syncthreads();
        const int n = sv.n;
        if (n == 0) break;
        dots(p, sv, i0);
        i0 = i0 + kBatch < n ? i0 + kBatch : 0;
      }
    }
    __syncthreads();
  }
}

// Batches of at least this many tokens and more than kListMinE experts gate in two steps (see
// gate_group_list_kernel).
constexpr int kListMinT = 4096, kListMinE = 128;

template <int NC>
__global__ void __launch_bounds__(G_WARPS * 32)
gate_group_kernel(const __grid_constant__ GateParams p, int n_group, int take) {
  pdl_trigger();
  pdl_wait();
  __shared__ GroupSmem sm[G_WARPS];
  __shared__ Service sv;
  __shared__ unsigned slow;
  const int warp = threadIdx.x >> 5, t0 = blockIdx.x * G_WARPS, t = t0 + warp;
  const Groups G(n_group, take, p.E, p.mode == MOE_GATING_SIGMOID_BIAS_RENORM);
  if (threadIdx.x == 0) slow = 0;
  __syncthreads();
  if (t < p.T && !gate_quick<NC>(p, G, t, nullptr, sm[warp]) && (threadIdx.x & 31) == 0)
    atomicOr(&slow, 1u << warp);
  __syncthreads();
  gate_slow_all<NC>(p, G, t0, slow, sm, sv);
}

// Large batches in two steps: the tokens that need re-scoring, one or two in a hundred, each take
// several times as long as the others, and their CTAs would be the last; so the first kernel lists
// them and a second gives each a CTA of its own.  (The whole routing of 256 experts: 8192 tokens
// 147 us with one kernel, 140 with two, 4096 104 / 98, 2048 80 / 86; of 60 experts, where fewer
// scores are close, 8192 tokens 65 / 67.)  The list's order varies from run to run; nothing else
// depends on it.
template <int NC>
__global__ void __launch_bounds__(G_WARPS * 32)
gate_group_list_kernel(const __grid_constant__ GateParams p, int n_group, int take,
                       int32_t* __restrict__ list) {
  pdl_trigger();
  pdl_wait();
  __shared__ GroupSmem sm[G_WARPS];
  const int warp = threadIdx.x >> 5, t = blockIdx.x * G_WARPS + warp;
  const Groups G(n_group, take, p.E, p.mode == MOE_GATING_SIGMOID_BIAS_RENORM);
  if (t < p.T && !gate_quick<NC>(p, G, t, nullptr, sm[warp]) && (threadIdx.x & 31) == 0)
    list[1 + atomicAdd(list, 1)] = t;
}
template <int NC>
__global__ void __launch_bounds__(G_WARPS * 32)
gate_group_rest_kernel(const __grid_constant__ GateParams p, int n_group, int take,
                       const int32_t* __restrict__ list) {
  pdl_trigger();
  pdl_wait();
  __shared__ GroupSmem sm;
  __shared__ Service sv;
  const Groups G(n_group, take, p.E, p.mode == MOE_GATING_SIGMOID_BIAS_RENORM);
  const int n = __ldcg(list);
#pragma unroll 1
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int t = __ldcg(list + 1 + i);
    if (threadIdx.x < 32) score_token<NC>(p, t, nullptr, sm);
    gate_slow_all<NC>(p, G, t, 1u, &sm, sv);
  }
}

// Everything after the router product for a batch of at most kSmallT tokens in one CTA, as
// route_tail_kernel: the slices of every logit summed in a fixed order, one warp a token gating,
// then the counts, scan, ranks and tables.
constexpr int kTailWarps = 32;
struct GroupTailSmem {
  TailSmem tail;                 // (lrow / exact_s unused)
  GroupSmem g[kSmallT];
  Service sv;
  unsigned slow;
  float sum[kTailWarps * 32];
  int wcnt[kMaxExperts / 32], wact[kMaxExperts / 32];
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
  // the logits: thread (g, li) sums slices g, g + G, ... of logit li (their loads in flight
  // together, neighbouring logits side by side), then the G sums in order
  const int G = max(1, NT / n);
  for (int i = tid; i < n * G; i += NT) {
    const int li = i % n, g = i / n;
    float a[4] = {0.f, 0.f, 0.f, 0.f};
    const float* q = p.part + li;
    int sp = g;
    for (; sp + 7 * G < S; sp += 8 * G) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __ldcg(q + (size_t)(sp + j * G) * stride);
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j & 3] += v[j];
    }
    for (int j = 0; sp < S; sp += G, ++j) a[j & 3] += __ldcg(q + (size_t)sp * stride);
    const float v = (a[0] + a[1]) + (a[2] + a[3]);
    if (G == 1) sm.tail.lg[li] = v;
    else sm.sum[i] = v;
  }
  if (G > 1) {
    __syncthreads();
    for (int li = tid; li < n; li += NT) {
      float v = 0.f;
      for (int g = 0; g < G; ++g) v += sm.sum[g * n + li];
      sm.tail.lg[li] = v;
    }
  }
  for (int e = tid; e < kMaxExperts; e += NT) sm.tail.hist[e] = 0;
  if (tid == 0) sm.slow = 0;
  __syncthreads();
  GateParams q = p;
  q.hist = sm.tail.hist;
  const Groups grp(n_group, take, E, p.mode == MOE_GATING_SIGMOID_BIAS_RENORM);
  if (warp < T && !gate_quick<EC>(q, grp, warp, sm.tail.lg + (size_t)warp * C, sm.g[warp]) &&
      (tid & 31) == 0)
    atomicOr(&sm.slow, 1u << warp);
  __syncthreads();
  gate_slow_all<EC>(q, grp, 0, sm.slow, sm.g, sm.sv);
  __syncthreads();
  // ---- counts, offsets, the experts with rows: a thread an expert, scans by warp and over the
  // eight warps
  const int lane = tid & 31, k = p.k;
  int cnt = 0, incl = 0;
  unsigned act = 0;
  if (warp < kMaxExperts / 32) {
    cnt = tid < E ? sm.tail.hist[tid] : 0;
    incl = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    act = __ballot_sync(0xffffffffu, cnt > 0);
    if (lane == 31) {
      sm.wcnt[warp] = incl;
      sm.wact[warp] = __popc(act);
    }
  }
  __syncthreads();
  if (warp < kMaxExperts / 32) {
    int before = 0, seen = 0;
    for (int w = 0; w < warp; ++w) {
      before += sm.wcnt[w];
      seen += sm.wact[w];
    }
    const int at = before + incl - cnt;
    seen += __popc(act & ((1u << lane) - 1u));
    sm.tail.excl[tid] = at;
    if (tid < E) {
      counts[tid] = cnt;
      offsets[tid] = at;
      if (cnt) active[seen] = tid;
      if (tid == E - 1) {
        offsets[E] = at + cnt;
        *n_active = seen + (cnt > 0);
      }
    }
  }
  if (tid < 4) shared_meta[tid] = tid == 1 ? T : tid == 3 ? 1 : 0;
  __syncthreads();
  // ---- stable ranks: pair i goes after every earlier pair of its expert
  if (tid < T * k) {
    const int t = tid / k, e = sm.g[t].ids[tid - t * k];
    int rank = 0;
    for (int i = 0; i < t; ++i)
      for (int j = 0; j < k; ++j) rank += sm.g[i].ids[j] == e;   // (a token's own are distinct)
    const int pp = sm.tail.excl[e] + rank;
    pos[tid] = pp;
    src[pp] = tid;
    sm.tail.srow[pp] = t;
  }
  if (!x_perm) return;
  __syncthreads();
  const int nvec = p.H / 8;
  for (int i = tid; i < T * k * nvec; i += NT) {
    const int r = i / nvec, v = i % nvec;
    reinterpret_cast<uint4*>(x_perm + (size_t)r * p.H)[v] =
        __ldg(reinterpret_cast<const uint4*>(p.x + (size_t)sm.tail.srow[r] * p.H) + v);
  }
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
  MOE_LAUNCH_NEXT(true, route_group_tail_kernel, dim3(1), dim3(kTailWarps * 32),
                  sizeof(GroupTailSmem), st, p, n_group, take, counts, offsets, pos, src, active,
                  n_active, shared_meta, x_perm);
  MOE_COUNT_LAUNCH();
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

template <int NC>
static int launch_gate_group_nc(const GateParams& p, int n_group, int take, int32_t* list,
                                cudaStream_t st) {
  const dim3 grid(ceil_div(p.T, G_WARPS)), block(G_WARPS * 32);
  if (!list || p.T < kListMinT || p.E <= kListMinE) {
    MOE_LAUNCH_NEXT(true, gate_group_kernel<NC>, grid, block, 0, st, p, n_group, take);
  } else {
    MOE_LAUNCH_NEXT(true, gate_group_list_kernel<NC>, grid, block, 0, st, p, n_group, take, list);
    MOE_COUNT_LAUNCH();
    MOE_LAUNCH_CHECK();
    MOE_LAUNCH_NEXT(true, gate_group_rest_kernel<NC>, dim3(2 * sm_count()), block, 0, st, p,
                    n_group, take, list);
  }
  MOE_COUNT_LAUNCH();
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

int launch_gate_group(const GateParams& p, int n_group, int take, int32_t* list, cudaStream_t st) {
  if (p.E <= 32) return launch_gate_group_nc<1>(p, n_group, take, list, st);
  if (p.E <= 64) return launch_gate_group_nc<2>(p, n_group, take, list, st);
  if (p.E <= 128) return launch_gate_group_nc<4>(p, n_group, take, list, st);
  return launch_gate_group_nc<EC>(p, n_group, take, list, st);
}

}  // namespace moe
