// Routing kernels' host interface (internal to libmoe).
#pragma once
#include "common.cuh"
#include <algorithm>

namespace moe {

constexpr int kMaxExperts = 256;  // E limit (expert slots per warp lane: 8)
constexpr int kMaxK = 8;          // top-k limit
constexpr int kTileT = 128;       // tokens per dispatch tile (histogram granularity)

struct GateParams {
  const float* part;         // router outputs: S slices [S][T][ldp], C columns used per row
  int S, C, ldp;
  const uint16_t* x;
  const float* w_r;
  const float* w_rT;         // [E][H] transposed router (tensor-core router path) or NULL
  const float* logit_bias;
  const float* sel_bias;
  const int32_t* forced;
  int T, H, E, k, mode;
  float scale;
  int32_t* ids;
  float* w;
  float* logits;
  float* shared_gate;
  int32_t* tie_flags;
  int32_t* hist;
  int tok_per_warp;          // warp-per-token gating: tokens per warp
  int32_t* ids_local;        // or NULL: the chosen ids are also stored here (shared memory)
};

struct RoutePlan {
  int C;            // logit columns (E, + 1 for the shared-expert gate)
  int S;            // H slices of the router product
  int h_per_split;
  int ntiles;       // 128-token dispatch tiles
  int tc;           // 1: router product on the tensor cores (bf16 x 3 pieces), S = 1
  int Mpad;         // rows of the tensor-core router image (C rounded up to 128)
  int tc_S;         // K splits of the tensor-core router product
  int own_tc;       // 1: the router product is route_tc.cu's, in tc_S >= 1 parts
  int small;        // 1: gating, scan, ranks and row copy in one CTA (T <= kSmallT)
};

// batches of at least this many tokens compute the router product on the tensor cores
constexpr int kTcRouterMinT = 256;
// ... and group-limited ones of at least this many by route_tc.cu's kernel (the whole routing of
// 7168 x 256 experts: 512 tokens 56 us instead of 65, 1024 71 / 82, 2048 80 / 93, 8192 140 / 180).
// It is the faster one for 256 tokens too (56 / 64), but there the logits stay moe_route_topk's to
// the bit.
constexpr int kOwnTcMinT = 512;
// batches of at most this many tokens run everything after the router product in one CTA
constexpr int kSmallT = 16;
// batches of at least this many tokens gather x_perm in a separate, GPU-wide kernel
constexpr int kSeparateGatherMinT = 1024;
// ... and so do batches whose permuted rows exceed this many bytes (one CTA per 128-token tile
// would copy them)
constexpr size_t kFusedGatherMaxBytes = size_t(512) << 10;

struct RouteScratch {
  float* part;      // [S][T][C] (own_tc: none)
  int32_t* hist;    // [ntiles][E] (own_tc: followed by the count and list of tokens to re-score)
  int32_t* base;    // [ntiles][E]
  int32_t* active;  // [E] experts with rows, ascending
  int32_t* n_active;
  int32_t* shared_meta;  // {0, T, 0, 1}: offsets / active list / count of the shared expert
  uint16_t* img;         // tensor-core router: [Mpad x 3H] tiled bf16 pieces
  float* w_rT;           // tensor-core router: [E][H] fp32
  float* tc_part;        // tensor-core router, tc_S > 1 or own_tc: [tc_S][T][Mpad] fp32 partials
};

struct RouteArgs {
  const uint16_t* x;
  const float* w_r;
  const float* logit_bias;
  const float* sel_bias;
  const uint16_t* w_gate;
  const int32_t* forced;
  int T, H, E, k, gating;
  float scale;
  int32_t *ids, *counts, *offsets, *pos, *src, *tie_flags;
  float *w, *logits, *shared_gate;
  uint16_t* x_perm;  // nullable: fused gather into expert order
  int32_t* err;      // device error word (bounded waits of the tensor-core router)
  int n_group, take; // group-limited selection: `take` of n_group groups; 0 = no groups
  int clear_err;     // group-limited: the first kernel clears *err
};

// launch_pdl, with programmatic stream serialization whatever MOE_OPT_PDL says when `chained`: for
// a kernel whose predecessor on the stream is one of the library's that the same call launched
// (group-limited routing's five launches, 60 experts and 333 tokens: 37 us plain, 31 chained).
template <typename... KArgs, typename... Args>
cudaError_t launch_next(bool chained, void (*kernel)(KArgs...), dim3 grid, dim3 block,
                        size_t smem, cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = chained || g_use_pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}
#define MOE_LAUNCH_NEXT(chained, kernel, grid, block, smem, st, ...) \
  MOE_CUDA_TRY(::moe::launch_next(chained, kernel, grid, block, smem, st, __VA_ARGS__))

RoutePlan plan_route(int T, int H, int E, int k, bool has_gate, bool grouped = false);
// moe_route_workspace_size without what group-limited routing needs beyond the rest
size_t route_workspace_ungrouped(int T, int H, int E, int k);
// The router product of a large group-limited batch (csrc/route_tc.cu): part [S][T][Mpad].
int route_tc_parts(int T, int H, int Mpad);
int launch_route_tc(const uint16_t* x, int T, int H, const uint16_t* img, int Mpad, int S,
                    float* part, int32_t* err, cudaStream_t st);
size_t route_scratch(WsCursor& c, const RoutePlan& r, int T, int E, RouteScratch* out);
int launch_route(const RouteArgs& a, const RoutePlan& r, const RouteScratch& s,
                 cudaStream_t st);
// Group-limited gating of p.T tokens (csrc/route_group.cu).
constexpr int kMaxGroups = 32;
// list: [1 + T], its first element zero; or NULL: tokens that need re-scoring are finished by the
// CTA that met them.
int launch_gate_group(const GateParams& p, int n_group, int take, int32_t* list, cudaStream_t st);
int launch_route_group_tail(const GateParams& p, int n_group, int take, int32_t* counts,
                            int32_t* offsets, int32_t* pos, int32_t* src, int32_t* active,
                            int32_t* n_active, int32_t* shared_meta, uint16_t* x_perm,
                            cudaStream_t st);
int launch_gather(const uint16_t* x, const int32_t* src, int rows, int k, int H,
                  uint16_t* x_perm, cudaStream_t st);

}  // namespace moe
