// moe_sort_tokens: the dispatch of token slots to experts for ids that come from elsewhere.
//
//   counts[e] = #{slots s : ids[s] = e},  offsets = exclusive scan of counts,
//   pos[s] = offsets[ids[s]] + #{s' < s : ids[s'] = ids[s]},  src[pos[s]] = s
//
// a stable counting sort of n = T k slots by expert.  A slot whose id lies outside [0, E) has no
// row: its pos is -1, and the entries of src that no slot takes (the last ones) are -1.
//
// A CTA takes a contiguous chunk of slots, each of its 32 warps a contiguous part of the chunk.
// The slots of an expert before a warp's are those of earlier chunks (from the chunks' histograms,
// which a first kernel leaves in the workspace), of earlier warps (a scan over the warps'
// histograms in shared memory) and of the warp itself (__match_any_sync, 32 slots at a time).  No
// result depends on the order of atomics: they only count.
// It needs 12 bytes a slot (id in, pos and src out), so a call is bound by its launches and the
// chain of steps within them: in graphs of calls one token 2 us, 1024 tokens of 8 slots on 256 experts 7,
// 32768 tokens 9.7 us (3 MB).  One launch with a barrier across the CTAs instead of the two took 0.7 us more.
#include "common.cuh"
#include "route.cuh"

namespace moe {
namespace {

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kSortParts = kSortThreads / kMaxExperts;   // threads an expert
// One chunk up to this many slots, else chunks of kSortChunk at least (8192 slots: one CTA 11.4 us, four
// 7.3), and at most kSortMaxChunks, whose histograms every CTA reads (262144 slots: 128 chunks 12.0 us,
// 64 9.5, 48 10.9).
constexpr int kSortOne = 2560, kSortChunk = 2048;
constexpr int kSortMaxChunks = 64;

struct SortPlan {
  int chunk, chunks;
};
SortPlan plan_sort(long long n) {
  SortPlan p;
  p.chunk = n <= kSortOne ? kSortOne
                          : (int)std::max<long long>(kSortChunk, (n + kSortMaxChunks - 1) / kSortMaxChunks);
  p.chunks = (int)((n + p.chunk - 1) / p.chunk);
  return p;
}

__global__ void __launch_bounds__(kSortThreads)
sort_histogram_kernel(const int32_t* __restrict__ ids, int n, int E, int chunk,
                      int32_t* __restrict__ hist) {
  __shared__ int s[kMaxExperts];
  if (threadIdx.x < kMaxExperts) s[threadIdx.x] = 0;
  __syncthreads();
  pdl_wait();
  pdl_trigger();   // (after the wait: the ranking kernel may read ids once it runs)
  const int lo = blockIdx.x * chunk, hi = min(n - lo, chunk);
  for (int i = threadIdx.x; i < hi; i += kSortThreads) {
    const int e = __ldg(ids + lo + i);
    if ((unsigned)e < (unsigned)E) atomicAdd(&s[e], 1);
  }
  __syncthreads();
  if (threadIdx.x < E) hist[(size_t)blockIdx.x * E + threadIdx.x] = s[threadIdx.x];
}

struct SortSmem {
  int base[kSortWarps][kMaxExperts];     // a warp's slots of e, then its next row of e in ...
  int before[kSortParts][kMaxExperts];   // slots of e in earlier chunks, by parts; then the row where ...
                                         // ... those of eight warps start
  int total[kSortParts][kMaxExperts], own[kSortParts][kMaxExperts];
  int scan[kMaxExperts / 32];
  int rows;
};
static_assert(sizeof(SortSmem) <= 48 * 1024, "static shared memory");

// hist: [gridDim.x][E] chunk histograms; chained: launched behind sort_histogram_kernel, else one chunk
// holds every slot.
__global__ void __launch_bounds__(kSortThreads)
sort_rank_kernel(const int32_t* __restrict__ ids, int n, int E, int chunk,
                 const int32_t* __restrict__ hist, int32_t* __restrict__ counts,
                 int32_t* __restrict__ offsets, int32_t* __restrict__ pos,
                 int32_t* __restrict__ src, bool chained) {
  constexpr int kParts = kSortParts, kPer = kSortWarps / kParts;
  __shared__ SortSmem sm;
  auto& base = sm.base;
  auto& before = sm.before;
  auto& total = sm.total;
  auto& own = sm.own;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();
  for (int i = tid; i < kSortWarps * kMaxExperts; i += kSortThreads) (&base[0][0])[i] = 0;
  __syncthreads();
  if (!chained) pdl_wait();
  const int lo = blockIdx.x * chunk, hi = min(n - lo, chunk);
  const int per = ((chunk + kSortWarps - 1) / kSortWarps + 31) & ~31;
  const int w0 = min(warp * per, hi), w1 = min(w0 + per, hi);
  for (int i = w0 + lane; i < w1; i += 32) {
    const int e = __ldg(ids + lo + i);
    if ((unsigned)e < (unsigned)E) atomicAdd(&base[warp][e], 1);
  }
  if (chained) pdl_wait();
  // slots of each expert in the chunks before this one and in all of them
  const int e = tid & (kMaxExperts - 1), part = tid / kMaxExperts;
  int b = 0, all = 0;
  if (chained && e < E) {
#pragma unroll
    for (int i = 0; i < kSortMaxChunks / kParts; ++i) {   // (all loads in flight together)
      const int c = part + kParts * i;
      const int h = c < gridDim.x ? hist[(size_t)c * E + e] : 0;
      all += h;
      b += c < blockIdx.x ? h : 0;
    }
  }
  before[part][e] = b;
  total[part][e] = all;
  __syncthreads();
  int run = 0;
#pragma unroll
  for (int w = part * kPer; w < (part + 1) * kPer; ++w) {
    const int h = base[w][e];
    base[w][e] = run;
    run += h;
  }
  own[part][e] = run;
  __syncthreads();
  int mine = 0, inc = 0;
  if (tid < kMaxExperts) {
#pragma unroll
    for (int p = 0; p < kParts; ++p) mine += chained ? total[p][e] : own[p][e];
    inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) sm.scan[warp] = inc;
  }
  __syncthreads();
  if (tid < kMaxExperts) {
    int off = inc - mine;
#pragma unroll
    for (int w = 0; w < kMaxExperts / 32; ++w) off += w < warp ? sm.scan[w] : 0;
    if (tid == kMaxExperts - 1) sm.rows = off + mine;
    if (blockIdx.x == 0 && e < E) {
      counts[e] = mine;
      offsets[e] = off;
      if (e == E - 1) offsets[E] = off + mine;
    }
#pragma unroll
    for (int p = 0; p < kParts; ++p) off += before[p][e];
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      before[p][e] = off;                  // (this thread's alone until the barrier)
      off += own[p][e];
    }
  }
  __syncthreads();
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const int id = i < w1 ? __ldg(ids + lo + i) : -1;
    const bool has = (unsigned)id < (unsigned)E;
    const unsigned same = __match_any_sync(0xffffffffu, has ? id : -1);
    const int rank = __popc(same & ((1u << lane) - 1u));
    int first = 0;
    if (has) first = base[warp][id];
    __syncwarp();
    if (has && rank == 0) base[warp][id] = first + __popc(same);
    __syncwarp();
    if (i < w1) {
      const int p = has ? before[warp / kPer][id] + first + rank : -1;
      pos[lo + i] = p;
      if (has) src[p] = lo + i;
    }
  }
  for (long long i = (long long)sm.rows + blockIdx.x * kSortThreads + tid; i < n;
       i += (long long)gridDim.x * kSortThreads)
    src[i] = -1;
}

bool valid_sort_shape(int T, int E, int k) {
  return T >= 0 && E >= 1 && E <= kMaxExperts && k >= 1 && k <= kMaxK &&
         (long long)T * k <= 0x7fffffffLL;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_sort_tokens_workspace_size(int T, int E, int k) {
  if (!valid_sort_shape(T, E, k)) return 0;
  const SortPlan p = plan_sort((long long)T * k);
  return round_up((size_t)std::max(1, p.chunks) * E * sizeof(int32_t), 256);
}

int moe_sort_tokens(const int32_t* ids, int T, int E, int k, int32_t* counts, int32_t* offsets,
                    int32_t* pos, int32_t* src, void* ws, size_t ws_bytes, void* stream) {
  MOE_REQUIRE(valid_sort_shape(T, E, k));
  MOE_REQUIRE(counts && offsets && aligned4(counts) && aligned4(offsets));
  cudaStream_t st = (cudaStream_t)stream;
  const int n = T * k;
  const SortPlan p = plan_sort(n);
  if (n > 0) {
    MOE_REQUIRE(ids && pos && src && aligned4(ids) && aligned4(pos) && aligned4(src));
    MOE_REQUIRE(ws && aligned4(ws) && ws_bytes >= moe_sort_tokens_workspace_size(T, E, k));
  }
  int32_t* hist = static_cast<int32_t*>(ws);
  if (p.chunks > 1) {
    MOE_LAUNCH_NEXT(true, sort_histogram_kernel, dim3(p.chunks), dim3(kSortThreads), 0, st, ids, n, E,
                   p.chunk, hist);
    MOE_COUNT_LAUNCH();
    MOE_LAUNCH_CHECK();
  }
  MOE_LAUNCH_NEXT(true, sort_rank_kernel, dim3(std::max(1, p.chunks)), dim3(kSortThreads),
                  0, st, ids, n, E, p.chunk, hist, counts, offsets, pos, src, p.chunks > 1);
  MOE_COUNT_LAUNCH();
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // extern "C"
