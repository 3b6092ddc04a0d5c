// moe_grouped_gemv_int4: products of few rows with 4-bit weights.
//
//   y[r][n] = sum_g s[e][n][g] * sum_{k in group g} (q[e][n][k] - z[e][n][g]) x[r][k]
//
// for the rows r of expert e; q a 4-bit code, s a bf16 scale and z a zero point of `G` codes along
// K.  A weight is read once and used for a few rows, so reading the codes bounds it.
//
// m16n8k16 products of bf16 values: 16 weight rows against eight token rows.  (tcgen05's smallest
// tile has 128 weight rows and wants its operand written to shared memory or TMEM first, which costs
// more than the few token rows' products.)  One group's products are added in fp32 before its scale
// is applied, in fp32, as moe_grouped_gemm_fp8 does.
//
// Codes to bf16.  Masked with 0x000F000F a code word is two bf16 of value q * 2^-133 (the bits of an
// integer below 256 read as a bf16 are that integer times 2^-133: subnormals and the first normal
// binade are one linear range), masked with 0x00F000F0 two of 16 q * 2^-133.  One bf16 fma,
// times 2^127 or 2^123 minus z 2^-6, gives (q - z) 2^-6 exactly; the sum is multiplied by 2^6 at the
// end.  Four pairs of a word take one shift, four masks and four fmas.
//
// The order of K inside a product is free as long as both operands agree.  A lane's codes for
// weight row n are the 8 of one 32-bit word, words of the four lanes of a row next to each other:
// 32 codes, which one group covers whatever its size.  Nibble pairs (i, i + 4) come out together,
// and the token row's eight values come from one 16-byte load.
//
// An item is 16, 32 or 48 weight rows of one expert against eight token rows, over the whole of K, so
// that no sum crosses CTAs; the height is the one whose rounds of items cost the least (launch_gemv).  A CTA's
// eight warps share an item's K, 256 codes at a time, and keep a step's token values in registers
// for all its weight rows.  Each warp has a ring of its own in shared memory, filled by TMA
// (boxes of the item's rows x 128 bytes, swizzled, so that the lanes' words lie in different
// banks) and running on from one item to the next; token values and scales are loaded ahead of their
// use.  The warps' sums are added in warp order in shared memory.
//
// Measured, groups of 128, in graphs of calls whose inputs change from call to call (the floor is what has
// to be read and written at the copy bandwidth): 14336 x 14336 codes, one token 22.6 us (floor 15.6; the
// same boxes loaded and not used 18.5), eight tokens 24.7; one row each on 8 experts of 4096 x 7168 30.9 us
// (17.9), two rows each on 256 of them, zero points, 762 us (581); 4096 x 7168, one token, 7.6 us, eight 8.6,
// of which launch, first loads and the last sums are about 6.  No pipe is full in the large ones: of about
// 280 instructions for 4096 codes 144 turn codes to bf16 and 20 are products and their loads, the issue slots
// are 60% busy with four warps a scheduler, the copy bandwidth 65 to 75%.  K that is no multiple of 256 takes
// scales one by one: 14304 x 14336, one token, 31.3 us.
// More than eight token rows are passes side by side, an expert's whole weights after one another in each: 64
// rows on 14336 x 14336 146 us.  16 rows a pass need registers that 16 warps a SM do not have, and a kernel
// for 64, codes turned once, won (1.1 to 1.6 times) only from 33 rows and 4096 weight rows on.
#include "common.cuh"
#include "route.cuh"
#include "tc_ptx.cuh"

#include <type_traits>

namespace moe {
namespace {

constexpr int kGvWarps = 8, kGvThreads = kGvWarps * 32;
constexpr int kGvUnit = 16;              // weight rows of a product
constexpr int kGvMaxTile = 3;            // units of an item at most (two boxes of four do not fit)
constexpr int kGvStep = 256;             // codes of K of a box (128 bytes a row)
constexpr int kGvWarpRing = 12288;       // bytes of a warp's ring: 6, 3 or 2 boxes
constexpr int kGvRing = kGvWarps * kGvWarpRing + 1024;
constexpr int kGvErrWait = 6;            // error word: a wait for weights ran out of time

struct GemvArgs {
  const uint16_t* x;
  const uint16_t* s;
  const uint8_t* z;
  const int32_t* offsets;
  int E, N, K, ng, max_rows;
  bool f32, wide;                              // wide: a step's scales of a row are one aligned load
  void* y;
  int32_t* err;
};

__device__ __forceinline__ void mma_bf16(float* d, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The four pairs of a code word as (q - z) 2^-6; nz: -z 2^-6 in both halves.
__device__ __forceinline__ void code_pairs(uint32_t w, uint32_t nz, uint32_t (&p)[4]) {
  const uint32_t h = w >> 8;
  const uint32_t v[4] = {w & 0x000F000Fu, w & 0x00F000F0u, h & 0x000F000Fu, h & 0x00F000F0u};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("fma.rn.bf16x2 %0, %1, %2, %3;"
        : "=r"(p[i])
        : "r"(v[i]), "r"(i & 1 ? 0x7D007D00u : 0x7F007F00u), "r"(nz));
}
// -z 2^-6 in both halves, z = byte I of `zeros`, 0..127: 128 + z by its bits, then an exact fma.
template <int I>
__device__ __forceinline__ uint32_t zero_pair(uint32_t zeros) {
  const uint32_t v = __byte_perm(zeros, 0x43434343u, 0x4040 | (I << 8) | I);
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(v), "r"(0xBC80BC80u), "r"(0x40004000u));
  return d;
}

struct GemvSmem {
  uint64_t full[kGvWarps][6];
  float red[kGvWarps][4][kGvMaxTile * kGvUnit + 4];   // the warps' sums of four token rows
  int lo[kMaxExperts], hi[kMaxExperts];        // token rows of the experts that have some
  int passes[kMaxExperts + 1];                 // eights of token rows of the experts before
  int16_t act[kMaxExperts];
  int wsum[2][kGvWarps];
};

// The experts with rows, ascending, with their ranges; returns how many there are.  CTA 0 records in
// the error word whether a range was clipped.
__device__ int active_experts(const GemvArgs& a, GemvSmem& sm) {
  const int e = threadIdx.x, lane = e & 31, warp = e >> 5;
  int b = 0, n = 0;
  bool clipped = false;
  if (e < a.E) {
    b = __ldg(a.offsets + e);
    const int end = __ldg(a.offsets + e + 1);
    const int cb = min(max(b, 0), a.max_rows), ce = min(max(end, 0), a.max_rows);
    clipped = end > b && (cb != b || ce != end);
    b = cb;
    n = max(ce - cb, 0);
  }
  const int mine = (n + 7) / 8;
  int before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  const unsigned m = __ballot_sync(0xffffffffu, n > 0);
  if (lane == 31) {
    sm.wsum[0][warp] = __popc(m);
    sm.wsum[1][warp] = before;
  }
  before -= mine;
  const int any = __syncthreads_or(clipped);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = any ? 8 : 0;
  int at = __popc(m & ((1u << lane) - 1u)), total = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kGvWarps; ++i) {
    at += i < warp ? sm.wsum[0][i] : 0;
    before += i < warp ? sm.wsum[1][i] : 0;
    total += sm.wsum[0][i];
    all += sm.wsum[1][i];
  }
  if (n > 0) {
    sm.act[at] = (int16_t)e;
    sm.lo[at] = b;
    sm.hi[at] = b + n;
    sm.passes[at] = before;
  }
  if (threadIdx.x == 0) sm.passes[total] = all;
  __syncthreads();
  return total;
}

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2,
                                       uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}


// The words of four 8 x 16-byte blocks: a lane gets word t of row gr of each.
__device__ __forceinline__ void load_words(uint32_t (&w)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(addr)
               : "memory");
}
// A token row's eight values in the order of a word's pairs: (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ uint4 pair_order(const uint4& v) {
  return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                    __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
}

// An item: weight rows from n0 on of expert e against token rows [rb, hi) (at most eight).
struct GemvItem {
  int e, n0, rb, hi;
};
template <int NT>
__device__ __forceinline__ GemvItem gemv_item(const GemvArgs& a, const GemvSmem& sm, int it, int ntile,
                                              int n_act) {
  const int pass = it / ntile, n0 = (it - pass * ntile) * (NT * kGvUnit);
  if (!a.offsets) return {0, n0, 8 * pass, min(a.max_rows, 8 * pass + 8)};
  int i = 0, end = n_act;                      // the last expert whose passes start at or before it
  while (end - i > 1) {
    const int c = (i + end) >> 1;
    if (sm.passes[c] <= pass) i = c;
    else end = c;
  }
  const int rb = sm.lo[i] + 8 * (pass - sm.passes[i]);
  return {sm.act[i], n0, rb, min(sm.hi[i], rb + 8)};
}

// G: codes a scale covers; NT: units of an item.
template <int G, bool ZERO, int NT>
__global__ void __launch_bounds__(kGvThreads, 2)
gemv_int4_kernel(const GemvArgs a, const __grid_constant__ CUtensorMap tm) {
  constexpr int NG = kGvStep / G;              // groups of a step: 2, 4, 8
  constexpr int CG = G / 32;                   // 32-code chunks of a group
  constexpr int kBox = NT * kGvUnit * kGvStep / 2, kBoxes = kGvWarpRing / kBox;
  static_assert(kMaxExperts <= kGvThreads, "one thread per expert");
  extern __shared__ uint8_t ring_raw[];
  __shared__ GemvSmem sm;
  const int lane = threadIdx.x & 31, gr = lane >> 2, t = lane & 3;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);   // (the same for every lane)
  uint64_t* full = sm.full[warp];
  // (the swizzle goes by address bits: the ring starts on a 1024-byte boundary)
  const uint32_t ring = ((smem_u32(ring_raw) + 1023u) & ~1023u) + warp * kGvWarpRing;
  pdl_trigger();
  if (lane == 0) {
    for (int i = 0; i < kBoxes; ++i) mbar_init(full + i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    prefetch_map(&tm);
  }
  pdl_wait();
  int n_act = 1, passes = (a.max_rows + 7) / 8;
  if (a.offsets) {
    n_act = __shfl_sync(0xffffffffu, active_experts(a, sm), 0);
    passes = sm.passes[n_act];
  } else {
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;
    __syncwarp();
  }
  const int ntile = (a.N + NT * kGvUnit - 1) / (NT * kGvUnit);
  const int steps = (a.K + kGvStep - 1) / kGvStep;
  const int items = passes * ntile;
  // A warp's steps of an item are first, first + 8, ...: dealt out from where the last item's ended.
  auto following = [&](int first) { return (first + kGvWarps - steps % kGvWarps) % kGvWarps; };

  // the next box to ask for
  int a_it = blockIdx.x;
  int a_first = warp, a_st = warp, put = 0, place = 0;
  GemvItem ai{0, 0, 0, 0};
  if (a_it < items) ai = gemv_item<NT>(a, sm, a_it, ntile, n_act);
  auto ask = [&] {
    while (a_st >= steps) {
      a_it += gridDim.x;
      if (a_it >= items) break;
      ai = gemv_item<NT>(a, sm, a_it, ntile, n_act);
      a_st = a_first = following(a_first);
    }
    if (a_it >= items) return;
    if (lane == 0) {
      mbar_expect_tx(full + place, kBox);
      tma_3d(ring + place * kBox, &tm, a_st * (kGvStep / 2), ai.n0, ai.e, full + place);
    }
    ++put;
    place = place + 1 == kBoxes ? 0 : place + 1;
    a_st += kGvWarps;
  };
  int got = 0, dead = -1;                      // boxes used; the first that did not come in time
  int slot = 0;
  uint32_t phase = 0;

  // Where the values of a step come from.  Token values: lane (gr, t) those of row gr that its words'
  // codes meet; rows past the item's last read that one (their sums are not stored), and what lies
  // past the end of K is set to zero when it is used.  A step's scales of the weight rows gr and gr + 8 of
  // a unit: lanes t = 0 and 1, two in a register; their zero points: lanes t = 2 and 3, four in a
  // register.  Rows past the end read the last one (they are not stored); the scales of groups past the
  // end are zero, so that an infinite last scale meets no product that is zero there.
  struct Source {
    const uint16_t* x;
    size_t s;
    int row, st;                               // the last weight row, counted from the item's first
  };
  auto source = [&](const GemvItem& i, int st) {
    return Source{a.x + (size_t)min(i.rb + gr, i.hi - 1) * a.K, ((size_t)i.e * a.N + i.n0) * a.ng,
                  a.N - 1 - i.n0, st};
  };
  uint4 xv[8];
  auto token_values = [&](const Source& f) {
    const int k = f.st * kGvStep + 8 * t;
    if ((f.st + 1) * kGvStep <= a.K) {
#pragma unroll
      for (int c = 0; c < 8; ++c) xv[c] = __ldg(reinterpret_cast<const uint4*>(f.x + k) + 4 * c);
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        xv[c] = __ldg(reinterpret_cast<const uint4*>(f.x + min(k + 32 * c, a.K - 8)));
    }
  };
  uint32_t rvs[NT][NG / 2];
  auto scale_values = [&](const Source& f, int i) {
    uint32_t(&rv)[NG / 2] = rvs[i];
    const size_t at = f.s + (size_t)((uint32_t)min(16 * i + gr + 8 * (t & 1), f.row) * a.ng);
    const int g0 = f.st * NG;
    if (a.wide) {
      const uint16_t* s = a.s + at + g0;
      const uint8_t* z = a.z + at + g0;
      if (t < 2) {
        if (NG == 2) {
          rv[0] = __ldg(reinterpret_cast<const uint32_t*>(s));
        } else if (NG == 4) {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(s));
          rv[0] = v.x;
          rv[1 % (NG / 2)] = v.y;
        } else {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(s));
          rv[0] = v.x;
          rv[1 % (NG / 2)] = v.y;
          rv[2 % (NG / 2)] = v.z;
          rv[3 % (NG / 2)] = v.w;
        }
      } else if (ZERO) {
        if (NG == 2) {
          rv[0] = __ldg(reinterpret_cast<const uint16_t*>(z));
        } else if (NG == 4) {
          rv[0] = __ldg(reinterpret_cast<const uint32_t*>(z));
        } else {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(z));
          rv[0] = v.x;
          rv[1 % (NG / 2)] = v.y;
        }
      }
    } else if (t < 2) {
#pragma unroll
      for (int j = 0; j < NG / 2; ++j) {
        const int g = g0 + 2 * j;
        const uint32_t lo = g < a.ng ? __ldg(a.s + at + g) : 0u;
        rv[j] = lo | (g + 1 < a.ng ? (uint32_t)__ldg(a.s + at + g + 1) << 16 : 0u);
      }
    } else if (ZERO) {
#pragma unroll
      for (int j = 0; j < (NG + 3) / 4; ++j) {
        uint32_t v = 0u;
#pragma unroll
        for (int b = 0; b < 4; ++b) v |= (uint32_t)__ldg(a.z + at + min(g0 + 4 * j + b, a.ng - 1)) << (8 * b);
        rv[j] = v;
      }
    }
  };
  // where the lane points ldmatrix: chunks 2 c, 2 c + 1 of weight rows 0..7 and 8..15
  uint32_t wa[4];
#pragma unroll
  for (int c = 0; c < 4; ++c)
    wa[c] = ring + (lane & 15) * 128 + (((2 * c + (lane >> 4)) ^ (lane & 7)) << 4);

  int first = warp;
  GemvItem next = ai;
  // The first item's first values ahead of the first boxes (one token on 4096 x 7168 8.8 -> 8.5 us), but
  // where that costs more registers than there are.
  constexpr bool kEarly = NT < 3 || !ZERO;
  bool loaded = kEarly && blockIdx.x < items && first < steps;   // are the item's first values under way?
  if (loaded) {
    const Source src = source(next, first);
#pragma unroll
    for (int i = 0; i < NT; ++i) scale_values(src, i);
    token_values(src);
  }
  for (int i = 0; i < kBoxes; ++i) ask();
  for (int it = blockIdx.x; it < items; it += gridDim.x) {
    const GemvItem cur = next;
    if (it + gridDim.x < items) next = gemv_item<NT>(a, sm, it + gridDim.x, ntile, n_act);
    Source src = source(cur, first);
    if (!loaded && first < steps) {
      token_values(src);
#pragma unroll
      for (int i = 0; i < NT; ++i) scale_values(src, i);
    }
    first = following(first);
    loaded = false;
    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[i][c] = 0.f;
    while (src.st < steps) {
      // the step whose values come next: this item's, or the next item's first
      Source nx = src;
      nx.st += kGvWarps;
      const bool last = nx.st >= steps;
      if (last) {
        if (it + gridDim.x < items && first < steps) {
          nx = source(next, first);
          loaded = true;
        } else {
          nx.st = src.st;                      // (none: values that no one uses)
        }
      }
#pragma unroll
      for (int c = 0; c < 8; ++c)
        xv[c] = pair_order(xv[c]);
      if ((src.st + 1) * kGvStep > a.K) {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (src.st * kGvStep + 8 * t + 32 * c >= a.K) xv[c] = make_uint4(0u, 0u, 0u, 0u);
      }
      if (dead < 0 && !warp_wait(full + slot, phase, a.err, kGvErrWait)) dead = got;
      const uint32_t box = slot * kBox;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        uint32_t sz[NG / 2];
#pragma unroll
        for (int j = 0; j < NG / 2; ++j) sz[j] = rvs[i][j];
        scale_values(nx, i);
        uint32_t f0 = 0u, f1 = 0u, zb0 = 0u, zb1 = 0u, w[4];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          if (g % 2 == 0) {
            f0 = __shfl_sync(0xffffffffu, sz[g / 2], lane & 28);
            f1 = __shfl_sync(0xffffffffu, sz[g / 2], (lane & 28) | 1);
          }
          if (ZERO && g % 4 == 0) {
            zb0 = __shfl_sync(0xffffffffu, sz[g / 4], (lane & 28) | 2);
            zb1 = __shfl_sync(0xffffffffu, sz[g / 4], (lane & 28) | 3);
          }
          uint32_t z0 = 0xBE00BE00u, z1 = 0xBE00BE00u;   // -8 * 2^-6
          if (ZERO) {
            z0 = g % 4 == 0 ? zero_pair<0>(zb0) : g % 4 == 1 ? zero_pair<1>(zb0)
               : g % 4 == 2 ? zero_pair<2>(zb0) : zero_pair<3>(zb0);
            z1 = g % 4 == 0 ? zero_pair<0>(zb1) : g % 4 == 1 ? zero_pair<1>(zb1)
               : g % 4 == 2 ? zero_pair<2>(zb1) : zero_pair<3>(zb1);
          }
          float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < CG; ++c) {
            const int ch = g * CG + c;
            if ((ch & 1) == 0) load_words(w, box + i * (kGvUnit * 128) + wa[ch / 2]);
            uint32_t p[4], q[4];
            code_pairs(w[2 * (ch & 1)], z0, p);
            code_pairs(w[2 * (ch & 1) + 1], z1, q);
            mma_bf16(d, p[0], q[0], p[1], q[1], xv[ch].x, xv[ch].y);
            mma_bf16(d, p[2], q[2], p[3], q[3], xv[ch].z, xv[ch].w);
          }
          const float s0 = __uint_as_float(g % 2 ? f0 & 0xFFFF0000u : f0 << 16);
          const float s1 = __uint_as_float(g % 2 ? f1 & 0xFFFF0000u : f1 << 16);
          acc[i][0] = fmaf(s0, d[0], acc[i][0]);
          acc[i][1] = fmaf(s0, d[1], acc[i][1]);
          acc[i][2] = fmaf(s1, d[2], acc[i][2]);
          acc[i][3] = fmaf(s1, d[3], acc[i][3]);
        }
      }
      token_values(nx);
      ++got;
      if (++slot == kBoxes) {
        slot = 0;
        phase ^= 1;
      }
      __syncwarp();                            // the box is read: its place is free
      if (dead < 0) ask();
      if (last) break;
      src = nx;
    }
    // the warps' sums, four token rows at a time
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int rows = cur.hi - cur.rb - 4 * h;
      if (rows <= 0) break;
      if ((t >> 1) == h) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            sm.red[warp][2 * (t & 1) + (c & 1)][16 * i + gr + 8 * (c >> 1)] = acc[i][c];
      }
      __syncthreads();
      const int n = threadIdx.x & 63, r = threadIdx.x >> 6;
      if (r < rows && n < NT * kGvUnit && cur.n0 + n < a.N) {
        float v = sm.red[0][r][n];
#pragma unroll
        for (int q = 1; q < kGvWarps; ++q) v += sm.red[q][r][n];
        const size_t at = (size_t)(cur.rb + 4 * h + r) * a.N + cur.n0 + n;
        v *= 0x1p6f;
        if (a.f32) static_cast<float*>(a.y)[at] = v;
        else static_cast<uint16_t*>(a.y)[at] = float_to_bf16_bits(v);
      }
      __syncthreads();
    }
  }
  // after a wait that ran out: what was asked for has to have landed before the memory goes
  if (dead >= 0)
    for (int i = dead; i < put; ++i)
      warp_wait(full + i % kBoxes, (i / kBoxes) & 1, a.err, kGvErrWait);
}

// (an item's rows are counted in eights, in 32 bits: the last eight of max_rows ends below 2^31)
bool valid_gemv_shape(int E, int N, int K, int max_rows) {
  return E > 0 && E <= kMaxExperts && N > 0 && K > 0 && K % 32 == 0 && max_rows >= 0 &&
         max_rows <= 0x7fffffff - 8 &&
         N <= (1 << 24) && K <= (1 << 24) && (long long)E * N < (1LL << 31);
}

bool encode_weights(CUtensorMap* m, const uint8_t* w, int E, int N, int K, int rows) {
  const cuuint64_t row = (cuuint64_t)K / 2;
  const cuuint64_t dims[3] = {row, (cuuint64_t)N, (cuuint64_t)E};
  const cuuint64_t strides[2] = {row, row * N};
  const cuuint32_t box[3] = {kGvStep / 2, (cuuint32_t)rows, 1}, step[3] = {1, 1, 1};
  auto enc = encode_fn();
  return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(w), dims, strides, box,
                    step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int G, bool ZERO, int NT>
int launch_gemv(const GemvArgs& a, int items, const CUtensorMap& tm, cudaStream_t st) {
  auto kernel = gemv_int4_kernel<G, ZERO, NT>;
  MOE_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kGvRing));
  MOE_LAUNCH_NEXT(true, kernel, dim3(std::min(items, 2 * sm_count())),
                 dim3(kGvThreads), kGvRing, st, a, tm);
  MOE_COUNT_LAUNCH();
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

template <int G, bool ZERO>
int launch_gemv(const GemvArgs& a, const uint8_t* w, cudaStream_t st) {
  // passes at most (an expert's last eight has one row at least), and as many as there will be when the
  // experts' last eights are half full
  const long long most = (a.max_rows + 7LL * std::min(a.E, a.max_rows)) / 8;
  const long long passes = std::min<long long>(most, (a.E + 1) / 2 + a.max_rows / 8);
  // the height whose rounds cost the least: its rows, and what a step costs beside them (about one unit:
  // 602, 680 and 952 us with 48, 32 and 16 rows for 64 tokens on 256 experts of 4096 x 7168); ties to
  // the higher
  long long best = 0;
  int nt = 0, items = 0;
  for (int n = 1; n <= kGvMaxTile; ++n) {
    const long long tiles = ceil_div(a.N, n * kGvUnit), slots = 2LL * sm_count();
    const long long cost = (std::max(1LL, passes) * tiles + slots - 1) / slots * (n + 1);
    if (most * tiles > 0x3fffffff) return MOE_ERR_INVALID_ARG;   // (items are counted in 32 bits)
    if (!nt || cost <= best) {
      nt = n;
      best = cost;
      items = (int)(most * tiles);
    }
  }
  CUtensorMap tm;
  if (!encode_weights(&tm, w, a.E, a.N, a.K, nt * kGvUnit)) return MOE_ERR_UNSUPPORTED;
  if (nt == 1) return launch_gemv<G, ZERO, 1>(a, items, tm, st);
  if (nt == 2) return launch_gemv<G, ZERO, 2>(a, items, tm, st);
  return launch_gemv<G, ZERO, 3>(a, items, tm, st);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_grouped_gemv_int4_workspace_size(int max_rows, int E, int N, int K) {
  return valid_gemv_shape(E, N, K, max_rows) ? 256 : 0;
}

int moe_grouped_gemv_int4(const uint16_t* x, const uint8_t* w, const uint16_t* w_scale,
                          const uint8_t* w_zero, const int32_t* offsets, int E, int N, int K,
                          int group, int max_rows, int out_f32, void* y, void* ws,
                          size_t ws_bytes, void* stream) {
  MOE_REQUIRE(valid_gemv_shape(E, N, K, max_rows) && (offsets || E == 1) &&
              (out_f32 == 0 || out_f32 == 1));
  MOE_REQUIRE(group == 32 || group == 64 || group == 128);
  if (max_rows == 0) return MOE_OK;
  MOE_REQUIRE(x && w && w_scale && y && ws);
  MOE_REQUIRE(aligned16(x) && aligned16(w) && aligned2(w_scale) && aligned16(y) &&
              aligned4(offsets) && aligned256(ws));
  MOE_REQUIRE(ws_bytes >= moe_grouped_gemv_int4_workspace_size(max_rows, E, N, K));
  const GemvArgs a{x, w_scale, w_zero, offsets, E, N, K, ceil_div(K, group), max_rows,
                   out_f32 != 0, K % kGvStep == 0 && aligned16(w_scale) && aligned16(w_zero), y,
                   static_cast<int32_t*>(ws)};
  cudaStream_t st = (cudaStream_t)stream;
  if (group == 32) return w_zero ? launch_gemv<32, true>(a, w, st) : launch_gemv<32, false>(a, w, st);
  if (group == 64) return w_zero ? launch_gemv<64, true>(a, w, st) : launch_gemv<64, false>(a, w, st);
  return w_zero ? launch_gemv<128, true>(a, w, st) : launch_gemv<128, false>(a, w, st);
}

}  // extern "C"
