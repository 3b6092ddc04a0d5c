// moe_grouped_gemv_int4 for more than eight token rows an expert: the mathematics of gemv_int4.cu, the
// codes of a chunk turned to bf16 once for up to 64 token rows.
//
// The products bound it here: m16n8k16 runs at one in two clocks a SM (1024 multiply-adds a clock),
// so 64 rows cannot take less than 45 us on 14336 x 14336 weights that are read in 16.  What
// matters is that nothing else takes longer:
//  - A first kernel lays the token rows out in the order in which the products' lanes want them, eight
//    rows of an expert and a step of 256 codes in 4 KB, so that the second one moves them with bulk
//    copies and reads them with one conflict-free 16-byte load a product pair.
//  - An item is 32 or 48 weight rows against all token rows of a pass, over the whole of K: a
//    token value that comes from L2 serves that many weight rows.  Its eight warps take one
//    32-code chunk each of every step, whose codes are in one group whatever its size.
// The ring's stages hold a step's codes (one TMA box) and its token rows; a ninth warp fills them, the
// first codes before the layout kernel has ended.  The warps' sums are added in warp order.
#include "gemv_int4.cuh"

#include <type_traits>

namespace moe {
namespace {

constexpr int kGvEight = 8 * kGvStep * 2;      // bytes of eight token rows' values of a step

// MT: units of 16 weight rows of an item; NE: eights of token rows of a pass.
template <int MT, int NE>
struct RowsCfg {
  static constexpr int kCtas = NE > 4 ? 1 : 2;
  static constexpr int kTogether = NE == 8 && MT == 2 ? 4 : 2;   // as many as the registers take
  static constexpr int kTokens = MT * 16 * kGvStep / 2;        // offset in a stage
  static constexpr int kStage = kTokens + NE * kGvEight;
  static constexpr int kStages = (kCtas == 1 ? 200 : 88) * 1024 / kStage;
  static constexpr int kRing = kStages * kStage + 1024;
  static_assert(kStages >= 2 && kStages <= 10 && kStage % 1024 == 0, "");
};

// acc[0..1] += s * d[0..1], in one instruction.
__device__ __forceinline__ void fma2(float* acc, float s, const float* d) {
  asm("{\n.reg .b64 a, b, c;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %4};\nmov.b64 c, {%0, %1};\n"
      "fma.rn.f32x2 c, a, b, c;\nmov.b64 {%0, %1}, c;\n}\n"
      : "+f"(acc[0]), "+f"(acc[1])
      : "f"(d[0]), "f"(d[1]), "f"(s));
}

// packed [eight][step][chunk][lane]: lane (gr, t) holds row gr's values k = 8 t .. 8 t + 7 of the chunk
// of 32, in pair order; rows and k past the end are zeros.
__global__ void __launch_bounds__(256)
pack_tokens_kernel(const GemvArgs a, int per, uint4* __restrict__ packed) {
  __shared__ GemvExperts ex;
  pdl_wait();
  pdl_trigger();   // (after the wait: the product reads the offsets as soon as it runs)
  const int n_act = active_experts(a, ex, per, true);
  const int lane = threadIdx.x & 31, gr = lane >> 2, t = lane & 3;
  const int steps = (a.K + kGvStep - 1) / kGvStep;
  const long long n = (long long)ex.eights[n_act] * steps;
  for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < n; i += gridDim.x * 8LL) {
    const int eight = (int)(i / steps), st = (int)(i % steps);
    const int x = find_expert(ex.eights, n_act, eight);
    const int row = ex.lo[x] + 8 * (eight - ex.eights[x]) + gr;
    const bool has = row < ex.hi[x];
    const uint16_t* from = a.x + (size_t)row * a.K + st * kGvStep + 8 * t;
    uint4 v[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      v[c] = make_uint4(0u, 0u, 0u, 0u);
      if (has && st * kGvStep + 32 * c + 8 * t < a.K)
        v[c] = __ldg(reinterpret_cast<const uint4*>(from + 32 * c));
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) packed[i * 256 + c * 32 + lane] = pair_order(v[c]);
  }
}

struct RowsSmem {
  uint64_t full[10], empty[10];
  float red[kGvWarps][8][3 * 16 + 4];          // the warps' sums of eight token rows
  GemvExperts ex;
};

// shift: log2 of the codes that a scale covers.
template <bool ZERO, int MT, int NE>
__global__ void __launch_bounds__((kGvWarps + 1) * 32, RowsCfg<MT, NE>::kCtas)
gemv_int4_rows_kernel(const GemvArgs a, const __grid_constant__ CUtensorMap tm, int shift,
                      const uint8_t* __restrict__ packed) {
  using C = RowsCfg<MT, NE>;
  extern __shared__ uint8_t ring_raw[];
  __shared__ RowsSmem sm;
  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  // (the swizzle goes by address bits: the ring starts on a 1024-byte boundary)
  const uint32_t ring = (smem_u32(ring_raw) + 1023u) & ~1023u;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(sm.full + i, 1);
      mbar_init(sm.empty + i, kGvWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    prefetch_map(&tm);
  }
  const int n_act = __shfl_sync(0xffffffffu, active_experts(a, sm.ex, NE, false), 0);
  const int ntile = (a.N + MT * 16 - 1) / (MT * 16), steps = (a.K + kGvStep - 1) / kGvStep;
  const int items = sm.ex.passes[n_act] * ntile;
  struct Item {
    int e, n0, rb, rows, eight;
  };
  auto item = [&](int it) {
    const int pass = it / ntile, x = find_expert(sm.ex.passes, n_act, pass);
    const int i = pass - sm.ex.passes[x], rb = sm.ex.lo[x] + 8 * NE * i;
    return Item{sm.ex.act[x], (it - pass * ntile) * (MT * 16), rb, min(sm.ex.hi[x] - rb, 8 * NE),
                sm.ex.eights[x] + NE * i};
  };

  if (warp == kGvWarps) {
    // ---- the ring's producer
    auto codes = [&](int q, const Item& w, int st, int nb) {
      if (lane == 0) {
        uint64_t* full = sm.full + q % C::kStages;
        mbar_expect_tx(full, C::kTokens + nb * kGvEight);
        tma_3d(ring + q % C::kStages * C::kStage, &tm, st * (kGvStep / 2), w.n0, w.e, full);
      }
    };
    auto tokens = [&](int q, const Item& w, int st, int nb) {
      if (lane < nb)
        bulk_g2s(ring + q % C::kStages * C::kStage + C::kTokens + lane * kGvEight,
                 packed + ((size_t)(w.eight + lane) * steps + st) * kGvEight, kGvEight,
                 sm.full + q % C::kStages);
    };
    int primed = 0;
    for (int it = blockIdx.x; it < items && primed < C::kStages; it += gridDim.x) {
      const Item w = item(it);
      for (int st = 0; st < steps && primed < C::kStages; ++st)
        codes(primed++, w, st, (w.rows + 7) / 8);
    }
    pdl_wait();                                // the token rows are laid out
    asm volatile("fence.proxy.async;" ::: "memory");
    int q = 0;
    bool ok = true;
    for (int it = blockIdx.x; it < items && ok; it += gridDim.x) {
      const Item w = item(it);
      const int nb = (w.rows + 7) / 8;
      for (int st = 0; st < steps; ++st, ++q) {
        if (q >= primed) {
          if (!(ok = warp_wait(sm.empty + q % C::kStages, (q / C::kStages - 1) & 1, a.err, kGvErrWait)))
            break;
          codes(q, w, st, nb);
          __syncwarp();
        }
        tokens(q, w, st, nb);
      }
    }
    // after a wait that ran out: what was asked for has to have landed before the memory goes
    if (!ok)
      for (int i = max(0, q - C::kStages); i < q; ++i)
        warp_wait(sm.full + i % C::kStages, (i / C::kStages) & 1, a.err, kGvErrWait);
    return;
  }

  // ---- the warps that multiply: chunk `warp` of every step
  const int gr = lane >> 2, t = lane & 3;
  bool ok = true;
  int slot = 0;
  uint32_t phase = 0;
  // where the lane points ldmatrix (weight row `lane` of 32) and its token values
  const uint32_t wa = ring + lane * 128 + ((warp ^ (lane & 7)) << 4);
  const uint32_t xa = ring + C::kTokens + warp * 512 + lane * 16;
  for (int it = blockIdx.x; it < items; it += gridDim.x) {
    const Item w = item(it);
    const int nb = (w.rows + 7) / 8;
    // Scales in the upper half, zero points in the lower, two steps ahead of their use: lane t of a
    // row reads those of the weight rows gr + 8 t and gr + 8 (t + 4); rows and groups past the end
    // read the last ones (those rows are not stored, those groups' products are zero).
    constexpr int NL = (2 * MT + 3) / 4;
    const size_t base = ((size_t)w.e * a.N + w.n0) * a.ng;
    size_t so[NL];
#pragma unroll
    for (int l = 0; l < NL; ++l)
      so[l] = base + (size_t)min(gr + 8 * (t + 4 * l), a.N - 1 - w.n0) * a.ng;
    auto scales = [&](int st, uint32_t (&v)[NL]) {
      const int g = min((st * kGvStep + 32 * warp) >> shift, a.ng - 1);
#pragma unroll
      for (int l = 0; l < NL; ++l) {
        v[l] = (uint32_t)__ldg(a.s + so[l] + g) << 16;
        if (ZERO) v[l] |= __ldg(a.z + so[l] + g);
      }
    };
    uint32_t sv[NL], sv1[NL];
    scales(0, sv);
    scales(min(1, steps - 1), sv1);
    float acc[MT][NE][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < NE; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[m][i][c] = 0.f;
    for (int st = 0; st < steps; ++st) {
      uint32_t sv2[NL];
      scales(min(st + 2, steps - 1), sv2);
      if (ok) ok = warp_wait(sm.full + slot, phase, a.err, kGvErrWait);
      const uint32_t off = slot * C::kStage;
      uint32_t p[MT][2][4];
      float f[MT][2];
#pragma unroll
      for (int u = 0; u < MT; u += 2) {
        uint32_t wd[4];
        load_words(wd, wa + off + u * 2048);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int m = u + j / 2, r = 2 * u + j;   // unit, eight of weight rows
          if (m < MT) {
            const uint32_t v = __shfl_sync(0xffffffffu, sv[r / 4], (lane & 28) | (r & 3));
            f[m][j & 1] = __uint_as_float(v & 0xFFFF0000u);
            code_pairs(wd[j], ZERO ? zero_pair<0>(v) : 0xBE00BE00u, p[m][j & 1]);   // -8 * 2^-6
          }
        }
      }
      // kTogether eights at a time, so that their products overlap (the last ones' may have no rows:
      // nothing stores what comes of them); all of them without a branch between where all have rows
      auto products = [&](auto first) {
        constexpr int i0 = decltype(first)::value;
        uint4 b[C::kTogether];
        float d[C::kTogether][MT][4];
#pragma unroll
        for (int i = 0; i < C::kTogether; ++i) b[i] = load_shared(xa + off + (i0 + i) * kGvEight);
#pragma unroll
        for (int i = 0; i < C::kTogether; ++i)
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            d[i][m][0] = d[i][m][1] = d[i][m][2] = d[i][m][3] = 0.f;
            mma_bf16(d[i][m], p[m][0][0], p[m][1][0], p[m][0][1], p[m][1][1], b[i].x, b[i].y);
          }
#pragma unroll
        for (int i = 0; i < C::kTogether; ++i)
#pragma unroll
          for (int m = 0; m < MT; ++m)
            mma_bf16(d[i][m], p[m][0][2], p[m][1][2], p[m][0][3], p[m][1][3], b[i].z, b[i].w);
#pragma unroll
        for (int i = 0; i < C::kTogether; ++i)
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            fma2(acc[m][i0 + i], f[m][0], d[i][m]);
            fma2(acc[m][i0 + i] + 2, f[m][1], d[i][m] + 2);
          }
      };
      constexpr int T = C::kTogether;
      if (nb > NE - T) {
        products(std::integral_constant<int, 0>{});
        if constexpr (NE > T) products(std::integral_constant<int, T>{});
        if constexpr (NE > 2 * T) products(std::integral_constant<int, 2 * T>{});
        if constexpr (NE > 3 * T) products(std::integral_constant<int, 3 * T>{});
      } else {
        products(std::integral_constant<int, 0>{});
        if constexpr (NE > 2 * T) {
          if (nb > T) products(std::integral_constant<int, T>{});
          if constexpr (NE > 3 * T)
            if (nb > 2 * T) products(std::integral_constant<int, 2 * T>{});
        }
      }
      __syncwarp();
      if (ok) warp_arrive(sm.empty + slot, lane);
      if (++slot == C::kStages) {
        slot = 0;
        phase ^= 1;
      }
#pragma unroll
      for (int l = 0; l < NL; ++l) {
        sv[l] = sv1[l];
        sv1[l] = sv2[l];
      }
    }
    // the warps' sums, eight token rows at a time
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      if (i >= nb) break;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          sm.red[warp][2 * t + (c & 1)][16 * m + gr + 8 * (c >> 1)] = acc[m][i][c];
      asm volatile("bar.sync 1, 256;" ::: "memory");
      for (int o = threadIdx.x; o < 8 * 64; o += kGvThreads) {
        const int r = o >> 6, n = o & 63;
        if (n < MT * 16 && w.n0 + n < a.N && 8 * i + r < w.rows) {
          float v = sm.red[0][r][n];
#pragma unroll
          for (int q = 1; q < kGvWarps; ++q) v += sm.red[q][r][n];
          const size_t at = (size_t)(w.rb + 8 * i + r) * a.N + w.n0 + n;
          v *= 0x1p6f;
          if (a.f32) static_cast<float*>(a.y)[at] = v;
          else static_cast<uint16_t*>(a.y)[at] = float_to_bf16_bits(v);
        }
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
    }
  }
}

long long most_eights(int max_rows, int E) {   // every expert's last one may have fewer rows
  return std::min<long long>(max_rows, (long long)E + max_rows / 8);
}

template <bool ZERO, int MT, int NE>
int launch_rows(const GemvArgs& a, const uint8_t* w, int items, int shift, const uint8_t* packed,
                cudaStream_t st) {
  using C = RowsCfg<MT, NE>;
  CUtensorMap tm;
  if (!encode_weights(&tm, w, a.E, a.N, a.K, MT * 16)) return MOE_ERR_UNSUPPORTED;
  auto kernel = gemv_int4_rows_kernel<ZERO, MT, NE>;
  MOE_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kRing));
  MOE_LAUNCH_NEXT(true, kernel, dim3(std::min(items, C::kCtas * sm_count())),
                  dim3((kGvWarps + 1) * 32), C::kRing, st, a, tm, shift, packed);
  MOE_COUNT_LAUNCH();
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

template <bool ZERO, int NE>
int launch_rows(const GemvArgs& a, const uint8_t* w, int shift, void* packed, cudaStream_t st) {
  const long long eights = most_eights(a.max_rows, a.E);
  const long long passes = std::min<long long>(eights, a.E + a.max_rows / (8 * NE));
  // the height whose rounds cost the least: its rows, and what a step costs beside them
  long long best = 0;
  int mt = 0, items = 0;
  for (int m = 2; m <= (NE == 4 ? 2 : 3); ++m) {   // (four eights and 48 rows spill)
    const long long c = passes * ceil_div(a.N, m * 16), slots = (NE > 4 ? 1LL : 2LL) * sm_count();
    const long long cost = (c + slots - 1) / slots * (10 * m + 8);
    if (c > 0x3fffffff) return MOE_ERR_INVALID_ARG;   // (y alone would not fit on the GPU)
    if (!mt || cost <= best) {
      mt = m;
      best = cost;
      items = (int)c;
    }
  }
  const long long blocks = (eights * ceil_div(a.K, kGvStep) + 7) / 8;
  MOE_LAUNCH_PDL(pack_tokens_kernel, dim3((unsigned)std::min<long long>(blocks, 8LL * sm_count())),
                 dim3(256), 0, st, a, NE, static_cast<uint4*>(packed));
  MOE_COUNT_LAUNCH();
  MOE_LAUNCH_CHECK();
  const uint8_t* px = static_cast<const uint8_t*>(packed);
  if constexpr (NE != 4)
    if (mt == 3) return launch_rows<ZERO, 3, NE>(a, w, items, shift, px, st);
  return launch_rows<ZERO, 2, NE>(a, w, items, shift, px, st);
}

template <bool ZERO>
int launch_rows(const GemvArgs& a, const uint8_t* w, int shift, void* packed, cudaStream_t st) {
  const int rows = ceil_div(a.max_rows, a.E);
  if (rows <= 16) return launch_rows<ZERO, 2>(a, w, shift, packed, st);
  if (rows <= 32) return launch_rows<ZERO, 4>(a, w, shift, packed, st);
  return launch_rows<ZERO, 8>(a, w, shift, packed, st);
}

}  // namespace

size_t gemv_packed_bytes(int max_rows, int E, int K) {
  if (ceil_div(max_rows, E) <= 8) return 0;
  return (size_t)most_eights(max_rows, E) * ceil_div(K, kGvStep) * kGvEight;
}

int launch_gemv_rows(const GemvArgs& a, const uint8_t* w, int group, void* packed, cudaStream_t st) {
  const int shift = group == 32 ? 5 : group == 64 ? 6 : 7;
  return a.z ? launch_rows<true>(a, w, shift, packed, st) : launch_rows<false>(a, w, shift, packed, st);
}

}  // namespace moe
