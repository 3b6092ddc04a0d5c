// Grouped matrix product of E4M3 token rows with E4M3 expert weights on the 5th-generation
// tensor cores (tcgen05 + TMEM), one fp32 scale per row and 128 columns of the activations and
// per 128 x 128 block of the weights:
//
//   acc[row][n] = sum_b xs[row][b] ws[n / 128][b] sum_{k in block b} xq[row][k] w[n][k]
//
// Each block's inner sum is formed by the tensor cores from zero and scaled into an fp32
// accumulator in registers, so arbitrary fp32 scales are exact to one rounding per block and the
// tensor cores' own accumulation never runs over more than 128 products.
//
// Tile: 128 token rows (the MMA's M, one TMEM lane each) x 256 weight rows (N: a gate tile and
// its up tile when fused, else two neighbouring tiles), one block of 128 k per step.  With tokens
// on the lanes a thread owns one token: its scale is one value per step, a weight block is one
// value per 128 columns, and the row's largest |h| (fused: h is requantised here) is a maximum
// over the thread's own registers.  (Weights on the lanes would need every token's scale in
// every thread, 128 shared-memory reads a step.)
//
// Persistent kernel, one CTA per SM, 384 threads:
//   warp 0     producer: per step 16 KB of token rows by 2-D TMA (128-byte swizzle; a tile that is
//              not full in boxes of 32 rows) and 32 KB of weights: two bundle tiles by bulk copy
//              (each is stored as its swizzled shared-memory image), or two TMA boxes of a
//              row-major weight; three stages;
//   warps 1, 3 MMA issuers, one per 256-column TMEM buffer: four tcgen05.mma (K = 32 each) per
//              step, the steps in turn;
//   warp 2     scale factors: xs * ws per token and weight tile of each step, to shared memory;
//   warps 4-11 two warps per TMEM lane quarter, 64 columns of each weight tile per thread: per
//              step, tcgen05.ld and a packed fp32 multiply-add by xs * ws into 128 accumulators
//              (they take the registers warps 0-3 give up).
//
// Work: tiles (expert, weight tile pair, token tile), token tile fastest so that CTAs running
// together share weights through L2.  With few tiles their steps are
// cut into equal ranges (see Cut): a tile of several ranges is finished by the last of its CTAs to
// arrive (a counter per lane quarter), which adds the pieces' fp32 sums in range order, so the
// result does not depend on the arrival order.
//
// Measured, inputs changing from call to call: 8192 rows of 8 experts x 4096 x 14336 in 457 us (2.1
// PFLOP/s); 65,536 rows of 256 SwiGLU experts of 7168 x 2048 in 3.6 ms (1.6 PFLOP/s, 3.5 TB/s of
// necessary bytes); 32 tokens of the same layer in 874 us, the copy bandwidth of HBM.  (The same
// inputs again and again: 418 us and 3.4 ms.)  What bounds the large ones is a step's way through shared memory (48 KB
// in, 48 KB out to the tensor cores: without the epilogue 2.8-3.0 PFLOP/s) and the epilogue warps'
// chain of wait, TMEM load, multiply-add and release, about 1000 clocks a step against 540 of
// tensor work (tensor pipe 52% busy, issue slots 42%).  Sixteen epilogue warps of half the columns
// were slower (468 us against 428 on the same inputs), half-step TMEM buffers no faster.  Of the small ones, launch,
// tile tables and first load take 3-5 us before the first product, joining pieces 2-5 after the last.
//
// Every wait is bounded (2 s; then an error word and the kernel ends).
#include "fp8.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int kStages = 3;
constexpr int kABytes = kFp8TileBytes, kBBytes = 2 * kFp8TileBytes;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kThreads = 384;
static_assert(kThreads >= kMaxExperts, "a thread looks up each expert's rows");
// Registers per thread after the split: warps 0-3 and warps 4-11 (128 * 56 + 256 * 224 = the
// 384 * 168 the block is launched with).
constexpr int kRegsLow = 56, kRegsHigh = 224;
static_assert(128 * kRegsLow + 256 * kRegsHigh <= kThreads * 168, "within the launch's registers");
constexpr int kAccCols = 256, kTmemCols = 512;
// Tiles are cut into ranges of steps where that spares the busiest CTA more than it costs, counted
// in steps: kJoinSteps for writing a piece and joining, kJoinRows for each piece of 128 rows read
// (few rows: 1 for 16 pieces), kPieceSteps where a CTA may write two pieces.  (1001 rows of 8 experts,
// 1200 x 1000, 10 steps a tile: joined from four pieces 33 us, whole 20.  One row, 7168 x 4096, 56
// steps a tile: 9 ranges a tile 19.4 us, ranges over all tiles 21.4.)
constexpr int kRangeTiles = 4, kJoinSteps = 4, kJoinRows = 3, kPieceSteps = 3;

// Output rows on their way out: per epilogue warp two boxes of 32 rows x 128 bytes.
constexpr int kBox = 4096, kOutBytes = 8 * 2 * kBox;
// Up to this many rows of a quarter are joined and finished a row at a time by the whole warp.
constexpr int kFewRows = 4;
struct Fp8Params {
  CUtensorMap tm_x, tm_x32;     // token rows [max_rows][K], boxes of 128 / 32 rows x 128 bytes
  CUtensorMap tm_out;           // y (or hq): boxes of 32 rows x 128 (hq: 64) bytes
  CUtensorMap tm_w;             // row-major weights [E * N][K], boxes of 128 x 128 bytes
  const float* xs;
  const int32_t* offsets;
  int E, N, K, KB, NT, max_rows, quarters;
  BundleTable tab;
  const void* const* dev_tab;
  size_t w_off, s_off;
  const float* ws;              // row-major weights: their scales (else the bundles')
  const int32_t* active;
  const int32_t* n_active;
  int host_n;
  int16_t host_ids[kMaxExperts];
  uint8_t* hq;
  float* hs;
  void* y;
  int y_f32, after;
  float* part;                  // [CTAs][2][quarters][2][32][32 lanes] groups of 4 columns
  int32_t* counters;            // [tiles][4], used when tiles are cut
  int32_t* err;
};
static_assert(sizeof(Fp8Params) <= 4096, "kernel parameters stay within 4 KB");

// Instruction descriptor of kind::f8f6f4: E4M3 A and B (type 0), fp32 D, both K-major, M x N.
__device__ __forceinline__ uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_fp8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
// 64 columns of the warp's 32 lanes, without the wait.
__device__ __forceinline__ void tmem_ld64_nw(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, "
      "%45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, "
      "%62, %63}, [%64];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]),
        "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]),
        "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]),
        "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]),
        "=r"(r[63])
      : "r"(taddr));
}
// acc[i] += v[i] * f, two at a time (fma.rn.f32x2: one issue slot).  Volatile, as the load and its
// wait are, so that no use of v moves above the wait.  The pairs are put together inside the
// asm: accumulators kept as 64-bit values make the compiler copy every operand each step
// (measured, 128 columns by two warps per scheduler: 613 clocks against 345).
template <int FROM = 0, int TO = 32>
__device__ __forceinline__ void fma64(float* acc, const uint32_t (&v)[64], uint64_t f) {
#pragma unroll
  for (int i = FROM; i < TO; ++i)
    asm volatile(
        "{\n.reg .b64 t, a;\nmov.b64 t, {%2, %3};\nmov.b64 a, {%0, %1};\n"
        "fma.rn.f32x2 a, t, %4, a;\nmov.b64 {%0, %1}, a;\n}\n"
        : "+f"(acc[2 * i]), "+f"(acc[2 * i + 1])
        : "r"(v[2 * i]), "r"(v[2 * i + 1]), "l"(f));
}
__device__ __forceinline__ uint64_t pack(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}

// silu(g) * u with the hardware exponential and reciprocal (relative error ~1e-6, far below
// E4M3's step); for g below about -88 e^-g is infinite and the quotient -0, the limit of silu.
__device__ __forceinline__ float silu_mul(float g, float u) {
  return __fdividef(g, 1.f + __expf(-g)) * u;
}

__device__ __forceinline__ int expert_of(const Fp8Params& p, int a) {
  return p.host_n >= 0 ? p.host_ids[a] : p.active ? p.active[a] : a;
}
// Rows [r0, r1) of expert e clipped to [0, max_rows); true when the clip changed anything.
__device__ __forceinline__ bool expert_rows(const Fp8Params& p, int e, int& r0, int& r1) {
  const int a = p.offsets ? p.offsets[e] : 0, b = p.offsets ? p.offsets[e + 1] : p.max_rows;
  r0 = min(max(a, 0), p.max_rows);
  r1 = min(max(b, r0), p.max_rows);
  return r0 != a || r1 != b;
}

// The CTA's share of the steps: whole tiles CTA, CTA + G, ..., or a range of all tiles' steps in
// order, the first `more` CTAs taking n + 1 steps and the others n; or, with no more tiles than
// CTAs, `per` equal ranges of every tile, so that no CTA writes two pieces.
struct Cut {
  int on, G, n, more, per, KB;
  // by a converged warp; rows: the most rows of any tile
  __device__ __forceinline__ void set(int U, int KB_, int rows, int lane) {
    const int ctas = gridDim.x;
    int best = 0;
    if (U > 0 && U < kRangeTiles * ctas) {
      // the busiest CTA's cost, in steps: of whole tiles, of ranges over all tiles, and of 2 .. 33
      // ranges a tile (one choice a lane); the least, or what comes first here.  (Quotients for the
      // choice only, so by fast division.)
      auto up = [](float a, float b) { return __float2uint_ru(__fdividef(a, b) - 1e-3f); };
      auto join = [&](float pieces) {
        const float each = rows <= kFewRows ? 0.0625f : kJoinRows / 128.f * rows;
        return kJoinSteps + __float2uint_rd(pieces * each);
      };
      const float fk = KB_, fu = U, fc = ctas;
      const unsigned whole = up(fu, fc) * KB_ << 8, all = up(fu * fk, fc);
      const unsigned over = (all + join(__fdividef(fk, all) + 1.f) + kPieceSteps) << 8 | 255u;
      unsigned c = min(whole, over);
      const int q = 2 + lane;
      if (q * U <= ctas && q <= KB_) c = min(c, (up(fk, q) + join(q)) << 8 | (unsigned)q);
      c = __reduce_min_sync(0xffffffffu, c);
      best = c & 255;
    }
    if (lane) return;
    per = best == 255 ? 0 : best;
    KB = KB_;
    on = best > 0;
    G = ctas;
    if (!on) return;
    G = per ? U * per : min(ctas, U * KB);      // no empty ranges
    const int steps = per ? KB : U * KB, parts = per ? per : G;
    n = steps / parts;
    more = steps - n * parts;
  }
  __device__ __forceinline__ int start(int cta) const {
    const int u = per ? cta / per : 0, i = cta - u * per;
    return u * KB + i * n + min(i, more);
  }
  __device__ __forceinline__ int count(int cta) const { return n + ((per ? cta % per : cta) < more); }
  __device__ __forceinline__ int owner(int step) const {
    const int u = per ? step / KB : 0, s = step - u * KB, i = s / (n + 1);
    return u * per + (i < more ? i : more + (s - more * (n + 1)) / n);
  }
};
struct Walk {
  int KB, U, G, u, lo, hi, left;   // left: steps (cut) still to do
  bool cut;
  __device__ __forceinline__ Walk(const Cut& c, int U_, int KB_) : KB(KB_), U(U_), G(c.G) {
    cut = c.on;
    lo = hi = left = 0;
    u = (int)blockIdx.x;
    if (cut) {
      const int pos = c.start(u);
      left = u < G ? c.count(u) : 0;
      u = pos / KB;
      lo = pos - u * KB;
    }
    u -= cut ? 1 : G;                           // next() steps on to the first
    hi = lo;
    if (cut && lo == 0) hi = KB;
  }
  __device__ __forceinline__ bool next() {
    if (cut) {
      if (left <= 0) return false;
      ++u;
      lo = hi == KB ? 0 : hi;
      hi = min(KB, lo + left);
      left -= hi - lo;
      return true;
    }
    u += G;
    lo = 0;
    hi = KB;
    return u < U;
  }
};

struct alignas(16) Ctl {
  uint64_t full[kStages], empty[kStages], tfull[2], tempty[2], pair[4], drain[2];
  uint32_t tmem;
  int last[4];
  Cut cut;
  int pref[kMaxExperts + 1];    // tiles before the a-th expert run
  int row0[kMaxExperts], rows[kMaxExperts], id[kMaxExperts];   // its rows and id
  float amax[2][2][128];
  float2 f[2][128];             // per TMEM buffer and token: xs * ws of the two weight tiles
};
constexpr int kSmem = kStages * kStageBytes + kOutBytes + 1024 + (int)sizeof(Ctl);
static_assert(kStages == 3, "the MMA issuers' order of waits covers a stage's use three steps back");
static_assert(kSmem <= 232448, "over the 227 KB shared-memory limit of a CTA");

struct Tile {
  int e, nt, r0, rows;
};
__device__ __forceinline__ Tile tile_of(const Ctl& c, int n_act, int u) {
  int lo = 0, hi = n_act - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (c.pref[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  Tile t;
  t.e = c.id[lo];
  const int n = c.rows[lo], mts = (n + 127) >> 7, rem = u - c.pref[lo];
  t.nt = mts == 1 ? rem : rem / mts;
  const int mt = rem - t.nt * mts;
  t.r0 = c.row0[lo] + mt * 128;
  t.rows = min(128, n - mt * 128);
  return t;
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int c0, int c1, uint32_t src) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(c0), "r"(c1), "r"(src)
      : "memory");
}
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// This thread's stores have read their shared memory (all: have also been written).
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}
__device__ __forceinline__ void proxy_fence() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Rows 32 q .. of the tile x 64 columns from `col` on leave from the box `st` (32 rows of kRow
// bytes, 16-byte piece i of row l at i ^ l's swizzle): one TMA store, which runs while the next
// tile's steps do, when all 32 rows exist; else coalesced stores of those that do (a box would
// reach into the next expert's rows).  (Stored from registers, a lane's 16 bytes a time, a tile
// took 9,000 clocks in which the tensor cores waited; by coalesced stores 4,300; by one bulk copy
// per row 6,000.)
template <int kRow>
__device__ __forceinline__ void store_box(const CUtensorMap* map, uint8_t* dst, size_t pitch,
                                          const uint8_t* st, int col, int row, int have, int bytes,
                                          int lane) {
  constexpr int kPer = kRow / 16;
  proxy_fence();
  __syncwarp();
  if (have >= 32) {
    if (lane == 0) {
      tma_store_2d(map, col, row, smem_u32(st));
      bulk_commit();
    }
  } else {
#pragma unroll 1
    for (int at = lane; at < have * kPer; at += 32) {
      const int l = at / kPer, i = at % kPer;
      if (16 * i < bytes)
        *reinterpret_cast<uint4*>(dst + l * pitch + 16 * i) = *reinterpret_cast<const uint4*>(
            st + l * kRow + ((i ^ (kRow == 128 ? l % 8 : (l >> 1) % 4)) << 4));
    }
  }
}

// A warp's 32 rows of y: 64 columns of the tile's first weight block (acc[0..63]) and 64 of the
// second, through its two boxes.  Rows that are not 16-byte aligned are stored element by
// element, the lanes side by side along one row after another.
template <bool F32>
__device__ __forceinline__ void store_y(const Fp8Params& p, uint8_t* box, const float (&acc)[128],
                                        int row, int n0, int half, int have, int lane) {
  constexpr int kElem = F32 ? 4 : 2, kCols = 128 / kElem;   // columns of a box
  const bool vec = (p.N * kElem) % 16 == 0;
  const size_t pitch = (size_t)p.N * kElem;
#pragma unroll
  for (int b = 0; b < 128 / kCols; ++b) {
    const int c0 = b * kCols, w = c0 / 64, col = n0 + 128 * w + 64 * half + c0 % 64;
    uint8_t* st = box + (b & 1) * kBox;
    if ((b & 1) == 0) {                       // both boxes free again
      if (lane == 0) bulk_wait_read();
      __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float* v = acc + c0 + i * (16 / kElem);
      const uint4 o =
          F32 ? make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                           __float_as_uint(v[3]))
              : make_uint4(float2_to_bf16x2(v[0], v[1]), float2_to_bf16x2(v[2], v[3]),
                           float2_to_bf16x2(v[F32 ? 0 : 4], v[F32 ? 0 : 5]),
                           float2_to_bf16x2(v[F32 ? 0 : 6], v[F32 ? 0 : 7]));
      *reinterpret_cast<uint4*>(st + lane * 128 + ((i ^ (lane & 7)) << 4)) = o;
    }
    const int left = min(kCols, p.N - col);   // columns of these that exist
    uint8_t* y = static_cast<uint8_t*>(p.y) + row * pitch + (size_t)col * kElem;
    if (left <= 0) continue;
    if (vec) {
      store_box<128>(&p.tm_out, y, pitch, st, col, row, have, left * kElem, lane);
    } else {
      __syncwarp();
#pragma unroll 1
      for (int l = 0; l < min(have, 32); ++l)
        for (int k = lane; k < left; k += 32) {
          const uint8_t* e = st + l * 128 + (((k * kElem / 16) ^ (l & 7)) << 4) + k * kElem % 16;
          if (F32) reinterpret_cast<float*>(y + l * pitch)[k] = *reinterpret_cast<const float*>(e);
          else reinterpret_cast<uint16_t*>(y + l * pitch)[k] = *reinterpret_cast<const uint16_t*>(e);
        }
    }
  }
  __syncwarp();
}

// Bytes a step of tile t brings in, and the request for its weights (into sb, completing on fb).
template <bool FUSED>
__device__ __forceinline__ uint32_t load_bytes(const Fp8Params& p, const Tile& t) {
  const bool two = FUSED || t.nt * 256 + 128 < p.N;
  return (t.rows > 96 ? kABytes : ((t.rows + 31) >> 5) * 4096) + (two ? kBBytes : kFp8TileBytes);
}
template <bool FUSED, bool PLAIN>
__device__ __forceinline__ void load_weights(const Fp8Params& p, const Tile& t, int kb, uint32_t sb,
                                             uint64_t* fb) {
  const int n0 = t.nt * (FUSED ? 128 : 256);
  const bool two = FUSED || n0 + 128 < p.N;
  if (PLAIN) {
    tma_2d(sb, &p.tm_w, kb * 128, t.e * p.N + n0, fb);
    if (two) tma_2d(sb + kFp8TileBytes, &p.tm_w, kb * 128, t.e * p.N + n0 + 128, fb);
  } else {
    const char* b = static_cast<const char*>(p.dev_tab ? p.dev_tab[t.e] : p.tab.p[t.e]) + p.w_off +
                    ((size_t)(n0 >> 7) * p.KB + kb) * kFp8TileBytes;
    bulk_g2s(sb, b, kFp8TileBytes, fb);
    if (two)
      bulk_g2s(sb + kFp8TileBytes, b + (size_t)(FUSED ? p.N >> 7 : 1) * p.KB * kFp8TileBytes,
               kFp8TileBytes, fb);
  }
}

// FUSED: N = columns of h (gate rows 0..N-1, up rows N..2N-1).  PLAIN: row-major weights by TMA.
template <bool FUSED, bool PLAIN>
__global__ void __launch_bounds__(kThreads, 1) fp8_gemm_kernel(const __grid_constant__ Fp8Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* out = smem + kStages * kStageBytes;
  Ctl& c = *reinterpret_cast<Ctl*>(out + kOutBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 32) {
    prefetch_map(&p.tm_x);
    prefetch_map(&p.tm_x32);
    if (PLAIN) prefetch_map(&p.tm_w);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&c.full[s], 1);
      mbar_init(&c.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&c.tfull[b], 2);   // the MMAs and the factors
      mbar_init(&c.tempty[b], 8);
    }
    for (int q = 0; q < 4; ++q) mbar_init(&c.pair[q], 2);
    for (int b = 0; b < 2; ++b) mbar_init(&c.drain[b], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&c.tmem)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  // A product after the clearing of its control words needs those first when it joins pieces; the
  // second product of an FFN starts while the first one ends: of what that writes it reads the
  // token rows and their scales only, and writes nothing itself, until pdl_wait (below, by the
  // warps concerned).  Experts, offsets and weights are older than both: the first product lets
  // the second go only after this wait, or itself follows a clearing that nothing ran beside.
  if (p.after == kAfterAny) pdl_wait();
  pdl_trigger();
  const int n_act = p.host_n >= 0 ? p.host_n : p.active ? *p.n_active : p.E;
  // the experts' rows, a thread each (one memory latency), then the prefix of their tile counts
  if ((int)threadIdx.x < n_act) {
    int r0, r1;
    const int a = threadIdx.x, e = expert_of(p, a);
    if (expert_rows(p, e, r0, r1)) {
      pdl_wait();
      atomicExch(p.err, 8);
    }
    if (!PLAIN && r1 > r0 && !(p.dev_tab ? p.dev_tab[e] : p.tab.p[e])) {
      r1 = r0;                                  // no weights: none of its rows is computed
      pdl_wait();
      atomicCAS(p.err, 0, 10);
    }
    c.row0[a] = r0;
    c.rows[a] = r1 - r0;
    c.id[a] = e;
  }
  __syncthreads();
  if (warp == 2) {
    int carry = 0, most = 0;
    for (int base = 0; base < n_act; base += 32) {
      const int a = base + lane, rows = a < n_act ? c.rows[a] : 0,
                cnt = p.NT * ((rows + 127) >> 7);
      most = max(most, __reduce_max_sync(0xffffffffu, min(rows, 128)));
      int incl = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (a < n_act) c.pref[a] = carry + incl - cnt;
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) c.pref[n_act] = carry;
    c.cut.set(carry, p.KB, most, lane);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;
  const int U = c.pref[n_act], KB = p.KB;
  Walk wk(c.cut, U, KB);

  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const int who = !elect_one();               // 0: the lane that waits and issues
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    bool ok = true;
    // the weights of the first stages are asked for before token rows still being written may be
    int ahead = 0;
    if (p.after == kAfterRows && wk.next()) {
      const Tile t = tile_of(c, n_act, wk.u);
      for (; ahead < min(kStages, wk.hi - wk.lo); ++ahead) {
        if (elect_one()) {
          const uint32_t sb = smem_u32(smem + ahead * kStageBytes) + kABytes;
          mbar_expect_tx(&c.full[ahead], load_bytes<FUSED>(p, t));
          load_weights<FUSED, PLAIN>(p, t, wk.lo + ahead, sb, &c.full[ahead]);
        }
        __syncwarp();
      }
    }
    if (p.after == kAfterRows) pdl_wait();
    wk = Walk(c.cut, U, KB);
    while (ok && wk.next()) {
      const Tile t = tile_of(c, n_act, wk.u);
      const int nsub = t.rows > 96 ? 0 : (t.rows + 31) >> 5;
      const uint32_t bytes = load_bytes<FUSED>(p, t);
      for (int kb = wk.lo; kb < wk.hi; ++kb) {
        if (!(ok = lead_wait(&c.empty[stage], phase ^ 1, p.err, 1, who))) break;
        uint64_t* fb = &c.full[stage];
        const uint32_t sa = smem_u32(smem + stage * kStageBytes);
        if (elect_one()) {
          if (issued >= ahead) {
            mbar_expect_tx(fb, bytes);
            load_weights<FUSED, PLAIN>(p, t, kb, sa + kABytes, fb);
          }
          if (nsub) {
            // 32-row boxes stacked at 4 KB: the same swizzled layout as one box of all rows
            for (int s = 0; s < nsub; ++s)
              tma_2d(sa + 4096 * s, &p.tm_x32, kb * 128, t.r0 + 32 * s, fb);
          } else {
            tma_2d(sa, &p.tm_x, kb * 128, t.r0, fb);
          }
        }
        __syncwarp();
        if (++stage == kStages) { stage = 0; phase ^= 1; }
        ++issued;
      }
    }
    // after a failed wait, copies may still be on their way to this CTA's shared memory: wait
    // (bounded) for the last of each stage
    for (int i = 0; !ok && i < min(issued, kStages); ++i) {
      if (--stage < 0) { stage = kStages - 1; phase ^= 1; }
      lead_wait(&c.full[stage], phase, p.err, 1, who);
    }
  } else if (warp == 1 || warp == 3) {
    // ------------------------------------------------------------ MMA issuers
    // warp 1 takes the even steps (TMEM buffer 0), warp 3 the odd ones (buffer 1): an issuer's
    // waits and loop run while the other's products do.  Always 256 columns, so that nothing of
    // a tile is needed but its steps (where a tile has one weight tile only, the second's
    // columns take what the stage held and are not stored).
    const uint32_t idesc = idesc_e4m3(128, kAccCols);
    const int buf = warp >> 1, who = !elect_one();
    const uint32_t d = tmem + buf * kAccCols;
    int stage = 0, turn = 0;
    uint32_t phase = 0, tphase = 0;
    bool ok = true;
    while (ok && wk.next()) {
      for (int kb = wk.lo; kb < wk.hi; ++kb, turn ^= 1) {
        if (turn == buf) {
          // In this order: once the buffer is back, step s - 2 has been through the epilogue, and
          // so has s - 3, the stage's last use, which the other issuer waited for.  Looked at
          // before that, the stage's barrier may still be two phases behind, where its parity
          // reads as complete.
          if (!(ok = lead_wait(&c.tempty[buf], tphase ^ 1, p.err, 2, who))) break;
          if (!(ok = lead_wait(&c.full[stage], phase, p.err, 3, who))) break;
          const uint32_t sa = smem_u32(smem + stage * kStageBytes);
          const uint64_t da = sdesc_sw128(sa), db = sdesc_sw128(sa + kABytes);
          if (elect_one()) {
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < 4; ++j) mma_fp8(d, da + 2 * j, db + 2 * j, idesc, j > 0);
            mma_commit(&c.empty[stage]);
            mma_commit(&c.tfull[buf]);
          }
          __syncwarp();
          tphase ^= 1;
        }
        if (++stage == kStages) { stage = 0; phase ^= 1; }
      }
    }
    if (!ok) {   // after a failed wait: the products still running write TMEM until they end
      if (elect_one()) mma_commit(&c.drain[buf]);
      __syncwarp();
      lead_wait(&c.drain[buf], 0, p.err, 7, who);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ scale factors
    if (p.after == kAfterRows) pdl_wait();
    // per step: xs * ws of every token and weight tile into the TMEM buffer's slot
    int buf = 0;
    uint32_t tphase = 0;
    bool ok = true;
    while (ok && wk.next()) {
      const Tile t = tile_of(c, n_act, wk.u);
      const int n0 = t.nt * (FUSED ? 128 : 256), NB = (p.N + 127) >> 7;
      const bool two = FUSED || n0 + 128 < p.N;
      const float* sw0;
      if (PLAIN) {
        sw0 = p.ws + ((size_t)t.e * NB + (n0 >> 7)) * KB;
      } else {
        const char* b = static_cast<const char*>(p.dev_tab ? p.dev_tab[t.e] : p.tab.p[t.e]);
        sw0 = reinterpret_cast<const float*>(b + p.s_off) + (size_t)(n0 >> 7) * KB;
      }
      const float* sw1 = two ? sw0 + (size_t)(FUSED ? NB : 1) * KB : sw0;
      const float* sx = p.xs + (size_t)(t.r0 + lane) * KB;
      const size_t step = (size_t)32 * KB;
      float x[2][4], a[2], b[2];      // two steps in turn: a step's loads go out a step ahead
      auto load = [&](int j, int kb) {
        a[j] = __ldg(sw0 + kb);
        b[j] = __ldg(sw1 + kb);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[j][i] = lane + 32 * i < t.rows ? __ldg(sx + i * step + kb) : 0.f;
      };
      load(0, wk.lo);
#pragma unroll 1
      for (int kb = wk.lo; ok && kb < wk.hi; kb += 2) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (kb + j >= wk.hi) break;
          load(j ^ 1, min(kb + j + 1, wk.hi - 1));
          if (!(ok = warp_wait(&c.tempty[buf], tphase ^ 1, p.err, 6))) break;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            c.f[buf][lane + 32 * i] = make_float2(x[j][i] * a[j], x[j][i] * b[j]);
          __syncwarp();
          warp_arrive(&c.tfull[buf], lane);
          buf ^= 1;
          if (buf == 0) tphase ^= 1;
        }
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ scaling and epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsHigh));
    const int q = warp & 3, half = (warp - 4) >> 2, r = q * 32 + lane;
    uint8_t* box = out + (warp - 4) * 2 * kBox;
    int buf = 0, flip = 0;
    uint32_t tphase = 0, pphase = 0;
    bool ok = true;
    // the two warps of a lane quarter meet (bounded, as every wait)
    auto meet = [&]() -> bool {
      __syncwarp();
      warp_arrive(&c.pair[q], lane);
      const bool w = warp_wait(&c.pair[q], pphase, p.err, 5);
      pphase ^= 1;
      return w;
    };
    if (p.after != kAfterAny) pdl_wait();
    while (ok && wk.next()) {
      const Tile t = tile_of(c, n_act, wk.u);
      const int n0 = t.nt * (FUSED ? 128 : 256);
      const bool here = q * 32 < t.rows, mine = r < t.rows;
      const int NB = (p.N + 127) >> 7;
      float acc[128];   // 64 columns of the first weight tile, 64 of the second
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i] = 0.f;
      if (!here) {
        // no token of the tile on this warp's lanes: only pass the buffers on
        for (int kb = wk.lo; kb < wk.hi; ++kb) {
          if (!(ok = lead_wait(&c.tfull[buf], tphase, p.err, 4, lane))) break;
          warp_arrive(&c.tempty[buf], lane);
          buf ^= 1;
          if (buf == 0) tphase ^= 1;
        }
        continue;
      }
      bool early = false;
      for (int kb = wk.lo; kb < wk.hi; ++kb) {
        if (!(ok = warp_wait(&c.tfull[buf], tphase, p.err, 4, early))) break;
        tc_fence_after();
        const uint32_t ta = tmem + ((uint32_t)(q * 32) << 16) + buf * kAccCols + half * 64;
        // straight-line: a condition around any part of it makes the compiler copy the
        // accumulators every step.  (A missing second weight tile leaves old values in its
        // columns, which are never stored.)  The warp's two loads of 64 columns each cost a latency
        // that the other warp of the scheduler fills (loads of 32, the next in flight while one is
        // added: 2% slower); the buffer is handed back, and the next one tried, before the second
        // half is added.
        uint32_t v[64];
        tmem_ld64_nw(ta, v);
        const float2 f = c.f[buf][r];
        const uint64_t f0 = pack(f.x, f.x), f1 = pack(f.y, f.y);
        tmem_wait_ld();
        fma64(acc, v, f0);
        tmem_ld64_nw(ta + 128, v);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        warp_arrive(&c.tempty[buf], lane);
        buf ^= 1;
        if (buf == 0) tphase ^= 1;
        fma64<0, 24>(acc + 64, v, f1);
        early = mbar_test(&c.tfull[buf], tphase, lane);
        fma64<24, 32>(acc + 64, v, f1);
      }
      if (!ok) break;
      if (wk.lo > 0 || wk.hi < KB) {
        // a piece of the tile: its sums to this CTA's slot (0: begins inside the tile, 1: ends
        // inside it); the last piece's CTA adds them all in range order
        // (per warp 32 groups of 4 columns x 32 lanes: a store covers 512 bytes in a row)
        const size_t slot = (size_t)p.quarters * 2 * 1024;
        float4* part = reinterpret_cast<float4*>(p.part) + (size_t)(q * 2 + half) * 1024 + lane;
        if (mine) {
          float4* mp = part + ((size_t)blockIdx.x * 2 + (wk.lo > 0 ? 0 : 1)) * slot;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            __stcg(mp + 32 * i,
                   make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]));
        }
        const int first = wk.u * KB;
        const int c_lo = c.cut.owner(first), c_hi = c.cut.owner(first + KB - 1);
        // both warps' pieces are written (meet), then published by one release at GPU scope
        if (!(ok = meet())) break;
        if (half == 0 && lane == 0) {
          int32_t* ctr = p.counters + (size_t)wk.u * 4 + q;
          int before;
          asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;"
                       : "=r"(before)
                       : "l"(ctr)
                       : "memory");
          const int l = before == c_hi - c_lo;
          if (l) *ctr = 0;
          c.last[q] = l;
        }
        if (!(ok = meet())) break;
        if (!c.last[q]) continue;
        // (the first CTA's piece begins at the tile's first step: its slot 1; the others' inside)
        const int have = t.rows - q * 32;
        if (have <= kFewRows) {
          // few rows: row by row, a lane takes 4 of the warp's columns (lanes 0-15 of the first
          // weight tile, 16-31 of the second), sums them over the pieces, whose loads are in flight
          // together, and finishes them; a lane per row would leave the others idle for it
          for (int l = 0; ok && l < have; ++l) {
            const float4* op = part - lane + 32 * lane + l;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
            for (int cc = c_lo; cc <= c_hi; ++cc) {
              const float4 o = __ldcg(op + ((size_t)cc * 2 + (cc > c_lo ? 0 : 1)) * slot);
              s.x += o.x;
              s.y += o.y;
              s.z += o.z;
              s.w += o.w;
            }
            const size_t row = (size_t)t.r0 + q * 32 + l;
            if (FUSED) {
              const float4 u = make_float4(__shfl_down_sync(0xffffffffu, s.x, 16),
                                           __shfl_down_sync(0xffffffffu, s.y, 16),
                                           __shfl_down_sync(0xffffffffu, s.z, 16),
                                           __shfl_down_sync(0xffffffffu, s.w, 16));
              s = make_float4(silu_mul(s.x, u.x), silu_mul(s.y, u.y), silu_mul(s.z, u.z),
                              silu_mul(s.w, u.w));
              float m = lane < 16 ? fmaxf(fmaxf(fabsf(s.x), fabsf(s.y)),
                                          fmaxf(fabsf(s.z), fabsf(s.w)))
                                  : 0.f;
#pragma unroll
              for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
              if (lane == 0) c.amax[flip][half][q * 32] = m;
              if (!(ok = meet())) break;
              m = fmaxf(fmaxf(c.amax[flip][0][q * 32], c.amax[flip][1][q * 32]), kFp8MinAmax);
              flip ^= 1;
              if (lane < 16)
                *reinterpret_cast<uint32_t*>(p.hq + row * p.N + n0 + 64 * half + 4 * lane) =
                    fp8_pack4(s.x, s.y, s.z, s.w, __fdiv_rn(kFp8Max, m));
              if (lane == 0 && half == 0) p.hs[row * NB + (n0 >> 7)] = __fdiv_rn(m, kFp8Max);
            } else {
              const int col = n0 + 128 * (lane >> 4) + 64 * half + 4 * (lane & 15);
              const float v[4] = {s.x, s.y, s.z, s.w};
              if (p.y_f32) {
                float* y = static_cast<float*>(p.y) + row * p.N + col;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  if (col + j < p.N) y[j] = v[j];
              } else {
                uint16_t* y = static_cast<uint16_t*>(p.y) + row * p.N + col;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  if (col + j < p.N) y[j] = float_to_bf16_bits(v[j]);
              }
            }
          }
          if (!ok) break;
          continue;
        } else {
#pragma unroll
          for (int i = 0; i < 128; ++i) acc[i] = 0.f;
          for (int cc = c_lo; mine && cc <= c_hi; ++cc) {
            const float4* op = part + ((size_t)cc * 2 + (cc > c_lo ? 0 : 1)) * slot;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float4 o = __ldcg(op + 32 * i);
              acc[4 * i] += o.x;
              acc[4 * i + 1] += o.y;
              acc[4 * i + 2] += o.z;
              acc[4 * i + 3] += o.w;
            }
          }
        }
      }
      const size_t row0 = (size_t)t.r0 + q * 32;     // the warp's first row, and how many exist
      const int have = t.rows - q * 32;
      if (FUSED) {
        // h over the gate sums; the row's largest |h| over both warps' 64 columns
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          acc[i] = silu_mul(acc[i], acc[64 + i]);
          m = fmaxf(m, fabsf(acc[i]));
        }
        c.amax[flip][half][r] = m;
        if (!(ok = meet())) break;
        m = fmaxf(fmaxf(m, c.amax[flip][half ^ 1][r]), kFp8MinAmax);
        flip ^= 1;
        const float inv = __fdiv_rn(kFp8Max, m);
        if (lane == 0) bulk_wait_read();
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float* h = acc + 16 * i + 4 * j;
            o[j] = fp8_pack4(h[0], h[1], h[2], h[3], inv);
          }
          *reinterpret_cast<uint4*>(box + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) =
              make_uint4(o[0], o[1], o[2], o[3]);
        }
        const int col = n0 + half * 64;
        store_box<64>(&p.tm_out, p.hq + row0 * p.N + col, p.N, box, col, (int)row0, have, 64, lane);
        __syncwarp();
        if (mine && half == 0) p.hs[(row0 + lane) * NB + (n0 >> 7)] = __fdiv_rn(m, kFp8Max);
      } else {
        if (p.y_f32) store_y<true>(p, box, acc, (int)row0, n0, half, have, lane);
        else store_y<false>(p, box, acc, (int)row0, n0, half, have, lane);
      }
    }
    if (lane == 0) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols));
  }
}

// Zeroes a product's control words.  A kernel, not a memset: the product's CTAs start beside it
// (one row x 7168 x 4096: with a memset before the product 20 us, this way 17).
__global__ void __launch_bounds__(256) clear_kernel(uint4* words, int n) {
  pdl_trigger();
  for (int i = threadIdx.x; i < n; i += 256) words[i] = make_uint4(0, 0, 0, 0);
}

// Map of byte rows [rows][K] with boxes of box_rows x 128 bytes, 128-byte swizzle; reads past K
// or the last row give zeros, writes there are dropped.  elem: bytes of an element (what
// coordinates count in); box_bytes = 64: 64-byte rows and swizzle.
bool encode_rows(CUtensorMap* m, const void* base, size_t K, size_t rows, int box_rows,
                 int elem = 1, int box_bytes = 128) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)(K * elem)};
  cuuint32_t box[2] = {(cuuint32_t)(box_bytes / elem), (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(m,
             elem == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                       : elem == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                   : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
             2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

template <bool FUSED, bool PLAIN>
int launch_variant(const Fp8Params& p, cudaStream_t st) {
  static bool attr = false;
  if (!attr) {
    MOE_CUDA_TRY(cudaFuncSetAttribute(fp8_gemm_kernel<FUSED, PLAIN>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem));
    attr = true;
  }
  if (p.after != kAfterAny) {
    // scheduled as the CTAs of the kernel before it end (see pdl_wait in the kernel)
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(sm_count());
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, fp8_gemm_kernel<FUSED, PLAIN>, p));
  } else {
    MOE_LAUNCH_PDL((fp8_gemm_kernel<FUSED, PLAIN>), dim3(sm_count()), dim3(kThreads), kSmem, st, p);
  }
  MOE_COUNT_LAUNCH();
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace

// lane quarters a tile can fill
static int quarters_of(int max_rows) { return ceil_div(std::min(std::max(max_rows, 1), 128), 32); }

int launch_clear(void* words, size_t bytes, cudaStream_t st) {
  clear_kernel<<<1, 256, 0, st>>>(static_cast<uint4*>(words), (int)(bytes / 16));
  MOE_COUNT_LAUNCH();
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

Fp8Plan plan_fp8(const Fp8Args& a) {
  Fp8Plan pl{};
  const int G = sm_count();
  pl.part_elems = (size_t)G * 2 * quarters_of(a.max_rows) * 2 * 4096;
  pl.counter_elems = (size_t)4 * kRangeTiles * G;
  return pl;
}

int launch_fp8(const Fp8Args& a, float* part, int32_t* counters, int32_t* err, cudaStream_t st) {
  if (a.max_rows <= 0 || a.host_n == 0) return MOE_OK;
  if (!encode_fn()) return MOE_ERR_UNSUPPORTED;
  Fp8Params p{};
  if (!encode_rows(&p.tm_x, a.xq, a.K, a.max_rows, 128) ||
      !encode_rows(&p.tm_x32, a.xq, a.K, a.max_rows, 32) ||
      (a.w && !encode_rows(&p.tm_w, a.w, a.K, (size_t)a.E * a.N, 128)))
    return MOE_ERR_INVALID_ARG;
  const int elem = a.fused ? 1 : a.y_f32 ? 4 : 2;
  if ((size_t)a.N * elem % 16 == 0 &&
      !encode_rows(&p.tm_out, a.fused ? a.hq : a.y, a.N, a.max_rows, 32, elem, a.fused ? 64 : 128))
    return MOE_ERR_INVALID_ARG;
  p.xs = a.xs; p.offsets = a.offsets; p.E = a.E; p.N = a.N; p.K = a.K;
  p.KB = ceil_div(a.K, 128); p.NT = a.fused ? a.N / 128 : ceil_div(a.N, 256);
  p.max_rows = a.max_rows; p.quarters = quarters_of(a.max_rows);
  if (a.tab) p.tab = *a.tab;
  p.dev_tab = a.dev_tab; p.w_off = a.w_off; p.s_off = a.s_off; p.ws = a.ws;
  p.active = a.active; p.n_active = a.n_active; p.host_n = a.host_n;
  for (int i = 0; i < (a.host_n > 0 ? a.host_n : 0); ++i) p.host_ids[i] = (int16_t)a.host_ids[i];
  p.hq = a.hq; p.hs = a.hs; p.y = a.y; p.y_f32 = a.y_f32; p.after = a.after;
  p.part = part; p.counters = counters; p.err = err;
  if (a.fused) return launch_variant<true, false>(p, st);
  return a.w ? launch_variant<false, true>(p, st) : launch_variant<false, false>(p, st);
}

}  // namespace moe
