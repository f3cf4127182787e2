// Products grouped by expert (include/moe_operators.h: moe_grouped_matmul,
// moe_grouped_matmul_fp4).
//
// The product is computed transposed: the weights are the M operand, the tokens the N
// operand, D[feature, token].  A CTA (CG = 1) or a pair of CTAs (CG = 2) multiplies 128 or
// 256 weight rows by up to 128 or 256 tokens of one expert.  An expert's last, ragged
// tile then costs only the columns it has (N is a multiple of 16 or 32 per
// instruction), and one decoded token costs 16 columns, not 128 rows.
//
// Persistent kernel, one CTA per SM:
//   warp 0       TMA: weight tiles, into a ring of K slices of 128 bytes a row
//   warp 1       one lane issues tcgen05.mma: kind::f16 (bf16) or the block-scaled 4-bit
//                kinds, whose scales go from shared memory to TMEM by tcgen05.cp first
//   warp 2       TMA: token tiles, or rows gathered four at a time by index
//   warp 3       TMA: 4-bit scale tiles
//   warps 4-7    with 4-bit SwiGLU, the weights' scales into the order of the rows (below)
//   warps 8-15   epilogue, two warps to a quarter of the TMEM lanes
// The issuing lane is picked by elect.sync in a converged warp: where the compiler has to
// allow for several lanes it issues each load, copy and product through a loop over lanes
// (16384 rows of 32 experts, K 7168, N 4096, NVFP4: 391 us from lane 0, 196 elected).
// Two accumulators in TMEM let the epilogue of a tile run under the products of the next.
// Two of 256 columns leave no room for 4-bit scales, so those of 4-bit pairs overlap by 64
// columns, which the epilogue reads first and then lets the next tile begin.
//
// SwiGLU: the weight rows of a tile alternate 16 gate rows and the 16 up rows of the same
// features (one 5-dimensional tensor map does it), so the two halves of a warp's TMEM lanes
// hold gate and up of one feature, and tcgen05.ld gives both to one thread.  A
// 16- or 32-element block of the result is requantised after a turn through shared memory.
//
// Every wait is bounded; one that runs out sets the flag moe_operators_check() reads.
#include "operators.cuh"
#include "tc.cuh"

#include <cudaTypedefs.h>

#include <algorithm>

namespace moe {

namespace {

using namespace tc;

__device__ uint32_t g_operator_err;

constexpr int FIRST_SORT = 4, FIRST_EPI = 8, EW = 8;           // EW epilogue warps (16 lose a stage of the ring and are slower)
constexpr int THREADS = 32 * (FIRST_EPI + EW);
constexpr int A_BYTES = 128 * 128;             // 128 weight rows, 128 bytes of K each
constexpr int MAX_STAGES = 12;
constexpr int TMEM_COLS = 512;
constexpr int TMEM_SCALES = 448, SCALE_SLOTS = 5;   // 12-column slots of block scales, a group of 4 blocks each, used in turn:
                                               // 4 columns of the weights' (128 rows), 8 of the tokens'
// An epilogue warp's buffer, 32 tokens: rows of 32 bf16 features, or 16 (SwiGLU), or 16 fp32 ones (requantising), with strides
// that reach all banks.  A warp needs no other, so that it waits for none.
constexpr int EPI_WARP = 32 * 80, ROW32 = 80, ROW16 = 48, ROW16F = 20 /* floats */;
constexpr int SUM_SLICES = 4;                  // fp32 results: K slices summed in TMEM before they are added in registers
constexpr int SMEM_LIMIT = 227 * 1024;

struct ProductArgs {
  int P, E, N, K, k, cols, groups, gw_count, act, gather, quant, wide, few;
  int m_blocks, kslices, stages, stage_bytes, b_rows, w_tiles, w_parts;   // w_parts: scale tiles one weight tile's rows are in
  int most_tiles;                // token tiles that P rows of E experts can make
  int64_t pad_rows;              // rows of the scale tiles that grouped rows have
  const float *gx, *gw, *g_out;
  const int32_t *offsets, *order;
  void* out;
  uint8_t *out_codes, *out_scales;
  const int32_t* tiles;
};

// expert, first grouped row, rows, weight block, scale tile of row0; tt: token tile, of all experts
struct Item { int e, row0, n, mb, tile, tt; };

template <int FMT, int CG>
struct Shape4 {
  static constexpr bool FP4 = FMT != MOE_BF16, NV = FMT == MOE_NVFP4;
  static constexpr int NMAX = 128 * CG;                 // tokens of a tile
  static constexpr int KS = FP4 ? 256 : 64;             // K of a slice
  static constexpr int KI = FP4 ? 64 : 16;              // K of an instruction
  static constexpr int GS = NV ? 4 : 2;                 // scale groups of a slice
  static constexpr int TILE_SCALES = GS * 512;          // bytes of a slice's scales of 128 rows
  // TMEM column of the second accumulator.  4-bit pairs: the two overlap in 64 columns, to leave room for the scales
  static constexpr int ACC_COLS = CG == 1 ? 128 : FP4 ? 192 : 256;
  static constexpr bool OVERLAP = FP4 && CG == 2;
  static constexpr bool GATHER = !FP4 && CG == 1;       // has the form for gathered rows
  static constexpr int BOX = 16 * CG;                   // token rows of a small load; a tile's 128 rows take one
};

// where expert e's rows start, whatever the offsets hold: a row number of the call's, or P
__device__ __forceinline__ int row_at(const ProductArgs& a, int e) { return min(max(__ldg(a.offsets + e), 0), a.P); }

// item `it` into o, which holds the one before (tt = -1: none)
template <int FMT, int CG>
__device__ __forceinline__ void item_at(const ProductArgs& a, const int32_t* first, int it, Item& o) {
  using S = Shape4<FMT, CG>;
  const int tt = it / a.m_blocks;
  o.mb = it - tt * a.m_blocks;
  if (tt == o.tt) return;
  o.tt = tt;
  int lo = 0, hi = a.E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= tt) lo = mid;
    else hi = mid;
  }
  o.e = lo;
  const int j = tt - first[lo], r0 = row_at(a, lo), n = max(row_at(a, lo + 1), r0) - r0;
  int chunk = S::NMAX;
  if constexpr (!S::FP4) {
    // even shares; 4-bit tiles start on their scales' 128-row tiles
    const int nt = first[lo + 1] - first[lo];
    chunk = min(S::NMAX, ((n + nt - 1) / nt + 16 * CG - 1) / (16 * CG) * (16 * CG));
  }
  o.row0 = r0 + j * chunk;
  o.n = min(chunk, n - j * chunk);
  o.tile = S::FP4 ? __ldg(a.tiles + lo) + j * CG : 0;
}

// token columns of a tile, and the rows of them that one CTA loads
template <int CG>
__device__ __forceinline__ int columns(int n) { return (n + 16 * CG - 1) / (16 * CG) * (16 * CG); }
template <int FMT, int CG>
__device__ __forceinline__ int token_rows(const ProductArgs& a, const Item& o) {
  using S = Shape4<FMT, CG>;
  const int mine = columns<CG>(o.n) / CG;
  if (S::GATHER && a.gather) return (o.n + 3) & ~3;   // single CTAs; the columns past the rows are not used
  return a.b_rows == 128 && mine > 3 * S::BOX ? 128 : (mine + S::BOX - 1) / S::BOX * S::BOX;
}

// The products of one K slice (descriptors da, db, ds of its weights, tokens and scales); `left`: the K that is there when
// the slice is not FULL.  Scales take the TMEM slots from `slot` on, so that copies do not wait for the last products.
template <int FMT, int CG, bool FULL>
__device__ __forceinline__ void issue_slice(uint32_t d, uint32_t tmem, uint64_t da, uint64_t db, uint64_t ds, uint32_t idesc, bool second,
                                            uint32_t acc, int left, uint32_t slot) {
  using S = Shape4<FMT, CG>;
  if constexpr (S::FP4) {
    uint32_t ts[S::GS];
#pragma unroll
    for (int g = 0; g < S::GS; ++g) {
      if (!FULL && g * (S::KS / S::GS) >= left) break;
      ts[g] = tmem + TMEM_SCALES + 12u * slot;
      if (++slot == SCALE_SLOTS) slot = 0;
      copy_scales<CG>(ts[g], ds + ((CG * S::TILE_SCALES) >> 4) + 32 * g);
      copy_scales<CG>(ts[g] + 4, ds + 32 * g);
      if (CG == 2 && second) copy_scales<CG>(ts[g] + 8, ds + (S::TILE_SCALES >> 4) + 32 * g);
    }
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      if (!FULL && kk * S::KI >= left) break;
      const uint32_t g = S::NV ? kk : kk >> 1, id = S::NV ? 0u : 2u * (kk & 1);
      mma_fp4<CG, S::NV>(d, da + 2 * kk, db + 2 * kk, idesc | (id << 4) | (id << 29), ts[g], ts[g] + 4, acc | (uint32_t)kk);
    }
  } else {
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      if (!FULL && kk * S::KI >= left) break;
      mma_bf16<CG>(d, da + 2 * kk, db + 2 * kk, idesc, acc | (uint32_t)kk);
    }
  }
}

// h[j] = silu(gate[j] g) * up[j] g of two values; e = -g log2 e.  exp by ex2.approx and one rcp.approx for both quotients
// (1 / a = b / (a b); the special function unit is what an epilogue of short K waits for).  Two units each, and the rounded
// argument adds |gate g| units: far inside bf16 and 4-bit results (fp32 ones: silu below).
// Past 2^60 the exponential stays there: silu is then below 1e-16 of the gate.
__device__ __forceinline__ void swiglu2(uint32_t gate0, uint32_t gate1, uint32_t up0, uint32_t up1, float g, float e, float& h0, float& h1) {
  const float a = __uint_as_float(gate0), b = __uint_as_float(gate1);
  float x, y, r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(x) : "f"(fminf(a * e, 60.0f)));
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(fminf(b * e, 60.0f)));
  x += 1.0f;
  y += 1.0f;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x * y));
  h0 = a * g * (r * y) * (__uint_as_float(up0) * g);
  h1 = b * g * (r * x) * (__uint_as_float(up1) * g);
}

// silu(x) = x / (1 + exp(-x)) of fp32 results, within ten half units.  exp(-x) = 2^t 2^r with t the rounded product -x log2 e and r
// what the rounding and log2 e's own have left out, |r| < 2^-16: 2^r = 1 + r ln 2.  (65536 rows of 128 experts, K 768, N 2048,
// MXFP4, fp32 results: 195 us, with expf and a division 293.)  Past -128 the exponential is infinite all the same, past 128 it is 0.
__device__ __forceinline__ float silu(float x) {
  constexpr double log2e = 1.4426950408889634;
  constexpr float near = (float)log2e, rest = (float)(log2e - (double)near);   // in two parts, as Cody and Waite have it
  const float c = fminf(fmaxf(x, -128.0f), 128.0f), t = c * -near, r = fmaf(c, -near, -t) - c * rest;
  float e;
  asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(t));
  if (e < INFINITY) e = fmaf(e, r * 0.693147181f, e);
  return __fdividef(x, 1.0f + e);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_bf16(uint32_t a, uint32_t b, float g) { return pack_bf16(__uint_as_float(a) * g, __uint_as_float(b) * g); }
__device__ __forceinline__ void store_one(const ProductArgs& a, size_t at, float v) { static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v); }

// The epilogue of fp32 results, times g.  The tensor cores truncate what they add to an accumulator: bf16 operands over K = 1944 are
// 2e-6 off, where fp32 additions that round leave 1e-7; 4-bit ones whose block scales vary by e^2 are 3e-6 off over K = 7168.  So an
// accumulator holds SUM_SLICES slices only (16 additions), and this adds them up in registers: 64 columns a warp, with the
// registers of the single-CTA form's 128.  false: a wait has run out.
template <bool FP4>
__device__ __forceinline__ bool exact_tile(const ProductArgs& a, const Item& o, float g, uint32_t tmem, uint32_t tfull, uint32_t tempty, int& acc,
                                           uint32_t& acc_phase, volatile int* abort_flag, int q, int part) {
  const int lane = threadIdx.x & 31;
  float lo[2][16] = {}, hi[2][16] = {};
  for (int k0 = 0; k0 < a.kslices; k0 += SUM_SLICES) {
    if (!warp_wait(tfull + 8 * acc, acc_phase, abort_flag)) {
      if (lane == 0) { *abort_flag = 1; atomicOr(&g_operator_err, 1u); }
      return false;
    }
    fence_after();
    const uint32_t tbase = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(acc * 128 + 64 * part);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (64 * part + 32 * h >= o.n) continue;
      uint32_t x[16], y[16];
      tmem_ld16x4(tbase + 32 * h, x);
      tmem_ld16x4(tbase + (16u << 16) + 32 * h, y);
      tmem_ld_wait(x, y);
#pragma unroll
      for (int i = 0; i < 16; ++i) { lo[h][i] += __uint_as_float(x[i]); hi[h][i] += __uint_as_float(y[i]); }
    }
    fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(tempty + 8 * acc);
    if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i0 = 0; i0 < 16; i0 += 4) {
      const int t0 = 64 * part + 32 * h + 2 * i0;
      if (t0 >= o.n) continue;   // eight tokens, of all lanes
#pragma unroll
      for (int i = i0; i < i0 + 4; ++i) {
        const int t = t0 + 2 * (lane & 3) + (i & 1), f = (lane >> 2) + 4 * (i & 2);
        float* out = static_cast<float*>(a.out) + (size_t)(o.row0 + t) * a.cols;
        const float x = FP4 ? lo[h][i] * g : lo[h][i], y = FP4 ? hi[h][i] * g : hi[h][i];
        if (a.act) {
          const int c = o.mb * 64 + 16 * q + f;
          const float v = silu(x) * y;
          if (t < o.n && c < a.cols) out[c] = v;
        } else {
          const int c = o.mb * 128 + 32 * q + f;
          if (t < o.n && c < a.cols) out[c] = x;
          if (t < o.n && c + 16 < a.cols) out[c + 16] = y;
        }
      }
    }
  return true;
}

// EXACT (CG = 1): fp32 results
template <int FMT, int CG, bool EXACT>
__global__ void __launch_bounds__(THREADS, 1)
product_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
               const __grid_constant__ CUtensorMap tmXall, const __grid_constant__ CUtensorMap tmSW, const __grid_constant__ CUtensorMap tmSX, const ProductArgs a) {
  using S = Shape4<FMT, CG>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const uint32_t ring = smem_u32(smem);
  uint8_t* tail = smem + (size_t)a.stages * a.stage_bytes;
  uint8_t* ebuf = tail;
  tail += EW * EPI_WARP + 1024;   // and the block maxima of requantised MXFP4
  const uint32_t full = smem_u32(tail), empty = full + 8 * MAX_STAGES, sfull = empty + 8 * MAX_STAGES, tfull = sfull + 8 * MAX_STAGES,
                 tempty = tfull + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail + 24 * MAX_STAGES + 32);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* gathered = reinterpret_cast<int32_t*>(tail + 24 * MAX_STAGES + 48);   // sources of a tile's 128 token rows
  int32_t* first = gathered + 128;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  const bool sorts = S::FP4 && a.act;   // warps 4 on sort the weights' scales
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(full + 8 * s, 1 + (sorts ? CG * S::GS : 0));
      mbar_init(empty + 8 * s, 1);
      mbar_init(sfull + 8 * s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(tfull + 8 * s, 1);
      mbar_init(tempty + 8 * s, EW * CG);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc<CG>(smem_u32(tmem_slot), TMEM_COLS);
  pdl_wait();
  pdl_trigger();
  if (warp == 2) {   // token tiles before each expert
    int run = 0;
    for (int b = 0; b < a.E; b += 32) {
      const int e = b + lane;
      const int c = e < a.E ? (max(row_at(a, e + 1) - row_at(a, e), 0) + S::NMAX - 1) / S::NMAX : 0;
      int x = c;
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += v;
      }
      // offsets that do not ascend could make more tiles than the rows do
      if (e < a.E) first[e] = min(run + x - c, a.most_tiles);
      run = min(run + __shfl_sync(0xffffffffu, x, 31), a.most_tiles);
    }
    if (lane == 0) first[a.E] = run;
  }
  fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  const int total = first[a.E] * a.m_blocks;
  // Every so many-th item, which mixes long and short tiles and lets neighbours share a token tile.  With few rows an expert, when
  // an item costs its weights: a run of items, mostly weight blocks of one token tile (16 tokens, K 768: 17.7 -> 15.2 us; with
  // 512 rows an expert runs read the weights again for every token tile, 500 -> 1090 us).
  const int units = gridDim.x / CG, unit = blockIdx.x / CG, share = total / units, more = total % units;
  const bool runs = CG == 1 && a.few;
  const int step = runs ? 1 : units, it0 = runs ? unit * share + min(unit, more) : unit;
  const int it1 = runs ? it0 + share + (unit < more) : total;
  Item o;
  o.tt = -1;

  if (warp == 0) {
    // ---------------- loads ----------------
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int it = it0; it < it1 && ok; it += step) {
      item_at<FMT, CG>(a, first, it, o);
      const int m = o.mb * CG + (int)rank;      // 128-row weight tile (64 gate + 64 up with SwiGLU)
      const uint32_t bytes = (uint32_t)CG * (A_BYTES + 128u * token_rows<FMT, CG>(a, o) + (S::FP4 ? (uint32_t)S::TILE_SCALES * (CG + (a.act ? 0 : 1)) : 0u));
      for (int ks = 0; ks < a.kslices; ++ks) {
        if (!warp_wait(empty + 8 * stage, phase ^ 1u, abort_flag)) { ok = false; break; }
        if (elect_one()) {
          const uint32_t bar = CG == 2 ? in_rank(full + 8 * stage, 0) : full + 8 * stage;
          if (rank == 0) mbar_expect(full + 8 * stage, bytes);
          // rows of one expert (dimensions K, row, expert), or with SwiGLU (K, 16 rows, gate / up, block of 16, expert)
          tma_5d<CG>(&tmW, bar, ring + stage * a.stage_bytes, ks * (S::FP4 ? 128 : 64), a.act ? 0 : 128 * m, 0, a.act ? 4 * m : 0, o.e);
        }
        if (++stage == a.stages) { stage = 0; phase ^= 1u; }
      }
    }
    if (!ok) {
      if (lane == 0) { *abort_flag = 1; atomicOr(&g_operator_err, 1u); }
      // copies in flight land long before this bound
      const unsigned long long t0 = gtimer();
      while (gtimer() - t0 < 1000000ull) {
      }
    }
    // every slice has been used, and no arrival on this CTA's barriers is outstanding, before it ends
    for (int i = 0; i < a.stages && ok; ++i) {
      ok = warp_wait(empty + 8 * stage, phase ^ 1u, abort_flag);
      if (++stage == a.stages) { stage = 0; phase ^= 1u; }
    }
  } else if (warp == 1) {
    // ---------------- products ----------------
    if (rank == 0) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0, slot = 0;
      bool ok = true;
      const int sum = EXACT ? SUM_SLICES : a.kslices;   // slices of an accumulator
      const uint64_t da = desc_sw128(ring), db = desc_sw128(ring + A_BYTES), ds = desc_scales(ring + A_BYTES + a.b_rows * 128);
      for (int it = it0; it < it1 && ok; it += step) {
        item_at<FMT, CG>(a, first, it, o);
        const int ncols = columns<CG>(o.n);
        // D fp32; bf16 operands, or e2m1 with e4m3 / e8m0 scales; both K-major; N; M = 128 CG
        const uint32_t idesc = ((uint32_t)(ncols >> 3) << 17) | ((uint32_t)(8 * CG) << 24) |
                               (S::FP4 ? (1u << 7) | (1u << 10) | (S::NV ? 0u : 1u << 23) : (1u << 4) | (1u << 7) | (1u << 10));
        for (int k0 = 0; k0 < a.kslices && ok; k0 += sum) {
          // overlapping accumulators: the tile before this one has let go of the overlap; otherwise: the one before that is read
          if (!warp_wait(tempty + (S::OVERLAP ? 0 : 8 * acc), S::OVERLAP ? (uint32_t)acc ^ 1u : acc_phase ^ 1u, abort_flag)) { ok = false; break; }
          fence_after();
          const uint32_t d = tmem + (uint32_t)(acc * S::ACC_COLS);
          const int k1 = min(a.kslices, k0 + sum);
          for (int ks = k0; ks < k1; ++ks) {
            if (!warp_wait(full + 8 * stage, phase, abort_flag)) { ok = false; break; }
            fence_after();
            const uint64_t at = (uint32_t)(stage * a.stage_bytes) >> 4;
            const int left = a.K - ks * S::KS;
            if (elect_one()) {
              if (left >= S::KS) issue_slice<FMT, CG, true>(d, tmem, da + at, db + at, ds + at, idesc, o.n > 128, ks - k0, 0, slot);
              else issue_slice<FMT, CG, false>(d, tmem, da + at, db + at, ds + at, idesc, o.n > 128, ks - k0, left, slot);
              commit<CG>(empty + 8 * stage);
            }
            __syncwarp();
            slot = (slot + S::GS) % SCALE_SLOTS;
            if (++stage == a.stages) { stage = 0; phase ^= 1u; }
          }
          if (!ok) break;
          if (elect_one()) commit<CG>(tfull + 8 * acc);
          __syncwarp();
          if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
        }
      }
      if (!ok && lane == 0) { *abort_flag = 1; atomicOr(&g_operator_err, 1u); }
    }
  } else if (warp == 2) {
    // ---------------- tokens ----------------
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int it = it0; it < it1 && ok; it += step) {
      item_at<FMT, CG>(a, first, it, o);
      const int row0 = o.row0 + (int)rank * (columns<CG>(o.n) / CG), rows = token_rows<FMT, CG>(a, o);
      if (S::GATHER && a.gather) {
        __syncwarp();
        for (int r = lane; r < rows; r += 32) gathered[r] = min(max(__ldg(a.order + row0 + min(r, o.n - 1)) / a.k, 0), a.P / a.k - 1);
        __syncwarp();
      }
      for (int ks = 0; ks < a.kslices; ++ks) {
        if (!warp_wait(empty + 8 * stage, phase ^ 1u, abort_flag)) { ok = false; break; }
        const uint32_t sb = ring + stage * a.stage_bytes + A_BYTES;
        const uint32_t bar = CG == 2 ? in_rank(full + 8 * stage, 0) : full + 8 * stage;
        const int x = ks * (S::FP4 ? 128 : 64);
        if (S::GATHER && a.gather) {
          if (elect_one()) {
#pragma unroll 4
            for (int r = 0; r < rows; r += 4)
              tma_gather4<CG>(&tmX, bar, sb + 128 * r, x, *reinterpret_cast<const int4*>(gathered + r));
          }
        } else if (elect_one()) {
          if (a.b_rows == 128 && rows == 128) tma_2d<CG>(&tmXall, bar, sb, x, row0);
          else
            for (int r = 0; r < rows; r += S::BOX) tma_2d<CG>(&tmX, bar, sb + r * 128, x, row0 + r);
        }
        if (++stage == a.stages) { stage = 0; phase ^= 1u; }
      }
    }
    if (!ok && lane == 0) { *abort_flag = 1; atomicOr(&g_operator_err, 1u); }
  } else if (S::FP4 && warp == 3) {
    // ---------------- scale tiles: the tokens' (CG of them), then the weights' ----------------
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int it = it0; it < it1 && ok; it += step) {
      item_at<FMT, CG>(a, first, it, o);
      const int m = o.mb * CG + (int)rank;
      const int wt = o.e * a.w_tiles + (a.act ? m >> 1 : m), ut = o.e * a.w_tiles + ((a.cols + 64 * m) >> 7);
      for (int ks = 0; ks < a.kslices; ++ks) {
        if (!warp_wait(empty + 8 * stage, phase ^ 1u, abort_flag)) { ok = false; break; }
        if (elect_one()) {
          const uint32_t ss = ring + stage * a.stage_bytes + A_BYTES + a.b_rows * 128, sw = ss + CG * S::TILE_SCALES;
          const uint32_t bar = CG == 2 ? in_rank(full + 8 * stage, 0) : full + 8 * stage;
          tma_3d<CG>(&tmSX, bar, ss, 0, ks * S::GS, o.tile);
          if (!a.act) {
            tma_3d<CG>(&tmSW, bar, sw, 0, ks * S::GS, wt);
          } else {   // the tile of the gate rows, and the one or two of the up rows
            mbar_expect(sfull + 8 * stage, a.w_parts * S::TILE_SCALES);
            tma_3d<1>(&tmSW, sfull + 8 * stage, sw, 0, ks * S::GS, wt);
            for (int i = 1; i < a.w_parts; ++i) tma_3d<1>(&tmSW, sfull + 8 * stage, sw + i * S::TILE_SCALES, 0, ks * S::GS, ut + i - 1);
          }
        }
        if (++stage == a.stages) { stage = 0; phase ^= 1u; }
      }
    }
    if (!ok && lane == 0) { *abort_flag = 1; atomicOr(&g_operator_err, 1u); }
  } else if (warp < FIRST_EPI) {
    // ---------------- 4-bit SwiGLU: a group of blocks a warp, the weights' scales in the order of the tile's rows ----------------
    const int grp = warp - FIRST_SORT;
    if (sorts && grp >= 0 && grp < S::GS) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int it = it0; it < it1 && ok; it += step) {
        item_at<FMT, CG>(a, first, it, o);
        const int m = o.mb * CG + (int)rank;
        uint32_t src[4];   // where the scales of row lane + 32 j of the weight tile are
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = (lane >> 4) * a.cols + m * 64 + 16 * j + (lane & 15);
          const int part = lane < 16 ? 0 : 1 + (row >> 7) - ((a.cols + 64 * m) >> 7);
          src[j] = part * S::TILE_SCALES + (row & 31) * 16 + ((row >> 5) & 3) * 4;
        }
        for (int ks = 0; ks < a.kslices; ++ks) {
          if (!warp_wait(sfull + 8 * stage, phase, abort_flag)) { ok = false; break; }
          const uint32_t sw = ring + stage * a.stage_bytes + A_BYTES + a.b_rows * 128 + CG * S::TILE_SCALES + 512 * grp;
          uint32_t r[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) r[j] = lds32(sw + src[j]);
          __syncwarp();   // in place: the group's 512 bytes of the first tile have been read
          sts128(sw + 16 * lane, r);
          fence_async_proxy();
          __syncwarp();
          if (lane == 0) {
            if (CG == 2) mbar_arrive_cluster(in_rank(full + 8 * stage, 0));
            else mbar_arrive(full + 8 * stage);
          }
          if (++stage == a.stages) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok && lane == 0) { *abort_flag = 1; atomicOr(&g_operator_err, 1u); }
    }
  } else if (warp >= FIRST_EPI) {
    // ---------------- epilogue: a TMEM lane is a weight row, a column a token ----------------
    // quarter of the TMEM lanes; which 32 columns of each round; a round's columns
    const int q = warp & 3, part = (warp - FIRST_EPI) >> 2;
    constexpr int RC = 8 * EW, ROUNDS = S::NMAX / RC;
    uint8_t* const buf = ebuf + (4 * part + q) * EPI_WARP;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int it = it0; it < it1; it += step) {
      item_at<FMT, CG>(a, first, it, o);
      // what the tile needs from memory, on its way while the products run
      float g = 1.0f;
      if (S::FP4) g = (a.gx ? __ldg(a.gx) : 1.0f) * (a.gw ? __ldg(a.gw + (a.gw_count > 1 ? o.e : 0)) : 1.0f);
      if constexpr (EXACT) {
        if (!exact_tile<S::FP4>(a, o, g, tmem, tfull, tempty, acc, acc_phase, abort_flag, q, part)) break;
        continue;
      }
      const float go = S::NV && a.quant && a.g_out ? __ldg(a.g_out) : 1.0f, up = fabsf(go) < 1e-30f ? 0x1p64f : 1.0f;
      const float rgo = __frcp_rn(go * up), sixth = kSixth * up;
      const int64_t pad0 = !(S::FP4 && a.quant) ? 0
          : min(max((int64_t)__ldg(a.tiles + o.e) * 128 + (o.row0 - row_at(a, o.e)), (int64_t)0), a.pad_rows - o.n);
      bool ok = warp_wait(tfull + 8 * acc, acc_phase, abort_flag);
      if (S::FP4 && !S::NV && a.quant) ok = named_and(1 + part, 128, ok);   // these four warps wait for one another below
      if (!ok) {
        if (lane == 0) { *abort_flag = 1; atomicOr(&g_operator_err, 1u); }
        break;
      }
      fence_after();
      const int m = o.mb * CG + (int)rank;
      const uint32_t tbase = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(acc * S::ACC_COLS);
      bool released = false;
      auto release = [&]() {   // the accumulator (or the part the next one needs) has been read
        fence_before();
        __syncwarp();
        if (lane == 0) {
          const uint32_t bar = tempty + (S::OVERLAP ? 0 : 8 * acc);
          if (CG == 2) mbar_arrive_cluster(in_rank(bar, 0));
          else mbar_arrive(bar);
        }
      };
      // The overlap of the accumulators, columns 192 on of the first and 0 to 63 of the second, first.  A thread gets, of the
      // 16 rows of its quarter's first half (lo) and second half (hi), rows lane / 4 and 8 on, columns 2 (lane % 4) and 1 on of
      // every 8: [4 k + 2 (row >= 8) + column].
#pragma unroll 1
      for (int round = 0; round < ROUNDS; ++round) {
        const int c = 32 * part + (S::OVERLAP && acc == 0 ? ROUNDS - 1 - round : round) * RC;
        uint32_t lo[16], hi[16];
        const bool some = c < o.n;
        if (some) {
          tmem_ld16x4(tbase + c, lo);
          tmem_ld16x4(tbase + (16u << 16) + c, hi);
          tmem_ld_wait(lo, hi);
        }
        if (S::OVERLAP ? round == 0 : !released && ((round + 1) * RC >= o.n || round + 1 == ROUNDS)) { release(); released = true; }
        if (!some) continue;
        const int left = o.n - c;
        const int tok = 2 * (lane & 3), feat = lane >> 2;    // token and row of register 0
        __syncwarp();                                        // the last round's buffer has been read
        if (!a.act) {
          if (a.wide) {
            // bf16: 32 tokens of 32 features through shared memory, transposed 8 x 8 by stmatrix, 16 bytes a lane to memory
            const uint32_t to = smem_u32(buf) + (lane & 7) * ROW32 + (lane >> 3) * 16;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              stmatrix4_trans(to + 8 * k * ROW32, pack_bf16(lo[4 * k], lo[4 * k + 1], g), pack_bf16(lo[4 * k + 2], lo[4 * k + 3], g),
                              pack_bf16(hi[4 * k], hi[4 * k + 1], g), pack_bf16(hi[4 * k + 2], hi[4 * k + 3], g));
            __syncwarp();
            const int f = m * 128 + 32 * q + (lane & 3) * 8;
#pragma unroll
            for (int r = lane >> 2; r < 32; r += 8)
              if (r < left && f < a.cols)
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + (size_t)(o.row0 + c + r) * a.cols + f) =
                    *reinterpret_cast<const uint4*>(buf + r * ROW32 + (lane & 3) * 16);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const uint32_t v = i < 16 ? lo[i & 15] : hi[i & 15];
              const int t = tok + 8 * ((i & 15) >> 2) + (i & 1), f = m * 128 + 32 * q + feat + (i & 16) + 4 * (i & 2);
              if (t < left && f < a.cols) store_one(a, (size_t)(o.row0 + c + t) * a.cols + f, __uint_as_float(v) * g);
            }
          }
          continue;
        }
        // lo: gate rows, hi: the up rows of the same 16 features
        float h[16];
#pragma unroll
        for (int i = 0; i < 16; i += 2) swiglu2(lo[i], lo[i + 1], hi[i], hi[i + 1], g, -1.44269504f * g, h[i], h[i + 1]);
        if (a.wide) {
          // matrices: features 0-7 and 8-15 of eight tokens, then of the next eight
          const uint32_t to = smem_u32(buf) + ((lane & 7) + 8 * (lane >> 4)) * ROW16 + (lane & 8) * 2;
#pragma unroll
          for (int k = 0; k < 4; k += 2)
            stmatrix4_trans(to + 8 * k * ROW16, pack_bf16(h[4 * k], h[4 * k + 1]), pack_bf16(h[4 * k + 2], h[4 * k + 3]),
                            pack_bf16(h[4 * k + 4], h[4 * k + 5]), pack_bf16(h[4 * k + 6], h[4 * k + 7]));
          __syncwarp();
          const int f = m * 64 + 16 * q + (lane & 1) * 8;
#pragma unroll
          for (int r = lane >> 1; r < 32; r += 16)
            if (r < left && f < a.cols)
              *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + (size_t)(o.row0 + c + r) * a.cols + f) =
                  *reinterpret_cast<const uint4*>(buf + r * ROW16 + (lane & 1) * 16);
          continue;
        }
        if (!a.quant) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int t = tok + 8 * (i >> 2) + (i & 1), f = m * 64 + 16 * q + feat + 4 * (i & 2);
            if (t < left && f < a.cols) store_one(a, (size_t)(o.row0 + c + t) * a.cols + f, h[i]);
          }
          continue;
        }
        if constexpr (S::FP4) {
          // Through shared memory, so that a lane has a token's 16 features: an NVFP4 block, or half an MXFP4 one, whose other
          // half another warp of the four has.
          float* hb = reinterpret_cast<float*>(buf);
#pragma unroll
          for (int i = 0; i < 16; ++i) hb[(tok + 8 * (i >> 2) + (i & 1)) * ROW16F + feat + 4 * (i & 2)] = h[i];
          __syncwarp();
          float x[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 w = *reinterpret_cast<const float4*>(hb + lane * ROW16F + 4 * i);
            x[4 * i] = w.x; x[4 * i + 1] = w.y; x[4 * i + 2] = w.z; x[4 * i + 3] = w.w;
          }
          uint32_t top = 0u;
#pragma unroll
          for (int i = 0; i < 16; i += 2)
            top = __vimax3_u32(top, __float_as_uint(x[i]) & 0x7fffffffu, __float_as_uint(x[i + 1]) & 0x7fffffffu);
          if constexpr (!S::NV) {
            uint32_t* tops = reinterpret_cast<uint32_t*>(ebuf + EW * EPI_WARP) + part * 128;
            tops[32 * q + lane] = top;
            named_sync(1 + part, 128);
            top = max(top, tops[32 * (q ^ 1) + lane]);
            named_sync(1 + part, 128);
          }
          float st;
          uint32_t code = block_scale<S::NV, false>(top, go, rgo, st, sixth);
          const uint2 codes = encode16<S::NV, false>(x, top, code, st);
          const int f = m * 64 + 16 * q, og = (a.cols + (S::NV ? 63 : 127)) / (S::NV ? 64 : 128);
          if (lane < left) {
            if (f < a.cols) *reinterpret_cast<uint2*>(a.out_codes + (size_t)(o.row0 + c + lane) * (a.cols / 2) + f / 2) = codes;
            // blocks past the end pad their group
            const int block = S::NV ? f / 16 : f / 32;
            if (block < 4 * og && (S::NV || !(q & 1))) {
              uint8_t* s = a.out_scales + scale_at((size_t)(pad0 + c + lane), block, og);
              *s = (uint8_t)(f < a.cols ? code : 0u);
              if (!S::NV && f + 64 >= a.cols && !(m & 1)) s[2] = 0;      // the group's second half has no tile of its own
            }
          }
        }
      }
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  if (warp == 1) {
    fence_after();
    tmem_free<CG>(tmem, TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 get_encode() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

bool make_map(CUtensorMap* m, CUtensorMapDataType type, int rank, const void* base, const cuuint64_t* dims, const cuuint64_t* strides,
              const cuuint32_t* box, bool swizzle) {
  auto enc = get_encode();
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  return enc && enc(m, type, rank, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct ProductMem { const void *x, *w, *x_scales, *w_scales; int x_rows; };

template <int FMT, int CG, bool EXACT>
moe_status launch_tiles(ProductArgs a, const ProductMem& mem, cudaStream_t s) {
  using S = Shape4<FMT, CG>;
  const uint64_t row_bytes = S::FP4 ? (uint64_t)a.K / 2 : (uint64_t)a.K * 2;
  const uint64_t row_elems = S::FP4 ? (uint64_t)a.K / 2 : (uint64_t)a.K;
  const CUtensorMapDataType type = S::FP4 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint32_t kbox = S::FP4 ? 128 : 64;
  a.m_blocks = (int)ceil_div64(a.act ? a.cols : a.N, (a.act ? 64 : 128) * CG);
  a.kslices = (a.K + S::KS - 1) / S::KS;
  a.w_tiles = (a.N + 127) / 128;
  a.wide = !a.quant && !EXACT && a.cols % 8 == 0;   // rows of out start on 16 bytes
  // rows of the token area: what the largest tile of P rows can need
  a.b_rows = std::min(128, (a.P + 15) / 16 * 16);
  if (CG == 2) a.b_rows = 128;
  // SwiGLU: the 64 gate rows of a tile lie in one scale tile, the 64 up rows in one or two
  a.w_parts = !a.act ? 1 : a.cols % 64 ? 3 : 2;
  a.stage_bytes = A_BYTES + a.b_rows * 128 + (S::FP4 ? (CG + a.w_parts) * S::TILE_SCALES : 0);
  const int fixed = 1024 + EW * EPI_WARP + 1024 + 24 * MAX_STAGES + 48 + 512 + 4 * (a.E + 1);
  a.stages = std::min(MAX_STAGES, (SMEM_LIMIT - fixed) / a.stage_bytes);
  const size_t smem = (size_t)fixed + (size_t)a.stages * a.stage_bytes;

  CUtensorMap tw, tx, txall, tsw, tsx;
  bool ok;
  if (a.act) {
    const cuuint64_t dims[5] = {row_elems, 16, 2, (cuuint64_t)a.cols / 16, (cuuint64_t)a.E};
    const cuuint64_t strides[4] = {row_bytes, row_bytes * a.cols, row_bytes * 16, row_bytes * a.N};
    const cuuint32_t box[5] = {kbox, 16, 2, 4, 1};
    ok = make_map(&tw, type, 5, mem.w, dims, strides, box, true);
  } else {
    const cuuint64_t dims[5] = {row_elems, (cuuint64_t)a.N, 1, 1, (cuuint64_t)a.E};
    const cuuint64_t strides[4] = {row_bytes, row_bytes * a.N, row_bytes * a.N, row_bytes * a.N};
    const cuuint32_t box[5] = {kbox, 128, 1, 1, 1};
    ok = make_map(&tw, type, 5, mem.w, dims, strides, box, true);
  }
  {
    const cuuint64_t dims[2] = {row_elems, (cuuint64_t)mem.x_rows};
    const cuuint64_t strides[1] = {row_bytes};
    const cuuint32_t box[2] = {kbox, a.gather ? 1u : (cuuint32_t)S::BOX}, all[2] = {kbox, 128};
    ok = ok && make_map(&tx, type, 2, mem.x, dims, strides, box, true) && make_map(&txall, type, 2, mem.x, dims, strides, all, true);
  }
  tsw = tsx = tx;
  if (S::FP4) {
    const cuuint64_t strides[2] = {512, 512ull * a.groups};
    const cuuint32_t bw[3] = {128, (cuuint32_t)S::GS, 1}, bx[3] = {128, (cuuint32_t)S::GS, CG};
    const cuuint64_t dw[3] = {128, (cuuint64_t)a.groups, (cuuint64_t)a.E * a.w_tiles};
    const cuuint64_t dx[3] = {128, (cuuint64_t)a.groups, (cuuint64_t)moe_grouped_tiles(a.P, a.E)};
    ok = ok && make_map(&tsw, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, mem.w_scales, dw, strides, bw, false) &&
         make_map(&tsx, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, mem.x_scales, dx, strides, bx, false);
  }
  if (!ok) return fail(MOE_ECUDA, "cuTensorMapEncodeTiled failed");

  // at most every token tile the rows can make, on every weight block
  const int64_t tiles = (a.P + (int64_t)(S::NMAX - 1) * std::min(a.P, a.E)) / S::NMAX, most = tiles * a.m_blocks;
  if (most > 0x7fffffff) return fail(MOE_EINVAL, "P = %d rows of N = %d columns are too many tiles", a.P, a.N);
  a.most_tiles = (int)tiles;
  a.pad_rows = moe_grouped_tiles(a.P, a.E) * 128;
  static bool allowed[64] = {};   // the kernel's shared memory, once per device
  int dev = 0;
  CK(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return fail(MOE_EINVAL, "device %d is out of range", dev);
  if (!allowed[dev]) {
    CK(cudaFuncSetAttribute(product_kernel<FMT, CG, EXACT>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_LIMIT));
    allowed[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG;
  // every unit of a persistent grid has to be resident: as many pairs as the device's clusters allow
  int resident = operator_sms();
  if (CG == 2) {
    static int pairs[64] = {};
    if (!pairs[dev]) {
      int n = 0;
      cfg.gridDim = dim3(operator_sms() / 2 * 2);
      cfg.dynamicSmemBytes = SMEM_LIMIT;
      CK(cudaOccupancyMaxActiveClusters(&n, product_kernel<FMT, CG, EXACT>, &cfg));
      if (n < 1) return fail(MOE_ECUDA, "no CTA pair fits the device");
      pairs[dev] = n;
      cfg.dynamicSmemBytes = smem;
    }
    resident = pairs[dev];
  }
  const int units = (int)std::min<int64_t>(most, resident);
  cfg.gridDim = dim3(units * CG);
  CK(cudaLaunchKernelEx(&cfg, product_kernel<FMT, CG, EXACT>, tw, tx, txall, tsw, tsx, a));
  return MOE_OK;
}

// Pairs of CTAs load half of the tokens each and fewer, larger slices; single CTAs start sooner and have twice the units of work.
// us of gate/up (K 2048, N 1536, 128 experts), single and in pairs, by rows an expert: bf16 1 row 75.9 / 73.7, 4 rows 114.3 / 109.1,
// 64 rows 178.9 / 138.4; rows gathered (before the product for pairs, in it otherwise) 1 row 75.9 / 80.2, 4 rows 119.0 / 118.6,
// 16 rows 249.7 / 136.0; NVFP4 4 rows 38.0 / 40.1, 64 rows 49.1 / 50.4, 128 rows 66.8 / 56.2 (K 7168, N 4096, 64 rows 32.7 / 28.5).
// With the same rows for every expert: NVFP4 64 rows 47.1 / 47.0, 256 rows 81.5 / 60.4, MXFP4 45.0 / 45.1 and 78.0 / 57.8; two experts
// of 2048 x 2048 stay below a wave of SMs, where pairs only start later: 256 rows 6.6 / 8.4.
// fp32 results take single CTAs (exact_tile): NVFP4, 65536 rows of 128 experts, K 2048, N 1536 184 us, in pairs without the short
// sums 199; 16384 rows of 32 experts, K 7168, N 4096 327 and 195.
bool use_pairs(int64_t P, int64_t E, bool fp4) { return P >= (fp4 ? 64 : 4) * E; }

template <int FMT>
moe_status launch_product(ProductArgs a, const ProductMem& mem, bool exact, cudaStream_t s) {
  a.few = a.P < 64 * (int64_t)a.E;
  if (exact) return launch_tiles<FMT, 1, true>(a, mem, s);
  return use_pairs(a.P, a.E, FMT != MOE_BF16) ? launch_tiles<FMT, 2, false>(a, mem, s) : launch_tiles<FMT, 1, false>(a, mem, s);
}

// xs[place[t, j]] = x[t]: a row is read once and stored k times, two 16-byte units a lane of a warp's segment.  A token
// tile gathered inside the product, once for every weight block, costs more than this pass: 8192 tokens, 8 of 128 experts, K 2048,
// N 1536 take 280 us from rows in order and 327 with this pass; single CTAs 429 from rows in order and 1488 gathered by TMA.
constexpr int GATHER_THREADS = 256, GATHER_SEG = 64;
__global__ void __launch_bounds__(GATHER_THREADS)
gather_kernel(const uint4* __restrict__ x, const int32_t* __restrict__ place, int T, int row16, int k, int P, uint4* __restrict__ xs) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, c = blockIdx.y * GATHER_SEG + lane;
  for (int t = blockIdx.x * (GATHER_THREADS / 32) + (threadIdx.x >> 5); t < T; t += gridDim.x * (GATHER_THREADS / 32)) {
    uint4 v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (c + 32 * h < row16) v[h] = __ldg(x + (size_t)t * row16 + c + 32 * h);
    for (int j = 0; j < k; ++j) {
      const int row = __ldg(place + (size_t)t * k + j);
      if ((unsigned)row >= (unsigned)P) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (c + 32 * h < row16) xs[(size_t)row * row16 + c + 32 * h] = v[h];
    }
  }
}

moe_status check_product(int32_t P, int32_t E, int32_t N, int32_t K, int32_t quantum, const int32_t* offsets,
                         const int32_t* tiles, int32_t act, int32_t out_dtype) {
  if (P < 0 || P > kMaxPairs || E < 1 || E > kMaxExperts || N < 1)
    return fail(MOE_EINVAL, "P >= 0 (at most %lld), 1 <= E <= %d and N >= 1 are needed, got P %d, E %d, N %d", (long long)kMaxPairs, kMaxExperts, P, E, N);
  if (K < 1 || K > 1 << 24 || K % quantum) return fail(MOE_EINVAL, "K = %d is not a multiple of %d", K, quantum);
  if (act != 0 && act != 1) return fail(MOE_EINVAL, "act must be 0 (none) or 1 (SwiGLU)");
  if (act == 1 && N % 32) return fail(MOE_EINVAL, "SwiGLU needs N a multiple of 32, got %d", N);
  if (out_dtype != MOE_F32 && out_dtype != MOE_BF16) return fail(MOE_EINVAL, "out_dtype must be MOE_F32 or MOE_BF16");
  if (!offsets || !tiles || !aligned_to(offsets, 4) || !aligned_to(tiles, 4))
    return fail(MOE_EINVAL, "offsets and tiles must not be NULL and be 4-byte aligned");
  return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" int64_t moe_grouped_matmul_workspace(int32_t P, int32_t E, int32_t K, int32_t gather) {
  // many rows of an expert are gathered once, before the product
  return gather && P > 0 && use_pairs(P, E, false) ? (int64_t)P * K * 2 : 0;
}

extern "C" moe_status moe_grouped_matmul(int32_t P, int32_t E, int32_t N, int32_t K, const void* x, int32_t x_rows,
                                         const int32_t* order, const int32_t* place, int32_t k, const void* w, const int32_t* offsets,
                                         const int32_t* tiles, int32_t act, int32_t out_dtype, void* out, void* workspace,
                                         int64_t workspace_bytes, void* stream) {
  moe_status st = check_product(P, E, N, K, 8, offsets, tiles, act, out_dtype);
  if (st != MOE_OK) return st;
  if (order && (!place || k < 1 || P % k || !aligned_to(order, 4) || !aligned_to(place, 4)))
    return fail(MOE_EINVAL, "order needs place, k >= 1 that divides P, and 4-byte alignment");
  if (P == 0) return MOE_OK;
  if (!x || !w || !out || x_rows < (order ? P / k : P)) return fail(MOE_EINVAL, "x, w and out must not be NULL and x must hold its rows");
  if (!aligned_to(x, 16) || !aligned_to(w, 16) || !aligned_to(out, 16)) return fail(MOE_EINVAL, "x, w and out must be 16-byte aligned");
  ProductArgs a{};
  a.P = P; a.E = E; a.N = N; a.K = K; a.k = k; a.act = act; a.cols = act ? N / 2 : N; a.gather = order != nullptr;
  a.order = order; a.offsets = offsets; a.tiles = tiles; a.out = out;
  const int64_t need = moe_grouped_matmul_workspace(P, E, K, a.gather);
  if (need) {
    if (!workspace || workspace_bytes < need || !aligned_to(workspace, 16))
      return fail(MOE_EINVAL, "workspace must hold %lld bytes, 16-byte aligned, holds %lld", (long long)need, (long long)workspace_bytes);
    const int T = P / k, warps = GATHER_THREADS / 32, segs = (K / 8 + GATHER_SEG - 1) / GATHER_SEG;
    const dim3 grid(std::min((T + warps - 1) / warps, std::max(1, operator_sms() * 64 / segs)), segs);
    CK(launch_pdl(gather_kernel, grid, dim3(GATHER_THREADS), 0, static_cast<cudaStream_t>(stream), static_cast<const uint4*>(x), place, T, K / 8, k, P,
                  static_cast<uint4*>(workspace)));
    a.gather = 0;
    x = workspace;
    x_rows = P;
  }
  return launch_product<MOE_BF16>(a, ProductMem{x, w, nullptr, nullptr, x_rows}, out_dtype == MOE_F32, static_cast<cudaStream_t>(stream));
}

extern "C" moe_status moe_grouped_matmul_fp4(int32_t P, int32_t E, int32_t N, int32_t K, int32_t wdtype,
                                             const uint8_t* x_codes, const uint8_t* x_scales, const float* gx,
                                             const uint8_t* w_codes, const uint8_t* w_scales, const float* gw,
                                             int32_t gw_count, const int32_t* offsets, const int32_t* tiles, int32_t act,
                                             int32_t out_dtype, void* out, uint8_t* out_codes, uint8_t* out_scales,
                                             const float* g_out, void* stream) {
  moe_status st = check_product(P, E, N, K, 32, offsets, tiles, act, out_dtype);
  if (st != MOE_OK) return st;
  if (wdtype != MOE_NVFP4 && wdtype != MOE_MXFP4) return fail(MOE_EINVAL, "wdtype must be MOE_NVFP4 or MOE_MXFP4");
  if (wdtype == MOE_MXFP4 && g_out) return fail(MOE_EINVAL, "an MXFP4 result has no matrix scale");
  if (gw && gw_count != 1 && gw_count != E) return fail(MOE_EINVAL, "gw_count must be 1 or E = %d, is %d", E, gw_count);
  if (P == 0) return MOE_OK;
  if (!x_codes || !x_scales || !w_codes || !w_scales) return fail(MOE_EINVAL, "codes and scales must not be NULL");
  if (!aligned_to(x_codes, 16) || !aligned_to(x_scales, 16) || !aligned_to(w_codes, 16) || !aligned_to(w_scales, 16))
    return fail(MOE_EINVAL, "codes and scales must be 16-byte aligned");
  if (!aligned_to(gx, 4) || !aligned_to(gw, 4) || !aligned_to(g_out, 4)) return fail(MOE_EINVAL, "gx, gw and g_out must be 4-byte aligned");
  if (out) {
    if (!aligned_to(out, 16)) return fail(MOE_EINVAL, "out must be 16-byte aligned");
  } else {
    if (!act || (N / 2) % 32) return fail(MOE_EINVAL, "a 4-bit result needs act = 1 and N / 2 a multiple of 32");
    if (!out_codes || !out_scales || !aligned_to(out_codes, 16) || !aligned_to(out_scales, 16))
      return fail(MOE_EINVAL, "out, or out_codes and out_scales (16-byte aligned), must not be NULL");
  }
  ProductArgs a{};
  a.P = P; a.E = E; a.N = N; a.K = K; a.k = 1; a.act = act; a.cols = act ? N / 2 : N;
  a.groups = wdtype == MOE_NVFP4 ? (K + 63) / 64 : (K + 127) / 128;
  a.quant = !out;
  a.gx = gx; a.gw = gw; a.gw_count = gw_count;
  a.offsets = offsets; a.tiles = tiles; a.out = out; a.out_codes = out_codes; a.out_scales = out_scales; a.g_out = g_out;
  const ProductMem mem{x_codes, w_codes, x_scales, w_scales, P};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool exact = out && out_dtype == MOE_F32;
  return wdtype == MOE_NVFP4 ? launch_product<MOE_NVFP4>(a, mem, exact, s) : launch_product<MOE_MXFP4>(a, mem, exact, s);
}

extern "C" moe_status moe_operators_check(void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t err = 0;
  CK(cudaMemcpyFromSymbolAsync(&err, g_operator_err, sizeof(err), 0, cudaMemcpyDeviceToHost, s));
  CK(cudaStreamSynchronize(s));
  if (!err) return MOE_OK;
  err = 0;
  CK(cudaMemcpyToSymbolAsync(g_operator_err, &err, sizeof(err), 0, cudaMemcpyHostToDevice, s));
  CK(cudaStreamSynchronize(s));
  return fail(MOE_EDEVICE, "a wait inside an operator kernel ran out");
}
