// 8-bit products grouped by expert (include/moe_operators.h: moe_grouped_matmul_fp8).
//
//   out[i, n] = sum_b sx[b, i] sw[n / 128, b] sum_{k in block b} x[i, k] w[n, k],   e4m3 x and w
//
// Transposed like the bf16 and 4-bit products (grouped.cu): D[feature, token], a CTA (CG = 1) or
// a pair (CG = 2) multiplies 128 or 256 weight rows by up to 128 or 256 tokens of one expert,
// so that ragged tiles and single tokens cost the columns they have.
//
// The scales are any fp32 numbers, of every 128 of K, so they cannot be left to the tensor cores
// (whose block scales are powers of two) nor to the end.  The tensor cores sum one block of K,
// one slice of the ring, into one of two TMEM accumulators; the epilogue's warps multiply it
// by its scales and add it up in fp32 registers while the next slice runs.  A tile of 256 x 256
// is 128 sums a thread, for which the other warps give up registers.  What a slice costs an SM:
// 512 cycles of products, and beside them 256 of reading TMEM and 256 of fused multiply-adds
// (two an instruction).
//
// Persistent kernel, one CTA per SM:
//   warp 0      TMA: weight tiles, into a ring of K slices of 128 bytes a row
//   warp 1      one lane issues tcgen05.mma kind::f8f6f4
//   warp 2      TMA: token tiles
//   warp 3      scales: products of the tokens' and the weights', a slice ahead, into a ring of their own
//   warps 4-11  sums and epilogue, two warps to a quarter of the TMEM lanes
//
// SwiGLU: the weight rows of a tile alternate 16 gate rows and the 16 up rows of the same features, as in
// grouped.cu.  A requantised result needs the largest of 128 features: both CTAs of a pair have 64 of
// them and tell one another their maxima, by stores that count on the other's barrier.
//
// Every wait is bounded; one that runs out sets the flag moe_operators_check() reads.
#include "grouped.cuh"

#include <algorithm>

namespace moe {

namespace {

using namespace tc;

__device__ uint32_t g_operator_err8;

constexpr int FIRST_EPI = 4, EW = 8;
constexpr int THREADS = 32 * (FIRST_EPI + EW);
constexpr int A_BYTES = 128 * 128;             // 128 weight rows, 128 bytes of K each
constexpr int MAX_STAGES = 12;
constexpr int SCALE_SLOTS = 8, SCALE_AHEAD = 4;   // slices of scales in the ring, and loaded at a time
// An epilogue warp's buffer, 32 tokens: rows of 32 bf16 features, or 16 (SwiGLU), with strides that reach all banks
constexpr int EPI_WARP = 32 * 80, ROW32 = 80, ROW16 = 48;
constexpr int SMEM_LIMIT = 227 * 1024;
// registers a thread: launched with LAUNCH_REGS, of which the pair form's epilogue takes EPI_REGS and the four other warps keep OTHER_REGS
constexpr int LAUNCH_REGS = 168, EPI_REGS = 216, OTHER_REGS = 72;
static_assert(EPI_REGS * 32 * EW + OTHER_REGS * 32 * FIRST_EPI <= LAUNCH_REGS * THREADS, "the shares are of the launch's registers");

struct Args8 {
  int P, E, N, K, cols, act, quant, out_f32, wide, few;
  int m_blocks, kslices, n_blocks, stages, stage_bytes, b_rows, most_tiles;   // n_blocks: 128-row blocks of a matrix, which its scales have
  const float *sx, *sw;
  const int32_t* offsets;       // NULL: one matrix, all rows
  void* out;
  uint8_t* out_codes;
  float* out_scales;
};

// expert, first row, rows, weight block; tt: token tile, of all experts
struct Item8 { int e, row0, n, mb, tt; };

// where expert e's rows start, whatever the offsets hold: a row number of the call's, or P
__device__ __forceinline__ int row_at(const Args8& a, int e) {
  return a.offsets ? min(max(__ldg(a.offsets + e), 0), a.P) : e ? a.P : 0;
}

// item `it` into o, which holds the one before (tt = -1: none)
template <int CG>
__device__ __forceinline__ void item_at(const Args8& a, const int32_t* first, int it, Item8& o) {
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
  // even shares of the expert's rows
  const int j = tt - first[lo], r0 = row_at(a, lo), n = max(row_at(a, lo + 1), r0) - r0, nt = first[lo + 1] - first[lo];
  const int chunk = min(128 * CG, ((n + nt - 1) / nt + 16 * CG - 1) / (16 * CG) * (16 * CG));
  o.row0 = r0 + j * chunk;
  o.n = min(chunk, n - j * chunk);
}

// token columns of a tile, and the rows of them that one CTA loads
template <int CG>
__device__ __forceinline__ int columns(int n) { return (n + 16 * CG - 1) / (16 * CG) * (16 * CG); }
template <int CG>
__device__ __forceinline__ int token_rows(const Args8& a, const Item8& o) {
  const int mine = columns<CG>(o.n) / CG;
  return a.b_rows == 128 && mine > 48 * CG ? 128 : (mine + 16 * CG - 1) / (16 * CG) * (16 * CG);
}

// place of column t's scale in a slot: a thread's eight of a chunk of 32 columns (2 (lane % 4), + 1 of every 8) lie together
__device__ __forceinline__ int scale_place(int t) { return (t & ~31) + ((t >> 1) & 3) * 8 + ((t >> 3) & 3) * 2 + (t & 1); }

__device__ __forceinline__ float2 unpack2(uint64_t p) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
  return f;
}

__device__ __forceinline__ uint32_t pair_bf16(uint64_t p) {
  const float2 f = unpack2(p);
  return pack_bf16(f.x, f.y);
}
__device__ __forceinline__ void put(const Args8& a, size_t row, int col, bool live, float v) {
  if (!live || col >= a.cols) return;
  if (a.out_f32) static_cast<float*>(a.out)[row + col] = v;
  else static_cast<__nv_bfloat16*>(a.out)[row + col] = __float2bfloat16_rn(v);
}

template <int CG>
__global__ void __launch_bounds__(THREADS, 1)
product8_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmXall, const Args8 a) {
  constexpr int NMAX = 128 * CG, CHUNKS = NMAX / 64;     // chunks of 32 columns that a warp has
  constexpr int SLOT = 2 * NMAX;                         // scales of a slice: for the first and second 16 rows of every 32
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const uint32_t ring = smem_u32(smem);
  uint8_t* tail = smem + (size_t)a.stages * a.stage_bytes;
  uint8_t* ebuf = tail;
  tail += EW * EPI_WARP;
  float* slots = reinterpret_cast<float*>(tail);
  tail += SCALE_SLOTS * SLOT * 4;
  const uint32_t full = smem_u32(tail), empty = full + 8 * MAX_STAGES, sfull = empty + 8 * MAX_STAGES, sempty = sfull + 8 * SCALE_SLOTS,
                 tfull = sempty + 8 * SCALE_SLOTS, tempty = tfull + 16, tops_full = tempty + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail + 16 * MAX_STAGES + 16 * SCALE_SLOTS + 64);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* first = reinterpret_cast<int32_t*>(tmem_slot + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    for (int s = 0; s < SCALE_SLOTS; ++s) {
      mbar_init(sfull + 8 * s, 1);
      mbar_init(sempty + 8 * s, EW);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(tfull + 8 * s, 1);
      mbar_init(tempty + 8 * s, EW * CG);
    }
    for (int s = 0; s < 4; ++s) mbar_init(tops_full + 8 * s, 4);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc<CG>(smem_u32(tmem_slot), 2 * NMAX);
  pdl_wait();
  pdl_trigger();
  if (warp == 2) {   // token tiles before each expert
    int run = 0;
    for (int b = 0; b < a.E; b += 32) {
      const int e = b + lane;
      const int c = e < a.E ? (max(row_at(a, e + 1) - row_at(a, e), 0) + NMAX - 1) / NMAX : 0;
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
  // Every so many-th item; with few rows an expert, runs of items, mostly weight blocks of one token tile (as in grouped.cu)
  const int units = gridDim.x / CG, unit = blockIdx.x / CG, share = total / units, more = total % units;
  const bool runs = CG == 1 && a.few;
  const int step = runs ? 1 : units, it0 = runs ? unit * share + min(unit, more) : unit;
  const int it1 = runs ? it0 + share + (unit < more) : total;
  Item8 o;
  o.tt = -1;

  if (warp < FIRST_EPI) {
    if constexpr (CG == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(OTHER_REGS));
    bool ok = true;
    if (warp == 0) {
      // ---------------- loads ----------------
      int stage = 0;
      uint32_t phase = 0;
      for (int it = it0; it < it1 && ok; it += step) {
        item_at<CG>(a, first, it, o);
        const int m = o.mb * CG + (int)rank;      // 128-row weight tile (64 gate + 64 up with SwiGLU)
        const uint32_t bytes = (uint32_t)CG * (A_BYTES + 128u * token_rows<CG>(a, o));
        for (int ks = 0; ks < a.kslices; ++ks) {
          if (!warp_wait(empty + 8 * stage, phase ^ 1u, abort_flag)) { ok = false; break; }
          if (elect_one()) {
            const uint32_t bar = CG == 2 ? in_rank(full + 8 * stage, 0) : full + 8 * stage;
            if (rank == 0) mbar_expect(full + 8 * stage, bytes);
            // rows of one expert (dimensions K, row, expert), or with SwiGLU (K, 16 rows, gate / up, block of 16, expert)
            tma_5d<CG>(&tmW, bar, ring + stage * a.stage_bytes, ks * 128, a.act ? 0 : 128 * m, 0, a.act ? 4 * m : 0, o.e);
          }
          if (++stage == a.stages) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok) {
        if (lane == 0) { *abort_flag = 1; atomicOr(&g_operator_err8, 1u); }
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
        uint32_t phase = 0, acc_phase = 0;
        const uint64_t da = desc_sw128(ring), db = desc_sw128(ring + A_BYTES);
        for (int it = it0; it < it1 && ok; it += step) {
          item_at<CG>(a, first, it, o);
          // D fp32; e4m3 operands, both K-major; N; M = 128 CG
          const uint32_t idesc = (1u << 4) | ((uint32_t)(columns<CG>(o.n) >> 3) << 17) | ((uint32_t)(8 * CG) << 24);
          for (int ks = 0; ks < a.kslices; ++ks) {
            if (!warp_wait(tempty + 8 * acc, acc_phase ^ 1u, abort_flag) || !warp_wait(full + 8 * stage, phase, abort_flag)) { ok = false; break; }
            fence_after();
            if (elect_one()) {
              const uint64_t at = (uint32_t)(stage * a.stage_bytes) >> 4;
              const uint32_t d = tmem + (uint32_t)(acc * NMAX);
              const int left = a.K - ks * 128;
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                if (kk * 32 < left) mma_f8<CG>(d, da + at + 2 * kk, db + at + 2 * kk, idesc, (uint32_t)kk);
              commit<CG>(empty + 8 * stage);
              commit<CG>(tfull + 8 * acc);
            }
            __syncwarp();
            if (++stage == a.stages) { stage = 0; phase ^= 1u; }
            if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
          }
        }
        if (!ok && lane == 0) { *abort_flag = 1; atomicOr(&g_operator_err8, 1u); }
      }
    } else if (warp == 2) {
      // ---------------- tokens ----------------
      int stage = 0;
      uint32_t phase = 0;
      for (int it = it0; it < it1 && ok; it += step) {
        item_at<CG>(a, first, it, o);
        const int row0 = o.row0 + (int)rank * (columns<CG>(o.n) / CG), rows = token_rows<CG>(a, o);
        for (int ks = 0; ks < a.kslices; ++ks) {
          if (!warp_wait(empty + 8 * stage, phase ^ 1u, abort_flag)) { ok = false; break; }
          if (elect_one()) {
            const uint32_t sb = ring + stage * a.stage_bytes + A_BYTES;
            const uint32_t bar = CG == 2 ? in_rank(full + 8 * stage, 0) : full + 8 * stage;
            if (a.b_rows == 128 && rows == 128) tma_2d<CG>(&tmXall, bar, sb, ks * 128, row0);
            else
              for (int r = 0; r < rows; r += 16 * CG) tma_2d<CG>(&tmX, bar, sb + r * 128, ks * 128, row0 + r);
          }
          if (++stage == a.stages) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok && lane == 0) { *abort_flag = 1; atomicOr(&g_operator_err8, 1u); }
    } else {
      // ---------------- scales ----------------
      int slot = 0;
      uint32_t phase = 0;
      for (int it = it0; it < it1 && ok; it += step) {
        item_at<CG>(a, first, it, o);
        const int m = o.mb * CG + (int)rank;
        // the weights' blocks of the first and second 16 rows of every 32: one block, or the gate rows' and the up rows'
        const int b0 = min(a.act ? m >> 1 : m, a.n_blocks - 1), b1 = a.act ? min((a.cols + 64 * m) >> 7, a.n_blocks - 1) : b0;
        const float *w0 = a.sw + ((size_t)o.e * a.n_blocks + b0) * a.kslices, *w1 = a.sw + ((size_t)o.e * a.n_blocks + b1) * a.kslices;
        const float* x = a.sx + o.row0;
        for (int k0 = 0; k0 < a.kslices && ok; k0 += SCALE_AHEAD) {
          float v[SCALE_AHEAD][NMAX / 32], g0[SCALE_AHEAD], g1[SCALE_AHEAD];
#pragma unroll
          for (int i = 0; i < SCALE_AHEAD; ++i) {
            const int ks = k0 + i;
            g0[i] = ks < a.kslices ? __ldg(w0 + ks) : 0.0f;
            g1[i] = ks < a.kslices && a.act ? __ldg(w1 + ks) : 0.0f;
#pragma unroll
            for (int c = 0; c < NMAX / 32; ++c) {
              const int t = 32 * c + lane;
              v[i][c] = ks < a.kslices && t < o.n ? __ldg(x + (size_t)ks * a.P + t) : 0.0f;
            }
          }
#pragma unroll
          for (int i = 0; i < SCALE_AHEAD; ++i) {
            if (k0 + i >= a.kslices || !ok) continue;
            if (!warp_wait(sempty + 8 * slot, phase ^ 1u, abort_flag)) { ok = false; continue; }
            float* to = slots + slot * SLOT + scale_place(lane);
#pragma unroll
            for (int c = 0; c < NMAX / 32; ++c) {
              if (32 * c >= o.n) continue;
              to[32 * c] = v[i][c] * g0[i];
              if (a.act) to[NMAX + 32 * c] = v[i][c] * g1[i];
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(sfull + 8 * slot);
            if (++slot == SCALE_SLOTS) { slot = 0; phase ^= 1u; }
          }
        }
      }
      if (!ok && lane == 0) { *abort_flag = 1; atomicOr(&g_operator_err8, 1u); }
    }
  } else {
    // ---------------- sums and epilogue: a TMEM lane is a weight row, a column a token ----------------
    if constexpr (CG == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPI_REGS));
    // quarter of the TMEM lanes; which of every two chunks of 32 columns
    const int q = warp & 3, part = (warp - FIRST_EPI) >> 2;
    uint8_t* const buf = ebuf + (4 * part + q) * EPI_WARP;
    int acc = 0, slot = 0, turn = 0;
    uint32_t acc_phase = 0, slot_phase = 0, tops_phase = 0;
    for (int it = it0; it < it1; it += step) {
      item_at<CG>(a, first, it, o);
      // Sums of the quarter's rows lane / 4 and + 8 (even and odd pairs) of its first 16 (lo) and second 16 (hi), columns
      // 2 (lane % 4) and + 1 of every 8, two columns a pair
      uint64_t lo[CHUNKS][8] = {}, hi[CHUNKS][8] = {};
      bool ok = true;
      for (int ks = 0; ks < a.kslices; ++ks) {
        ok = warp_wait(sfull + 8 * slot, slot_phase, abort_flag) && warp_wait(tfull + 8 * acc, acc_phase, abort_flag);
        if (!ok) break;
        fence_after();
        const uint32_t tbase = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(acc * NMAX + 32 * part);
        const float* sc = slots + slot * SLOT + 32 * part + 8 * (lane & 3);
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
          if (64 * c + 32 * part >= o.n) continue;
          uint32_t x[16], y[16];
          tmem_ld16x4(tbase + 64 * c, x);
          tmem_ld16x4(tbase + (16u << 16) + 64 * c, y);
          const ulonglong2 s0 = *reinterpret_cast<const ulonglong2*>(sc + 64 * c), s1 = *reinterpret_cast<const ulonglong2*>(sc + 64 * c + 4);
          const uint64_t s[4] = {s0.x, s0.y, s1.x, s1.y};
          uint64_t u[4] = {s0.x, s0.y, s1.x, s1.y};
          if (a.act) {
            const ulonglong2 u0 = *reinterpret_cast<const ulonglong2*>(sc + NMAX + 64 * c), u1 = *reinterpret_cast<const ulonglong2*>(sc + NMAX + 64 * c + 4);
            u[0] = u0.x; u[1] = u0.y; u[2] = u1.x; u[3] = u1.y;
          }
          tmem_ld_wait(x, y);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            lo[c][i] = fma2(pack2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), s[i >> 1], lo[c][i]);
            hi[c][i] = fma2(pack2(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1])), u[i >> 1], hi[c][i]);
          }
        }
        fence_before();
        __syncwarp();
        if (lane == 0) {
          if (CG == 2) mbar_arrive_cluster(in_rank(tempty + 8 * acc, 0));
          else mbar_arrive(tempty + 8 * acc);
          mbar_arrive(sempty + 8 * slot);
        }
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
        if (++slot == SCALE_SLOTS) { slot = 0; slot_phase ^= 1u; }
      }
      if (!ok) {
        if (lane == 0) { *abort_flag = 1; atomicOr(&g_operator_err8, 1u); }
        break;
      }
      const int m = o.mb * CG + (int)rank, tok = 2 * (lane & 3), feat = lane >> 2;
      if (a.act) {
        // lo: gate rows, hi: the up rows of the same 16 features
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
          if (64 * c + 32 * part >= o.n) continue;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 g = unpack2(lo[c][i]), u = unpack2(hi[c][i]);
            float h0, h1;
            if (a.out_f32) {
              h0 = silu(g.x) * u.x;
              h1 = silu(g.y) * u.y;
            } else {
              swiglu2(__float_as_uint(g.x), __float_as_uint(g.y), __float_as_uint(u.x), __float_as_uint(u.y), 1.0f, -1.44269504f, h0, h1);
            }
            lo[c][i] = pack2(h0, h1);
          }
        }
      }
      if constexpr (CG == 2) {
        if (a.quant) {
          // ---- the largest of the pair's 128 features for every token: [CTA][quarter][column], columns as scales lie in a slot ----
          uint32_t* const top = reinterpret_cast<uint32_t*>(ebuf) + turn * (8 * NMAX);
          uint8_t* const bytes = ebuf + 2 * 8 * NMAX * 4 + (4 * part + q) * (32 * 16);
          const uint32_t bar = tops_full + 8 * (2 * turn + part);
#pragma unroll
          for (int c = 0; c < CHUNKS; ++c) {
            if (64 * c + 32 * part >= o.n) continue;
            uint32_t b[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 f = unpack2(lo[c][2 * i]), g = unpack2(lo[c][2 * i + 1]);
              b[2 * i] = max(__float_as_uint(f.x) & 0x7fffffffu, __float_as_uint(g.x) & 0x7fffffffu);
              b[2 * i + 1] = max(__float_as_uint(f.y) & 0x7fffffffu, __float_as_uint(g.y) & 0x7fffffffu);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
              for (int s = 4; s < 32; s <<= 1) b[i] = max(b[i], __shfl_xor_sync(0xffffffffu, b[i], s));
            if (lane < 4) {
              uint32_t* const at = top + (4 * (int)rank + q) * NMAX + 64 * c + 32 * part + 8 * lane;
              const uint32_t v[4] = {b[0], b[1], b[2], b[3]}, w[4] = {b[4], b[5], b[6], b[7]};
              *reinterpret_cast<uint4*>(at) = make_uint4(v[0], v[1], v[2], v[3]);
              *reinterpret_cast<uint4*>(at + 4) = make_uint4(w[0], w[1], w[2], w[3]);
              const uint32_t to = in_rank(smem_u32(at), rank ^ 1u), tobar = in_rank(bar, rank ^ 1u);
              st_async16(to, tobar, v);
              st_async16(to + 16, tobar, w);
            }
          }
          __syncwarp();
          if (lane == 0) {   // four warps arrive; the other CTA's four send 128 bytes a chunk
            if (q == 0) mbar_expect(bar, (uint32_t)((o.n - 32 * part + 63) / 64) * 4 * 128);
            else mbar_arrive(bar);
          }
          if (!warp_wait(bar, tops_phase, abort_flag)) {
            if (lane == 0) { *abort_flag = 1; atomicOr(&g_operator_err8, 1u); }
            break;
          }
          // Two turns: the other CTA's warps send a turn's next maxima only after these have sent the other turn's, and so read this
          // one's.
          if (turn) tops_phase ^= 1u;
          turn ^= 1;
          const int f = m * 64 + 16 * q;
#pragma unroll
          for (int c = 0; c < CHUNKS; ++c) {
            const int c0 = 64 * c + 32 * part, left = o.n - c0;
            if (left <= 0) continue;
            uint32_t b[8] = {};
#pragma unroll
            for (int w = 0; w < 8; ++w) {
              const uint4* const at = reinterpret_cast<const uint4*>(top + w * NMAX + c0 + 8 * (lane & 3));
              const uint4 x = at[0], y = at[1];
              b[0] = max(b[0], x.x); b[1] = max(b[1], x.y); b[2] = max(b[2], x.z); b[3] = max(b[3], x.w);
              b[4] = max(b[4], y.x); b[5] = max(b[5], y.y); b[6] = max(b[6], y.z); b[7] = max(b[7], y.w);
            }
            float r[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float top_i = fmaxf(__uint_as_float(b[i]), kLeast8);   // NaN counts as kLeast8
              asm("rcp.approx.f32 %0, %1;" : "=f"(r[i]) : "f"(top_i));
              r[i] *= 448.0f;
              const int t = tok + 8 * (i >> 1) + (i & 1);
              if (rank == 0 && q == 0 && lane < 4 && t < left)
                a.out_scales[(size_t)o.mb * a.P + o.row0 + c0 + t] = b[i] >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : top_i * (1.0f / 448.0f);
            }
            __syncwarp();   // the last chunk's bytes have been read
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 h = unpack2(lo[c][i]);
              const uint32_t codes = to_e4m3x2(h.x * r[i & ~1], h.y * r[i | 1]);
              uint8_t* const at = bytes + (tok + 8 * (i >> 1)) * 16 + feat + 8 * (i & 1);
              at[0] = (uint8_t)codes;
              at[16] = (uint8_t)(codes >> 8);
            }
            __syncwarp();
            if (lane < left && f < a.cols)
              *reinterpret_cast<uint4*>(a.out_codes + (size_t)(o.row0 + c0 + lane) * a.cols + f) = *reinterpret_cast<const uint4*>(bytes + lane * 16);
          }
          continue;
        }
      }
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c) {
        const int c0 = 64 * c + 32 * part, left = o.n - c0;
        if (left <= 0) continue;
        __syncwarp();   // the last chunk's buffer has been read
        if (a.wide && !a.act) {
          // bf16: 32 tokens of 32 features through shared memory, transposed 8 x 8 by stmatrix, 16 bytes a lane to memory
          const uint32_t to = smem_u32(buf) + (lane & 7) * ROW32 + (lane >> 3) * 16;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            stmatrix4_trans(to + 8 * k * ROW32, pair_bf16(lo[c][2 * k]), pair_bf16(lo[c][2 * k + 1]), pair_bf16(hi[c][2 * k]), pair_bf16(hi[c][2 * k + 1]));
          __syncwarp();
          const int f = m * 128 + 32 * q + (lane & 3) * 8;
#pragma unroll
          for (int r = lane >> 2; r < 32; r += 8)
            if (r < left && f < a.cols)
              *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + (size_t)(o.row0 + c0 + r) * a.cols + f) =
                  *reinterpret_cast<const uint4*>(buf + r * ROW32 + (lane & 3) * 16);
        } else if (a.wide) {
          // matrices: features 0-7 and 8-15 of eight tokens, then of the next eight
          const uint32_t to = smem_u32(buf) + ((lane & 7) + 8 * (lane >> 4)) * ROW16 + (lane & 8) * 2;
#pragma unroll
          for (int k = 0; k < 4; k += 2)
            stmatrix4_trans(to + 8 * k * ROW16, pair_bf16(lo[c][2 * k]), pair_bf16(lo[c][2 * k + 1]), pair_bf16(lo[c][2 * k + 2]), pair_bf16(lo[c][2 * k + 3]));
          __syncwarp();
          const int f = m * 64 + 16 * q + (lane & 1) * 8;
#pragma unroll
          for (int r = lane >> 1; r < 32; r += 16)
            if (r < left && f < a.cols)
              *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + (size_t)(o.row0 + c0 + r) * a.cols + f) =
                  *reinterpret_cast<const uint4*>(buf + r * ROW16 + (lane & 1) * 16);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int t = tok + 8 * (i >> 1), f = feat + 8 * (i & 1);
            const size_t row = (size_t)(o.row0 + c0 + t) * a.cols;
            const float2 x = unpack2(lo[c][i]), y = unpack2(hi[c][i]);
            const int col = a.act ? m * 64 + 16 * q + f : m * 128 + 32 * q + f;
            put(a, row, col, t < left, x.x);
            put(a, row + a.cols, col, t + 1 < left, x.y);
            if (!a.act) {
              put(a, row, col + 16, t < left, y.x);
              put(a, row + a.cols, col + 16, t + 1 < left, y.y);
            }
          }
        }
      }
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  if (warp == 1) {
    fence_after();
    tmem_free<CG>(tmem, 2 * NMAX);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
struct Mem8 { const uint8_t *x, *w; };

template <int CG>
moe_status launch8(Args8 a, const Mem8& mem, cudaStream_t s) {
  constexpr int NMAX = 128 * CG;
  const auto kernel = product8_kernel<CG>;
  const uint64_t K = a.K;
  a.m_blocks = (int)ceil_div64(a.act ? a.cols : a.N, (a.act ? 64 : 128) * CG);
  a.kslices = (a.K + 127) / 128;
  a.n_blocks = (a.N + 127) / 128;
  a.wide = !a.quant && !a.out_f32 && a.cols % 8 == 0;   // rows of out start on 16 bytes
  // rows of the token area: what the largest tile of P rows can need
  a.b_rows = CG == 2 ? 128 : std::min(128, (a.P + 15) / 16 * 16);
  a.stage_bytes = A_BYTES + a.b_rows * 128;
  const int fixed = 1024 + EW * EPI_WARP + SCALE_SLOTS * 2 * NMAX * 4 + 16 * MAX_STAGES + 16 * SCALE_SLOTS + 64 + 16 + 4 * (a.E + 1);
  a.stages = std::min(MAX_STAGES, (SMEM_LIMIT - fixed) / a.stage_bytes);
  const size_t smem = (size_t)fixed + (size_t)a.stages * a.stage_bytes;

  CUtensorMap tw, tx, txall;
  bool ok;
  if (a.act) {
    const cuuint64_t dims[5] = {K, 16, 2, (cuuint64_t)a.cols / 16, (cuuint64_t)a.E};
    const cuuint64_t strides[4] = {K, K * a.cols, K * 16, K * a.N};
    const cuuint32_t box[5] = {128, 16, 2, 4, 1};
    ok = make_map(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, mem.w, dims, strides, box, true);
  } else {
    const cuuint64_t dims[5] = {K, (cuuint64_t)a.N, 1, 1, (cuuint64_t)a.E};
    const cuuint64_t strides[4] = {K, K * a.N, K * a.N, K * a.N};
    const cuuint32_t box[5] = {128, 128, 1, 1, 1};
    ok = make_map(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, mem.w, dims, strides, box, true);
  }
  {
    const cuuint64_t dims[2] = {K, (cuuint64_t)a.P};
    const cuuint64_t strides[1] = {K};
    const cuuint32_t box[2] = {128, 16 * CG}, all[2] = {128, 128};
    ok = ok && make_map(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, mem.x, dims, strides, box, true) &&
         make_map(&txall, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, mem.x, dims, strides, all, true);
  }
  if (!ok) return fail(MOE_ECUDA, "cuTensorMapEncodeTiled failed");

  // at most every token tile the rows can make, on every weight block
  const int64_t tiles = (a.P + (int64_t)(NMAX - 1) * std::min(a.P, a.E)) / NMAX, most = tiles * a.m_blocks;
  if (most > 0x7fffffff) return fail(MOE_EINVAL, "P = %d rows of N = %d columns are too many tiles", a.P, a.N);
  a.most_tiles = (int)tiles;
  static bool allowed[64] = {};   // the kernel's shared memory and registers, once per device
  int dev = 0;
  CK(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return fail(MOE_EINVAL, "device %d is out of range", dev);
  if (!allowed[dev]) {
    cudaFuncAttributes attr;
    CK(cudaFuncGetAttributes(&attr, kernel));
    if (CG == 2 && attr.numRegs < LAUNCH_REGS) return fail(MOE_ECUDA, "the kernel was built with %d registers, %d are shared out", attr.numRegs, LAUNCH_REGS);
    CK(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_LIMIT));
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
      CK(cudaOccupancyMaxActiveClusters(&n, kernel, &cfg));
      if (n < 1) return fail(MOE_ECUDA, "no CTA pair fits the device");
      pairs[dev] = n;
      cfg.dynamicSmemBytes = smem;
    }
    resident = pairs[dev];
  }
  const int units = (int)std::min<int64_t>(most, resident);
  cfg.gridDim = dim3(units * CG);
  CK(cudaLaunchKernelEx(&cfg, kernel, tw, tx, txall, a));
  return MOE_OK;
}

// Pairs of CTAs load half of the tokens each; single CTAs start sooner and have twice the units of work.
bool use_pairs8(int64_t P, int64_t E) { return P >= 16 * E; }

}  // namespace

moe_status operators_check8(cudaStream_t s) {
  uint32_t err = 0;
  CK(cudaMemcpyFromSymbolAsync(&err, g_operator_err8, sizeof(err), 0, cudaMemcpyDeviceToHost, s));
  CK(cudaStreamSynchronize(s));
  if (!err) return MOE_OK;
  err = 0;
  CK(cudaMemcpyToSymbolAsync(g_operator_err8, &err, sizeof(err), 0, cudaMemcpyHostToDevice, s));
  CK(cudaStreamSynchronize(s));
  return fail(MOE_EDEVICE, "a wait inside an operator kernel ran out");
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_grouped_matmul_fp8(int32_t P, int32_t E, int32_t N, int32_t K, const uint8_t* x_codes, const float* x_scales, const uint8_t* w_codes,
                                             const float* w_scales, const int32_t* offsets, int32_t act, int32_t out_dtype, void* out, uint8_t* out_codes,
                                             float* out_scales, void* stream) {
  if (P < 0 || P > kMaxPairs || E < 1 || E > kMaxExperts || N < 1)
    return fail(MOE_EINVAL, "P >= 0 (at most %lld), 1 <= E <= %d and N >= 1 are needed, got P %d, E %d, N %d", (long long)kMaxPairs, kMaxExperts, P, E, N);
  if (K < 16 || K > 1 << 24 || K % 16) return fail(MOE_EINVAL, "K = %d is not a multiple of 16 (at most 2^24)", K);
  if (act != 0 && act != 1) return fail(MOE_EINVAL, "act must be 0 (none) or 1 (SwiGLU)");
  if (act == 1 && N % 128) return fail(MOE_EINVAL, "SwiGLU needs N a multiple of 128, got %d", N);
  if (out_dtype != MOE_F32 && out_dtype != MOE_BF16) return fail(MOE_EINVAL, "out_dtype must be MOE_F32 or MOE_BF16");
  if (!offsets && E != 1) return fail(MOE_EINVAL, "without offsets E must be 1, got %d", E);
  if (!aligned_to(offsets, 4)) return fail(MOE_EINVAL, "offsets must be 4-byte aligned");
  if (P == 0) return MOE_OK;
  if (!x_codes || !x_scales || !w_codes || !w_scales) return fail(MOE_EINVAL, "codes and scales must not be NULL");
  if (!aligned_to(x_codes, 16) || !aligned_to(w_codes, 16) || !aligned_to(x_scales, 4) || !aligned_to(w_scales, 4))
    return fail(MOE_EINVAL, "codes must be 16-byte aligned, scales 4-byte aligned");
  if (out) {
    if (!aligned_to(out, 16)) return fail(MOE_EINVAL, "out must be 16-byte aligned");
  } else {
    if (!act) return fail(MOE_EINVAL, "an 8-bit result needs act = 1");
    if (!out_codes || !out_scales || !aligned_to(out_codes, 16) || !aligned_to(out_scales, 4))
      return fail(MOE_EINVAL, "out, or out_codes (16-byte aligned) and out_scales (4-byte aligned), must not be NULL");
  }
  Args8 a{};
  a.P = P; a.E = E; a.N = N; a.K = K; a.act = act; a.cols = act ? N / 2 : N; a.quant = !out; a.out_f32 = out && out_dtype == MOE_F32;
  a.few = P < 64 * (int64_t)E;
  a.sx = x_scales; a.sw = w_scales; a.offsets = offsets; a.out = out; a.out_codes = out_codes; a.out_scales = out_scales;
  const Mem8 mem{x_codes, w_codes};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // the block of an 8-bit result is a pair's
  return a.quant || use_pairs8(P, E) ? launch8<2>(a, mem, s) : launch8<1>(a, mem, s);
}
