// 8-bit products grouped by expert (include/moe_operators.h: moe_grouped_matmul_fp8).
//
//   out[i, n] = sum_b sx[b, i] sw[n / 128, b] sum_{k in block b} x[i, k] w[n, k],   e4m3 x and w
//
// The scales are any fp32 numbers, of every 128 of K, so they cannot be left to the tensor cores
// (whose block scales are powers of two) nor to the end.  The tensor cores sum one block of K,
// one slice of the ring, into one of two TMEM accumulators; the epilogue's warps multiply it
// by its scales and add it up in fp32 registers while the next slice runs: 128 sums a thread, for
// which the other warps give up registers.
//
// So D[token, feature], unlike the bf16 and 4-bit products (grouped.cu): a TMEM lane is a token, whose scale is
// one register, and the features of a warp share theirs.  That leaves reading TMEM (32x32b loads, 256 cycles
// a slice of 128 tokens x 256 features) and the additions (256 more, beside them), under the 512 of the
// slice's products.  With the features as lanes the columns' scales come from shared memory: 660 cycles with
// broadcast loads, more with 16x256b loads, which read TMEM at half the rate (709 us for 16384 rows of 8
// experts, K 7168, N 4096; now 317, 3.0 PFLOP/s, and 301 with nothing added up).  What it costs: a ragged tile of tokens takes a
// whole one's products.  These are bursts, at 1785 MHz and 727 cycles a slice; in loops of seconds power leaves 1567 MHz, 723 cycles,
// 362 us.  Single CTAs take 736 to 777 cycles a slice at 1.33 to 1.66 GHz; with six slices a tile (K 768) it is 1240 to 1310, start and
// end of the tile among them.
//
// What an epilogue warp does once a slice counts as much: two warps a scheduler hide little of it.  Scales come for four slices at a
// time (a barrier of their own a slice: 500 us), arrivals are elected without a branch and both accumulators' addresses and
// phases are registers (410), the warp's number is uniform to the compiler and scales stay single registers until used (338); the second
// issuing warp took it to 317.
//
// A CTA (CG = 1) takes up to 128 tokens of one expert, a pair (CG = 2) up to 256, by TILE weight rows.
// Persistent kernel, one CTA per SM:
//   warp 0      TMA: weight tiles, and the token rows there are (the products of the rows behind them are not looked at), into a ring of
//               K slices of 128 bytes a row
//   warps 1-2   one lane each issues tcgen05.mma kind::f8f6f4, for every other slice: waiting for a slice and issuing it takes 500 to
//               650 cycles, more than the products of a small tile
//   warp 3      scales, some slices ahead, into a ring of groups of slices
//   warps 4-11  sums and epilogue: a quarter of the lanes, half of the columns each
//
// SwiGLU: the weight rows of a tile alternate 16 gate rows and the 16 up rows of the same features, as in
// grouped.cu, so a thread has both.  A requantised block is a token's 128 features: a tile's two halves, in two warps.
//
// Every wait is bounded; one that runs out sets the flag moe_operators_check() reads.
#include "grouped.cuh"

#include <algorithm>

namespace moe {

namespace {

using namespace tc;

constexpr int FIRST_EPI = 4, EW = 8;
constexpr int THREADS = 32 * (FIRST_EPI + EW);
constexpr int MAX_STAGES = 12;
// Accumulators, and columns between them: a slice's products and its sums take turns on one, so that with small tiles, whose slices are
// short, it is the way from one to the other and back that counts.
template <int TILE> constexpr int accs() { return TILE == 256 ? 2 : 4; }
constexpr int TMEM_COLS = 512, MAX_ACCS = 4;
// Stages, of `room` that fit.  Two warps issue alternate slices, so an odd number makes them share each stage, and a warp may test slice g's
// data while its stage's use before that, the other warp's slice g - stages, has not landed: by parity, that looks like data that has.  With
// ACCS + 2 stages it has landed: the warp is done with slice g - 2, so the sums with g - 2 - ACCS.  With fewer each warp keeps its own stages.
template <int TILE> int stages_of(int room) {
  const int n = std::min(MAX_STAGES, room);
  return n >= accs<TILE>() + 2 ? n : n & ~1;
}
constexpr int GROUP = 4;                       // slices whose scales go together, a multiple of the accumulators
constexpr int SLOT = GROUP * 128 + 4 * GROUP;  // a group's scales: [slice][token of the CTA], then [half of the columns][even, odd 16 columns][slice]
constexpr int SCALE_SLOTS = 3;
// What the epilogue has to know of the items (looking it up there, between two items, took 1500 cycles): the scales' warp, SCALE_SLOTS
// groups ahead at most, leaves it with an item's first group.
constexpr int HEADS = 8;
static_assert(HEADS > SCALE_SLOTS + 1, "an item's head stays until its epilogue has read it");
// An epilogue warp's buffer.  Single CTAs: 64 bytes of 32 tokens' rows, with a stride that reaches all banks; four lanes a row store them.
// Pairs: two boxes of 32 rows x 128 bytes in the 128-byte swizzle, which TMA stores while the next item's products run (a ragged
// warp's rows are stored by its lanes).
constexpr int ROW = 64, ROW_STRIDE = 80, EPI_WARP = 32 * ROW_STRIDE, BOX = 32 * 128;
template <int CG> constexpr int epi_warp() { return CG == 2 ? 2 * BOX : EPI_WARP; }
constexpr int SMEM_LIMIT = 227 * 1024;
// registers a thread: launched with LAUNCH_REGS, of which the epilogue takes EPI_REGS and the four other warps keep OTHER_REGS
constexpr int LAUNCH_REGS = 168, EPI_REGS = 224, OTHER_REGS = 56;
static_assert(EPI_REGS * 32 * EW + OTHER_REGS * 32 * FIRST_EPI <= LAUNCH_REGS * THREADS, "the shares are of the launch's registers");

struct Args8 {
  int P, E, N, K, cols, act, quant, out_f32, few;
  int m_blocks, kslices, n_blocks, stages, stage_bytes, box, most_tiles;   // n_blocks: 128-row blocks of a matrix; box: token rows of a load
  int whole;                    // rows of out start on 16 bytes
  const float *sx, *sw;
  const int32_t* offsets;       // NULL: one matrix, all rows
  void* out;
  uint8_t* out_codes;
  float* out_scales;
  uint32_t* err;                // operator_flag()
};

// expert, first row, rows, weight block; tt: token tile, of all experts
struct Item8 { int e, row0, n, mb, tt; };

// where expert e's rows start, whatever the offsets hold: a row number of the call's, or P
__device__ __forceinline__ int row_at(const Args8& a, int e) {
  return a.offsets ? min(max(__ldg(a.offsets + e), 0), a.P) : e ? a.P : 0;
}

// item `it` into o, which holds the one before (tt = -1: none), by a whole warp.  at[e]: the token tiles, and rows, before expert e.
template <int CG>
__device__ __forceinline__ void item_at(const Args8& a, const int2* at, int it, Item8& o) {
  const int tt = it / a.m_blocks;
  o.mb = it - tt * a.m_blocks;
  if (tt == o.tt) return;
  o.tt = tt;
  int lo = 0;
  if (a.E <= 256) {   // how many experts start at tt or before: the steps of a search would wait for one another
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int b = 0; b < 256; b += 32)
      if (b < a.E) lo += __popc(__ballot_sync(0xffffffffu, b + lane < a.E && at[b + lane].x <= tt));
    --lo;
  } else {
    int hi = a.E;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (at[mid].x <= tt) lo = mid;
      else hi = mid;
    }
  }
  o.e = lo;
  // even shares of the expert's rows: they are what is loaded
  const int2 s0 = at[lo], s1 = at[lo + 1];
  const int n = max(s1.y - s0.y, 0), nt = s1.x - s0.x, j = tt - s0.x;
  const int chunk = nt == 1 ? min(128 * CG, n) : min(128 * CG, (n + nt - 1) / nt);
  o.row0 = s0.y + j * chunk;
  o.n = min(chunk, n - j * chunk);
}

// of an item's rows: where CTA `rank`'s start, how many it has, how many it loads
template <int CG>
__device__ __forceinline__ int rows_from(const Args8& a, const Item8& o, int rank) {
  return CG == 1 || rank == 0 ? 0 : min(o.n, (((o.n + 1) >> 1) + a.box - 1) / a.box * a.box);
}
template <int CG>
__device__ __forceinline__ int rows_of(const Args8& a, const Item8& o, int rank) {
  const int split = rows_from<CG>(a, o, 1);
  return CG == 1 ? o.n : rank == 0 ? split : o.n - split;
}
__device__ __forceinline__ int rows_loaded(const Args8& a, int rows) { return (rows + a.box - 1) / a.box * a.box; }

template <int N>
__device__ __forceinline__ void rotate(uint32_t (&v)[N]) {
  const uint32_t t = v[0];
#pragma unroll
  for (int i = 1; i < N; ++i) v[i - 1] = v[i];
  v[N - 1] = t;
}
// acc += {a, b} * s, behind the wait for a and b
__device__ __forceinline__ void add2(uint64_t& acc, uint32_t a, uint32_t b, uint64_t s) {
  asm volatile("{\n .reg .b64 t;\n mov.b64 t, {%1, %2};\n fma.rn.f32x2 %0, t, %3, %0;\n}\n" : "+l"(acc) : "r"(a), "r"(b), "l"(s));
}
__device__ __forceinline__ float2 unpack2(uint64_t p) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
  return f;
}
// 64 bytes of each lane's row to memory: `rows` rows of `stride` bytes from `out` on, `bytes` of each (64 or less), SIZE bytes an element
template <int SIZE>
__device__ __forceinline__ void put_rows(uint8_t* buf, const uint32_t (&w)[16], uint8_t* out, size_t stride, int rows, int bytes, bool whole) {
  const int lane = threadIdx.x & 31;
  __syncwarp();   // the last rows have been read
#pragma unroll
  for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(buf + lane * ROW_STRIDE + 16 * i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  __syncwarp();
  if (whole) {
    const int at = 16 * (lane & 3);
    uint8_t* to = out + (size_t)(lane >> 2) * stride + at;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = (lane >> 2) + 8 * i;
      if (r < rows && at < bytes) *reinterpret_cast<uint4*>(to + 8 * i * stride) = *reinterpret_cast<const uint4*>(buf + r * ROW_STRIDE + at);
    }
  } else {
    constexpr int N = ROW / SIZE;   // elements of a row here
    const int at = SIZE * (lane % N);
    for (int r = lane / N; r < rows; r += 32 / N) {
      if (at >= bytes) continue;
      if constexpr (SIZE == 4) *reinterpret_cast<uint32_t*>(out + (size_t)r * stride + at) = *reinterpret_cast<const uint32_t*>(buf + r * ROW_STRIDE + at);
      else *reinterpret_cast<uint16_t*>(out + (size_t)r * stride + at) = *reinterpret_cast<const uint16_t*>(buf + r * ROW_STRIDE + at);
    }
  }
}
// 64 bytes of a row: 16 fp32 columns, or 32 bf16 ones of two chunks
template <int CHUNKS, int STEP>
__device__ __forceinline__ void pack64(const uint64_t (&v)[CHUNKS][8], int c, bool f32, uint32_t (&w)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (f32) {
      const float2 p = unpack2(v[c * STEP][i >> 1]);
      w[i] = __float_as_uint(i & 1 ? p.y : p.x);
    } else {
      const float2 p = (c + (i >> 3)) * STEP < CHUNKS ? unpack2(v[(c + (i >> 3)) * STEP < CHUNKS ? (c + (i >> 3)) * STEP : 0][i & 7]) : make_float2(0.0f, 0.0f);
      w[i] = pack_bf16(p.x, p.y);
    }
  }
}
// The results of a warp's 32 tokens, from `token` on: every STEP-th of CHUNKS chunks of 16 columns, from column f on
template <int CG, int CHUNKS, int STEP, bool F32>
__device__ __forceinline__ void put_results(const Args8& a, const CUtensorMap& map, uint8_t* buf, const uint64_t (&v)[CHUNKS][8], int token, int rows, int f) {
  constexpr int SIZE = F32 ? 4 : 2, ONE = F32 ? 1 : 2, PIECES = (CHUNKS / STEP + ONE - 1) / ONE;   // pieces of 64 bytes
  const int lane = threadIdx.x & 31;
  const size_t stride = (size_t)a.cols * SIZE;
  uint8_t* const out = static_cast<uint8_t*>(a.out) + (size_t)token * stride + (size_t)f * SIZE;
  const int bytes = min(a.cols - f, CHUNKS / STEP * 16) * SIZE;   // of a row from column f on
  if constexpr (CG == 2) {
    if (a.whole) {
#pragma unroll
      for (int p0 = 0; p0 < PIECES; p0 += 4) {
        if (p0 * 64 >= bytes) continue;
        constexpr int N = PIECES < 4 ? PIECES : 4;
        store_wait_read();   // the last boxes have been read
        __syncwarp();
#pragma unroll
        for (int p = 0; p < N; ++p) {
          uint32_t w[16];
          pack64<CHUNKS, STEP>(v, (p0 + p) * ONE, F32, w);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(buf + (p >> 1) * BOX + lane * 128 + ((4 * (p & 1) + i) ^ (lane & 7)) * 16) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
        if (rows == 32) {
          fence_async_proxy();
          __syncwarp();
          if (elect_one()) {
#pragma unroll
            for (int b = 0; b < (N + 1) / 2; ++b)
              if ((p0 + 2 * b) * 64 < bytes) tma_store_2d(&map, smem_u32(buf) + b * BOX, f + (p0 + 2 * b) * 64 / SIZE, token);
            store_commit();
          }
          __syncwarp();
        } else {
          __syncwarp();
#pragma unroll
          for (int b = 0; b < (N + 1) / 2; ++b)
            for (int r = lane >> 3; r < rows; r += 4) {
              const int at = (p0 + 2 * b) * 64 + 16 * (lane & 7);
              if (at < bytes && (lane & 7) < 4 * (N - 2 * b))
                *reinterpret_cast<uint4*>(out + (size_t)r * stride + at) = *reinterpret_cast<const uint4*>(buf + b * BOX + r * 128 + ((lane ^ r) & 7) * 16);
            }
        }
      }
      return;
    }
  }
#pragma unroll
  for (int p = 0; p < PIECES; ++p) {
    if (p * 64 >= bytes) continue;
    uint32_t w[16];
    pack64<CHUNKS, STEP>(v, p * ONE, F32, w);
    put_rows<SIZE>(buf, w, out + 64 * p, stride, rows, min(64, bytes - 64 * p), a.whole);
  }
}
template <int CG, int CHUNKS, int STEP>
__device__ __forceinline__ void put_results(const Args8& a, const CUtensorMap& map, uint8_t* buf, const uint64_t (&v)[CHUNKS][8], int token, int rows, int f) {
  if (a.out_f32) put_results<CG, CHUNKS, STEP, true>(a, map, buf, v, token, rows, f);
  else put_results<CG, CHUNKS, STEP, false>(a, map, buf, v, token, rows, f);
}

// desc_sw128 in two halves: what an address adds is in the lower one
__device__ __forceinline__ uint32_t desc_low(uint32_t addr) { return (uint32_t)desc_sw128(addr); }
__device__ __forceinline__ uint64_t desc_of(uint32_t low) { return (desc_sw128(0) & 0xffffffff00000000ull) | low; }
// whether both phases are over, for the whole warp.  Both tests are on their way at once, and each may be held until its phase ends: an outcome
// can be older than the other one's (stages_of).
__device__ __forceinline__ bool test_both(uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p, q;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n"
      " and.pred p, p, q;\n vote.sync.all.pred q, p, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(ok) : "r"(b0), "r"(p0), "r"(b1), "r"(p1) : "memory");
  return ok != 0;
}
template <int CG, int TILE>
__global__ void __launch_bounds__(THREADS, 1)
product8_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmO, const Args8 a) {
  constexpr int HALF = TILE / 2, CHUNKS = HALF / 16;     // a thread's columns: half of the tile's, 16 a chunk
  constexpr int ACCS = accs<TILE>(), ACC_COLS = TMEM_COLS / ACCS;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const uint32_t ring = smem_u32(smem);
  constexpr int w_bytes = TILE / CG * 128;     // a stage: the CTA's weight rows, then its token rows
  uint8_t* tail = smem + (size_t)a.stages * a.stage_bytes;
  uint8_t* ebuf = tail;
  tail += EW * epi_warp<CG>();
  float* slots = reinterpret_cast<float*>(tail);
  tail += SCALE_SLOTS * SLOT * 4;
  int4* heads = reinterpret_cast<int4*>(tail);          // an item's first token and number of tokens in this CTA, and its weight block
  tail += HEADS * 16;
  uint32_t* tops = reinterpret_cast<uint32_t*>(tail);   // [turn][half of the columns][token]
  tail += 2 * 2 * 128 * 4;
  const uint32_t full = smem_u32(tail), empty = full + 8 * MAX_STAGES, sfull = empty + 8 * MAX_STAGES, sempty = sfull + 8 * SCALE_SLOTS,
                 tfull = sempty + 8 * SCALE_SLOTS, tempty = tfull + 8 * MAX_ACCS, tops_full = tempty + 8 * MAX_ACCS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail + 16 * MAX_STAGES + 16 * SCALE_SLOTS + 16 * MAX_ACCS + 32);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int2* first = reinterpret_cast<int2*>(tmem_slot + 4);   // of each expert, and behind the last one: item_at's

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = CG == 2 ? (int)cluster_rank() : 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    for (int s = 0; s < SCALE_SLOTS; ++s) {
      mbar_init(sfull + 8 * s, 1);
      mbar_init(sempty + 8 * s, EW);
    }
    for (int s = 0; s < ACCS; ++s) {
      mbar_init(tfull + 8 * s, 1);
      mbar_init(tempty + 8 * s, EW * CG);
    }
    for (int s = 0; s < 4; ++s) mbar_init(tops_full + 8 * s, 2);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc<CG>(smem_u32(tmem_slot), TMEM_COLS);
  if (warp == 3 && lane == 0) {
    prefetch_map(&tmW);
    prefetch_map(&tmX);
    prefetch_map(&tmO);
  }
  pdl_wait();
  pdl_trigger();
  if (warp == 2) {   // token tiles and rows before each expert, four experts a lane
    int run = 0;
    for (int b = 4 * lane; b < a.E + 1 + 4 * lane; b += 128) {
      int row[5], tiles[4], sum = 0;
#pragma unroll
      for (int i = 0; i < 5; ++i) row[i] = b + i <= a.E ? row_at(a, b + i) : 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        tiles[i] = b + i < a.E ? (max(row[i + 1] - row[i], 0) + 128 * CG - 1) / (128 * CG) : 0;
        sum += tiles[i];
      }
      int x = sum;
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += v;
      }
      int before = run + x - sum;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // offsets that do not ascend could make more tiles than the rows do
        if (b + i <= a.E) first[b + i] = make_int2(min(before, a.most_tiles), row[i]);
        before += tiles[i];
      }
      run = min(run + __shfl_sync(0xffffffffu, x, 31), a.most_tiles);
    }
  }
  fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  const int total = first[a.E].x * a.m_blocks;
  // Every so many-th item; with few rows an expert, runs of items, mostly weight blocks of one token tile (as in grouped.cu)
  const int units = gridDim.x / CG, unit = blockIdx.x / CG, share = total / units, more = total % units;
  const bool runs = CG == 1 && a.few;
  const int step = runs ? 1 : units, it0 = runs ? unit * share + min(unit, more) : unit;
  const int it1 = runs ? it0 + share + (unit < more) : total;
  Item8 o;
  o.tt = -1;

  if (warp < FIRST_EPI) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(OTHER_REGS));
    bool ok = true;
    if (warp == 0) {
      // ---------------- loads ----------------
      int stage = 0;
      uint32_t phase = 0;
      constexpr int boxes = (TILE / CG + 127) / 128;
      for (int it = it0; it < it1 && ok; it += step) {
        item_at<CG>(a, first, it, o);
        uint32_t bytes = (uint32_t)(CG * w_bytes);
        for (int r = 0; r < CG; ++r) bytes += 128u * rows_loaded(a, rows_of<CG>(a, o, r));
        const int row0 = o.row0 + rows_from<CG>(a, o, rank), rows = rows_of<CG>(a, o, rank);
        for (int ks = 0; ks < a.kslices; ++ks) {
          if (!warp_wait(empty + 8 * stage, phase ^ 1u, abort_flag)) { ok = false; break; }
          if (elect_one()) {
            const uint32_t bar = CG == 2 ? in_rank(full + 8 * stage, 0) : full + 8 * stage, to = ring + stage * a.stage_bytes;
            if (rank == 0) mbar_expect(full + 8 * stage, bytes);
            // rows of one expert (dimensions K, row, expert), or with SwiGLU (K, 16 rows, gate / up, block of 16, expert)
            for (int b = 0; b < boxes; ++b) {
              const int row = o.mb * TILE + rank * (TILE / CG) + 128 * b;
              tma_5d<CG>(&tmW, bar, to + b * 128 * 128, ks * 128, a.act ? 0 : row, 0, a.act ? row >> 5 : 0, o.e);
            }
            for (int r = 0; r < rows; r += a.box) tma_2d<CG>(&tmX, bar, to + w_bytes + r * 128, ks * 128, row0 + r);
          }
          if (++stage == a.stages) { stage = 0; phase ^= 1u; }
        }
      }
      // every slice has been used, and no arrival on this CTA's barriers is outstanding, before it ends
      for (int i = 0; i < a.stages && ok; ++i) {
        ok = warp_wait(empty + 8 * stage, phase ^ 1u, abort_flag);
        if (++stage == a.stages) { stage = 0; phase ^= 1u; }
      }
      if (!ok) {
        if (lane == 0) { *abort_flag = 1; atomicOr(a.err, 1u); }
        // copies and products in flight end long before this bound
        const unsigned long long t0 = gtimer();
        while (gtimer() - t0 < 1000000ull) {
        }
      }
    } else if (warp < 3) {
      // ---------------- products: every other slice ----------------
      if (rank == 0) {
        const int p = warp - 1, items = it0 < it1 ? (it1 - it0 + step - 1) / step : 0, slices = items * a.kslices;
        int stage = p, acc = p, ks = p;
        uint32_t phase = 0, acc_phase = 1;
        const uint32_t lw = desc_low(ring), lx = desc_low(ring + w_bytes);
        const int whole = a.K >> 7, rest = a.K & 127;
        // D fp32; e4m3 operands, both K-major; N = TILE; M = 128 CG
        constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(TILE >> 3) << 17) | ((uint32_t)(8 * CG) << 24);
        for (int g = p; g < slices; g += 2) {
          while (ks >= a.kslices) ks -= a.kslices;   // of its item
          const uint32_t at = (uint32_t)(stage * a.stage_bytes) >> 4;
          // The other CTA's arrivals on tempty stand for its TMEM reads, which the fences order; no memory is handed over.
          if (!test_both(full + 8 * stage, phase, tempty + 8 * acc, acc_phase) &&
              (!warp_wait(full + 8 * stage, phase, abort_flag) || !warp_wait(tempty + 8 * acc, acc_phase, abort_flag))) { ok = false; break; }
          fence_after();
          const uint32_t d = tmem + (uint32_t)(acc * ACC_COLS);
          if (elect_one()) {
            if (ks < whole) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) mma_f8<CG>(d, desc_of(lx + at + 2 * kk), desc_of(lw + at + 2 * kk), idesc, (uint32_t)kk);
            } else {
              for (int kk = 0; kk * 32 < rest; ++kk) mma_f8<CG>(d, desc_of(lx + at + 2 * kk), desc_of(lw + at + 2 * kk), idesc, (uint32_t)kk);
            }
            commit<CG>(tfull + 8 * acc);
            commit<CG>(empty + 8 * stage);
          }
          __syncwarp();
          ks += 2;
          if ((stage += 2) >= a.stages) { stage -= a.stages; phase ^= 1u; }
          if ((acc += 2) >= ACCS) { acc -= ACCS; acc_phase ^= 1u; }
        }
        if (!ok && lane == 0) { *abort_flag = 1; atomicOr(a.err, 1u); }
      }
    } else {
      // ---------------- scales ----------------
      int slot = 0, head = 0;
      uint32_t phase = 0;
      for (int it = it0; it < it1 && ok; it += step, head = (head + 1) % HEADS) {
        item_at<CG>(a, first, it, o);
        const int rows = rows_of<CG>(a, o, rank);
        // lane 8 half + 4 odd + slice: the weights' blocks of each half of the columns, one or the gate rows' and the up rows'
        const int half = lane >> 3 & 1, odd = lane >> 2 & 1;
        const int f = a.act ? (o.mb * 2 + half) * (HALF / 2) + odd * a.cols : (o.mb * 2 + half) * HALF;
        const float* w = a.sw + ((size_t)o.e * a.n_blocks + min(f >> 7, a.n_blocks - 1)) * a.kslices;
        const float* x = a.sx + o.row0 + rows_from<CG>(a, o, rank);
        for (int k0 = 0; k0 < a.kslices && ok; k0 += GROUP) {
          float v[GROUP][4];
#pragma unroll
          for (int i = 0; i < GROUP; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              v[i][c] = k0 + i < a.kslices && 32 * c + lane < rows ? __ldg(x + (size_t)(k0 + i) * a.P + 32 * c + lane) : 0.0f;
          const float g = lane < 4 * GROUP && k0 + (lane & 3) < a.kslices ? __ldg(w + k0 + (lane & 3)) : 0.0f;
          ok = warp_wait_cta(sempty + 8 * slot, phase ^ 1u, abort_flag);
          if (!ok) continue;
          float* to = slots + slot * SLOT + lane;
#pragma unroll
          for (int i = 0; i < GROUP; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (32 * c < rows) to[128 * i + 32 * c] = v[i][c];
          if (lane < 4 * GROUP) to[GROUP * 128] = g;
          if (k0 == 0 && lane == 0) heads[head] = make_int4(o.row0 + rows_from<CG>(a, o, rank), rows, o.mb, 0);
          __syncwarp();
          if (lane == 0) mbar_arrive(sfull + 8 * slot);
          if (++slot == SCALE_SLOTS) { slot = 0; phase ^= 1u; }
        }
      }
      if (!ok && lane == 0) { *abort_flag = 1; atomicOr(a.err, 1u); }
    }
  } else {
    // ---------------- sums and epilogue: a TMEM lane is a token, a column a weight row ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPI_REGS));
    // quarter of the TMEM lanes, half of the columns
    const int q = warp & 3, part = (warp - FIRST_EPI) >> 2;
    int slot = 0, turn = 0, head = 0;
    uint32_t slot_phase = 0, tops_phase = 0;
    // of the accumulator of an item's every ACCS-th slice: where the warp reads it, its barriers, the phase of the next use
    uint32_t from[ACCS], ready[ACCS], done[ACCS], phase[ACCS] = {};
#pragma unroll
    for (int i = 0; i < ACCS; ++i) {
      from[i] = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(i * ACC_COLS + HALF * part);
      ready[i] = tfull + 8 * i;
      done[i] = CG == 2 ? in_rank(tempty + 8 * i, 0) : tempty + 8 * i;
    }
    uint8_t* const buf = ebuf + (4 * part + q) * epi_warp<CG>();
    for (int it = it0; it < it1; it += step, head = (head + 1) % HEADS) {
      uint64_t sum[CHUNKS][8] = {};   // of the thread's token: two columns a pair, 16 a chunk
      bool ok = true, some = false;   // some: tokens of this warp's
      for (int k0 = 0; k0 < a.kslices; k0 += GROUP) {
        ok = warp_wait_cta(sfull + 8 * slot, slot_phase, abort_flag);
        if (!ok) break;
        const float* sc = slots + slot * SLOT;
        if (k0 == 0) some = 32 * q < heads[head].y;
        float s0[GROUP], s1[GROUP];   // of even and odd chunks
        if (some) {
          const float4 w0 = *reinterpret_cast<const float4*>(sc + GROUP * 128 + 8 * part), w1 = *reinterpret_cast<const float4*>(sc + GROUP * 128 + 8 * part + 4);
          const float u0[GROUP] = {w0.x, w0.y, w0.z, w0.w}, u1[GROUP] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
          for (int j = 0; j < GROUP; ++j) {
            const float v = sc[128 * j + 32 * q + lane];
            s0[j] = u0[j] * v;
            s1[j] = u1[j] * v;
          }
        }
        __syncwarp();
        arrive_elected<1>(sempty + 8 * slot);
        if (++slot == SCALE_SLOTS) { slot = 0; slot_phase ^= 1u; }
#pragma unroll
        for (int j = 0; j < GROUP; ++j) {
          if (k0 + j >= a.kslices) break;
          ok = warp_wait_cta(ready[j % ACCS], phase[j % ACCS], abort_flag);
          if (!ok) break;
          phase[j % ACCS] ^= 1u;
          fence_after();
          if (some) {
            const uint64_t t0 = pack2(s0[j], s0[j]), t1 = pack2(s1[j], s1[j]);
            uint32_t x[2][16];
            tmem_ld32(from[j % ACCS], x[0]);
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c) {
              tmem_wait();
              if (c + 1 < CHUNKS) {
                tmem_ld32(from[j % ACCS] + 16 * (c + 1), x[(c + 1) & 1]);
              } else {   // the accumulator has been read
                fence_before();
                arrive_elected<CG>(done[j % ACCS]);
              }
#pragma unroll
              for (int i = 0; i < 8; ++i) add2(sum[c][i], x[c & 1][2 * i], x[c & 1][2 * i + 1], c & 1 ? t1 : t0);
            }
          } else {
            fence_before();
            arrive_elected<CG>(done[j % ACCS]);
          }
        }
        if (!ok) break;
      }
      for (int i = a.kslices % ACCS; i > 0; --i) {   // the accumulator that the next item starts with
        rotate(from);
        rotate(ready);
        rotate(done);
        rotate(phase);
      }
      if (!ok) {
        if (lane == 0) { *abort_flag = 1; atomicOr(a.err, 1u); }
        break;
      }
      const int4 o = heads[head];
      const int token = o.x + 32 * q, rows = min(32, o.y - 32 * q);   // the warp's
      if (!a.act) {
        if (some) put_results<CG, CHUNKS, 1>(a, tmO, buf, sum, token, rows, o.z * TILE + part * HALF);
        continue;
      }
      // gate and up of 16 features alternate
      const int f0 = (o.z * 2 + part) * (HALF / 2);
      uint32_t top = 0u;
      if (some) {
#pragma unroll
        for (int c = 0; c < CHUNKS; c += 2) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 g = unpack2(sum[c][i]), u = unpack2(sum[c + 1][i]);
            float h0, h1;
            if (a.out_f32) {
              h0 = silu(g.x) * u.x;
              h1 = silu(g.y) * u.y;
            } else {
              swiglu2(__float_as_uint(g.x), __float_as_uint(g.y), __float_as_uint(u.x), __float_as_uint(u.y), 1.0f, -1.44269504f, h0, h1);
            }
            sum[c][i] = pack2(h0, h1);
            top = __vimax3_u32(top, __float_as_uint(h0) & 0x7fffffffu, __float_as_uint(h1) & 0x7fffffffu);
          }
        }
      }
      if (!a.quant) {
        if (some) put_results<CG, CHUNKS, 2>(a, tmO, buf, sum, token, rows, f0);
        continue;
      }
      if constexpr (TILE == 256) {
        // ---- the largest of the token's 128 features: this warp's 64, and those of the warp with the other half ----
        uint32_t* const at = tops + turn * 256 + 32 * q + lane;
        at[128 * part] = top;
        __syncwarp();
        if (lane == 0) mbar_arrive(tops_full + 8 * q);
        if (!warp_wait_cta(tops_full + 8 * q, tops_phase, abort_flag)) {
          if (lane == 0) { *abort_flag = 1; atomicOr(a.err, 1u); }
          break;
        }
        top = max(top, at[128 * (part ^ 1)]);
        // two turns: the other warp writes this turn again only after this one has arrived for the next, and so read this
        tops_phase ^= 1u;
        turn ^= 1;
        if (!some || f0 >= a.cols) continue;
        const float most = fmaxf(__uint_as_float(top), kLeast8);
        const bool bad = top >= 0x7f800000u;   // a NaN or an infinity: scale NaN, codes 0
        if (part == 0 && lane < rows) a.out_scales[(size_t)o.z * a.P + token + lane] = bad ? __uint_as_float(0x7fffffffu) : most * (1.0f / 448.0f);
        // Codes by a reciprocal good to three units, not the quantiser's rounded quotient: h carries the sums' and SwiGLU's errors, so no tie
        // of the 8-bit grid is exact here (512 x 2048 results of K 7168: the codes are those of quantising the fp32 results, each one).
        float r;
        asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(most));
        r *= 448.0f;
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float2 h = unpack2(sum[2 * (i >> 3)][i & 7]);
          const uint32_t two = to_e4m3x2(h.x * r, h.y * r);
          w[i >> 1] = bad ? 0u : i & 1 ? w[i >> 1] | two << 16 : two;
        }
        put_rows<2>(buf, w, a.out_codes + (size_t)token * a.cols + f0, a.cols, rows, ROW, true);
      }
    }
    if (CG == 2) store_wait();
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
struct Mem8 { const uint8_t *x, *w; };

// Shared memory of a CTA: rows of the token area, what the largest tile of P rows can need; bytes of a stage, and of all else; stages
struct Room8 { int x_rows, stage_bytes, fixed, stages; };
template <int CG, int TILE>
Room8 room8(int P, int E) {
  Room8 m;
  m.x_rows = CG == 2 ? 128 : std::min(128, (int)(((int64_t)P + 15) / 16 * 16));
  m.stage_bytes = (TILE / CG + m.x_rows) * 128;
  // behind the last stage as much as the products read past its token rows
  m.fixed = 1024 + std::max(EW * epi_warp<CG>() + SCALE_SLOTS * SLOT * 4 + HEADS * 16 + 2 * 2 * 128 * 4 + 16 * MAX_STAGES + 16 * SCALE_SLOTS + 16 * MAX_ACCS + 32 + 16 + 8 * (E + 1), (128 - m.x_rows) * 128);
  m.stages = stages_of<TILE>((SMEM_LIMIT - m.fixed) / m.stage_bytes);
  return m;
}

template <int CG, int TILE>
moe_status launch8(Args8 a, const Mem8& mem, cudaStream_t s) {
  const auto kernel = product8_kernel<CG, TILE>;
  const uint64_t K = a.K;
  a.m_blocks = (int)ceil_div64(a.N, TILE);
  a.kslices = (a.K + 127) / 128;
  a.n_blocks = (a.N + 127) / 128;
  a.whole = a.cols * (a.out_f32 ? 4 : 2) % 16 == 0;
  const Room8 m = room8<CG, TILE>(a.P, a.E);
  if (m.stages < 2) return fail(MOE_EINVAL, "the table of E = %d experts leaves no room for two stages", a.E);   // a warp that issues starts at its own
  a.box = std::min(32, m.x_rows & -m.x_rows);
  a.stage_bytes = m.stage_bytes;
  a.stages = m.stages;
  const size_t smem = (size_t)m.fixed + (size_t)a.stages * a.stage_bytes;

  CUtensorMap tw, tx, to;
  bool ok;
  const cuuint32_t w_rows = (cuuint32_t)std::min(128, TILE / CG);
  if (a.act) {
    const cuuint64_t dims[5] = {K, 16, 2, (cuuint64_t)a.cols / 16, (cuuint64_t)a.E};
    const cuuint64_t strides[4] = {K, K * a.cols, K * 16, K * a.N};
    const cuuint32_t box[5] = {128, 16, 2, w_rows / 32, 1};
    ok = make_map(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, mem.w, dims, strides, box, true);
  } else {
    const cuuint64_t dims[5] = {K, (cuuint64_t)a.N, 1, 1, (cuuint64_t)a.E};
    const cuuint64_t strides[4] = {K, K * a.N, K * a.N, K * a.N};
    const cuuint32_t box[5] = {128, w_rows, 1, 1, 1};
    ok = make_map(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, mem.w, dims, strides, box, true);
  }
  {
    const cuuint64_t dims[2] = {K, (cuuint64_t)a.P};
    const cuuint64_t strides[1] = {K};
    const cuuint32_t box[2] = {128, (cuuint32_t)a.box};
    ok = ok && make_map(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, mem.x, dims, strides, box, true);
  }
  to = tx;
  if (CG == 2 && !a.quant && a.whole) {
    const int size = a.out_f32 ? 4 : 2;
    const cuuint64_t dims[2] = {(cuuint64_t)a.cols, (cuuint64_t)a.P}, strides[1] = {(cuuint64_t)a.cols * size};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / size), 32};
    ok = ok && make_map(&to, a.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.out, dims, strides, box, true);
  }
  if (!ok) return fail(MOE_ECUDA, "cuTensorMapEncodeTiled failed");

  // at most every token tile the rows can make, on every weight block
  const int64_t tiles = (a.P + (int64_t)(128 * CG - 1) * std::min(a.P, a.E)) / (128 * CG), most = tiles * a.m_blocks;
  if (most > 0x7fffffff) return fail(MOE_EINVAL, "P = %d rows of N = %d columns are too many tiles", a.P, a.N);
  a.most_tiles = (int)tiles;
  static bool allowed[64] = {};   // the kernel's shared memory and registers, once per device
  int dev = 0;
  CK(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return fail(MOE_EINVAL, "device %d is out of range", dev);
  if (!allowed[dev]) {
    cudaFuncAttributes attr;
    CK(cudaFuncGetAttributes(&attr, kernel));
    if (attr.numRegs < LAUNCH_REGS) return fail(MOE_ECUDA, "the kernel was built with %d registers, %d are shared out", attr.numRegs, LAUNCH_REGS);
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
  CK(cudaLaunchKernelEx(&cfg, kernel, tw, tx, to, a));
  return MOE_OK;
}

// Pairs of CTAs take twice the tokens with the same weight rows, and store their tiles under the next one's products; single ones waste less on
// ragged tiles.  us, pairs / single, by the experts' mean rows, spread as a router spreads them (bursts; in brackets loops of 0.7 s,
// where power bounds both and pairs gain):
//   K 768, N 2048, 128 experts                256 86 / 81, 384 111 / 112, 512 136 / 143, 1024 233 / 267
//   K 2048, N 2048, 128                       384 217 / 211, 704 347 / 346 (387 / 406), 1024 466 / 482
//   K 7168, N 4096, 32                        512 416 / 405, 704 531 / 519 (604 / 615), 1024 733 / 734 (829 / 873)
//   K 7168, N 4096, 32, SwiGLU                512 445 / 415, 704 539 / 538 (608 / 638), 1024 749 / 729 (857 / 866)
//   K 2048, N 1536, 128, requantised          512 219 / 201, 1024 385 / 369 (416 / 418), 1536 552 / 533 (597 / 599), 2048 709 / 696 (766 / 783)
// Experts of 512 rows each, no tile ragged, are faster in pairs already (111 / 133, 222 / 241, 350 / 374, 355 / 373 in the order above); a
// rule on sizes does not see that.  Nor does this one see how many items there are: one matrix of 1001 rows, K 7168, N 2048 takes
// 26 us in 32 pairs, 19 single.
bool use_pairs8(const Args8& a) { return a.P > (int64_t)(a.act ? a.K >= 4096 ? 704 : 1536 : a.K <= 1024 ? 384 : 704) * a.E; }

// Weight rows of a single CTA's tile: as many as leave items for half of the SMs.  With one tile a unit a call lasts as long as its slices take in
// turn, a quarter of a microsecond and more.  us with 256, 128 and 64 rows: one row, K 7168, N 4096 23.0 / 17.2 / 15.6; 256 rows, K 2048,
// N 7168 10.8 / 9.0 / 11.5; one row of 8 experts, K 768, N 2048 7.4 / 6.8 / 7.8.
int tile8(const Args8& a, int64_t tiles, int sms) {
  if (a.quant) return 256;   // a block of 128 features is one tile's
  int tile = 256;
  while (tile > 64 && tiles * ((a.N + tile - 1) / tile) < sms / 2) tile /= 2;
  return tile;
}

// what a call runs on a device of so many SMs
struct Form8 { int ctas, tile; };
Form8 form8(const Args8& a, int sms) {
  if (use_pairs8(a)) return Form8{2, 256};
  return Form8{1, tile8(a, (a.P + 127 * (int64_t)std::min(a.P, a.E)) / 128, sms)};
}

}  // namespace

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
  a.err = operator_flag();
  if (!a.err) return fail(MOE_ECUDA, "the library's flag has no address on this device");
  const Mem8 mem{x_codes, w_codes};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Form8 f = form8(a, operator_sms());
  return f.ctas == 2 ? launch8<2, 256>(a, mem, s) : f.tile == 256 ? launch8<1, 256>(a, mem, s) : f.tile == 128 ? launch8<1, 128>(a, mem, s) : launch8<1, 64>(a, mem, s);
}

extern "C" void moe_product8_form(int32_t P, int32_t E, int32_t N, int32_t K, int32_t act, int32_t quant, int32_t sms, int32_t* form) {
  Args8 a{};
  a.P = P; a.E = E; a.N = N; a.K = K; a.act = act; a.quant = quant;
  const Form8 f = form8(a, sms);
  const Room8 m = f.ctas == 2 ? room8<2, 256>(P, E) : f.tile == 256 ? room8<1, 256>(P, E) : f.tile == 128 ? room8<1, 128>(P, E) : room8<1, 64>(P, E);
  form[0] = f.ctas;
  form[1] = f.tile;
  form[2] = m.stages;
  form[3] = f.tile == 256 ? accs<256>() : f.tile == 128 ? accs<128>() : accs<64>();
}
