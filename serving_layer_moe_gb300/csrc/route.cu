// The router, the grouping of (token, expert) pairs by expert, and the weighted
// sum of the experts' rows (include/moe_operators.h: moe_route, moe_group_pairs,
// moe_combine).
//
// Router: one warp per token.  A lane holds E / 32 neighbouring scores in registers as
// order-preserving integers, and its two best; each of the k picks is a warp-wide integer
// maximum, and the lowest lane that holds it gives it up, so equal scores go to the lower
// index and the result is the same on every run.
//
// Grouping is a stable counting sort of the T*k pairs by expert in three launches: the
// router's blocks count the pairs they pick per expert, those counts become starts, and
// blocks rank their own pairs, 32 at a time by match.  Ranks follow the pair index, so no
// atomic decides an order.  Calls of at most 256 pairs of 32 tokens do all of it, router
// included, in one block, where a pair counts the pairs before it in expert order; pairs
// that come with their ids up to 256, whatever their tokens.
//
// Bounds: a prompt chunk of 8192 tokens and 256 experts reads 8.4 MB of logits; one
// decoded token is one launch's latency.
#include "operators.cuh"

#include <algorithm>
#include <type_traits>

namespace moe {

namespace {

constexpr int ROUTE_THREADS = 256;          // 8 warps, a token each at a time
constexpr int ROUTE_WARPS = ROUTE_THREADS / 32;
constexpr int PLACE_THREADS = 256;          // 8 warps rank a segment of pairs each
constexpr int PLACE_WARPS = PLACE_THREADS / 32;
constexpr int kMaxBlocks = 1024;            // counting blocks
// Up to here one block groups; and routes, up to kSmallTokens, four a warp.  us of one block / of three launches: top-8 of 128
// experts, 1 token 2.8 / 5.8, 16 tokens 5.3 / 7.0, 32 tokens 9.8 / 7.3; best of 128, 32 tokens 5.0 / 5.9, 64 tokens 8.8 / 5.9, 256
// tokens 32 / 6.4; best of 4096, 32 tokens 31 / 25, 256 tokens 146 / 27.
constexpr int kSmallPairs = 256, kSmallTokens = 32;

struct RouteArgs {
  int T, E, k, scoring, n_group, topk_group, renorm, tokens_per_block, bf16;
  float scale;
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* w;
  int32_t *offsets, *tiles, *order, *place;   // NULL: no grouping
  int32_t* counts;                            // [blocks, E + 1] pairs of each block of each expert; bin E: dropped ones
};

// larger float <=> larger integer; -0 and +0 are one value; NaN is below -inf
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 1u;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}

__device__ __forceinline__ float warp_sum(float v) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// the softmax numerator, with the row's largest value taken out; infinities and NaN as the header says
__device__ __forceinline__ float softmax_term(float l, float top) {
  if (!(l > -INFINITY)) return 0.0f;
  return expf(fminf(l, 3.402823466e38f) - top);
}
__device__ __forceinline__ float sigmoid_of(float l) { return 1.0f / (1.0f + expf(-l)); }

// a row's logit e
__device__ __forceinline__ float logit_at(const RouteArgs& a, size_t at) {
  return a.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[at]) : static_cast<const float*>(a.logits)[at];
}

// Routes token t; lane j % 32 hands pick j to `found(j, expert)`.  FULL: NPL experts to every lane, on addresses that hold
// logits and bias four (or two) at a time.  scratch [E + E / 32 + 1]: the warp's, where not FULL or the groups are not whole lanes.
template <int NPL, bool FULL, typename F>
__device__ __forceinline__ void route_token(const RouteArgs& a, int t, float* scratch, F found) {
  constexpr int U = NPL >= 4 ? 4 : 2;
  const int lane = threadIdx.x & 31, per = FULL ? NPL : (a.E + 31) / 32, e0 = lane * per;
  const size_t row = (size_t)t * a.E;
  auto has = [&](int i) { return FULL || (i < per && e0 + i < a.E); };
  alignas(16) float v[NPL];
  if constexpr (FULL) {
    if (a.bf16) {
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.logits) + row + e0;
#pragma unroll
      for (int i = 0; i < NPL; i += U) {
        alignas(8) __nv_bfloat16 x[U];
        if constexpr (U == 4) *reinterpret_cast<uint2*>(x) = *reinterpret_cast<const uint2*>(src + i);
        else *reinterpret_cast<uint32_t*>(x) = *reinterpret_cast<const uint32_t*>(src + i);
#pragma unroll
        for (int u = 0; u < U; ++u) v[i + u] = __bfloat162float(x[u]);
      }
    } else {
      const float* src = static_cast<const float*>(a.logits) + row + e0;
#pragma unroll
      for (int i = 0; i < NPL; i += U) {
        if constexpr (U == 4) *reinterpret_cast<float4*>(v + i) = *reinterpret_cast<const float4*>(src + i);
        else *reinterpret_cast<float2*>(v + i) = *reinterpret_cast<const float2*>(src + i);
      }
    }
  } else {
    for (int e = lane; e < a.E; e += 32) scratch[e + (e >> 5)] = logit_at(a, row + e);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < NPL; ++i) v[i] = has(i) ? scratch[e0 + i + ((e0 + i) >> 5)] : 0.0f;
    __syncwarp();
  }

  uint32_t key[NPL];   // 0: no expert, or one that may not be picked
  if (a.scoring != 0) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) v[i] = sigmoid_of(v[i]);
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < NPL; i += U) {
        alignas(16) float b[U];
        if constexpr (!FULL) {
#pragma unroll
          for (int u = 0; u < U; ++u) b[u] = has(i + u) ? __ldg(a.bias + e0 + i + u) : 0.0f;
        } else if constexpr (U == 4) {
          *reinterpret_cast<float4*>(b) = __ldg(reinterpret_cast<const float4*>(a.bias + e0 + i));
        } else {
          *reinterpret_cast<float2*>(b) = __ldg(reinterpret_cast<const float2*>(a.bias + e0 + i));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) v[i + u] += b[u];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NPL; ++i) key[i] = has(i) ? order_key(v[i]) : 0u;

  // a group is a power of two of whole lanes: its two best come from the lanes' own two best, below
  const bool lanes = a.n_group > 1 && a.E == 32 * per && !(a.n_group & (a.n_group - 1));
  // score of a group: the sum of its two best; a NaN (key 1) or an absent second value adds nothing, a group of NaN ranks last
  auto live_groups = [&](int sub, uint32_t b1, uint32_t b2) {
    for (int o = 1; o < sub; o <<= 1) {
      const uint32_t c1 = __shfl_xor_sync(0xffffffffu, b1, o), c2 = __shfl_xor_sync(0xffffffffu, b2, o);
      b2 = max(min(b1, c1), max(b2, c2));
      b1 = max(b1, c1);
    }
    uint32_t gkey = 0u, live = 0u;
    if (lane / sub < a.n_group && lane % sub == 0)
      gkey = b1 <= 1u ? 1u : order_key(b2 <= 1u ? key_value(b1) : key_value(b1) + key_value(b2));
    for (int r = 0; r < a.topk_group; ++r) {
      const uint32_t best = __reduce_max_sync(0xffffffffu, gkey);
      const int who = __ffs(__ballot_sync(0xffffffffu, gkey == best)) - 1;
      live |= 1u << (who / sub);
      if (lane == who) gkey = 0u;
    }
    return live;
  };
  if (a.n_group > 1 && !lanes) {
    // a power of two of lanes looks through each group
    const int gs = a.E / a.n_group;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (has(i)) scratch[e0 + i + ((e0 + i) >> 5)] = __uint_as_float(key[i]);
    __syncwarp();
    int sub = 1;
    while (2 * sub * a.n_group <= 32) sub *= 2;
    const int g = lane / sub;
    uint32_t b1 = 0u, b2 = 0u;
    if (g < a.n_group)
      for (int i = lane % sub; i < gs; i += sub) {
        const int e = g * gs + i;
        const uint32_t x = __float_as_uint(scratch[e + (e >> 5)]);
        b2 = max(min(b1, x), b2);
        b1 = max(b1, x);
      }
    const uint32_t live = live_groups(sub, b1, b2);
    const float step = 1.0f / (float)gs;
#pragma unroll
    for (int i = 0; i < NPL; ++i)   // e / gs: e < 4096 and half a unit away from the next quotient
      if (!((live >> (min((int)(((float)(e0 + i) + 0.5f) * step), 31))) & 1u)) key[i] = 0u;
    __syncwarp();
  }

  // A lane keeps its two best, m1 at i1 and m2 at i2 (the lower index where they are equal), of its experts that come after
  // (last, at_last) in that order: what it has lost needs no mark, and it looks through its keys again only after two losses.
  uint32_t m1, m2;
  int i1, i2, kept;
  auto best_two = [&](auto all, uint32_t last, int at_last) {
    m1 = m2 = 0u;
    i1 = i2 = 0;
    kept = 2;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const uint32_t x = decltype(all)::value || key[i] < last || (key[i] == last && i > at_last) ? key[i] : 0u;
      const bool first = x > m1, second = x > m2;
      i2 = first ? i1 : second ? i : i2;
      m2 = max(min(m1, x), m2);
      i1 = first ? i : i1;
      m1 = max(m1, x);
    }
  };
  best_two(std::true_type{}, 0u, 0);
  if (lanes) {
    const int sub = 32 / a.n_group;
    if (!((live_groups(sub, m1, m2) >> (lane / sub)) & 1u)) m1 = 0u;
  }

  // the largest score of a softmax row is the first pick's
  float top = 0.0f, denom = 0.0f, sum = 0.0f;
  auto term_of = [&](uint32_t x) { return x <= 1u ? 0.0f : softmax_term(key_value(x), top); };
  if (a.scoring == 0) {
    const uint32_t best = __reduce_max_sync(0xffffffffu, m1);
    top = best <= 1u ? 0.0f : fminf(key_value(best), 3.402823466e38f);
    if (!a.renorm) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) denom += term_of(key[i]);
      denom = warp_sum(denom);
    }
  }

  // The k picks: the warp's largest key, of the lowest lane that has it.  Lane j % 32 keeps pick j.
  int32_t* ids = a.ids + (size_t)t * a.k;
  float* w = a.w + (size_t)t * a.k;
  const bool divide = a.renorm || a.scoring == 0;
  auto gate = [&](float x) { return (divide ? (denom > 0.0f ? x / denom : 0.0f) : x) * a.scale; };
  for (int j0 = 0; j0 < a.k; j0 += 32) {
    const int nj = min(32, a.k - j0);
    int my_at = 0;
    uint32_t my_key = 0u;
    for (int j = 0; j < nj; ++j) {
      const uint32_t best = __reduce_max_sync(0xffffffffu, m1);
      const int who = __ffs(__ballot_sync(0xffffffffu, m1 == best)) - 1;
      const int at = __shfl_sync(0xffffffffu, e0 + i1, who);
      if (lane == j) { my_at = at; my_key = best; }
      if (lane == who) {
        if (--kept == 0) {
          best_two(std::false_type{}, best, i1);
        } else {
          m1 = m2;
          i1 = i2;
        }
      }
    }
    float term = 0.0f;
    if (lane < nj) {
      if (a.scoring == 0) term = term_of(my_key);
      else if (!a.bias) term = my_key <= 1u ? 0.0f : key_value(my_key);
      else if (my_key > 1u) term = sigmoid_of(logit_at(a, row + my_at));   // the gate has no bias in it
      ids[j0 + lane] = my_at;
      found(j0 + lane, my_at);
    }
    if (a.renorm) sum += warp_sum(term);
    if (a.k <= 32) {
      if (a.renorm) denom = sum;
      if (lane < nj) w[lane] = gate(term);
      return;
    }
    if (lane < nj) w[j0 + lane] = term;
  }
  if (a.renorm) denom = sum;
  for (int j = lane; j < a.k; j += 32) w[j] = gate(w[j]);   // its own picks
}

// Exclusive prefixes over the E + 1 bins of `count` by a block of 256 threads: of the counts into `first` (and `offsets`), of
// ceil(count / 128) into `tiles`.  A thread adds up a run of bins, the threads' sums are scanned by shuffles.  Bin E, the
// dropped pairs, comes last, so first[E] is the number of rows.
__device__ __forceinline__ void scan_bins(const int32_t* count, int E, int32_t* first, int32_t* offsets, int32_t* tiles) {
  __shared__ int2 warps[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (E + 1 + 255) / 256, e0 = threadIdx.x * per, e1 = min(E + 1, e0 + per);
  int c = 0, t = 0;
  for (int e = e0; e < e1; ++e) { c += count[e]; t += (count[e] + 127) >> 7; }
  int x = c, y = t;
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) { x += u; y += v; }
  }
  if (lane == 31) warps[warp] = make_int2(x, y);
  __syncthreads();
  x -= c;
  y -= t;
#pragma unroll
  for (int w = 0; w < 8; ++w)
    if (w < warp) { x += warps[w].x; y += warps[w].y; }
  for (int e = e0; e < e1; ++e) {
    first[e] = x;
    if (offsets) { offsets[e] = x; tiles[e] = y; }
    x += count[e];
    y += (count[e] + 127) >> 7;
  }
}

// Groups at most kSmallPairs pairs in one block.  smem: the pairs' bins [kSmallPairs], count [E + 1], room for starts [E + 1].
__device__ __forceinline__ void group_small(int P, int E, int32_t* offsets, int32_t* tiles, int32_t* order, int32_t* place,
                                            int32_t* smem) {
  const int32_t* id = smem;
  const int32_t* count = id + kSmallPairs;
  int32_t* first = smem + kSmallPairs + E + 1;
  const int p = threadIdx.x;      // blockDim.x >= kSmallPairs
  if (p < P) {
    const int mine = id[p];
    int row = 0;
    for (int i = 0; i < P; ++i) row += id[i] < mine || (id[i] == mine && i < p);
    order[row] = mine < E ? p : -1;
    place[p] = mine < E ? row : -1;
  }
  scan_bins(count, E, first, offsets, tiles);
}

// Registers for 5 blocks an SM (3 with 16 scores a lane): 8192 tokens of 256 experts in 4 of 8 groups take 10.7 us, 11.4 without a
// bound, 10.9 with 6 blocks; 8192 tokens of 384 experts 13.7, 17.1 with 2.
template <int NPL, bool FULL>
__global__ void __launch_bounds__(ROUTE_THREADS, NPL <= 8 ? 5 : NPL == 16 ? 3 : 1) route_kernel(RouteArgs a, int scratch_at) {
  extern __shared__ int32_t smem[];
  // the block's own pairs by expert; a block that groups them all keeps their bins before that
  const bool small = a.offsets && !a.counts;
  int32_t* count = smem + (small ? kSmallPairs : 0);
  if (a.offsets)
    for (int i = threadIdx.x; i <= a.E; i += ROUTE_THREADS) count[i] = 0;
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  const int warp = threadIdx.x >> 5;
  const int t0 = blockIdx.x * a.tokens_per_block, t1 = min(a.T, t0 + a.tokens_per_block);
  float* scratch = reinterpret_cast<float*>(smem + scratch_at) + (size_t)warp * (a.E + a.E / 32 + 1);
  for (int t = t0 + warp; t < t1; t += ROUTE_WARPS)
    route_token<NPL, FULL>(a, t, scratch, [&](int j, int e) {
      if (!a.offsets) return;
      atomicAdd(&count[e], 1);
      if (small) smem[t * a.k + j] = e;
    });
  if (!a.offsets) return;
  __syncthreads();
  if (small) group_small(a.T * a.k, a.E, a.offsets, a.tiles, a.order, a.place, smem);
  else
    for (int i = threadIdx.x; i <= a.E; i += ROUTE_THREADS) a.counts[(size_t)blockIdx.x * (a.E + 1) + i] = count[i];
}

__global__ void __launch_bounds__(ROUTE_THREADS)
count_kernel(const int32_t* __restrict__ ids, int P, int E, int per_block, int32_t* __restrict__ counts) {
  extern __shared__ int32_t smem[];
  for (int i = threadIdx.x; i <= E; i += ROUTE_THREADS) smem[i] = 0;
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  const int p0 = blockIdx.x * per_block, p1 = min(P, p0 + per_block);
  for (int p = p0 + threadIdx.x; p < p1; p += ROUTE_THREADS) {
    const int e = ids[p];
    atomicAdd(&smem[(unsigned)e < (unsigned)E ? e : E], 1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i <= E; i += ROUTE_THREADS) counts[(size_t)blockIdx.x * (E + 1) + i] = smem[i];
}

__global__ void __launch_bounds__(ROUTE_THREADS)
group_small_kernel(const int32_t* __restrict__ ids, int P, int E, int32_t* offsets, int32_t* tiles, int32_t* order, int32_t* place) {
  extern __shared__ int32_t smem[];
  int32_t* count = smem + kSmallPairs;
  for (int e = threadIdx.x; e <= E; e += ROUTE_THREADS) count[e] = 0;
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  if (threadIdx.x < P) {
    const int e = ids[threadIdx.x], bin = (unsigned)e < (unsigned)E ? e : E;
    smem[threadIdx.x] = bin;
    atomicAdd(&count[bin], 1);
  }
  __syncthreads();
  group_small(P, E, offsets, tiles, order, place, smem);
}

// counts [blocks, E + 1] -> what comes before each block, in place, and each expert's total.  A block of 1024 threads takes 8
// bins, a sector of each row; a thread holds the counts of a run of at most kMaxBlocks / 128 blocks.
__global__ void __launch_bounds__(1024) starts_kernel(int32_t* __restrict__ counts, int E, int blocks, int32_t* __restrict__ total) {
  constexpr int ROWS = kMaxBlocks / 128;
  __shared__ int32_t sums[32][8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, bin = lane & 7, e = blockIdx.x * 8 + bin;
  const int rows = (blocks + 127) / 128, r0 = (int)(threadIdx.x >> 3) * rows, n = e <= E ? min(rows, blocks - r0) : 0;
  int32_t* at = counts + (size_t)r0 * (E + 1) + e;
  pdl_wait();
  pdl_trigger();
  int c[ROWS], sum = 0;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) c[r] = r < n ? at[(size_t)r * (E + 1)] : 0;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) sum += c[r];
  int run = sum;   // over the warp's four runs of the bin
  for (int o = 8; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += u;
  }
  if (lane >= 24) sums[warp][bin] = run;
  __syncthreads();
  run -= sum;
#pragma unroll
  for (int w = 0; w < 32; ++w) run += w < warp ? sums[w][bin] : 0;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    if (r < n) at[(size_t)r * (E + 1)] = run;
    run += c[r];
  }
  if (threadIdx.x >= 1016 && e <= E) total[e] = run;
}

// Ranks the pairs of `per` counting blocks; warps take consecutive segments.  smem: start [E + 1], total [E + 1], a count per
// warp and bin.
__global__ void __launch_bounds__(PLACE_THREADS)
place_kernel(const int32_t* __restrict__ ids, int P, int E, int per_block, int per, const int32_t* __restrict__ starts,
             const int32_t* __restrict__ totals, int32_t* offsets, int32_t* tiles, int32_t* __restrict__ order, int32_t* __restrict__ place) {
  extern __shared__ int32_t smem[];
  const int bins = E + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t* start = smem;
  int32_t* total = start + bins;
  int32_t* cnt = total + bins;
  for (int i = threadIdx.x; i < PLACE_WARPS * bins; i += PLACE_THREADS) cnt[i] = 0;
  pdl_wait();
  pdl_trigger();
  const int p0 = blockIdx.x * per * per_block, p1 = min(P, p0 + per * per_block);
  const int seg = ((p1 - p0 + PLACE_WARPS - 1) / PLACE_WARPS + 31) & ~31;
  const int s0 = p0 + warp * seg, s1 = min(p1, s0 + seg);
  int32_t* mine = cnt + warp * bins;
  for (int e = threadIdx.x; e < bins; e += PLACE_THREADS) total[e] = totals[e];
  __syncthreads();
  scan_bins(total, E, start, blockIdx.x == 0 ? offsets : nullptr, tiles);
  for (int p = s0; p < s1; p += 32) {
    const int q = p + lane;
    int e = q < s1 ? __ldg(ids + q) : -2;
    if (q < s1 && (unsigned)e >= (unsigned)E) e = E;
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    if (q < s1 && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  for (int e = threadIdx.x; e < bins; e += PLACE_THREADS) {
    int run = start[e] + starts[(size_t)blockIdx.x * per * bins + e];
#pragma unroll
    for (int w = 0; w < PLACE_WARPS; ++w) {
      const int c = cnt[w * bins + e];
      cnt[w * bins + e] = run;
      run += c;
    }
  }
  __syncthreads();
  for (int p = s0; p < s1; p += 32) {
    const int q = p + lane;
    int e = q < s1 ? __ldg(ids + q) : -2;
    if (q < s1 && (unsigned)e >= (unsigned)E) e = E;
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    if (q < s1) {
      const int row = mine[e] + __popc(same & ((1u << lane) - 1u));
      order[row] = e < E ? q : -1;
      place[q] = e < E ? row : -1;
    }
    __syncwarp();
    if (q < s1 && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
  }
}

// out[t, n] = sum_j w[t, j] y[place[t, j], n], in j order: V columns a thread.  Four rows' loads are in flight before the first is
// used: 4096 tokens, 8 experts, N 7168 in bf16 take 89 us a row at a time, 81 so, 102 by eights, whose registers cost warps.
constexpr int COMBINE_ROWS = 4;
template <typename Y, typename O, int V>
__global__ void __launch_bounds__(256)
combine_kernel(int T, int k, int N, const Y* __restrict__ y, const int32_t* __restrict__ place,
               const float* __restrict__ w, O* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const int cols = N / V, rows = T * k;
  const int64_t units = (int64_t)T * cols;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < units; u += (int64_t)gridDim.x * 256) {
    // a 64-bit division only where it is needed (4 us of 85)
    const int t = units <= 0x7fffffff ? (int)((uint32_t)u / (uint32_t)cols) : (int)(u / cols), c = (int)(u - (int64_t)t * cols) * V;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += COMBINE_ROWS) {
      alignas(16) Y tmp[COMBINE_ROWS][V];
      int row[COMBINE_ROWS];
      float g[COMBINE_ROWS];
#pragma unroll
      for (int j = 0; j < COMBINE_ROWS; ++j) {
        row[j] = j0 + j < k ? __ldg(place + (size_t)t * k + j0 + j) : -1;
        g[j] = j0 + j < k ? __ldg(w + (size_t)t * k + j0 + j) : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < COMBINE_ROWS; ++j) {
        if ((unsigned)row[j] >= (unsigned)rows) continue;
        const Y* src = y + (size_t)row[j] * N + c;
        if constexpr (sizeof(Y) * V % 16 == 0) {
#pragma unroll
          for (int i = 0; i < (int)sizeof(Y) * V / 16; ++i) reinterpret_cast<uint4*>(tmp[j])[i] = __ldg(reinterpret_cast<const uint4*>(src) + i);
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) tmp[j][i] = src[i];
        }
      }
#pragma unroll
      for (int j = 0; j < COMBINE_ROWS; ++j) {
        if ((unsigned)row[j] >= (unsigned)rows) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(g[j], (float)tmp[j][i], acc[i]);
      }
    }
    alignas(16) O res[V];
#pragma unroll
    for (int i = 0; i < V; ++i) res[i] = (O)acc[i];
    O* dst = out + (size_t)t * N + c;
    if constexpr (sizeof(O) * V == 16) *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<uint4*>(res);
    else if constexpr (sizeof(O) * V == 32) {
      reinterpret_cast<uint4*>(dst)[0] = reinterpret_cast<uint4*>(res)[0];
      reinterpret_cast<uint4*>(dst)[1] = reinterpret_cast<uint4*>(res)[1];
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) dst[i] = res[i];
    }
  }
}

template <typename Y, typename O>
cudaError_t launch_combine_rows(int T, int k, int N, const void* y, const int32_t* place, const float* w, void* out,
                                cudaStream_t s) {
  const bool wide = N % 8 == 0;   // every row of y and out starts on 16 bytes
  const int64_t units = (int64_t)T * (wide ? N / 8 : N);
  const int grid = (int)std::min<int64_t>((units + 255) / 256, (int64_t)operator_sms() * 32);
  return wide ? launch_pdl(combine_kernel<Y, O, 8>, dim3(grid), dim3(256), 0, s, T, k, N, (const Y*)y, place, w, (O*)out)
              : launch_pdl(combine_kernel<Y, O, 1>, dim3(grid), dim3(256), 0, s, T, k, N, (const Y*)y, place, w, (O*)out);
}

// tokens of one counting block when T tokens are spread over at most kMaxBlocks
int tokens_per_block(int T) { return ROUTE_WARPS * std::max(1, (T + ROUTE_WARPS * kMaxBlocks - 1) / (ROUTE_WARPS * kMaxBlocks)); }
bool small_group(int64_t T, int64_t k) { return T * k <= kSmallPairs; }
bool small_route(int64_t T, int64_t k) { return small_group(T, k) && T <= kSmallTokens; }

moe_status check_group_args(int32_t T, int64_t need, const void* offsets, const void* tiles, const void* order,
                            const void* place, const void* ws, int64_t ws_bytes) {
  if (!offsets || !tiles || (T > 0 && (!order || !place)))
    return fail(MOE_EINVAL, "offsets, tiles, order and place are all needed for grouping");
  if (!aligned_to(offsets, 4) || !aligned_to(tiles, 4) || !aligned_to(order, 4) || !aligned_to(place, 4) || !aligned_to(ws, 4))
    return fail(MOE_EINVAL, "offsets, tiles, order, place and workspace must be 4-byte aligned");
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(MOE_EINVAL, "workspace holds %lld bytes, %lld are needed", (long long)ws_bytes, (long long)need);
  return MOE_OK;
}

moe_status check_sizes(int32_t T, int32_t E, int32_t k) {
  if (T < 0 || E < 1 || E > kMaxExperts || k < 1) return fail(MOE_EINVAL, "T >= 0, 1 <= E <= %d and k >= 1 are needed, got T %d, E %d, k %d", kMaxExperts, T, E, k);
  if ((int64_t)T * k > kMaxPairs) return fail(MOE_EINVAL, "T * k = %lld pairs do not fit 31 bits with room for a block", (long long)T * k);
  return MOE_OK;
}

cudaError_t allow_smem(const void* fn, size_t bytes) {
  if (bytes <= 48 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

size_t small_smem(int E) { return (size_t)(kSmallPairs + 2 * (E + 1)) * 4; }

template <int NPL>
moe_status run_route(const RouteArgs& a, int blocks, cudaStream_t s) {
  constexpr int U = NPL >= 4 ? 4 : 2;
  const bool full = a.E == 32 * NPL && aligned_to(a.logits, U * (a.bf16 ? 2 : 4)) && aligned_to(a.bias, 4 * U);
  const bool whole_lanes = a.n_group == 1 || (a.E % 32 == 0 && !(a.n_group & (a.n_group - 1)));
  const size_t bins = !a.offsets ? 0 : a.counts ? (size_t)(a.E + 1) * 4 : small_smem(a.E);
  const size_t smem = bins + (full && whole_lanes ? 0 : (size_t)ROUTE_WARPS * (a.E + a.E / 32 + 1) * 4);
  const auto kernel = full ? route_kernel<NPL, true> : route_kernel<NPL, false>;
  CK(allow_smem((const void*)kernel, smem));
  CK(launch_pdl(kernel, dim3(blocks), dim3(ROUTE_THREADS), smem, s, a, (int)(bins / 4)));
  return MOE_OK;
}

// counts [blocks, E + 1] of the blocks' pairs -> the grouping; the totals follow the counts in the workspace
moe_status run_place(const int32_t* ids, int P, int E, int per_block, int blocks, int32_t* counts, int32_t* offsets, int32_t* tiles,
                     int32_t* order, int32_t* place, cudaStream_t s) {
  int32_t* total = counts + (size_t)(E + 1) * blocks;
  CK(launch_pdl(starts_kernel, dim3((E + 8) / 8), dim3(1024), 0, s, counts, E, blocks, total));
  const size_t smem = (size_t)(2 + PLACE_WARPS) * (E + 1) * 4;
  CK(allow_smem((const void*)place_kernel, smem));
  const int per = std::max(1, PLACE_THREADS / per_block);   // about a pair a thread
  CK(launch_pdl(place_kernel, dim3((blocks + per - 1) / per), dim3(PLACE_THREADS), smem, s, ids, P, E, per_block, per,
                (const int32_t*)counts, (const int32_t*)total, offsets, tiles, order, place));
  return MOE_OK;
}

moe_status run_small(const int32_t* ids, int P, int E, int32_t* offsets, int32_t* tiles, int32_t* order, int32_t* place, cudaStream_t s) {
  const size_t smem = small_smem(E);
  CK(allow_smem((const void*)group_small_kernel, smem));
  CK(launch_pdl(group_small_kernel, dim3(1), dim3(ROUTE_THREADS), smem, s, ids, P, E, offsets, tiles, order, place));
  return MOE_OK;
}

}  // namespace

int operator_sms() {
  static int sms[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  if (!sms[dev]) {
    int n = 1;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    sms[dev] = n;
  }
  return sms[dev];
}

}  // namespace moe

using namespace moe;

extern "C" int64_t moe_grouped_tiles(int64_t P, int32_t E) { return P < 0 || E < 0 ? 0 : (P + 127 * std::min<int64_t>(P, E)) / 128; }

extern "C" int64_t moe_group_workspace(int32_t T, int32_t k, int32_t E) {
  if (T <= 0 || k < 0 || E < 0 || small_route(T, k)) return 0;
  const int64_t blocks = (T + tokens_per_block(T) - 1) / tokens_per_block(T);
  return (blocks + 1) * ((int64_t)E + 1) * 4;
}

extern "C" moe_status moe_route(int32_t T, int32_t E, int32_t k, int32_t logits_dtype, const void* logits, int32_t scoring,
                                const float* bias, int32_t n_group, int32_t topk_group, int32_t renormalize, float scale,
                                int32_t* ids, float* w, int32_t* offsets, int32_t* tiles, int32_t* order, int32_t* place,
                                void* workspace, int64_t workspace_bytes, void* stream) {
  moe_status st = check_sizes(T, E, k);
  if (st != MOE_OK) return st;
  if (k > E) return fail(MOE_EINVAL, "k = %d is more than E = %d", k, E);
  if (logits_dtype != MOE_F32 && logits_dtype != MOE_BF16) return fail(MOE_EINVAL, "logits_dtype must be MOE_F32 or MOE_BF16");
  if (scoring != 0 && scoring != 1) return fail(MOE_EINVAL, "scoring must be 0 (softmax) or 1 (sigmoid)");
  if (scoring == 0 && (bias || n_group != 1)) return fail(MOE_EINVAL, "softmax scoring takes no bias and n_group = 1");
  if (n_group < 1 || n_group > 32 || E % n_group || topk_group < 1 || topk_group > n_group ||
      (int64_t)topk_group * (E / n_group) < k)
    return fail(MOE_EINVAL, "n_group = %d (1 to 32) must divide E = %d and topk_group = %d of them hold k = %d experts",
                n_group, E, topk_group, k);
  const bool group = offsets || tiles || order || place;
  if (group && (st = check_group_args(T, moe_group_workspace(T, k, E), offsets, tiles, order, place, workspace, workspace_bytes)) != MOE_OK) return st;
  if (T > 0 && (!logits || !ids || !w)) return fail(MOE_EINVAL, "logits, topk_ids and topk_w must not be NULL");
  if (!aligned_to(logits, logits_dtype == MOE_F32 ? 4 : 2) || !aligned_to(bias, 4) || !aligned_to(ids, 4) || !aligned_to(w, 4))
    return fail(MOE_EINVAL, "logits, bias, topk_ids and topk_w must be aligned to their element size");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) return group ? run_small(nullptr, 0, E, offsets, tiles, order, place, s) : MOE_OK;
  RouteArgs a{};
  a.T = T; a.E = E; a.k = k; a.scoring = scoring; a.n_group = n_group; a.topk_group = topk_group;
  a.renorm = renormalize != 0; a.scale = scale; a.logits = logits; a.bias = bias; a.ids = ids; a.w = w;
  a.offsets = offsets; a.tiles = tiles; a.order = order; a.place = place;
  const bool small = group && small_route(T, k);
  a.counts = group && !small ? static_cast<int32_t*>(workspace) : nullptr;
  a.tokens_per_block = small ? T : tokens_per_block(T);
  const int blocks = (T + a.tokens_per_block - 1) / a.tokens_per_block;
  a.bf16 = logits_dtype == MOE_BF16;
  const int npl = (E + 31) / 32;
  st = npl <= 2 ? run_route<2>(a, blocks, s) : npl <= 4 ? run_route<4>(a, blocks, s) : npl <= 8 ? run_route<8>(a, blocks, s)
       : npl <= 16 ? run_route<16>(a, blocks, s) : npl <= 32 ? run_route<32>(a, blocks, s)
       : npl <= 64 ? run_route<64>(a, blocks, s) : run_route<128>(a, blocks, s);
  if (st != MOE_OK || !a.counts) return st;
  return run_place(ids, T * k, E, a.tokens_per_block * k, blocks, a.counts, offsets, tiles, order, place, s);
}

extern "C" moe_status moe_group_pairs(int32_t T, int32_t E, int32_t k, const int32_t* ids, int32_t* offsets, int32_t* tiles,
                                      int32_t* order, int32_t* place, void* workspace, int64_t workspace_bytes, void* stream) {
  moe_status st = check_sizes(T, E, k);
  if (st != MOE_OK) return st;
  if ((st = check_group_args(T, small_group(T, k) ? 0 : moe_group_workspace(T, k, E), offsets, tiles, order, place, workspace, workspace_bytes)) != MOE_OK) return st;
  if (T > 0 && !ids) return fail(MOE_EINVAL, "topk_ids must not be NULL");
  if (!aligned_to(ids, 4)) return fail(MOE_EINVAL, "topk_ids must be 4-byte aligned");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (small_group(T, k)) return run_small(ids, T * k, E, offsets, tiles, order, place, s);
  const int tpb = tokens_per_block(T), blocks = (T + tpb - 1) / tpb;
  int32_t* counts = static_cast<int32_t*>(workspace);
  const size_t smem = (size_t)(E + 1) * 4;
  CK(launch_pdl(count_kernel, dim3(blocks), dim3(ROUTE_THREADS), smem, s, ids, T * k, E, tpb * k, counts));
  return run_place(ids, T * k, E, tpb * k, blocks, counts, offsets, tiles, order, place, s);
}

extern "C" moe_status moe_combine(int32_t T, int32_t k, int32_t N, int32_t y_dtype, const void* y, const int32_t* place,
                                  const float* w, int32_t out_dtype, void* out, void* stream) {
  if (T < 0 || k < 1 || N < 1 || (int64_t)T * k > kMaxPairs)
    return fail(MOE_EINVAL, "T >= 0, k >= 1, N >= 1 and at most %lld pairs are needed, got T %d, k %d, N %d", (long long)kMaxPairs, T, k, N);
  if ((y_dtype != MOE_F32 && y_dtype != MOE_BF16) || (out_dtype != MOE_F32 && out_dtype != MOE_BF16))
    return fail(MOE_EINVAL, "y_dtype and out_dtype must be MOE_F32 or MOE_BF16");
  if (T == 0) return MOE_OK;
  if (!y || !place || !w || !out) return fail(MOE_EINVAL, "y, place, topk_w and out must not be NULL");
  const uintptr_t ya = N % 8 == 0 ? 16 : y_dtype == MOE_BF16 ? 2 : 4, oa = N % 8 == 0 ? 16 : out_dtype == MOE_BF16 ? 2 : 4;
  if (!aligned_to(y, ya) || !aligned_to(out, oa) || !aligned_to(place, 4) || !aligned_to(w, 4))
    return fail(MOE_EINVAL, "y and out must be 16-byte aligned (N a multiple of 8; else to their elements), place and topk_w 4-byte aligned");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool yb = y_dtype == MOE_BF16, ob = out_dtype == MOE_BF16;
  CK(yb ? (ob ? launch_combine_rows<__nv_bfloat16, __nv_bfloat16>(T, k, N, y, place, w, out, s)
              : launch_combine_rows<__nv_bfloat16, float>(T, k, N, y, place, w, out, s))
        : (ob ? launch_combine_rows<float, __nv_bfloat16>(T, k, N, y, place, w, out, s)
              : launch_combine_rows<float, float>(T, k, N, y, place, w, out, s)));
  return MOE_OK;
}
