// The router, the grouping of (token, expert) pairs by expert, and the weighted
// sum of the experts' rows (include/moe_operators.h: moe_route, moe_group_pairs,
// moe_combine).
//
// Router: one warp per token.  A lane holds E / 32 scores in registers as order-
// preserving integers; each of the k picks is a warp-wide integer maximum and then
// a minimum over the indices that hold it, so equal scores go to the lower index
// and the result is the same on every run.
//
// Grouping is a stable counting sort of the T*k pairs by expert in at most two
// launches: blocks of tokens count their pairs per expert (the router's blocks count
// what they have just picked), then each block adds up the counts of the blocks
// before it and ranks its own pairs, 32 at a time by match.  Ranks follow the pair
// index, so no atomic decides an order.  Calls whose pairs fit one block do all of
// it, router included, in one launch.
//
// Bounds: a prompt chunk of 8192 tokens and 256 experts reads 8.4 MB of logits; one
// decoded token is one launch's latency.
#include "operators.cuh"

#include <algorithm>

namespace moe {

namespace {

constexpr int ROUTE_THREADS = 256;          // 8 warps, a token each at a time
constexpr int ROUTE_WARPS = ROUTE_THREADS / 32;
constexpr int PLACE_THREADS = 512;          // 256 above 1024 experts: a count per warp and expert in shared memory
constexpr int kMaxBlocks = 304;             // two blocks on each of 152 SMs
constexpr int kOneBlockTokens = 32;         // up to here one block routes and groups

struct RouteArgs {
  int T, E, k, scoring, n_group, topk_group, renorm, tokens_per_block;
  float scale;
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* w;
  int32_t *offsets, *tiles, *order, *place;   // NULL: no grouping
  int32_t* counts;                            // [blocks, E + 1]
};

// larger float <=> larger integer; -0 and +0 are one value; NaN is below -inf
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 1u;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}

__device__ __forceinline__ float warp_max(float v) {
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
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
__device__ __forceinline__ float sigmoid_of(float l) { return l != l ? 0.0f : 1.0f / (1.0f + expf(-l)); }

template <int NPL>
__device__ __forceinline__ void route_token(const RouteArgs& a, int logits_bf16, int t, float* group_scratch) {
  const int lane = threadIdx.x & 31;
  float v[NPL];
  uint32_t key[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = i * 32 + lane;
    const size_t at = (size_t)t * a.E + e;
    v[i] = e >= a.E ? -INFINITY
           : logits_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[at])
                         : static_cast<const float*>(a.logits)[at];
  }
  float top = -INFINITY, denom = 0.0f;
  if (a.scoring == 0) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      key[i] = i * 32 + lane < a.E ? order_key(v[i]) : 0u;
      top = fmaxf(top, v[i]);   // fmaxf passes NaN over
    }
    top = fminf(warp_max(top), 3.402823466e38f);
    if (!a.renorm) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) denom += softmax_term(v[i], top);
      denom = warp_sum(denom);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = i * 32 + lane;
      const bool nan = v[i] != v[i];
      v[i] = sigmoid_of(v[i]);
      const float s = a.bias && e < a.E ? v[i] + a.bias[e] : v[i];
      key[i] = e >= a.E ? 0u : nan ? 1u : order_key(s);
    }
    if (a.n_group > 1) {
      // score of a group: the sum of its two best; a power of two of lanes looks through each group
      const int gs = a.E / a.n_group;
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const int e = i * 32 + lane;
        if (e < a.E) group_scratch[e + (e >> 5)] = __uint_as_float(key[i]);
      }
      __syncwarp();
      int sub = 1;
      while (2 * sub * a.n_group <= 32) sub *= 2;
      const int g = lane / sub, j = lane % sub;
      uint32_t b1 = 0u, b2 = 0u;
      if (g < a.n_group) {
        for (int i = j; i < gs; i += sub) {
          const int e = g * gs + i;
          const uint32_t x = __float_as_uint(group_scratch[e + (e >> 5)]);
          if (x > b1) { b2 = b1; b1 = x; }
          else if (x > b2) b2 = x;
        }
      }
      for (int o = 1; o < sub; o <<= 1) {
        const uint32_t c1 = __shfl_xor_sync(0xffffffffu, b1, o), c2 = __shfl_xor_sync(0xffffffffu, b2, o);
        b2 = b1 > c1 ? max(b2, c1) : max(b1, c2);
        b1 = max(b1, c1);
      }
      // a NaN (key 1) or an absent second value adds nothing; a group of NaN ranks last
      uint32_t gkey = 0u;
      if (g < a.n_group && j == 0)
        gkey = b1 <= 1u ? 1u : order_key(b2 <= 1u ? key_value(b1) : key_value(b1) + key_value(b2));
      uint32_t live = 0u;
      for (int r = 0; r < a.topk_group; ++r) {
        const uint32_t best = __reduce_max_sync(0xffffffffu, gkey);
        const uint32_t who = __reduce_min_sync(0xffffffffu, gkey == best && gkey ? (uint32_t)lane : 0xffu);
        live |= 1u << (who / sub);
        if (lane == (int)who) gkey = 0u;
      }
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const int e = i * 32 + lane;
        if (e < a.E && !((live >> (e / gs)) & 1u)) key[i] = 0u;
      }
      __syncwarp();
    }
  }

  // the k picks; lane j % 32 keeps pick j's id, its weight term goes to w
  float sum = 0.0f;
  for (int j = 0; j < a.k; ++j) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < NPL; ++i) m = max(m, key[i]);
    const uint32_t best = __reduce_max_sync(0xffffffffu, m);
    uint32_t at = 0xffffffffu;
#pragma unroll
    for (int i = NPL - 1; i >= 0; --i)
      if (key[i] == best) at = (uint32_t)(i * 32 + lane);
    at = __reduce_min_sync(0xffffffffu, at);
    float term = 0.0f;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (at == (uint32_t)(i * 32 + lane)) {
        key[i] = 0u;
        term = a.scoring == 0 ? softmax_term(v[i], top) : v[i];
      }
    term = __shfl_sync(0xffffffffu, term, (int)(at & 31u));
    sum += term;
    if (lane == 0) {
      a.ids[(size_t)t * a.k + j] = (int32_t)at;
      a.w[(size_t)t * a.k + j] = term;
    }
  }
  if (a.renorm) denom = sum;
  __syncwarp();
  const bool divide = a.renorm || a.scoring == 0;
  for (int j = lane; j < a.k; j += 32) {
    float* w = a.w + (size_t)t * a.k + j;
    const float x = *w;
    *w = (divide ? (denom > 0.0f ? x / denom : 0.0f) : x) * a.scale;
  }
}

// Rank the pairs of one block of tokens: pairs p0 .. p1 - 1, experts `ids`.  base[e]
// (shared, E + 1) is the row of the block's first pair of expert e; bin E holds the pairs whose id is
// out of range.  Warps take consecutive segments, so ranks follow the pair index.
__device__ __forceinline__ void count_segments(const int32_t* __restrict__ ids, int p0, int p1, int E, int32_t* cnt,
                                               int warps) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int seg = ((p1 - p0 + warps - 1) / warps + 31) & ~31;
  int32_t* mine = cnt + warp * (E + 1);
  const int s0 = p0 + warp * seg, s1 = min(p1, s0 + seg);
  for (int p = s0; p < s1; p += 32) {
    const int q = p + lane;
    const bool live = q < s1;
    int e = live ? ids[q] : -2;
    if (live && (unsigned)e >= (unsigned)E) e = E;
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    if (live && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
  }
}

__device__ __forceinline__ void place_segments(const int32_t* __restrict__ ids, int p0, int p1, int E, int32_t* cnt,
                                               int warps, int32_t* __restrict__ order, int32_t* __restrict__ place) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int seg = ((p1 - p0 + warps - 1) / warps + 31) & ~31;
  int32_t* mine = cnt + warp * (E + 1);
  const int s0 = p0 + warp * seg, s1 = min(p1, s0 + seg);
  for (int p = s0; p < s1; p += 32) {
    const int q = p + lane;
    const bool live = q < s1;
    int e = live ? ids[q] : -2;
    if (live && (unsigned)e >= (unsigned)E) e = E;
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    if (live) {
      const int row = mine[e] + __popc(same & ((1u << lane) - 1u));
      order[row] = e < E ? q : -1;
      place[q] = e < E ? row : -1;
    }
    __syncwarp();
    if (live && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
  }
}

// exclusive prefix over E + 1 bins of shared `total` into `first` and, for tiles, of ceil(total / 128); one warp
__device__ __forceinline__ void scan_bins(const int32_t* total, int E, int32_t* first, int32_t* offsets, int32_t* tiles,
                                          bool write) {
  const int lane = threadIdx.x & 31;
  int run = 0, trun = 0;
  for (int b = 0; b <= E; b += 32) {
    const int e = b + lane;
    const int c = e <= E ? total[e] : 0;
    const int tl = (c + 127) >> 7;
    int x = c, y = tl;
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) { x += u; y += v; }
    }
    if (e <= E) {
      first[e] = run + x - c;
      if (write) { offsets[e] = run + x - c; tiles[e] = trun + y - tl; }
    }
    run += __shfl_sync(0xffffffffu, x, 31);
    trun += __shfl_sync(0xffffffffu, y, 31);
  }
}

// Ranks the pairs of block `b` of `blocks`; smem: total[E+1], first[E+1], cnt[warps][E+1].
__device__ __forceinline__ void place_block(const int32_t* __restrict__ ids, int p0, int p1, int E, int b, int blocks,
                                            const int32_t* __restrict__ counts, int32_t* offsets, int32_t* tiles,
                                            int32_t* order, int32_t* place, int32_t* smem) {
  const int nt = blockDim.x, tid = threadIdx.x, warps = nt >> 5, bins = E + 1;
  int32_t* total = smem;
  int32_t* first = total + bins;
  int32_t* before = first + bins;
  int32_t* cnt = before + bins;
  for (int i = tid; i < (3 + warps) * bins; i += nt) smem[i] = 0;
  __syncthreads();
  count_segments(ids, p0, p1, E, cnt, warps);
  if (blocks > 1) {
    // the other blocks' counts: `parts` threads to a bin
    const int parts = max(1, nt / bins);
    for (int i = tid; i < parts * bins; i += nt) {
      const int e = i % bins, part = i / bins;
      int all = 0, bef = 0;
      for (int r = part; r < blocks; r += parts) {
        const int c = __ldcg(counts + (size_t)r * bins + e);
        all += c;
        if (r < b) bef += c;
      }
      atomicAdd(&total[e], all);
      if (bef) atomicAdd(&before[e], bef);
    }
    __syncthreads();
  } else {
    __syncthreads();
    for (int e = tid; e < bins; e += nt) {
      int c = 0;
      for (int w = 0; w < warps; ++w) c += cnt[w * bins + e];
      total[e] = c;
    }
    __syncthreads();
  }
  if (tid < 32) scan_bins(total, E, first, offsets, tiles, b == 0);
  __syncthreads();
  for (int e = tid; e < bins; e += nt) {
    int run = first[e] + before[e];
    for (int w = 0; w < warps; ++w) {
      const int c = cnt[w * bins + e];
      cnt[w * bins + e] = run;
      run += c;
    }
  }
  __syncthreads();
  place_segments(ids, p0, p1, E, cnt, warps, order, place);
}

int place_threads(int E) { return E <= 1024 ? PLACE_THREADS : 256; }
size_t place_smem(int E, int threads) { return (size_t)(3 + threads / 32) * (E + 1) * 4; }

template <int NPL>
__global__ void __launch_bounds__(ROUTE_THREADS) route_kernel(RouteArgs a, int logits_bf16) {
  extern __shared__ int32_t smem[];
  const int warp = threadIdx.x >> 5;
  const int t0 = blockIdx.x * a.tokens_per_block, t1 = min(a.T, t0 + a.tokens_per_block);
  float* scratch = reinterpret_cast<float*>(smem) + (size_t)warp * (a.E + a.E / 32 + 1);
  for (int t = t0 + warp; t < t1; t += ROUTE_WARPS) route_token<NPL>(a, logits_bf16, t, scratch);
  if (!a.offsets) return;
  __syncthreads();   // this block's ids are written, the scratch is free
  if (gridDim.x == 1) {
    place_block(a.ids, 0, a.T * a.k, a.E, 0, 1, nullptr, a.offsets, a.tiles, a.order, a.place, smem);
    return;
  }
  for (int i = threadIdx.x; i <= a.E; i += ROUTE_THREADS) smem[i] = 0;
  __syncthreads();
  for (int p = t0 * a.k + threadIdx.x; p < t1 * a.k; p += ROUTE_THREADS) atomicAdd(&smem[a.ids[p]], 1);
  __syncthreads();
  for (int i = threadIdx.x; i <= a.E; i += ROUTE_THREADS) a.counts[(size_t)blockIdx.x * (a.E + 1) + i] = smem[i];
}

__global__ void __launch_bounds__(ROUTE_THREADS)
count_kernel(const int32_t* __restrict__ ids, int P, int E, int per_block, int32_t* __restrict__ counts) {
  extern __shared__ int32_t smem[];
  for (int i = threadIdx.x; i <= E; i += ROUTE_THREADS) smem[i] = 0;
  __syncthreads();
  const int p0 = blockIdx.x * per_block, p1 = min(P, p0 + per_block);
  for (int p = p0 + threadIdx.x; p < p1; p += ROUTE_THREADS) {
    const int e = ids[p];
    atomicAdd(&smem[(unsigned)e < (unsigned)E ? e : E], 1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i <= E; i += ROUTE_THREADS) counts[(size_t)blockIdx.x * (E + 1) + i] = smem[i];
}

__global__ void __launch_bounds__(PLACE_THREADS)
place_kernel(const int32_t* __restrict__ ids, int P, int E, int per_block, const int32_t* __restrict__ counts,
             int32_t* offsets, int32_t* tiles, int32_t* order, int32_t* place) {
  extern __shared__ int32_t smem[];
  const int p0 = blockIdx.x * per_block, p1 = min(P, p0 + per_block);
  place_block(ids, p0, p1, E, blockIdx.x, gridDim.x, counts, offsets, tiles, order, place, smem);
}

// out[t, n] = sum_j w[t, j] y[place[t, j], n]: V columns a thread
template <typename Y, typename O, int V>
__global__ void __launch_bounds__(256)
combine_kernel(int T, int k, int N, const Y* __restrict__ y, const int32_t* __restrict__ place,
               const float* __restrict__ w, O* __restrict__ out) {
  const int cols = N / V;
  const int64_t units = (int64_t)T * cols;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < units; u += (int64_t)gridDim.x * 256) {
    const int t = (int)(u / cols), c = (int)(u % cols) * V;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    for (int j = 0; j < k; ++j) {
      const int row = __ldg(place + (size_t)t * k + j);
      if (row < 0) continue;
      const float g = __ldg(w + (size_t)t * k + j);
      const Y* src = y + (size_t)row * N + c;
      Y tmp[V];
      if constexpr (sizeof(Y) * V == 16) *reinterpret_cast<uint4*>(tmp) = __ldg(reinterpret_cast<const uint4*>(src));
      else if constexpr (sizeof(Y) * V == 32) {
        reinterpret_cast<uint4*>(tmp)[0] = __ldg(reinterpret_cast<const uint4*>(src));
        reinterpret_cast<uint4*>(tmp)[1] = __ldg(reinterpret_cast<const uint4*>(src) + 1);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) tmp[i] = src[i];
      }
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = fmaf(g, (float)tmp[i], acc[i]);
    }
    O res[V];
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
  if (wide)
    combine_kernel<Y, O, 8><<<grid, 256, 0, s>>>(T, k, N, (const Y*)y, place, w, (O*)out);
  else
    combine_kernel<Y, O, 1><<<grid, 256, 0, s>>>(T, k, N, (const Y*)y, place, w, (O*)out);
  return cudaGetLastError();
}

// tokens of one block when T tokens are spread over at most kMaxBlocks
int tokens_per_block(int T) {
  const int want = (T + kMaxBlocks - 1) / kMaxBlocks;
  return std::max(ROUTE_WARPS, (want + ROUTE_WARPS - 1) / ROUTE_WARPS * ROUTE_WARPS);
}

moe_status check_group_args(int32_t T, int32_t E, int32_t k, const void* offsets, const void* tiles, const void* order,
                            const void* place, const void* ws, int64_t ws_bytes) {
  if (!offsets || !tiles || (T > 0 && (!order || !place)))
    return fail(MOE_EINVAL, "offsets, tiles, order and place are all needed for grouping");
  if (!aligned_to(offsets, 4) || !aligned_to(tiles, 4) || !aligned_to(order, 4) || !aligned_to(place, 4) || !aligned_to(ws, 4))
    return fail(MOE_EINVAL, "offsets, tiles, order, place and workspace must be 4-byte aligned");
  const int64_t need = moe_group_workspace(T, k, E);
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(MOE_EINVAL, "workspace holds %lld bytes, %lld are needed", (long long)ws_bytes, (long long)need);
  return MOE_OK;
}

moe_status check_sizes(int32_t T, int32_t E, int32_t k) {
  if (T < 0 || E < 1 || E > kMaxExperts || k < 1) return fail(MOE_EINVAL, "T >= 0, 1 <= E <= %d and k >= 1 are needed, got T %d, E %d, k %d", kMaxExperts, T, E, k);
  if ((int64_t)T * k > 0x7fffff00ll) return fail(MOE_EINVAL, "T * k = %lld pairs do not fit 31 bits", (long long)T * k);
  return MOE_OK;
}

cudaError_t allow_smem(const void* fn, size_t bytes) {
  if (bytes <= 48 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <int NPL>
moe_status run_route(const RouteArgs& a, int bf16, int blocks, cudaStream_t s) {
  size_t smem = a.n_group > 1 ? (size_t)ROUTE_WARPS * (a.E + a.E / 32 + 1) * 4 : 0;
  if (a.offsets) smem = std::max(smem, blocks == 1 ? place_smem(a.E, ROUTE_THREADS) : (size_t)(a.E + 1) * 4);
  CK(allow_smem((const void*)route_kernel<NPL>, smem));
  route_kernel<NPL><<<blocks, ROUTE_THREADS, smem, s>>>(a, bf16);
  CK(cudaGetLastError());
  return MOE_OK;
}

moe_status run_place(const int32_t* ids, int P, int E, int per_block, int blocks, const int32_t* counts, int32_t* offsets,
                     int32_t* tiles, int32_t* order, int32_t* place, cudaStream_t s) {
  const size_t smem = place_smem(E, place_threads(E));
  CK(allow_smem((const void*)place_kernel, smem));
  place_kernel<<<blocks, place_threads(E), smem, s>>>(ids, P, E, per_block, counts, offsets, tiles, order, place);
  CK(cudaGetLastError());
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
  (void)k;
  if (T < 0 || E < 0) return 0;
  const int64_t blocks = T ? (T + tokens_per_block(T) - 1) / tokens_per_block(T) : 1;
  return blocks * ((int64_t)E + 1) * 4;
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
  if (group && (st = check_group_args(T, E, k, offsets, tiles, order, place, workspace, workspace_bytes)) != MOE_OK) return st;
  if (T > 0 && (!logits || !ids || !w)) return fail(MOE_EINVAL, "logits, topk_ids and topk_w must not be NULL");
  if (!aligned_to(logits, logits_dtype == MOE_F32 ? 4 : 2) || !aligned_to(bias, 4) || !aligned_to(ids, 4) || !aligned_to(w, 4))
    return fail(MOE_EINVAL, "logits, bias, topk_ids and topk_w must be aligned to their element size");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0)
    return group ? run_place(nullptr, 0, E, 1, 1, nullptr, offsets, tiles, order, place, s) : MOE_OK;
  RouteArgs a{};
  a.T = T; a.E = E; a.k = k; a.scoring = scoring; a.n_group = n_group; a.topk_group = topk_group;
  a.renorm = renormalize != 0; a.scale = scale; a.logits = logits; a.bias = bias; a.ids = ids; a.w = w;
  a.offsets = offsets; a.tiles = tiles; a.order = order; a.place = place;
  a.counts = static_cast<int32_t*>(workspace);
  a.tokens_per_block = group && T <= kOneBlockTokens ? T : tokens_per_block(T);
  const int blocks = (T + a.tokens_per_block - 1) / a.tokens_per_block;
  const int bf16 = logits_dtype == MOE_BF16;
  const int npl = (E + 31) / 32;
  st = npl <= 2 ? run_route<2>(a, bf16, blocks, s) : npl <= 4 ? run_route<4>(a, bf16, blocks, s)
       : npl <= 8 ? run_route<8>(a, bf16, blocks, s) : npl <= 16 ? run_route<16>(a, bf16, blocks, s)
       : npl <= 32 ? run_route<32>(a, bf16, blocks, s) : run_route<128>(a, bf16, blocks, s);
  if (st != MOE_OK || !group || blocks == 1) return st;
  return run_place(ids, T * k, E, a.tokens_per_block * k, blocks, a.counts, offsets, tiles, order, place, s);
}

extern "C" moe_status moe_group_pairs(int32_t T, int32_t E, int32_t k, const int32_t* ids, int32_t* offsets, int32_t* tiles,
                                      int32_t* order, int32_t* place, void* workspace, int64_t workspace_bytes, void* stream) {
  moe_status st = check_sizes(T, E, k);
  if (st != MOE_OK) return st;
  if ((st = check_group_args(T, E, k, offsets, tiles, order, place, workspace, workspace_bytes)) != MOE_OK) return st;
  if (T > 0 && !ids) return fail(MOE_EINVAL, "topk_ids must not be NULL");
  if (!aligned_to(ids, 4)) return fail(MOE_EINVAL, "topk_ids must be 4-byte aligned");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T <= kOneBlockTokens)
    return run_place(ids, T * k, E, std::max(1, T * k), 1, nullptr, offsets, tiles, order, place, s);
  const int tpb = tokens_per_block(T), blocks = (T + tpb - 1) / tpb;
  int32_t* counts = static_cast<int32_t*>(workspace);
  const size_t smem = (size_t)(E + 1) * 4;
  count_kernel<<<blocks, ROUTE_THREADS, smem, s>>>(ids, T * k, E, tpb * k, counts);
  CK(cudaGetLastError());
  return run_place(ids, T * k, E, tpb * k, blocks, counts, offsets, tiles, order, place, s);
}

extern "C" moe_status moe_combine(int32_t T, int32_t k, int32_t N, int32_t y_dtype, const void* y, const int32_t* place,
                                  const float* w, int32_t out_dtype, void* out, void* stream) {
  if (T < 0 || k < 1 || N < 1 || (int64_t)T * k > 0x7fffff00ll)
    return fail(MOE_EINVAL, "T >= 0, k >= 1, N >= 1 and at most 2^31 pairs are needed, got T %d, k %d, N %d", T, k, N);
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
