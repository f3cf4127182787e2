// 4-bit quantisation and its inverse (include/moe_operators.h: moe_fp4_scale,
// moe_quantize_fp4, moe_dequantize_fp4).
//
// A thread holds 16 consecutive elements of a row: one NVFP4 block, or half an MXFP4
// block, whose largest value it shares with its neighbour.  The largest |x| is taken
// over the bit patterns, so NaN shows up above infinity.  Rounding is the format's:
// NVFP4 divides by the step in correctly rounded 32-bit divisions, MXFP4 multiplies by
// a power of two, which is exact.  Scales go straight into the tile order that the
// tensor cores take.
//
// Bound by memory: 2 bytes read and 0.53 or 0.56 written an element (bf16), the other way
// round for the inverse.
#include "operators.cuh"

#include <algorithm>

namespace moe {

namespace {

constexpr int Q_THREADS = 256;
constexpr int Q_ROWS = 8;       // rows of one step of a block

// where an output row comes from and which padded row holds its scales; src < 0: no pair
struct RowAt { int64_t src, pad; int g; };

struct QuantArgs {
  int64_t rows;      // output rows
  int N, K, E, k, block_groups, g_count;
  const void* x;
  const float* g;
  const int32_t *offsets, *tiles, *order;   // NULL: a stack of matrices
  uint8_t *codes, *scales;
};

__device__ __forceinline__ RowAt row_at(const QuantArgs& a, int64_t r) {
  RowAt o;
  if (a.offsets) {
    o.g = 0;
    const int i = (int)r;
    if (i >= __ldg(a.offsets + a.E)) { o.src = -1; o.pad = 0; return o; }
    const int e = expert_of(a.offsets, a.E, i);
    o.src = a.order ? __ldg(a.order + i) / a.k : i;
    o.pad = (int64_t)__ldg(a.tiles + e) * 128 + (i - __ldg(a.offsets + e));
    return o;
  }
  const int64_t m = r / a.N;
  o.src = r;
  o.pad = m * (ceil_div64(a.N, 128) * 128) + (r - m * a.N);
  o.g = a.g_count > 1 ? (int)m : 0;
  return o;
}

template <typename X>
__device__ __forceinline__ void load16(const X* p, float (&v)[16]) {
  if constexpr (sizeof(X) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(p) + i);
      v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(p) + i);
      const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[8 * i + 2 * j] = __uint_as_float(u[j] << 16);
        v[8 * i + 2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
      }
    }
  }
}

template <typename X, bool NV>
__global__ void __launch_bounds__(Q_THREADS) quantize_kernel(QuantArgs a) {
  __shared__ RowAt at[Q_ROWS];
  const int per_row = a.K / 16;
  for (int64_t r0 = (int64_t)blockIdx.x * Q_ROWS; r0 < a.rows; r0 += (int64_t)gridDim.x * Q_ROWS) {
    const int n = (int)min((int64_t)Q_ROWS, a.rows - r0);
    __syncthreads();
    if (threadIdx.x < n) at[threadIdx.x] = row_at(a, r0 + threadIdx.x);
    __syncthreads();
    // units past the last one do the last again, so that a warp's shuffles are whole
    const int units = n * per_row, padded = (units + 31) & ~31;
    for (int u = threadIdx.x; u < padded; u += Q_THREADS) {
      const int uu = min(u, units - 1);
      const int r = uu / per_row, c = uu - r * per_row;
      const RowAt o = at[r];
      float v[16];
      load16(static_cast<const X*>(a.x) + (size_t)max(o.src, (int64_t)0) * a.K + c * 16, v);
      uint32_t m = 0u;
#pragma unroll
      for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
      if (!NV) m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));   // per_row is even: the pair is one block
      float step;
      const float g = NV && a.g ? __ldg(a.g + o.g) : 1.0f;
      const uint32_t code = block_scale<NV>(m, g, step);
      const uint2 q = encode16<NV>(v, m, code, step);
      if (u >= units || o.src < 0) continue;
      *reinterpret_cast<uint2*>(a.codes + (size_t)(r0 + r) * (a.K / 2) + c * 8) = q;
      const int b = NV ? c : c >> 1;
      if (NV || !(c & 1)) {
        uint8_t* s = a.scales + scale_at((size_t)o.pad, b, a.block_groups);
        *s = (uint8_t)code;
        // the row's last block also pads its group
        if (b == (NV ? per_row : per_row / 2) - 1)
          for (int i = 1; i < 4 - (b & 3); ++i) s[i] = 0;
      }
    }
  }
}

template <typename O, bool NV>
__global__ void __launch_bounds__(Q_THREADS) dequantize_kernel(QuantArgs a, O* __restrict__ out) {
  __shared__ RowAt at[Q_ROWS];
  const int per_row = a.K / 16;
  for (int64_t r0 = (int64_t)blockIdx.x * Q_ROWS; r0 < a.rows; r0 += (int64_t)gridDim.x * Q_ROWS) {
    const int n = (int)min((int64_t)Q_ROWS, a.rows - r0);
    __syncthreads();
    if (threadIdx.x < n) at[threadIdx.x] = row_at(a, r0 + threadIdx.x);
    __syncthreads();
    for (int u = threadIdx.x; u < n * per_row; u += Q_THREADS) {
      const int r = u / per_row, c = u - r * per_row;
      const RowAt o = at[r];
      O res[16];
      if (o.src < 0) {
#pragma unroll
        for (int i = 0; i < 16; ++i) res[i] = (O)0.0f;
      } else {
        const uint2 q = __ldg(reinterpret_cast<const uint2*>(a.codes + (size_t)(r0 + r) * (a.K / 2) + c * 8));
        const uint32_t sc = a.scales[scale_at((size_t)o.pad, NV ? c : c >> 1, a.block_groups)];
        const float step = (NV ? e4m3_value(sc) : e8m0_value(sc)) * (a.g ? __ldg(a.g + o.g) : 1.0f);
#pragma unroll
        for (int i = 0; i < 16; ++i) res[i] = (O)(e2m1_value(((i < 8 ? q.x : q.y) >> (4 * (i & 7))) & 15u) * step);
      }
      uint4* dst = reinterpret_cast<uint4*>(out + (size_t)(r0 + r) * a.K + c * 16);
#pragma unroll
      for (int i = 0; i < (int)sizeof(O); ++i) dst[i] = reinterpret_cast<const uint4*>(res)[i];
    }
  }
}

// Largest |x| of each matrix, as bits, into g (zeroed before); integer maxima, so any order gives the same.
template <typename X>
__global__ void __launch_bounds__(Q_THREADS) amax_kernel(const X* __restrict__ x, int64_t count, int blocks_each,
                                                         uint32_t* __restrict__ top) {
  const int m = blockIdx.x / blocks_each, part = blockIdx.x % blocks_each;
  const X* p = x + (size_t)m * count;
  uint32_t best = 0u;
  const bool wide = ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(count * sizeof(X))) & 15) == 0;
  if (wide) {
    const int64_t n = count * sizeof(X) / 16;
    for (int64_t i = (int64_t)part * Q_THREADS + threadIdx.x; i < n; i += (int64_t)blocks_each * Q_THREADS) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(p) + i);
      const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(X) == 4) best = max(best, u[j] & 0x7fffffffu);
        else best = max(best, max((u[j] << 16) & 0x7fffffffu, u[j] & 0x7fff0000u));
      }
    }
  } else {
    for (int64_t i = (int64_t)part * Q_THREADS + threadIdx.x; i < count; i += (int64_t)blocks_each * Q_THREADS)
      best = max(best, __float_as_uint((float)p[i]) & 0x7fffffffu);
  }
  best = __reduce_max_sync(0xffffffffu, best);
  if ((threadIdx.x & 31) == 0 && best) atomicMax(top + m, best);
}

__global__ void finish_scale_kernel(int G, float* g) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= G) return;
  const float a = g[i];
  g[i] = a == 0.0f ? 1.0f : __fdiv_rn(a, 2688.0f);
}

moe_status check_fp4(int32_t G, int32_t N, int32_t K, int32_t dtype, int32_t wdtype, const float* g, int32_t g_count) {
  if (G < 0 || N < 0) return fail(MOE_EINVAL, "G and N must not be negative, got %d and %d", G, N);
  if (K < 32 || K % 32) return fail(MOE_EINVAL, "K = %d is not a multiple of 32", K);
  if (dtype != MOE_F32 && dtype != MOE_BF16) return fail(MOE_EINVAL, "dtype must be MOE_F32 or MOE_BF16");
  if (wdtype != MOE_NVFP4 && wdtype != MOE_MXFP4) return fail(MOE_EINVAL, "wdtype must be MOE_NVFP4 or MOE_MXFP4");
  if (g && g_count != 1 && g_count != G) return fail(MOE_EINVAL, "g_count must be 1 or G = %d, is %d", G, g_count);
  return MOE_OK;
}

int row_grid(int64_t rows) { return (int)std::min<int64_t>((rows + Q_ROWS - 1) / Q_ROWS, (int64_t)operator_sms() * 8); }

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_fp4_scale(int32_t G, int64_t count, int32_t dtype, const void* x, float* g, void* stream) {
  if (G < 0 || count < 1) return fail(MOE_EINVAL, "G >= 0 matrices of at least one element are needed, got %d of %lld", G, (long long)count);
  if (dtype != MOE_F32 && dtype != MOE_BF16) return fail(MOE_EINVAL, "dtype must be MOE_F32 or MOE_BF16");
  if (G == 0) return MOE_OK;
  if (!x || !g || !aligned_to(x, dtype == MOE_F32 ? 4 : 2) || !aligned_to(g, 4))
    return fail(MOE_EINVAL, "x and g must not be NULL and be aligned to their elements");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  CK(cudaMemsetAsync(g, 0, (size_t)G * 4, s));
  const int64_t most = std::max<int64_t>(1, (int64_t)operator_sms() * 8 / G);
  const int each = (int)std::min<int64_t>(most, (count + Q_THREADS * 32 - 1) / (Q_THREADS * 32));
  if ((int64_t)G * each > 0x7fffffffll) return fail(MOE_EINVAL, "G = %d matrices are too many", G);
  if (dtype == MOE_F32)
    amax_kernel<float><<<G * each, Q_THREADS, 0, s>>>(static_cast<const float*>(x), count, each, reinterpret_cast<uint32_t*>(g));
  else
    amax_kernel<__nv_bfloat16><<<G * each, Q_THREADS, 0, s>>>(static_cast<const __nv_bfloat16*>(x), count, each,
                                                              reinterpret_cast<uint32_t*>(g));
  CK(cudaGetLastError());
  finish_scale_kernel<<<(G + 255) / 256, 256, 0, s>>>(G, g);
  CK(cudaGetLastError());
  return MOE_OK;
}

extern "C" moe_status moe_quantize_fp4(int32_t G, int32_t N, int32_t K, int32_t dtype, const void* x, int32_t wdtype,
                                       const float* g, int32_t g_count, int32_t E, int32_t k, const int32_t* offsets,
                                       const int32_t* tiles, const int32_t* order, uint8_t* codes, uint8_t* scales,
                                       void* stream) {
  moe_status st = check_fp4(G, N, K, dtype, wdtype, g, g_count);
  if (st != MOE_OK) return st;
  if (g && wdtype == MOE_MXFP4) return fail(MOE_EINVAL, "MXFP4 has no matrix scale");
  if (offsets && (G != 1 || !tiles || (N > 0 && !order) || E < 1 || k < 1))
    return fail(MOE_EINVAL, "grouped rows need G = 1, tiles, order, E >= 1 and k >= 1");
  if (G == 0 || N == 0) return MOE_OK;
  if (!x || !codes || !scales) return fail(MOE_EINVAL, "x, codes and scales must not be NULL");
  if (!aligned_to(x, 16) || !aligned_to(codes, 16) || !aligned_to(scales, 16) || !aligned_to(g, 4))
    return fail(MOE_EINVAL, "x, codes and scales must be 16-byte aligned, g 4-byte aligned");
  if (!aligned_to(offsets, 4) || !aligned_to(tiles, 4) || !aligned_to(order, 4))
    return fail(MOE_EINVAL, "offsets, tiles and order must be 4-byte aligned");
  QuantArgs a{};
  a.rows = (int64_t)G * N; a.N = N; a.K = K; a.E = E; a.k = k; a.g_count = g_count; a.x = x; a.g = g;
  a.block_groups = wdtype == MOE_NVFP4 ? (K + 63) / 64 : (K + 127) / 128;
  a.offsets = offsets; a.tiles = tiles; a.order = order; a.codes = codes; a.scales = scales;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int grid = row_grid(a.rows);
  const bool f32 = dtype == MOE_F32, nv = wdtype == MOE_NVFP4;
  if (f32 && nv) quantize_kernel<float, true><<<grid, Q_THREADS, 0, s>>>(a);
  else if (f32) quantize_kernel<float, false><<<grid, Q_THREADS, 0, s>>>(a);
  else if (nv) quantize_kernel<__nv_bfloat16, true><<<grid, Q_THREADS, 0, s>>>(a);
  else quantize_kernel<__nv_bfloat16, false><<<grid, Q_THREADS, 0, s>>>(a);
  CK(cudaGetLastError());
  return MOE_OK;
}

extern "C" moe_status moe_dequantize_fp4(int32_t G, int32_t N, int32_t K, int32_t wdtype, const uint8_t* codes,
                                         const uint8_t* scales, const float* g, int32_t g_count, int32_t E,
                                         const int32_t* offsets, const int32_t* tiles, int32_t dtype, void* out,
                                         void* stream) {
  moe_status st = check_fp4(G, N, K, dtype, wdtype, g, g_count);
  if (st != MOE_OK) return st;
  if (offsets && (G != 1 || !tiles || E < 1)) return fail(MOE_EINVAL, "grouped rows need G = 1, tiles and E >= 1");
  if (G == 0 || N == 0) return MOE_OK;
  if (!codes || !scales || !out) return fail(MOE_EINVAL, "codes, scales and out must not be NULL");
  if (!aligned_to(codes, 16) || !aligned_to(scales, 16) || !aligned_to(out, 16) || !aligned_to(g, 4))
    return fail(MOE_EINVAL, "codes, scales and out must be 16-byte aligned, g 4-byte aligned");
  if (!aligned_to(offsets, 4) || !aligned_to(tiles, 4)) return fail(MOE_EINVAL, "offsets and tiles must be 4-byte aligned");
  QuantArgs a{};
  a.rows = (int64_t)G * N; a.N = N; a.K = K; a.E = E; a.k = 1; a.g_count = g_count; a.g = g;
  a.block_groups = wdtype == MOE_NVFP4 ? (K + 63) / 64 : (K + 127) / 128;
  a.offsets = offsets; a.tiles = tiles;
  a.codes = const_cast<uint8_t*>(codes); a.scales = const_cast<uint8_t*>(scales);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int grid = row_grid(a.rows);
  const bool f32 = dtype == MOE_F32, nv = wdtype == MOE_NVFP4;
  if (f32 && nv) dequantize_kernel<float, true><<<grid, Q_THREADS, 0, s>>>(a, static_cast<float*>(out));
  else if (f32) dequantize_kernel<float, false><<<grid, Q_THREADS, 0, s>>>(a, static_cast<float*>(out));
  else if (nv) dequantize_kernel<__nv_bfloat16, true><<<grid, Q_THREADS, 0, s>>>(a, static_cast<__nv_bfloat16*>(out));
  else dequantize_kernel<__nv_bfloat16, false><<<grid, Q_THREADS, 0, s>>>(a, static_cast<__nv_bfloat16*>(out));
  CK(cudaGetLastError());
  return MOE_OK;
}
