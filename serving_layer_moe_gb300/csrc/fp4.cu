// 4-bit quantisation and its inverse (include/moe_operators.h: moe_fp4_scale,
// moe_quantize_fp4, moe_dequantize_fp4).
//
// A thread holds 16 consecutive elements of a row: one NVFP4 block, or half an MXFP4
// block, whose largest value it shares with its neighbour.  The largest |x| is taken
// over the bit patterns, so NaN shows up above infinity.  Rounding is the format's:
// NVFP4 takes the correctly rounded quotient by the step, MXFP4 multiplies by a power of
// two, which is exact.  Scales go straight into the tile order that the tensor cores
// take, a word for each row's group of four blocks.
//
// Rows for the experts are read and converted once a token and stored once an expert
// (converting once a pair took 95 us for 8192 tokens, 8 experts each, K 2048).
//
// Bound by memory: 2 bytes read and 0.53 or 0.56 written an element (bf16), the other way
// round for the inverse.
#include "operators.cuh"

#include <algorithm>

namespace moe {

namespace {

constexpr int Q_THREADS = 256;
constexpr int Q_UNITS = 1024;   // 16-element units of one step of a block, about
constexpr int Q_PLACES = 256;   // output rows of one step, at most

struct QuantArgs {
  int64_t rows;      // input rows
  int N, K, E, k, block_groups, g_count, step_rows;
  const void* x;
  const float* g;
  const int32_t *offsets, *tiles, *place;   // NULL: a stack of matrices
  uint8_t *codes, *scales;
};

// an output row, the padded row of its scales, its matrix's scale; row < 0: none
struct RowAt { int64_t row, pad; float g; };

__device__ __forceinline__ RowAt row_at(const QuantArgs& a, int64_t r) {
  RowAt o{r, 0, 1.0f};
  if (a.offsets) {
    const int i = (int)r, e = expert_of(a.offsets, a.E, i);
    o.pad = (int64_t)__ldg(a.tiles + e) * 128 + (i - __ldg(a.offsets + e));
    if (a.g) o.g = __ldg(a.g);
  } else {
    const int64_t m = r / a.N;
    o.pad = m * (ceil_div64(a.N, 128) * 128) + (r - m * a.N);
    if (a.g) o.g = __ldg(a.g + (a.g_count > 1 ? m : 0));
  }
  return o;
}

// 16 elements of a row; a row of K starts on 16 elements' bytes from its 16-byte aligned matrix
template <typename X>
__device__ __forceinline__ void load16(const X* p, float (&v)[16]) {
  constexpr int W = sizeof(X) == 4 ? 4 : 2;   // 16-byte words
  uint4 q[W];
  if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {   // 32 bytes an instruction
#pragma unroll
    for (int i = 0; i < W / 2; ++i)
      asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(q[2 * i].x), "=r"(q[2 * i].y), "=r"(q[2 * i].z), "=r"(q[2 * i].w), "=r"(q[2 * i + 1].x), "=r"(q[2 * i + 1].y),
                     "=r"(q[2 * i + 1].z), "=r"(q[2 * i + 1].w)
                   : "l"(reinterpret_cast<const uint4*>(p) + 2 * i));
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) q[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const uint32_t u[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(X) == 4) {
        v[4 * i + j] = __uint_as_float(u[j]);
      } else {
        v[8 * i + 2 * j] = __uint_as_float(u[j] << 16);
        v[8 * i + 2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
      }
    }
  }
}

template <typename X, bool NV>
__global__ void __launch_bounds__(Q_THREADS) quantize_kernel(QuantArgs a) {
  __shared__ RowAt at[Q_PLACES];
  pdl_wait();
  pdl_trigger();
  constexpr int G = NV ? 4 : 8;                       // units of a group of four blocks
  const int units_row = a.K / 16, per_row = (units_row + G - 1) / G * G;
  const int kk = min(a.k, Q_PLACES / a.step_rows);    // copies of a row handled at a time
  for (int64_t r0 = (int64_t)blockIdx.x * a.step_rows; r0 < a.rows; r0 += (int64_t)gridDim.x * a.step_rows) {
    const int n = (int)min((int64_t)a.step_rows, a.rows - r0);
    for (int j0 = 0; j0 < a.k; j0 += kk) {
      const int nj = min(kk, a.k - j0);
      __syncthreads();
      for (int i = threadIdx.x; i < n * nj; i += Q_THREADS) {
        const int64_t r = r0 + i / nj;
        const int64_t row = a.place ? (int64_t)__ldg(a.place + r * a.k + j0 + i % nj) : r;
        at[i] = row < 0 ? RowAt{-1, 0, 1.0f} : row_at(a, row);
      }
      __syncthreads();
      // whole groups a row, so that four (eight) neighbouring lanes make a group's word of scales; past the row's end: no block
      for (int u0 = 0; u0 < n * per_row; u0 += Q_THREADS) {
        const int u = u0 + threadIdx.x;
        const bool some = u < n * per_row;
        const int r = some ? u / per_row : 0, c = some ? u - r * per_row : 0;
        const bool live = some && c < units_row;
        float v[16];
        uint32_t m = 0u, code = 0u;
        uint2 q = make_uint2(0u, 0u);
        if (live) {
          load16(static_cast<const X*>(a.x) + (size_t)(r0 + r) * a.K + c * 16, v);
#pragma unroll
          for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
        }
        if (!NV) m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        if (live) {
          float step;
          code = block_scale<NV>(m, a.place ? (a.g ? __ldg(a.g) : 1.0f) : at[r].g, step);
          q = encode16<NV>(v, m, code, step);
        }
        if (NV) {
          code |= __shfl_xor_sync(0xffffffffu, code, 1) << 8;      // lane 0 of 4: bytes of lanes 0, 1
          code |= __shfl_xor_sync(0xffffffffu, code, 2) << 16;
        } else {
          code |= __shfl_xor_sync(0xffffffffu, code, 2) << 8;
          code |= __shfl_xor_sync(0xffffffffu, code, 4) << 16;
        }
        if (!some) continue;
        for (int j = 0; j < nj; ++j) {
          const RowAt o = at[r * nj + j];
          if (o.row < 0) continue;
          if (live) *reinterpret_cast<uint2*>(a.codes + (size_t)o.row * (a.K / 2) + c * 8) = q;
          if (c % G == 0) *reinterpret_cast<uint32_t*>(a.scales + scale_at((size_t)o.pad, c / (G / 4), a.block_groups)) = code;
        }
      }
    }
  }
}

// 8 values a thread: 16 bytes of bf16
template <typename O, bool NV>
__global__ void __launch_bounds__(Q_THREADS) dequantize_kernel(QuantArgs a, O* __restrict__ out) {
  __shared__ RowAt at[Q_PLACES];
  pdl_wait();
  pdl_trigger();
  const int per_row = a.K / 8;
  for (int64_t r0 = (int64_t)blockIdx.x * a.step_rows; r0 < a.rows; r0 += (int64_t)gridDim.x * a.step_rows) {
    const int n = (int)min((int64_t)a.step_rows, a.rows - r0);
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += Q_THREADS) {
      at[i] = a.offsets && r0 + i >= __ldg(a.offsets + a.E) ? RowAt{-1, 0, 1.0f} : row_at(a, r0 + i);
    }
    __syncthreads();
    for (int u = threadIdx.x; u < n * per_row; u += Q_THREADS) {
      const int r = u / per_row, c = u - r * per_row;
      const RowAt o = at[r];
      O res[8];
      if (o.row < 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) res[i] = (O)0.0f;
      } else {
        const uint32_t q = __ldg(reinterpret_cast<const uint32_t*>(a.codes + (size_t)o.row * (a.K / 2)) + c);
        const uint32_t sc = __ldg(a.scales + scale_at((size_t)o.pad, NV ? c >> 1 : c >> 2, a.block_groups));
        const float step = (NV ? e4m3_value(sc) : e8m0_value(sc)) * o.g;
#pragma unroll
        for (int i = 0; i < 8; ++i) res[i] = (O)(e2m1_value((q >> (4 * i)) & 15u) * step);
      }
      uint4* dst = reinterpret_cast<uint4*>(out + (size_t)(r0 + r) * a.K + c * 8);
#pragma unroll
      for (int i = 0; i < (int)sizeof(O) / 2; ++i) dst[i] = reinterpret_cast<const uint4*>(res)[i];
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

// rows of a step of a block, and the blocks
void set_steps(QuantArgs& a, int unit) {
  const int64_t share = a.rows / ((int64_t)operator_sms() * 4) + 1;   // small calls: a few rows a block, on every SM
  const int most = std::min({Q_PLACES / std::min(a.k, Q_PLACES), Q_UNITS * 16 / unit / std::max(1, a.K / unit), 64});
  a.step_rows = (int)std::max<int64_t>(1, std::min<int64_t>(most, share));
}
int steps_grid(const QuantArgs& a) {
  return (int)std::min<int64_t>((a.rows + a.step_rows - 1) / a.step_rows, (int64_t)operator_sms() * 8);
}

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
                                       const int32_t* tiles, const int32_t* place, uint8_t* codes, uint8_t* scales,
                                       void* stream) {
  moe_status st = check_fp4(G, N, K, dtype, wdtype, g, g_count);
  if (st != MOE_OK) return st;
  if (g && wdtype == MOE_MXFP4) return fail(MOE_EINVAL, "MXFP4 has no matrix scale");
  if (offsets && (G != 1 || !tiles || (N > 0 && !place) || E < 1 || k < 1 || N % k))
    return fail(MOE_EINVAL, "grouped rows need G = 1, tiles, place, E >= 1 and N pairs of k a row");
  if (G == 0 || N == 0) return MOE_OK;
  if (!x || !codes || !scales) return fail(MOE_EINVAL, "x, codes and scales must not be NULL");
  if (!aligned_to(x, 16) || !aligned_to(codes, 16) || !aligned_to(scales, 16) || !aligned_to(g, 4))
    return fail(MOE_EINVAL, "x, codes and scales must be 16-byte aligned, g 4-byte aligned");
  if (!aligned_to(offsets, 4) || !aligned_to(tiles, 4) || !aligned_to(place, 4))
    return fail(MOE_EINVAL, "offsets, tiles and place must be 4-byte aligned");
  QuantArgs a{};
  a.k = offsets ? k : 1;
  a.rows = offsets ? N / k : (int64_t)G * N; a.N = N; a.K = K; a.E = E; a.g_count = g_count; a.x = x; a.g = g;
  a.block_groups = wdtype == MOE_NVFP4 ? (K + 63) / 64 : (K + 127) / 128;
  a.offsets = offsets; a.tiles = tiles; a.place = offsets ? place : nullptr; a.codes = codes; a.scales = scales;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  set_steps(a, 16);
  const dim3 grid(steps_grid(a)), block(Q_THREADS);
  const bool f32 = dtype == MOE_F32, nv = wdtype == MOE_NVFP4;
  CK(f32 ? (nv ? launch_pdl(quantize_kernel<float, true>, grid, block, 0, s, a) : launch_pdl(quantize_kernel<float, false>, grid, block, 0, s, a))
         : (nv ? launch_pdl(quantize_kernel<__nv_bfloat16, true>, grid, block, 0, s, a)
               : launch_pdl(quantize_kernel<__nv_bfloat16, false>, grid, block, 0, s, a)));
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
  set_steps(a, 8);
  const dim3 grid(steps_grid(a)), block(Q_THREADS);
  const bool f32 = dtype == MOE_F32, nv = wdtype == MOE_NVFP4;
  float* of = static_cast<float*>(out);
  __nv_bfloat16* ob = static_cast<__nv_bfloat16*>(out);
  CK(f32 ? (nv ? launch_pdl(dequantize_kernel<float, true>, grid, block, 0, s, a, of) : launch_pdl(dequantize_kernel<float, false>, grid, block, 0, s, a, of))
         : (nv ? launch_pdl(dequantize_kernel<__nv_bfloat16, true>, grid, block, 0, s, a, ob)
               : launch_pdl(dequantize_kernel<__nv_bfloat16, false>, grid, block, 0, s, a, ob)));
  return MOE_OK;
}
