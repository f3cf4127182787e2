// 4-bit quantisation and its inverse (include/moe_operators.h: moe_fp4_scale,
// moe_quantize_fp4, moe_dequantize_fp4).
//
// A thread holds 16 consecutive elements of a row: one NVFP4 block, or half an MXFP4
// block, whose largest value it shares with its neighbour.  The largest |x| is taken
// over the bit patterns, so NaN shows up above infinity.  Rounding is the format's:
// NVFP4's codes are those of the correctly rounded quotient by the step, MXFP4 multiplies by a
// power of two, which is exact.  Scales go straight into the tile order that the tensor cores
// take, a word for each row's group of four blocks.
//
// Rows for the experts are read and converted once a token and stored once an expert
// (converting once a pair took 95 us for 8192 tokens, 8 experts each, K 2048).
//
// Bound by memory: 2 bytes read and 0.53 or 0.56 written an element (bf16), the other way
// round for the inverse.
#include "operators.cuh"

#include <algorithm>
#include <type_traits>

namespace moe {

namespace {

constexpr int Q_THREADS = 256;
constexpr int Q_WARPS = Q_THREADS / 32;
// A warp takes a segment of a row (blockIdx.y): a unit of 16 elements a lane when quantising, four of 8 when dequantising,
// loaded before any is used.  Rows, segments and matrices (blockIdx.z) come from the grid: 64-bit divisions were half of
// the instructions (391 us for 805 MB of bf16, against 152 of its bytes).
constexpr int Q_SEG = 32, D_SEG = 128;

struct QuantArgs {
  int64_t rows;      // input rows (of each matrix)
  int K, E, k, block_groups, g_count;
  int64_t pairs, pad_rows;   // grouped rows, and the rows of their scale tiles
  const void* x;
  const float* g;
  const int32_t *offsets, *tiles, *place;   // NULL: a stack of matrices
  uint8_t *codes, *scales;
};

struct RowAt { int64_t row, pad; };   // an output row and the padded row of its scales; row < 0: none

// row i of the rows in expert order; none where i, or what offsets and tiles make of it, is not one of them
__device__ __forceinline__ RowAt grouped_row(const QuantArgs& a, int i) {
  if ((unsigned)i >= (unsigned)a.pairs) return RowAt{-1, 0};
  const int e = expert_of(a.offsets, a.E, i);
  const int64_t pad = (int64_t)__ldg(a.tiles + e) * 128 + i - __ldg(a.offsets + e);
  return RowAt{(uint64_t)pad < (uint64_t)a.pad_rows ? i : -1, pad};
}

// GROUPED: rows become the rows of their pairs in expert order; otherwise a stack of matrices.
// Blocks an SM: loads in flight against registers.  805 MB of bf16 to NVFP4 takes 211 us with 4, 178 with 6 and 214 with 8, where
// registers spill; to MXFP4 186, 157 and 147 (150 at the copy rate); 403 MB of fp32 84 with 3, 74 with 4, 69 with 5 or 6 (68).
template <typename X, bool NV, bool GROUPED>
__global__ void __launch_bounds__(Q_THREADS, sizeof(X) == 4 ? 5 : NV ? 6 : 8) quantize_kernel(QuantArgs a) {
  __shared__ RowAt places[Q_WARPS][GROUPED ? 32 : 1];
  pdl_wait();
  pdl_trigger();
  constexpr int G = NV ? 4 : 8;                       // units of a group of four blocks
  const int units = a.K / 16, padded = (units + G - 1) / G * G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = (int)blockIdx.y * Q_SEG + lane;
  const bool live = c < units, word = c % G == 0 && c < padded;
  const int64_t m = blockIdx.z;
  const float g = NV && a.g ? __ldg(a.g + (a.g_count > 1 ? m : 0)) : 1.0f, rg = __frcp_rn(g);
  const size_t word_at = ((size_t)(c / (G / 4)) >> 2) * 512;
  auto store = [&](int64_t row, int64_t pad, uint2 q, uint32_t code) {
    if (live) *reinterpret_cast<uint2*>(a.codes + (size_t)row * (a.K / 2) + c * 8) = q;
    if (word) *reinterpret_cast<uint32_t*>(a.scales + scale_at((size_t)pad, 0, a.block_groups) + word_at) = code;
  };
  for (int64_t r = (int64_t)blockIdx.x * Q_WARPS + warp; r < a.rows; r += (int64_t)gridDim.x * Q_WARPS) {
    Raw16<X> x;
    if (live) x.load(static_cast<const X*>(a.x) + (size_t)(m * a.rows + r) * a.K + c * 16);
    uint32_t top = live ? x.top() : 0u, code = 0u;
    uint2 q = make_uint2(0u, 0u);
    if (!NV) top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    if (live) {
      float step, v[16];
      x.values(v);
      code = block_scale<NV>(top, g, rg, step);
      q = encode16<NV>(v, top, code, step);
    }
    // four (eight) neighbouring lanes make a group's word of scales; past the row's end there is no block
    code |= __shfl_xor_sync(0xffffffffu, code, NV ? 1 : 2) << 8;
    code |= __shfl_xor_sync(0xffffffffu, code, NV ? 2 : 4) << 16;
    if constexpr (!GROUPED) {
      store(m * a.rows + r, m * ((a.rows + 127) & ~127ll) + r, q, code);
    } else {
      RowAt* at = places[warp];
      for (int j0 = 0; j0 < a.k; j0 += 32) {
        const int nj = min(32, a.k - j0);
        __syncwarp();
        if (lane < nj) at[lane] = grouped_row(a, __ldg(a.place + r * a.k + j0 + lane));
        __syncwarp();
        for (int j = 0; j < nj; ++j)
          if (at[j].row >= 0) store(at[j].row, at[j].pad, q, code);
      }
    }
  }
}

// two e2m1 codes (low nibble first) as fp16 values, exact
__device__ __forceinline__ float2 e2m1x2_values(uint32_t byte) {
  uint32_t h;
  asm("{\n .reg .b8 t;\n cvt.u8.u32 t, %1;\n cvt.rn.f16x2.e2m1x2 %0, t;\n}\n" : "=r"(h) : "r"(byte));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

template <typename O, bool NV>
__global__ void __launch_bounds__(Q_THREADS) dequantize_kernel(QuantArgs a, O* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const int units = a.K / 8, lane = threadIdx.x & 31;
  const int c0 = (int)blockIdx.y * D_SEG + lane;
  const int64_t m = blockIdx.z;
  const float g = a.g ? __ldg(a.g + (a.g_count > 1 ? m : 0)) : 1.0f;
  for (int64_t r = (int64_t)blockIdx.x * Q_WARPS + (threadIdx.x >> 5); r < a.rows; r += (int64_t)gridDim.x * Q_WARPS) {
    const int64_t row = m * a.rows + r;
    const RowAt at = !a.offsets ? RowAt{row, m * ((a.rows + 127) & ~127ll) + r} : r < __ldg(a.offsets + a.E) ? grouped_row(a, (int)r) : RowAt{-1, 0};
    const bool none = at.row < 0;   // no pair fills the row
    const int64_t pad = at.pad;
    uint32_t q[D_SEG / 32], sc[D_SEG / 32];
#pragma unroll
    for (int h = 0; h < D_SEG / 32; ++h) {
      const int c = c0 + 32 * h;
      q[h] = sc[h] = 0u;
      if (c < units && !none) {
        q[h] = __ldg(reinterpret_cast<const uint32_t*>(a.codes + (size_t)row * (a.K / 2)) + c);
        sc[h] = __ldg(a.scales + scale_at((size_t)pad, NV ? c >> 1 : c >> 2, a.block_groups));
      }
    }
#pragma unroll
    for (int h = 0; h < D_SEG / 32; ++h) {
      const int c = c0 + 32 * h;
      if (c >= units) continue;
      const float step = none ? 0.0f : (NV ? e4m3_value(sc[h]) : e8m0_value(sc[h])) * g;
      O res[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 x = e2m1x2_values((q[h] >> (8 * i)) & 255u);
        res[2 * i] = (O)(x.x * step);
        res[2 * i + 1] = (O)(x.y * step);
      }
      uint4* dst = reinterpret_cast<uint4*>(out + (size_t)row * a.K + c * 8);
      const uint4* src = reinterpret_cast<const uint4*>(res);
      if (sizeof(O) == 4 && (reinterpret_cast<uintptr_t>(dst) & 31) == 0) {   // 32 bytes an instruction
        asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(src[0].x), "r"(src[0].y), "r"(src[0].z), "r"(src[0].w),
                     "r"(src[sizeof(O) / 4].x), "r"(src[sizeof(O) / 4].y), "r"(src[sizeof(O) / 4].z), "r"(src[sizeof(O) / 4].w), "l"(dst)
                     : "memory");
      } else {
#pragma unroll
        for (int i = 0; i < (int)sizeof(O) / 2; ++i) dst[i] = src[i];
      }
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
  g[i] = a == 0.0f ? 1.0f : a * (1.0f / 2688.0f);
}

moe_status check_fp4(int32_t G, int32_t N, int32_t K, int32_t dtype, int32_t wdtype, const float* g, int32_t g_count) {
  if (G < 0 || G > 65535 || N < 0) return fail(MOE_EINVAL, "G (at most 65535) and N must not be negative, got %d and %d", G, N);
  if (K < 32 || K % 32 || K > 1 << 24) return fail(MOE_EINVAL, "K = %d is not a multiple of 32 (at most 2^24)", K);
  if (dtype != MOE_F32 && dtype != MOE_BF16) return fail(MOE_EINVAL, "dtype must be MOE_F32 or MOE_BF16");
  if (wdtype != MOE_NVFP4 && wdtype != MOE_MXFP4) return fail(MOE_EINVAL, "wdtype must be MOE_NVFP4 or MOE_MXFP4");
  if (g && g_count != 1 && g_count != G) return fail(MOE_EINVAL, "g_count must be 1 or G = %d, is %d", G, g_count);
  return MOE_OK;
}

// blocks: rows in x, a row's segments in y, matrices in z
dim3 segment_grid(const QuantArgs& a, int G, int units, int seg) {
  const int segs = (units + seg - 1) / seg;
  const int64_t most = std::max<int64_t>(1, (int64_t)operator_sms() * 64 / segs / G);
  return dim3((unsigned)std::min<int64_t>((a.rows + Q_WARPS - 1) / Q_WARPS, most), (unsigned)segs, (unsigned)G);
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
  a.rows = offsets ? N / k : N; a.K = K; a.E = E; a.g_count = g_count; a.x = x; a.g = g;
  a.block_groups = wdtype == MOE_NVFP4 ? (K + 63) / 64 : (K + 127) / 128;
  a.offsets = offsets; a.tiles = tiles; a.place = offsets ? place : nullptr; a.codes = codes; a.scales = scales;
  a.pairs = N; a.pad_rows = offsets ? moe_grouped_tiles(N, E) * 128 : 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid = segment_grid(a, G, (K / 16 + 7) / 8 * 8, Q_SEG), block(Q_THREADS);   // whole groups of blocks
  const bool f32 = dtype == MOE_F32, nv = wdtype == MOE_NVFP4;
  auto run = [&](auto dtype_of, auto nvfp4) {
    using X = decltype(dtype_of);
    constexpr bool NV = decltype(nvfp4)::value;
    return offsets ? launch_pdl(quantize_kernel<X, NV, true>, grid, block, 0, s, a) : launch_pdl(quantize_kernel<X, NV, false>, grid, block, 0, s, a);
  };
  CK(f32 ? (nv ? run(float{}, std::true_type{}) : run(float{}, std::false_type{}))
         : (nv ? run(__nv_bfloat16{}, std::true_type{}) : run(__nv_bfloat16{}, std::false_type{})));
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
  a.rows = N; a.K = K; a.E = E; a.k = 1; a.g_count = g_count; a.g = g;
  a.block_groups = wdtype == MOE_NVFP4 ? (K + 63) / 64 : (K + 127) / 128;
  a.offsets = offsets; a.tiles = tiles;
  a.pairs = N; a.pad_rows = offsets ? moe_grouped_tiles(N, E) * 128 : 0;
  a.codes = const_cast<uint8_t*>(codes); a.scales = const_cast<uint8_t*>(scales);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid = segment_grid(a, G, K / 8, D_SEG), block(Q_THREADS);
  const bool f32 = dtype == MOE_F32, nv = wdtype == MOE_NVFP4;
  float* of = static_cast<float*>(out);
  __nv_bfloat16* ob = static_cast<__nv_bfloat16*>(out);
  CK(f32 ? (nv ? launch_pdl(dequantize_kernel<float, true>, grid, block, 0, s, a, of) : launch_pdl(dequantize_kernel<float, false>, grid, block, 0, s, a, of))
         : (nv ? launch_pdl(dequantize_kernel<__nv_bfloat16, true>, grid, block, 0, s, a, ob)
               : launch_pdl(dequantize_kernel<__nv_bfloat16, false>, grid, block, 0, s, a, ob)));
  return MOE_OK;
}
