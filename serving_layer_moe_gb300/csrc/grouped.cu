// Products grouped by expert (include/moe_operators.h: moe_grouped_matmul,
// moe_grouped_matmul_fp4).
//
// A block computes 64 rows of one expert's 128-row tile against 64 columns (with
// SwiGLU: 64 gate columns and their 64 up columns) on the CUDA cores, from fp32 copies of
// 32-deep slices in shared memory.
#include "operators.cuh"

#include <algorithm>

namespace moe {

namespace {

constexpr int TM = 64, TN = 64, TK = 32;

struct ProductArgs {
  int P, E, N, K, k, cols, block_groups, gw_count, act;
  const void* x;             // bf16 rows or codes
  const uint8_t* x_scales;
  const void* w;
  const uint8_t* w_scales;
  const float *gx, *gw, *g_out;
  const int32_t *offsets, *tiles, *order;
  void* out;
  uint8_t *out_codes, *out_scales;
};

// element of a 4-bit matrix: row r of `codes`, padded row `pad` of `scales`
template <int FMT>
__device__ __forceinline__ float fp4_at(const uint8_t* codes, const uint8_t* scales, size_t r, size_t pad, int c, int K, int groups) {
  const uint32_t q = codes[r * (size_t)(K / 2) + (c >> 1)] >> (4 * (c & 1));
  const uint32_t s = scales[scale_at(pad, FMT == MOE_NVFP4 ? c >> 4 : c >> 5, groups)];
  return e2m1_value(q & 15u) * (FMT == MOE_NVFP4 ? e4m3_value(s) : e8m0_value(s));
}

// OUT: MOE_BF16, MOE_F32, or -1 = 4-bit rows of FMT
template <int FMT, int OUT, bool SWIGLU>
__global__ void __launch_bounds__(256) product_kernel(ProductArgs a) {
  constexpr int NB = SWIGLU ? 2 : 1;
  __shared__ float xs[TK][TM + 1], ws[NB][TK][TN + 1];
  __shared__ float hs[OUT < 0 ? TM : 1][TN + 1];
  const int tile = blockIdx.y >> 1;
  if (tile >= __ldg(a.tiles + a.E)) return;
  const int e = expert_of(a.tiles, a.E, tile);
  const int in_e = (tile - __ldg(a.tiles + e)) * 128 + (blockIdx.y & 1) * TM;
  const int row0 = __ldg(a.offsets + e) + in_e, row1 = __ldg(a.offsets + e + 1);
  if (row0 >= row1) return;
  const int col0 = blockIdx.x * TN;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const size_t wpad = (size_t)e * (size_t)(ceil_div64(a.N, 128) * 128), xpad = (size_t)tile * 128 + (blockIdx.y & 1) * TM;
  float acc[NB][4][4] = {};
  for (int k0 = 0; k0 < a.K; k0 += TK) {
    for (int i = threadIdx.x; i < TM * TK; i += 256) {
      const int r = i / TK, c = i % TK;
      float v = 0.0f;
      if (row0 + r < row1 && k0 + c < a.K) {
        if constexpr (FMT == MOE_BF16) {
          const size_t src = a.order ? (size_t)(__ldg(a.order + row0 + r) / a.k) : (size_t)(row0 + r);
          v = __bfloat162float(static_cast<const __nv_bfloat16*>(a.x)[src * a.K + k0 + c]);
        } else {
          v = fp4_at<FMT>(static_cast<const uint8_t*>(a.x), a.x_scales, row0 + r, xpad + r, k0 + c, a.K, a.block_groups);
        }
      }
      xs[c][r] = v;
    }
    for (int b = 0; b < NB; ++b)
      for (int i = threadIdx.x; i < TN * TK; i += 256) {
        const int r = i / TK, c = i % TK;
        float v = 0.0f;
        if (col0 + r < a.cols && k0 + c < a.K) {
          const int n = col0 + r + b * a.cols;
          if constexpr (FMT == MOE_BF16)
            v = __bfloat162float(static_cast<const __nv_bfloat16*>(a.w)[((size_t)e * a.N + n) * a.K + k0 + c]);
          else
            v = fp4_at<FMT>(static_cast<const uint8_t*>(a.w), a.w_scales, (size_t)e * a.N + n, wpad + n, k0 + c, a.K, a.block_groups);
        }
        ws[b][c][r] = v;
      }
    __syncthreads();
#pragma unroll 8
    for (int c = 0; c < TK; ++c)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[b][i][j] = fmaf(xs[c][ty * 4 + i], ws[b][c][tx + 16 * j], acc[b][i][j]);
    __syncthreads();
  }
  float g = 1.0f;
  if (FMT != MOE_BF16) g = (a.gx ? *a.gx : 1.0f) * (a.gw ? a.gw[a.gw_count > 1 ? e : 0] : 1.0f);
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int r = row0 + ty * 4 + i, c = col0 + tx + 16 * j;
      float v = acc[0][i][j] * g;
      if (SWIGLU) v = v / (1.0f + expf(-v)) * (acc[NB - 1][i][j] * g);
      if constexpr (OUT < 0) hs[ty * 4 + i][tx + 16 * j] = v;
      else if (r < row1 && c < a.cols) {
        if constexpr (OUT == MOE_F32) static_cast<float*>(a.out)[(size_t)r * a.cols + c] = v;
        else static_cast<__nv_bfloat16*>(a.out)[(size_t)r * a.cols + c] = __float2bfloat16_rn(v);
      }
    }
  if constexpr (OUT < 0) {
    __syncthreads();
    constexpr bool NV = FMT == MOE_NVFP4;
    constexpr int B = NV ? 16 : 32;
    const int og = (a.cols + 4 * B - 1) / (4 * B);
    const float go = NV && a.g_out ? *a.g_out : 1.0f;
    for (int u = threadIdx.x; u < TM * (TN / B); u += 256) {
      const int r = u / (TN / B), b = u % (TN / B), c = col0 + b * B;
      if (row0 + r >= row1 || c >= a.cols) continue;
      uint32_t m = 0u;
      for (int i = 0; i < B; ++i) m = max(m, __float_as_uint(hs[r][b * B + i]) & 0x7fffffffu);
      float step;
      const uint32_t code = block_scale<NV>(m, go, step);
      const float inv = NV ? 0.0f : e8m0_inverse(code);
      for (int i = 0; i < B; i += 2) {
        const float lo = hs[r][b * B + i], hi = hs[r][b * B + i + 1];
        const uint32_t q = !(step > 0.0f) ? 0u : NV ? to_e2m1x2(__fdiv_rn(lo, step), __fdiv_rn(hi, step)) : to_e2m1x2(lo * inv, hi * inv);
        a.out_codes[(size_t)(row0 + r) * (a.cols / 2) + (c + i) / 2] = (uint8_t)q;
      }
      uint8_t* s = a.out_scales + scale_at(xpad + r, c / B, og);
      *s = (uint8_t)code;
      if (c + B >= a.cols)
        for (int i = 1; i < 4 - ((c / B) & 3); ++i) s[i] = 0;
    }
  }
}

template <int FMT>
moe_status launch_product(const ProductArgs& a, int out_dtype, cudaStream_t s) {
  const dim3 grid((a.cols + TN - 1) / TN, (unsigned)(2 * moe_grouped_tiles(a.P, a.E)));
  if (grid.y > 65535) return fail(MOE_EINVAL, "P = %d rows are too many", a.P);
  if (!a.out) {
    if constexpr (FMT != MOE_BF16) product_kernel<FMT, -1, true><<<grid, 256, 0, s>>>(a);
  } else if (a.act) {
    if (out_dtype == MOE_F32) product_kernel<FMT, MOE_F32, true><<<grid, 256, 0, s>>>(a);
    else product_kernel<FMT, MOE_BF16, true><<<grid, 256, 0, s>>>(a);
  } else {
    if (out_dtype == MOE_F32) product_kernel<FMT, MOE_F32, false><<<grid, 256, 0, s>>>(a);
    else product_kernel<FMT, MOE_BF16, false><<<grid, 256, 0, s>>>(a);
  }
  CK(cudaGetLastError());
  return MOE_OK;
}

moe_status check_product(int32_t P, int32_t E, int32_t N, int32_t K, int32_t quantum, const int32_t* offsets,
                         const int32_t* tiles, int32_t act, int32_t out_dtype) {
  if (P < 0 || E < 1 || E > kMaxExperts || N < 1) return fail(MOE_EINVAL, "P >= 0, 1 <= E <= %d and N >= 1 are needed, got P %d, E %d, N %d", kMaxExperts, P, E, N);
  if (K < 1 || K % quantum) return fail(MOE_EINVAL, "K = %d is not a multiple of %d", K, quantum);
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

extern "C" moe_status moe_grouped_matmul(int32_t P, int32_t E, int32_t N, int32_t K, const void* x, int32_t x_rows,
                                         const int32_t* order, int32_t k, const void* w, const int32_t* offsets,
                                         const int32_t* tiles, int32_t act, int32_t out_dtype, void* out, void* stream) {
  moe_status st = check_product(P, E, N, K, 8, offsets, tiles, act, out_dtype);
  if (st != MOE_OK) return st;
  if (order && (k < 1 || !aligned_to(order, 4))) return fail(MOE_EINVAL, "order needs k >= 1 and 4-byte alignment");
  if (P == 0) return MOE_OK;
  if (!x || !w || !out || x_rows < 1) return fail(MOE_EINVAL, "x, w and out must not be NULL and x must hold rows");
  if (!aligned_to(x, 16) || !aligned_to(w, 16) || !aligned_to(out, 16)) return fail(MOE_EINVAL, "x, w and out must be 16-byte aligned");
  ProductArgs a{};
  a.P = P; a.E = E; a.N = N; a.K = K; a.k = k; a.act = act; a.cols = act ? N / 2 : N;
  a.x = x; a.w = w; a.order = order; a.offsets = offsets; a.tiles = tiles; a.out = out;
  return launch_product<MOE_BF16>(a, out_dtype, static_cast<cudaStream_t>(stream));
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
  if (wdtype == MOE_MXFP4 && (gx || gw || g_out)) return fail(MOE_EINVAL, "MXFP4 has no matrix scale");
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
  a.block_groups = wdtype == MOE_NVFP4 ? (K + 63) / 64 : (K + 127) / 128;
  a.x = x_codes; a.x_scales = x_scales; a.gx = gx; a.w = w_codes; a.w_scales = w_scales; a.gw = gw; a.gw_count = gw_count;
  a.offsets = offsets; a.tiles = tiles; a.out = out; a.out_codes = out_codes; a.out_scales = out_scales; a.g_out = g_out;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return wdtype == MOE_NVFP4 ? launch_product<MOE_NVFP4>(a, out_dtype, s) : launch_product<MOE_MXFP4>(a, out_dtype, s);
}

extern "C" moe_status moe_operators_check(void* stream) {
  CK(cudaStreamSynchronize(static_cast<cudaStream_t>(stream)));
  return MOE_OK;
}
