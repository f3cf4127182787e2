// What the products grouped by expert share: SwiGLU of their epilogues, and tensor maps.
#pragma once

#include "operators.cuh"
#include "tc.cuh"

#include <cudaTypedefs.h>

namespace moe {

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
// __fdividef gives 0 for a divisor past 2^126: x below -87.3, where silu is under 1.1e-36.
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

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
inline PFN_cuTensorMapEncodeTiled_v12000 get_encode() {
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

inline bool make_map(CUtensorMap* m, CUtensorMapDataType type, int rank, const void* base, const cuuint64_t* dims, const cuuint64_t* strides,
              const cuuint32_t* box, bool swizzle) {
  auto enc = get_encode();
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  return enc && enc(m, type, rank, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace moe
