// Declarations shared by the operators of include/moe_operators.h.
#pragma once

#include "cache.cuh"
#include "../../include/moe_operators.h"

namespace moe {

constexpr int64_t kMaxPairs = 0x70000000;   // T * k: row numbers, and those a block past them, fit 31 bits

// SMs of the current device (looked up once per device).
int operator_sms();

// Address of the current device's flag that waits which run out set, for kernels outside grouped.cu (looked up once per device;
// NULL where that fails).  One flag, so that moe_operators_check waits for one copy.
uint32_t* operator_flag();

// For tests, outside the ABI: what moe_grouped_matmul_fp8 runs for such a call on a device of so many SMs, as {CTAs a tile, weight
// rows of a tile, stages of the ring, accumulators}.
extern "C" void moe_product8_form(int32_t P, int32_t E, int32_t N, int32_t K, int32_t act, int32_t quant, int32_t sms, int32_t* form);

__host__ __device__ __forceinline__ int64_t ceil_div64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// expert of a grouped row, or of a row tile: the e with first[e] <= i < first[e + 1]
__device__ __forceinline__ int expert_of(const int32_t* __restrict__ first, int E, int i) {
  int lo = 0, hi = E;   // first[lo] <= i < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(first + mid) <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ---------------------------------------------------------------------------
// 4-bit blocks
// ---------------------------------------------------------------------------
// byte of the scale of block b of padded row r: tiles of 128 rows x 4 blocks
__host__ __device__ __forceinline__ size_t scale_at(size_t r, int b, int block_groups) {
  const uint32_t t = (uint32_t)(r & 127);
  return ((r >> 7) * (size_t)block_groups + (size_t)(b >> 2)) * 512 + (t & 31) * 16 + (t >> 5) * 4 + (b & 3);
}

// value of an e4m3 code, exact in fp16
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  uint32_t h;
  asm("{\n .reg .b16 t;\n cvt.u16.u32 t, %1;\n cvt.rn.f16x2.e4m3x2 %0, t;\n}\n" : "=r"(h) : "r"(code));
  return __low2float(*reinterpret_cast<const __half2*>(&h));
}
// 2^(code - 127); 255 is NaN.  Code 0 is the subnormal 2^-127.
__device__ __forceinline__ float e8m0_value(uint32_t code) {
  return code == 255u ? __uint_as_float(0x7fffffffu) : code ? __uint_as_float(code << 23) : __uint_as_float(0x00400000u);
}
// nearest e4m3, ties to even, at most 448; x >= 0 or NaN (which gives the code of NaN)
__device__ __forceinline__ uint32_t to_e4m3(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(x));
  return r & 0xffu;
}
// two e2m1 codes, lo in the low nibble: nearest, ties to even, at most 6
__device__ __forceinline__ uint32_t to_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n cvt.u32.u8 %0, t;\n}\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 16 elements of a row as they are; a row of K starts on 16 elements' bytes from its 16-byte aligned matrix
template <typename X>
struct Raw16 {
  static constexpr int W = sizeof(X) == 4 ? 16 : 8;
  uint32_t w[W];
  __device__ __forceinline__ void load(const X* p) {
    const uint32_t* src = reinterpret_cast<const uint32_t*>(p);
    if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {   // 32 bytes an instruction
#pragma unroll
      for (int i = 0; i < W; i += 8)
        asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]), "=r"(w[i + 4]), "=r"(w[i + 5]), "=r"(w[i + 6]), "=r"(w[i + 7])
                     : "l"(src + i));
    } else {
#pragma unroll
      for (int i = 0; i < W; i += 4) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(src + i));
        w[i] = q.x; w[i + 1] = q.y; w[i + 2] = q.z; w[i + 3] = q.w;
      }
    }
  }
  // bits of the largest |x| as fp32
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0u;
    if constexpr (sizeof(X) == 4) {
#pragma unroll
      for (int i = 0; i < W; ++i) m = max(m, w[i] & 0x7fffffffu);
    } else {   // two at a time: bf16 patterns without their signs order like the values
#pragma unroll
      for (int i = 0; i < W; i += 2) m = __vimax3_u16x2(m, w[i] & 0x7fff7fffu, w[i + 1] & 0x7fff7fffu);
      m = max(m << 16, m & 0xffff0000u);
    }
    return m;
  }
  __device__ __forceinline__ void values(float (&v)[16]) const {
    if constexpr (sizeof(X) == 4) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
};

// Correctly rounded x / d from r = 1 / d rounded to nearest, without a division (Markstein 1990): with q = x r, the
// remainder x - q d is exact in one fma, and q + remainder * r rounds to the quotient.  Away from the ends of the exponent
// range (`regular`); a zero comes out positive.
__device__ __forceinline__ float quotient(float x, float d, float r) {
  const float q = x * r;
  return fmaf(fmaf(-q, d, x), r, q);
}
// two fp32 an instruction (codes of 805 MB of bf16 from quotients: 230 us one at a time, 211 so)
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(a), "f"(b));
  return p;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t p;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(a), "l"(b));
  return p;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t p;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p) : "l"(a), "l"(b), "l"(c));
  return p;
}
// for every |x| <= most; a remainder too small to be exact belongs to a quotient that rounds to code 0
__device__ __forceinline__ bool regular(float most, float d, float r) { return d > 1e-24f && d < 1e24f && most * r < 1e30f; }

// Scale code of a block and the value of one step, from the bits of its largest |x|; rg = 1 / g rounded.
// EXACT: as the format defines them, by correctly rounded divisions.  Otherwise (values that carry rounding errors of their
// own) by multiplications, good to three units; rg is then 1 / (g up) and sixth is up / 6 for an `up` that keeps 1 / g finite.
constexpr float kSixth = 0.16666667f;   // the fp32 nearest to 1 / 6
template <bool NV, bool EXACT = true>
__device__ __forceinline__ uint32_t block_scale(uint32_t amax_bits, float g, float rg, float& step, float sixth = kSixth) {
  if (NV) {
    if (amax_bits > 0x7f800000u) { step = 0.0f; return 0x7fu; }
    const float a = __uint_as_float(amax_bits) * sixth;
    const uint32_t code = to_e4m3(!EXACT ? a * rg : a > 1e-20f && regular(a, g, rg) ? quotient(a, g, rg) : __fdiv_rn(a, g));
    step = e4m3_value(code) * g;
    return code;
  }
  if (amax_bits > 0x7f800000u) { step = 0.0f; return 255u; }
  const int x = amax_bits ? max((int)(amax_bits >> 23) - 129, -127) : 0;
  step = e8m0_value((uint32_t)(x + 127));
  return (uint32_t)(x + 127);
}
// what a value is multiplied by (MXFP4: 2^-X, exact) -- NVFP4 divides by the step
__device__ __forceinline__ float e8m0_inverse(uint32_t code) { return e8m0_value(254u - code); }

// 16 values -> 8 bytes of codes
template <bool NV, bool EXACT = true>
__device__ __forceinline__ uint2 encode16(const float (&v)[16], uint32_t amax_bits, uint32_t code, float step) {
  if (!(step > 0.0f)) return make_uint2(0u, 0u);
  uint32_t w[2] = {0u, 0u};
  auto put = [&](int i, float lo, float hi) { w[i >> 2] |= to_e2m1x2(lo, hi) << (8 * (i & 3)); };
  auto put2 = [&](int i, uint64_t p) {
    float lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
    put(i, lo, hi);
  };
  float r;
  if (!NV) r = e8m0_inverse(code);
  else if (EXACT) r = __frcp_rn(step);
  else asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(step));
  if (!NV || (!EXACT && r < 1e38f)) {
    const uint64_t rr = pack2(r, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) put2(i, mul2(pack2(v[2 * i], v[2 * i + 1]), rr));
    return make_uint2(w[0], w[1]);
  }
  // (comparing the codes of quotients rounded down and up first, and doing this only where they differ, was no faster where
  // the matrix scale comes from the same bf16 values: ties are common there, 259 against 240 us for 805 MB one at a time)
  if (regular(__uint_as_float(amax_bits), step, r)) {
    // quotient() of -x, two at a time and by -r: so a zero keeps its sign, and the codes' signs are turned at the end
    const uint64_t nr = pack2(-r, -r), d = pack2(step, step);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t x = pack2(v[2 * i], v[2 * i + 1]), q = mul2(x, nr);
      put2(i, fma2(fma2(q, d, x), nr, q));
    }
    return make_uint2(w[0] ^ 0x88888888u, w[1] ^ 0x88888888u);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) put(i, __fdiv_rn(v[2 * i], step), __fdiv_rn(v[2 * i + 1], step));
  return make_uint2(w[0], w[1]);
}

// ---------------------------------------------------------------------------
// 8-bit blocks
// ---------------------------------------------------------------------------
constexpr float kLeast8 = 0x1p-100f;   // a block's largest |x| counts as this at least, so that no scale is 0
// two values -> two e4m3 codes, lo in the low byte
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace moe
