// 8-bit blocks (include/moe_operators.h: moe_quantize_fp8, moe_quantize_fp8_weights,
// moe_dequantize_fp8): e4m3 codes with one fp32 scale for 128 elements of a row, or for
// 128 x 128 elements of a matrix.
//
// Rows: a lane holds 16 elements, eight lanes a block; the largest |x| is taken over the bit
// patterns, so NaN and infinity show up above every number.  Rows for the experts are read and
// converted once a token and stored once an expert.  Weights: a block of threads holds a whole
// 128 x 128 tile in registers between finding its largest element and converting it.
//
// Codes are those of the correctly rounded quotient 448 x / a: with bf16 inputs 448 x is exact,
// and exact ties, which a reciprocal would break either way, are common (1 to 4 % of the
// codes of some rows).  Bound by memory: 2 bytes read and 1.03 written an element (bf16).
#include "operators.cuh"

#include <algorithm>

namespace moe {

namespace {

constexpr int Q_THREADS = 256;
constexpr int Q_WARPS = Q_THREADS / 32;
constexpr int Q_SEG = 32;          // units of 16 elements a warp takes of a row (blockIdx.y)

// What a block of largest |x| `bits` is scaled by: 448 x c over a c, c a power of two that keeps the quotient's steps in range.
struct Block8 { float mul, d, r, scale; bool bad; };
__device__ __forceinline__ Block8 block8(uint32_t bits) {
  Block8 b;
  b.bad = bits >= 0x7f800000u;
  const float a = fmaxf(__uint_as_float(b.bad ? 0u : bits), kLeast8), c = a > 1e24f ? 0x1p-64f : a < 1e-24f ? 0x1p64f : 1.0f;
  b.mul = 448.0f * c;
  b.d = a * c;
  b.r = __frcp_rn(b.d);
  b.scale = b.bad ? __uint_as_float(0x7fffffffu) : a * (1.0f / 448.0f);
  return b;
}
// 16 values -> 16 bytes.  quotient() of -x two at a time, by -r, so that a zero keeps its sign; the codes' signs turn at the end.
__device__ __forceinline__ uint4 encode16_8(const float (&v)[16], const Block8& b) {
  if (b.bad) return make_uint4(0u, 0u, 0u, 0u);
  const uint64_t m = pack2(b.mul, b.mul), nr = pack2(-b.r, -b.r), d = pack2(b.d, b.d);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t x = mul2(pack2(v[2 * i], v[2 * i + 1]), m), q = mul2(x, nr), y = fma2(fma2(q, d, x), nr, q);
    float lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(y));
    const uint32_t c = to_e4m3x2(lo, hi) ^ 0x8080u;
    w[i >> 1] = i & 1 ? w[i >> 1] | c << 16 : c;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

struct Rows8 {
  int64_t rows, out_rows;
  int K, k;
  const void* x;
  const int32_t* place;   // NULL: rows as they are
  uint8_t* codes;
  float* scales;
};

template <typename X, bool GROUPED>
__global__ void __launch_bounds__(Q_THREADS, sizeof(X) == 4 ? 4 : 6) quantize_rows8_kernel(Rows8 a) {
  pdl_wait();
  pdl_trigger();
  const int units = a.K / 16, lane = threadIdx.x & 31, c = (int)blockIdx.y * Q_SEG + lane;
  const bool live = c < units;
  auto store = [&](int64_t row, uint4 q, float scale) {
    if (!live) return;
    reinterpret_cast<uint4*>(a.codes + (size_t)row * a.K)[c] = q;
    if ((c & 7) == 0) a.scales[(size_t)(c >> 3) * a.out_rows + row] = scale;
  };
  for (int64_t r = (int64_t)blockIdx.x * Q_WARPS + (threadIdx.x >> 5); r < a.rows; r += (int64_t)gridDim.x * Q_WARPS) {
    Raw16<X> x;
    if (live) x.load(static_cast<const X*>(a.x) + (size_t)r * a.K + c * 16);
    uint32_t top = live ? x.top() : 0u;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const Block8 b = block8(top);
    uint4 q = make_uint4(0u, 0u, 0u, 0u);
    if (live) {
      float v[16];
      x.values(v);
      q = encode16_8(v, b);
    }
    if constexpr (!GROUPED) {
      store(r, q, b.scale);
    } else {
      for (int j = 0; j < a.k; ++j) {
        const int row = __ldg(a.place + r * a.k + j);
        if ((uint32_t)row < (uint32_t)a.out_rows) store(row, q, b.scale);
      }
    }
  }
}

// a tile of 128 x 128 a block: eight lanes a row, four rows a thread
template <typename X>
__global__ void __launch_bounds__(Q_THREADS, sizeof(X) == 4 ? 2 : 4)
quantize_tiles8_kernel(const X* __restrict__ w, int N, int K, int k_blocks, uint8_t* __restrict__ codes, float* __restrict__ scales) {
  __shared__ uint32_t tops[Q_WARPS];
  pdl_wait();
  pdl_trigger();
  const int nb = blockIdx.x / k_blocks, kb = blockIdx.x % k_blocks, g = blockIdx.y, tiles = gridDim.x;
  const int unit = kb * 8 + (threadIdx.x & 7), row0 = nb * 128 + (threadIdx.x >> 3);
  const bool live = unit < K / 16;
  const size_t at = ((size_t)g * N + row0) * K + unit * 16;
  Raw16<X> x[4];
  uint32_t top = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (live && row0 + 32 * i < N) x[i].load(w + at + (size_t)(32 * i) * K);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (live && row0 + 32 * i < N) top = max(top, x[i].top());
  top = __reduce_max_sync(0xffffffffu, top);
  if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < Q_WARPS; ++i) top = max(top, tops[i]);
  const Block8 b = block8(top);
  if (threadIdx.x == 0) scales[(size_t)g * tiles + blockIdx.x] = b.scale;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (live && row0 + 32 * i < N) {
      float v[16];
      x[i].values(v);
      *reinterpret_cast<uint4*>(codes + at + (size_t)(32 * i) * K) = encode16_8(v, b);
    }
}

// two e4m3 codes as fp32, exact (through fp16)
__device__ __forceinline__ float2 e4m3x2_values(uint32_t codes) {
  uint32_t h;
  asm("{\n .reg .b16 t;\n cvt.u16.u32 t, %1;\n cvt.rn.f16x2.e4m3x2 %0, t;\n}\n" : "=r"(h) : "r"(codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// scale of row r, block b of matrix g: scales[g * per + (r / high) * rs + b * bs]
struct Scales8 { int64_t per, rs, bs; int high; };

template <typename O>
__global__ void __launch_bounds__(Q_THREADS) dequantize8_kernel(const uint8_t* __restrict__ codes, const float* __restrict__ scales, Scales8 sc,
                                                                int64_t rows, int K, O* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const int64_t g = blockIdx.z;
  if constexpr (sizeof(O) == 4) {
    // four elements of each of four blocks a lane, so that a store's 512 bytes are in one place (32 x 4096 x 2000: 267 us with 16 in a row, now 195)
    const int e0 = (int)blockIdx.y * (Q_SEG * 16) + 4 * (threadIdx.x & 31);
    for (int64_t r = (int64_t)blockIdx.x * Q_WARPS + (threadIdx.x >> 5); r < rows; r += (int64_t)gridDim.x * Q_WARPS) {
      const size_t at = (size_t)(g * rows + r) * K + e0;
      const float* sp = scales + g * sc.per + r / sc.high * sc.rs + (e0 >> 7) * sc.bs;
      uint32_t w[4];
      float s[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e0 + 128 * i < K) {
          w[i] = __ldg(reinterpret_cast<const uint32_t*>(codes + at + 128 * i));
          s[i] = __ldg(sp + i * sc.bs);
        }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e0 + 128 * i < K) {
          const float2 x = e4m3x2_values(w[i] & 0xffffu), y = e4m3x2_values(w[i] >> 16);
          *reinterpret_cast<float4*>(out + at + 128 * i) = make_float4(x.x * s[i], x.y * s[i], y.x * s[i], y.y * s[i]);
        }
    }
  } else {
    const int units = K / 16, c = (int)blockIdx.y * Q_SEG + (threadIdx.x & 31);
    if (c >= units) return;
    for (int64_t r = (int64_t)blockIdx.x * Q_WARPS + (threadIdx.x >> 5); r < rows; r += (int64_t)gridDim.x * Q_WARPS) {
      const size_t at = (size_t)(g * rows + r) * K + c * 16;
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(codes + at));
      const float s = __ldg(scales + g * sc.per + r / sc.high * sc.rs + (c >> 3) * sc.bs);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
      O res[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 x = e4m3x2_values((w[i >> 1] >> (16 * (i & 1))) & 0xffffu);
        res[2 * i] = (O)(x.x * s);
        res[2 * i + 1] = (O)(x.y * s);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) reinterpret_cast<uint4*>(out + at)[i] = reinterpret_cast<const uint4*>(res)[i];
    }
  }
}

dim3 rows_grid(int64_t rows, int G, int K) {
  const int segs = (K / 16 + Q_SEG - 1) / Q_SEG;
  const int64_t most = std::max<int64_t>(1, (int64_t)operator_sms() * 64 / segs / G);
  return dim3((unsigned)std::min<int64_t>((rows + Q_WARPS - 1) / Q_WARPS, most), (unsigned)segs, (unsigned)G);
}

moe_status check_fp8(int32_t G, int64_t rows, int32_t K, int32_t dtype) {
  if (G < 0 || G > 65535 || rows < 0) return fail(MOE_EINVAL, "matrices (at most 65535) and rows must not be negative, got %d of %lld", G, (long long)rows);
  if (K < 16 || K % 16 || K > 1 << 24) return fail(MOE_EINVAL, "K = %d is not a multiple of 16 (at most 2^24)", K);
  if (dtype != MOE_F32 && dtype != MOE_BF16) return fail(MOE_EINVAL, "dtype must be MOE_F32 or MOE_BF16");
  return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_quantize_fp8(int32_t T, int32_t K, int32_t dtype, const void* x, int32_t k, const int32_t* place, uint8_t* codes,
                                       float* scales, void* stream) {
  moe_status st = check_fp8(1, T, K, dtype);
  if (st != MOE_OK) return st;
  if (k < 1 || (!place && k != 1) || (int64_t)T * k > kMaxPairs)
    return fail(MOE_EINVAL, "k >= 1 (1 without place) and at most %lld rows are needed, got T %d, k %d", (long long)kMaxPairs, T, k);
  if (T == 0) return MOE_OK;
  if (!x || !codes || !scales) return fail(MOE_EINVAL, "x, codes and scales must not be NULL");
  if (!aligned_to(x, 16) || !aligned_to(codes, 16) || !aligned_to(scales, 4) || !aligned_to(place, 4))
    return fail(MOE_EINVAL, "x and codes must be 16-byte aligned, scales and place 4-byte aligned");
  const Rows8 a{T, (int64_t)T * k, K, k, x, place, codes, scales};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid = rows_grid(T, 1, K), block(Q_THREADS);
  const bool f32 = dtype == MOE_F32;
  CK(place ? (f32 ? launch_pdl(quantize_rows8_kernel<float, true>, grid, block, 0, s, a) : launch_pdl(quantize_rows8_kernel<__nv_bfloat16, true>, grid, block, 0, s, a))
           : (f32 ? launch_pdl(quantize_rows8_kernel<float, false>, grid, block, 0, s, a) : launch_pdl(quantize_rows8_kernel<__nv_bfloat16, false>, grid, block, 0, s, a)));
  return MOE_OK;
}

extern "C" moe_status moe_quantize_fp8_weights(int32_t G, int32_t N, int32_t K, int32_t dtype, const void* w, uint8_t* codes, float* scales, void* stream) {
  moe_status st = check_fp8(G, N, K, dtype);
  if (st != MOE_OK) return st;
  const int64_t kb = (K + 127) / 128, tiles = ((int64_t)N + 127) / 128 * kb;
  if (tiles > 0x7fffffff) return fail(MOE_EINVAL, "N = %d rows of K = %d are too many blocks", N, K);
  if (G == 0 || N == 0) return MOE_OK;
  if (!w || !codes || !scales) return fail(MOE_EINVAL, "w, codes and scales must not be NULL");
  if (!aligned_to(w, 16) || !aligned_to(codes, 16) || !aligned_to(scales, 4)) return fail(MOE_EINVAL, "w and codes must be 16-byte aligned, scales 4-byte aligned");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)tiles, (unsigned)G), block(Q_THREADS);
  CK(dtype == MOE_F32 ? launch_pdl(quantize_tiles8_kernel<float>, grid, block, 0, s, static_cast<const float*>(w), N, K, (int)kb, codes, scales)
                      : launch_pdl(quantize_tiles8_kernel<__nv_bfloat16>, grid, block, 0, s, static_cast<const __nv_bfloat16*>(w), N, K, (int)kb, codes, scales));
  return MOE_OK;
}

extern "C" moe_status moe_dequantize_fp8(int32_t G, int32_t N, int32_t K, int32_t tiles, const uint8_t* codes, const float* scales, int32_t dtype, void* out,
                                         void* stream) {
  moe_status st = check_fp8(G, N, K, dtype);
  if (st != MOE_OK) return st;
  if (!tiles && G != 1) return fail(MOE_EINVAL, "rows are one matrix, got %d", G);
  if (G == 0 || N == 0) return MOE_OK;
  if (!codes || !scales || !out) return fail(MOE_EINVAL, "codes, scales and out must not be NULL");
  if (!aligned_to(codes, 16) || !aligned_to(out, 16) || !aligned_to(scales, 4)) return fail(MOE_EINVAL, "codes and out must be 16-byte aligned, scales 4-byte aligned");
  const int64_t kb = (K + 127) / 128;
  const Scales8 sc = tiles ? Scales8{((int64_t)N + 127) / 128 * kb, kb, 1, 128} : Scales8{0, 1, N, 1};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid = rows_grid(N, G, K), block(Q_THREADS);
  CK(dtype == MOE_F32 ? launch_pdl(dequantize8_kernel<float>, grid, block, 0, s, codes, scales, sc, (int64_t)N, K, static_cast<float*>(out))
                      : launch_pdl(dequantize8_kernel<__nv_bfloat16>, grid, block, 0, s, codes, scales, sc, (int64_t)N, K, static_cast<__nv_bfloat16*>(out)));
  return MOE_OK;
}
