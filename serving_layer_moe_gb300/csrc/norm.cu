// The end of a block (include/moe_operators.h: moe_combine_norm): the experts' rows summed by
// their gates, the shared expert's rows, the norm behind the block, its gate, the scaled
// residual, and the norm before the next block, in one pass.
//
//   c = sum_j w[j] y[place[j]] + shared;   c = c / sqrt(mean c^2 + eps) * post;   c = gate c
//   h = alpha r + c;                       z = h / sqrt(mean h^2 + eps) * pre
//
// A block of threads holds a token's row in fp32 registers from the first load to the last
// store, so each row is read and written once.  The two means are the only points where its
// threads wait for one another; other blocks' loads fill that time.  Bound by memory.
#include "operators.cuh"

#include <algorithm>

namespace moe {

namespace {

constexpr int MAX_THREADS = 1024;
constexpr int MAX_WIDTH = 32768;

struct EndArgs {
  int T, k, N;
  const void *y, *shared, *residual, *post, *pre;   // any but residual may be NULL
  const int32_t* place;                             // NULL: row t of y as it is
  const float *w, *gate;
  int gate_rows;                                    // gate holds a value for each token, otherwise for each channel
  int post_bf16, pre_bf16, z_bf16;
  float alpha, eps;
  void *h, *z;                                      // either may be NULL
};

// U consecutive values as fp32
template <int U, typename X>
__device__ __forceinline__ void load(const X* p, float (&v)[U]) {
  if constexpr (U == 1) {
    v[0] = (float)*p;
  } else if constexpr (sizeof(X) == 2) {
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 q = __ldg(reinterpret_cast<const float4*>(p) + i);
      v[4 * i] = q.x; v[4 * i + 1] = q.y; v[4 * i + 2] = q.z; v[4 * i + 3] = q.w;
    }
  }
}
// of a norm's weights, in either type
template <int U>
__device__ __forceinline__ void load_any(const void* p, int bf16, size_t at, float (&v)[U]) {
  if (bf16) load(static_cast<const __nv_bfloat16*>(p) + at, v);
  else load(static_cast<const float*>(p) + at, v);
}
template <int U, typename X>
__device__ __forceinline__ void store(X* p, const float (&v)[U]) {
  if constexpr (U == 1) {
    *p = (X)v[0];
  } else if constexpr (sizeof(X) == 2) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  }
}

// sum over the block, the same in every thread and whatever the order in which warps run; `part` holds a value a warp
__device__ __forceinline__ float block_sum(float v, float* part) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (warps == 1) return v;
  if (lane == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? part[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// V units of U values a thread, unit threadIdx.x first and then every blockDim.x-th
template <typename Y, typename R, int U, int V>
__global__ void __launch_bounds__(MAX_THREADS) block_end_kernel(EndArgs a) {
  __shared__ float parts[2][32];
  pdl_wait();
  pdl_trigger();
  const int units = a.N / U;
  const Y *y = static_cast<const Y*>(a.y), *shared = static_cast<const Y*>(a.shared);
  const R* residual = static_cast<const R*>(a.residual);
  const float per = 1.0f / (float)a.N;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    float c[V][U] = {}, r[V][U];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int u = threadIdx.x + v * blockDim.x;
      if (u < units) load(residual + (size_t)t * a.N + u * U, r[v]);
    }
    if (y) {
      const int P = a.place ? a.T * a.k : a.T;
      for (int j = 0; j < (a.place ? a.k : 1); ++j) {
        const int row = a.place ? __ldg(a.place + (size_t)t * a.k + j) : t;
        if ((unsigned)row >= (unsigned)P) continue;
        const float w = a.place ? __ldg(a.w + (size_t)t * a.k + j) : 1.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int u = threadIdx.x + v * blockDim.x;
          if (u >= units) continue;
          float x[U];
          load(y + (size_t)row * a.N + u * U, x);
#pragma unroll
          for (int i = 0; i < U; ++i) c[v][i] = fmaf(w, x[i], c[v][i]);
        }
      }
      if (shared) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int u = threadIdx.x + v * blockDim.x;
          if (u >= units) continue;
          float x[U];
          load(shared + (size_t)t * a.N + u * U, x);
#pragma unroll
          for (int i = 0; i < U; ++i) c[v][i] += x[i];
        }
      }
      if (a.post) {
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int i = 0; i < U; ++i) s = fmaf(c[v][i], c[v][i], s);
        const float inv = rsqrtf(fmaf(block_sum(s, parts[0]), per, a.eps));
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int u = threadIdx.x + v * blockDim.x;
          if (u >= units) continue;
          float x[U];
          load_any(a.post, a.post_bf16, (size_t)u * U, x);
#pragma unroll
          for (int i = 0; i < U; ++i) c[v][i] *= inv * x[i];
        }
      }
      if (a.gate) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int u = threadIdx.x + v * blockDim.x;
          if (u >= units) continue;
          float x[U];
          if (a.gate_rows) {
            const float g = __ldg(a.gate + t);
#pragma unroll
            for (int i = 0; i < U; ++i) x[i] = g;
          } else {
            load(a.gate + (size_t)u * U, x);
          }
#pragma unroll
          for (int i = 0; i < U; ++i) c[v][i] *= x[i];
        }
      }
    }
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int u = threadIdx.x + v * blockDim.x;
      if (u >= units) continue;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        c[v][i] = fmaf(a.alpha, r[v][i], c[v][i]);
        s = fmaf(c[v][i], c[v][i], s);
      }
      if (a.h) store(static_cast<R*>(a.h) + (size_t)t * a.N + u * U, c[v]);
    }
    if (a.z) {
      const float inv = rsqrtf(fmaf(block_sum(s, parts[1]), per, a.eps));
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int u = threadIdx.x + v * blockDim.x;
        if (u >= units) continue;
        float x[U];
        load_any(a.pre, a.pre_bf16, (size_t)u * U, x);
#pragma unroll
        for (int i = 0; i < U; ++i) x[i] *= inv * c[v][i];
        const size_t at = (size_t)t * a.N + u * U;
        if (a.z_bf16) store(static_cast<__nv_bfloat16*>(a.z) + at, x);
        else store(static_cast<float*>(a.z) + at, x);
      }
    }
    __syncthreads();   // the parts have been read
  }
}

template <typename Y, typename R, int U, int V>
moe_status launch_end(const EndArgs& a, int threads, cudaStream_t s) {
  const int grid = (int)std::min<int64_t>(a.T, (int64_t)operator_sms() * std::max(1, 2048 / threads));
  CK(launch_pdl(block_end_kernel<Y, R, U, V>, dim3(grid), dim3(threads), 0, s, a));
  return MOE_OK;
}

// Units a thread: as few as reach the row with 1024 threads, and more, down to 256 threads, when there are tokens for every SM.
template <typename Y, typename R>
moe_status run_end(const EndArgs& a, bool wide, cudaStream_t s) {
  const int units = wide ? a.N / 8 : a.N;
  const int most = a.T >= 2 * operator_sms() ? 256 : MAX_THREADS;
  int v = 1;
  while (v < (wide ? 4 : 32) && (units + v - 1) / v > most) v *= 2;
  const int threads = ((units + v - 1) / v + 31) / 32 * 32;
  if (wide)
    return v == 1 ? launch_end<Y, R, 8, 1>(a, threads, s) : v == 2 ? launch_end<Y, R, 8, 2>(a, threads, s) : launch_end<Y, R, 8, 4>(a, threads, s);
  return v <= 4 ? launch_end<Y, R, 1, 4>(a, ((units + 3) / 4 + 31) / 32 * 32, s) : v == 8 ? launch_end<Y, R, 1, 8>(a, threads, s)
         : v == 16 ? launch_end<Y, R, 1, 16>(a, threads, s) : launch_end<Y, R, 1, 32>(a, threads, s);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_combine_norm(int32_t T, int32_t k, int32_t N, int32_t y_dtype, const void* y, const int32_t* place, const float* w,
                                       const void* shared, int32_t post_dtype, const void* post, int32_t gate_rows, const float* gate, float alpha,
                                       int32_t r_dtype, const void* residual, int32_t pre_dtype, const void* pre, float eps, void* h,
                                       int32_t z_dtype, void* z, void* stream) {
  auto is_float = [](int32_t d) { return d == MOE_F32 || d == MOE_BF16; };
  if (T < 0 || k < 1 || N < 1 || N > MAX_WIDTH || (int64_t)T * k > kMaxPairs)
    return fail(MOE_EINVAL, "T >= 0, k >= 1, 1 <= N <= %d and at most %lld pairs are needed, got T %d, k %d, N %d", MAX_WIDTH, (long long)kMaxPairs, T, k, N);
  if (!is_float(y_dtype) || !is_float(r_dtype) || !is_float(post_dtype) || !is_float(pre_dtype) || !is_float(z_dtype))
    return fail(MOE_EINVAL, "every dtype must be MOE_F32 or MOE_BF16");
  if (!(eps >= 1.1754944e-38f) || !(eps < INFINITY) || !(alpha - alpha == 0.0f)) return fail(MOE_EINVAL, "eps must be a positive normal number and alpha finite");
  if ((place && (!y || !w)) || (!place && k != 1)) return fail(MOE_EINVAL, "place needs y and topk_w; without place k must be 1");
  if (!y && (shared || post || gate)) return fail(MOE_EINVAL, "shared, post and gate need y");
  if ((pre != nullptr) != (z != nullptr) || (!h && !z)) return fail(MOE_EINVAL, "pre and z go together, and h or z must not be NULL");
  if (T == 0) return MOE_OK;
  if (!residual) return fail(MOE_EINVAL, "residual must not be NULL");
  const bool wide = N % 8 == 0;
  auto ok = [&](const void* p, int32_t d) { return aligned_to(p, wide ? 16 : d == MOE_BF16 ? 2 : 4); };
  if (!ok(y, y_dtype) || !ok(shared, y_dtype) || !ok(residual, r_dtype) || !ok(h, r_dtype) || !ok(post, post_dtype) || !ok(pre, pre_dtype) ||
      !ok(z, z_dtype) || !(gate_rows ? aligned_to(gate, 4) : ok(gate, MOE_F32)) || !aligned_to(place, 4) || !aligned_to(w, 4))
    return fail(MOE_EINVAL, "rows and weights must be 16-byte aligned (N a multiple of 8; else to their elements), place and topk_w 4-byte aligned");
  EndArgs a{};
  a.T = T; a.k = k; a.N = N; a.y = y; a.shared = shared; a.residual = residual; a.post = post; a.pre = pre; a.place = place; a.w = w; a.gate = gate;
  a.gate_rows = gate_rows; a.post_bf16 = post_dtype == MOE_BF16; a.pre_bf16 = pre_dtype == MOE_BF16; a.z_bf16 = z_dtype == MOE_BF16;
  a.alpha = alpha; a.eps = eps; a.h = h; a.z = z;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool yb = y_dtype == MOE_BF16, rb = r_dtype == MOE_BF16;
  return yb ? (rb ? run_end<__nv_bfloat16, __nv_bfloat16>(a, wide, s) : run_end<__nv_bfloat16, float>(a, wide, s))
            : (rb ? run_end<float, __nv_bfloat16>(a, wide, s) : run_end<float, float>(a, wide, s));
}
