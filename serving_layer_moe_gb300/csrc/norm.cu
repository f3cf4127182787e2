// The end of a block (include/moe_operators.h: moe_combine_norm): the experts' rows summed by
// their gates, the shared expert's rows, the norm behind the block, its gate, the scaled
// residual, and the norm before the next block, in one pass.
//
//   c = sum_j w[j] y[place[j]] + shared;   c = c / sqrt(mean c^2 + eps) * post;   c = gate c
//   h = alpha r + c;                       z = h / sqrt(mean h^2 + eps) * pre
//
// A block of threads holds a token's row in fp32, in registers or shared memory, from the first load to the last
// store, so each row is read and written once.  The two means are the only points where its
// threads wait for one another; other blocks' loads fill that time.  Bound by memory.
#include "operators.cuh"

#include <algorithm>

namespace moe {

namespace {

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

// U consecutive values (8, 16-byte aligned) as they are, so that many can be on their way, and as fp32
template <int U, typename X>
struct Raw {
  static constexpr int Q = U * (int)sizeof(X) / 16;
  uint4 q[Q];
  __device__ __forceinline__ void load(const X* p) {
#pragma unroll
    for (int i = 0; i < Q; ++i) q[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void read(const X* p) {   // from shared memory
#pragma unroll
    for (int i = 0; i < Q; ++i) q[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void values(float (&v)[U]) const {
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const uint32_t u[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        if constexpr (sizeof(X) == 2) {
          v[8 * i + 2 * h] = __uint_as_float(u[h] << 16);
          v[8 * i + 2 * h + 1] = __uint_as_float(u[h] & 0xffff0000u);
        } else {
          v[4 * i + h] = __uint_as_float(u[h]);
        }
      }
    }
  }
};
template <int U, typename X>
__device__ __forceinline__ void load(const X* p, float (&v)[U]) {
  Raw<U, X> r;
  r.load(p);
  r.values(v);
}
// of a norm's weights, in either type
template <int U>
__device__ __forceinline__ void load_any(const void* p, int bf16, size_t at, float (&v)[U]) {
  if (bf16) load(static_cast<const __nv_bfloat16*>(p) + at, v);
  else load(static_cast<const float*>(p) + at, v);
}
template <int U, typename X>
__device__ __forceinline__ void store(X* p, const float (&v)[U]) {
  if constexpr (sizeof(X) == 2) {
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

// V units of 8 values a thread, unit threadIdx.x first and then every blockDim.x-th; J rows of y on their way at a time
template <typename Y, typename R, int V, int J>
__global__ void __launch_bounds__(1024, 1) block_end_kernel(EndArgs a) {
  constexpr int U = 8;
  __shared__ float parts[2][32];
  pdl_wait();
  pdl_trigger();
  const int units = a.N / U;
  const Y *y = static_cast<const Y*>(a.y), *shared = static_cast<const Y*>(a.shared);
  const R* residual = static_cast<const R*>(a.residual);
  const float per = 1.0f / (float)a.N;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    float c[V][U] = {};
    Raw<U, R> r[V];
    auto each = [&](auto f) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int u = threadIdx.x + v * blockDim.x;
        if (u < units) f(v, (size_t)u * U);
      }
    };
    // Rows are loaded without a test of the width, so that a row's loads do not wait for one another: behind it, its last unit again.
    // us of 250 tokens, N 7168, 8 rows each and all parts 12.4 with the test, 10.3 without.
    auto place_of = [&](int v) { return (size_t)min((int)(threadIdx.x + v * blockDim.x), units - 1) * U; };
    if (y) {
      const int k = a.place ? a.k : 1, P = a.T * k;
      for (int j0 = 0; j0 < k; j0 += J) {
        int row[J];
        float w[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const bool there = j0 + j < k;
          row[j] = !there ? -1 : a.place ? __ldg(a.place + (size_t)t * k + j0 + j) : t;
          if ((unsigned)row[j] >= (unsigned)P) row[j] = -1;
          w[j] = there && a.place ? __ldg(a.w + (size_t)t * k + j0 + j) : 1.0f;
        }
        Raw<U, Y> x[J][V];
#pragma unroll
        for (int j = 0; j < J; ++j)
          if (row[j] >= 0)
#pragma unroll
            for (int v = 0; v < V; ++v) x[j][v].load(y + (size_t)row[j] * a.N + place_of(v));
#pragma unroll
        for (int j = 0; j < J; ++j)
          if (row[j] >= 0)
#pragma unroll
            for (int v = 0; v < V; ++v) {
              float f[U];
              x[j][v].values(f);
#pragma unroll
              for (int i = 0; i < U; ++i) c[v][i] = fmaf(w[j], f[i], c[v][i]);
            }
      }
      if (shared) {
        Raw<U, Y> x[V];
#pragma unroll
        for (int v = 0; v < V; ++v) x[v].load(shared + (size_t)t * a.N + place_of(v));
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float f[U];
          x[v].values(f);
#pragma unroll
          for (int i = 0; i < U; ++i) c[v][i] += f[i];
        }
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) r[v].load(residual + (size_t)t * a.N + place_of(v));   // on its way during the first mean
    if (a.post) {
      float s = 0.0f;
      each([&](int v, size_t) {
#pragma unroll
        for (int i = 0; i < U; ++i) s = fmaf(c[v][i], c[v][i], s);
      });
      const float inv = rsqrtf(fmaf(block_sum(s, parts[0]), per, a.eps));
      each([&](int v, size_t at) {
        float x[U];
        load_any(a.post, a.post_bf16, at, x);
#pragma unroll
        for (int i = 0; i < U; ++i) c[v][i] *= inv * x[i];
      });
    }
    if (a.gate) {
      const float g = a.gate_rows ? __ldg(a.gate + t) : 1.0f;
      each([&](int v, size_t at) {
        float x[U];
        if (!a.gate_rows) load(a.gate + at, x);
#pragma unroll
        for (int i = 0; i < U; ++i) c[v][i] *= a.gate_rows ? g : x[i];
      });
    }
    float s = 0.0f;
    each([&](int v, size_t at) {
      float x[U];
      r[v].values(x);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        c[v][i] = fmaf(a.alpha, x[i], c[v][i]);
        s = fmaf(c[v][i], c[v][i], s);
      }
      if (a.h) store(static_cast<R*>(a.h) + (size_t)t * a.N + at, c[v]);
    });
    if (a.z) {
      const float inv = rsqrtf(fmaf(block_sum(s, parts[1]), per, a.eps));
      each([&](int v, size_t at) {
        float x[U];
        load_any(a.pre, a.pre_bf16, at, x);
#pragma unroll
        for (int i = 0; i < U; ++i) x[i] *= inv * c[v][i];
        at += (size_t)t * a.N;
        if (a.z_bf16) store(static_cast<__nv_bfloat16*>(a.z) + at, x);
        else store(static_cast<float*>(a.z) + at, x);
      });
    }
    __syncthreads();   // the parts have been read
  }
}

// Any width: single values, which start anywhere.  The row is in shared memory as fp32, each value its thread's own, so that a thread needs
// few registers, none of them for values it has yet to use, and has W loads on their way.  us with the row in registers / so: 4096 tokens, N
// 1001, 2 rows each and all parts 26 / 23; 2000 tokens, N 8191 150 / 105 (bound 29); 1000 tokens, N 16383 414 / 108; one token, N 8191 15 / 13.
// Four values of two rows at a time 25, 107, 112 and 14, eight of two rows 39, 158, 164 and 18 (spilled).
constexpr int ANY_THREADS = 512, ANY_VALUES = 8;
template <typename Y, typename R>
__global__ void __launch_bounds__(ANY_THREADS, 2) block_end_any_kernel(EndArgs a) {
  constexpr int W = ANY_VALUES;
  extern __shared__ float c_row[];
  __shared__ float parts[2][32];
  pdl_wait();
  pdl_trigger();
  const Y *y = static_cast<const Y*>(a.y), *shared = static_cast<const Y*>(a.shared);
  const R* residual = static_cast<const R*>(a.residual);
  const float per = 1.0f / (float)a.N;
  const int k = a.place ? a.k : 1, P = a.T * k, stride = blockDim.x;
  // f(values' places, of which the thread's i-th is there if there[i]; behind the row's end they are its last one)
  auto each = [&](auto f) {
    for (int u0 = threadIdx.x; u0 < a.N; u0 += W * stride) {
      int at[W];
      bool there[W];
#pragma unroll
      for (int i = 0; i < W; ++i) {
        there[i] = u0 + i * stride < a.N;
        at[i] = min(u0 + i * stride, a.N - 1);
      }
      f(at, there);
    }
  };
  auto weights = [&](const void* p, int bf16, const int (&at)[W], float (&x)[W]) {
    if (bf16)
#pragma unroll
      for (int i = 0; i < W; ++i) x[i] = (float)static_cast<const __nv_bfloat16*>(p)[at[i]];
    else
#pragma unroll
      for (int i = 0; i < W; ++i) x[i] = static_cast<const float*>(p)[at[i]];
  };
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const size_t row0 = (size_t)t * a.N;
    float s = 0.0f;
    if (y)
      each([&](const int (&at)[W], const bool (&there)[W]) {
        float c[W] = {};
        for (int j = 0; j < k; ++j) {
          const int row = a.place ? __ldg(a.place + (size_t)t * k + j) : t;
          if ((unsigned)row >= (unsigned)P) continue;
          const float w = a.place ? __ldg(a.w + (size_t)t * k + j) : 1.0f;
          Y x[W];
#pragma unroll
          for (int i = 0; i < W; ++i) x[i] = y[(size_t)row * a.N + at[i]];
#pragma unroll
          for (int i = 0; i < W; ++i) c[i] = fmaf(w, (float)x[i], c[i]);
        }
        if (shared) {
          Y x[W];
#pragma unroll
          for (int i = 0; i < W; ++i) x[i] = shared[row0 + at[i]];
#pragma unroll
          for (int i = 0; i < W; ++i) c[i] += (float)x[i];
        }
#pragma unroll
        for (int i = 0; i < W; ++i)
          if (there[i]) {
            c_row[at[i]] = c[i];
            s = fmaf(c[i], c[i], s);
          }
      });
    const float inv_post = a.post ? rsqrtf(fmaf(block_sum(s, parts[0]), per, a.eps)) : 1.0f, token_gate = a.gate && a.gate_rows ? __ldg(a.gate + t) : 1.0f;
    s = 0.0f;
    each([&](const int (&at)[W], const bool (&there)[W]) {
      R r[W];
      float c[W] = {}, x[W];
#pragma unroll
      for (int i = 0; i < W; ++i) r[i] = residual[row0 + at[i]];
      if (y)
#pragma unroll
        for (int i = 0; i < W; ++i) c[i] = there[i] ? c_row[at[i]] : 0.0f;
      if (a.post) {
        weights(a.post, a.post_bf16, at, x);
#pragma unroll
        for (int i = 0; i < W; ++i) c[i] *= inv_post * x[i];
      }
      if (a.gate) {
        if (!a.gate_rows) weights(a.gate, 0, at, x);
#pragma unroll
        for (int i = 0; i < W; ++i) c[i] *= a.gate_rows ? token_gate : x[i];
      }
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float h = fmaf(a.alpha, (float)r[i], c[i]);
        if (!there[i]) continue;
        if (a.h) static_cast<R*>(a.h)[row0 + at[i]] = (R)h;
        if (a.z) c_row[at[i]] = h;
        s = fmaf(h, h, s);
      }
    });
    if (a.z) {
      const float inv = rsqrtf(fmaf(block_sum(s, parts[1]), per, a.eps));
      each([&](const int (&at)[W], const bool (&there)[W]) {
        float x[W];
        weights(a.pre, a.pre_bf16, at, x);
#pragma unroll
        for (int i = 0; i < W; ++i)
          if (there[i]) {
            const float z = x[i] * (inv * c_row[at[i]]);
            if (a.z_bf16) static_cast<__nv_bfloat16*>(a.z)[row0 + at[i]] = (__nv_bfloat16)z;
            else static_cast<float*>(a.z)[row0 + at[i]] = z;
          }
      });
    }
    __syncthreads();   // the parts have been read
  }
}

// ---------------------------------------------------------------------------
// The same for many tokens: rows come ahead, in a ring of D of them in shared memory, so that loads never wait for a mean.
// A thread copies what it will read itself (cp.async), so nothing is waited for but its own copies.  A token's rows are
// its pairs', the shared one, the residual; the norms' weights stay in registers.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void copy16(uint32_t to, const void* from) { asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory"); }

// D steps of two rows in the ring.  us of 4096 tokens, N 7168, 8 rows each and all parts (bound 104 bf16, 201 fp32): one row a step 154
// and 204; two rows, the norms' weights in registers and one block an SM 138 and 202; weights read for each token (KEEP
// false), registers for two blocks an SM 129 and 237.  Without the ring, bf16: 147 to 203.
template <typename Y, typename R, int V, int D, bool KEEP, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) block_stream_kernel(EndArgs a) {
  constexpr int U = 8;
  extern __shared__ uint4 ring[];
  __shared__ float parts[2][32];
  pdl_wait();
  pdl_trigger();
  // A unit's place is the same whatever the row's type: it stays the thread's own.
  constexpr int WIDE = sizeof(Y) > sizeof(R) ? sizeof(Y) : sizeof(R);
  const int units = a.N / U, lane = threadIdx.x & 31;
  const int k = a.y ? a.place ? a.k : 1 : 0, sums = k + (a.shared ? 1 : 0), steps = sums / 2 + 1, last = 2 * steps - 1, P = a.T * max(k, 1);
  const uint32_t row_bytes = (uint32_t)(a.N * WIDE), base = (uint32_t)__cvta_generic_to_shared(ring);
  const float per = 1.0f / (float)a.N;
  float post[KEEP ? V : 1][U], pre[KEEP ? V : 1][U], gate[KEEP ? V : 1][U];
  auto each = [&](auto f) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int u = threadIdx.x + v * blockDim.x;
      if (u < units) f(v, u * U);
    }
  };
  auto load_post = [&](int at, float (&x)[U]) { load_any(a.post, a.post_bf16, (size_t)at, x); };
  auto load_pre = [&](int at, float (&x)[U]) { load_any(a.pre, a.pre_bf16, (size_t)at, x); };
  auto load_gate = [&](int at, float (&x)[U]) {
    if (a.gate && !a.gate_rows) load(a.gate + at, x);
  };
  if (KEEP)
    each([&](int v, int at) {
      if (a.post) load_post(at, post[v]);
      if (a.z) load_pre(at, pre[v]);
      load_gate(at, gate[v]);
    });
  // Lane j has row j of a token: its pairs', the shared one, and the residual as the last of the last step.  row_of: the pair's row, as
  // it is loaded; address: where the row is, 0 where there is none.
  auto row_of = [&](int t) { return t >= a.T || lane >= k ? -1 : a.place ? __ldg(a.place + (size_t)t * k + lane) : t; };
  auto address = [&](int t, int row) {
    return t >= a.T ? 0ull
           : lane < k ? (unsigned)row < (unsigned)P ? (unsigned long long)(static_cast<const Y*>(a.y) + (size_t)row * a.N) : 0ull
           : lane < sums ? (unsigned long long)(static_cast<const Y*>(a.shared) + (size_t)t * a.N)
           : lane == last ? (unsigned long long)(static_cast<const R*>(a.residual) + (size_t)t * a.N) : 0ull;
  };

  int pt = blockIdx.x, ps = 0, p_slot = 0;   // the next step to copy
  int p_row = row_of(pt + gridDim.x);
  unsigned long long p_at = address(pt, row_of(pt));
  auto copy = [&]() {
    if (pt < a.T) {
      const uint32_t to = base + (uint32_t)p_slot * (2 * row_bytes);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const char* from = reinterpret_cast<const char*>(__shfl_sync(0xffffffffu, p_at, 2 * ps + h));
        if (!from) continue;
        each([&](int, int at) {
          const int size = h == 1 && sizeof(Y) != sizeof(R) && ps == steps - 1 ? sizeof(R) : sizeof(Y), bytes = sizeof(Y) == sizeof(R) ? (int)sizeof(Y) : size;
#pragma unroll
          for (int i = 0; i < WIDE / 2; ++i)
            if (i < bytes / 2) copy16(to + h * row_bytes + at * WIDE + 16 * i, from + at * bytes + 16 * i);
        });
      }
      if (++ps == steps) {
        ps = 0;
        pt += gridDim.x;
        p_at = address(pt, p_row);
        p_row = row_of(pt + gridDim.x);
      }
      if (++p_slot == D) p_slot = 0;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int i = 0; i < D - 1; ++i) copy();

  int slot = 0, row = row_of(blockIdx.x);
  auto weight_of = [&](int t) { return t < a.T && lane < k && a.place ? __ldg(a.w + (size_t)t * k + lane) : 1.0f; };
  float weight = weight_of(blockIdx.x);
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const unsigned there = __ballot_sync(0xffffffffu, lane < k ? (unsigned)row < (unsigned)P : lane < sums);
    const int next_row = row_of(t + gridDim.x);
    const float next_weight = weight_of(t + gridDim.x), token_gate = a.gate && a.gate_rows ? __ldg(a.gate + t) : 1.0f;
    float c[V][U] = {};
    const uint8_t* from;
    auto add = [&](int j, const uint8_t* src) {
      const float w = __shfl_sync(0xffffffffu, weight, j);
      if (there >> j & 1)
        each([&](int v, int at) {
          Raw<U, Y> x;
          x.read(reinterpret_cast<const Y*>(src + at * WIDE));
          float f[U];
          x.values(f);
#pragma unroll
          for (int i = 0; i < U; ++i) c[v][i] = fmaf(w, f[i], c[v][i]);
        });
    };
    for (int j = 0; j < steps; ++j) {
      copy();   // into the slot that was read last
      asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
      from = reinterpret_cast<const uint8_t*>(ring) + (size_t)slot * (2 * row_bytes);
      if (++slot == D) slot = 0;
      add(2 * j, from);
      if (j < steps - 1) add(2 * j + 1, from + row_bytes);
    }
    float s = 0.0f;
    if (a.post) {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < U; ++i) s = fmaf(c[v][i], c[v][i], s);
      const float inv = rsqrtf(fmaf(block_sum(s, parts[0]), per, a.eps));
      each([&](int v, int at) {
        const int w = KEEP ? v : 0;
        if (!KEEP) load_post(at, post[w]);
#pragma unroll
        for (int i = 0; i < U; ++i) c[v][i] *= inv * post[w][i];
      });
    }
    s = 0.0f;
    each([&](int v, int at) {
      Raw<U, R> r;
      r.read(reinterpret_cast<const R*>(from + row_bytes + at * WIDE));
      float x[U];
      r.values(x);
      const int w = KEEP ? v : 0;
      if (!KEEP) load_gate(at, gate[w]);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (a.gate) c[v][i] *= a.gate_rows ? token_gate : gate[w][i];
        c[v][i] = fmaf(a.alpha, x[i], c[v][i]);
        s = fmaf(c[v][i], c[v][i], s);
      }
      if (a.h) store(static_cast<R*>(a.h) + (size_t)t * a.N + at, c[v]);
    });
    if (a.z) {
      const float inv = rsqrtf(fmaf(block_sum(s, parts[1]), per, a.eps));
      each([&](int v, int at) {
        float x[U];
        const int w = KEEP ? v : 0;
        if (!KEEP) load_pre(at, pre[w]);
#pragma unroll
        for (int i = 0; i < U; ++i) x[i] = inv * c[v][i] * pre[w][i];
        if (a.z_bf16) store(static_cast<__nv_bfloat16*>(a.z) + (size_t)t * a.N + at, x);
        else store(static_cast<float*>(a.z) + (size_t)t * a.N + at, x);
      });
    }
    if (!(a.post && a.z)) __syncthreads();   // the parts have been read: with two means a token, the other one's barrier says so
    row = next_row;
    weight = next_weight;
  }
}

template <typename Y, typename R, int V, int D, bool KEEP, int THREADS, int BLOCKS>
moe_status launch_stream(const EndArgs& a, int threads, cudaStream_t s) {
  const auto kernel = block_stream_kernel<Y, R, V, D, KEEP, THREADS, BLOCKS>;
  const size_t smem = (size_t)D * 2 * a.N * std::max(sizeof(Y), sizeof(R));
  static bool allowed[64] = {};
  int dev = 0;
  CK(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return fail(MOE_EINVAL, "device %d is out of range", dev);
  if (!allowed[dev]) {
    CK(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 224 * 1024));
    allowed[dev] = true;
  }
  int blocks = 1;
  CK(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&blocks, kernel, threads, smem));
  const int grid = (int)std::min<int64_t>(a.T, (int64_t)operator_sms() * std::max(1, blocks));
  CK(launch_pdl(kernel, dim3(grid), dim3(threads), smem, s, a));
  return MOE_OK;
}

template <typename Y, typename R, int V, int J>
moe_status launch_end(const EndArgs& a, int threads, cudaStream_t s) {
  const int grid = (int)std::min<int64_t>(a.T, (int64_t)operator_sms() * std::max(1, 2048 / threads));
  CK(launch_pdl(block_end_kernel<Y, R, V, J>, dim3(grid), dim3(threads), 0, s, a));
  return MOE_OK;
}

template <typename Y, typename R>
moe_status launch_any(const EndArgs& a, cudaStream_t s) {
  const auto kernel = block_end_any_kernel<Y, R>;
  const int threads = std::min(ANY_THREADS, ((a.N + ANY_VALUES - 1) / ANY_VALUES + 31) / 32 * 32);
  const size_t smem = (size_t)a.N * 4;
  static bool allowed[64] = {};
  int dev = 0;
  CK(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return fail(MOE_EINVAL, "device %d is out of range", dev);
  if (!allowed[dev]) {
    CK(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_WIDTH * 4));
    allowed[dev] = true;
  }
  int blocks = 1;
  CK(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&blocks, kernel, threads, smem));
  const int grid = (int)std::min<int64_t>(a.T, (int64_t)operator_sms() * std::max(1, blocks));
  CK(launch_pdl(kernel, dim3(grid), dim3(threads), smem, s, a));
  return MOE_OK;
}

template <typename Y, typename R>
moe_status run_end(const EndArgs& a, bool wide, cudaStream_t s) {
  const int units = a.N / 8;
  auto threads = [&](int v) { return ((units + v - 1) / v + 31) / 32 * 32; };
  constexpr int H = sizeof(Y) == 2 ? 2 : 1;   // rows on their way: twice as many of half the bytes
  if (wide) {
    if (a.T >= 2 * operator_sms() && (!a.place || a.k <= 30)) {   // a lane a row
      if constexpr (sizeof(Y) + sizeof(R) == 4) {
        // with few rows a token three weights a channel, read each time, hold it up: us, kept in registers / read, 8192 dense rows of 7168
        // with all parts 107 / 118, 16384 of 2048 54 / 63; without post 86 / 79 and 43 / 45; 8192 tokens of 2 rows, N 7168 142 / 108
        if (!a.place && a.post && units <= 1024) return launch_stream<Y, R, 2, 3, true, 512, 1>(a, threads(2), s);
        if (units <= 512) return launch_stream<Y, R, 2, 3, false, 256, 4>(a, threads(2), s);
        if (units <= 1024) return launch_stream<Y, R, 2, 3, false, 512, 2>(a, threads(2), s);
      } else {
        if (units <= 256) return launch_stream<Y, R, 1, 3, true, 256, 2>(a, threads(1), s);
        if (units <= 1024) return launch_stream<Y, R, 2, 3, true, 512, 1>(a, threads(2), s);
      }
    }
    if (units <= 1024) return launch_end<Y, R, 1, 4 * H>(a, threads(1), s);
    if (units <= 2048) return launch_end<Y, R, 2, H>(a, threads(2), s);
    return launch_end<Y, R, 4, 1>(a, threads(4), s);
  }
  return launch_any<Y, R>(a, s);
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
