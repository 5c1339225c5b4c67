// Combine ("MoE Forward", eq. y_n): y_n = sum over the k slots of the weighted expert rows (already
// scaled by w in the down GEMM) + the shared expert's row, accumulated in float32 in slot order and
// then the shared term, rounded once to the output type. When alpha sits on the routed output
// ("MoE Forward", Official code) the slot sum is multiplied by it before the shared term is added.
// Empty slots (inv_row < 0) add nothing. No atomics: the same inputs always give the same bits.
#include <hip/hip_runtime.h>

#include "ops_internal.h"
#include "row_ops.h"

namespace moe {
namespace {

constexpr int MAX_K = 32;

// 8 consecutive elements of a row, as loaded
template <typename T>
struct V8;
template <>
struct V8<uint16_t> {
  uint4 v;
};
template <>
struct V8<float> {
  float4 a, b;
};
__device__ inline V8<uint16_t> load8(const uint16_t* p) {
  const u32x4 v = __builtin_nontemporal_load((const u32x4*)p);  // each expert row is read once
  return V8<uint16_t>{make_uint4(v.x, v.y, v.z, v.w)};
}
__device__ inline V8<float> load8(const float* p) { return V8<float>{*(const float4*)p, *(const float4*)(p + 4)}; }
__device__ inline void add8(float* acc, const V8<uint16_t>& x) {
  const uint32_t w[4] = {x.v.x, x.v.y, x.v.z, x.v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc[2 * i] += __uint_as_float(w[i] << 16);
    acc[2 * i + 1] += __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ inline void add8(float* acc, const V8<float>& x) {
  acc[0] += x.a.x; acc[1] += x.a.y; acc[2] += x.a.z; acc[3] += x.a.w;
  acc[4] += x.b.x; acc[5] += x.b.y; acc[6] += x.b.z; acc[7] += x.b.w;
}
template <typename T>
__device__ inline void add8(float* acc, const T* p) {
  add8(acc, load8(p));
}
__device__ inline void store8(uint16_t* p, const float* acc) {
  uint4 v;
  v.x = (uint32_t)bf16_rne(acc[0]) | ((uint32_t)bf16_rne(acc[1]) << 16);
  v.y = (uint32_t)bf16_rne(acc[2]) | ((uint32_t)bf16_rne(acc[3]) << 16);
  v.z = (uint32_t)bf16_rne(acc[4]) | ((uint32_t)bf16_rne(acc[5]) << 16);
  v.w = (uint32_t)bf16_rne(acc[6]) | ((uint32_t)bf16_rne(acc[7]) << 16);
  const u32x4 w = {v.x, v.y, v.z, v.w};
  __builtin_nontemporal_store(w, (u32x4*)p);
}
__device__ inline void store8(float* p, const float* acc) {
  *(float4*)p = make_float4(acc[0], acc[1], acc[2], acc[3]);
  *(float4*)(p + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
}

// One block per token; each thread owns 8 consecutive features per pass (the launch sizes the block so
// that a row of up to 8192 features takes one pass).
template <typename T>
__global__ __launch_bounds__(1024) void combine_kernel(const T* __restrict__ Y, const T* __restrict__ Ysh,
                                                      const int32_t* __restrict__ inv_row, int k, int D,
                                                      float alpha_out, T* __restrict__ y) {
  __shared__ int rows[MAX_K];
  const int64_t n = blockIdx.x;
  if (threadIdx.x < k) rows[threadIdx.x] = inv_row[n * k + threadIdx.x];
  __syncthreads();
  for (int c = threadIdx.x * 8; c < D; c += blockDim.x * 8) {
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    V8<T> vsh;
    if (Ysh) vsh = load8(Ysh + n * D + c);  // in flight with the slot rows
    // slots in groups of 8: the group's row loads are all issued before the first add (a loop of
    // load-then-add waited out one memory latency per slot); the adds keep slot order
    for (int s0 = 0; s0 < k; s0 += 8) {
      V8<T> v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int r = s0 + u < k ? rows[s0 + u] : -1;
        if (r >= 0) v[u] = load8(Y + (int64_t)r * D + c);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (s0 + u < k && rows[s0 + u] >= 0) add8(acc, v[u]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = __fmul_rn(acc[i], alpha_out);  // exact when alpha_out == 1
    if (Ysh) add8(acc, vsh);
    store8(y + n * D + c, acc);
  }
}

// moe_combine: the same sum for rows that are not yet weighted, y = alpha sum_s w_s rows[inv_s] + shared. Bound by
// HBM: 1,000 tokens x 8 rows of 4,096 float32, 164 MB, 26 us (30 with non-temporal loads, which pass by the
// last-level cache where the product before left the rows).
// inv_row comes from the caller: an entry outside [0, R) is an empty slot.
template <typename T>
__global__ __launch_bounds__(1024) void combine_rows_kernel(const T* __restrict__ rows_in, int64_t R,
                                                           const int32_t* __restrict__ inv_row,
                                                           const float* __restrict__ w, const T* shared,
                                                           int k, int D, float alpha, T* y) {
  __shared__ int rows[MAX_K];
  __shared__ float wt[MAX_K];
  const int64_t n = blockIdx.x;
  if (threadIdx.x < k) {
    const int r = inv_row[n * k + threadIdx.x];
    rows[threadIdx.x] = r >= 0 && r < R ? r : -1;
    wt[threadIdx.x] = w ? w[n * k + threadIdx.x] : 1.0f;
  }
  __syncthreads();
  for (int c = threadIdx.x * 8; c < D; c += blockDim.x * 8) {
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    Raw8<T> vsh;
    if (shared) vsh = raw_load8(shared + n * D + c);
    for (int s0 = 0; s0 < k; s0 += 8) {  // as above: a group's loads first, the sums in slot order
      Raw8<T> v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int r = s0 + u < k ? rows[s0 + u] : -1;
        if (r >= 0) v[u] = raw_load8(rows_in + (int64_t)r * D + c);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (s0 + u < k && rows[s0 + u] >= 0) {
          float f[8];
          widen8(v[u], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] += wt[s0 + u] * f[i];
        }
    }
    float sh[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (shared) widen8(vsh, sh);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = alpha * acc[i] + sh[i];
    raw_store8(y + n * D + c, acc);
  }
}

// Gradients of moe_combine: drows[inv_s] = alpha w_s dy and dw_s = alpha <dy, rows[inv_s]>, one block per
// token. A token's dy stays in registers over its slots (rows of up to 8192 features); the slots' dot
// products are summed over the block together, eight at a time. Every row is written by the one slot
// that names it, so nothing is accumulated in memory. Bound by HBM: 4,096 tokens x 8 rows of 4,096 bf16, 571 MB,
// 106 us.
template <typename T>
__global__ __launch_bounds__(1024) void combine_rows_backward_kernel(const T* __restrict__ dy,
                                                                    const T* __restrict__ rows_in, int64_t R,
                                                                    const int32_t* __restrict__ inv_row,
                                                                    const float* __restrict__ w, int k, int D,
                                                                    float alpha, T* __restrict__ drows,
                                                                    float* __restrict__ dw) {
  __shared__ int rows[MAX_K];
  __shared__ float wt[MAX_K];
  __shared__ float buf[2][16][8];
  const int64_t n = blockIdx.x;
  const int waves = blockDim.x >> 6;
  if (threadIdx.x < k) {
    const int r = inv_row[n * k + threadIdx.x];
    rows[threadIdx.x] = r >= 0 && r < R ? r : -1;
    wt[threadIdx.x] = alpha * (w ? w[n * k + threadIdx.x] : 1.0f);
  }
  __syncthreads();
  for (int s0 = 0; s0 < k; s0 += 8) {
    float dot[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int c = threadIdx.x * 8; c < D; c += blockDim.x * 8) {
      Raw8<T> v[8];
      if (dw) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int r = s0 + u < k ? rows[s0 + u] : -1;
          if (r >= 0) v[u] = raw_load8(rows_in + (int64_t)r * D + c);
        }
      }
      float g[8];
      widen8(raw_load8(dy + n * D + c), g);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int r = s0 + u < k ? rows[s0 + u] : -1;
        if (r < 0) continue;
        float f[8];
        if (dw) {
          widen8(v[u], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) dot[u] += g[i] * f[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = wt[s0 + u] * g[i];
        raw_store8(drows + (int64_t)r * D + c, f);
      }
    }
    if (!dw) continue;
    block_sums<8>(dot, buf[(s0 >> 3) & 1], waves);
    if (threadIdx.x == 0) {
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (s0 + u < k) dw[n * k + s0 + u] = rows[s0 + u] >= 0 ? alpha * dot[u] : 0.f;
    }
  }
}

}  // namespace

int combine_threads(int D) {
  const int threads = (D / 8 + 63) / 64 * 64;
  return threads > 1024 ? 1024 : threads;
}

hipError_t launch_combine_rows(int dtype, const void* rows, int64_t R, const int32_t* inv_row, const float* w,
                               const void* shared, int64_t N, int k, int D, float alpha, void* y, hipStream_t s) {
  const dim3 grid((unsigned)N), block(combine_threads(D));
  if (dtype == MOE_F32)
    hipLaunchKernelGGL(combine_rows_kernel<float>, grid, block, 0, s, (const float*)rows, R, inv_row, w,
                       (const float*)shared, k, D, alpha, (float*)y);
  else
    hipLaunchKernelGGL(combine_rows_kernel<uint16_t>, grid, block, 0, s, (const uint16_t*)rows, R, inv_row, w,
                       (const uint16_t*)shared, k, D, alpha, (uint16_t*)y);
  return hipGetLastError();
}

hipError_t launch_combine_rows_backward(int dtype, const void* dy, const void* rows, int64_t R,
                                        const int32_t* inv_row, const float* w, int64_t N, int k, int D, float alpha,
                                        void* drows, float* dw, hipStream_t s) {
  const dim3 grid((unsigned)N), block(combine_threads(D));
  if (dtype == MOE_F32)
    hipLaunchKernelGGL(combine_rows_backward_kernel<float>, grid, block, 0, s, (const float*)dy, (const float*)rows, R,
                       inv_row, w, k, D, alpha, (float*)drows, dw);
  else
    hipLaunchKernelGGL(combine_rows_backward_kernel<uint16_t>, grid, block, 0, s, (const uint16_t*)dy,
                       (const uint16_t*)rows, R, inv_row, w, k, D, alpha, (uint16_t*)drows, dw);
  return hipGetLastError();
}

hipError_t launch_combine(int dtype, const void* Y, const void* Ysh, const int32_t* inv_row, int64_t N, int k, int D,
                          float alpha_out, void* y, hipStream_t s) {
  // one thread per 8 features, whole waves, at most 1024 (D is a multiple of 64)
  int threads = (D / 8 + 63) / 64 * 64;
  if (threads > 1024) threads = 1024;
  if (dtype == MOE_F32)
    hipLaunchKernelGGL(combine_kernel<float>, dim3((unsigned)N), dim3(threads), 0, s, (const float*)Y,
                       (const float*)Ysh, inv_row, k, D, alpha_out, (float*)y);
  else
    hipLaunchKernelGGL(combine_kernel<uint16_t>, dim3((unsigned)N), dim3(threads), 0, s, (const uint16_t*)Y,
                       (const uint16_t*)Ysh, inv_row, k, D, alpha_out, (uint16_t*)y);
  return hipGetLastError();
}

}  // namespace moe
