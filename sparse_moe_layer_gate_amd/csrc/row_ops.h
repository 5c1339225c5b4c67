// Row helpers shared by the kernels that stream whole rows (block norms, combine): eight consecutive
// elements of a row per thread, and sums over a thread block in a fixed order.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_internal.h"

namespace moe {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4v __attribute__((ext_vector_type(4)));

// Eight consecutive elements as loaded (bf16: 16 bytes, float32: 32 bytes).
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  u32x4 v;
};
template <>
struct Raw8<float> {
  f32x4v a, b;
};

__device__ inline Raw8<uint16_t> raw_load8(const uint16_t* p) { return Raw8<uint16_t>{*(const u32x4*)p}; }
__device__ inline Raw8<float> raw_load8(const float* p) {
  return Raw8<float>{*(const f32x4v*)p, *((const f32x4v*)p + 1)};
}
__device__ inline void widen8(const Raw8<uint16_t>& r, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(r.v[i] << 16);
    f[2 * i + 1] = __uint_as_float(r.v[i] & 0xffff0000u);
  }
}
__device__ inline void widen8(const Raw8<float>& r, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = r.a[i];
    f[4 + i] = r.b[i];
  }
}
// float32 -> bfloat16 bits, to nearest even, infinities and NaN kept (two per instruction)
__device__ inline uint32_t bf16_pair(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  bf16x2 v;
  v[0] = (__bf16)lo;
  v[1] = (__bf16)hi;
  return __builtin_bit_cast(uint32_t, v);
}
// NT: non-temporal, for bytes that nothing reads soon.
template <bool NT = true>
__device__ inline void raw_store8(uint16_t* p, const float* f) {
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = bf16_pair(f[2 * i], f[2 * i + 1]);
  if (NT)
    __builtin_nontemporal_store(v, (u32x4*)p);
  else
    *(u32x4*)p = v;
}
template <bool NT = true>
__device__ inline void raw_store8(float* p, const float* f) {
  f32x4v a, b;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = f[i];
    b[i] = f[4 + i];
  }
  if (NT) {
    __builtin_nontemporal_store(a, (f32x4v*)p);
    __builtin_nontemporal_store(b, (f32x4v*)p + 1);
  } else {
    *(f32x4v*)p = a;
    *((f32x4v*)p + 1) = b;
  }
}

__device__ inline float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

// Sums of NV values over the block, the same in every thread: butterflies in each wave, then the waves'
// totals in wave order. `buf` holds NV floats per wave (at most 16 waves); a caller alternates between two
// buffers, so that one barrier per call is enough: a buffer is written again only after the barrier of
// the call in between, which every wave reaches after its reads.
template <int NV>
__device__ inline void block_sums(float (&v)[NV], float (*buf)[NV], int waves) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = wave_sum(v[i]);
  if (waves == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) buf[wave][i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = 0.f;
  for (int w = 0; w < waves; ++w) {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] += buf[w][i];
  }
}

}  // namespace moe
