// Products grouped by expert, and their gradients, over rows sorted by expert (the order moe_dispatch
// gives). With e(r) the expert whose range [offsets[e], offsets[e + 1]) holds row r:
//
//   fwd    y[r]  = W[e(r)] x[src(r)]                       (reduction over the input features)
//   dgrad  dx[r] = W[e(r)]^T dy[r]                         (reduction over the output features)
//   wgrad  dW[e] = sum over the expert's rows of dy[r] x[src(r)]^T
//
// W is [E, M, K] row-major, as the layer's own matrices. The tile lists (fwd, dgrad) come from the device
// (launch_offset_lists); wgrad needs none, its tiles are those of dW.
#include <hip/hip_runtime.h>

#include "moe_internal.h"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ inline void load8f(const float* p, float* f) {
  const f32x4 a = *(const f32x4*)p, b = *(const f32x4*)(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = a[i];
    f[4 + i] = b[i];
  }
}
__device__ inline void load8f(const uint16_t* p, float* f) {
  const uint4 v = *(const uint4*)p;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ inline void store1(float* p, float v) { *p = v; }
__device__ inline void store1(uint16_t* p, float v) { *p = __builtin_bit_cast(uint16_t, (__bf16)v); }

// 128 x 128 tile of C[i, j] = sum_t A(i, t) B(j, t) in float32: both operands go through LDS as
// [t][i] / [t][j] (16 t per step), four waves of 64 x 64 as 4 x 4 tiles of v_mfma_f32_16x16x4_f32
// (A: row lane % 16, k lane / 16; C: column lane % 16, rows 4 (lane / 16) + r).
//   fwd:   i = row, j = output feature, t = input feature;   both operands contiguous in t
//   dgrad: i = row, j = input feature,  t = output feature;  B contiguous in j
//   wgrad: i = output feature, j = input feature, t = row;   both contiguous in i / j
template <typename T, int MODE>
__global__ __launch_bounds__(256) void grouped_any(GradArgs a, int col_tiles) {
  constexpr bool A_T = MODE == GM_WGRAD;              // A contiguous in i
  constexpr bool B_T = MODE != GM_FWD;                // B contiguous in j
  constexpr int BT = 16, PITCH = 128 + 4;
  __shared__ float sa[BT][PITCH], sb[BT][PITCH];
  const int M = a.M, K = a.K;
  int64_t row0;   // first grouped row of the tile (fwd, dgrad) or of the expert (wgrad)
  int expert, rows, i0 = 0, j0;
  if (MODE == GM_WGRAD) {
    const int mt = (M + 127) / 128;
    const int64_t b = blockIdx.x;
    j0 = (int)(b % col_tiles) * 128;
    i0 = (int)(b / col_tiles % mt) * 128;
    expert = (int)(b / col_tiles / mt);
    const int64_t lo = min(max((int64_t)a.offsets[expert], (int64_t)0), a.R);
    const int64_t hi = min(max((int64_t)a.offsets[expert + 1], lo), a.R);
    row0 = lo;
    rows = (int)(hi - lo);
  } else {
    const int64_t L = xcd_logical_block((int64_t)*a.n_tiles * col_tiles);
    if (L < 0) return;
    const Tile tile = a.tiles[L / col_tiles];
    j0 = (int)(L % col_tiles) * 128;
    row0 = tile.row_start;
    rows = tile.rows;
    expert = tile.expert;
    if (rows <= 0) return;
  }
  const int ni = MODE == GM_WGRAD ? M : rows, nj = MODE == GM_FWD ? M : K;
  const int nt = MODE == GM_FWD ? K : MODE == GM_DGRAD ? M : rows;
  const T* A = (const T*)a.a;
  const T* B = (const T*)a.b;
  const int64_t wbase = (int64_t)expert * M * K;

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wi = (wave >> 1) * 64, wj = (wave & 1) * 64;
  // this thread's eight elements of each operand per step
  const int ai = A_T ? (tid & 15) * 8 : tid >> 1, at = A_T ? tid >> 4 : (tid & 1) * 8;
  const int bj = B_T ? (tid & 15) * 8 : tid >> 1, bt = B_T ? tid >> 4 : (tid & 1) * 8;
  auto src = [&](int64_t r) -> int64_t { return a.src_row ? a.src_row[r] : r; };
  int64_t a_row = 0;
  if (MODE == GM_FWD && ai < rows) a_row = src(row0 + ai);

  f32x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  float ra[8], rb[8];
  auto load = [&](int t0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) ra[i] = rb[i] = 0.f;
    if (MODE == GM_FWD) {
      if (ai < rows) load8f(A + a_row * K + t0 + at, ra);
      if (j0 + bj < nj) load8f(B + wbase + (int64_t)(j0 + bj) * K + t0 + bt, rb);
    } else if (MODE == GM_DGRAD) {
      if (ai < rows) load8f(A + (row0 + ai) * M + t0 + at, ra);
      if (j0 + bj < nj) load8f(B + wbase + (int64_t)(t0 + bt) * K + j0 + bj, rb);
    } else {
      if (t0 + at < nt && i0 + ai < ni) load8f(A + (row0 + t0 + at) * M + i0 + ai, ra);
      if (t0 + bt < nt && j0 + bj < nj) load8f(B + src(row0 + t0 + bt) * K + j0 + bj, rb);
    }
  };
  auto put = [&](float (*s)[PITCH], bool contiguous_row, int i, int t, const float* r) {
    if (contiguous_row) {
      *(f32x4*)&s[t][i] = f32x4{r[0], r[1], r[2], r[3]};
      *(f32x4*)&s[t][i + 4] = f32x4{r[4], r[5], r[6], r[7]};
    } else {
#pragma unroll
      for (int u = 0; u < 8; ++u) s[t + u][i] = r[u];
    }
  };
  if (nt > 0) load(0);
  for (int t0 = 0; t0 < nt; t0 += BT) {
    __syncthreads();
    put(sa, A_T, ai, at, ra);
    put(sb, B_T, bj, bt, rb);
    __syncthreads();
    if (t0 + BT < nt) load(t0 + BT);
#pragma unroll
    for (int k = 0; k < BT; k += 4) {
      float av[4], bv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) av[i] = sa[k + (lane >> 4)][wi + 16 * i + (lane & 15)];
#pragma unroll
      for (int j = 0; j < 4; ++j) bv[j] = sb[k + (lane >> 4)][wj + 16 * j + (lane & 15)];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(av[i], bv[j], acc[i][j], 0, 0, 0);
    }
  }
  T* out = (T*)a.out;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int ii = i0 + wi + 16 * i + 4 * (lane >> 4) + q;
      if (ii >= ni) continue;
      const int64_t base = MODE == GM_WGRAD ? wbase + (int64_t)ii * K : (row0 + ii) * (int64_t)nj;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int jj = j0 + wj + 16 * j + (lane & 15);
        if (jj < nj) store1(out + base + jj, acc[i][j][q]);
      }
    }
}

template <typename T>
hipError_t launch_any(GroupedMode mode, const GradArgs& a, int64_t max_tile_count, hipStream_t s) {
  const int cols = ((mode == GM_FWD ? a.M : a.K) + 127) / 128;
  const int64_t tiles = mode == GM_WGRAD ? (int64_t)a.E * ((a.M + 127) / 128) : max_tile_count;
  int64_t blocks = tiles * cols;
  if (mode != GM_WGRAD) blocks = (blocks + 7) / 8 * 8;
  if (blocks == 0) return hipSuccess;
  if (blocks >= (int64_t)1 << 31) return hipErrorInvalidValue;
  const dim3 grid((unsigned)blocks), block(256);
  if (mode == GM_FWD)
    hipLaunchKernelGGL((grouped_any<T, GM_FWD>), grid, block, 0, s, a, cols);
  else if (mode == GM_DGRAD)
    hipLaunchKernelGGL((grouped_any<T, GM_DGRAD>), grid, block, 0, s, a, cols);
  else
    hipLaunchKernelGGL((grouped_any<T, GM_WGRAD>), grid, block, 0, s, a, cols);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_bf16(GroupedMode mode, const GradArgs& a, int64_t max_tile_count, hipStream_t s) {
  return launch_any<uint16_t>(mode, a, max_tile_count, s);
}
hipError_t launch_grouped_f32(GroupedMode mode, const GradArgs& a, int64_t max_tile_count, hipStream_t s) {
  return launch_any<float>(mode, a, max_tile_count, s);
}

}  // namespace moe
