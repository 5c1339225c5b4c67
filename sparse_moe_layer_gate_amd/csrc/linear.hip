// Dense linear maps with bias, activation and residual in the epilogue:
//
//   z = x W^T + bias      y = act(z) + residual
//
// Both operands are contiguous in the reduction index (W is [out, in] row-major). Forms, picked by linear_plan:
//  - linear_w8 (bfloat16, many rows): 256 x 256 tiles on the eight-wave K loop of the expert GEMMs (gemm_w8.h), a
//    static walk over the tiles, one block per CU;
//  - linear_tile (both types): 32 to 256 rows x 128 columns, the reduction split over blocks where the tiles alone
//    would not fill the CUs; linear_join then adds the parts in order and runs the epilogue.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "activation.h"
#include "gemm_w8.h"
#include "ops_internal.h"
#include "row_ops.h"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <typename T>
struct LinArgs {
  const T *x, *w, *bias, *residual;
  T *z, *y;
  float* part;  // [splits][R][M] when splits > 1
  int64_t R;
  int M, K, act, splits;
  int64_t row_tiles;
  int col_tiles;
};

// Loads and stores of N = 4 or 8 consecutive values of a row, in float32 registers.
template <int N>
__device__ inline void load_row(const float* p, float* f) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const f32x4 v = *(const f32x4*)(p + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) f[i + j] = v[j];
  }
}
template <int N>
__device__ inline void load_row(const uint16_t* p, float* f) {
  typedef uint32_t words __attribute__((ext_vector_type(N / 2)));
  const words v = *(const words*)p;
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
  }
}
template <int N>
__device__ inline void store_row(float* p, const float* f) {
#pragma unroll
  for (int i = 0; i < N; i += 4) *(f32x4*)(p + i) = f32x4{f[i], f[i + 1], f[i + 2], f[i + 3]};
}
template <int N>
__device__ inline void store_row(uint16_t* p, const float* f) {
  typedef uint32_t words __attribute__((ext_vector_type(N / 2)));
  words v;
#pragma unroll
  for (int i = 0; i < N / 2; ++i) v[i] = bf16_pair(f[2 * i], f[2 * i + 1]);
  *(words*)p = v;
}

// bias, z, activation, residual and y of N consecutive columns of one row; v holds the sums.
template <int N, typename T>
__device__ inline void epilogue(const LinArgs<T>& a, int64_t row, int col, float* v, const float* bias) {
  const int64_t at = row * a.M + col;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] += bias[i];
  if (a.z) store_row<N>(a.z + at, v);
  act_apply<std::is_same<T, uint16_t>::value, N>(a.act, v);
  if (a.residual) {
    float r[N];
    load_row<N>(a.residual + at, r);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += r[i];
  }
  store_row<N>(a.y + at, v);
}
template <int N, typename T>
__device__ inline void load_bias(const LinArgs<T>& a, int col, float* b) {
#pragma unroll
  for (int i = 0; i < N; ++i) b[i] = 0.f;
  if (a.bias) load_row<N>(a.bias + col, b);
}

// ---- tiles of 32 to 256 rows x 128 columns ----
//
// A stage of the ring holds 128 bytes of every row of x and of W that the tile covers (whole lines per load), copied
// global -> LDS by direct loads, chunk-swizzled as in gemm_w8.h. Each wave multiplies a share of TM x TN tiles of
// 16 x 16: W rows are the first operand, so that a lane ends up with four consecutive output columns of one row. A
// lane of both operands holds the 16 bytes of chunk lane / 16 of its row: eight k of v_mfma_f32_16x16x32_bf16, or four k
// that four steps of v_mfma_f32_16x16x4_f32 take one by one (which k of a chunk meet in one step does not matter as
// long as both operands agree).
// One barrier per step: it follows the wait for the step's own loads, and the stage that is refilled behind it was
// read in the step before.
template <typename T, int BM_, int WM_, int WN_, int S_>
struct LinTile {
  static constexpr int BM = BM_, BN = 128, WM = WM_, WN = WN_, S = S_;
  static constexpr int NW = WM * WN;
  static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
  static constexpr int BK = 128 / (int)sizeof(T);  // elements of a 128-byte row
  static constexpr int NA = BM / 8 / NW, NB = BN / 8 / NW;  // direct loads per wave and step (8 rows each)
  static constexpr int STAGE = (BM + BN) * 128;
  static_assert(NA * 8 * NW == BM && NB * 8 * NW == BN, "whole loads per wave");
  static_assert(S * STAGE <= 160 * 1024, "LDS");
  __device__ static int swz(int r) {
    r &= 31;
    return (r ^ (r >> 3)) & 7;
  }
};

template <typename T, int BM, int WM, int WN, int S>
__global__ __launch_bounds__(64 * WM * WN) void linear_tile(LinArgs<T> a) {
  using L = LinTile<T, BM, WM, WN, S>;
  constexpr int TM = L::TM, TN = L::TN, NW = L::NW, NA = L::NA, NB = L::NB, PER = NA + NB;
  __shared__ __attribute__((aligned(1024))) char lds[S * L::STAGE];
  // splits outermost (an XCD's run of blocks then shares one part of x in its L2), row tiles innermost (blocks on the
  // same rows of W run together)
  const int64_t id = xcd_logical_block(gridDim.x);
  const int64_t rt = id % a.row_tiles, rest = id / a.row_tiles;
  const int ct = (int)(rest % a.col_tiles), split = (int)(rest / a.col_tiles);
  const int64_t row0 = rt * BM;
  const int col0 = ct * L::BN;
  const int rows = (int)min((int64_t)BM, a.R - row0);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;

  // rows past the end repeat the last one (never stored); offsets are from the tile's first row and stay below 2^32
  const __amdgpu_buffer_rsrc_t ra =
      __builtin_amdgcn_make_buffer_rsrc((void*)(a.x + row0 * a.K), (short)0, -1, kRawBufferWord3);
  const __amdgpu_buffer_rsrc_t rb =
      __builtin_amdgcn_make_buffer_rsrc((void*)(a.w + (int64_t)col0 * a.K), (short)0, -1, kRawBufferWord3);
  uint32_t oa[NA], ob[NB];
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    const int r = (wave + NW * i) * 8 + (lane >> 3), c = (lane & 7) ^ L::swz(r);
    oa[i] = (uint32_t)min(r, rows - 1) * (uint32_t)(a.K * (int)sizeof(T)) + 16 * c;
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int r = (wave + NW * i) * 8 + (lane >> 3), c = (lane & 7) ^ L::swz(r);
    ob[i] = (uint32_t)min(r, a.M - 1 - col0) * (uint32_t)(a.K * (int)sizeof(T)) + 16 * c;
  }
  const int nk_all = a.K / L::BK;
  const int k0 = (int)((int64_t)nk_all * split / a.splits), nk = (int)((int64_t)nk_all * (split + 1) / a.splits) - k0;

  auto issue = [&](int t) {
    char* st = lds + (t % S) * L::STAGE;
    const int off = (k0 + t) * 128;
#pragma unroll
    for (int i = 0; i < NA; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(st + (wave + NW * i) * 1024), 16, (int)oa[i], off, 0, 0);
#pragma unroll
    for (int i = 0; i < NB; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(st + BM * 128 + (wave + NW * i) * 1024), 16, (int)ob[i],
                                               off, 0, 0);
  };
  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int r16 = lane & 15, kq = lane >> 4;
  const bool live = wm * TM * 16 < rows;  // this wave has rows at all
  int arow[TM], brow[TN], asw[TM], bsw[TN];
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int r = (wm * TM + i) * 16 + r16;
    arow[i] = r * 128;
    asw[i] = L::swz(r);
  }
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int r = (wn * TN + j) * 16 + r16;
    brow[j] = BM * 128 + r * 128;
    bsw[j] = L::swz(r);
  }
  auto step = [&](int t) {
    const char* st = lds + (t % S) * L::STAGE;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = 4 * h + kq;
      if constexpr (std::is_same<T, uint16_t>::value) {
        bf16x8 av[TM], bv[TN];
#pragma unroll
        for (int i = 0; i < TM; ++i) av[i] = *(const bf16x8*)(st + arow[i] + 16 * (c ^ asw[i]));
#pragma unroll
        for (int j = 0; j < TN; ++j) bv[j] = *(const bf16x8*)(st + brow[j] + 16 * (c ^ bsw[j]));
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv[j], av[i], acc[i][j], 0, 0, 0);
      } else {
        f32x4 av[TM], bv[TN];
#pragma unroll
        for (int i = 0; i < TM; ++i) av[i] = *(const f32x4*)(st + arow[i] + 16 * (c ^ asw[i]));
#pragma unroll
        for (int j = 0; j < TN; ++j) bv[j] = *(const f32x4*)(st + brow[j] + 16 * (c ^ bsw[j]));
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(bv[j][u], av[i][u], acc[i][j], 0, 0, 0);
      }
    }
  };
#pragma unroll
  for (int t = 0; t < S - 1; ++t)
    if (t < nk) issue(t);
  for (int t = 0; t < nk; ++t) {
    // step t has landed: at most the S - 2 steps behind it are still in flight
    if (t + S - 1 <= nk)
      wait_vmcnt<(S - 2) * PER>();
    else
      wait_vmcnt<0>();
    wait_lgkm0();
    bare_barrier();
    if (t + S - 1 < nk) issue(t + S - 1);
    if (live) step(t);
  }

  const bool whole = a.splits == 1;
  float* part = a.part + (int64_t)split * a.R * a.M;
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int col = col0 + (wn * TN + j) * 16 + 4 * kq;
    if (col >= a.M) continue;
    float bias[4];
    if (whole) load_bias<4>(a, col, bias);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int r = (wm * TM + i) * 16 + r16;
      if (r >= rows) continue;
      float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
      if (whole)
        epilogue<4>(a, row0 + r, col, v, bias);
      else
        store_row<4>(part + (row0 + r) * a.M + col, v);
    }
  }
}

// The parts of a split reduction in order, then the epilogue: eight columns per thread.
template <typename T>
__global__ __launch_bounds__(256) void linear_join(LinArgs<T> a) {
  const int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x, per_row = a.M / 8;
  if (p >= a.R * per_row) return;
  const int64_t row = p / per_row;
  const int col = (int)(p % per_row) * 8;
  const float* src = a.part + row * a.M + col;
  const int64_t stride = a.R * a.M;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, bias[8];
  load_bias<8>(a, col, bias);
  int s = 0;
  for (; s + 4 <= a.splits; s += 4) {
    float q[4][8];
#pragma unroll
    for (int u = 0; u < 4; ++u) load_row<8>(src + (s + u) * stride, q[u]);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += q[u][i];
  }
  for (; s < a.splits; ++s) {
    float q[8];
    load_row<8>(src + s * stride, q);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += q[i];
  }
  epilogue<8>(a, row, col, v, bias);
}

// ---- 256 x 256 tiles ----
//
// The tiles cost the same but for the last row tile's, so each block walks them without claiming: per XCD a run of
// logical ids of nearly equal length (xcd_logical_block), its blocks taking every 32nd. The epilogue goes through LDS
// in float32, 32 rows of a wave's 64 at a time, so that a lane holds eight consecutive columns of a row: bias, z,
// activation and residual are applied there, with whole 16-byte loads and stores, and y is rounded once.
constexpr int kStagePitch = 128 + 8;  // floats: rows four apart, which one store writes together, lie 32 banks apart

__global__ __launch_bounds__(512, 1) void linear_w8(LinArgs<uint16_t> a) {
  using T = Wave8Tile<false>;
  __shared__ __attribute__((aligned(1024))) char lds[T::RING];
  static_assert(8 * 32 * kStagePitch * 4 <= T::RING, "staged outputs fit the ring");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int grp = wave >> 2, q = wave & 3, m0 = grp * 128 + (q & 1) * 64, wn = q >> 1;
  const int64_t tiles = a.row_tiles * a.col_tiles;
  const int64_t xq = tiles >> 3, xr = tiles & 7, xcd = blockIdx.x & 7;
  const int64_t start = xcd * xq + min(xcd, xr), len = xq + (xcd < xr ? 1 : 0);
  for (int64_t id = blockIdx.x >> 3; id < len; id += gridDim.x >> 3) {
    int64_t rt;
    int ct;
    raster<4, 8>(start + id, a.col_tiles, a.row_tiles, rt, ct);
    const int64_t row0 = rt * 256;
    const int col0 = ct * 256, rows = (int)min((int64_t)256, a.R - row0);
    const __amdgpu_buffer_rsrc_t ra =
        __builtin_amdgcn_make_buffer_rsrc((void*)(a.x + row0 * a.K), (short)0, -1, kRawBufferWord3);
    const __amdgpu_buffer_rsrc_t rb =
        __builtin_amdgcn_make_buffer_rsrc((void*)(a.w + (int64_t)col0 * a.K), (short)0, -1, kRawBufferWord3);
    uint32_t oa[4], ob[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = (i * 4 + q) * 64 + lane, r = grp * 128 + (p >> 3), c = (p & 7) ^ T::swz(r);
      oa[i] = ((uint32_t)min(r, rows - 1) * (uint32_t)a.K + 8 * c) * 2;
      ob[i] = ((uint32_t)min(r, a.M - 1 - col0) * (uint32_t)a.K + 8 * c) * 2;
    }
    const int na = max(0, min(4, (rows - grp * 128 - 8 * q + 31) / 32));
    f32x16 acc[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    const int nk = a.K / T::BK;
    const int mi = max(0, min(2, (rows - m0 + 31) / 32));
    __syncthreads();  // the previous tile's staged outputs have been read
    if (mi == 2)
      wave8_loop<false, 2>(lds, ra, oa, na, rb, ob, acc, nk, grp, q, lane, m0, wn);
    else if (mi == 1)
      wave8_loop<false, 1>(lds, ra, oa, na, rb, ob, acc, nk, grp, q, lane, m0, wn);
    else
      wave8_loop<false, 0>(lds, ra, oa, na, rb, ob, acc, nk, grp, q, lane, m0, wn);

    // each wave in its own part of the ring (every wave has passed the loop's last barrier, behind the last read)
    float* stage = (float*)lds + wave * (32 * kStagePitch);
    const int ch = lane & 15, col = col0 + wn * 128 + ch * 8;
    const bool in = col < a.M;
    float bias[8];
    if (in) load_bias<8>(a, col, bias);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (i >= mi) continue;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
#pragma unroll
        for (int j = 0; j < 4; ++j) stage[row * kStagePitch + j * 32 + (lane & 31)] = acc[i][j][r];
      }
      __builtin_amdgcn_wave_barrier();
      const int here = min(32, rows - m0 - i * 32);
      for (int row = lane >> 4; row < here; row += 4) {
        float v[8];
        load_row<8>(stage + row * kStagePitch + ch * 8, v);
        if (in) epilogue<8>(a, row0 + m0 + i * 32 + row, col, v, bias);
      }
      __builtin_amdgcn_wave_barrier();
    }
  }
}

// Blocks of linear_tile: rows per tile and the parts of the reduction.
template <typename T, int BM, int WM, int WN, int S>
hipError_t run_tile(const LinArgs<T>& a, hipStream_t s) {
  const int64_t blocks = a.row_tiles * a.col_tiles * a.splits;
  hipLaunchKernelGGL((linear_tile<T, BM, WM, WN, S>), dim3((unsigned)blocks), dim3(64 * WM * WN), 0, s, a);
  return hipGetLastError();
}

template <typename T>
hipError_t linear_t(const LinearCall& c, const LinearPlan& p, hipStream_t s) {
  LinArgs<T> a{};
  a.x = (const T*)c.x;
  a.w = (const T*)c.w;
  a.bias = (const T*)c.bias;
  a.residual = (const T*)c.residual;
  a.z = (T*)c.z;
  a.y = (T*)c.y;
  a.part = c.part;
  a.R = c.R;
  a.M = c.out;
  a.K = c.in;
  a.act = c.act;
  a.splits = p.splits;
  a.row_tiles = (c.R + p.bm - 1) / p.bm;
  a.col_tiles = (c.out + p.bn - 1) / p.bn;
  hipError_t e = hipErrorInvalidValue;
  if constexpr (std::is_same<T, uint16_t>::value) {
    if (p.bn == 256) {
      const int64_t grid = std::min((a.row_tiles * a.col_tiles + 7) / 8 * 8, persistent_grid());
      hipLaunchKernelGGL(linear_w8, dim3((unsigned)grid), dim3(512), 0, s, a);
      return hipGetLastError();
    }
    if (p.bm == 256) e = run_tile<T, 256, 4, 2, 3>(a, s);
  }
  if (p.bm == 32) e = run_tile<T, 32, 1, 4, 4>(a, s);
  if (p.bm == 64) e = run_tile<T, 64, 2, 2, 3>(a, s);
  if (p.bm == 128) e = run_tile<T, 128, 2, 4, 4>(a, s);
  if (e != hipSuccess || p.splits == 1) return e;
  hipLaunchKernelGGL(linear_join<T>, dim3((unsigned)linear_join_blocks(c.R, c.out)), dim3(256), 0, s, a);
  return hipGetLastError();
}

// ---- the gradients of the epilogue ----
//
// Eight columns per thread; the four waves of a block take rows in turn of a run of kBackRows, and the run's column sums
// go to one row of the partial array, which launch_column_sums adds in order.
constexpr int kBackRows = 64;

template <typename T>
__global__ __launch_bounds__(256) void linear_back(int64_t R, int M, int act, const T* __restrict__ dy, const T* z, T* dz,
                                                   float* part, int64_t runs) {
  __shared__ float join[4][512];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t run = blockIdx.x % runs;
  const int col = (int)(blockIdx.x / runs) * 512 + lane * 8;
  const int64_t first = run * kBackRows, last = min(first + kBackRows, R);
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (col < M) {
    for (int64_t n = first + wave; n < last; n += 16) {
      Raw8<T> rd[4], rz[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (n + 4 * u < last) {
          rd[u] = raw_load8(dy + (n + 4 * u) * M + col);
          if (act != MOE_ACT_NONE) rz[u] = raw_load8(z + (n + 4 * u) * M + col);
        }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (n + 4 * u < last) {
          float d[8], v[8];
          widen8(rd[u], d);
          if (act != MOE_ACT_NONE) {
            widen8(rz[u], v);
            act_slope_times<std::is_same<T, uint16_t>::value, 8>(act, v, d);
          }
          if (dz) raw_store8<false>(dz + (n + 4 * u) * M + col, d);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[i] += d[i];
        }
    }
  }
  if (!part) return;
  raw_store8<false>(&join[wave][lane * 8], sum);
  __syncthreads();
  for (int c = threadIdx.x; c < 512; c += 256) {
    const int at = (int)(blockIdx.x / runs) * 512 + c;
    if (at < M) part[run * M + at] = ((join[0][c] + join[1][c]) + join[2][c]) + join[3][c];
  }
}

template <typename T>
hipError_t linear_back_t(const LinearBackCall& c, hipStream_t s) {
  const int64_t runs = linear_back_runs(c.R);
  hipLaunchKernelGGL(linear_back<T>, dim3((unsigned)(runs * ((c.out + 511) / 512))), dim3(256), 0, s, c.R, c.out, c.act,
                     (const T*)c.dy, (const T*)c.z, (T*)c.dz, c.dbias ? c.part : nullptr, runs);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !c.dbias) return e;
  return launch_column_sums(c.part, c.dbias, nullptr, nullptr, runs, c.out, s);
}

}  // namespace

int64_t linear_join_blocks(int64_t R, int out) { return (R * (out / 8) + 255) / 256; }
int64_t linear_back_runs(int64_t R) { return (R + kBackRows - 1) / kBackRows; }

namespace {
constexpr int kMaxSplits = 16;
int tile_rows(int dtype, int64_t R) {
  if (R <= 32) return 32;
  if (R <= 64) return 64;
  return R <= 128 || dtype == MOE_F32 ? 128 : 256;
}
}  // namespace

LinearPlan linear_plan(int dtype, int64_t R, int in, int out) {
  LinearPlan p{tile_rows(dtype, R), 128, 1};
  if (dtype == MOE_BF16 && (R + 255) / 256 * ((out + 255) / 256) >= 192) {
    p.bn = 256;
    p.bm = 256;
    return p;
  }
  const int64_t tiles = (R + p.bm - 1) / p.bm * ((out + 127) / 128);
  const int64_t slots = p.bm <= 64 ? 512 : 256;
  const int steps = in / (dtype == MOE_F32 ? 32 : 64);
  int64_t splits = std::min<int64_t>(slots / tiles, steps / 4);
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(splits, kMaxSplits));
  return p;
}

// A split call has at most 512 / tiles parts (256 / tiles for tiles of 128 rows and more) of R x out floats, and R x out
// is at most tiles x the tile's size (linear_plan); kMaxSplits parts at most. Both bounds never fall as R grows.
size_t linear_part_bytes(int dtype, int64_t R, int out) {
  const int64_t bm = tile_rows(dtype, R), slots = bm <= 64 ? 512 : 256;
  const int64_t by_tiles = slots * bm * 128;
  const int64_t rows = std::min<int64_t>(R, (int64_t)1 << 22);
  const int64_t by_rows = rows * out * kMaxSplits;
  return sizeof(float) * (size_t)std::min(by_tiles, by_rows);
}

hipError_t launch_linear(int dtype, const LinearCall& c, hipStream_t s) {
  const LinearPlan p = linear_plan(dtype, c.R, c.in, c.out);
  return dtype == MOE_F32 ? linear_t<float>(c, p, s) : linear_t<uint16_t>(c, p, s);
}

hipError_t launch_linear_back(int dtype, const LinearBackCall& c, hipStream_t s) {
  return dtype == MOE_F32 ? linear_back_t<float>(c, s) : linear_back_t<uint16_t>(c, s);
}

}  // namespace moe
