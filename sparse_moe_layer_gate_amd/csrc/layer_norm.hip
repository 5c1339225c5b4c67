// Layer norm, optionally with the residual sum in front of it, and its gradients:
//
//   h = x + residual    m = mean(h)    r = 1 / sqrt(mean((h - m)^2) + eps)    n = (h - m) r    y = n w + b
//   t = dy w            dh = dh_out + r (t - mean(t) - n mean(t n))           dw = sum_rows dy n    db = sum_rows dy
//
// Everything between the loads and the stores is float32. Both passes are bound by HBM: a row is read once into
// registers (pieces of eight consecutive features), so the sums and the second use of a row cost no second read.
// Rows of up to 2,048 features belong to a group of 8 to 64 lanes of one wave, which needs no barrier and fills the
// wave with several narrow rows; wider ones to a block. In bfloat16, 8,191 x 5,120 with the residual take 62 us, 5.4 TB/s,
// and the gradients of 4,096 x 4,096 25 and 5 for the join of the sums, 5.7 TB/s of the first.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "ops_internal.h"
#include "row_ops.h"

namespace moe {
namespace {

template <typename T>
struct LnArgs {
  int N, D;
  float eps;
  const T *x, *residual, *w, *b;  // backward: x is h
  T *h_out, *y;
  float* stats;  // [N, 2]
  // backward
  const T *dh_out, *dy;
  T* dh;
  float* part;  // [2][nblocks][D] partial sums: dw, db
  int64_t nblocks;
  int want;  // bit 0: dw, 1: db
};

constexpr int kRowThreads = 256;     // of a block whose rows belong to groups of lanes
constexpr int kBlockThreads = 512;   // most of a block whose rows belong to it whole
constexpr int kNarrowThreads = 640;  // and with one piece per thread, in the backward pass

// Sums over the threads of a row: G lanes of a wave, or (G = 0) the block. Every thread of the row gets them.
template <int NV, int G>
__device__ inline void row_sums(float (&v)[NV], float (*buf)[NV], int waves) {
  if constexpr (G == 0) {
    block_sums<NV>(v, buf, waves);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int off = G / 2; off > 0; off >>= 1) v[i] += __shfl_xor(v[i], off);
  }
}

// VPT pieces of eight features per thread. The variance is the mean square around a first mean, less the square of
// what that mean is off by, so that neither a large common offset nor its rounding reaches it. h_out may be x or
// residual: a thread writes only what it has read.
template <typename T, int VPT, int G>
__global__ __launch_bounds__(G ? kRowThreads : kBlockThreads) void layer_norm_forward(LnArgs<T> p) {
  __shared__ float buf0[16][1], buf1[16][2];
  const int waves = blockDim.x >> 6;
  const int t = G ? threadIdx.x % (G ? G : 1) : threadIdx.x, step = G ? G : blockDim.x;
  const int64_t n = G ? (int64_t)blockIdx.x * (kRowThreads / (G ? G : 1)) + threadIdx.x / (G ? G : 1) : blockIdx.x;
  if (n >= p.N) return;  // whole groups: the shuffles of the others stay within theirs
  const float inv_d = 1.0f / (float)p.D;
  float h[VPT][8];
  Raw8<T> rx[VPT], rr[VPT], rw[VPT], rb[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = (t + v * step) * 8;
    if (c >= p.D) continue;
    rx[v] = raw_load8(p.x + n * p.D + c);
    if (p.residual) rr[v] = raw_load8(p.residual + n * p.D + c);
  }
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = (t + v * step) * 8;
    if (c >= p.D) continue;
    if (p.w) rw[v] = raw_load8(p.w + c);
    if (p.b) rb[v] = raw_load8(p.b + c);
  }
  float s[1] = {0.f};
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = (t + v * step) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[v][i] = 0.f;
    if (c >= p.D) continue;
    widen8(rx[v], h[v]);
    if (p.residual) {
      float r[8];
      widen8(rr[v], r);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[v][i] += r[i];
      raw_store8(p.h_out + n * p.D + c, h[v]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s[0] += h[v][i];
  }
  row_sums<1, G>(s, buf0, waves);
  const float m0 = s[0] * inv_d;
  float q[2] = {0.f, 0.f};
#pragma unroll
  for (int v = 0; v < VPT; ++v)
    if ((t + v * step) * 8 < p.D) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[v][i] -= m0;
        q[0] += h[v][i];
        q[1] += h[v][i] * h[v][i];
      }
    }
  row_sums<2, G>(q, buf1, waves);
  const float off = q[0] * inv_d;
  const float r = 1.0f / sqrtf(fmaxf(q[1] * inv_d - off * off, 0.f) + p.eps);
  if (p.stats && t == 0) {
    p.stats[2 * n] = m0 + off;
    p.stats[2 * n + 1] = r;
  }
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = (t + v * step) * 8;
    if (c >= p.D) continue;
    float w[8], b[8];
    if (p.w) widen8(rw[v], w);
    if (p.b) widen8(rb[v], b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float y = (h[v][i] - off) * r;
      if (p.w) y *= w[i];
      if (p.b) y += b[i];
      h[v][i] = y;
    }
    raw_store8<false>(p.y + n * p.D + c, h[v]);  // the next block reads y at once
  }
}

// p + i by a 32-bit offset from a base that a block shares: one register instead of an address per array and piece.
template <typename T>
__device__ inline T* offset(T* p, int i) {
  return (T*)((uintptr_t)p + (uint32_t)i * (uint32_t)sizeof(T));
}

template <typename T>
__device__ inline Raw8<T> raw_of8(const float* f) {
  Raw8<T> r;
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[i] = bf16_pair(f[2 * i], f[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.a[i] = f[i];
      r.b[i] = f[4 + i];
    }
  }
  return r;
}

// Keeps the compiler from holding widened copies of loaded values across a use.
__device__ inline void opaque(Raw8<uint16_t>& r) { asm volatile("" : "+v"(r.v)); }
__device__ inline void opaque(Raw8<float>& r) { asm volatile("" : "+v"(r.a), "+v"(r.b)); }

// A block takes rows in turn (one, or one per group of lanes, at a time), so that those at work at once lie side by side
// in memory (against a run of rows per block: 4,096 features 5.2 TB/s to 5.0, 8,192 5.6 to 5.2), and keeps its
// features' parameter gradients in registers; its sums go to one row of the partial arrays, which launch_column_sums adds
// in order. A row's values stay as loaded, and both passes over them widen them anew; without that and the pinned sums
// (the compiler else moves the additions behind the barrier, with all their operands) rows of 12,288 features spilled
// 130 registers and ran at 1.5 TB/s, now 5.0.
template <typename T, int VPT, int G>
__global__ __launch_bounds__(G ? kRowThreads : VPT == 1 ? kNarrowThreads : kBlockThreads) void layer_norm_backward(LnArgs<T> p) {
  __shared__ float buf[2][16][2];
  __shared__ float join[G ? 4 : 1][2][G ? VPT * G * 8 : 1];  // G: one row of sums per wave
  constexpr int GG = G ? G : 1;
  const int waves = blockDim.x >> 6;
  const int t = G ? threadIdx.x % GG : threadIdx.x, step = G ? G : blockDim.x;
  const int rows_at_once = G ? kRowThreads / GG : 1;
  const float inv_d = 1.0f / (float)p.D;
  const int64_t b = blockIdx.x;
  const int64_t stride = p.nblocks * rows_at_once;
  float aw[VPT][8], ab[VPT][8];
#pragma unroll
  for (int v = 0; v < VPT; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) aw[v][i] = ab[v][i] = 0.f;
  Raw8<T> rw[VPT];
  // The next row's pieces: its loads run under this row's sums. Not with four pieces of float32 per thread (rows of more
  // than 12,288 features), whose registers hold one row only.
  constexpr bool AHEAD = sizeof(T) == 2 || VPT < 4;
  Raw8<T> nh[VPT], ny[VPT], nd[VPT];
  const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, one[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    nh[v] = ny[v] = nd[v] = raw_of8<T>(zero);
    rw[v] = raw_of8<T>(one);
  }
  float mean = 0.f, rstd = 0.f;
  auto fetch = [&](int64_t n) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (t + v * step) * 8;
      if (c >= p.D) continue;
      nh[v] = raw_load8(offset(p.x + n * p.D, c));
      ny[v] = raw_load8(offset(p.dy + n * p.D, c));
      if (p.dh_out) nd[v] = raw_load8(offset(p.dh_out + n * p.D, c));
    }
    mean = p.stats[2 * n];
    rstd = p.stats[2 * n + 1];
  };
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = (t + v * step) * 8;
    if (p.w && c < p.D) rw[v] = raw_load8(p.w + c);
  }
  int64_t n = b * rows_at_once + (G ? threadIdx.x / GG : 0);
  if (AHEAD && n < p.N) fetch(n);
  for (int it = 0; n < p.N; n += stride, ++it) {
    if (!AHEAD) fetch(n);
    Raw8<T> rh[VPT], ry[VPT], rd[VPT];
    const float m = mean, r = rstd;
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      rh[v] = nh[v];
      ry[v] = ny[v];
      rd[v] = nd[v];
    }
    if (AHEAD && n + stride < p.N) fetch(n + stride);
#pragma unroll
    for (int v = 0; v < VPT; ++v) opaque(rw[v]);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float h[8], y[8], w[8];
      widen8(rh[v], h);
      widen8(ry[v], y);
      widen8(rw[v], w);
      const bool in = (t + v * step) * 8 < p.D;  // behind the row's end all are 0, so that nothing is added
      const float mv = in ? m : 0.f, rv = in ? r : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[i] = (h[i] - mv) * rv;
        aw[v][i] += y[i] * h[i];
        ab[v][i] += y[i];
        y[i] *= w[i];
        s[0] += y[i];
        s[1] += y[i] * h[i];
      }
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) asm volatile("" : "+v"(aw[v][i]), "+v"(ab[v][i]));
    row_sums<2, G>(s, buf[it & 1], waves);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      opaque(rh[v]);
      opaque(ry[v]);
      opaque(rw[v]);
    }
    const float c0 = s[0] * inv_d, c1 = s[1] * inv_d;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (t + v * step) * 8;
      float d[8];
      widen8(rd[v], d);
      float h[8], y[8], w[8];
      widen8(rh[v], h);
      widen8(ry[v], y);
      widen8(rw[v], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[i] *= w[i];
        d[i] += r * (y[i] - c0 - (h[i] - m) * r * c1);
      }
      if (c < p.D) raw_store8(offset(p.dh + n * p.D, c), d);
    }
  }
  if (p.want == 0) return;
  if constexpr (G != 0) {
    // the groups of a wave, then the waves in order
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int off = G; off < 64; off <<= 1) {
          aw[v][i] += __shfl_xor(aw[v][i], off);
          ab[v][i] += __shfl_xor(ab[v][i], off);
        }
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) < G) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        raw_store8<false>(&join[wave][0][(t + v * G) * 8], aw[v]);
        raw_store8<false>(&join[wave][1][(t + v * G) * 8], ab[v]);
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.D; c += kRowThreads) {
      if (p.want & 1) p.part[b * p.D + c] = ((join[0][0][c] + join[1][0][c]) + join[2][0][c]) + join[3][0][c];
      if (p.want & 2)
        p.part[(p.nblocks + b) * p.D + c] = ((join[0][1][c] + join[1][1][c]) + join[2][1][c]) + join[3][1][c];
    }
  } else {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (t + v * step) * 8;
      if (c >= p.D) continue;
      if (p.want & 1) raw_store8<false>(p.part + b * p.D + c, aw[v]);
      if (p.want & 2) raw_store8<false>(p.part + (p.nblocks + b) * p.D + c, ab[v]);
    }
  }
}

// Columns of up to two arrays [rows, D]: 64 columns per block, 64 row lanes, four rows of a lane in flight, then the
// lanes in a fixed order.
struct ColumnJob {
  const float* src;
  float* dst;
};
__global__ __launch_bounds__(1024) void column_sums(ColumnJob j0, ColumnJob j1, int64_t rows, int D) {
  __shared__ f32x4v acc[16][16];
  const ColumnJob job = blockIdx.y == 0 ? j0 : j1;
  const int col = blockIdx.x * 64 + (threadIdx.x & 15) * 4, lane = threadIdx.x >> 4, wave = threadIdx.x >> 6;
  f32x4v s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = f32x4v{0.f, 0.f, 0.f, 0.f};
  if (col < D) {
    const float* src = job.src + col;
    for (int64_t r = lane; r < rows; r += 256) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r + 64 * i < rows) s[i] += *(const f32x4v*)(src + (r + 64 * i) * D);
    }
  }
  f32x4v v = (s[0] + s[1]) + (s[2] + s[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] += __shfl_xor(v[i], 16);
    v[i] += __shfl_xor(v[i], 32);
  }
  if ((threadIdx.x & 63) < 16) acc[wave][threadIdx.x & 15] = v;
  __syncthreads();
  if (threadIdx.x < 16 && col < D) {
    v = acc[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < 16; ++w) v += acc[w][threadIdx.x];
    *(f32x4v*)(job.dst + col) = v;
  }
}

// Lanes of a row's group (0: the block takes the row), threads of a block, pieces per thread. Several pieces per thread
// keep more of a row in flight per block and need fewer waves at its barriers: forward, 5,120 features of bfloat16 with
// one piece (640 threads) 3.3 TB/s, with four (192) 5.6; four in three waves of 12,288 features 4.9 and three in eight
// waves 5.6. The backward pass, which has the next row's loads in flight, takes one piece up to 640 threads (5,120
// features 5.0 TB/s, with two 3.6 and with three 4.8), then as many as its registers hold.
struct Shape {
  int lanes, threads, vpt;
};
Shape shape_of(int D, bool backward) {
  if (D <= 512) {
    int g = 8;
    while (g * 8 < D) g *= 2;
    return {g, kRowThreads, 1};
  }
  if (D <= (backward ? 1024 : 2048)) return {64, kRowThreads, D <= 1024 ? 2 : 4};
  const int vpt = backward ? (D <= 8 * kNarrowThreads ? 1 : D <= 24 * kBlockThreads ? 3 : 4)
                           : (D <= 8192 || D > 24 * kBlockThreads ? 4 : 3);
  return {0, ((D / 8 + vpt - 1) / vpt + 63) / 64 * 64, vpt};
}

template <typename T, bool BACKWARD, int VPT, int G>
hipError_t run(const LnArgs<T>& p, int64_t blocks, int threads, hipStream_t s) {
  if constexpr (BACKWARD)
    hipLaunchKernelGGL((layer_norm_backward<T, VPT, G>), dim3((unsigned)blocks), dim3(threads), 0, s, p);
  else
    hipLaunchKernelGGL((layer_norm_forward<T, VPT, G>), dim3((unsigned)blocks), dim3(threads), 0, s, p);
  return hipGetLastError();
}

template <typename T, bool BACKWARD>
hipError_t pick(const LnArgs<T>& p, const Shape& sh, int64_t blocks, hipStream_t s) {
  if (sh.lanes == 8) return run<T, BACKWARD, 1, 8>(p, blocks, sh.threads, s);
  if (sh.lanes == 16) return run<T, BACKWARD, 1, 16>(p, blocks, sh.threads, s);
  if (sh.lanes == 32) return run<T, BACKWARD, 1, 32>(p, blocks, sh.threads, s);
  if (sh.lanes == 64) {
    if (sh.vpt == 1) return run<T, BACKWARD, 1, 64>(p, blocks, sh.threads, s);
    if (sh.vpt == 2) return run<T, BACKWARD, 2, 64>(p, blocks, sh.threads, s);
    if constexpr (!BACKWARD) return run<T, BACKWARD, 4, 64>(p, blocks, sh.threads, s);
  }
  if constexpr (BACKWARD)
    if (sh.vpt == 1) return run<T, BACKWARD, 1, 0>(p, blocks, sh.threads, s);
  if (sh.vpt == 3) return run<T, BACKWARD, 3, 0>(p, blocks, sh.threads, s);
  return run<T, BACKWARD, 4, 0>(p, blocks, sh.threads, s);
}

template <typename T>
hipError_t layer_norm_t(const LayerNormCall& c, bool backward, hipStream_t s) {
  LnArgs<T> p{};
  p.N = (int)c.N;
  p.D = c.D;
  p.eps = c.eps;
  p.x = (const T*)c.x;
  p.residual = (const T*)c.residual;
  p.w = (const T*)c.w;
  p.b = (const T*)c.b;
  p.h_out = (T*)c.h_out;
  p.y = (T*)c.y;
  p.stats = c.stats;
  if (!backward) {
    return pick<T, false>(p, shape_of(c.D, false), layer_norm_blocks(c.N, c.D), s);
  }
  p.dh_out = (const T*)c.dh_out;
  p.dy = (const T*)c.dy;
  p.dh = (T*)c.dh;
  p.part = c.part;
  p.want = (c.dw ? 1 : 0) | (c.db ? 2 : 0);
  const Shape sh = shape_of(c.D, true);
  const int64_t rows = sh.lanes ? kRowThreads / sh.lanes : 1;
  p.nblocks = std::min((c.N + rows - 1) / rows, layer_norm_runs(c.D));
  const hipError_t e = pick<T, true>(p, sh, p.nblocks, s);
  if (e != hipSuccess || p.want == 0) return e;
  const float* pw = p.part;
  const float* pb = p.part + p.nblocks * c.D;
  return launch_column_sums(c.dw ? pw : pb, c.dw ? c.dw : c.db, p.want == 3 ? pb : nullptr, c.db, p.nblocks, c.D, s);
}

}  // namespace

int layer_norm_threads(int D) { return shape_of(D, false).threads; }
int64_t layer_norm_blocks(int64_t N, int D) {
  const Shape sh = shape_of(D, false);
  return sh.lanes ? (N + kRowThreads / sh.lanes - 1) / (kRowThreads / sh.lanes) : N;
}
// Blocks of the backward pass: two per CU, or one of more than 320 threads (2,560 features: 4.4 and 5.4 TB/s with one and
// two; 4,096: 6.0 and 5.4).
int64_t layer_norm_runs(int D) { return shape_of(D, true).threads <= 320 ? 512 : 256; }

hipError_t launch_layer_norm(int dtype, const LayerNormCall& c, bool backward, hipStream_t s) {
  return dtype == MOE_F32 ? layer_norm_t<float>(c, backward, s) : layer_norm_t<uint16_t>(c, backward, s);
}

hipError_t launch_column_sums(const float* src0, float* dst0, const float* src1, float* dst1, int64_t rows, int D,
                              hipStream_t s) {
  hipLaunchKernelGGL(column_sums, dim3((D + 63) / 64, src1 ? 2 : 1), dim3(1024), 0, s, ColumnJob{src0, dst0},
                     ColumnJob{src1, dst1}, rows, D);
  return hipGetLastError();
}

}  // namespace moe
