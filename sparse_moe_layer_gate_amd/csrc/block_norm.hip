// Norms before and after a block, fused with the block's gate and the residual scale:
//
//   h_out = a h + g * (o rho(o)) w_post      u = (h_out rho(h_out)) w_pre      rho(v) = 1 / sqrt(mean(v^2) + eps)
//
// and the gradients. With d = dh_out + [gradient of u through the second norm], t = du w_pre,
// n = h_out rho(h_out), m = o rho(o):
//
//   d      = dh_out + rho(h_out) (t - n mean(t n))     dw_pre  = sum_rows du n
//   dh     = a d                                        dgate   = sum over the gate row's rows of d m w_post
//   do     = rho(o) (z - m mean(z m)), z = d g w_post   dw_post = sum_rows d g m
//
// Everything between the loads and the stores is float32. Both passes are bound by HBM: each row is read
// once into registers (eight consecutive features per thread and pass over the row), so the sums and the
// second use of a row cost no second read. Rows come straight from the kernel before, so the loads keep the
// default policy and may hit the last-level cache (8,191 x 5,120 forward 72 us with non-temporal loads, 61
// without); the stores are non-temporal where nothing reads them soon (61 against 75). On inputs that are not in
// that cache the forward takes 69 us, 4.9 TB/s, the rate of a large copy; the gradients of 4,096 x 4,096 take 56 us,
// 3.6 TB/s (two barriers and the partial sums of the parameter gradients cost the rest).
#include <hip/hip_runtime.h>

#include "ops_internal.h"
#include "row_ops.h"

namespace moe {
namespace {

template <typename T>
struct NormArgs {
  int N;
  int D;
  float eps, a;
  const T* h;       // forward: h; backward: h_out
  const T* o;       // or nullptr
  const T* w_post;  // or nullptr
  const T* gate;    // or nullptr; row n uses gate row n / gate_rows
  int gate_rows;
  const T* w_pre;  // or nullptr
  T* h_out;        // forward; nullptr without o
  T* u;            // forward; nullptr without w_pre
  // backward
  const T* dh_out;  // or nullptr
  const T* du;      // nullptr without w_pre
  T* dh;
  T* d_o;
  float* part;    // [3][nblocks][D] partial sums: dw_post, dw_pre, dgate
  float* dgate;   // written directly when a block holds whole gate groups
  int chunk;  // rows per block
  int chunks_per_group;  // > 0: blocks split one gate group; 0: chunks run over all rows
  int64_t nblocks;
  int want;  // bit 0: dw_post, 1: dw_pre, 2: dgate
};

// One block per row; the row's 8-feature pieces stay in registers between the sums and the outputs. VPT
// pieces per thread (2 only for rows of more than 8192 features). h_out may be h itself: a thread
// writes only what it has read.
template <typename T, int VPT, bool POST, bool PRE>
__global__ __launch_bounds__(1024) void norm_forward(NormArgs<T> p) {
  __shared__ float buf0[16][1], buf1[16][1];
  const int64_t n = blockIdx.x;
  const int waves = blockDim.x >> 6;
  const float inv_d = 1.0f / (float)p.D;
  float h[VPT][8], o[POST ? VPT : 1][8];
  Raw8<T> rw[VPT], rg[VPT], rp[VPT];
  const T* gate = POST && p.gate ? p.gate + (int64_t)((int)blockIdx.x / p.gate_rows) * p.D : nullptr;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = (threadIdx.x + v * blockDim.x) * 8;
    if (c >= p.D) continue;
    const Raw8<T> rh = raw_load8(p.h + n * p.D + c);
    if (POST) {
      const Raw8<T> ro = raw_load8(p.o + n * p.D + c);
      if (p.w_post) rw[v] = raw_load8(p.w_post + c);
      if (gate) rg[v] = raw_load8(gate + c);
      if (PRE) rp[v] = raw_load8(p.w_pre + c);
      widen8(ro, o[v]);
    } else if (PRE) {
      rp[v] = raw_load8(p.w_pre + c);
    }
    widen8(rh, h[v]);
  }
  if (POST) {
    float s[1] = {0.f};
    if (p.w_post) {  // without w_post the block's output is added as it is
#pragma unroll
      for (int v = 0; v < VPT; ++v)
        if ((threadIdx.x + v * blockDim.x) * 8 < p.D) {
#pragma unroll
          for (int i = 0; i < 8; ++i) s[0] += o[v][i] * o[v][i];
        }
      block_sums<1>(s, buf0, waves);
    }
    const float r = p.w_post ? 1.0f / sqrtf(s[0] * inv_d + p.eps) : 1.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (threadIdx.x + v * blockDim.x) * 8;
      if (c >= p.D) continue;
      float w[8], g[8];
      if (p.w_post) widen8(rw[v], w);
      if (gate) widen8(rg[v], g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float m = o[v][i] * r;
        if (p.w_post) m *= w[i];
        if (gate) m *= g[i];
        h[v][i] = p.a * h[v][i] + m;
      }
      raw_store8(p.h_out + n * p.D + c, h[v]);
    }
  }
  if (PRE) {
    // of the float32 row, before its rounding to h_out's type: u is rounded once
    float s[1] = {0.f};
#pragma unroll
    for (int v = 0; v < VPT; ++v)
      if ((threadIdx.x + v * blockDim.x) * 8 < p.D) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] += h[v][i] * h[v][i];
      }
    block_sums<1>(s, buf1, waves);
    const float r = 1.0f / sqrtf(s[0] * inv_d + p.eps);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (threadIdx.x + v * blockDim.x) * 8;
      if (c >= p.D) continue;
      float w[8], out[8];
      widen8(rp[v], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) out[i] = h[v][i] * r * w[i];
      raw_store8<false>(p.u + n * p.D + c, out);  // the next block reads u at once
    }
  }
}

// A block walks a run of rows and keeps its features' parameter gradients in registers; the run's sums go
// to one row of the partial arrays, which norm_reduce adds in block order (no atomics: the same inputs
// give the same bits). With gate rows of no more than a run, a run holds whole gate groups and dgate is
// written when a group ends; otherwise a run lies inside one group.
template <typename T, int VPT, int MAXT, bool POST, bool PRE>
__global__ __launch_bounds__(MAXT) void norm_backward(NormArgs<T> p) {
  __shared__ float buf0[2][16][3], buf1[16][1];
  const int waves = blockDim.x >> 6;
  const float inv_d = 1.0f / (float)p.D;
  const int64_t b = blockIdx.x;
  int first, last;  // rows; a last run may be empty
  if (p.chunks_per_group > 0) {
    const int g = blockIdx.x / p.chunks_per_group, c = blockIdx.x % p.chunks_per_group;
    const int64_t at = (int64_t)g * p.gate_rows + (int64_t)c * p.chunk;
    first = (int)min(at, (int64_t)p.N);
    last = (int)min(min(at + p.chunk, (int64_t)(g + 1) * p.gate_rows), (int64_t)p.N);
  } else {
    first = blockIdx.x * p.chunk;
    last = (int)min((int64_t)first + p.chunk, (int64_t)p.N);
  }
  float aw[POST ? VPT : 1][8], ag[POST ? VPT : 1][8], ap[PRE ? VPT : 1][8];
#pragma unroll
  for (int v = 0; v < VPT; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (POST) aw[v][i] = ag[v][i] = 0.f;
      if (PRE) ap[v][i] = 0.f;
    }
  const bool norm_o = POST && p.w_post;
  // the weights of this thread's features, and the current gate row's
  Raw8<T> rwp[PRE ? VPT : 1], rwo[POST ? VPT : 1], rg[POST ? VPT : 1];
  // the next row's pieces: its loads run under this row's sums (28% of the pass waited for them otherwise)
  Raw8<T> nd[VPT], nh[PRE ? VPT : 1], nt[PRE ? VPT : 1], no[POST ? VPT : 1];
  auto fetch = [&](int n) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (threadIdx.x + v * blockDim.x) * 8;
      if (c >= p.D) continue;
      const int64_t at = (int64_t)n * p.D + c;
      if (p.dh_out) nd[v] = raw_load8(p.dh_out + at);
      if (PRE) {
        nh[v] = raw_load8(p.h + at);
        nt[v] = raw_load8(p.du + at);
      }
      if (POST) no[v] = raw_load8(p.o + at);
    }
  };
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = (threadIdx.x + v * blockDim.x) * 8;
    if (c >= p.D) continue;
    if (PRE) rwp[v] = raw_load8(p.w_pre + c);
    if (norm_o) rwo[v] = raw_load8(p.w_post + c);
  }
  if (first < last) fetch(first);
  int gate_row = -1;
  for (int n = first; n < last; ++n) {
    float h[PRE ? VPT : 1][8], t[PRE ? VPT : 1][8], o[POST ? VPT : 1][8], d[VPT][8];
    float s[3] = {0.f, 0.f, 0.f};
    if (POST && p.gate && n / p.gate_rows != gate_row) {
      gate_row = n / p.gate_rows;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = (threadIdx.x + v * blockDim.x) * 8;
        if (c < p.D) rg[v] = raw_load8(p.gate + (int64_t)gate_row * p.D + c);
      }
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (threadIdx.x + v * blockDim.x) * 8;
      if (c >= p.D) continue;
      if (p.dh_out)
        widen8(nd[v], d[v]);
      else {
#pragma unroll
        for (int i = 0; i < 8; ++i) d[v][i] = 0.f;
      }
      if (PRE) {
        widen8(nh[v], h[v]);
        widen8(nt[v], t[v]);
      }
      if (POST) widen8(no[v], o[v]);
    }
    if (n + 1 < last) fetch(n + 1);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (threadIdx.x + v * blockDim.x) * 8;
      if (c >= p.D) continue;
      if (PRE) {
        float w[8];
        widen8(rwp[v], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s[0] += h[v][i] * h[v][i];
          s[1] += t[v][i] * w[i] * h[v][i];
        }
      }
      if (norm_o) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[2] += o[v][i] * o[v][i];
      }
    }
    if (PRE || norm_o) block_sums<3>(s, buf0[n & 1], waves);
    const float rh = PRE ? 1.0f / sqrtf(s[0] * inv_d + p.eps) : 0.f;
    const float ch = PRE ? s[1] * inv_d * rh * rh : 0.f;  // mean(t n) rho
    const float ro = norm_o ? 1.0f / sqrtf(s[2] * inv_d + p.eps) : 1.0f;
    float z[1] = {0.f};
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (threadIdx.x + v * blockDim.x) * 8;
      if (c >= p.D) continue;
      if (PRE) {
        float w[8];
        widen8(rwp[v], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ap[v][i] += t[v][i] * (h[v][i] * rh);
          d[v][i] += rh * (t[v][i] * w[i] - h[v][i] * ch);
        }
      }
      if (!POST) {
        raw_store8(p.dh + (int64_t)n * p.D + c, d[v]);
        continue;
      }
      float out[8], g[8], w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) out[i] = p.a * d[v][i];
      raw_store8(p.dh + (int64_t)n * p.D + c, out);
      const bool gate = p.gate != nullptr;
      if (gate) widen8(rg[v], g);
      if (norm_o) widen8(rwo[v], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float m = o[v][i] * ro;
        if (gate) ag[v][i] += d[v][i] * m * (norm_o ? w[i] : 1.0f);
        float q = gate ? d[v][i] * g[i] : d[v][i];
        aw[v][i] += q * m;
        if (norm_o) q *= w[i];
        d[v][i] = q;
        z[0] += q * o[v][i];
      }
    }
    if (POST) {
      if (norm_o) block_sums<1>(z, buf1, waves);
      const float cz = norm_o ? z[0] * inv_d * ro * ro : 0.f;  // mean(z m) rho
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = (threadIdx.x + v * blockDim.x) * 8;
        if (c >= p.D) continue;
        float out[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) out[i] = ro * (d[v][i] - o[v][i] * cz);
        raw_store8(p.d_o + (int64_t)n * p.D + c, out);
        // the gate group ends with this row
        if (p.dgate && p.chunks_per_group == 0 && ((n + 1) % p.gate_rows == 0 || n + 1 == p.N)) {
          raw_store8<false>(p.dgate + (int64_t)(n / p.gate_rows) * p.D + c, ag[v]);
#pragma unroll
          for (int i = 0; i < 8; ++i) ag[v][i] = 0.f;
        }
      }
    }
  }
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = (threadIdx.x + v * blockDim.x) * 8;
    if (c >= p.D) continue;
    if (POST && (p.want & 1)) raw_store8<false>(p.part + b * p.D + c, aw[v]);
    if (PRE && (p.want & 2)) raw_store8<false>(p.part + (p.nblocks + b) * p.D + c, ap[v]);
    if (POST && (p.want & 4) && p.chunks_per_group > 0)
      raw_store8<false>(p.part + (2 * p.nblocks + b) * p.D + c, ag[v]);
  }
}

// Sums of the partial rows: 32 features per block, 32 row lanes, eight rows of a lane in flight, then the lanes
// in order.
struct ReduceJob {
  const float* src;  // first partial row of group 0
  float* dst;        // [groups, D]
  int64_t rows;      // partial rows per group
  int64_t groups;
};
// Blocks of the backward pass have at most 512 threads (two pieces per thread above 4,096 features): with up
// to 1,024, the register budget of 128 spilled (4,096 x 4,096: 68 -> 63 us). Some forms still spill: with both norms
// in float32 above 4,096 features (31 registers; 4,096 x 5,120: 168 us, a copy of its bytes 104), and every form of
// rows of more than 8,192 features, which take 1,024 threads (both norms: 228 registers in bfloat16, 297 in float32;
// 1,024 x 16,384: 231 and 363 us, against 41 and 83).
constexpr int kBackwardThreads = 512;
struct ReduceArgs {
  ReduceJob job[3];
  int D;
};
__global__ __launch_bounds__(1024) void norm_reduce(ReduceArgs a) {
  __shared__ float acc[32][33];
  int64_t g = blockIdx.y;
  int which = 0;
  while (which < 2 && g >= a.job[which].groups) g -= a.job[which++].groups;
  const ReduceJob& job = which == 0 ? a.job[0] : which == 1 ? a.job[1] : a.job[2];
  if (g >= job.groups) return;
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), lane = threadIdx.x >> 5;
  const float* src = job.src + g * job.rows * a.D + col;
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int64_t r = lane; r < job.rows; r += 256) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (r + 32 * i < job.rows) s[i] += src[(r + 32 * i) * a.D];
  }
  acc[lane][threadIdx.x & 31] = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
  __syncthreads();
  if (lane == 0) {
    float t = 0.f;
#pragma unroll
    for (int l = 0; l < 32; ++l) t += acc[l][threadIdx.x];
    job.dst[g * a.D + col] = t;
  }
}

// Threads of a block and pieces per thread: one piece each while the block has at most `limit` threads, else two.
struct Shape {
  int threads, vpt;
};
Shape shape_of(int D, int limit) {
  const int t = (D / 8 + 63) / 64 * 64;
  if (t <= limit) return {t, 1};
  return {(D / 16 + 63) / 64 * 64, 2};
}

template <typename T, int VPT>
hipError_t forward_vpt(const NormArgs<T>& p, int threads, hipStream_t s) {
  const dim3 grid((unsigned)p.N), block(threads);
  if (p.o && p.w_pre)
    hipLaunchKernelGGL((norm_forward<T, VPT, true, true>), grid, block, 0, s, p);
  else if (p.o)
    hipLaunchKernelGGL((norm_forward<T, VPT, true, false>), grid, block, 0, s, p);
  else
    hipLaunchKernelGGL((norm_forward<T, VPT, false, true>), grid, block, 0, s, p);
  return hipGetLastError();
}

template <typename T, int VPT, int MAXT>
hipError_t backward_vpt(const NormArgs<T>& p, int threads, hipStream_t s) {
  const dim3 grid((unsigned)p.nblocks), block(threads);
  if (p.o && p.w_pre)
    hipLaunchKernelGGL((norm_backward<T, VPT, MAXT, true, true>), grid, block, 0, s, p);
  else if (p.o)
    hipLaunchKernelGGL((norm_backward<T, VPT, MAXT, true, false>), grid, block, 0, s, p);
  else
    hipLaunchKernelGGL((norm_backward<T, VPT, MAXT, false, true>), grid, block, 0, s, p);
  return hipGetLastError();
}

// Rows that share a gate row, at most N (one group then holds every row).
int64_t gate_rows_of(const NormCall& c) { return c.gate ? (c.gate_rows < c.N ? c.gate_rows : c.N) : 1; }

template <typename T>
hipError_t forward_t(const NormCall& c, hipStream_t s) {
  NormArgs<T> p{};
  p.N = (int)c.N;
  p.D = c.D;
  p.eps = c.eps;
  p.a = c.a;
  p.h = (const T*)c.h;
  p.o = (const T*)c.o;
  p.w_post = (const T*)c.w_post;
  p.gate = (const T*)c.gate;
  p.gate_rows = (int)gate_rows_of(c);
  p.w_pre = (const T*)c.w_pre;
  p.h_out = (T*)c.h_out;
  p.u = (T*)c.u;
  const Shape sh = shape_of(c.D, 1024);
  return sh.vpt == 1 ? forward_vpt<T, 1>(p, sh.threads, s) : forward_vpt<T, 2>(p, sh.threads, s);
}

template <typename T>
hipError_t backward_t(const NormCall& c, hipStream_t s) {
  const NormPlan pl = norm_plan(c.N, c.D, c.gate ? c.gate_rows : 0);
  NormArgs<T> p{};
  p.N = (int)c.N;
  p.D = c.D;
  p.eps = c.eps;
  p.a = c.a;
  p.h = (const T*)c.h;
  p.o = (const T*)c.o;
  p.w_post = (const T*)c.w_post;
  p.gate = (const T*)c.gate;
  p.gate_rows = (int)gate_rows_of(c);
  p.w_pre = (const T*)c.w_pre;
  p.dh_out = (const T*)c.dh_out;
  p.du = (const T*)c.du;
  p.dh = (T*)c.dh;
  p.d_o = (T*)c.d_o;
  p.part = c.part;
  p.dgate = c.dgate;
  p.chunk = (int)pl.chunk;
  p.chunks_per_group = (int)pl.chunks_per_group;
  p.nblocks = pl.nblocks;
  p.want = (c.dw_post ? 1 : 0) | (c.dw_pre ? 2 : 0) | (c.dgate ? 4 : 0);
  const Shape sh = shape_of(c.D, kBackwardThreads);
  const hipError_t e = sh.vpt == 1 ? backward_vpt<T, 1, kBackwardThreads>(p, sh.threads, s)
                       : sh.threads <= kBackwardThreads ? backward_vpt<T, 2, kBackwardThreads>(p, sh.threads, s)
                                                        : backward_vpt<T, 2, 1024>(p, sh.threads, s);
  if (e != hipSuccess) return e;
  ReduceArgs r{};
  r.D = c.D;
  int64_t groups = 0;
  if (c.dw_post) groups += (r.job[0] = ReduceJob{p.part, c.dw_post, pl.nblocks, 1}).groups;
  if (c.dw_pre) groups += (r.job[1] = ReduceJob{p.part + pl.nblocks * c.D, c.dw_pre, pl.nblocks, 1}).groups;
  if (c.dgate && pl.chunks_per_group > 0)
    groups += (r.job[2] = ReduceJob{p.part + 2 * pl.nblocks * c.D, c.dgate, pl.chunks_per_group,
                                    pl.nblocks / pl.chunks_per_group}).groups;
  if (groups == 0) return hipSuccess;
  hipLaunchKernelGGL(norm_reduce, dim3(c.D / 32, (unsigned)groups), dim3(1024), 0, s, r);
  return hipGetLastError();
}

}  // namespace

int norm_forward_threads(int D) { return shape_of(D, 1024).threads; }

// Runs of the backward pass: blocks of 512 threads, or as many smaller ones as make no more, per CU (256 CUs): eight
// waves at 4,096 and 8,192 features, five at 2,560 and 5,120, six at 1,536 and 6,144. More runs mean more partial rows
// (three of D floats per run) to write and add: 4,096 x 4,096 with 256 / 512 runs 51 / 59 us, the one width where both
// were measured (4,096 rows of 5,120 and 6,144, the call: 73 and 82 us, copies of their bytes 52 and 62).
int64_t norm_runs(int D) {
  const int threads = shape_of(D, kBackwardThreads).threads;
  return threads >= 512 ? 256 : 256 * (512 / threads);
}

// With gate rows of no more than a run, runs are whole gate groups and may then be nearly twice an even share: 8,191
// rows of 4,096 with 31 rows a gate make 133 runs and take 149 us, 90 without a gate.
NormPlan norm_plan(int64_t N, int D, int64_t gate_rows) {
  const int64_t kBlocks = norm_runs(D);
  NormPlan p{};
  int64_t c = (N + kBlocks - 1) / kBlocks;
  if (c < 1) c = 1;
  const int64_t T = gate_rows < N ? gate_rows : N;
  if (gate_rows > 0 && T > c) {
    p.chunks_per_group = (T + c - 1) / c;
    p.chunk = (T + p.chunks_per_group - 1) / p.chunks_per_group;
    p.nblocks = (N + T - 1) / T * p.chunks_per_group;
  } else {
    if (gate_rows > 0) c = (c + T - 1) / T * T;
    p.chunk = c;
    p.nblocks = (N + c - 1) / c;
  }
  return p;
}

hipError_t launch_norm_forward(int dtype, const NormCall& c, hipStream_t s) {
  return dtype == MOE_F32 ? forward_t<float>(c, s) : forward_t<uint16_t>(c, s);
}

hipError_t launch_norm_backward(int dtype, const NormCall& c, hipStream_t s) {
  return dtype == MOE_F32 ? backward_t<float>(c, s) : backward_t<uint16_t>(c, s);
}

}  // namespace moe
