// The balance loss of a routed batch, per sequence, with the counts behind it, and the gradient of the router's
// logits. For a sequence of V live tokens, with p = s / sum(s) over a token's scores:
//
//   c_i = slots that name i    f_i = E c_i / (k V)    P_i = sum_tokens p_i / V    loss = weight / S sum_seq sum_i f_i P_i
//
// The loss is linear in p once the counts are constants: d loss / d p_i = weight / S f_i / V = coef_i, and through
// the normalisation d loss / d s_i = (coef_i - sum_j coef_j p_j) / sum(s). The weights w_m = alpha s_m / D give
// ds_m = alpha / D (dw_m - sum_l dw_l s_l / D); both meet in dlogit = ds s (1 - s).
//
// Both directions read the scores once (N E float32) and are bound by that, or for usual batches, which fit the
// caches, by latency: a row belongs to a group of 8 to 64 lanes, so that its sums are shuffles. 8,192 x 256 in sequences of
// 1,024: 6 us and 5.5 for the join; gradient of 8,000 x 160: 6; 1 M x 64 54 (5.4 TB/s) and 143 (4.1 TB/s).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "ops_internal.h"
#include "row_ops.h"

namespace moe {
namespace {

// Sum over the G lanes of a group, the same in each.
template <int G>
__device__ inline float group_sum(float v) {
#pragma unroll
  for (int off = G / 2; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

struct BalanceArgs {
  int64_t N, T;  // T <= N
  int E, k;
  int64_t S;
  int64_t chunk, chunks;  // rows per block, blocks per sequence
  float weight;           // over S
  const float* scores;
  const int32_t* idx;
  const uint8_t* mask;
  int32_t* counts;  // [S, E] or nullptr
  float* coef;      // [S, E] or nullptr
  float* loss;
  float* part_p;    // [S chunks, E] sums of p
  int32_t* part_c;  // [S chunks, E] slots
  int32_t* part_v;  // [S chunks] live tokens
  float* part_l;    // losses of the sequences, or of the blocks of balance_join
  int32_t* done;    // blocks of balance_join that have ended; nullptr: balance_total adds their shares
};

// The end of a sequence: f and P of one expert from its sums; returns f P weight / S.
__device__ inline float finish_expert(const BalanceArgs& a, int64_t q, int e, float p, int32_t c, int32_t v) {
  const float live = (float)max(v, 1);
  const float f = (float)c * (float)a.E / ((float)a.k * live);
  if (a.counts) a.counts[q * a.E + e] = c;
  if (a.coef) a.coef[q * a.E + e] = a.weight * f / live;
  return a.weight * f * (p / live);
}

// Sum of one float per thread over the block, in a fixed order, valid in thread 0.
__device__ inline float block_total(float v, float* buf) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
  float t = 0.f;
  if (threadIdx.x == 0)
    for (int w = 0; w < (int)(blockDim.x >> 6); ++w) t += buf[w];
  return t;
}

// The scores of a row lie with a group of G lanes: piece i of lane j holds the V experts from V (j + G i) on, one load of V
// floats. V = 4 needs E to be a multiple of 4; 16 lanes then take a row of up to 64 experts in one load and a wave four
// rows (one row of 64 lanes and single floats: 1 M rows of 64 experts, gradient 407 us, so 143).
template <int G, int PL, int V>
struct Row {
  static constexpr int N = PL * V;  // values per lane
  __device__ static int expert(int lane, int x) { return V * (lane + G * (x / V)) + x % V; }
  __device__ static void load(const float* row, int E, int lane, float* v) {
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = V * (lane + G * i);
      if constexpr (V == 4) {
        const f32x4v q = e < E ? *(const f32x4v*)(row + e) : f32x4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j) v[4 * i + j] = q[j];
      } else {
        v[i] = e < E ? row[e] : 0.f;
      }
    }
  }
};

// Float32 holds no reciprocal of a sum below 2^-128. Rows whose scores sum to less than kSmallSum are scaled up first, which
// is exact and leaves the shares p = s / sum as they are.
constexpr float kSmallSum = 0x1p-100f, kScaleUp = 0x1p64f;

// One chunk of a sequence's rows. Live tokens add to the sums in registers, the slots to a histogram in LDS (whole numbers:
// the order does not matter). A sequence of one chunk is finished here.
template <int G, int PL, int V>
__global__ __launch_bounds__(1024) void balance_chunks(BalanceArgs a) {
  using R = Row<G, PL, V>;
  __shared__ float sum[16][G * R::N];
  __shared__ int32_t hist[G * R::N];
  __shared__ int32_t live_rows;
  __shared__ float buf[16];
  if (a.done && blockIdx.x == 0 && threadIdx.x == 0) *a.done = 0;  // for balance_join, the next launch
  const int64_t q = blockIdx.x / a.chunks, ch = blockIdx.x % a.chunks;
  const int64_t first = q * a.T + ch * a.chunk;
  const int64_t last = min(min(first + a.chunk, (q + 1) * a.T), a.N);
  const int waves = blockDim.x >> 6, wave = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < G * R::N; e += blockDim.x) hist[e] = 0;
  if (threadIdx.x == 0) live_rows = 0;
  __syncthreads();
  const int lane = threadIdx.x % G;
  const int groups = blockDim.x / G;
  float acc[R::N];
  int mine = 0;
#pragma unroll
  for (int i = 0; i < R::N; ++i) acc[i] = 0.f;
  // two rows at a time, all their loads first: a block has only a few rows per group, each a trip to memory
  for (int64_t n0 = first + threadIdx.x / G; n0 < last; n0 += 2 * groups) {
    float v[2][R::N];
    int32_t id[2];
    bool live[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t n = n0 + u * groups;
      const bool have = n < last;
      live[u] = have && (!a.mask || a.mask[n] != 0);
      id[u] = have && lane < a.k ? a.idx[n * a.k + lane] : -1;
      if (have) R::load(a.scores + n * a.E, a.E, lane, v[u]);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (!live[u]) continue;  // the same for the lanes of a group
      float total = 0.f;
#pragma unroll
      for (int i = 0; i < R::N; ++i) total += v[u][i];
      total = group_sum<G>(total);
      if (fabsf(total) < kSmallSum) {
#pragma unroll
        for (int i = 0; i < R::N; ++i) v[u][i] *= kScaleUp;
        total *= kScaleUp;
      }
      const float inv = total != 0.f ? 1.0f / total : 0.f;
#pragma unroll
      for (int i = 0; i < R::N; ++i) acc[i] += v[u][i] * inv;
      if (id[u] >= 0 && id[u] < a.E) atomicAdd(&hist[id[u]], 1);
      for (int m = lane + G; m < a.k; m += G) {  // more slots than lanes
        const int32_t e = a.idx[(n0 + u * groups) * a.k + m];
        if (e >= 0 && e < a.E) atomicAdd(&hist[e], 1);
      }
      mine += lane == 0;
    }
  }
  if (mine) atomicAdd(&live_rows, mine);
  // the groups of a wave, then the waves in order
#pragma unroll
  for (int i = 0; i < R::N; ++i) {
#pragma unroll
    for (int off = G; off < 64; off <<= 1) acc[i] += __shfl_xor(acc[i], off);
    if ((threadIdx.x & 63) < G) sum[wave][R::expert(lane, i)] = acc[i];
  }
  __syncthreads();
  float loss = 0.f;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    float p = 0.f;
    for (int w = 0; w < waves; ++w) p += sum[w][e];
    if (a.chunks == 1) {
      loss += finish_expert(a, q, e, p, hist[e], live_rows);
    } else {
      a.part_p[(int64_t)blockIdx.x * a.E + e] = p;
      a.part_c[(int64_t)blockIdx.x * a.E + e] = hist[e];
    }
  }
  if (a.chunks == 1) {
    loss = block_total(loss, buf);
    if (threadIdx.x == 0) (a.S == 1 ? a.loss : a.part_l + q)[0] = loss;
  } else if (threadIdx.x == 0) {
    a.part_v[blockIdx.x] = live_rows;
  }
}

// The chunks of one sequence, in order: a block takes kJoin experts, up to 32 lanes each, so that few of its loads wait
// for one another (32,768 x 256 in one sequence: 27 -> 24 us). Of a few blocks the one that
// ends last adds their shares of the loss, in order (0.5 us less than one more launch); more take balance_total, since they
// would wait at the count (512 blocks: 25 us for 21).
constexpr int kJoin = 32, kCountedBlocks = 128;
static_assert(kJoin == 32, "two lanes of every expert per wave");
__global__ __launch_bounds__(1024) void balance_join(BalanceArgs a, int parts) {
  __shared__ float sp[16][kJoin];
  __shared__ int32_t sc[16][kJoin];
  __shared__ int32_t sv[16];
  __shared__ float buf[16];
  __shared__ int last;
  const int64_t q = blockIdx.x / parts, base = q * a.chunks;
  const int lanes = blockDim.x / kJoin;
  const int e = (int)(blockIdx.x % parts) * kJoin + threadIdx.x % kJoin, l = threadIdx.x / kJoin;
  float p = 0.f;
  int32_t c = 0, v = threadIdx.x < a.chunks ? a.part_v[base + threadIdx.x] : 0;  // no more chunks than threads
  if (e < a.E) {
    for (int64_t ch = l; ch < a.chunks; ch += 8 * lanes) {
      float rp[8];
      int32_t rc[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const bool have = ch + u * lanes < a.chunks;
        const int64_t at = (base + ch + u * lanes) * a.E + e;
        rp[u] = have ? a.part_p[at] : 0.f;
        rc[u] = have ? a.part_c[at] : 0;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        p += rp[u];
        c += rc[u];
      }
    }
  }
  // the two lanes of a wave, then the waves
  const int waves = blockDim.x >> 6, wave = threadIdx.x >> 6;
  p += __shfl_xor(p, kJoin);
  c += __shfl_xor(c, kJoin);
  if ((threadIdx.x & 63) < kJoin) {
    sp[wave][threadIdx.x % kJoin] = p;
    sc[wave][threadIdx.x % kJoin] = c;
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  if ((threadIdx.x & 63) == 0) sv[wave] = v;
  __syncthreads();
  float loss = 0.f;
  if (threadIdx.x < kJoin && e < a.E) {
    v = sv[0];
#pragma unroll
    for (int w = 1; w < 16; ++w)
      if (w < waves) {
        p += sp[w][threadIdx.x];
        c += sc[w][threadIdx.x];
        v += sv[w];
      }
    loss = finish_expert(a, q, e, p, c, v);
  }
  if (threadIdx.x < 64) loss = wave_sum(loss);
  if (threadIdx.x == 0) {
    // The one value that another block reads goes past the caches of this XCD (what a store of agent scope does on gfx950)
    // and, by the wait, is there before the count rises. That order is the chip's: the language's would be a release fence,
    // which writes back all that the caches hold (9.4 us for the launch at 8,192 x 256 in sequences of 1,024, 5.8 without).
    __hip_atomic_store(a.part_l + blockIdx.x, loss, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (a.done) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      last = __hip_atomic_fetch_add(a.done, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
    }
  }
  if (!a.done) return;
  __syncthreads();
  if (!last) return;
  float s = 0.f;
  for (int64_t i = threadIdx.x; i < gridDim.x; i += blockDim.x)
    s += __hip_atomic_load(a.part_l + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  s = block_total(s, buf);
  if (threadIdx.x == 0) *a.loss = s;
}

__global__ __launch_bounds__(1024) void balance_total(const float* part, int64_t n, float* loss) {
  __shared__ float buf[16];
  float s = 0.f;
  for (int64_t i = threadIdx.x; i < n; i += 1024) s += part[i];
  s = block_total(s, buf);
  if (threadIdx.x == 0) *loss = s;
}

struct RouteBackArgs {
  int64_t N, T;
  int E, k;
  float alpha, eps;
  int norm;
  const float* scores;
  const int32_t* idx;
  const float* dw;
  const float* coef;
  const float* dloss;
  const uint8_t* mask;
  float* out;
};

// A group of G lanes per token, a slot's owner lane m % G. The slots' scores are read again (they have just been loaded),
// their gradients go to the lanes of their experts one slot after the other. dlogits may be the scores: a group reads its
// row before it writes it.
template <int G, int PL, int V>
__global__ __launch_bounds__(256) void route_backward(RouteBackArgs a) {
  using R = Row<G, PL, V>;
  constexpr int SPL = (32 + G - 1) / G;  // slots per lane (k <= 32)
  const int lane = threadIdx.x % G;
  const int64_t n = (int64_t)blockIdx.x * (256 / G) + threadIdx.x / G;
  if (n >= a.N) return;  // whole groups
  // every load first
  const float* row = a.scores + n * a.E;
  const float* co = a.coef ? a.coef + n / a.T * a.E : nullptr;
  float s[R::N], c[R::N], ds[R::N];
  int32_t id[SPL];
  float w[SPL], sw[SPL];
#pragma unroll
  for (int m = 0; m < SPL; ++m) {
    const int slot = lane + G * m;
    const bool have = a.dw && slot < a.k;
    id[m] = have ? a.idx[n * a.k + slot] : -1;
    w[m] = have ? a.dw[n * a.k + slot] : 0.f;
  }
  R::load(row, a.E, lane, s);
#pragma unroll
  for (int i = 0; i < R::N; ++i) c[i] = ds[i] = 0.f;
  if (co) R::load(co, a.E, lane, c);
#pragma unroll
  for (int m = 0; m < SPL; ++m) {
    const bool ok = id[m] >= 0 && id[m] < a.E;
    sw[m] = ok ? row[id[m]] : 0.f;
    if (!ok) w[m] = 0.f;
  }
  const bool live = !a.mask || a.mask[n] != 0;
  const float g = a.dloss ? *a.dloss : 1.0f;
  float sum = 1.0f, dot = 0.f, total = 1.0f, dot_w = 0.f, down = 1.0f;
  auto add_scores = [&] {
    sum = dot = 0.f;
#pragma unroll
    for (int i = 0; i < R::N; ++i) {
      sum += s[i];
      dot += c[i] * s[i];
    }
    sum = group_sum<G>(sum);
    dot = group_sum<G>(dot);
  };
  auto add_slots = [&](float eps) {
    total = dot_w = 0.f;
#pragma unroll
    for (int m = 0; m < SPL; ++m) {
      total += sw[m];
      dot_w += sw[m] * w[m];
    }
    total = group_sum<G>(total) + eps;
    dot_w = group_sum<G>(dot_w);
  };
  if (co && live) add_scores();
  if (a.dw && a.norm) add_slots(a.eps);
  if (fminf(fabsf(sum), fabsf(total)) < kSmallSum) {  // ds s is the same with s times kScaleUp and ds over it
#pragma unroll
    for (int i = 0; i < R::N; ++i) s[i] *= kScaleUp;
#pragma unroll
    for (int m = 0; m < SPL; ++m) sw[m] *= kScaleUp;
    down = 1.0f / kScaleUp;
    if (co && live) add_scores();
    if (a.dw && a.norm) add_slots(a.eps * kScaleUp);
  }
  if (co && live) {
    const float inv = sum != 0.f ? 1.0f / sum : 0.f;
#pragma unroll
    for (int i = 0; i < R::N; ++i) ds[i] = g * inv * (c[i] - dot * inv);
  }
  if (a.dw) {
    if (a.norm) {
      // divided, not multiplied by a rounded reciprocal: with one slot the two terms are equal
      const float mean = total != 0.f ? dot_w / total : 0.f, scale = total != 0.f ? a.alpha / total : 0.f;
#pragma unroll
      for (int m = 0; m < SPL; ++m) w[m] = scale * (w[m] - mean);
    } else {
#pragma unroll
      for (int m = 0; m < SPL; ++m) w[m] *= a.alpha * down;
    }
    // every slot to the lane and value of its expert (an id may come up twice: each adds)
#pragma unroll
    for (int m = 0; m < SPL; ++m) {
      for (int l = 0; l < G && l + G * m < a.k; ++l) {
        const int32_t e = __shfl(id[m], l, G);
        const float b = __shfl(w[m], l, G);
        const int vec = e / V, at = e >= 0 && vec % G == lane ? vec / G * V + e % V : -1;
#pragma unroll
        for (int i = 0; i < R::N; ++i) ds[i] += at == i ? b : 0.f;
      }
    }
  }
  float* out = a.out + n * a.E;
#pragma unroll
  for (int i = 0; i < R::N; ++i)  // whatever a dead token holds
    ds[i] = ds[i] == 0.f ? 0.f : ds[i] * s[i] * fmaf(-s[i], down, 1.0f);
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = V * (lane + G * i);
    if (e >= a.E) continue;
    if constexpr (V == 4)
      *(f32x4v*)(out + e) = f32x4v{ds[4 * i], ds[4 * i + 1], ds[4 * i + 2], ds[4 * i + 3]};
    else
      out[e] = ds[i];
  }
}

// Lanes of a row's group.
int lanes_of(int E) { return E % 4 == 0 ? (E <= 32 ? 8 : 16) : E <= 8 ? 8 : E <= 16 ? 16 : E <= 32 ? 32 : 64; }

// Calls f with lanes, pieces and floats per piece as compile-time values.
template <typename F>
hipError_t with_shape(int E, F f) {
  using std::integral_constant;
  const integral_constant<int, 1> c1{};
  const integral_constant<int, 4> c4{};
  const integral_constant<int, 8> g8{};
  const integral_constant<int, 16> g16{};
  const integral_constant<int, 32> g32{};
  const integral_constant<int, 64> g64{};
  const int G = lanes_of(E);
  auto pieces = [&](auto g, auto v) {
    switch ((E + 63) / 64) {
      case 1: return f(g, integral_constant<int, 1>{}, v);
      case 2: return f(g, integral_constant<int, 2>{}, v);
      case 3: return f(g, integral_constant<int, 3>{}, v);
      case 4: return f(g, integral_constant<int, 4>{}, v);
      case 5: return f(g, integral_constant<int, 5>{}, v);
      case 6: return f(g, integral_constant<int, 6>{}, v);
      case 7: return f(g, integral_constant<int, 7>{}, v);
      case 8: return f(g, integral_constant<int, 8>{}, v);
    }
    return hipErrorInvalidValue;
  };
  if (E % 4 == 0) return G == 8 ? f(g8, c1, c4) : pieces(g16, c4);
  if (G == 8) return f(g8, c1, c1);
  if (G == 16) return f(g16, c1, c1);
  if (G == 32) return f(g32, c1, c1);
  return pieces(g64, c1);
}

}  // namespace

// Rows of a block: a few per group of lanes, with two to four blocks per CU in a large batch (1 M rows of 64 experts in
// sequences of 512: 59 us, with 32 rows per block 299). One block takes a sequence of up to 512 rows, or one of 256
// sequences and more (65,536 x 256 in sequences of 512: 17 us, with 64 rows per block 42). A sequence is never shared by
// more than 512 blocks.
BalancePlan balance_plan(int64_t N, int64_t T, int E) {
  BalancePlan p{};
  p.T = T < N ? T : N;
  if (p.T < 1) p.T = 1;
  p.S = (N + p.T - 1) / p.T;
  const int64_t wide = std::max((p.T + 511) / 512, (N + 1023) / 1024);
  p.chunk = wide > 32 ? wide : 32;
  if (p.chunk > p.T) p.chunk = p.T;
  if (p.T <= 512 || p.S >= 256) p.chunk = p.T;
  p.chunks = (p.T + p.chunk - 1) / p.chunk;
  const int64_t rows = 64 / lanes_of(E);  // of a wave at a time
  const int64_t waves = (p.chunk + 2 * rows - 1) / (2 * rows);
  p.threads = 64 * (int)(waves < 1 ? 1 : waves > 16 ? 16 : waves);
  p.join_parts = (E + kJoin - 1) / kJoin;
  p.join_threads = p.chunks >= 32 ? 1024 : 64;
  while (p.join_threads < kJoin * p.chunks && p.join_threads < 1024) p.join_threads *= 2;
  return p;
}

hipError_t launch_balance(const BalanceCall& c, hipStream_t s) {
  const BalancePlan p = balance_plan(c.N, c.T, c.E);
  BalanceArgs a{};
  a.N = c.N;
  a.T = p.T;
  a.E = c.E;
  a.k = c.k;
  a.S = p.S;
  a.chunk = p.chunk;
  a.chunks = p.chunks;
  a.weight = c.weight / (float)p.S;
  a.scores = c.scores;
  a.idx = c.idx;
  a.mask = c.mask;
  a.counts = c.counts;
  a.coef = c.coef;
  a.loss = c.loss;
  a.part_p = c.part_p;
  a.part_c = c.part_c;
  a.part_v = c.part_v;
  a.part_l = c.part_l;
  const bool few = p.S * p.join_parts <= kCountedBlocks;
  a.done = p.chunks > 1 && few ? c.done : nullptr;
  hipError_t e = with_shape(c.E, [&](auto g, auto pl, auto v) {
    hipLaunchKernelGGL((balance_chunks<decltype(g)::value, decltype(pl)::value, decltype(v)::value>),
                       dim3((unsigned)(p.S * p.chunks)), dim3(p.threads), 0, s, a);
    return hipGetLastError();
  });
  if (e == hipSuccess && p.chunks > 1) {
    hipLaunchKernelGGL(balance_join, dim3((unsigned)(p.S * p.join_parts)), dim3(p.join_threads), 0, s, a, p.join_parts);
    e = hipGetLastError();
  }
  if (e == hipSuccess && (p.chunks == 1 ? p.S > 1 : !few)) {
    hipLaunchKernelGGL(balance_total, dim3(1), dim3(1024), 0, s, (const float*)a.part_l,
                       p.chunks == 1 ? p.S : p.S * p.join_parts, a.loss);
    e = hipGetLastError();
  }
  return e;
}

int64_t route_backward_blocks(int64_t N, int E) { return (N + 256 / lanes_of(E) - 1) / (256 / lanes_of(E)); }

hipError_t launch_route_backward(const RouteBackCall& c, hipStream_t s) {
  RouteBackArgs a{c.N, c.T < c.N ? c.T : c.N, c.E, c.k, c.alpha, c.eps, c.norm, c.scores, c.idx, c.dw, c.coef, c.dloss, c.mask,
                  c.out};
  return with_shape(c.E, [&](auto g, auto pl, auto v) {
    hipLaunchKernelGGL((route_backward<decltype(g)::value, decltype(pl)::value, decltype(v)::value>),
                       dim3((unsigned)route_backward_blocks(c.N, c.E)), dim3(256), 0, s, a);
    return hipGetLastError();
  });
}

}  // namespace moe
