// The 2-norm over many tensors, and the tensors scaled to at most a given norm:
//
//   norm = sqrt(sum over all values of g^2)      out = g min(1, max_norm / (norm + eps))
//
// Squares and sums are float64: a square of a float32 is exact in it and cannot overflow, and the vector unit's
// float64 rate leaves the pass bound by HBM. Tensors of any length, type and alignment of their own are cut into
// chunks, one block each; a block finds its tensor in the launch's table (kernel arguments, so
// nothing has to outlive the call) by bisection. The clip walks the chunks backwards: what the norm's pass read last
// is still in the last-level cache (256 MiB). 290 M values of bfloat16 into float32: norm 92 us, the join of
// its partial sums 8, clip 284: 6.3 and 6.1 TB/s.
#include <hip/hip_runtime.h>

#include <utility>

#include "ops_internal.h"
#include "row_ops.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
// Pieces of eight values per thread and chunk of a long list (8 instead of 4: clip of 290 M float32 values 444 us, so 416;
// 2: norm of as many bfloat16 ones 133, so 100).
constexpr int kPieces = 4;
// Values of a chunk: 8,192, or 2,048 in lists of up to 4 M values, which would otherwise leave CUs without a block
// (1.6 M values: norm 6.0 -> 4.2, clip 7.0 -> 5.6 us).
int64_t chunk_values(int64_t all) { return (int64_t)kThreads * 8 * (all <= (int64_t)1 << 22 ? 1 : kPieces); }
constexpr int kTable = 100;  // tensors per launch: the table stays below the 4 KiB of kernel arguments

struct Table {
  const void* in[kTable];
  void* out[kTable];
  int64_t numel[kTable];
  int32_t first[kTable + 1];  // first chunk of each tensor; [n]: chunks in all
  uint8_t in_bf16[kTable], out_bf16[kTable];
  uint8_t skip[kTable];  // clip: values in front of the tensor that its first piece leaves out
  int n;
};
static_assert(sizeof(Table) <= 4000, "kernel arguments");

// Eight values at an address that has the alignment of their type alone.
template <typename T>
struct Unaligned8;
template <>
struct __attribute__((packed, aligned(2))) Unaligned8<uint16_t> {
  u32x4 v;
};
template <>
struct __attribute__((packed, aligned(4))) Unaligned8<float> {
  f32x4v a, b;
};
__device__ inline void load8u(const uint16_t* p, float* f) {
  widen8(Raw8<uint16_t>{((const Unaligned8<uint16_t>*)p)->v}, f);
}
__device__ inline void load8u(const float* p, float* f) {
  const auto* q = (const Unaligned8<float>*)p;
  widen8(Raw8<float>{q->a, q->b}, f);
}
// Four values, and stores of whole pieces: non-temporal, since the optimizer reads them after everything else is written.
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef f32x4v f32x4_any __attribute__((aligned(4)));
__device__ inline void load4u(const uint16_t* p, float* f) {
  const u32x2 v = *(const u32x2_any*)p;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
  }
}
__device__ inline void load4u(const float* p, float* f) {
  const f32x4v v = *(const f32x4_any*)p;
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = v[i];
}
__device__ inline void store4u(uint16_t* p, const float* f) {
  __builtin_nontemporal_store(u32x2{bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3])}, (u32x2_any*)p);
}
__device__ inline void store4u(float* p, const float* f) {
  __builtin_nontemporal_store(f32x4v{f[0], f[1], f[2], f[3]}, (f32x4_any*)p);
}
__device__ inline void store8u(uint16_t* p, const float* f) {
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = bf16_pair(f[2 * i], f[2 * i + 1]);
  __builtin_nontemporal_store(v, (u32x4_any*)p);
}
__device__ inline float load1(const uint16_t* p) { return bf16_f32(*p); }
__device__ inline float load1(const float* p) { return *p; }
__device__ inline void store1(uint16_t* p, float f) { *p = (uint16_t)(bf16_pair(f, 0.f) & 0xffffu); }
__device__ inline void store1(float* p, float f) { *p = f; }

// The tensor that holds chunk c (uniform over the block).
__device__ inline int tensor_of(const Table& t, int c) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= c)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Chunks begin at the tensor's first value wherever it lies, so that the order of the sums, and with it the norm's last bit,
// does not depend on its address. (290 M values of bfloat16 at an odd multiple of 2 bytes: 120 us, at any other address 98;
// float32: the same anywhere.)
template <typename T, int PIECES>
__device__ inline double chunk_squares(const T* p, int64_t n) {
  double s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = 0.0;
  if (n == kThreads * 8 * PIECES) {  // a whole chunk: every load in flight before the first sum
    float f[PIECES][8];
#pragma unroll
    for (int v = 0; v < PIECES; ++v) load8u(p + (threadIdx.x + v * kThreads) * 8, f[v]);
#pragma unroll
    for (int v = 0; v < PIECES; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] += (double)f[v][i] * (double)f[v][i];
  } else {
    for (int64_t at = threadIdx.x * 8; at < n; at += kThreads * 8) {
      float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (at + 8 <= n) {
        load8u(p + at, f);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (at + i < n) f[i] = load1(p + at + i);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] += (double)f[i] * (double)f[i];
    }
  }
  return ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
}

// Sum over the block in a fixed order, valid in thread 0.
__device__ inline double block_sum(double v, double* buf) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < (int)(blockDim.x >> 6); ++w) t += buf[w];
  return t;
}

template <int PIECES>
__global__ __launch_bounds__(kThreads) void norm_chunks(Table t, double* part) {
  __shared__ double buf[kThreads / 64];
  constexpr int64_t CHUNK = kThreads * 8 * PIECES;
  const int c = blockIdx.x, i = tensor_of(t, c);
  const int64_t at = (int64_t)(c - t.first[i]) * CHUNK, n = min(CHUNK, t.numel[i] - at);
  const double s = t.in_bf16[i] ? chunk_squares<uint16_t, PIECES>((const uint16_t*)t.in[i] + at, n)
                                : chunk_squares<float, PIECES>((const float*)t.in[i] + at, n);
  const double b = block_sum(s, buf);
  if (threadIdx.x == 0) part[c] = b;
}

__global__ __launch_bounds__(1024) void norm_total(const double* part, int64_t n, float* norm) {
  __shared__ double buf[16];
  double s[8] = {0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0};
  for (int64_t i = threadIdx.x; i < n; i += 8192) {
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] += i + 1024 * j < n ? part[i + 1024 * j] : 0.0;
  }
  const double b = block_sum(((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7])), buf);
  if (threadIdx.x == 0) *norm = (float)sqrt(b);
}

// A thread's values in a whole chunk: eight in a row where both sides are bfloat16, else four and four a wave's run apart,
// so that a load or store of float32 covers whole lines in one instruction (290 M values of bfloat16 into float32, norm
// and clip: 470 us with eight in a row and ordinary stores, 540 with non-temporal ones).
template <int PIECES, typename T, typename U>
__device__ inline void scale_chunk(const T* p, U* o, int64_t n, int skip, float scale) {
  constexpr int W = sizeof(T) == 2 && sizeof(U) == 2 ? 8 : 4, M = PIECES * 8 / W;
  if (n == kThreads * PIECES * 8 && skip == 0) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    auto place = [&](int m) {
      return W == 8 ? (m * kThreads + (int)threadIdx.x) * 8 : (m >> 1) * kThreads * 8 + wave * 512 + (m & 1) * 256 + lane * 4;
    };
    float f[M][W];
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if constexpr (W == 8)
        load8u(p + place(m), f[m]);
      else
        load4u(p + place(m), f[m]);
    }
#pragma unroll
    for (int m = 0; m < M; ++m) {
#pragma unroll
      for (int i = 0; i < W; ++i) f[m][i] *= scale;
      if constexpr (W == 8)
        store8u(o + place(m), f[m]);
      else
        store4u(o + place(m), f[m]);
    }
    return;
  }
  // the first and the last chunk of a tensor
  for (int64_t at = threadIdx.x * 4; at < n; at += kThreads * 4) {
    if (at >= skip && at + 4 <= n) {
      float f[4];
      load4u(p + at, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] *= scale;
      store4u(o + at, f);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (at + i >= skip && at + i < n) store1(o + at + i, load1(p + at + i) * scale);
    }
  }
}

template <int PIECES>
__global__ __launch_bounds__(kThreads) void clip_chunks(Table t, const float* norm, float max_norm, float eps,
                                                        int in_place) {
  constexpr int64_t CHUNK = kThreads * 8 * PIECES;
  const float total = *norm + eps, ratio = max_norm / total;
  const float scale = ratio >= 1.0f || total == 0.f ? 1.0f : ratio;  // 0 / 0 is not below 1; a NaN in norm stays one
  if (in_place && scale == 1.0f) return;
  const int c = t.first[t.n] - 1 - (int)blockIdx.x, i = tensor_of(t, c);
  const int64_t at = (int64_t)(c - t.first[i]) * CHUNK, n = min(CHUNK, t.numel[i] - at);
  const int skip = at == 0 ? t.skip[i] : 0;
  const uint16_t* pb = (const uint16_t*)t.in[i] + at;
  const float* pf = (const float*)t.in[i] + at;
  uint16_t* ob = (uint16_t*)t.out[i] + at;
  float* of = (float*)t.out[i] + at;
  if (t.in_bf16[i])
    t.out_bf16[i] ? scale_chunk<PIECES>(pb, ob, n, skip, scale) : scale_chunk<PIECES>(pb, of, n, skip, scale);
  else
    t.out_bf16[i] ? scale_chunk<PIECES>(pf, ob, n, skip, scale) : scale_chunk<PIECES>(pf, of, n, skip, scale);
}

// The clip walks a tensor from the start of the 128-byte line that it begins in, so that the blocks' loads and stores cover
// whole lines (non-temporal stores of float32 that straddle lines made norm and clip of 290 M values 429 us, 391 without).
int lead_of(const moe_tensor& t) {
  return t.numel == 0 ? 0 : (int)((uintptr_t)t.data & 127) / (t.dtype == MOE_BF16 ? 2 : 4);
}
int64_t chunks_of(const moe_tensor& t, int lead, int64_t chunk) {
  return t.numel == 0 ? 0 : (t.numel + lead + chunk - 1) / chunk;
}
int64_t all_values(const moe_tensor* t, int n) {
  int64_t all = 0;
  for (int i = 0; i < n; ++i) all += t[i].numel;
  return all;
}

// Tables of up to kTable tensors and kMost chunks (a longer tensor is cut); f(table, the chunks of the tables before it).
// For the clip from the last tensor to the first, each from the start of its line.
template <typename F>
hipError_t for_tables(const moe_tensor* in, const moe_tensor* out, int n, int64_t chunk, bool clip, F f) {
  constexpr int64_t kMost = (int64_t)1 << 22;
  int i = clip ? n - 1 : 0;  // the tensor at hand, and how many of its chunks earlier tables hold
  int64_t cut = 0, before = 0;
  Table t;
  while (i >= 0 && i < n) {
    int64_t count = 0, size[kTable];
    t.n = 0;
    for (; i >= 0 && i < n && t.n < kTable && count < kMost; ) {
      const moe_tensor& o = out ? out[i] : in[i];
      const int64_t lead = clip ? lead_of(o) : 0, values = in[i].numel + lead;
      const int64_t left = chunks_of(in[i], (int)lead, chunk) - cut, take = left < kMost - count ? left : kMost - count;
      if (take > 0) {
        const int j = t.n++;
        // whole tables leave the end of a tensor to the next one, or in the clip its beginning
        const int64_t at = (clip ? left - take : cut) * chunk;
        t.in_bf16[j] = in[i].dtype == MOE_BF16;
        t.out_bf16[j] = o.dtype == MOE_BF16;
        t.in[j] = (const char*)in[i].data + (at - lead) * (t.in_bf16[j] ? 2 : 4);
        t.out[j] = (char*)o.data + (at - lead) * (t.out_bf16[j] ? 2 : 4);
        t.numel[j] = values - at < take * chunk ? values - at : take * chunk;
        t.skip[j] = at == 0 ? (uint8_t)lead : 0;
        size[j] = take;
        count += take;
      }
      if (take < left) {
        cut += take;
        break;
      }
      cut = 0;
      i += clip ? -1 : 1;
    }
    if (t.n == 0) break;
    if (clip) {
      for (int a = 0, b = t.n - 1; a < b; ++a, --b) {
        std::swap(t.in[a], t.in[b]);
        std::swap(t.out[a], t.out[b]);
        std::swap(t.numel[a], t.numel[b]);
        std::swap(t.in_bf16[a], t.in_bf16[b]);
        std::swap(t.out_bf16[a], t.out_bf16[b]);
        std::swap(t.skip[a], t.skip[b]);
        std::swap(size[a], size[b]);
      }
    }
    t.first[0] = 0;
    for (int j = 0; j < t.n; ++j) t.first[j + 1] = (int32_t)(t.first[j] + size[j]);
    const hipError_t e = f(t, before, count);
    if (e != hipSuccess) return e;
    before += count;
  }
  return hipSuccess;
}

}  // namespace

int64_t tensor_chunks(const moe_tensor* t, int n) {
  const int64_t chunk = chunk_values(all_values(t, n));
  int64_t c = 0;
  for (int i = 0; i < n; ++i) c += chunks_of(t[i], 0, chunk);
  return c;
}

hipError_t launch_grad_norm(const moe_tensor* t, int n, double* part, float* norm, hipStream_t s) {
  const int64_t chunk = chunk_values(all_values(t, n));
  int64_t chunks = 0;
  const hipError_t e = for_tables(t, nullptr, n, chunk, false, [&](const Table& tab, int64_t before, int64_t count) {
    if (chunk == kThreads * 8)
      hipLaunchKernelGGL(norm_chunks<1>, dim3((unsigned)count), dim3(kThreads), 0, s, tab, part + before);
    else
      hipLaunchKernelGGL(norm_chunks<kPieces>, dim3((unsigned)count), dim3(kThreads), 0, s, tab, part + before);
    chunks = before + count;
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(norm_total, dim3(1), dim3(1024), 0, s, (const double*)part, chunks, norm);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const moe_tensor* t, const moe_tensor* out, int n, const float* norm, float max_norm,
                            float eps, hipStream_t s) {
  const int64_t chunk = chunk_values(all_values(t, n));
  return for_tables(t, out, n, chunk, true, [&](const Table& tab, int64_t, int64_t count) {
    if (chunk == kThreads * 8)
      hipLaunchKernelGGL(clip_chunks<1>, dim3((unsigned)count), dim3(kThreads), 0, s, tab, norm, max_norm, eps, out ? 0 : 1);
    else
      hipLaunchKernelGGL(clip_chunks<kPieces>, dim3((unsigned)count), dim3(kThreads), 0, s, tab, norm, max_norm, eps,
                         out ? 0 : 1);
    return hipGetLastError();
  });
}

}  // namespace moe
