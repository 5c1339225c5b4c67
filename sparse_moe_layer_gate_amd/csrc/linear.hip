// Dense linear maps with bias, activation and residual in the epilogue:
//
//   z = x W^T + bias      y = act(z) + residual
//
// Both operands are contiguous in the reduction index (W is [out, in] row-major). Forms, picked by linear_plan:
//  - linear_few (both types, up to 16 rows, and up to 64 where x is small): a stream of W, the reduction split over a
//    block's waves;
//  - linear_w8 (bfloat16, many rows): 256 x 256 tiles of eight waves in the expert GEMMs' layout (gemm_w8.h), a static
//    walk over the tiles, one block per CU;
//  - linear_tile (both types): 64 rows (bfloat16: to 256) x 64 or 128 columns, the reduction split over blocks where the
//    tiles alone would not fill the CUs; linear_join then adds the parts in order and runs the epilogue.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
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

// Cache policy of weights that are read once per call: non-temporal (the NT bit, 2 on gfx950).
constexpr int kStreamW = 2;

// Waits until at most min(n, MOST) steps of PER loads each are in flight.
template <int PER, int MOST>
__device__ inline void wait_steps(int n) {
  if constexpr (MOST == 0) {
    wait_vmcnt<0>();
  } else {
    if (n >= MOST)
      wait_vmcnt<PER * MOST>();
    else
      wait_steps<PER, MOST - 1>(n);
  }
}

// ---- up to 64 rows ----
//
// A stream of W: a block holds 16 columns, its waves a run of the reduction each, with a ring of their own and no barrier
// until the end, where their sums meet in LDS. A step is 128 bytes of every row, whole lines per load, as in the tiles
// below; of x only the first 8 NX rows are copied, and what the products make of the others is not stored. Bound by HBM
// with few rows (1 x 5,120 -> 12,288 in bfloat16: 20 us, 6.3 TB/s of W), with more by x, copied for every 16 columns.
template <typename T, int NX, int NW, int S>
struct LinFew {
  static constexpr int STAGE = (2 + NX) * 1024, PER = 2 + NX;
  static constexpr int LDS = NW * S * STAGE;
  static constexpr int TM = (NX + 1) / 2;  // 16-row tiles
  static_assert(LDS <= 80 * 1024 && LDS >= NW * TM * 1024 && TM <= NW, "two blocks per CU; the sums, a tile per wave");
};

template <typename T, int NX, int NW, int S>
__global__ __launch_bounds__(64 * NW) void linear_few(LinArgs<T> a) {
  using L = LinFew<T, NX, NW, S>;
  constexpr bool BF16 = std::is_same<T, uint16_t>::value;
  __shared__ __attribute__((aligned(1024))) char lds[L::LDS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int col0 = (int)blockIdx.x * 16, rows = (int)a.R;
  const int nk_all = a.K / (128 / (int)sizeof(T));
  const int k0 = nk_all * wave / NW, nk = nk_all * (wave + 1) / NW - k0;
  // rows past the end repeat the last one
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc((void*)a.x, (short)0, -1, kRawBufferWord3);
  const __amdgpu_buffer_rsrc_t rb =
      __builtin_amdgcn_make_buffer_rsrc((void*)(a.w + (int64_t)col0 * a.K), (short)0, -1, kRawBufferWord3);
  auto swz = [](int r) { return (r >> 1) & 7; };
  constexpr int TM = L::TM;
  uint32_t ox[NX], ow[2];
#pragma unroll
  for (int i = 0; i < NX; ++i) {
    const int r = 8 * i + (lane >> 3), c = (lane & 7) ^ swz(r);
    ox[i] = (uint32_t)min(r, rows - 1) * (uint32_t)(a.K * (int)sizeof(T)) + 16 * c;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 8 * i + (lane >> 3), c = (lane & 7) ^ swz(r);
    ow[i] = (uint32_t)min(r, a.M - 1 - col0) * (uint32_t)(a.K * (int)sizeof(T)) + 16 * c;
  }
  char* const ring = lds + wave * (S * L::STAGE);
  int put = 0, get = 0, at = k0 * 128;
  auto issue = [&] {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(ring + put + i * 1024), 16, (int)ow[i], at, 0, kStreamW);
#pragma unroll
    for (int i = 0; i < NX; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(ring + put + (2 + i) * 1024), 16, (int)ox[i], at, 0, 0);
    put = put == (S - 1) * L::STAGE ? 0 : put + L::STAGE;
    at += 128;
  };
  const int r16 = lane & 15, kq = lane >> 4;
  int fw[2], fx[TM][2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    fw[h] = r16 * 128 + 16 * ((4 * h + kq) ^ swz(r16));
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      const int r = NX == 1 ? r16 & 7 : 16 * j + r16;
      fx[j][h] = 2048 + r * 128 + 16 * ((4 * h + kq) ^ swz(r));
    }
  }
  typedef typename std::conditional<BF16, bf16x8, f32x4>::type frag;
  f32x4 acc[TM];
#pragma unroll
  for (int j = 0; j < TM; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto step = [&](bool refill) {
    frag w[2], x[TM][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      w[h] = *(const frag*)(ring + get + fw[h]);
#pragma unroll
      for (int j = 0; j < TM; ++j) x[j][h] = *(const frag*)(ring + get + fx[j][h]);
    }
    get = get == (S - 1) * L::STAGE ? 0 : get + L::STAGE;
    wait_lgkm0();  // in registers: the stage may be refilled
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    if (refill) issue();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int u = 0; u < (BF16 ? 1 : 4); ++u)
#pragma unroll
        for (int j = 0; j < TM; ++j) {
          if constexpr (BF16)
            acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[h], x[j][h], acc[j], 0, 0, 0);
          else
            acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(w[h][u], x[j][h][u], acc[j], 0, 0, 0);
        }
    }
  };
  const int ahead = min(S, nk);
  for (int t = 0; t < ahead; ++t) issue();
  int t = 0;
  for (; t + S < nk; ++t) {
    wait_vmcnt<(S - 1) * L::PER>();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    step(true);
  }
  for (; t < nk; ++t) {
    wait_steps<L::PER, S - 1>(nk - 1 - t);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    step(false);
  }
  __syncthreads();  // every ring has been read
  f32x4* sums = (f32x4*)lds;
#pragma unroll
  for (int j = 0; j < TM; ++j) sums[(wave * TM + j) * 64 + lane] = acc[j];
  __syncthreads();
  const int col = col0 + 4 * kq, row = 16 * wave + r16;  // wave j ends the j-th tile
  if (wave >= TM || row >= rows || col >= a.M) return;
  f32x4 sum = sums[wave * 64 + lane];
#pragma unroll
  for (int w = 1; w < NW; ++w) sum += sums[(w * TM + wave) * 64 + lane];
  float v[4] = {sum[0], sum[1], sum[2], sum[3]}, bias[4];
  load_bias<4>(a, col, bias);
  epilogue<4>(a, row, col, v, bias);
}

// ---- tiles of 64 to 256 rows x 64 or 128 columns ----
//
// Eight waves, two per SIMD. A step covers 128 bytes of every row of x and of W in the tile (64 k of bfloat16, 32 of
// float32; whole lines per load), copied global -> LDS by direct loads into a ring of S stages, chunk-swizzled. Waves 0-3
// multiply the first half of each step and waves 4-7 the second, each wave a quarter of the tile,
// so that a wave's share is as large as the registers allow and LDS is read least; at the end the halves exchange sums.
//  - One barrier per step: behind it the next step has landed and every wave has read the present one into registers,
//    so its stage is refilled at once, and the next fragments are read while the present products run.
//  - The steps that refill run in a loop of their own, free of branches and with a fixed wait: with the conditions of
//    the last steps inside, a step of little work took 0.42 us of branches alone.
//  - W rows are the first operand of the products, so that a lane ends up with four consecutive output columns of one
//    row. A lane of both operands holds the 16 bytes of one chunk of its row: eight k of v_mfma_f32_16x16x32_bf16, or
//    four k that four steps of v_mfma_f32_16x16x4_f32 take one by one (which k of a chunk meet in one step does not
//    matter as long as both operands agree).
// In bfloat16 with few rows bound by the loads into LDS, x's for every BN columns among them (201 x 12,288 -> 5,120 with
// 128 x 128 tiles in three parts: 45 us, matrix cores 28% busy, 2.8 TB/s of W; 5 us for the join), in float32
// by the matrix cores (1,000 x 1,536 -> 4,096: 96 us back to back, 103 in a kernel trace, 78% busy).
template <typename T, int BM_, int BN_>
struct LinTile {
  static constexpr int BM = BM_, BN = BN_;
  static constexpr int WM = 2, WN = 2;
  static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
  static constexpr int BK = 128 / (int)sizeof(T);  // elements of a 128-byte row
  static constexpr int NA = BM / 64, NB = BN / 64, PER = NA + NB;  // direct loads per wave and step (8 rows each)
  static constexpr int STAGE = (BM + BN) * 128;
  static constexpr int S = BM == 128 || BN == 64 ? 4 : 3;  // BM = 64: two blocks per CU
  static constexpr int XCH = 8 * (TM * TN / 2) * 1024;  // the exchange of sums
  static constexpr int LDS = S * STAGE > XCH ? S * STAGE : XCH;
  static_assert(LDS <= 160 * 1024 && TM % 2 == 0, "LDS; the halves end half the tiles each");
  // Over the 16 rows of a fragment no two of the lanes that LDS serves together share banks (with the pattern of gemm_w8.h,
  // made for 32 rows, half the cycles of the reads were conflicts).
  __device__ static int swz(int r) { return (r >> 1) & 7; }
};

template <typename T, int BM, int BN>
__global__ __launch_bounds__(512) void linear_tile(LinArgs<T> a) {
  using L = LinTile<T, BM, BN>;
  constexpr int TM = L::TM, TN = L::TN, NA = L::NA, NB = L::NB, S = L::S;
  __shared__ __attribute__((aligned(1024))) char lds[L::LDS];
  // splits outermost (an XCD's run of blocks then shares one part of x in its L2), row tiles innermost (blocks on the
  // same rows of W run together)
  const int64_t id = xcd_logical_block(gridDim.x);
  const int64_t rt = id % a.row_tiles, rest = id / a.row_tiles;
  const int ct = (int)(rest % a.col_tiles), split = (int)(rest / a.col_tiles);
  const int64_t row0 = rt * BM;
  const int col0 = ct * BN;
  const int rows = (int)min((int64_t)BM, a.R - row0);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int half = wave >> 2, wm = (wave >> 1) & 1, wn = wave & 1;
  const int nk_all = a.K / L::BK;
  const int k0 = (int)((int64_t)nk_all * split / a.splits), nk = (int)((int64_t)nk_all * (split + 1) / a.splits) - k0;

  // A load covers eight rows; this wave's i-th those from (wave + 8 i) 8 on. Rows past the end repeat the last one (never
  // stored); offsets are from the tile's first row and stay below 2^32.
  const __amdgpu_buffer_rsrc_t ra =
      __builtin_amdgcn_make_buffer_rsrc((void*)(a.x + row0 * a.K), (short)0, -1, kRawBufferWord3);
  const __amdgpu_buffer_rsrc_t rb =
      __builtin_amdgcn_make_buffer_rsrc((void*)(a.w + (int64_t)col0 * a.K), (short)0, -1, kRawBufferWord3);
  uint32_t oa[NA], ob[NB];
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    const int r = (wave + 8 * i) * 8 + (lane >> 3), c = (lane & 7) ^ L::swz(r);
    oa[i] = (uint32_t)min(r, rows - 1) * (uint32_t)(a.K * (int)sizeof(T)) + 16 * c;
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int r = (wave + 8 * i) * 8 + (lane >> 3), c = (lane & 7) ^ L::swz(r);
    ob[i] = (uint32_t)min(r, a.M - 1 - col0) * (uint32_t)(a.K * (int)sizeof(T)) + 16 * c;
  }
  // byte offsets: the stage to fill next, the step's place in a row. The columns' tiles begin at different steps of their
  // part and go round: where rows of W lie a multiple of 8 KiB apart, all of them would ask the same few memory channels at
  // one step (12,288 -> 5,120 with 40 rows 36 -> 31 us, with 128 40 -> 37)
  int put = 0, at = (k0 + (int)((int64_t)nk * ct / a.col_tiles)) * 128;
  auto load = [&](int i) {  // the i-th of a step's PER loads
    char* st = lds + put + wave * 1024 + i * 8192;  // W's rows lie behind x's
    if (i < NA)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)st, 16, (int)oa[i < NA ? i : 0], at, 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)st, 16, (int)ob[i < NA ? 0 : i - NA], at, 0, 0);
  };
  auto loaded = [&] {
    put = put + L::STAGE == S * L::STAGE ? 0 : put + L::STAGE;
    at = at + 128 == (k0 + nk) * 128 ? k0 * 128 : at + 128;
  };
  auto issue = [&] {
#pragma unroll
    for (int i = 0; i < L::PER; ++i) load(i);
    loaded();
  };

  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int r16 = lane & 15, kq = lane >> 4;
  // fragment addresses: 16-row tiles lie 2 KiB apart
  const int fc = r16 * 128 + 16 * ((4 * half + kq) ^ L::swz(r16));
  const int fa = wm * TM * 2048 + fc, fb = BM * 128 + wn * TN * 2048 + fc;
  typedef typename std::conditional<std::is_same<T, uint16_t>::value, bf16x8, f32x4>::type frag;
  frag av[2][TM], bv[2][TN];
  constexpr int FRAGS = TM + TN;
  constexpr int PRODUCTS = TM * TN * (std::is_same<T, uint16_t>::value ? 1 : 4);
  int get = 0;  // byte offset of the stage to read next
  auto read_one = [&](auto buf, int f) {  // the f-th of a step's FRAGS fragments
    constexpr int b = decltype(buf)::value;
    if (f < TN)
      bv[b][f] = *(const frag*)(lds + get + fb + f * 2048);
    else
      av[b][f - TN] = *(const frag*)(lds + get + fa + (f - TN) * 2048);
  };
  auto got = [&] { get = get + L::STAGE == S * L::STAGE ? 0 : get + L::STAGE; };
  auto read = [&](auto buf) {
#pragma unroll
    for (int f = 0; f < FRAGS; ++f) read_one(buf, f);
    got();
  };
  auto product = [&](auto buf, int m) {  // the m-th of a step's PRODUCTS
    constexpr int b = decltype(buf)::value;
    const int i = m % (TM * TN) / TN, j = m % TN;
    if constexpr (std::is_same<T, uint16_t>::value)
      acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv[b][j], av[b][i], acc[i][j], 0, 0, 0);
    else
      acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(bv[b][j][m / (TM * TN)], av[b][i][m / (TM * TN)], acc[i][j], 0, 0, 0);
  };
  auto products = [&](auto buf) {
#pragma unroll
    for (int m = 0; m < PRODUCTS; ++m) product(buf, m);
  };
  auto fence = [] { __builtin_amdgcn_sched_barrier(0); };
  // LIVE: the wave has rows at all (one without keeps loading and meeting the others)
  auto loop = [&](auto live) {
    constexpr bool LIVE = decltype(live)::value;
    const int ahead = min(S, nk);
    for (int t = 0; t < ahead; ++t) issue();
    wait_steps<L::PER, S - 1>(ahead - 1);
    bare_barrier();
    if (LIVE) read(IntC<0>{});
    int t = 0;
    auto steady = [&](auto buf) {  // step t is being read into buf; steps up to t + S - 1 are issued
      wait_lgkm0();
      wait_vmcnt<L::PER*(S - 2)>();
      bare_barrier();
      fence();
      if (LIVE) {
        // one fragment read or load at a time, the products spread evenly behind them: the wave would otherwise stand
        // at its reads until LDS had taken all of them, its matrix core idle
        constexpr int OPS = FRAGS + L::PER;
#pragma unroll
        for (int o = 0; o < OPS; ++o) {
          const int loads = (o + 1) * L::PER / OPS;
          if (loads != o * L::PER / OPS)
            load(loads - 1);
          else
            read_one(IntC<1 - decltype(buf)::value>{}, o - loads);
          fence();
#pragma unroll
          for (int m = o * PRODUCTS / OPS; m < (o + 1) * PRODUCTS / OPS; ++m) product(buf, m);
          fence();
        }
        loaded();
        got();
      } else {
        issue();
        got();
      }
      fence();
    };
    for (; t + S + 1 < nk; t += 2) {
      steady(IntC<0>{});
      steady(IntC<1>{});
    }
    auto tail = [&](int t, auto buf) {
      if (t + 1 < nk) {
        wait_lgkm0();
        wait_steps<L::PER, S - 2>(min(nk - 1, t + S - 1) - (t + 1));
        bare_barrier();
        if (t + S < nk) issue();
        fence();
        if (LIVE) read(IntC<1 - decltype(buf)::value>{});
      }
      fence();
      if (LIVE) products(buf);
      fence();
    };
    for (; t < nk; t += 2) {
      tail(t, IntC<0>{});
      if (t + 1 < nk) tail(t + 1, IntC<1>{});
    }
  };
  if (wm * TM * 16 < rows)
    loop(BoolC<true>{});
  else
    loop(BoolC<false>{});

  // The halves' sums: waves 0-3 end with the first TM / 2 tile rows, waves 4-7 with the others.
  constexpr int HT = TM / 2;
  f32x4* mine = (f32x4*)lds + (wave * HT * TN) * 64 + lane;
  f32x4* theirs = (f32x4*)lds + ((wave ^ 4) * HT * TN) * 64 + lane;
  __syncthreads();  // the last fragments have been read
#pragma unroll
  for (int i = 0; i < HT; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) mine[(i * TN + j) * 64] = half == 0 ? acc[i + HT][j] : acc[i][j];
  __syncthreads();
  f32x4 sum[HT][TN];
#pragma unroll
  for (int i = 0; i < HT; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const f32x4 other = theirs[(i * TN + j) * 64];
      sum[i][j] = half == 0 ? acc[i][j] + other : other + acc[i + HT][j];
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
    for (int i = 0; i < HT; ++i) {
      const int r = (wm * TM + half * HT + i) * 16 + r16;
      if (r >= rows) continue;
      float v[4] = {sum[i][j][0], sum[i][j][1], sum[i][j][2], sum[i][j][3]};
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
// activation and residual are applied there, with whole 16-byte loads and stores, and y is rounded once. Bound by the
// matrix cores: 8,191 x 5,120 -> 12,288 with gelu and z 814 to 823 us, 1,250 to 1,270 TFLOP/s,
// 71% busy.
constexpr int kStagePitch = 128 + 8;  // floats: rows four apart, which one store writes together, lie 32 banks apart

// The K loop of one wave on the ring of Wave8Tile (two stages of x rows, three of W rows): the wave's 64 rows x 128
// columns as MI x 4 tiles. Between two barriers a wave multiplies the last 16-wide slice of step kt and the first three
// of step kt + 1, each while it reads the next slice's fragments, and issues its loads of x for step kt + 2 and of W for
// step kt + 3, whose stages every wave has left when the barrier opens. One read or load at a time, the products spread
// behind them: issued together, the reads of a slice hold the wave until LDS has taken all of them, and the matrix core
// waits. na: the wave's loads of x that reach a valid row (the others are not issued; W's always are, so the newest
// four loads are W's).
template <int MI>
__device__ __attribute__((always_inline)) inline void w8_spread_loop(char* lds, __amdgpu_buffer_rsrc_t ra,
                                                                     const uint32_t (&oa)[4], int na,
                                                                     __amdgpu_buffer_rsrc_t rb, const uint32_t (&ob)[4],
                                                                     f32x16 (&acc)[2][4], int nk, int grp, int q, int lane,
                                                                     int m0, int wn) {
  using T = Wave8Tile<false>;
  constexpr int TN = 4, ROWB = T::ROWB, OPB = T::OPB;
  const int sw = T::swz(lane & 31);
  const int a_off = (m0 + (lane & 31)) * ROWB;
  const int b_off = T::B_BASE + (wn * 128 + (lane & 31)) * ROWB;  // column tiles lie 32 rows apart
  int coff[4];
#pragma unroll
  for (int sl = 0; sl < 4; ++sl) coff[sl] = ((2 * sl + (lane >> 5)) ^ sw) * 16;
  const int fill = grp * (OPB / 2) + q * 1024;  // this wave's first chunk run in a stage
  int a_put = 0, b_put = 0, a_at = 0, b_at = 0;  // stages to fill next (bytes), places in a row of their steps
  auto load_a = [&](int i) {
    if (i < na)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(lds + a_put + fill + i * 4096), 16, (int)oa[i], a_at, 0, 0);
  };
  auto load_b = [&](int i) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(lds + T::B_BASE + b_put + fill + i * 4096), 16, (int)ob[i], b_at,
                                             0, 0);
  };
  auto loaded_a = [&] {
    a_put ^= OPB;
    a_at += 128;
  };
  auto loaded_b = [&] {
    b_put = b_put == 2 * OPB ? 0 : b_put + OPB;
    b_at += 128;
  };
  bf16x8 af[2][MI > 0 ? MI : 1], bfr[2][TN];
  int a_get = 0, b_get = 0;
  auto read_one = [&](int sl, int f) {  // the f-th fragment of slice sl, into buffer sl % 2
    if (MI == 0) return;
    if (f < TN)
      bfr[sl & 1][f] = *(const bf16x8*)(lds + b_get + b_off + f * 32 * ROWB + coff[sl]);
    else
      af[sl & 1][f - TN] = *(const bf16x8*)(lds + a_get + a_off + (f - TN) * 32 * ROWB + coff[sl]);
  };
  auto next_stage = [&] {
    a_get ^= OPB;
    b_get = b_get == 2 * OPB ? 0 : b_get + OPB;
  };
  auto fence = [] { __builtin_amdgcn_sched_barrier(0); };
  // the products of slice `cur`, the reads of slice `next` and `loads` loads among them
  auto phase = [&](auto cur_, auto next_, auto loads_, auto&& load) {
    constexpr int cur = decltype(cur_)::value, next = decltype(next_)::value, loads = decltype(loads_)::value;
    constexpr int FR = MI > 0 ? MI + TN : 0, OPS = FR + loads > 0 ? FR + loads : 1, P = MI * TN;
    wait_lgkm0();  // slice `cur` is in registers
    fence();
#pragma unroll
    for (int o = 0; o < OPS; ++o) {
      if (o < FR)
        read_one(next, o);
      else if (o - FR < loads)
        load(o - FR);
      fence();
#pragma unroll
      for (int m = o * P / OPS; m < (o + 1) * P / OPS; ++m)
        acc[m / TN][m % TN] =
            __builtin_amdgcn_mfma_f32_32x32x16_bf16(af[cur & 1][m / TN], bfr[cur & 1][m % TN], acc[m / TN][m % TN], 0, 0, 0);
      fence();
    }
  };
  auto compute = [&](auto cur_) {
    constexpr int cur = decltype(cur_)::value;
#pragma unroll
    for (int m = 0; m < MI * TN; ++m)
      acc[m / TN][m % TN] =
          __builtin_amdgcn_mfma_f32_32x32x16_bf16(af[cur & 1][m / TN], bfr[cur & 1][m % TN], acc[m / TN][m % TN], 0, 0, 0);
  };
  auto all_a = [&] {
#pragma unroll
    for (int i = 0; i < 4; ++i) load_a(i);
    loaded_a();
  };
  auto all_b = [&] {
#pragma unroll
    for (int i = 0; i < 4; ++i) load_b(i);
    loaded_b();
  };
  auto none = [](int) {};
  const IntC<0> c0;
  const IntC<1> c1;
  const IntC<2> c2;
  const IntC<3> c3;
  const IntC<4> c4;

  // steps 0 and 1 of both operands, step 2 of W; wait for step 0
  all_a();
  all_b();
  if (nk > 1) {
    all_a();
    all_b();
  }
  if (nk > 2) all_b();
  // x of step 1 may not have been issued by this wave at all: only W's loads can be counted on
  if (nk > 2)
    wait_vmcnt<8>();
  else if (nk > 1)
    wait_vmcnt<4>();
  else
    wait_vmcnt<0>();
  bare_barrier();
#pragma unroll
  for (int f = 0; f < (MI > 0 ? MI + TN : 0); ++f) read_one(0, f);
  phase(c0, c1, c0, none);
  phase(c1, c2, c0, none);
  phase(c2, c3, c0, none);
  // steps kt and kt + 1: x of kt + 2 and W of kt + 3 are issued
  int kt = 0;
  for (; kt + 3 < nk; ++kt) {
    wait_lgkm0();
    wait_vmcnt<4>();  // all but W of step kt + 2 has landed
    bare_barrier();
    next_stage();
    phase(c3, c0, c4, load_a);
    loaded_a();
    phase(c0, c1, c2, load_b);
    phase(c1, c2, c2, [&](int i) { load_b(i + 2); });
    loaded_b();
    phase(c2, c3, c0, none);
  }
  for (; kt + 1 < nk; ++kt) {
    wait_lgkm0();
    if (kt + 2 < nk)
      wait_vmcnt<4>();
    else
      wait_vmcnt<0>();
    bare_barrier();
    next_stage();
    if (kt + 2 < nk) all_a();
    phase(c3, c0, c0, none);
    phase(c0, c1, c0, none);
    phase(c1, c2, c0, none);
    phase(c2, c3, c0, none);
  }
  wait_lgkm0();
  fence();
  compute(c3);
  bare_barrier();  // every wave has read its last fragments
}

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
      w8_spread_loop<2>(lds, ra, oa, na, rb, ob, acc, nk, grp, q, lane, m0, wn);
    else if (mi == 1)
      w8_spread_loop<1>(lds, ra, oa, na, rb, ob, acc, nk, grp, q, lane, m0, wn);
    else
      w8_spread_loop<0>(lds, ra, oa, na, rb, ob, acc, nk, grp, q, lane, m0, wn);

    // each wave in its own part of the ring (the loop ends on a barrier behind the last read)
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
template <typename T, int BM, int BN>
hipError_t run_tile(const LinArgs<T>& a, hipStream_t s) {
  const int64_t blocks = a.row_tiles * a.col_tiles * a.splits;
  hipLaunchKernelGGL((linear_tile<T, BM, BN>), dim3((unsigned)blocks), dim3(512), 0, s, a);
  return hipGetLastError();
}

template <typename T>
hipError_t run_few(const LinArgs<T>& a, hipStream_t s) {
  const dim3 grid((a.M + 15) / 16);
  if (a.R <= 8)
    hipLaunchKernelGGL((linear_few<T, 1, 8, 3>), grid, dim3(512), 0, s, a);
  else if (a.R > 48)
    hipLaunchKernelGGL((linear_few<T, 8, 4, 2>), grid, dim3(256), 0, s, a);
  else if (a.R > 32)
    hipLaunchKernelGGL((linear_few<T, 6, 4, 2>), grid, dim3(256), 0, s, a);
  else if (a.R > 16)
    hipLaunchKernelGGL((linear_few<T, 4, 4, 3>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((linear_few<T, 2, 4, 4>), grid, dim3(256), 0, s, a);
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
  if (p.bm == 16) return run_few<T>(a, s);
  if constexpr (std::is_same<T, uint16_t>::value) {
    if (p.bn == 256) {
      const int64_t grid = std::min((a.row_tiles * a.col_tiles + 7) / 8 * 8, persistent_grid());
      hipLaunchKernelGGL(linear_w8, dim3((unsigned)grid), dim3(512), 0, s, a);
      return hipGetLastError();
    }
    if (p.bm == 256) e = run_tile<T, 256, 128>(a, s);
    if (p.bm == 128) e = run_tile<T, 128, 128>(a, s);
  }
  if (p.bm == 64) e = p.bn == 64 ? run_tile<T, 64, 64>(a, s) : run_tile<T, 64, 128>(a, s);
  if (e != hipSuccess || p.splits == 1) return e;
  hipLaunchKernelGGL(linear_join<T>, dim3((unsigned)((c.R * (c.out / 8) + 255) / 256)), dim3(256), 0, s, a);
  return hipGetLastError();
}

// ---- the gradients of the epilogue ----
//
// Eight columns per thread, up to 64 lanes per row, several rows per wave where the rows are narrower. A block takes the
// rows of every runs-th step, so that the blocks at work lie side by side in memory; its column sums go to one row of the
// partial array, which launch_column_sums adds in order. One row of a lane in flight and not four, whose unrolled
// exponentials also made small float32 calls twice as long: 8,192 x 12,288 in bfloat16 134 -> 119 us, 131,072 x 1,024 in
// float32 355 -> 295. Bound by HBM: 4,096 x 12,288 in bfloat16 with gelu 58 us and 4.5 for the join, 5.2 TB/s.
// The blocks of a large call have as many bytes in flight in both types (524,288 x 256 with 1,024 blocks: bfloat16
// 169 us for 160, float32 319 for 300).
constexpr int kBackBlocks = 1536, kBackBlocksF32 = 768;

int back_lanes(int M) {
  int lanes = 1;
  while (lanes < 64 && lanes * 8 < M) lanes *= 2;
  return lanes;
}

template <typename T>
__global__ __launch_bounds__(256) void linear_back(int64_t R, int M, int act, const T* dy, const T* z, T* dz, float* part,
                                                   int64_t runs, int lanes) {
  __shared__ float join[4][512];
  const int wave = threadIdx.x >> 6, rows = 256 / lanes;  // of a step
  const int64_t run = blockIdx.x % runs;
  const int first_col = (int)(blockIdx.x / runs) * 512, c8 = (threadIdx.x & (lanes - 1)) * 8, col = first_col + c8;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (col < M) {
    for (int64_t n = run * rows + threadIdx.x / lanes; n < R; n += runs * rows) {
      const int64_t at = n * M + col;
      const Raw8<T> rd = raw_load8(dy + at);
      float d[8], v[8];
      if (act != MOE_ACT_NONE) {
        const Raw8<T> rz = raw_load8(z + at);
        widen8(rd, d);
        widen8(rz, v);
        act_slope_times<std::is_same<T, uint16_t>::value, 8>(act, v, d);
      } else {
        widen8(rd, d);
      }
      if (dz) raw_store8<false>(dz + at, d);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += d[i];
    }
  }
  if (!part) return;
  for (int off = lanes; off < 64; off <<= 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += __shfl_xor(sum[i], off);
  }
  if ((threadIdx.x & 63) < lanes) raw_store8<false>(&join[wave][c8], sum);
  __syncthreads();
  for (int c = threadIdx.x; c < 512; c += 256) {
    if (first_col + c < M) part[run * M + first_col + c] = ((join[0][c] + join[1][c]) + join[2][c]) + join[3][c];
  }
}

template <typename T>
hipError_t linear_back_t(const LinearBackCall& c, hipStream_t s) {
  const int rows = 256 / back_lanes(c.out);
  const int dtype = std::is_same<T, float>::value ? MOE_F32 : MOE_BF16;
  const int64_t steps = (c.R + rows - 1) / rows, most = linear_back_runs(dtype, c.R, c.out);
  const int64_t each = (steps + most - 1) / most, runs = (steps + each - 1) / each;  // as many steps for each block
  hipLaunchKernelGGL(linear_back<T>, dim3((unsigned)(runs * ((c.out + 511) / 512))), dim3(256), 0, s, c.R, c.out, c.act,
                     (const T*)c.dy, (const T*)c.z, (T*)c.dz, c.dbias ? c.part : nullptr, runs, back_lanes(c.out));
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !c.dbias) return e;
  return launch_column_sums(c.part, c.dbias, nullptr, nullptr, runs, c.out, s);
}

}  // namespace

int64_t linear_back_runs(int dtype, int64_t R, int out) {
  const int64_t columns = (out + 511) / 512, blocks = dtype == MOE_F32 ? kBackBlocksF32 : kBackBlocks;
  const int64_t most = std::max<int64_t>(64, blocks / columns);
  const int rows = 256 / back_lanes(out);
  return std::min((R + rows - 1) / rows, most);
}

namespace {

constexpr int kFewRows = 16, kMostFewRows = 64;
constexpr int kSplits[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 24, 32}, kMostSplits = 32;
constexpr int64_t kMostPart = (int64_t)1 << 23;  // floats of a split call's parts: 32 MiB of workspace

// What a call takes with tiles of bm x bn, in microseconds: rounds of blocks over the CUs, each of a fixed time and a time
// per step (less in a last round that leaves CUs idle); or the copies of all tiles into LDS, at the 14.3 TB/s that all CUs
// together reach, where those take longer (the shorter of the two hides all but an eighth); and the parts written, read
// and joined. Fitted to the timings of every tile and number of parts at 2,122 shapes (66 to 11,585 rows, 128 to 13,312
// input and 88 to 16,384 output features, a quarter in float32). On 2,139 others its choice is 0.9% slower than the best on
// average and 34% at most (the rule before, without the copies and the idle CUs: 2.2%; 8,192 x 12,288 -> 5,120 in bfloat16
// 1,130 us, so 828).
struct TileCost {
  int bm, bn;
  double start, idle;  // idle: a step's time with few blocks over that with one on every CU
  double step[2], both[2];  // bfloat16 and float32, of 64 and 32 k: one block on a CU, two of 64 rows
};
constexpr TileCost kTiles[] = {{64, 64, 2.2, 0.9, {0.245, 0.67}, {0.615, 1.36}},
                               {64, 128, 2.0, 0.9, {0.424, 1.39}, {0.72, 2.65}},
                               {128, 128, 4.0, 0.9, {0.571, 0}, {0, 0}},
                               {256, 128, 10.0, 0.7, {0.878, 0}, {0, 0}},
                               {256, 256, 9.5, 0.85, {1.39, 0}, {0, 0}}};  // 0: not for float32, where 64 rows do as much

double tile_cost(const TileCost& c, bool f32, int64_t tiles, int64_t R, int in, int out, int splits) {
  const int64_t blocks = tiles * splits, round = c.bm == 64 ? 512 : 256, rest = blocks % round;
  const int all = in / (f32 ? 32 : 64), steps = (all + splits - 1) / splits;
  const double one = c.step[f32], most = c.bm == 64 ? c.both[f32] : one;
  double work = (double)(blocks / round) * (c.start + steps * most);
  if (rest > 0) work += c.start + steps * (rest > 256 ? most : one * (c.idle + (1.0 - c.idle) * (double)rest / 256));
  const double copies = c.start + (double)tiles * (c.bm + c.bn) * in * (f32 ? 4.0 : 2.0) / 1.43e7;
  double t = std::max(work, copies) + 0.125 * std::min(work, copies);
  if (splits > 1) t += 2.5 + 0.2 * splits + 1.7e-6 * splits * R * out;
  return t;
}

}  // namespace

LinearPlan linear_plan(int dtype, int64_t R, int in, int out) {
  const LinearPlan few{16, 16, 1};
  if (R <= kFewRows) return few;
  const bool f32 = dtype == MOE_F32;
  LinearPlan best{0, 0, 1};
  double least = 0;
  for (const TileCost& c : kTiles) {
    if (c.step[f32] == 0) continue;
    const int64_t tiles = (R + c.bm - 1) / c.bm * ((out + c.bn - 1) / c.bn);
    for (int splits : kSplits) {
      if (splits > 1 && (c.bn == 256 || tiles * splits > 1024 || in / (f32 ? 32 : 64) < splits || splits * R * out > kMostPart))
        break;
      const double t = tile_cost(c, f32, tiles, R, in, out, splits);
      if (best.bm == 0 || t < least) {
        least = t;
        best = LinearPlan{c.bm, c.bn, splits};
      }
    }
  }
  // Up to 64 rows the tiles and linear_few come close. It reads the weights at 5.5 TB/s, but x again for every 16 columns, at
  // 60 GB/s into a CU's LDS and 12 TB/s into all; and the tiles' cost, fitted to more rows, is a little off. Fitted to 300
  // shapes of 17 to 64 rows: 0.2% slower than the better one on average (tiles alone 31%, linear_few alone 9%).
  if (R <= kMostFewRows) {
    const double size = f32 ? 4.0 : 2.0, weights = size * in * out, blocks = (out + 15) / 16, each = (16.0 + R) * size * in;
    const double stream = std::max({std::ceil(blocks / 256) * each / 6.0e4, blocks * each / 1.2e7, weights / 5.5e6});
    if (1.5 + stream < (f32 ? 0.8 : 1.15) * least) return few;
  }
  return best;
}

// At most kMostSplits parts and kMostPart floats; never falls as R grows.
size_t linear_part_bytes(int64_t R, int out) {
  if (R <= kFewRows) return 0;
  const int64_t rows = std::min<int64_t>(R, kMostPart);
  return sizeof(float) * (size_t)std::min<int64_t>(rows * out * kMostSplits, kMostPart);
}

hipError_t launch_linear(int dtype, const LinearCall& c, hipStream_t s) {
  const LinearPlan p = linear_plan(dtype, c.R, c.in, c.out);
  return dtype == MOE_F32 ? linear_t<float>(c, p, s) : linear_t<uint16_t>(c, p, s);
}

hipError_t launch_linear_back(int dtype, const LinearBackCall& c, hipStream_t s) {
  return dtype == MOE_F32 ? linear_back_t<float>(c, s) : linear_back_t<uint16_t>(c, s);
}

}  // namespace moe
