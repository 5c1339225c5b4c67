// Products grouped by expert, and their gradients, over rows sorted by expert (the order moe_dispatch
// gives). With e(r) the expert whose range [offsets[e], offsets[e + 1]) holds row r:
//
//   fwd    y[r]  = W[e(r)] x[src(r)]                       (reduction over the input features)
//   dgrad  dx[r] = W[e(r)]^T dy[r]                         (reduction over the output features)
//   wgrad  dW[e] = sum over the expert's rows of dy[r] x[src(r)]^T
//
// W is [E, M, K] row-major, as the layer's own matrices. The tile lists (fwd, dgrad) come from the device
// (launch_offset_lists); wgrad needs none, its tiles are those of dW. The bf16 forward runs on the layer's expert
// GEMMs (gemm_bf16.hip, gemm_decode.hip); here are the float32 products and the bf16 gradients.
//
// What bounds them, measured on whole calls: the Air gate_up shape (128 experts, 4,096 -> 2,816, 4,096 tokens of
// eight experts) wgrad 1.09-1.15 ms, 660-690 TFLOP/s while it writes 2.95 GB of dW (skipping the stores alone 0.85 ms,
// the products alone 0.75: neither hides wholly behind the other); the GLM-4.5 down shape (160 experts, 1,536 <- 5,120,
// 3,001 tokens) dgrad 0.58-0.61 ms, 4.6-4.9 TB/s of its 2.84 GB, the rate of a large copy: bound by the weights' stream.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "ops_internal.h"
#include "row_ops.h"

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
// 128 x 128 tile of C[i, j] = sum_t A(i, t) B(j, t) in float32: both operands go through LDS as
// [t][i] / [t][j] (16 t per step), four waves of 64 x 64 as 4 x 4 tiles of v_mfma_f32_16x16x4_f32
// (A: row lane % 16, k lane / 16; C: column lane % 16, rows 4 (lane / 16) + r).
//   fwd:   i = row, j = output feature, t = input feature;   both operands contiguous in t
//   dgrad: i = row, j = input feature,  t = output feature;  B contiguous in j
//   wgrad: i = output feature, j = input feature, t = row;   both contiguous in i / j
// (60 experts, 704 -> 1,024, 1,024 tokens of four: 116 / 155 / 94 us; one matrix step per LDS round trip and two
// barriers bound it, not the matrix cores.)
// FEW, for groups of few rows (launch_grouped_f32): the waves stand side by side, 128 rows x 32 columns each as 8 x 2
// tiles, and multiply only the row tiles that hold rows (rounded up to 1, 2, 4 or 8).
template <int MODE, bool FEW>
__global__ __launch_bounds__(256) void grouped_f32_tile(GradArgs a, int col_tiles) {
  constexpr bool A_T = MODE == GM_WGRAD;              // A contiguous in i
  constexpr bool B_T = MODE != GM_FWD;                // B contiguous in j
  constexpr int BT = 16, PITCH = 128 + 4;
  __shared__ float sa[BT][PITCH], sb[BT][PITCH];
  const int M = a.M, K = a.K;
  int64_t row0;   // first grouped row of the tile (fwd, dgrad) or of the expert (wgrad)
  int expert, rows, i0 = 0, j0, split;
  if (MODE == GM_WGRAD) {
    const int mt = (M + 127) / 128;
    const int64_t b = blockIdx.x / a.splits;
    split = (int)(blockIdx.x % a.splits);
    j0 = (int)(b % col_tiles) * 128;
    i0 = (int)(b / col_tiles % mt) * 128;
    expert = (int)(b / col_tiles / mt);
    const int64_t lo = min(max((int64_t)a.offsets[expert], (int64_t)0), a.R);
    const int64_t hi = min(max((int64_t)a.offsets[expert + 1], lo), a.R);
    row0 = lo;
    rows = (int)(hi - lo);
  } else {
    int64_t L = xcd_logical_block((int64_t)*a.n_tiles * col_tiles * a.splits);
    if (L < 0) return;
    split = (int)(L % a.splits);
    L /= a.splits;
    const Tile tile = a.tiles[L / col_tiles];
    j0 = (int)(L % col_tiles) * 128;
    row0 = tile.row_start;
    rows = tile.rows;
    expert = tile.expert;
    if (rows <= 0) return;
  }
  const int ni = MODE == GM_WGRAD ? M : rows, nj = MODE == GM_FWD ? M : K;
  const int nt_all = MODE == GM_FWD ? K : MODE == GM_DGRAD ? M : rows;
  // this part of the reduction (the last ones may be empty: they write zeros)
  const int part = (nt_all + a.splits * BT - 1) / (a.splits * BT) * BT;
  const int nt0 = min(split * part, nt_all), nt = min(nt0 + part, nt_all);
  const float* A = (const float*)a.a;
  const float* B = (const float*)a.b;
  const int64_t wbase = (int64_t)expert * M * K;

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int TI = FEW ? 8 : 4, TJ = FEW ? 2 : 4;  // 16 x 16 tiles of a wave
  const int wi = FEW ? 0 : (wave >> 1) * 64, wj = FEW ? wave * 32 : (wave & 1) * 64;
  // this thread's eight elements of each operand per step
  const int ai = A_T ? (tid & 15) * 8 : tid >> 1, at = A_T ? tid >> 4 : (tid & 1) * 8;
  const int bj = B_T ? (tid & 15) * 8 : tid >> 1, bt = B_T ? tid >> 4 : (tid & 1) * 8;
  auto src = [&](int64_t r) -> int64_t { return a.src_row ? a.src_row[r] : r; };
  int64_t a_row = 0;
  if (MODE == GM_FWD && ai < rows) a_row = src(row0 + ai);

  f32x4 acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int live = __builtin_amdgcn_readfirstlane((min(ni - i0, 128) + 15) / 16);  // row tiles that hold rows

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
  if (nt > nt0) load(nt0);
  for (int t0 = nt0; t0 < nt; t0 += BT) {
    __syncthreads();
    put(sa, A_T, ai, at, ra);
    put(sb, B_T, bj, bt, rb);
    __syncthreads();
    if (t0 + BT < nt) load(t0 + BT);
    auto products = [&](auto tiles) {
      constexpr int TILES = decltype(tiles)::value;
#pragma unroll
      for (int k = 0; k < BT; k += 4) {
        float av[TILES], bv[TJ];
#pragma unroll
        for (int i = 0; i < TILES; ++i) av[i] = sa[k + (lane >> 4)][wi + 16 * i + (lane & 15)];
#pragma unroll
        for (int j = 0; j < TJ; ++j) bv[j] = sb[k + (lane >> 4)][wj + 16 * j + (lane & 15)];
#pragma unroll
        for (int i = 0; i < TILES; ++i)
#pragma unroll
          for (int j = 0; j < TJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(av[i], bv[j], acc[i][j], 0, 0, 0);
      }
    };
    if constexpr (!FEW) {
      products(std::integral_constant<int, TI>{});
    } else {
      if (live > 4)
        products(std::integral_constant<int, TI>{});
      else if (live > 2)
        products(std::integral_constant<int, TI / 2>{});
      else if (live == 2)
        products(std::integral_constant<int, 2>{});
      else
        products(std::integral_constant<int, 1>{});
    }
  }
  const int64_t part_elems = MODE == GM_WGRAD ? (int64_t)a.E * M * K : a.R * nj;
  float* out = a.splits > 1 ? a.part + split * part_elems : (float*)a.out;
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int ii = i0 + wi + 16 * i + 4 * (lane >> 4) + q;
      if (ii >= ni) continue;
      const int64_t base = MODE == GM_WGRAD ? wbase + (int64_t)ii * K : (row0 + ii) * (int64_t)nj;
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        const int jj = j0 + wj + 16 * j + (lane & 15);
        if (jj < nj) out[base + jj] = acc[i][j][q];
      }
    }
}

// ---- bfloat16 gradients ----
//
// Both gradients reduce over an index that is not contiguous in one operand (dgrad: W over its rows) or in
// both (wgrad: dy and x over their rows). Such an operand goes to LDS as it lies in memory, whole rows of
// the reduction index, and is turned on the way to the matrix cores: ds_read_b64_tr_b16 gives lane i of 16
// the four elements of column i from four rows of 16 columns, so two of them make the eight consecutive
// reduction elements that a lane of v_mfma_f32_32x32x16_bf16 holds of its column.
//  - a row's 32-byte pieces are XOR-swizzled by twice the row's position modulo 4: the four rows x two
//    neighbouring pieces that half a wave reads at a time then lie in distinct banks;
//  - operands go global -> LDS directly (1 KiB of LDS per wave and load), no register staging;
//  - each wave holds 64 x 128 of C as 2 x 4 tiles; the fragments of the next 16-wide slice are read while
//    the present one's products run.
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kRawBufferWord3 = 0x00020000;  // raw buffer, 32-bit data format

__device__ inline void wait_lgkm0() { __builtin_amdgcn_s_waitcnt((15) | (3 << 14) | (7 << 4) | (0 << 8)); }
template <int N>
__device__ inline void wait_lgkm() {
  static_assert(N >= 0 && N <= 15, "lgkmcnt is 4 bits");
  __builtin_amdgcn_s_waitcnt((15) | (3 << 14) | (7 << 4) | (N << 8));
}
__device__ inline void bare_barrier() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// Both: 256 x 256 tile, eight waves, one block per CU.
// dgrad: 64 reduction elements per step (whole lines of dy), dy in a two-stage ring and W in a three-stage
// one: all 160 KiB of LDS.
// wgrad: 32 rows per step, four stages of both operands (128 KiB).
template <int MODE>
struct GradTile {
  static constexpr bool A_T = MODE == GM_WGRAD;
  static constexpr int NW = 8;  // waves
  static constexpr int BM = 256, BN = 256, BK = A_T ? 32 : 64;
  static constexpr int SA = A_T ? 4 : 2, SB = A_T ? 4 : 3;  // stages
  static constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2;
  static constexpr int NLA = A_BYTES / 1024 / NW, NLB = B_BYTES / 1024 / NW;  // loads per wave and step
  static constexpr int B_BASE = SA * A_BYTES;
  static constexpr int RING = SA * A_BYTES + SB * B_BYTES;
  static constexpr int SLICES = BK / 16;
  static constexpr int OPITCH = 128 + 8;  // staged output row of a wave (dgrad)
  static constexpr int A_RB = BM * 2, B_RB = BN * 2;  // bytes per reduction row of a turned operand
  static_assert(RING <= 160 * 1024 && SLICES % 2 == 0, "LDS; the last slice of a step is in buffer 1");
};

// Byte offset, within a stage of turned rows of RB bytes, of the fragment of 32 columns from col0: slice s adds
// 16 rows, the second half of a lane's eight elements 4 rows.
template <int RB>
__device__ inline int turned_offset(int col0, int lane) {
  const int h = lane >> 5, piece = col0 / 16 + ((lane >> 4) & 1), i = lane & 15;
  return (h * 8 + (i >> 2)) * RB + ((piece ^ (2 * (i >> 2))) * 32) + (i & 3) * 8;
}
// The restrict pointer says what the ring's waits ensure: the direct loads in flight write other stages. Without
// it the compiler puts a vmcnt(0) before each of these reads (it treats the builtin, unlike an ordinary LDS
// load, as a possible reader of whatever is still being loaded).
__device__ inline s16x4 read_tr16(const lds_s16x4* __restrict__ p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
}
// The same for writes into a stage with no loads under way.
typedef __attribute__((address_space(3))) uint2 lds_uint2;
__device__ inline void write_lds8(lds_uint2* __restrict__ p, uint32_t x, uint32_t y) {
  p->x = x;
  p->y = y;
}
template <int RB>
__device__ inline bf16x8 read_turned(const char* p) {
  const s16x4 lo = read_tr16((const lds_s16x4*)p);
  const s16x4 hi = read_tr16((const lds_s16x4*)(p + 4 * RB));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}
// Row (of the reduction) and first column of this lane's 16 bytes in load i of a turned operand.
template <int RB, int NW>
__device__ inline int turned_row(int i, int wave, int lane) {
  return (i * NW + wave) * (1024 / RB) + lane / (RB / 16);
}
template <int RB>
__device__ inline int turned_col(int t, int lane) {
  const int pos = lane % (RB / 16);
  return (((pos >> 1) ^ (2 * (t & 3))) * 2 + (pos & 1)) * 8;
}

__device__ inline int line_swz(int r) {
  r &= 31;
  return (r ^ (r >> 3)) & 7;
}

template <bool V>
struct BoolC {
  static constexpr bool value = V;
};

// One wave's fragments of a 16-wide slice, double-buffered, and its products: 32 MI x 128 of C^T (the column
// operand first, so that a lane holds four neighbouring columns of one row).
template <int MODE, int MI>
struct GradWave {
  using T = GradTile<MODE>;
  static constexpr int NR = MI > 0 ? MI * (T::A_T ? 2 : 1) + 8 : 0;  // LDS reads per slice
  int a_off[MI > 0 ? MI : 1], b_off[4], sw, half;
  bf16x8 af[2][MI > 0 ? MI : 1], bf[2][4];
  __device__ __attribute__((always_inline)) inline void init(int lane, int m0, int n0) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
      a_off[i] = T::A_T ? turned_offset<T::A_RB>(m0 + 32 * i, lane) : (m0 + 32 * i + (lane & 31)) * (T::BK * 2);
#pragma unroll
    for (int j = 0; j < 4; ++j) b_off[j] = turned_offset<T::B_RB>(n0 + 32 * j, lane);
    sw = line_swz(lane);
    half = lane >> 5;
  }
  // slice sl of the step in A stage sta and B stage stb
  __device__ __attribute__((always_inline)) inline void read(const char* lds, int sta, int stb, int sl, int buf) {
    if (MI == 0) return;
    // the stage's place is a scalar to the compiler, which otherwise keeps an address register per read
    int oa = sta * T::A_BYTES, ob = T::B_BASE + stb * T::B_BYTES;
    asm("" : "+s"(oa));
    asm("" : "+s"(ob));
    const char* sa = lds + oa;
    const char* sb = lds + ob;
#pragma unroll
    for (int j = 0; j < 4; ++j) bf[buf][j] = read_turned<T::B_RB>(sb + b_off[j] + sl * 16 * T::B_RB);
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      if (T::A_T)
        af[buf][i] = read_turned<T::A_RB>(sa + a_off[i] + sl * 16 * T::A_RB);
      else
        af[buf][i] = *(const bf16x8*)(sa + a_off[i] + ((2 * sl + half) ^ sw) * 16);
    }
  }
  __device__ __attribute__((always_inline)) inline void compute(f32x16 (&acc)[2][4], int buf) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf[buf][j], af[buf][i], acc[i][j], 0, 0, 0);
  }
};
__device__ inline void sched_fence() { __builtin_amdgcn_sched_barrier(0); }

// dgrad's reduction loop of one wave. issue_a(step) / issue_b(step) start this wave's loads of a step into its
// stage; the newest NLB loads are those of the step after the next.
template <int MI, class IA, class IB>
__device__ __attribute__((always_inline)) inline void dgrad_loop(char* lds, IA&& issue_a, IB&& issue_b,
                                                                 f32x16 (&acc)[2][4], int nk, int lane, int m0,
                                                                 int n0) {
  using T = GradTile<GM_DGRAD>;
  GradWave<GM_DGRAD, MI> w;
  constexpr int NR = GradWave<GM_DGRAD, MI>::NR, AHEAD = T::NLB;
  w.init(lane, m0, n0);
  auto fence = [] { sched_fence(); };
  auto read_slice = [&](int step, int sl, int buf) { w.read(lds, step % T::SA, step % T::SB, sl, buf); };
  auto compute = [&](int buf) { w.compute(acc, buf); };

  // prologue: the steps before the first compute, oldest first
  issue_a(0);
  issue_b(0);
  if (nk > 1) {
    issue_b(1);
    wait_vmcnt<AHEAD>();
  } else {
    wait_vmcnt<0>();
  }
  bare_barrier();
  read_slice(0, 0, 0);
  fence();
  auto step = [&](int kt, auto more_a, auto more_b, auto last) {
    constexpr bool MA = decltype(more_a)::value, MB = decltype(more_b)::value, LAST = decltype(last)::value;
    if (MA) issue_a(kt + T::SA - 1);  // into the stage that step kt - 1 used
#pragma unroll
    for (int sl = 0; sl < T::SLICES; ++sl) {
      if (sl + 1 < T::SLICES) {
        read_slice(kt, sl + 1, (sl + 1) & 1);
        fence();
        wait_lgkm<NR>();
        if (sl == 0 && MB) issue_b(kt + T::SB - 1);
        compute(sl & 1);
        fence();
      } else {
        wait_lgkm0();  // every read of this step has landed
        if (MA && MB)
          wait_vmcnt<AHEAD>();
        else if (!LAST)
          wait_vmcnt<0>();
        bare_barrier();
        if (!LAST) read_slice(kt + 1, 0, 0);
        fence();
        compute(sl & 1);  // while the next step's first reads land
        fence();
      }
    }
  };
  int kt = 0;
  for (; kt + T::SB - 1 < nk; ++kt) step(kt, BoolC<true>{}, BoolC<true>{}, BoolC<false>{});
  if (kt + 1 < nk) step(kt++, BoolC<true>{}, BoolC<false>{}, BoolC<false>{});
  step(kt, BoolC<false>{}, BoolC<false>{}, BoolC<true>{});
}

// Results of one wave through its part of the (idle) ring: whole 16-byte pieces of `rows` rows of up to 128
// columns, `ld` elements apart.
__device__ __attribute__((always_inline)) inline void store_dgrad(char* lds, const f32x16 (&acc)[2][4], int wave,
                                                                  int lane, int rows, int cols, uint16_t* out,
                                                                  int64_t ld) {
  using T = GradTile<GM_DGRAD>;
  static_assert(T::NW * 64 * T::OPITCH * 2 <= T::RING - 16, "the staged outputs fit the ring");
  uint16_t* st = (uint16_t*)lds + wave * (64 * T::OPITCH);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (32 * i >= rows) continue;
    uint16_t* row = st + (i * 32 + (lane & 31)) * T::OPITCH + 4 * (lane >> 5);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint2 v = make_uint2(bf16_pair(acc[i][j][4 * q], acc[i][j][4 * q + 1]),
                                   bf16_pair(acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]));
        *(uint2*)(row + j * 32 + 8 * q) = v;
      }
  }
  // the region is this wave's own: its writes need only be in order with its reads
  wait_lgkm0();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  // 4 rows of 16 pieces at a time, eight reads ahead of their stores
  const int row0 = lane >> 4, ch = lane & 15;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    u32x4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = *(const u32x4*)(st + (h * 32 + u * 4 + row0) * T::OPITCH + ch * 8);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int row = h * 32 + u * 4 + row0;
      if (row < rows && ch * 8 < cols) __builtin_nontemporal_store(v[u], (u32x4*)(out + row * ld + ch * 8));
    }
  }
}

// Float32 results of one wave straight to a part of a split reduction: four columns a lane.
__device__ __attribute__((always_inline)) inline void store_part(const f32x16 (&acc)[2][4], int lane, int rows, int cols,
                                                                 float* out, int64_t ld) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = i * 32 + (lane & 31);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int col = j * 32 + 8 * q + 4 * (lane >> 5);
        if (row < rows && col < cols)
          *(f32x4*)(out + row * ld + col) =
              f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
      }
  }
}

// One 256 x 256 tile of dx: rows of `tile`, columns from col0, part `split` of the reduction.
__device__ __forceinline__ void dgrad_block(const GradArgs& a, const Tile tile, int col0, int split, char* lds) {
  using T = GradTile<GM_DGRAD>;
  const int t = threadIdx.x;
  int lane = t & 63;
  // keeps what depends on the lane inside this tile: kept over the claiming loop, it spilled 42 registers
  asm volatile("" : "+v"(lane));
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int m0 = (wave & 3) * 64, n0 = (wave >> 2) * 128;
  const int M = a.M, K = a.K;
  // this part's steps (never none: grouped_splits)
  const int all = M / T::BK, per = (all + a.splits - 1) / a.splits, k0 = split * per, nk = min(per, all - k0);
  const uint16_t* abase = (const uint16_t*)a.a + (int64_t)tile.row_start * M + k0 * T::BK;
  const uint16_t* bbase = (const uint16_t*)a.b + ((int64_t)tile.expert * M + k0 * T::BK) * K;
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc((void*)abase, (short)0, -1, kRawBufferWord3);
  const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc((void*)bbase, (short)0, -1, kRawBufferWord3);
  uint32_t oa[T::NLA], ob[T::NLB];
#pragma unroll
  for (int i = 0; i < T::NLA; ++i) {
    const int r = (i * T::NW + wave) * 8 + (lane >> 3), c = (lane & 7) ^ line_swz(r);
    oa[i] = ((uint32_t)min(r, tile.rows - 1) * (uint32_t)M + 8 * c) * 2;  // rows past the tile repeat its last
  }
#pragma unroll
  for (int i = 0; i < T::NLB; ++i) {
    const int r = turned_row<T::B_RB, T::NW>(i, wave, lane);
    const int c = min(col0 + turned_col<T::B_RB>(r, lane), K - 8);  // columns past K repeat the last piece
    ob[i] = ((uint32_t)r * (uint32_t)K + c) * 2;
  }
  // loads that reach a valid row (8 rows per load)
  const int na = max(0, min(T::NLA, (tile.rows - wave * 8 + 63) / 64));
  auto issue_a = [&](int k) {
    char* dst = lds + (k % T::SA) * T::A_BYTES + wave * 1024;
#pragma unroll
    for (int i = 0; i < T::NLA; ++i)
      if (i < na)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(dst + i * T::NW * 1024), 16, (int)oa[i], k * T::BK * 2,
                                                 0, 0);
  };
  auto issue_b = [&](int k) {
    char* dst = lds + T::B_BASE + (k % T::SB) * T::B_BYTES + wave * 1024;
    const uint32_t soff = (uint32_t)k * T::BK * (uint32_t)K * 2;
#pragma unroll
    for (int i = 0; i < T::NLB; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(dst + i * T::NW * 1024), 16, (int)ob[i], (int)soff, 0, 0);
  };
  f32x16 acc[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  const int live = tile.rows - m0;
  if (live > 32)
    dgrad_loop<2>(lds, issue_a, issue_b, acc, nk, lane, m0, n0);
  else if (live > 0)
    dgrad_loop<1>(lds, issue_a, issue_b, acc, nk, lane, m0, n0);
  else
    dgrad_loop<0>(lds, issue_a, issue_b, acc, nk, lane, m0, n0);
  if (a.splits > 1) {
    store_part(acc, lane, max(0, min(64, live)), min(128, K - col0 - n0),
               a.part + (split * a.R + tile.row_start + m0) * K + col0 + n0, K);
    return;
  }
  // the loop ended on a barrier after the last operand read
  uint16_t* out = (uint16_t*)a.out + ((int64_t)tile.row_start + m0) * K + col0 + n0;
  store_dgrad(lds, acc, wave, lane, max(0, min(64, live)), min(128, K - col0 - n0), out, K);
}

// Logical block L over n_rows x n_cols tiles -> rectangles of GR x GC tiles, rows fastest.
template <int GR, int GC>
__device__ inline void grad_raster(int64_t L, int64_t n_rows, int n_cols, int64_t& row, int& col) {
  const int64_t sg = L / ((int64_t)GR * n_cols), within = L % ((int64_t)GR * n_cols);
  const int64_t gr = min((int64_t)GR, n_rows - sg * GR);
  const int64_t cg = within / (gr * GC), w2 = within % (gr * GC);
  row = sg * GR + w2 % gr;
  col = (int)(cg * GC + w2 / gr);
}

// Persistent: one block per CU claims tiles, of its own XCD's run of the list first and then of the others',
// and exits once all eight runs are empty.
__global__ __launch_bounds__(512, 1) void grouped_dgrad_bf16(GradArgs a, int ncol) {
  using T = GradTile<GM_DGRAD>;
  __shared__ __attribute__((aligned(1024))) char lds[T::RING];
  int* claim = (int*)(lds + T::RING - 4);  // outside the staged outputs; written when the loop's reads are over
  const int64_t n_tiles = *a.n_tiles, nvalid = n_tiles * ncol * a.splits, q = nvalid >> 3, r = nvalid & 7;
  const int x = blockIdx.x & 7;
  for (int v = 0; v < 8; ++v) {
    const int y = (x + v) & 7;
    const int64_t start = y * q + min((int64_t)y, r), len = q + (y < r ? 1 : 0);
    for (;;) {
      if (threadIdx.x == 0) *claim = atomicAdd(&a.work_ctr[y], 1);
      __syncthreads();
      const int64_t j = *claim;
      __syncthreads();
      if (j >= len) break;
      int64_t tid;
      int ct;
      grad_raster<2, 16>((start + j) / a.splits, n_tiles, ncol, tid, ct);
      const Tile tile = a.tiles[tid];
      if (tile.rows > 0) dgrad_block(a, tile, ct * T::BN, (int)((start + j) % a.splits), lds);
      __syncthreads();  // every wave's stores have read the LDS
    }
  }
}

// wgrad. An expert's few hundred rows make a short loop (eight steps at 256 rows) and every tile ends in 128 KiB
// of dW, so what counts is that neither the first loads of a tile nor its stores are waited for: a block is
// persistent and its ring runs across tile borders. While a tile's last steps compute and its results are
// stored, the next tile's first three steps are already being loaded; the results pass through the one
// stage that is free at that point. Tiles are dealt in runs of one per CU of an XCD, runs to the XCDs in turn:
// the blocks of an XCD work on one rectangle of one expert's dW and share its rows in L2, and experts of
// different sizes spread over all XCDs.
//
// Rows past the expert's are read as zeros: dy through the descriptor's range (the step's rows of dy and nothing
// behind them), gathered x through an offset past the range.
struct WgradTile {
  int expert, split, i0, j0, cnt, nk;
  int64_t row0;
};
template <bool GATHER, bool SPLIT>
__global__ __launch_bounds__(512, 1) void grouped_wgrad_bf16(GradArgs a, int mt, int kt_tiles) {
  using T = GradTile<GM_WGRAD>;
  constexpr int S = T::SA, PER = T::NLA + T::NLB, NST = SPLIT ? 32 : 16;  // stages, loads per step, stores per tile
  static_assert(T::SA == T::SB && (S & (S - 1)) == 0 && (S - 2) * PER + NST < 64, "ring indices and vmcnt");
  __shared__ __attribute__((aligned(1024))) char lds[T::RING];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m0 = (wave & 3) * 64, n0 = (wave >> 2) * 128;
  const int M = a.M, K = a.K;
  typedef const __attribute__((address_space(4))) int32_t* const_i32;  // scalar loads: none counts in vmcnt
  const uint32_t slots = gridDim.x >> 3, stride = gridDim.x;
  const uint32_t per_expert = (uint32_t)(mt * kt_tiles);
  const uint32_t total = per_expert * (uint32_t)a.E * (uint32_t)(SPLIT ? a.splits : 1);
  const uint32_t first = (blockIdx.x & 7) * slots + (blockIdx.x >> 3);

  auto decode = [&](uint32_t id) {
    WgradTile t;
    t.expert = (int)(id / per_expert);
    t.split = 0;
    if (SPLIT) {
      t.split = t.expert % a.splits;
      t.expert /= a.splits;
    }
    // rectangles of 4 x 8 tiles, rows fastest
    const uint32_t in = id % per_expert, sg = in / (4u * kt_tiles), within = in % (4u * kt_tiles);
    const uint32_t gr = min(4u, (uint32_t)mt - sg * 4), cg = within / (gr * 8), w2 = within % (gr * 8);
    t.i0 = (int)(sg * 4 + w2 % gr) * T::BM;
    t.j0 = (int)(cg * 8 + w2 / gr) * T::BN;
    const int64_t lo = ((const_i32)a.offsets)[t.expert], hi = ((const_i32)a.offsets)[t.expert + 1];
    t.row0 = min(max(lo, (int64_t)0), a.R);
    t.cnt = (int)(min(max(hi, t.row0), a.R) - t.row0);
    if (SPLIT) {  // this part of the expert's rows, in whole steps; perhaps none
      const int per = (t.cnt + a.splits * T::BK - 1) / (a.splits * T::BK) * T::BK, from = min(t.split * per, t.cnt);
      t.row0 += from;
      t.cnt = min(per, t.cnt - from);
    }
    t.nk = (t.cnt + T::BK - 1) / T::BK;
    return t;
  };

  // ---- the load stream: its own tile and step, up to three steps ahead of the products ----
  uint32_t load_id = first;
  int load_k = 0;
  int issued = 0;  // steps
  WgradTile lt{};
  uint32_t oa[T::NLA], ob[T::NLB];
  auto load_tile = [&](uint32_t id) {  // the first tile from id on that has rows
    for (; id < total; id += stride) {
      lt = decode(id);
      if (lt.nk > 0) break;
    }
    load_id = id;
    load_k = 0;
    if (id >= total) return;
#pragma unroll
    for (int i = 0; i < T::NLA; ++i) {
      const int r = turned_row<T::A_RB, T::NW>(i, wave, lane);
      oa[i] = ((uint32_t)r * (uint32_t)M + min(lt.i0 + turned_col<T::A_RB>(r, lane), M - 8)) * 2;
    }
#pragma unroll
    for (int i = 0; i < T::NLB; ++i) {
      const int r = turned_row<T::B_RB, T::NW>(i, wave, lane);
      const int c = min(lt.j0 + turned_col<T::B_RB>(r, lane), K - 8);
      ob[i] = GATHER ? (uint32_t)c * 2 : ((uint32_t)r * (uint32_t)K + c) * 2;
    }
  };
  // source rows of the next issued step's x loads: a wave's load i takes two rows, so their indices are scalar
  // loads, made a step ahead; fold() turns them into this lane's offsets once they are there
  int32_t idx[T::NLB][2];
  uint32_t ox[T::NLB];
  auto fetch_index = [&]() {
    if (!GATHER || load_id >= total) return;
#pragma unroll
    for (int i = 0; i < T::NLB; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = load_k * T::BK + (i * T::NW + wave) * 2 + h;
        idx[i][h] = ((const_i32)a.src_row)[lt.row0 + min(r, lt.cnt - 1)];
      }
  };
  auto fold = [&]() {
    if (!GATHER || load_id >= total) return;
    const int left = lt.cnt - load_k * T::BK;
#pragma unroll
    for (int i = 0; i < T::NLB; ++i) {
      const uint32_t r = (uint32_t)(lane < 32 ? idx[i][0] : idx[i][1]);
      ox[i] = turned_row<T::B_RB, T::NW>(i, wave, lane) < left ? r * (uint32_t)K * 2 + ob[i] : 0xfffffff0u;
    }
  };
  // the stream's next step into its stage; nothing at its end
  auto issue = [&]() {
    if (load_id >= total) return;
    const int left = min(lt.cnt - load_k * T::BK, T::BK);
    const int64_t row = lt.row0 + (int64_t)load_k * T::BK;
    char* da = lds + (issued & (S - 1)) * T::A_BYTES + wave * 1024;
    char* db = lds + T::B_BASE + (issued & (S - 1)) * T::B_BYTES + wave * 1024;
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc((void*)((const uint16_t*)a.a + row * M), (short)0,
                                                                        left * M * 2, kRawBufferWord3);
#pragma unroll
    for (int i = 0; i < T::NLA; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(da + i * T::NW * 1024), 16, (int)oa[i], 0, 0, 0);
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
        (void*)((const uint16_t*)a.b + (GATHER ? 0 : row * K)), (short)0,
        GATHER ? (int)(uint32_t)(a.x_rows * K * 2) : left * K * 2, kRawBufferWord3);
#pragma unroll
    for (int i = 0; i < T::NLB; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(db + i * T::NW * 1024), 16, (int)(GATHER ? ox[i] : ob[i]),
                                               0, 0, 0);
    ++issued;
    if (++load_k == lt.nk) load_tile(load_id + stride);
  };

  GradWave<GM_WGRAD, 2> w;
  constexpr int NR = GradWave<GM_WGRAD, 2>::NR;
  w.init(lane, m0, n0);
  load_tile(first);
#pragma unroll
  for (int i = 0; i < S - 1; ++i) {
    fetch_index();
    fold();
    issue();
  }
  fetch_index();
  fold();
  wait_vmcnt<0>();
  bare_barrier();
  int done = 0;         // steps whose products ran
  int mark = 0;         // steps issued before this wave's last stores
  bool stored = false;  // the previous tile's results were stored by this wave
  if (issued > 0) w.read(lds, 0, 0, 0, 0);
  sched_fence();

  for (uint32_t id = first; id < total; id += stride) {
    const WgradTile t = decode(id);
    f32x16 acc[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    for (int k = 0; k < t.nk; ++k) {
      const int st = done & (S - 1), nx = (done + 1) & (S - 1);
      // into the stage of the step before this one (of the tile before: behind its epilogue's barrier)
      issue();
      fetch_index();
      w.read(lds, st, st, 1, 1);
      sched_fence();
      wait_lgkm<NR>();
      w.compute(acc, 0);
      sched_fence();
      wait_lgkm0();  // this step's reads have landed, and the indices
      fold();
      // the next step has landed: of the loads behind its own, `ahead` steps may be in flight, and the stores of
      // the last tile if they were issued after it
      const int ahead = issued - done - 2;
      ++done;
      if (ahead < S - 2)
        wait_vmcnt<0>();
      else if (stored && issued - mark <= ahead)
        wait_vmcnt<(S - 2) * PER + NST>();
      else
        wait_vmcnt<(S - 2) * PER>();
      bare_barrier();
      if (done < issued) w.read(lds, nx, nx, 0, 0);
      sched_fence();
      w.compute(acc, 1);
      sched_fence();
    }
    // Epilogue in the stage the last step used (free until the next issue): each wave has 4 KiB of it (two in
    // each operand's part), 32 rows x 64 columns a pass, 16-byte pieces swizzled by the row. Every pass issues four
    // stores in any case (lanes past the columns through an offset past the range): the counts above rely on it.
    const int free_st = (done + S - 1) & (S - 1);
    stored = t.i0 + m0 < M;
    mark = issued;
    if (SPLIT && stored) {  // float32 parts, straight from the registers
      const __amdgpu_buffer_rsrc_t ro = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(a.part + (((int64_t)t.split * a.E + t.expert) * M + t.i0 + m0) * K), (short)0, 64 * K * 4,
          kRawBufferWord3);
      const int cols = K - t.j0 - n0;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int row = i * 32 + (lane & 31), col = j * 32 + 8 * q + 4 * (lane >> 5);
            const uint32_t off = col < cols ? ((uint32_t)row * (uint32_t)K + t.j0 + n0 + col) * 4 : 0xfffffff0u;
            const f32x4 c = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, c), ro, (int)off, 0, 0);
          }
    }
    if (!SPLIT && stored) {
      char* sp = lds + (wave < 4 ? free_st * T::A_BYTES + wave * 4096 : T::B_BASE + free_st * T::B_BYTES + (wave - 4) * 4096);
      const __amdgpu_buffer_rsrc_t ro = __builtin_amdgcn_make_buffer_rsrc(
          (void*)((uint16_t*)a.out + ((int64_t)t.expert * M + t.i0 + m0) * K), (short)0, 64 * K * 2, kRawBufferWord3);
      const int cols = K - t.j0 - n0;  // of this wave's 128
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int jp = 0; jp < 2; ++jp) {
          const int r = lane & 31;
#pragma unroll
          for (int jj = 0; jj < 2; ++jj)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const f32x16& c = acc[i][2 * jp + jj];
              write_lds8((lds_uint2*)(sp + r * 128 + (((4 * jj + q) ^ (r & 7)) * 16) + (lane >> 5) * 8),
                         bf16_pair(c[4 * q], c[4 * q + 1]), bf16_pair(c[4 * q + 2], c[4 * q + 3]));
            }
          __atomic_signal_fence(__ATOMIC_SEQ_CST);  // a wave's LDS accesses are in order
          u32x4 v[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int row = u * 8 + (lane >> 3);
            v[u] = *(const u32x4*)(sp + row * 128 + (((lane & 7) ^ (row & 7)) * 16));
          }
          __atomic_signal_fence(__ATOMIC_SEQ_CST);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int row = i * 32 + u * 8 + (lane >> 3), col = jp * 64 + (lane & 7) * 8;
            const uint32_t off = col < cols ? ((uint32_t)row * (uint32_t)K + t.j0 + n0 + col) * 2 : 0xfffffff0u;
            __builtin_amdgcn_raw_buffer_store_b128(v[u], ro, (int)off, 0, 2);
          }
        }
    }
    wait_lgkm0();
    bare_barrier();  // the stage is free again
  }
}

int grad_cus() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 8) n = 256;
    n = n / 8 * 8;
    cached[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

}  // namespace

hipError_t launch_grouped_bf16(GroupedMode mode, const GradArgs& a, int64_t max_tile_count, hipStream_t s) {
  if (mode == GM_DGRAD) {
    const int nc = (a.K + 255) / 256;
    const int64_t blocks = (max_tile_count * nc * a.splits + 7) / 8 * 8;
    if (blocks == 0) return hipSuccess;
    if (!a.work_ctr) return hipErrorInvalidValue;
    hipLaunchKernelGGL(grouped_dgrad_bf16, dim3((unsigned)std::min<int64_t>(blocks, grad_cus())), dim3(512), 0, s, a,
                       nc);
    return hipGetLastError();
  }
  if (mode != GM_WGRAD) return hipErrorInvalidValue;
  const int mt = (a.M + 255) / 256, kt = (a.K + 255) / 256;
  const int64_t tiles = ((int64_t)a.E * mt * kt * a.splits + 7) / 8 * 8;
  if (tiles >= (int64_t)1 << 30) return hipErrorInvalidValue;  // 32-bit tile ids, with a stride to spare
  const dim3 grid((unsigned)std::min<int64_t>(tiles, grad_cus())), block(512);
  if (a.splits > 1) {
    if (a.src_row)
      hipLaunchKernelGGL((grouped_wgrad_bf16<true, true>), grid, block, 0, s, a, mt, kt);
    else
      hipLaunchKernelGGL((grouped_wgrad_bf16<false, true>), grid, block, 0, s, a, mt, kt);
  } else if (a.src_row) {
    hipLaunchKernelGGL((grouped_wgrad_bf16<true, false>), grid, block, 0, s, a, mt, kt);
  } else {
    hipLaunchKernelGGL((grouped_wgrad_bf16<false, false>), grid, block, 0, s, a, mt, kt);
  }
  return hipGetLastError();
}

// Parts of the reduction. A call with few tiles (few rows and narrow outputs; wgrad: few experts and small
// matrices) leaves most CUs idle while a few walk a long reduction, so it is cut until there is a block for every
// CU (two for the smaller float32 tiles), in parts of at least four steps, as long as the parts' float32 outputs
// fit `part_bytes`. With the tile counts known only on the device, fwd and dgrad assume the most there can be.
int grouped_splits(GroupedMode mode, int dtype, int E, int64_t R, int M, int K, size_t part_bytes) {
  const bool f32 = dtype == MOE_F32;
  const int64_t bm = f32 ? kF32Rows : kGradRows, bn = f32 ? 128 : 256;
  const int64_t target = f32 ? 512 : 256;
  if (R == 0) return 1;
  auto up = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
  const int64_t used = std::min<int64_t>(R, E);  // experts with rows, at most
  int64_t items, red, step, elems;
  if (mode == GM_WGRAD) {
    items = (int64_t)E * up(M, bm) * up(K, bn);
    red = up(R, used);
    step = f32 ? 16 : 32;
    elems = (int64_t)E * M * K;
  } else {
    const int64_t J = mode == GM_FWD ? M : K;
    items = (used + R / bm) * up(J, bn);
    red = mode == GM_FWD ? K : M;
    step = f32 ? 16 : 64;
    elems = R * J;
  }
  int64_t n = std::min(target / items, red / (4 * step));
  n = std::min<int64_t>(n, (int64_t)(part_bytes / 4) / elems);
  n = std::min<int64_t>(n, 32);
  if (n < 2) return 1;
  if (mode != GM_WGRAD) {  // equal whole steps, none of the parts empty
    const int64_t steps = up(red, step), per = up(steps, n);
    n = up(steps, per);
  }
  return (int)n;
}

namespace {

// out = the sum of the parts, in order; eight elements a thread. Rows outside the grouped ones are left alone.
template <typename T>
__global__ __launch_bounds__(256) void grouped_join_kernel(const float* __restrict__ part, int splits, int64_t elems,
                                                           int64_t row_elems, const int32_t* __restrict__ row_range,
                                                           T* __restrict__ out) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  const int64_t lo = row_range ? row_range[0] * row_elems : 0, hi = row_range ? row_range[1] * row_elems : elems;
  if (i < lo || i >= hi) return;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int s0 = 0; s0 < splits; s0 += 4) {
    Raw8<float> v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (s0 + u < splits) v[u] = raw_load8(part + (s0 + u) * elems + i);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (s0 + u < splits) {
        float f[8];
        widen8(v[u], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += f[e];
      }
  }
  raw_store8<false>(out + i, acc);
}

}  // namespace

hipError_t launch_grouped_join(GroupedMode mode, int dtype, const GradArgs& a, hipStream_t s) {
  const int64_t row = mode == GM_FWD ? a.M : a.K;
  const int64_t elems = mode == GM_WGRAD ? (int64_t)a.E * a.M * a.K : a.R * row;
  const int64_t blocks = (elems / 8 + 255) / 256;
  if (blocks >= (int64_t)1 << 31) return hipErrorInvalidValue;
  const int32_t* range = mode == GM_WGRAD ? nullptr : a.row_range;
  if (dtype == MOE_F32)
    hipLaunchKernelGGL(grouped_join_kernel<float>, dim3((unsigned)blocks), dim3(256), 0, s, a.part, a.splits, elems, row,
                       range, (float*)a.out);
  else
    hipLaunchKernelGGL(grouped_join_kernel<uint16_t>, dim3((unsigned)blocks), dim3(256), 0, s, a.part, a.splits, elems,
                       row, range, (uint16_t*)a.out);
  return hipGetLastError();
}

int64_t grouped_f32_blocks(GroupedMode mode, int E, int M, int K, int splits, int64_t max_tile_count) {
  const int64_t cols = ((mode == GM_FWD ? M : K) + 127) / 128;
  const int64_t blocks = (mode == GM_WGRAD ? (int64_t)E * ((M + 127) / 128) : max_tile_count) * cols * splits;
  return mode == GM_WGRAD ? blocks : (blocks + 7) / 8 * 8;
}

hipError_t launch_grouped_f32(GroupedMode mode, const GradArgs& a, int64_t max_tile_count, hipStream_t s) {
  const int cols = ((mode == GM_FWD ? a.M : a.K) + 127) / 128;
  const int64_t blocks = grouped_f32_blocks(mode, a.E, a.M, a.K, a.splits, max_tile_count);
  if (blocks == 0) return hipSuccess;
  const dim3 grid((unsigned)blocks), block(256);
  // Groups of few rows on average: most of a 128-row tile is empty, and the form that skips its empty row tiles wins
  // up to about 32 rows per group (60 experts, 704 -> 1,024, us with / without: fwd of 8 / 16 / 32 / 40 rows 54 / 113,
  // 72 / 111, 108 / 112, 124 / 113; dgrad 78 / 149, 91 / 151, 148 / 155, 175 / 154). With full tiles it is slower
  // (dgrad, 48 rows: 176 / 158): it holds 196 registers instead of 108, so fewer waves hide the loads.
  const bool few = a.R <= 32 * (int64_t)a.E;
  if (mode == GM_FWD && few)
    hipLaunchKernelGGL((grouped_f32_tile<GM_FWD, true>), grid, block, 0, s, a, cols);
  else if (mode == GM_FWD)
    hipLaunchKernelGGL((grouped_f32_tile<GM_FWD, false>), grid, block, 0, s, a, cols);
  else if (mode == GM_DGRAD && few)
    hipLaunchKernelGGL((grouped_f32_tile<GM_DGRAD, true>), grid, block, 0, s, a, cols);
  else if (mode == GM_DGRAD)
    hipLaunchKernelGGL((grouped_f32_tile<GM_DGRAD, false>), grid, block, 0, s, a, cols);
  else
    hipLaunchKernelGGL((grouped_f32_tile<GM_WGRAD, false>), grid, block, 0, s, a, cols);
  return hipGetLastError();
}

}  // namespace moe
