// Products with 4-bit weights and one scale per group of a weight row, dense or grouped by expert:
//
//   y[r, m] = sum_k x[src(r), k] (q[e, m, k] - 8) s[e, m, k / group]
//
// q holds two 4-bit values a byte, even k in the low half; groups of 32, 64 or 128. With few rows per
// expert the product is a stream of the weights (half a byte each), so the weights go straight from
// memory to registers in 16-byte pieces of 32 values, several pieces ahead of their use, and are made
// into matrix operands there:
//  - q - 8 becomes a bfloat16, exactly, in twelve instructions per eight values (unpack8); the activations are
//    laid out in LDS in the order that this gives the values;
//  - v_mfma_f32_16x16x32_bf16 sums one group in float32, and the group's sum is scaled in float32 and added.
//    Neither a weight nor a scaled partial sum is ever rounded to bfloat16, and a weight of 0 adds exactly
//    nothing, however large its activation. (A cheaper unpacking to 128 + q with 136 sum(x) taken off a group's sum
//    cancels: 5,120 features, groups of 128, weights of 0 beside an activation 10,000 times the others: 30% of
//    the outputs were not the exact value rounded; now all are.)
// A lane's 16 bytes are 32 consecutive k of one weight row. Groups of 128 take them as they are (four
// matrix steps that each cross the four 32-value pieces); smaller groups first exchange the four words
// among the four lanes of a row (permlane swaps), so that a step's 32 values are consecutive.
//
// What bounds it: 32 tokens over 256 experts, 6,144 -> 4,096, groups of 32: 0.44-0.46 ms, 4.7 TB/s of the weights and
// scales that it fetches, about a large copy's rate, with the vector unit busy 70% of the cycles; one token,
// 5,120 -> 24,576, groups of 128: 14.5-16 us, of which the 65 MB would take 13 (the launch's ramp, few rounds of loads
// per wave); 1,021 rows, 12,288 -> 5,120, groups of 64: 0.23 ms, 556 TFLOP/s: per 48 x 64 x 256 values of a wave 96
// matrix instructions (16 cycles each) and 760 vector ones (4 each) of two waves per SIMD that overlap in part.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ops_internal.h"
#include "row_ops.h"

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int SEG = 128;  // k per 16-byte piece of the four lanes of a row

// TT: 16-row activation tiles per block; KS: waves that split k (the other factor of the four waves splits
// the weight rows); RT: 16-row weight tiles per wave (with SWIGLU, gate tiles and their up tiles in turn);
// NSEG: pieces per batch, a wave's weight loads in flight per weight tile; LDS: activations held at a time.
template <int TT_, int KS_, int RT_, int NSEG_, int LDS_, int BLOCKS_>
struct QTile {
  static constexpr int BLOCKS = BLOCKS_;  // per CU, for the register budget
  static constexpr int TT = TT_, KS = KS_, RT = RT_, NSEG = NSEG_;
  static constexpr int ROWS = 16 * TT;
  static constexpr int WAVE_N = 4 / KS;            // waves over weight rows
  static constexpr int BATCH = SEG * NSEG;         // k per wave and batch
  static constexpr int STEP = KS * BATCH;          // k per batch of the block
  static constexpr int LDS_ELEMS = LDS_ + 8 * ROWS;  // activations of a chunk, rows padded by 8
  static_assert(ROWS * STEP <= LDS_, "a full tile's step fits");
  // k per chunk for a tile of `rows` activation rows: what the LDS holds, no more than the row needs
  __device__ static int chunk(int rows, int K) { return min(LDS_ / rows / STEP * STEP, (K + STEP - 1) / STEP * STEP); }
};

// Eight values of a word as the bfloat16 q - 8, exactly, in the order 0 2 4 6 1 3 5 7. First the sign (n: 8 where
// q < 8) and the magnitude of all eight nibbles at once: where q < 8 the three low bits inverted and one added, 8 - q,
// elsewhere bit 3 taken off. Then bytes of a sign and four magnitude bits: as e4m3 such a byte is its magnitude times
// 2^-9 (subnormal up to 7, and linear up to 15), so the conversion of a pair to bfloat16, scaled by 2^9, is exact. The
// compiler is kept from seeing through n and mag: it then forms n three times (16 instructions; one token,
// 5,120 -> 24,576: 21 us, 19.5 with 12).
__device__ inline bf16x8 unpack8(uint32_t w) {
  uint32_t n = ~w & 0x88888888u;
  asm("" : "+v"(n));
  const uint32_t r = n >> 3;
  uint32_t mag = (w ^ (0x88888888u - r)) + r;  // per nibble: no borrow, no carry
  asm("" : "+v"(mag));
  const uint32_t n4 = n << 4, mag4 = mag >> 4;
  const uint32_t even = (mag & 0x0f0f0f0fu) | (n4 & 0xf0f0f0f0u), odd = (mag4 & 0x0f0f0f0fu) | (n & 0xf0f0f0f0u);
  u32x4 v;
  v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(even, 512.f, false));
  v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(even, 512.f, true));
  v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(odd, 512.f, false));
  v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(odd, 512.f, true));
  return __builtin_bit_cast(bf16x8, v);
}

// The four words of the four lanes of a row, transposed: lane group j receives word j of lane groups 0..3.
__device__ inline void exchange4(u32x4& d) {
  auto a = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
  auto b = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
  auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto e = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  d[0] = c[0];
  d[1] = c[1];
  d[2] = e[0];
  d[3] = e[1];
}

// SwiGLU of the products, clamped as swiglu_bf16 does. By comparisons, which leave a NaN as it is: fminf would make it
// the bound, and a damaged weight's output an ordinary number.
__device__ inline uint16_t gated(float g, float u, float lim) {
  if (lim > 0.f) {
    g = g > lim ? lim : g;
    u = u > lim ? lim : u < -lim ? -lim : u;
  }
  return (uint16_t)bf16_pair(swiglu_bf16(g, u, 0.f), 0.f);
}

template <int V>
struct IntC {
  static constexpr int value = V;
};

template <class T, int G, bool SWIGLU>
__global__ __launch_bounds__(256, T::BLOCKS) void qlinear_kernel(QuantArgs a) {
  constexpr int TT = T::TT, KS = T::KS, RT = T::RT, NSEG = T::NSEG, BATCH = T::BATCH;
  constexpr int GPS = SEG / G;                // groups per piece
  constexpr int STEPS = G / 32;               // matrix steps per group
  __shared__ __attribute__((aligned(16))) uint16_t xs[T::LDS_ELEMS];
  __shared__ int src_rows[T::ROWS];

  const int expert = blockIdx.y;
  int64_t row0 = 0, cnt = a.R;
  if (a.offsets) {
    row0 = min(max((int64_t)a.offsets[expert], (int64_t)0), a.R);
    cnt = min(max((int64_t)a.offsets[expert + 1], row0), a.R) - row0;
  }
  const int K = a.K;
  const int half = a.M / 2;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kw = wave % KS, nw = wave / KS;   // this wave's k share and weight rows
  // output columns of the block, and this wave's two weight tiles
  constexpr int WCOLS = SWIGLU ? 8 * RT : 16 * RT;
  const int ncols = SWIGLU ? half : a.M;
  const int col0 = (blockIdx.x * T::WAVE_N + nw) * WCOLS;
  // an expert's matrix is below 4 GiB: one scalar base and 32-bit offsets
  const uint8_t* qb = a.q + (int64_t)expert * a.M * (K / 2);
  const uint16_t* sb = a.s + (int64_t)expert * a.M * (K / G);

  for (int64_t tile0 = (int64_t)blockIdx.z * T::ROWS; tile0 < cnt; tile0 += (int64_t)gridDim.z * T::ROWS) {
    const int rows = (int)min((int64_t)T::ROWS, cnt - tile0);
    const int kc = T::chunk(rows, K);
    const int pitch = kc + 8;
    // what depends on the lane stays inside the tile: kept over this loop (mostly one turn), it spilled
    int ln = lane;
    asm volatile("" : "+v"(ln));
    const int r16 = ln & 15, j = ln >> 4;
    uint32_t wq[RT], ws[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int c = min(col0, ncols - WCOLS);
      const int m = SWIGLU ? (t & 1) * half + c + 16 * (t >> 1) : c + 16 * t;
      wq[t] = (uint32_t)(m + r16) * (uint32_t)(K / 2);
      ws[t] = (uint32_t)(m + r16) * (uint32_t)(K / G);
    }
    __syncthreads();  // the previous tile's LDS reads are over
    if (tid < rows) {
      int64_t r = row0 + tile0 + tid;
      if (a.row_index) {
        r = a.row_index[r] / a.div;
        r = min(max(r, (int64_t)0), a.x_rows - 1);
      }
      src_rows[tid] = (int)r;
    }
    f32x4 acc[TT][RT];
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
      for (int t = 0; t < RT; ++t) acc[i][t] = f32x4{0.f, 0.f, 0.f, 0.f};

    u32x4 q[RT][NSEG];
    constexpr int SW = (NSEG * GPS + 1) / 2;  // words of a batch's scales, two a word
    uint32_t sc[RT][SW];
    // this wave's batch at k0: 16 bytes per piece and weight tile, and the batch's scales; past K the last
    // valid piece again (the activations there are zero)
    auto load = [&](int k0) {
#pragma unroll
      for (int p = 0; p < NSEG; ++p) {
        const int k = min(k0 + p * SEG + j * 32, K - 32);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          // (not non-temporal: a load takes half of each row's line, and with the hint the line was fetched again
          // for the other half: 32 tokens over 256 experts 451 -> 479 us, one token 20 -> 24 us)
          q[t][p] = *(const u32x4*)(qb + (wq[t] + (uint32_t)(k >> 1)));
        }
      }
      if (k0 + BATCH <= K) {  // the wave's scales of the batch lie together: wide loads
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          sc[t][SW - 1] = 0;
          __builtin_memcpy(sc[t], sb + (ws[t] + (uint32_t)(k0 / G)), 2 * NSEG * GPS);
        }
      } else {
#pragma unroll
        for (int t = 0; t < RT; ++t) {
#pragma unroll
          for (int g = 0; g < SW; ++g) {
            sc[t][g] = sb[ws[t] + (uint32_t)min(k0 / G + 2 * g, K / G - 1)];
            sc[t][g] |= (uint32_t)sb[ws[t] + (uint32_t)min(k0 / G + 2 * g + 1, K / G - 1)] << 16;
          }
        }
      }
    };
    load(kw * BATCH);
    for (int c0 = 0; c0 < K; c0 += kc) {
      __syncthreads();  // src_rows is written; the previous chunk's reads are over
      // stage rows x kc activations (zeros past K), values 0 2 4 6 1 3 5 7 of every eight: a wave takes 512 of one
      // row at a time (its row address is scalar), four of these loads ahead of their writes
      const int runs = (kc + 511) / 512;
      int r = 0, run = wave;
      auto settle = [&]() {
        while (run >= runs) {
          run -= runs;
          ++r;
        }
      };
      for (settle(); r < rows;) {
        u32x4 v[4];
        int to[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int kk = run * 512 + ln * 8;
          to[u] = r < rows && kk < kc ? r * pitch + kk : -1;
          v[u] = u32x4{0, 0, 0, 0};
          if (r < rows) {
            const uint16_t* xr = a.x + (int64_t)__builtin_amdgcn_readfirstlane(src_rows[r]) * K + c0;
            if (kk < kc && c0 + kk < K) v[u] = *(const u32x4*)(xr + kk);
          }
          run += 4;
          settle();
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          u32x4 w;
          w[0] = __builtin_amdgcn_perm(v[u][1], v[u][0], 0x05040100);
          w[1] = __builtin_amdgcn_perm(v[u][3], v[u][2], 0x05040100);
          w[2] = __builtin_amdgcn_perm(v[u][1], v[u][0], 0x07060302);
          w[3] = __builtin_amdgcn_perm(v[u][3], v[u][2], 0x07060302);
          if (to[u] >= 0) *(u32x4*)(xs + to[u]) = w;
        }
      }
      __syncthreads();
      for (int b0 = kw * BATCH; b0 < kc && c0 + b0 < K; b0 += T::STEP) {
        u32x4 cq[RT][NSEG];
        uint32_t cs[RT][SW];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
#pragma unroll
          for (int p = 0; p < NSEG; ++p) cq[t][p] = q[t][p];
#pragma unroll
          for (int g = 0; g < SW; ++g) cs[t][g] = sc[t][g];
        }
        // the next batch is STEP further on, within the chunk or at the next one's start (chunks are
        // whole steps); nothing is read past the row
        if (c0 + b0 + T::STEP < K) load(c0 + b0 + T::STEP);
        // of a 32-row tile with at most 16 rows only the first half (32 tokens over 256 experts, groups of 32: 472 ->
        // 446 us). Groups of 128 hold more activations at a time and spilled with both bodies: they always run the
        // whole tile (one token, 5,120 -> 24,576: 19 us, 25 with both bodies).
        auto batch = [&](auto tiles) {
          constexpr int NT = decltype(tiles)::value;
#pragma unroll
          for (int p = 0; p < NSEG; ++p) {
            if (c0 + b0 + p * SEG >= K) break;
            if (G < SEG) {
#pragma unroll
              for (int t = 0; t < RT; ++t) exchange4(cq[t][p]);
            }
            const uint16_t* xp = xs + b0 + p * SEG;
#pragma unroll
            for (int g = 0; g < GPS; ++g) {
              bf16x8 xf[STEPS][NT];
#pragma unroll
              for (int i = 0; i < NT; ++i) {
#pragma unroll
                for (int u = 0; u < STEPS; ++u) {
                  const int piece = G < SEG ? 4 * (g * STEPS + u) + j : 4 * j + u;
                  xf[u][i] = *(const bf16x8*)(xp + min(16 * i + r16, rows - 1) * pitch + piece * 8);
                }
              }
#pragma unroll
              for (int t = 0; t < RT; ++t) {
                f32x4 sum[NT];
#pragma unroll
                for (int u = 0; u < STEPS; ++u) {
                  const bf16x8 w = unpack8(cq[t][p][g * STEPS + u]);
#pragma unroll
                  for (int i = 0; i < NT; ++i)
                    sum[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[u][i], w, u == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : sum[i],
                                                                     0, 0, 0);
                }
                const uint32_t sw = cs[t][(p * GPS + g) / 2];
                const float s = __uint_as_float((p * GPS + g) & 1 ? sw & 0xffff0000u : sw << 16);
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                  for (int r = 0; r < 4; ++r) acc[i][t][r] += s * sum[i][r];
              }
              // keeps the compiler from reading several groups' activations ahead, which spilled
              __builtin_amdgcn_sched_barrier(0);
            }
          }
        };
        if (TT == 2 && G < SEG && rows <= 16)
          batch(IntC<1>{});
        else
          batch(IntC<TT>{});
      }
    }
    // the waves that split k: partial sums through LDS, added in wave order by the first of them
    {
      constexpr int PER = TT * RT * 4;
      float* red = (float*)xs;  // [4 waves][PER][64 lanes]
      static_assert(4 * PER * 64 * 4 <= T::LDS_ELEMS * 2, "the partial sums fit the activations' space");
      __syncthreads();
#pragma unroll
      for (int i = 0; i < TT; ++i)
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) red[(wave * PER + (i * RT + t) * 4 + r) * 64 + lane] = acc[i][t][r];
      __syncthreads();
      if (kw == 0) {
#pragma unroll
        for (int i = 0; i < TT; ++i)
#pragma unroll
          for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              float v = acc[i][t][r];
              for (int w = 1; w < KS; ++w) v += red[((wave + w) * PER + (i * RT + t) * 4 + r) * 64 + lane];
              acc[i][t][r] = v;
            }
      }
    }
    if (kw == 0 && col0 < ncols) {
#pragma unroll
      for (int i = 0; i < TT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * i + 4 * j + r;
          if (row >= rows) continue;
          uint16_t* y = a.y + (row0 + tile0 + row) * ncols + col0 + r16;
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            if (SWIGLU) {
              if (t & 1) y[8 * (t - 1)] = gated(acc[i][t - 1][r], acc[i][t][r], a.limit);
            } else {
              y[16 * t] = (uint16_t)bf16_pair(acc[i][t][r], 0.f);
            }
          }
        }
    }
  }
}

// Many rows: TT 16-row activation tiles and 256 weight rows per block, all of k in every wave, so that a wave uses
// each value it unpacks for 16 TT rows. The activations pass through two LDS stages of 256 k: half of the next
// stage's rows is in flight in registers during each of the two 128-wide batches of the present one. A batch's
// weights are loaded while the batch before it runs. No load is behind a branch (past the end the last valid piece
// is read again), so every wait names its own loads. Against one stage of twice the length that is loaded, waited
// for and then used: 1,021 rows, 12,288 -> 5,120, groups of 64, 254 -> 230 us; 2,048 rows, 5,120 -> 24,576 SwiGLU,
// groups of 128, 690 -> 590; 1,021 rows, 4,096 -> 4,096, groups of 32, 86 -> 64. (Weights loaded one batch earlier
// into copies of their own: 3% faster with groups of 64, 5-12% slower with 32 and 128; the next group's
// activations read ahead of the present one's products: nothing, or spills.)
//
// One tile of `rows` activation rows, at most 16 TT, from row0 on.
template <int TT, int G, bool SWIGLU>
__device__ __forceinline__ void wide_tile(const QuantArgs& a, int expert, int64_t row0, int rows, int wave, int lane,
                                          uint16_t* lds, int* src_rows) {
  constexpr int RT = 4, ROWS = 16 * TT, STAGE = 2 * SEG, PITCH = STAGE + 8;
  constexpr int GPS = SEG / G, STEPS = G / 32;  // groups per piece, matrix steps per group
  constexpr int XL = TT;                        // this thread's 16-byte loads of half a stage
  constexpr int SW = (GPS + 1) / 2;
  constexpr int WCOLS = SWIGLU ? 8 * RT : 16 * RT;
  const int K = a.K, half = a.M / 2, ncols = SWIGLU ? half : a.M;
  const int tid = wave * 64 + lane;
  const int col0 = (blockIdx.x * 4 + wave) * WCOLS;
  const uint8_t* qb = a.q + (int64_t)expert * a.M * (K / 2);
  const uint16_t* sb = a.s + (int64_t)expert * a.M * (K / G);
  const int stages = (K + STAGE - 1) / STAGE;
  int ln = lane;
  asm volatile("" : "+v"(ln));  // what depends on the lane stays inside the tile
  const int r16 = ln & 15, j = ln >> 4;
  uint32_t wq[RT], ws[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int c = min(col0, ncols - WCOLS);
    const int m = SWIGLU ? (t & 1) * half + c + 16 * (t >> 1) : c + 16 * t;
    wq[t] = (uint32_t)(m + r16) * (uint32_t)(K / 2);
    ws[t] = (uint32_t)(m + r16) * (uint32_t)(K / G);
  }
  __syncthreads();  // the previous tile's LDS reads are over
  if (tid < ROWS) {
    int64_t r = row0 + min(tid, rows - 1);  // rows past the tile repeat its last
    if (a.row_index) {
      r = a.row_index[r] / a.div;
      r = min(max(r, (int64_t)0), a.x_rows - 1);
    }
    src_rows[tid] = (int)r;
  }
  __syncthreads();
  f32x4 acc[TT][RT];
#pragma unroll
  for (int i = 0; i < TT; ++i)
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[i][t] = f32x4{0.f, 0.f, 0.f, 0.f};

  // rows 8 i + tid / 32 of half a stage's rows, values 8 (tid % 32) .. of the stage
  const int xr = wave * 2 + (ln >> 5), xk = (ln & 31) * 8;
  u32x4 xv[XL];
  auto load_x = [&](int stage, int h) {
    const int k = min(stage * STAGE + xk, K - 8);
#pragma unroll
    for (int i = 0; i < XL; ++i)
      xv[i] = *(const u32x4*)(a.x + (int64_t)src_rows[h * (ROWS / 2) + 8 * i + xr] * K + k);
  };
  // zeros past K; values 0 2 4 6 1 3 5 7 of every eight
  auto put_x = [&](int stage, int h) {
    const bool in = stage * STAGE + xk < K;
#pragma unroll
    for (int i = 0; i < XL; ++i) {
      u32x4 v = xv[i], w;
      if (!in) v = u32x4{0, 0, 0, 0};
      w[0] = __builtin_amdgcn_perm(v[1], v[0], 0x05040100);
      w[1] = __builtin_amdgcn_perm(v[3], v[2], 0x05040100);
      w[2] = __builtin_amdgcn_perm(v[1], v[0], 0x07060302);
      w[3] = __builtin_amdgcn_perm(v[3], v[2], 0x07060302);
      *(u32x4*)&lds[((stage & 1) * ROWS + h * (ROWS / 2) + 8 * i + xr) * PITCH + xk] = w;
    }
  };
  static_assert(ROWS / 2 == 8 * XL, "half a stage's rows");

  u32x4 q[2][RT];
  uint32_t sc[2][RT][SW];
  auto load_w = [&](int h, int k0) {
    const int k = min(k0 + j * 32, K - 32);
#pragma unroll
    for (int t = 0; t < RT; ++t) q[h][t] = *(const u32x4*)(qb + (wq[t] + (uint32_t)(k >> 1)));
    // the piece's scales lie together; at the row's end the row's last ones, moved down to where they belong
    const int g = min(k0 / G, K / G - GPS), sh = 16 * (k0 / G - g);
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      if constexpr (GPS == 4) {
        uint64_t v;
        __builtin_memcpy(&v, sb + (ws[t] + (uint32_t)g), 8);
        v >>= sh & 63;
        sc[h][t][0] = (uint32_t)v;
        sc[h][t][1] = (uint32_t)(v >> 32);
      } else if constexpr (GPS == 2) {
        uint32_t v;
        __builtin_memcpy(&v, sb + (ws[t] + (uint32_t)g), 4);
        sc[h][t][0] = v >> (sh & 31);
      } else {
        sc[h][t][0] = sb[ws[t] + (uint32_t)g];
      }
    }
  };
  load_x(0, 0);
  put_x(0, 0);
  load_x(0, 1);
  load_w(0, 0);
  load_w(1, SEG);
  put_x(0, 1);
  for (int st = 0; st < stages; ++st) {
    __syncthreads();  // this stage is written; the reads of the stage that the next one replaces are over
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k0 = st * STAGE + h * SEG;
      if (k0 >= K) break;
      load_x(st + 1, h);
      if (G < SEG) {
#pragma unroll
        for (int t = 0; t < RT; ++t) exchange4(q[h][t]);
      }
      const uint16_t* xp = &lds[((st & 1) * ROWS + r16) * PITCH + h * SEG];
#pragma unroll
      for (int g = 0; g < GPS; ++g) {
        bf16x8 xf[STEPS][TT];
#pragma unroll
        for (int i = 0; i < TT; ++i) {
#pragma unroll
          for (int u = 0; u < STEPS; ++u) {
            const int piece = G < SEG ? 4 * (g * STEPS + u) + j : 4 * j + u;
            xf[u][i] = *(const bf16x8*)(xp + 16 * i * PITCH + piece * 8);
          }
        }
        // the next word is unpacked under the present one's products; with groups of 128 (four steps per sum) the
        // order is set, a product and then a share of the unpacking: with one wave per SIMD nothing else fills the
        // matrix core's time (128 rows, 5,120 -> 24,576: 73 -> 63 us). With fewer steps the compiler's own order is
        // faster (512 rows, 12,288 -> 5,120, groups of 64: 152 us, 184 with the order set).
        bf16x8 next = unpack8(q[h][0][g * STEPS]);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          f32x4 sum[TT];
#pragma unroll
          for (int u = 0; u < STEPS; ++u) {
            const bf16x8 w = next;
            const int n = t * STEPS + u + 1;
            if (n < RT * STEPS) next = unpack8(q[h][n / STEPS][g * STEPS + n % STEPS]);
#pragma unroll
            for (int i = 0; i < TT; ++i)
              sum[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[u][i], w, u == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : sum[i], 0,
                                                               0, 0);
            if (G == SEG) {
#pragma unroll
              for (int i = 0; i < TT; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);        // matrix instructions
                __builtin_amdgcn_sched_group_barrier(0x002, 12 / TT, 0);  // vector ones
              }
            }
          }
          const uint32_t sw = sc[h][t][g / 2];
          const float s = __uint_as_float(g & 1 ? sw & 0xffff0000u : sw << 16);
#pragma unroll
          for (int i = 0; i < TT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[i][t][r] += s * sum[i][r];
        }
      }
      load_w(h, k0 + STAGE);
      put_x(st + 1, h);
    }
  }
  if (col0 < ncols) {
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * i + 4 * j + r;
        if (row >= rows) continue;
        uint16_t* y = a.y + (row0 + row) * ncols + col0 + r16;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          if (SWIGLU) {
            if (t & 1) y[8 * (t - 1)] = gated(acc[i][t - 1][r], acc[i][t][r], a.limit);
          } else {
            y[16 * t] = (uint16_t)bf16_pair(acc[i][t][r], 0.f);
          }
        }
      }
  }
}

// EXPERTS: a tile of at most 32 rows runs a body of its own (256 experts 6,144 -> 4,096, 24 / 64 rows each: 1,480 ->
// 1,379, 2,527 -> 2,412 us). A dense product has at most one such tile and keeps one body, which takes fewer
// registers (12,288 -> 5,120, 1,021 rows: 231 us, 239 with both); so does the form that both would make spill. Two
// waves per SIMD at most: the 48-row form with groups of 32 has the registers for three blocks per CU and is slower with
// them (256 experts 6,144 -> 4,096, 32 rows each: 1,628 us, 1,940 with three).
template <int TT, int G, bool SWIGLU, bool EXPERTS>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void qlinear_wide_kernel(QuantArgs a) {
  constexpr int ROWS = 16 * TT;
  __shared__ __attribute__((aligned(16))) uint16_t lds[2 * ROWS * (2 * SEG + 8)];
  __shared__ int src_rows[ROWS];
  const int expert = blockIdx.y;
  int64_t row0 = 0, cnt = a.R;
  if (a.offsets) {
    row0 = min(max((int64_t)a.offsets[expert], (int64_t)0), a.R);
    cnt = min(max((int64_t)a.offsets[expert + 1], row0), a.R) - row0;
  }
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int64_t tile0 = (int64_t)blockIdx.z * ROWS; tile0 < cnt; tile0 += (int64_t)gridDim.z * ROWS) {
    const int rows = (int)min((int64_t)ROWS, cnt - tile0);
    if (EXPERTS && !(TT == 4 && G == SEG) && rows <= 32)
      wide_tile<2, G, SWIGLU>(a, expert, row0 + tile0, rows, wave, lane, lds, src_rows);
    else
      wide_tile<TT, G, SWIGLU>(a, expert, row0 + tile0, rows, wave, lane, lds, src_rows);
  }
}

template <int TT, int G>
hipError_t launch_wide_group(const QuantArgs& a, hipStream_t s) {
  constexpr int ROWS = 16 * TT;
  const int wcols = a.swiglu ? 128 : 256, ncols = a.swiglu ? a.M / 2 : a.M;
  int64_t z = (a.R + (int64_t)a.E * ROWS - 1) / ((int64_t)a.E * ROWS);  // as in launch_q
  if (a.E > 1 && z > 1) z *= 2;
  if (z > 65535) z = 65535;
  const dim3 grid((ncols + wcols - 1) / wcols, a.E, (unsigned)z);
  auto launch = [&](auto swiglu, auto experts) {
    hipLaunchKernelGGL((qlinear_wide_kernel<TT, G, decltype(swiglu)::value, decltype(experts)::value>), grid, dim3(256), 0,
                       s, a);
  };
  if (a.E > 1 && a.swiglu)
    launch(std::true_type{}, std::true_type{});
  else if (a.E > 1)
    launch(std::false_type{}, std::true_type{});
  else if (a.swiglu)
    launch(std::true_type{}, std::false_type{});
  else
    launch(std::false_type{}, std::false_type{});
  return hipGetLastError();
}

template <int TT>
hipError_t launch_wide(const QuantArgs& a, hipStream_t s) {
  if (a.group == 32) return launch_wide_group<TT, 32>(a, s);
  if (a.group == 64) return launch_wide_group<TT, 64>(a, s);
  return launch_wide_group<TT, 128>(a, s);
}

template <class T, int G>
hipError_t launch_q(const QuantArgs& a, hipStream_t s) {
  const int wcols = (a.swiglu ? 8 : 16) * T::RT * T::WAVE_N, ncols = a.swiglu ? a.M / 2 : a.M;
  // row tiles side by side: what an even load needs, twice that for experts with more rows than the others (a
  // block takes every z-th tile of its expert)
  int64_t z = (a.R + (int64_t)a.E * T::ROWS - 1) / ((int64_t)a.E * T::ROWS);
  if (a.E > 1 && z > 1) z *= 2;
  if (z > 65535) z = 65535;
  const dim3 grid((ncols + wcols - 1) / wcols, a.E, (unsigned)z);
  if (a.swiglu)
    hipLaunchKernelGGL((qlinear_kernel<T, G, true>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((qlinear_kernel<T, G, false>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

template <class T>
hipError_t launch_group(const QuantArgs& a, hipStream_t s) {
  if (a.group == 32) return launch_q<T, 32>(a, s);
  if (a.group == 64) return launch_q<T, 64>(a, s);
  return launch_q<T, 128>(a, s);
}

// One thread per eight values, group / 8 neighbouring lanes per group: the group's largest magnitude over
// 7, rounded to bfloat16, is the scale; a value is the nearest integer (ties to even) of its quotient by
// that scale, kept within [-8, 7]. A group of zeros has the scale 0 and the values 0. The largest magnitude is taken of
// the bits, where a NaN is above an infinity and that above every number, so that a group with either has it as its
// scale and shows in every product; its values are 0.
template <typename T>
__global__ __launch_bounds__(256) void quantize_kernel(const T* __restrict__ w, int64_t pieces, int lanes_per_group,
                                                       uint32_t* __restrict__ q, uint16_t* __restrict__ s) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const bool live = i < pieces;
  float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (live) widen8(raw_load8(w + i * 8), f);
  int m = 0;
#pragma unroll
  for (int u = 0; u < 8; ++u) m = max(m, __float_as_int(f[u]) & 0x7fffffff);
  for (int off = 1; off < lanes_per_group; off <<= 1) m = max(m, __shfl_xor(m, off));
  const uint16_t sb = (uint16_t)bf16_pair(__int_as_float(m) / 7.0f, 0.f);
  const float sf = bf16_f32(sb);
  const bool usable = sf > 0.f && sf < __builtin_inff();
  uint32_t word = 0;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const float v = usable ? fminf(fmaxf(rintf(f[u] / sf), -8.f), 7.f) : 0.f;
    word |= (uint32_t)((int)v + 8) << (4 * u);
  }
  if (!live) return;
  q[i] = word;
  if (i % lanes_per_group == 0) s[i / lanes_per_group] = sb;
}

}  // namespace

// Which form runs, by the average rows per expert r and the blocks a form makes (256 CUs). Measured, us, on
// dense 12,288 -> 5,120 (groups of 64), dense 5,120 -> 24,576 (SwiGLU, groups of 128) and 256 experts 6,144 -> 4,096
// with eight rows a token (SwiGLU, groups of 32):
//   narrow, 16 rows, k over four waves      1 / 64 / 128 rows: 17 / 59 / 95 | 16 / 79 / 144 | 1 / 32 / 256 tokens: 36 / 435 / 1,006
//   middle, 32 rows, k over two waves       28 / 85 / 99                    | 20 / 52 / 96  | 41 / 447 / 904
//   wide, 64 or 48 rows, all of k per wave  149 / 150 / 149                 | 52 / 55 / 62  | 121 / 736 / 1,163
// The narrow form reads the activations most often but makes the most and shortest blocks. It wins while the middle
// form makes fewer than one block per CU (experts without rows make none that count), and for up to 16 rows in all,
// when no expert has more than one of its tiles, unless k is shorter than two of its steps of 1,024 (16 rows,
// narrow / middle: 12,288 -> 16,384 47 / 54, 4,096 -> 16,384 20 / 22; 1 row, 4,096 -> 16,384 12 / 15; one token, 128
// experts 4,096 -> 2,816 19 / 25 and 1,408 -> 4,096 15 / 14). The wide form shares each unpacked value among 48 or 64 rows. For
// a dense product it wins from about 96 rows on, once it makes blocks for five eighths of the CUs (12,288 -> 5,120,
// middle / wide: 256 rows, 120 blocks, 122 / 148; 384 rows, 160 blocks, 180 / 149; 512 rows 200 / 150). For experts it
// wins from 24 rows each (128 experts 1,408 -> 4,096, 24 rows: 195 / 154; of 256 experts 6,144 -> 4,096 with groups of
// 32 24 rows 1,427 / 1,433, 32 rows 1,736 / 1,643).
// Of its two heights a dense product takes the one whose last round of blocks leaves less idle (1,021 rows,
// 12,288 -> 5,120: 262 with 64 rows, 235 with 48; 768 rows 168 and 235), experts the lower one up to 64 rows each
// (128 experts, 24 / 64 / 128 rows: 147 / 241 / 371 with 64 rows, 154 / 238 / 431 with 48).
hipError_t launch_qlinear(const QuantArgs& a, hipStream_t s) {
  constexpr int64_t kCus = 256;
  auto up = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
  const int64_t r = up(a.R, a.E), live = a.R < a.E ? a.R : a.E;  // live: experts with rows, at most
  const int64_t blocks64 = up(a.M, 256) * a.E * up(r, 64), blocks48 = up(a.M, 256) * a.E * up(r, 48);
  const bool low = a.E > 1 ? r <= 64 : up(blocks48, kCus) * 3 < up(blocks64, kCus) * 4;
  if (a.K >= SEG && r >= (a.E > 1 ? 24 : 96) && (low ? blocks48 : blocks64) * 8 >= kCus * 5)
    return low ? launch_wide<3>(a, s) : launch_wide<4>(a, s);
  const bool few = a.R <= 16 && a.K >= 2048;
  if (!few && up(a.M, 64) * live * up(r, 32) >= kCus) return launch_group<QTile<2, 2, 2, 2, 16384, 3>>(a, s);
  return launch_group<QTile<1, 4, 2, 2, 16384, 4>>(a, s);
}

hipError_t launch_quantize(int dtype, const void* w, int64_t rows, int K, int group, uint8_t* q, uint16_t* s,
                           hipStream_t st) {
  const int64_t pieces = rows * (K / 8);
  const int64_t blocks = (pieces + 255) / 256;
  if (blocks == 0) return hipSuccess;
  if (dtype == MOE_F32)
    hipLaunchKernelGGL(quantize_kernel<float>, dim3((unsigned)blocks), dim3(256), 0, st, (const float*)w, pieces,
                       group / 8, (uint32_t*)q, s);
  else
    hipLaunchKernelGGL(quantize_kernel<uint16_t>, dim3((unsigned)blocks), dim3(256), 0, st, (const uint16_t*)w, pieces,
                       group / 8, (uint32_t*)q, s);
  return hipGetLastError();
}

}  // namespace moe
