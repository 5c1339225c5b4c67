// The eight-wave bf16 K loop for 256 x 256 tiles, shared by the grouped expert GEMMs and the dense linear maps, with
// the walk over tiles that keeps an XCD's blocks on common operands.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>

#include "moe_internal.h"

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// ---- eight-wave kernel for 256-row tiles ----
//
// With one wave per SIMD, the wave that issues a K step's direct loads stalls while the texture path
// accepts them (the CU's waves issue theirs within a short window of the step, so they queue behind
// one another), and its SIMD's matrix core idles meanwhile. Here each SIMD runs two waves (w and w + 4),
// each with its own 64 x 128 share of the tile, its own fragment reads and an eighth of every step's
// loads: while one of them waits on the load path, the other keeps the matrix core busy.
//  - block tile 256 x 256, BK = 64 (whole 128-byte lines per row and load); A in a two-stage ring, B
//    in a three-stage ring, together all 160 KiB of LDS; rows chunk-swizzled (Wave8Tile::swz);
//  - half g = w / 4 owns tile rows [128 g, 128 g + 128); wave w % 4 = 2 wn + mh owns 64 rows (mh) of
//    that half and 128 B rows (wn), as 2 x 4 tiles of v_mfma_f32_32x32x16_bf16 (gate_up: 64 gate rows
//    and the matching 64 up rows, so SwiGLU pairs stay in one wave);
//  - the waves of half g load rows [128 g, 128 g + 128) of both operands, four direct loads per lane
//    of each per step (buffer_load_dwordx4 ... lds through raw buffer descriptors);
//  - per K step t a wave issues its A loads of step t + 1 and works through the step's four 16-wide K
//    slices with the fragments double-buffered by slice: the reads of slice s + 1 are in flight while
//    slice s's MFMAs run. It issues its B loads of step t + 2 with the second slice, waits for its
//    loads of step t + 1, meets the others at a barrier, and then reads step t + 1's first slice while
//    the last slice's MFMAs run. A stage is refilled only after every wave has passed the barrier that
//    follows its last read; A loads get about one step to land and B loads two.
template <bool GATE_UP>
struct Wave8Tile {
  static constexpr int BM = 256, BN = 256, BK = 64;
  static constexpr int ROWB = BK * 2;          // bytes per LDS row
  static constexpr int OPB = 256 * ROWB;       // one operand's bytes per stage (32 KiB)
  static constexpr int A_STAGES = 2, B_STAGES = 3;
  static constexpr int B_BASE = A_STAGES * OPB;
  static constexpr int RING = (A_STAGES + B_STAGES) * OPB;
  static constexpr int NL = 4;                 // direct loads per lane and quarter (128 rows of one operand)
  static constexpr int COLS = GATE_UP ? BN / 2 : BN;  // output columns per block
  static constexpr int OC = GATE_UP ? 64 : 128;       // output columns per wave
  __device__ static int swz(int r) {
    r &= 31;
    return (r ^ (r >> 3)) & 7;
  }
  // LDS row (within a B stage) of the wave's column tile j
  __device__ static int b_row(int j, int wn) {
    if (GATE_UP) return (j < 2 ? 0 : BN / 2) + wn * 64 + (j & 1) * 32;
    return wn * 128 + j * 32;
  }
};

template <bool V>
struct BoolC {
  static constexpr bool value = V;
};
template <int V>
struct IntC {
  static constexpr int value = V;
};

// Word 3 of a raw (untyped, stride 0) buffer descriptor on gfx9-family parts: 32-bit data format, no
// swizzle, no index stride.
constexpr int kRawBufferWord3 = 0x00020000;

// s_waitcnt lgkmcnt(0), other counters at their maximum
__device__ inline void wait_lgkm0() { __builtin_amdgcn_s_waitcnt((15) | (3 << 14) | (7 << 4) | (0 << 8)); }
// Workgroup barrier without the memory-counter waits __syncthreads() adds (callers wait for exactly
// what they need first); the signal fences keep the compiler from moving memory accesses across it.
__device__ inline void bare_barrier() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// The K loop of one wave. offA / offB: byte offsets of this wave's direct-load sources in its half's
// rows; na: how many of its A loads reach a valid row (the others are not issued; lanes of an issued
// load past the tile repeat its last row). B is never skipped, so a wave's newest NL loads are always
// B loads, which is what the vmcnt(NL) waits rely on.
template <bool GATE_UP, int MI>
__device__ __attribute__((always_inline)) inline void wave8_loop(char* lds, __amdgpu_buffer_rsrc_t rsrcA,
                                                                 const uint32_t (&offA)[4], int na,
                                                                 __amdgpu_buffer_rsrc_t rsrcB, const uint32_t (&offB)[4],
                                                                 f32x16 (&acc)[2][4], int nk, int grp, int q, int lane,
                                                                 int m0, int wn) {
  using T = Wave8Tile<GATE_UP>;
  constexpr int NL = T::NL, TN = 4, ROWB = T::ROWB;
  const int sw = T::swz(lane & 31);
  const int a_off = (m0 + (lane & 31)) * ROWB;
  int b_off[TN];
#pragma unroll
  for (int j = 0; j < TN; ++j) b_off[j] = (T::b_row(j, wn) + (lane & 31)) * ROWB;
  const int half_off = grp * (T::OPB / 2) + q * 1024;  // this wave's first LDS chunk run in a stage

  // this wave's loads of step kstep: load i fills chunks [(4 i + q) 64, + 64) of its half's rows; the K
  // offset rides in the scalar offset
  auto issue_a = [&](int kstep) {
    char* dst = lds + (kstep % T::A_STAGES) * T::OPB + half_off;
#pragma unroll
    for (int i = 0; i < NL; ++i)
      if (i < na)  // wave-uniform: loads wholly past the tile's rows are not issued
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrcA, (lds_void*)(dst + i * 4096), 16, (int)offA[i], kstep * T::BK * 2,
                                                 0, 0);
  };
  auto issue_b = [&](int kstep) {
    char* dst = lds + T::B_BASE + (kstep % T::B_STAGES) * T::OPB + half_off;
#pragma unroll
    for (int i = 0; i < NL; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrcB, (lds_void*)(dst + i * 4096), 16, (int)offB[i], kstep * T::BK * 2,
                                               0, 0);
  };
  // Fragments of one 16-wide K slice (kstep's slice sl) into buffer buf; the reads are only issued
  // here, and the waits below order them. A wave with no valid rows reads nothing.
  constexpr int NR = MI > 0 ? MI + TN : 0;  // LDS reads per slice
  bf16x8 af[2][MI > 0 ? MI : 1], bfr[2][TN];
  auto read_slice = [&](int kstep, int sl, int buf) {
    if (MI == 0) return;
    const char* sa = lds + (kstep % T::A_STAGES) * T::OPB;
    const char* sb = lds + T::B_BASE + (kstep % T::B_STAGES) * T::OPB;
    const int coff = ((2 * sl + (lane >> 5)) ^ sw) * 16;
#pragma unroll
    for (int j = 0; j < TN; ++j) bfr[buf][j] = *(const bf16x8*)(sb + b_off[j] + coff);
#pragma unroll
    for (int i = 0; i < MI; ++i) af[buf][i] = *(const bf16x8*)(sa + a_off + i * 32 * ROWB + coff);
  };
  auto compute = [&](int buf) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(af[buf][i], bfr[buf][j], acc[i][j], 0, 0, 0);
  };
  // Scheduling fence: without it the compiler sinks each fragment read next to its first MFMA and
  // waits for it there, so the matrix core idles for an LDS round trip per read.
  auto fence = [] { __builtin_amdgcn_sched_barrier(0); };
  // s_waitcnt lgkmcnt(NR): all but the newest slice's reads have landed
  auto wait_older_slices = [] { __builtin_amdgcn_s_waitcnt((15) | (3 << 14) | (7 << 4) | (NR << 8)); };

  // prologue: this wave's rows of A(0), B(0), B(1); wait for step 0; read its first slice
  issue_a(0);
  issue_b(0);
  if (nk > 1) {
    issue_b(1);
    wait_vmcnt<NL>();  // B loads are never skipped: the newest NL are step 1's
  } else {
    wait_vmcnt<0>();
  }
  bare_barrier();
  read_slice(0, 0, 0);
  fence();
  // The steps that issue both operands' loads run in a loop of their own, free of the branches and of
  // the variable waits of the last two steps, which are peeled (with the small-tile loop peeled the same
  // way, against one loop with the conditions inside: dense FFN gate_up 1.74 -> 1.65 ms, skewed GLM-4.5
  // layer 4.22 -> 4.08 ms, Air 1.75 -> 1.63 ms; 239 -> 207 VGPRs in gate_up). The slice double buffer
  // against reading whole K halves, which the compiler had interleaved read by read with the MFMAs:
  // gate_up 1-2% faster on every layer (skewed GLM-4.5 2.35 -> 2.34 ms, mild skew 2.23 -> 2.19,
  // GLM-5 3.88 -> 3.83, Air 0.90 -> 0.89).
  auto step = [&](int kt, auto more_a, auto more_b, auto last) {
    constexpr bool MA = decltype(more_a)::value, MB = decltype(more_b)::value, LAST = decltype(last)::value;
    // step kt is in LDS (A stage kt % 2, B stage kt % 3), its slice 0 being read into buffer 0
    if (MA) issue_a(kt + 1);  // into the A stage step kt - 1 used (every wave is done with it)
    read_slice(kt, 1, 1);
    fence();
    wait_older_slices();
    compute(0);
    fence();
    read_slice(kt, 2, 0);
    fence();
    wait_older_slices();
    if (MB) issue_b(kt + 2);  // into the B stage step kt - 1 used
    compute(1);
    fence();
    read_slice(kt, 3, 1);
    fence();
    wait_older_slices();
    compute(0);
    fence();
    wait_lgkm0();
    // step kt + 1 has landed (only this wave's B loads of step kt + 2 may still be in flight)
    if (MB)
      wait_vmcnt<NL>();
    else if (MA)
      wait_vmcnt<0>();
    bare_barrier();
    if (!LAST) read_slice(kt + 1, 0, 0);
    fence();
    compute(1);  // the last slice, while the next step's first reads land
    fence();
  };
  int kt = 0;
  for (; kt + 2 < nk; ++kt) step(kt, BoolC<true>{}, BoolC<true>{}, BoolC<false>{});
  if (kt + 1 < nk) step(kt++, BoolC<true>{}, BoolC<false>{}, BoolC<false>{});
  step(kt, BoolC<false>{}, BoolC<false>{}, BoolC<true>{});
}

// Logical block L of a region of n_region row tiles -> (row tile within the region, column tile): walk
// rectangles of GR row tiles x GC column tiles (the last ones of a row group or of the region smaller),
// row tiles fastest.
template <int GR, int GC>
__device__ inline void raster(int64_t L, int ncol_max, int64_t n_region, int64_t& tile_rel, int& ct) {
  const int64_t sg = L / ((int64_t)GR * ncol_max), within = L % ((int64_t)GR * ncol_max);
  const int64_t gr = min((int64_t)GR, n_region - sg * GR);
  const int64_t cg = within / (gr * GC), w2 = within % (gr * GC);
  tile_rel = sg * GR + w2 % gr;
  ct = (int)(cg * GC + w2 / gr);
}

// Blocks of the persistent kernel: one per CU of the current device (a multiple of 8: every XCD gets
// the same number), queried once per device.
int64_t persistent_grid() {
  static std::atomic<int> cached[64];  // 0 until queried; callers on several threads may race to fill it
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
}  // namespace moe
