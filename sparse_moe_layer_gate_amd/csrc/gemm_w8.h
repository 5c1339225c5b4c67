// 256 x 256 tiles of eight waves in bf16: the LDS ring's layout, the waits, the walk over tiles that keeps an XCD's
// blocks on common operands. Shared by the grouped expert GEMMs and the dense linear maps, which have a K loop each.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>

#include "moe_internal.h"

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// ---- eight-wave kernels for 256-row tiles ----
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
//    of each per step (buffer_load_dwordx4 ... lds through raw buffer descriptors).
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
