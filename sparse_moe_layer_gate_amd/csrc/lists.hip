// Row-tile lists and source rows of the grouped products, from offsets and indices that the caller gives.
#include <hip/hip_runtime.h>

#include "ops_internal.h"

namespace moe {
namespace {

// Inclusive running sum / maximum of one int per thread over a 512-thread block: shuffles inside each wave, then
// the waves before it. `tmp` holds one int per wave and is free again when the call returns.
template <bool MAX>
__device__ int block_running(int v, int* tmp) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int y = __shfl_up(v, off);
    if (lane >= off) v = MAX ? max(v, y) : v + y;
  }
  if (lane == 63) tmp[wave] = v;
  __syncthreads();
  for (int w = 0; w < wave; ++w) v = MAX ? max(v, tmp[w]) : v + tmp[w];
  __syncthreads();
  return v;
}

// One list: the tiles of the experts with more than small_max rows, in expert order, each expert's padded with
// empty tiles to MOE_TILE_ALIGN in the 256-row lists (its tiles then share a rasterization rectangle of the
// expert GEMM), then the single tiles of the smaller ones, which mostly stream their expert's weights.
__device__ void write_list(const TileSpec& ts, int e, int start, int cnt, int* tmp, int* total) {
  const int nt = (cnt + ts.bm - 1) / ts.bm;
  const bool small = cnt >= 1 && cnt <= ts.small_max && cnt <= ts.bm;
  const int align = ts.small_max > 0 ? MOE_TILE_ALIGN : 1;
  const int slots = small ? 0 : (nt + align - 1) / align * align;
  const int first = block_running<false>(slots, tmp) - slots;
  const int rank = block_running<false>(small ? 1 : 0, tmp) - (small ? 1 : 0);
  if (threadIdx.x == blockDim.x - 1) {  // the last thread's running sums are the totals
    total[0] = first + slots;
    total[1] = rank + (small ? 1 : 0);
  }
  __syncthreads();
  if (small) {
    ts.tiles[total[0] + rank] = Tile{0, e, start, cnt};
  } else {
    for (int j = 0; j < slots; ++j)
      ts.tiles[first + j] = Tile{0, e, j < nt ? start + j * ts.bm : start, j < nt ? min(ts.bm, cnt - j * ts.bm) : 0};
  }
  if (threadIdx.x == 0) {
    *ts.n_tiles = total[0] + total[1];
    if (ts.n_hot) *ts.n_hot = 0;
  }
  if (ts.work_ctr && threadIdx.x < 8) ts.work_ctr[threadIdx.x] = 0;
  __syncthreads();  // `total` is reused by the next list
}

// Block 0: the lists of the rows that `offsets` [E + 1] groups; the other blocks: the source row of every grouped
// row. Ranges are kept within [0, R] and in order (each start is the largest offset so far), so that the lists
// never hold more than R rows, and source rows within [0, x_rows).
__global__ __launch_bounds__(512) void offset_lists_kernel(const int32_t* __restrict__ offsets, int E, int64_t R,
                                                           TileSpec t0, TileSpec t1, int pick_rows,
                                                           const int32_t* __restrict__ row_index, int32_t div,
                                                           int64_t x_rows, int32_t* __restrict__ src_row,
                                                           int32_t* __restrict__ row_range) {
  if (blockIdx.x > 0) {
    const int64_t r = (int64_t)(blockIdx.x - 1) * 512 + threadIdx.x;
    if (r < R) src_row[r] = (int32_t)min(max((int64_t)(row_index[r] / div), (int64_t)0), x_rows - 1);
    return;
  }
  __shared__ int tmp[8], total[2];
  __shared__ int max_cnt;
  if (threadIdx.x == 0) max_cnt = 0;
  const int e = threadIdx.x;  // E <= 512: one expert per thread
  const int lo = e < E ? (int)min(max((int64_t)offsets[e], (int64_t)0), R) : 0;
  const int hi = e < E ? (int)min(max((int64_t)offsets[e + 1], (int64_t)0), R) : 0;
  const int start = block_running<true>(lo, tmp);
  const int cnt = e < E ? max(hi - start, 0) : 0;
  if (row_range && e == 0) row_range[0] = lo;
  if (row_range && e == E - 1) row_range[1] = max(start, hi);  // the experts' ranges lie end to end
  if (pick_rows > 0 && cnt > 0) atomicMax(&max_cnt, cnt);  // read after the lists' barriers
  if (t0.tiles) write_list(t0, e, start, cnt, tmp, total);
  if (t1.tiles) write_list(t1, e, start, cnt, tmp, total);
  // both lists written: empty the one whose kernels do not run (thread 0 wrote both counts)
  if (pick_rows > 0 && threadIdx.x == 0) *(max_cnt <= pick_rows ? t1.n_tiles : t0.n_tiles) = 0;
}

}  // namespace

hipError_t launch_offset_lists(const int32_t* offsets, int E, int64_t R, TileSpec t0, TileSpec t1, int pick_rows,
                               const int32_t* row_index, int32_t div, int64_t x_rows, int32_t* src_row,
                               int32_t* row_range, hipStream_t s) {
  if (E > 512) return hipErrorInvalidValue;
  const int64_t blocks = 1 + (row_index ? (R + 511) / 512 : 0);
  hipLaunchKernelGGL(offset_lists_kernel, dim3((unsigned)blocks), dim3(512), 0, s, offsets, E, R, t0, t1, pick_rows,
                     row_index, div, x_rows, src_row, row_range);
  return hipGetLastError();
}

}  // namespace moe
