// Internal declarations of the operators around the layer (block norms, combine, grouped products, 4-bit
// products) and of a training step (layer norm, linear maps, balance loss, gradient norm), shared by their
// translation units.
#pragma once

#include "moe_internal.h"

namespace moe {

// Timing slots of these operators, behind the forward's (moe_combine and its gradients use ST_COMBINE).
enum OpStage {
  ST_BLOCK_NORM = ST_COUNT_STAGES,  // moe_block_norm and its gradients
  ST_GROUPED_LISTS,                 // tile lists and source rows of the moe_grouped_* calls
  ST_GROUPED_LINEAR,                // moe_grouped_linear and its gradients
  ST_QLINEAR,                       // moe_qlinear
  ST_QUANTIZE,                      // moe_quantize
  ST_LAYER_NORM,                    // moe_layer_norm and its gradients
  ST_LINEAR,                        // moe_linear and its gradients
  ST_BALANCE,                       // moe_balance_loss
  ST_ROUTE_BACKWARD,                // moe_route_backward
  ST_GRAD_NORM,                     // moe_grad_norm
  ST_GRAD_CLIP,                     // moe_grad_clip
  ST_ALL_STAGES
};

// A launch of an entry point, as one recorded stage on the call's stream `s`.
#define MOE_TRY(stage, expr)                 \
  do {                                       \
    prof_before((stage), s);                 \
    const hipError_t e_ = (expr);            \
    prof_after((stage), s);                  \
    if (e_ != hipSuccess) return MOE_ERR_HIP; \
  } while (0)

// ---- argument checks ----
constexpr int64_t kInt31 = (int64_t)1 << 31, kGiB4 = (int64_t)1 << 32;
inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
template <typename... P>
bool all_aligned16(P... p) {
  return (aligned16(p) && ...);
}
// A launch holds fewer than 2^32 threads: what would take more is refused here, before anything is launched.
inline bool launch_fits(int64_t blocks, int64_t threads) { return blocks <= (kGiB4 - 1) / threads; }
inline bool dtype_ok(int32_t t) { return t == MOE_F32 || t == MOE_BF16; }

// ---- combine ----
int combine_threads(int D);  // of the one block per token
// y = alpha * sum over slots of w rows[inv_row] + shared (w or shared may be null)
hipError_t launch_combine_rows(int dtype, const void* rows, int64_t R, const int32_t* inv_row, const float* w,
                               const void* shared, int64_t N, int k, int D, float alpha, void* y, hipStream_t s);
// drows[inv_row] = alpha w dy, dw = alpha <dy, rows[inv_row]> (w, and with it dw, may be null)
hipError_t launch_combine_rows_backward(int dtype, const void* dy, const void* rows, int64_t R,
                                        const int32_t* inv_row, const float* w, int64_t N, int k, int D, float alpha,
                                        void* drows, float* dw, hipStream_t s);

// ---- block norms ----
struct NormCall {
  int64_t N;
  int D;
  float eps, a;
  const void *h, *o, *w_post, *gate, *w_pre;  // backward: h is h_out
  int64_t gate_rows;
  void *h_out, *u;  // forward
  const void *dh_out, *du;  // backward
  void *dh, *d_o;
  float *dw_post, *dgate, *dw_pre, *part;
};
struct NormPlan {
  int64_t chunk;             // rows per block of the backward pass
  int64_t chunks_per_group;  // > 0: the blocks of one gate group; 0: blocks hold whole groups (or no gate)
  int64_t nblocks;
};
int norm_forward_threads(int D);  // of the one block per row
int64_t norm_runs(int D);  // most runs of rows without a gate
NormPlan norm_plan(int64_t N, int D, int64_t gate_rows);  // gate_rows 0: no gate
hipError_t launch_norm_forward(int dtype, const NormCall& c, hipStream_t s);
hipError_t launch_norm_backward(int dtype, const NormCall& c, hipStream_t s);

// ---- grouped products and their gradients ----
// Row-tile lists of rows grouped by `offsets` [E + 1] (made monotone and kept within [0, R]), and, with
// row_index, the source row of every grouped row, kept within [0, x_rows). row_range (or nullptr): the first grouped
// row and the one behind the last.
hipError_t launch_offset_lists(const int32_t* offsets, int E, int64_t R, TileSpec t0, TileSpec t1, int pick_rows,
                               const int32_t* row_index, int32_t div, int64_t x_rows, int32_t* src_row,
                               int32_t* row_range, hipStream_t s);
enum GroupedMode {
  GM_FWD = 0,  // y = x W^T    (float32 only: the bf16 product runs on the expert GEMMs)
  GM_DGRAD,    // dx = dy W
  GM_WGRAD     // dW = dy^T x over each expert's rows
};
struct GradArgs {
  const void* a;            // x or dy rows
  const void* b;            // W [E, M, K], or x rows (wgrad)
  void* out;
  int64_t R;
  int M, K, E;
  const int32_t* offsets;   // wgrad
  const int32_t* src_row;   // x rows of the grouped rows, or nullptr
  int64_t x_rows;
  const Tile* tiles;        // fwd / dgrad
  const int32_t* n_tiles;
  int32_t* work_ctr;        // bf16 dgrad: 8 counters, zero at launch
  // splits > 1: the reduction in that many parts, each writing its own float32 output (fwd / dgrad [R, J], wgrad
  // [E, M, K]) into `part`; launch_grouped_join adds them in order
  int splits;
  float* part;
  const int32_t* row_range;  // fwd / dgrad: first grouped row and the one behind the last
};
hipError_t launch_grouped_bf16(GroupedMode mode, const GradArgs& a, int64_t max_tile_count, hipStream_t s);
hipError_t launch_grouped_f32(GroupedMode mode, const GradArgs& a, int64_t max_tile_count, hipStream_t s);
int64_t grouped_f32_blocks(GroupedMode mode, int E, int M, int K, int splits, int64_t max_tile_count);  // of 256 threads
int grouped_splits(GroupedMode mode, int dtype, int E, int64_t R, int M, int K, size_t part_bytes);
hipError_t launch_grouped_join(GroupedMode mode, int dtype, const GradArgs& a, hipStream_t s);
constexpr int kGradRows = 256;  // rows per tile of the bf16 dgrad list
constexpr int kF32Rows = 128;   // rows per tile of the float32 lists

// ---- 4-bit weights ----
struct QuantArgs {
  const uint16_t* x;       // [x_rows, K] bf16
  const uint8_t* q;        // [E, M, K / 2]
  const uint16_t* s;       // [E, M, K / group] bf16
  const int32_t* offsets;  // [E + 1], or nullptr: one expert with all R rows
  const int32_t* row_index;
  int32_t div;
  int64_t x_rows, R;
  int E, M, K, group;
  int swiglu;
  float limit;
  uint16_t* y;
};
hipError_t launch_qlinear(const QuantArgs& a, hipStream_t s);
hipError_t launch_quantize(int dtype, const void* w, int64_t rows, int K, int group, uint8_t* q, uint16_t* s,
                           hipStream_t st);

// ---- layer norm ----
struct LayerNormCall {
  int64_t N;
  int D;
  float eps;
  const void *x, *residual, *w, *b;  // backward: x is h
  void *h_out, *y;
  float* stats;
  const void *dh_out, *dy;  // backward
  void* dh;
  float *dw, *db, *part;
};
int layer_norm_threads(int D);  // of a block of the forward pass
int64_t layer_norm_blocks(int64_t N, int D);
int64_t layer_norm_runs(int D);  // most runs of rows, each with a partial row of dw and of db
hipError_t launch_layer_norm(int dtype, const LayerNormCall& c, bool backward, hipStream_t s);
// dst[c] = sum over rows of src[r, c], in a fixed order, for one or two (src1 not null) arrays [rows, D]; D a multiple
// of 4
hipError_t launch_column_sums(const float* src0, float* dst0, const float* src1, float* dst1, int64_t rows, int D,
                              hipStream_t s);

// ---- linear maps ----
struct LinearCall {
  int64_t R;
  int in, out, act;
  const void *x, *w, *bias, *residual;
  void *z, *y;
  float* part;
};
struct LinearPlan {
  int bm, bn;  // rows and columns of a tile
  int splits;  // parts of the reduction
};
LinearPlan linear_plan(int dtype, int64_t R, int in, int out);
size_t linear_part_bytes(int64_t R, int out);  // workspace; never falls as R grows
hipError_t launch_linear(int dtype, const LinearCall& c, hipStream_t s);
struct LinearBackCall {
  int64_t R;
  int out, act;
  const void *dy, *z;
  void* dz;
  float *dbias, *part;
};
int64_t linear_back_runs(int dtype, int64_t R, int out);  // most partial rows of dbias
hipError_t launch_linear_back(int dtype, const LinearBackCall& c, hipStream_t s);

// ---- balance loss and the router's gradient ----
struct BalancePlan {
  int64_t T, S;           // rows per sequence (at most N), sequences
  int64_t chunk, chunks;  // rows per block, blocks per sequence
  int threads;
  int join_parts, join_threads;  // blocks per sequence of the second launch, where chunks > 1; S is below 256 then
};
BalancePlan balance_plan(int64_t N, int64_t T, int E);
struct BalanceCall {
  int64_t N, T;
  int E, k;
  float weight;
  const float* scores;
  const int32_t* idx;
  const uint8_t* mask;
  int32_t* counts;
  float *coef, *loss;
  float* part_p;    // [S chunks, E], with more than one chunk
  int32_t* part_c;  // [S chunks, E]
  int32_t* part_v;  // [S chunks]
  float* part_l;    // [S], with more than one sequence of one chunk; [S join_parts] of several
  int32_t* done;    // [1], with more than one chunk
};
hipError_t launch_balance(const BalanceCall& c, hipStream_t s);
struct RouteBackCall {
  int64_t N, T;
  int E, k;
  float alpha, eps;
  int norm;
  const float* scores;
  const int32_t* idx;
  const float *dw, *coef, *dloss;
  const uint8_t* mask;
  float* out;
};
int64_t route_backward_blocks(int64_t N, int E);  // of 256 threads
hipError_t launch_route_backward(const RouteBackCall& c, hipStream_t s);

// ---- gradient norm and clipping ----
int64_t tensor_chunks(const moe_tensor* t, int n);  // partial sums of the norm of a list
hipError_t launch_grad_norm(const moe_tensor* t, int n, double* part, float* norm, hipStream_t s);
hipError_t launch_grad_clip(const moe_tensor* t, const moe_tensor* out, int n, const float* norm, float max_norm,
                            float eps, hipStream_t s);

}  // namespace moe
