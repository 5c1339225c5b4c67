// C ABI entry points of the operators around the layer (declared and documented in include/moe.h): block
// norms, combine, grouped products, 4-bit products. Argument checks on the host, the workspace carve-up,
// and the launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "ops_internal.h"

using namespace moe;

namespace {

constexpr int kMaxE = 512, kMaxK = 32, kMaxNormD = 16384;
constexpr int64_t kInt31 = (int64_t)1 << 31, kGiB4 = (int64_t)1 << 32;

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
template <typename... P>
bool all_aligned16(P... p) {
  return (aligned16(p) && ...);
}
size_t align_up(size_t v) { return (v + 255) & ~(size_t)255; }
// A launch holds fewer than 2^32 threads: what would take more is refused here, before anything is launched.
bool launch_fits(int64_t blocks, int64_t threads) { return blocks <= (kGiB4 - 1) / threads; }
bool dtype_ok(int32_t t) { return t == MOE_F32 || t == MOE_BF16; }

moe_status check_norm(int64_t N, int32_t D, int32_t dtype, float eps, float a) {
  if (N < 0 || D < 1 || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.f || !std::isfinite(a)) return MOE_ERR_INVALID_ARG;
  if (D % 64 != 0 || D > kMaxNormD || N >= kInt31) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Most blocks norm_plan can choose for at most N rows, with B = norm_runs(D) and c = ceil(N / B) rows a run: B
// without a gate or with whole gate groups in a run; otherwise (T > c) ceil(N / T) groups of ceil(T / c) runs, at
// most N / c + N / T + T / c + 1, each term at most B; and no more than 2 N, reached with c = 1.
int64_t norm_blocks_bound(int64_t N, int D, bool gate) {
  const int64_t B = norm_runs(D);
  return gate ? std::min<int64_t>(2 * N, 3 * B + 1) : std::min<int64_t>(N, B);
}

moe_status check_combine(int64_t N, int32_t k, int32_t D, int32_t dtype, int64_t R, float alpha) {
  if (N < 0 || k < 1 || D < 1 || R < 0 || !dtype_ok(dtype) || !std::isfinite(alpha)) return MOE_ERR_INVALID_ARG;
  if (k > kMaxK || D % 64 != 0 || N >= kInt31 || N * k >= kInt31 || R >= kInt31) return MOE_ERR_UNSUPPORTED;
  if (!launch_fits(N, combine_threads(D))) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_grouped(int32_t E, int64_t R, int32_t in, int32_t out, int32_t dtype) {
  if (E < 1 || R < 0 || in < 1 || out < 1 || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
  if (E > kMaxE || in % 64 != 0 || out % 64 != 0 || R >= kInt31) return MOE_ERR_UNSUPPORTED;
  // the bf16 kernels address an expert's matrix with 32-bit byte offsets
  if (dtype == MOE_BF16 && (int64_t)in * out * 2 >= kGiB4) return MOE_ERR_UNSUPPORTED;
  if ((int64_t)in * out >= kInt31 || in > (1 << 22) || out > (1 << 22)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// The rows a grouped call reads: x_rows rows of x, through row_index or one for one.
moe_status check_source(int64_t R, int64_t x_rows, const int32_t* row_index, int32_t index_div, int32_t in,
                        int32_t dtype) {
  if (x_rows < 0) return MOE_ERR_INVALID_ARG;
  if (x_rows >= kInt31) return MOE_ERR_UNSUPPORTED;
  if (row_index) {
    if (index_div < 1 || (R > 0 && x_rows < 1)) return MOE_ERR_INVALID_ARG;
    // gathered rows are addressed with 32-bit byte offsets from x
    if (dtype == MOE_BF16 && x_rows * in * 2 >= kGiB4) return MOE_ERR_UNSUPPORTED;
  } else if (x_rows < R) {
    return MOE_ERR_INVALID_ARG;
  }
  return MOE_OK;
}

struct GroupedLayout {
  size_t tiles0, tiles1, ntiles, src_row, part, part_bytes, total;
  int64_t max_tiles0, max_tiles1;
  int bm0, bm1, pick;
};

// Lists of the forward product: as the layer's own (moe_forward) for bf16, 128-row tiles for float32. List 1
// serves dgrad too (256-row tiles). What depends on R is sized so that it never falls as R grows: the tile
// height drops to 16 rows only below a threshold of rows, and the larger of the two counts is taken.
GroupedLayout grouped_layout(int32_t E, int64_t R, int32_t dtype) {
  GroupedLayout w{};
  const bool f32 = dtype == MOE_F32;
  w.pick = f32 ? 0 : device_pick_rows(dtype, R, 1, E);
  w.bm0 = f32 ? kF32Rows : w.pick ? 16 : gemm_bm(dtype, R, 1, E);
  w.bm1 = f32 ? kF32Rows : kGradRows;
  w.max_tiles0 = max_tiles(R, 1, E, 0, f32 ? kF32Rows : w.bm0);
  w.max_tiles1 = max_tiles(R, 1, E, 0, w.bm1);
  // 16-row lists hold at most R / 16 + E tiles, and only while R < MOE_PICK_BAND_ROWS * E; 256-row lists
  // with their padding at most R / 256 + 4 E
  const int64_t small_rows = std::min<int64_t>(R, (int64_t)tile_plan_rows(1) * E);
  const int64_t room0 = f32 ? w.max_tiles0 : std::max(w.max_tiles1, max_tiles(small_rows, 1, E, 0, 16));
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes);
    return at;
  };
  w.tiles0 = take(sizeof(Tile) * room0);
  w.tiles1 = take(f32 ? 0 : sizeof(Tile) * w.max_tiles1);
  w.ntiles = take(sizeof(int32_t) * 22);  // two tile counts, 8 work counters per list, two hot counts, row range
  w.src_row = take(sizeof(int32_t) * R);
  // float32 parts of a reduction that is split (grouped_splits): a call with few rows needs little of it
  w.part_bytes = (size_t)std::min<int64_t>(R, 32) << 19;
  w.part = take(w.part_bytes);
  w.total = o;
  return w;
}

template <typename T>
T* at(void* ws, size_t off) {
  return (T*)((char*)ws + off);
}

}  // namespace

extern "C" {

// ---- block norms ----
size_t moe_block_norm_workspace_size(int64_t N, int32_t D, int32_t dtype, int64_t gate_rows) {
  if (check_norm(N, D, dtype, 0.f, 0.f) != MOE_OK || gate_rows < 0) return 0;
  return sizeof(float) * (gate_rows > 0 ? 3 : 2) * (size_t)norm_blocks_bound(N, D, gate_rows > 0) * D;
}

moe_status moe_block_norm(int64_t N, int32_t D, int32_t dtype, float eps, float residual_scale, const void* h,
                          const void* o, const void* w_post, const void* gate, int64_t gate_rows, const void* w_pre,
                          void* h_out, void* u, void* stream) {
  const moe_status st = check_norm(N, D, dtype, eps, residual_scale);
  if (st != MOE_OK) return st;
  if (gate && gate_rows < 1) return MOE_ERR_INVALID_ARG;
  if (!launch_fits(N, norm_forward_threads(D))) return MOE_ERR_UNSUPPORTED;
  if (N == 0) return MOE_OK;
  if (!h || (!o && (w_post || gate || h_out)) || (o && !h_out)) return MOE_ERR_INVALID_ARG;
  if ((w_pre == nullptr) != (u == nullptr) || (!o && !w_pre)) return MOE_ERR_INVALID_ARG;
  if (!all_aligned16(h, o, w_post, gate, w_pre, h_out, u)) return MOE_ERR_INVALID_ARG;
  if (h_out && h_out == o) return MOE_ERR_INVALID_ARG;
  if (u && (u == h || u == o || u == h_out)) return MOE_ERR_INVALID_ARG;
  hipStream_t s = (hipStream_t)stream;
  NormCall c{};
  c.N = N;
  c.D = D;
  c.eps = eps;
  c.a = residual_scale;
  c.h = h;
  c.o = o;
  c.w_post = w_post;
  c.gate = gate;
  c.gate_rows = gate_rows;
  c.w_pre = w_pre;
  c.h_out = h_out;
  c.u = u;
  MOE_TRY(ST_BLOCK_NORM, launch_norm_forward(dtype, c, s));
  return MOE_OK;
}

moe_status moe_block_norm_backward(int64_t N, int32_t D, int32_t dtype, float eps, float residual_scale,
                                   const void* h_out, const void* o, const void* w_post, const void* gate,
                                   int64_t gate_rows, const void* w_pre, const void* dh_out, const void* du, void* dh,
                                   void* d_o, float* dw_post, float* dgate, float* dw_pre, void* workspace,
                                   size_t ws_bytes, void* stream) {
  const moe_status st = check_norm(N, D, dtype, eps, residual_scale);
  if (st != MOE_OK) return st;
  if (gate && gate_rows < 1) return MOE_ERR_INVALID_ARG;
  if ((dw_post && !w_post) || (dgate && !gate) || (dw_pre && !w_pre)) return MOE_ERR_INVALID_ARG;
  if (!all_aligned16(dw_post, dgate, dw_pre)) return MOE_ERR_INVALID_ARG;
  hipStream_t s = (hipStream_t)stream;
  if (N == 0) {  // sums over no rows
    const int64_t n = dw_post ? D : 0, m = dw_pre ? D : 0;
    if (launch_fill2_i32((int32_t*)dw_post, n, (int32_t*)dw_pre, m, 0, s) != hipSuccess) return MOE_ERR_HIP;
    return MOE_OK;
  }
  if (!o && (w_post || gate || d_o)) return MOE_ERR_INVALID_ARG;
  if ((o && !d_o) || !dh || (!dh_out && !du) || (!o && !w_pre)) return MOE_ERR_INVALID_ARG;
  if ((w_pre == nullptr) != (du == nullptr) || (w_pre && !h_out)) return MOE_ERR_INVALID_ARG;
  if (!all_aligned16(h_out, o, w_post, gate, w_pre, dh_out, du, dh, d_o)) return MOE_ERR_INVALID_ARG;
  if (dh == h_out || dh == o || dh == du || dh == d_o) return MOE_ERR_INVALID_ARG;
  if (d_o && (d_o == h_out || d_o == o || d_o == du || d_o == dh_out)) return MOE_ERR_INVALID_ARG;
  const bool sums = dw_post || dgate || dw_pre;
  if (sums && (!workspace || !aligned16(workspace) ||
               ws_bytes < moe_block_norm_workspace_size(N, D, dtype, gate ? gate_rows : 0)))
    return MOE_ERR_WORKSPACE;
  NormCall c{};
  c.N = N;
  c.D = D;
  c.eps = eps;
  c.a = residual_scale;
  c.h = h_out;
  c.o = o;
  c.w_post = w_post;
  c.gate = gate;
  c.gate_rows = gate_rows;
  c.w_pre = w_pre;
  c.dh_out = dh_out;
  c.du = du;
  c.dh = dh;
  c.d_o = d_o;
  c.dw_post = dw_post;
  c.dgate = dgate;
  c.dw_pre = dw_pre;
  c.part = (float*)workspace;
  MOE_TRY(ST_BLOCK_NORM, launch_norm_backward(dtype, c, s));
  return MOE_OK;
}

// ---- combine ----
moe_status moe_combine(int64_t N, int32_t k, int32_t D, int32_t dtype, const void* rows, int64_t R,
                       const int32_t* inv_row, const float* topk_w, const void* shared, float alpha, void* y,
                       void* stream) {
  const moe_status st = check_combine(N, k, D, dtype, R, alpha);
  if (st != MOE_OK) return st;
  if (N == 0) return MOE_OK;
  if (!inv_row || !y || (R > 0 && !rows) || (rows && rows == y)) return MOE_ERR_INVALID_ARG;
  if (!all_aligned16(rows, shared, y)) return MOE_ERR_INVALID_ARG;
  hipStream_t s = (hipStream_t)stream;
  MOE_TRY(ST_COMBINE, launch_combine_rows(dtype, rows, R, inv_row, topk_w, shared, N, k, D, alpha, y, s));
  return MOE_OK;
}

moe_status moe_combine_backward(int64_t N, int32_t k, int32_t D, int32_t dtype, const void* dy, const void* rows,
                                int64_t R, const int32_t* inv_row, const float* topk_w, float alpha, void* drows,
                                float* dtopk_w, void* stream) {
  const moe_status st = check_combine(N, k, D, dtype, R, alpha);
  if (st != MOE_OK) return st;
  if (N == 0) return MOE_OK;
  if (!dy || !inv_row || (R > 0 && !drows) || (dtopk_w && !topk_w)) return MOE_ERR_INVALID_ARG;
  if (dtopk_w && R > 0 && !rows) return MOE_ERR_INVALID_ARG;
  if (drows && (drows == dy || drows == rows)) return MOE_ERR_INVALID_ARG;
  if (!all_aligned16(dy, rows, drows)) return MOE_ERR_INVALID_ARG;
  hipStream_t s = (hipStream_t)stream;
  MOE_TRY(ST_COMBINE,
          launch_combine_rows_backward(dtype, dy, rows, R, inv_row, topk_w, N, k, D, alpha, drows, dtopk_w, s));
  return MOE_OK;
}

// ---- grouped products ----
size_t moe_grouped_workspace_size(int32_t E, int64_t R, int32_t dtype) {
  if (check_grouped(E, R, 64, 64, dtype) != MOE_OK) return 0;
  return grouped_layout(E, R, dtype).total;
}

moe_status moe_grouped_linear(int32_t E, int64_t R, int32_t in, int32_t out, int32_t dtype, const void* x,
                              int64_t x_rows, const int32_t* row_index, int32_t index_div, const void* w,
                              const int32_t* offsets, void* y, void* workspace, size_t ws_bytes, void* stream) {
  moe_status st = check_grouped(E, R, in, out, dtype);
  if (st != MOE_OK) return st;
  if ((st = check_source(R, x_rows, row_index, index_div, in, dtype)) != MOE_OK) return st;
  if (R == 0) return MOE_OK;
  if (!x || !w || !offsets || !y || x == y || !all_aligned16(x, w, y)) return MOE_ERR_INVALID_ARG;
  const GroupedLayout L = grouped_layout(E, R, dtype);
  const int splits = dtype == MOE_F32 ? grouped_splits(GM_FWD, dtype, E, R, out, in, L.part_bytes) : 1;
  // (the 16-row form of the expert GEMMs takes 128 columns per block; the others launch one block per CU)
  if (dtype == MOE_F32 ? !launch_fits(grouped_f32_blocks(GM_FWD, E, out, in, splits, L.max_tiles0), 256)
                       : L.bm0 == 16 && !launch_fits(L.max_tiles0 * ((out + 127) / 128) + 7, 256))
    return MOE_ERR_UNSUPPORTED;
  if (!workspace || ws_bytes < L.total || !aligned16(workspace)) return MOE_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  void* ws = workspace;
  int32_t* ntiles = at<int32_t>(ws, L.ntiles);
  int32_t* src = row_index ? at<int32_t>(ws, L.src_row) : nullptr;
  const TileSpec none{0, nullptr, nullptr, 0, nullptr, nullptr};
  const TileSpec t0{L.bm0, at<Tile>(ws, L.tiles0), ntiles, small_expert_rows(dtype, L.bm0), ntiles + 2, ntiles + 18};
  const TileSpec t1{L.bm1, at<Tile>(ws, L.tiles1), ntiles + 1, small_expert_rows(dtype, L.bm1), ntiles + 10,
                    ntiles + 19};
  MOE_TRY(ST_GROUPED_LISTS, launch_offset_lists(offsets, E, R, t0, L.pick ? t1 : none, L.pick, row_index, index_div,
                                                x_rows, src, ntiles + 20, s));
  if (dtype == MOE_F32) {
    const GradArgs g{x, w, y, R, out, in, E, offsets, src, x_rows, t0.tiles, ntiles, nullptr,
                     splits, at<float>(ws, L.part), ntiles + 20};
    MOE_TRY(ST_GROUPED_LINEAR, launch_grouped_f32(GM_FWD, g, L.max_tiles0, s));
    if (g.splits > 1) MOE_TRY(ST_GROUPED_LINEAR, launch_grouped_join(GM_FWD, dtype, g, s));
    return MOE_OK;
  }
  // the layer's expert GEMM without its row scale; source rows are resolved already (k = 1)
  GroupedArgs g{};
  g.sorted_pair = src;
  g.k = 1;
  g.gather_rows = x_rows;
  g.prob[0] = ExpertProblem{x, in, row_index ? 1 : 0, w, nullptr, (int64_t)out * in, in, out, y, out, 0};
  for (int list = 0; list < (L.pick ? 2 : 1); ++list) {
    g.tiles = list ? t1.tiles : t0.tiles;
    g.n_tiles = ntiles + list;
    g.work_ctr = ntiles + (list ? 10 : 2);
    g.n_hot = ntiles + 18 + list;
    g.bm = list ? L.bm1 : L.bm0;
    MOE_TRY(ST_GROUPED_LINEAR, launch_down(dtype, g, list ? L.max_tiles1 : L.max_tiles0, s));
  }
  return MOE_OK;
}

moe_status moe_grouped_linear_dgrad(int32_t E, int64_t R, int32_t in, int32_t out, int32_t dtype, const void* dy,
                                    const void* w, const int32_t* offsets, void* dx, void* workspace, size_t ws_bytes,
                                    void* stream) {
  const moe_status st = check_grouped(E, R, in, out, dtype);
  if (st != MOE_OK) return st;
  if (R == 0) return MOE_OK;
  if (!dy || !w || !offsets || !dx || dy == dx || !all_aligned16(dy, w, dx)) return MOE_ERR_INVALID_ARG;
  const GroupedLayout L = grouped_layout(E, R, dtype);
  const int splits = grouped_splits(GM_DGRAD, dtype, E, R, out, in, L.part_bytes);
  if (dtype == MOE_F32 && !launch_fits(grouped_f32_blocks(GM_DGRAD, E, out, in, splits, L.max_tiles1), 256))
    return MOE_ERR_UNSUPPORTED;
  if (!workspace || ws_bytes < L.total || !aligned16(workspace)) return MOE_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  void* ws = workspace;
  int32_t* ntiles = at<int32_t>(ws, L.ntiles);
  const TileSpec none{0, nullptr, nullptr, 0, nullptr, nullptr};
  const TileSpec t0{L.bm1, at<Tile>(ws, L.tiles0), ntiles, small_expert_rows(dtype, L.bm1), ntiles + 2, ntiles + 18};
  MOE_TRY(ST_GROUPED_LISTS, launch_offset_lists(offsets, E, R, t0, none, 0, nullptr, 1, 0, nullptr, ntiles + 20, s));
  const GradArgs g{dy, w, dx, R, out, in, E, offsets, nullptr, 0, t0.tiles, ntiles, ntiles + 2,
                   splits, at<float>(ws, L.part), ntiles + 20};
  MOE_TRY(ST_GROUPED_LINEAR, dtype == MOE_F32 ? launch_grouped_f32(GM_DGRAD, g, L.max_tiles1, s)
                                              : launch_grouped_bf16(GM_DGRAD, g, L.max_tiles1, s));
  if (g.splits > 1) MOE_TRY(ST_GROUPED_LINEAR, launch_grouped_join(GM_DGRAD, dtype, g, s));
  return MOE_OK;
}

moe_status moe_grouped_linear_wgrad(int32_t E, int64_t R, int32_t in, int32_t out, int32_t dtype, const void* dy,
                                    const void* x, int64_t x_rows, const int32_t* row_index, int32_t index_div,
                                    const int32_t* offsets, void* dw, void* workspace, size_t ws_bytes,
                                    void* stream) {
  moe_status st = check_grouped(E, R, in, out, dtype);
  if (st != MOE_OK) return st;
  if ((st = check_source(R, x_rows, row_index, index_div, in, dtype)) != MOE_OK) return st;
  if (!dw || !offsets || (R > 0 && (!dy || !x))) return MOE_ERR_INVALID_ARG;
  if (dw == dy || dw == x || !all_aligned16(dy, x, dw)) return MOE_ERR_INVALID_ARG;
  const GroupedLayout L = grouped_layout(E, R, dtype);
  const int splits = grouped_splits(GM_WGRAD, dtype, E, R, out, in, L.part_bytes);
  if (dtype == MOE_F32 && !launch_fits(grouped_f32_blocks(GM_WGRAD, E, out, in, splits, 0), 256))
    return MOE_ERR_UNSUPPORTED;
  if (!workspace || ws_bytes < L.total || !aligned16(workspace)) return MOE_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  int32_t* src = nullptr;
  if (row_index && R > 0) {
    src = at<int32_t>(workspace, L.src_row);
    const TileSpec none{0, nullptr, nullptr, 0, nullptr, nullptr};
    MOE_TRY(ST_GROUPED_LISTS, launch_offset_lists(offsets, E, R, none, none, 0, row_index, index_div, x_rows, src, nullptr, s));
  }
  const GradArgs g{dy, x, dw, R, out, in, E, offsets, src, x_rows, nullptr, nullptr, nullptr,
                   splits, at<float>(workspace, L.part), nullptr};
  MOE_TRY(ST_GROUPED_LINEAR,
          dtype == MOE_F32 ? launch_grouped_f32(GM_WGRAD, g, 0, s) : launch_grouped_bf16(GM_WGRAD, g, 0, s));
  if (g.splits > 1) MOE_TRY(ST_GROUPED_LINEAR, launch_grouped_join(GM_WGRAD, dtype, g, s));
  return MOE_OK;
}

// ---- 4-bit weights ----
moe_status moe_qlinear(int32_t E, int64_t R, int32_t in, int32_t out, int32_t group, const void* x, int64_t x_rows,
                       const int32_t* row_index, int32_t index_div, const void* wq, const void* scales,
                       const int32_t* offsets, int32_t swiglu, float swiglu_limit, void* y, void* stream) {
  moe_status st = check_grouped(E, R, in, out, MOE_BF16);
  if (st != MOE_OK) return st;
  if (group != 32 && group != 64 && group != 128) return group < 1 ? MOE_ERR_INVALID_ARG : MOE_ERR_UNSUPPORTED;
  if (in % group != 0) return MOE_ERR_INVALID_ARG;
  if (swiglu != 0 && swiglu != 1) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(swiglu_limit) || swiglu_limit < 0.f || (swiglu_limit > 0.f && !swiglu)) return MOE_ERR_INVALID_ARG;
  if (swiglu && out % 128 != 0) return MOE_ERR_UNSUPPORTED;
  if ((st = check_source(R, x_rows, row_index, index_div, in, MOE_F32)) != MOE_OK) return st;
  if (E > 1 && !offsets) return MOE_ERR_INVALID_ARG;
  if (R == 0) return MOE_OK;
  if (!x || !wq || !scales || !y || x == y || !all_aligned16(x, wq, scales, y)) return MOE_ERR_INVALID_ARG;
  hipStream_t s = (hipStream_t)stream;
  const QuantArgs a{(const uint16_t*)x, (const uint8_t*)wq, (const uint16_t*)scales, offsets, row_index, index_div,
                    x_rows, R, E, out, in, group, swiglu, swiglu_limit, (uint16_t*)y};
  MOE_TRY(ST_QLINEAR, launch_qlinear(a, s));
  return MOE_OK;
}

moe_status moe_quantize(int32_t dtype, int64_t rows, int32_t in, int32_t group, const void* w, void* wq, void* scales,
                        void* stream) {
  if (!dtype_ok(dtype) || rows < 0 || in < 1) return MOE_ERR_INVALID_ARG;
  if (group != 32 && group != 64 && group != 128) return group < 1 ? MOE_ERR_INVALID_ARG : MOE_ERR_UNSUPPORTED;
  if (in % group != 0) return MOE_ERR_INVALID_ARG;
  // a thread per eight values, in whole blocks of 256
  if (in % 64 != 0 || rows > (kGiB4 - 256) / (in / 8)) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!w || !wq || !scales || !all_aligned16(w, wq, scales)) return MOE_ERR_INVALID_ARG;
  if (wq == w || scales == w || wq == scales) return MOE_ERR_INVALID_ARG;
  hipStream_t s = (hipStream_t)stream;
  MOE_TRY(ST_QUANTIZE, launch_quantize(dtype, w, rows, in, group, (uint8_t*)wq, (uint16_t*)scales, s));
  return MOE_OK;
}

}  // extern "C"
