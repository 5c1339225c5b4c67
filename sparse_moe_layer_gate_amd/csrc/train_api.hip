// C ABI entry points of a training step around the layer (declared and documented in include/moe.h): layer norm,
// linear maps, the balance loss and the router's gradient, the gradient norm and clipping. Argument checks on the
// host, the workspace carve-up, and the launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <memory>
#include <new>

#include "ops_internal.h"

using namespace moe;

namespace {

constexpr int64_t kInt40 = (int64_t)1 << 40;
size_t align_up(size_t v) { return (v + 255) & ~(size_t)255; }

// A workspace that has to hold `need` bytes (0: it may be missing).
bool workspace_ok(const void* p, size_t have, size_t need) {
  return need == 0 || (p && aligned16(p) && have >= need);
}

// ---- layer norm ----
moe_status check_layer_norm(int64_t N, int32_t D, int32_t dtype) {
  if (N < 0 || D < 1 || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
  if (D % 8 != 0 || D > 16384 || N >= kInt31) return MOE_ERR_UNSUPPORTED;
  if (!launch_fits(layer_norm_blocks(N, D), layer_norm_threads(D))) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// ---- linear maps ----
moe_status check_linear(int64_t R, int32_t in, int32_t out, int32_t dtype) {
  if (R < 0 || in < 1 || out < 1 || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
  if (in % 64 != 0 || out % 8 != 0 || in > (1 << 22) || out > (1 << 22)) return MOE_ERR_UNSUPPORTED;
  if ((int64_t)in * out >= kInt31 || R >= kInt31 || R > (kInt40 - 1) / out) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
bool activation_ok(int32_t a) { return a >= MOE_ACT_NONE && a <= MOE_ACT_GELU_TANH; }

// ---- balance loss ----
moe_status check_routing(const moe_config* cfg, int64_t N, int64_t seq_rows) {
  const moe_status st = moe_check_config(cfg);
  if (st != MOE_OK) return st;
  if (N < 0 || seq_rows < 1) return MOE_ERR_INVALID_ARG;
  if (N >= kInt31 / cfg->num_experts_per_tok || N > (kInt40 - 1) / cfg->n_routed_experts) return MOE_ERR_UNSUPPORTED;
  if (!launch_fits(route_backward_blocks(N, cfg->n_routed_experts), 256)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

struct BalanceLayout {
  size_t part_p, part_c, part_v, part_l, done, total;
};
BalanceLayout balance_layout(const BalancePlan& p, int E) {
  BalanceLayout w{};
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes);
    return at;
  };
  const size_t parts = p.chunks > 1 ? (size_t)p.S * p.chunks : 0;
  w.part_p = take(4 * parts * E);
  w.part_c = take(4 * parts * E);
  w.part_v = take(4 * parts);
  w.part_l = take(parts ? 4 * (size_t)p.S * p.join_parts : p.S > 1 ? 4 * (size_t)p.S : 0);
  w.done = take(parts ? 4 : 0);
  w.total = o;
  return w;
}
// What any batch of up to N rows may need: sequences of at most 512 rows, or 256 of them, have a block each, and the others
// share at most 1,024 chunks of 32 rows and more, the last sequence counted as long as the others.
size_t balance_bytes(const BalancePlan& p, int64_t N, int E) {
  BalancePlan most = p;
  most.S = std::min<int64_t>(p.S, 255);
  most.chunks = 1;
  if (p.T <= 512) {
    most.S = p.S;
    return balance_layout(most, E).total;
  }
  const int64_t parts = 2 * std::min<int64_t>((N + 31) / 32, 1024) + most.S;
  const size_t shares = 4 * (size_t)std::max(p.S, most.S * p.join_parts);
  return 2 * align_up(4 * (size_t)parts * E) + align_up(4 * (size_t)parts) + align_up(shares) + 256;
}
bool balance_fits(const BalancePlan& p) { return launch_fits(p.S * p.chunks, p.threads); }

// ---- tensor lists ----
size_t value_bytes(const moe_tensor& t) { return t.dtype == MOE_BF16 ? 2 : 4; }

moe_status check_tensors(const moe_tensor* t, int32_t n) {
  if (n < 0 || (n > 0 && !t)) return MOE_ERR_INVALID_ARG;
  if (n > 65536) return MOE_ERR_UNSUPPORTED;
  int64_t all = 0;
  for (int i = 0; i < n; ++i) {
    if (t[i].numel < 0 || !dtype_ok(t[i].dtype)) return MOE_ERR_INVALID_ARG;
    if (t[i].numel > 0 && (!t[i].data || (uintptr_t)t[i].data % value_bytes(t[i]) != 0)) return MOE_ERR_INVALID_ARG;
    if (t[i].numel > kInt40) return MOE_ERR_UNSUPPORTED;
    all += t[i].numel;
  }
  return all > kInt40 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// Non-empty tensors one behind the other in memory, as views of a buffer usually are.
bool ascending(const moe_tensor* t, int32_t n) {
  uintptr_t end = 0;
  for (int i = 0; i < n; ++i) {
    if (t[i].numel == 0) continue;
    if ((uintptr_t)t[i].data < end) return false;
    end = (uintptr_t)t[i].data + t[i].numel * value_bytes(t[i]);
  }
  return true;
}

// Whether no tensor that a clip writes overlaps another one of either list (an out[i] that is tensors[i] aside). Lists
// that lie in order and apart need no sorting.
enum class Overlap { None, Some, Unknown };
Overlap clip_overlap(const moe_tensor* in, const moe_tensor* out, int32_t n) {
  struct Range {
    uintptr_t begin, end;
    bool written;
  };
  const moe_tensor* w = out ? out : in;
  auto end_of = [](const moe_tensor& t) { return (uintptr_t)t.data + t.numel * value_bytes(t); };
  if (ascending(w, n)) {
    if (!out) return Overlap::None;
    uintptr_t lo[2] = {~(uintptr_t)0, ~(uintptr_t)0}, hi[2] = {0, 0};
    for (int k = 0; k < 2; ++k)
      for (int i = 0; i < n; ++i) {
        const moe_tensor& t = k ? out[i] : in[i];
        if (t.numel == 0) continue;
        lo[k] = std::min(lo[k], (uintptr_t)t.data);
        hi[k] = std::max(hi[k], end_of(t));
      }
    if (lo[0] >= hi[1] || lo[1] >= hi[0]) return Overlap::None;
  }
  std::unique_ptr<Range[]> r(new (std::nothrow) Range[2 * (size_t)n]);
  if (!r) return Overlap::Unknown;
  size_t m = 0;
  for (int i = 0; i < n; ++i) {
    if (w[i].numel == 0) continue;
    r[m++] = {(uintptr_t)w[i].data, end_of(w[i]), true};
    if (out && !(out[i].data == in[i].data && out[i].dtype == in[i].dtype))
      r[m++] = {(uintptr_t)in[i].data, end_of(in[i]), false};
  }
  std::sort(r.get(), r.get() + m, [](const Range& a, const Range& b) { return a.begin < b.begin; });
  uintptr_t written = 0, read = 0;  // the furthest ends so far
  for (size_t i = 0; i < m; ++i) {
    if (r[i].begin < written || (r[i].written && r[i].begin < read)) return Overlap::Some;
    (r[i].written ? written : read) = std::max(r[i].written ? written : read, r[i].end);
  }
  return Overlap::None;
}

}  // namespace

extern "C" {

// ---- layer norm ----
size_t moe_layer_norm_workspace_size(int64_t N, int32_t D, int32_t dtype) {
  if (check_layer_norm(N, D, dtype) != MOE_OK) return 0;
  return sizeof(float) * 2 * (size_t)std::min(N, layer_norm_runs(D)) * D;
}

moe_status moe_layer_norm(int64_t N, int32_t D, int32_t dtype, float eps, const void* x, const void* residual,
                          const void* w, const void* b, void* h_out, void* y, float* stats, void* stream) {
  const moe_status st = check_layer_norm(N, D, dtype);
  if (st != MOE_OK) return st;
  if (!std::isfinite(eps) || eps < 0.f) return MOE_ERR_INVALID_ARG;
  if (N == 0) return MOE_OK;
  if (!x || !y || (residual == nullptr) != (h_out == nullptr)) return MOE_ERR_INVALID_ARG;
  if (!all_aligned16(x, residual, w, b, h_out, y, stats)) return MOE_ERR_INVALID_ARG;
  if (y == x || y == residual || y == h_out) return MOE_ERR_INVALID_ARG;
  hipStream_t s = (hipStream_t)stream;
  LayerNormCall c{};
  c.N = N;
  c.D = D;
  c.eps = eps;
  c.x = x;
  c.residual = residual;
  c.w = w;
  c.b = b;
  c.h_out = h_out;
  c.y = y;
  c.stats = stats;
  MOE_TRY(ST_LAYER_NORM, launch_layer_norm(dtype, c, false, s));
  return MOE_OK;
}

moe_status moe_layer_norm_backward(int64_t N, int32_t D, int32_t dtype, const void* h, const float* stats,
                                   const void* w, const void* dh_out, const void* dy, void* dh, float* dw, float* db,
                                   void* workspace, size_t ws_bytes, void* stream) {
  const moe_status st = check_layer_norm(N, D, dtype);
  if (st != MOE_OK) return st;
  if (!all_aligned16(dw, db) || (dw && dw == db)) return MOE_ERR_INVALID_ARG;
  hipStream_t s = (hipStream_t)stream;
  if (N == 0) {  // sums over no rows
    MOE_TRY(ST_LAYER_NORM, launch_fill2_i32((int32_t*)dw, dw ? D : 0, (int32_t*)db, db ? D : 0, 0, s));
    return MOE_OK;
  }
  if (!h || !stats || !dy || !dh) return MOE_ERR_INVALID_ARG;
  if (!all_aligned16(h, stats, w, dh_out, dy, dh)) return MOE_ERR_INVALID_ARG;
  if (dh == h || dh == dy) return MOE_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, ws_bytes, dw || db ? moe_layer_norm_workspace_size(N, D, dtype) : 0))
    return MOE_ERR_WORKSPACE;
  LayerNormCall c{};
  c.N = N;
  c.D = D;
  c.x = h;
  c.stats = (float*)stats;
  c.w = w;
  c.dh_out = dh_out;
  c.dy = dy;
  c.dh = dh;
  c.dw = dw;
  c.db = db;
  c.part = (float*)workspace;
  MOE_TRY(ST_LAYER_NORM, launch_layer_norm(dtype, c, true, s));
  return MOE_OK;
}

// ---- linear maps ----
size_t moe_linear_workspace_size(int64_t R, int32_t in, int32_t out, int32_t dtype) {
  if (check_linear(R, in, out, dtype) != MOE_OK) return 0;
  return linear_part_bytes(R, out);
}

moe_status moe_linear(int64_t R, int32_t in, int32_t out, int32_t dtype, int32_t activation, const void* x,
                      const void* w, const void* bias, const void* residual, void* z, void* y, void* workspace,
                      size_t ws_bytes, void* stream) {
  const moe_status st = check_linear(R, in, out, dtype);
  if (st != MOE_OK) return st;
  if (!activation_ok(activation)) return MOE_ERR_INVALID_ARG;
  if (R == 0) return MOE_OK;
  const LinearPlan p = linear_plan(dtype, R, in, out);
  const int64_t blocks = (R + p.bm - 1) / p.bm * ((out + p.bn - 1) / p.bn) * p.splits;
  if (p.bn != 256 && !launch_fits(blocks, 512)) return MOE_ERR_UNSUPPORTED;  // 256-column tiles: one block per CU
  if (!x || !w || !y || !all_aligned16(x, w, bias, residual, z, y)) return MOE_ERR_INVALID_ARG;
  if (y == x || y == w || y == bias || y == z || (z && (z == x || z == w || z == bias || z == residual)))
    return MOE_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, ws_bytes, linear_part_bytes(R, out))) return MOE_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  const LinearCall c{R, in, out, activation, x, w, bias, residual, z, y, (float*)workspace};
  MOE_TRY(ST_LINEAR, launch_linear(dtype, c, s));
  return MOE_OK;
}

size_t moe_linear_backward_workspace_size(int64_t R, int32_t out, int32_t dtype) {
  if (check_linear(R, 64, out, dtype) != MOE_OK) return 0;
  return sizeof(float) * (size_t)linear_back_runs(dtype, R, out) * out;
}

moe_status moe_linear_backward(int64_t R, int32_t out, int32_t dtype, int32_t activation, const void* dy,
                               const void* z, void* dz, float* dbias, void* workspace, size_t ws_bytes, void* stream) {
  const moe_status st = check_linear(R, 64, out, dtype);
  if (st != MOE_OK) return st;
  if (!activation_ok(activation) || !aligned16(dbias)) return MOE_ERR_INVALID_ARG;
  hipStream_t s = (hipStream_t)stream;
  if (R == 0) {  // a sum over no rows
    MOE_TRY(ST_LINEAR, launch_fill2_i32((int32_t*)dbias, dbias ? out : 0, nullptr, 0, 0, s));
    return MOE_OK;
  }
  if (!dy || (!dz && !dbias) || (!z && activation != MOE_ACT_NONE)) return MOE_ERR_INVALID_ARG;
  if (!all_aligned16(dy, z, dz)) return MOE_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, ws_bytes, dbias ? moe_linear_backward_workspace_size(R, out, dtype) : 0))
    return MOE_ERR_WORKSPACE;
  const LinearBackCall c{R, out, activation, dy, z, dz, dbias, (float*)workspace};
  MOE_TRY(ST_LINEAR, launch_linear_back(dtype, c, s));
  return MOE_OK;
}

// ---- balance loss and the router's gradient ----
size_t moe_balance_workspace_size(const moe_config* cfg, int64_t N, int64_t seq_rows) {
  if (check_routing(cfg, N, seq_rows) != MOE_OK) return 0;
  const BalancePlan p = balance_plan(N, seq_rows, cfg->n_routed_experts);
  return balance_fits(p) ? balance_bytes(p, N, cfg->n_routed_experts) : 0;
}

moe_status moe_balance_loss(const moe_config* cfg, int64_t N, int64_t seq_rows, float weight, const float* scores,
                            const int32_t* topk_idx, const uint8_t* token_mask, int32_t* counts, float* coef,
                            float* loss, void* workspace, size_t ws_bytes, void* stream) {
  const moe_status st = check_routing(cfg, N, seq_rows);
  if (st != MOE_OK) return st;
  if (!std::isfinite(weight) || !loss || !aligned16(loss)) return MOE_ERR_INVALID_ARG;
  const int E = cfg->n_routed_experts;
  const BalancePlan p = balance_plan(N, seq_rows, E);
  if (!balance_fits(p)) return MOE_ERR_UNSUPPORTED;
  hipStream_t s = (hipStream_t)stream;
  if (N == 0) {
    MOE_TRY(ST_BALANCE, launch_fill2_i32((int32_t*)loss, 1, nullptr, 0, 0, s));
    return MOE_OK;
  }
  if (!scores || !topk_idx || !all_aligned16(scores, topk_idx, token_mask, counts, coef)) return MOE_ERR_INVALID_ARG;
  if (loss == coef || (counts && (void*)counts == coef) || (void*)counts == loss) return MOE_ERR_INVALID_ARG;
  if (scores == coef || (const void*)scores == counts || scores == loss || topk_idx == counts) return MOE_ERR_INVALID_ARG;
  const BalanceLayout L = balance_layout(p, E);
  if (!workspace_ok(workspace, ws_bytes, std::max(L.total, balance_bytes(p, N, E)))) return MOE_ERR_WORKSPACE;
  char* ws = (char*)workspace;
  const BalanceCall c{N, seq_rows, E, cfg->num_experts_per_tok, weight, scores, topk_idx, token_mask, counts, coef, loss,
                      (float*)(ws + L.part_p), (int32_t*)(ws + L.part_c), (int32_t*)(ws + L.part_v),
                      (float*)(ws + L.part_l), (int32_t*)(ws + L.done)};
  MOE_TRY(ST_BALANCE, launch_balance(c, s));
  return MOE_OK;
}

moe_status moe_route_backward(const moe_config* cfg, int64_t N, const float* scores, const int32_t* topk_idx,
                              const float* dtopk_w, int64_t seq_rows, const float* coef, const float* dloss,
                              const uint8_t* token_mask, float* dlogits, void* stream) {
  const moe_status st = check_routing(cfg, N, coef ? seq_rows : 1);
  if (st != MOE_OK) return st;
  if (N == 0) return MOE_OK;
  if (!dtopk_w && !coef) return MOE_ERR_INVALID_ARG;
  if (!scores || !dlogits || (dtopk_w && !topk_idx)) return MOE_ERR_INVALID_ARG;
  if (!all_aligned16(scores, topk_idx, dtopk_w, coef, dloss, token_mask, dlogits)) return MOE_ERR_INVALID_ARG;
  if (dlogits == dtopk_w || dlogits == coef || dlogits == dloss || (const void*)dlogits == topk_idx)
    return MOE_ERR_INVALID_ARG;
  hipStream_t s = (hipStream_t)stream;
  const float alpha = cfg->alpha_on_output ? 1.0f : cfg->routed_scaling_factor;
  const RouteBackCall c{N, coef ? seq_rows : N, cfg->n_routed_experts, cfg->num_experts_per_tok, alpha, cfg->eps,
                        cfg->norm_topk_prob, scores, topk_idx, dtopk_w, coef, dloss, token_mask, dlogits};
  MOE_TRY(ST_ROUTE_BACKWARD, launch_route_backward(c, s));
  return MOE_OK;
}

// ---- gradient norm and clipping ----
size_t moe_grad_norm_workspace_size(const moe_tensor* tensors, int32_t n) {
  if (check_tensors(tensors, n) != MOE_OK) return 0;
  return align_up(sizeof(double) * std::max<int64_t>(1, tensor_chunks(tensors, n)));
}

moe_status moe_grad_norm(const moe_tensor* tensors, int32_t n, float* norm, void* workspace, size_t ws_bytes,
                         void* stream) {
  const moe_status st = check_tensors(tensors, n);
  if (st != MOE_OK) return st;
  if (!norm || (uintptr_t)norm % 4 != 0) return MOE_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, ws_bytes, moe_grad_norm_workspace_size(tensors, n))) return MOE_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  MOE_TRY(ST_GRAD_NORM, launch_grad_norm(tensors, n, (double*)workspace, norm, s));
  return MOE_OK;
}

moe_status moe_grad_clip(const moe_tensor* tensors, const moe_tensor* out, int32_t n, const float* norm, float max_norm,
                         float eps, void* stream) {
  moe_status st = check_tensors(tensors, n);
  if (st != MOE_OK) return st;
  if (!std::isfinite(max_norm) || max_norm < 0.f || !std::isfinite(eps) || eps < 0.f) return MOE_ERR_INVALID_ARG;
  if (out) {
    if ((st = check_tensors(out, n)) != MOE_OK) return st;
    for (int i = 0; i < n; ++i)
      if (out[i].numel != tensors[i].numel) return MOE_ERR_INVALID_ARG;
  }
  if (!norm || (uintptr_t)norm % 4 != 0) return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {  // a block might read the norm after another one has scaled it
    const moe_tensor& w = out ? out[i] : tensors[i];
    const uintptr_t begin = (uintptr_t)w.data, end = begin + w.numel * value_bytes(w);
    if ((uintptr_t)norm < end && (uintptr_t)norm + 4 > begin) return MOE_ERR_INVALID_ARG;
  }
  const Overlap o = clip_overlap(tensors, out, n);
  if (o != Overlap::None) return o == Overlap::Some ? MOE_ERR_INVALID_ARG : MOE_ERR_UNSUPPORTED;
  hipStream_t s = (hipStream_t)stream;
  MOE_TRY(ST_GRAD_CLIP, launch_grad_clip(tensors, out, n, norm, max_norm, eps, s));
  return MOE_OK;
}

}  // extern "C"
