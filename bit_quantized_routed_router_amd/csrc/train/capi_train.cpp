// C ABI of a training step's operators: argument validation and dispatch.
// Nothing is enqueued unless every check passes.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "../trace.h"
#include "train.h"

namespace ds4 {

static bool al(const void* p, int n) { return ((uintptr_t)p & (n - 1)) == 0; }
static bool dt_ok(int dt) { return dt == DS4MOE_DT_F32 || dt == DS4MOE_DT_BF16; }
static int dt_size(int dt) { return dt == DS4MOE_DT_F32 ? 4 : 2; }
static bool dim_ok(int64_t v) { return v >= 256 && v <= 16384 && v % 256 == 0; }
static int status(hipError_t e) { return e == hipSuccess ? DS4MOE_OK : DS4MOE_EHIP; }

static int check_balance(int64_t T, int32_t E, int32_t seqs) {
  if (T < 1 || T > kOpsMaxT || E < 1 || E > 1024 || T * E >= (1ll << 31)) return DS4MOE_ESHAPE;
  return seqs >= 1 && seqs <= kBalMaxSeqs ? DS4MOE_OK : DS4MOE_ESHAPE;
}
static int check_balance_args(const BalanceCall& c) {
  const int rc = check_balance(c.T, c.E, c.seqs);
  if (rc) return rc;
  if (c.k < 1 || c.k > 16) return DS4MOE_ESHAPE;
  if (!c.z || !c.idx || !c.counts || !c.tokens || !dt_ok(c.z_dt)) return DS4MOE_EINVAL;
  if (!c.off && c.seqs != 1) return DS4MOE_EINVAL;
  if (!al(c.z, dt_size(c.z_dt)) || !al(c.idx, 4) || !al(c.off, 4) || !al(c.counts, 4) || !al(c.tokens, 4))
    return DS4MOE_EALIGN;
  return DS4MOE_OK;
}

static int check_xent(int dt, int64_t T, int64_t V, int32_t d) {
  if (!dt_ok(dt)) return DS4MOE_EINVAL;
  return T >= 1 && T <= kOpsMaxT && V >= 1 && V <= kXentMaxV && dim_ok(d) ? DS4MOE_OK : DS4MOE_ESHAPE;
}
static int check_xent_args(const XentCall& c, bool grad, size_t ws_bytes) {
  const int rc = check_xent(c.dt, c.T, c.V, c.d);
  if (rc) return rc;
  if (!c.h || !c.w || !c.target || !c.ws || !std::isfinite(c.scale)) return DS4MOE_EINVAL;
  if (!al(c.h, 16) || !al(c.w, 16) || !al(c.target, 4) || !al(c.ws, 256)) return DS4MOE_EALIGN;
  return ws_bytes < xent_ws_bytes(c.dt, c.T, c.V, c.d, grad) ? DS4MOE_EWORKSPACE : DS4MOE_OK;
}

static bool params_ok(const ds4moe_param* p, int32_t n) {
  if (n < 0 || n > kAdamMaxTensors) return false;
  int64_t all = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (p[i].n < 0 || p[i].n > kAdamMaxN) return false;
    all += p[i].n;
  }
  return all <= kAdamMaxN;
}
static int check_options(const ds4moe_adamw* A) {
  if (!A || !dt_ok(A->grad_dtype) || !dt_ok(A->param_dtype)) return DS4MOE_EINVAL;
  if (A->state != DS4MOE_STATE_F32 && A->state != DS4MOE_STATE_FP8) return DS4MOE_EINVAL;
  // (below fp32's normal numbers the reciprocal of eps would be infinite, and a value without moments NaN)
  if (!std::isfinite(A->lr) || !std::isfinite(A->eps) || !((float)A->eps >= 1.17549435e-38f)) return DS4MOE_EINVAL;
  if (!(A->beta1 >= 0.0 && A->beta1 < 1.0) || !(A->beta2 >= 0.0 && A->beta2 < 1.0)) return DS4MOE_EINVAL;
  return al(A->lr_dev, 4) && al(A->step_dev, 4) ? DS4MOE_OK : DS4MOE_EALIGN;
}
// types and states that a table was made for
static int64_t kinds_of(const ds4moe_adamw* A) { return 8 | A->param_dtype | A->grad_dtype << 1 | A->state << 2; }
// Whether a range that a step writes overlaps another, or a gradient.  Gradients may share memory: they are read only.
static bool overlap(const ds4moe_adamw* A, const ds4moe_param* p, int32_t n) {
  const bool fp8 = A->state == DS4MOE_STATE_FP8;
  struct Range {
    uintptr_t at, end;
    bool written;
  };
  std::vector<Range> r;
  r.reserve((size_t)n * (fp8 ? 7 : 5));
  for (int32_t i = 0; i < n; ++i) {
    const ds4moe_param& q = p[i];
    if (q.n == 0) continue;
    auto add = [&](const void* at, int64_t bytes, bool written) {
      if (at) r.push_back({(uintptr_t)at, (uintptr_t)at + (uintptr_t)bytes, written});
    };
    add(q.grad, q.n * dt_size(A->grad_dtype), false);
    add(q.param, q.n * dt_size(A->param_dtype), true);
    add(q.master, q.n * 4, true);
    add(q.m, q.n * (fp8 ? 1 : 4), true);
    add(q.v, q.n * (fp8 ? 1 : 4), true);
    if (fp8) {
      add(q.m_scale, (q.n + 255) / 256 * 4, true);
      add(q.v_scale, (q.n + 255) / 256 * 4, true);
    }
  }
  std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.at < b.at; });
  uintptr_t written = 0, read = 0;  // where those before end
  for (const Range& x : r) {
    if (x.at < written || (x.written && x.at < read)) return true;
    uintptr_t& end = x.written ? written : read;
    end = std::max(end, x.end);
  }
  return false;
}
static int check_params(const ds4moe_adamw* A, const ds4moe_param* p, int32_t n) {
  const bool fp8 = A->state == DS4MOE_STATE_FP8;
  for (int32_t i = 0; i < n; ++i) {
    const ds4moe_param& q = p[i];
    if (!std::isfinite(q.weight_decay)) return DS4MOE_EINVAL;
    if (q.n == 0) continue;
    if (!q.param || !q.grad || !q.m || !q.v || (fp8 && (!q.m_scale || !q.v_scale))) return DS4MOE_EINVAL;
    if (!al(q.param, dt_size(A->param_dtype)) || !al(q.grad, dt_size(A->grad_dtype)) || !al(q.master, 4) ||
        !al(q.m, fp8 ? 1 : 4) || !al(q.v, fp8 ? 1 : 4) || (fp8 && (!al(q.m_scale, 4) || !al(q.v_scale, 4))))
      return DS4MOE_EALIGN;
  }
  return DS4MOE_OK;
}
// a descriptor that ds4moe_adamw_table has filled in, and its table
static int check_table(const ds4moe_adamw* A, const void* table) {
  const int rc = check_options(A);
  if (rc) return rc;
  if (A->n_params < 0 || A->n_params > kAdamMaxTensors || A->blocks < 0 || A->blocks > kAdamMaxBlocks || A->run < 256 ||
      A->run % 256)
    return DS4MOE_ESHAPE;
  if (!table || A->kinds != kinds_of(A)) return DS4MOE_EINVAL;
  return al(table, 16) ? DS4MOE_OK : DS4MOE_EALIGN;
}

}  // namespace ds4

using namespace ds4;

extern "C" {

// ---------------------------------------------------------------- balance loss
size_t ds4moe_balance_workspace_bytes(int64_t T, int32_t n_experts, int32_t n_seqs) {
  return check_balance(T, n_experts, n_seqs) ? 0 : balance_ws_bytes(T, n_experts, n_seqs);
}

int ds4moe_balance(const void* logits, int l_dtype, int64_t T, int32_t n_experts, const int32_t* topk_idx, int32_t k,
                   const int32_t* seq_offsets, int32_t n_seqs, int32_t* counts, int32_t* tokens, float* loss, void* ws,
                   size_t ws_bytes, void* stream) {
  BalanceCall c{};
  c.z = logits;
  c.z_dt = l_dtype;
  c.T = T;
  c.E = n_experts;
  c.k = k;
  c.seqs = n_seqs;
  c.idx = topk_idx;
  c.off = seq_offsets;
  c.counts = counts;
  c.tokens = tokens;
  c.loss = loss;
  c.ws = ws;
  c.st = (hipStream_t)stream;
  const int rc = check_balance_args(c);
  if (rc) return rc;
  if (!loss || !ws) return DS4MOE_EINVAL;
  if (!al(loss, 4) || !al(ws, 256)) return DS4MOE_EALIGN;
  if (ws_bytes < balance_ws_bytes(T, n_experts, n_seqs)) return DS4MOE_EWORKSPACE;
  return status(launch_balance(c));
}

int ds4moe_balance_grad(const void* logits, int l_dtype, int64_t T, int32_t n_experts, const int32_t* topk_idx,
                        int32_t k, const int32_t* seq_offsets, int32_t n_seqs, const int32_t* counts,
                        const int32_t* tokens, const float* dloss, const float* dslots, void* dlogits, void* stream) {
  BalanceCall c{};
  c.z = logits;
  c.z_dt = l_dtype;
  c.T = T;
  c.E = n_experts;
  c.k = k;
  c.seqs = n_seqs;
  c.idx = topk_idx;
  c.off = seq_offsets;
  c.counts = const_cast<int32_t*>(counts);
  c.tokens = const_cast<int32_t*>(tokens);
  c.dloss = dloss;
  c.dslots = dslots;
  c.dz = dlogits;
  c.st = (hipStream_t)stream;
  const int rc = check_balance_args(c);
  if (rc) return rc;
  if (!dlogits) return DS4MOE_EINVAL;
  if (!al(dlogits, dt_size(l_dtype)) || !al(dloss, 4) || !al(dslots, 4)) return DS4MOE_EALIGN;
  return status(launch_balance_grad(c));
}

// ---------------------------------------------------------------- cross entropy
size_t ds4moe_xent_workspace_bytes(int dtype, int64_t T, int64_t vocab, int32_t d, int with_grad) {
  if (check_xent(dtype, T, vocab, d)) return 0;
  const size_t fwd = xent_ws_bytes(dtype, T, vocab, d, false);
  return with_grad ? std::max(fwd, xent_ws_bytes(dtype, T, vocab, d, true)) : fwd;
}

int ds4moe_xent(const void* h, const void* w, int dtype, int64_t T, int64_t vocab, int32_t d, float scale,
                const int32_t* target, float* loss, float* lse, void* ws, size_t ws_bytes, void* stream) {
  XentCall c{};
  c.h = h;
  c.w = w;
  c.dt = dtype;
  c.T = T;
  c.V = vocab;
  c.d = d;
  c.scale = scale;
  c.target = target;
  c.loss = loss;
  c.lse = lse;
  c.ws = (uint8_t*)ws;
  c.st = (hipStream_t)stream;
  const int rc = check_xent_args(c, false, ws_bytes);
  if (rc) return rc;
  if (!loss || !lse) return DS4MOE_EINVAL;
  if (!al(loss, 4) || !al(lse, 4)) return DS4MOE_EALIGN;
  return status(launch_xent(c));
}

int ds4moe_xent_grad(const void* h, const void* w, int dtype, int64_t T, int64_t vocab, int32_t d, float scale,
                     const int32_t* target, const float* lse, const float* dloss, void* dh, void* dw, void* ws,
                     size_t ws_bytes, void* stream) {
  XentCall c{};
  c.h = h;
  c.w = w;
  c.dt = dtype;
  c.T = T;
  c.V = vocab;
  c.d = d;
  c.scale = scale;
  c.target = target;
  c.lse_in = lse;
  c.dloss = dloss;
  c.dh = dh;
  c.dw = dw;
  c.ws = (uint8_t*)ws;
  c.st = (hipStream_t)stream;
  const int rc = check_xent_args(c, true, ws_bytes);
  if (rc) return rc;
  if (!lse || (!dh && !dw)) return DS4MOE_EINVAL;
  if (!al(lse, 4) || !al(dloss, 4) || !al(dh, 16) || !al(dw, 16)) return DS4MOE_EALIGN;
  return status(launch_xent_grad(c));
}

// ---------------------------------------------------------------- AdamW
size_t ds4moe_adamw_table_bytes(const ds4moe_param* params, int32_t n_params) {
  if ((!params && n_params != 0) || !params_ok(params, n_params)) return 0;
  return adam_table_bytes(params, n_params);
}

int ds4moe_adamw_table(ds4moe_adamw* A, const ds4moe_param* params, int32_t n_params, void* table, size_t table_bytes) {
  int rc = check_options(A);
  if (rc) return rc;
  if (!table || (!params && n_params != 0)) return DS4MOE_EINVAL;
  if (!params_ok(params, n_params)) return DS4MOE_ESHAPE;
  if ((rc = check_params(A, params, n_params))) return rc;
  if (!al(table, 8)) return DS4MOE_EALIGN;
  if (table_bytes < adam_table_bytes(params, n_params)) return DS4MOE_EWORKSPACE;
  try {  // (the ranges take host memory)
    if (overlap(A, params, n_params)) return DS4MOE_EINVAL;
  } catch (...) {
    return DS4MOE_EWORKSPACE;
  }
  adam_table(A, params, n_params, table);
  A->kinds = kinds_of(A);
  return DS4MOE_OK;
}

int ds4moe_adamw_step(const ds4moe_adamw* A, const void* table, int64_t step, const float* grad_scale, void* stream) {
  const int rc = check_table(A, table);
  if (rc) return rc;
  if (step < 1 && !A->step_dev) return DS4MOE_EINVAL;
  if (!al(grad_scale, 4)) return DS4MOE_EALIGN;
  AdamCall c{};
  c.A = *A;
  c.table = table;
  c.step = step;
  c.grad_scale = grad_scale;
  c.st = (hipStream_t)stream;
  return status(launch_adamw_step(c));
}

size_t ds4moe_adamw_workspace_bytes(const ds4moe_adamw* A) {
  if (!A || A->blocks < 0 || A->blocks > kAdamMaxBlocks) return 0;
  return adam_ws_bytes(*A);
}

int ds4moe_adamw_norm(const ds4moe_adamw* A, const void* table, float max_norm, float* out, void* ws, size_t ws_bytes,
                      void* stream) {
  const int rc = check_table(A, table);
  if (rc) return rc;
  if (!(max_norm > 0.0f) || !out || !ws) return DS4MOE_EINVAL;
  if (!al(out, 4) || !al(ws, 256)) return DS4MOE_EALIGN;
  if (ws_bytes < adam_ws_bytes(*A)) return DS4MOE_EWORKSPACE;
  AdamCall c{};
  c.A = *A;
  c.table = table;
  c.max_norm = max_norm;
  c.out = out;
  c.ws = (double*)ws;
  c.st = (hipStream_t)stream;
  return status(launch_adamw_norm(c));
}

}  // extern "C"
