// C ABI of the operators around the layer: argument validation and dispatch.
// Nothing is enqueued unless every check passes.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../trace.h"
#include "ops.h"

namespace ds4 {

static bool al(const void* p, int n) { return ((uintptr_t)p & (n - 1)) == 0; }
static bool dt_ok(int dt) { return dt == DS4MOE_DT_F32 || dt == DS4MOE_DT_BF16; }
static bool dim_ok(int64_t v) { return v >= 256 && v <= 16384 && v % 256 == 0; }
static int status(hipError_t e) { return e == hipSuccess ? DS4MOE_OK : DS4MOE_EHIP; }

static int check_norm(const ds4moe_norm* N, int64_t T) {
  if (!N) return DS4MOE_EINVAL;
  if (!(N->eps > 0.0f) || !std::isfinite(N->eps) || !std::isfinite(N->res_scale)) return DS4MOE_EINVAL;
  if (N->gate < DS4MOE_GATE_NONE || N->gate > DS4MOE_GATE_FULL) return DS4MOE_EINVAL;
  if (!dim_ok(N->d_model) || T < 1 || T > kOpsMaxT) return DS4MOE_ESHAPE;
  if (!al(N->w_pre, 16) || !al(N->w_post, 16) || !al(N->w_next, 16)) return DS4MOE_EALIGN;
  return DS4MOE_OK;
}
// [0] the gate is there exactly when the descriptor has one, and aligned
static int check_gate(const ds4moe_norm* N, const float* gate) {
  if ((N->gate != DS4MOE_GATE_NONE) != (gate != nullptr)) return DS4MOE_EINVAL;
  return al(gate, N->gate == DS4MOE_GATE_TOKEN ? 4 : 16) ? DS4MOE_OK : DS4MOE_EALIGN;
}
static size_t norm_ws(const ds4moe_norm& N, int64_t T) { return (size_t)2 * norm_parts(N.d_model, T) * N.d_model * sizeof(float); }
static int check_norm_ws(const ds4moe_norm& N, int64_t T, const void* ws, size_t ws_bytes) {
  if (!ws) return DS4MOE_EINVAL;
  if (!al(ws, 256)) return DS4MOE_EALIGN;
  return ws_bytes < norm_ws(N, T) ? DS4MOE_EWORKSPACE : DS4MOE_OK;
}

// tokens, slots and width of a sorted call
static int check_slots(int64_t T, int32_t k) {
  if (T < 1 || T > kOpsMaxT || k < 1 || k > 16) return DS4MOE_ESHAPE;
  return DS4MOE_OK;
}
static int check_rows(int64_t T, int32_t k, int32_t d, int64_t n_rows) {
  const int rc = check_slots(T, k);
  if (rc) return rc;
  return dim_ok(d) && n_rows >= 1 && n_rows <= kOpsMaxRows ? DS4MOE_OK : DS4MOE_ESHAPE;
}

// the shapes of a product with E packed [rows, cols] matrices
static int check_product(int64_t n, int32_t rows, int32_t cols, int32_t E, const int32_t* offsets) {
  if (n < 1 || n > kOpsMaxRows || !dim_ok(cols)) return DS4MOE_ESHAPE;
  if (rows < 16 || rows > 16384 || rows % 16 || E < 1 || E > 1024) return DS4MOE_ESHAPE;
  if (!offsets && E != 1) return DS4MOE_EINVAL;
  return DS4MOE_OK;
}

}  // namespace ds4

using namespace ds4;

extern "C" {

// ---------------------------------------------------------------- norms
size_t ds4moe_norm_workspace_bytes(const ds4moe_norm* N, int64_t T) {
  return check_norm(N, T) ? 0 : norm_ws(*N, T);
}

int ds4moe_norm_pre(const ds4moe_norm* N, const void* h, int h_dtype, int64_t T, void* x, int x_dtype, void* stream) {
  const int rc = check_norm(N, T);
  if (rc) return rc;
  if (!h || !x || !dt_ok(h_dtype) || !dt_ok(x_dtype)) return DS4MOE_EINVAL;
  if (!al(h, 16) || !al(x, 16)) return DS4MOE_EALIGN;
  NormCall c{};
  c.N = *N;
  c.h = h;
  c.h_dt = h_dtype;
  c.T = T;
  c.x = x;
  c.x_dt = x_dtype;
  c.st = (hipStream_t)stream;
  return status(launch_norm_pre(c));
}

int ds4moe_norm_post(const ds4moe_norm* N, const void* h, int h_dtype, const void* y, int y_dtype, const float* gate,
                     int64_t T, void* h_out, void* x_next, int x_dtype, void* stream) {
  int rc = check_norm(N, T);
  if (rc) return rc;
  if (!h || !y || !h_out || !dt_ok(h_dtype) || !dt_ok(y_dtype) || !dt_ok(x_dtype)) return DS4MOE_EINVAL;
  if ((rc = check_gate(N, gate))) return rc;
  if (!al(h, 16) || !al(y, 16) || !al(h_out, 16) || !al(x_next, 16)) return DS4MOE_EALIGN;
  NormCall c{};
  c.N = *N;
  c.h = h;
  c.h_dt = h_dtype;
  c.y = y;
  c.y_dt = y_dtype;
  c.gate = gate;
  c.T = T;
  c.h_out = h_out;
  c.x = x_next;
  c.x_dt = x_dtype;
  c.st = (hipStream_t)stream;
  return status(launch_norm_post(c));
}

int ds4moe_norm_pre_grad(const ds4moe_norm* N, const void* h, int h_dtype, const void* dx, int x_dtype,
                         const void* dh_out, int64_t T, void* dh, float* dw_pre, void* ws, size_t ws_bytes,
                         void* stream) {
  int rc = check_norm(N, T);
  if (rc) return rc;
  if (!h || !dx || !dh || !dt_ok(h_dtype) || !dt_ok(x_dtype)) return DS4MOE_EINVAL;
  if (!al(h, 16) || !al(dx, 16) || !al(dh_out, 16) || !al(dh, 16) || !al(dw_pre, 16)) return DS4MOE_EALIGN;
  if (dw_pre && (rc = check_norm_ws(*N, T, ws, ws_bytes))) return rc;
  NormCall c{};
  c.N = *N;
  c.h = h;
  c.h_dt = h_dtype;
  c.dx = dx;
  c.x_dt = x_dtype;
  c.dh_out = dh_out;
  c.T = T;
  c.dh = dh;
  c.dw = dw_pre;
  c.part = (float*)ws;
  c.st = (hipStream_t)stream;
  return status(launch_norm_pre_grad(c));
}

int ds4moe_norm_post_grad(const ds4moe_norm* N, const void* dh_out, int h_dtype, const void* y, int y_dtype,
                          const float* gate, int64_t T, void* dy, float* dw_post, float* dgate, void* ws,
                          size_t ws_bytes, void* stream) {
  int rc = check_norm(N, T);
  if (rc) return rc;
  if (!dh_out || !y || !dy || !dt_ok(h_dtype) || !dt_ok(y_dtype)) return DS4MOE_EINVAL;
  if ((rc = check_gate(N, gate))) return rc;
  if (dgate && N->gate == DS4MOE_GATE_NONE) return DS4MOE_EINVAL;
  if (!al(dh_out, 16) || !al(y, 16) || !al(dy, 16) || !al(dw_post, 16) ||
      !al(dgate, N->gate == DS4MOE_GATE_TOKEN ? 4 : 16))
    return DS4MOE_EALIGN;
  if ((dw_post || (dgate && N->gate == DS4MOE_GATE_CHANNEL)) && (rc = check_norm_ws(*N, T, ws, ws_bytes))) return rc;
  NormCall c{};
  c.N = *N;
  c.dh_out = dh_out;
  c.h_dt = h_dtype;
  c.y = y;
  c.y_dt = y_dtype;
  c.gate = gate;
  c.T = T;
  c.dy = dy;
  c.dw = dw_post;
  c.dgate = dgate;
  c.part = (float*)ws;
  c.st = (hipStream_t)stream;
  return status(launch_norm_post_grad(c));
}

// ---------------------------------------------------------------- sorted tokens
size_t ds4moe_group_workspace_bytes(int64_t T, int32_t k, int32_t n_experts) {
  if (check_slots(T, k) || n_experts < 1 || n_experts > 1024) return 0;
  return group_ws_bytes(T * k, n_experts);
}

int ds4moe_group(const int32_t* topk_idx, int64_t T, int32_t k, int32_t n_experts, int32_t* counts, int32_t* offsets,
                 int32_t* perm, int32_t* inv, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_slots(T, k);
  if (rc) return rc;
  if (n_experts < 1 || n_experts > 1024) return DS4MOE_ESHAPE;
  if (!topk_idx || !counts || !offsets || !perm || !inv || !ws) return DS4MOE_EINVAL;
  if (!al(topk_idx, 4) || !al(counts, 4) || !al(offsets, 4) || !al(perm, 4) || !al(inv, 4) || !al(ws, 256))
    return DS4MOE_EALIGN;
  if (ws_bytes < group_ws_bytes(T * k, n_experts)) return DS4MOE_EWORKSPACE;
  return status(launch_group(topk_idx, T * k, n_experts, counts, offsets, perm, inv, (int32_t*)ws, (hipStream_t)stream));
}

int ds4moe_dispatch(const void* x, int x_dtype, int64_t T, int32_t k, int32_t d, const int32_t* inv, void* xs,
                    int64_t n_rows, void* stream) {
  const int rc = check_rows(T, k, d, n_rows);
  if (rc) return rc;
  if (!x || !inv || !xs || !dt_ok(x_dtype)) return DS4MOE_EINVAL;
  if (!al(x, 16) || !al(xs, 16) || !al(inv, 4)) return DS4MOE_EALIGN;
  return status(launch_dispatch(x, x_dtype, T, k, d, inv, xs, n_rows, (hipStream_t)stream));
}

int ds4moe_combine(const void* ys, int ys_dtype, int64_t n_rows, const int32_t* inv, const float* topk_w,
                   const void* base, int64_t T, int32_t k, int32_t d, void* y, int y_dtype, void* stream) {
  const int rc = check_rows(T, k, d, n_rows);
  if (rc) return rc;
  if (!ys || !inv || !y || !dt_ok(ys_dtype) || !dt_ok(y_dtype)) return DS4MOE_EINVAL;
  if (!al(ys, 16) || !al(base, 16) || !al(y, 16) || !al(inv, 4) || !al(topk_w, 4)) return DS4MOE_EALIGN;
  return status(launch_combine(ys, ys_dtype, n_rows, inv, topk_w, base, T, k, d, y, y_dtype, (hipStream_t)stream));
}

int ds4moe_combine_grad(const void* dy, int y_dtype, const void* ys, int ys_dtype, int64_t n_rows, const int32_t* inv,
                        const float* topk_w, int64_t T, int32_t k, int32_t d, void* dys, float* dw, float* dlogits,
                        void* stream) {
  const int rc = check_rows(T, k, d, n_rows);
  if (rc) return rc;
  if (!dy || !ys || !inv || !dt_ok(ys_dtype) || !dt_ok(y_dtype)) return DS4MOE_EINVAL;
  if (!dys && !dw && !dlogits) return DS4MOE_EINVAL;
  if (!al(dy, 16) || !al(ys, 16) || !al(dys, 16) || !al(inv, 4) || !al(topk_w, 4) || !al(dw, 4) || !al(dlogits, 4))
    return DS4MOE_EALIGN;
  return status(launch_combine_grad(dy, y_dtype, ys, ys_dtype, n_rows, inv, topk_w, T, k, d, dys, dw, dlogits,
                                    (hipStream_t)stream));
}

// ---------------------------------------------------------------- MXFP4 rows
int ds4moe_mx_quantize(const void* x, int x_dtype, int64_t T, const int32_t* inv, int32_t k, int64_t n, int32_t cols,
                       void* packed, void* stream) {
  if (inv && check_slots(T, k)) return DS4MOE_ESHAPE;
  if (!dim_ok(cols) || n < 1 || n > kOpsMaxRows) return DS4MOE_ESHAPE;
  if (!inv && (k != 1 || T < 1 || n < T)) return DS4MOE_ESHAPE;
  if (!x || !packed || !dt_ok(x_dtype)) return DS4MOE_EINVAL;
  if (!al(x, 16) || !al(packed, 16) || !al(inv, 4)) return DS4MOE_EALIGN;
  return status(launch_mx_quantize(x, x_dtype, T, inv, k, n, cols, packed, (hipStream_t)stream));
}

int ds4moe_mx_dequantize(const void* packed, int64_t n, int32_t cols, void* out, int out_dtype, void* stream) {
  if (n < 1 || n > kOpsMaxRows || !dim_ok(cols)) return DS4MOE_ESHAPE;
  if (!packed || !out || !dt_ok(out_dtype)) return DS4MOE_EINVAL;
  if (!al(packed, 16) || !al(out, 16)) return DS4MOE_EALIGN;
  return status(launch_mx_dequantize(packed, n, cols, out, out_dtype, (hipStream_t)stream));
}

int ds4moe_mx_product(const void* a, int64_t n, int32_t cols, const void* w, const void* w_up, int32_t rows,
                      int32_t n_experts, const int32_t* offsets, void* y, int y_dtype, void* stream) {
  const int rc = check_product(n, rows, cols, n_experts, offsets);
  if (rc) return rc;
  if (!a || !w || !y || !dt_ok(y_dtype)) return DS4MOE_EINVAL;
  if (!al(a, 16) || !al(w, 16) || !al(w_up, 16) || !al(y, 16) || !al(offsets, 4)) return DS4MOE_EALIGN;
  MxProduct p{};
  p.a = (const uint8_t*)a;
  p.n = n;
  p.rows = rows;
  p.cols = cols;
  p.E = n_experts;
  p.w = (const uint8_t*)w;
  p.w2 = (const uint8_t*)w_up;
  p.offsets = offsets;
  p.out = y;
  p.out_dt = y_dtype;
  p.st = (hipStream_t)stream;
  return status(launch_mx_product(p));
}

int ds4moe_mx_product_grad(const void* dy, int dy_dtype, int64_t n, int32_t rows, const void* w, int32_t cols,
                           int32_t n_experts, const int32_t* offsets, void* da, int da_dtype, void* stream) {
  const int rc = check_product(n, rows, cols, n_experts, offsets);
  if (rc) return rc;
  if (n * cols > kOpsMaxGrad) return DS4MOE_ESHAPE;
  if (!dy || !w || !da || !dt_ok(dy_dtype) || !dt_ok(da_dtype)) return DS4MOE_EINVAL;
  if (!al(dy, 16) || !al(w, 16) || !al(da, 16) || !al(offsets, 4)) return DS4MOE_EALIGN;
  MxProduct p{};
  p.dy = dy;
  p.dy_dt = dy_dtype;
  p.n = n;
  p.rows = rows;
  p.cols = cols;
  p.E = n_experts;
  p.w = (const uint8_t*)w;
  p.offsets = offsets;
  p.out = da;
  p.out_dt = da_dtype;
  p.st = (hipStream_t)stream;
  return status(launch_mx_product_grad(p));
}

}  // extern "C"
