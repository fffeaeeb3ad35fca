// Norms before and after a block, fused with the block's gate and residual
// scale, and their gradients.  For a row t of d values (all sums in fp32):
//
//   pre        r = 1 / sqrt(sum_c h^2 / d + eps)       x  = h r w_pre
//   post       q = 1 / sqrt(sum_c y^2 / d + eps)       h' = rho h + g (y q w_post)
//              and, of h' before its rounding,          x' = h' r' w_next
//   pre_grad   v = dx w_pre      dh = rho dh' + r (v - h r^2 sum_c(h v) / d)
//              dw_pre = sum_t dx h r
//   post_grad  u = dh' g w_post  dy = q (u - y q^2 sum_c(y u) / d)
//              dw_post = sum_t dh' g y q   dg = dh' y q w_post summed over what g is shared by
//
// Every kernel reads its rows once and keeps them in registers between the
// sums and the outputs, so all of them are bound by memory for many tokens
// and by the latency of load, sum, store for few.
#include <algorithm>

#include "../trace.h"
#include "ops.h"

namespace ds4 {

// Sums NV values over the NT threads of a block (or of one of its teams);
// every thread gets the same result.  red is written once per call and slot
// (the caller alternates slots between barriers).
template <int NV, int NW>
__device__ inline void team_sum(float (&v)[NV], float* red, int wave) {
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = wave_sum(v[i]);
  if (NW == 1) return;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) red[i * NW + wave] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) s += red[i * NW + w];
    v[i] = s;
  }
}

__device__ inline float inv_rms(float ss, int d, float eps) { return 1.0f / sqrtf(ss / (float)d + eps); }

__device__ inline void ld_w(const float* w, int c, float (&v)[8]) {
  if (w) {
    unpack8(ld8<false>(w, c), v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 1.0f;
  }
}

// gate values of row t, columns c .. c + 7 (the per-token value is in gt)
__device__ inline void ld_gate(const float* g, int mode, int64_t t, int d, int c, float gt, float (&v)[8]) {
  if (mode == DS4MOE_GATE_CHANNEL) {
    unpack8(ld8<false>(g, c), v);
  } else if (mode == DS4MOE_GATE_FULL) {
    unpack8(ld8<false>(g, t * d + c), v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = gt;
  }
}

// ---------------------------------------------------------------- forward
// One block of NT threads per row; thread i holds columns 8 (i + s NT) .. + 7
// for s < NS.
template <int NT, int NS, bool HB, bool XB>
__global__ __launch_bounds__(NT) void k_norm_pre(const void* __restrict__ h, const float* __restrict__ w, int d,
                                                 float eps, void* __restrict__ x) {
  __shared__ float red[NT / 64];
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, d8 = d / 8;
  float v[NS][8];
  float ss[1] = {0.f};
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int i = min(tid + s * NT, d8 - 1);
    unpack8(ld8<HB>(h, t * d + 8 * i), v[s]);
  }
#pragma unroll
  for (int s = 0; s < NS; ++s)
    if (tid + s * NT < d8)
#pragma unroll
      for (int e = 0; e < 8; ++e) ss[0] = fmaf(v[s][e], v[s][e], ss[0]);
  team_sum<1, NT / 64>(ss, red, tid >> 6);
  const float r = inv_rms(ss[0], d, eps);
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int i = tid + s * NT;
    if (i < d8) {
      float wv[8];
      ld_w(w, 8 * i, wv);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[s][e] = v[s][e] * r * wv[e];
      st8<XB>(x, t * d + 8 * i, v[s]);
    }
  }
}

// The next block's norm takes h' before its rounding: its error is then that
// of x's own rounding alone.
template <int NT, int NS, bool HB, bool YB, bool XB>
__global__ __launch_bounds__(NT) void k_norm_post(const void* h, const void* __restrict__ y,
                                                  const float* __restrict__ gate, int gmode,
                                                  const float* __restrict__ w, const float* __restrict__ wn, int d,
                                                  float eps, float rho, void* ho, void* __restrict__ x) {
  __shared__ float red[2][NT / 64];
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, d8 = d / 8;
  float v[NS][8];
  Raw8<HB> hr[NS];
  float ss[1] = {0.f};
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int i = min(tid + s * NT, d8 - 1);
    unpack8(ld8<YB>(y, t * d + 8 * i), v[s]);
    hr[s] = ld8<HB>(h, t * d + 8 * i);
  }
  const float gt = gmode == DS4MOE_GATE_TOKEN ? gate[t] : 1.0f;
#pragma unroll
  for (int s = 0; s < NS; ++s)
    if (tid + s * NT < d8)
#pragma unroll
      for (int e = 0; e < 8; ++e) ss[0] = fmaf(v[s][e], v[s][e], ss[0]);
  team_sum<1, NT / 64>(ss, red[0], tid >> 6);
  const float q = inv_rms(ss[0], d, eps);
  ss[0] = 0.f;
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int i = tid + s * NT;
    if (i < d8) {
      float wv[8], gv[8], hv[8];
      ld_w(w, 8 * i, wv);
      ld_gate(gate, gmode, t, d, 8 * i, gt, gv);
      unpack8(hr[s], hv);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[s][e] = fmaf(rho, hv[e], gv[e] * (v[s][e] * q * wv[e]));
        ss[0] = fmaf(v[s][e], v[s][e], ss[0]);
      }
      st8<HB>(ho, t * d + 8 * i, v[s]);
    }
  }
  if (!x) return;
  team_sum<1, NT / 64>(ss, red[1], tid >> 6);
  const float r = inv_rms(ss[0], d, eps);
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int i = tid + s * NT;
    if (i < d8) {
      float wv[8];
      ld_w(wn, 8 * i, wv);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[s][e] = v[s][e] * r * wv[e];
      st8<XB>(x, t * d + 8 * i, v[s]);
    }
  }
}

// ---------------------------------------------------------------- backward
// Blocks of kTeams teams of 256 threads; team m of the grid takes rows m,
// m + M, ... and keeps its share of the sums over tokens in registers, which
// it writes to row m of part at the end.  k_norm_colsum adds those rows in
// order, so the result does not depend on how the blocks ran.
constexpr int kTeamT = 256, kTeams = 2, kMaxParts = 512;
int norm_parts(int64_t T) { return (int)std::min<int64_t>(T, kMaxParts); }

template <int NS, bool HB, bool XB>
__global__ __launch_bounds__(kTeamT * kTeams) void k_norm_pre_grad(
    const void* __restrict__ h, const void* __restrict__ dx, const void* dho, const float* __restrict__ w, int d,
    float eps, float rho, int64_t T, int M, void* dh, float* __restrict__ dw) {
  __shared__ float red[2][kTeams][2 * (kTeamT / 64)];
  const int team = threadIdx.x / kTeamT, tid = threadIdx.x % kTeamT, d8 = d / 8;
  const int m = blockIdx.x * kTeams + team;
  float acc[NS][8] = {};
  int slot = 0;
  for (int64_t t0 = 0; t0 < T; t0 += M, slot ^= 1) {
    const int64_t t = t0 + m;
    const bool live = m < M && t < T;
    float hv[NS][8], xv[NS][8];
    Raw8<HB> ho[NS] = {};
    float ss[2] = {0.f, 0.f};
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int i = tid + s * kTeamT;
      if (live && i < d8) {
        unpack8(ld8<HB>(h, t * d + 8 * i), hv[s]);
        unpack8(ld8<XB>(dx, t * d + 8 * i), xv[s]);
        if (dho) ho[s] = ld8<HB>(dho, t * d + 8 * i);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) hv[s][e] = xv[s][e] = 0.f;
      }
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      float wv[8];
      ld_w(w, 8 * min(tid + s * kTeamT, d8 - 1), wv);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss[0] = fmaf(hv[s][e], hv[s][e], ss[0]);
        ss[1] = fmaf(hv[s][e], xv[s][e] * wv[e], ss[1]);
      }
    }
    team_sum<2, kTeamT / 64>(ss, red[slot][team], tid >> 6);
    const float r = inv_rms(ss[0], d, eps), c = ss[1] / (float)d * r * r;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int i = tid + s * kTeamT;
      if (live && i < d8) {
        float wv[8], o[8];
        ld_w(w, 8 * i, wv);
        unpack8(ho[s], o);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          acc[s][e] = fmaf(xv[s][e], hv[s][e] * r, acc[s][e]);
          o[e] = (dho ? rho * o[e] : 0.f) + r * (xv[s][e] * wv[e] - hv[s][e] * c);
        }
        st8<HB>(dh, t * d + 8 * i, o);
      }
    }
  }
  if (dw && m < M) {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int i = tid + s * kTeamT;
      if (i < d8) st8<false>(dw, (int64_t)m * d + 8 * i, acc[s]);
    }
  }
}

template <int NS, bool HB, bool YB>
__global__ __launch_bounds__(kTeamT * kTeams) void k_norm_post_grad(
    const void* __restrict__ dho, const void* y, const float* __restrict__ gate, int gmode,
    const float* __restrict__ w, int d, float eps, int64_t T, int M, void* dy, float* __restrict__ dw,
    float* __restrict__ dgate) {
  __shared__ float red[2][kTeams][3 * (kTeamT / 64)];
  const int team = threadIdx.x / kTeamT, tid = threadIdx.x % kTeamT, d8 = d / 8;
  const int m = blockIdx.x * kTeams + team;
  float acc[NS][8] = {}, accg[NS][8] = {};
  int slot = 0;
  for (int64_t t0 = 0; t0 < T; t0 += M, slot ^= 1) {
    const int64_t t = t0 + m;
    const bool live = m < M && t < T;
    float yv[NS][8], ov[NS][8];
    float ss[3] = {0.f, 0.f, 0.f};
    float gt = 1.0f;
    if (live && gmode == DS4MOE_GATE_TOKEN) gt = gate[t];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int i = tid + s * kTeamT;
      if (live && i < d8) {
        unpack8(ld8<YB>(y, t * d + 8 * i), yv[s]);
        unpack8(ld8<HB>(dho, t * d + 8 * i), ov[s]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) yv[s][e] = ov[s][e] = 0.f;
      }
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int i = min(tid + s * kTeamT, d8 - 1);
      float wv[8], gv[8];
      ld_w(w, 8 * i, wv);
      ld_gate(gate, gmode, min(t, T - 1), d, 8 * i, gt, gv);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float o = ov[s][e] * wv[e];
        ss[0] = fmaf(yv[s][e], yv[s][e], ss[0]);
        ss[1] = fmaf(yv[s][e], o * gv[e], ss[1]);
        ss[2] = fmaf(yv[s][e], o, ss[2]);
      }
    }
    team_sum<3, kTeamT / 64>(ss, red[slot][team], tid >> 6);
    const float q = inv_rms(ss[0], d, eps), c = ss[1] / (float)d * q * q;
    if (live && tid == 0 && dgate && gmode == DS4MOE_GATE_TOKEN) dgate[t] = ss[2] * q;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int i = tid + s * kTeamT;
      if (live && i < d8) {
        float wv[8], gv[8], o[8], gg[8];
        ld_w(w, 8 * i, wv);
        ld_gate(gate, gmode, t, d, 8 * i, gt, gv);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float yq = yv[s][e] * q;
          acc[s][e] = fmaf(ov[s][e] * gv[e], yq, acc[s][e]);
          gg[e] = ov[s][e] * (yq * wv[e]);
          accg[s][e] += gg[e];
          o[e] = q * (ov[s][e] * gv[e] * wv[e] - yv[s][e] * c);
        }
        if (dgate && gmode == DS4MOE_GATE_FULL) st8<false>(dgate, t * d + 8 * i, gg);
        st8<YB>(dy, t * d + 8 * i, o);
      }
    }
  }
  if (m < M) {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int i = tid + s * kTeamT;
      if (i < d8) {
        if (dw) st8<false>(dw, (int64_t)m * d + 8 * i, acc[s]);
        if (dgate && gmode == DS4MOE_GATE_CHANNEL) st8<false>(dgate, (int64_t)m * d + 8 * i, accg[s]);
      }
    }
  }
}

// Sum of the M rows of part: a block adds 64 columns, sixteen threads of four
// columns each per row and sixteen rows at a time.  blockIdx.y picks one of
// two arrays.
__global__ __launch_bounds__(256) void k_norm_colsum(const float* __restrict__ p0, const float* __restrict__ p1,
                                                     int M, int d, float* __restrict__ o0, float* __restrict__ o1) {
  __shared__ float4_t red[16][16];
  const float* p = blockIdx.y ? p1 : p0;
  float* o = blockIdx.y ? o1 : o0;
  const int c = threadIdx.x & 15, g = threadIdx.x >> 4;
  const float4_t* src = (const float4_t*)(p + blockIdx.x * 64) + c;
  float4_t s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int m = g; m < M; m += 16) s += src[(int64_t)m * (d / 4)];
  red[g][c] = s;
  __syncthreads();
  if (g == 0) {
#pragma unroll
    for (int j = 1; j < 16; ++j) s += red[j][c];
    ((float4_t*)(o + blockIdx.x * 64))[c] = s;
  }
}

// ---------------------------------------------------------------- launchers
// Steps of NT threads x 8 columns that cover d, rounded up to a power of two.
static int steps(int d, int nt) {
  int s = 1;
  while (s * nt * 8 < d) s *= 2;
  return s;
}
#define DS4_STEPS(ns, ...)                          \
  do {                                              \
    if (ns == 1) {                                  \
      constexpr int NS = 1;                         \
      __VA_ARGS__                                   \
    } else if (ns == 2) {                           \
      constexpr int NS = 2;                         \
      __VA_ARGS__                                   \
    } else if (ns == 4) {                           \
      constexpr int NS = 4;                         \
      __VA_ARGS__                                   \
    } else {                                        \
      constexpr int NS = 8;                         \
      __VA_ARGS__                                   \
    }                                               \
  } while (0)
#define DS4_BOOL(cond, NAME, ...) \
  do {                            \
    if (cond) {                   \
      constexpr bool NAME = true; \
      __VA_ARGS__                 \
    } else {                      \
      constexpr bool NAME = false; \
      __VA_ARGS__                 \
    }                             \
  } while (0)

static bool bf(int dt) { return dt == DS4MOE_DT_BF16; }

hipError_t launch_norm_pre(const NormCall& c) {
  const int d = c.N.d_model;
  const dim3 grid((unsigned)c.T);
  DS4_STEPS(steps(d, 256), DS4_BOOL(bf(c.h_dt), HB, DS4_BOOL(bf(c.x_dt), XB, {
    DS4_LAUNCH((k_norm_pre<256, NS, HB, XB>), grid, dim3(256), 0, c.st, c.h, c.N.w_pre, d, c.N.eps, c.x);
  });););
  return hipGetLastError();
}

hipError_t launch_norm_post(const NormCall& c) {
  const int d = c.N.d_model;
  const dim3 grid((unsigned)c.T);
  DS4_STEPS(steps(d, 256), DS4_BOOL(bf(c.h_dt), HB, DS4_BOOL(bf(c.y_dt), YB, DS4_BOOL(bf(c.x_dt), XB, {
    DS4_LAUNCH((k_norm_post<256, NS, HB, YB, XB>), grid, dim3(256), 0, c.st, c.h, c.y, c.gate, c.N.gate, c.N.w_post,
               c.N.w_next, d, c.N.eps, c.N.res_scale, c.h_out, c.x);
  }););););
  return hipGetLastError();
}

hipError_t launch_norm_pre_grad(const NormCall& c) {
  const int d = c.N.d_model, M = norm_parts(c.T);
  const dim3 grid((M + kTeams - 1) / kTeams);
  float* dw = c.dw ? (M == 1 ? c.dw : c.part) : nullptr;
  DS4_STEPS(steps(d, kTeamT), DS4_BOOL(bf(c.h_dt), HB, DS4_BOOL(bf(c.x_dt), XB, {
    DS4_LAUNCH((k_norm_pre_grad<NS, HB, XB>), grid, dim3(kTeamT * kTeams), 0, c.st, c.h, c.dx, c.dh_out, c.N.w_pre, d,
               c.N.eps, c.N.res_scale, c.T, M, c.dh, dw);
  });););
  if (c.dw && M > 1)
    DS4_LAUNCH(k_norm_colsum, dim3(d / 64), dim3(256), 0, c.st, (const float*)dw, (const float*)nullptr, M, d, c.dw,
               (float*)nullptr);
  return hipGetLastError();
}

hipError_t launch_norm_post_grad(const NormCall& c) {
  const int d = c.N.d_model, M = norm_parts(c.T);
  const dim3 grid((M + kTeams - 1) / kTeams);
  const bool channel = c.dgate && c.N.gate == DS4MOE_GATE_CHANNEL;
  float* dw = c.dw ? (M == 1 ? c.dw : c.part) : nullptr;
  float* dg = channel && M > 1 ? c.part + (int64_t)M * d : c.dgate;
  DS4_STEPS(steps(d, kTeamT), DS4_BOOL(bf(c.h_dt), HB, DS4_BOOL(bf(c.y_dt), YB, {
    DS4_LAUNCH((k_norm_post_grad<NS, HB, YB>), grid, dim3(kTeamT * kTeams), 0, c.st, c.dh_out, c.y, c.gate, c.N.gate,
               c.N.w_post, d, c.N.eps, c.T, M, c.dy, dw, dg);
  });););
  if (M > 1 && (c.dw || channel)) {
    const float *p0 = dw, *p1 = dg;
    float *o0 = c.dw, *o1 = c.dgate;
    if (!c.dw) p0 = dg, o0 = c.dgate;
    DS4_LAUNCH(k_norm_colsum, dim3(d / 64, c.dw && channel ? 2 : 1), dim3(256), 0, c.st, p0, p1, M, d, o0, o1);
  }
  return hipGetLastError();
}

}  // namespace ds4
