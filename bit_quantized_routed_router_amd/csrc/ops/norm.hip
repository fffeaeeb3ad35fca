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
// and by the latency of load, sum, store for few.  Kernel times: post with the
// next pre-norm, one fp32 row of 4096 3.4 us, 2048 bf16 rows with fp32 y 84 MB
// in 14 us (6 TB/s); 2047 bf16 rows of 1792: post_grad 22 MB in 10.3 us,
// pre_grad 29 MB in 9.1 us, each with 3.4 us for the sum over tokens.  Above
// 8192 columns post_grad spills 51 to 65 registers a thread, on 4096 fp32
// columns 3.
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
// Blocks of 1024 threads in TEAMS teams of TT; team m of the grid's M takes
// rows m, m + M, ..., the next row's loads under way while a row is summed
// and written, and keeps its share of the sums over tokens in registers.  The
// block's teams add theirs up through LDS in order into the block's row of
// part, and k_norm_colsum adds those rows in order, so the result does not
// depend on how the blocks ran.
constexpr int kGradT = 1024, kMaxParts = 256;
static int grad_team(int d) { return d <= 2048 ? 256 : d <= 4096 ? 512 : 1024; }
int norm_parts(int d, int64_t T) {
  const int teams = kGradT / grad_team(d);
  return (int)std::min<int64_t>((T + teams - 1) / teams, kMaxParts);
}

// Adds the teams' acc in order and writes the block's sum to out: each team
// lays its share into lds (8 TT columns of it), then every thread adds pairs
// of columns.
template <int TT, int NS>
__device__ inline void add_teams(const float (&acc)[NS][8], float* lds, int team, int tid, int d, float* out) {
  constexpr int TEAMS = kGradT / TT;
  if constexpr (TEAMS == 1) {
#pragma unroll
    for (int s = 0; s < NS; ++s)
      if (8 * (tid + s * TT) < d) st8<false>(out, 8 * (tid + s * TT), acc[s]);
  } else {
    static_assert(NS == 1, "one step per team");
    __syncthreads();  // lds may still be read
    st8<false>(lds + team * 8 * TT, 8 * tid, acc[0]);
    __syncthreads();
    for (int c = 2 * threadIdx.x; c < d; c += 2 * kGradT) {
      float2_t v = *(const float2_t*)(lds + c);
#pragma unroll
      for (int m = 1; m < TEAMS; ++m) v += *(const float2_t*)(lds + m * 8 * TT + c);
      *(float2_t*)(out + c) = v;
    }
  }
}

template <int TT, int NS, bool HB, bool XB>
__global__ __launch_bounds__(kGradT) void k_norm_pre_grad(const void* __restrict__ h, const void* __restrict__ dx,
                                                          const void* dho, const float* __restrict__ w, int d,
                                                          float eps, float rho, int64_t T, void* dh,
                                                          float* __restrict__ dw) {
  constexpr int TEAMS = kGradT / TT, NW = TT / 64;
  constexpr bool AHEAD = NS == 1;  // two steps leave no registers for the next row
  __shared__ float red[2][TEAMS][2 * NW];
  __shared__ __align__(16) float lds[TEAMS > 1 ? kGradT * 8 : 4];
  const int team = threadIdx.x / TT, tid = threadIdx.x % TT, d8 = d / 8;
  const int64_t M = (int64_t)gridDim.x * TEAMS;
  int64_t t = (int64_t)blockIdx.x * TEAMS + team;
  float acc[NS][8] = {}, wv[NS][8];
  Raw8<HB> hr[NS], ho[NS];
  Raw8<XB> xr[NS];
  auto load = [&](int64_t row) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int64_t i = row * d + 8 * min(tid + s * TT, d8 - 1);
      hr[s] = ld8<HB>(h, i);
      xr[s] = ld8<XB>(dx, i);
      ho[s] = dho ? ld8<HB>(dho, i) : Raw8<HB>{};
    }
  };
#pragma unroll
  for (int s = 0; s < NS; ++s) ld_w(w, 8 * min(tid + s * TT, d8 - 1), wv[s]);
  if (AHEAD) load(min(t, T - 1));
  int slot = 0;
  for (int64_t t0 = (int64_t)blockIdx.x * TEAMS; t0 < T; t0 += M, t += M, slot ^= 1) {
    float hv[NS][8], xv[NS][8], o[NS][8];
    float ss[2] = {0.f, 0.f};
    if (!AHEAD) load(min(t, T - 1));
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      unpack8(hr[s], hv[s]);
      unpack8(xr[s], xv[s]);
      unpack8(ho[s], o[s]);
      if (t >= T || tid + s * TT >= d8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) hv[s][e] = xv[s][e] = 0.f;
      }
    }
    if (AHEAD) load(min(t + M, T - 1));
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss[0] = fmaf(hv[s][e], hv[s][e], ss[0]);
        ss[1] = fmaf(hv[s][e], xv[s][e] * wv[s][e], ss[1]);
      }
    team_sum<2, NW>(ss, red[slot][team], tid >> 6);
    const float r = inv_rms(ss[0], d, eps), c = ss[1] / (float)d * r * r;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        acc[s][e] = fmaf(xv[s][e], hv[s][e] * r, acc[s][e]);
        o[s][e] = (dho ? rho * o[s][e] : 0.f) + r * (xv[s][e] * wv[s][e] - hv[s][e] * c);
      }
      if (t < T && tid + s * TT < d8) st8<HB>(dh, t * d + 8 * (tid + s * TT), o[s]);
    }
  }
  if (dw) add_teams<TT, NS>(acc, lds, team, tid, d, dw + (int64_t)blockIdx.x * d);
}

template <int TT, int NS, bool HB, bool YB>
__global__ __launch_bounds__(kGradT) void k_norm_post_grad(const void* __restrict__ dho, const void* y,
                                                           const float* __restrict__ gate, int gmode,
                                                           const float* __restrict__ w, int d, float eps, int64_t T,
                                                           void* dy, float* __restrict__ dw,
                                                           float* __restrict__ dgate) {
  constexpr int TEAMS = kGradT / TT, NW = TT / 64;
  constexpr bool AHEAD = NS == 1;  // two steps leave no registers for the next row
  __shared__ float red[2][TEAMS][3 * NW];
  __shared__ __align__(16) float lds[TEAMS > 1 ? kGradT * 8 : 4];
  const int team = threadIdx.x / TT, tid = threadIdx.x % TT, d8 = d / 8;
  const int64_t M = (int64_t)gridDim.x * TEAMS;
  int64_t t = (int64_t)blockIdx.x * TEAMS + team;
  const bool full = gmode == DS4MOE_GATE_FULL;
  float acc[NS][8] = {}, accg[NS][8] = {}, wv[NS][8], gv[NS][8];
  Raw8<YB> yr[NS];
  Raw8<HB> hr[NS];
  Raw8<false> gr[NS];
  float gt = 1.0f;
  auto load = [&](int64_t row) __attribute__((always_inline)) {
    if (gmode == DS4MOE_GATE_TOKEN) gt = gate[row];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int64_t i = row * d + 8 * min(tid + s * TT, d8 - 1);
      yr[s] = ld8<YB>(y, i);
      hr[s] = ld8<HB>(dho, i);
      if (full) gr[s] = ld8<false>(gate, i);
    }
  };
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int c = 8 * min(tid + s * TT, d8 - 1);
    ld_w(w, c, wv[s]);
    if (gmode == DS4MOE_GATE_CHANNEL) unpack8(ld8<false>(gate, c), gv[s]);
  }
  if (AHEAD) load(min(t, T - 1));
  int slot = 0;
  for (int64_t t0 = (int64_t)blockIdx.x * TEAMS; t0 < T; t0 += M, t += M, slot ^= 1) {
    float yv[NS][8], ov[NS][8];
    float ss[3] = {0.f, 0.f, 0.f};
    if (!AHEAD) load(min(t, T - 1));
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      unpack8(yr[s], yv[s]);
      unpack8(hr[s], ov[s]);
      if (full) {
        unpack8(gr[s], gv[s]);
      } else if (gmode != DS4MOE_GATE_CHANNEL) {
#pragma unroll
        for (int e = 0; e < 8; ++e) gv[s][e] = gt;
      }
      if (t >= T || tid + s * TT >= d8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) yv[s][e] = ov[s][e] = 0.f;
        if (gmode != DS4MOE_GATE_CHANNEL) {
#pragma unroll
          for (int e = 0; e < 8; ++e) gv[s][e] = 0.f;
        }
      }
    }
    if (AHEAD) load(min(t + M, T - 1));
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float o = ov[s][e] * wv[s][e];
        ss[0] = fmaf(yv[s][e], yv[s][e], ss[0]);
        ss[1] = fmaf(yv[s][e], o * gv[s][e], ss[1]);
        ss[2] = fmaf(yv[s][e], o, ss[2]);
      }
    team_sum<3, NW>(ss, red[slot][team], tid >> 6);
    const float q = inv_rms(ss[0], d, eps), c = ss[1] / (float)d * q * q;
    if (t < T && tid == 0 && dgate && gmode == DS4MOE_GATE_TOKEN) dgate[t] = ss[2] * q;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const bool on = t < T && tid + s * TT < d8;
      const int64_t i = t * d + 8 * (tid + s * TT);
      float o[8], gg[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float yq = yv[s][e] * q;
        acc[s][e] = fmaf(ov[s][e] * gv[s][e], yq, acc[s][e]);
        gg[e] = ov[s][e] * (yq * wv[s][e]);
        accg[s][e] += gg[e];
        o[e] = q * (ov[s][e] * gv[s][e] * wv[s][e] - yv[s][e] * c);
      }
      if (on && full && dgate) st8<false>(dgate, i, gg);
      if (on) st8<YB>(dy, i, o);
    }
  }
  if (dw) add_teams<TT, NS>(acc, lds, team, tid, d, dw + (int64_t)blockIdx.x * d);
  if (dgate && gmode == DS4MOE_GATE_CHANNEL)
    add_teams<TT, NS>(accg, lds, team, tid, d, dgate + (int64_t)blockIdx.x * d);
}

// Sum of the M rows of part: a block adds 32 columns, eight threads of four
// columns each per row and 32 rows at a time.  blockIdx.y picks one of two
// arrays.
__global__ __launch_bounds__(256) void k_norm_colsum(const float* __restrict__ p0, const float* __restrict__ p1,
                                                     int M, int d, float* __restrict__ o0, float* __restrict__ o1) {
  __shared__ float4_t red[32][8];
  const float* p = blockIdx.y ? p1 : p0;
  float* o = blockIdx.y ? o1 : o0;
  const int c = threadIdx.x & 7, g = threadIdx.x >> 3;
  const float4_t* src = (const float4_t*)(p + blockIdx.x * 32) + c;
  float4_t s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int m = g; m < M; m += 32) s += src[(int64_t)m * (d / 4)];
  red[g][c] = s;
  __syncthreads();
  if (g == 0) {
#pragma unroll
    for (int j = 1; j < 32; ++j) s += red[j][c];
    ((float4_t*)(o + blockIdx.x * 32))[c] = s;
  }
}

// ---------------------------------------------------------------- launchers
// Threads of a row and their steps of 8 columns.  256 threads keep more rows
// on a CU (2048 rows of 4096: 14.1 us, 15.2 with 512); above 8 K columns 512
// halve the longest part of a row (2048 rows of 16384 67.8 us, 73.8 with 256;
// one row 6.3 and 8.4).
#define DS4_ROW(d, ...)                  \
  do {                                   \
    if (d <= 2048) {                     \
      constexpr int NT = 256, NS = 1;    \
      __VA_ARGS__                        \
    } else if (d <= 4096) {              \
      constexpr int NT = 256, NS = 2;    \
      __VA_ARGS__                        \
    } else if (d <= 8192) {              \
      constexpr int NT = 256, NS = 4;    \
      __VA_ARGS__                        \
    } else {                             \
      constexpr int NT = 512, NS = 4;    \
      __VA_ARGS__                        \
    }                                    \
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
  DS4_ROW(d, DS4_BOOL(bf(c.h_dt), HB, DS4_BOOL(bf(c.x_dt), XB, {
    DS4_LAUNCH((k_norm_pre<NT, NS, HB, XB>), grid, dim3(NT), 0, c.st, c.h, c.N.w_pre, d, c.N.eps, c.x);
  });););
  return hipGetLastError();
}

hipError_t launch_norm_post(const NormCall& c) {
  const int d = c.N.d_model;
  const dim3 grid((unsigned)c.T);
  DS4_ROW(d, DS4_BOOL(bf(c.h_dt), HB, DS4_BOOL(bf(c.y_dt), YB, DS4_BOOL(bf(c.x_dt), XB, {
    DS4_LAUNCH((k_norm_post<NT, NS, HB, YB, XB>), grid, dim3(NT), 0, c.st, c.h, c.y, c.gate, c.N.gate, c.N.w_post,
               c.N.w_next, d, c.N.eps, c.N.res_scale, c.h_out, c.x);
  }););););
  return hipGetLastError();
}

// the team that a width takes, and its steps
#define DS4_TEAM(d, ...)                  \
  do {                                    \
    if (d <= 2048) {                      \
      constexpr int TT = 256, NS = 1;     \
      __VA_ARGS__                         \
    } else if (d <= 4096) {               \
      constexpr int TT = 512, NS = 1;     \
      __VA_ARGS__                         \
    } else if (d <= 8192) {               \
      constexpr int TT = 1024, NS = 1;    \
      __VA_ARGS__                         \
    } else {                              \
      constexpr int TT = 1024, NS = 2;    \
      __VA_ARGS__                         \
    }                                     \
  } while (0)

hipError_t launch_norm_pre_grad(const NormCall& c) {
  const int d = c.N.d_model, M = norm_parts(d, c.T);
  float* dw = c.dw ? (M == 1 ? c.dw : c.part) : nullptr;
  DS4_TEAM(d, DS4_BOOL(bf(c.h_dt), HB, DS4_BOOL(bf(c.x_dt), XB, {
    DS4_LAUNCH((k_norm_pre_grad<TT, NS, HB, XB>), dim3(M), dim3(kGradT), 0, c.st, c.h, c.dx, c.dh_out, c.N.w_pre, d,
               c.N.eps, c.N.res_scale, c.T, c.dh, dw);
  });););
  if (c.dw && M > 1)
    DS4_LAUNCH(k_norm_colsum, dim3(d / 32), dim3(256), 0, c.st, (const float*)dw, (const float*)nullptr, M, d, c.dw,
               (float*)nullptr);
  return hipGetLastError();
}

hipError_t launch_norm_post_grad(const NormCall& c) {
  const int d = c.N.d_model, M = norm_parts(d, c.T);
  const bool channel = c.dgate && c.N.gate == DS4MOE_GATE_CHANNEL;
  float* dw = c.dw ? (M == 1 ? c.dw : c.part) : nullptr;
  float* dg = channel && M > 1 ? c.part + (int64_t)M * d : c.dgate;
  DS4_TEAM(d, DS4_BOOL(bf(c.h_dt), HB, DS4_BOOL(bf(c.y_dt), YB, {
    DS4_LAUNCH((k_norm_post_grad<TT, NS, HB, YB>), dim3(M), dim3(kGradT), 0, c.st, c.dh_out, c.y, c.gate, c.N.gate,
               c.N.w_post, d, c.N.eps, c.T, c.dy, dw, dg);
  });););
  if (M > 1 && (c.dw || channel)) {
    const float *p0 = dw, *p1 = dg;
    float *o0 = c.dw, *o1 = c.dgate;
    if (!c.dw) p0 = dg, o0 = c.dgate;
    DS4_LAUNCH(k_norm_colsum, dim3(d / 32, c.dw && channel ? 2 : 1), dim3(256), 0, c.st, p0, p1, M, d, o0, o1);
  }
  return hipGetLastError();
}

}  // namespace ds4
