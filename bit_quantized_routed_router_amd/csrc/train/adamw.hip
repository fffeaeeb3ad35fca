// AdamW over many tensors at once, and the norm of all their gradients:
//
//   g' = s g,  m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
//   p  = p - lr (wd p + (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps))
//   norm = sqrt(sum g^2),  s = min(1, max_norm / norm)
//
// States in fp32, or m and sqrt(v) as E4M3 codes with an fp32 scale (largest
// magnitude times the fp32 nearest to 1/448) per 256 values.  The root halves
// the exponents that v spans, and what is positive of it is held as the lowest
// code at least: a v that became 0 would make its value's next step as large as
// eps allows.  The scale is no power of two, so that a block that only decays is
// still followed.
// m, v, the root, the scale and the quotient by it are each rounded as IEEE
// operations are, so that the codes can be computed elsewhere bit for bit.
//
// A block takes a run of one tensor, 8 values to a thread: 32 lanes hold a
// block of 256, so its largest value stays within half a wave.  Which run is
// read from a table on the device that the program lays out once: passed with
// the launch instead, 46 tensors fit, and finding one among arguments in host
// memory took 8 us a launch (512 tensors of 32768: 236 us in 25 launches).
//
// Memory bounds it where there is much of it.  268 M bf16 values with 8-bit
// states (10 bytes a value): norm and step 647 us; in a trace the step 504 us,
// 5.3 TB/s (583 in the mean, first runs among them), the norm 115 to 132 us, 4.1
// to 4.7 TB/s.  512 tensors of 32768 bf16 values with masters and 8-bit states:
// norm and step 68 us (in a trace 10 and 5, 43).  129 tensors of 4096 in fp32:
// 11 to 12 us in three launches.
#include <algorithm>
#include <cmath>

#include "../trace.h"
#include "train.h"

namespace ds4 {

constexpr int kAdamThreads = 256;
// Values of a block: 4096, or a power of two more where that many blocks are
// enough.  Norm and step of one bf16 tensor, us, with runs of 4096 / 8192 /
// 16384 / 32768 values (* what the rule takes):
//   8-bit states  201 M    503 /  488*
//                 268 M    658 /  631*
//                 537 M   1294 / 1235 / 1254*
//                1074 M          2457 / 2467 / 2510*
//   fp32 states   268 M   1227 / 1244*
//                 537 M   2434 / 2467 / 2497*
//                1074 M          4893 / 4957 / 5036*
// 61 tensors of 1 to 5 M with fp32 states 26* / 29 / 31 (2048: 30).
constexpr int64_t kAdamRun = 4096;
constexpr int64_t kAdamBlocks = 1 << 15;
constexpr int64_t kAdamParts = 1 << 13;  // sums of squares, at most

// The table: ds4moe_param [n], then for each block (tensor, run).
struct AdamRun {
  int32_t tensor, run;
};
static size_t adam_map_at(int64_t n) { return (size_t)(n * sizeof(ds4moe_param) + 15) / 16 * 16; }
static int64_t adam_blocks(const ds4moe_param* p, int n, int64_t run) {
  int64_t blocks = 0;
  for (int i = 0; i < n; ++i) blocks += (p[i].n + run - 1) / run;
  return blocks;
}
static int64_t adam_run(const ds4moe_param* p, int n) {
  int64_t run = kAdamRun;
  // (a tensor has a block at least, however long the runs)
  while (adam_blocks(p, n, run) > kAdamBlocks + n) run *= 2;
  return run;
}
size_t adam_table_bytes(const ds4moe_param* p, int n) {
  return adam_map_at(n) + std::max<size_t>(16, sizeof(AdamRun) * (size_t)adam_blocks(p, n, adam_run(p, n)));
}
void adam_table(ds4moe_adamw* A, const ds4moe_param* p, int n, void* table) {
  A->n_params = n;
  A->run = adam_run(p, n);
  A->blocks = 0;
  std::copy(p, p + n, (ds4moe_param*)table);
  AdamRun* map = (AdamRun*)((uint8_t*)table + adam_map_at(n));
  for (int i = 0; i < n; ++i)
    for (int64_t r = 0; r * A->run < p[i].n; ++r) map[A->blocks++] = {i, (int32_t)r};
}
// blocks whose squares are summed together, and how many such groups there are
static int adam_group(const ds4moe_adamw& A) { return (int)((A.blocks + kAdamParts - 1) / kAdamParts); }
static int64_t adam_groups(const ds4moe_adamw& A) {
  const int g = adam_group(A);
  return g ? (A.blocks + g - 1) / g : 0;
}
size_t adam_ws_bytes(const ds4moe_adamw& A) { return std::max<size_t>(256, 8 * (size_t)adam_groups(A)); }

// Eight values from i on, `left` of them there; zeros for the others.
template <bool BF>
__device__ inline void get8(const void* p, int64_t i, int left, bool whole, float (&v)[8]) {
  if (whole) {
    unpack8<BF>(ld8<BF>(p, i), v);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    v[e] = 0.f;
    if (e < left) {
      if constexpr (BF) v[e] = __builtin_bit_cast(float, (uint32_t)((const uint16_t*)p)[i + e] << 16);
      else v[e] = ((const float*)p)[i + e];
    }
  }
}
template <bool BF>
__device__ inline void put8(void* p, int64_t i, int left, bool whole, const float (&v)[8]) {
  if (whole) {
    st8<BF>(p, i, v);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < left) {
      if constexpr (BF) ((uint16_t*)p)[i + e] = (uint16_t)bf16_pair(v[e], 0.f);
      else ((float*)p)[i + e] = v[e];
    }
}

// E4M3 codes times a scale, and back.
__device__ inline void get8_codes(const void* p, int64_t i, int left, bool whole, float scale, float (&v)[8]) {
  uint32_t w[2] = {0, 0};
  if (whole) {
    const u32x2_t x = *(const u32x2_t*)((const uint8_t*)p + i);
    w[0] = x.x;
    w[1] = x.y;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) w[e >> 2] |= (uint32_t)((const uint8_t*)p)[i + e] << (8 * (e & 3));
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const float2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[q], false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[q], true);
    v[4 * q] = a.x * scale;
    v[4 * q + 1] = a.y * scale;
    v[4 * q + 2] = b.x * scale;
    v[4 * q + 3] = b.y * scale;
  }
}
// The block of 256 that 32 lanes hold.  Its scale: largest times 1/448; 0 (and
// codes of 0) where that is below fp32's normal numbers; NaN, and so the whole
// block, where a value is not finite.
template <bool ROOT>
__device__ inline float put8_codes(void* p, int64_t i, int left, bool whole, const float (&v)[8]) {
  float top = 0.f;
  bool bad = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    top = fmaxf(top, fabsf(v[e]));
    bad |= !(fabsf(v[e]) <= 3.402823466e38f);
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
  const uint64_t half = 0xFFFFFFFFull << (threadIdx.x & 32);
  bad = (__ballot(bad) & half) != 0;
  float scale = top * (1.0f / 448.0f);
  if (scale < 1.17549435e-38f) scale = 0.f;
  const float r = scale > 0.f && !bad ? 1.0f / scale : 0.f;
  uint32_t w[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = v[4 * q + e], y0 = x * r;
      // the quotient x / scale rounded to nearest: r is, and one correction by
      // the remainder makes the product so (Markstein 1990)
      y[e] = bad ? 0.f : fmaf(fmaf(-y0, scale, x), r, y0);
      if constexpr (ROOT) y[e] = y[e] > 0.f ? fmaxf(y[e], 0.001953125f) : 0.f;  // 2^-9, the lowest code
    }
    int c = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    w[q] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], c, true);
  }
  if (whole) {
    *(u32x2_t*)((uint8_t*)p + i) = u32x2_t{w[0], w[1]};
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) ((uint8_t*)p)[i + e] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
  }
  return bad ? NAN : scale;
}

// The root within a step.  The instruction takes a subnormal argument as zero,
// which would leave eps alone in the denominator, so small ones are scaled.
// (sqrtf, which rounds to nearest: 129 tensors of 4096 6.6 us a step instead of 6.2.)
__device__ inline float root_near(float x) {
  const bool low = x < 0x1p-96f;
  const float r = __builtin_amdgcn_sqrtf(low ? x * 0x1p64f : x);
  return low ? r * 0x1p-32f : r;
}

struct AdamScalars {
  float b1, b1m, b2, b2m, eps;
  double lr, c1, c2, log_b1, log_b2;  // lr; 1 - b1^t and 1 - b2^t; for a step on the device
  const float *lr_dev, *grad_scale;
  const int32_t* step_dev;
};

template <bool PBF, bool GBF, bool FP8>
__global__ __launch_bounds__(kAdamThreads) void k_adamw(const ds4moe_param* __restrict__ params,
                                                        const AdamRun* __restrict__ map, int64_t run, AdamScalars s) {
  const float gs = s.grad_scale ? *s.grad_scale : 1.0f;
  const AdamRun r = map[blockIdx.x];
  const ds4moe_param q = params[r.tensor];
  const int64_t at = r.run * run;
  if (!(fabsf(gs) <= 3.402823466e38f)) return;  // a step without finite gradients changes nothing
  const double lr = s.lr_dev ? (double)*s.lr_dev : s.lr;
  double c1 = s.c1, c2 = s.c2;
  if (s.step_dev) {
    const double step = max(*s.step_dev, 1);
    c1 = 1.0 - exp(step * s.log_b1);
    c2 = 1.0 - exp(step * s.log_b2);
  }
  const float decay = (float)(lr * q.weight_decay), up = (float)(lr / c1), root = (float)(1.0 / sqrt(c2));
  const uintptr_t align = (uintptr_t)q.param | (uintptr_t)q.grad | (uintptr_t)q.master |
                          (FP8 ? ((uintptr_t)q.m | (uintptr_t)q.v) << 1 : (uintptr_t)q.m | (uintptr_t)q.v);
  const bool vec = (align & 15) == 0;
  const int64_t end = min(at + run, q.n);
  // FP8: every lane of a block of 256 stays, so that its largest value is known
  for (int64_t i0 = at; i0 < end; i0 += 8 * kAdamThreads) {
    const int64_t i = i0 + 8 * threadIdx.x;
    const int left = (int)max((int64_t)0, min((int64_t)8, end - i));
    const bool whole = vec && left == 8;
    if (!FP8 && left == 0) break;
    float g[8], m[8], v[8], p[8];
    float ms = 0.f, vs = 0.f;
    if (FP8 && left > 0) {
      ms = q.m_scale[i >> 8];
      vs = q.v_scale[i >> 8];
    }
    get8<GBF>(q.grad, i, left, whole, g);
    if (q.master) get8<false>(q.master, i, left, whole, p);
    else get8<PBF>(q.param, i, left, whole, p);
    if constexpr (FP8) {
      get8_codes(q.m, i, left, whole, ms, m);
      get8_codes(q.v, i, left, whole, vs, v);
    } else {
      get8<false>(q.m, i, left, whole, m);
      get8<false>(q.v, i, left, whole, v);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      {
#pragma clang fp contract(off)
        const float d = gs * g[e];
        if (FP8) v[e] = v[e] * v[e];
        m[e] = s.b1 * m[e] + s.b1m * d;
        v[e] = s.b2 * v[e] + s.b2m * (d * d);
      }
      const float r = FP8 ? sqrtf(v[e]) : root_near(v[e]);
      // (1 - decay as an fp32 would be 1 for a decay below 3e-8, and a fifth off at 1e-7)
      p[e] -= fmaf(decay, p[e], up * m[e] * __builtin_amdgcn_rcpf(root * r + s.eps));
      if (FP8) v[e] = r;
    }
    put8<PBF>(q.param, i, left, whole, p);
    if (q.master) put8<false>(q.master, i, left, whole, p);
    if constexpr (FP8) {
      ms = put8_codes<false>(q.m, i, left, whole, m);
      vs = put8_codes<true>(q.v, i, left, whole, v);
      if ((threadIdx.x & 31) == 0 && left > 0) {
        q.m_scale[i >> 8] = ms;
        q.v_scale[i >> 8] = vs;
      }
    } else {
      put8<false>(q.m, i, left, whole, m);
      put8<false>(q.v, i, left, whole, v);
    }
  }
}

// ---------------------------------------------------------------- norm
// Sums of squares in fp64: fp32 squares overflow above 2^64, and the sum over
// 10^9 values keeps its digits.
__device__ inline double block_sum(double x, double* lds, int waves) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) x += __shfl_xor(x, o);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  x = 0.0;
  for (int w = 0; w < waves; ++w) x += lds[w];
  return x;
}
template <bool GBF>
__global__ __launch_bounds__(kAdamThreads) void k_adamw_squares(const ds4moe_param* __restrict__ params,
                                                                const AdamRun* __restrict__ map, int64_t blocks,
                                                                int group, int64_t run, double* __restrict__ part) {
  __shared__ double lds[kAdamThreads / 64];
  double sum = 0.0;
  const int64_t last = min(blocks, ((int64_t)blockIdx.x + 1) * group);
  for (int64_t b = (int64_t)blockIdx.x * group; b < last; ++b) {
    const AdamRun r = map[b];
    const void* grad = params[r.tensor].grad;
    const int64_t at = r.run * run, end = min(at + run, params[r.tensor].n);
    const bool vec = ((uintptr_t)grad & 15) == 0;
    constexpr int U = 2;
    for (int64_t i0 = at + 8 * threadIdx.x; i0 < end; i0 += U * 8 * kAdamThreads) {
      float g[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t i = i0 + u * 8 * kAdamThreads;
        const int left = (int)max((int64_t)0, min((int64_t)8, end - i));
        get8<GBF>(grad, i, left, vec && left == 8, g[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += (double)g[u][e] * (double)g[u][e];
    }
  }
  sum = block_sum(sum, lds, kAdamThreads / 64);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}
__global__ __launch_bounds__(1024) void k_adamw_norm(const double* __restrict__ part, int64_t n, float max_norm,
                                                     float* __restrict__ out) {
  __shared__ double lds[16];
  double sum = 0.0;
#pragma unroll 8
  for (int64_t i = threadIdx.x; i < n; i += 1024) sum += part[i];
  sum = block_sum(sum, lds, 16);
  if (threadIdx.x != 0) return;
  const float norm = (float)sqrt(sum);
  out[0] = norm;
  out[1] = !(norm <= 3.402823466e38f) ? NAN : norm > max_norm ? max_norm / norm : 1.0f;
}

// ---------------------------------------------------------------- launches
static const ds4moe_param* adam_params(const AdamCall& c) { return (const ds4moe_param*)c.table; }
static const AdamRun* adam_map(const AdamCall& c) {
  return (const AdamRun*)((const uint8_t*)c.table + adam_map_at(c.A.n_params));
}
template <bool PBF, bool GBF, bool FP8>
static hipError_t adam_step(const AdamCall& c) {
  AdamScalars s{};
  const ds4moe_adamw& A = c.A;
  s.b1 = (float)A.beta1;
  s.b1m = (float)(1.0 - A.beta1);
  s.b2 = (float)A.beta2;
  s.b2m = (float)(1.0 - A.beta2);
  s.eps = (float)A.eps;
  s.lr = A.lr;
  s.log_b1 = std::log(A.beta1);
  s.log_b2 = std::log(A.beta2);
  s.c1 = -std::expm1(c.step * s.log_b1);
  s.c2 = -std::expm1(c.step * s.log_b2);
  s.lr_dev = A.lr_dev;
  s.step_dev = A.step_dev;
  s.grad_scale = c.grad_scale;
  if (A.blocks == 0) return hipSuccess;
  DS4_LAUNCH((k_adamw<PBF, GBF, FP8>), dim3((unsigned)A.blocks), dim3(kAdamThreads), 0, c.st, adam_params(c), adam_map(c),
             A.run, s);
  return hipGetLastError();
}
template <bool PBF, bool GBF>
static hipError_t adam_step_state(const AdamCall& c) {
  return c.A.state == DS4MOE_STATE_FP8 ? adam_step<PBF, GBF, true>(c) : adam_step<PBF, GBF, false>(c);
}
template <bool PBF>
static hipError_t adam_step_grad(const AdamCall& c) {
  return c.A.grad_dtype == DS4MOE_DT_BF16 ? adam_step_state<PBF, true>(c) : adam_step_state<PBF, false>(c);
}
hipError_t launch_adamw_step(const AdamCall& c) {
  return c.A.param_dtype == DS4MOE_DT_BF16 ? adam_step_grad<true>(c) : adam_step_grad<false>(c);
}

template <bool GBF>
static hipError_t adam_norm(const AdamCall& c) {
  const int64_t groups = adam_groups(c.A);
  if (groups > 0)
    DS4_LAUNCH((k_adamw_squares<GBF>), dim3((unsigned)groups), dim3(kAdamThreads), 0, c.st, adam_params(c), adam_map(c),
               c.A.blocks, adam_group(c.A), c.A.run, c.ws);
  DS4_LAUNCH(k_adamw_norm, dim3(1), dim3(1024), 0, c.st, (const double*)c.ws, groups, c.max_norm, c.out);
  return hipGetLastError();
}
hipError_t launch_adamw_norm(const AdamCall& c) {
  return c.A.grad_dtype == DS4MOE_DT_BF16 ? adam_norm<true>(c) : adam_norm<false>(c);
}

}  // namespace ds4
