// Internal declarations of the operators around the layer: block norms,
// tokens sorted by expert and back, MXFP4 rows and products.  They are apart
// from the layer's own sources (one folder up) and share only its small
// device helpers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../common.h"
#include "ds4moe.h"

namespace ds4 {

constexpr int64_t kOpsMaxT = 1 << 20;     // tokens of a norm, sort, dispatch or combine call
constexpr int64_t kOpsMaxRows = 1 << 24;  // rows of an MXFP4 call, and T * top_k of a sorted one
// values of a product gradient: its blocks of 256 threads take 256 columns and
// 32 rows (and one more tile an expert), and a launch fewer than 2^32 threads
constexpr int64_t kOpsMaxGrad = (1ll << 37) - (1ll << 29);

// ---------------------------------------------------------------- typed rows
// Eight consecutive elements (index i, a multiple of 8) of an fp32 or
// bfloat16 array as fp32, and back.  The conversion to bfloat16 rounds to
// nearest, ties to even, and keeps NaN.
template <bool BF>
struct Raw8;
template <>
struct Raw8<true> {
  u32x4_t a;
};
template <>
struct Raw8<false> {
  float4_t a, b;
};
template <bool BF>
__device__ inline Raw8<BF> ld8(const void* p, int64_t i) {
  Raw8<BF> r;
  if constexpr (BF) {
    r.a = *(const u32x4_t*)((const uint16_t*)p + i);
  } else {
    const float4_t* s = (const float4_t*)((const float*)p + i);
    r.a = s[0];
    r.b = s[1];
  }
  return r;
}
template <bool BF>
__device__ inline void unpack8(const Raw8<BF>& r, float (&v)[8]) {
  if constexpr (BF) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      v[2 * p] = __builtin_bit_cast(float, r.a[p] << 16);
      v[2 * p + 1] = __builtin_bit_cast(float, r.a[p] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      v[p] = r.a[p];
      v[4 + p] = r.b[p];
    }
  }
}
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float float2_t __attribute__((ext_vector_type(2)));
__device__ inline uint32_t bf16_pair(float lo, float hi) {
  const float2_t f = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2_t));
}
template <bool BF>
__device__ inline void st8(void* p, int64_t i, const float (&v)[8]) {
  if constexpr (BF) {
    u32x4_t o;
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = bf16_pair(v[2 * q], v[2 * q + 1]);
    *(u32x4_t*)((uint16_t*)p + i) = o;
  } else {
    float4_t* d = (float4_t*)((float*)p + i);
    d[0] = float4_t{v[0], v[1], v[2], v[3]};
    d[1] = float4_t{v[4], v[5], v[6], v[7]};
  }
}

// ---------------------------------------------------------------- sums over a wave
template <int CTRL>
__device__ inline float dpp_add(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}
// The sum over the 64 lanes, the same value in every lane: quads, rows of 16
// by rotation, then the four rows through scalar registers.
__device__ inline float wave_sum(float v) {
  v = dpp_add<0xB1>(v);   // quad_perm [1,0,3,2]
  v = dpp_add<0x4E>(v);   // quad_perm [2,3,0,1]
  v = dpp_add<0x124>(v);  // row_ror:4
  v = dpp_add<0x128>(v);  // row_ror:8
  const int b = __builtin_bit_cast(int, v);
  const float r0 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 0));
  const float r1 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 16));
  const float r2 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 32));
  const float r3 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 48));
  return (r0 + r1) + (r2 + r3);
}

// ---------------------------------------------------------------- a token's slots
// Lane j holds the position of the token's slot j (k <= 16 of them; -1 for
// none or one outside [0, rows)): one load for all, read back lane by lane,
// where a loop of scalar loads would wait for each in turn.
__device__ inline int slot_positions(const int32_t* inv, int64_t t, int k, int rows) {
  const int j = min((int)(threadIdx.x & 63), k - 1);
  const int p = inv[t * k + j];
  return p >= 0 && p < rows ? p : -1;
}
__device__ inline float lane_float(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

// ---------------------------------------------------------------- launchers
struct NormCall {
  ds4moe_norm N;
  const void *h, *y, *dx, *dh_out;  // inputs (those that the call has)
  const float* gate;
  int h_dt, y_dt, x_dt;
  int64_t T;
  void *x, *h_out, *dy, *dh;  // outputs
  float *dw, *dgate, *part;
  hipStream_t st;
};
int norm_parts(int d, int64_t T);  // partial rows of the gradients summed over tokens
hipError_t launch_norm_pre(const NormCall& c);
hipError_t launch_norm_post(const NormCall& c);
hipError_t launch_norm_pre_grad(const NormCall& c);
hipError_t launch_norm_post_grad(const NormCall& c);

size_t group_ws_bytes(int64_t S, int E);
hipError_t launch_group(const int32_t* idx, int64_t S, int E, int32_t* counts, int32_t* offsets, int32_t* perm,
                        int32_t* inv, int32_t* ws, hipStream_t st);
hipError_t launch_dispatch(const void* x, int dt, int64_t T, int k, int d, const int32_t* inv, void* xs, int64_t rows,
                           hipStream_t st);
hipError_t launch_combine(const void* ys, int ys_dt, int64_t rows, const int32_t* inv, const float* w,
                          const void* base, int64_t T, int k, int d, void* y, int y_dt, hipStream_t st);
hipError_t launch_combine_grad(const void* dy, int dy_dt, const void* ys, int ys_dt, int64_t rows, const int32_t* inv,
                               const float* w, int64_t T, int k, int d, void* dys, float* dw, float* dl,
                               hipStream_t st);

hipError_t launch_mx_quantize(const void* x, int dt, int64_t T, const int32_t* inv, int k, int64_t rows, int cols,
                              void* packed, hipStream_t st);
hipError_t launch_mx_dequantize(const void* packed, int64_t rows, int cols, void* out, int dt, hipStream_t st);

struct MxProduct {
  const uint8_t* a;  // packed rows (forward)
  const void* dy;    // rows of gradients (backward)
  int64_t n;
  int rows, cols, E;
  const uint8_t *w, *w2;
  const int32_t* offsets;
  void* out;
  int dy_dt, out_dt;
  hipStream_t st;
};
hipError_t launch_mx_product(const MxProduct& c);
hipError_t launch_mx_product_grad(const MxProduct& c);

}  // namespace ds4
