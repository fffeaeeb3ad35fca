// MXFP4 rows of activations (format in include/ds4moe.h): quantisation into a
// packed matrix, at the rows that a sort gives, and the values back.
//
// A lane takes 8 columns, four lanes a block of 32: the block's largest
// magnitude comes from two exchanges within the quad, as an integer maximum
// of the bits without their sign (so a NaN counts as the largest), and the
// conversion instruction rounds to E2M1 to nearest, ties to the even code,
// beyond 6 to 6.  Codes leave as one word per lane and scales as one byte per
// quad.  Both kernels are bound by memory: 2048 bf16 tokens of 4096 to 6 rows
// each 44 MB in 10.7 us, back to bf16 127 MB in 19 us (6.6 TB/s); six rows 2.6
// and 2.3 us.
#include <algorithm>

#include "../trace.h"
#include "ops.h"

namespace ds4 {

template <int CTRL>
__device__ inline uint32_t dpp_max(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false));
}

// 2^(sc - 127), by the exponent field (sc = 0: the subnormal 2^-127)
__device__ inline float pow2_scale(uint32_t sc) {
  return __builtin_bit_cast(float, sc ? sc << 23 : 0x00400000u);
}

// E8M0 code of a block whose largest magnitude has the fp32 bits m:
// floor(log2) - 2 + 127 within 0 .. 254; 255 where the block holds an
// infinity or a NaN, 0 where all of it is zero.
__device__ inline uint32_t block_scale(uint32_t m) {
  if (m >= 0x7F800000u) return 255u;
  // a subnormal's exponent is below the range's: it gives 0 as well
  return (uint32_t)max((int)(m >> 23) - 2, 0);
}

// Codes of -0 become +0, as the format's quantiser has them.
__device__ inline uint32_t no_minus_zero(uint32_t c) {
  const uint32_t m = c & 0x77777777u;
  const uint32_t any = (m | (m >> 1) | (m >> 2)) & 0x11111111u;
  return m | (c & (any << 3));
}

// Block b: token b / nb, columns 2048 (b % nb) onward, eight per thread.
template <bool BF>
__global__ __launch_bounds__(256) void k_mx_quantize(const void* __restrict__ x, const int32_t* __restrict__ inv,
                                                     int k, int cols, int nb, int rows,
                                                     uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const int64_t t = blockIdx.x / nb;
  const int c = ((blockIdx.x % nb) * 256 + threadIdx.x) * 8;
  const int pos = inv ? slot_positions(inv, t, k, rows) : (int)t;
  if (c >= cols) return;  // whole half waves: cols is a multiple of 256
  const Raw8<BF> v = ld8<BF>(x, t * cols + c);
  uint32_t m = 0;
  float f[8];
  unpack8(v, f);
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, __builtin_bit_cast(uint32_t, f[e]) & 0x7FFFFFFFu);
  m = dpp_max<0xB1>(m);
  m = dpp_max<0x4E>(m);
  const uint32_t sc = block_scale(m);
  uint32_t w = 0;
  if (sc != 255u) {
    const float s = pow2_scale(sc);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[0], f[1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[2], f[3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[4], f[5], s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[6], f[7], s, 3);
    w = no_minus_zero(w);
  }
  for (int j = 0; j < k; ++j) {
    const int64_t p = __builtin_amdgcn_readlane(pos, j);
    if (p < 0) continue;
    const int64_t i = p * cols + c;
    *(uint32_t*)(codes + i / 2) = w;
    if ((threadIdx.x & 3) == 0) scales[i / 32] = (uint8_t)sc;
  }
}

template <bool BF>
__global__ __launch_bounds__(256) void k_mx_dequantize(const uint8_t* __restrict__ codes,
                                                       const uint8_t* __restrict__ scales, int64_t n8,
                                                       void* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n8) return;
  const uint32_t w = ((const uint32_t*)codes)[i];
  const uint32_t sc = scales[i / 4];
  // the conversion takes the exponent field as an E8M0 code: 0 is 2^-127, 255 NaN
  const float s = __builtin_bit_cast(float, sc << 23);
  if constexpr (BF) {
    u32x4_t o;
    o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
    o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
    o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
    o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
    ((u32x4_t*)out)[i] = o;
    return;
  }
  const float2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0), p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
  const float2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2), p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
  const float v[8] = {p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
  st8<BF>(out, i * 8, v);
}

hipError_t launch_mx_quantize(const void* x, int dt, int64_t T, const int32_t* inv, int k, int64_t rows, int cols,
                              void* packed, hipStream_t st) {
  const int nb = (cols + 2047) / 2048;
  uint8_t* codes = (uint8_t*)packed;
  uint8_t* scales = codes + rows * cols / 2;
  // a launch takes fewer than 2^32 threads: 2^20 tokens, as many as a sorted
  // call has at most
  for (int64_t t = 0; t < T; t += kOpsMaxT) {
    const int64_t n = std::min(T - t, kOpsMaxT), i = t * cols;
    const dim3 grid((unsigned)(n * nb));
    if (dt == DS4MOE_DT_BF16)
      DS4_LAUNCH(k_mx_quantize<true>, grid, dim3(256), 0, st, (const void*)((const uint16_t*)x + i), inv, k, cols, nb,
                 (int)rows, codes + i / 2, scales + i / 32);
    else
      DS4_LAUNCH(k_mx_quantize<false>, grid, dim3(256), 0, st, (const void*)((const float*)x + i), inv, k, cols, nb,
                 (int)rows, codes + i / 2, scales + i / 32);
  }
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const void* packed, int64_t rows, int cols, void* out, int dt, hipStream_t st) {
  // a launch takes fewer than 2^32 threads: 2^31 words of 8 values each
  constexpr int64_t kWords = 1ll << 31;
  const int64_t words = rows * cols / 8;
  const uint8_t* codes = (const uint8_t*)packed;
  const uint8_t* scales = codes + rows * cols / 2;
  for (int64_t i = 0; i < words; i += kWords) {
    const int64_t n8 = std::min(words - i, kWords);
    const dim3 grid((unsigned)((n8 + 255) / 256));
    if (dt == DS4MOE_DT_BF16)
      DS4_LAUNCH(k_mx_dequantize<true>, grid, dim3(256), 0, st, codes + 4 * i, scales + i / 4, n8,
                 (void*)((uint16_t*)out + 8 * i));
    else
      DS4_LAUNCH(k_mx_dequantize<false>, grid, dim3(256), 0, st, codes + 4 * i, scales + i / 4, n8,
                 (void*)((float*)out + 8 * i));
  }
  return hipGetLastError();
}

}  // namespace ds4
