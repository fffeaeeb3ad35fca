// Products of MXFP4 rows with the experts' MXFP4 weights on the block-scaled
// matrix instruction:
//
//   y[p][r] = sum_c A[p][c] W_e[r][c]        rows p of expert e
//   y[p][r] = silu(g) u                      g, u: the products with two matrices
//
// v_mfma_scale_f32_16x16x128_f8f6f4 with both operands in FP4: lane l holds
// row (l & 15) and one block of 32 along c per step, 16 bytes, and the
// block's scale code in one byte of a register; the products and the scales
// are exact and the sum is fp32.  Blocks are dealt to the steps so that
// lane group q = l >> 4 has the neighbouring blocks 4 q .. 4 q + 3 of 512
// columns in four steps (2 q, 2 q + 1 of 256 in two): 64 consecutive bytes of
// codes, and one word with the four scale codes that the steps select.
// The weights are the first operand, so a lane ends with four neighbouring
// outputs 4 q .. 4 q + 3 of one row p = l & 15.
#include <algorithm>

#include "../trace.h"
#include "ops.h"
#include "rowtile.h"

namespace ds4 {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// step J's scale code is byte J of sa and sb
template <int J>
__device__ inline float4_t mfma_mx(u32x4_t a, u32x4_t b, float4_t c, uint32_t sa, uint32_t sb) {
  const i32x8_t av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8_t bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, J, (int)sa, J, (int)sb);
}

// ---------------------------------------------------------------- few rows
// A block takes 16 outputs of a tile of up to 16 NT rows; its four waves each
// take every fourth piece of 512 columns and add up through LDS.
template <int NT, bool GLU, bool BF>
__global__ __launch_bounds__(256) void k_mx_rows(const uint8_t* __restrict__ a, const uint8_t* __restrict__ w,
                                                 const uint8_t* __restrict__ w2, const int32_t* __restrict__ offsets,
                                                 int n, int rows, int cols, int E, void* __restrict__ y) {
  constexpr int NM = GLU ? 2 : 1;
  __shared__ int lds[16];
  __shared__ float4_t red[3][64][NM * NT];
  const RowTile rt = find_tile(offsets, E, n, 16 * NT, blockIdx.x / (rows / 16), lds);
  if (rt.cnt <= 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, q = lane >> 4;
  const int r0 = blockIdx.x % (rows / 16) * 16;
  const int64_t wb = (int64_t)rt.e * ((int64_t)rows * cols / 32 * 17);
  const uint8_t* wc[NM];
  const uint8_t* ws[NM];
#pragma unroll
  for (int m = 0; m < NM; ++m) {
    const uint8_t* base = (m ? w2 : w) + wb;
    wc[m] = base + (int64_t)(r0 + c) * (cols / 2);
    ws[m] = base + (int64_t)rows * (cols / 2) + (int64_t)(r0 + c) * (cols / 32);
  }
  const uint8_t* ac[NT];
  const uint8_t* as[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int64_t p = rt.lo + min(16 * i + c, rt.cnt - 1);
    ac[i] = a + p * (cols / 2);
    as[i] = a + (int64_t)n * (cols / 2) + p * (cols / 32);
  }
  float4_t acc[NM][NT] = {};
  const int pieces = cols / 512;
  for (int k = wave; k < pieces; k += 4) {
    const int oc = k * 256 + q * 64, os = k * 16 + q * 4;
    u32x4_t wv[NM][4], av[NT][4];
    uint32_t wsc[NM], asc[NT];
#pragma unroll
    for (int m = 0; m < NM; ++m) {
#pragma unroll
      for (int j = 0; j < 4; ++j) wv[m][j] = *(const u32x4_t*)(wc[m] + oc + 16 * j);
      wsc[m] = *(const uint32_t*)(ws[m] + os);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) av[i][j] = *(const u32x4_t*)(ac[i] + oc + 16 * j);
      asc[i] = *(const uint32_t*)(as[i] + os);
    }
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        acc[m][i] = mfma_mx<0>(wv[m][0], av[i][0], acc[m][i], wsc[m], asc[i]);
        acc[m][i] = mfma_mx<1>(wv[m][1], av[i][1], acc[m][i], wsc[m], asc[i]);
        acc[m][i] = mfma_mx<2>(wv[m][2], av[i][2], acc[m][i], wsc[m], asc[i]);
        acc[m][i] = mfma_mx<3>(wv[m][3], av[i][3], acc[m][i], wsc[m], asc[i]);
      }
  }
  if (cols % 512 && wave == pieces % 4) {  // the last 256 columns
    const int oc = pieces * 256 + q * 32, os = pieces * 16 + q * 2;
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      const u32x4_t w0 = *(const u32x4_t*)(wc[m] + oc), w1 = *(const u32x4_t*)(wc[m] + oc + 16);
      const uint32_t sw = *(const uint16_t*)(ws[m] + os);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const u32x4_t a0 = *(const u32x4_t*)(ac[i] + oc), a1 = *(const u32x4_t*)(ac[i] + oc + 16);
        const uint32_t sa = *(const uint16_t*)(as[i] + os);
        acc[m][i] = mfma_mx<0>(w0, a0, acc[m][i], sw, sa);
        acc[m][i] = mfma_mx<1>(w1, a1, acc[m][i], sw, sa);
      }
    }
  }
  if (wave > 0) {
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int i = 0; i < NT; ++i) red[wave - 1][lane][m * NT + i] = acc[m][i];
  }
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int v = 0; v < 3; ++v) acc[m][i] += red[v][lane][m * NT + i];
    if (16 * i + c >= rt.cnt) continue;
    float4_t o = acc[0][i];
    if constexpr (GLU) {
#pragma unroll
      for (int v = 0; v < 4; ++v) o[v] = silu(o[v]) * acc[1][i][v];
    }
    const int64_t at = (int64_t)(rt.lo + 16 * i + c) * rows + r0 + 4 * q;
    if constexpr (BF)
      *(u32x2_t*)((uint16_t*)y + at) = u32x2_t{bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3])};
    else
      *(float4_t*)((float*)y + at) = o;
  }
}

hipError_t launch_mx_product(const MxProduct& p) {
  const bool glu = p.w2 != nullptr, b16 = p.out_dt == DS4MOE_DT_BF16;
  const int nt = p.n > 16 * (int64_t)p.E ? 4 : 1;
  const dim3 grid((unsigned)(p.rows / 16 * max_tiles(p.n, p.E, p.offsets != nullptr, 16 * nt)));
#define DS4_MXROWS(NT, GLU, BF)                                                                                      \
  DS4_LAUNCH((k_mx_rows<NT, GLU, BF>), grid, dim3(256), 0, p.st, p.a, p.w, p.w2, p.offsets, (int)p.n, p.rows, p.cols, \
             p.E, p.out)
#define DS4_MXROWS_T(NT)                   \
  do {                                     \
    if (glu && b16) DS4_MXROWS(NT, true, true);   \
    else if (glu) DS4_MXROWS(NT, true, false);    \
    else if (b16) DS4_MXROWS(NT, false, true);    \
    else DS4_MXROWS(NT, false, false);            \
  } while (0)
  if (nt == 4) DS4_MXROWS_T(4);
  else DS4_MXROWS_T(1);
  return hipGetLastError();
}

}  // namespace ds4
