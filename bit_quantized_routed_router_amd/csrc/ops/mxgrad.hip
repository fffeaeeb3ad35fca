// Gradient of the MXFP4 product to its rows: dA[p][c] = sum_r dY[p][r] W_e[r][c]
// for the rows p of expert e.
//
// The sum runs over the weights' rows, across which the block scales differ,
// so the block-scaled instruction does not apply: the weights become bfloat16
// (exact: two significant bits and a power of two) and v_mfma_f32_16x16x32_bf16
// multiplies them.  A bfloat16 dY goes in as it is; an fp32 dY is cut into
// three bfloat16 parts of 8 significant bits each, which hold it exactly, and
// takes three instructions.  The sum is fp32.
//
// A block takes 256 columns and a tile of rows p.  A thread decodes 8 rows r
// by 8 columns, pairs neighbouring rows by byte permutation and writes, per
// column, 8 consecutive r as 16 bytes into LDS: the layout that the operands
// are read in.  16-byte pieces are XOR-swizzled so that both the writes (a
// column step of 8 between lanes) and the reads (16 neighbouring columns)
// spread over the banks.
#include "../trace.h"
#include "ops.h"
#include "rowtile.h"

namespace ds4 {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr int kGradBN = 256;  // columns of a block
constexpr int kGradKC = 64;   // weight rows per step

__device__ inline float4_t mfma_bf16(u32x4_t a, u32x4_t b, float4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0,
                                                 0, 0);
}
// pieces of 16 bytes (8 r) of row i within the 128 bytes of a step
__device__ inline int swz_w(int c, int piece) { return c * 8 + (piece ^ ((c ^ (c >> 3)) & 7)); }
__device__ inline int swz_a(int p, int piece) { return p * 8 + (piece ^ (p & 7)); }

// the 8 elements of a code word as four bfloat16 pairs
__device__ inline u32x4_t mx_bf16(uint32_t w, uint32_t sc) {
  const float s = sc == 255u ? __builtin_nanf("") : __builtin_bit_cast(float, sc ? sc << 23 : 0x00400000u);
  u32x4_t r;
  r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
  r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
  r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
  r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
  return r;
}

// x = the sum of three bfloat16 values, by truncation: 8 + 8 + 8 bits
__device__ inline void split3(float x, uint32_t (&h)[3]) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  if ((u & 0x7F800000u) == 0x7F800000u) {  // infinity or NaN: one part holds it
    h[0] = (u & 0x7FFFFFu) ? (u | 0x00400000u) >> 16 : u >> 16;
    h[1] = h[2] = 0;
    return;
  }
  h[0] = u >> 16;
  const float r1 = x - __builtin_bit_cast(float, u & 0xFFFF0000u);
  const uint32_t u1 = __builtin_bit_cast(uint32_t, r1);
  h[1] = u1 >> 16;
  const float r2 = r1 - __builtin_bit_cast(float, u1 & 0xFFFF0000u);
  h[2] = __builtin_bit_cast(uint32_t, r2) >> 16;
}

// BM: rows of a tile (16 or 64); PARTS: 1 (bfloat16 dY) or 3 (fp32 dY)
template <int BM, int PARTS, bool OB>
__global__ __launch_bounds__(256) void k_mx_grad(const void* __restrict__ dy, const uint8_t* __restrict__ w,
                                                 const int32_t* __restrict__ offsets, int n, int rows, int cols,
                                                 int E, void* __restrict__ out) {
  constexpr int NF = BM / 16;
  __shared__ int lds[16];
  __shared__ u32x4_t ws[kGradBN * 8];
  __shared__ u32x4_t as[PARTS][BM * 8];
  const int nc = cols / kGradBN;
  const RowTile rt = find_tile(offsets, E, n, BM, nc, lds);
  if (rt.cnt <= 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = lane & 15, q = lane >> 4;
  const int c0 = rt.part * kGradBN;
  const int rg = tid >> 5, cw = tid & 31;
  const uint8_t* wb = w + (int64_t)rt.e * ((int64_t)rows * cols / 32 * 17);
  const uint8_t* wcode = wb + (c0 + 8 * cw) / 2;
  const uint8_t* wscale = wb + (int64_t)rows * (cols / 2) + (c0 + 8 * cw) / 32;
  float4_t acc[4][NF] = {};
  for (int r0 = 0; r0 < rows; r0 += kGradKC) {
    uint32_t cd[8], sc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // rows is a multiple of 16, so eight rows are all there or none is
      const int64_t r = min(r0 + 8 * rg, rows - 8) + i;
      cd[i] = *(const uint32_t*)(wcode + r * (cols / 2));
      sc[i] = wscale[r * (cols / 32)];
    }
    const bool past = r0 + 8 * rg >= rows;
    __syncthreads();  // the previous step's reads are done
    {
      u32x4_t col[8];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const u32x4_t a = mx_bf16(cd[i], sc[i]), b = mx_bf16(cd[i + 1], sc[i + 1]);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          col[2 * p][i / 2] = past ? 0u : __builtin_amdgcn_perm(b[p], a[p], 0x05040100u);
          col[2 * p + 1][i / 2] = past ? 0u : __builtin_amdgcn_perm(b[p], a[p], 0x07060302u);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ws[swz_w(8 * cw + j, rg)] = col[j];
    }
    for (int i = tid; i < BM * 8; i += 256) {
      const int p = i >> 3, piece = i & 7;
      const int r = r0 + 8 * piece;
      const int64_t at = (int64_t)(rt.lo + min(p, rt.cnt - 1)) * rows + r;
      if constexpr (PARTS == 1) {
        u32x4_t v = {0u, 0u, 0u, 0u};
        if (r < rows) v = *(const u32x4_t*)((const uint16_t*)dy + at);
        as[0][swz_a(p, piece)] = v;
      } else {
        float v[8] = {};
        if (r < rows) unpack8(ld8<false>(dy, at), v);
        u32x4_t o[3];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          uint32_t x[3], y[3];
          split3(v[e], x);
          split3(v[e + 1], y);
#pragma unroll
          for (int s = 0; s < 3; ++s) o[s][e / 2] = x[s] | (y[s] << 16);
        }
#pragma unroll
        for (int s = 0; s < 3; ++s) as[s][swz_a(p, piece)] = o[s];
      }
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < kGradKC / 32; ++kk) {
      u32x4_t wf[4];
#pragma unroll
      for (int f = 0; f < 4; ++f) wf[f] = ws[swz_w(64 * wave + 16 * f + c, 4 * kk + q)];
#pragma unroll
      for (int s = PARTS - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NF; ++i) {
          const u32x4_t af = as[s][swz_a(16 * i + c, 4 * kk + q)];
#pragma unroll
          for (int f = 0; f < 4; ++f) acc[f][i] = mfma_bf16(wf[f], af, acc[f][i]);
        }
    }
  }
#pragma unroll
  for (int i = 0; i < NF; ++i) {
    if (16 * i + c >= rt.cnt) continue;
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const int64_t at = (int64_t)(rt.lo + 16 * i + c) * cols + c0 + 64 * wave + 16 * f + 4 * q;
      const float4_t o = acc[f][i];
      if constexpr (OB)
        *(u32x2_t*)((uint16_t*)out + at) = u32x2_t{bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3])};
      else
        *(float4_t*)((float*)out + at) = o;
    }
  }
}

hipError_t launch_mx_product_grad(const MxProduct& p) {
  const bool f32 = p.dy_dt == DS4MOE_DT_F32, ob = p.out_dt == DS4MOE_DT_BF16;
  const int bm = p.n > 16 * (int64_t)p.E ? 64 : 16;
  const dim3 grid((unsigned)(p.cols / kGradBN * max_tiles(p.n, p.E, p.offsets != nullptr, bm)));
#define DS4_MXGRAD(BM, PARTS, OB)                                                                                 \
  DS4_LAUNCH((k_mx_grad<BM, PARTS, OB>), grid, dim3(256), 0, p.st, p.dy, p.w, p.offsets, (int)p.n, p.rows, p.cols, \
             p.E, p.out)
#define DS4_MXGRAD_T(BM)                      \
  do {                                        \
    if (f32 && ob) DS4_MXGRAD(BM, 3, true);   \
    else if (f32) DS4_MXGRAD(BM, 3, false);   \
    else if (ob) DS4_MXGRAD(BM, 1, true);     \
    else DS4_MXGRAD(BM, 1, false);            \
  } while (0)
  if (bm == 64) DS4_MXGRAD_T(64);
  else DS4_MXGRAD_T(16);
  return hipGetLastError();
}

}  // namespace ds4
