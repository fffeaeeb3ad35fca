// Gradient of the MXFP4 product to its rows: dA[p][c] = sum_r dY[p][r] W_e[r][c]
// for the rows p of expert e.
//
// The sum runs over the weights' rows, across which the block scales differ,
// so the block-scaled instruction does not apply: the weights become bfloat16
// (exact: two significant bits and a power of two) and v_mfma_f32_16x16x32_bf16
// multiplies them.  A bfloat16 dY goes in as it is; an fp32 dY is cut into
// three bfloat16 parts of 8 significant bits each, which hold it exactly
// (below 2^-110 to less than 2^-133, bfloat16's smallest number), and takes
// three instructions.  The sum is fp32.
//
// A block takes 256 columns and a tile of rows p.  A thread decodes 8 rows r
// by 8 columns, pairs neighbouring rows by byte permutation and writes, per
// column, 8 consecutive r as 16 bytes into LDS: the layout that the operands
// are read in.  16-byte pieces are XOR-swizzled so that both the writes (a
// column step of 8 between lanes) and the reads (16 neighbouring columns)
// spread over the banks.
//
// 2001 rows over 32 experts of 2048 x 4096: 95 us, 1.8 TB/s of the bytes that
// it needs (a copy moves 4.5) and 0.35 PFLOP/s; 85 us where a pass before left
// the weights in the last-level cache.  What bounds it is the chain
// of a step within a block (load, barrier, decode, barrier, products).  Tried
// and left: codes through LDS copies (98 us), the next step's decode beside
// the products of the same wave with one block to a CU (153 us), scale codes
// as words handed out by lane exchange (102 us where bytes take 90).
#include "../trace.h"
#include "ops.h"
#include "rowtile.h"
#include "../ring.h"

namespace ds4 {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr int kGradBN = 256;  // columns of a block
constexpr int kGradKC = 64;   // weight rows per step

__device__ inline float4_t mfma_bf16(u32x4_t a, u32x4_t b, float4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0,
                                                 0, 0);
}
// pieces of 16 bytes (8 r) of row i within the 128 bytes of a step
__device__ inline int swz_w(int c, int piece) { return c * 8 + (piece ^ (((c >> 1) ^ (c >> 3)) & 7)); }
__device__ inline int swz_a(int p, int piece) { return p * 8 + (piece ^ (p & 7)); }

// The 8 elements of a code word as four bfloat16 pairs.  The instruction takes
// the scale's exponent field as an E8M0 code: 0 is 2^-127, 255 NaN.
__device__ inline u32x4_t mx_bf16(uint32_t w, uint32_t sc) {
  const float s = __builtin_bit_cast(float, sc << 23);
  u32x4_t r;
  r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
  r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
  r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
  r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
  return r;
}

// The bfloat16 values of which x and y are the sum, by truncation (8 + 8 + 8
// bits; what lies under 2^-133 is lost), as three pairs.  An infinity or a NaN is its first part (a NaN made
// quiet before, so that its upper half says NaN), the others are zero.
__device__ inline void split3(float x, float y, uint32_t (&h)[3]) {
  x = __builtin_canonicalizef(x);
  y = __builtin_canonicalizef(y);
  const bool fx = fabsf(x) <= 3.402823466e38f, fy = fabsf(y) <= 3.402823466e38f;
#pragma unroll
  for (int s = 0; s < 3; ++s) {
    const uint32_t ux = __builtin_bit_cast(uint32_t, x), uy = __builtin_bit_cast(uint32_t, y);
    h[s] = __builtin_amdgcn_perm(uy, ux, 0x07060302u);
    if (s == 2) break;
    x -= __builtin_bit_cast(float, ux & 0xFFFF0000u);
    y -= __builtin_bit_cast(float, uy & 0xFFFF0000u);
    if (s == 0) {
      x = fx ? x : 0.f;
      y = fy ? y : 0.f;
    }
  }
}

// Bytes of LDS of a step: the weights, then the parts of the rows.
constexpr int grad_lds(int nf, int parts) { return kGradBN * 128 + parts * nf * 16 * 128; }

// One tile of up to 16 NF rows.  PARTS: 1 (bfloat16 dY) or 3 (fp32 dY).
// While a step is multiplied the next is on its way into registers, from
// which it is decoded into LDS once everyone is done.  One slot and more
// blocks to a CU hide a step's latency better than two slots (2001 rows over
// 32 experts: 96 us with three blocks, 100 with two blocks of two slots).
template <int NF, int PARTS, bool OB>
__device__ __attribute__((always_inline)) inline void grad_tile(const RowTile& rt, uint8_t* smem,
                                                                const void* __restrict__ dy,
                                                                const uint8_t* __restrict__ w, int rows, int cols,
                                                                void* __restrict__ out) {
  constexpr int BM = 16 * NF, AP = (BM * 8 + 255) / 256;  // 16-byte pieces of the rows per thread
  const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c0 = rt.part * kGradBN, rg = tid >> 5, cw = tid & 31;
  const int64_t mat = (int64_t)rows * cols / 32 * 17;
  const __amdgpu_buffer_rsrc_t wr = buf_rsrc(w + rt.e * mat, (uint32_t)mat);
  const uint32_t wo = (uint32_t)(8 * rg) * (cols / 2) + 4 * cw, so = (uint32_t)(8 * rg) * (cols / 32) + cw / 4;
  uint32_t cd[8], sc[8];
  Raw8<PARTS == 1> av[AP];
  auto load = [&](int r0) __attribute__((always_inline)) {
    // rows is a multiple of 16, so a thread's eight weight rows are all there
    // or none is; none reads as zeros
    const bool on = r0 + 8 * rg < rows;
    const uint32_t vo = on ? wo : kOob, vs = on ? so : kOob;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cd[i] = buf_ld32(wr, vo, (r0 + i) * (cols / 2) + c0 / 2);
      sc[i] = (uint32_t)__builtin_bit_cast(
          uint8_t, __builtin_amdgcn_raw_buffer_load_b8(wr, (int)vs, rows * (cols / 2) + (r0 + i) * (cols / 32) + c0 / 32, 0));
    }
#pragma unroll
    for (int i = 0; i < AP; ++i) {
      const int p = (tid + 256 * i) >> 3, r = r0 + 8 * (tid & 7);
      av[i] = Raw8<PARTS == 1>{};
      if (p < rt.cnt && r < rows) av[i] = ld8<PARTS == 1>(dy, (int64_t)(rt.lo + p) * rows + r);
    }
  };
  auto store = [&](uint8_t* slot) __attribute__((always_inline)) {
    u32x4_t* ws = (u32x4_t*)slot;
    u32x4_t* as = ws + kGradBN * 8;
    u32x4_t col[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const u32x4_t a = mx_bf16(cd[i], sc[i]), b = mx_bf16(cd[i + 1], sc[i + 1]);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        col[2 * p][i / 2] = __builtin_amdgcn_perm(b[p], a[p], 0x05040100u);
        col[2 * p + 1][i / 2] = __builtin_amdgcn_perm(b[p], a[p], 0x07060302u);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ws[swz_w(8 * cw + j, rg)] = col[j];
#pragma unroll
    for (int i = 0; i < AP; ++i) {
      const int p = (tid + 256 * i) >> 3, piece = tid & 7;
      if (p >= BM) break;
      if constexpr (PARTS == 1) {
        as[swz_a(p, piece)] = av[i].a;
      } else {
        float v[8];
        unpack8(av[i], v);
        u32x4_t o[3];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          uint32_t x[3];
          split3(v[e], v[e + 1], x);
#pragma unroll
          for (int s = 0; s < 3; ++s) o[s][e / 2] = x[s];
        }
#pragma unroll
        for (int s = 0; s < 3; ++s) as[s * BM * 8 + swz_a(p, piece)] = o[s];
      }
    }
  };
  float4_t acc[4][NF] = {};
  load(0);
  store(smem);
  ring_barrier();  // (orders LDS; loads into registers stay in flight)
#pragma unroll 1
  for (int r0 = 0; r0 < rows; r0 += kGradKC) {
    load(r0 + kGradKC);
    pin();
    const u32x4_t* ws = (const u32x4_t*)smem;
    const u32x4_t* as = ws + kGradBN * 8;
#pragma unroll
    for (int kk = 0; kk < kGradKC / 32; ++kk) {
      u32x4_t wf[4];
#pragma unroll
      for (int f = 0; f < 4; ++f) wf[f] = ws[swz_w(64 * wave + 16 * f + c, 4 * kk + q)];
#pragma unroll
      for (int s = PARTS - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NF; ++i) {
          const u32x4_t af = as[s * BM * 8 + swz_a(16 * i + c, 4 * kk + q)];
#pragma unroll
          for (int f = 0; f < 4; ++f) acc[f][i] = mfma_bf16(wf[f], af, acc[f][i]);
        }
    }
    pin();
    ring_barrier();  // everyone is done with the step
    store(smem);     // (zeros past the last one)
    ring_barrier();
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

template <int NF, int PARTS, bool OB>
__global__ __launch_bounds__(256, PARTS == 3 ? 2 : NF == 2 ? 4 : 3) void k_mx_grad(const void* __restrict__ dy, const uint8_t* __restrict__ w,
                                                    const int32_t* __restrict__ offsets, int n, int rows, int cols,
                                                    int E, void* __restrict__ out) {
  extern __shared__ uint8_t smem[];  // one slot: 36 KB (2, 1), 40 (4, 1) or 44 (2, 3)
  const RowTile rt = find_tile(offsets, E, n, 16 * NF, cols / kGradBN, (int*)smem);
  if (rt.cnt <= 0) return;
  __syncthreads();  // everyone has read the tile
  if (rt.cnt <= 16)
    grad_tile<1, PARTS, OB>(rt, smem, dy, w, rows, cols, out);
  else if (NF > 2 && rt.cnt <= 32)
    grad_tile<2, PARTS, OB>(rt, smem, dy, w, rows, cols, out);
  else
    grad_tile<NF, PARTS, OB>(rt, smem, dy, w, rows, cols, out);
}

template <int NF, int PARTS, bool OB>
static hipError_t launch_grad(const MxProduct& p) {
  const int64_t blocks = p.cols / kGradBN * max_tiles(p.n, p.E, p.offsets != nullptr, 16 * NF);
  DS4_LAUNCH((k_mx_grad<NF, PARTS, OB>), dim3((unsigned)blocks), dim3(256), grad_lds(NF, PARTS), p.st, p.dy, p.w,
             p.offsets, (int)p.n, p.rows, p.cols, p.E, p.out);
  return hipGetLastError();
}
// Tiles of 32 rows (36 KB, four blocks to a CU), or of 64 (40 KB, three; 32 or
// 16 where a tile has no more) so that a decoded weight serves twice as many:
// where an expert has rows for them on average, or where there are two rounds
// of them anyway.  2001 rows over 32 experts 88 / 94 us, 12288 rows over 256
// experts 273 / 245, 4000 rows of one 121 / 96.  fp32 dY: 32 rows (44 KB), 138
// us on the first; 16 or 64 take 167 and 182.
hipError_t launch_mx_product_grad(const MxProduct& p) {
  const bool ob = p.out_dt == DS4MOE_DT_BF16;
  if (p.dy_dt == DS4MOE_DT_F32) return ob ? launch_grad<2, 3, true>(p) : launch_grad<2, 3, false>(p);
  const int64_t E = p.offsets ? p.E : 1, blocks = (p.n / 64 + E / 2) * (p.cols / kGradBN);
  if (p.n < 128 * E && blocks <= 2 * 3 * 256) return ob ? launch_grad<2, 1, true>(p) : launch_grad<2, 1, false>(p);
  return ob ? launch_grad<4, 1, true>(p) : launch_grad<4, 1, false>(p);
}

}  // namespace ds4
