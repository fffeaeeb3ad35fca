// Products of MXFP4 rows with the experts' MXFP4 weights on the block-scaled
// matrix instruction:
//
//   y[p][r] = sum_c A[p][c] W_e[r][c]        rows p of expert e
//   y[p][r] = silu(g) u                      g, u: the products with two matrices
//
// v_mfma_scale_f32_16x16x128_f8f6f4 with both operands in FP4: lane l holds
// row (l & 15) and the block of 32 number q = l >> 4 of a step's 128 columns
// (16 bytes), and its scale code in the low byte of a register; the products
// and the scales are exact and the sum is fp32.  A step's loads cover 64
// consecutive bytes of each of 16 rows.  The scale codes of a row's four
// steps (512 columns, a piece) are read as four words, of which each lane
// shifts down the byte of its block.
// The weights are the first operand, so a lane ends with four neighbouring
// outputs 4 q .. 4 q + 3 of one row p = l & 15.
#include <algorithm>
#include <type_traits>

#include "../trace.h"
#include "ops.h"
#include "rowtile.h"
#include "../ring.h"

namespace ds4 {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

__device__ inline float4_t mfma_mx(u32x4_t a, u32x4_t b, float4_t c, uint32_t sa, uint32_t sb) {
  const i32x8_t av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8_t bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

// g / (1 + e^-g) with the reciprocal instruction: within 2 steps of the
// quotient, which the output's rounding or the sum's own error covers.
__device__ inline float silu_rcp(float g) { return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

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
  const RowTile rt = find_tile(offsets, E, n, 16 * NT, rows / 16, lds);
  if (rt.cnt <= 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, q = lane >> 4;
  const int r0 = rt.part * 16;
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
    const int oc = k * 256 + q * 16, os = k * 16;
    u32x4_t wv[NM][4], av[NT][4];
    u32x2_t wsc[NM][2], asc[NT][2];
#pragma unroll
    for (int m = 0; m < NM; ++m) {
#pragma unroll
      for (int j = 0; j < 4; ++j) wv[m][j] = *(const u32x4_t*)(wc[m] + oc + 64 * j);
#pragma unroll
      for (int j = 0; j < 2; ++j) wsc[m][j] = *(const u32x2_t*)(ws[m] + os + 8 * j);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) av[i][j] = *(const u32x4_t*)(ac[i] + oc + 64 * j);
#pragma unroll
      for (int j = 0; j < 2; ++j) asc[i][j] = *(const u32x2_t*)(as[i] + os + 8 * j);
    }
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[m][i] = mfma_mx(wv[m][j], av[i][j], acc[m][i], wsc[m][j / 2][j & 1] >> (8 * q), asc[i][j / 2][j & 1] >> (8 * q));
  }
  if (cols % 512 && wave == pieces % 4) {  // the last 256 columns
    const int oc = pieces * 256 + q * 16, os = pieces * 16;
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      const u32x2_t sw = *(const u32x2_t*)(ws[m] + os);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const u32x2_t sa = *(const u32x2_t*)(as[i] + os);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[m][i] = mfma_mx(*(const u32x4_t*)(wc[m] + oc + 64 * j), *(const u32x4_t*)(ac[i] + oc + 64 * j), acc[m][i],
                              sw[j] >> (8 * q), sa[j] >> (8 * q));
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
      for (int v = 0; v < 4; ++v) o[v] = silu_rcp(o[v]) * acc[1][i][v];
    }
    const int64_t at = (int64_t)(rt.lo + 16 * i + c) * rows + r0 + 4 * q;
    if constexpr (BF)
      *(u32x2_t*)((uint16_t*)y + at) = u32x2_t{bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3])};
    else
      *(float4_t*)((float*)y + at) = o;
  }
}

// ---------------------------------------------------------------- many rows
// A block of four waves takes a tile of up to 16 NT rows and 64 NW weight
// rows (GLU: half of them gate, half up, of the same outputs).  Each wave
// owns 16 NW weight rows, which come straight into its registers, and all of
// the tile's rows, which the block shares through LDS (copied there by
// buffer loads to LDS): a piece of 256 columns at a time, R pieces in the
// ring.  A row's 128 bytes of a piece are 8 pieces of 16 bytes, XOR-swizzled
// by row pair so that the 16 rows that a fragment reads cover all banks once.
template <int NT, int NW, int R, bool GLU, bool BF>
__device__ __attribute__((always_inline)) inline void mx_tile(const RowTile& rt, uint8_t* smem,
                                                              const uint8_t* __restrict__ a,
                                                              const uint8_t* __restrict__ w,
                                                              const uint8_t* __restrict__ w2, int n, int rows, int cols,
                                                              void* __restrict__ y) {
  constexpr int NO = GLU ? NW / 2 : NW;                // fragments of outputs per wave
  constexpr int CI = (NT + 1) / 2, SI = (NT + 7) / 8;  // copies of codes and scales per thread
  constexpr int kLoads = 3 * NW + CI + SI;             // vector loads per lane and piece
  constexpr int kSlot = CI * 4096 + SI * 1024;
  static_assert((R - 1) * kLoads <= 63, "ring depth");
  static_assert(!GLU || NW % 2 == 0, "gate and up fragments come in pairs");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = lane & 15, q = lane >> 4;
  const int r0 = rt.part * (64 * NO) + wave * (16 * NO);  // the wave's first output
  const int64_t mat = (int64_t)rows * cols / 32 * 17;
  // Offsets within a matrix or a tile of rows fit 32 bits.  Weight rows past
  // the last are read within the matrix, and past it the buffers give zeros;
  // they are not stored.
  const __amdgpu_buffer_rsrc_t wr[2] = {buf_rsrc(w + rt.e * mat, (uint32_t)mat),
                                        buf_rsrc((GLU ? w2 : w) + rt.e * mat, (uint32_t)mat)};
  const __amdgpu_buffer_rsrc_t ar = buf_rsrc(a + (int64_t)rt.lo * (cols / 2), (uint32_t)rt.cnt * (cols / 2));
  const __amdgpu_buffer_rsrc_t sr =
      buf_rsrc(a + (int64_t)n * (cols / 2) + (int64_t)rt.lo * (cols / 32), (uint32_t)rt.cnt * (cols / 32));
  const uint32_t wvo = (uint32_t)c * (cols / 2) + q * 16;
  const uint32_t wso = (uint32_t)rows * (cols / 2) + (uint32_t)c * (cols / 32);
  // copies: thread i of copy u fills 16-byte slot s = 256 u + i, which holds
  // piece (s ^ (row / 2)) & 7 of row s / 8; rows past the tile's read nothing
  const int prow = tid >> 3;
  const uint32_t avo = (uint32_t)prow * (cols / 2) + ((tid ^ (prow >> 1)) & 7) * 16;
  const uint32_t svo = (uint32_t)(tid >> 1) * (cols / 32) + (tid & 1) * 4;

  float4_t acc[NW][NT] = {};
  u32x4_t W[R][NW][2];
  u32x2_t S[R][NW];

  const int pieces = cols / 256;
  auto issue = [&](int k, int u) __attribute__((always_inline)) {
#pragma unroll
    for (int f = 0; f < NW; ++f) {
      const int r = r0 + 16 * (GLU ? f / 2 : f), m = GLU ? f & 1 : 0;
#pragma unroll
      for (int j = 0; j < 2; ++j) W[u][f][j] = buf_ld128(wr[m], wvo + 64 * j, r * (cols / 2) + k * 128);
      S[u][f] = buf_ld64(wr[m], wso, r * (cols / 32) + k * 8);
    }
    uint8_t* dst = smem + u * kSlot + wave * 1024;
#pragma unroll
    for (int i = 0; i < CI; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ar, (__attribute__((address_space(3))) void*)(dst + i * 4096), 16,
                                               (int)avo, i * 32 * (cols / 2) + k * 128, 0, 0);
    dst = smem + u * kSlot + CI * 4096 + wave * 256;
#pragma unroll
    for (int i = 0; i < SI; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(sr, (__attribute__((address_space(3))) void*)(dst + i * 1024), 4,
                                               (int)svo, i * 128 * (cols / 32) + k * 8, 0, 0);
  };
  auto compute = [&](int u) __attribute__((always_inline)) {
    const uint8_t* src = smem + u * kSlot;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const uint8_t* rp = src + (16 * i + c) * 128;
      const u32x2_t sa = *(const u32x2_t*)(src + CI * 4096 + (16 * i + c) * 8);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const u32x4_t av = *(const u32x4_t*)(rp + (((4 * j + q) ^ (c >> 1)) * 16));
        const uint32_t sj = sa[j] >> (8 * q);
#pragma unroll
        for (int f = 0; f < NW; ++f) acc[f][i] = mfma_mx(W[u][f][j], av, acc[f][i], S[u][f][j] >> (8 * q), sj);
      }
    }
  };
  // At each step a wave waits for its own loads of the piece, the barrier
  // makes everyone's copies visible and shows that all waves are done with
  // the piece before, whose slot then takes the piece R - 1 ahead.
#pragma unroll
  for (int u = 0; u < R - 1; ++u)
    if (u < pieces) issue(u, u);
  for (int k0 = 0; k0 < pieces; k0 += R) {
#pragma unroll
    for (int u = 0; u < R; ++u) {
      const int k = k0 + u;
      if (k >= pieces) break;
      pin();
      if (k + R - 2 < pieces) vm_wait<(R - 2) * kLoads>();
      else vm_wait<0>();
      ring_barrier();
      pin();
      if (k + R - 1 < pieces) issue(k + R - 1, (u + R - 1) % R);
      pin();
      compute(u);
    }
  }

#pragma unroll
  for (int i = 0; i < NT; ++i) {
    if (16 * i + c >= rt.cnt) continue;
    const int64_t at = (int64_t)(rt.lo + 16 * i + c) * rows;
#pragma unroll
    for (int f = 0; f < NO; ++f) {
      const int r = r0 + 16 * f + 4 * q;
      if (r >= rows) continue;
      float4_t o = acc[GLU ? 2 * f : f][i];
      if constexpr (GLU) {
#pragma unroll
        for (int v = 0; v < 4; ++v) o[v] = silu_rcp(o[v]) * acc[2 * f + 1][i][v];
      }
      if constexpr (BF)
        *(u32x2_t*)((uint16_t*)y + at + r) = u32x2_t{bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3])};
      else
        *(float4_t*)((float*)y + at + r) = o;
    }
  }
}

// Rings are as deep as the registers and LDS of the block's largest form allow.
constexpr size_t ring_bytes(int nt, int r) { return (size_t)r * ((nt + 1) / 2 * 4096 + (nt + 7) / 8 * 1024); }

template <int NT, int NW, int R, bool GLU, bool BF, int WPE>
__global__ __launch_bounds__(256, WPE) void k_mx_tiles(const uint8_t* __restrict__ a, const uint8_t* __restrict__ w,
                                                       const uint8_t* __restrict__ w2,
                                                       const int32_t* __restrict__ offsets, int n, int rows, int cols,
                                                       int E, void* __restrict__ y) {
  constexpr int NO = GLU ? NW / 2 : NW;
  extern __shared__ uint8_t smem[];
  __shared__ int lds[16];
  const RowTile rt = find_tile(offsets, E, n, 16 * NT, (rows + 64 * NO - 1) / (64 * NO), lds);
  if (rt.cnt <= 0) return;
  if (NT == 4 && rt.cnt <= 16)
    mx_tile<1, NW, R, GLU, BF>(rt, smem, a, w, w2, n, rows, cols, y);
  else if (NT == 4 && rt.cnt <= 32)
    mx_tile<2, NW, R, GLU, BF>(rt, smem, a, w, w2, n, rows, cols, y);
  else
    mx_tile<NT, NW, R, GLU, BF>(rt, smem, a, w, w2, n, rows, cols, y);
}

template <int NT, int NW, int R, bool GLU, bool BF, int WPE>
static hipError_t launch_tiles(const MxProduct& p) {
  constexpr int no = GLU ? NW / 2 : NW;
  constexpr size_t shmem = ring_bytes(NT, R);
  const int64_t parts = (p.rows + 64 * no - 1) / (64 * no);
  const int64_t blocks = parts * max_tiles(p.n, p.E, p.offsets != nullptr, 16 * NT);
  DS4_LAUNCH((k_mx_tiles<NT, NW, R, GLU, BF, WPE>), dim3((unsigned)blocks), dim3(256), shmem, p.st, p.a, p.w, p.w2,
             p.offsets, (int)p.n, p.rows, p.cols, p.E, p.out);
  return hipGetLastError();
}
template <int NT, int NW, int R, int WPE>
static hipError_t tiles(const MxProduct& p) {
  const bool b16 = p.out_dt == DS4MOE_DT_BF16;
  if (p.w2) return b16 ? launch_tiles<NT, NW, R, true, true, WPE>(p) : launch_tiles<NT, NW, R, true, false, WPE>(p);
  return b16 ? launch_tiles<NT, NW, R, false, true, WPE>(p) : launch_tiles<NT, NW, R, false, false, WPE>(p);
}

// ---------------------------------------------------------------- large tiles
// A block of four waves takes 256 rows by 256 weight rows (GLU: 128 gate and
// the same 128 up), each wave 128 by 128 of them as 4 x 4 tiles of
// v_mfma_scale_f32_32x32x64_f8f6f4: lane l holds row (l & 31) and block
// h = l >> 5 of a step's 64 columns.  Both operands go through LDS, a piece
// of 256 columns at a time and two pieces in turn.  The tile is this large
// because FP4 products outrun what feeds them: per 256 columns it loads 68 KB
// for 2048 cycles of products (33 of a CU's 64 bytes a cycle from the L2),
// and its fragment reads take half of the LDS rate.
typedef float float16_t __attribute__((ext_vector_type(16)));

template <int SEL>
__device__ inline float16_t mfma_mx32(u32x4_t a, u32x4_t b, float16_t c, uint32_t sa, uint32_t sb) {
  const i32x8_t av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8_t bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, SEL, (int)sa, SEL, (int)sb);
}

constexpr int kBig = 256;                        // rows, and weight rows, of a block
constexpr int kBigSlot = 2 * kBig * 128;         // bytes of a piece's codes of both
constexpr int kBigScales = 2 * kBig * 16;        // bytes of the scales of two pieces
constexpr int kBigLds = 2 * (kBigSlot + kBigScales);
template <bool GLU, bool BF>
__global__ __launch_bounds__(256, 1) void k_mx_big(const uint8_t* __restrict__ a, const uint8_t* __restrict__ w,
                                                   const uint8_t* __restrict__ w2,
                                                   const int32_t* __restrict__ offsets, int n, int rows, int cols,
                                                   int E, void* __restrict__ y) {
  constexpr int NOB = GLU ? kBig / 2 : kBig;  // outputs of a block
  // codes of 256 weight rows and 256 rows, two pieces; scales of both, two pairs of pieces
  extern __shared__ uint8_t smem[];
  __shared__ int lds[16];
  const RowTile rt = find_tile(offsets, E, n, kBig, (rows + NOB - 1) / NOB, lds);
  if (rt.cnt <= 0) return;
  const int tid = threadIdx.x, lane = tid & 63, c = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave & 1, wn = wave >> 1;  // the wave's half of the weight rows and of the rows
  const int r0 = rt.part * NOB;
  const int64_t mat = (int64_t)rows * cols / 32 * 17;
  const __amdgpu_buffer_rsrc_t wr[2] = {buf_rsrc(w + rt.e * mat, (uint32_t)mat),
                                        buf_rsrc((GLU ? w2 : w) + rt.e * mat, (uint32_t)mat)};
  const __amdgpu_buffer_rsrc_t ar = buf_rsrc(a + (int64_t)rt.lo * (cols / 2), (uint32_t)rt.cnt * (cols / 2));
  const __amdgpu_buffer_rsrc_t sr =
      buf_rsrc(a + (int64_t)n * (cols / 2) + (int64_t)rt.lo * (cols / 32), (uint32_t)rt.cnt * (cols / 32));
  // copy i of a thread: row 32 i + tid / 8 of an operand, swizzled by row pair
  const int prow = tid >> 3;
  const uint32_t cvo = (uint32_t)prow * (cols / 2) + ((tid ^ (prow >> 1)) & 7) * 16;
  // scale copies: a thread takes a row's 16 bytes
  const uint32_t svo = (uint32_t)tid * (cols / 32);
  const bool up = GLU && wave >= 2;
  const __amdgpu_buffer_rsrc_t wsr = wr[up];
  const uint32_t wso = (uint32_t)rows * (cols / 2) + (uint32_t)(r0 - (up ? kBig / 2 : 0)) * (cols / 32);
  auto copy16 = [&](__amdgpu_buffer_rsrc_t r, uint8_t* dst, uint32_t vo, uint32_t so) __attribute__((always_inline)) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)(dst + wave * 1024), 16,
                                             (int)vo, (int)so, 0, 0);
  };
  // Copy i of piece k's kCopies: codes of the weights, of the rows, and the
  // scales of a pair of pieces: those of the weights with its first piece,
  // those of the rows with the piece before it.  Past the last piece a copy
  // reads nothing, so that the loop below has no branches and its order of
  // reads, copies and products stays as written.
  constexpr int kCopies = 17;
  const int pieces = cols / 256;
  uint8_t* const scales = smem + 2 * kBigSlot;
  auto issue_scales = [&](int k) __attribute__((always_inline)) {  // with piece k
    const bool of_rows = k & 1;
    const int pair = (k + 1) >> 1;
    copy16(of_rows ? sr : wsr, scales + (pair & 1) * kBigScales + (of_rows ? kBigScales / 2 : 0),
           2 * pair < pieces ? svo : kOob, (of_rows ? 0 : wso) + pair * 16);
  };
  auto issue = [&](int k, int i) __attribute__((always_inline)) {
    uint8_t* dst = smem + (k & 1) * kBigSlot;
    const uint32_t co = k < pieces ? cvo : kOob;
    if (i < 8) {
      const int m = GLU && i >= 4, r = r0 + 32 * i - m * (kBig / 2);
      copy16(wr[m], dst + i * 4096, co, r * (cols / 2) + k * 128);
    } else {
      copy16(ar, dst + i * 4096, co, 32 * (i - 8) * (cols / 2) + k * 128);
    }
  };
  // the wave's weight fragment f: rows of the piece in LDS
  auto wrow = [&](int f) __attribute__((always_inline)) {
    return GLU ? (f >> 1) * 128 + wm * 64 + (f & 1) * 32 + c : wm * 128 + f * 32 + c;
  };
  // The fragments of a step are read while the products of the step before
  // run, across pieces too: the barrier and the first reads of the next piece
  // come before the last step's products.
  struct Frags {
    u32x4_t w[4], a[4];
  };
  struct Scales {  // word i, byte 0 and 2: steps 2 i and 2 i + 1
    u32x2_t w[4], a[4];
  };
  auto read = [&](Frags& F, const uint8_t* slot, int j) __attribute__((always_inline)) {
    const int ph = ((2 * j + h) ^ ((c >> 1) & 7)) * 16;  // fragments are multiples of 32 rows apart
#pragma unroll
    for (int f = 0; f < 4; ++f) F.w[f] = *(const u32x4_t*)(slot + wrow(f) * 128 + ph);
#pragma unroll
    for (int i = 0; i < 4; ++i) F.a[i] = *(const u32x4_t*)(slot + 32768 + (wn * 128 + 32 * i + c) * 128 + ph);
  };
  auto read_scales = [&](Scales& S, int k) __attribute__((always_inline)) {
    const uint8_t* sc = scales + ((k >> 1) & 1) * kBigScales + (k & 1) * 8;
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      S.w[f] = *(const u32x2_t*)(sc + wrow(f) * 16) >> (8 * h);
      S.a[f] = *(const u32x2_t*)(sc + kBigScales / 2 + (wn * 128 + 32 * f + c) * 16) >> (8 * h);
    }
  };
  float16_t acc[4][4] = {};
  // A step's 16 products, with copies first .. last - 1 of piece k issued
  // between them: issued in one run, the copies would hold up the products
  // behind them while the address unit works them off.
  auto products = [&](const Frags& F, const Scales& S, auto J, int k, int first, int last) __attribute__((always_inline)) {
    constexpr int j = decltype(J)::value;
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      const int i = x / 4, f = x % 4;
      acc[f][i] = mfma_mx32<(j & 1) * 2>(F.w[f], F.a[i], acc[f][i], S.w[f][j / 2], S.a[i][j / 2]);
      if (first + x < last) {
        pin();
        issue(k, first + x);
        pin();
      }
    }
  };
  Frags F0, F1;
  Scales S;
#pragma unroll
  for (int i = 0; i < 16; ++i) issue(0, i);
  issue_scales(-1);
  issue_scales(0);
  vm_wait<0>();
  ring_barrier();
  read(F0, smem, 0);
  read_scales(S, 0);
  issue_scales(1);
#pragma unroll
  for (int i = 0; i < kCopies / 2; ++i) issue(1, i);
#pragma unroll 1
  for (int k = 0; k < pieces; ++k) {
    const uint8_t* slot = smem + (k & 1) * kBigSlot;
    const uint8_t* next = smem + ((k + 1) & 1) * kBigSlot;
    pin();
    read(F1, slot, 1);
    pin();
    products(F0, S, std::integral_constant<int, 0>{}, k + 1, kCopies / 2, 16);
    pin();
    read(F0, slot, 2);
    pin();
    products(F1, S, std::integral_constant<int, 1>{}, k, 0, 0);
    pin();
    read(F1, slot, 3);
    pin();
    products(F0, S, std::integral_constant<int, 2>{}, k, 0, 0);
    pin();
    const Scales T = S;
    vm_wait<0>();    // this wave's copies of the next piece
    ring_barrier();  // everyone's, and everyone has read this piece
    pin();
    read(F0, next, 0);  // (not used after the last piece)
    read_scales(S, k + 1);
    pin();
    issue_scales(k + 2);
    products(F1, T, std::integral_constant<int, 3>{}, k + 2, 0, kCopies / 2);
  }
  vm_wait<0>();
  ring_barrier();

  // A wave turns 32 rows of its outputs at a time through its share of LDS,
  // so that they leave as whole runs of a row.
  constexpr int NOW = GLU ? 64 : 128, ES = BF ? 2 : 4;  // outputs of a wave, bytes of one
  constexpr int RB = NOW * ES, PITCH = RB + 16;
  uint8_t* turn = smem + wave * (32 * PITCH);
  static_assert(4 * 32 * PITCH <= kBigLds, "the waves' shares fit");
  const int rw = r0 + wm * NOW;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int f = 0; f < NOW / 32; ++f)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float4_t o;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          o[v] = acc[f][i][4 * g + v];
          if constexpr (GLU) o[v] = silu_rcp(o[v]) * acc[f + 2][i][4 * g + v];
        }
        uint8_t* at = turn + c * PITCH + (32 * f + 8 * g + 4 * h) * ES;
        if constexpr (BF)
          *(u32x2_t*)at = u32x2_t{bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3])};
        else
          *(float4_t*)at = o;
      }
    __builtin_amdgcn_wave_barrier();
    constexpr int LPR = RB / 16;  // lanes of a row
#pragma unroll
    for (int x = 0; x < 32 * LPR / 64; ++x) {
      const int row = x * (64 / LPR) + lane / LPR, ch = lane % LPR;
      const int p = wn * 128 + 32 * i + row, r = rw + ch * (16 / ES);
      const u32x4_t v = *(const u32x4_t*)(turn + row * PITCH + ch * 16);
      if (p < rt.cnt && r < rows) *(u32x4_t*)((uint8_t*)y + ((int64_t)(rt.lo + p) * rows + r) * ES) = v;
    }
    __builtin_amdgcn_wave_barrier();
  }
}

template <bool GLU, bool BF>
static hipError_t launch_big(const MxProduct& p) {
  const int nob = GLU ? kBig / 2 : kBig;
  const int64_t blocks = (p.rows + nob - 1) / nob * max_tiles(p.n, p.E, p.offsets != nullptr, kBig);
  DS4_LAUNCH((k_mx_big<GLU, BF>), dim3((unsigned)blocks), dim3(256), kBigLds, p.st, p.a, p.w, p.w2, p.offsets,
             (int)p.n, p.rows, p.cols, p.E, p.out);
  return hipGetLastError();
}

hipError_t launch_mx_product(const MxProduct& p) {
  if (p.n >= 256 * (int64_t)p.E) {
    if (p.w2) return p.out_dt == DS4MOE_DT_BF16 ? launch_big<true, true>(p) : launch_big<true, false>(p);
    return p.out_dt == DS4MOE_DT_BF16 ? launch_big<false, true>(p) : launch_big<false, false>(p);
  }
  if (p.n > 16 * (int64_t)p.E) return tiles<4, 2, 3, 2>(p);
  const bool glu = p.w2 != nullptr, b16 = p.out_dt == DS4MOE_DT_BF16;
  const dim3 grid((unsigned)(p.rows / 16 * max_tiles(p.n, p.E, p.offsets != nullptr, 16)));
#define DS4_MXROWS(NT, GLU, BF)                                                                                      \
  DS4_LAUNCH((k_mx_rows<NT, GLU, BF>), grid, dim3(256), 0, p.st, p.a, p.w, p.w2, p.offsets, (int)p.n, p.rows, p.cols, \
             p.E, p.out)
  if (glu && b16) DS4_MXROWS(1, true, true);
  else if (glu) DS4_MXROWS(1, true, false);
  else if (b16) DS4_MXROWS(1, false, true);
  else DS4_MXROWS(1, false, false);
  return hipGetLastError();
}

}  // namespace ds4
