// Products of MXFP4 rows with the experts' MXFP4 weights on the block-scaled
// matrix instruction:
//
//   y[p][r] = sum_c A[p][c] W_e[r][c]        rows p of expert e
//   y[p][r] = silu(g) u                      g, u: the products with two matrices
//
// v_mfma_scale_f32_16x16x128_f8f6f4 (few rows) and _32x32x64_ (the rest) with
// both operands in FP4: a lane holds one row and one block of 32 columns of a
// step, 16 bytes, and the block's scale code in a byte of a register; the
// products and the scales are exact and the sum is fp32.  A row's scale codes
// are read as whole words, of which each lane shifts down the bytes of its
// blocks.  The weights are the first operand, so a lane ends with runs of four
// neighbouring outputs of one row.
//
// The lanes hold different rows side by side, and loads in that order move 15
// bytes a cycle and CU (hot in the L2), against 52 for copies into LDS with
// eight lanes to a row: so everything but a few rows goes through LDS, its 16
// byte pieces XOR-swizzled by row pair.
//
// Measured: 6 rows of 256 experts, gate and up, 53 MB in 11.5 us (4.6 TB/s);
// 12288 rows of 256 experts, down, 1.36 GB in 280 us (4.9 TB/s; a kernel that
// only reads as much takes 276); 4001 rows of one expert, gate and up 4096 x
// 4096, 75 to 81 us (3.3 to 3.6 PFLOP/s; the instruction alone reaches 8).
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

// g / (1 + e^-g) with the reciprocal instruction (within 2 steps of the
// quotient) and the fast exponential, whose argument is off by |g| half steps:
// (16 + |g|) half steps in all bound it.
__device__ inline float silu_rcp(float g) { return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

typedef float float16_t __attribute__((ext_vector_type(16)));

template <int SEL>
__device__ inline float16_t mfma_mx32(u32x4_t a, u32x4_t b, float16_t c, uint32_t sa, uint32_t sb) {
  const i32x8_t av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8_t bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, SEL, (int)sa, SEL, (int)sb);
}

// Bytes of LDS in which a wave turns 32 rows of NOW outputs.
template <int NOW, bool BF>
constexpr int turn_bytes() {
  return 32 * (NOW * (BF ? 2 : 4) + 16);
}
// Stores a wave's 32 rows (p0 onward of the tile) by 32 NF / (GLU ? 2 : 1)
// outputs (r0 onward): the accumulators leave four neighbouring outputs in a
// lane, so the wave turns them through its share of LDS and stores whole runs
// of each row.  GLU: the fragments' first half is gate, the second up.
template <int NF, bool GLU, bool BF>
__device__ __attribute__((always_inline)) inline void store_tile(const float16_t (&acc)[NF], uint8_t* turn,
                                                                 const RowTile& rt, int p0, int r0, int rows,
                                                                 int lane, void* y) {
  constexpr int NO = GLU ? NF / 2 : NF, ES = BF ? 2 : 4, RB = 32 * NO * ES, PITCH = RB + 16;
  const int c = lane & 31, h = lane >> 5;
#pragma unroll
  for (int f = 0; f < NO; ++f)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float4_t o;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        o[v] = acc[f][4 * g + v];
        if constexpr (GLU) o[v] = silu_rcp(o[v]) * acc[f + NO][4 * g + v];
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
    const int p = p0 + row, r = r0 + ch * (16 / ES);
    const u32x4_t v = *(const u32x4_t*)(turn + row * PITCH + ch * 16);
    if (p < rt.cnt && r < rows) *(u32x4_t*)((uint8_t*)y + ((int64_t)(rt.lo + p) * rows + r) * ES) = v;
  }
  __builtin_amdgcn_wave_barrier();
}

// ---------------------------------------------------------------- few rows
// A block takes 32 weight rows (GLU: 16 gate and the same 16 up) and a tile
// of up to 16 rows; its four waves each take a quarter of the columns, a
// piece of 256 at a time, and add up through LDS.  The weights pass through
// the wave's own LDS, two pieces in flight, because the lanes of the matrix
// instruction hold 16 different rows side by side and a load in that order
// moves 15 bytes a cycle against the copies' 52 (8 lanes to a row).  Their
// scales come four pieces at a time and wait in registers, so that the next
// four's copy has the same LDS again: 36 KB, four blocks to a CU.  The few
// rows themselves are loaded straight into registers.
constexpr int kRowsAhead = 2;                        // pieces in flight
constexpr int kRowsWave = kRowsAhead * 4096 + 1024;  // their codes, scales of four pieces
constexpr int kRowsBlocks = 4;                       // blocks to a CU
template <bool GLU, bool BF>
__global__ __launch_bounds__(256, kRowsBlocks) void k_mx_rows(const uint8_t* a, const uint8_t* __restrict__ w,
                                                              const uint8_t* __restrict__ w2,
                                                              const int32_t* __restrict__ offsets, int n, int rows,
                                                              int cols, int E, void* __restrict__ y) {
  constexpr int NO = GLU ? 16 : 32;
  // (sized at the launch: for an array of fixed size the compiler puts a wait
  // for the copies under way before reads that it cannot tell apart from them)
  extern __shared__ uint8_t smem[];
  __shared__ int lds[16];
  static_assert(kRowsBlocks * (sizeof(lds) + 4 * kRowsWave) <= 160 * 1024, "the CU's LDS");
  const RowTile rt = find_tile(offsets, E, n, 16, (rows + NO - 1) / NO, lds);
  if (rt.cnt <= 0) return;
  const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r0 = rt.part * NO;
  const int64_t mat = (int64_t)rows * cols / 32 * 17;
  const __amdgpu_buffer_rsrc_t wr[2] = {buf_rsrc(w + rt.e * mat, (uint32_t)mat),
                                        buf_rsrc((GLU ? w2 : w) + rt.e * mat, (uint32_t)mat)};
  const __amdgpu_buffer_rsrc_t ar = buf_rsrc(a + (int64_t)rt.lo * (cols / 2), (uint32_t)rt.cnt * (cols / 2));
  const __amdgpu_buffer_rsrc_t sr =
      buf_rsrc(a + (int64_t)n * (cols / 2) + (int64_t)rt.lo * (cols / 32), (uint32_t)rt.cnt * (cols / 32));
  // the wave's pieces: k0 .. k1 - 1
  const int pieces = cols / 256, k0 = pieces * wave / 4, k1 = pieces * (wave + 1) / 4;
  uint8_t* const wl = smem + wave * kRowsWave;
  const int prow = lane >> 3;
  // copies take 8 rows by 128 bytes, swizzled by row pair (rows 8 i + prow)
  auto copy_codes = [&](int k) __attribute__((always_inline)) {
    uint8_t* dst = wl + ((k - k0) & (kRowsAhead - 1)) * 4096;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = GLU && i >= 2, r = r0 + 8 * i - 16 * m;
      const uint32_t vo = (uint32_t)prow * (cols / 2) + (((lane & 7) ^ (4 * i + (prow >> 1))) & 7) * 16;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wr[m], (__attribute__((address_space(3))) void*)(dst + i * 1024), 16,
                                               k < k1 ? (int)vo : (int)kOob, r * (cols / 2) + k * 128, 0, 0);
    }
  };
  // scales of four pieces: 32 bytes of each of 32 rows, two lanes to a row
  uint8_t* const sl = wl + kRowsAhead * 4096;
  auto copy_scales = [&](int k) __attribute__((always_inline)) {
    const uint32_t vo = (uint32_t)((lane >> 1) & (GLU ? 15 : 31)) * (cols / 32) + (lane & 1) * 16;
    const uint32_t so = rows * (cols / 2) + r0 * (cols / 32) + k * 8;
    const int off = k < k1 ? (int)vo : (int)kOob;
    auto copy = [&](int m) __attribute__((always_inline)) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wr[m], (__attribute__((address_space(3))) void*)sl, 16, off, so, 0, 0);
    };
    if constexpr (GLU) {  // half of the lanes from each matrix; a copy fills what its active lanes name
      if (lane < 32) copy(0);
      asm volatile("" ::: "memory");  // (two copies, not one with a choice of matrix)
      if (lane >= 32) copy(1);
    } else {
      copy(0);
    }
  };
  u32x4_t A[kRowsAhead][2];
  u32x2_t AS[kRowsAhead];
  auto load_rows = [&](int k, int u) __attribute__((always_inline)) {  // rows past the tile's: zeros
    const bool on = c < rt.cnt && k < k1;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      A[u][j] = buf_ld128(ar, on ? (uint32_t)c * (cols / 2) + q * 16 + 64 * j : kOob, k * 128);
    AS[u] = buf_ld64(sr, on ? (uint32_t)c * (cols / 32) : kOob, k * 8);
  };
  constexpr int kCopies = 4 + 3;  // loads per piece
  float4_t acc[2] = {};
  // The waits below count loads in this order.  The fences keep it (and that a
  // is not __restrict__: loads of what nothing writes may pass them).
  auto fence = [] { asm volatile("" ::: "memory"); };
  copy_scales(k0);
#pragma unroll
  for (int u = 0; u < kRowsAhead; ++u) {
    pin();
    fence();
    copy_codes(k0 + u);
    load_rows(k0 + u, u);
  }
  fence();
#pragma unroll 1
  for (int kb = k0; kb < k1; kb += 4) {
    u32x4_t ws[2][2];  // scales of the group's pieces, two words a piece
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = kb + u, v = u % kRowsAhead;
      // past the last piece the rows are zeros and what LDS holds does not count
      pin();
      // Younger than piece k: the pieces ahead, and for the group's second piece
      // the next group's scales.  This group's are older than its first piece.
      if (u == 1) vm_wait<(kRowsAhead - 1) * kCopies + 1>();
      else vm_wait<(kRowsAhead - 1) * kCopies>();
      asm volatile("" ::: "memory");
      pin();
      u32x4_t wv[2][2];
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const int row = 16 * f + c;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          wv[f][j] = *(const u32x4_t*)(wl + v * 4096 + row * 128 + (((4 * j + q) ^ (row >> 1)) & 7) * 16);
        if (u == 0) {
#pragma unroll
          for (int j = 0; j < 2; ++j) ws[f][j] = *(const u32x4_t*)(sl + row * 32 + 16 * j);
        }
      }
      if (k < k1) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int f = 0; f < 2; ++f)
            acc[f] = mfma_mx(wv[f][j], A[v][j], acc[f], ws[f][u / 2][2 * (u & 1) + j] >> (8 * q), AS[v][j] >> (8 * q));
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slot (and the scales) have been read
      pin();
      if (u == 0) copy_scales(kb + 4);
      copy_codes(k + kRowsAhead);
      load_rows(k + kRowsAhead, v);
    }
  }
  vm_wait<0>();
  // sums of the four waves
  __syncthreads();
  float4_t(*red)[64][2] = (float4_t(*)[64][2])smem;
  if (wave > 0) {
#pragma unroll
    for (int f = 0; f < 2; ++f) red[wave - 1][lane][f] = acc[f];
  }
  __syncthreads();
  if (wave > 0 || c >= rt.cnt) return;
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int v = 0; v < 3; ++v) acc[f] += red[v][lane][f];
  const int64_t at = (int64_t)(rt.lo + c) * rows + r0 + 4 * q;
#pragma unroll
  for (int f = 0; f < (GLU ? 1 : 2); ++f) {
    if (r0 + 16 * f >= rows) continue;
    float4_t o = acc[f];
    if constexpr (GLU) {
#pragma unroll
      for (int v = 0; v < 4; ++v) o[v] = silu_rcp(o[v]) * acc[1][v];
    }
    if constexpr (BF)
      *(u32x2_t*)((uint16_t*)y + at + 16 * f) = u32x2_t{bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3])};
    else
      *(float4_t*)((float*)y + at + 16 * f) = o;
  }
}

// ---------------------------------------------------------------- many rows
// A block of four waves takes a tile of up to 64 NT rows and 128 weight rows
// (GLU: 64 gate and the same 64 up); a wave takes 64 of the weight rows (32
// of each) and half of the rows.  Both operands pass through LDS, a piece of
// 256 columns at a time with R pieces in the ring, and their scales two
// pieces at a time.
template <int NT>
constexpr int mid_slot() {
  return (128 + 64 * NT) * 128;
}
template <int NT>
constexpr int mid_scales() {
  return (128 + 64 * NT) * 16;
}
template <int NT, int R>
constexpr int mid_lds() {
  return R * mid_slot<NT>() + 2 * mid_scales<NT>() + 1024;
}
template <int NT, int R, bool GLU, bool BF>
__global__ __launch_bounds__(256, 2) void k_mx_mid(const uint8_t* __restrict__ a, const uint8_t* __restrict__ w,
                                                   const uint8_t* __restrict__ w2,
                                                   const int32_t* __restrict__ offsets, int n, int rows, int cols,
                                                   int E, void* __restrict__ y) {
  constexpr int BM = 64 * NT, NOB = GLU ? 64 : 128;
  extern __shared__ uint8_t smem[];
  __shared__ int lds[16];
  const RowTile rt = find_tile(offsets, E, n, BM, (rows + NOB - 1) / NOB, lds);
  if (rt.cnt <= 0) return;
  const int tid = threadIdx.x, lane = tid & 63, c = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave & 1, wn = wave >> 1;
  const int r0 = rt.part * NOB;
  const int64_t mat = (int64_t)rows * cols / 32 * 17;
  const __amdgpu_buffer_rsrc_t wr[2] = {buf_rsrc(w + rt.e * mat, (uint32_t)mat),
                                        buf_rsrc((GLU ? w2 : w) + rt.e * mat, (uint32_t)mat)};
  const __amdgpu_buffer_rsrc_t ar = buf_rsrc(a + (int64_t)rt.lo * (cols / 2), (uint32_t)rt.cnt * (cols / 2));
  const __amdgpu_buffer_rsrc_t sr =
      buf_rsrc(a + (int64_t)n * (cols / 2) + (int64_t)rt.lo * (cols / 32), (uint32_t)rt.cnt * (cols / 32));
  const int pieces = cols / 256;
  // copies of codes: row 32 i + tid / 8, swizzled by row pair
  const int prow = tid >> 3;
  const uint32_t cvo = (uint32_t)prow * (cols / 2) + ((tid ^ (prow >> 1)) & 7) * 16;
  // Copies of scales: waves 0 and 1 take the weights' 128 rows, the next NT
  // the rows' (64 lanes each); a wave without any reads nothing into a spare
  // KB, so that all waves count the same loads.
  uint8_t* const scales = smem + R * mid_slot<NT>();
  const bool up = GLU && wave == 1, of_w = wave < 2, idle = wave >= 2 + NT;
  const __amdgpu_buffer_rsrc_t scr = of_w ? wr[up] : sr;
  const uint32_t scv = idle ? kOob : (uint32_t)lane * (cols / 32);
  const uint32_t sco = of_w ? (uint32_t)rows * (cols / 2) + (uint32_t)(r0 + (!GLU && wave == 1 ? 64 : 0)) * (cols / 32)
                            : (uint32_t)(wave - 2) * 64 * (cols / 32);
  constexpr int kCopies = 4 + 2 * NT;
  auto issue = [&](int k, int u) __attribute__((always_inline)) {
    if (!(k & 1)) {
      uint8_t* dst = idle ? scales + 2 * mid_scales<NT>() : scales + ((k >> 1) & 1) * mid_scales<NT>() + wave * 1024;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(scr, (__attribute__((address_space(3))) void*)dst, 16, (int)scv,
                                               sco + k * 8, 0, 0);
    }
    uint8_t* dst = smem + u * mid_slot<NT>() + wave * 1024;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = GLU && i >= 2, r = r0 + 32 * i - 64 * m;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wr[m], (__attribute__((address_space(3))) void*)(dst + i * 4096), 16,
                                               (int)cvo, r * (cols / 2) + k * 128, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ar, (__attribute__((address_space(3))) void*)(dst + 16384 + i * 4096), 16,
                                               (int)cvo, 32 * i * (cols / 2) + k * 128, 0, 0);
  };
  auto wrow = [&](int f) __attribute__((always_inline)) { return GLU ? 64 * f + 32 * wm + c : 64 * wm + 32 * f + c; };
  const int arow = 32 * NT * wn + c;
  const bool none = 32 * NT * wn >= rt.cnt;  // no rows for this wave
  float16_t acc[2][NT] = {};
  auto compute = [&](int k, int u) __attribute__((always_inline)) {
    const uint8_t* slot = smem + u * mid_slot<NT>();
    const uint8_t* sc = scales + ((k >> 1) & 1) * mid_scales<NT>() + (k & 1) * 8;
    u32x2_t sw[2], sa[NT];
#pragma unroll
    for (int f = 0; f < 2; ++f) sw[f] = *(const u32x2_t*)(sc + wrow(f) * 16) >> (8 * h);
#pragma unroll
    for (int i = 0; i < NT; ++i) sa[i] = *(const u32x2_t*)(sc + 2048 + (arow + 32 * i) * 16) >> (8 * h);
    auto step = [&](auto J) __attribute__((always_inline)) {
      constexpr int j = decltype(J)::value;
      const int ph = ((2 * j + h) ^ ((c >> 1) & 7)) * 16;
      u32x4_t wv[2], av[NT];
#pragma unroll
      for (int f = 0; f < 2; ++f) wv[f] = *(const u32x4_t*)(slot + wrow(f) * 128 + ph);
#pragma unroll
      for (int i = 0; i < NT; ++i) av[i] = *(const u32x4_t*)(slot + 16384 + (arow + 32 * i) * 128 + ph);
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int f = 0; f < 2; ++f)
          acc[f][i] = mfma_mx32<(j & 1) * 2>(wv[f], av[i], acc[f][i], sw[f][j / 2], sa[i][j / 2]);
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
  };
  // At each step a wave waits for its own copies of the piece, the barrier
  // makes everyone's visible and shows that all waves are done with the piece
  // before, whose slot then takes the piece R - 1 ahead.
#pragma unroll
  for (int u = 0; u < R - 1; ++u)
    if (u < pieces) issue(u, u);
  int u = 0;
#pragma unroll 1
  for (int k = 0; k < pieces; ++k) {
    pin();
    if (k + R - 2 < pieces) vm_wait<(R - 2) * kCopies>();
    else vm_wait<0>();
    ring_barrier();
    pin();
    if (k + R - 1 < pieces) issue(k + R - 1, u == 0 ? R - 1 : u - 1);
    pin();
    if (!none) compute(k, u);
    u = u + 1 == R ? 0 : u + 1;
  }
  ring_barrier();
  constexpr int NOW = GLU ? 32 : 64;
  static_assert(4 * turn_bytes<NOW, BF>() <= mid_lds<NT, R>(), "the waves' shares fit");
  if (none) return;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    float16_t o[2] = {acc[0][i], acc[1][i]};
    store_tile<2, GLU, BF>(o, smem + wave * turn_bytes<NOW, BF>(), rt, 32 * NT * wn + 32 * i, r0 + wm * NOW, rows, lane, y);
  }
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

  constexpr int NOW = GLU ? 64 : 128;
  static_assert(4 * turn_bytes<NOW, BF>() <= kBigLds, "the waves' shares fit");
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float16_t o[4] = {acc[0][i], acc[1][i], acc[2][i], acc[3][i]};
    store_tile<4, GLU, BF>(o, smem + wave * turn_bytes<NOW, BF>(), rt, wn * 128 + 32 * i, r0 + wm * NOW, rows, lane, y);
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

template <bool GLU, bool BF>
static hipError_t launch_rows(const MxProduct& p) {
  const int no = GLU ? 16 : 32;
  const int64_t blocks = (p.rows + no - 1) / no * max_tiles(p.n, p.E, p.offsets != nullptr, 16);
  DS4_LAUNCH((k_mx_rows<GLU, BF>), dim3((unsigned)blocks), dim3(256), 4 * kRowsWave, p.st, p.a, p.w, p.w2, p.offsets,
             (int)p.n, p.rows, p.cols, p.E, p.out);
  return hipGetLastError();
}
template <int NT, int R, bool GLU, bool BF>
static hipError_t launch_mid(const MxProduct& p) {
  const int nob = GLU ? 64 : 128;
  const int64_t blocks = (p.rows + nob - 1) / nob * max_tiles(p.n, p.E, p.offsets != nullptr, 64 * NT);
  // (the number of rows as written, so that the timer's names tell the forms apart)
#define DS4_MID(nt)                                                                                                  \
  DS4_LAUNCH((k_mx_mid<nt, R, GLU, BF>), dim3((unsigned)blocks), dim3(256), (mid_lds<nt, R>()), p.st, p.a, p.w, p.w2, \
             p.offsets, (int)p.n, p.rows, p.cols, p.E, p.out)
  static_assert(NT == 1 || NT == 2, "64 or 128 rows");
  if constexpr (NT == 1) DS4_MID(1);
  else DS4_MID(2);
#undef DS4_MID
  return hipGetLastError();
}

// Which form: by the blocks that each would have (the experts' last, partly
// filled tiles counted as a half each) and the rows an expert has on average.
// Times of 4096 x 4096 weights on one expert, in us: rows / 64-row / 128-row /
// 256-row tiles.
//   few rows   while its blocks fit the chip at once (four on each of 256
//              CUs): 32 rows (256 blocks) 5.2 / 11.3, 96 rows (768) 9.7 / 11.6,
//              128 rows (1024) 11.8 / 11.7
//   256 rows   when its blocks, one to a CU, fill at least 3/4 of their last
//              round: 4096 rows (256 blocks) 63 / 50 / 40, 2000 rows (128
//              blocks) 32 / 26.6 / 32.5
//   128 rows   with rows to fill the tiles and more 64-row blocks than two to
//              a CU: 1500 rows 27.9 / 22.7, 600 rows (320 blocks) 14.6 / 15.7;
//              256 experts with 48 rows each 277 / 284
template <bool GLU, bool BF>
static hipError_t product(const MxProduct& p) {
  constexpr int kCus = 256;
  const int64_t E = p.offsets ? p.E : 1, mean = p.n / E;
  auto blocks = [&](int64_t outputs, int64_t bm) {
    return (p.rows + outputs - 1) / outputs * std::max<int64_t>(1, p.n / bm + (E > 1 ? E / 2 : p.n % bm != 0));
  };
  constexpr int g = GLU ? 2 : 1;  // weight rows per output
  if ((p.rows + 32 / g - 1) / (32 / g) * max_tiles(p.n, p.E, p.offsets != nullptr, 16) <= kRowsBlocks * kCus)
    return launch_rows<GLU, BF>(p);
  const int64_t big = blocks(kBig / g, kBig);
  if (mean >= 192 && 4 * big >= 3 * ((big + kCus - 1) / kCus * kCus)) return launch_big<GLU, BF>(p);
  if (mean >= 96 && blocks(128 / g, 64) > 2 * kCus) return launch_mid<2, 2, GLU, BF>(p);
  return launch_mid<1, 3, GLU, BF>(p);
}
hipError_t launch_mx_product(const MxProduct& p) {
  const bool b16 = p.out_dt == DS4MOE_DT_BF16;
  if (p.w2) return b16 ? product<true, true>(p) : product<true, false>(p);
  return b16 ? product<false, true>(p) : product<false, false>(p);
}

}  // namespace ds4
