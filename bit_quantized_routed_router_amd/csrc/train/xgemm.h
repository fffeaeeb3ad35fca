// The products of the cross entropy on v_mfma_f32_32x32x16_bf16:
//
//   acc[a][b] = sum_k A[a][k] B[b][k]
//
// over tiles of BM a's by BN b's, four waves, both operands through LDS a
// chunk of 64 k at a time with R chunks in the ring.  An operand lies in
// memory either by rows (k contiguous: 128 bytes of a row per chunk) or by
// columns (its own index contiguous: 64 rows of the tile's width per chunk,
// turned by the transposing LDS read).  fp32 operands come as three bfloat16
// planes whose sum they are, and a chunk is multiplied six times: hi hi, hi
// mid, mid hi, mid mid, hi lo, lo hi.  What is left out (mid lo, lo mid, lo lo)
// is within 2^-24 of the product, fp32's own rounding, and of either sign,
// since each plane is what is left rounded to nearest.  For few rows, where
// reading the operands is what takes time, they stay fp32 and go through
// v_mfma_f32_32x32x2_f32, 32 k a chunk: lane l's four values of a 16-byte piece
// take four products, in which the two halves of the wave hold k's four apart
// in both operands.
//
// Measured, 4096 rows x 65536 words x 4096 in bf16: 1.62 to 1.70 ms for the forward
// pass's product (1.30 to 1.36 PFLOP/s; a library's product alone 1.48 ms),
// 0.82 to 0.88 ms for each of its halves' ds, dw and dh.  The matrix unit is busy
// 78 % of the cycles in the forward product, 74 in ds and dw, 81 in dh, at the
// 1.65 GHz or so that the card holds under this load.
//
// LDS: 16-byte pieces, swizzled on their way in by choosing which piece a
// lane copies.  By rows piece p of row r lies at p ^ (r / 2 & 7), so that the
// 16 rows that a quarter of a wave reads lie in different banks; by columns
// piece p of row k lies at p ^ 4 (k & 3) (as far as its row has pieces), since
// half a wave reads four neighbouring pieces of four rows; in fp32 at
// p ^ 8 (k / 4 & 1), since its halves read eight pieces of rows four apart.
#pragma once

#include "../ring.h"
#include "train.h"

namespace ds4 {

typedef float float16_t __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));

__device__ inline float16_t mfma32(u32x4_t a, u32x4_t b, float16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0,
                                                 0, 0);
}

__device__ inline float16_t mfma32_f32(u32x4_t a, u32x4_t b, float16_t c) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t x = a[e], y = b[e];
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__builtin_bit_cast(float, x), __builtin_bit_cast(float, y), c, 0, 0, 0);
  }
  return c;
}

// The transposing read.  The argument's __restrict__ is what the compiler knows
// about the read: without it, it would wait for every copy under way before.
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;
__device__ __attribute__((always_inline)) inline u32x2_t read_turned(lds_s16x4_t* __restrict__ p) {
  return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p));
}

// waves along a and b, 32x32 fragments of a wave along both, chunks in the ring
template <int WM_, int WN_, int FM_, int FN_, int R_>
struct XShape {
  static constexpr int WM = WM_, WN = WN_, FM = FM_, FN = FN_, R = R_;
  static constexpr int BM = 32 * WM * FM, BN = 32 * WN * FN;
  static constexpr int slot = (BM + BN) * 128, lds = FM * FN == 16 ? 160 * 1024 : R * slot;
  static constexpr int copies = (BM + BN) / 32;  // a thread's copies per chunk
  static_assert(WM * WN == 4 && lds <= 160 * 1024 && (R - 2) * copies < 64, "four waves, LDS, copies in flight");
};

struct XOperand {
  const uint8_t* p;
  int64_t plane;  // bytes from one bfloat16 plane to the next
  int64_t pitch;  // bytes of a row (a k of an operand by columns); 256 of them below 2^31
};

// One operand's side of a tile of B indices, from index i0 on.
template <int B, bool COL, bool F32>
struct XSide {
  static constexpr int ES = F32 ? 4 : 2, KC = 128 / ES;  // bytes of a value, k of a chunk
  static constexpr int RB = B * ES, P = RB / 16;         // by columns: bytes and pieces of a k
  static constexpr int kStep = COL ? 4096 / RB : 32;     // rows from one copy to the next
  static_assert(!COL || !F32 || kStep % 8 == 0, "the swizzle of a thread's copies is one");
  const uint8_t* base;
  int64_t plane, pitch;
  uint32_t records;  // by rows: bytes that the tile has; by columns: what a row's end leaves out
  uint32_t vo;       // the lane's piece
  static __device__ inline int swizzle(int k) { return (F32 ? 8 * (k >> 2 & 1) : 4 * (k & 3)) & (P - 1); }
  __device__ inline void init(const XOperand& o, int64_t i0, int64_t rows, int tid) {
    plane = o.plane;
    pitch = o.pitch;
    if constexpr (!COL) {
      base = o.p + i0 * pitch;
      records = (uint32_t)((rows - i0 < B ? rows - i0 : B) * pitch);
      const int r = tid >> 3;
      vo = (uint32_t)(r * pitch) + ((tid ^ (r >> 1)) & 7) * 16;
    } else {
      base = o.p + i0 * ES;
      records = (uint32_t)i0 * ES;
      const int k = tid / P, p = tid % P;
      vo = (uint32_t)(k * pitch) + (p ^ swizzle(k)) * 16;
    }
  }
  // chunk kc of plane q; K: how many k there are
  __device__ __attribute__((always_inline)) inline __amdgpu_buffer_rsrc_t chunk(int kc, int q, int64_t K) const {
    const uint8_t* src = base + q * plane;
    if constexpr (!COL) {
      return buf_rsrc(src + (int64_t)kc * 128, kc * 128 < (int)records ? records - kc * 128 : 0);
    } else {
      const int64_t left = K - (int64_t)kc * KC;
      return buf_rsrc(src + (int64_t)kc * KC * pitch, left > 0 ? (uint32_t)((left < KC ? left : KC) * pitch) - records : 0);
    }
  }
  // copy i of the thread (B / 32 in all), of a chunk that lies at dst
  __device__ __attribute__((always_inline)) inline void copy(__amdgpu_buffer_rsrc_t r, bool on, int i, uint8_t* dst,
                                                             int wave) const {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)(dst + i * 4096 + wave * 1024),
                                             16, on ? (int)vo : (int)kOob, (int)(i * kStep * pitch), 0, 0);
  }
  // Fragment f (32 indices from first on) of step j, a quarter of the chunk:
  // lane l gets index l & 31 and k 8 (l >> 5) .. + 7 of the step's 16; in fp32
  // k 4 (l >> 5) .. + 3 of its 8.
  static __device__ __attribute__((always_inline)) inline u32x4_t read(const uint8_t* at, int first, int f, int j,
                                                                       int lane) {
    if constexpr (!COL) {
      const int c = lane & 31, h = lane >> 5;
      return *(const u32x4_t*)(at + (first + 32 * f + c) * 128 + (((2 * j + h) ^ (c >> 1)) & 7) * 16);
    } else if constexpr (F32) {
      const int c = lane & 31, h = lane >> 5, piece = (first / 4 + 8 * f + (c >> 2)) ^ swizzle(4 * h);
      u32x4_t v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = *(const uint32_t*)(at + (8 * j + 4 * h + e) * RB + piece * 16 + 4 * (c & 3));
      return v;
    } else {
      // Of a quarter's 16 lanes, four hold 16 neighbouring indices of one k,
      // four k in all; the read hands lane i index i of the four.
      const int i = lane & 15, s = (lane >> 4) & 1, h = lane >> 5;
      u32x4_t v;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int k = 4 * r + (i >> 2);  // its last three bits
        const int piece = (first / 8 + 4 * f + 2 * s + ((i & 3) >> 1)) ^ swizzle(k);
        const u32x2_t x = read_turned((lds_s16x4_t*)(at + (16 * j + 8 * h + k) * RB + piece * 16 + 8 * (i & 1)));
        v[2 * r] = x.x;
        v[2 * r + 1] = x.y;
      }
      return v;
    }
  }
};

// Planes of a chunk's q-th product.
__device__ inline int plane_a(int q) { return (0x200110 >> (4 * (5 - q))) & 3; }
__device__ inline int plane_b(int q) { return (0x021010 >> (4 * (5 - q))) & 3; }

// Chunks kc0 .. kc1 - 1 of the tile into acc[FM][FN] of this wave.  PARTS: the
// bfloat16 planes of an operand, 0 for fp32 as it is.
//
// One chunk after another, with R - 1 of them under way.  256 x 256 tiles are
// written out further: with one wave to a SIMD nothing else hides a wait, so a
// step's fragments are read while the products of the step before run, across
// the chunk's border too, and the copies are dealt out between products, which
// would otherwise wait behind a run of them.  (4096 x 65536 x 4096,
// forward and back: 9.05 ms before; 7.2 with this, no wait at the transposing
// reads and dh's sum started from its slab; 6.8 with B's copies a chunk further
// ahead and the masks and exponentials made cheaper.)
template <class S, bool ACOL, bool BCOL, int PARTS>
__device__ __attribute__((always_inline)) inline void xgemm(const XSide<S::BM, ACOL, PARTS == 0>& A,
                                                            const XSide<S::BN, BCOL, PARTS == 0>& B, int64_t K, int kc0, int kc1, uint8_t* smem,
                                                            float16_t (&acc)[S::FM][S::FN], int wave, int lane) {
  constexpr int Q = PARTS == 3 ? 6 : 1;
  const int n = (kc1 - kc0) * Q;
  const int am = (wave % S::WM) * 32 * S::FM, bn = (wave / S::WM) * 32 * S::FN;
  struct Chunk {
    __amdgpu_buffer_rsrc_t a, b;
    bool on;  // a chunk past the last copies nothing
  };
  auto chunk = [&](int ch) __attribute__((always_inline)) {
    const int kc = kc0 + ch / Q, q = ch % Q;
    return Chunk{A.chunk(kc, PARTS == 3 ? plane_a(q) : 0, K), B.chunk(kc, PARTS == 3 ? plane_b(q) : 0, K), ch < n};
  };
  struct Frags {
    u32x4_t a[S::FM], b[S::FN];
  };
  if constexpr (S::FM * S::FN == 16) {
    // LDS: two chunks of A in turn, and three of B.  Once everyone has read a
    // chunk, the A after next takes its place; the B after next has had a place
    // since the chunk before, so its copies go out while nothing else does.
    static_assert(S::R == 2 && S::copies == 16, "eight copies of either");
    constexpr int kSide = S::BM * 128;
    auto copy_a = [&](const Chunk& x, int i, uint8_t* dst) __attribute__((always_inline)) { A.copy(x.a, x.on, i, dst, wave); };
    auto copy_b = [&](const Chunk& x, int i, uint8_t* dst) __attribute__((always_inline)) { B.copy(x.b, x.on, i, dst, wave); };
    auto read1 = [&](Frags& N, int p, const uint8_t* sa, const uint8_t* sb, int j) __attribute__((always_inline)) {
      if (p < 4) N.a[p] = XSide<S::BM, ACOL, PARTS == 0>::read(sa, am, p, j, lane);
      else if (p < 8) N.b[p - 4] = XSide<S::BN, BCOL, PARTS == 0>::read(sb, bn, p - 4, j, lane);
    };
    // A step's 16 products; between them the reads of the next step's
    // fragments (step j of the chunk at sa and sb), and copies.
    auto step = [&](const Frags& F, Frags& N, const uint8_t* sa, const uint8_t* sb, int j, auto copies)
                    __attribute__((always_inline)) {
#pragma unroll
      for (int p = 0; p < 16; ++p) {
        acc[p % 4][p / 4] = mfma32(F.a[p % 4], F.b[p / 4], acc[p % 4][p / 4]);
        pin();
        read1(N, p, sa, sb, j);
        copies(p);
        pin();
      }
    };
    Frags F0, F1;
    uint8_t *a0 = smem, *a1 = smem + kSide;  // chunk ch's, the next one's
    uint8_t *b0 = smem + 2 * kSide, *b1 = b0 + kSide, *b2 = b1 + kSide;
    Chunk x = chunk(0);
#pragma unroll
    for (int i = 0; i < 8; ++i) copy_a(x, i, a0);
#pragma unroll
    for (int i = 0; i < 8; ++i) copy_b(x, i, b0);
    x = chunk(1);
#pragma unroll
    for (int i = 0; i < 8; ++i) copy_b(x, i, b1);
#pragma unroll
    for (int i = 0; i < 8; ++i) copy_a(x, i, a1);
    vm_wait<16>();
    ring_barrier();
#pragma unroll
    for (int p = 0; p < 8; ++p) read1(F0, p, a0, b0, 0);
    x = chunk(2);
#pragma unroll 1
    for (int ch = 0; ch < n; ++ch) {
      pin();
      step(F0, F1, a0, b0, 1, [&](int p) __attribute__((always_inline)) { if (p % 4 == 3) copy_b(x, p / 4, b2); });
      step(F1, F0, a0, b0, 2, [&](int p) __attribute__((always_inline)) { if (p % 4 == 3) copy_b(x, 4 + p / 4, b2); });
      step(F0, F1, a0, b0, 3, [](int) {});
      vm_wait<8>();    // this wave's copies of the next chunk; those of the B after it may be under way
      ring_barrier();  // everyone's, and everyone has read this one
      pin();
      // (what it reads is not used after the last chunk)
      step(F1, F0, a1, b1, 0, [&](int p) __attribute__((always_inline)) { if (p % 2) copy_a(x, p / 2, a0); });
      uint8_t* const u = a0;
      a0 = a1;
      a1 = u;
      uint8_t* const v = b0;
      b0 = b1;
      b1 = b2;
      b2 = v;
      x = chunk(ch + 3);
    }
  } else {
    auto copy = [&](const Chunk& x, int i, uint8_t* dst) __attribute__((always_inline)) {
      if (i < S::BM / 32) A.copy(x.a, x.on, i, dst, wave);
      else B.copy(x.b, x.on, i - S::BM / 32, dst + S::BM * 128, wave);
    };
    auto read = [&](Frags& F, const uint8_t* slot, int j) __attribute__((always_inline)) {
  #pragma unroll
      for (int f = 0; f < S::FM; ++f) F.a[f] = XSide<S::BM, ACOL, PARTS == 0>::read(slot, am, f, j, lane);
  #pragma unroll
      for (int f = 0; f < S::FN; ++f) F.b[f] = XSide<S::BN, BCOL, PARTS == 0>::read(slot + S::BM * 128, bn, f, j, lane);
    };
#pragma unroll
    for (int u = 0; u < S::R - 1; ++u) {
      const Chunk x = chunk(u);
#pragma unroll
      for (int i = 0; i < S::copies; ++i) copy(x, i, smem + u * S::slot);
    }
    int u = 0;
#pragma unroll 1
    for (int ch = 0; ch < n; ++ch) {
      pin();
      vm_wait<(S::R - 2) * S::copies>();  // this wave's copies of the chunk
      ring_barrier();                      // everyone's, and everyone is done with the chunk before
      pin();
      const Chunk x = chunk(ch + S::R - 1);
      uint8_t* const dst = smem + (u == 0 ? S::R - 1 : u - 1) * S::slot;
#pragma unroll
      for (int i = 0; i < S::copies; ++i) copy(x, i, dst);
      pin();
      const uint8_t* slot = smem + u * S::slot;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        Frags F;
        read(F, slot, j);
#pragma unroll
        for (int i = 0; i < S::FN; ++i)
#pragma unroll
          for (int f = 0; f < S::FM; ++f)
            acc[f][i] = PARTS == 0 ? mfma32_f32(F.a[f], F.b[i], acc[f][i]) : mfma32(F.a[f], F.b[i], acc[f][i]);
      }
      u = u + 1 == S::R ? 0 : u + 1;
    }
  }
  vm_wait<0>();
  ring_barrier();
}

// A wave's 32 b's by 32 FM a's (fragment i of its b's) through its share of
// LDS, so that runs of a are stored whole: put(f, g, four values) fills, and
// store(row, piece, sixteen bytes) gets every piece of a row.
template <int FM, int ES>
constexpr int xturn_pitch() {
  return 32 * FM * ES + 16;
}
template <int FM, int ES, typename Value, typename Store>
__device__ __attribute__((always_inline)) inline void xturn(uint8_t* turn, int lane, Value value, Store store) {
  constexpr int PITCH = xturn_pitch<FM, ES>(), LPR = 32 * FM * ES / 16;
  const int c = lane & 31, h = lane >> 5;
#pragma unroll
  for (int f = 0; f < FM; ++f)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float4_t o;
#pragma unroll
      for (int v = 0; v < 4; ++v) o[v] = value(f, 4 * g + v);
      uint8_t* at = turn + c * PITCH + (32 * f + 8 * g + 4 * h) * ES;
      if constexpr (ES == 2)
        *(u32x2_t*)at = u32x2_t{bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3])};
      else
        *(float4_t*)at = o;
    }
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int x = 0; x < 32 * LPR / 64; ++x) {
    const int row = x * (64 / LPR) + lane / LPR, ch = lane % LPR;
    store(row, ch, *(const u32x4_t*)(turn + row * PITCH + ch * 16));
  }
  __builtin_amdgcn_wave_barrier();
}

}  // namespace ds4
