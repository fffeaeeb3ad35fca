// Softmax cross entropy of rows h [T][d] against a vocabulary w [V][d], in
// pieces of the vocabulary and without keeping the logits:
//
//   z = scale h w^T,  lse = log sum_v e^z_v,  loss = lse - z_target
//   ds = dloss scale (e^(z - lse) - [v = target]),  dh = ds w,  dw = ds^T h
//
// Forward: a tile of the product leaves, for each of its rows, the maximum and
// the sum of e^(z - maximum) over its words, and a second kernel joins them.
// Backward: for each piece, the product again with ds as its epilogue (bfloat16,
// or three planes of it for fp32), then the two products with ds.  Rows without
// a target take no part: those that do are copied together first, so a masked
// prompt costs nothing and what its rows hold (NaN, too) reaches nothing.  ds is
// held over the largest |dloss scale|, by which the products are multiplied in
// fp32: 1 / rows, which most losses have there, would otherwise be rounded the
// same way in every value (dh 0.0034 off, against 0.002).  Rounding ds to
// bfloat16 costs each value at most half a step, 2^-8 of it; dh and dw, themselves
// bfloat16, are 0.0018 off where a form with fp32 in between has 0.0017.
//
// Measured (rates count the four products, ds's logits formed again): 4096 x
// 65536 x 4096 in bf16, forward and back, 6.7 to 6.8 ms, 1.3 PFLOP/s; 2047 x 50001 x
// 2048 with a tenth of the rows masked 1.38 to 1.42 ms; 16 rows x 65536 x 4096
// forward 107 us, 5 TB/s of reading w.  fp32: 512 x 60000 x 1024 1.51 to 1.61 ms, 0.16
// PFLOP/s (a library product in fp32 has 0.154); 127 x 1003 x 256 41 us, seven
// launches of 3 to 10 us.
#include <algorithm>
#include <numeric>
#include <type_traits>

#include "../trace.h"
#include "../ops/rowtile.h"
#include "xgemm.h"

namespace ds4 {

// ---------------------------------------------------------------- workspace
// What grows with rows and words is bounded by taking words a piece at a time
// (ds, and the planes of an fp32 w) and, in the forward pass, rows (the partial
// sums).
constexpr int64_t kXentPiece = 256 << 20;   // bytes that either aims at
// fp32 operands of up to so many rows go through the fp32 instruction as they
// are, of more as planes.  The rows at which planes are faster depend on d; this
// is between them.  Forward / forward and back, us, as they are and as planes:
//   256 x 30000 x 1024   134 /  544    157 /  537
//   384 x 30000 x 1024   212 /  811    215 /  768
//   384 x 65536 x  512   203 /  846    218 /  824
//   384 x 10000 x 4096   272 / 1051    378 / 1163
//   512 x 60000 x 1024   578 / 2081    461 / 1609
//   512 x 10000 x 4096   359 / 1365    428 / 1297
constexpr int64_t kXentF32Rows = 384;
constexpr int64_t kXentCounted = 2048;      // rows up to which every block counts the live ones before it
constexpr int kXentSlabs = 32;              // parts of the sum over words in dh, at most

template <typename T>
static T round_up(T v, T m) {
  return (v + m - 1) / m * m;
}

// Shapes of a product's tiles (a's by b's), and the words that a wave of one
// has, which a partial sum covers.
enum { kFew, kNarrow, kSmall, kMid, kBig };  // 128 x 32, 128 x 64, 64 x 64, 128 x 128, 256 x 256
constexpr int kXentPart[] = {32, 32, 32, 64, 128};

// Relative time of a product's blocks in a shape: rounds of 512 blocks, two to
// a CU, and a last one that has up to 256 CUs to themselves; 256 x 256 tiles have
// one to a CU, and are faster where not all CUs have any.  Measured against a
// round of 256 x 256 tiles, 4096 x 65536 x 4096: 128 x 128 tiles 0.62 of the time for
// half of the work, 64 x 64 0.33 for an eighth; alone on a CU little more than
// half of that.  In fp32 the instruction is what takes time.
static double xent_time(int parts, int shape, int64_t a, int64_t b, int64_t splits) {
  const int64_t m = shape == kBig ? 256 : shape == kMid ? 128 : 64;
  const int64_t n = (a + m - 1) / m * ((b + m - 1) / m) * splits;
  if (shape == kBig) return (double)(n / 256) + (n % 256 ? 0.75 + 0.25 / 256 * (double)(n % 256) : 0.0);
  const double pair = parts == 0 ? (shape == kMid ? 2.0 : 0.55) : shape == kMid ? 0.62 : 0.33;
  const int64_t rest = n % 512;
  return (double)(n / 512) * pair + (rest == 0 ? 0.0 : rest <= 256 ? 0.55 * pair : pair);
}
static int xent_shape(int parts, int64_t a, int64_t b, int64_t splits) {
  if (b <= 64) return b <= 32 ? kFew : kNarrow;
  int best = kSmall;
  for (int s = kMid; s <= (parts > 0 ? kBig : kMid); ++s)
    if (xent_time(parts, s, a, b, splits) <= xent_time(parts, best, a, b, splits)) best = s;
  return best;
}

// A product over `words` words by `rows` rows (or columns) as one launch, or
// as two where that is faster: full rounds of 256 x 256 tiles, and the rest in smaller ones.
struct XentLaunch {
  int shape;
  int64_t w0, words;
};
static int xent_launches(int parts, int64_t words, int64_t rows, XentLaunch (&l)[2]) {
  l[0] = {xent_shape(parts, words, rows, 1), 0, words};
  if (parts == 0 || rows <= 64) return 1;
  const int64_t per = (rows + 255) / 256, blocks = (words + 255) / 256 * per;
  const int64_t first = blocks / 256 * 256 / per * 256;
  if (first == 0 || first >= words) return 1;
  const int rest = xent_shape(parts, words - first, rows, 1);
  const double one = xent_time(parts, l[0].shape, words, rows, 1);
  if (xent_time(parts, kBig, first, rows, 1) + xent_time(parts, rest, words - first, rows, 1) >= 0.97 * one) return 1;
  l[0] = {kBig, 0, first};
  l[1] = {rest, first, words - first};
  return 2;
}

struct XentPlan {
  int parts;          // bfloat16 planes of an operand; 0: fp32 as it is
  int es;             // bytes of its values, in all planes
  int64_t piece;      // words of a piece, a multiple of 256
  int pieces;
  int64_t rows;       // rows of a forward pass over the vocabulary
  int slabs;
  // offsets into the workspace
  size_t hc, wp, n, live, y, lse, g, ds, slab, zt, part, bytes;
};

static XentPlan xent_plan(int dt, int64_t T, int64_t V, int d, bool grad) {
  XentPlan p{};
  p.parts = dt != DS4MOE_DT_F32 ? 1 : T <= kXentF32Rows ? 0 : 3;
  p.es = p.parts == 0 ? 4 : 2 * p.parts;
  // bytes per word of what a piece keeps: ds, and the planes of an fp32 w
  const int64_t per = p.es * std::max<int64_t>(grad ? T : 0, p.parts == 3 ? d : 0);
  const int64_t all = round_up<int64_t>(V, 256), tr = (T + 255) / 256, td = d / 256;
  const int64_t most = per ? std::max<int64_t>(2048, kXentPiece / per / 256 * 256) : all;
  // words of a piece whose products are full rounds of blocks
  const int64_t unit = 256 * std::max(256 / std::gcd<int64_t>(256, tr), 256 / std::gcd<int64_t>(256, td));
  if (most >= all) p.piece = all;
  else if (most >= unit) p.piece = most / unit * unit;
  else p.piece = round_up<int64_t>((all + (all + most - 1) / most - 1) / ((all + most - 1) / most), 256);
  p.pieces = (int)((all + p.piece - 1) / p.piece);
  // Parts of dh's sum: the fewer rounds of tiles (26 ns a word, six times that
  // as planes and ten times in fp32) against writing the parts and reading them
  // again.  1500 x 40000 x 1024 in bf16: 8 parts 542 us forward and back, 32 589;
  // 16 x 65536 x 256: 83 and 61.
  const double word = p.parts == 1 ? 0.026 : p.parts == 3 ? 0.156 : 0.26;
  auto cost = [&](int s) {
    return (double)((tr * td * s + 255) / 256) / s * (double)p.piece * word + (double)s * (double)T * d * 8 / 4.8e6;
  };
  p.slabs = 1;
  for (int s = 2; s <= kXentSlabs && p.piece / s >= 256; s *= 2)
    if (cost(s) < cost(p.slabs)) p.slabs = s;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += round_up<size_t>(bytes, 256);
    return here;
  };
  if (p.parts == 3 || grad) p.hc = take((size_t)p.es * T * d);
  if (p.parts == 3) p.wp = take((size_t)6 * p.piece * d);
  if (grad) {
    p.n = take(8);
    p.live = take(4 * T);
    p.y = take(4 * T);
    p.lse = take(4 * T);
    p.g = take(4 * T);
    p.ds = take((size_t)p.es * T * p.piece);
    p.slab = take((size_t)4 * p.slabs * T * d);
  } else {
    p.rows = std::min(T, std::max<int64_t>(1024, kXentPiece / (8 * (all / 128)) / 256 * 256));
    p.zt = take(4 * p.rows);
    auto sums = [&](int64_t rows) {  // partial sums of that many rows
      int64_t n = 0;
      for (int64_t v0 = 0; v0 < V; v0 += p.piece) {
        XentLaunch l[2];
        const int m = xent_launches(p.parts, std::min(p.piece, V - v0), rows, l);
        for (int i = 0; i < m; ++i) {
          const int per = kXentPart[l[i].shape];
          n += (l[i].words + per - 1) / per;
        }
      }
      return n * rows;
    };
    p.part = take((size_t)8 * std::max(sums(p.rows), T % p.rows ? sums(T % p.rows) : 0));
  }
  p.bytes = at;
  return p;
}
size_t xent_ws_bytes(int dt, int64_t T, int64_t V, int d, bool grad) { return xent_plan(dt, T, V, d, grad).bytes; }

// ---------------------------------------------------------------- rows that have a target
// The largest |g|, where its reciprocal has fp32's range too.
__device__ inline float xent_top(float top) {
  return top >= 1.17549435e-38f && top <= 8.507059e37f ? top : 1.0f;
}
// live: the rows with a target in order, then the others from the end; n: how
// many; y, lse, g: theirs; top: the largest |g|, or 1.  One block: rows are
// few beside the products.
__global__ __launch_bounds__(1024) void k_xent_live(const int32_t* __restrict__ target, int T, int V, float scale,
                                                    const float* __restrict__ lse, const float* __restrict__ dloss,
                                                    int32_t* __restrict__ n, int32_t* __restrict__ live,
                                                    int32_t* __restrict__ y, float* __restrict__ lse_c,
                                                    float* __restrict__ g_c) {
  __shared__ int sums[2][16];
  __shared__ float tops[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int base = 0;
  float top = 0.f;
  for (int t0 = 0, b = 0; t0 < T; t0 += 1024, b ^= 1) {
    const int t = t0 + tid;
    const int v = t < T ? target[t] : -1;
    const bool on = v >= 0 && v < V;
    const uint64_t m = __ballot(on);
    if (lane == 0) sums[b][wave] = __popcll(m);
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
      before += w < wave ? sums[b][w] : 0;
      total += sums[b][w];
    }
    const int at = base + before + __popcll(m & ((1ull << lane) - 1));
    if (on) {
      const float g = scale * (dloss ? dloss[t] : 1.0f);
      live[at] = t;
      y[at] = v;
      lse_c[at] = lse[t];
      g_c[at] = g;
      top = fmaxf(top, fabsf(g));
    } else if (t < T) {
      live[T - 1 - (t - at)] = t;  // t - at rows without a target lie before it
    }
    base += total;
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
  if (lane == 0) tops[wave] = top;
  __syncthreads();
  if (tid != 0) return;
  for (int w = 1; w < 16; ++w) top = fmaxf(top, tops[w]);
  n[0] = base;
  ((float*)n)[1] = xent_top(top);
}

// x as three bfloat16 values whose sum it is, each to the nearest of what is left
// (what lies under 2^-133 is lost).  So the second and third are within 2^-8 and
// 2^-17 of the power of two below x, of either sign: what xgemm leaves out is
// within 2^-24 of the product and has no bias.  (By truncation it would be up to
// 2^-21, always towards zero: 0.7 x 2^-24 in the mean.)  Finite values above
// bfloat16's largest have that as their first part; an infinity or a NaN is its
// first part.
__device__ inline void xsplit8(const float (&x)[8], u32x4_t (&o)[3]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    float v[2] = {x[2 * p], x[2 * p + 1]};
    bool finite[2];
    float first[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      finite[e] = fabsf(v[e]) <= 3.402823466e38f;
      first[e] = finite[e] ? __builtin_amdgcn_fmed3f(v[e], -0x1.FEp127f, 0x1.FEp127f) : v[e];
    }
#pragma unroll
    for (int s = 0; s < 3; ++s) {
      const uint32_t w = s == 0 ? bf16_pair(first[0], first[1]) : bf16_pair(v[0], v[1]);
      o[s][p] = w;
      v[0] -= __builtin_bit_cast(float, w << 16);
      v[1] -= __builtin_bit_cast(float, w & 0xFFFF0000u);
      if (s == 0) {
        v[0] = finite[0] ? v[0] : 0.f;
        v[1] = finite[1] ? v[1] : 0.f;
      }
    }
  }
}

// Row `from` of src as row r of the live rows, as planes; dh of a row without a
// target is zero.
template <int PARTS>
__device__ inline void xent_row(const void* __restrict__ src, int64_t from, int64_t r, bool on, int d,
                                uint8_t* __restrict__ dst, int64_t plane, void* __restrict__ dh) {
  constexpr bool BF = PARTS == 1;
  for (int i = 8 * threadIdx.x; i < d; i += 2048) {
    if (on) {
      const Raw8<BF> v = ld8<BF>(src, from * d + i);
      if constexpr (PARTS == 3) {
        float x[8];
        u32x4_t o[3];
        unpack8<BF>(v, x);
        xsplit8(x, o);
#pragma unroll
        for (int s = 0; s < 3; ++s) *(u32x4_t*)(dst + s * plane + (r * d + i) * 2) = o[s];
      } else {
        *(Raw8<BF>*)(dst + (r * d + i) * (BF ? 2 : 4)) = v;
      }
    } else if (dh) {
      const float zero[8] = {};
      st8<BF>(dh, from * d + i, zero);
    }
  }
}
template <int PARTS>
__global__ __launch_bounds__(256) void k_xent_rows(const void* __restrict__ src, const int32_t* __restrict__ n,
                                                   const int32_t* __restrict__ live, int64_t rows, int d,
                                                   uint8_t* __restrict__ dst, int64_t plane, void* __restrict__ dh) {
  const int n_live = *n;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) xent_row<PARTS>(src, live[r], r, r < n_live, d, dst, plane, dh);
}
// k_xent_live and k_xent_rows in one, for as many rows as a block counts in a
// moment: block t counts the live rows before row t, the last one all of them.
template <int PARTS>
__global__ __launch_bounds__(256) void k_xent_live_rows(const int32_t* __restrict__ target, int T, int V, float scale,
                                                        const float* __restrict__ lse, const float* __restrict__ dloss,
                                                        int32_t* __restrict__ n, int32_t* __restrict__ live,
                                                        int32_t* __restrict__ y, float* __restrict__ lse_c,
                                                        float* __restrict__ g_c, const void* __restrict__ src, int d,
                                                        uint8_t* __restrict__ dst, int64_t plane, void* __restrict__ dh) {
  __shared__ int counts[4];
  __shared__ float tops[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, t = blockIdx.x;
  int count = 0;
  float top = 0.f;
  for (int i0 = 0; i0 < t; i0 += 256) {
    const int i = i0 + tid;
    const int v = i < t ? target[i] : -1;
    const bool on = v >= 0 && v < V;
    count += on;
    if (t == T && on) top = fmaxf(top, fabsf(scale * (dloss ? dloss[i] : 1.0f)));
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    count += __shfl_xor(count, o);
    top = fmaxf(top, __shfl_xor(top, o));
  }
  if (lane == 0) {
    counts[wave] = count;
    tops[wave] = top;
  }
  __syncthreads();
  count = (counts[0] + counts[1]) + (counts[2] + counts[3]);
  if (t == T) {
    if (tid == 0) {
      n[0] = count;
      ((float*)n)[1] = xent_top(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])));
    }
    return;
  }
  const int v = target[t];
  const bool on = v >= 0 && v < V;
  const int r = on ? count : T - 1 - (t - count);
  if (tid == 0) {
    live[r] = t;
    if (on) {
      y[r] = v;
      lse_c[r] = lse[t];
      g_c[r] = scale * (dloss ? dloss[t] : 1.0f);
    }
  }
  xent_row<PARTS>(src, t, r, on, d, dst, plane, dh);
}
// All of n fp32 values (a multiple of 8) as planes.
__global__ __launch_bounds__(256) void k_xent_split(const float* __restrict__ src, int64_t n, uint8_t* __restrict__ dst,
                                                    int64_t plane) {
  const int64_t step = (int64_t)gridDim.x * 2048;
#pragma unroll 2
  for (int64_t i = (int64_t)blockIdx.x * 2048 + 8 * threadIdx.x; i < n; i += step) {
    float x[8];
    u32x4_t o[3];
    unpack8<false>(ld8<false>(src, i), x);
    xsplit8(x, o);
#pragma unroll
    for (int s = 0; s < 3; ++s) *(u32x4_t*)(dst + s * plane + i * 2) = o[s];
  }
}

// ---------------------------------------------------------------- products
struct XArgs {
  XOperand a, b;
  int64_t a_rows, b_rows;  // how many a's and b's there are (b's: at most)
  int64_t K;
  const int32_t* n;  // live rows, backward: b's, or the k of dw
  int splits;        // of k
  // epilogues
  float scale;
  int V;             // words of the launch
  const int32_t* y;
  int v0;            // its first word
  int rows, part0;   // partial sums: rows of one, and the first of this launch
  float2* part;
  float* zt;
  const float *lse, *g, *top;
  uint8_t* out;
  int64_t out_pitch, out_plane;  // bytes
  bool add;
};
enum { XE_SUM = 0, XE_DS = 1, XE_ROWS = 2, XE_SLAB = 3 };

// Tile of this block: (split, a tile, b tile).  Each XCD takes a contiguous run
// of them (block_item), in which four a tiles meet all b tiles before the next
// four: the 32 blocks that an XCD runs at once read 4 + 8 tiles' operands.
__device__ inline bool xtile(int ta, int tb, int splits, int& a, int& b, int& s) {
  int64_t item;
  if (!block_item((int64_t)ta * tb * splits, item)) return false;
  const int per = ta * tb;
  s = (int)(item / per);
  const int left = (int)(item - (int64_t)s * per);
  const int g = left / (4 * tb), in = left - g * 4 * tb;
  const int wide = min(4, ta - 4 * g);
  b = in / wide;
  a = 4 * g + in - b * wide;
  return true;
}

template <class S, int EPI, int PARTS, bool OBF>
__global__ __launch_bounds__(256, S::lds > 80 * 1024 ? 1 : 2) void k_xent_gemm(XArgs x) {
  constexpr bool ACOL = EPI == XE_ROWS || EPI == XE_SLAB, BCOL = EPI == XE_ROWS;
  extern __shared__ uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63, c = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int64_t b_rows = x.b_rows, K = x.K;
  if (x.n) {
    const int64_t n = ld_uniform(x.n);
    if constexpr (BCOL) K = n;
    else b_rows = n;
  }
  if (b_rows <= 0) return;
  int ta, tb, s;
  if (!xtile((int)((x.a_rows + S::BM - 1) / S::BM), (int)((b_rows + S::BN - 1) / S::BN), x.splits, ta, tb, s)) return;
  const int64_t a0 = (int64_t)ta * S::BM, b0 = (int64_t)tb * S::BN;
  XSide<S::BM, ACOL, PARTS == 0> A;
  XSide<S::BN, BCOL, PARTS == 0> B;
  A.init(x.a, a0, x.a_rows, tid);
  B.init(x.b, b0, b_rows, tid);
  constexpr int KC = PARTS == 0 ? 32 : 64;
  const int nk = (int)((K + KC - 1) / KC);
  const int kc0 = (int)((int64_t)nk * s / x.splits), kc1 = (int)((int64_t)nk * (s + 1) / x.splits);
  const int am = (wave % S::WM) * 32 * S::FM, bn = (wave / S::WM) * 32 * S::FN;
  float16_t acc[S::FM][S::FN] = {};
  if constexpr (EPI == XE_SLAB) {  // on top of the pieces before; zeros without any
    const int64_t rows = min((int64_t)S::BN, b_rows - b0);
    const __amdgpu_buffer_rsrc_t r = buf_rsrc(x.out + s * x.out_plane + b0 * x.out_pitch, (uint32_t)(rows * x.out_pitch));
#pragma unroll
    for (int i = 0; i < S::FN; ++i) {
      const uint32_t at = x.add ? (uint32_t)((bn + 32 * i + c) * x.out_pitch + (a0 + am + 4 * h) * 4) : kOob;
#pragma unroll
      for (int f = 0; f < S::FM; ++f)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float4_t u = __builtin_bit_cast(float4_t, buf_ld128(r, at, 128 * f + 32 * g));
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[f][i][4 * g + v] = u[v];
        }
      pin();
    }
  }
  xgemm<S, ACOL, BCOL, PARTS>(A, B, K, kc0, kc1, smem, acc, wave, lane);

  // Exponentials to base 2, the scale in the same multiply-add.  Words past the
  // vocabulary's end are only in its last tile, a row's target in few.
  const float k2 = x.scale * 1.44269504f;
  const int left = x.V - (int)a0 - am;  // words from the wave's first on
  auto word = [&](int f, int v) { return 32 * f + 8 * (v >> 2) + 4 * h + (v & 3); };
  if constexpr (EPI == XE_SUM) {
    const int a1 = (int)a0 + am;
    const bool whole = left >= 32 * S::FM, falling = k2 < 0.f;
#pragma unroll
    for (int i = 0; i < S::FN; ++i) {
      const int64_t t = b0 + bn + 32 * i + c;
      const bool on = t < b_rows;
      float m = -INFINITY;  // the largest product, or that of their negatives where the scale turns them
      float sum = 0.f;
      auto top = [&](auto all, float sign) __attribute__((always_inline)) {
#pragma unroll
        for (int f = 0; f < S::FM; ++f)
#pragma unroll
          for (int v = 0; v < 16; ++v)
            if (decltype(all)::value) m = fmaxf(m, sign * acc[f][i][v]);
            else m = fmaxf(m, word(f, v) < left ? sign * acc[f][i][v] : -INFINITY);
        m = fmaxf(m, __shfl_xor(m, 32));
      };
      if (!whole) top(std::false_type{}, falling ? -1.f : 1.f);
      else if (falling) top(std::true_type{}, -1.f);
      else top(std::true_type{}, 1.f);
      const float z = fabsf(k2) * m, mm = m == -INFINITY ? 0.f : z;
      auto add = [&](auto all) __attribute__((always_inline)) {
#pragma unroll
        for (int f = 0; f < S::FM; ++f)
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            const float e = __builtin_amdgcn_exp2f(fmaf(k2, acc[f][i][v], -mm));
            sum += decltype(all)::value || word(f, v) < left ? e : 0.f;
          }
      };
      if (whole) add(std::true_type{});
      else add(std::false_type{});
      pin();
      sum += __shfl_xor(sum, 32);
      if (on && left > 0 && h == 0)
        x.part[(int64_t)(x.part0 + a1 / (32 * S::FM)) * x.rows + t] = float2{m == -INFINITY ? m : fabsf(x.scale) * m, sum};
      const int y = on ? x.y[t] - x.v0 - a1 : -1;  // the target among the wave's words
      const bool mine = y >= 0 && y < 32 * S::FM && y < left && ((y >> 2) & 1) == h;
      if (__ballot(mine)) {
        float z = 0.f;
#pragma unroll
        for (int f = 0; f < S::FM; ++f)
#pragma unroll
          for (int v = 0; v < 16; ++v) z = y == word(f, v) ? acc[f][i][v] : z;
        if (mine) x.zt[t] = x.scale * z;
      }
    }
  } else if constexpr (EPI == XE_DS) {
    // words past the vocabulary's end are zeros: the products with ds run over whole pieces
    constexpr int ES = PARTS == 0 ? 4 : 2;
    uint8_t* const turn = smem + wave * 32 * xturn_pitch<S::FM, ES>();
    const float by = 1.0f / *x.top;
#pragma unroll
    for (int i = 0; i < S::FN; ++i) {
      const int64_t t = b0 + bn + 32 * i + c;
      const bool on = t < b_rows;
      const float lse = on ? x.lse[t] : 0.f, g = on ? x.g[t] * by : 0.f;
      const int y = on ? x.y[t] - x.v0 - (int)a0 - am : -1;
      // lse to base 2 in two parts where the values are held to fp32
      const float l = 1.44269504f * lse, ll = PARTS != 1 ? fmaf(1.44269504f, lse, -l) + 1.92596299e-8f * lse : 0.f;
#pragma unroll
      for (int f = 0; f < S::FM; ++f)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          float e = fmaf(k2, acc[f][i][v], -l);
          if (PARTS != 1) e -= ll;
          acc[f][i][v] = __builtin_amdgcn_exp2f(e);
        }
      if (__ballot(y >= 0 && y < 32 * S::FM)) {
#pragma unroll
        for (int f = 0; f < S::FM; ++f)
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[f][i][v] -= word(f, v) == y ? 1.f : 0.f;
      }
      if (left < 32 * S::FM) {
#pragma unroll
        for (int f = 0; f < S::FM; ++f)
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[f][i][v] = word(f, v) < left ? acc[f][i][v] : 0.f;
      }
#pragma unroll
      for (int f = 0; f < S::FM; ++f)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[f][i][v] *= g;
      // by planes: what the bfloat16 before leaves
#pragma unroll
      for (int q = 0; q < std::max(PARTS, 1); ++q) {
        xturn<S::FM, ES>(
            turn, lane, [&](int f, int v) { return acc[f][i][v]; },
            [&](int row, int ch, u32x4_t v) {
              const int64_t r = b0 + bn + 32 * i + row;
              if (r < b_rows) *(u32x4_t*)(x.out + q * x.out_plane + r * x.out_pitch + (a0 + am) * ES + ch * 16) = v;
            });
        if (q + 1 < PARTS) {
#pragma unroll
          for (int f = 0; f < S::FM; ++f)
#pragma unroll
            for (int v = 0; v < 16; v += 2) {
              const uint32_t b = bf16_pair(acc[f][i][v], acc[f][i][v + 1]);
              acc[f][i][v] -= __builtin_bit_cast(float, b << 16);
              acc[f][i][v + 1] -= __builtin_bit_cast(float, b & 0xFFFF0000u);
            }
        }
      }
    }
  } else {
    constexpr int ES = EPI == XE_ROWS && OBF ? 2 : 4;
    uint8_t* const turn = smem + wave * 32 * xturn_pitch<S::FM, ES>();
    uint8_t* const out = x.out + s * x.out_plane;
    const float by = EPI == XE_ROWS ? *x.top : 1.f;
#pragma unroll
    for (int i = 0; i < S::FN; ++i)
      xturn<S::FM, ES>(
          turn, lane, [&](int f, int v) { return EPI == XE_ROWS ? by * acc[f][i][v] : acc[f][i][v]; },
          [&](int row, int ch, u32x4_t v) {
            const int64_t r = b0 + bn + 32 * i + row;
            if (r >= b_rows) return;
            *(u32x4_t*)(out + r * x.out_pitch + (a0 + am) * ES + ch * 16) = v;
          });
  }
}

// ---------------------------------------------------------------- joins
// loss and lse of the rows from their partial sums: R rows by 1024 / R shares
// of the parts to a block (R = 4 where few rows have many parts: 16 rows of
// 2048 parts 13 -> 5 us).
__device__ inline void xent_add(float2& a, float2 b) {
  const float top = fmaxf(a.x, b.x), mm = top == -INFINITY ? 0.f : top;
  // (a sum that is no number stays one, whatever it is multiplied by)
  a = float2{top, a.y * __expf(a.x - mm) + b.y * __expf(b.x - mm)};
}
template <int R>
__global__ __launch_bounds__(1024) void k_xent_join(const float2* __restrict__ part, int parts, int64_t rows,
                                                    const int32_t* __restrict__ target, int V,
                                                    const float* __restrict__ zt, float* __restrict__ loss,
                                                    float* __restrict__ lse) {
  constexpr int S = 1024 / R;
  __shared__ float2 lds[1024];
  const int tid = threadIdx.x, c = tid % R, s = tid / R;
  const int64_t r = (int64_t)blockIdx.x * R + c;
  const bool on = r < rows;
  float2 a = {-INFINITY, 0.f};
  if (on) {
#pragma unroll 8
    for (int p = s; p < parts; p += S) xent_add(a, part[(int64_t)p * rows + r]);
  }
  lds[tid] = a;
  __syncthreads();
#pragma unroll 1
  for (int o = 512; o >= R; o >>= 1) {
    if (tid < o) xent_add(lds[tid], lds[tid + o]);
    __syncthreads();
  }
  if (s != 0 || !on) return;
  const float l = lds[tid].x + logf(lds[tid].y);
  lse[r] = l;
  const int y = target[r];
  loss[r] = y >= 0 && y < V ? l - zt[r] : 0.f;
}

// dh of the live rows from the slabs.
template <bool BF>
__global__ __launch_bounds__(256) void k_xent_dh(const float* __restrict__ slab, int slabs, int64_t stride,
                                                 const int32_t* __restrict__ n, const int32_t* __restrict__ live,
                                                 int d, const float* __restrict__ top, void* __restrict__ dh) {
  const int rows = *n;
  const float by = *top;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const int64_t t = live[r];
    for (int i = 8 * threadIdx.x; i < d; i += 2048) {
      float v[8];
      unpack8<false>(ld8<false>(slab, r * d + i), v);
      for (int s = 1; s < slabs; ++s) {
        float u[8];
        unpack8<false>(ld8<false>(slab + s * stride, r * d + i), u);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += u[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= by;
      st8<BF>(dh, t * d + i, v);
    }
  }
}

// ---------------------------------------------------------------- launches
using XFew = XShape<4, 1, 1, 1, 3>;    // two blocks to a CU, as the next three have
using XNarrow = XShape<4, 1, 1, 2, 3>;
using XSmall = XShape<2, 2, 1, 1, 4>;
using XMid = XShape<2, 2, 2, 2, 2>;
using XBig = XShape<2, 2, 4, 4, 2>;

template <class S, int EPI, int PARTS, bool OBF>
static hipError_t xent_launch(const XArgs& x, hipStream_t st) {
  const int64_t blocks = (x.a_rows + S::BM - 1) / S::BM * ((x.b_rows + S::BN - 1) / S::BN) * x.splits;
  DS4_LAUNCH((k_xent_gemm<S, EPI, PARTS, OBF>), dim3((unsigned)blocks), dim3(256), S::lds, st, x);
  return hipGetLastError();
}
template <int EPI, int PARTS, bool OBF>
static hipError_t xent_shaped(int shape, const XArgs& x, hipStream_t st) {
  if constexpr (EPI != XE_ROWS) {
    if (shape == kFew) return xent_launch<XFew, EPI, PARTS, OBF>(x, st);
    if (shape == kNarrow) return xent_launch<XNarrow, EPI, PARTS, OBF>(x, st);
  }
  if (shape == kSmall) return xent_launch<XSmall, EPI, PARTS, OBF>(x, st);
  if constexpr (PARTS > 0) {
    if (shape == kBig) return xent_launch<XBig, EPI, PARTS, OBF>(x, st);
  }
  return xent_launch<XMid, EPI, PARTS, OBF>(x, st);
}
// The product of a piece: its words are a's, or b's (dw); the sum over words
// of dh is one launch.
template <int EPI, int PARTS, bool OBF>
static hipError_t xent_gemm(XArgs& x, hipStream_t st) {
  if (EPI == XE_SLAB) return xent_shaped<EPI, PARTS, OBF>(xent_shape(PARTS, x.a_rows, x.b_rows, x.splits), x, st);
  constexpr bool of_b = EPI == XE_ROWS;
  constexpr int kES = PARTS == 0 ? 4 : 2;
  XentLaunch l[2];
  const int n = xent_launches(PARTS, of_b ? x.b_rows : x.a_rows, of_b ? x.a_rows : x.b_rows, l);
  for (int i = 0; i < n; ++i) {
    XArgs y = x;
    const int shape = of_b && l[i].shape < kSmall ? kSmall : l[i].shape;
    if (of_b) {
      y.b.p += kES * l[i].w0;
      y.b_rows = l[i].words;
      y.out += l[i].w0 * y.out_pitch;
    } else {
      y.a.p += l[i].w0 * y.a.pitch;
      y.a_rows = l[i].words;
      y.V = (int)l[i].words;
      y.v0 += (int)l[i].w0;
      y.out += kES * l[i].w0;
      x.part0 += (int)((l[i].words + kXentPart[shape] - 1) / kXentPart[shape]);
    }
    const hipError_t e = xent_shaped<EPI, PARTS, OBF>(shape, y, st);
    if (e) return e;
  }
  return hipSuccess;
}
static unsigned xent_row_blocks(int64_t rows) { return (unsigned)std::min<int64_t>(rows, 8192); }

static void xent_split(const void* src, int64_t n, uint8_t* dst, int64_t plane, hipStream_t st) {
  DS4_LAUNCH(k_xent_split, dim3((unsigned)std::min<int64_t>((n + 2047) / 2048, 4096)), dim3(256), 0, st, (const float*)src,
             n, dst, plane);
}

template <int PARTS>
static hipError_t xent_forward(const XentCall& c) {
  const XentPlan p = xent_plan(c.dt, c.T, c.V, c.d, false);
  uint8_t* w = c.ws;
  constexpr int kES = PARTS == 0 ? 4 : 2, kIn = PARTS == 1 ? 2 : 4;  // bytes of an operand's value, of an input's
  const int64_t pitch = kES * (int64_t)c.d;
  XOperand h = {(const uint8_t*)c.h, 0, pitch};
  if (PARTS == 3) {
    h = {w + p.hc, c.T * pitch, pitch};
    xent_split(c.h, c.T * c.d, w + p.hc, h.plane, c.st);
  }
  for (int64_t r0 = 0; r0 < c.T; r0 += p.rows) {
    const int64_t rows = std::min(c.T - r0, p.rows);
    int parts = 0;
    for (int i = 0; i < p.pieces; ++i) {
      const int64_t v0 = i * p.piece, words = std::min(p.piece, c.V - v0);
      const uint8_t* src = (const uint8_t*)c.w + v0 * c.d * kIn;
      XArgs x{};
      x.a = {src, 0, pitch};
      if (PARTS == 3) {
        xent_split(src, words * c.d, w + p.wp, p.piece * pitch, c.st);
        x.a = {w + p.wp, p.piece * pitch, pitch};
      }
      x.b = {h.p + r0 * h.pitch, h.plane, h.pitch};
      x.a_rows = words;
      x.b_rows = rows;
      x.K = c.d;
      x.splits = 1;
      x.scale = c.scale;
      x.V = (int)words;
      x.y = c.target + r0;
      x.v0 = (int)v0;
      x.rows = (int)rows;
      x.part = (float2*)(w + p.part);
      x.part0 = parts;
      x.zt = (float*)(w + p.zt);
      const hipError_t e = xent_gemm<XE_SUM, PARTS, false>(x, c.st);
      if (e) return e;
      parts = x.part0;
    }
#define DS4_JOIN(R)                                                                                                 \
  DS4_LAUNCH(k_xent_join<R>, dim3((unsigned)((rows + R - 1) / R)), dim3(1024), 0, c.st, (const float2*)(w + p.part), \
             parts, rows, c.target + r0, (int)c.V, (const float*)(w + p.zt), c.loss + r0, c.lse + r0)
    if (rows <= 256 && parts > 64) DS4_JOIN(4);
    else DS4_JOIN(32);
#undef DS4_JOIN
  }
  return hipGetLastError();
}

template <int PARTS>
static hipError_t xent_backward(const XentCall& c) {
  constexpr bool BF = PARTS == 1;
  constexpr int kES = PARTS == 0 ? 4 : 2, kIn = PARTS == 1 ? 2 : 4;
  const XentPlan p = xent_plan(c.dt, c.T, c.V, c.d, true);
  uint8_t* w = c.ws;
  const int64_t pitch = kES * (int64_t)c.d;
  int32_t* const n = (int32_t*)(w + p.n);
  int32_t* const live = (int32_t*)(w + p.live);
  hipError_t e;
  if (c.T <= kXentCounted) {
    DS4_LAUNCH((k_xent_live_rows<PARTS>), dim3((unsigned)c.T + 1), dim3(256), 0, c.st, c.target, (int)c.T, (int)c.V, c.scale,
               c.lse_in, c.dloss, n, live, (int32_t*)(w + p.y), (float*)(w + p.lse), (float*)(w + p.g), c.h, c.d, w + p.hc,
               c.T * pitch, c.dh);
  } else {
    DS4_LAUNCH(k_xent_live, dim3(1), dim3(1024), 0, c.st, c.target, (int)c.T, (int)c.V, c.scale, c.lse_in, c.dloss, n, live,
               (int32_t*)(w + p.y), (float*)(w + p.lse), (float*)(w + p.g));
    DS4_LAUNCH((k_xent_rows<PARTS>), dim3(xent_row_blocks(c.T)), dim3(256), 0, c.st, c.h, (const int32_t*)n,
               (const int32_t*)live, c.T, c.d, w + p.hc, c.T * pitch, c.dh);
  }
  for (int i = 0; i < p.pieces; ++i) {
    const int64_t v0 = i * p.piece, words = std::min(p.piece, c.V - v0);
    const uint8_t* src = (const uint8_t*)c.w + v0 * c.d * kIn;
    XOperand wop = {src, 0, pitch};
    if (PARTS == 3) {
      xent_split(src, words * c.d, w + p.wp, p.piece * pitch, c.st);
      wop = {w + p.wp, p.piece * pitch, pitch};
    }
    const XOperand hop = {w + p.hc, c.T * pitch, pitch}, dsop = {w + p.ds, kES * c.T * p.piece, kES * p.piece};
    XArgs x{};
    x.a = wop;
    x.b = hop;
    x.a_rows = words;
    x.b_rows = c.T;
    x.K = c.d;
    x.n = n;
    x.splits = 1;
    x.scale = c.scale;
    x.V = (int)words;
    x.y = (const int32_t*)(w + p.y);
    x.v0 = (int)v0;
    x.lse = (const float*)(w + p.lse);
    x.g = (const float*)(w + p.g);
    x.top = (const float*)n + 1;
    x.out = w + p.ds;
    x.out_pitch = dsop.pitch;
    x.out_plane = dsop.plane;
    // the last tile's words past the end are written too: as zeros
    if ((e = xent_gemm<XE_DS, PARTS, false>(x, c.st))) return e;
    if (c.dh) {
      XArgs u{};
      u.a = wop;
      u.b = dsop;
      u.a_rows = c.d;
      u.b_rows = c.T;
      u.K = words;
      u.n = n;
      u.splits = p.slabs;
      u.out = w + p.slab;
      u.out_pitch = 4 * (int64_t)c.d;
      u.out_plane = 4 * c.T * c.d;
      u.add = i > 0;
      if ((e = xent_gemm<XE_SLAB, PARTS, false>(u, c.st))) return e;
    }
    if (c.dw) {
      XArgs u{};
      u.a = hop;
      u.b = dsop;
      u.a_rows = c.d;
      u.b_rows = words;
      u.K = c.T;
      u.n = n;
      u.top = (const float*)n + 1;
      u.splits = 1;
      u.out = (uint8_t*)c.dw + v0 * c.d * kIn;
      u.out_pitch = c.d * (int64_t)kIn;
      if ((e = xent_gemm<XE_ROWS, PARTS, BF>(u, c.st))) return e;
    }
  }
  if (c.dh)
    DS4_LAUNCH(k_xent_dh<BF>, dim3(xent_row_blocks(c.T)), dim3(256), 0, c.st, (const float*)(w + p.slab), p.slabs,
               c.T * (int64_t)c.d, (const int32_t*)n, (const int32_t*)live, c.d, (const float*)n + 1, c.dh);
  return hipGetLastError();
}

static int xent_parts(const XentCall& c) { return xent_plan(c.dt, c.T, c.V, c.d, false).parts; }
hipError_t launch_xent(const XentCall& c) {
  const int parts = xent_parts(c);
  return parts == 0 ? xent_forward<0>(c) : parts == 1 ? xent_forward<1>(c) : xent_forward<3>(c);
}
hipError_t launch_xent_grad(const XentCall& c) {
  const int parts = xent_parts(c);
  return parts == 0 ? xent_backward<0>(c) : parts == 1 ? xent_backward<1>(c) : xent_backward<3>(c);
}

}  // namespace ds4
