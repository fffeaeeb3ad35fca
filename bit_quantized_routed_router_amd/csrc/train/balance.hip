// Balance loss of the router and its gradient to the routing logits:
//
//   p_te = e^(z_te - max) / sum,   c_be = slots of sequence b on expert e,
//   n_b = tokens of b with a slot on any expert (the others take no part)
//   loss_b  = E / (k n_b^2) sum_e c_be sum_t p_te
//   dz_te   = dloss_b E / (k n_b^2) p_te (c_be - sum_j p_tj c_bj) + the
//             gradients of the token's slots on e
//
// A row of logits is held by G lanes, NV runs of four each, and read once; a
// block takes a run of one sequence's tokens, adds up probabilities in
// registers and counts in LDS, and a second kernel joins the runs of each
// sequence in order.  Nothing floating is added by atomics, so results repeat.
//
// Measured, forward and back: 2048 tokens of 256 experts 17 us in three launches
// (in a trace 6, join 6, gradient 5); 16381 tokens in 13 sequences, bf16, 28 us
// (10, 7, 12); 262144 tokens of 64 experts 61 to 62 us (19, 6, 30: 3.6 TB/s of logits
// read, 4.4 of logits read and gradients written; a 4 GB copy has 4.8).
#include <algorithm>

#include "../ops/rowtile.h"
#include "../trace.h"
#include "train.h"

namespace ds4 {

constexpr int kBalThreads = 256;

// Lanes of a row: a quarter of its experts, from 4 to 64.
static int bal_lanes(int E) { return E <= 16 ? 4 : E <= 64 ? 16 : 64; }

// Tokens of a block: 16, and 32 where there are enough blocks, so that the join
// has few runs to add; no more than 2048 blocks, so that it need not add many.
static int bal_run(int64_t T) { return (int)std::max<int64_t>(T <= 8192 ? 16 : 32, (T + 2047) / 2048); }
// Up to this many tokens a sequence is one run and needs no join.
static bool bal_one(int64_t T) { return T <= 32; }

struct BalRow {  // of the ws: (sum of probabilities, count) [E, to an even number], tokens; 16-byte aligned
  static __host__ __device__ inline int64_t pairs(int E) { return ((int64_t)E + 1) / 2 * 2 + 2; }
};
size_t balance_ws_bytes(int64_t T, int E, int seqs) {
  if (bal_one(T)) return 256;
  const int run = bal_run(T);
  return (size_t)(T / run + seqs + 1) * BalRow::pairs(E) * 8;
}

// Largest value and sum over the G lanes of a row, in every lane: quads, rows
// of 16 by rotation, the wave's four rows through scalar registers.
template <int CTRL>
__device__ inline float dpp_move(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}
template <int G>
__device__ inline float group_max(float v) {
  v = fmaxf(v, dpp_move<0xB1>(v));
  v = fmaxf(v, dpp_move<0x4E>(v));
  if constexpr (G >= 16) {
    v = fmaxf(v, dpp_move<0x124>(v));
    v = fmaxf(v, dpp_move<0x128>(v));
  }
  if constexpr (G == 64)
    v = fmaxf(fmaxf(lane_float(v, 0), lane_float(v, 16)), fmaxf(lane_float(v, 32), lane_float(v, 48)));
  return v;
}
template <int G>
__device__ inline float group_sum(float v) {
  if constexpr (G == 64) return wave_sum(v);
  v += dpp_move<0xB1>(v);
  v += dpp_move<0x4E>(v);
  if constexpr (G >= 16) {
    v += dpp_move<0x124>(v);
    v += dpp_move<0x128>(v);
  }
  return v;
}
// Lane J's value of the row, in all of its lanes (16 or 64 of them).
template <int G, int J>
__device__ inline int group_lane(int v) {
  if constexpr (G == 64) return __builtin_amdgcn_readlane(v, J);
  return __builtin_amdgcn_update_dpp(0, v, 0x150 + J, 0xF, 0xF, false);  // row_newbcast:J
}

// The lane's logits of row t: elements 4 (g + G v) .. + 3; -inf past the last.
template <int G, int NV, bool BF>
struct BalZ {
  float z[NV][4];
  __device__ inline void load(const void* p, int64_t t, int E, bool vec, int g, bool on) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = 4 * (g + G * v);
#pragma unroll
      for (int i = 0; i < 4; ++i) z[v][i] = -INFINITY;
      if (!on || e >= E) continue;
      const int64_t at = t * E + e;
      if (vec) {
        if constexpr (BF) {
          const u32x2_t w = *(const u32x2_t*)((const uint16_t*)p + at);
          z[v][0] = __builtin_bit_cast(float, w.x << 16);
          z[v][1] = __builtin_bit_cast(float, w.x & 0xFFFF0000u);
          z[v][2] = __builtin_bit_cast(float, w.y << 16);
          z[v][3] = __builtin_bit_cast(float, w.y & 0xFFFF0000u);
        } else {
          const float4_t w = *(const float4_t*)((const float*)p + at);
#pragma unroll
          for (int i = 0; i < 4; ++i) z[v][i] = w[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (e + i < E) {
            if constexpr (BF) z[v][i] = __builtin_bit_cast(float, (uint32_t)((const uint16_t*)p)[at + i] << 16);
            else z[v][i] = ((const float*)p)[at + i];
          }
      }
    }
  }
  // to probabilities; zeros for a row without any finite or NaN logit
  __device__ inline void softmax() {
    float m = -INFINITY;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) m = fmaxf(m, z[v][i]);
    m = group_max<G>(m);
    const float mm = m == -INFINITY ? 0.f : m;
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        z[v][i] = __expf(z[v][i] - mm);
        s += z[v][i];
      }
    s = group_sum<G>(s);
    const float r = s == 0.f ? 0.f : 1.0f / s;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) z[v][i] *= r;
  }
};

// ---------------------------------------------------------------- forward
template <int G, int NV, bool BF, bool ONE>
__global__ __launch_bounds__(kBalThreads) void k_balance(const void* __restrict__ z, int64_t T, int E, int k,
                                                         const int32_t* __restrict__ idx,
                                                         const int32_t* __restrict__ off, int seqs, int run, bool vec,
                                                         float2* __restrict__ ws, int32_t* __restrict__ counts,
                                                         int32_t* __restrict__ tokens, float* __restrict__ loss) {
  constexpr int ROWS = 64 / G, W = kBalThreads / 64, EM = 4 * G * NV;
  __shared__ float psum[W][EM];
  __shared__ int cnt[EM];
  __shared__ int lds[16];
  __shared__ int live_n[W];
  __shared__ double lsum[W];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane % G, rg = lane / G;
  RowTile rt{};
  if constexpr (ONE) {
    rt.e = blockIdx.x;
    rt.lo = off ? min(max(off[rt.e], 0), (int)T) : 0;
    rt.cnt = (off ? min(max(off[rt.e + 1], 0), (int)T) : (int)T) - rt.lo;
  } else {
    rt = find_tile(off, seqs, (int)T, run, 1, lds);
    if (rt.cnt <= 0) return;
  }
  for (int e = tid; e < EM; e += kBalThreads) cnt[e] = 0;
  __syncthreads();
  float acc[NV][4] = {};
  int live = 0;
  constexpr int U = NV == 1 ? 4 : 2;  // rows of a group in flight
  for (int t0 = wave * ROWS + rg; t0 - rg < rt.cnt; t0 += U * W * ROWS) {
    BalZ<G, NV, BF> r[U];
    int named[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + u * W * ROWS;
      r[u].load(z, rt.lo + t, E, vec, g, t < rt.cnt);
      named[u] = -1;
      if (G >= 16 && t < rt.cnt && g < k) named[u] = idx[(int64_t)(rt.lo + t) * k + g];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + u * W * ROWS;
      r[u].softmax();
      bool any = false;
      if constexpr (G >= 16) {
        any = named[u] >= 0 && named[u] < E;
        if (any) atomicAdd(&cnt[named[u]], 1);
      } else if (t < rt.cnt) {
        for (int j = g; j < k; j += G) {
          const int e = idx[(int64_t)(rt.lo + t) * k + j];
          if (e < 0 || e >= E) continue;
          any = true;
          atomicAdd(&cnt[e], 1);
        }
      }
      const uint64_t mask = (G == 64 ? ~0ull : ((1ull << (G % 64)) - 1) << (rg * G));
      const bool on = (__ballot(any) & mask) != 0;
      live += on && g == 0;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[v][i] += on ? r[u].z[v][i] : 0.f;
    }
  }
  // over the wave's rows, then over the waves
#pragma unroll
  for (int o = G; o < 64; o <<= 1) {
    live += __shfl_xor(live, o);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[v][i] += __shfl_xor(acc[v][i], o);
  }
  if (rg == 0) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) psum[wave][4 * (g + G * v) + i] = acc[v][i];
  }
  if (lane == 0) live_n[wave] = live;
  __syncthreads();
  const int n = live_n[0] + live_n[1] + live_n[2] + live_n[3];
  if constexpr (ONE) {
    double s = 0.0;
    for (int e = tid; e < E; e += kBalThreads) {
      const float p = (psum[0][e] + psum[1][e]) + (psum[2][e] + psum[3][e]);
      counts[(int64_t)rt.e * E + e] = cnt[e];
      s += (double)cnt[e] * p;
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o);
    if (lane == 0) lsum[wave] = s;
    __syncthreads();
    if (tid == 0) {
      tokens[rt.e] = n;
      loss[rt.e] = n ? (float)((lsum[0] + lsum[1] + lsum[2] + lsum[3]) * E / ((double)k * n * n)) : 0.f;
    }
  } else {
    // run i of sequence b has row lo / run + b: ascending, and no two alike
    float2* row = ws + (int64_t)(rt.lo / run + rt.e) * BalRow::pairs(E);
    for (int e = tid; e < E; e += kBalThreads)
      row[e] = float2{(psum[0][e] + psum[1][e]) + (psum[2][e] + psum[3][e]), __builtin_bit_cast(float, cnt[e])};
    if (tid == 0) row[BalRow::pairs(E) - 1].x = __builtin_bit_cast(float, n);
  }
}

// A block joins the runs of a sequence: two experts to a thread, cb threads (a
// power of two) to a run, 1024 / cb runs at a time.
__global__ __launch_bounds__(1024) void k_balance_join(const float2* __restrict__ ws, int T, int E, int cb, int k,
                                                       const int32_t* __restrict__ off, int run,
                                                       int32_t* __restrict__ counts, int32_t* __restrict__ tokens,
                                                       float* __restrict__ loss) {
  __shared__ double sums[2][1024];
  __shared__ int cnts[2][1024];
  __shared__ double lsum[16];
  __shared__ int ltok[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, b = blockIdx.x;
  const int col = tid & (cb - 1), share = tid / cb, shares = 1024 / cb;
  const int lo = off ? min(max(off[b], 0), T) : 0, hi = off ? min(max(off[b + 1], 0), T) : T;
  const int runs = hi > lo ? (hi - lo + run - 1) / run : 0;
  const int64_t pairs = BalRow::pairs(E);
  const float2* row = ws + (int64_t)(lo / run + b) * pairs;
  double p0 = 0.0, p1 = 0.0;
  int c0 = 0, c1 = 0, n = 0;
  if (tid < runs) n = __builtin_bit_cast(int, row[tid * pairs + pairs - 1].x);
  for (int i = tid + 1024; i < runs; i += 1024) n += __builtin_bit_cast(int, row[i * pairs + pairs - 1].x);
  if (2 * col < E) {
    constexpr int U = 8;
    for (int i0 = share; i0 < runs; i0 += U * shares) {
      float4_t v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {  // (a run's second may be past the last expert)
        const int i = i0 + u * shares;
        v[u] = float4_t{0.f, 0.f, 0.f, 0.f};
        if (i < runs) v[u] = *(const float4_t*)(row + i * pairs + 2 * col);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float n0 = v[u].y, n1 = v[u].w;  // (a bit cast of an element would take the vector's first)
        p0 += v[u].x;
        c0 += __builtin_bit_cast(int, n0);
        p1 += v[u].z;
        c1 += __builtin_bit_cast(int, n1);
      }
    }
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) n += __shfl_xor(n, o);
  if (lane == 0) ltok[wave] = n;
  sums[0][tid] = p0;
  sums[1][tid] = p1;
  cnts[0][tid] = c0;
  cnts[1][tid] = c1;
  __syncthreads();
  for (int o = 512; o >= cb; o >>= 1) {
    if (tid < o) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        sums[q][tid] += sums[q][tid + o];
        cnts[q][tid] += cnts[q][tid + o];
      }
    }
    __syncthreads();
  }
  double s = 0.0;
  if (tid < cb) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (2 * tid + q >= E) continue;
      counts[(int64_t)b * E + 2 * tid + q] = cnts[q][tid];
      s += cnts[q][tid] * sums[q][tid];
    }
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o);
  if (lane == 0) lsum[wave] = s;
  __syncthreads();
  if (tid != 0) return;
  s = 0.0;
  n = 0;
  for (int i = 0; i < 16; ++i) {
    s += lsum[i];
    n += ltok[i];
  }
  tokens[b] = n;
  loss[b] = n ? (float)(s * E / ((double)k * n * n)) : 0.f;
}

// ---------------------------------------------------------------- backward
// The number of sequences that end at or before token t, by a search of 64
// places at a time.
__device__ inline int ends_before(const int32_t* __restrict__ off, int seqs, int t, int lane) {
  int lo = 0, hi = seqs;  // the answer lies in lo .. hi
  while (hi - lo > 0) {
    const int step = (hi - lo + 63) / 64;
    const int at = lo + (lane + 1) * step;  // off[at] <= t: at least `at` of them
    const bool yes = at <= hi && off[at] <= t;
    const int more = __popcll(__ballot(yes));
    lo += more * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

template <int G, int NV, bool BF>
// (z and dz may be one: a wave reads its rows before it writes them)
__global__ __launch_bounds__(kBalThreads) void k_balance_grad(const void* z, int T, int E, int k,
                                                              const int32_t* __restrict__ idx,
                                                              const int32_t* __restrict__ off, int seqs, bool vec,
                                                              const int32_t* __restrict__ counts,
                                                              const int32_t* __restrict__ tokens,
                                                              const float* __restrict__ dloss,
                                                              const float* __restrict__ dslots, int run,
                                                              void* dz) {
  constexpr int ROWS = 64 / G, W = kBalThreads / 64;
  const int lane = threadIdx.x & 63, g = lane % G, rg = lane / G;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int w0 = (blockIdx.x * W + wave) * run;  // the wave's tokens: run of them, a multiple of its rows
  if (w0 >= T) return;
  constexpr int U = NV == 1 ? 2 : 1;
  const int end = min(T, w0 + run);
  BalZ<G, NV, BF> r[U];
  int named[U];
  float slot[U];
  auto load = [&](int t0) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + u * ROWS;
      r[u].load(z, t, E, vec, g, t < end);
      named[u] = -1;
      slot[u] = 0.f;
      if (G >= 16 && t < end && g < k) {
        named[u] = idx[(int64_t)t * k + g];
        if (dslots) slot[u] = dslots[(int64_t)t * k + g];
      }
    }
  };
  load(w0 + rg);  // under way while the sequence is searched for
  int b = off ? ends_before(off, seqs, w0, lane) : 0;
  // the sequence's first token, and the next one's
  int first = off && b < seqs ? off[b] : 0, next = !off ? T : b < seqs ? off[b + 1] : INT32_MAX;
  int of = -1;  // the sequence that c holds
  float c[NV][4] = {}, factor = 0.f;
  for (int t0 = w0 + rg;;) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + u * ROWS;
      const bool on = t < end;
      r[u].softmax();
      while (on && t >= next) {
        first = next;
        next = ++b < seqs ? off[b + 1] : INT32_MAX;
      }
      const bool in = on && b < seqs && t >= first;
      if (in && b != of) {
        of = b;
        const int n = tokens[b];
        factor = n > 0 ? (float)((double)(dloss ? dloss[b] : 1.0f) * E / ((double)k * n * n)) : 0.f;
        // Counts less their mean: a constant less changes nothing, since the
        // probabilities add up to one, and what is left is small and exact.
        const int mean = (int)((int64_t)k * n / E);
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = 4 * (g + G * v) + i;
            c[v][i] = e < E ? (float)(counts[(int64_t)b * E + e] - mean) : 0.f;
          }
      }
      float dot = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) dot += r[u].z[v][i] * c[v][i];
      dot = group_sum<G>(dot);
      bool any = false;
      if constexpr (G >= 16) {
        any = named[u] >= 0 && named[u] < E;
      } else if (on) {
        for (int j = g; j < k; j += G) {
          const int e = idx[(int64_t)t * k + j];
          any |= e >= 0 && e < E;
        }
      }
      const uint64_t mask = (G == 64 ? ~0ull : ((1ull << (G % 64)) - 1) << (rg * G));
      const bool live = in && (__ballot(any) & mask) != 0;
      float o[NV][4];
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[v][i] = live ? factor * r[u].z[v][i] * (c[v][i] - dot) : 0.f;
      if (dslots) {
        // (an expert out of range is no lane's, or that of places past the last)
        auto add = [&](int e, float s) __attribute__((always_inline)) {
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[v][i] += e == 4 * (g + G * v) + i ? s : 0.f;
        };
        if constexpr (G >= 16) {
          const int sb = __builtin_bit_cast(int, slot[u]);
#define DS4_SLOT(J) \
  if (J < k) add(group_lane<G, J>(named[u]), __builtin_bit_cast(float, group_lane<G, J>(sb)))
          DS4_SLOT(0); DS4_SLOT(1); DS4_SLOT(2); DS4_SLOT(3); DS4_SLOT(4); DS4_SLOT(5); DS4_SLOT(6); DS4_SLOT(7);
          if (k > 8) {
            DS4_SLOT(8); DS4_SLOT(9); DS4_SLOT(10); DS4_SLOT(11); DS4_SLOT(12); DS4_SLOT(13); DS4_SLOT(14); DS4_SLOT(15);
          }
#undef DS4_SLOT
        } else {
          for (int j = 0; j < k; ++j)
            add(on ? idx[(int64_t)t * k + j] : -1, on ? dslots[(int64_t)t * k + j] : 0.f);
        }
      }
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int e = 4 * (g + G * v);
        if (!on || e >= E) continue;
        const int64_t at = (int64_t)t * E + e;
        if (vec) {
          if constexpr (BF)
            *(u32x2_t*)((uint16_t*)dz + at) = u32x2_t{bf16_pair(o[v][0], o[v][1]), bf16_pair(o[v][2], o[v][3])};
          else
            *(float4_t*)((float*)dz + at) = float4_t{o[v][0], o[v][1], o[v][2], o[v][3]};
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (e + i < E) {
              if constexpr (BF) ((uint16_t*)dz)[at + i] = (uint16_t)bf16_pair(o[v][i], 0.f);
              else ((float*)dz)[at + i] = o[v][i];
            }
        }
      }
    }
    t0 += U * ROWS;
    if (t0 - rg >= end) break;
    load(t0);
  }
}

// ---------------------------------------------------------------- launches
static bool bal_vec(const BalanceCall& c) {
  const uintptr_t a = c.z_dt == DS4MOE_DT_BF16 ? 7 : 15;
  return c.E % 4 == 0 && (((uintptr_t)c.z | (uintptr_t)c.dz) & a) == 0;
}

template <int G, int NV, bool BF>
static hipError_t balance_fwd(const BalanceCall& c) {
  const int run = bal_run(c.T);
  if (bal_one(c.T)) {
    DS4_LAUNCH((k_balance<G, NV, BF, true>), dim3(c.seqs), dim3(kBalThreads), 0, c.st, c.z, c.T, c.E, c.k, c.idx, c.off,
               c.seqs, run, bal_vec(c), (float2*)nullptr, c.counts, c.tokens, c.loss);
    return hipGetLastError();
  }
  const int64_t blocks = max_tiles(c.T, c.seqs, c.off != nullptr, run);
  DS4_LAUNCH((k_balance<G, NV, BF, false>), dim3((unsigned)blocks), dim3(kBalThreads), 0, c.st, c.z, c.T, c.E, c.k,
             c.idx, c.off, c.seqs, run, bal_vec(c), (float2*)c.ws, c.counts, c.tokens, c.loss);
  int cb = 64;
  while (2 * cb < c.E) cb *= 2;
  DS4_LAUNCH(k_balance_join, dim3(c.seqs), dim3(1024), 0, c.st, (const float2*)c.ws, (int)c.T, c.E, cb, c.k, c.off, run,
             c.counts, c.tokens, c.loss);
  return hipGetLastError();
}
template <int G, int NV, bool BF>
static hipError_t balance_bwd(const BalanceCall& c) {
  // a wave's tokens: enough waves to fill the chip, then more tokens each, a
  // multiple of the rows that it takes at a time
  constexpr int rows = 64 / G * 2, W = kBalThreads / 64;
  const int run = (int)std::max<int64_t>(1, std::min<int64_t>(16, c.T / (rows * 8192))) * rows;
  const int64_t waves = (c.T + run - 1) / run;
  DS4_LAUNCH((k_balance_grad<G, NV, BF>), dim3((unsigned)((waves + W - 1) / W)), dim3(kBalThreads), 0, c.st, c.z,
             (int)c.T, c.E, c.k, c.idx, c.off, c.seqs, bal_vec(c), (const int32_t*)c.counts, (const int32_t*)c.tokens,
             c.dloss, c.dslots, run, c.dz);
  return hipGetLastError();
}
template <bool BF>
static hipError_t balance_call(const BalanceCall& c, bool grad) {
#define DS4_BAL(g, nv) return grad ? balance_bwd<g, nv, BF>(c) : balance_fwd<g, nv, BF>(c)
  switch (bal_lanes(c.E)) {
    case 4: DS4_BAL(4, 1);
    case 16: DS4_BAL(16, 1);
  }
  if (c.E <= 256) DS4_BAL(64, 1);
  if (c.E <= 512) DS4_BAL(64, 2);
  DS4_BAL(64, 4);
#undef DS4_BAL
}
hipError_t launch_balance(const BalanceCall& c) {
  return c.z_dt == DS4MOE_DT_BF16 ? balance_call<true>(c, false) : balance_call<false>(c, false);
}
hipError_t launch_balance_grad(const BalanceCall& c) {
  return c.z_dt == DS4MOE_DT_BF16 ? balance_call<true>(c, true) : balance_call<false>(c, true);
}

}  // namespace ds4
