// Tokens sorted by expert and back.
//
//   group         slots s = t k + j in order of (expert, slot): counts, exclusive
//                 offsets, perm (position -> slot) and inv (slot -> position)
//   dispatch      xs[inv[s]] = x[t]
//   combine       y[t] = base[t] + sum_j w[t, j] ys[inv[t k + j]], j ascending
//   combine_grad  dys[inv[s]] = w_s dy[t],  dw_s = sum_c dy[t] ys[inv[s]],
//                 dl_s = w_s (dw_s - sum_j w_j dw_j)
//
// A slot whose expert lies outside [0, E) has no position: inv is -1, its
// weight and rows are never read, and its gradients are zero.  The row
// kernels go by token, so a token's row is read once for all its slots, and
// no sum depends on the order in which blocks run.
#include <algorithm>

#include "../trace.h"
#include "ops.h"

namespace ds4 {

constexpr int kMaxK = 16;    // slots of a token
constexpr int kMaxE = 1024;  // experts

// ---------------------------------------------------------------- sort
// Lanes of the wave with the same key (keys below 2^bits): a mask per lane.
__device__ inline uint64_t same_key(int key, int bits) {
  uint64_t m = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const uint64_t v = __ballot((key >> b) & 1);
    m &= (key >> b) & 1 ? v : ~v;
  }
  return m;
}

// Exclusive scan of one value per thread of an NT-thread block.
template <int NT>
__device__ inline int block_scan(int v, int* tmp, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  if (lane == 63) tmp[wave] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) {
    const int s = tmp[w];
    if (w < wave) before += s;
    all += s;
  }
  __syncthreads();
  *total = all;
  return before + x - v;
}

// A chunk of slots per block, a contiguous run of 64 * PER of them per wave.
constexpr int kSortPer = 8;
constexpr int kSortT = 512;
constexpr int kSortWaves = kSortT / 64;
constexpr int kSortChunk = kSortT * kSortPer;

__device__ inline int expert_key(const int32_t* idx, int64_t s, int64_t S, int E) {
  if (s >= S) return -1;
  const int e = idx[s];
  return e >= 0 && e < E ? e : E;
}

// Slots of every expert in each chunk: hist[chunk][E].
__global__ __launch_bounds__(kSortT) void k_group_hist(const int32_t* __restrict__ idx, int64_t S, int E,
                                                       int32_t* __restrict__ hist) {
  __shared__ int cnt[kMaxE + 1];
  for (int e = threadIdx.x; e <= E; e += kSortT) cnt[e] = 0;
  __syncthreads();
  const int64_t s0 = (int64_t)blockIdx.x * kSortChunk;
#pragma unroll
  for (int u = 0; u < kSortPer; ++u) {
    const int key = expert_key(idx, s0 + u * kSortT + threadIdx.x, S, E);
    if (key >= 0) atomicAdd(&cnt[key], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kSortT) hist[(int64_t)blockIdx.x * E + e] = cnt[e];
}

// hist -> slots of the expert in earlier chunks; counts.  A block takes 16
// experts, sixteen groups of chunks each.
__global__ __launch_bounds__(256) void k_group_scan(int32_t* __restrict__ hist, int chunks, int E,
                                                    int32_t* __restrict__ counts) {
  __shared__ int part[16][17];
  const int e = blockIdx.x * 16 + (threadIdx.x & 15), g = threadIdx.x >> 4;
  const int per = (chunks + 15) / 16, c0 = min(g * per, chunks), c1 = min(c0 + per, chunks);
  int s = 0;
  if (e < E)
#pragma unroll 8
    for (int c = c0; c < c1; ++c) s += hist[(int64_t)c * E + e];
  part[g][threadIdx.x & 15] = s;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const int v = part[j][threadIdx.x & 15];
    if (j < g) before += v;
    all += v;
  }
  if (e >= E) return;
  if (g == 0) counts[e] = all;
#pragma unroll 4
  for (int c = c0; c < c1; ++c) {
    const int v = hist[(int64_t)c * E + e];
    hist[(int64_t)c * E + e] = before;
    before += v;
  }
}

// Positions of the block's chunk of slots.  The chunk's slots are ranked
// stably: each wave counts its own run, the waves' counts are added up in
// order, and each wave then goes through its run again, 64 slots at a time,
// a slot's rank among equal keys being the count of lower lanes that hold
// the same key.  ONE: there is only this chunk, and counts come from here.
// LDS holds kSortWaves counters per expert.
template <bool ONE>
__global__ __launch_bounds__(kSortT) void k_group_place(const int32_t* __restrict__ idx, int64_t S, int E, int bits,
                                                        const int32_t* __restrict__ hist,
                                                        int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
                                                        int32_t* __restrict__ perm, int32_t* __restrict__ inv) {
  extern __shared__ int lds[];
  __shared__ int tmp[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t s0 = (int64_t)blockIdx.x * kSortChunk + wave * (64 * kSortPer) + lane;
  for (int i = tid; i < kSortWaves * E; i += kSortT) lds[i] = 0;
  int key[kSortPer];
#pragma unroll
  for (int u = 0; u < kSortPer; ++u) key[u] = expert_key(idx, s0 + u * 64, S, E);
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kSortPer; ++u)
    if (key[u] >= 0 && key[u] < E) atomicAdd(&lds[wave * E + key[u]], 1);
  __syncthreads();
  // a thread takes up to two neighbouring experts: kMaxE == 2 kSortT
  static_assert(kMaxE == 2 * kSortT, "experts per thread of the scan");
  int c[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = 2 * tid + i;
    if (e >= E) continue;
    if (ONE) {
      int sum = 0;
      for (int w = 0; w < kSortWaves; ++w) {
        const int v = lds[w * E + e];
        lds[w * E + e] = sum;
        sum += v;
      }
      c[i] = sum;
      counts[e] = sum;
    } else {
      int sum = hist[(int64_t)blockIdx.x * E + e];
      for (int w = 0; w < kSortWaves; ++w) {
        const int v = lds[w * E + e];
        lds[w * E + e] = sum;
        sum += v;
      }
      c[i] = counts[e];
    }
  }
  int live;
  const int off = block_scan<kSortT>(c[0] + c[1], tmp, &live);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = 2 * tid + i, o = off + (i ? c[0] : 0);
    if (e >= E) continue;
    for (int w = 0; w < kSortWaves; ++w) lds[w * E + e] += o;
    if (blockIdx.x == 0) {
      offsets[e] = o;
      if (e == E - 1) offsets[E] = o + c[i];
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kSortPer; ++u) {
    const int64_t s = s0 + u * 64;
    // keys of lanes past the last slot match nothing that is counted
    const uint64_t m = same_key(key[u] < 0 ? E : key[u], bits);
    const int leader = __ffsll((unsigned long long)m) - 1;
    const bool mine = key[u] >= 0 && key[u] < E;
    int base = 0;
    if (mine && lane == leader) base = atomicAdd(&lds[wave * E + key[u]], __popcll(m));
    base = __shfl(base, leader);
    if (key[u] < 0) continue;
    int pos = -1;
    if (mine) {
      pos = base + __popcll(m & ((1ull << lane) - 1));
      perm[pos] = (int)s;
    }
    inv[s] = pos;
  }
  // positions without a slot
#pragma unroll
  for (int u = 0; u < kSortPer; ++u) {
    const int64_t s = s0 + u * 64;
    if (s < S && s >= live) perm[s] = -1;
  }
}

// counters of the chunks, when there is more than one
size_t group_ws_bytes(int64_t S, int E) {
  const int64_t chunks = (S + kSortChunk - 1) / kSortChunk;
  return (size_t)((chunks > 1 ? chunks * E * 4 : 0) + 256 + 255) & ~(size_t)255;
}

hipError_t launch_group(const int32_t* idx, int64_t S, int E, int32_t* counts, int32_t* offsets, int32_t* perm,
                        int32_t* inv, int32_t* ws, hipStream_t st) {
  const int chunks = (int)((S + kSortChunk - 1) / kSortChunk);
  int bits = 0;
  while ((1 << bits) <= E) ++bits;
  const size_t shmem = (size_t)kSortWaves * E * 4;
  if (chunks == 1) {
    DS4_LAUNCH(k_group_place<true>, dim3(1), dim3(kSortT), shmem, st, idx, S, E, bits, (const int32_t*)nullptr, counts,
               offsets, perm, inv);
    return hipGetLastError();
  }
  DS4_LAUNCH(k_group_hist, dim3(chunks), dim3(kSortT), 0, st, idx, S, E, ws);
  DS4_LAUNCH(k_group_scan, dim3((E + 15) / 16), dim3(256), 0, st, ws, chunks, E, counts);
  DS4_LAUNCH(k_group_place<false>, dim3(chunks), dim3(kSortT), shmem, st, idx, S, E, bits, (const int32_t*)ws, counts,
             offsets, perm, inv);
  return hipGetLastError();
}

// ---------------------------------------------------------------- rows
// Block b: token b / nb, columns 2048 (b % nb) onward, eight per thread.
template <bool BF>
__global__ __launch_bounds__(256) void k_dispatch(const void* __restrict__ x, const int32_t* __restrict__ inv, int k,
                                                  int d, int nb, int rows, void* __restrict__ xs) {
  const int64_t t = blockIdx.x / nb;
  const int c = ((blockIdx.x % nb) * 256 + threadIdx.x) * 8;
  if (c >= d) return;
  const Raw8<BF> v = ld8<BF>(x, t * d + c);
  for (int j = 0; j < k; ++j) {
    const int p = inv[t * k + j];
    if (p < 0 || p >= rows) continue;
    if constexpr (BF) {
      *(u32x4_t*)((uint16_t*)xs + (int64_t)p * d + c) = v.a;
    } else {
      float4_t* o = (float4_t*)((float*)xs + (int64_t)p * d + c);
      o[0] = v.a;
      o[1] = v.b;
    }
  }
}

// Loads of up to four slots' rows are in flight at once.
template <bool SB, bool YB>
__global__ __launch_bounds__(256) void k_combine_rows(const void* __restrict__ ys, const int32_t* __restrict__ inv,
                                                      const float* __restrict__ w, const void* base, int k, int d,
                                                      int nb, int rows, void* y) {
  const int64_t t = blockIdx.x / nb;
  const int c = ((blockIdx.x % nb) * 256 + threadIdx.x) * 8;
  if (c >= d) return;
  float acc[8] = {};
  if (base) unpack8(ld8<YB>(base, t * d + c), acc);
  for (int j0 = 0; j0 < k; j0 += 4) {
    Raw8<SB> v[4];
    float wj[4];
    bool on[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = min(j0 + u, k - 1);
      const int p = inv[t * k + j];
      on[u] = j0 + u < k && p >= 0 && p < rows;
      wj[u] = 1.0f;
      if (on[u]) {
        v[u] = ld8<SB>(ys, (int64_t)p * d + c);
        if (w) wj[u] = w[t * k + j];
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (!on[u]) continue;
      float f[8];
      unpack8(v[u], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(wj[u], f[e], acc[e]);
    }
  }
  st8<YB>(y, t * d + c, acc);
}

// One block per token: its row of dy stays in registers (NS pieces of 8
// columns per thread) while the slots' rows pass by.
template <int NS, bool YB, bool SB>
__global__ __launch_bounds__(256) void k_combine_grad(const void* __restrict__ dy, const void* ys,
                                                      const int32_t* __restrict__ inv, const float* __restrict__ w,
                                                      int k, int d, int rows, void* dys, float* __restrict__ dw,
                                                      float* __restrict__ dl) {
  __shared__ float red[kMaxK][4];
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, d8 = d / 8;
  float g[NS][8];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int i = tid + s * 256;
    if (i < d8) {
      unpack8(ld8<YB>(dy, t * d + 8 * i), g[s]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) g[s][e] = 0.f;
    }
  }
  for (int j = 0; j < k; ++j) {
    const int p = inv[t * k + j];
    float dot = 0.f;
    if (p >= 0 && p < rows) {
      const float wj = w ? w[t * k + j] : 1.0f;
      Raw8<SB> v[NS];
#pragma unroll
      for (int s = 0; s < NS; ++s) v[s] = ld8<SB>(ys, (int64_t)p * d + 8 * min(tid + s * 256, d8 - 1));
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        float f[8];
        unpack8(v[s], f);
        if (tid + s * 256 < d8) {
#pragma unroll
          for (int e = 0; e < 8; ++e) dot = fmaf(g[s][e], f[e], dot);
          if (dys) {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = wj * g[s][e];
            st8<SB>(dys, (int64_t)p * d + 8 * (tid + s * 256), f);
          }
        }
      }
    }
    dot = wave_sum(dot);
    if ((tid & 63) == 0) red[j][tid >> 6] = dot;
  }
  __syncthreads();
  if (tid < k) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) v += red[tid][i];
    if (dw) dw[t * k + tid] = v;
    red[tid][0] = v;
  }
  if (!dl) return;
  __syncthreads();
  if (tid < k) {
    float mean = 0.f, mine = 0.f;
    for (int j = 0; j < k; ++j) {
      const int p = inv[t * k + j];
      const float wj = p >= 0 && p < rows ? (w ? w[t * k + j] : 1.0f) : 0.f;
      mean = fmaf(wj, red[j][0], mean);
      if (j == tid) mine = wj;
    }
    const int p = inv[t * k + tid];
    dl[t * k + tid] = p >= 0 && p < rows ? mine * (red[tid][0] - mean) : 0.f;
  }
}

// ---------------------------------------------------------------- launchers
static bool bf(int dt) { return dt == DS4MOE_DT_BF16; }

hipError_t launch_dispatch(const void* x, int dt, int64_t T, int k, int d, const int32_t* inv, void* xs, int64_t rows,
                           hipStream_t st) {
  const int nb = (d + 2047) / 2048;
  const dim3 grid((unsigned)(T * nb));
  if (bf(dt))
    DS4_LAUNCH(k_dispatch<true>, grid, dim3(256), 0, st, x, inv, k, d, nb, (int)rows, xs);
  else
    DS4_LAUNCH(k_dispatch<false>, grid, dim3(256), 0, st, x, inv, k, d, nb, (int)rows, xs);
  return hipGetLastError();
}

hipError_t launch_combine(const void* ys, int ys_dt, int64_t rows, const int32_t* inv, const float* w,
                          const void* base, int64_t T, int k, int d, void* y, int y_dt, hipStream_t st) {
  const int nb = (d + 2047) / 2048;
  const dim3 grid((unsigned)(T * nb));
#define DS4_COMBINE(SB, YB) \
  DS4_LAUNCH((k_combine_rows<SB, YB>), grid, dim3(256), 0, st, ys, inv, w, base, k, d, nb, (int)rows, y)
  if (bf(ys_dt)) {
    if (bf(y_dt)) DS4_COMBINE(true, true);
    else DS4_COMBINE(true, false);
  } else {
    if (bf(y_dt)) DS4_COMBINE(false, true);
    else DS4_COMBINE(false, false);
  }
#undef DS4_COMBINE
  return hipGetLastError();
}

template <int NS>
static hipError_t combine_grad_steps(const void* dy, int dy_dt, const void* ys, int ys_dt, int64_t rows,
                                     const int32_t* inv, const float* w, int64_t T, int k, int d, void* dys, float* dw,
                                     float* dl, hipStream_t st) {
  const dim3 grid((unsigned)T);
#define DS4_CGRAD(YB, SB) \
  DS4_LAUNCH((k_combine_grad<NS, YB, SB>), grid, dim3(256), 0, st, dy, ys, inv, w, k, d, (int)rows, dys, dw, dl)
  if (bf(dy_dt)) {
    if (bf(ys_dt)) DS4_CGRAD(true, true);
    else DS4_CGRAD(true, false);
  } else {
    if (bf(ys_dt)) DS4_CGRAD(false, true);
    else DS4_CGRAD(false, false);
  }
#undef DS4_CGRAD
  return hipGetLastError();
}

hipError_t launch_combine_grad(const void* dy, int dy_dt, const void* ys, int ys_dt, int64_t rows, const int32_t* inv,
                               const float* w, int64_t T, int k, int d, void* dys, float* dw, float* dl,
                               hipStream_t st) {
  const int n = (d + 2047) / 2048;
  if (n <= 1) return combine_grad_steps<1>(dy, dy_dt, ys, ys_dt, rows, inv, w, T, k, d, dys, dw, dl, st);
  if (n <= 2) return combine_grad_steps<2>(dy, dy_dt, ys, ys_dt, rows, inv, w, T, k, d, dys, dw, dl, st);
  if (n <= 4) return combine_grad_steps<4>(dy, dy_dt, ys, ys_dt, rows, inv, w, T, k, d, dys, dw, dl, st);
  return combine_grad_steps<8>(dy, dy_dt, ys, ys_dt, rows, inv, w, T, k, d, dys, dw, dl, st);
}

}  // namespace ds4
