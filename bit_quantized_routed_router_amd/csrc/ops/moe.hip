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
// no sum depends on the order in which blocks run.  They are bound by memory:
// 2048 tokens of 4096, 6 slots each: dispatch 117 MB in 21 us (5.5 TB/s),
// combine 168 MB in 31 us (5.4 TB/s); combine_grad in fp32 (1021 tokens of
// 2048, 4 slots) 72 MB in 13 us (5.5 TB/s).  A 4 GB copy moves 4.5 TB/s, one
// of 128 MB, which the last-level cache holds, 6.8.
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

__device__ inline int expert_key(const int32_t* idx, int64_t s, int64_t S, int E) {
  if (s >= S) return -1;
  const int e = idx[s];
  return e >= 0 && e < E ? e : E;
}

// Slots that one block sorts by itself, with one wave or sixteen, and those
// of a chunk when there are more.
constexpr int kSortWaveT = 64, kSortWavePer = 8;
constexpr int kSortBlockT = 1024, kSortBlockPer = 4;
constexpr int kSortChunkT = 512, kSortChunkPer = 4;
constexpr int kSortChunk = kSortChunkT * kSortChunkPer;
constexpr int kSortFew = 32;  // chunks up to which each block adds up the ones before it itself
// where k_group_place has the slots of earlier chunks from: there are none,
// the chunks' counters, or those already scanned
enum { kSortOne = 0, kSortCounted = 1, kSortScanned = 2 };

// Slots of every expert in each chunk: hist[chunk][E].
__global__ __launch_bounds__(kSortChunkT) void k_group_hist(const int32_t* __restrict__ idx, int64_t S, int E,
                                                            int32_t* __restrict__ hist) {
  __shared__ int cnt[kMaxE + 1];
  for (int e = threadIdx.x; e <= E; e += kSortChunkT) cnt[e] = 0;
  __syncthreads();
  const int64_t s0 = (int64_t)blockIdx.x * kSortChunk;
#pragma unroll
  for (int u = 0; u < kSortChunkPer; ++u) {
    const int key = expert_key(idx, s0 + u * kSortChunkT + threadIdx.x, S, E);
    if (key >= 0) atomicAdd(&cnt[key], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kSortChunkT) hist[(int64_t)blockIdx.x * E + e] = cnt[e];
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

// Positions of the block's slots, stable.  Each wave takes a contiguous run,
// 64 slots at a time in order: the lanes with a key find each other by
// ballots, their first one adds their number to the wave's counter of the key
// and so learns how many of the run came before.  The counters are then added
// up over the waves and scanned over the experts, and a slot's position is
// its wave's start for the key plus its place in the run.  EP: experts of a
// thread in the scan.  Dynamic LDS: a counter per wave and expert.
template <int NT, int PER, int EP, int FROM>
__global__ __launch_bounds__(NT) void k_group_place(const int32_t* __restrict__ idx, int64_t S, int E, int bits,
                                                    const int32_t* __restrict__ hist, int chunks,
                                                    int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
                                                    int32_t* __restrict__ perm, int32_t* __restrict__ inv) {
  constexpr int NW = NT / 64;
  extern __shared__ int lds[];
  __shared__ int tmp[NW];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t c0 = (int64_t)blockIdx.x * (NT * PER), c1 = min(c0 + NT * PER, S);
  const int steps = (int)((c1 - c0 + NT - 1) / NT);  // 64 slots of every wave each
  const int64_t s0 = c0 + wave * (64 * steps) + lane;
  int key[PER], place[PER];
#pragma unroll
  for (int u = 0; u < PER; ++u) key[u] = u < steps ? expert_key(idx, s0 + u * 64, c1, E) : -1;
  // the expert's slots in earlier chunks, and in all
  int earlier[EP], total[EP];
#pragma unroll
  for (int i = 0; i < EP; ++i) {
    const int e = EP * tid + i;
    earlier[i] = total[i] = 0;
    if (FROM == kSortScanned && e < E) {
      earlier[i] = hist[(int64_t)blockIdx.x * E + e];
      total[i] = counts[e];
    }
    if (FROM == kSortCounted && e < E) {
#pragma unroll 8
      for (int c = 0; c < chunks; ++c) {
        const int v = hist[c * E + e];
        if (c < (int)blockIdx.x) earlier[i] += v;
        total[i] += v;
      }
    }
  }
  for (int i = tid; i < NW * E; i += NT) lds[i] = 0;
  __syncthreads();
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    if (u < steps) {
      // lanes past the last slot join those without an expert
      const uint64_t m = same_key(key[u] < 0 ? E : key[u], bits);
      const int leader = __ffsll((unsigned long long)m) - 1;
      int before = 0;
      if (lane == leader && key[u] >= 0 && key[u] < E) before = atomicAdd(&lds[wave * E + key[u]], __popcll(m));
      place[u] = __shfl(before, leader) + __popcll(m & ((1ull << lane) - 1));
    }
  }
  __syncthreads();
  // a thread takes EP neighbouring experts
  int v[EP][NW], sum = 0;
#pragma unroll
  for (int i = 0; i < EP; ++i) {
    const int e = EP * tid + i;
    if (e < E) {
      int all = 0;
#pragma unroll
      for (int w = 0; w < NW; ++w) v[i][w] = lds[w * E + e];
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const int x = v[i][w];
        v[i][w] = all;
        all += x;
      }
      if (FROM == kSortOne) total[i] = all;
      if (FROM != kSortScanned && blockIdx.x == 0) counts[e] = total[i];
    }
    sum += total[i];
  }
  int live, off = block_scan<NT>(sum, tmp, &live);
#pragma unroll
  for (int i = 0; i < EP; ++i) {
    const int e = EP * tid + i;
    if (e < E) {
#pragma unroll
      for (int w = 0; w < NW; ++w) lds[w * E + e] = off + earlier[i] + v[i][w];
      if (blockIdx.x == 0) {
        offsets[e] = off;
        if (e == E - 1) offsets[E] = off + total[i];
      }
    }
    off += total[i];
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int64_t s = s0 + u * 64;
    if (key[u] >= 0) {
      int pos = -1;
      if (key[u] < E) {
        pos = lds[wave * E + key[u]] + place[u];
        perm[pos] = (int)s;
      }
      inv[s] = pos;
      if (s >= live) perm[s] = -1;  // positions without a slot
    }
  }
}

// counters of the chunks, when there is more than one
static bool sorts_alone(int64_t S) { return S <= kSortBlockT * kSortBlockPer; }
size_t group_ws_bytes(int64_t S, int E) {
  const int64_t chunks = sorts_alone(S) ? 0 : (S + kSortChunk - 1) / kSortChunk;
  return (size_t)(chunks * E * 4 + 256 + 255) & ~(size_t)255;
}

// Kernel times: 96 slots of 256 experts 3.7 us with one wave (7.4 with eight);
// 4084 slots of 64 experts 7.5 us with sixteen; 12288 slots of 256 experts 4.7
// + 7.7 us in two launches (one block of sixteen waves: 21.8, bound by its one
// CU; scanning in a launch of its own: 17 in three).
hipError_t launch_group(const int32_t* idx, int64_t S, int E, int32_t* counts, int32_t* offsets, int32_t* perm,
                        int32_t* inv, int32_t* ws, hipStream_t st) {
  int bits = 0;
  while ((1 << bits) <= E) ++bits;
#define DS4_PLACE(NT, PER, EP, FROM, blocks, hist, chunks)                                                     \
  DS4_LAUNCH((k_group_place<NT, PER, EP, FROM>), dim3(blocks), dim3(NT), (size_t)(NT / 64) * E * 4, st, idx, S, E, \
             bits, (const int32_t*)(hist), chunks, counts, offsets, perm, inv)
  if (S <= kSortWaveT * kSortWavePer) {
    if (E <= 4 * kSortWaveT) DS4_PLACE(kSortWaveT, kSortWavePer, 4, kSortOne, 1, nullptr, 1);
    else DS4_PLACE(kSortWaveT, kSortWavePer, kMaxE / kSortWaveT, kSortOne, 1, nullptr, 1);
    return hipGetLastError();
  }
  if (sorts_alone(S)) {
    DS4_PLACE(kSortBlockT, kSortBlockPer, kMaxE / kSortBlockT, kSortOne, 1, nullptr, 1);
    return hipGetLastError();
  }
  const int chunks = (int)((S + kSortChunk - 1) / kSortChunk);
  DS4_LAUNCH(k_group_hist, dim3(chunks), dim3(kSortChunkT), 0, st, idx, S, E, ws);
  if (chunks <= kSortFew) {
    if (E <= kSortChunkT) DS4_PLACE(kSortChunkT, kSortChunkPer, 1, kSortCounted, chunks, ws, chunks);
    else DS4_PLACE(kSortChunkT, kSortChunkPer, kMaxE / kSortChunkT, kSortCounted, chunks, ws, chunks);
    return hipGetLastError();
  }
  DS4_LAUNCH(k_group_scan, dim3((E + 15) / 16), dim3(256), 0, st, ws, chunks, E, counts);
  DS4_PLACE(kSortChunkT, kSortChunkPer, kMaxE / kSortChunkT, kSortScanned, chunks, ws, chunks);
#undef DS4_PLACE
  return hipGetLastError();
}

// ---------------------------------------------------------------- rows
// Block b: token b / nb, columns 2048 (b % nb) onward, eight per thread.
template <bool BF>
__global__ __launch_bounds__(256) void k_dispatch(const void* __restrict__ x, const int32_t* __restrict__ inv, int k,
                                                  int d, int nb, int rows, void* __restrict__ xs) {
  const int64_t t = blockIdx.x / nb;
  const int c = ((blockIdx.x % nb) * 256 + threadIdx.x) * 8;
  const int pos = slot_positions(inv, t, k, rows);
  if (c >= d) return;  // (whole waves or their upper lanes, so lanes 0 .. 15 stay: d is a multiple of 256)
  const Raw8<BF> v = ld8<BF>(x, t * d + c);
  for (int j = 0; j < k; ++j) {
    const int p = __builtin_amdgcn_readlane(pos, j);
    if (p < 0) continue;
    if constexpr (BF) {
      *(u32x4_t*)((uint16_t*)xs + (int64_t)p * d + c) = v.a;
    } else {
      float4_t* o = (float4_t*)((float*)xs + (int64_t)p * d + c);
      o[0] = v.a;
      o[1] = v.b;
    }
  }
}

// The rows of up to eight slots are in flight at once.
template <bool SB, bool YB>
__global__ __launch_bounds__(256) void k_combine_rows(const void* __restrict__ ys, const int32_t* __restrict__ inv,
                                                      const float* __restrict__ w, const void* base, int k, int d,
                                                      int nb, int rows, void* y) {
  constexpr int B = 8;
  const int64_t t = blockIdx.x / nb;
  const int c = ((blockIdx.x % nb) * 256 + threadIdx.x) * 8;
  const int pos = slot_positions(inv, t, k, rows);
  float weight = 1.0f;
  if (w && pos >= 0) weight = w[t * k + min((int)(threadIdx.x & 63), k - 1)];
  if (c >= d) return;
  float acc[8] = {};
  if (base) unpack8(ld8<YB>(base, t * d + c), acc);
  for (int j0 = 0; j0 < k; j0 += B) {
    Raw8<SB> v[B];
    bool on[B];
#pragma unroll
    for (int u = 0; u < B; ++u) {
      const int p = __builtin_amdgcn_readlane(pos, min(j0 + u, k - 1));
      on[u] = j0 + u < k && p >= 0;
      if (on[u]) v[u] = ld8<SB>(ys, (int64_t)p * d + c);
    }
#pragma unroll
    for (int u = 0; u < B; ++u) {
      if (!on[u]) continue;
      const float wj = lane_float(weight, j0 + u);
      float f[8];
      unpack8(v[u], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(wj, f[e], acc[e]);
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
