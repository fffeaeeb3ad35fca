// Internal declarations of a training step's operators: the router's balance
// loss, the cross entropy over a vocabulary and AdamW over many tensors.
// They share the typed rows and wave sums of the operators around the layer.
#pragma once

#include "../ops/ops.h"

namespace ds4 {

// ---------------------------------------------------------------- limits
constexpr int kBalMaxSeqs = 16384;         // sequences of a balance call
constexpr int64_t kXentMaxV = 1 << 20;     // words of a vocabulary
constexpr int64_t kAdamMaxN = 1ll << 40;   // values of all tensors
constexpr int kAdamMaxTensors = 1 << 20;
constexpr int64_t kAdamMaxBlocks = (1 << 15) + 2 * kAdamMaxTensors;

// ---------------------------------------------------------------- balance
struct BalanceCall {
  const void* z;
  int z_dt;
  int64_t T;
  int E, k, seqs;
  const int32_t *idx, *off;
  int32_t *counts, *tokens;
  float* loss;
  void* ws;
  const float *dloss, *dslots;
  void* dz;
  hipStream_t st;
};
size_t balance_ws_bytes(int64_t T, int E, int seqs);
hipError_t launch_balance(const BalanceCall& c);
hipError_t launch_balance_grad(const BalanceCall& c);

// ---------------------------------------------------------------- cross entropy
struct XentCall {
  const void *h, *w;
  int dt;
  int64_t T, V;
  int d;
  float scale;
  const int32_t* target;
  float *loss, *lse;         // forward
  const float *lse_in, *dloss;  // backward
  void *dh, *dw;
  uint8_t* ws;
  hipStream_t st;
};
size_t xent_ws_bytes(int dt, int64_t T, int64_t V, int d, bool grad);
hipError_t launch_xent(const XentCall& c);
hipError_t launch_xent_grad(const XentCall& c);

// ---------------------------------------------------------------- AdamW
struct AdamCall {
  ds4moe_adamw A;
  const void* table;
  int64_t step;
  const float* grad_scale;
  float max_norm;
  float* out;
  double* ws;
  hipStream_t st;
};
size_t adam_table_bytes(const ds4moe_param* p, int n);
void adam_table(ds4moe_adamw* A, const ds4moe_param* p, int n, void* table);
size_t adam_ws_bytes(const ds4moe_adamw& A);
hipError_t launch_adamw_step(const AdamCall& c);
hipError_t launch_adamw_norm(const AdamCall& c);

}  // namespace ds4
