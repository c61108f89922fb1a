// Internal declarations of the norms, dropout and the batched router with its balance loss,
// and their backward passes, shared with the C ABI (not installed).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "linear.h"

namespace ada {

constexpr int kMaxNorm = 32768;  // columns of a normed row: one workgroup holds it in registers
constexpr int kMaxExperts = 64;

// Elements whose 16-bit number is below `least` are dropped, the others scaled; least = 0
// drops nothing.  With `state` (device) the key is state[0] and the offset counts from state[1].
struct DropParams {
  uint32_t least;
  float scale;
  uint64_t seed;
  uint64_t offset;
  const uint64_t* state;
};

struct DropoutParams {
  MatIn x;
  MatIn res;  // null: nothing is added
  MatOut y;
  int64_t rows;
  int32_t d;
  DropParams drop;
};
hipError_t launch_dropout(const DropoutParams& p, int dtype, hipStream_t s);

// h = res + dropout(x), to hidden; y = (h - mean) rstd w + b.  Unused operands are null.
struct NormParams {
  MatIn x;
  MatIn res;
  const void* w;
  const void* b;
  MatOut y;
  MatOut hidden;
  float* mean;
  float* rstd;
  int64_t rows;
  int32_t d;
  int32_t rms;
  float eps;
  DropParams drop;
};
hipError_t launch_norm(const NormParams& p, int dtype, hipStream_t s);

// Gradients of NormParams' outputs; dx, dres, dw and db are written where they are not null.
struct NormGradParams {
  MatIn dy;
  MatIn hidden;
  MatIn dhidden;
  const void* w;
  const float* mean;  // null: rms
  const float* rstd;
  MatOut dx;
  MatOut dres;
  void* dw;
  void* db;
  int64_t rows;
  int32_t d;
  DropParams drop;
};
int64_t norm_grad_workspace(int64_t rows, int32_t d);
hipError_t launch_norm_grad(const NormGradParams& p, int dtype, void* ws, hipStream_t s);

struct RouteParams {
  MatIn logits;
  const uint8_t* valid;  // null: every row counts
  int32_t* idx;
  float* gate;
  int32_t* counts;  // the four of the balance are null together
  float* prob;
  float* loss;
  int32_t* used;
  int64_t rows;
  int32_t E;
  int32_t k;
  int32_t renorm;
  double per_pick;  // E / k, the loss's factor
};
int64_t route_workspace(int64_t rows, int32_t E);
hipError_t launch_route(const RouteParams& p, int dtype, void* ws, hipStream_t s);

struct RouteGradParams {
  MatIn logits;
  const int32_t* idx;
  const float* gate;
  const int32_t* counts;
  const int32_t* used;
  const float* dgate;  // null: no gradient of the gates
  const float* dloss;  // null: no gradient of the loss
  MatOut dlogits;
  int64_t rows;
  int32_t E;
  int32_t k;
  int32_t renorm;
};
hipError_t launch_route_grad(const RouteGradParams& p, int dtype, hipStream_t s);

}  // namespace ada
