// Internal declarations of the linear and gated feed-forward products and their
// backward passes, shared with the C ABI (not installed).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ada {

// A row-major matrix of the storage type: element (i, j) at p[i * ld + j].
struct MatIn {
  const void* p;
  int64_t ld;
};
struct MatOut {
  void* p;
  int64_t ld;
};

// z = x w^T + bias; y = act(z) + res; z to pre.  Unused operands are null.  With `gated`,
// z_h = x w[h]^T + bias[h] for h = 0 (gate), 1 (up), y = act(z_0) z_1 and z_h to pre[h].
struct LinearParams {
  MatIn x;
  MatIn w[2];
  const void* bias[2];
  MatIn res;
  MatOut y;
  MatOut pre[2];
  int64_t rows;
  int32_t d_out;
  int32_t d_in;
  int32_t act;
  int32_t gated;
};

// Gradients of LinearParams' products given dy and the saved pre; dx, dw and dbias are
// written where they are not null.
struct LinearGradParams {
  MatIn dy;
  MatIn x;
  MatIn w[2];
  MatIn pre[2];
  MatOut dx;
  MatOut dw[2];
  void* dbias[2];
  int64_t rows;
  int32_t d_out;
  int32_t d_in;
  int32_t act;
  int32_t gated;
};

// Device bytes a launch needs for its intermediates (0: none).
int64_t linear_workspace(int64_t rows, int32_t d_out, int32_t d_in, int gated, int dtype);
int64_t linear_grad_workspace(int64_t rows, int32_t d_out, int32_t d_in, int act, int gated, int dtype);

hipError_t launch_linear(const LinearParams& p, int dtype, void* ws, hipStream_t s);
hipError_t launch_linear_grad(const LinearGradParams& p, int dtype, void* ws, hipStream_t s);

}  // namespace ada
