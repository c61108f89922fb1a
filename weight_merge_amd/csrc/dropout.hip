// Dropout from a counter-based generator, with the residual added in the same pass:
//   y = residual + x keep / (1 - p).  The backward pass is the same on dy, with no residual.
// The mask is never stored: it is a function of (seed, offset, element), so the backward pass,
// or a norm that drops the same matrix, makes it again.
//
// Bound by memory: 2 (3 with a residual) values moved an element.  A lane takes blocks of eight
// elements, one 16-byte vector in bf16 and one draw of the generator; kBlocks of them a workgroup
// apart, all loads in flight before the first draw.  4096 x 28672 bf16: 78.5 us, 6.0 TB/s (with one
// round of the generator instead of ten 1 us less, so its instructions hide behind the stream).
#include "elements.h"

namespace ada {
namespace {

constexpr int kBlocks = 4;
constexpr int kThreads = 256;

// Where block g of a matrix with row stride ld begins.  DENSE: rows follow each other.
// Otherwise the row is g / per_row, by the reciprocal `inv` = ceil(2^64 / per_row) (0: per_row
// is 1): exact, for its error, below g per_row / 2^64, stays under 1 / per_row with g < 2^32 and
// per_row <= 2^19.
template <bool DENSE>
__device__ __forceinline__ int64_t block_at(uint64_t g, uint32_t per_row, uint64_t inv, int64_t ld) {
  if constexpr (DENSE) return int64_t(g) * 8;
  const uint64_t row = inv == 0 ? g : __umul64hi(g, inv);
  return int64_t(row) * ld + int64_t(g - row * per_row) * 8;
}

// y may be x or the residual: a block's elements are read and written by one lane, reads first.
template <typename T, bool DENSE, bool RES, bool STREAM>
__global__ void __launch_bounds__(kThreads) dropout_kernel(DropoutParams p, uint64_t blocks, uint32_t per_row,
                                                           uint64_t inv) {
  const uint64_t g0 = uint64_t(blockIdx.x) * (kThreads * kBlocks) + threadIdx.x;
  const T* x = static_cast<const T*>(p.x.p);
  const T* res = static_cast<const T*>(p.res.p);
  T* y = static_cast<T*>(p.y.p);
  const DropKey key = drop_key(p.drop);
  const auto one = [&](uint64_t g, const Eight<T>& in, const Eight<T>& add) {
    float f[8];
    unpack(in, f);
    drop_eight(f, uint32_t(g), key, p.drop.least, p.drop.scale);
    if constexpr (RES) {
      float r[8];
      unpack(add, r);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] += r[i];
    }
    store_eight(y + block_at<DENSE>(g, per_row, inv, p.y.ld), f);
  };
  if (uint64_t(blockIdx.x + 1) * (kThreads * kBlocks) <= blocks) {
    Eight<T> in[kBlocks], add[kBlocks];
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) {
      const uint64_t g = g0 + u * kThreads;
      in[u] = load_eight<STREAM>(x + block_at<DENSE>(g, per_row, inv, p.x.ld));
      if constexpr (RES) add[u] = load_eight<STREAM>(res + block_at<DENSE>(g, per_row, inv, p.res.ld));
    }
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) one(g0 + u * kThreads, in[u], add[u]);
    return;
  }
  for (uint64_t g = g0; g < blocks; g += kThreads) {  // the last workgroup
    Eight<T> in, add;
    in = load_eight<STREAM>(x + block_at<DENSE>(g, per_row, inv, p.x.ld));
    if constexpr (RES) add = load_eight<STREAM>(res + block_at<DENSE>(g, per_row, inv, p.res.ld));
    one(g, in, add);
  }
}

template <typename T, bool RES, bool STREAM>
hipError_t launch(const DropoutParams& p, hipStream_t s) {
  const uint32_t per_row = uint32_t(p.d / 8);
  const uint64_t blocks = uint64_t(p.rows) * per_row;
  const bool dense = p.x.ld == p.d && p.y.ld == p.d && (!RES || p.res.ld == p.d);
  const uint64_t inv = per_row == 1 ? 0 : ~uint64_t(0) / per_row + 1;
  // at most 2^32 blocks: 2^22 workgroups
  const dim3 grid(static_cast<unsigned>((blocks + kThreads * kBlocks - 1) / (kThreads * kBlocks)));
  if (dense)
    hipLaunchKernelGGL((dropout_kernel<T, true, RES, STREAM>), grid, dim3(kThreads), 0, s, p, blocks, per_row, inv);
  else
    hipLaunchKernelGGL((dropout_kernel<T, false, RES, STREAM>), grid, dim3(kThreads), 0, s, p, blocks, per_row, inv);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const DropoutParams& p, int dtype, hipStream_t s) {
  if (p.rows == 0) return hipSuccess;
  const bool res = p.res.p != nullptr;
  if (dtype != 1) return res ? launch<float, true, false>(p, s) : launch<float, false, false>(p, s);
  if (streams(p.rows * p.d, dtype)) return res ? launch<uint16_t, true, true>(p, s) : launch<uint16_t, false, true>(p, s);
  return res ? launch<uint16_t, true, false>(p, s) : launch<uint16_t, false, false>(p, s);
}

}  // namespace ada
