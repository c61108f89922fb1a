// Dropout from a counter-based generator, with the residual added in the same pass:
//   y = residual + x keep / (1 - p).  The backward pass is the same on dy, with no residual.
// The mask is never stored: it is a function of (seed, offset, element), so the backward pass,
// or a norm that drops the same matrix, makes it again.
//
// Bound by memory: 2 (3 with a residual) values moved an element.  A lane takes kBlocks blocks of
// eight elements (as load_block deals them), one draw of the generator each; all loads are in flight
// before the first draw.  4096 x 28672 bf16: 78.5 us, 6.0 TB/s (with one
// round of the generator instead of ten 1 us less, so its instructions hide behind the stream);
// 4096 x 14336 fp32: 77.9 us (with each lane's eight in a row 85.4).
#include "elements.h"

namespace ada {
namespace {

constexpr int kBlocks = 4;
constexpr int kThreads = 256;

// Where block g of a matrix with row stride ld begins.  The row is g / per_row, by the reciprocal
// `inv` = ceil(2^64 / per_row) (0: per_row is 1): inv is above 2^64 / per_row by less than one, so the product
// above g / per_row by less than g / 2^64 < 2^-32, while g / per_row is below the next whole number by
// 1 / per_row >= 2^-19 or more: exact.
__device__ __forceinline__ int64_t block_at(uint64_t g, uint32_t per_row, uint64_t inv, int64_t ld) {
  const uint64_t row = inv == 0 ? g : __umul64hi(g, inv);
  return int64_t(row) * ld + int64_t(g - row * per_row) * 8;
}

// y may be x or the residual: a block's elements are read and written by one lane, reads first.
template <typename T, bool DENSE, bool RES, bool STREAM>
__global__ void __launch_bounds__(kThreads) dropout_kernel(DropoutParams p, uint64_t blocks, uint32_t per_row,
                                                           uint64_t inv) {
  constexpr int PER = kVectors<T>;
  const uint64_t first = uint64_t(blockIdx.x) * (kThreads * kBlocks);  // this workgroup's first block of eight
  const int vectors = int(min(blocks - first, uint64_t(kThreads * kBlocks))) * PER;
  const T* x = static_cast<const T*>(p.x.p);
  const T* res = static_cast<const T*>(p.res.p);
  T* y = static_cast<T*>(p.y.p);
  const DropKey key = drop_key(p.drop);
  // vector v of the workgroup's, of a matrix with row stride ld
  const auto place = [&](int v, int64_t ld) {
    if constexpr (DENSE) return int64_t(first) * 8 + int64_t(v) * kVector<T>;
    return block_at(first + v / PER, per_row, inv, ld) + v % PER * kVector<T>;
  };
  const auto fetch = [&](const T* m, int64_t ld, int u, bool whole) {
    Eight<T> e;
    zero_eight(e);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int v = vector_of<T>(threadIdx.x, kThreads, u, i);
      if (whole || v < vectors) e.v[i] = load_vector<STREAM>(reinterpret_cast<const u32x4*>(m + place(v, ld)));
    }
    return e;
  };
  const auto finish = [&](const Eight<T>& in, const Eight<T>& add, int u, bool whole) {
    float f[8];
    unpack(in, f);
    drop_block<false, T>(f, uint32_t(first), threadIdx.x, kThreads, u, key, p.drop.least, p.drop.scale);
    if constexpr (RES) {
      float r[8];
      unpack(add, r);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] += r[i];
    }
    const Eight<T> out = pack(f, T());
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int v = vector_of<T>(threadIdx.x, kThreads, u, i);
      if (whole || v < vectors) store_vector<false>(reinterpret_cast<u32x4*>(y + place(v, p.y.ld)), out.v[i]);
    }
  };
  if (vectors == kThreads * kBlocks * PER) {
    Eight<T> in[kBlocks], add[kBlocks];
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) {
      in[u] = fetch(x, p.x.ld, u, true);
      if constexpr (RES) add[u] = fetch(res, p.res.ld, u, true);
    }
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) finish(in[u], add[u], u, true);
    return;
  }
  for (int u = 0; vector_of<T>(threadIdx.x, kThreads, u, 0) < vectors; ++u) {  // the last workgroup
    Eight<T> add;
    const Eight<T> in = fetch(x, p.x.ld, u, false);
    if constexpr (RES) add = fetch(res, p.res.ld, u, false);
    finish(in, add, u, false);
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
  const bool stream = streams(p.rows * p.d);
  if (dtype == 1 && stream) return res ? launch<uint16_t, true, true>(p, s) : launch<uint16_t, false, true>(p, s);
  if (dtype == 1) return res ? launch<uint16_t, true, false>(p, s) : launch<uint16_t, false, false>(p, s);
  if (stream) return res ? launch<float, true, true>(p, s) : launch<float, false, true>(p, s);
  return res ? launch<float, true, false>(p, s) : launch<float, false, false>(p, s);
}

}  // namespace ada
