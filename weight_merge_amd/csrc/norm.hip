// Layer and root-mean-square norms with the residual stream and the dropout before them, and
// their backward pass.
//
//   h = residual + dropout(x), y = (h - mean) rstd w + b over each row; "rms": mean is 0
//   dh = dhidden + rstd (t - mean(t) - xhat mean(t xhat)),  t = dy w, xhat = (h - mean) rstd
//   ("rms": without mean(t)); dresidual = dh, dx = dropout(dh), dw = sum over rows of dy xhat,
//   db = sum over rows of dy
//
// Bound by memory: every matrix is read once and written once.  A row lives in the registers of
// one group of lanes from its load to its store, in blocks of eight elements a lane: a power of
// two of lanes for rows of up to 256 elements, otherwise whole waves, whose sums meet in LDS.
#include "elements.h"

namespace ada {
namespace {

constexpr int kMaxWaves = 16;

// Lanes that share a row: `lanes` below 64 is a power of two, otherwise a multiple of 64.
struct RowShape {
  int lanes;
  int groups;  // rows in flight in one workgroup
  int chunks;  // blocks of eight elements a lane holds
};

// ---- sums over the lanes of a row ------------------------------------------------------
// N sums at once, the same on every lane of the row.  `slot` is LDS of kMaxWaves x N floats that
// nothing else uses until after the next barrier; WIDE: several waves share a row.
template <int N, bool SUB, bool WIDE>
__device__ __forceinline__ void row_totals(float (&v)[N], int lanes, float (*slot)[N]) {
  if constexpr (SUB) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = group_total(v[i], lanes);
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_total(v[i]);
  if constexpr (WIDE) {
    const int wave = threadIdx.x >> 6, per_row = lanes >> 6, first = wave / per_row * per_row;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) slot[wave][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
    for (int w = 0; w < per_row; ++w) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += slot[first + w][i];
    }
  }
}

// ---- forward ---------------------------------------------------------------------------
// One row at a time per group of lanes.  The variance is the mean square of h - m with m the
// first sum's mean, and that sum's rounding is taken out of both with the mean of h - m
// (Chan, Golub, LeVeque, "Algorithms for computing the sample variance", 1983), so rows far from
// zero keep their accuracy.  y and hidden may be x or the residual: a lane reads what it writes.
template <typename T, int CH, bool SUB, bool WIDE, bool DROP>
__global__ void __launch_bounds__(1024) norm_kernel(NormParams p, int lanes) {
  __shared__ float mean_slot[kMaxWaves][1];
  __shared__ float square_slot[kMaxWaves][2];
  const int group = threadIdx.x / lanes, lane = threadIdx.x - group * lanes, groups = blockDim.x / lanes;
  const int per_row = p.d >> 3;
  const T* w = static_cast<const T*>(p.w);
  const T* b = static_cast<const T*>(p.b);
  const float over = 1.f / float(p.d);
  DropKey key{};
  if constexpr (DROP) key = drop_key(p.drop);

  for (int64_t row0 = int64_t(blockIdx.x) * groups; row0 < p.rows; row0 += int64_t(gridDim.x) * groups) {
    const bool live = row0 + group < p.rows;
    const int64_t row = live ? row0 + group : p.rows - 1;
    const T* x = static_cast<const T*>(p.x.p) + row * p.x.ld;
    const T* res = static_cast<const T*>(p.res.p) + row * p.res.ld;
    T* y = static_cast<T*>(p.y.p) + row * p.y.ld;
    T* hidden = static_cast<T*>(p.hidden.p) + row * p.hidden.ld;
    Eight<T> in[CH], add[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int g = lane + c * lanes;
      zero_eight(in[c]);
      zero_eight(add[c]);
      if (g < per_row) {
        in[c] = load_eight(x + g * 8);
        if (p.res.p != nullptr) add[c] = load_eight(res + g * 8);
      }
    }
    float h[CH][8], sum[1] = {0.f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float r[8];
      unpack(in[c], h[c]);
      if constexpr (DROP)
        drop_eight(h[c], uint32_t(row * per_row + lane + c * lanes), key, p.drop.least, p.drop.scale);
      unpack(add[c], r);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (p.res.p != nullptr) h[c][i] += r[i];
        sum[0] += h[c][i];
      }
    }
    float mean = 0.f, rest = 0.f;
    if (!p.rms) {
      row_totals<1, SUB, WIDE>(sum, lanes, mean_slot);
      mean = sum[0] * over;
    }
    float second[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (lane + c * lanes < per_row) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a = h[c][i] - mean;
          second[0] = fmaf(a, a, second[0]);
          second[1] += a;
        }
      }
    }
    row_totals<2, SUB, WIDE>(second, lanes, square_slot);
    float square = second[0] * over;
    if (!p.rms) {
      rest = second[1] * over;
      square -= rest * rest;
      square = square < 0.f ? 0.f : square;  // NaN stays
    }
    const float rstd = 1.f / sqrtf(square + p.eps);
    if (live) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int g = lane + c * lanes;
        if (g >= per_row) continue;
        if (p.hidden.p != nullptr) store_eight(hidden + g * 8, h[c]);
        float wv[8], bv[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          wv[i] = 1.f;
          bv[i] = 0.f;
        }
        if (w != nullptr) unpack(load_eight(w + g * 8), wv);
        if (b != nullptr) unpack(load_eight(b + g * 8), bv);
        float out[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) out[i] = fmaf((h[c][i] - mean - rest) * rstd, wv[i], bv[i]);
        store_eight(y + g * 8, out);
      }
      if (lane == 0) {
        if (p.mean != nullptr) p.mean[row] = mean + rest;
        if (p.rstd != nullptr) p.rstd[row] = rstd;
      }
    }
  }
}

// ---- backward --------------------------------------------------------------------------
// A workgroup takes every gridDim.x-th set of rows, keeps dw and db of a lane's columns in
// registers over all of them, and writes them once: part[0][block][d] and part[1][block][d], which
// norm_join_kernel sums in a fixed order.  The next row's loads are in flight while this one is
// summed where registers allow it (CH sizeof(T) <= 4); rows of more than 16384 fp32 elements are
// read again behind their sums instead of being held.  dx and dres may be dy or dhidden.
template <typename T, int CH>
struct GradRow {
  Eight<T> dy[CH], h[CH], add[CH];
  float mean, rstd;

  __device__ __forceinline__ void load(const NormGradParams& p, int64_t row, int lane, int lanes, int per_row) {
    const bool live = row < p.rows;
    const T* pdy = static_cast<const T*>(p.dy.p) + row * p.dy.ld;
    const T* ph = static_cast<const T*>(p.hidden.p) + row * p.hidden.ld;
    const T* pd = static_cast<const T*>(p.dhidden.p) + row * p.dhidden.ld;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int g = lane + c * lanes;
      zero_eight(dy[c]);
      zero_eight(h[c]);
      zero_eight(add[c]);
      if (live && g < per_row) {
        dy[c] = load_eight(pdy + g * 8);
        h[c] = load_eight(ph + g * 8);
        if (p.dhidden.p != nullptr) add[c] = load_eight(pd + g * 8);
      }
    }
    mean = live && p.mean != nullptr ? p.mean[row] : 0.f;
    rstd = live ? p.rstd[row] : 0.f;  // a row past the end adds zeros
  }
};

template <typename T, int CH, bool SUB, bool WIDE, bool DROP>
__global__ void __launch_bounds__(1024) norm_grad_kernel(NormGradParams p, int lanes, float* part) {
  constexpr bool AHEAD = CH * sizeof(T) <= 4, AGAIN = CH * sizeof(T) > 8;
  __shared__ float slot[2][kMaxWaves][2];
  extern __shared__ float meet[];  // [threads][8] where several groups of a workgroup meet
  const int group = threadIdx.x / lanes, lane = threadIdx.x - group * lanes, groups = blockDim.x / lanes;
  const int per_row = p.d >> 3;
  const float over = 1.f / float(p.d);
  DropKey key{};
  if constexpr (DROP) key = drop_key(p.drop);

  Eight<T> wraw[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    zero_eight(wraw[c]);
    if (p.w != nullptr && lane + c * lanes < per_row)
      wraw[c] = load_eight(static_cast<const T*>(p.w) + (lane + c * lanes) * 8);
  }
  float dw[CH][8], db[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[c][i] = db[c][i] = 0.f;

  GradRow<T, CH> now, next;
  const int64_t step = int64_t(gridDim.x) * groups;
  int64_t row = int64_t(blockIdx.x) * groups + group;
  now.load(p, row, lane, lanes, per_row);
  int turn = 0;
  for (int64_t row0 = row - group; row0 < p.rows; row0 += step, row += step, turn ^= 1) {
    if constexpr (AHEAD) next.load(p, row + step, lane, lanes, per_row);
    float sums[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float dy[8], h[8], w[8];
      unpack(now.dy[c], dy);
      unpack(now.h[c], h);
      unpack(wraw[c], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float t = p.w != nullptr ? dy[i] * w[i] : dy[i], xhat = (h[i] - now.mean) * now.rstd;
        sums[0] += t;
        sums[1] = fmaf(t, xhat, sums[1]);
        dw[c][i] = fmaf(dy[i], xhat, dw[c][i]);
        db[c][i] += dy[i];
      }
    }
    row_totals<2, SUB, WIDE>(sums, lanes, slot[turn]);
    const float c1 = p.mean != nullptr ? sums[0] * over : 0.f, c2 = sums[1] * over;
    if (row < p.rows && (p.dx.p != nullptr || p.dres.p != nullptr)) {
      T* dx = static_cast<T*>(p.dx.p) + row * p.dx.ld;
      T* dres = static_cast<T*>(p.dres.p) + row * p.dres.ld;
      if constexpr (AGAIN) {
        asm volatile("" ::: "memory");
        now.load(p, row, lane, lanes, per_row);
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int g = lane + c * lanes;
        if (g >= per_row) continue;
        float dy[8], h[8], w[8], add[8];
        unpack(now.dy[c], dy);
        unpack(now.h[c], h);
        unpack(wraw[c], w);
        unpack(now.add[c], add);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float t = p.w != nullptr ? dy[i] * w[i] : dy[i], xhat = (h[i] - now.mean) * now.rstd;
          h[i] = fmaf(now.rstd, t - c1 - xhat * c2, add[i]);
        }
        if (p.dres.p != nullptr) store_eight(dres + g * 8, h);
        if (p.dx.p != nullptr) {
          if constexpr (DROP) drop_eight(h, uint32_t(row * per_row + g), key, p.drop.least, p.drop.scale);
          store_eight(dx + g * 8, h);
        }
      }
    }
    if constexpr (AHEAD)
      now = next;
    else
      now.load(p, row + step, lane, lanes, per_row);
  }

  // the groups' sums meet in LDS, a block of eight columns at a time, and go to part
  for (int which = 0; which < 2; ++which) {
    if ((which == 0 ? p.dw : p.db) == nullptr) continue;
    float* to = part + (int64_t(which) * gridDim.x + blockIdx.x) * p.d;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = which == 0 ? dw[c][i] : db[c][i];
      if (groups > 1) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) meet[i * blockDim.x + threadIdx.x] = v[i];
        __syncthreads();
        if (group == 0) {
          for (int q = 1; q < groups; ++q)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += meet[i * blockDim.x + q * lanes + lane];
        }
      }
      const int g = lane + c * lanes;
      if (group == 0 && g < per_row) store_eight(to + g * 8, v);
    }
  }
}

// dw (blockIdx.y = 0) and db (1) from `parts` rows of d sums each: 64 columns a workgroup, four a
// lane, the rows dealt to 16 sets of lanes whose sums meet in LDS.
constexpr int kJoinSets = 16;
template <typename T>
__global__ void __launch_bounds__(256) norm_join_kernel(const float* part, int parts, int d, T* dw, T* db) {
  __shared__ float meet[kJoinSets][64];
  T* out = blockIdx.y == 0 ? dw : db;
  if (out == nullptr) return;
  const float* from = part + int64_t(blockIdx.y) * parts * d;
  const int quad = threadIdx.x & 15, set = threadIdx.x >> 4, col = blockIdx.x * 64 + quad * 4;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  if (col < d) {
    for (int r = set; r < parts; r += kJoinSets) {
      const float4 f = *reinterpret_cast<const float4*>(from + int64_t(r) * d + col);
      v[0] += f.x;
      v[1] += f.y;
      v[2] += f.z;
      v[3] += f.w;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) meet[set][quad * 4 + i] = v[i];
  __syncthreads();
  const int c = blockIdx.x * 64 + threadIdx.x;
  if (threadIdx.x < 64 && c < d) {
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < kJoinSets; ++q) sum += meet[q][threadIdx.x];
    if constexpr (sizeof(T) == 2)
      out[c] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(sum));
    else
      out[c] = sum;
  }
}

// ---- rules on sizes --------------------------------------------------------------------
int round64(int v) { return (v + 63) / 64 * 64; }

RowShape row_shape(int d, int threads) {
  const int per_row = d / 8;
  RowShape s{};
  s.chunks = per_row <= 1024 ? 1 : per_row <= 2048 ? 2 : 4;
  if (per_row <= 32) {
    s.lanes = 1;
    while (s.lanes < per_row) s.lanes *= 2;
  } else {
    s.lanes = round64((per_row + s.chunks - 1) / s.chunks);
  }
  s.groups = s.lanes < threads ? threads / s.lanes : 1;
  return s;
}

int norm_grad_blocks(int64_t rows, int d) {
  const RowShape s = row_shape(d, 512);
  const int64_t sets = (rows + s.groups - 1) / s.groups;
  return static_cast<int>(sets < 256 ? sets : 256);
}

template <typename T, int CH, bool DROP>
hipError_t forward(const NormParams& p, const RowShape& r, hipStream_t s) {
  const int64_t sets = (p.rows + r.groups - 1) / r.groups;
  const dim3 grid(static_cast<unsigned>(sets < (1 << 20) ? sets : 1 << 20)), block(r.lanes * r.groups);
  if (r.lanes < 64)
    hipLaunchKernelGGL((norm_kernel<T, CH, true, false, DROP>), grid, block, 0, s, p, r.lanes);
  else if (r.lanes == 64)
    hipLaunchKernelGGL((norm_kernel<T, CH, false, false, DROP>), grid, block, 0, s, p, r.lanes);
  else
    hipLaunchKernelGGL((norm_kernel<T, CH, false, true, DROP>), grid, block, 0, s, p, r.lanes);
  return hipGetLastError();
}

template <typename T, bool DROP>
hipError_t forward(const NormParams& p, hipStream_t s) {
  const RowShape r = row_shape(p.d, 256);
  if (r.chunks == 1) return forward<T, 1, DROP>(p, r, s);
  if (r.chunks == 2) return forward<T, 2, DROP>(p, r, s);
  return forward<T, 4, DROP>(p, r, s);
}

template <typename T, int CH, bool DROP>
hipError_t backward(const NormGradParams& p, const RowShape& r, int blocks, float* part, hipStream_t s) {
  const dim3 grid(blocks), block(r.lanes * r.groups);
  const size_t meet = r.groups > 1 ? size_t(r.lanes) * r.groups * 8 * sizeof(float) : 0;
  if (r.lanes < 64)
    hipLaunchKernelGGL((norm_grad_kernel<T, CH, true, false, DROP>), grid, block, meet, s, p, r.lanes, part);
  else if (r.lanes == 64)
    hipLaunchKernelGGL((norm_grad_kernel<T, CH, false, false, DROP>), grid, block, meet, s, p, r.lanes, part);
  else
    hipLaunchKernelGGL((norm_grad_kernel<T, CH, false, true, DROP>), grid, block, meet, s, p, r.lanes, part);
  return hipGetLastError();
}

template <typename T, bool DROP>
hipError_t backward(const NormGradParams& p, float* part, hipStream_t s) {
  const RowShape r = row_shape(p.d, 512);
  const int blocks = norm_grad_blocks(p.rows, p.d);
  hipError_t e = hipSuccess;
  if (p.rows > 0)
    e = r.chunks == 1   ? backward<T, 1, DROP>(p, r, blocks, part, s)
        : r.chunks == 2 ? backward<T, 2, DROP>(p, r, blocks, part, s)
                        : backward<T, 4, DROP>(p, r, blocks, part, s);
  if (e != hipSuccess || (p.dw == nullptr && p.db == nullptr)) return e;
  hipLaunchKernelGGL(norm_join_kernel<T>, dim3((p.d + 63) / 64, 2), dim3(256), 0, s, part, blocks, p.d,
                     static_cast<T*>(p.dw), static_cast<T*>(p.db));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormParams& p, int dtype, hipStream_t s) {
  if (p.rows == 0) return hipSuccess;
  const bool drop = p.drop.least != 0;
  if (dtype == 1) return drop ? forward<uint16_t, true>(p, s) : forward<uint16_t, false>(p, s);
  return drop ? forward<float, true>(p, s) : forward<float, false>(p, s);
}

int64_t norm_grad_workspace(int64_t rows, int32_t d, int dtype) {
  (void)dtype;
  return int64_t(2) * norm_grad_blocks(rows, d) * d * int64_t(sizeof(float));
}

hipError_t launch_norm_grad(const NormGradParams& p, int dtype, void* ws, hipStream_t s) {
  float* part = static_cast<float*>(ws);
  const bool drop = p.drop.least != 0;
  if (dtype == 1) return drop ? backward<uint16_t, true>(p, part, s) : backward<uint16_t, false>(p, part, s);
  return drop ? backward<float, true>(p, part, s) : backward<float, false>(p, part, s);
}

}  // namespace ada
