// Layer and root-mean-square norms with the residual stream and the dropout before them, and
// their backward pass.
//
//   h = residual + dropout(x), y = (h - mean) rstd w + b over each row; "rms": mean is 0
//   dh = dhidden + rstd (t - mean(t) - xhat mean(t xhat)),  t = dy w, xhat = (h - mean) rstd
//   ("rms": without mean(t)); dresidual = dh, dx = dropout(dh), dw = sum over rows of dy xhat,
//   db = sum over rows of dy
//
// Bound by memory: every matrix is read once and written once, but for dy and h of the backward pass
// for few or wide rows (norm_apart_kernel), which reads them twice.  A row lives in the registers of
// one group of lanes from its load to its store, in blocks of eight elements a lane: a power of
// two of lanes for rows of up to 256 elements, otherwise whole waves, whose sums meet in LDS.
// 4096 x 8192 bf16 with residual and dropout: forward 47.0 us, backward 58.9, 5.7 TB/s either way.
// Four fp32 blocks a lane are the exception: a bound of 1024 threads leaves 128 registers, and 36 bytes a
// lane go to scratch (forward; 100 with dropout, 80 and 112 in the backward pass): 585 x 28672 writes 151 MB
// for 134 in 58 us, and 106 for 67 in 84.
#include "elements.h"

namespace ada {
namespace {

constexpr int kMaxWaves = 16;
constexpr int kGradThreads = 1024;  // of a workgroup of norm_grad_kernel, about
constexpr int kGradBlocks = 256;    // one a CU: twice as many write and join twice the partial sums
// Rows that a lane's sums for dw and db take one after the other before they are put aside: fp32 sums of
// hundreds of terms, and of hundreds of such, instead of one of up to 10^5 (2^20 x 8200 fp32: error of db 3e-7, else 3e-6)
constexpr int kRun = 256;

// Lanes that share a row: `lanes` below 64 is a power of two, otherwise a multiple of 64.
struct RowShape {
  int lanes;
  int groups;  // rows in flight in one workgroup
  int chunks;  // blocks of eight elements a lane holds
};

// ---- sums over the lanes of a row ------------------------------------------------------
// N sums at once, the same on every lane of the row.  `slot` is LDS of kMaxWaves x N floats that
// nothing else uses until after the next barrier, not even the next row's sums: a wave may be there
// while others still read.  WIDE: several waves share a row.
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
    // at most 16 waves: their sums come back on 16 lanes, which add up as a row of lanes does
    const int wave = threadIdx.x >> 6, waves = lanes >> 6, first = wave / waves * waves, from = threadIdx.x & 15;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) slot[wave][i] = v[i];
    }
    __syncthreads();
    const float* at = slot[first + (from < waves ? from : 0)];
    float part[N];
#pragma unroll
    for (int i = 0; i < N; ++i) part[i] = at[i];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = row16_total(from < waves ? part[i] : 0.f);
  }
}

// ---- forward ---------------------------------------------------------------------------
// One row at a time per group of lanes.  The variance is the mean square of h - m with m the
// first sum's mean, and that sum's rounding is taken out of both with the mean of h - m
// (Chan, Golub, LeVeque, "Algorithms for computing the sample variance", 1983), so rows far from
// zero keep their accuracy.  y and hidden may be x or the residual: a lane reads what it writes.
template <typename T, int CH, bool STREAM>
struct NormRow {
  Eight<T> x[CH], res[CH];

  __device__ __forceinline__ void load(const NormParams& p, int64_t row, int lane, int lanes, int vectors) {
    const T* px = static_cast<const T*>(p.x.p) + row * p.x.ld;
    const T* pr = static_cast<const T*>(p.res.p) + row * p.res.ld;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      zero_eight(x[c]);
      zero_eight(res[c]);
#pragma unroll
      for (int i = 0; i < kVectors<T>; ++i) {
        const int v = vector_of<T>(lane, lanes, c, i);
        if (row >= p.rows || v >= vectors) continue;
        x[c].v[i] = load_vector<STREAM>(reinterpret_cast<const u32x4*>(px) + v);
        if (p.res.p != nullptr) res[c].v[i] = load_vector<STREAM>(reinterpret_cast<const u32x4*>(pr) + v);
      }
    }
  }
};

template <typename T, int CH, bool SUB, bool WIDE, bool DROP, bool STREAM>
__global__ void __launch_bounds__(1024) norm_kernel(NormParams p, int lanes) {
  __shared__ float mean_slot[kMaxWaves][1];
  __shared__ float square_slot[2][kMaxWaves][2];  // by turns: rms has no other barrier between two rows' sums
  const int group = threadIdx.x / lanes, lane = threadIdx.x - group * lanes, groups = blockDim.x / lanes;
  const int per_row = p.d >> 3, vectors = p.d / kVector<T>;
  const T* w = static_cast<const T*>(p.w);
  const T* b = static_cast<const T*>(p.b);
  const float over = 1.f / float(p.d);
  DropKey key{};
  if constexpr (DROP) key = drop_key(p.drop);

  // lanes of one block hold their weights from the start, one trip to memory less behind the sums
  // (16384 x 2048: 46.8 against 49.3 us); of two it costs more waves than it saves
  constexpr bool HOLD = CH == 1;
  Eight<T> wheld[HOLD ? CH : 1], bheld[HOLD ? CH : 1];
  const auto load_affine = [&](const T* v, int c) {
    Eight<T> e;
    zero_eight(e);
    if (v != nullptr) e = load_anyway(v, lane, lanes, c, vectors);
    return e;
  };
  if constexpr (HOLD) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      wheld[c] = load_affine(w, c);
      bheld[c] = load_affine(b, c);
    }
  }
  NormRow<T, CH, STREAM> now;
  const int64_t step = int64_t(gridDim.x) * groups;
  int64_t row = int64_t(blockIdx.x) * groups + group;
  now.load(p, row, lane, lanes, vectors);
  int turn = 0;
  for (int64_t row0 = row - group; row0 < p.rows; row0 += step, row += step, turn ^= 1) {
    T* y = static_cast<T*>(p.y.p) + row * p.y.ld;
    T* hidden = static_cast<T*>(p.hidden.p) + row * p.hidden.ld;
    float h[CH][8], sum[1] = {0.f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      unpack(now.x[c], h[c]);
      if constexpr (DROP)
        drop_block<SUB, T>(h[c], uint32_t(row * per_row), lane, lanes, c, key, p.drop.least, p.drop.scale);
      if (p.res.p != nullptr) {
        float r[8];
        unpack(now.res[c], r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[c][i] += r[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[0] += h[c][i];
    }
    float mean = 0.f, rest = 0.f;
    if (!p.rms) {
      row_totals<1, SUB, WIDE>(sum, lanes, mean_slot);
      mean = sum[0] * over;
    }
    float second[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
      for (int v = 0; v < kVectors<T>; ++v) {
        if (vector_of<T>(lane, lanes, c, v) >= vectors) continue;
#pragma unroll
        for (int i = v * kVector<T>; i < (v + 1) * kVector<T>; ++i) {
          const float a = h[c][i] - mean;
          second[0] = fmaf(a, a, second[0]);
          second[1] += a;
        }
      }
    }
    row_totals<2, SUB, WIDE>(second, lanes, square_slot[turn]);
    float square = second[0] * over;
    if (!p.rms) {
      rest = second[1] * over;
      square -= rest * rest;
      square = square < 0.f ? 0.f : square;  // NaN stays
    }
    const float rstd = 1.f / sqrtf(square + p.eps);
    if (row < p.rows) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (vector_of<T>(lane, lanes, c, 0) >= vectors) continue;
        if (p.hidden.p != nullptr) store_block<STREAM>(hidden, lane, lanes, c, vectors, h[c]);
        float out[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) out[i] = (h[c][i] - mean - rest) * rstd;
        if (w != nullptr) {
          float v[8];
          unpack(HOLD ? wheld[HOLD ? c : 0] : load_affine(w, c), v);
#pragma unroll
          for (int i = 0; i < 8; ++i) out[i] *= v[i];
        }
        if (b != nullptr) {
          float v[8];
          unpack(HOLD ? bheld[HOLD ? c : 0] : load_affine(b, c), v);
#pragma unroll
          for (int i = 0; i < 8; ++i) out[i] += v[i];
        }
        store_block(y, lane, lanes, c, vectors, out);
      }
      if (lane == 0) {
        if (p.mean != nullptr) p.mean[row] = mean + rest;
        if (p.rstd != nullptr) p.rstd[row] = rstd;
      }
    }
    now.load(p, row + step, lane, lanes, vectors);
  }
}

// ---- backward --------------------------------------------------------------------------
// A lane's part of a row's operands; a row past the end adds zeros.
template <typename T, int CH, bool STREAM>
struct GradRow {
  struct {
    Eight<T> dy, h, add;
  } c[CH];
  float mean, rstd;

  __device__ __forceinline__ void load(const NormGradParams& p, int64_t row, int lane, int lanes, int vectors) {
    const bool live = row < p.rows;
    const int in_row = live ? vectors : 0;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      c[i].dy = load_block<STREAM>(static_cast<const T*>(p.dy.p) + row * p.dy.ld, lane, lanes, i, in_row);
      c[i].h = load_block<STREAM>(static_cast<const T*>(p.hidden.p) + row * p.hidden.ld, lane, lanes, i, in_row);
      zero_eight(c[i].add);
      if (p.dhidden.p != nullptr)
        c[i].add = load_block<STREAM>(static_cast<const T*>(p.dhidden.p) + row * p.dhidden.ld, lane, lanes, i, in_row);
    }
    mean = live && p.mean != nullptr ? p.mean[row] : 0.f;
    rstd = live ? p.rstd[row] : 0.f;
  }

  // Makes the loads' results wanted here.
  __device__ __forceinline__ void arrived() {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
#pragma unroll
      for (unsigned j = 0; j < sizeof(T) / 2; ++j) {
        asm volatile("" : "+v"(c[i].dy.v[j]), "+v"(c[i].h.v[j]), "+v"(c[i].add.v[j]));
      }
    }
    asm volatile("" : "+v"(mean), "+v"(rstd));
  }

  // The eight values of dh from block i, given the means of t and of t xhat.
  __device__ __forceinline__ void gradient(int i, const float (&w)[8], float c1, float c2, float (&dh)[8]) const {
    float dy[8], add[8];
    unpack(c[i].dy, dy);
    unpack(c[i].h, dh);
    unpack(c[i].add, add);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float xhat = (dh[e] - mean) * rstd;
      dh[e] = fmaf(rstd, dy[e] * w[e] - c1 - xhat * c2, add[e]);
    }
  }
};

// What block c of a row's gradient goes to; dx and dres may be dy or dhidden: a lane has read what it
// writes.
template <typename T, bool SUB, bool DROP, bool STREAM, bool STREAM_DX>
__device__ __forceinline__ void store_gradient(const NormGradParams& p, int64_t row, int lane, int lanes, int c,
                                               const DropKey& key, float (&dh)[8]) {
  const int vectors = p.d / kVector<T>;
  if (p.dres.p != nullptr)
    store_block<STREAM>(static_cast<T*>(p.dres.p) + row * p.dres.ld, lane, lanes, c, vectors, dh);
  if (p.dx.p == nullptr) return;
  if constexpr (DROP)
    drop_block<SUB, T>(dh, uint32_t(row * (p.d >> 3)), lane, lanes, c, key, p.drop.least, p.drop.scale);
  store_block<STREAM_DX>(static_cast<T*>(p.dx.p) + row * p.dx.ld, lane, lanes, c, vectors, dh);
}

// Eight weights; ones where there are none.
template <typename T>
__device__ __forceinline__ void weight_of(const void* w, const Eight<T>& raw, float (&f)[8]) {
  unpack(raw, f);
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 1.f;
  }
}

// Rows and columns in one pass, for many rows of up to 8192 columns.  A workgroup takes every
// gridDim.x-th set of rows, keeps the sums dw and db of a lane's eight columns in registers over all
// of them, and writes them once: part[0][block][d] and part[1][block][d], which norm_join_kernel
// adds up in a fixed order.  The next row's loads are in flight while this one is summed.
template <typename T, bool SUB, bool WIDE, bool DROP, bool STREAM>
__global__ void __launch_bounds__(1024) norm_grad_kernel(NormGradParams p, int lanes, float* part) {
  __shared__ float slot[2][kMaxWaves][2];
  __shared__ f32x4 meet[4 * kGradThreads];  // sums put aside, then where the groups of a workgroup meet
  const int group = threadIdx.x / lanes, lane = threadIdx.x - group * lanes, groups = blockDim.x / lanes;
  const int vectors = p.d / kVector<T>;
  const float over = 1.f / float(p.d);
  DropKey key{};
  if constexpr (DROP) key = drop_key(p.drop);
  float dw[8] = {}, db[8] = {};
  Eight<T> weight;  // unpacked anew for each row (2047 x 4096: 20 us; held as floats 24)
  zero_eight(weight);
  if (p.w != nullptr) weight = load_block(static_cast<const T*>(p.w), lane, lanes, 0, vectors);

  GradRow<T, 1, STREAM> now, next;
  const int64_t step = int64_t(gridDim.x) * groups;
  int64_t row = int64_t(blockIdx.x) * groups + group;
  now.load(p, row, lane, lanes, vectors);
  int turn = 0;
  for (int64_t row0 = row - group; row0 < p.rows; row0 += step, row += step, ++turn) {
    next.load(p, row + step, lane, lanes, vectors);
    float sums[2] = {0.f, 0.f}, dy[8], h[8], w[8];
    weight_of(p.w, weight, w);
    unpack(now.c[0].dy, dy);
    unpack(now.c[0].h, h);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = dy[i] * w[i], xhat = (h[i] - now.mean) * now.rstd;
      sums[0] += t;
      sums[1] = fmaf(t, xhat, sums[1]);
      dw[i] = fmaf(dy[i], xhat, dw[i]);
      db[i] += dy[i];
    }
    row_totals<2, SUB, WIDE>(sums, lanes, slot[turn & 1]);
    now.gradient(0, w, p.mean != nullptr ? sums[0] * over : 0.f, sums[1] * over, h);
    // the next row's loads are waited for before this row's stores: the counter holds both, and behind
    // the stores the wait would be for them too
    now = next;
    now.arrived();
    if (row < p.rows) store_gradient<T, SUB, DROP, STREAM, false>(p, row, lane, lanes, 0, key, h);
    if (turn % kRun == kRun - 1) {
      const f32x4 sum[4] = {{dw[0], dw[1], dw[2], dw[3]}, {dw[4], dw[5], dw[6], dw[7]},
                            {db[0], db[1], db[2], db[3]}, {db[4], db[5], db[6], db[7]}};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f32x4& at = meet[j * blockDim.x + threadIdx.x];
        at = turn < kRun ? sum[j] : at + sum[j];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) dw[i] = db[i] = 0.f;
    }
  }
  if (turn >= kRun) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dw[i] += meet[(i >> 2) * blockDim.x + threadIdx.x][i & 3];
      db[i] += meet[(2 + (i >> 2)) * blockDim.x + threadIdx.x][i & 3];
    }
  }

  for (int which = 0; which < 2; ++which) {
    if ((which == 0 ? p.dw : p.db) == nullptr) continue;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = which == 0 ? dw[i] : db[i];
    if (groups > 1) {
      __syncthreads();
      meet[threadIdx.x] = f32x4{v[0], v[1], v[2], v[3]};
      meet[blockDim.x + threadIdx.x] = f32x4{v[4], v[5], v[6], v[7]};
      __syncthreads();
      if (group == 0) {
        for (int q = 1; q < groups; ++q) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] += meet[(i >> 2) * blockDim.x + q * lanes + lane][i & 3];
        }
      }
    }
    if (group != 0) continue;
    float* to = part + (int64_t(which) * gridDim.x + blockIdx.x) * p.d;
#pragma unroll
    for (int q = 0; q < 2; ++q) {  // the lane's columns, four at a time: of one vector in bf16, of two in fp32
      const int at = vector_of<T>(lane, lanes, 0, q * kVectors<T> / 2);
      if (at < vectors)
        *reinterpret_cast<f32x4*>(to + at * kVector<T> + (kVectors<T> == 1 ? 4 * q : 0)) =
            f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
    }
  }
}

// Rows and columns apart, in one grid: dw and db need no sums over a row, since mean and rstd are
// given.  The first `stripes` workgroups sum 64 columns each over all rows, eight columns a lane, the
// rows dealt to sets of eight lanes; the others take a set of rows each.  dy and h are read twice,
// but there are no partial sums to write and join, so few rows need one launch; and a row is only
// held until it is summed, so wide ones fit the registers.  Large calls stream dx too: what stays in the
// caches is dy and h for their second reading (1170 x 28672: 96 us, with dx kept 111).
constexpr int kStripe = 64;
template <typename T, int CH, bool SUB, bool WIDE, bool DROP, bool STREAM>
__global__ void __launch_bounds__(1024) norm_apart_kernel(NormGradParams p, int lanes, int stripes) {
  const int per_row = p.d >> 3, vectors = p.d / kVector<T>;
  if (int(blockIdx.x) < stripes) {
    __shared__ f32x4 meet[kMaxWaves][8][4];
    const int quad = threadIdx.x & 7, sets = blockDim.x >> 3, g = blockIdx.x * 8 + quad;
    const bool inside = g < per_row;
    const T* dyp = static_cast<const T*>(p.dy.p) + (inside ? g : 0) * 8;
    const T* hp = static_cast<const T*>(p.hidden.p) + (inside ? g : 0) * 8;
    f32x4 sum[4] = {};  // dw, dw, db, db
    constexpr int U = 4;
    constexpr bool LONG = CH == 4;  // of those alone more than kRun rows a lane come here (apart())
    f32x4 aside[4] = {};
    int run = 0;
    for (int64_t row0 = threadIdx.x >> 3; row0 < p.rows; row0 += int64_t(sets) * U) {
      Eight<T> a[U], b[U];
      float mean[U], rstd[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {  // past the last row the last again, and nothing of it is added
        const int64_t at = row0 + int64_t(u) * sets, row = at < p.rows ? at : p.rows - 1;
        a[u] = load_eight(dyp + row * p.dy.ld);
        b[u] = load_eight(hp + row * p.hidden.ld);
        mean[u] = p.mean != nullptr ? p.mean[row] : 0.f;
        rstd[u] = p.rstd[row];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (row0 + int64_t(u) * sets >= p.rows) break;
        float dy[8], h[8];
        unpack(a[u], dy);
        unpack(b[u], h);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sum[i >> 2][i & 3] = fmaf(dy[i], (h[i] - mean[u]) * rstd[u], sum[i >> 2][i & 3]);
          sum[2 + (i >> 2)][i & 3] += dy[i];
        }
      }
      if constexpr (LONG) {
        run += U;
        if (run == kRun) {
          run = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            aside[j] += sum[j];
            sum[j] = f32x4{0.f, 0.f, 0.f, 0.f};
          }
        }
      }
    }
    if constexpr (LONG) {
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] += aside[j];
    }
    // the eight sets of a wave, then the waves
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        for (int m = 8; m < 64; m <<= 1) sum[j][e] += __shfl_xor(sum[j][e], m, 64);
      }
      if ((threadIdx.x & 63) < 8) meet[threadIdx.x >> 6][quad][j] = sum[j];
    }
    __syncthreads();
    if (threadIdx.x < 8 && inside) {
      for (unsigned v = 1; v < blockDim.x >> 6; ++v) {
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] += meet[v][quad][j];
      }
      float f[8];
#pragma unroll
      for (int which = 0; which < 2; ++which) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = sum[2 * which + (i >> 2)][i & 3];
        T* to = static_cast<T*>(which == 0 ? p.dw : p.db);
        if (to != nullptr) store_eight(to + g * 8, f);
      }
    }
    return;
  }
  __shared__ float slot[kMaxWaves][2];
  const int group = threadIdx.x / lanes, lane = threadIdx.x - group * lanes, groups = blockDim.x / lanes;
  const float over = 1.f / float(p.d);
  DropKey key{};
  if constexpr (DROP) key = drop_key(p.drop);
  const int64_t row = int64_t(blockIdx.x - stripes) * groups + group;
  GradRow<T, CH, STREAM> now;
  // the weights come with the row and stay for its second use; of the widest rows they are read twice
  constexpr bool HOLD = CH < 4;
  Eight<T> held[HOLD ? CH : 1];
  const auto load_weight = [&](int c) {
    Eight<T> w;
    zero_eight(w);
    if (p.w != nullptr) w = load_anyway(static_cast<const T*>(p.w), lane, lanes, c, vectors);
    return w;
  };
  if constexpr (HOLD) {
#pragma unroll
    for (int c = 0; c < CH; ++c) held[c] = load_weight(c);
  }
  now.load(p, row, lane, lanes, vectors);
  float sums[2] = {0.f, 0.f};
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    float dy[8], h[8], w[8];
    unpack(now.c[c].dy, dy);
    unpack(now.c[c].h, h);
    weight_of(p.w, HOLD ? held[HOLD ? c : 0] : load_weight(c), w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = dy[i] * w[i];
      sums[0] += t;
      sums[1] = fmaf(t, (h[i] - now.mean) * now.rstd, sums[1]);
    }
  }
  row_totals<2, SUB, WIDE>(sums, lanes, slot);
  if (row >= p.rows) return;
  const float c1 = p.mean != nullptr ? sums[0] * over : 0.f, c2 = sums[1] * over;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    if (vector_of<T>(lane, lanes, c, 0) >= vectors) continue;
    float w[8], dh[8];
    weight_of(p.w, HOLD ? held[HOLD ? c : 0] : load_weight(c), w);
    now.gradient(c, w, c1, c2, dh);
    store_gradient<T, SUB, DROP, STREAM, STREAM>(p, row, lane, lanes, c, key, dh);
  }
}

// dw (blockIdx.y = 0) and db (1) from `parts` (at most kGradBlocks) rows of d sums each: 32 columns a
// workgroup (one line of each row), four a lane, the rows dealt to 32 sets of lanes, all of a lane's
// loads in flight at once; the sets meet in LDS.
constexpr int kJoinSets = 32;
template <typename T>
__global__ void __launch_bounds__(256) norm_join_kernel(const float* part, int parts, int d, T* dw, T* db) {
  constexpr int EACH = (kGradBlocks + kJoinSets - 1) / kJoinSets;
  __shared__ f32x4 meet[4][8];
  T* out = blockIdx.y == 0 ? dw : db;
  if (out == nullptr) return;
  const int quad = threadIdx.x & 7, set = threadIdx.x >> 3, col = blockIdx.x * 32 + quad * 4;
  const float* from = part + int64_t(blockIdx.y) * parts * d + (col < d ? col : 0);
  f32x4 v[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int r = set + i * kJoinSets;
    v[i] = *reinterpret_cast<const f32x4*>(from + int64_t(r < parts ? r : 0) * d);
  }
  f32x4 sum{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] += set + i * kJoinSets < parts ? v[i][e] : 0.f;
  }
  // the eight sets of a wave, then the waves
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    for (int m = 8; m < 64; m <<= 1) sum[e] += __shfl_xor(sum[e], m, 64);
  }
  if ((threadIdx.x & 63) < 8) meet[threadIdx.x >> 6][quad] = sum;
  __syncthreads();
  const int c = blockIdx.x * 32 + threadIdx.x;
  if (threadIdx.x < 32 && c < d) {
    const int q = threadIdx.x >> 2, e = threadIdx.x & 3;
    const float sum = (meet[0][q][e] + meet[1][q][e]) + (meet[2][q][e] + meet[3][q][e]);
    if constexpr (sizeof(T) == 2)
      out[c] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(sum));
    else
      out[c] = sum;
  }
}

// ---- rules on sizes --------------------------------------------------------------------
int round64(int v) { return (v + 63) / 64 * 64; }

// Lanes of a row of `chunks` blocks a lane, and rows of a workgroup of about `threads` threads.
RowShape row_shape(int per_row, int chunks, int threads) {
  RowShape s{};
  s.chunks = chunks;
  if (per_row <= 32) {
    s.lanes = 1;
    while (s.lanes < per_row) s.lanes *= 2;
  } else {
    s.lanes = round64((per_row + chunks - 1) / chunks);
  }
  s.groups = s.lanes < threads ? threads / s.lanes : 1;
  return s;
}

// Blocks a lane: one up to 4096 columns, two up to 8192, else four.  More waves of fewer blocks
// each are the faster (4096 x 4096 bf16: 26 us with one, 28 with two), until a row takes 1024
// threads, of which a CU holds two rows only (4096 x 8192: 48 us with two blocks, 61 with one, 49 with
// four; one row of 4096: 3.0, 3.3 and 4.1 us).  Many rows of up to 1536 columns take a wave each, without
// barriers and with less of the last wave idle (16384 x 1032: 32 against 35 us, x 520: 18
// against 21); few rows do not (300 x 1032 fp32: 4.4 against 3.6).
RowShape forward_shape(int64_t rows, int d) {
  const int per_row = d / 8;
  if (per_row > 32 && per_row <= 192 && rows >= 2048) return row_shape(per_row, (per_row + 63) / 64, 256);
  return row_shape(per_row, per_row <= 512 ? 1 : per_row <= 1024 ? 2 : 4, 256);
}

// Rows and columns apart, or in one pass.  Apart reads 7 matrices for 5 but has no partial sums and
// one launch; it is the faster from 512 up to 550 to 1400 rows, more with more columns: 512 x 4096 bf16 8.0
// against 13.6 us, 1024 x 4096 14.7 against 15.9, 1536 x 4096 20.3 against 17.7; 512 x 1032 7.4 against
// 8.4, 1024 x 1032 11.3 against 9.8; 1024 x 8192 19.7 against 22.9, 4096 x 8192 67 against 54.  Past 8192
// columns a lane of the one pass, 1024 threads to a workgroup, would hold two blocks or more with their sums in
// the 128 registers that leaves, which spilled: 1170 x 28672 in 96 us apart, 218 in one pass.  So there is a step
// behind 8192 columns, the larger the more rows: 8192 and 8200 columns bf16 11.7 and 15.3 us at 512 rows,
// 31 and 46 at 2048, 54 and 85 at 4096, 182 and 321 at 16384.
bool apart(int64_t rows, int d) { return d > 8192 || rows <= 512 + d / 8; }

// The rows' part as in the forward pass, in workgroups of as many rows as 512 threads hold, one at least: 320
// (2056 to 2560 columns, and twice and four times that) to 1024 threads, for the columns' part too.
RowShape apart_shape(int d) {
  const int per_row = d / 8;
  return row_shape(per_row, per_row <= 512 ? 1 : per_row <= 1024 ? 2 : 4, 512);
}

int norm_grad_blocks(int64_t rows, int d) {
  const RowShape s = row_shape(d / 8, 1, kGradThreads);
  const int64_t sets = (rows + s.groups - 1) / s.groups;
  return static_cast<int>(sets < kGradBlocks ? sets : kGradBlocks);
}

template <typename T, int CH, bool DROP, bool STREAM>
hipError_t forward(const NormParams& p, const RowShape& r, hipStream_t s) {
  const int64_t sets = (p.rows + r.groups - 1) / r.groups, most = 1 << 20;
  const dim3 grid(static_cast<unsigned>(sets < most ? sets : most)), block(r.lanes * r.groups);
  // three blocks a lane are a wave's only, four a wide row's
  if (r.lanes < 64)
    hipLaunchKernelGGL((norm_kernel<T, 1, true, false, DROP, STREAM>), grid, block, 0, s, p, r.lanes);
  else if (CH < 4 && r.lanes == 64)
    hipLaunchKernelGGL((norm_kernel<T, CH < 4 ? CH : 1, false, false, DROP, STREAM>), grid, block, 0, s, p, r.lanes);
  else
    hipLaunchKernelGGL((norm_kernel<T, CH != 3 ? CH : 1, false, true, DROP, STREAM>), grid, block, 0, s, p, r.lanes);
  return hipGetLastError();
}

template <typename T, bool DROP, bool STREAM>
hipError_t forward(const NormParams& p, hipStream_t s) {
  const RowShape r = forward_shape(p.rows, p.d);
  if (r.chunks == 1) return forward<T, 1, DROP, STREAM>(p, r, s);
  if (r.chunks == 2) return forward<T, 2, DROP, STREAM>(p, r, s);
  if (r.chunks == 3) return forward<T, 3, DROP, STREAM>(p, r, s);
  return forward<T, 4, DROP, STREAM>(p, r, s);
}

template <typename T, int CH, bool DROP, bool STREAM>
hipError_t launch_apart(const NormGradParams& p, const RowShape& r, int stripes, int64_t sets, hipStream_t s) {
  if (stripes + sets == 0) return hipSuccess;
  const dim3 grid(static_cast<unsigned>(stripes + sets)), block(r.lanes * r.groups);
  if (r.lanes > 64)
    hipLaunchKernelGGL((norm_apart_kernel<T, CH, false, true, DROP, STREAM>), grid, block, 0, s, p, r.lanes, stripes);
  else if (r.lanes == 64)
    hipLaunchKernelGGL((norm_apart_kernel<T, 1, false, false, DROP, STREAM>), grid, block, 0, s, p, r.lanes, stripes);
  else
    hipLaunchKernelGGL((norm_apart_kernel<T, 1, true, false, DROP, STREAM>), grid, block, 0, s, p, r.lanes, stripes);
  return hipGetLastError();
}

template <typename T, int CH, bool DROP, bool STREAM>
hipError_t rows_apart(const NormGradParams& p, const RowShape& r, hipStream_t s) {
  const int64_t sets = p.dx.p == nullptr && p.dres.p == nullptr ? 0 : (p.rows + r.groups - 1) / r.groups;
  const int stripes = p.dw == nullptr && p.db == nullptr ? 0 : (p.d + kStripe - 1) / kStripe;
  // the columns' workgroups read dy: where a gradient takes its place, they go first
  const bool over_dy = p.dy.p != nullptr && (p.dx.p == p.dy.p || p.dres.p == p.dy.p);
  if (!over_dy) return launch_apart<T, CH, DROP, STREAM>(p, r, stripes, sets, s);
  const hipError_t e = launch_apart<T, CH, DROP, STREAM>(p, r, stripes, 0, s);
  return e == hipSuccess ? launch_apart<T, CH, DROP, STREAM>(p, r, 0, sets, s) : e;
}

template <typename T, bool DROP, bool STREAM>
hipError_t backward(const NormGradParams& p, float* part, hipStream_t s) {
  if (apart(p.rows, p.d)) {
    const RowShape r = apart_shape(p.d);
    if (r.chunks == 1) return rows_apart<T, 1, DROP, STREAM>(p, r, s);
    if (r.chunks == 2) return rows_apart<T, 2, DROP, STREAM>(p, r, s);
    return rows_apart<T, 4, DROP, STREAM>(p, r, s);
  }
  const RowShape r = row_shape(p.d / 8, 1, kGradThreads);
  const int blocks = norm_grad_blocks(p.rows, p.d);
  const dim3 grid(blocks), block(r.lanes * r.groups);
  if (r.lanes > 64)
    hipLaunchKernelGGL((norm_grad_kernel<T, false, true, DROP, STREAM>), grid, block, 0, s, p, r.lanes, part);
  else if (r.lanes == 64)
    hipLaunchKernelGGL((norm_grad_kernel<T, false, false, DROP, STREAM>), grid, block, 0, s, p, r.lanes, part);
  else
    hipLaunchKernelGGL((norm_grad_kernel<T, true, false, DROP, STREAM>), grid, block, 0, s, p, r.lanes, part);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || (p.dw == nullptr && p.db == nullptr)) return e;
  hipLaunchKernelGGL(norm_join_kernel<T>, dim3((p.d + 31) / 32, 2), dim3(256), 0, s, part, blocks, p.d,
                     static_cast<T*>(p.dw), static_cast<T*>(p.db));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormParams& p, int dtype, hipStream_t s) {
  if (p.rows == 0) return hipSuccess;
  const bool drop = p.drop.least != 0;
  const bool stream = streams(p.rows * p.d);
  if (dtype == 1 && stream) return drop ? forward<uint16_t, true, true>(p, s) : forward<uint16_t, false, true>(p, s);
  if (dtype == 1) return drop ? forward<uint16_t, true, false>(p, s) : forward<uint16_t, false, false>(p, s);
  if (stream) return drop ? forward<float, true, true>(p, s) : forward<float, false, true>(p, s);
  return drop ? forward<float, true, false>(p, s) : forward<float, false, false>(p, s);
}

int64_t norm_grad_workspace(int64_t rows, int32_t d) {
  return apart(rows, d) ? 0 : int64_t(2) * norm_grad_blocks(rows, d) * d * int64_t(sizeof(float));
}

hipError_t launch_norm_grad(const NormGradParams& p, int dtype, void* ws, hipStream_t s) {
  // without rows only dw and db are written
  if (p.rows == 0 && p.dw == nullptr && p.db == nullptr) return hipSuccess;
  float* part = static_cast<float*>(ws);
  const bool drop = p.drop.least != 0;
  const bool stream = streams(p.rows * p.d);
  if (dtype == 1 && stream)
    return drop ? backward<uint16_t, true, true>(p, part, s) : backward<uint16_t, false, true>(p, part, s);
  if (dtype == 1)
    return drop ? backward<uint16_t, true, false>(p, part, s) : backward<uint16_t, false, false>(p, part, s);
  if (stream) return drop ? backward<float, true, true>(p, part, s) : backward<float, false, true>(p, part, s);
  return drop ? backward<float, true, false>(p, part, s) : backward<float, false, false>(p, part, s);
}

}  // namespace ada
