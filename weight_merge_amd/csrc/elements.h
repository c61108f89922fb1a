// Device code shared by the norms, dropout and the router: eight consecutive elements as one
// unit of work, the counter-based generator, and sums over lanes.
#pragma once

#include "layer.h"

namespace ada {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// ---- eight consecutive elements, 16-byte aligned ---------------------------------------
template <typename T>
struct Eight {
  u32x4 v[sizeof(T) / 2];  // bf16: one vector, fp32: two
};
template <typename T>
constexpr int kVectors = sizeof(T) / 2;  // of a block
template <typename T>
constexpr int kVector = 16 / sizeof(T);  // elements of a vector

// STREAM: past the caches' ordinary policy (streams() below).
template <bool STREAM>
__device__ __forceinline__ u32x4 load_vector(const u32x4* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(p);
  return *p;
}
template <bool STREAM>
__device__ __forceinline__ void store_vector(u32x4* p, u32x4 v) {
  if constexpr (STREAM)
    __builtin_nontemporal_store(v, p);
  else
    *p = v;
}

// Eight elements in a row.
template <typename T>
__device__ __forceinline__ Eight<T> load_eight(const T* p) {
  Eight<T> e;
#pragma unroll
  for (int i = 0; i < kVectors<T>; ++i) e.v[i] = load_vector<false>(reinterpret_cast<const u32x4*>(p) + i);
  return e;
}

template <typename T>
__device__ __forceinline__ void zero_eight(Eight<T>& e) {
#pragma unroll
  for (unsigned i = 0; i < sizeof(T) / 2; ++i) e.v[i] = u32x4{0, 0, 0, 0};
}

__device__ __forceinline__ void unpack(const Eight<float>& e, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(e.v[i >> 2][i & 3]);
}
__device__ __forceinline__ void unpack(const Eight<uint16_t>& e, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(e.v[0][i] << 16);
    f[2 * i + 1] = __uint_as_float(e.v[0][i] & 0xffff0000u);
  }
}

__device__ __forceinline__ Eight<float> pack(const float (&f)[8], float) {
  Eight<float> e;
#pragma unroll
  for (int i = 0; i < 8; ++i) e.v[i >> 2][i & 3] = __float_as_uint(f[i]);
  return e;
}
__device__ __forceinline__ Eight<uint16_t> pack(const float (&f)[8], uint16_t) {  // to nearest-even
  Eight<uint16_t> e;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = __builtin_bit_cast(uint16_t, static_cast<__bf16>(f[2 * i]));
    const uint32_t hi = __builtin_bit_cast(uint16_t, static_cast<__bf16>(f[2 * i + 1]));
    e.v[0][i] = lo | hi << 16;
  }
  return e;
}

template <typename T>
__device__ __forceinline__ void store_eight(T* p, const float (&f)[8]) {
  const Eight<T> e = pack(f, T());
#pragma unroll
  for (int i = 0; i < kVectors<T>; ++i) store_vector<false>(reinterpret_cast<u32x4*>(p) + i, e.v[i]);
}

// Eight elements of a row that `lanes` lanes share, the lane's block c: in bf16 vector c lanes + lane of
// the row's, in fp32 vectors 2 c lanes + lane and (2 c + 1) lanes + lane, so that an instruction's lanes
// lie side by side in either.  Vectors past the row's `vectors` are zero, and are not stored.
template <typename T>
__device__ __forceinline__ int vector_of(int lane, int lanes, int c, int i) {
  return lane + (c * kVectors<T> + i) * lanes;
}
template <bool STREAM = false, typename T>
__device__ __forceinline__ Eight<T> load_block(const T* row, int lane, int lanes, int c, int vectors) {
  Eight<T> e;
#pragma unroll
  for (int i = 0; i < kVectors<T>; ++i) {
    const int v = vector_of<T>(lane, lanes, c, i);
    e.v[i] = u32x4{0, 0, 0, 0};
    if (v < vectors) e.v[i] = load_vector<STREAM>(reinterpret_cast<const u32x4*>(row) + v);
  }
  return e;
}
// The same with some vector in place of one past the end: no branch.
template <typename T>
__device__ __forceinline__ Eight<T> load_anyway(const T* row, int lane, int lanes, int c, int vectors) {
  Eight<T> e;
#pragma unroll
  for (int i = 0; i < kVectors<T>; ++i) {
    const int v = vector_of<T>(lane, lanes, c, i);
    e.v[i] = reinterpret_cast<const u32x4*>(row)[v < vectors ? v : 0];
  }
  return e;
}
template <bool STREAM = false, typename T>
__device__ __forceinline__ void store_block(T* row, int lane, int lanes, int c, int vectors, const float (&f)[8]) {
  const Eight<T> e = pack(f, T());
#pragma unroll
  for (int i = 0; i < kVectors<T>; ++i) {
    const int v = vector_of<T>(lane, lanes, c, i);
    if (v < vectors) store_vector<STREAM>(reinterpret_cast<u32x4*>(row) + v, e.v[i]);
  }
}

// Whether a call on matrices of this many elements streams what it will not need again soon: its
// inputs, the residual stream and that stream's gradient, but not y and dx, which the next call reads
// (norm_apart_kernel streams dx, so that dy and h stay for its second reading of them).
// Between products (norm, projection, norm, ..) of 4096 columns ordinary accesses throughout take 33.6 us
// a layer at 509 rows (streamed: 33.6; with y too 35.0), 81.6 at 2047 (79.6; 80.9), 1800 at 16384 rows
// of 8192 columns (1776; 1814); the backward pass at 509 rows 35.2 (37.5).  The same number in fp32:
// dropout of 4096 x 14336 85.4 us ordinary, 77.9 streamed, of 2047 x 1032 5.2 and 6.8.
inline bool streams(int64_t elements) { return elements >= int64_t(1) << 22; }

// ---- dropout ---------------------------------------------------------------------------
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3",
// 2011).  Counter (g, 0, offset), key = seed: the four words are the eight 16-bit numbers of
// elements 8 g .. 8 g + 7, low half first.  16 bits an element rather than 32 halve the
// generator's products, which would otherwise bound the pass (20 of 32 x 32 bits at a quarter
// of the rate of other instructions for every block of eight instead of four elements); p is
// then a multiple of 2^-16 and the scale is exactly that multiple's.
struct DropKey {
  uint32_t k0, k1, o0, o1;
};
__device__ __forceinline__ DropKey drop_key(const DropParams& d) {
  uint64_t seed = d.seed, offset = d.offset;
  if (d.state != nullptr) {
    seed = d.state[0];
    offset += d.state[1];
  }
  return {uint32_t(seed), uint32_t(seed >> 32), uint32_t(offset), uint32_t(offset >> 32)};
}

// One instruction; the compiler makes two of it where a key is uniform.
__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
  return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96);
}

__device__ __forceinline__ u32x4 philox(uint32_t g, const DropKey& key) {
  uint32_t c0 = g, c1 = 0, c2 = key.o0, c3 = key.o1, k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = uint64_t(c0) * 0xD2511F53u, b = uint64_t(c2) * 0xCD9E8D57u;
    c0 = xor3(uint32_t(b >> 32), c1, k0);
    c1 = uint32_t(b);
    c2 = xor3(uint32_t(a >> 32), c3, k1);
    c3 = uint32_t(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4{c0, c1, c2, c3};
}

// Four elements with the numbers of two words: kept ones times the scale, dropped ones zero whatever
// they were.
__device__ __forceinline__ void drop_four(float* f, uint32_t w0, uint32_t w1, uint32_t least, float scale) {
  f[0] = (w0 & 0xffffu) >= least ? f[0] * scale : 0.f;
  f[1] = (w0 >> 16) >= least ? f[1] * scale : 0.f;
  f[2] = (w1 & 0xffffu) >= least ? f[2] * scale : 0.f;
  f[3] = (w1 >> 16) >= least ? f[3] * scale : 0.f;
}

// Block c of a lane (as load_block) of a row whose first eight elements are the matrix's block g0.  In
// fp32 a lane holds halves of two of the generator's blocks, whose other halves its neighbour holds: the
// even lane draws for the first, the odd one for the second, and they exchange two words each (`lanes`
// is even, and so is a row's number of vectors: a pair holds or lacks a vector together).  APART: fewer
// lanes, each draws for both.
template <bool APART, typename T>
__device__ __forceinline__ void drop_block(float (&f)[8], uint32_t g0, int lane, int lanes, int c, const DropKey& key,
                                           uint32_t least, float scale) {
  if constexpr (sizeof(T) == 2) {
    const u32x4 w = philox(g0 + vector_of<T>(lane, lanes, c, 0), key);
    drop_four(f, w[0], w[1], least, scale);
    drop_four(f + 4, w[2], w[3], least, scale);
  } else if constexpr (APART) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int v = vector_of<T>(lane, lanes, c, i);
      const u32x4 w = philox(g0 + (v >> 1), key);
      drop_four(f + 4 * i, v & 1 ? w[2] : w[0], v & 1 ? w[3] : w[1], least, scale);
    }
  } else {
    const bool odd = lane & 1;
    const u32x4 w = philox(g0 + (vector_of<T>(lane, lanes, c, odd) >> 1), key);
    const auto theirs = [](uint32_t v) {  // quad_perm [1, 0, 3, 2]
      return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0xB1, 0xf, 0xf, true));
    };
    const uint32_t t0 = theirs(odd ? w[0] : w[2]), t1 = theirs(odd ? w[1] : w[3]);
    drop_four(f, odd ? t0 : w[0], odd ? t1 : w[1], least, scale);
    drop_four(f + 4, odd ? w[2] : t0, odd ? w[3] : t1, least, scale);
  }
}

// ---- sums over lanes -------------------------------------------------------------------
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_or_zero(float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, int(__float_as_uint(v)), CTRL, ROWS, 0xf, true));
}

// Sum over the wave's 64 lanes, on every lane: within rows of 16 lanes by shifts, then each
// row's last lane into the next row and the half's into the other half (DPP: no LDS traffic).
__device__ __forceinline__ float wave_total(float v) {
  v += dpp_or_zero<0x111, 0xf>(v);  // row_shr:1
  v += dpp_or_zero<0x112, 0xf>(v);  // row_shr:2
  v += dpp_or_zero<0x114, 0xf>(v);  // row_shr:4
  v += dpp_or_zero<0x118, 0xf>(v);  // row_shr:8
  v += dpp_or_zero<0x142, 0xa>(v);  // row_bcast:15 into rows 1 and 3
  v += dpp_or_zero<0x143, 0xc>(v);  // row_bcast:31 into rows 2 and 3
  return __uint_as_float(__builtin_amdgcn_readlane(int(__float_as_uint(v)), 63));
}

// Sum over 16 neighbouring lanes that hold the same in every row of 16, on every lane.
__device__ __forceinline__ float row16_total(float v) {
  v += dpp_or_zero<0x111, 0xf>(v);
  v += dpp_or_zero<0x112, 0xf>(v);
  v += dpp_or_zero<0x114, 0xf>(v);
  v += dpp_or_zero<0x118, 0xf>(v);
  return __uint_as_float(__builtin_amdgcn_readlane(int(__float_as_uint(v)), 15));
}

// Sum over groups of `lanes` lanes (a power of two up to 32), on each of them.
__device__ __forceinline__ float group_total(float v, int lanes) {
  for (int m = 1; m < lanes; m <<= 1) v += __shfl_xor(v, m, 64);
  return v;
}

}  // namespace
}  // namespace ada
