// Linear and gated feed-forward products with their epilogues, and their backward passes.
//
//   linear   z = x W^T + b,  y = act(z) + residual                       [rows, d_out]
//   glu      g = x Wg^T + bg, u = x Wu^T + bu,  y = act(g) u
//   backward dz = dy act'(z) (dg = dy u act'(g), du = dy act(g)),
//            dx = dz W (dg Wg + du Wu), dW = dz^T x, db = sum over rows of dz
//
// Every product is D(i, j) = sum_k P(i, k) Q(j, k) on the matrix instructions with fp32
// sums and both operands read along k: x and W of the forward pass as they are, W of dx and
// dz and x of dW from transposed copies in the workspace.  Matrix instruction layout (16 x
// 16 tile): lane l = 16 q + c supplies Q(c, k) as the row operand and P(c, k) as the column
// operand for its k slice, and receives D(i = c, j = 4 q .. 4 q + 3), four consecutive
// columns of an output row.  A 16-byte vector per lane feeds one 16x16x32 instruction in
// bf16 and four 16x16x4 ones in fp32 (the instruction's k order is free as long as both
// operands share it).
#include "linear.h"

#include "adafuse.h"

namespace ada {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// ---- storage types -------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<uint16_t>(uint16_t v) { return __uint_as_float(uint32_t(v) << 16); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t from_f32<uint16_t>(float v) {  // to nearest-even
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

template <typename T>
__device__ __forceinline__ void load4(const T* p, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = to_f32<T>(p[i]);
}
template <typename T>
__device__ __forceinline__ void store4(T* p, const float* v) {
  struct alignas(4 * sizeof(T)) Quad { T e[4]; } q;
#pragma unroll
  for (int i = 0; i < 4; ++i) q.e[i] = from_f32<T>(v[i]);
  *reinterpret_cast<Quad*>(p) = q;
}

// ---- activations: value and slope in fp32 --------------------------------------------
constexpr float kSqrt1_2 = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kSqrt2OverPi = 0.79788456080286536f;
constexpr float kCubic = 0.044715f;

__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case ADA_ACT_RELU: return z < 0.f ? 0.f : z;  // NaN stays NaN
    case ADA_ACT_SILU: return z / (1.f + expf(-z));
    case ADA_ACT_GELU: return 0.5f * z * erfcf(-kSqrt1_2 * z);  // erfc: no cancellation for z << 0
    case ADA_ACT_GELU_TANH: return 0.5f * z * (1.f + tanhf(kSqrt2OverPi * (z + kCubic * z * z * z)));
    default: return z;
  }
}

__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case ADA_ACT_RELU: return z > 0.f ? 1.f : 0.f;
    case ADA_ACT_SILU: {
      const float s = 1.f / (1.f + expf(-z));
      return s * (1.f + z * (1.f - s));
    }
    case ADA_ACT_GELU: return 0.5f * erfcf(-kSqrt1_2 * z) + z * kInvSqrt2Pi * expf(-0.5f * z * z);
    case ADA_ACT_GELU_TANH: {
      const float t = tanhf(kSqrt2OverPi * (z + kCubic * z * z * z));
      const float sech2 = 1.f - t * t;  // 0 far out, where z * z may be infinite
      const float inner = kSqrt2OverPi * (1.f + 3.f * kCubic * z * z);
      return 0.5f * (1.f + t) + (sech2 > 0.f ? 0.5f * z * sech2 * inner : 0.f);
    }
    default: return 1.f;
  }
}

// ---- tiled product -------------------------------------------------------------------
#define ADA_GLOBAL __attribute__((address_space(1)))
#define ADA_LDS __attribute__((address_space(3)))

struct GemmParams {
  MatIn p;                // [rows][depth]
  MatIn q[2];             // [cols][depth]; gated: the gate's and the up projection's weights
  const void* bias[2];
  MatIn res;
  MatOut y[2];            // rows from row_split on go to y[1] (the two halves of dW)
  MatOut pre[2];
  float* part;            // split contraction: fp32 sums [split][h][rows][cols]
  int64_t rows;
  int64_t row_split;
  int64_t depth;
  int32_t cols;           // output columns (gated: of one of the two products)
  int32_t act;
  int32_t splits;
  int32_t tiles_m;
  int32_t tiles_n;
};

// y, pre of four consecutive columns n of row m, from the sums without the bias.
template <typename T, bool GATED>
__device__ __forceinline__ void finish4(const GemmParams& a, int64_t m, int64_t n, const f32x4 (&acc)[GATED ? 2 : 1]) {
  constexpr int NQ = GATED ? 2 : 1;
  float z[NQ][4], o[4];
#pragma unroll
  for (int h = 0; h < NQ; ++h) {
    float b[4] = {0.f, 0.f, 0.f, 0.f};
    if (a.bias[h] != nullptr) load4(static_cast<const T*>(a.bias[h]) + n, b);
#pragma unroll
    for (int e = 0; e < 4; ++e) z[h][e] = acc[h][e] + b[e];
    if (a.pre[h].p != nullptr) store4(static_cast<T*>(a.pre[h].p) + m * a.pre[h].ld + n, z[h]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    o[e] = act_value(z[0][e], a.act);
    if constexpr (GATED) o[e] *= z[1][e];
  }
  if (a.res.p != nullptr) {
    float r[4];
    load4(static_cast<const T*>(a.res.p) + m * a.res.ld + n, r);
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] += r[e];
  }
  const int second = m >= a.row_split;
  store4(static_cast<T*>(a.y[second].p) + (m - (second ? a.row_split : 0)) * a.y[second].ld + n, o);
}

// Sixteen bytes per lane from global memory to LDS, lane l's at lds + 16 l (lds is the same
// in every lane of the wave).
__device__ __forceinline__ void copy_to_lds(const unsigned char* g, unsigned char* lds) {
  __builtin_amdgcn_global_load_lds((const ADA_GLOBAL void*)g, (ADA_LDS void*)lds, 16, 0, 0);
}

// Wait until at most N of the wave's copies to LDS are in flight and all its LDS reads and
// writes are done, then meet the workgroup's other waves.
template <int N>
__device__ __forceinline__ void copies_then_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <typename T>
__device__ __forceinline__ f32x4 mfma16(u32x4 q, u32x4 p, f32x4 acc) {
  if constexpr (sizeof(T) == 2) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, q), __builtin_bit_cast(bf16x8, p), acc,
                                                   0, 0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(q[j]), __uint_as_float(p[j]), acc, 0, 0, 0);
    return acc;
  }
}

// A tile of BM x BN outputs (gated: BN counts the columns of both products, 16 of the gate's
// next to 16 of the up projection's, so a wave holds both for its columns) by WM x WN waves.
// A step stages 128 bytes of k of every operand row (BM + BN rows) in LDS by direct copies,
// S buffers deep; vector v of row r lies at r * 128 + 16 (v ^ (r >> 1 & 7)), which spreads
// the 16 rows of a fragment read over all banks.  The depth's last part of a step (depth is
// a multiple of 16 bytes) goes through registers, zeros behind its end.  Rows past an
// operand's end repeat its last row and are not stored.
template <typename T, int BM_, int BN_, int WM_, int WN_, int S_, int WAVES_PER_SIMD_>
struct TileConfig {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, S = S_, waves = WM_ * WN_;
  static constexpr int threads = 64 * waves, per_simd = WAVES_PER_SIMD_;
  static constexpr int rows = BM + BN;           // staged rows per step
  static constexpr int copies = rows / 8 / waves;  // direct copies per wave and step
  static constexpr int lds = S * rows * 128;
  static_assert(rows % (8 * waves) == 0 && BM % 8 == 0, "a copy holds rows of one operand");
};

template <typename T, typename C, bool GATED, bool PARTIAL>
__global__ void __launch_bounds__(C::threads, C::per_simd) gemm_kernel(GemmParams a) {
  constexpr int NQ = GATED ? 2 : 1;
  constexpr int FM = C::BM / C::WM / 16, FN = C::BN / C::WN / 16;
  constexpr int CC = C::BN / NQ;  // output columns of a tile
  static_assert(!GATED || FN % 2 == 0, "a wave holds both products of its columns");
  __shared__ __attribute__((aligned(16))) unsigned char lds[C::lds];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, q = lane >> 4;

  // consecutive workgroups go to the 8 XCDs in turn: give each XCD a run of tiles, walked
  // down groups of 8 row bands so that its L2 serves a compact block of the output
  const int total = a.tiles_m * a.tiles_n;
  const int split = blockIdx.x / total, b = blockIdx.x - split * total;
  const int xcd = b & 7, per = total >> 3, more = total & 7;
  const int tile = xcd * per + (xcd < more ? xcd : more) + (b >> 3);
  constexpr int kGroup = 8;
  const int group = tile / (kGroup * a.tiles_n), in = tile - group * kGroup * a.tiles_n;
  const int first = group * kGroup, height = a.tiles_m - first < kGroup ? a.tiles_m - first : kGroup;
  const int64_t row0 = int64_t(first + in % height) * C::BM, col0 = int64_t(in / height) * CC;

  // this split's steps
  const int64_t bytes = a.depth * sizeof(T);
  const int all = static_cast<int>((bytes + 127) >> 7);
  const int step0 = static_cast<int>(int64_t(all) * split / a.splits);
  const int steps = static_cast<int>(int64_t(all) * (split + 1) / a.splits) - step0;
  const int tail = step0 + steps == all ? static_cast<int>(bytes & 127) : 0;  // bytes of the last step if short
  const int full = steps - (tail != 0);

  // where this lane reads: copy j of the wave fills staged rows 8 (wave copies + j) + lane / 8
  const unsigned char* src[C::copies];
#pragma unroll
  for (int j = 0; j < C::copies; ++j) {
    const int r = 8 * (wave * C::copies + j) + (lane >> 3);
    const int v = (lane & 7) ^ ((r >> 1) & 7);
    const MatIn* m;
    int64_t i, n;
    if (r < C::BM) {
      m = &a.p;
      i = row0 + r;
      n = a.rows;
    } else {
      const int rq = r - C::BM;
      m = &a.q[GATED ? (rq >> 4) & 1 : 0];
      i = col0 + (GATED ? (rq >> 5) * 16 + (rq & 15) : rq);
      n = a.cols;
    }
    if (i >= n) i = n - 1;
    src[j] = static_cast<const unsigned char*>(m->p) + i * m->ld * int64_t(sizeof(T)) + int64_t(step0) * 128 + v * 16;
  }
  auto stage = [&](int t) {
    const int at = (t % C::S) * C::rows * 128 + wave * C::copies * 1024;
    if (t < full) {
#pragma unroll
      for (int j = 0; j < C::copies; ++j) {
        copy_to_lds(src[j], lds + at + j * 1024);
        src[j] += 128;
      }
    } else {
#pragma unroll
      for (int j = 0; j < C::copies; ++j) {
        const int r = 8 * (wave * C::copies + j) + (lane >> 3);
        const int v = (lane & 7) ^ ((r >> 1) & 7);
        u32x4 d = {0, 0, 0, 0};
        if (v * 16 < tail) d = *reinterpret_cast<const u32x4*>(src[j]);
        *reinterpret_cast<u32x4*>(lds + at + j * 1024 + lane * 16) = d;
      }
    }
  };

  f32x4 acc[FM][FN] = {};
  const int wm = wave / C::WN, wn = wave % C::WN;
  const int rd = 16 * (q ^ (c >> 1));  // vectors 4 .. 7 of a row lie at rd ^ 64
  const int rp = (wm * FM * 16 + c) * 128, rq = (C::BM + wn * FN * 16 + c) * 128;
#pragma unroll
  for (int t = 0; t < C::S - 1; ++t)
    if (t < steps) stage(t);
  for (int t = 0; t < steps; ++t) {
    if (t + C::S - 2 < full)
      copies_then_barrier<(C::S - 2) * C::copies>();
    else
      copies_then_barrier<0>();
    if (t + C::S - 1 < steps) stage(t + C::S - 1);
    const unsigned char* buf = lds + (t % C::S) * C::rows * 128;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      u32x4 pv[FM], qv[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j) qv[j] = *reinterpret_cast<const u32x4*>(buf + rq + (rd ^ (kk * 64)) + j * 2048);
#pragma unroll
      for (int i = 0; i < FM; ++i) pv[i] = *reinterpret_cast<const u32x4*>(buf + rp + (rd ^ (kk * 64)) + i * 2048);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = mfma16<T>(qv[j], pv[i], acc[i][j]);
    }
  }

#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int64_t m = row0 + (wm * FM + i) * 16 + c;
    if (m >= a.rows) continue;
#pragma unroll
    for (int j = 0; j < FN; j += NQ) {
      const int64_t n = col0 + (wn * FN + j) / NQ * 16 + 4 * q;
      if (n >= a.cols) continue;
      if constexpr (PARTIAL) {
#pragma unroll
        for (int h = 0; h < NQ; ++h)
          *reinterpret_cast<f32x4*>(a.part + ((int64_t(split) * NQ + h) * a.rows + m) * a.cols + n) = acc[i][j + h];
      } else {
        f32x4 z[NQ];
#pragma unroll
        for (int h = 0; h < NQ; ++h) z[h] = acc[i][j + h];
        finish4<T, GATED>(a, m, n, z);
      }
    }
  }
}

// Join a split contraction: the parts' sums in order, then the epilogue.
template <typename T, bool GATED>
__global__ void __launch_bounds__(256) join_kernel(GemmParams a) {
  constexpr int NQ = GATED ? 2 : 1;
  const int64_t quads = a.rows * (a.cols / 4);
  const int64_t v = blockIdx.x * 256ll + threadIdx.x;
  if (v >= quads) return;
  const int64_t m = v / (a.cols / 4);
  const int64_t n = (v - m * (a.cols / 4)) * 4;
  f32x4 z[NQ] = {};
  for (int s = 0; s < a.splits; ++s)
#pragma unroll
    for (int h = 0; h < NQ; ++h)
      z[h] += *reinterpret_cast<const f32x4*>(a.part + ((int64_t(s) * NQ + h) * a.rows + m) * a.cols + n);
  finish4<T, GATED>(a, m, n, z);
}

template <typename T>
struct Tiles {
  using Big = TileConfig<T, 256, 256, 2, 4, 2, 2>;
  using Mid = TileConfig<T, 128, 128, 2, 2, 2, 2>;
  using Small = TileConfig<T, 64, 64, 2, 2, 3, 2>;
};

template <typename T, typename C, bool GATED>
hipError_t launch_tiles(GemmParams a, hipStream_t s) {
  a.tiles_m = static_cast<int32_t>((a.rows + C::BM - 1) / C::BM);
  a.tiles_n = (a.cols + C::BN / (GATED ? 2 : 1) - 1) / (C::BN / (GATED ? 2 : 1));
  const unsigned grid = static_cast<unsigned>(a.tiles_m) * a.tiles_n * a.splits;
  if (a.splits > 1) {
    gemm_kernel<T, C, GATED, true><<<grid, C::threads, 0, s>>>(a);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    const int64_t quads = a.rows * (a.cols / 4);
    join_kernel<T, GATED><<<static_cast<unsigned>((quads + 255) / 256), 256, 0, s>>>(a);
  } else {
    gemm_kernel<T, C, GATED, false><<<grid, C::threads, 0, s>>>(a);
  }
  return hipGetLastError();
}

// Which tile, and into how many parts the contraction is split.
struct Plan {
  int tile;    // 0: 256 x 256, 1: 128 x 128, 2: 64 x 64
  int splits;
};
constexpr int kMaxSplits = 16;

Plan plan_gemm(int64_t rows, int64_t cols, int64_t depth, int gated, int esz) {
  const int64_t n = gated ? 2 * cols : cols;
  auto tiles = [&](int64_t t) { return ((rows + t - 1) / t) * ((n + t - 1) / t); };
  const int64_t steps = (depth * esz + 127) / 128;
  if (tiles(256) >= 192) return {0, 1};
  const int tile = tiles(128) >= 192 ? 1 : 2;
  const int64_t have = tiles(tile == 1 ? 128 : 64);
  int64_t splits = 512 / have;
  if (splits > steps / 8) splits = steps / 8;
  if (splits > kMaxSplits) splits = kMaxSplits;
  return {tile, static_cast<int>(splits < 1 ? 1 : splits)};
}

int64_t plan_bytes(const Plan& p, int64_t rows, int64_t cols, int gated) {
  return p.splits > 1 ? int64_t(p.splits) * (gated ? 2 : 1) * rows * cols * 4 : 0;
}

template <typename T, bool GATED>
hipError_t launch_gemm(GemmParams a, float* part, hipStream_t s) {
  const Plan p = plan_gemm(a.rows, a.cols, a.depth, GATED, sizeof(T));
  a.splits = p.splits;
  a.part = part;
  if (p.tile == 0) return launch_tiles<T, typename Tiles<T>::Big, GATED>(a, s);
  if (p.tile == 1) return launch_tiles<T, typename Tiles<T>::Mid, GATED>(a, s);
  return launch_tiles<T, typename Tiles<T>::Small, GATED>(a, s);
}

// ---- slopes and transposed copies ----------------------------------------------------
// 64 x 64 tiles; a transposed copy goes through LDS so that both sides move 16-byte vectors.
constexpr int kSide = 64;

template <typename T>
struct alignas(16) Vec16 {
  T e[16 / sizeof(T)];
};

// Store the tile t[row][col] as out[col][row]: columns n0 .. (< cols), rows m0 .. (< m_end).
template <typename T>
__device__ __forceinline__ void store_transposed(const T (*t)[kSide + 16 / sizeof(T)], T* out, int64_t ld, int64_t m0,
                                                 int64_t m_end, int64_t n0, int64_t cols) {
  constexpr int VEC = 16 / sizeof(T), PER = kSide / VEC;
  for (int v = threadIdx.x; v < kSide * PER; v += 256) {
    const int n = v / PER, m = (v % PER) * VEC;
    if (n0 + n >= cols || m0 + m >= m_end) continue;
    Vec16<T> d;
#pragma unroll
    for (int e = 0; e < VEC; ++e) d.e[e] = t[m + e][n];
    *reinterpret_cast<Vec16<T>*>(out + (n0 + n) * ld + m0 + m) = d;
  }
}

// out[j][i] = m[i][j] for an [n_rows][cols] matrix and i < n_out, a multiple of 16 bytes; zeros
// from n_rows on.
template <typename T>
__global__ void __launch_bounds__(256) transpose_kernel(MatIn m, T* out, int64_t ld_out, int64_t n_out,
                                                        int64_t n_rows, int64_t cols, int64_t tiles_n) {
  constexpr int VEC = 16 / sizeof(T), PER = kSide / VEC;
  __shared__ __attribute__((aligned(16))) T t[kSide][kSide + VEC];
  const int64_t m0 = (blockIdx.x / tiles_n) * kSide, n0 = (blockIdx.x % tiles_n) * kSide;
  for (int v = threadIdx.x; v < kSide * PER; v += 256) {
    const int r = v / PER, n = (v % PER) * VEC;
    Vec16<T> d = {};
    if (m0 + r < n_rows && n0 + n < cols)
      d = *reinterpret_cast<const Vec16<T>*>(static_cast<const T*>(m.p) + (m0 + r) * m.ld + n0 + n);
    *reinterpret_cast<Vec16<T>*>(&t[r][n]) = d;
  }
  __syncthreads();
  store_transposed<T>(t, out, ld_out, m0, n_out, n0, cols);
}

struct SlopeParams {
  MatIn dy;
  MatIn pre[2];
  void* dz;        // null or [rows][ld_z]: dz, or dg in columns 0 .., du in columns cols ..
  int64_t ld_z;
  void* dzt;       // null or [cols (x 2)][ld_t]: the same transposed, zeros behind rows
  int64_t ld_t;
  float* sums;     // null or [tile rows][cols (x 2)]: column sums of each 64-row tile
  int64_t rows;
  int32_t cols;
  int32_t tiles_n;
  int32_t act;
};

// dz = dy act'(z), or dg = dy u act'(g), du = dy act(g), in every form the products and the
// bias gradients read, in one pass over dy and the saved pre-activations.
template <typename T, bool GATED>
__global__ void __launch_bounds__(256) slope_kernel(SlopeParams a) {
  constexpr int VEC = 16 / sizeof(T), PER = kSide / VEC, RSTEP = 256 / PER;
  constexpr int NQ = GATED ? 2 : 1;
  __shared__ __attribute__((aligned(16))) T t[NQ][kSide][kSide + VEC];
  __shared__ float part[RSTEP][kSide];
  const int64_t m0 = int64_t(blockIdx.x / a.tiles_n) * kSide, n0 = int64_t(blockIdx.x % a.tiles_n) * kSide;
  const int n = (threadIdx.x % PER) * VEC;
  float sum[NQ][VEC] = {};
  for (int r = threadIdx.x / PER; r < kSide; r += RSTEP) {
    const int64_t m = m0 + r;
    const bool in = m < a.rows && n0 + n < a.cols;
    Vec16<T> d = {}, z = {}, u = {}, out[NQ] = {};
    if (in) {
      d = *reinterpret_cast<const Vec16<T>*>(static_cast<const T*>(a.dy.p) + m * a.dy.ld + n0 + n);
      if (GATED || a.act != ADA_ACT_NONE)
        z = *reinterpret_cast<const Vec16<T>*>(static_cast<const T*>(a.pre[0].p) + m * a.pre[0].ld + n0 + n);
      if constexpr (GATED)
        u = *reinterpret_cast<const Vec16<T>*>(static_cast<const T*>(a.pre[1].p) + m * a.pre[1].ld + n0 + n);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float dv = to_f32<T>(d.e[e]), zv = to_f32<T>(z.e[e]);
        float g = dv * act_slope(zv, a.act);
        if constexpr (GATED) {
          g *= to_f32<T>(u.e[e]);
          const float w = dv * act_value(zv, a.act);
          sum[1][e] += w;
          out[1].e[e] = from_f32<T>(w);
        }
        sum[0][e] += g;
        out[0].e[e] = from_f32<T>(g);
      }
      if (a.dz != nullptr) {
#pragma unroll
        for (int h = 0; h < NQ; ++h)
          *reinterpret_cast<Vec16<T>*>(static_cast<T*>(a.dz) + m * a.ld_z + h * a.cols + n0 + n) = out[h];
      }
    }
#pragma unroll
    for (int h = 0; h < NQ; ++h) *reinterpret_cast<Vec16<T>*>(&t[h][r][n]) = out[h];
  }
  __syncthreads();
  if (a.dzt != nullptr) {
#pragma unroll
    for (int h = 0; h < NQ; ++h)
      store_transposed<T>(t[h], static_cast<T*>(a.dzt) + int64_t(h) * a.cols * a.ld_t, a.ld_t, m0, a.ld_t, n0,
                          a.cols);
  }
  if (a.sums != nullptr) {
#pragma unroll
    for (int h = 0; h < NQ; ++h) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < VEC; ++e) part[threadIdx.x / PER][n + e] = sum[h][e];
      __syncthreads();
      if (threadIdx.x < kSide && n0 + threadIdx.x < a.cols) {
        float s = 0.f;
        for (int r = 0; r < RSTEP; ++r) s += part[r][threadIdx.x];
        a.sums[(int64_t(blockIdx.x / a.tiles_n) * NQ + h) * a.cols + n0 + threadIdx.x] = s;
      }
    }
  }
}

// dbias: the tiles' column sums in a fixed order, four chains per column.
template <typename T>
__global__ void __launch_bounds__(256) bias_grad_kernel(const float* sums, int64_t tiles, int parts, int cols, T* db0,
                                                        T* db1) {
  __shared__ float part[4][64];
  const int c = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int h = blockIdx.y, n = blockIdx.x * 64 + c;
  float s = 0.f;
  if (n < cols)
    for (int64_t i = w; i < tiles; i += 4) s += sums[(i * parts + h) * cols + n];
  part[w][c] = s;
  __syncthreads();
  T* db = h == 0 ? db0 : db1;
  if (w == 0 && n < cols && db != nullptr) db[n] = from_f32<T>((part[0][c] + part[1][c]) + (part[2][c] + part[3][c]));
}

template <typename T>
hipError_t launch_linear_t(const LinearParams& p, void* ws, hipStream_t s) {
  GemmParams a{};
  a.p = p.x;
  a.q[0] = p.w[0];
  a.q[1] = p.w[1];
  a.bias[0] = p.bias[0];
  a.bias[1] = p.bias[1];
  a.res = p.res;
  a.y[0] = p.y;
  a.pre[0] = p.pre[0];
  a.pre[1] = p.pre[1];
  a.rows = p.rows;
  a.row_split = p.rows;
  a.cols = p.d_out;
  a.depth = p.d_in;
  a.act = p.act;
  return p.gated ? launch_gemm<T, true>(a, static_cast<float*>(ws), s)
                 : launch_gemm<T, false>(a, static_cast<float*>(ws), s);
}

// Workspace of a backward pass (byte offsets): dz [rows][parts d_out] and the weights'
// transposed copy [d_in][parts d_out] for dx; dz transposed [parts d_out][ld_t] and x
// transposed [d_in][ld_t] for dW; column sums for dbias; parts of a split contraction.
struct GradPlan {
  int64_t dz, wt, dzt, xt, sums, part, total;
  int64_t ld_t;
};

GradPlan plan_grad(int64_t rows, int64_t n, int64_t k, int act, int gated, int esz) {
  GradPlan g{};
  const int64_t parts = gated ? 2 : 1;
  auto take = [&](int64_t bytes) {
    const int64_t at = g.total;
    g.total += (bytes + 255) / 256 * 256;
    return at;
  };
  g.ld_t = (rows + 16 / esz - 1) / (16 / esz) * (16 / esz);
  g.dz = take(gated || act != ADA_ACT_NONE ? rows * parts * n * esz : 0);
  g.wt = take(k * parts * n * esz);
  g.dzt = take(parts * n * g.ld_t * esz);
  g.xt = take(k * g.ld_t * esz);
  g.sums = take((rows + kSide - 1) / kSide * parts * n * 4);
  const int64_t dx = plan_bytes(plan_gemm(rows, k, parts * n, 0, esz), rows, k, 0);
  const int64_t dw2 = plan_bytes(plan_gemm(parts * n, k, g.ld_t, 0, esz), parts * n, k, 0);
  const int64_t dw1 = plan_bytes(plan_gemm(n, k, g.ld_t, 0, esz), n, k, 0);
  g.part = take(dx > dw2 ? (dx > dw1 ? dx : dw1) : (dw2 > dw1 ? dw2 : dw1));
  return g;
}

template <typename T>
hipError_t launch_transpose(const MatIn& m, T* out, int64_t ld_out, int64_t n_out, int64_t n_rows, int64_t cols,
                            hipStream_t s) {
  const int64_t tm = (n_out + kSide - 1) / kSide, tn = (cols + kSide - 1) / kSide;
  transpose_kernel<T><<<static_cast<unsigned>(tm * tn), 256, 0, s>>>(m, out, ld_out, n_out, n_rows, cols, tn);
  return hipGetLastError();
}

template <typename T>
__global__ void __launch_bounds__(256) zero_kernel(MatOut y, int64_t rows, int64_t cols) {
  for (int64_t v = blockIdx.x * 256ll + threadIdx.x; v < rows * cols; v += gridDim.x * 256ll)
    static_cast<T*>(y.p)[(v / cols) * y.ld + v % cols] = from_f32<T>(0.f);
}

template <typename T>
hipError_t launch_zero(const MatOut& y, int64_t rows, int64_t cols, hipStream_t s) {
  if (y.p == nullptr) return hipSuccess;
  const int64_t blocks = (rows * cols + 255) / 256;
  zero_kernel<T><<<static_cast<unsigned>(blocks < 4096 ? blocks : 4096), 256, 0, s>>>(y, rows, cols);
  return hipGetLastError();
}

#define ADA_TRY(call) \
  if (const hipError_t e_ = (call); e_ != hipSuccess) return e_

template <typename T>
hipError_t launch_linear_grad_t(const LinearGradParams& p, void* ws, hipStream_t s) {
  const int parts = p.gated ? 2 : 1;
  const int64_t n = p.d_out, k = p.d_in;
  if (p.rows == 0) {  // sums over no rows
    for (int h = 0; h < parts; ++h) {
      ADA_TRY(launch_zero<T>(p.dw[h], n, k, s));
      ADA_TRY(launch_zero<T>(MatOut{p.dbias[h], n}, 1, n, s));
    }
    return hipSuccess;
  }
  const GradPlan g = plan_grad(p.rows, n, k, p.act, p.gated, sizeof(T));
  unsigned char* base = static_cast<unsigned char*>(ws);
  T* wt = reinterpret_cast<T*>(base + g.wt);
  T* dzt = reinterpret_cast<T*>(base + g.dzt);
  T* xt = reinterpret_cast<T*>(base + g.xt);
  float* part = reinterpret_cast<float*>(base + g.part);
  const bool want_dx = p.dx.p != nullptr, want_dw = p.dw[0].p != nullptr || p.dw[1].p != nullptr;
  const bool want_db = p.dbias[0] != nullptr || p.dbias[1] != nullptr;
  const bool own_dz = p.gated || p.act != ADA_ACT_NONE;  // else dz is dy

  SlopeParams sl{};
  sl.dy = p.dy;
  sl.pre[0] = p.pre[0];
  sl.pre[1] = p.pre[1];
  sl.dz = own_dz && want_dx ? base + g.dz : nullptr;
  sl.ld_z = parts * n;
  sl.dzt = want_dw ? dzt : nullptr;
  sl.ld_t = g.ld_t;
  sl.sums = want_db ? reinterpret_cast<float*>(base + g.sums) : nullptr;
  sl.rows = p.rows;
  sl.cols = p.d_out;
  sl.tiles_n = (p.d_out + kSide - 1) / kSide;
  sl.act = p.act;
  const int64_t tiles_m = (p.rows + kSide - 1) / kSide;
  if (sl.dz != nullptr || sl.dzt != nullptr || sl.sums != nullptr) {
    const unsigned grid = static_cast<unsigned>(tiles_m * sl.tiles_n);
    if (p.gated)
      slope_kernel<T, true><<<grid, 256, 0, s>>>(sl);
    else
      slope_kernel<T, false><<<grid, 256, 0, s>>>(sl);
    ADA_TRY(hipGetLastError());
  }
  if (want_db) {
    bias_grad_kernel<T><<<dim3((p.d_out + 63) / 64, parts), 256, 0, s>>>(sl.sums, tiles_m, parts, p.d_out,
                                                                         static_cast<T*>(p.dbias[0]),
                                                                         static_cast<T*>(p.dbias[1]));
    ADA_TRY(hipGetLastError());
  }
  if (want_dx) {
    for (int h = 0; h < parts; ++h) ADA_TRY(launch_transpose<T>(p.w[h], wt + h * n, parts * n, n, n, k, s));
    GemmParams a{};
    a.p = own_dz ? MatIn{base + g.dz, parts * n} : p.dy;
    a.q[0] = MatIn{wt, parts * n};
    a.y[0] = p.dx;
    a.rows = p.rows;
    a.row_split = p.rows;
    a.cols = p.d_in;
    a.depth = parts * n;
    ADA_TRY((launch_gemm<T, false>(a, part, s)));
  }
  if (want_dw) {
    ADA_TRY(launch_transpose<T>(p.x, xt, g.ld_t, g.ld_t, p.rows, k, s));
    const bool both = p.gated && p.dw[0].p != nullptr && p.dw[1].p != nullptr;
    const int h = p.dw[0].p != nullptr ? 0 : 1;
    GemmParams a{};
    a.p = MatIn{dzt + h * n * g.ld_t, g.ld_t};
    a.q[0] = MatIn{xt, g.ld_t};
    a.y[0] = p.dw[h];
    a.y[1] = p.dw[1];
    a.rows = both ? 2 * n : n;
    a.row_split = n;
    a.cols = p.d_in;
    a.depth = g.ld_t;
    ADA_TRY((launch_gemm<T, false>(a, part, s)));
  }
  return hipSuccess;
}

}  // namespace

int64_t linear_workspace(int64_t rows, int32_t d_out, int32_t d_in, int gated, int dtype) {
  if (rows == 0) return 0;
  return plan_bytes(plan_gemm(rows, d_out, d_in, gated, dtype == ADA_BF16 ? 2 : 4), rows, d_out, gated);
}

int64_t linear_grad_workspace(int64_t rows, int32_t d_out, int32_t d_in, int act, int gated, int dtype) {
  return rows == 0 ? 0 : plan_grad(rows, d_out, d_in, act, gated, dtype == ADA_BF16 ? 2 : 4).total;
}

hipError_t launch_linear(const LinearParams& p, int dtype, void* ws, hipStream_t s) {
  if (p.rows == 0) return hipSuccess;
  return dtype == ADA_BF16 ? launch_linear_t<uint16_t>(p, ws, s) : launch_linear_t<float>(p, ws, s);
}

hipError_t launch_linear_grad(const LinearGradParams& p, int dtype, void* ws, hipStream_t s) {
  return dtype == ADA_BF16 ? launch_linear_grad_t<uint16_t>(p, ws, s) : launch_linear_grad_t<float>(p, ws, s);
}

}  // namespace ada
