// Linear and gated feed-forward products with their epilogues, and their backward passes.
//
//   linear   z = x W^T + b,  y = act(z) + residual                       [rows, d_out]
//   glu      g = x Wg^T + bg, u = x Wu^T + bu,  y = act(g) u
//   backward dz = dy act'(z) (dg = dy u act'(g), du = dy act(g)),
//            dx = dz W (dg Wg + du Wu), dW = dz^T x, db = sum over rows of dz
//
// Every product is D(i, j) = sum_k P(i, k) Q(j, k) on the matrix instructions with fp32
// sums; an operand is read along k (x and W of the forward pass) or across it (W of dx,
// dz and x of dW).  Matrix instruction layout (16 x 16 tile): lane l = 16 q + c supplies
// Q(c, k) as the row operand and P(c, k) as the column operand for its k slice, and
// receives D(i = c, j = 4 q .. 4 q + 3), four consecutive columns of an output row.  A
// 16-byte vector per lane feeds one 16x16x32 instruction in bf16 and four 16x16x4 ones in
// fp32 (the instruction's k order is free as long as both operands share it).
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
// 64 x 64 outputs per workgroup of four waves (32 x 32 each); a step stages 64 rows x 128
// bytes of k of each operand in LDS.
constexpr int kTile = 64;
constexpr int kPitch = 128 + 16;  // bytes of a staged row: 16-byte vectors of 16 rows fall on all banks

struct GemmParams {
  MatIn p[2];  // P of contraction segment s
  MatIn q[2];  // Q of segment s (gated: q[0], q[1] are the two weights of one segment)
  const void* bias[2];
  MatIn res;
  MatOut y;
  MatOut pre[2];
  int64_t rows;
  int32_t cols;
  int64_t depth;  // k per segment
  int32_t segs;
  int32_t act;
};

// Stage rows row0 .. row0 + 63 of an operand, k0 .. k0 + KB - 1, zero outside.  Across:
// the operand's memory runs along its rows (element (i, k) at p[k * ld + i]).
template <typename T, bool ACROSS>
__device__ __forceinline__ void stage_tile(unsigned char* lds, const MatIn& m, int64_t row0, int64_t n_rows, int64_t k0,
                                           int64_t depth) {
  constexpr int VEC = 16 / sizeof(T), KB = 128 / sizeof(T);
  const T* base = static_cast<const T*>(m.p);
  for (int v = threadIdx.x; v < kTile * 8; v += 256) {
    if constexpr (!ACROSS) {
      const int r = v >> 3, c = v & 7;
      const int64_t i = row0 + r, k = k0 + c * VEC;
      u32x4 d = {0, 0, 0, 0};
      if (i < n_rows && k < depth) d = *reinterpret_cast<const u32x4*>(base + i * m.ld + k);
      *reinterpret_cast<u32x4*>(lds + r * kPitch + c * 16) = d;
    } else {
      constexpr int PER = kTile / VEC;
      const int kk = v / PER, r = (v % PER) * VEC;
      const int64_t i = row0 + r, k = k0 + kk;
      struct alignas(16) Vec { T e[VEC]; } d = {};
      if (i < n_rows && k < depth) d = *reinterpret_cast<const Vec*>(base + k * m.ld + i);
#pragma unroll
      for (int e = 0; e < VEC; ++e) *reinterpret_cast<T*>(lds + (r + e) * kPitch + kk * sizeof(T)) = d.e[e];
    }
  }
  static_assert(KB * sizeof(T) == 128, "a staged row is 128 bytes");
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

template <typename T, bool P_ACROSS, bool Q_ACROSS, bool GATED>
__global__ void __launch_bounds__(256) gemm_kernel(GemmParams a) {
  constexpr int KB = 128 / sizeof(T);
  constexpr int NQ = GATED ? 2 : 1;
  __shared__ __attribute__((aligned(16))) unsigned char lds[(1 + NQ) * kTile * kPitch];
  const int64_t row0 = int64_t(blockIdx.y) * kTile;
  const int64_t col0 = int64_t(blockIdx.x) * kTile;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane & 15, q = lane >> 4;
  const int wr = (wave & 1) * 32, wc = (wave >> 1) * 32;
  f32x4 acc[NQ][2][2] = {};
  for (int s = 0; s < a.segs; ++s) {
    for (int64_t k0 = 0; k0 < a.depth; k0 += KB) {
      __syncthreads();
      stage_tile<T, P_ACROSS>(lds, a.p[s], row0, a.rows, k0, a.depth);
      for (int h = 0; h < NQ; ++h)
        stage_tile<T, Q_ACROSS>(lds + (1 + h) * kTile * kPitch, a.q[GATED ? h : s], col0, a.cols, k0, a.depth);
      __syncthreads();
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        u32x4 pv[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          pv[i] = *reinterpret_cast<const u32x4*>(lds + (wr + 16 * i + c) * kPitch + (4 * kk + q) * 16);
#pragma unroll
        for (int h = 0; h < NQ; ++h)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const u32x4 qv = *reinterpret_cast<const u32x4*>(lds + (1 + h) * kTile * kPitch +
                                                             (wc + 16 * j + c) * kPitch + (4 * kk + q) * 16);
#pragma unroll
            for (int i = 0; i < 2; ++i) acc[h][i][j] = mfma16<T>(qv, pv[i], acc[h][i][j]);
          }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t m = row0 + wr + 16 * i + c;
    if (m >= a.rows) continue;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t n = col0 + wc + 16 * j + 4 * q;
      if (n >= a.cols) continue;
      float z[NQ][4], o[4];
#pragma unroll
      for (int h = 0; h < NQ; ++h) {
        float b[4] = {0.f, 0.f, 0.f, 0.f};
        if (a.bias[h] != nullptr) load4(static_cast<const T*>(a.bias[h]) + n, b);
#pragma unroll
        for (int e = 0; e < 4; ++e) z[h][e] = acc[h][i][j][e] + b[e];
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
      store4(static_cast<T*>(a.y.p) + m * a.y.ld + n, o);
    }
  }
}

template <typename T, bool PA, bool QA, bool GATED>
hipError_t launch_gemm(const GemmParams& a, hipStream_t s) {
  const dim3 grid((a.cols + kTile - 1) / kTile, static_cast<unsigned>((a.rows + kTile - 1) / kTile));
  gemm_kernel<T, PA, QA, GATED><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

// ---- slopes: dz = dy act'(z), or dg = dy u act'(g), du = dy act(g) --------------------
template <typename T, bool GATED>
__global__ void __launch_bounds__(256) slope_kernel(MatIn dy, MatIn g, MatIn u, T* dz, T* du, int64_t rows, int cols,
                                                    int act) {
  const int64_t quads = rows * (cols / 4);
  for (int64_t v = blockIdx.x * 256ll + threadIdx.x; v < quads; v += gridDim.x * 256ll) {
    const int64_t m = v / (cols / 4);
    const int n = static_cast<int>(v - m * (cols / 4)) * 4;
    float d[4], z[4], up[4], a[4], b[4];
    load4(static_cast<const T*>(dy.p) + m * dy.ld + n, d);
    load4(static_cast<const T*>(g.p) + m * g.ld + n, z);
    if constexpr (GATED) load4(static_cast<const T*>(u.p) + m * u.ld + n, up);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[e] = d[e] * act_slope(z[e], act);
      if constexpr (GATED) {
        a[e] *= up[e];
        b[e] = d[e] * act_value(z[e], act);
      }
    }
    store4(dz + m * cols + n, a);
    if constexpr (GATED) store4(du + m * cols + n, b);
  }
}

// dbias: one workgroup per 64 columns walks every row; the sums take the unrounded dz, in a
// fixed order.
template <typename T, bool GATED>
__global__ void __launch_bounds__(256) bias_grad_kernel(MatIn dy, MatIn g, MatIn u, T* db0, T* db1, int64_t rows,
                                                        int cols, int act) {
  __shared__ float part[2][4][64];
  const int c = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int n = blockIdx.x * 64 + c;
  float s0 = 0.f, s1 = 0.f;
  if (n < cols) {
    for (int64_t m = w; m < rows; m += 4) {
      const float d = to_f32<T>(static_cast<const T*>(dy.p)[m * dy.ld + n]);
      const float z = act == ADA_ACT_NONE && !GATED ? 0.f : to_f32<T>(static_cast<const T*>(g.p)[m * g.ld + n]);
      float a = d * act_slope(z, act);
      if constexpr (GATED) {
        a *= to_f32<T>(static_cast<const T*>(u.p)[m * u.ld + n]);
        s1 += d * act_value(z, act);
      }
      s0 += a;
    }
  }
  part[0][w][c] = s0;
  part[1][w][c] = s1;
  __syncthreads();
  if (w == 0 && n < cols) {
    if (db0 != nullptr) db0[n] = from_f32<T>((part[0][0][c] + part[0][1][c]) + (part[0][2][c] + part[0][3][c]));
    if (db1 != nullptr) db1[n] = from_f32<T>((part[1][0][c] + part[1][1][c]) + (part[1][2][c] + part[1][3][c]));
  }
}

template <typename T>
hipError_t launch_linear_t(const LinearParams& p, hipStream_t s) {
  GemmParams a{};
  a.p[0] = p.x;
  a.q[0] = p.w[0];
  a.q[1] = p.w[1];
  a.bias[0] = p.bias[0];
  a.bias[1] = p.bias[1];
  a.res = p.res;
  a.y = p.y;
  a.pre[0] = p.pre[0];
  a.pre[1] = p.pre[1];
  a.rows = p.rows;
  a.cols = p.d_out;
  a.depth = p.d_in;
  a.segs = 1;
  a.act = p.act;
  return p.gated ? launch_gemm<T, false, false, true>(a, s) : launch_gemm<T, false, false, false>(a, s);
}

template <typename T>
hipError_t launch_linear_grad_t(const LinearGradParams& p, void* ws, hipStream_t s) {
  const int parts = p.gated ? 2 : 1;
  MatIn dz[2] = {p.dy, p.dy};
  const bool want_bias = p.dbias[0] != nullptr || p.dbias[1] != nullptr;
  const bool want_dz = p.dx.p != nullptr || p.dw[0].p != nullptr || p.dw[1].p != nullptr;
  if (want_bias) {
    const unsigned grid = (p.d_out + 63) / 64;
    T* b0 = static_cast<T*>(p.dbias[0]);
    T* b1 = static_cast<T*>(p.dbias[1]);
    if (p.gated)
      bias_grad_kernel<T, true><<<grid, 256, 0, s>>>(p.dy, p.pre[0], p.pre[1], b0, b1, p.rows, p.d_out, p.act);
    else
      bias_grad_kernel<T, false><<<grid, 256, 0, s>>>(p.dy, p.pre[0], p.pre[0], b0, b1, p.rows, p.d_out, p.act);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (want_dz && (p.gated || p.act != ADA_ACT_NONE)) {
    T* z = static_cast<T*>(ws);
    for (int h = 0; h < parts; ++h) dz[h] = MatIn{z + h * p.rows * p.d_out, p.d_out};
    if (p.rows > 0) {
      const int64_t blocks = (p.rows * (p.d_out / 4) + 255) / 256;
      const unsigned grid = static_cast<unsigned>(blocks < 4096 ? blocks : 4096);
      if (p.gated)
        slope_kernel<T, true><<<grid, 256, 0, s>>>(p.dy, p.pre[0], p.pre[1], z, z + p.rows * p.d_out, p.rows, p.d_out,
                                                   p.act);
      else
        slope_kernel<T, false><<<grid, 256, 0, s>>>(p.dy, p.pre[0], p.pre[0], z, z, p.rows, p.d_out, p.act);
      if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
  }
  if (p.dx.p != nullptr && p.rows > 0) {
    GemmParams a{};
    for (int h = 0; h < parts; ++h) {
      a.p[h] = dz[h];
      a.q[h] = p.w[h];
    }
    a.y = p.dx;
    a.rows = p.rows;
    a.cols = p.d_in;
    a.depth = p.d_out;
    a.segs = parts;
    if (const hipError_t e = launch_gemm<T, false, true, false>(a, s); e != hipSuccess) return e;
  }
  for (int h = 0; h < parts; ++h) {
    if (p.dw[h].p == nullptr) continue;
    GemmParams a{};
    a.p[0] = dz[h];
    a.q[0] = p.x;
    a.y = p.dw[h];
    a.rows = p.d_out;
    a.cols = p.d_in;
    a.depth = p.rows;
    a.segs = 1;
    if (const hipError_t e = launch_gemm<T, true, true, false>(a, s); e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

int64_t linear_workspace(int64_t, int32_t, int32_t, int, int) { return 0; }

int64_t linear_grad_workspace(int64_t rows, int32_t d_out, int32_t, int act, int gated, int dtype) {
  if (!gated && act == ADA_ACT_NONE) return 0;
  return rows * d_out * (gated ? 2 : 1) * (dtype == ADA_BF16 ? 2 : 4);
}

hipError_t launch_linear(const LinearParams& p, int dtype, void*, hipStream_t s) {
  if (p.rows == 0) return hipSuccess;
  return dtype == ADA_BF16 ? launch_linear_t<uint16_t>(p, s) : launch_linear_t<float>(p, s);
}

hipError_t launch_linear_grad(const LinearGradParams& p, int dtype, void* ws, hipStream_t s) {
  return dtype == ADA_BF16 ? launch_linear_grad_t<uint16_t>(p, ws, s) : launch_linear_grad_t<float>(p, ws, s);
}

}  // namespace ada
