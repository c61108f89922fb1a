// Linear and gated feed-forward products with their epilogues, and their backward passes.
//
//   linear   z = x W^T + b,  y = act(z) + residual                       [rows, d_out]
//   glu      g = x Wg^T + bg, u = x Wu^T + bu,  y = act(g) u
//   backward dz = dy act'(z) (dg = dy u act'(g), du = dy act(g)),
//            dx = dz W (dg Wg + du Wu), dW = dz^T x, db = sum over rows of dz
//
// Every product is D(i, j) = sum_k P(i, k) Q(j, k) on the matrix instructions with fp32
// sums; an operand is read along k (x and W of the forward pass, dz of dx) or across it, k being
// the row of its memory (W of dx, dz and x of dW).  Matrix instruction layout (32 x
// 32 tile): lane l = 32 q + c supplies Q(c, k) as the row operand and P(c, k) as the column
// operand for its k slice, and receives D(i = c, j = 8 g + 4 q + e) in register 4 g + e:
// groups of four consecutive columns of an output row.  A 16-byte vector per lane feeds one
// 32x32x16 instruction in bf16 and four 32x32x2 ones in fp32 (the instruction's k order is
// free as long as both operands share it).
#include "linear.h"
#include "linear_plan.h"

#include "adafuse.h"

namespace ada {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
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

// Eight consecutive elements (16-byte aligned) as floats, and back.
template <typename T>
struct alignas(16) Vec16 {
  T e[16 / sizeof(T)];
};
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  constexpr int VEC = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < 8; i += VEC) {
    const Vec16<T> d = *reinterpret_cast<const Vec16<T>*>(p + i);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[i + e] = to_f32<T>(d.e[e]);
  }
}
template <bool STREAM = false, typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  constexpr int VEC = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < 8; i += VEC) {
    Vec16<T> d;
#pragma unroll
    for (int e = 0; e < VEC; ++e) d.e[e] = from_f32<T>(v[i + e]);
    if constexpr (STREAM)
      __builtin_nontemporal_store(__builtin_bit_cast(u32x4, d), reinterpret_cast<u32x4*>(p + i));
    else
      *reinterpret_cast<Vec16<T>*>(p + i) = d;
  }
}

// ---- activations: value and slope in fp32 --------------------------------------------
// At +inf the values are +inf; at -inf they are the formula's -inf * 0 = NaN (relu 0).  The
// slopes take their limits, 1 and 0: far out, where the part that falls off is 0, its factor z
// may be infinite and is left out.  NaN stays NaN (relu's slope is a comparison).
// Outputs stored in bf16 take everything from one exponential and one reciprocal, as the
// instructions give them: in the epilogue of a short contraction the activation is a large part
// of the time (1838 x 14248 x 192: gelu 58 us, with erfcf 86; silu 44, with expf and a division
// 62; none 37).  The exponent's rounding makes their tails up to (|z| + 8) 2^-23 (silu) or
// (z^2 + 20) 2^-23 (gelu) of the value off, a small part of bf16's half step of 2^-8 wherever the
// value is not 0.  Outputs stored in fp32 (T = float) are owed those bits: expf, a division, and
// the exponent of gelu's tail with its rounding made good (silu 143 us, gelu 177, none 130).
constexpr float kLog2E = 1.44269504088896340f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kSqrt2OverPi = 0.79788456080286536f;
constexpr float kCubic = 0.044715f;

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }
__device__ __forceinline__ float rcp_fast(float v) { return __builtin_amdgcn_rcpf(v); }

// Phi(-|z|) for the normal distribution's Phi, and e = exp(-z^2 / 2), from
// Phi(-|z|) = erfc(|z| / sqrt 2) / 2 = e t P(t), t = 1 / (1 + 0.38 |z| / sqrt 2): P is fitted to
// exp(x^2) erfc(x) / (2 t), x up to 14, within 3e-8 of it.  No cancellation for z << 0.
template <typename T>
__device__ __forceinline__ float normal_tail(float z, float& e) {
  const float d = 1.f + 0.26870057685088807f * fabsf(z);
  float t;
  if constexpr (sizeof(T) == 4) {
    const float zz = z * z;
    e = expf(-0.5f * zz);
    if (e > 0.f) e = fmaf(e, -0.5f * fmaf(z, z, -zz), e);  // what z * z was rounded by
    t = 1.f / d;
  } else {
    e = exp2_fast(-0.5f * kLog2E * z * z);
    t = rcp_fast(d);
  }
  float q = 0.029212618f;
  q = q * t - 0.12993799f;
  q = q * t + 0.17968433f;
  q = q * t - 0.07843517f;
  q = q * t + 0.1136192f;
  q = q * t + 0.06983649f;
  q = q * t + 0.10184348f;
  q = q * t + 0.10697212f;
  q = q * t + 0.10720492f;
  return q * t * e;
}

// 1 / (1 + e), e = exp(-z).
template <typename T>
__device__ __forceinline__ float logistic(float z, float& e) {
  if constexpr (sizeof(T) == 4) {
    e = expf(-z);
    return 1.f / (1.f + e);
  }
  e = exp2_fast(-kLog2E * z);
  return rcp_fast(1.f + e);
}

// What gelu_tanh's tanh is taken of, twice: (1 + tanh v) / 2 = logistic(2 v).
__device__ __forceinline__ float twice_inner(float z) { return 2.f * kSqrt2OverPi * (z + kCubic * z * z * z); }

template <typename T>
__device__ __forceinline__ float act_value(float z, int act) {
  float e;
  switch (act) {
    case ADA_ACT_RELU: return z < 0.f ? 0.f : z;  // NaN stays NaN
    case ADA_ACT_SILU: return z * logistic<T>(z, e);
    case ADA_ACT_GELU: {
      const float tail = normal_tail<T>(z, e);  // 0 from 15 on, so an infinite z need not meet it
      return z < 0.f ? z * tail : z - fminf(z, 16.f) * tail;
    }
    case ADA_ACT_GELU_TANH: return z * logistic<T>(twice_inner(z), e);
    default: return z;
  }
}

// One choice of the activation for eight values.
template <typename T>
__device__ __forceinline__ void act_values(float (&z)[8], int act) {
#define ADA_EACH(a)                                         \
  case a:                                                   \
    _Pragma("unroll") for (int e = 0; e < 8; ++e) z[e] = act_value<T>(z[e], a); \
    break;
  switch (act) {
    ADA_EACH(ADA_ACT_RELU)
    ADA_EACH(ADA_ACT_SILU)
    ADA_EACH(ADA_ACT_GELU)
    ADA_EACH(ADA_ACT_GELU_TANH)
    default: break;
  }
#undef ADA_EACH
}

template <typename T>
__device__ __forceinline__ float act_slope(float z, int act) {
  float e;
  switch (act) {
    case ADA_ACT_RELU: return z > 0.f ? 1.f : 0.f;
    case ADA_ACT_SILU: {
      const float s = logistic<T>(z, e), fall = e * s;  // 1 - s
      return s == 0.f ? 0.f : fall == 0.f ? s : s * (1.f + z * fall);
    }
    case ADA_ACT_GELU: {
      const float tail = normal_tail<T>(z, e);
      return (z < 0.f ? tail : 1.f - tail) + (e == 0.f ? 0.f : z * kInvSqrt2Pi * e);
    }
    case ADA_ACT_GELU_TANH: {
      const float s = logistic<T>(twice_inner(z), e);
      const float fall = e * s * s;  // s (1 - s): 0 far out, where z * z may be infinite
      return s == 0.f ? 0.f : s + (fall > 0.f ? 2.f * kSqrt2OverPi * z * fall * (1.f + 3.f * kCubic * z * z) : 0.f);
    }
    default: return 1.f;
  }
}

// ---- tiled product -------------------------------------------------------------------
#define ADA_GLOBAL __attribute__((address_space(1)))
#define ADA_LDS __attribute__((address_space(3)))

struct GemmParams {
  MatIn p;                // [rows][depth]; dW: [depth][rows]
  MatIn q[2];             // [cols][depth]; gated: the gate's and the up projection's weights;
                          // dx: [depth][cols], q[1] from row `seam` on; dW: [depth][cols]
  int64_t seam;
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
  int32_t form;           // a Form
};

// How a product reads its operands.
enum Form : int32_t {
  kForward = 0,  // both along k
  kDx = 1,       // P along, Q across
  kDw = 2        // both across
};

// One or two products in a grid: workgroups from `first` on belong to the second.
struct GemmPair {
  GemmParams a[2];
  int32_t first;
};

// A value held in scalar registers from here on: the kernel's arguments lie in memory, and the
// compiler would otherwise load them again in every iteration of an epilogue.
template <typename V>
__device__ __forceinline__ V held(V v) {
  asm volatile("" : "+s"(v));
  return v;
}

// What an epilogue needs of its product.
template <typename T, bool GATED>
struct Epilogue {
  static constexpr int NQ = GATED ? 2 : 1;
  const T* bias[NQ];
  T* pre[NQ];
  int64_t ld_pre[NQ];
  const T* res;
  int64_t ld_res;
  T* y[2];
  int64_t ld_y[2];
  int64_t row_split;
  int act;

  __device__ __forceinline__ explicit Epilogue(const GemmParams& a) {
#pragma unroll
    for (int h = 0; h < NQ; ++h) {
      bias[h] = held(static_cast<const T*>(a.bias[h]));
      pre[h] = held(static_cast<T*>(a.pre[h].p));
      ld_pre[h] = held(a.pre[h].ld);
    }
    res = held(static_cast<const T*>(a.res.p));
    ld_res = held(a.res.ld);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      y[h] = held(static_cast<T*>(a.y[h].p));
      ld_y[h] = held(a.y[h].ld);
    }
    row_split = held(a.row_split);
    act = held(a.act);
  }

  // y, pre of eight consecutive columns n of row m, from the sums without the bias.  STREAM: past
  // the caches, for outputs of whole tiles (gated pair with both saved, 4096 x 11008 x 4096: 656
  // to 641 us).
  template <bool STREAM = false>
  __device__ __forceinline__ void finish8(int64_t m, int64_t n, float (&z)[NQ][8]) const {
#pragma unroll
    for (int h = 0; h < NQ; ++h) {
      if (bias[h] != nullptr) {
        float b[8];
        load8(bias[h] + n, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[h][e] += b[e];
      }
      if (pre[h] != nullptr) store8<STREAM>(pre[h] + m * ld_pre[h] + n, z[h]);
    }
    act_values<T>(z[0], act);
    if constexpr (GATED) {
#pragma unroll
      for (int e = 0; e < 8; ++e) z[0][e] *= z[1][e];
    }
    if (res != nullptr) {
      float r[8];
      load8(res + m * ld_res + n, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) z[0][e] += r[e];
    }
    if (m < row_split)
      store8<STREAM>(y[0] + m * ld_y[0] + n, z[0]);
    else
      store8<STREAM>(y[1] + (m - row_split) * ld_y[1] + n, z[0]);
  }
};

// Sixteen bytes per lane from global memory to LDS, lane l's at lds + 16 l (lds is the same
// in every lane of the wave).
__device__ __forceinline__ void copy_to_lds(const unsigned char* g, unsigned char* lds) {
  __builtin_amdgcn_global_load_lds((const ADA_GLOBAL void*)g, (ADA_LDS void*)lds, 16, 0, 0);
}

// Order the LDS accesses of one wave: what its lanes wrote before is what they read after.
__device__ __forceinline__ void lds_wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Wait until at most N of the wave's copies to LDS are in flight and all its LDS reads and
// writes are done, then meet the workgroup's other waves.
template <int N>
__device__ __forceinline__ void copies_then_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <typename T>
__device__ __forceinline__ f32x16 mfma32(u32x4 q, u32x4 p, f32x16 acc) {
  if constexpr (sizeof(T) == 2) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, q), __builtin_bit_cast(bf16x8, p), acc,
                                                   0, 0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(q[j]), __uint_as_float(p[j]), acc, 0, 0, 0);
    return acc;
  }
}

// A tile of BM x BN outputs (gated: BN counts the columns of both products, 16 of the gate's
// next to 16 of the up projection's, so a wave holds both for its columns) by WM x WN waves.
// A step is 64 (bf16) or 32 (fp32) of k.  One operand's rows of one step are a unit; units go to
// LDS by direct copies into a ring of U slots: 2 t holds P of step t, 2 t + 1 holds Q.  The
// depth's last part of a step goes through registers, zeros behind its end.  Rows past an
// operand's end repeat its last ones and are not stored.
// A unit along k holds 128 bytes of every row: vector v of row r at r * 128 + 16 (v ^ (r >> 1 & 7)),
// which spreads the 32 rows of a fragment read over all banks.  A unit across k holds the operand's
// memory rows, one k each, read one k at a time: in bf16 a lane reads as many neighbouring columns
// as its wave has fragments (F = 4: 8 bytes, F = 2: 4 bytes), fragment x taking columns F c + x,
// and byte permutes pair the k of each column while the matrix instructions run.  Vector v of row
// k lies at v ^ spread(k), so that the two halves of a wave, eight k apart, read different banks.
//
// The large tiles are bound by the matrix pipes at the clock that their power allows (256 x 256
// at 4096 x 8192 x 28672: 1.40 ms, 1375 TFLOP/s, pipes 84% busy; with its copies taken out, 1640).
// One wave per SIMD with 128 x 128 sums in its accumulation registers reads two thirds of the LDS
// bytes of two waves with 128 x 64 each (1280 TFLOP/s).  128 bytes of k a row, because 64-byte
// segments cost the caches a third of their rate (1130 TFLOP/s).  The smaller tiles, for fewer
// rows, are bound by the latency of their copies, hence the longer rings.
template <int BM_, int BN_, int U_, int WAVES_PER_SIMD_>
struct TileConfig {
  static constexpr int BM = BM_, BN = BN_, WM = 2, WN = 2, U = U_, waves = WM * WN;
  static constexpr int threads = 64 * waves, per_simd = WAVES_PER_SIMD_;
  static constexpr int copies_p = BM / 8 / waves, copies_q = BN / 8 / waves;  // direct copies per wave and unit
  static constexpr int win_pitch = BN / WN + 4;       // floats of a row of a wave's epilogue window
  static constexpr int window = 32 * win_pitch * 4;   // its bytes
  static constexpr int ring = BM == BN ? U * BM * 128 : U / 2 * (BM + BN) * 128;
  static constexpr int lds = ring > waves * window ? ring : waves * window;
  // where slot s lies (an even ring keeps P in even slots)
  __device__ static int slot(int s) { return BM == BN ? s * BM * 128 : (s >> 1) * (BM + BN) * 128 + (s & 1) * BM * 128; }
  // of a unit across k with B rows: vectors of a k, and where vector v of k lies
  template <typename T, int B>
  struct Across {
    static constexpr int vecs = B * int(sizeof(T)) / 16;
    __device__ static int spread(int k) { return sizeof(T) == 2 ? (8 * ((k >> 3) & 1)) & (vecs - 1) : 0; }
  };
  // copies of n units from a P unit on
  static constexpr int copies(int n) { return (n + 1) / 2 * copies_p + n / 2 * copies_q; }
  static_assert((BM == BN || U % 2 == 0) && U >= 5 && lds <= 160 * 1024 && copies(U - 3) < 64, "ring");
};

template <typename T, typename C, bool GATED, int FORM>
__device__ __forceinline__ void product(const GemmParams& a, int block, unsigned char* lds) {
  constexpr bool kAcross[2] = {FORM == kDw, FORM != kForward};
  constexpr int KS = 128 / sizeof(T), VEC = 16 / sizeof(T);  // k of a step, elements of a vector
  using AP = typename C::template Across<T, C::BM>;
  using AQ = typename C::template Across<T, C::BN>;
  constexpr int NQ = GATED ? 2 : 1;
  constexpr int FM = C::BM / C::WM / 32, FN = C::BN / C::WN / 32;
  constexpr int CC = C::BN / NQ;  // output columns of a tile
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 31, q = lane >> 5;

  // consecutive workgroups go to the 8 XCDs in turn: give each XCD a run of tiles, walked
  // down groups of 8 row bands so that its L2 serves a compact block of the output
  const int total = a.tiles_m * a.tiles_n;
  const int split = block / total, b = block - split * total;
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

  // With one row band no W is shared between workgroups: each starts elsewhere in k, or all of
  // them would read the same few memory channels at a time.
  const int turn = FORM == kForward && a.tiles_m == 1 && full > 0 ? block % 4096 * 61 % full : 0;

  // Where this lane reads.  Along k, copy j of the wave fills rows 8 (wave copies + j) + lane / 8
  // of a unit; across it, rows of k.
  constexpr int kCopies[2] = {C::copies_p, C::copies_q};
  constexpr int kMost = C::copies_p > C::copies_q ? C::copies_p : C::copies_q;
  constexpr int kVecs[2] = {AP::vecs, AQ::vecs};
  auto unit_row = [&](int h, int j) {  // the unit's row (of its k) that copy j reads in this lane
    const int per = kAcross[h] ? kVecs[h] : 8;
    return 64 / per * (wave * kCopies[h] + j) + lane / per;
  };
  const unsigned char* src[2][kMost];
  int64_t by[2];                     // from a step to the next
  const unsigned char* cross[kMost];  // dx: where a copy goes on in the second weight,
  int cross_at[kMost];                // and from which step
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    by[h] = kAcross[h] ? (h == 0 ? a.p : a.q[0]).ld * int64_t(128) : 128;
#pragma unroll
    for (int j = 0; j < kCopies[h]; ++j) {
      const int r = unit_row(h, j);
      const int64_t n = h == 0 ? a.rows : a.cols;
      if constexpr (kAcross[0] || kAcross[1]) {
        if (kAcross[h]) {
          const int v = (lane % kVecs[h]) ^ (h == 0 ? AP::spread(r) : AQ::spread(r));
          const int64_t at = (h == 0 ? row0 : col0) + v * VEC, i = at < n ? at : n - VEC;
          const int64_t k = int64_t(step0) * KS + r;
          const MatIn& m = h == 0 ? a.p : a.q[0];
          src[h][j] = static_cast<const unsigned char*>(m.p) + (k * m.ld + i) * int64_t(sizeof(T));
          if (FORM == kDx && h == 1) {
            // k = seam and on lie in the second weight
            const int64_t over = a.seam - k, at_step = over <= 0 ? 0 : (over + KS - 1) / KS;
            cross[j] = static_cast<const unsigned char*>(a.q[1].p) +
                       ((k + at_step * KS - a.seam) * a.q[1].ld + i) * int64_t(sizeof(T));
            cross_at[j] = at_step < (1 << 30) ? static_cast<int>(at_step) : 1 << 30;
            if (at_step == 0) src[h][j] = cross[j];
          }
          continue;
        }
      }
      const MatIn& m = h == 0 ? a.p : a.q[GATED ? (r >> 4) & 1 : 0];
      const int64_t at = h == 0 ? row0 + r : col0 + (GATED ? (r >> 5) * 16 + (r & 15) : r);
      src[h][j] = static_cast<const unsigned char*>(m.p) + (at < n ? at : n - 1) * m.ld * int64_t(sizeof(T)) +
                  int64_t(step0 + turn) * 128 + ((lane & 7) ^ ((r >> 1) & 7)) * 16;
    }
  }
  const int64_t by_seam = FORM == kDx ? a.q[1].ld * int64_t(128) : 0;
  // the lane's place in step t + 1, from its place in step t
  auto advance = [&](int h, int j, int t) {
    if (FORM == kDx && h == 1) {
      const unsigned char* next = src[h][j] + (t >= cross_at[j] ? by_seam : by[h]);
      src[h][j] = t + 1 == cross_at[j] ? cross[j] : next;
    } else {
      src[h][j] += FORM == kForward && t == full - 1 - turn ? 128 - full * 128 : by[h];
    }
  };
  auto copy_unit = [&](int t, int slot, int h) {
    unsigned char* at = lds + C::slot(slot) + wave * kCopies[h] * 1024;
#pragma unroll
    for (int j = 0; j < kCopies[h]; ++j) {
      copy_to_lds(src[h][j], at + j * 1024);
      advance(h, j, t);
    }
  };
  auto copy_unit_or_tail = [&](int u, int slot, int h) {
    if ((u >> 1) < full) {
      copy_unit(u >> 1, slot, h);
    } else if ((u >> 1) < steps) {
      unsigned char* at = lds + C::slot(slot) + wave * kCopies[h] * 1024;
#pragma unroll
      for (int j = 0; j < kCopies[h]; ++j) {
        const int r = unit_row(h, j);
        const bool in = kAcross[h] ? r * int(sizeof(T)) < tail : ((lane & 7) ^ ((r >> 1) & 7)) * 16 < tail;
        const int64_t back = FORM == kForward ? (full - turn) * 128 : 0;
        u32x4 d = {0, 0, 0, 0};
        if (in) d = *reinterpret_cast<const u32x4*>(src[h][j] + back);
        *reinterpret_cast<u32x4*>(at + j * 1024 + lane * 16) = d;
      }
    }
  };

  f32x16 acc[FM][FN] = {};
  const int wm = wave / C::WN, wn = wave % C::WN;
  // Fragments of an operand read along k, or in fp32: the x-th, slice s = 0 .. 3 of a step.
  const int rd = 16 * (q ^ ((c >> 1) & 7));  // along: vector 2 s + q of the row lies at rd ^ 32 s
  const int along[2] = {(wm * FM * 32 + c) * 128, (wn * FN * 32 + c) * 128};
  constexpr int kFrags[2] = {FM, FN};
  constexpr bool kPaired[2] = {kAcross[0] && sizeof(T) == 2, kAcross[1] && sizeof(T) == 2};
  int across[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int base = (h == 0 ? wm : wn) * kFrags[h] * 32, width = kVecs[h] * 16;  // first column, bytes of a k
    if constexpr (sizeof(T) == 2) {
      const int col = base + (kFrags[h] > 1 ? kFrags[h] * c : c & ~1);
      across[h] = 8 * q * width + ((col / 8) ^ (h == 0 ? AP::spread(8 * q) : AQ::spread(8 * q))) * 16 + col % 8 * 2;
    } else {
      across[h] = 4 * q * width + (base + c) * 4;
    }
  }
  auto fragment = [&](int h, int slot, int x, int s) -> u32x4 {
    const unsigned char* unit = lds + C::slot(slot);
    if (!kAcross[h]) return *reinterpret_cast<const u32x4*>(unit + along[h] + (rd ^ (s * 32)) + x * 4096);
    const int width = kVecs[h] * 16;
    u32x4 d;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      d[r] = *reinterpret_cast<const uint32_t*>(unit + across[h] + x * 128 + (8 * s + r) * width);
    return d;
  };
  // bf16 across k: the lane's columns of k = 16 s + 8 q + kk, and word d (k = 2 d, 2 d + 1) of
  // fragment x paired from them.
  auto columns = [&](int h, int slot, int s, int kk, uint32_t (&to)[2]) {
    const unsigned char* from = lds + C::slot(slot) + across[h] + (16 * s + kk) * kVecs[h] * 16;
    if (kFrags[h] == 4) {
      typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
      const u32x2 d = *reinterpret_cast<const u32x2*>(from);
      to[0] = d[0];
      to[1] = d[1];
    } else {
      to[0] = *reinterpret_cast<const uint32_t*>(from);
    }
  };
  constexpr uint32_t kLow = 0x05040100, kHigh = 0x07060302;  // low and high halves of two words
  const uint32_t mine = c & 1 ? kHigh : kLow;
  auto paired = [&](int h, const uint32_t (&raw)[8][2], int x, int d) {
    const int w = kFrags[h] == 4 ? x >> 1 : 0;
    return __builtin_amdgcn_perm(raw[2 * d + 1][w], raw[2 * d][w], kFrags[h] == 1 ? mine : x & 1 ? kHigh : kLow);
  };
  // A step has two halves; the fragments of one are read while the other is multiplied.  One
  // barrier a step, between them: behind it every wave has read step t's units, and step t + 1's
  // are complete for every wave.  Unit 2 t + U takes unit 2 t's slot from there on, unit
  // 2 t + U + 1 the next one in the first half of step t + 1: the copies spread evenly over
  // the multiplications, and the last of a step's own has half a step to arrive.
  u32x4 p0[2][FM], q0[2][FN], p1[2][FM], q1[2][FN];
  auto read = [&](int slot_p, int slot_q, u32x4 (&pv)[2][FM], u32x4 (&qv)[2][FN]) {  // the first half of a step
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int slot = h == 0 ? slot_p : slot_q;
        uint32_t raw[8][2];
        if (kPaired[h]) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) columns(h, slot, s, kk, raw[kk]);
        }
#pragma unroll
        for (int x = 0; x < kFrags[h]; ++x) {
          u32x4 d;
          if (kPaired[h]) {
#pragma unroll
            for (int w = 0; w < 4; ++w) d[w] = paired(h, raw, x, w);
          } else {
            d = fragment(h, slot, x, s);
          }
          if (h == 0)
            pv[s][x] = d;
          else
            qv[s][x] = d;
        }
      }
  };
  // One half multiplied, with the other's fragment reads and one unit's copies spread evenly
  // between the multiplications, in exactly this order: the reads over the first three quarters,
  // or, where columns are paired, over the first half, and the pairing over the second.  A burst
  // of copies holds up the wave that issues it, and with it its matrix instructions: with them
  // issued together the 256 x 256 tile reached 1100 TFLOP/s at 4096 x 8192 x 28672, spread 1400.
  constexpr bool kPairs = kPaired[0] || kPaired[1];
  constexpr int kMults = 2 * FM * FN;
  constexpr int kReadsOf[2] = {kPaired[0] ? 8 : FM, kPaired[1] ? 8 : FN}, kReads = 2 * (kReadsOf[0] + kReadsOf[1]);
  constexpr int kPairsOf[2] = {kPaired[0] ? 4 * FM : 0, kPaired[1] ? 4 * FN : 0};
  constexpr int kPairings = 2 * (kPairsOf[0] + kPairsOf[1]);
  constexpr int kEarly = kMults * (kPairs ? 2 : 3) / 4 > 0 ? kMults * (kPairs ? 2 : 3) / 4 : 1;
  auto half_step = [&](const u32x4 (&pa)[2][FM], const u32x4 (&qa)[2][FN], int slot_p, int slot_q, int half,
                       u32x4 (&pb)[2][FM], u32x4 (&qb)[2][FN], int step, int slot_copy, int h, bool copies) {
    unsigned char* at = lds + C::slot(slot_copy) + wave * kCopies[h] * 1024;
    uint32_t raw_p[2][8][2], raw_q[2][8][2];
#pragma unroll
    for (int m = 0; m < kMults; ++m) {
      const int s = m / (FM * FN), i = m / FN % FM, j = m % FN;
      acc[i][j] = mfma32<T>(qa[s][j], pa[s][i], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int r = m < kEarly ? kReads * m / kEarly : kReads; r < (m < kEarly ? kReads * (m + 1) / kEarly : kReads); ++r) {
        const int rs = r / (kReads / 2), x = r % (kReads / 2), y = x - kReadsOf[1];
        if (x < kReadsOf[1]) {
          if (kPaired[1])
            columns(1, slot_q, 2 * half + rs, x, raw_q[rs][x]);
          else
            qb[rs][x] = fragment(1, slot_q, x, 2 * half + rs);
        } else {
          if (kPaired[0])
            columns(0, slot_p, 2 * half + rs, y, raw_p[rs][y]);
          else
            pb[rs][y] = fragment(0, slot_p, y, 2 * half + rs);
        }
      }
      if (copies) {
#pragma unroll
        for (int k = kCopies[h] * m / kMults; k < kCopies[h] * (m + 1) / kMults; ++k) {
          copy_to_lds(src[h][k], at + k * 1024);
          advance(h, k, step);
        }
      }
      if constexpr (kPairs) {
        constexpr int kLate = kMults - kEarly;
        const int l = m - kEarly;
#pragma unroll
        for (int r = l < 0 ? 0 : kPairings * l / kLate; r < (l < 0 ? 0 : kPairings * (l + 1) / kLate); ++r) {
          const int rs = r / (kPairings / 2), x = r % (kPairings / 2), y = x - kPairsOf[1];
          if (x < kPairsOf[1])
            qb[rs][x / 4][x % 4] = paired(1, raw_q[rs], x / 4, x % 4);
          else
            pb[rs][y / 4][y % 4] = paired(0, raw_p[rs], y / 4, y % 4);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto after = [](int slot, int by) { return slot + by >= C::U ? slot + by - C::U : slot + by; };
  if ((C::U - 2) / 2 < full) {
#pragma unroll
    for (int u = 0; u < C::U - 1; ++u) copy_unit(u >> 1, u, u & 1);
    copies_then_barrier<C::copies(C::U - 3)>();
  } else {
#pragma unroll
    for (int u = 0; u < C::U - 1; ++u) copy_unit_or_tail(u, u, u & 1);
    copies_then_barrier<0>();
  }
  read(0, 1, p0, q0);
  int t = 0, slot = 0;  // slot of unit 2 t
  for (; (2 * t + C::U) / 2 < full; ++t) {
    half_step(p0, q0, slot, after(slot, 1), 1, p1, q1, (2 * t + C::U - 1) / 2, after(slot, C::U - 1),
              (C::U - 1) & 1, true);
    copies_then_barrier<C::copies(C::U - 4)>();
    const int next = after(slot, 2);
    half_step(p1, q1, next, after(next, 1), 0, p0, q0, (2 * t + C::U) / 2, slot, C::U & 1, true);
    slot = next;
  }
  for (; t < steps; ++t) {
    copy_unit_or_tail(2 * t + C::U - 1, after(slot, C::U - 1), (C::U - 1) & 1);
    half_step(p0, q0, slot, after(slot, 1), 1, p1, q1, 0, 0, 0, false);
    copies_then_barrier<0>();
    copy_unit_or_tail(2 * t + C::U, slot, C::U & 1);
    slot = after(slot, 2);
    half_step(p1, q1, slot, after(slot, 1), 0, p0, q0, 0, 0, 0, false);
  }

  // Epilogue: each wave passes its sums, 32 rows at a time, through an LDS window of its own,
  // so that a lane has eight consecutive columns and a row's lanes write whole lines.
  __syncthreads();
  float* win = reinterpret_cast<float*>(lds + wave * C::window);
  const Epilogue<T, GATED> ep(a);
  float* const part = held(a.part);
  const int64_t rows = held(a.rows);
  const int cols = held(a.cols), splits = held(a.splits);
  constexpr int CW = FN * 32 / NQ, LANES = CW / 8;  // output columns of the wave, lanes per row
  // (the rows' loop stays rolled: its body holds every activation)
#pragma unroll 1
  for (int i = 0; i < FM; ++i) {
    lds_wave_sync();
#pragma unroll
    for (int f = 0; f < FM; ++f) {
      if (f != i) continue;
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          float* row = win + c * C::win_pitch;
          if constexpr (kPaired[1] && FN == 4) {  // fragment x holds columns 4 r + x: here those of r = 8 g + 4 q + j
            const int r = 4 * g + j;
            *reinterpret_cast<f32x4*>(row + 4 * (8 * g + 4 * q + j)) =
                f32x4{acc[f][0][r], acc[f][1][r], acc[f][2][r], acc[f][3][r]};
          } else if constexpr (kPaired[1] && FN == 2) {
#pragma unroll
            for (int e = 0; e < 4; ++e) row[2 * (8 * g + 4 * q + e) + j] = acc[f][j][4 * g + e];
          } else {
            *reinterpret_cast<f32x4*>(row + 32 * j + 8 * g + 4 * q) =
                f32x4{acc[f][j][4 * g], acc[f][j][4 * g + 1], acc[f][j][4 * g + 2], acc[f][j][4 * g + 3]};
          }
        }
    }
    lds_wave_sync();
    constexpr int kRounds = LANES / 2 > 0 ? LANES / 2 : 1, kTogether = kRounds > 1 ? 2 : 1;
#pragma unroll 1
    for (int v0 = 0; v0 < kRounds; v0 += kTogether) {
      float z[kTogether][NQ][8];
#pragma unroll
      for (int u = 0; u < kTogether; ++u) {
        const int v = (v0 + u) * 64 + lane, r = v / LANES, nc = (v % LANES) * 8;
#pragma unroll
        for (int h = 0; h < NQ; ++h)
          load8(win + r * C::win_pitch + (GATED ? (nc >> 4) * 32 + h * 16 + (nc & 15) : nc), z[u][h]);
      }
#pragma unroll
      for (int u = 0; u < kTogether; ++u) {
        const int v = (v0 + u) * 64 + lane, r = v / LANES, nc = (v % LANES) * 8;
        const int64_t m = row0 + wm * FM * 32 + (kPaired[0] ? FM * r + i : 32 * i + r), n = col0 + wn * CW + nc;
        if (m >= rows || n >= cols) continue;
        if (splits > 1) {
#pragma unroll
          for (int h = 0; h < NQ; ++h) store8(part + ((int64_t(split) * NQ + h) * rows + m) * cols + n, z[u][h]);
        } else {
          ep.template finish8<true>(m, n, z[u]);
        }
      }
    }
  }
}

// The forward products, or those of a backward pass (GRAD).
template <typename T, typename C, bool GATED, bool GRAD>
__global__ void __launch_bounds__(C::threads, C::per_simd) gemm_kernel(GemmPair pair) {
  __shared__ __attribute__((aligned(16))) unsigned char lds[C::lds];
  const int second = static_cast<int>(blockIdx.x) >= pair.first;
  const GemmParams& a = pair.a[second];
  const int block = static_cast<int>(blockIdx.x) - (second ? pair.first : 0);
  if constexpr (!GRAD) {
    product<T, C, GATED, kForward>(a, block, lds);
  } else {
    if (a.form == kDx)
      product<T, C, false, kDx>(a, block, lds);
    else
      product<T, C, false, kDw>(a, block, lds);
  }
}

// Lanes that share eight columns' parts in a join: with many parts of a small matrix there are
// few threads, each with a long chain of loads (dx of 17 x 18048 x 1784 in 32 parts: 31.3 us with
// one lane, 24.1 with four).
__host__ __device__ inline int join_lanes(int splits) { return splits >= 8 ? 4 : 1; }

// Join a split contraction: eight columns per thread or four threads, the parts' sums in a fixed
// order, then the epilogue.
template <typename T, bool GATED>
__device__ __forceinline__ void join_parts(const GemmParams& a, int block) {
  constexpr int NQ = GATED ? 2 : 1;
  const int64_t groups = a.rows * (a.cols / 8);
  const int lanes = join_lanes(a.splits), lane = threadIdx.x & (lanes - 1);
  const int64_t v = block * int64_t(256 / lanes) + threadIdx.x / lanes;
  if (v >= groups) return;
  const int64_t m = v / (a.cols / 8);
  const int64_t n = (v - m * (a.cols / 8)) * 8;
  const Epilogue<T, GATED> ep(a);
  float z[NQ][8] = {};
  constexpr int kAhead = GATED ? 4 : 8;  // parts whose loads are in flight together
  for (int s0 = lane; s0 < a.splits; s0 += kAhead * lanes) {
    float t[kAhead][NQ][8];
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
#pragma unroll
      for (int h = 0; h < NQ; ++h) {
        const int from = s0 + s * lanes < a.splits ? s0 + s * lanes : s0;
        load8(a.part + ((int64_t(from) * NQ + h) * a.rows + m) * a.cols + n, t[s][h]);
      }
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
#pragma unroll
      for (int h = 0; h < NQ; ++h)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (s0 + s * lanes < a.splits) z[h][e] += t[s][h][e];
  }
  if (lanes > 1) {  // the four threads of a group are next to each other, and all here
#pragma unroll
    for (int h = 0; h < NQ; ++h)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        z[h][e] += __shfl_xor(z[h][e], 1, 64);
        z[h][e] += __shfl_xor(z[h][e], 2, 64);
      }
    if (lane != 0) return;
  }
  ep.finish8(m, n, z);
}

// dbias: the slope tiles' column sums in a fixed order, four chains per column; blocks of 64
// columns, first dbias[0]'s, then dbias[1]'s.
struct BiasParams {
  const float* sums;  // [tiles][parts][cols]
  int64_t tiles;
  int32_t parts;
  int32_t cols;
  void* db[2];
};

template <typename T>
__device__ __forceinline__ void join_bias(const BiasParams& b, int block) {
  __shared__ float part[4][64];
  const int per = (b.cols + 63) / 64, h = block >= per;
  const int c = threadIdx.x & 63, w = threadIdx.x >> 6, n = (block - h * per) * 64 + c;
  float s = 0.f;
  if (n < b.cols)
    for (int64_t i = w; i < b.tiles; i += 4) s += b.sums[(i * b.parts + h) * b.cols + n];
  part[w][c] = s;
  __syncthreads();
  T* db = static_cast<T*>(b.db[h]);
  if (w == 0 && n < b.cols && db != nullptr)
    db[n] = from_f32<T>((part[0][c] + part[1][c]) + (part[2][c] + part[3][c]));
}

// What is left after the products, in one launch: up to two joins, then dbias.
struct JoinParams {
  GemmPair pair;       // first: blocks of the first join
  int32_t bias_first;  // blocks of both joins
  BiasParams bias;
};

template <typename T, bool GATED>
__global__ void __launch_bounds__(256) join_kernel(JoinParams j) {
  const int block = static_cast<int>(blockIdx.x);
  if constexpr (!GATED) {
    if (block >= j.bias_first) {
      join_bias<T>(j.bias, block - j.bias_first);
      return;
    }
  }
  const int second = block >= j.pair.first;
  join_parts<T, GATED>(j.pair.a[second], block - (second ? j.pair.first : 0));
}

// ---- few rows ------------------------------------------------------------------------
// Two to 48 rows, in TB blocks of 16: bound by reading W once (24 x 4096 x 11008: 20.4 us, 4.5
// TB/s).  A workgroup takes 16 output columns (gated: of both
// products) and its NW waves share the contraction in windows of 256 bytes of k, dealt out in
// turn.  A wave streams its windows of W and of x through an LDS ring of its own, S windows
// deep, by direct copies (4 rows x 256 bytes each), so no barrier is met before the end.
// Vector v of row r lies at r * 256 + 16 (v ^ r): the 16 rows of a fragment read fall on all
// banks.  The waves' sums meet in LDS in a fixed order.  16 x 16 instructions: lane l = 16 q + c
// supplies W(c, k) and x(c, k) of vector 4 s + q, and receives columns 4 q .. 4 q + 3 of row c.
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

template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

template <bool GATED, int TB, int NW, int S>
struct FewRows {
  static constexpr int NQ = GATED ? 2 : 1;
  static constexpr int window = (NQ + TB) * 4096;  // bytes of a window: 16 rows of each W, then blocks of x
  static constexpr int pitch = 20;                 // floats of a row of 16 sums
  static constexpr int sums = NQ * TB * 16 * pitch * 4;
  static constexpr int lds = NW * S * window;
  static_assert(S >= 2 && S * window >= sums && lds <= 160 * 1024 && 4 * (S - 1) * (NQ + TB) < 64, "ring");
};

template <typename T, bool GATED, int TB, int NW, int S>
__device__ __forceinline__ void few_rows_product(const GemmParams& a, unsigned char* lds) {
  using F = FewRows<GATED, TB, NW, S>;
  constexpr int NQ = F::NQ, NO = NQ + TB;  // operands: the weights, then x's blocks
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, q = lane >> 4;
  const int blocks = (a.cols + 15) / 16, split = __builtin_amdgcn_readfirstlane(static_cast<int>(blockIdx.x) / blocks);
  const int column = static_cast<int>(blockIdx.x) - split * blocks;  // of workgroups: the same for all splits
  const int64_t col0 = column * int64_t(16);
  const int64_t bytes = a.depth * sizeof(T);
  const int whole = static_cast<int>(bytes >> 8), windows = static_cast<int>((bytes + 255) >> 8);
  const int tail = static_cast<int>(bytes & 255);  // bytes of the last window if short
  // this wave's windows: place, place + stride, ...
  const int place = split * NW + wave, stride = NW * a.splits;
  const int n = place < windows ? (windows - place + stride - 1) / stride : 0;
  const int full = n - (tail != 0 && n > 0 && place + (n - 1) * stride == windows - 1);
  // Each column starts elsewhere in k: side by side, their 16 rows a stride apart, they would
  // read the same few memory channels at a time (11008-long rows: 20.3 us, turned 16.6 us).
  const int turn = whole > 0 ? column % 4096 * 61 % whole : 0;
  auto window = [&](int i) {  // byte offset of this wave's window i
    const int p = place + i * stride, r = p + turn;
    return __builtin_amdgcn_readfirstlane(256 * (p >= whole ? p : r >= whole ? r - whole : r));
  };

  // buffer copies: an operand's first row as base, 32-bit offsets to its others (rows past its
  // end repeat the last)
  __amdgpu_buffer_rsrc_t m[NO];
  int off[NO][4];
#pragma unroll
  for (int h = 0; h < NO; ++h) {
    const MatIn& o = h < NQ ? a.q[h] : a.p;
    const int64_t ld = o.ld * int64_t(sizeof(T)), first = h < NQ ? col0 : 16 * (h - NQ), rows = h < NQ ? a.cols : a.rows;
    const int64_t last = rows - 1 - first < 15 ? rows - 1 - first : 15;
    m[h] = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<unsigned char*>(static_cast<const unsigned char*>(o.p) + first * ld), 0,
        static_cast<int>(last * ld + bytes), 0x00020000);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = 4 * j + (lane >> 4);
      off[h][j] = static_cast<int>((r < last ? r : last) * ld) + ((lane & 15) ^ r) * 16;
    }
  }
  unsigned char* ring = lds + wave * S * F::window;
  auto copy_or_tail = [&](int i) {  // window i of this wave; W is streamed past the caches
    unsigned char* at = ring + (i % S) * F::window;
    if (i < full) {
#pragma unroll
      for (int h = 0; h < NO; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          ADA_LDS void* to = (ADA_LDS void*)(at + h * 4096 + j * 1024);
          if (h < NQ)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(m[h], to, 16, off[h][j], window(i), 0, 2);
          else
            __builtin_amdgcn_raw_ptr_buffer_load_lds(m[h], to, 16, off[h][j], window(i), 0, 0);
        }
    } else if (i < n) {
#pragma unroll
      for (int h = 0; h < NO; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          u32x4 d = {0, 0, 0, 0};
          if (((lane & 15) ^ (4 * j + (lane >> 4))) * 16 < tail)
            d = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(m[h], off[h][j], window(i), 0));
          *reinterpret_cast<u32x4*>(at + h * 4096 + j * 1024 + lane * 16) = d;
        }
    }
  };
  f32x4 acc[NQ][TB] = {};
#pragma unroll
  for (int i = 0; i < S - 1; ++i) copy_or_tail(i);
  for (int i = 0; i < n; ++i) {
    copy_or_tail(i + S - 1);
    if (i + S - 1 < full)  // all but the S - 1 windows behind this one have arrived
      wait_copies<4 * (S - 1) * NO>();
    else
      wait_copies<0>();
    lds_wave_sync();  // a tail window went through registers
    const unsigned char* at = ring + (i % S) * F::window + c * 256;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int v = ((4 * s + q) ^ c) * 16;
      u32x4 x[TB];
#pragma unroll
      for (int b = 0; b < TB; ++b) x[b] = *reinterpret_cast<const u32x4*>(at + (NQ + b) * 4096 + v);
#pragma unroll
      for (int h = 0; h < NQ; ++h) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(at + h * 4096 + v);
#pragma unroll
        for (int b = 0; b < TB; ++b) acc[h][b] = mfma16<T>(w, x[b], acc[h][b]);
      }
    }
    // the window's reads are done before its slot is copied to again
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }

  __syncthreads();
  float* sums = reinterpret_cast<float*>(lds);
  constexpr int kWave = F::sums / 4;
#pragma unroll
  for (int h = 0; h < NQ; ++h)
#pragma unroll
    for (int b = 0; b < TB; ++b)
      *reinterpret_cast<f32x4*>(sums + wave * kWave + ((h * TB + b) * 16 + c) * F::pitch + 4 * q) = acc[h][b];
  __syncthreads();
  const Epilogue<T, GATED> ep(a);
  for (int v = threadIdx.x; v < 2 * a.rows; v += 64 * NW) {
    const int r = v >> 1, nc = (v & 1) * 8;
    if (col0 + nc >= a.cols) continue;
    float z[NQ][8] = {};
#pragma unroll
    for (int w = 0; w < NW; ++w)
#pragma unroll
      for (int h = 0; h < NQ; ++h) {
        float t[8];
        load8(sums + w * kWave + (h * TB * 16 + r) * F::pitch + nc, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[h][e] += t[e];
      }
    if (a.splits > 1) {
#pragma unroll
      for (int h = 0; h < NQ; ++h)
        store8(a.part + ((int64_t(split) * NQ + h) * a.rows + r) * a.cols + col0 + nc, z[h]);
    } else {
      ep.finish8(r, col0 + nc, z);
    }
  }
}

template <typename T, bool GATED, int TB, int NW, int S>
__global__ void __launch_bounds__(64 * NW) few_rows_kernel(GemmParams a) {
  __shared__ __attribute__((aligned(16))) unsigned char lds[FewRows<GATED, TB, NW, S>::lds];
  few_rows_product<T, GATED, TB, NW, S>(a, lds);
}

// ... and whose operands lie within the 32-bit offsets of its buffer copies.
bool few_rows(const GemmParams& a, bool gated, int esz) {
  if (!few_rows_sizes(a.rows, a.cols, a.depth, gated, esz)) return false;
  for (int h = 0; h < (gated ? 3 : 2); ++h)
    if ((15 * (h == 0 ? a.p : a.q[h - 1]).ld + a.depth) * esz >= (int64_t(1) << 31)) return false;
  return true;
}

template <typename T, bool GATED, int TB, int NW>
hipError_t launch_few_rows_waves(const GemmParams& a, hipStream_t s) {
  const unsigned grid = static_cast<unsigned>((a.cols + 15) / 16 * a.splits);
  few_rows_kernel<T, GATED, TB, NW, 2><<<grid, 64 * NW, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T, bool GATED, int TB>
hipError_t launch_few_rows_block(const GemmParams& a, hipStream_t s) {
  if (few_rows_two_waves(a.cols, a.depth, GATED, TB, sizeof(T))) return launch_few_rows_waves<T, GATED, TB, 2>(a, s);
  return launch_few_rows_waves<T, GATED, TB, (!GATED && TB == 1 ? 8 : 4)>(a, s);
}

template <typename T, bool GATED>
hipError_t launch_few_rows(const GemmParams& a, hipStream_t s) {
  if (a.rows <= 16) return launch_few_rows_block<T, GATED, 1>(a, s);
  if (a.rows <= 32) return launch_few_rows_block<T, GATED, 2>(a, s);
  return launch_few_rows_block<T, GATED, 3>(a, s);
}

// ---- one row -------------------------------------------------------------------------
// Bound by reading W once (4096 x 4096: 7.1 us, 4.7 TB/s; gated 11008 x 4096: 30.4 us, 5.9 TB/s):
// one wave per W row (gated: per pair), lanes along it with 16-byte loads, U vectors of each row
// in flight before any is used, x from the caches.  Eight waves hold eight consecutive columns,
// which the epilogue takes together.  Past the row's end a lane re-reads its first vector and
// drops the product (a zero x would make an infinite weight there NaN).
template <typename T>
__device__ __forceinline__ float dot16(u32x4 w, u32x4 x, float acc) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      acc = fmaf(__uint_as_float(w[i] << 16), __uint_as_float(x[i] << 16), acc);
      acc = fmaf(__uint_as_float(w[i] & 0xffff0000u), __uint_as_float(x[i] & 0xffff0000u), acc);
    } else {
      acc = fmaf(__uint_as_float(w[i]), __uint_as_float(x[i]), acc);
    }
  }
  return acc;
}

template <typename T, bool GATED>
__global__ void __launch_bounds__(512) one_row_kernel(GemmParams a) {
  constexpr int NQ = GATED ? 2 : 1, VEC = 16 / sizeof(T), U = GATED ? 4 : 8;
  __shared__ float sums[NQ][8];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n = int64_t(blockIdx.x) * 8 + wave;
  const int nvec = static_cast<int>(a.depth / VEC);
  const u32x4* x = static_cast<const u32x4*>(a.p.p);
  const u32x4* w[NQ];
#pragma unroll
  for (int h = 0; h < NQ; ++h)
    w[h] = reinterpret_cast<const u32x4*>(static_cast<const T*>(a.q[h].p) + n * a.q[h].ld);
  float acc[NQ] = {};
  for (int v0 = 0; v0 < nvec; v0 += 64 * U) {
    u32x4 wv[NQ][U], xv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = v0 + 64 * u + lane, at = v < nvec ? v : 0;
#pragma unroll
      for (int h = 0; h < NQ; ++h) wv[h][u] = __builtin_nontemporal_load(w[h] + at);
      xv[u] = x[at];
    }
    __builtin_amdgcn_sched_barrier(0);  // every load before the first use
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = v0 + 64 * u + lane < nvec;
#pragma unroll
      for (int h = 0; h < NQ; ++h) {
        const float sum = dot16<T>(wv[h][u], xv[u], acc[h]);
        acc[h] = in ? sum : acc[h];
      }
    }
  }
#pragma unroll
  for (int h = 0; h < NQ; ++h) {
    float v = acc[h];
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
    if (lane == 0) sums[h][wave] = v;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    const Epilogue<T, GATED> ep(a);
    float z[NQ][8];
#pragma unroll
    for (int h = 0; h < NQ; ++h)
#pragma unroll
      for (int e = 0; e < 8; ++e) z[h][e] = sums[h][e];
    ep.finish8(0, int64_t(blockIdx.x) * 8, z);
  }
}

template <typename T, bool GATED>
hipError_t launch_one_row(const GemmParams& a, hipStream_t s) {
  one_row_kernel<T, GATED><<<a.cols / 8, 512, 0, s>>>(a);
  return hipGetLastError();
}

// The tiles that the plan chooses from.
using Tile0 = TileConfig<256, 256, 5, 1>;
using Tile1 = TileConfig<256, 128, 6, 1>;
using Tile2 = TileConfig<128, 256, 6, 1>;
using Tile3 = TileConfig<128, 128, 10, 1>;
using Tile4 = TileConfig<64, 128, 12, 1>;
using Tile5 = TileConfig<64, 64, 10, 2>;
constexpr int kRowsOf[] = {Tile0::BM, Tile1::BM, Tile2::BM, Tile3::BM, Tile4::BM, Tile5::BM};
constexpr int kColsOf[] = {Tile0::BN, Tile1::BN, Tile2::BN, Tile3::BN, Tile4::BN, Tile5::BN};
constexpr bool planned_tiles() {
  for (int t = 0; t < kTiles; ++t)
    if (kRowsOf[t] != kTileRows[t] || kColsOf[t] != kTileCols[t]) return false;
  return sizeof(kRowsOf) == sizeof(kTileRows);
}
static_assert(planned_tiles(), "the plan's tiles are these");

#define ADA_TRY(call)                                              \
  do {                                                             \
    if (const hipError_t e_ = (call); e_ != hipSuccess) return e_; \
  } while (0)

// Launch n = 1 or 2 products (their splits set) as one grid of this tile.
template <typename T, typename C, bool GATED, bool GRAD>
hipError_t launch_tiles(const GemmParams* a, int n, hipStream_t s) {
  constexpr int cc = C::BN / (GATED ? 2 : 1);
  GemmPair pair{};
  int64_t grid = 0;
  for (int i = 0; i < n; ++i) {
    pair.a[i] = a[i];
    pair.a[i].tiles_m = static_cast<int32_t>((a[i].rows + C::BM - 1) / C::BM);
    pair.a[i].tiles_n = (a[i].cols + cc - 1) / cc;
    if (i == 1) pair.first = static_cast<int32_t>(grid);
    grid += int64_t(pair.a[i].tiles_m) * pair.a[i].tiles_n * a[i].splits;
  }
  if (n == 1) pair.first = static_cast<int32_t>(grid);
  gemm_kernel<T, C, GATED, GRAD><<<static_cast<unsigned>(grid), C::threads, 0, s>>>(pair);
  return hipGetLastError();
}

template <typename T, bool GATED, bool GRAD>
hipError_t launch_products(int tile, const GemmParams* a, int n, hipStream_t s) {
  switch (tile) {
    case 0: return launch_tiles<T, Tile0, GATED, GRAD>(a, n, s);
    case 1: return launch_tiles<T, Tile1, GATED, GRAD>(a, n, s);
    case 2: return launch_tiles<T, Tile2, GATED, GRAD>(a, n, s);
    case 3: return launch_tiles<T, Tile3, GATED, GRAD>(a, n, s);
    case 4: return launch_tiles<T, Tile4, GATED, GRAD>(a, n, s);
    default: return launch_tiles<T, Tile5, GATED, GRAD>(a, n, s);
  }
}

// The joins of n products (those with splits > 1), and dbias where asked for.
template <typename T, bool GATED>
hipError_t launch_joins(const GemmParams* a, int n, const BiasParams* bias, hipStream_t s) {
  JoinParams j{};
  int64_t grid = 0;
  int used = 0;
  for (int i = 0; i < n; ++i) {
    if (a[i].splits <= 1) continue;
    j.pair.a[used++] = a[i];
    grid += (a[i].rows * (a[i].cols / 8) * join_lanes(a[i].splits) + 255) / 256;
    if (used == 1) j.pair.first = static_cast<int32_t>(grid);
  }
  j.bias_first = static_cast<int32_t>(grid);
  if (bias != nullptr) {
    j.bias = *bias;
    grid += int64_t(bias->parts) * ((bias->cols + 63) / 64);
  }
  if (grid == 0) return hipSuccess;
  join_kernel<T, GATED><<<static_cast<unsigned>(grid), 256, 0, s>>>(j);
  return hipGetLastError();
}

template <typename T, bool GATED>
hipError_t launch_forward(GemmParams a, float* part, hipStream_t s) {
  if (a.rows == 1) return launch_one_row<T, GATED>(a, s);
  const Plan p = plan_forward(a.rows, a.cols, a.depth, GATED, sizeof(T));
  a.splits = p.splits;
  a.part = part;
  const hipError_t e = few_rows(a, GATED, sizeof(T)) ? launch_few_rows<T, GATED>(a, s)
                                                     : launch_products<T, GATED, false>(p.tile, &a, 1, s);
  if (e != hipSuccess) return e;
  return launch_joins<T, GATED>(&a, 1, nullptr, s);
}

// ---- gradients of few rows -------------------------------------------------------------
// Up to 32 or 64 rows: dx is bound by reading W once, dW by writing it once (32 x 11008 x 4096: 29
// and 21 us, both in one grid 40, 4.5 TB/s; on the tiles 57, 77 and 95), so no operand goes
// through LDS.  Both products have an operand whose rows lie across the contraction (W, x): a
// lane reads VEC neighbouring columns of VEC such rows, 16 bytes each, and has with them VEC
// fragments whose x-th column is its VEC c + x; the sums of all fragments in a lane are then VEC
// neighbouring outputs of a row, again 16 bytes.  32 x 32 instructions: lane l = 32 h + c supplies
// the contraction's elements 2 VEC t + VEC h + i of step t, i = 0 .. VEC - 1.
template <typename T>
struct FewGrad {
  static constexpr int VEC = 16 / sizeof(T);
  static constexpr int cols = 32 * VEC;            // a wave's output columns
  static constexpr int step = 2 * VEC;             // of the contraction
  static constexpr int ahead = sizeof(T) == 2 ? 2 : 4;  // dx: steps of W in flight in a wave
  static constexpr int dw_rows = 256;              // dW: rows of a workgroup, 64 a wave
};

// The x-th fragment of VEC rows of VEC columns.
template <typename T>
__device__ __forceinline__ u32x4 across_fragment(const u32x4 (&raw)[16 / sizeof(T)], int x) {
  u32x4 f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (sizeof(T) == 2)
      f[j] = __builtin_amdgcn_perm(raw[2 * j + 1][x >> 1], raw[2 * j][x >> 1], x & 1 ? 0x07060302u : 0x05040100u);
    else
      f[j] = raw[j][x];
  }
  return f;
}

// VEC outputs of a row.
template <typename T>
__device__ __forceinline__ void store_vec(T* p, const float (&z)[16 / sizeof(T)]) {
  Vec16<T> d;
#pragma unroll
  for (int e = 0; e < int(16 / sizeof(T)); ++e) d.e[e] = from_f32<T>(z[e]);
  __builtin_nontemporal_store(__builtin_bit_cast(u32x4, d), (ADA_GLOBAL u32x4*)p);
}

// dW = dz^T x over up to ROWS rows: a wave holds x's fragments of its columns for all of them.
template <typename T, int ROWS>
__device__ __forceinline__ void few_rows_dw(const GemmParams& a, int block) {
  using F = FewGrad<T>;
  constexpr int VEC = F::VEC, kSteps = ROWS / F::step;
  typedef uint32_t Two __attribute__((ext_vector_type(sizeof(T) / 2)));  // two neighbours of dz
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 31, h = lane >> 5;
  const int strips = (a.cols + F::cols - 1) / F::cols;
  const int64_t n0 = int64_t(block / strips) * F::dw_rows + wave * 64, rows = held(a.rows);
  if (n0 >= rows) return;
  const int col = block % strips * F::cols + VEC * c;
  const bool in = col < a.cols;
  const int depth = static_cast<int>(a.depth);
  const int64_t ld_z = held(a.p.ld), ld_x = held(a.q[0].ld);
  // rows 2 c and 2 c + 1 of this wave's 64: the 0th and 1st fragment of dz
  const T* dz = static_cast<const T*>(a.p.p) + (n0 + 2 * c < rows ? n0 + 2 * c : 0);
  const T* xs = static_cast<const T*>(a.q[0].p) + (in ? col : 0);
  u32x4 raw[kSteps][VEC];
  Two two[kSteps][VEC];
#pragma unroll
  for (int t = 0; t < kSteps; ++t)
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int r = t * F::step + VEC * h + i;
      const int64_t at = r < depth ? r : 0;
      two[t][i] = *(const ADA_GLOBAL Two*)(dz + at * ld_z);
      raw[t][i] = *(const ADA_GLOBAL u32x4*)(xs + at * ld_x);
    }
  T* const y[2] = {held(static_cast<T*>(a.y[0].p)), held(static_cast<T*>(a.y[1].p))};
  const int64_t ld_y[2] = {held(a.y[0].ld), held(a.y[1].ld)}, row_split = held(a.row_split);
  __builtin_amdgcn_sched_barrier(0);  // all loads in flight before the first is used
  u32x4 x[kSteps][VEC], z[kSteps][2];
#pragma unroll
  for (int t = 0; t < kSteps; ++t) {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (t * F::step + VEC * h + i >= depth) {  // behind the last row: zeros on both sides
        raw[t][i] = u32x4{0, 0, 0, 0};
        two[t][i] = Two(0);
      }
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 2)
          z[t][f][j] = __builtin_amdgcn_perm(two[t][2 * j + 1][0], two[t][2 * j][0], f ? 0x07060302u : 0x05040100u);
        else
          z[t][f][j] = two[t][j][f];
      }
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[t][e] = across_fragment<T>(raw[t], e);
  }
#pragma unroll 1  // straight-line code once through waits for its instructions
  for (int f = 0; f < 2; ++f) {
    f32x16 acc[VEC] = {};
#pragma unroll
    for (int t = 0; t < kSteps; ++t) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] = mfma32<T>(z[t][0], x[t][e], acc[e]);
      z[t][0] = z[t][1];
    }
#pragma unroll
    for (int g = 0; g < 16; ++g) {
      const int64_t n = n0 + 2 * (8 * (g >> 2) + 4 * h + (g & 3)) + f;
      float v[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = acc[e][g];
      const bool up = n >= row_split;
      T* row = (up ? y[1] : y[0]) + (n - (up ? row_split : 0)) * (up ? ld_y[1] : ld_y[0]);
      if (in && n < rows) store_vec<T>(row + col, v);
    }
  }
}

// dx = dz W, QF blocks of 32 rows: the waves of all workgroups of a strip of columns share W's
// rows, step by step in turn; a workgroup's sums meet in LDS in a fixed order, and the workgroups'
// in the join.
template <typename T, int QF>
__device__ __forceinline__ void few_rows_dx(const GemmParams& a, int block, f32x4* lds) {
  using F = FewGrad<T>;
  constexpr int VEC = F::VEC, D = F::ahead;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 31, h = lane >> 5;
  const int cols = held(a.cols), strips = (cols + F::cols - 1) / F::cols, splits = held(a.splits);
  const int split = block / strips;
  const int col = block % strips * F::cols + VEC * c;
  const bool in = col < cols;
  const int64_t depth = held(a.depth), rows = held(a.rows), seam = held(a.seam);
  const int64_t stride = int64_t(4) * splits * F::step;  // of the contraction, from step to step
  const int64_t first = (int64_t(split) * 4 + wave) * F::step;
  const int64_t steps = first < depth ? (depth - first + stride - 1) / stride : 0;
  // rows behind the last repeat it and are not stored
  const T* zs[QF];
#pragma unroll
  for (int f = 0; f < QF; ++f)
    zs[f] = static_cast<const T*>(a.p.p) + (32 * f + c < rows ? 32 * f + c : rows - 1) * a.p.ld;
  const T* const q[2] = {held(static_cast<const T*>(a.q[0].p)), held(static_cast<const T*>(a.q[1].p))};
  const int64_t ld_q[2] = {held(a.q[0].ld), held(a.q[1].ld)};
  u32x4 w[D][VEC], z[D][QF];
  auto load = [&](int slot, int64_t t) {
    const int64_t k = first + t * stride + VEC * h;
    const int64_t at = k < depth ? k : 0;
    const bool up = at >= seam;
    const int64_t ld = up ? ld_q[1] : ld_q[0];
    const T* row = (up ? q[1] : q[0]) + (at - (up ? seam : 0)) * ld + (in ? col : 0);
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      w[slot][i] = __builtin_nontemporal_load((const ADA_GLOBAL u32x4*)(row + i * ld));
#pragma unroll
    for (int f = 0; f < QF; ++f) z[slot][f] = *(const ADA_GLOBAL u32x4*)(zs[f] + at);
    __builtin_amdgcn_sched_barrier(0);
  };
  f32x16 acc[QF][VEC] = {};
  if (steps > 0) {
#pragma unroll
    for (int d = 0; d < D; ++d) load(d, d);
    for (int64_t t = 0; t < steps; t += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        const bool live = first + (t + d) * stride + VEC * h < depth;  // else zeros on both sides
        u32x4 raw[VEC], zf[QF];
#pragma unroll
        for (int i = 0; i < VEC; ++i) raw[i] = live ? w[d][i] : u32x4{0, 0, 0, 0};
#pragma unroll
        for (int f = 0; f < QF; ++f) zf[f] = live ? z[d][f] : u32x4{0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const u32x4 wf = across_fragment<T>(raw, e);
#pragma unroll
          for (int f = 0; f < QF; ++f) acc[f][e] = mfma32<T>(zf[f], wf, acc[f][e]);
        }
        load(d, t + d + D);
      }
    }
  }
  float* const part = held(a.part);
  T* const y = held(static_cast<T*>(a.y[0].p));
  const int64_t ld_y = held(a.y[0].ld);
#pragma unroll
  for (int f = 0; f < QF; ++f) {
    // waves 2 and 3 to 0 and 1, then 1 to 0
#pragma unroll 1
    for (int half = 2; half >= 1; half >>= 1) {
      if (wave >= half && wave < 2 * half) {
        f32x4* to = lds + (wave - half) * VEC * 256 + lane;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            to[(e * 4 + v) * 64] =
                f32x4{acc[f][e][4 * v], acc[f][e][4 * v + 1], acc[f][e][4 * v + 2], acc[f][e][4 * v + 3]};
      }
      __syncthreads();
      if (wave < half) {
        const f32x4* from = lds + wave * VEC * 256 + lane;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const f32x4 o = from[(e * 4 + v) * 64];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[f][e][4 * v + i] += o[i];
          }
      }
      __syncthreads();
    }
    if (wave != 0 || !in) continue;
#pragma unroll
    for (int g = 0; g < 16; ++g) {
      const int64_t r = 32 * f + 8 * (g >> 2) + 4 * h + (g & 3);
      if (r >= rows) continue;
      float v[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = acc[f][e][g];
      if (splits > 1) {
        float* to = part + (split * rows + r) * cols + col;
#pragma unroll
        for (int e = 0; e < VEC; e += 4) *(ADA_GLOBAL f32x4*)(to + e) = f32x4{v[e], v[e + 1], v[e + 2], v[e + 3]};
      } else {
        store_vec<T>(y + r * ld_y + col, v);
      }
    }
  }
}

// dx and dW, or one of them, in one grid: the one reads while the other writes.
template <typename T, int ROWS>
__global__ void __launch_bounds__(256, ROWS > 32 ? 1 : 2) few_rows_grad_kernel(GemmPair pair) {
  __shared__ f32x4 lds[2 * FewGrad<T>::VEC * 256];
  const int second = static_cast<int>(blockIdx.x) >= pair.first;
  const GemmParams& a = pair.a[second];
  const int block = static_cast<int>(blockIdx.x) - (second ? pair.first : 0);
  if (a.form == kDx)
    few_rows_dx<T, (ROWS + 31) / 32>(a, block, lds);
  else
    few_rows_dw<T, ROWS>(a, block);
}

template <typename T, int ROWS>
hipError_t launch_few_rows_grad(const GemmParams* a, int n, hipStream_t s) {
  using F = FewGrad<T>;
  GemmPair pair{};
  int64_t grid = 0;
  for (int i = 0; i < n; ++i) {
    pair.a[i] = a[i];
    if (i == 1) pair.first = static_cast<int32_t>(grid);
    const int64_t strips = (a[i].cols + F::cols - 1) / F::cols;
    grid += strips * (a[i].form == kDx ? a[i].splits : (a[i].rows + F::dw_rows - 1) / F::dw_rows);
  }
  if (n == 1) pair.first = static_cast<int32_t>(grid);
  few_rows_grad_kernel<T, ROWS><<<static_cast<unsigned>(grid), 256, 0, s>>>(pair);
  return hipGetLastError();
}

// ---- slopes ---------------------------------------------------------------------------
// Tiles of kSide x kSide of dz.
struct SlopeParams {
  MatIn dy;
  MatIn pre[2];
  void* dz;        // null or [rows][ld_z]: dz, or dg in columns 0 .., du in columns cols ..
  int64_t ld_z;
  float* sums;     // null or [tile rows][cols (x 2)]: column sums of each 64-row tile
  int64_t rows;
  int32_t cols;
  int32_t tiles_n;
  int32_t act;
};

// dz = dy act'(z), or dg = dy u act'(g), du = dy act(g), and the tile's column sums, in one pass
// over dy and the saved pre-activations: bound by memory (gated, 4096 x 11008: 450 MB in 75 us,
// 6.0 TB/s).
// dz is stored in the storage type, an operand of matrix instructions that take that type: in bf16
// each is off by up to 2^-8 of itself, once, before dx and dW sum over it.  Gradients are then
// within 2.35e-3 of the exact ones (2-norm) where rounding them alone leaves 1.66e-3: the two
// roundings, 1.66e-3 each.  Carrying dz as a sum of two bf16 numbers would take that away for
// twice the matrix instructions (gated backward at 4096 x 11008 x 4096: 1.3 ms, of which they bind
// 1.24); fp32 storage has no such rounding.  The column sums take dz as it was computed.
template <typename T, bool GATED>
__global__ void __launch_bounds__(256) slope_kernel(SlopeParams a) {
  constexpr int VEC = 16 / sizeof(T), PER = kSide / VEC, RSTEP = 256 / PER;
  constexpr int NQ = GATED ? 2 : 1;
  __shared__ float part[RSTEP][kSide];
  const int block = static_cast<int>(blockIdx.x);
  const int64_t m0 = int64_t(block / a.tiles_n) * kSide, n0 = int64_t(block % a.tiles_n) * kSide;
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
        float g = dv * act_slope<T>(zv, a.act);
        if constexpr (GATED) {
          g *= to_f32<T>(u.e[e]);
          const float w = dv * act_value<T>(zv, a.act);
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
        a.sums[(int64_t(block / a.tiles_n) * NQ + h) * a.cols + n0 + threadIdx.x] = s;
      }
    }
  }
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
  return p.gated ? launch_forward<T, true>(a, static_cast<float*>(ws), s)
                 : launch_forward<T, false>(a, static_cast<float*>(ws), s);
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
  const bool want_dx = p.dx.p != nullptr, want_dw = p.dw[0].p != nullptr || p.dw[1].p != nullptr;
  const bool want_db = p.dbias[0] != nullptr || p.dbias[1] != nullptr;
  const bool own_dz = p.gated || p.act != ADA_ACT_NONE;  // else dz is dy

  SlopeParams sl{};
  sl.dy = p.dy;
  sl.pre[0] = p.pre[0];
  sl.pre[1] = p.pre[1];
  sl.dz = own_dz && (want_dx || want_dw) ? base + g.dz : nullptr;
  sl.ld_z = parts * n;
  sl.sums = want_db ? reinterpret_cast<float*>(base + g.sums) : nullptr;
  sl.rows = p.rows;
  sl.cols = p.d_out;
  sl.tiles_n = (p.d_out + kSide - 1) / kSide;
  sl.act = p.act;
  const int64_t tiles_m = (p.rows + kSide - 1) / kSide;
  if (sl.dz != nullptr || sl.sums != nullptr) {
    const unsigned grid = static_cast<unsigned>(tiles_m * sl.tiles_n);
    if (p.gated)
      slope_kernel<T, true><<<grid, 256, 0, s>>>(sl);
    else
      slope_kernel<T, false><<<grid, 256, 0, s>>>(sl);
    ADA_TRY(hipGetLastError());
  }
  const MatIn dz = own_dz ? MatIn{base + g.dz, parts * n} : p.dy;

  GemmParams a[2] = {};
  int tile[2], count = 0;
  auto add = [&](int i) {  // product i of the pair is a[count]
    a[count].splits = g.pair.plan[i].splits;
    a[count].part = reinterpret_cast<float*>(base + g.part[i]);
    tile[count] = g.pair.plan[i].tile;
    return &a[count++];
  };
  // longer workgroups first
  for (int i : {g.pair.plan[0].us >= g.pair.plan[1].us ? 0 : 1, g.pair.plan[0].us >= g.pair.plan[1].us ? 1 : 0}) {
    if (i == 0 && want_dx) {
      GemmParams* d = add(0);
      d->form = kDx;
      d->p = dz;
      d->q[0] = p.w[0];
      d->q[1] = p.gated ? p.w[1] : p.w[0];
      d->seam = p.gated ? n : INT64_MAX / 2;
      d->y[0] = p.dx;
      d->rows = p.rows;
      d->row_split = p.rows;
      d->cols = p.d_in;
      d->depth = parts * n;
    } else if (i == 1 && want_dw) {
      const bool both = p.gated && p.dw[0].p != nullptr && p.dw[1].p != nullptr;
      const int h = p.dw[0].p != nullptr ? 0 : 1;
      GemmParams* d = add(1);
      d->form = kDw;
      d->p = MatIn{static_cast<const T*>(dz.p) + h * n, dz.ld};
      d->q[0] = p.x;
      d->y[0] = p.dw[h];
      d->y[1] = p.dw[1];
      d->rows = both ? 2 * n : n;
      d->row_split = n;
      d->cols = p.d_in;
      d->depth = p.rows;
    }
  }
  if (count > 0 && g.few) {
    if (p.rows <= 16) {
      ADA_TRY((launch_few_rows_grad<T, 16>(a, count, s)));
    } else if (p.rows <= 32) {
      ADA_TRY((launch_few_rows_grad<T, 32>(a, count, s)));
    } else if constexpr (sizeof(T) == 2) {
      ADA_TRY((launch_few_rows_grad<T, 64>(a, count, s)));
    }
  } else if (count == 2 && g.pair.together) {
    ADA_TRY((launch_products<T, false, true>(tile[0], a, 2, s)));
  } else {
    for (int i = 0; i < count; ++i) ADA_TRY((launch_products<T, false, true>(tile[i], a + i, 1, s)));
  }
  BiasParams bias{sl.sums, tiles_m, parts, p.d_out, {p.dbias[0], p.dbias[1]}};
  return launch_joins<T, false>(a, count, want_db ? &bias : nullptr, s);
}

}  // namespace

int64_t linear_workspace(int64_t rows, int32_t d_out, int32_t d_in, int gated, int dtype) {
  if (rows == 0) return 0;
  const int esz = dtype == ADA_BF16 ? 2 : 4;
  return part_bytes({rows, gated ? 2 * int64_t(d_out) : d_out, d_in, esz},
                    plan_forward(rows, d_out, d_in, gated, esz).splits);
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
