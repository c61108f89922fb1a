// The router's choice for many rows, its balance loss and both gradients, from the logits
// z [rows][E] of a router product.
//
//   p = softmax(z); the k largest z of a row in descending order, equal ones lower index first;
//   g = softmax over the picked logits (renorm) or p at the picked; counts_e = rows that picked e,
//   prob_e = mean of p_e over the n rows that count; loss = E sum_e (counts_e / (k n)) prob_e
//   dp_e = dloss E counts_e / (k n^2) (+ dg_j at the picked, without renorm)
//   dz = p (dp - sum p dp) (+ g_j (dg_j - sum g dg) at the picked, with renorm)
//
// A logit of -inf is an expert closed to the row: probability 0, never picked.  A row counts
// if its flag says so and one expert is open to it; the others get index -1, gate 0, gradient 0.
//
// A row is shared by 1, 2, 4 or 8 neighbouring lanes, eight experts each, so one 16-byte load a
// lane (bf16) brings a wave 8 to 64 rows and the softmax needs at most three steps across
// lanes.  A pick is a maximum over a lane's eight keys and the row's lanes, then the lowest index that
// holds it.  Bound by launches and latency up to some ten thousand rows (16384 rows of 64 experts
// are 5 MB), by the picks' instructions past that (262144 x 64 fp32, eight picks: 41 us for 84 MB, 48 with the balance).
#include "elements.h"

namespace ada {
namespace {

constexpr int kThreads = 1024;
constexpr int kMostBlocks = 256;

// Order-preserving map of a logit to an integer: -0 and +0 are equal, NaN is above everything (a
// row that holds one still picks inside its range), and -inf, a closed expert, gives kClosed, next below
// the lowest finite one.
constexpr uint32_t kClosed = 0x007fffffu;
__device__ __forceinline__ uint32_t rank_key(float f) {
  const uint32_t u = __float_as_uint(f + 0.f);
  const uint32_t k = u ^ (uint32_t(int(u) >> 31) | 0x80000000u);
  return f == f ? k : 0xffffffffu;
}
__device__ __forceinline__ float value_of_key(uint32_t k) {  // of an open expert; NaN of 0xffffffff
  return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

template <int V>
struct Int {
  static constexpr int value = V;
};
template <int CTRL>
__device__ __forceinline__ uint32_t swapped(uint32_t v) {
  return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, 0xf, 0xf, true));
}
// The value of the lane 1, 2 or (where groups of four lanes already agree) 4 away.
template <int STEP>
__device__ __forceinline__ uint32_t across(uint32_t v) {
  if constexpr (STEP == 1) return swapped<0xB1>(v);  // quad_perm [1, 0, 3, 2]
  if constexpr (STEP == 2) return swapped<0x4E>(v);  // quad_perm [2, 3, 0, 1]
  return swapped<0x141>(v);                          // row_half_mirror: lane 7 - l of eight
}
template <int L>
__device__ __forceinline__ float row_sum(float v) {
  if constexpr (L > 1) v += __uint_as_float(across<1>(__float_as_uint(v)));
  if constexpr (L > 2) v += __uint_as_float(across<2>(__float_as_uint(v)));
  if constexpr (L > 4) v += __uint_as_float(across<4>(__float_as_uint(v)));
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  if constexpr (L > 1) v = max(v, across<1>(v));
  if constexpr (L > 2) v = max(v, across<2>(v));
  if constexpr (L > 4) v = max(v, across<4>(v));
  return v;
}

template <int L>
__device__ __forceinline__ uint32_t row_min(uint32_t v) {
  if constexpr (L > 1) v = min(v, across<1>(v));
  if constexpr (L > 2) v = min(v, across<2>(v));
  if constexpr (L > 4) v = min(v, across<4>(v));
  return v;
}
// Sum over the lanes of 16 that hold the same part of their rows, on each of them (rotations by
// L, 2 L, .. 8 of the row of 16).
template <int L, typename V>
__device__ __forceinline__ V same_part_sum(V v) {
  const auto turned = [](auto ctrl, V a) {
    return __builtin_bit_cast(
        V, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, a), decltype(ctrl)::value, 0xf, 0xf, true));
  };
  if constexpr (L <= 1) v += turned(Int<0x121>(), v);
  if constexpr (L <= 2) v += turned(Int<0x122>(), v);
  if constexpr (L <= 4) v += turned(Int<0x124>(), v);
  v += turned(Int<0x128>(), v);
  return v;
}

__device__ __forceinline__ float value_of(float v) { return v; }
__device__ __forceinline__ float value_of(uint16_t v) { return __uint_as_float(uint32_t(v) << 16); }

// A lane's eight logits; experts past E are closed.  VEC: 16-byte vectors (E a multiple of eight,
// rows aligned).
template <typename T, bool VEC>
__device__ __forceinline__ void load_logits(const T* row, int first, int E, float (&z)[8]) {
  if constexpr (VEC) {
    if (first < E) {
      unpack(load_eight(row + first), z);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = -__builtin_inff();
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = first + i < E ? value_of(row[first + i]) : -__builtin_inff();
  }
}

// Softmax of a row from a lane's eight logits, x over sums to 1, and their keys; a row that does not
// count has every expert closed.  Whether any is open.
template <int L>
__device__ __forceinline__ bool softmax8(const float (&z)[8], bool counts, uint32_t (&key)[8], float (&x)[8],
                                         float& m, float& over) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    key[i] = counts ? rank_key(z[i]) : 0u;
    top = max(top, key[i]);
  }
  top = row_max<L>(top);
  m = value_of_key(top);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // a closed expert's is zero also where the largest logit is infinite
    x[i] = key[i] > kClosed ? expf(z[i] - m) : 0.f;
    sum += x[i];
  }
  sum = row_sum<L>(sum);
  over = top > kClosed ? 1.f / sum : 0.f;
  return top > kClosed;
}

// ---- forward ---------------------------------------------------------------------------
__device__ __forceinline__ double wave_total(double v) {
  const auto part = [&](auto ctrl, auto rows) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    constexpr int CTRL = decltype(ctrl)::value, ROWS = decltype(rows)::value;
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, int(uint32_t(u)), CTRL, ROWS, 0xf, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, int(u >> 32), CTRL, ROWS, 0xf, true);
    return __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
  };
  v += part(Int<0x111>(), Int<0xf>());
  v += part(Int<0x112>(), Int<0xf>());
  v += part(Int<0x114>(), Int<0xf>());
  v += part(Int<0x118>(), Int<0xf>());
  v += part(Int<0x142>(), Int<0xa>());
  v += part(Int<0x143>(), Int<0xc>());
  return v;  // on lane 63
}

// The last step of the balance: counts, mean probabilities and the loss from the sums over every
// row, expert e on lane e of one wave.
__device__ __forceinline__ void finish_balance(const RouteParams& p, int lane, int count, double sum, int used) {
  const double over = used > 0 ? 1.0 / double(used) : 1.0, mean = sum * over;
  if (lane < p.E) {
    p.counts[lane] = count;
    p.prob[lane] = float(mean);
  }
  const double total = wave_total(lane < p.E ? double(count) * mean : 0.0);
  if (lane == 63) {
    p.loss[0] = float(total * over * p.per_pick);
    p.used[0] = used;
  }
}

// Partial sums of the balance, one of each for every workgroup.
struct BalanceParts {
  uint2* experts;  // [blocks][kMaxExperts]: sum of probabilities (fp32 bits), picks
  int32_t* used;   // [blocks]: rows that count
};

// The next pick of a row, known to all its lanes: the largest key, the lowest index among equals.  It
// is marked as taken.  `best` is at most kClosed where no open expert is left.
constexpr uint32_t kTaken = 1;  // no logit's key
template <int L>
__device__ __forceinline__ uint32_t next_pick(uint32_t (&key)[8], int first, uint32_t& best) {
  best = key[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) best = max(best, key[i]);
  best = row_max<L>(best);
  uint32_t at = kMaxExperts;  // none
#pragma unroll
  for (int i = 7; i >= 0; --i) at = key[i] == best ? first + i : at;
  at = best > kClosed ? row_min<L>(at) : kMaxExperts;
#pragma unroll
  for (int i = 0; i < 8; ++i) key[i] = at == uint32_t(first + i) ? kTaken : key[i];
  return at;
}

template <typename T, int L, bool VEC>
__global__ void __launch_bounds__(kThreads) route_kernel(RouteParams p, BalanceParts parts) {
  const int lane = threadIdx.x & 63, l = lane & (L - 1), first = l * 8;
  const int rows_at_once = blockDim.x / L;
  const bool balance = p.counts != nullptr;
  float probs[8] = {};
  int counts[8] = {}, used = 0;
  for (int64_t row0 = int64_t(blockIdx.x) * rows_at_once; row0 < p.rows; row0 += int64_t(gridDim.x) * rows_at_once) {
    const int64_t row = row0 + threadIdx.x / L;
    const bool inside = row < p.rows;
    const int64_t at = inside ? row : p.rows - 1;
    float z[8], x[8], over;
    uint32_t key[8];
    load_logits<T, VEC>(static_cast<const T*>(p.logits.p) + at * p.logits.ld, first, p.E, z);
    float m;
    const bool open = softmax8<L>(z, inside && (p.valid == nullptr || p.valid[at] != 0), key, x, m, over);
    // pick j = q L + l stays on lane l
    uint32_t pick[8];
    float e[8], picked = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (q * L >= p.k) break;
      uint32_t mine = 0;
      pick[q] = kMaxExperts;
#pragma unroll 1  // little code: a workgroup walks through it once or twice, and every line of it is fetched
      for (int t = 0; t < L && q * L + t < p.k; ++t) {
        uint32_t best;
        const uint32_t one = next_pick<L>(key, first, best);
        pick[q] = t == l ? one : pick[q];
        mine = t == l ? best : mine;
      }
      e[q] = pick[q] < kMaxExperts ? expf(value_of_key(mine) - m) : 0.f;
      picked += e[q];
    }
    picked = row_sum<L>(picked);
    const float share = p.renorm ? (open ? 1.f / picked : 0.f) : over;
    if (inside) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int j = q * L + l;
        if (q * L >= p.k) break;
        if (j < p.k) {
          const bool some = pick[q] < kMaxExperts;
          p.idx[row * p.k + j] = some ? int32_t(pick[q]) : -1;
          p.gate[row * p.k + j] = some ? e[q] * share : 0.f;
        }
      }
    }
    if (balance) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        probs[i] = fmaf(x[i], over, probs[i]);
        counts[i] += key[i] == kTaken;
      }
      used += open && l == 0;
    }
  }
  if (!balance) return;

  // the same experts of 16 lanes' rows, of a wave's four such sets, of the waves
  constexpr int WAVES = kThreads / 64;
  __shared__ float set_prob[WAVES][4][kMaxExperts], wave_prob[WAVES][kMaxExperts];
  __shared__ int set_count[WAVES][4][kMaxExperts], wave_count[WAVES][kMaxExperts], wave_used[WAVES];
  const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    probs[i] = same_part_sum<L>(probs[i]);
    counts[i] = same_part_sum<L>(counts[i]);
  }
  if ((lane & 15) < L) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      set_prob[wave][lane >> 4][first + i] = probs[i];
      set_count[wave][lane >> 4][first + i] = counts[i];
    }
  }
  for (int s = 1; s < 64; s <<= 1) used += __shfl_xor(used, s, 64);
  __syncthreads();
  {
    const float* sp = set_prob[wave][0] + lane;
    const int* sc = set_count[wave][0] + lane;
    const bool real = lane < 8 * L;
    wave_prob[wave][lane] = real ? (sp[0] + sp[64]) + (sp[128] + sp[192]) : 0.f;
    wave_count[wave][lane] = real ? (sc[0] + sc[64]) + (sc[128] + sc[192]) : 0;
    if (lane == 0) wave_used[wave] = used;
  }
  __syncthreads();
  if (wave != 0) return;
  double sum = 0.0;
  int count = 0, rows = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    if (w >= waves) break;
    sum += wave_prob[w][lane];
    count += wave_count[w][lane];
    rows += wave_used[w];
  }
  if (gridDim.x == 1) {
    finish_balance(p, lane, count, sum, rows);
  } else {
    parts.experts[blockIdx.x * kMaxExperts + lane] = make_uint2(__float_as_uint(float(sum)), uint32_t(count));
    if (lane == 0) parts.used[blockIdx.x] = rows;
  }
}

// One workgroup: expert e on lane e of each wave, the parts dealt to the waves, all of a lane's loads
// in flight at once.
__global__ void __launch_bounds__(kThreads) balance_join_kernel(RouteParams p, BalanceParts parts, int blocks) {
  constexpr int WAVES = kThreads / 64, EACH = kMostBlocks / WAVES;
  __shared__ double wave_prob[WAVES][64];
  __shared__ int wave_count[WAVES][64], wave_used[WAVES];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint2 part[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int b = wave + i * WAVES;
    if (i * WAVES >= blocks) break;
    part[i] = parts.experts[(b < blocks ? b : 0) * kMaxExperts + lane];
  }
  static_assert(kMostBlocks <= kThreads);
  int used = int(threadIdx.x) < blocks ? parts.used[threadIdx.x] : 0;
  double sum = 0.0;
  int count = 0;
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    if (i * WAVES >= blocks) break;
    const bool some = wave + i * WAVES < blocks;
    sum += some ? __uint_as_float(part[i].x) : 0.f;
    count += some ? int(part[i].y) : 0;
  }
  for (int s = 1; s < 64; s <<= 1) used += __shfl_xor(used, s, 64);
  wave_prob[wave][lane] = sum;
  wave_count[wave][lane] = count;
  if (lane == 0) wave_used[wave] = used;
  __syncthreads();
  if (wave != 0) return;
  sum = 0.0;
  count = used = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    sum += wave_prob[w][lane];
    count += wave_count[w][lane];
    used += wave_used[w];
  }
  finish_balance(p, lane, count, sum, used);
}

// ---- backward --------------------------------------------------------------------------
// The lanes of a row share its picks, add each one's part to the row in LDS (an index outside
// [0, E) is passed over, one that is there twice is added twice), and take their eight experts' back.  The
// additions are atomic: of two parts their order does not matter, of three, which the forward pass never
// writes, it would.  262144 x 64 fp32, eight picks: 47 us for 159 MB; a lane's eight logits in a row
// make each 16-byte access touch half of every line (bf16, whole lines: 38 us for 92 MB).
template <typename T, int L, bool VEC>
__global__ void __launch_bounds__(256) route_grad_kernel(RouteGradParams p) {
  __shared__ float at_expert[256][8];  // rows of 8 L, one to L lanes
  const int l = threadIdx.x & (L - 1), first = l * 8;
  const int64_t row = (int64_t(blockIdx.x) * 256 + threadIdx.x) / L;
  const bool inside = row < p.rows;
  const int64_t at = inside ? row : p.rows - 1;
  float* mine = at_expert[threadIdx.x];
  float* theirs = at_expert[threadIdx.x - l];
  float z[8], x[8], m, over, dp[8], dz[8];
  uint32_t key[8];
  load_logits<T, VEC>(static_cast<const T*>(p.logits.p) + at * p.logits.ld, first, p.E, z);
  const bool counts = p.idx[at * p.k] >= 0;
  int e[8];
  float g[8], d[8];
  if (p.dgate != nullptr) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (q * L >= p.k) break;
      const bool some = q * L + l < p.k;
      const int64_t j = at * p.k + (some ? q * L + l : 0);
      e[q] = some ? p.idx[j] : -1;
      g[q] = p.renorm ? p.gate[j] : 1.f;
      d[q] = p.dgate[j];
    }
  }
  float per_count = 0.f;
  if (p.dloss != nullptr) {
    const int used = p.used[0];
    if (used > 0) per_count = float(double(p.dloss[0]) * p.E / (double(p.k) * used * used));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    dp[i] = p.dloss != nullptr && first + i < p.E ? per_count * float(p.counts[first + i]) : 0.f;
    dz[i] = 0.f;
  }
  const bool open = softmax8<L>(z, counts, key, x, m, over);
  if (p.dgate != nullptr) {
    float along = 0.f;
    if (p.renorm) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (q * L >= p.k) break;
        along += uint32_t(e[q]) < uint32_t(p.E) ? g[q] * d[q] : 0.f;
      }
      along = row_sum<L>(along);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) mine[i] = 0.f;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (q * L >= p.k) break;
      if (uint32_t(e[q]) < uint32_t(p.E)) atomicAdd(theirs + e[q], g[q] * (d[q] - along));
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) (p.renorm ? dz[i] : dp[i]) += mine[i];
  }
  float along = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] *= over;
    along = fmaf(x[i], dp[i], along);
  }
  along = row_sum<L>(along);
#pragma unroll
  for (int i = 0; i < 8; ++i) dz[i] = open ? fmaf(x[i], dp[i] - along, dz[i]) : 0.f;
  if (!inside) return;
  T* out = static_cast<T*>(p.dlogits.p) + row * p.dlogits.ld + first;
  if constexpr (VEC) {
    if (first < p.E) store_eight(out, dz);
  } else {
    const Eight<T> e = pack(dz, T());
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (first + i >= p.E) continue;
      if constexpr (sizeof(T) == 2)
        out[i] = uint16_t(e.v[0][i >> 1] >> (16 * (i & 1)));
      else
        out[i] = dz[i];
    }
  }
}

// ---- rules on sizes --------------------------------------------------------------------
int row_lanes(int E) { return E <= 8 ? 1 : E <= 16 ? 2 : E <= 32 ? 4 : 8; }

struct RouteGrid {
  int blocks;
  int threads;
};

// One workgroup where its waves suffice: it needs no second launch to join the balance (512 x 16: 6.4 us;
// 1024 x 16 in 16 workgroups and a join 7.3, in one workgroup of two steps 9.4).  Otherwise the rows spread
// over all CUs, four waves a workgroup or more.
RouteGrid route_grid(int64_t rows, int E) {
  const int64_t waves = (rows * row_lanes(E) + 63) / 64;
  if (waves <= kThreads / 64) return {1, static_cast<int>(waves < 1 ? 64 : 64 * waves)};
  const int64_t each = (waves + kMostBlocks - 1) / kMostBlocks, most = each < 4 ? 4 : each < 16 ? each : 16;
  const int64_t blocks = (waves + most - 1) / most;
  return {static_cast<int>(blocks < kMostBlocks ? blocks : kMostBlocks), static_cast<int>(64 * most)};
}

// Whether eight logits may be moved as 16-byte vectors.
bool vectors(const void* p, int64_t ld, int E, int dtype) {
  const int64_t esz = dtype == 1 ? 2 : 4;
  return E % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * esz % 16 == 0;
}

template <typename T, int L>
void forward(const RouteParams& p, const BalanceParts& parts, const RouteGrid& g, bool vec, hipStream_t s) {
  if (vec)
    hipLaunchKernelGGL((route_kernel<T, L, true>), dim3(g.blocks), dim3(g.threads), 0, s, p, parts);
  else
    hipLaunchKernelGGL((route_kernel<T, L, false>), dim3(g.blocks), dim3(g.threads), 0, s, p, parts);
}
template <typename T>
void forward(const RouteParams& p, const BalanceParts& parts, const RouteGrid& g, bool vec, hipStream_t s) {
  switch (row_lanes(p.E)) {
    case 1: return forward<T, 1>(p, parts, g, vec, s);
    case 2: return forward<T, 2>(p, parts, g, vec, s);
    case 4: return forward<T, 4>(p, parts, g, vec, s);
    default: return forward<T, 8>(p, parts, g, vec, s);
  }
}

template <typename T, int L>
void backward(const RouteGradParams& p, bool vec, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>((p.rows * L + 255) / 256));
  if (vec)
    hipLaunchKernelGGL((route_grad_kernel<T, L, true>), grid, dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((route_grad_kernel<T, L, false>), grid, dim3(256), 0, s, p);
}
template <typename T>
void backward(const RouteGradParams& p, bool vec, hipStream_t s) {
  switch (row_lanes(p.E)) {
    case 1: return backward<T, 1>(p, vec, s);
    case 2: return backward<T, 2>(p, vec, s);
    case 4: return backward<T, 4>(p, vec, s);
    default: return backward<T, 8>(p, vec, s);
  }
}

}  // namespace

int64_t route_workspace(int64_t rows, int32_t E) {
  const int blocks = route_grid(rows, E).blocks;
  return blocks == 1 ? 0 : int64_t(blocks) * (2 * kMaxExperts + 1) * 4;
}

hipError_t launch_route(const RouteParams& p, int dtype, void* ws, hipStream_t s) {
  // no rows: one workgroup that writes a balance of nothing
  if (p.rows == 0 && p.counts == nullptr) return hipSuccess;
  const RouteGrid g = route_grid(p.rows, p.E);
  const bool join = g.blocks > 1 && p.counts != nullptr;
  BalanceParts parts{};
  if (join) {
    parts.experts = static_cast<uint2*>(ws);
    parts.used = reinterpret_cast<int32_t*>(parts.experts + g.blocks * kMaxExperts);
  }
  const bool vec = vectors(p.logits.p, p.logits.ld, p.E, dtype);
  if (dtype == 1)
    forward<uint16_t>(p, parts, g, vec, s);
  else
    forward<float>(p, parts, g, vec, s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !join) return e;
  hipLaunchKernelGGL(balance_join_kernel, dim3(1), dim3(kThreads), 0, s, p, parts, g.blocks);
  return hipGetLastError();
}

hipError_t launch_route_grad(const RouteGradParams& p, int dtype, hipStream_t s) {
  if (p.rows == 0) return hipSuccess;
  const bool vec = vectors(p.logits.p, p.logits.ld, p.E, dtype) && vectors(p.dlogits.p, p.dlogits.ld, p.E, dtype);
  if (dtype == 1)
    backward<uint16_t>(p, vec, s);
  else
    backward<float>(p, vec, s);
  return hipGetLastError();
}

}  // namespace ada
