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
// lanes.  A pick is a maximum over a lane's eight keys, the same steps across lanes, and a
// ballot that names the first lane that holds it.  Bound by launches and latency at the sizes of a
// training step (16384 rows of 64 experts are 5 MB).
#include "elements.h"

namespace ada {
namespace {

constexpr int kThreads = 1024;
constexpr int kMostBlocks = 256;
#ifndef ONE
#define ONE 32
#endif

// Order-preserving map of fp32 bits to nonzero integers, 0 for -inf (closed); -0 and +0 are equal,
// and NaN is above everything, so a row that holds one still picks experts inside its range.
__device__ __forceinline__ uint32_t rank_key(float f) {
  if (f != f) return 0xffffffffu;
  if (f == -__builtin_inff()) return 0u;
  const uint32_t u = f == 0.f ? 0u : __float_as_uint(f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

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

// Softmax of a row from a lane's eight logits: x over sums to 1.  Whether any expert is open.
template <int L>
__device__ __forceinline__ bool softmax8(const float (&z)[8], uint32_t (&key)[8], float (&x)[8], float& over) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    key[i] = rank_key(z[i]);
    top = max(top, key[i]);
  }
  top = row_max<L>(top);
  const bool open = top != 0;
  const float m = top == 0xffffffffu ? __builtin_nanf("")
                                     : __uint_as_float((top & 0x80000000u) ? top & 0x7fffffffu : ~top);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // a closed expert's is zero also where the largest logit is infinite
    x[i] = key[i] != 0 ? expf(z[i] - m) : 0.f;
    sum += x[i];
  }
  sum = row_sum<L>(sum);
  over = open ? 1.f / sum : 0.f;
  return open;
}

// ---- forward ---------------------------------------------------------------------------
// The last step of the balance: counts, mean probabilities and the loss from the sums over every
// row, expert e on lane e of the first wave.
__device__ __forceinline__ void finish_balance(const RouteParams& p, int lane, int count, double sum, int used) {
  const double n = used > 0 ? double(used) : 1.0;
  if (lane < p.E) {
    p.counts[lane] = count;
    p.prob[lane] = float(sum / n);
  }
  double part = lane < p.E ? double(count) / (double(p.k) * n) * (sum / n) : 0.0;
  for (int m = 1; m < 64; m <<= 1) part += __shfl_xor(part, m, 64);
  if (lane == 0) {
    p.loss[0] = float(double(p.E) * part);
    p.used[0] = used;
  }
}

// Partial sums of the balance of one workgroup, [blocks] of each: probabilities, counts, rows.
struct BalanceParts {
  float* prob;
  int32_t* counts;
  int32_t* used;
};

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
    load_logits<T, VEC>(static_cast<const T*>(p.logits.p) + at * p.logits.ld, first, p.E, z);
    const bool counts_row = inside && (p.valid == nullptr || p.valid[at] != 0);
    uint32_t key[8];
    const bool open = softmax8<L>(z, key, x, over) && counts_row;
#pragma unroll
    for (int i = 0; i < 8; ++i) key[i] = open ? key[i] : 0u;
    uint32_t taken = 0;                     // bit i: expert first + i is picked
    unsigned long long slots = 0;           // byte i: its place among the picks
    int n = 0;
    for (int j = 0; j < p.k; ++j) {
      uint32_t mine = key[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) mine = max(mine, key[i]);
      const uint32_t best = row_max<L>(mine);
      const unsigned long long holders = __ballot(mine == best) >> (lane - l) & ((1ull << L) - 1);
      n += best != 0;
      if (best != 0 && __builtin_ctzll(holders) == l) {
        bool found = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (!found && key[i] == best) {
            found = true;
            key[i] = 0;
            taken |= 1u << i;
            slots |= static_cast<unsigned long long>(j) << (8 * i);
          }
        }
      }
    }
    float picked = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) picked += (taken >> i & 1) ? x[i] : 0.f;
    picked = row_sum<L>(picked);
    const float share = p.renorm ? 1.f / picked : over;
    if (inside) {
      int32_t* idx = p.idx + row * p.k;
      float* gate = p.gate + row * p.k;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (taken >> i & 1) {
          const int j = int(slots >> (8 * i)) & 0xff;
          idx[j] = first + i;
          gate[j] = x[i] * share;
        }
      }
      for (int j = n + l; j < p.k; j += L) {
        idx[j] = -1;
        gate[j] = 0.f;
      }
    }
    if (balance) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        probs[i] += open ? x[i] * over : 0.f;
        counts[i] += taken >> i & 1;
      }
      used += open && l == 0;
    }
  }
  if (!balance) return;

  // the same experts of a wave's rows, then the waves
  __shared__ float wave_prob[kThreads / 64][kMaxExperts];
  __shared__ int wave_count[kThreads / 64][kMaxExperts], wave_used[kThreads / 64];
  const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  for (int m = L; m < 64; m <<= 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      probs[i] += __shfl_xor(probs[i], m, 64);
      counts[i] += __shfl_xor(counts[i], m, 64);
    }
    used += __shfl_xor(used, m, 64);
  }
  if (lane < L) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      wave_prob[wave][first + i] = probs[i];
      wave_count[wave][first + i] = counts[i];
    }
    if (lane == 0) wave_used[wave] = used;
  }
  __syncthreads();
  if (wave != 0) return;
  double sum = 0.0;
  int count = 0, rows = 0;
  if (lane < 8 * L)
    for (int w = 0; w < waves; ++w) {
      sum += wave_prob[w][lane];
      count += wave_count[w][lane];
    }
  for (int w = 0; w < waves; ++w) rows += wave_used[w];
  if (gridDim.x == 1) {
    finish_balance(p, lane, count, sum, rows);
  } else {
    parts.prob[blockIdx.x * kMaxExperts + lane] = float(sum);
    parts.counts[blockIdx.x * kMaxExperts + lane] = count;
    if (lane == 0) parts.used[blockIdx.x] = rows;
  }
}

// One workgroup: expert e on lane e of each wave, the parts dealt to the waves.
__global__ void __launch_bounds__(kThreads) balance_join_kernel(RouteParams p, BalanceParts parts, int blocks) {
  __shared__ double wave_prob[kThreads / 64][64];
  __shared__ int wave_count[kThreads / 64][64], wave_used[kThreads / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  constexpr int EACH = kMostBlocks / (kThreads / 64);
  double sum = 0.0;
  int count = 0, used = 0;
  float prob[EACH];
  int counts[EACH], rows[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) {  // all loads in flight at once
    const int b = wave + i * (kThreads / 64);
    prob[i] = b < blocks ? parts.prob[b * kMaxExperts + lane] : 0.f;
    counts[i] = b < blocks ? parts.counts[b * kMaxExperts + lane] : 0;
    rows[i] = b < blocks ? parts.used[b] : 0;
  }
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    sum += prob[i];
    count += counts[i];
    used += rows[i];
  }
  wave_prob[wave][lane] = sum;
  wave_count[wave][lane] = count;
  if (lane == 0) wave_used[wave] = used;
  __syncthreads();
  if (wave != 0) return;
  sum = 0.0;
  count = used = 0;
  for (int w = 0; w < kThreads / 64; ++w) {
    sum += wave_prob[w][lane];
    count += wave_count[w][lane];
    used += wave_used[w];
  }
  finish_balance(p, lane, count, sum, used);
}

// ---- backward --------------------------------------------------------------------------
// Eight of a row's picks, loaded together; past the k-th none (index -1).
struct Picks {
  int e[8];
  float gate[8], dgate[8];

  __device__ __forceinline__ void load(const RouteGradParams& p, int64_t at, int j0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool some = j0 + j < p.k;
      const int64_t i = at * p.k + (some ? j0 + j : 0);
      e[j] = some ? p.idx[i] : -1;
      gate[j] = p.renorm ? p.gate[i] : 1.f;
      dgate[j] = p.dgate[i];
    }
  }
};

// The lanes of a row read the same picks, and each keeps what falls on its eight experts; an index
// outside [0, E) is passed over.  The first eight picks stay in registers between the sum over
// them and its use.
template <typename T, int L, bool VEC>
__global__ void __launch_bounds__(256) route_grad_kernel(RouteGradParams p) {
  const int l = threadIdx.x & (L - 1), first = l * 8;
  const int64_t row = (int64_t(blockIdx.x) * 256 + threadIdx.x) / L;
  const bool inside = row < p.rows;
  const int64_t at = inside ? row : p.rows - 1;
  float z[8], x[8], over, dp[8], dz[8];
  uint32_t key[8];
  Picks picks;
  load_logits<T, VEC>(static_cast<const T*>(p.logits.p) + at * p.logits.ld, first, p.E, z);
  const int top = p.idx[at * p.k];
  if (p.dgate != nullptr) picks.load(p, at, 0);
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
  const bool open = softmax8<L>(z, key, x, over) && top >= 0;
  if (p.dgate != nullptr) {
    float along = 0.f;
    if (p.renorm) {
      for (int j0 = 0; j0 < p.k; j0 += 8) {
        if (j0 > 0) picks.load(p, at, j0);
#pragma unroll
        for (int j = 0; j < 8; ++j) along += picks.e[j] >= 0 ? picks.gate[j] * picks.dgate[j] : 0.f;
      }
    }
    for (int j0 = 0; j0 < p.k; j0 += 8) {
      if (p.k > 8) picks.load(p, at, j0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = picks.e[j] - first;
        const float d = p.renorm ? picks.gate[j] * (picks.dgate[j] - along) : picks.dgate[j];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (p.renorm)
            dz[i] += e == i ? d : 0.f;
          else
            dp[i] += e == i ? d : 0.f;
        }
      }
    }
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

RouteGrid route_grid(int64_t rows, int E) {
  const int64_t waves = (rows * row_lanes(E) + 63) / 64;
  if (waves <= ONE) return {1, static_cast<int>(waves < 1 ? 64 : waves < 16 ? 64 * waves : kThreads)};
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
    parts.prob = static_cast<float*>(ws);
    parts.counts = reinterpret_cast<int32_t*>(parts.prob + g.blocks * kMaxExperts);
    parts.used = parts.counts + g.blocks * kMaxExperts;
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
