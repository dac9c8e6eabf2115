// Layer norm of rows, and its gradients.
//   y = n * w + b, n = (x - mean) * rstd;  dx = rstd * (g - mean(g) - n * mean(g n)), g = dy * w;
//   dw = sum over rows of dy * n;  db = sum over rows of dy
//
// Bound by memory: a row is read once and stays in registers, so its mean, the differences from it (their squares are the
// variance: no difference of large numbers), and the result cost no second read.
// - The mean. The row's sum times 1 / dim is off by a few steps of fp32, which every difference would have; their sum, which
//   comes with that of their squares, says by how much (stats_of; 1 us of 43 for 131071 rows of 128).
// - The split. A row belongs to a group of 8 to 256 lanes, as few as hold it in at most 4 pieces of 16 bytes each:
//   narrow rows need no barrier and no idle lanes, wide ones need few registers. Rows that fit no group (more than 8192
//   columns of 16 bits) or start on no 16-byte boundary are read value by value, the longest of them several times.
// - The parameters' gradients. A lane holds the same columns of all of its rows, so a CTA, which walks over many rows,
//   adds up both sums in registers, joins its groups once at its end in a fixed order, and leaves one row of partial
//   sums; a second kernel adds those up. No atomics: the same sums in every run.
// Measured in bf16, in a graph: 131071 rows of 128, forward 15.5 us (10 at the copy rate), with all gradients 44 (25); 16384
// rows of 1536 23.5 (15) and 68 (37); a decode step's 48 rows of 128, forward, 1.5. What bounds it is instructions as much as
// loads: of narrow rows the forward has 3.0 issued a clock and SM (of four), the ALU busy half of the time, the gradient 2.4, and
// each row's loads come before its two sums, with nothing of the next row under way. Two rows at once (57 us), the next row's loads
// ahead of this one's sums (62 and 35 us for the gradients alone) and a CTA or a warp for each wide row were slower: their registers
// cost as many resident warps. Rows on no 16-byte boundary are read a value at a time: 16384 rows of 1002 31 and 91 us (of 1000: 18
// and 53), of 1537, which no group holds, 69 and 249; long rows are read three times, and twice more for the parameters'
// gradients: 4096 rows of 16384 133 us (40) and 631 (99).

#include <algorithm>

#include "indexer_common.cuh"

namespace indexer_gb300 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct NormParams {
  const void* x;
  const void* dy;      // gradient: that of the result
  const void* weight;
  const void* bias;    // may be NULL
  void* out;           // forward: the result; gradient: that of x, may be NULL
  float* stats;        // mean and rstd of each row; forward: may be NULL
  float* partial;      // gradient: [parts][2][dim], or NULL
  int64_t x_ts, x_hs, dy_ts, dy_hs;
  Divisor heads;
  uint32_t rows;
  int32_t dim, params32;  // params32: fp32 parameters, else the rows' type
  float eps, inv_dim;
};

// A row's mean and 1 / sqrt(variance + eps). `about`: the sum of the row times 1 / dim, which is off by the sum's rounding and
// by that of 1 / dim, a step or more of fp32 that each difference from it would have, times rstd (a constant row of 200 in 7168
// columns came out as -0.015). sums: of the differences from `about`, and of their squares: the first one is what `about` lacks.
__device__ __forceinline__ float2 stats_of(const NormParams& p, float about, const float (&sums)[2]) {
  const float rest = sums[0] * p.inv_dim;
  float var = sums[1] * p.inv_dim;
  if (var < 3.0e38f) var = fmaxf(fmaf(-rest, rest, var), 0.0f);  // (an infinity or a NaN stays one)
  return make_float2(about + rest, rsqrtf(var + p.eps));
}

__device__ __forceinline__ float param_at(const void* p, bool wide, int i, float) { return static_cast<const float*>(p)[i]; }
template <typename T>
__device__ __forceinline__ float param_at(const void* p, bool wide, int i, T) {
  return wide ? static_cast<const float*>(p)[i] : to_float(static_cast<const T*>(p)[i]);
}

// V consecutive parameters.
template <typename T, int V>
__device__ __forceinline__ void params_at(const void* p, bool wide, int col, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = param_at(p, wide, col, T());
  } else if (sizeof(T) == 4 || wide) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + col + i);
      f[i] = a.x, f[i + 1] = a.y, f[i + 2] = a.z, f[i + 3] = a.w;
    }
  } else {
    const Pack<T, V> a = *reinterpret_cast<const Pack<T, V>*>(static_cast<const T*>(p) + col);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = to_float(a.v[i]);
  }
}

// Sums of N values over groups of L lanes; every lane of a group takes part, and waits for no other group. `turn` tells one
// use of the scratch from the next: a lane that writes at turn t + 2 has passed the barrier of t + 1, which all reached
// after their reads of t.
template <int L, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float (&scratch)[2][N][kWarps], int& turn) {
#pragma unroll
  for (int d = (L < 32 ? L : 32) / 2; d > 0; d /= 2)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], d);
  if constexpr (L > 32) {
    constexpr int kPart = L / 32;
    const int warp = threadIdx.x / 32;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int k = 0; k < N; ++k) scratch[turn][k][warp] = v[k];
    asm volatile("bar.sync %0, %1;" ::"r"(warp / kPart + 1), "n"(L) : "memory");
#pragma unroll
    for (int k = 0; k < N; ++k) {
      v[k] = 0.0f;
#pragma unroll
      for (int w = 0; w < kPart; ++w) v[k] += scratch[turn][k][warp / kPart * kPart + w];
    }
    turn ^= 1;
  }
}

template <typename T>
__device__ __forceinline__ const T* row_at(const void* base, const NormParams& p, uint32_t row, int64_t ts, int64_t hs) {
  const uint32_t t = quotient(p.heads, row);
  return static_cast<const T*>(base) + t * ts + (row - t * p.heads.d) * hs;
}

template <typename T, int V, int L, int P>
__global__ void __launch_bounds__(kThreads) norm_kernel(const NormParams p) {
  constexpr int kGroups = kThreads / L;
  constexpr bool kHold = P * V <= 16;  // the parameters stay in registers
  __shared__ float scratch[2][1][kWarps], scratch2[2][2][kWarps];
  begin_after_prior_grids();
  const int lane = threadIdx.x % L;
  const bool wide = p.params32 != 0, shift = p.bias != nullptr;
  int turn = 0;
  float w[kHold ? P : 1][V], b[kHold ? P : 1][V];
  auto params = [&](int q, int col) {
    params_at<T, V>(p.weight, wide, col, w[kHold ? q : 0]);
#pragma unroll
    for (int i = 0; i < V; ++i) b[kHold ? q : 0][i] = 0.0f;
    if (shift) params_at<T, V>(p.bias, wide, col, b[kHold ? q : 0]);
  };
  if constexpr (kHold) {
#pragma unroll
    for (int q = 0; q < P; ++q) {
      const int col = (q * L + lane) * V;
      if (col < p.dim) params(q, col);
    }
  }
  for (uint32_t r0 = blockIdx.x * kGroups; r0 < p.rows; r0 += gridDim.x * kGroups) {
    const uint32_t row = r0 + threadIdx.x / L;
    const bool live = row < p.rows;
    const T* src = row_at<T>(p.x, p, live ? row : 0, p.x_ts, p.x_hs);
    Pack<T, V> raw[P];
    float sum[1] = {0.0f};
#pragma unroll
    for (int q = 0; q < P; ++q) {
      const int col = (q * L + lane) * V;
      if (live && col < p.dim) {
        raw[q] = *reinterpret_cast<const Pack<T, V>*>(src + col);
#pragma unroll
        for (int i = 0; i < V; ++i) sum[0] += to_float(raw[q].v[i]);
      }
    }
    group_sum<L, 1>(sum, scratch, turn);
    const float about = sum[0] * p.inv_dim;
    float sums[2] = {0.0f, 0.0f};
#pragma unroll
    for (int q = 0; q < P; ++q) {
      const int col = (q * L + lane) * V;
      if (live && col < p.dim)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float d = to_float(raw[q].v[i]) - about;
          sums[0] += d;
          sums[1] = fmaf(d, d, sums[1]);
        }
    }
    group_sum<L, 2>(sums, scratch2, turn);
    const float2 stat = stats_of(p, about, sums);
    const float mean = stat.x, rstd = stat.y;
    if (!live) continue;
    if (p.stats != nullptr && lane == 0)
      *reinterpret_cast<float2*>(p.stats + 2 * static_cast<int64_t>(row)) = stat;
    T* dst = static_cast<T*>(p.out) + static_cast<int64_t>(row) * p.dim;
#pragma unroll
    for (int q = 0; q < P; ++q) {
      const int col = (q * L + lane) * V, at = kHold ? q : 0;
      if (col < p.dim) {
        if constexpr (!kHold) params(q, col);
        Pack<T, V> y;
#pragma unroll
        for (int i = 0; i < V; ++i) y.v[i] = from_float<T>(fmaf((to_float(raw[q].v[i]) - mean) * rstd, w[at][i], b[at][i]));
        *reinterpret_cast<Pack<T, V>*>(dst + col) = y;
      }
    }
  }
}

// Any row, one a CTA, read three times (from L1 or L2 after the first).
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_long_kernel(const NormParams p) {
  __shared__ float scratch[2][1][kWarps], scratch2[2][2][kWarps];
  begin_after_prior_grids();
  const bool wide = p.params32 != 0;
  int turn = 0;
  for (uint32_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* src = row_at<T>(p.x, p, row, p.x_ts, p.x_hs);
    float sum[1] = {0.0f}, sums[2] = {0.0f, 0.0f};
    for (int c = threadIdx.x; c < p.dim; c += kThreads) sum[0] += to_float(src[c]);
    group_sum<kThreads, 1>(sum, scratch, turn);
    const float about = sum[0] * p.inv_dim;
    for (int c = threadIdx.x; c < p.dim; c += kThreads) {
      const float d = to_float(src[c]) - about;
      sums[0] += d;
      sums[1] = fmaf(d, d, sums[1]);
    }
    group_sum<kThreads, 2>(sums, scratch2, turn);
    const float2 stat = stats_of(p, about, sums);
    const float mean = stat.x, rstd = stat.y;
    if (p.stats != nullptr && threadIdx.x == 0)
      *reinterpret_cast<float2*>(p.stats + 2 * static_cast<int64_t>(row)) = stat;
    T* dst = static_cast<T*>(p.out) + static_cast<int64_t>(row) * p.dim;
    for (int c = threadIdx.x; c < p.dim; c += kThreads)
      dst[c] = from_float<T>(fmaf((to_float(src[c]) - mean) * rstd, param_at(p.weight, wide, c, T()),
                                  p.bias != nullptr ? param_at(p.bias, wide, c, T()) : 0.0f));
  }
}

// Gradients of rows; and of the parameters one row of partial sums for each CTA.
template <typename T, int V, int L, int P>
__global__ void __launch_bounds__(kThreads) norm_grad_kernel(const NormParams p) {
  constexpr int kGroups = kThreads / L;
  extern __shared__ float joined[];  // [2][dim]
  __shared__ float scratch[2][2][kWarps];
  begin_after_prior_grids();
  const int lane = threadIdx.x % L;
  const bool wide = p.params32 != 0;
  int turn = 0;
  float dw[P][V], db[P][V];
#pragma unroll
  for (int q = 0; q < P; ++q)
#pragma unroll
    for (int i = 0; i < V; ++i) dw[q][i] = db[q][i] = 0.0f;
  for (uint32_t r0 = blockIdx.x * kGroups; r0 < p.rows; r0 += gridDim.x * kGroups) {
    const uint32_t row = r0 + threadIdx.x / L;
    const bool live = row < p.rows;
    const T* src = row_at<T>(p.x, p, live ? row : 0, p.x_ts, p.x_hs);
    const T* up = row_at<T>(p.dy, p, live ? row : 0, p.dy_ts, p.dy_hs);
    const float2 stat = live ? *reinterpret_cast<const float2*>(p.stats + 2 * static_cast<int64_t>(row)) : make_float2(0.0f, 0.0f);
    Pack<T, V> x[P], dy[P];
#pragma unroll
    for (int q = 0; q < P; ++q) {
      const int col = (q * L + lane) * V;
      if (live && col < p.dim) {
        x[q] = *reinterpret_cast<const Pack<T, V>*>(src + col);
        dy[q] = *reinterpret_cast<const Pack<T, V>*>(up + col);
      }
    }
    float sums[2] = {0.0f, 0.0f};  // of g and of g n
#pragma unroll
    for (int q = 0; q < P; ++q) {
      const int col = (q * L + lane) * V;
      if (live && col < p.dim) {
        float w[V];
        params_at<T, V>(p.weight, wide, col, w);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float n = (to_float(x[q].v[i]) - stat.x) * stat.y, d = to_float(dy[q].v[i]), g = d * w[i];
          sums[0] += g;
          sums[1] = fmaf(g, n, sums[1]);
          dw[q][i] = fmaf(d, n, dw[q][i]);
          db[q][i] += d;
        }
      }
    }
    if (p.out == nullptr) continue;
    group_sum<L, 2>(sums, scratch, turn);
    if (!live) continue;
    const float mean_g = sums[0] * p.inv_dim, mean_gn = sums[1] * p.inv_dim;
    T* dst = static_cast<T*>(p.out) + static_cast<int64_t>(row) * p.dim;
#pragma unroll
    for (int q = 0; q < P; ++q) {
      const int col = (q * L + lane) * V;
      if (col < p.dim) {
        float w[V];
        params_at<T, V>(p.weight, wide, col, w);
        Pack<T, V> y;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float n = (to_float(x[q].v[i]) - stat.x) * stat.y;
          y.v[i] = from_float<T>(stat.y * (fmaf(to_float(dy[q].v[i]), w[i], -mean_g) - n * mean_gn));
        }
        *reinterpret_cast<Pack<T, V>*>(dst + col) = y;
      }
    }
  }
  if (p.partial == nullptr) return;
  // the groups of a warp, then the warps (groups, where they are larger) one after the other
  constexpr int kJoin = L < 32 ? 32 : L;
#pragma unroll
  for (int d = 16; d >= L; d /= 2)
#pragma unroll
    for (int q = 0; q < P; ++q)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        dw[q][i] += __shfl_xor_sync(0xffffffffu, dw[q][i], d);
        db[q][i] += __shfl_xor_sync(0xffffffffu, db[q][i], d);
      }
  float* const part = p.partial + static_cast<int64_t>(blockIdx.x) * 2 * p.dim;
  constexpr int kRounds = kThreads / kJoin;
#pragma unroll 1
  for (int round = 0; round < kRounds; ++round) {
    if (static_cast<int>(threadIdx.x) / kJoin == round && static_cast<int>(threadIdx.x) % kJoin < L) {
#pragma unroll
      for (int q = 0; q < P; ++q) {
        const int col = (q * L + lane) * V;
        if (col < p.dim)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float a = dw[q][i], b = db[q][i];
            if (round > 0) a += joined[col + i], b += joined[p.dim + col + i];
            float* const to = round == kRounds - 1 ? part : joined;
            to[col + i] = a;
            to[p.dim + col + i] = b;
          }
      }
    }
    if (kRounds > 1) __syncthreads();
  }
}

// The gradient of any row, one a CTA.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_grad_long_kernel(const NormParams p) {
  __shared__ float scratch[2][2][kWarps];
  begin_after_prior_grids();
  const bool wide = p.params32 != 0;
  int turn = 0;
  for (uint32_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* src = row_at<T>(p.x, p, row, p.x_ts, p.x_hs);
    const T* up = row_at<T>(p.dy, p, row, p.dy_ts, p.dy_hs);
    const float2 stat = *reinterpret_cast<const float2*>(p.stats + 2 * static_cast<int64_t>(row));
    float sums[2] = {0.0f, 0.0f};
    for (int c = threadIdx.x; c < p.dim; c += kThreads) {
      const float n = (to_float(src[c]) - stat.x) * stat.y, g = to_float(up[c]) * param_at(p.weight, wide, c, T());
      sums[0] += g;
      sums[1] = fmaf(g, n, sums[1]);
    }
    group_sum<kThreads, 2>(sums, scratch, turn);
    const float mean_g = sums[0] * p.inv_dim, mean_gn = sums[1] * p.inv_dim;
    T* dst = static_cast<T*>(p.out) + static_cast<int64_t>(row) * p.dim;
    for (int c = threadIdx.x; c < p.dim; c += kThreads) {
      const float n = (to_float(src[c]) - stat.x) * stat.y;
      dst[c] = from_float<T>(stat.y * (fmaf(to_float(up[c]), param_at(p.weight, wide, c, T()), -mean_g) - n * mean_gn));
    }
  }
}

// Partial sums of the parameters' gradients by columns, for rows that no group holds: a thread owns a column of every
// parts-th row.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_columns_kernel(const NormParams p, const uint32_t parts) {
  begin_after_prior_grids();
  const uint32_t part = blockIdx.x % parts;
  const int c = static_cast<int>(blockIdx.x / parts) * kThreads + threadIdx.x;
  if (c >= p.dim) return;
  float dw = 0.0f, db = 0.0f;
  for (uint32_t row = part; row < p.rows; row += parts) {
    const float2 stat = *reinterpret_cast<const float2*>(p.stats + 2 * static_cast<int64_t>(row));
    const float d = to_float(row_at<T>(p.dy, p, row, p.dy_ts, p.dy_hs)[c]);
    dw = fmaf(d, (to_float(row_at<T>(p.x, p, row, p.x_ts, p.x_hs)[c]) - stat.x) * stat.y, dw);
    db += d;
  }
  p.partial[static_cast<int64_t>(part) * 2 * p.dim + c] = dw;
  p.partial[static_cast<int64_t>(part) * 2 * p.dim + p.dim + c] = db;
}

struct JoinParams {
  const float* partial;
  void* dw;
  void* db;
  uint32_t parts;
  int32_t dim, dtype;
};

// The sum of the parts, 32 columns a CTA, every 32nd part a thread.
__global__ void __launch_bounds__(1024) norm_join_kernel(const JoinParams p) {
  __shared__ float sums[32][33];
  begin_after_prior_grids();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane, all = 2 * static_cast<int64_t>(p.dim);
  float sum = 0.0f;
  if (c < all) {
#pragma unroll 8
    for (uint32_t k = warp; k < p.parts; k += 32) sum += p.partial[k * all + c];
  }
  sums[warp][lane] = sum;
  __syncthreads();
  sum = sums[lane][warp];
#pragma unroll
  for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  const int64_t mine = static_cast<int64_t>(blockIdx.x) * 32 + warp;
  if (lane != 0 || mine >= all) return;
  void* const to = mine < p.dim ? p.dw : p.db;
  const int64_t at = mine < p.dim ? mine : mine - p.dim;
  if (to == nullptr) return;
  if (p.dtype == INDEXER_BF16) static_cast<__nv_bfloat16*>(to)[at] = from_float<__nv_bfloat16>(sum);
  else if (p.dtype == INDEXER_FP16) static_cast<__half*>(to)[at] = from_float<__half>(sum);
  else static_cast<float*>(to)[at] = sum;
}

// CTAs of an SM for the gradients of rows of `held` values a lane: what its registers allow, for a second round of a few
// takes as long as the first (16384 rows of 1536: 40 us with two of an SM, 49 with four; 131071 rows of 128: 24.5 with
// four, 38 with two), and each leaves a row of partial sums.
constexpr int grad_ctas(int held) { return held <= 8 ? 4 : held <= 24 ? 2 : 1; }
constexpr int kGradCtas = grad_ctas(1);
constexpr int kMaxDim = 65536;

// How rows are split: groups of `lanes` with `pieces` pieces of V values each; 0 lanes: the long rows' kernels.
struct Split {
  int lanes, pieces;
  bool vec;
};

Split split_of(const NormParams& p, int32_t dtype, bool grad) {
  const int64_t size = static_cast<int64_t>(dtype_bytes(dtype)), v = 16 / size;
  uintptr_t all = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.out) |
                  reinterpret_cast<uintptr_t>(p.weight) | reinterpret_cast<uintptr_t>(p.bias);
  int64_t steps = p.dim | p.x_ts | p.x_hs;
  if (grad) all |= reinterpret_cast<uintptr_t>(p.dy), steps |= p.dy_ts | p.dy_hs;
  const bool vec = (all & 15u) == 0 && steps % v == 0;
  const int64_t n = vec ? p.dim / v : p.dim;
  if (!vec) return n <= 32 ? Split{32, 1, false} : n <= 128 ? Split{32, 4, false} : n <= 1024 ? Split{256, 4, false} : Split{0, 0, false};
  return n <= 8     ? Split{8, 1, true}
         : n <= 16  ? Split{16, 1, true}
         : n <= 32  ? Split{32, 1, true}
         : n <= 64  ? Split{32, 2, true}
         : n <= 128 ? Split{64, 2, true}
         : n <= 192 ? Split{64, 3, true}
         : n <= 256 ? Split{64, 4, true}
         : n <= 512 ? Split{256, 2, true}
         : n <= 1024 ? Split{256, 4, true}
                     : Split{0, 0, true};
}

template <typename T, int V, int L, int P>
cudaError_t launch_split(const NormParams& p, bool grad, unsigned grid, cudaStream_t stream) {
  if (!grad) return launch(norm_kernel<T, V, L, P>, grid, kThreads, 0, stream, p);
  const size_t smem = p.partial != nullptr && L < kThreads ? 8u * static_cast<size_t>(p.dim) : 0;
  return launch(norm_grad_kernel<T, V, L, P>, grid, kThreads, smem, stream, p);
}

template <typename T>
cudaError_t launch_rows(const NormParams& p, const Split& s, bool grad, unsigned grid, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  if (s.vec) {
    if (s.lanes == 8) return launch_split<T, V, 8, 1>(p, grad, grid, stream);
    if (s.lanes == 16) return launch_split<T, V, 16, 1>(p, grad, grid, stream);
    if (s.lanes == 32 && s.pieces == 1) return launch_split<T, V, 32, 1>(p, grad, grid, stream);
    if (s.lanes == 32) return launch_split<T, V, 32, 2>(p, grad, grid, stream);
    if (s.lanes == 64 && s.pieces == 2) return launch_split<T, V, 64, 2>(p, grad, grid, stream);
    if (s.lanes == 64 && s.pieces == 3) return launch_split<T, V, 64, 3>(p, grad, grid, stream);
    if (s.lanes == 64) return launch_split<T, V, 64, 4>(p, grad, grid, stream);
    if (s.pieces == 2) return launch_split<T, V, 256, 2>(p, grad, grid, stream);
    return launch_split<T, V, 256, 4>(p, grad, grid, stream);
  }
  if (s.lanes == 32 && s.pieces == 1) return launch_split<T, 1, 32, 1>(p, grad, grid, stream);
  if (s.lanes == 32) return launch_split<T, 1, 32, 4>(p, grad, grid, stream);
  return launch_split<T, 1, 256, 4>(p, grad, grid, stream);
}

// Partial sums of a call: CTAs of the gradient's kernel, or parts of the rows of the long rows' one.
int64_t parts_of(int64_t rows, int sms) { return std::min<int64_t>(rows, static_cast<int64_t>(sms) * kGradCtas); }

template <typename T>
cudaError_t run_rows(const NormParams& p, int32_t dtype, bool grad, int sms, cudaStream_t stream, uint32_t* parts) {
  const Split s = split_of(p, dtype, grad);
  const int64_t groups = s.lanes > 0 ? kThreads / s.lanes : 1;
  const int64_t blocks = (p.rows + groups - 1) / groups;
  const int held = s.pieces * (s.vec ? 16 / static_cast<int>(sizeof(T)) : 1);
  const unsigned most = static_cast<unsigned>(sms) * (grad ? grad_ctas(held) : 32);
  const unsigned grid = blocks < most ? static_cast<unsigned>(blocks) : most;
  if (s.lanes > 0) {
    *parts = grid;
    return launch_rows<T>(p, s, grad, grid, stream);
  }
  if (!grad) return launch(norm_long_kernel<T>, grid, kThreads, 0, stream, p);
  cudaError_t e = cudaSuccess;
  if (p.out != nullptr) e = launch(norm_grad_long_kernel<T>, grid, kThreads, 0, stream, p);
  if (e != cudaSuccess || p.partial == nullptr) return e;
  const int64_t columns = (p.dim + kThreads - 1) / kThreads;
  *parts = static_cast<uint32_t>(std::min<int64_t>(parts_of(p.rows, sms), (sms * 8 + columns - 1) / columns));
  return launch(norm_columns_kernel<T>, static_cast<unsigned>(columns * *parts), kThreads, 0, stream, p, *parts);
}

cudaError_t run_norm(const NormParams& p, int32_t dtype, bool grad, int sms, cudaStream_t stream, uint32_t* parts) {
  if (dtype == INDEXER_BF16) return run_rows<__nv_bfloat16>(p, dtype, grad, sms, stream, parts);
  if (dtype == INDEXER_FP16) return run_rows<__half>(p, dtype, grad, sms, stream, parts);
  return run_rows<float>(p, dtype, grad, sms, stream, parts);
}

bool aligned(const void* p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// What both calls have; rows a constant step apart need no division.
bool rows_ok(int32_t dtype, int32_t param_dtype, int64_t tokens, int32_t heads, int32_t dim, int64_t ts, int64_t hs) {
  return dtype >= INDEXER_BF16 && dtype <= INDEXER_FP32 && (param_dtype == dtype || param_dtype == INDEXER_FP32) &&
         tokens >= 0 && heads >= 0 && dim >= 1 && dim <= kMaxDim && ts >= 0 && hs >= 0 &&
         tokens <= INT32_MAX && (heads == 0 || tokens <= INT32_MAX / heads);
}

void place_rows(NormParams& p, int64_t tokens, int32_t heads, int64_t x_ts, int64_t x_hs, int64_t dy_ts, int64_t dy_hs) {
  p.x_ts = tokens > 1 ? x_ts : 0;
  p.x_hs = heads > 1 ? x_hs : 0;
  p.dy_ts = tokens > 1 ? dy_ts : 0;
  p.dy_hs = heads > 1 ? dy_hs : 0;
  p.rows = static_cast<uint32_t>(tokens * heads);
  p.heads = divisor(heads);
  const bool x_even = heads == 1 || tokens == 1 || p.x_ts == heads * p.x_hs;
  const bool dy_even = heads == 1 || tokens == 1 || p.dy_ts == heads * p.dy_hs;
  if (heads > 1 && x_even && dy_even) {
    p.x_ts = p.x_hs, p.dy_ts = p.dy_hs;
    p.x_hs = p.dy_hs = 0;
    p.heads = divisor(1);
  }
}

}  // namespace
}  // namespace indexer_gb300

extern "C" {

int indexer_layer_norm(const void* x, int64_t x_token_stride, int64_t x_head_stride, int32_t dtype, int64_t tokens,
                       int32_t heads, int32_t dim, const void* weight, const void* bias, int32_t param_dtype, float eps,
                       void* out, float* stats, cudaStream_t stream) {
  using namespace indexer_gb300;
  if (!rows_ok(dtype, param_dtype, tokens, heads, dim, x_token_stride, x_head_stride) || !(eps >= 0.0f) || eps > 3.4e38f)
    return TOPK_ERR_INVALID_ARGUMENT;
  if (tokens == 0 || heads == 0) return TOPK_OK;
  if (x == nullptr || weight == nullptr || out == nullptr || !aligned(x, dtype_bytes(dtype)) ||
      !aligned(out, dtype_bytes(dtype)) || !aligned(weight, dtype_bytes(param_dtype)) ||
      !aligned(bias, dtype_bytes(param_dtype)) || !aligned(stats, 8))
    return TOPK_ERR_INVALID_ARGUMENT;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return status_of(e);
  NormParams p = {};
  p.x = x;
  p.weight = weight;
  p.bias = bias;
  p.out = out;
  p.stats = stats;
  p.dim = dim;
  p.params32 = param_dtype == INDEXER_FP32;
  p.eps = eps;
  p.inv_dim = 1.0f / static_cast<float>(dim);
  place_rows(p, tokens, heads, x_token_stride, x_head_stride, 0, 0);
  uint32_t parts = 0;
  return status_of(run_norm(p, dtype, false, sms, stream, &parts));
}

size_t indexer_layer_norm_grad_workspace_bytes(int64_t tokens, int32_t heads, int32_t dim) {
  using namespace indexer_gb300;
  int sms = 0;
  if (!rows_ok(INDEXER_FP32, INDEXER_FP32, tokens, heads, dim, 0, 0) || sm_count(&sms) != cudaSuccess) return 0;
  return static_cast<size_t>(parts_of(tokens * heads, sms)) * 8u * static_cast<size_t>(dim);
}

int indexer_layer_norm_grad(const void* x, int64_t x_token_stride, int64_t x_head_stride, const void* grad,
                            int64_t grad_token_stride, int64_t grad_head_stride, int32_t dtype, int64_t tokens,
                            int32_t heads, int32_t dim, const void* weight, int32_t param_dtype, const float* stats,
                            void* grad_x, void* grad_weight, void* grad_bias, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream) {
  using namespace indexer_gb300;
  if (!rows_ok(dtype, param_dtype, tokens, heads, dim, x_token_stride, x_head_stride) || grad_token_stride < 0 ||
      grad_head_stride < 0)
    return TOPK_ERR_INVALID_ARGUMENT;
  const bool params = grad_weight != nullptr || grad_bias != nullptr;
  const int64_t rows = tokens * heads;
  const size_t size = dtype_bytes(dtype), param_size = dtype_bytes(param_dtype);
  if (!aligned(grad_weight, param_size) || !aligned(grad_bias, param_size)) return TOPK_ERR_INVALID_ARGUMENT;
  if (rows > 0 && (x == nullptr || grad == nullptr || weight == nullptr || stats == nullptr || !aligned(x, size) ||
                   !aligned(grad, size) || !aligned(grad_x, size) || !aligned(weight, param_size) || !aligned(stats, 8)))
    return TOPK_ERR_INVALID_ARGUMENT;
  if (!params && (rows == 0 || grad_x == nullptr)) return TOPK_OK;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return status_of(e);
  if (params && rows > 0) {
    if (workspace_bytes < static_cast<size_t>(parts_of(rows, sms)) * 8u * static_cast<size_t>(dim)) return TOPK_ERR_WORKSPACE_TOO_SMALL;
    if (workspace == nullptr || !aligned(workspace, 16)) return TOPK_ERR_INVALID_ARGUMENT;
  }
  uint32_t parts = 0;
  if (rows > 0) {
    NormParams p = {};
    p.x = x;
    p.dy = grad;
    p.weight = weight;
    p.out = grad_x;
    p.stats = const_cast<float*>(stats);
    p.partial = params ? static_cast<float*>(workspace) : nullptr;
    p.dim = dim;
    p.params32 = param_dtype == INDEXER_FP32;
    p.inv_dim = 1.0f / static_cast<float>(dim);
    place_rows(p, tokens, heads, x_token_stride, x_head_stride, grad_token_stride, grad_head_stride);
    e = run_norm(p, dtype, true, sms, stream, &parts);
    if (e != cudaSuccess || !params) return status_of(e);
  }
  JoinParams j = {static_cast<const float*>(workspace), grad_weight, grad_bias, parts, dim, param_dtype};
  return status_of(launch(norm_join_kernel, static_cast<unsigned>((2 * static_cast<int64_t>(dim) + 31) / 32), 1024, 0, stream, j));
}

}  // extern "C"
