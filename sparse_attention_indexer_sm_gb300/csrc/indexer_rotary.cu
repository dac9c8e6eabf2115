// Rotary positions: pairs of columns turned by an angle of their own, position * frequency.
//
// Bound by memory: every element is read once and written once, about 10 operations each.
// - The angle. position * frequency in radians loses the fraction of a turn for far
//   positions in fp32 (2^20 positions leave 4 bits of it), and GB300 has almost no fp64
//   rate. A frequency is therefore turned into a 64-bit fixed-point fraction of a turn,
//   once for each CTA (the only fp64 operations); position * fraction wraps modulo one turn
//   by itself, in integers and without any rounding, and its top 32 bits are the angle.
// - The split. A thread keeps the angles of one token's few pairs in registers and walks
//   over a group of heads with them, so that sine and cosine are computed once for the
//   group. Lanes cover a row's columns, so accesses are coalesced.

#include "indexer_common.cuh"

namespace indexer_gb300 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairsShared = 1024;  // pairs whose steps fit the shared array

struct RotaryParams {
  const void* x;
  void* out;
  const int32_t* positions;
  const double* freqs;
  int64_t x_ts, x_hs, out_ts, out_hs;
  int64_t units;     // tokens * head groups * items
  int32_t heads, dim, pairs, start;
  int32_t group, groups;  // heads of a group, groups
  int32_t items, rot_items;  // threads' shares of a row; the first rot_items of them rotate
  float scale, sign;
};

// One position step as a fraction of a turn, in 2^-64 turns.
__device__ __forceinline__ uint64_t turn_step(double freq) {
  double t = freq * 0.15915494309189533577;  // 1 / (2 pi)
  t -= floor(t);
  return static_cast<uint64_t>(t * 18446744073709551616.0);
}

// V: values of one access. kHalf: the layout. A rotating item is V pairs (half layout, two
// accesses) or V / 2 pairs (interleaved, one access; one pair and two accesses at V = 1).
template <typename T, int V, bool kHalf>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryParams p) {
  constexpr int kPairs = kHalf || V == 1 ? V : V / 2;
  __shared__ uint64_t steps[kMaxPairsShared];
  begin_after_prior_grids();
  const bool shared_steps = p.pairs <= kMaxPairsShared;
  if (shared_steps) {
    for (int i = threadIdx.x; i < p.pairs; i += kThreads) steps[i] = turn_step(p.freqs[i]);
    __syncthreads();
  }
  using P = Pack<T, V>;
  const T* x = static_cast<const T*>(p.x);
  T* out = static_cast<T*>(p.out);
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; u < p.units;
       u += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t row = u / p.items;
    const int item = static_cast<int>(u - row * p.items);
    const int64_t t = row / p.groups;
    const int h0 = static_cast<int>(row - t * p.groups) * p.group;
    const int h1 = min(h0 + p.group, p.heads);
    const T* src = x + t * p.x_ts + static_cast<int64_t>(h0) * p.x_hs;
    T* dst = out + t * p.out_ts + static_cast<int64_t>(h0) * p.out_hs;
    if (item >= p.rot_items) {
      int col = (item - p.rot_items) * V;
      if (col >= p.start) col += 2 * p.pairs;
      for (int h = h0; h < h1; ++h, src += p.x_hs, dst += p.out_hs)
        *reinterpret_cast<P*>(dst + col) = *reinterpret_cast<const P*>(src + col);
      continue;
    }
    const int first = item * kPairs;
    const int64_t pos = p.positions[t];
    float c[kPairs], s[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const uint64_t step = shared_steps ? steps[first + i] : turn_step(p.freqs[first + i]);
      const uint64_t phase = static_cast<uint64_t>(pos) * step;
      // top 32 bits, signed: half turns in [-1, 1)
      const float half_turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f;
      sincospif(half_turns, &s[i], &c[i]);
      c[i] *= p.scale;
      s[i] *= p.scale * p.sign;
    }
    if constexpr (kHalf || V == 1) {
      const int ca = p.start + (kHalf ? first : 2 * first);
      const int cb = ca + (kHalf ? p.pairs : 1);
#pragma unroll 4
      for (int h = h0; h < h1; ++h, src += p.x_hs, dst += p.out_hs) {
        const P a = *reinterpret_cast<const P*>(src + ca);
        const P b = *reinterpret_cast<const P*>(src + cb);
        P ya, yb;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float fa = to_float(a.v[i]), fb = to_float(b.v[i]);
          ya.v[i] = from_float<T>(fmaf(fa, c[i], -fb * s[i]));
          yb.v[i] = from_float<T>(fmaf(fa, s[i], fb * c[i]));
        }
        *reinterpret_cast<P*>(dst + ca) = ya;
        *reinterpret_cast<P*>(dst + cb) = yb;
      }
    } else {
      const int col = p.start + 2 * first;
#pragma unroll 4
      for (int h = h0; h < h1; ++h, src += p.x_hs, dst += p.out_hs) {
        const P a = *reinterpret_cast<const P*>(src + col);
        P y;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const float fa = to_float(a.v[2 * i]), fb = to_float(a.v[2 * i + 1]);
          y.v[2 * i] = from_float<T>(fmaf(fa, c[i], -fb * s[i]));
          y.v[2 * i + 1] = from_float<T>(fmaf(fa, s[i], fb * c[i]));
        }
        *reinterpret_cast<P*>(dst + col) = y;
      }
    }
  }
}

template <typename T>
cudaError_t launch_rotary(RotaryParams p, int64_t tokens, bool half, bool in_place, int sms,
                          cudaStream_t stream) {
  // 16-byte accesses where every row, and the pairs' two halves, start on 16 bytes
  constexpr int kV = 16 / sizeof(T);
  const int64_t all = p.x_ts | p.x_hs | p.out_ts | p.out_hs | p.dim | p.start | (half ? p.pairs : 2 * p.pairs);
  const bool wide = all % kV == 0 &&
                    ((reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.out)) & 15u) == 0;
  const int v = wide ? kV : 1;
  const int pairs_of_item = half || v == 1 ? v : v / 2;
  p.rot_items = p.pairs / pairs_of_item;
  p.items = p.rot_items + (in_place ? 0 : (p.dim - 2 * p.pairs) / v);
  // Heads of a group: eight share a sine, fewer where that leaves threads of the chip idle.
  p.group = 8;
  while (p.group > 1 && tokens * ((p.heads + p.group - 1) / p.group) * p.items < int64_t(sms) * 2048) p.group /= 2;
  p.groups = (p.heads + p.group - 1) / p.group;
  p.units = tokens * p.groups * p.items;
  const int64_t blocks = (p.units + kThreads - 1) / kThreads;
  const unsigned grid = static_cast<unsigned>(blocks < int64_t(sms) * 8 ? blocks : int64_t(sms) * 8);
  if (wide) {
    return half ? launch(rotary_kernel<T, kV, true>, grid, kThreads, 0, stream, p)
                : launch(rotary_kernel<T, kV, false>, grid, kThreads, 0, stream, p);
  }
  return half ? launch(rotary_kernel<T, 1, true>, grid, kThreads, 0, stream, p)
              : launch(rotary_kernel<T, 1, false>, grid, kThreads, 0, stream, p);
}

}  // namespace
}  // namespace indexer_gb300

extern "C" int indexer_rotary(const void* x, int64_t x_token_stride, int64_t x_head_stride,
                              const int32_t* positions, const double* freqs, int32_t dtype,
                              int64_t tokens, int32_t heads, int32_t dim, int32_t rot_dim,
                              int32_t start, int32_t layout, float scale, int32_t transpose,
                              void* out, int64_t out_token_stride, int64_t out_head_stride,
                              cudaStream_t stream) {
  using namespace indexer_gb300;
  if (dtype < INDEXER_BF16 || dtype > INDEXER_FP32 || layout < INDEXER_LAYOUT_HALF ||
      layout > INDEXER_LAYOUT_INTERLEAVED)
    return TOPK_ERR_INVALID_ARGUMENT;
  if (tokens < 0 || tokens > INT32_MAX || heads < 0 || dim < 2 || dim > 65536 || rot_dim < 2 ||
      rot_dim % 2 != 0 || start < 0 || start > dim || rot_dim > dim - start)
    return TOPK_ERR_INVALID_ARGUMENT;
  if (x_token_stride < 0 || x_head_stride < 0 || out_token_stride < 0 || out_head_stride < 0)
    return TOPK_ERR_INVALID_ARGUMENT;
  if (tokens == 0 || heads == 0) return TOPK_OK;
  if (x == nullptr || positions == nullptr || freqs == nullptr || out == nullptr)
    return TOPK_ERR_INVALID_ARGUMENT;
  // rows of out apart from each other: the axis of the smaller stride lies inside the other
  const int64_t ots = tokens > 1 ? out_token_stride : INT64_MAX;
  const int64_t ohs = heads > 1 ? out_head_stride : INT64_MAX;
  const int64_t inner = ots < ohs ? ots : ohs, outer = ots < ohs ? ohs : ots;
  const int64_t inner_n = ots < ohs ? tokens : heads;
  if (inner < dim || (outer != INT64_MAX && (outer - dim) / inner < inner_n - 1))
    return TOPK_ERR_INVALID_ARGUMENT;
  const uintptr_t low = static_cast<uintptr_t>(dtype_bytes(dtype)) - 1;
  if (((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out)) & low) != 0)
    return TOPK_ERR_INVALID_ARGUMENT;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return status_of(e);
  RotaryParams p = {};
  p.x = x;
  p.out = out;
  p.positions = positions;
  p.freqs = freqs;
  // strides of axes of one entry are never stepped over: they decide nothing
  p.x_ts = tokens > 1 ? x_token_stride : 0;
  p.x_hs = heads > 1 ? x_head_stride : 0;
  p.out_ts = tokens > 1 ? out_token_stride : 0;
  p.out_hs = heads > 1 ? out_head_stride : 0;
  p.heads = heads;
  p.dim = dim;
  p.pairs = rot_dim / 2;
  p.start = start;
  p.scale = scale;
  p.sign = transpose != 0 ? -1.0f : 1.0f;
  const bool half = layout == INDEXER_LAYOUT_HALF;
  const bool in_place = x == out && p.x_ts == p.out_ts && p.x_hs == p.out_hs;
  if (dtype == INDEXER_BF16) e = launch_rotary<__nv_bfloat16>(p, tokens, half, in_place, sms, stream);
  else if (dtype == INDEXER_FP16) e = launch_rotary<__half>(p, tokens, half, in_place, sms, stream);
  else e = launch_rotary<float>(p, tokens, half, in_place, sms, stream);
  return status_of(e);
}
