// Rotary positions: pairs of columns turned by an angle of their own, position * frequency.
//
// Bound by memory: every element is read once and written once, with a few operations each.
// - The angle. position * frequency in radians loses the fraction of a turn for far positions in fp32 (2^20
//   positions leave 4 bits of it), and GB300 has almost no fp64 rate. A frequency's bits are therefore turned
//   into a 64-bit fixed-point fraction of a turn by one integer product, cut off at 2^-64; position * fraction
//   wraps modulo one turn by itself, without any rounding, and its top 32 bits are the angle: within 2^-31 of a
//   turn at any position, for frequencies of a few radians. Sine and cosine are taken of its 24 leading bits
//   past a quarter's multiple, 2^-28 of a turn at most: the step of an fp32 angle within a turn.
// - The split. A CTA owns a tile of tokens and heads. Its threads first leave the tile's sines and cosines in
//   shared memory, each computed once, then walk over the rows in pieces of 32 bytes (interleaved) or twice 16
//   (half layout; twice 32 needs too many registers). Many small CTAs hide the loads' latency better than
//   several pieces in flight in each thread (one piece and six CTAs an SM against two and five: 8192 x 64 x 128
//   in bf16, half of each row turned, 48 against 52 us). Sines kept in registers over a thread's heads took up to
//   232 registers and left the loads' latency bare (the same rows: 89 us).
// - A decode step (48 x 64 x 128: 3.0 us) is one chain: frequency and position behind the row's load, the
//   64-bit product, the series, shared memory, a barrier, the store. Columns that pass through are a second loop
//   behind that barrier (32768 rows of 192 in fp32, a third turned: 8.9 us where its bytes take 7.4).

#include "indexer_common.cuh"

namespace indexer_gb300 {
namespace {

constexpr int kThreads = 256;

// CTAs of an SM: what registers allow of pieces of 32 bytes, or of two accesses of 16 bytes each.
constexpr int resident(int bytes) { return bytes == 32 ? 5 : 6; }
constexpr int kMaxAngles = 2048;   // sines of a tile

struct RotaryParams {
  const void* x;
  void* out;
  const int32_t* positions;
  const double* freqs;
  int64_t x_ts, x_hs, out_ts, out_hs;
  Divisor pairs, turn_items, copy_items;  // pairs of a segment; a row's pieces that turn, and that are copied
  Divisor tile_heads, head_tiles, segments;
  int32_t tokens, heads, all_pairs, start, tile_tokens;
  float scale, sign;
};

// One position step as a fraction of a turn, in 2^-64 turns: the frequency's 53 bits times 2^66 / (2 pi).
__device__ __forceinline__ uint64_t turn_step(double freq) {
  constexpr uint64_t kPerTurn = 0xa2f9836e4e441529ull;  // floor(2^66 / (2 pi))
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(freq));
  const int field = static_cast<int>(bits >> 52) & 0x7ff;
  const uint64_t m = (bits & 0xfffffffffffffull) | (field != 0 ? 1ull << 52 : 0ull);
  const uint64_t high = __umul64hi(m, kPerTurn), low = m * kPerTurn;
  const int shift = 54 + 1023 - (field != 0 ? field : 1);  // to the right
  uint64_t r;
  if (shift >= 128) r = 0;
  else if (shift >= 64) r = high >> (shift - 64);
  else if (shift > 0) r = high << (64 - shift) | low >> shift;
  else r = shift > -64 ? low << -shift : 0;
  return bits >> 63 ? 0 - r : r;
}

// Sine and cosine of u * 2^-32 turns: an eighth of a turn to either side of a quarter's multiple, by the Taylor
// series (the first terms left out are below 2e-9 and 2e-10), then turned by the quarters.
__device__ __forceinline__ void sincos_turns(uint32_t u, float* sine, float* cosine) {
  const uint32_t quarters = (u + 0x20000000u) >> 30;
  constexpr float kRadians = 1.46291807926715968e-9f;  // 2 pi / 2^32
  const float x = static_cast<float>(static_cast<int32_t>(u - (quarters << 30))) * kRadians;
  const float y = x * x;
  float s = fmaf(y, 1.0f / 362880.0f, -1.0f / 5040.0f);
  s = fmaf(s, y, 1.0f / 120.0f);
  s = fmaf(s, y, -1.0f / 6.0f);
  s = fmaf(s * y, x, x);
  float c = fmaf(y, -1.0f / 3628800.0f, 1.0f / 40320.0f);
  c = fmaf(c, y, -1.0f / 720.0f);
  c = fmaf(c, y, 1.0f / 24.0f);
  c = fmaf(c, y, -0.5f);
  c = fmaf(c, y, 1.0f);
  const bool odd = (quarters & 1u) != 0;
  const float a = odd ? c : s, b = odd ? s : c;
  *sine = (quarters & 2u) != 0 ? -a : a;
  *cosine = ((quarters + 1u) & 2u) != 0 ? -b : b;
}

// V: values of one access. kHalf: the layout. A piece that turns is V pairs (half layout, two
// accesses) or V / 2 pairs (interleaved, one access; one pair and two accesses at V = 1).
template <typename T, int V, bool kHalf>
__global__ void __launch_bounds__(kThreads, resident(V * sizeof(T))) rotary_kernel(const RotaryParams p) {
  constexpr bool kTwo = kHalf || V == 1;
  constexpr int kPairs = kTwo ? V : V / 2;
  __shared__ __align__(16) float cosines[kMaxAngles], sines[kMaxAngles];
  begin_after_prior_grids();
  // this CTA's segment of pairs, tile of heads and tile of tokens
  const uint32_t block = quotient(p.segments, blockIdx.x), segment = blockIdx.x - block * p.segments.d;
  const uint32_t tile = quotient(p.head_tiles, block);
  const int h0 = static_cast<int>((block - tile * p.head_tiles.d) * p.tile_heads.d);
  const int t0 = static_cast<int>(tile) * p.tile_tokens;
  const uint32_t heads = min(static_cast<int>(p.tile_heads.d), p.heads - h0);
  const uint32_t tokens = min(p.tile_tokens, p.tokens - t0);
  const uint32_t first_pair = segment * p.pairs.d, pairs = min(p.pairs.d, p.all_pairs - first_pair);

  struct alignas(sizeof(T) * V) P {
    T v[V];
  };
  const T* const x = static_cast<const T*>(p.x) + t0 * p.x_ts + h0 * p.x_hs;
  T* const out = static_cast<T*>(p.out) + t0 * p.out_ts + h0 * p.out_hs;
  const uint32_t rows = tokens * heads;
  // row r of the tile: token t, and the head that is returned
  auto place = [&](uint32_t r, uint32_t* t) {
    *t = heads == p.tile_heads.d ? quotient(p.tile_heads, r) : r / heads;
    return r - *t * heads;
  };
  const uint32_t turning = rows * p.turn_items.d;
  P a, b;
  uint32_t angle = 0;
  T* dst = nullptr;
  auto load = [&](uint32_t u) {
    dst = nullptr;
    if (u >= turning) return;
    const uint32_t r = quotient(p.turn_items, u), first = (u - r * p.turn_items.d) * kPairs;
    if (first >= pairs) return;
    uint32_t t;
    const uint32_t h = place(r, &t);
    angle = t * p.pairs.d + first;
    const uint32_t col = p.start + (kHalf ? 1 : 2) * (first_pair + first);
    const T* src = x + t * p.x_ts + h * p.x_hs + col;
    dst = out + t * p.out_ts + h * p.out_hs + col;
    a = *reinterpret_cast<const P*>(src);
    if constexpr (kTwo) b = *reinterpret_cast<const P*>(src + (kHalf ? p.all_pairs : 1));
  };
  load(threadIdx.x);  // on its way while the angles are computed

  uint32_t last_pair = 0xffffffffu;
  uint64_t step = 0;
  for (uint32_t i = threadIdx.x; i < tokens * p.pairs.d; i += kThreads) {
    const uint32_t t = quotient(p.pairs, i), k = i - t * p.pairs.d;
    if (k >= pairs) continue;
    if (k != last_pair) step = turn_step(p.freqs[first_pair + k]);  // mostly one for all of a thread's tokens
    last_pair = k;
    const int64_t pos = p.positions[t0 + t];
    float s, c;
    sincos_turns(static_cast<uint32_t>(static_cast<uint64_t>(pos) * step >> 32), &s, &c);
    cosines[i] = c * p.scale;
    sines[i] = s * p.scale * p.sign;
  }
  __syncthreads();

  for (uint32_t u = threadIdx.x; u < turning; u += kThreads) {
    if (u != threadIdx.x) load(u);
    if (dst == nullptr) continue;
    float c[kPairs], s[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; i += kPairs % 4 == 0 ? 4 : 1) {
      if constexpr (kPairs % 4 == 0) {
        const float4 fc = *reinterpret_cast<const float4*>(&cosines[angle + i]);
        const float4 fs = *reinterpret_cast<const float4*>(&sines[angle + i]);
        c[i] = fc.x, c[i + 1] = fc.y, c[i + 2] = fc.z, c[i + 3] = fc.w;
        s[i] = fs.x, s[i + 1] = fs.y, s[i + 2] = fs.z, s[i + 3] = fs.w;
      } else {
        c[i] = cosines[angle + i];
        s[i] = sines[angle + i];
      }
    }
    P ya, yb;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const float fa = to_float(kTwo ? a.v[i] : a.v[2 * i]);
      const float fb = to_float(kTwo ? b.v[i] : a.v[2 * i + 1]);
      (kTwo ? ya.v[i] : ya.v[2 * i]) = from_float<T>(fmaf(fa, c[i], -fb * s[i]));
      (kTwo ? yb.v[i] : ya.v[2 * i + 1]) = from_float<T>(fmaf(fa, s[i], fb * c[i]));
    }
    *reinterpret_cast<P*>(dst) = ya;
    if constexpr (kTwo) *reinterpret_cast<P*>(dst + (kHalf ? p.all_pairs : 1)) = yb;
  }

  if (segment != 0) return;
  const uint32_t copying = rows * p.copy_items.d;
  for (uint32_t u = threadIdx.x; u < copying; u += kThreads) {
    const uint32_t r = quotient(p.copy_items, u);
    int col = static_cast<int>(u - r * p.copy_items.d) * V;
    if (col >= p.start) col += 2 * p.all_pairs;
    uint32_t t;
    const uint32_t h = place(r, &t);
    *reinterpret_cast<P*>(out + t * p.out_ts + h * p.out_hs + col) =
        *reinterpret_cast<const P*>(x + t * p.x_ts + h * p.x_hs + col);
  }
}

template <typename T>
cudaError_t launch_rotary(RotaryParams p, int64_t tokens, int32_t dim, bool half, bool in_place, int sms,
                          cudaStream_t stream) {
  // The widest accesses on whose boundaries every row starts, and the turned columns' parts: 32 bytes
  // (interleaved only: 8191 x 64 x 128 in bf16 44 us against 52 with 16 bytes), 16, 4 (two 16-bit values: 4096
  // x 7 x 130, 68 columns turned, half layout, 7.7 us against 10.4 with single ones), or single values.
  const int64_t all = p.x_ts | p.x_hs | p.out_ts | p.out_hs | dim | p.start | (half ? p.all_pairs : 2 * p.all_pairs);
  const uintptr_t bases = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.out);
  constexpr int kV = 16 / sizeof(T);
  const int v = !half && all % (2 * kV) == 0 && (bases & 31u) == 0 ? 2 * kV : all % kV == 0 && (bases & 15u) == 0 ? kV
                : sizeof(T) == 2 && all % 2 == 0 && (bases & 3u) == 0                     ? 2
                                                                                          : 1;
  const int pairs_of_item = half || v == 1 ? v : v / 2;
  const int64_t segments = (p.all_pairs + kMaxAngles - 1) / kMaxAngles;
  const int64_t pairs = segments > 1 ? kMaxAngles : p.all_pairs;
  const int64_t turn_items = pairs / pairs_of_item, copy_items = in_place ? 0 : (dim - 2 * p.all_pairs) / v;
  // A CTA owns all heads of some tokens, or a part of one token's heads: from one piece to about eight for each
  // thread, in whole rounds of the CTAs that the chip holds (a last round of a few CTAs takes as long as a full
  // one).
  const int64_t row = turn_items + copy_items, total = tokens * p.heads * row, slots = int64_t(sms) * resident(v * sizeof(T));
  const int64_t rounds = (total + slots * 8 * kThreads - 1) / (slots * 8 * kThreads);
  int64_t pieces = total / (slots * rounds);
  if (pieces < kThreads) pieces = kThreads;
  int64_t heads = pieces / row < 1 ? 1 : pieces / row < p.heads ? pieces / row : p.heads;
  const int64_t head_tiles = (p.heads + heads - 1) / heads;
  heads = (p.heads + head_tiles - 1) / head_tiles;
  int64_t tile_tokens = 1;
  if (heads == p.heads) {
    tile_tokens = (tokens + slots * rounds - 1) / (slots * rounds);
    if (tile_tokens * heads * row < kThreads) tile_tokens = kThreads / (heads * row);
  }
  if (tile_tokens > kMaxAngles / pairs) tile_tokens = kMaxAngles / pairs;
  if (tile_tokens < 1) tile_tokens = 1;
  p.tile_tokens = static_cast<int32_t>(tile_tokens);
  p.tile_heads = divisor(heads);
  p.head_tiles = divisor(head_tiles);
  p.segments = divisor(segments);
  p.pairs = divisor(pairs);
  p.turn_items = divisor(turn_items);
  p.copy_items = copy_items > 0 ? divisor(copy_items) : Divisor{0, 0, 0};
  p.tokens = static_cast<int32_t>(tokens);
  // more CTAs than a launch takes would need an output of more than the device's memory
  const int64_t blocks = (tokens + tile_tokens - 1) / tile_tokens * head_tiles * segments;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(blocks);
  if (v == 2 * kV) return launch(rotary_kernel<T, 2 * kV, false>, grid, kThreads, 0, stream, p);
  if (v == kV)
    return half ? launch(rotary_kernel<T, kV, true>, grid, kThreads, 0, stream, p)
                : launch(rotary_kernel<T, kV, false>, grid, kThreads, 0, stream, p);
  if constexpr (sizeof(T) == 2) {
    if (v == 2)
      return half ? launch(rotary_kernel<T, 2, true>, grid, kThreads, 0, stream, p)
                  : launch(rotary_kernel<T, 2, false>, grid, kThreads, 0, stream, p);
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
  if (((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out)) & low) != 0 ||
      (reinterpret_cast<uintptr_t>(positions) & 3u) != 0 || (reinterpret_cast<uintptr_t>(freqs) & 7u) != 0)
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
  p.all_pairs = rot_dim / 2;
  p.start = start;
  p.scale = scale;
  p.sign = transpose != 0 ? -1.0f : 1.0f;
  const bool half = layout == INDEXER_LAYOUT_HALF;
  const bool in_place = x == out && p.x_ts == p.out_ts && p.x_hs == p.out_hs;
  if (dtype == INDEXER_BF16) e = launch_rotary<__nv_bfloat16>(p, tokens, dim, half, in_place, sms, stream);
  else if (dtype == INDEXER_FP16) e = launch_rotary<__half>(p, tokens, dim, half, in_place, sms, stream);
  else e = launch_rotary<float>(p, tokens, dim, half, in_place, sms, stream);
  return status_of(e);
}
