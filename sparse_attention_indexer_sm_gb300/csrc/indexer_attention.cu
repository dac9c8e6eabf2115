// Attention over a paged cache of e4m3 keys and values with one scale for each block of tokens and head:
//   out = sum_j p_j sv_j v_j / sum_j p_j,  p_j = exp(c sk_j q . k_j)
// in one pass over the keys, with the running maximum and sum of the softmax.
//
// - The values' scales. With t_j = log2 p_j + log2 sv_j a weight p_j sv_j is 2^(t_j - m) for a running bound m of the
//   t_j: one exponential for both sums, and the weights that are rounded to 16 bits for the products with the codes are
//   relative to the largest of them, whatever the scales are. The sum of p_j is that of 2^(t_j - m) / sv_j, in fp32.
// - The products run on the tensor cores in fp16 with fp32 sums. Codes are fp16 numbers. A query row is scaled by a power
//   of two that brings its largest value to [2^14, 2^15): of 16-bit values nothing is lost down to 2^-28 of the
//   largest, and no more than 2^-39 of it below. m follows the largest t_j only when that is kSlack above it, so weights
//   of up to 2^kSlack times 2^kShift stay below fp16's largest number, and none is rounded to zero above 2^-32 of the
//   largest: many small ones still count. Sums are rescaled once or twice a tile instead of at every new maximum.
// - Operands. Keys and columns of values are the rows of the products (16), query rows their columns (8 and more): a step
//   converts its codes once for all query rows, and few query rows leave little of the tensor cores unused. The order of
//   what a product sums over is free, and so is that of its rows and columns, as long as both operands agree. So a lane's
//   part of a row of the cache is 16 consecutive bytes, which become its operands' registers by conversions (and byte
//   permutes, for values) alone; the weights change lanes by two transposing moves.
// - Work. A tile is 8 or 16 query rows (queries of a sequence * heads that share a head of keys) of each of up to four
//   warps that share keys. The CTA's other warps lie along the keys, each (or each set on the same keys) with a ring of
//   stages of 16 keys and values, which cp.async fills some steps ahead and across the ends of tiles. CTAs
//   take equal spans of all the steps of all tiles, which each finds by adding up the lengths. A tile cut by a span's end
//   leaves its unscaled sums, bounds and sums of weights in the workspace; a second kernel joins these, in order.
// What bounds it: one query row, or a few, read the keys at 73% of the copy rate (64 sequences of up to 32768 keys of 8
// heads, 8 query heads on each, 1054085 keys and 2.16 GB in all: 435 us). From 9 rows on it is the instructions of a step, 1050 for 32 rows on 16
// keys, of which conversions of the codes and the products' operands are most: 256 rows of 2048 picks, 2 heads, 32 query
// heads on each (270 MB) take 135 us. Picked rows of 128 bytes arrive at 4.5 TB/s at best (a kernel of copies alone). The
// codes as e4m3 operands of the logits' products, with queries in parts, cost more than they save (134 -> 168 us).
// Heads of 64 columns, and of more than 128, take these tiles at any number of query rows, and are far from their floor with many: a
// prompt's chunk of 1024 queries behind 15360 keys, 8 heads, 4 query heads on each, 1171 us with 64 columns and 2741 with 256, for
// 70 and 281 us of products.

#include <algorithm>

#include "indexer_attention.cuh"

namespace indexer_gb300 {
namespace {

constexpr int kMaxCtas = 2;         // of an SM
constexpr int kStep = 16;           // keys of a warp's step

// Pages and slots outside the cache that were met (see indexer_guard_hits).
__device__ unsigned int g_guard_hits;

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The transpose of 8 x 8 values of 16 bits: a lane has two neighbours of row lane / 4.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

constexpr int kMaxShared = 226 * 1024;  // of an SM's CTAs, beside what is declared in the kernel

// How the columns of a head are laid out: kDim columns (the cache's and zeros).
template <int kDim> struct Shape {
  static constexpr int kChunks = kDim / 16;                  // 16-byte pieces of a row
  static constexpr int kTileBytes = kStep * kDim;            // of keys or values of a stage
  static constexpr int kStageBytes = 2 * kTileBytes + 8 * kStep + 16;  // and their scales, and which are there
  static constexpr int kOut = kDim / 16;                     // m-tiles of the result
  static constexpr int kRowsAtOnce = 32 / kChunks;           // rows that a warp copies at once
  // Where a piece lies in its tile. Eight lanes read at once: keys two rows * four pieces in a row, values four rows two
  // apart * two pieces; each eight fall on different banks.
  static __device__ __forceinline__ int place(int row, int chunk) {
    if constexpr (kDim == 64) return (row >> 1) * 128 + ((((row & 1) << 2) | chunk) ^ ((row >> 1 & 3) << 1)) * 16;
    else return row * kDim + (chunk ^ ((row & 6) ^ ((row & 1) << 2))) * 16;
  }
  // The column of value e (0, 1) of m-tile t that lane 4 g + c holds.
  static __device__ __forceinline__ int column(int t, int g, int e) {
    if constexpr (kDim == 64) return g * 8 + 2 * t + e;
    else return (t >> 3) * 128 + g * 16 + 2 * (t & 7) + e;
  }
};

// o += values * weights (of 16 keys). A lane reads 4 keys' pieces of 16 bytes (8 for 64 columns): pairs of neighbouring
// keys of two neighbouring columns are its operands. kScrub: NaN codes count as 0.
template <int kDim, int kTiles, bool kScrub>
__device__ __forceinline__ void weigh(float (&o)[kDim / 16][kTiles][4], const uint32_t (&weights)[kTiles][2], const uint8_t* values,
                                      int g, int c) {
  using S = Shape<kDim>;
  constexpr int kWords = kDim == 64 ? 2 : 4;
#pragma unroll
  for (int i = 0; i < (kDim + 127) / 128; ++i) {
    uint32_t v[4][kWords];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int row = (k >> 1) * 8 + 2 * c + (k & 1);
      if constexpr (kDim == 64) {
        const uint2 x = *reinterpret_cast<const uint2*>(values + S::place(row, g >> 1) + (g & 1) * 8);
        v[k][0] = x.x, v[k][1] = x.y;
      } else {
        const uint4 x = *reinterpret_cast<const uint4*>(values + S::place(row, 8 * i + g));
        v[k][0] = x.x, v[k][1] = x.y, v[k][2] = x.z, v[k][3] = x.w;
      }
      if constexpr (kScrub) {
#pragma unroll
        for (int w = 0; w < kWords; ++w) v[k][w] &= ~((nan_codes(v[k][w]) >> 7) * 0xffu);
      }
    }
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t lo = __byte_perm(v[0][w], v[1][w], h ? 0x7362 : 0x5140);
        const uint32_t hi = __byte_perm(v[2][w], v[3][w], h ? 0x7362 : 0x5140);
        const uint32_t a[4] = {halves_of(lo), halves_of(lo >> 16), halves_of(hi), halves_of(hi >> 16)};
#pragma unroll
        for (int t = 0; t < kTiles; ++t) mma(o[8 * i + 2 * w + h][t], a, weights[t][0], weights[t][1]);
      }
    }
  }
}

// What weigh left out of `bad` keys (of a step from position j0 on): a NaN code of a value makes its column NaN for the rows that see
// the key, and nothing else. columns: for each of the warp's rows, row0 on, a bit for each column, in shared memory, which the tile's
// end looks at. A call, as its registers would be spilled in the loop (64 sequences of up to 8192 keys of 8 heads of 256 columns, 16
// query heads on each: 307 us, 294 so).
template <int kDim, int kWarpRows>
__device__ __noinline__ void mark(const AttendParams& p, uint32_t* columns, uint32_t bad, const uint8_t* values, int32_t j0, int32_t list,
                                  int32_t row0) {
  using S = Shape<kDim>;
  const int lane = threadIdx.x & 31, chunk = lane % S::kChunks;  // a lane a piece of the key's row
  int32_t len = INT32_MAX;
  if (p.seq_lens != nullptr && lane < kWarpRows && row0 + lane < p.list_queries * static_cast<int32_t>(p.group.d))
    len = p.seq_lens[static_cast<int64_t>(list) * p.list_queries + quotient(p.group, row0 + lane)];
#pragma unroll 1
  for (; bad != 0u; bad &= bad - 1u) {
    const int key = __ffs(bad) - 1;
    const uint8_t* const codes = values + S::place(key, chunk);
    uint32_t bits = 0;
#pragma unroll 1
    for (int i = 0; i < 16; ++i)
      if ((codes[i] & 0x7fu) == 0x7fu) bits |= 1u << i;
#pragma unroll 1
    for (int r = 0; r < kWarpRows; ++r) {
      const int32_t seen = __shfl_sync(0xffffffffu, len, r);
      if (bits != 0u && lane < S::kChunks && j0 + key < seen) atomicOr(columns + r * (kDim / 32) + chunk / 2, bits << (chunk & 1) * 16);
    }
  }
}

// kTiles: tiles of 8 query rows of a warp. kRowWarps: warps that share keys.
template <int kDim, int kTiles, int kRowWarps> struct Layout {
  using S = Shape<kDim>;
  // Warps of an SM: what the registers allow. In two CTAs, of which one goes on while the other passes from one tile to the
  // next (256 x 2048 picks, 32 query heads on one of keys: 169 us in one CTA, 146 in two).
  static constexpr int kCtas = kDim <= 128 && kTiles == 2 && kRowWarps < 4 ? 2 : 1;
  static constexpr int kWarps = (kDim <= 128 ? 12 : 8) / kCtas;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kKeyWarps = kWarps / kRowWarps;
  static constexpr int kWarpRows = 8 * kTiles, kRows = kWarpRows * kRowWarps;
  static constexpr int kKeys = kStep * kKeyWarps;
  static constexpr int kSent = kRows * kDim <= 1024 ? 4 : kRows * kDim <= 2048 ? 2 : 1;  // warps whose sums are handed on at once
  static constexpr int kQueryBytes = kRows * kDim * 2;
  static constexpr int kFactorBytes = kRows * 4;
  static constexpr int kStatBytes = kWarps * kWarpRows * 8;
  static constexpr int kRowFloats = kDim + 4;                            // four rows two apart lie 8 banks from each other
  static constexpr int kSumBytes = kSent * kRows * kRowFloats * 4;
  static constexpr int kColumnBytes = kRows * kDim / 8;
  static constexpr int kRest = kQueryBytes + kFactorBytes + kStatBytes + kSumBytes + kColumnBytes;
  static constexpr int kFit = (kMaxShared / kCtas - kRest) / (kKeyWarps * S::kStageBytes);
  static constexpr int kStages = kFit > 12 ? 12 : kFit;
  static_assert(kStages >= 3, "stages ahead");
  static constexpr int kRing = kStages * S::kStageBytes;                 // of one group of warps
  static constexpr int kQuery = kKeyWarps * kRing;                       // then the queries' operands,
  static constexpr int kFactor = kQuery + kQueryBytes;                   // the factor of each row,
  static constexpr int kStats = kFactor + kFactorBytes;                  // bound and sum of each row and warp,
  static constexpr int kSums = kStats + kStatBytes;                      // warps' sums,
  static constexpr int kColumns = kSums + kSumBytes;                     // and each row's columns that are NaN
  static constexpr int kBytes = kColumns + kColumnBytes;
  static constexpr int64_t kPartial = kRows * (kDim + 2);                // floats of a piece in the workspace
};

template <int kDim, int kTiles, int kRowWarps>
__global__ void __launch_bounds__(Layout<kDim, kTiles, kRowWarps>::kThreads, Layout<kDim, kTiles, kRowWarps>::kCtas) attend_kernel(const __grid_constant__ AttendParams p) {
  using S = Shape<kDim>;
  using L = Layout<kDim, kTiles, kRowWarps>;
  constexpr int kStages = L::kStages, kThreads = L::kThreads, kWarps = L::kWarps;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Spans span;
  __shared__ int64_t sums[kWarps];
  const float none = __uint_as_float(0xff800000u);
  // columns that the cache does not have are zeros, which no copy touches
  if (p.dim < kDim)
    for (int i = threadIdx.x; i < L::kQuery / 16; i += kThreads) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
  for (int i = threadIdx.x; i < L::kColumnBytes / 4; i += kThreads) reinterpret_cast<uint32_t*>(smem + L::kColumns)[i] = 0u;
  begin_after_prior_grids();
  find_span<L::kRows, L::kKeys>(p, sums, span);
  if (threadIdx.x == 0) p.cuts[blockIdx.x] = Cut{span.total, 0, 0, 0, 0};
  if (span.at[0] >= span.at[1]) return;

  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, g = lane >> 2, c = lane & 3;
  const int mw = warp % kRowWarps, kw = warp / kRowWarps;
  uint8_t* const ring = smem + kw * L::kRing;
  float* const factors = reinterpret_cast<float*>(smem + L::kFactor);
  float2* const stats = reinterpret_cast<float2*>(smem + L::kStats);
  const int32_t group = static_cast<int32_t>(p.group.d), rows_of_list = p.list_queries * group;
  const bool listed = p.seq_lens == nullptr;

  auto group_barrier = [&]() {
    if constexpr (kRowWarps == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(kw + 1), "n"(32 * kRowWarps) : "memory");
  };
  auto enter = [&](Cursor& k) {  // a slice
    k.list = k.slice / p.tiles;
    k.longest = listed ? p.row_len : max(__reduce_max_sync(0xffffffffu, longest_of(p, k.slice, L::kRows, lane, 32)), 0);
    k.steps = steps_of(k.longest, L::kKeys);
  };
  auto advance = [&](Cursor& k, int32_t n) {  // n steps of this tile and head; true where it ends
    k.left -= n;
    k.step += n;
    if (k.step < k.steps || k.left <= 0) return false;
    k.step = 0;
    if (++k.head == p.kv_heads) {
      k.head = 0;
      ++k.slice;
      enter(k);
    }
    return true;
  };
  Cursor use;
  use.left = span.at[1] - span.at[0];
  use.slice = span.slice[0];
  enter(use);
  use.head = static_cast<int32_t>(span.rest[0] / use.steps);
  use.step = static_cast<int32_t>(span.rest[0] - static_cast<int64_t>(use.head) * use.steps);
  Cursor ask = use;

  // ---- copies: keys and values by a warp, or by one of a pair each; scales by the first one, a lane each
  const int copy_row = lane / S::kChunks, copy_chunk = lane % S::kChunks;
  const bool copy_in = copy_chunk * 16 < p.dim;
  const uint32_t ring_addr = smem_addr(ring);
  const Side& scale_side = p.side[lane >> 4];
  const uint32_t scale_ps = scale_side.scale_ps, scale_bs = scale_side.scale_bs;
  const Divisor block = scale_side.block;
  const uint8_t* bases[2];   // this lane's part of the first rows of the head; where each key has a page of its own, its row's
  const float* scales_base;  // likewise
  const int32_t* entries;    // the list
  auto set_bases = [&]() {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const Side& side = p.side[p.whole_steps ? s : kRowWarps > 1 ? mw & 1 : lane >> 4];
      bases[s] = side.codes + ask.head * side.code_hs;
      if (p.whole_steps) bases[s] += 16 * (static_cast<uint64_t>(copy_row) * side.code_ts + copy_chunk);
    }
    scales_base = scale_side.scales + ask.head * scale_side.scale_hs;
    entries = p.index + static_cast<int64_t>(ask.list) * p.index_stride;
  };
  // Pages of the next 32 steps, one a lane; or, where the keys of a step have pages of their own, of the next step.
  int32_t ids = -1;
  int ids_used = 0;
  auto look_up = [&]() {
    ids = -1;
    ids_used = 0;
    if (ask.left <= 0) return;
    if (p.whole_steps) {
      const int64_t j = (static_cast<int64_t>(ask.step) + lane) * L::kKeys + kw * kStep;
      if (j < ask.longest) ids = entries[quotient(p.page_size, static_cast<uint32_t>(j))];
    } else {
      const int32_t j = ask.step * L::kKeys + kw * kStep + (lane & 15);
      if (j < ask.longest) ids = entries[listed ? j : static_cast<int32_t>(quotient(p.page_size, j))];
    }
  };
  auto send = [&](int stage) {
    if (ask.left > 0) {
      const int32_t j0 = ask.step * L::kKeys + kw * kStep;
      const uint32_t at = ring_addr + stage * S::kStageBytes;
      uint32_t present, page, off;
      if (p.whole_steps) {
        if (ids_used == 32) look_up();
        page = __shfl_sync(0xffffffffu, ids, ids_used++);
        const bool there = page < static_cast<uint32_t>(p.num_pages);
        const int32_t n = min(ask.longest - j0, kStep);
        present = there && n > 0 ? (1u << n) - 1u : 0u;
        off = j0 - quotient(p.page_size, j0) * p.page_size.d;
        if (present != 0u) {
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (kRowWarps > 1 && s != mw) continue;
            const uint32_t ts = p.side[s].code_ts;
            const uint8_t* from = bases[s] + 16 * (static_cast<uint64_t>(page) * p.side[s].code_ps + static_cast<uint64_t>(off) * ts);
            const uint64_t step = static_cast<uint64_t>(ts) * (16 * S::kRowsAtOnce);
#pragma unroll
            for (int row = 0; row < kStep; row += S::kRowsAtOnce, from += step)
              if (copy_in) copy16(at + s * S::kTileBytes + S::place(row + copy_row, copy_chunk), from);
          }
          off += lane & 15;
        } else if (n > 0 && mw == 0 && lane == 0) {
          atomicAdd(&g_guard_hits, 1u);
        }
      } else {
        const int32_t j = j0 + (lane & 15);
        const bool asked = j < ask.longest;
        const bool there = asked && static_cast<int64_t>(static_cast<uint32_t>(ids)) < (listed ? p.capacity : p.num_pages);
        if (asked && !there && lane < 16 && mw == 0 && (!listed || ids != -1)) atomicAdd(&g_guard_hits, 1u);
        const uint32_t of = listed ? (there ? ids : 0) : (there ? j : 0), entry = quotient(p.page_size, of);
        page = listed ? entry : there ? ids : 0;
        off = of - entry * p.page_size.d;
        present = __ballot_sync(0xffffffffu, there) & 0xffffu;
        if (present != 0u) {  // keys that are not there take a row that is, which is not looked at
          const Side& side = p.side[kRowWarps > 1 ? mw & 1 : lane >> 4];
          const unsigned long long mine = reinterpret_cast<unsigned long long>(
              bases[0] + 16 * (static_cast<uint64_t>(page) * side.code_ps + static_cast<uint64_t>(off) * side.code_ts));
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (kRowWarps > 1 && s != mw) continue;
#pragma unroll
            for (int row = 0; row < kStep; row += S::kRowsAtOnce) {
              const unsigned long long from = __shfl_sync(0xffffffffu, mine, row + copy_row + (kRowWarps > 1 ? 0 : 16 * s));
              if (copy_in)
                copy16(at + s * S::kTileBytes + S::place(row + copy_row, copy_chunk), reinterpret_cast<const uint8_t*>(from) + copy_chunk * 16);
            }
          }
        }
      }
      if (mw == 0) {
        if (present != 0u)
          copy4(at + 2 * S::kTileBytes + 4 * lane,
                scales_base + (static_cast<uint64_t>(page) * scale_ps + static_cast<uint64_t>(quotient(block, off)) * scale_bs));
        if (lane == 0) *reinterpret_cast<uint32_t*>(ring + stage * S::kStageBytes + 2 * S::kTileBytes + 8 * kStep) = present;
      }
      const bool ended = advance(ask, 1);
      if (ended) set_bases();
      if (ended || !p.whole_steps) look_up();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  set_bases();
  look_up();
  for (int k = 0; k < kStages - 1; ++k) send(k);

  int stage = 0;
  while (use.left > 0) {
    const int32_t r0 = (use.slice - use.list * p.tiles) * L::kRows;
    const int32_t n_steps = static_cast<int32_t>(min(static_cast<int64_t>(use.steps - use.step), use.left));
    const bool from_start = use.step == 0, to_end = use.step + n_steps == use.steps;
    const int64_t first_query = static_cast<int64_t>(use.list) * p.list_queries;
    // row r of the list: its number among all rows of q
    auto row_at = [&](int32_t r) {
      const int32_t n = quotient(p.group, r);
      return (first_query + n) * p.heads + use.head * group + (r - n * group);
    };
    // ---- the queries as operands, a warp a row; all of a warp's rows are asked for at once
    constexpr int kPer = (L::kRows + kWarps - 1) / kWarps;
    uint32_t got[kPer][kDim / 64];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = warp + i * kWarps;
      const bool in = r < L::kRows && r0 + r < rows_of_list;
      const uint32_t* const src = static_cast<const uint32_t*>(p.q) + (in ? row_at(r0 + r) : 0) * (p.dim / 2);
#pragma unroll
      for (int k = 0; k < kDim / 64; ++k) got[i][k] = in && 2 * (k * 32 + lane) < p.dim ? src[k * 32 + lane] : 0u;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = warp + i * kWarps;
      if (r >= L::kRows) break;
      float2 v[kDim / 64];
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < kDim / 64; ++k) {
        if (p.fp16) {
          __half2 h;
          memcpy(&h, &got[i][k], 4);
          v[k] = __half22float2(h);
        } else {
          v[k] = make_float2(__uint_as_float(got[i][k] << 16), __uint_as_float(got[i][k] & 0xffff0000u));
        }
        top = max(top, max(__float_as_uint(v[k].x) & 0x7fffffffu, __float_as_uint(v[k].y) & 0x7fffffffu));
      }
      top = __reduce_max_sync(0xffffffffu, top);
      // 2^e the largest value's power: 2^(14 - e) in fp32 for e from -112 on
      const int e = max(static_cast<int>(top >> 23) - 127, -112);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - min(e, 127)) << 23);
      const float down = __uint_as_float(static_cast<uint32_t>(max(e - 14 + 127, 1)) << 23);
      if (lane == 0) factors[r] = top >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : p.scale * down;
      uint32_t* const to = reinterpret_cast<uint32_t*>(smem + L::kQuery);
#pragma unroll
      for (int k = 0; k < kDim / 64; ++k) {
        const int d = k * 64 + 2 * lane;  // column d: piece d / 16 = 4 i + c, byte 4 w + 2 h of it; product 4 i + w, register h
        const int s = (d >> 6) * 4 + (d >> 2 & 3), at = (r & 7) * 4 + (d >> 4 & 3), reg = (s & 1) * 2 + (d >> 1 & 1);
        const __half2 h = __floats2half2_rn(v[k].x * up, v[k].y * up);
        uint32_t word;
        memcpy(&word, &h, 4);
        to[(((s >> 1) * (kTiles * kRowWarps) + (r >> 3)) * 32 + at) * 4 + reg] = word;
      }
    }
    __syncthreads();

    // this lane's rows: 2 c and 2 c + 1 of each of its warp's tiles
    float factor[kTiles][2], bound[kTiles][2], sum[kTiles][2];
    int32_t len[kTiles][2], shortest = INT32_MAX;
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int32_t r = mw * L::kWarpRows + t * 8 + 2 * c + e;
        factor[t][e] = factors[r];
        bound[t][e] = none;
        sum[t][e] = 0.0f;
        // rows behind the last one are not written: they may see everything
        len[t][e] = listed || r0 + r >= rows_of_list ? INT32_MAX : p.seq_lens[first_query + quotient(p.group, r0 + r)];
        shortest = min(shortest, len[t][e]);
      }
    shortest = __reduce_min_sync(0xffffffffu, shortest);
    float o[S::kOut][kTiles][4];
#pragma unroll
    for (int t = 0; t < S::kOut; ++t)
#pragma unroll
      for (int n = 0; n < kTiles; ++n) o[t][n][0] = o[t][n][1] = o[t][n][2] = o[t][n][3] = 0.0f;
    const uint4* const query = reinterpret_cast<const uint4*>(smem + L::kQuery) + mw * kTiles * 32 + lane;

    for (int32_t n = 0; n < n_steps; ++n) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      group_barrier();
      send(stage == 0 ? kStages - 1 : stage - 1);  // its last contents were read to their end before the barrier
      const uint8_t* const at = ring + stage * S::kStageBytes;
      stage = stage + 1 == kStages ? 0 : stage + 1;
      const int32_t j0 = (use.step + n) * L::kKeys + kw * kStep;
      // ---- keys . queries
      float s[kTiles][4];
#pragma unroll
      for (int t = 0; t < kTiles; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.0f;
#pragma unroll
      for (int i = 0; i < kDim / 64; ++i) {
        const uint4 ka = *reinterpret_cast<const uint4*>(at + S::place(g, 4 * i + c));
        const uint4 kb = *reinterpret_cast<const uint4*>(at + S::place(g + 8, 4 * i + c));
        const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
        for (int w = 0; w < 4; w += 2) {
          const uint32_t a0[4] = {halves_of(wa[w]), halves_of(wb[w]), halves_of(wa[w] >> 16), halves_of(wb[w] >> 16)};
          const uint32_t a1[4] = {halves_of(wa[w + 1]), halves_of(wb[w + 1]), halves_of(wa[w + 1] >> 16), halves_of(wb[w + 1] >> 16)};
#pragma unroll
          for (int t = 0; t < kTiles; ++t) {
            const uint4 b = query[((2 * i + w / 2) * (kTiles * kRowWarps) + t) * 32];
            mma(s[t], a0, b.x, b.y);
            mma(s[t], a1, b.z, b.w);
          }
        }
      }
      // ---- logits (in log2) with the values' scales, of keys g and g + 8
      const float* const scales = reinterpret_cast<const float*>(at + 2 * S::kTileBytes);
      const uint8_t* const values = at + S::kTileBytes;
      const uint32_t present = *reinterpret_cast<const uint32_t*>(scales + 2 * kStep);
      const bool whole = present == 0xffffu && j0 + kStep <= shortest;
      float more[2], inverse[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float sk = scales[g + 8 * h], sv = max_or_nan(scales[kStep + g + 8 * h], 0x1p-100f);  // no logarithm of zero
        more[h] = log2_fast(sv);
        inverse[h] = inverse_fast(sv);
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) s[t][2 * h + e] = fmaf(s[t][2 * h + e], sk * factor[t][e], more[h]);
      }
      uint32_t bad = 0;
      if (!whole) {
        // Where some rows see a key and others do not, a NaN among its value's codes would reach all of them through a
        // weight of 0: there it counts as 0, and the rows that see it are marked.
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          bool found = false;
          const int row = (k >> 1) * 8 + 2 * c + (k & 1);
          for (int piece = g; piece < S::kChunks; piece += 8) {
            const uint4 v = *reinterpret_cast<const uint4*>(values + S::place(row, piece));
            found = found || ((nan_codes(v.x) | nan_codes(v.y) | nan_codes(v.z) | nan_codes(v.w)) != 0u);
          }
          const uint32_t lanes = __ballot_sync(0xffffffffu, found);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if ((lanes & (0x11111111u << q)) != 0u) bad |= 1u << ((k >> 1) * 8 + 2 * q + (k & 1));
        }
        bad |= (bad & present) << 16;  // above: those that some row may see
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = g + 8 * h;
          const bool there = (present >> key & 1u) != 0u;
#pragma unroll
          for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!there || j0 + key >= len[t][e]) s[t][2 * h + e] = none;
        }
      }
      // ---- weights
      bool above = false;
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) above = above || fmaxf(s[t][e], s[t][2 + e]) > bound[t][e] + kSlack;
      if (__any_sync(0xffffffffu, above)) {
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = fmaxf(s[t][e], s[t][2 + e]);
#pragma unroll
            for (int d = 4; d < 32; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float now = fmaxf(bound[t][e], top), f = now == none ? 1.0f : exp2_fast(bound[t][e] - now);
            bound[t][e] = now;
            sum[t][e] *= f;
#pragma unroll
            for (int m = 0; m < S::kOut; ++m) o[m][t][e] *= f, o[m][t][2 + e] *= f;
          }
      }
      uint32_t weights[kTiles][2];
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float base = bound[t][e] == none ? 0.0f : bound[t][e] - kShift;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            w[2 * h + e] = exp2_fast(s[t][2 * h + e] - base);
            // a hidden key's scale may be anything
            if (whole || s[t][2 * h + e] != none) sum[t][e] = fmaf(w[2 * h + e], inverse[h], sum[t][e]);
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const __half2 two = __floats2half2_rn(w[2 * h], w[2 * h + 1]);
          uint32_t word;
          memcpy(&word, &two, 4);
          weights[t][h] = transposed(word);
        }
      }
      // ---- values . weights
      if (bad != 0u) {
        weigh<kDim, kTiles, true>(o, weights, values, g, c);
        mark<kDim, L::kWarpRows>(p, reinterpret_cast<uint32_t*>(smem + L::kColumns) + mw * L::kWarpRows * (kDim / 32), bad >> 16, values, j0,
                                 use.list, r0 + mw * L::kWarpRows);
      } else {
        weigh<kDim, kTiles, false>(o, weights, values, g, c);
      }
    }

    // ---- the end of the tile, or of the span: the warps along the keys, joined in a fixed order
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d *= 2) sum[t][e] += __shfl_xor_sync(0xffffffffu, sum[t][e], d);
        if (g == 0) stats[warp * L::kWarpRows + t * 8 + 2 * c + e] = make_float2(bound[t][e], sum[t][e]);
      }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2* const row = stats + mw * L::kWarpRows + t * 8 + 2 * c + e;
        float top = none, total = 0.0f;
        for (int k = 0; k < L::kKeyWarps; ++k) top = fmaxf(top, row[k * L::kRows].x);
        for (int k = 0; k < L::kKeyWarps; ++k) {
          const float2 part = row[k * L::kRows];
          // a warp whose keys are all hidden from a row has no bound; its sum is 0, or NaN
          total += part.x == none ? part.y : part.y * exp2_fast(part.x - top);
        }
        const float f = bound[t][e] == none ? 1.0f : exp2_fast(bound[t][e] - top);
#pragma unroll
        for (int m = 0; m < S::kOut; ++m) o[m][t][e] *= f, o[m][t][2 + e] *= f;
        bound[t][e] = top;
        sum[t][e] = total;
      }
    float* const mine = reinterpret_cast<float*>(smem + L::kSums) + (mw * L::kWarpRows + 2 * c) * L::kRowFloats + 2 * g;
#pragma unroll 1
    for (int rest = L::kKeyWarps; rest > 1;) {  // the last ones hand their sums to those before them
      const int sent = min(rest / 2, L::kSent);
      if (kw >= rest - sent && kw < rest) {
        float* const to = mine + (kw - (rest - sent)) * L::kRows * L::kRowFloats;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int m = 0; m < S::kOut; ++m)
              *reinterpret_cast<float2*>(to + (t * 8 + e) * L::kRowFloats + m * 16) = make_float2(o[m][t][e], o[m][t][2 + e]);
      }
      __syncthreads();
      if (kw >= rest - 2 * sent && kw < rest - sent) {
        const float* const from = mine + (kw - (rest - 2 * sent)) * L::kRows * L::kRowFloats;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int m = 0; m < S::kOut; ++m) {
              const float2 v = *reinterpret_cast<const float2*>(from + (t * 8 + e) * L::kRowFloats + m * 16);
              o[m][t][e] += v.x;
              o[m][t][2 + e] += v.y;
            }
      }
      rest -= sent;
      if (rest > 1) __syncthreads();
    }
    if (kw == 0) {
      uint32_t* const columns = reinterpret_cast<uint32_t*>(smem + L::kColumns) + mw * L::kWarpRows * (kDim / 32);
      uint32_t spoiled[kTiles][2][(kDim + 127) / 128], any = 0;  // of this lane's columns: neighbouring bits
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < (kDim + 127) / 128; ++i) {
            const int col = S::column(8 * i, g, 0);
            spoiled[t][e][i] = columns[(t * 8 + 2 * c + e) * (kDim / 32) + col / 32] >> (col % 32);
            any |= spoiled[t][e][i];
          }
      if (__any_sync(0xffffffffu, any != 0u)) {
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int m = 0; m < S::kOut; ++m) {
              const uint32_t two = spoiled[t][e][m / 8] >> (2 * (m % 8));
              if ((two & 1u) != 0u) o[m][t][e] = __uint_as_float(0x7fffffffu);
              if ((two & 2u) != 0u) o[m][t][2 + e] = __uint_as_float(0x7fffffffu);
            }
        for (int i = lane; i < L::kWarpRows * (kDim / 32); i += 32) columns[i] = 0u;  // (all of the warp have read theirs)
      }
      if (from_start && to_end) {
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int32_t r = r0 + mw * L::kWarpRows + t * 8 + 2 * c + e;
            if (r >= rows_of_list) continue;
            const int64_t row = row_at(r);
            const float f = sum[t][e] == 0.0f ? 0.0f : 1.0f / sum[t][e];
            if (p.lse != nullptr && g == 0) p.lse[row] = log_sum(bound[t][e], sum[t][e]);
#pragma unroll
            for (int m = 0; m < S::kOut; ++m) {
              const int col = S::column(m, g, 0);
              if (col < p.dim) store_pair(p.out, row * p.dim + col, p.fp16 != 0, o[m][t][e] * f, o[m][t][2 + e] * f);
            }
          }
      } else {
        // the piece without its tile's start is a span's first, the one with it (and without the end) its last
        float* const piece = p.partial + (2 * static_cast<int64_t>(blockIdx.x) + (from_start ? 1 : 0)) * L::kPartial;
        if (from_start && threadIdx.x == 0) {
          // the last span that has steps of this tile
          const int64_t end = span.at[1] - n_steps + use.steps, spans = gridDim.x;
          const int64_t last = min((end * spans + span.total - 1) / span.total - 1, spans - 1);
          p.cuts[blockIdx.x] = Cut{span.total, use.slice, use.head, static_cast<int32_t>(last), 1};
        }
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = mw * L::kWarpRows + t * 8 + 2 * c + e;
            if (g == 0) *reinterpret_cast<float2*>(piece + L::kRows * kDim + 2 * r) = make_float2(bound[t][e], sum[t][e]);
#pragma unroll
            for (int m = 0; m < S::kOut; ++m)
              *reinterpret_cast<float2*>(piece + r * kDim + m * 16 + 2 * g) = make_float2(o[m][t][e], o[m][t][2 + e]);
          }
      }
    }
    advance(use, n_steps);
    __syncthreads();
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Columns of a row's sums as a tile's warps leave them: m-tiles of 16, in them pairs of lanes 4 g + c.
template <int kDim> struct Held {
  static __device__ __forceinline__ int column(int at) { return Shape<kDim>::column(at / 16, at / 2 % 8, at % 2); }
};

template <int kDim, int kTiles, int kRowWarps>
cudaError_t launch_attention(AttendParams p, int sms, cudaStream_t stream) {
  using L = Layout<kDim, kTiles, kRowWarps>;
  const int64_t tiles = (static_cast<int64_t>(p.list_queries) * p.group.d + L::kRows - 1) / L::kRows;
  if (tiles * p.lists > INT32_MAX / 2) return cudaErrorInvalidValue;
  p.tiles = static_cast<int32_t>(tiles);
  p.slices = static_cast<int32_t>(tiles * p.lists);
  // no more spans than there can be steps
  const int64_t most = static_cast<int64_t>(p.slices) * p.kv_heads * ((static_cast<int64_t>(p.row_len) + L::kKeys) / L::kKeys);
  const int spans = static_cast<int>(std::min<int64_t>(sms * L::kCtas, most));
  static thread_local int known = -1;  // the device whose kernel may use so much shared memory
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess && known != device) {
    e = cudaFuncSetAttribute(attend_kernel<kDim, kTiles, kRowWarps>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
    if (e == cudaSuccess) known = device;
  }
  if (e == cudaSuccess) e = launch(attend_kernel<kDim, kTiles, kRowWarps>, spans, L::kThreads, L::kBytes, stream, p);
  if (e != cudaSuccess || spans == 1) return e;
  return launch_join<kDim, Held<kDim>>(p, spans, L::kRows, stream);
}

int padded_dim(int32_t dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

// The tile for so many rows that share keys: 8 or 16 of a warp, in as many warps as hold them: at most four, of more than
// 64 columns two (of 128 the wide tiles take what is above that).
struct Tile {
  int tiles, row_warps;
  int rows() const { return 8 * tiles * row_warps; }
};

Tile tile_of(int64_t rows, int dim) {
  if (rows <= 8) return Tile{1, 1};
  return Tile{2, static_cast<int>(std::min<int64_t>((rows + 15) / 16, dim == 64 ? 4 : 2))};
}

template <int kDim>
cudaError_t run_rows(const AttendParams& p, int sms, cudaStream_t stream) {
  const Tile t = tile_of(static_cast<int64_t>(p.list_queries) * p.group.d, kDim);
  if (t.tiles == 1) return launch_attention<kDim, 1, 1>(p, sms, stream);
  if (t.row_warps == 1) return launch_attention<kDim, 2, 1>(p, sms, stream);
  if constexpr (kDim == 64) {
    if (t.row_warps == 3) return launch_attention<kDim, 2, 3>(p, sms, stream);
    if (t.row_warps == 4) return launch_attention<kDim, 2, 4>(p, sms, stream);
  }
  return launch_attention<kDim, 2, 2>(p, sms, stream);
}

// More query rows on the same keys than two warps of a tile: the kernel of wide tiles, whose rows have 128 columns (64
// sequences of up to 8192 keys of 8 heads, 40 query heads on each: 279 us there, 323 in tiles of three warps; 32 query heads:
// 248 in tiles of two warps, 299 there).
bool wide_tile(int64_t rows, int32_t dim) { return padded_dim(dim) == 128 && rows > 32; }

cudaError_t run_attention(const AttendParams& p, int sms, cudaStream_t stream) {
  const int dim = padded_dim(p.dim);
  if (wide_tile(static_cast<int64_t>(p.list_queries) * p.group.d, p.dim)) return launch_wide_attention(p, sms, stream);
  if (dim == 64) return run_rows<64>(p, sms, stream);
  if (dim == 128) return run_rows<128>(p, sms, stream);
  return run_rows<256>(p, sms, stream);
}

Side side_of(const indexer_block_cache_t& c) {
  Side s = {};
  s.codes = c.codes;
  s.scales = c.scales;
  const auto step = [](int64_t n, int64_t stride) { return static_cast<uint32_t>(n > 1 ? stride : 0); };
  s.code_ps = step(c.num_pages, c.code_page_stride / 16), s.code_ts = step(c.page_size, c.code_token_stride / 16);
  s.scale_ps = step(c.num_pages, c.scale_page_stride), s.scale_bs = step(c.page_size / c.block, c.scale_block_stride);
  s.code_hs = c.code_head_stride, s.scale_hs = c.scale_head_stride;
  s.block = divisor(c.block);
  return s;
}

// Strides that the kernel steps over fit its 32 bits.
bool strides_ok(const indexer_block_cache_t& c) {
  const auto fits = [](int64_t n, int64_t stride) { return n <= 1 || stride <= INT64_C(0xffffffff); };
  return fits(c.num_pages, c.code_page_stride / 16) && fits(c.page_size, c.code_token_stride / 16) &&
         fits(c.num_pages, c.scale_page_stride) && fits(c.page_size / c.block, c.scale_block_stride);
}

bool aligned(const void* p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

size_t workspace_of(int64_t rows, int32_t dim, int sms) {
  const int padded = padded_dim(dim), tile = wide_tile(rows, dim) ? wide_rows(rows) : tile_of(rows, padded).rows();
  return static_cast<size_t>(kMaxCtas * sms) * (sizeof(Cut) + 2u * static_cast<size_t>(tile) * static_cast<size_t>(padded + 2) * 4u);
}

}  // namespace

cudaError_t attention_guard_hits(unsigned int* hits) {
  unsigned int more = 0;
  cudaError_t e = cudaMemcpyFromSymbol(hits, g_guard_hits, sizeof(unsigned int));
  if (e == cudaSuccess) e = wide_attention_guard_hits(&more);
  *hits += more;
  return e;
}

cudaError_t reset_attention_guard_hits() {
  const unsigned int zero = 0;
  const cudaError_t e = cudaMemcpyToSymbol(g_guard_hits, &zero, sizeof(unsigned int));
  return e == cudaSuccess ? reset_wide_attention_guard_hits() : e;
}

}  // namespace indexer_gb300

extern "C" {

size_t indexer_attention_workspace_bytes(int32_t queries, int32_t heads, int32_t cache_heads, int32_t dim, int32_t picked) {
  using namespace indexer_gb300;
  int sms = 0;
  if (queries < 1 || cache_heads < 1 || heads < cache_heads || heads % cache_heads != 0 || dim < 16 || dim % 16 != 0 ||
      dim > INDEXER_MAX_HEAD_DIM || sm_count(&sms) != cudaSuccess)
    return 0;
  return workspace_of(static_cast<int64_t>(picked != 0 ? 1 : queries) * (heads / cache_heads), dim, sms);
}

int indexer_attention(const void* q, int32_t dtype, const indexer_block_cache_t* keys, const indexer_block_cache_t* values,
                      const int32_t* index, int64_t index_stride, int64_t width, const int32_t* seq_lens, int32_t batch,
                      int32_t queries, int32_t heads, float softmax_scale, void* out, float* lse, void* workspace,
                      size_t workspace_bytes, cudaStream_t stream) {
  using namespace indexer_gb300;
  if ((dtype != INDEXER_BF16 && dtype != INDEXER_FP16) || !block_cache_ok(keys) || !block_cache_ok(values))
    return TOPK_ERR_INVALID_ARGUMENT;
  if (values->num_pages != keys->num_pages || values->page_size != keys->page_size || values->heads != keys->heads ||
      values->dim != keys->dim || !strides_ok(*keys) || !strides_ok(*values))
    return TOPK_ERR_INVALID_ARGUMENT;
  if (batch < 0 || queries < 0 || heads < 1 || heads % keys->heads != 0 || width < 0 || index_stride < 0 ||
      !(softmax_scale > -3.0e38f && softmax_scale < 3.0e38f))
    return TOPK_ERR_INVALID_ARGUMENT;
  if (batch == 0 || queries == 0) return TOPK_OK;
  if (queries > INT32_MAX / batch || queries > (1 << 30) / (heads / keys->heads)) return TOPK_ERR_INVALID_ARGUMENT;
  const int64_t lists = seq_lens != nullptr ? batch : static_cast<int64_t>(batch) * queries;
  if (lists > 1 && index_stride < width) return TOPK_ERR_INVALID_ARGUMENT;
  if (seq_lens == nullptr && width > INT32_MAX - 65536) return TOPK_ERR_INVALID_ARGUMENT;
  if (q == nullptr || out == nullptr || (index == nullptr && width > 0) || !aligned(q, 16) || !aligned(out, 16) ||
      !aligned(index, 4) || !aligned(seq_lens, 4) || !aligned(lse, 4))
    return TOPK_ERR_INVALID_ARGUMENT;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return status_of(e);
  AttendParams p = {};
  p.list_queries = seq_lens != nullptr ? queries : 1;
  p.group = divisor(heads / keys->heads);
  const size_t need = workspace_of(static_cast<int64_t>(p.list_queries) * p.group.d, keys->dim, sms);
  if (workspace_bytes < need) return TOPK_ERR_WORKSPACE_TOO_SMALL;
  if (workspace == nullptr || !aligned(workspace, 16)) return TOPK_ERR_INVALID_ARGUMENT;
  p.side[0] = side_of(*keys);
  p.side[1] = side_of(*values);
  p.q = q;
  p.out = out;
  p.lse = lse;
  p.index = index;
  p.seq_lens = seq_lens;
  p.partial = static_cast<float*>(workspace);  // of 16-byte multiples; what describes the cuts lies behind it
  p.cuts = reinterpret_cast<Cut*>(static_cast<char*>(workspace) + need - static_cast<size_t>(kMaxCtas * sms) * sizeof(Cut));
  p.index_stride = lists > 1 ? index_stride : 0;
  p.num_pages = keys->num_pages;
  p.capacity = keys->num_pages * keys->page_size;
  p.page_size = divisor(keys->page_size);
  p.lists = static_cast<int32_t>(lists);
  p.kv_heads = keys->heads;
  p.heads = heads;
  p.dim = keys->dim;
  constexpr int64_t kLongest = INT32_MAX - 65536;  // steps are numbered in 31 bits
  p.fp16 = dtype == INDEXER_FP16;
  p.whole_steps = seq_lens != nullptr && keys->page_size % kStep == 0;
  p.row_len = static_cast<int32_t>(seq_lens == nullptr ? width : width > kLongest / keys->page_size ? kLongest : width * keys->page_size);
  p.scale = softmax_scale * 1.44269504088896340736f;
  return status_of(run_attention(p, sms, stream));
}

}  // extern "C"
