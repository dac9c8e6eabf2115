// The indexer's scores over a paged cache of e4m3 keys:
//   score[j] = scale_j * sum_h weight_h * max(q_h . k_j, 0)
//
// The products are one matrix product: A a tile of 128 keys (one key a row of 128 bytes), B the
// heads of a group of queries of one sequence (N = queries * heads, up to 256 columns),
// both K-major in 128-byte swizzled shared memory, accumulated in fp32 in TMEM by tcgen05.mma
// kind::f8f6f4. A key is a TMEM lane, so the thread that reads a lane holds all of its key's
// products and sums its heads without any exchange between threads.
//
// What bounds it: one query a sequence (decode) reads 132 bytes a key for 2 * 128 * heads
// operations and is bound by memory; a prompt's chunk shares a key tile between the queries of a group
// and is bound by the relu-sum of the epilogue and by the tensor cores, about evenly.
//
// One CTA an SM, persistent over (sequence, query group, chunk of tiles); its warps share out the work:
//   warp 0      page ids and TMA copies: a ring of key tiles, two buffers of queries
//   warp 1      tcgen05.mma
//   warps 2, 3  the keys' scales into a ring, four tiles at once: they are a dependent load
//               behind the page id, which no warp with other work should wait for
//   warps 4-7, 8-11  two epilogue groups that take the tiles in turn
// A page is copied in pieces of the largest power of two of rows that divides its size, so
// every page size takes the same path.

#include <cuda.h>

#include <atomic>

#include "indexer_common.cuh"

namespace indexer_gb300 {
namespace {

constexpr int kDim = INDEXER_SCORE_DIM;  // bytes of a key's codes: one swizzled row
constexpr int kTile = 128;               // keys of a tile: the rows of one MMA, the lanes of TMEM
constexpr int kThreads = 384;
constexpr int kMaxColumns = 256;         // N of one MMA
constexpr int kTmemColumns = 512;
constexpr int kKeyStages = 8;
constexpr int kMaxTmemStages = 8;
constexpr int kScaleStages = 8;          // of each epilogue group
constexpr int kScaleBatch = 4;
constexpr int kMaxGroup = 16;            // queries of a group
constexpr int kEpilogueWarps = 8;
constexpr int kWaitLimit = 1 << 20;      // tries of a wait before it is given up

// A scale that stands for a page outside the cache; NaN scales of the cache get other bits.
constexpr uint32_t kNoPage = 0x7fc00001u;
constexpr uint32_t kNan = 0x7fffffffu;

// Pages outside the cache that were met, and waits that ran out (see indexer_guard_hits).
__device__ unsigned int g_guard_hits;

struct ScoresParams {
  const float* weights;
  const float* scales;
  const int32_t* page_table;
  const int32_t* seq_lens;
  float* out;
  int64_t num_pages, scale_ps, scale_ts, pt_stride;
  int64_t row_len, items, slices;  // slices: items of one chunk of tiles (sequences * groups)
  int32_t page_size, piece_rows;
  int32_t queries, heads, group, groups;
  int32_t tiles, chunk;            // tiles of a row; tiles of an item
  int32_t tmem_stages, tmem_stride;
};

struct Shared {
  alignas(1024) uint8_t keys[kKeyStages][kTile * kDim];
  alignas(1024) uint8_t queries[2][kMaxColumns * kDim];
  alignas(16) float scales[2][kScaleStages][kTile];
  alignas(16) float weights[kEpilogueWarps][kMaxColumns];  // each warp's own copy: no barrier among them
  int32_t lens[kEpilogueWarps][kMaxGroup];
  alignas(8) uint64_t key_full[kKeyStages], key_empty[kKeyStages];
  uint64_t query_full[2], query_empty[2];
  uint64_t tmem_full[kMaxTmemStages], tmem_empty[kMaxTmemStages];
  uint64_t scale_full[2][kScaleStages], scale_empty[2][kScaleStages];
  uint64_t drained;
  uint32_t tmem_base;
  int32_t aborted;
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void bar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void bar_expect(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)),
               "r"(bytes)
               : "memory");
}

// Waits for the end of a barrier's phase, for the whole warp. False when this or another wait of
// the CTA ran out: then every role leaves its loop.
__device__ __forceinline__ bool bar_wait(Shared& s, uint64_t* bar, uint32_t parity) {
  const uint32_t addr = smem_addr(bar);
  bool done = false;
  for (int i = 0; i < kWaitLimit; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\n"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n"
        "selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(addr), "r"(parity)
        : "memory");
    if (ok != 0u) {
      done = true;
      break;
    }
    if ((i & 255) == 255 && *const_cast<volatile int32_t*>(&s.aborted) != 0) break;
  }
  if (__all_sync(0xffffffffu, done)) return true;
  if ((threadIdx.x & 31) == 0 && atomicExch(&s.aborted, 1) == 0) atomicAdd(&g_guard_hits, 1u);
  return false;
}

__device__ __forceinline__ void tma_load_3d(const CUtensorMap* map, void* dst, uint64_t* bar, int x, int y,
                                            int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
      ::"r"(smem_addr(dst)), "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// K-major rows of 128 bytes, 128-byte swizzle: groups of 8 rows are 1024 bytes apart.
__device__ __forceinline__ uint64_t matrix_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}

__device__ __forceinline__ void tmem_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// 16 or 32 consecutive columns of this thread's lane.
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&r)[N]) {
  static_assert(N == 16 || N == 32, "columns of one load");
  if constexpr (N == 32) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
          "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
          "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
          "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(addr));
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
          "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(addr));
  }
}

// Completes the loads into r: its values may be used from here on, and not before.
template <int N>
__device__ __forceinline__ void tmem_wait(float (&r)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(r[i]));
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// One item: `count` queries from `query` on (rows of seq_lens and out, all of sequence b)
// against tiles [first, end); tiles from `seen` on have no key that any of the queries sees.
struct Item {
  int64_t query;
  int32_t b, count, first, seen, end, longest;
};

__device__ __forceinline__ int32_t clamp_len(const ScoresParams& p, int32_t len) {
  return static_cast<int32_t>(min(max(static_cast<int64_t>(len), int64_t(0)), p.row_len));
}

// Whole warps call this. Items are ordered with the chunk of tiles outermost, so that the CTAs work on
// the same tiles of a sequence at about the same time and find them in L2.
__device__ __forceinline__ Item item_at(const ScoresParams& p, int64_t index) {
  Item it;
  const int64_t c = index / p.slices;
  const int64_t slice = index - c * p.slices;
  it.b = static_cast<int32_t>(slice / p.groups);
  const int g0 = static_cast<int>(slice - static_cast<int64_t>(it.b) * p.groups) * p.group;
  it.count = min(p.group, p.queries - g0);
  it.query = static_cast<int64_t>(it.b) * p.queries + g0;
  it.first = static_cast<int32_t>(c) * p.chunk;
  it.end = min(it.first + p.chunk, p.tiles);
  const int lane = threadIdx.x & 31;
  const int32_t len = lane < it.count ? clamp_len(p, p.seq_lens[it.query + lane]) : 0;
  it.longest = __reduce_max_sync(0xffffffffu, len);
  it.seen = max(it.first, min(it.end, static_cast<int32_t>((static_cast<int64_t>(it.longest) + kTile - 1) / kTile)));
  return it;
}

__device__ __forceinline__ void load_keys(const ScoresParams& p, Shared& s, const CUtensorMap* key_map,
                                          const CUtensorMap* query_map, int head_rows) {
  const int lane = threadIdx.x & 31;
  const int pieces = kTile / p.piece_rows;
  const uint32_t piece_bytes = static_cast<uint32_t>(p.piece_rows) * kDim;
  int64_t tile_count = 0, item_count = 0;
  bool ok = true;
  for (int64_t i = blockIdx.x; ok && i < p.items; i += gridDim.x) {
    const Item it = item_at(p, i);
    if (it.seen <= it.first) continue;
    const int qb = static_cast<int>(item_count & 1);
    ok = bar_wait(s, &s.query_empty[qb], static_cast<uint32_t>((item_count >> 1) & 1) ^ 1u);
    if (!ok) break;
    if (lane == 0) {
      bar_expect(&s.query_full[qb], static_cast<uint32_t>(head_rows * p.group) * kDim);
      tma_load_3d(query_map, s.queries[qb], &s.query_full[qb], 0, 0, static_cast<int>(it.query));
    }
    ++item_count;
    const int32_t* table = p.page_table + static_cast<int64_t>(it.b) * p.pt_stride;
    int32_t page[4], next[4];
    auto pages_of = [&](int t, int32_t (&ids)[4]) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int piece = lane + 32 * k;
        const int64_t row = static_cast<int64_t>(t) * kTile + piece * p.piece_rows;
        ids[k] = t < it.seen && piece < pieces && row < it.longest
                     ? table[static_cast<uint32_t>(row) / static_cast<uint32_t>(p.page_size)]
                     : -1;
      }
    };
    pages_of(it.first, next);
    for (int t = it.first; t < it.seen; ++t) {
#pragma unroll
      for (int k = 0; k < 4; ++k) page[k] = next[k];
      pages_of(t + 1, next);
      const int st = static_cast<int>(tile_count % kKeyStages);
      ok = bar_wait(s, &s.key_empty[st], static_cast<uint32_t>((tile_count / kKeyStages) & 1) ^ 1u);
      if (!ok) break;
      ++tile_count;
      uint32_t bytes = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        bytes += piece_bytes * __popc(__ballot_sync(0xffffffffu, page[k] >= 0 && page[k] < p.num_pages));
      if (lane == 0) bar_expect(&s.key_full[st], bytes);
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (page[k] < 0 || page[k] >= p.num_pages) continue;
        const int piece = lane + 32 * k;
        const uint32_t row = static_cast<uint32_t>(t) * kTile + piece * p.piece_rows;
        tma_load_3d(key_map, s.keys[st] + piece * piece_bytes, &s.key_full[st], 0,
                    static_cast<int>(row % static_cast<uint32_t>(p.page_size)), page[k]);
      }
      __syncwarp();
    }
  }
  // no copy outlives the CTA, whatever ended the loop
  const int64_t tiles = tile_count < kKeyStages ? tile_count : kKeyStages, items = item_count < 2 ? item_count : 2;
  for (int64_t k = 1; k <= tiles; ++k) {
    const int64_t c = tile_count - k;
    bar_wait(s, &s.key_full[c % kKeyStages], static_cast<uint32_t>((c / kKeyStages) & 1));
  }
  for (int64_t k = 1; k <= items; ++k) {
    const int64_t c = item_count - k;
    bar_wait(s, &s.query_full[c & 1], static_cast<uint32_t>((c >> 1) & 1));
  }
}

__device__ __forceinline__ void multiply(const ScoresParams& p, Shared& s, uint32_t tmem, int head_rows) {
  const int lane = threadIdx.x & 31;
  int64_t tile_count = 0, item_count = 0;
  int ts = 0;
  uint32_t ts_phase = 0;
  bool ok = true;
  for (int64_t i = blockIdx.x; ok && i < p.items; i += gridDim.x) {
    const Item it = item_at(p, i);
    if (it.seen <= it.first) continue;
    const int qb = static_cast<int>(item_count & 1);
    ok = bar_wait(s, &s.query_full[qb], static_cast<uint32_t>((item_count >> 1) & 1));
    if (!ok) break;
    ++item_count;
    // fp32 accumulators, e4m3 operands, both K-major, M = 128
    const uint32_t columns = static_cast<uint32_t>(it.count * head_rows);
    const uint32_t idesc = (1u << 4) | ((columns >> 3) << 17) | ((kTile >> 4) << 24);
    const uint64_t b = matrix_desc(smem_addr(s.queries[qb]));
    for (int t = it.first; t < it.seen; ++t) {
      const int st = static_cast<int>(tile_count % kKeyStages);
      ok = bar_wait(s, &s.key_full[st], static_cast<uint32_t>((tile_count / kKeyStages) & 1)) &&
           bar_wait(s, &s.tmem_empty[ts], ts_phase ^ 1u);
      if (!ok) break;
      ++tile_count;
      tmem_fence_after();
      if (lane == 0) {
        const uint64_t a = matrix_desc(smem_addr(s.keys[st]));
        const uint32_t d = tmem + static_cast<uint32_t>(ts * p.tmem_stride);
#pragma unroll
        for (int k = 0; k < kDim / 32; ++k) mma_e4m3(d, a + k * 2, b + k * 2, idesc, k > 0 ? 1u : 0u);
        mma_commit(&s.key_empty[st]);
        mma_commit(&s.tmem_full[ts]);
        if (t + 1 == it.seen) mma_commit(&s.query_empty[qb]);
      }
      __syncwarp();
      if (++ts == p.tmem_stages) {
        ts = 0;
        ts_phase ^= 1u;
      }
    }
  }
  // no MMA outlives the CTA
  if (lane == 0) mma_commit(&s.drained);
  __syncwarp();
  bar_wait(s, &s.drained, 0u);
}

// The scales of the tiles of epilogue group `wg` (every second one), kScaleBatch tiles at once: the
// page ids of all of them, then the scales, so that each latency is met once in a batch.
__device__ __forceinline__ void load_scales(const ScoresParams& p, Shared& s, int wg) {
  constexpr int kKeys = kTile / 32;  // keys of a lane
  const int lane = threadIdx.x & 31;
  int64_t index = blockIdx.x, tile_count = 0, stored = 0;
  Item it = {};
  int t = 0;
  bool more = index < p.items;
  if (more) {
    it = item_at(p, index);
    t = it.first;
  }
  while (more) {
    uint32_t got[kScaleBatch][kKeys];
    int32_t page[kScaleBatch][kKeys];
    int tiles = 0;
#pragma unroll
    for (int u = 0; u < kScaleBatch; ++u) {
      // on to the next tile of this group
      bool found = false;
      while (more && !found) {
        if (t >= it.seen) {
          index += gridDim.x;
          more = index < p.items;
          if (more) {
            it = item_at(p, index);
            t = it.first;
          }
          continue;
        }
        found = (tile_count & 1) == wg;
        ++tile_count;
        if (!found) ++t;
      }
#pragma unroll
      for (int k = 0; k < kKeys; ++k) {
        const uint32_t j = static_cast<uint32_t>(t) * kTile + k * 32 + lane;
        const bool seen = found && j < static_cast<uint32_t>(it.longest);
        // past the longest query: 0, and never used
        got[u][k] = seen ? j % static_cast<uint32_t>(p.page_size) : 0xffffffffu;
        page[u][k] = seen ? p.page_table[static_cast<int64_t>(it.b) * p.pt_stride +
                                         j / static_cast<uint32_t>(p.page_size)]
                          : 0;
      }
      if (found) {
        ++tiles;
        ++t;
      }
    }
#pragma unroll
    for (int u = 0; u < kScaleBatch; ++u) {
#pragma unroll
      for (int k = 0; k < kKeys; ++k) {
        const uint32_t off = got[u][k];
        if (off == 0xffffffffu) {
          got[u][k] = 0u;
        } else if (page[u][k] < 0 || page[u][k] >= p.num_pages) {
          got[u][k] = kNoPage;
          atomicAdd(&g_guard_hits, 1u);
        } else {
          got[u][k] = __float_as_uint(p.scales[page[u][k] * p.scale_ps + off * p.scale_ts]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kScaleBatch; ++u) {
      if (u >= tiles) break;
      const int st = static_cast<int>(stored % kScaleStages);
      if (!bar_wait(s, &s.scale_empty[wg][st], static_cast<uint32_t>((stored / kScaleStages) & 1) ^ 1u)) return;
      ++stored;
#pragma unroll
      for (int k = 0; k < kKeys; ++k) {
        const uint32_t v = got[u][k];
        s.scales[wg][st][k * 32 + lane] =
            __uint_as_float((v & 0x7fffffffu) > 0x7f800000u && v != kNoPage ? kNan : v);
      }
      __syncwarp();
      if (lane == 0) bar_arrive(&s.scale_full[wg][st]);
    }
  }
}

// Adds weight * relu(product) of N columns to two pairs of sums.
template <int N>
__device__ __forceinline__ void add_heads(const float (&r)[N], const float* weights, uint64_t (&acc)[2]) {
  const float4* w = reinterpret_cast<const float4*>(weights);
#pragma unroll
  for (int h = 0; h < N / 4; ++h) {
    const float4 f = w[h];
    acc[0] = fma2(pack2(fmaxf(r[4 * h], 0.0f), fmaxf(r[4 * h + 1], 0.0f)), pack2(f.x, f.y), acc[0]);
    acc[1] = fma2(pack2(fmaxf(r[4 * h + 2], 0.0f), fmaxf(r[4 * h + 3], 0.0f)), pack2(f.z, f.w), acc[1]);
  }
}

// One epilogue warp: relu, weights and the sum over heads of its 32 lanes (keys), for the tiles of
// group `wg`. kHeads: columns of a query.
template <int kHeads>
__device__ __forceinline__ void reduce(const ScoresParams& p, Shared& s, uint32_t tmem, int wg) {
  constexpr int kHalf = kHeads <= 32 ? kHeads : 32;   // columns of a load
  constexpr int kStep = kHeads <= 32 ? kHeads : 64;   // columns of a round: one load, or two
  constexpr int kWeights = kMaxColumns / 32;          // weights that a lane brings
  const int tid = threadIdx.x & 127, lane = tid & 31, warp = threadIdx.x / 32 - 4;
  float* const weights = s.weights[warp];
  int32_t* const lens = s.lens[warp];
  const uint32_t lane_base = tmem + (static_cast<uint32_t>(tid & ~31) << 16);
  const float minus_inf = __int_as_float(0xff800000);
  float w[kWeights];
  auto weights_of = [&](int64_t index) {
    if (index >= p.items) return;
    const int64_t slice = index % p.slices, b = slice / p.groups;
    const int g0 = static_cast<int>(slice - b * p.groups) * p.group;
    const float* src = p.weights + (b * p.queries + g0) * p.heads;
#pragma unroll
    for (int k = 0; k < kWeights; ++k) {
      const int g = (lane + 32 * k) / kHeads, h = (lane + 32 * k) % kHeads;
      w[k] = g < p.group && g0 + g < p.queries && h < p.heads ? src[g * p.heads + h] : 0.0f;
    }
  };
  weights_of(blockIdx.x);
  int64_t tile_count = 0, taken = 0;
  for (int64_t i = blockIdx.x; i < p.items; i += gridDim.x) {
    const Item it = item_at(p, i);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kWeights; ++k) weights[lane + 32 * k] = w[k];
    if (lane < it.count) lens[lane] = clamp_len(p, p.seq_lens[it.query + lane]);
    __syncwarp();
    weights_of(i + gridDim.x);  // on their way while this item is worked on
    float* const out = p.out + it.query * p.row_len;
    for (int t = it.first; t < it.seen; ++t, ++tile_count) {
      if ((tile_count & 1) != wg) continue;
      const int64_t j = static_cast<int64_t>(t) * kTile + tid;
      const int ss = static_cast<int>(taken % kScaleStages);
      if (!bar_wait(s, &s.scale_full[wg][ss], static_cast<uint32_t>((taken / kScaleStages) & 1))) return;
      const float scale = s.scales[wg][ss][tid];
      __syncwarp();
      if (lane == 0) bar_arrive(&s.scale_empty[wg][ss]);
      ++taken;
      const int ts = static_cast<int>(tile_count % p.tmem_stages);
      if (!bar_wait(s, &s.tmem_full[ts], static_cast<uint32_t>((tile_count / p.tmem_stages) & 1))) return;
      tmem_fence_after();
      const uint32_t at = lane_base + static_cast<uint32_t>(ts * p.tmem_stride);
      const bool no_page = __float_as_uint(scale) == kNoPage;
      const int columns = it.count * kHeads;
      auto release = [&](int next) {  // every column of the tile is in registers: its stage is free
        if (next < columns) return;
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&s.tmem_empty[ts]);
      };
      uint64_t acc[2] = {0, 0};
      for (int c = 0; c < columns; c += kStep) {
        float r0[kHalf];
        tmem_load<kHalf>(at + c, r0);
        tmem_wait<kHalf>(r0);
        if constexpr (kStep > kHalf) {
          float r1[kHalf];
          tmem_load<kHalf>(at + c + kHalf, r1);
          add_heads<kHalf>(r0, weights + c, acc);
          tmem_wait<kHalf>(r1);
          release(c + kStep);
          add_heads<kHalf>(r1, weights + c + kHalf, acc);
        } else {
          release(c + kStep);
          add_heads<kHalf>(r0, weights + c, acc);
        }
        if ((c + kStep) % kHeads == 0) {
          const int g = c / kHeads;
          const float2 a = unpack2(acc[0]), b = unpack2(acc[1]);
          const float y = ((a.x + a.y) + (b.x + b.y)) * scale;
          if (j < p.row_len) out[g * p.row_len + j] = j < lens[g] && !no_page ? y : minus_inf;
          acc[0] = acc[1] = 0;
        }
      }
    }
    // tiles that no query of the group sees
    for (int t = it.seen + wg; t < it.end; t += 2) {
      const int64_t j = static_cast<int64_t>(t) * kTile + tid;
      if (j < p.row_len)
        for (int g = 0; g < it.count; ++g) out[g * p.row_len + j] = minus_inf;
    }
  }
}

// kHeads: heads rounded up to 16, 32, 64 or 128. The rounding's rows of B are zeros (beyond the
// tensor map's heads) and their weights are 0.
template <int kHeads>
__global__ void __launch_bounds__(kThreads, 1)
    scores_kernel(const ScoresParams p, const __grid_constant__ CUtensorMap key_map,
                  const __grid_constant__ CUtensorMap query_map) {
  extern __shared__ uint8_t raw[];
  Shared& s = *reinterpret_cast<Shared*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x / 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kKeyStages; ++i) {
      bar_init(&s.key_full[i], 1);
      bar_init(&s.key_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&s.query_full[i], 1);
      bar_init(&s.query_empty[i], 1);
      for (int k = 0; k < kScaleStages; ++k) {
        bar_init(&s.scale_full[i][k], 1);
        bar_init(&s.scale_empty[i][k], 4);
      }
    }
    for (int i = 0; i < kMaxTmemStages; ++i) {
      bar_init(&s.tmem_full[i], 1);
      bar_init(&s.tmem_empty[i], 4);
    }
    bar_init(&s.drained, 1);
    s.aborted = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    // one CTA an SM (its shared memory sees to that), so the columns are free
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s.tmem_base)),
                 "r"(kTmemColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    tmem_fence_before();
  }
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = s.tmem_base;
  begin_after_prior_grids();

  if (warp == 0) load_keys(p, s, &key_map, &query_map, kHeads);
  else if (warp == 1) multiply(p, s, tmem, kHeads);
  else if (warp < 4) load_scales(p, s, warp - 2);
  else reduce<kHeads>(p, s, tmem, (warp - 4) / 4);

  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemColumns));
}

constexpr size_t kSmemBytes = sizeof(Shared) + 1024;

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

cudaError_t encode_fn(EncodeTiled* out) {
  static std::atomic<void*> known{nullptr};
  void* fn = known.load(std::memory_order_acquire);
  if (fn == nullptr) {
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (found != cudaDriverEntryPointSuccess || fn == nullptr) return cudaErrorNotSupported;
    known.store(fn, std::memory_order_release);
  }
  *out = reinterpret_cast<EncodeTiled>(fn);
  return cudaSuccess;
}

// A map of rows of 128 bytes on two outer axes, copied `box1` by `box2` rows at once.
cudaError_t row_map(EncodeTiled encode, CUtensorMap* map, const uint8_t* base, int64_t n1, int64_t stride1, int64_t n2,
                    int64_t stride2, int box1, int box2) {
  const cuuint64_t dims[3] = {kDim, static_cast<cuuint64_t>(n1), static_cast<cuuint64_t>(n2)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(stride1), static_cast<cuuint64_t>(stride2)};
  const cuuint32_t box[3] = {kDim, static_cast<cuuint32_t>(box1), static_cast<cuuint32_t>(box2)};
  const cuuint32_t steps[3] = {1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(base), dims, strides, box, steps,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int kHeads>
cudaError_t launch_scores(ScoresParams p, const CUtensorMap& key_map, const CUtensorMap& query_map, unsigned grid,
                          cudaStream_t stream) {
  // set once for each device and kernel: the attribute belongs to the function on that device
  static std::atomic<uint64_t> prepared{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev > 63 || (prepared.load(std::memory_order_acquire) >> dev & 1u) == 0) {
    e = cudaFuncSetAttribute(scores_kernel<kHeads>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmemBytes));
    if (e != cudaSuccess) return e;
    if (dev <= 63) prepared.fetch_or(uint64_t(1) << dev, std::memory_order_release);
  }
  return launch(scores_kernel<kHeads>, grid, kThreads, kSmemBytes, stream, p, key_map, query_map);
}

}  // namespace

cudaError_t scores_guard_hits(unsigned int* hits) {
  return cudaMemcpyFromSymbol(hits, g_guard_hits, sizeof(unsigned int));
}

cudaError_t reset_scores_guard_hits() {
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_guard_hits, &zero, sizeof(unsigned int));
}

}  // namespace indexer_gb300

extern "C" int indexer_scores(const uint8_t* q, const float* weights, const indexer_cache_t* cache,
                              const int32_t* page_table, int64_t page_table_stride,
                              const int32_t* seq_lens, int32_t batch, int32_t queries, int32_t heads,
                              int64_t row_len, float* out, cudaStream_t stream) {
  using namespace indexer_gb300;
  if (!cache_ok(cache) || cache->dim != INDEXER_SCORE_DIM) return TOPK_ERR_INVALID_ARGUMENT;
  if (batch < 0 || queries < 0 || heads < 1 || heads > INDEXER_MAX_HEADS || row_len < 1 ||
      row_len > INT32_MAX || static_cast<int64_t>(batch) * queries > INT32_MAX)
    return TOPK_ERR_INVALID_ARGUMENT;
  if (batch == 0 || queries == 0) return TOPK_OK;
  if (q == nullptr || weights == nullptr || page_table == nullptr || seq_lens == nullptr || out == nullptr)
    return TOPK_ERR_INVALID_ARGUMENT;
  const int64_t pages = (row_len + cache->page_size - 1) / cache->page_size;
  if (page_table_stride < (batch > 1 ? pages : 1)) return TOPK_ERR_INVALID_ARGUMENT;
  const int64_t code_ts = cache->page_size > 1 ? cache->code_token_stride : kDim;
  const int64_t code_ps = cache->num_pages > 1 ? cache->code_page_stride : kDim;
  const uintptr_t low = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(cache->codes) |
                        static_cast<uintptr_t>(code_ts) | static_cast<uintptr_t>(code_ps);
  const uintptr_t low4 = reinterpret_cast<uintptr_t>(weights) | reinterpret_cast<uintptr_t>(page_table) |
                         reinterpret_cast<uintptr_t>(seq_lens) | reinterpret_cast<uintptr_t>(out);
  if ((low & 15u) != 0 || (low4 & 3u) != 0) return TOPK_ERR_INVALID_ARGUMENT;
  if (code_ts >= INT64_C(1) << 40 || code_ps >= INT64_C(1) << 40) return TOPK_ERR_INVALID_ARGUMENT;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return status_of(e);
  EncodeTiled encode = nullptr;
  e = encode_fn(&encode);
  if (e != cudaSuccess) return status_of(e);

  ScoresParams p = {};
  p.weights = weights;
  p.scales = cache->scales;
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.out = out;
  p.num_pages = cache->num_pages;
  p.scale_ps = cache->scale_page_stride;
  p.scale_ts = cache->scale_token_stride;
  p.pt_stride = page_table_stride;
  p.row_len = row_len;
  p.page_size = cache->page_size;
  p.piece_rows = cache->page_size & -cache->page_size;
  if (p.piece_rows > kTile) p.piece_rows = kTile;
  p.queries = queries;
  p.heads = heads;
  const int head_rows = heads <= 16 ? 16 : heads <= 32 ? 32 : heads <= 64 ? 64 : 128;
  p.group = kMaxColumns / head_rows < queries ? kMaxColumns / head_rows : queries;
  p.groups = (queries + p.group - 1) / p.group;
  p.tiles = static_cast<int32_t>((row_len + kTile - 1) / kTile);
  // Tensor-memory stages of 32 columns or a larger power of two.
  p.tmem_stride = 32;
  while (p.tmem_stride < p.group * head_rows) p.tmem_stride *= 2;
  p.tmem_stages = kTmemColumns / p.tmem_stride < kMaxTmemStages ? kTmemColumns / p.tmem_stride : kMaxTmemStages;
  // Tiles of an item: one while there are fewer tiles than SMs; otherwise so many that each SM gets
  // 16 items or more (its share of uneven items evens out), 32 tiles at most.
  p.slices = static_cast<int64_t>(batch) * p.groups;
  const int64_t chunk = p.slices * p.tiles / (int64_t(sms) * 16);
  p.chunk = static_cast<int32_t>(chunk < 1 ? 1 : chunk > 32 ? 32 : chunk);
  p.items = p.slices * ((p.tiles + p.chunk - 1) / p.chunk);

  CUtensorMap key_map, query_map;
  // a cache of no pages has none that passes the kernel's check: its map is never used
  e = cache->num_pages > 0
          ? row_map(encode, &key_map, cache->codes, cache->page_size, code_ts, cache->num_pages, code_ps, p.piece_rows, 1)
          : row_map(encode, &key_map, q, 1, kDim, 1, kDim, 1, 1);
  if (e == cudaSuccess)
    e = row_map(encode, &query_map, q, heads, kDim, static_cast<int64_t>(batch) * queries,
                static_cast<int64_t>(heads) * kDim, head_rows, p.group);
  if (e != cudaSuccess) return status_of(e);
  const unsigned grid = static_cast<unsigned>(p.items < sms ? p.items : sms);
  if (head_rows == 16) e = launch_scores<16>(p, key_map, query_map, grid, stream);
  else if (head_rows == 32) e = launch_scores<32>(p, key_map, query_map, grid, stream);
  else if (head_rows == 64) e = launch_scores<64>(p, key_map, query_map, grid, stream);
  else e = launch_scores<128>(p, key_map, query_map, grid, stream);
  return status_of(e);
}
