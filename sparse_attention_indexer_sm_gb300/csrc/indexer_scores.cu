// The indexer's scores over a paged cache of e4m3 keys:
//   score[j] = scale_j * sum_h weight_h * max(q_h . k_j, 0)
//
// The products are one matrix product: A a tile of 128 keys (one key a row of 128 bytes), B the
// heads of a group of queries of one sequence (N = queries * heads, up to 256 columns),
// both K-major in 128-byte swizzled shared memory, accumulated in fp32 in TMEM by tcgen05.mma
// kind::f8f6f4. A key is a TMEM lane, so the thread that reads a lane holds all of its key's
// products and sums its heads without any exchange between threads.
//
// What bounds it: one query a sequence (decode) reads 132 bytes a key for 2 * 128 * heads operations and is
// bound by memory (256 rows of 32768 keys, 64 heads: 175 us, 6.5 TB/s). A prompt's chunk shares a key tile
// between the queries of a group and is bound by the epilogue's relu-sum (2048 queries over 32768 keys:
// 512 us, 2.1 PFLOP/s); so are several drafted tokens (64 rows of 4 queries: 83 us against 46 for the memory).
//
// One CTA an SM, persistent: over items (sequence, query group, chunk of tiles) in turn, or over an equal span
// of all tiles that some query sees, which each CTA finds by adding up the lengths. A tile's products are one
// unit of columns, or two (the same number for a whole launch). The warps of a CTA share out the work:
//   loaders      page ids and TMA copies: a ring of key tiles, two buffers of queries
//   multipliers  tcgen05.mma
//   scalers      the keys' scales, two tiles at once: they are a dependent load behind the page id,
//                which no warp with other work should wait for
//   epilogue     groups of four warps, each with a weight for every one of its columns in registers: from
//                shared memory a weight costs as much as four columns' arithmetic
// in one of two plans. A lone warp takes some 50 cycles for each barrier that it looks at, so with up to 128
// columns, where a tile is soon done, every role that a tile passes through has two warps or four that take
// turns. With more columns an epilogue group's work on a tile outlasts that, and what counts is how many warps
// hide each other's latencies: four groups, of a quarter of the columns each (2048 queries over 32768 keys, 16,
// 32 and 64 heads: 151, 275 and 511 us, with two groups 183, 297 and 540). There the epilogue still bounds the
// kernel, at 66% of the issue slots and 64% of the integer pipe (relu is one of its instructions); the tensor
// pipe is at 43%. Its warps wait for a tile 5% of their time. Of some 200 instructions a warp and tile 96 are
// relus and products and 54 are left in an epilogue without them; the rest, some 50, is not accounted for
// (spilled registers, and places that are worked out at every tile, are among it). No pipe is full: the
// instructions' own latencies are, and fewer of them would show.
// A barrier's parity tells a phase from the next one, but not from the one after that. So each place of a ring
// belongs to the same warp of a role throughout: tiles and units are dealt out by their running numbers over the
// whole launch, and the rings' lengths are multiples of the numbers of warps.
// A page is copied in pieces of the largest power of two of rows that divides its size, so every page size takes
// the same path; but pages of one row are gathered, four by one copy (64 rows of 32768 keys, 64 heads: 90 us; a
// copy for each took two and a half times that).

#include <cuda.h>

#include <atomic>
#include <type_traits>

#include "indexer_common.cuh"

namespace indexer_gb300 {
namespace {

constexpr int kDim = INDEXER_SCORE_DIM;  // bytes of a key's codes: one swizzled row
constexpr int kTile = 128;               // keys of a tile: the rows of one MMA, the lanes of TMEM
constexpr int kMaxColumns = 256;         // heads of a group's queries
// How a CTA's warps share out its work, by the number of epilogue groups. Registers of a thread: what a launch
// of so many threads has of 65536, moved from the first warps to the epilogue (512 * 128 = 256 * 64 + 256 * 192,
// and 640 * 96 = 128 * 64 + 512 * 104).
template <int kGroups> struct Plan;
template <> struct Plan<2> {  // the groups take units in turn
  static constexpr int kLoaders = 2, kMultipliers = 2, kScalers = 4, kFewRegisters = 64, kManyRegisters = 192;
  static constexpr int kColumns = 128;  // of a unit, N of its MMAs: a register each in the epilogue
};
template <> struct Plan<4> {  // each group takes a quarter of the columns of every tile
  static constexpr int kLoaders = 1, kMultipliers = 1, kScalers = 2, kFewRegisters = 64, kManyRegisters = 104;
  static constexpr int kColumns = 64;
};
template <int kGroups> constexpr int kFirstWarp = Plan<kGroups>::kLoaders + Plan<kGroups>::kMultipliers + Plan<kGroups>::kScalers;
template <int kGroups> constexpr int kThreads = 32 * (kFirstWarp<kGroups> + 4 * kGroups);

constexpr int kTmemColumns = 512;
constexpr int kKeyStages = 8;
constexpr int kMaxTmemStages = 8;
constexpr int kScaleBatch = 2;
constexpr int kMaxSpanSlices = 8192;     // slices whose lengths a CTA adds up for its span
constexpr int kMaxChunk = 64;            // tiles of an item
constexpr int kItemCost = 4;             // tiles that the start of an item costs
constexpr int kMaxGroup = 16;            // queries of a group
constexpr int kEpilogueWarps = 16;       // at most
static_assert(kMaxSpanSlices * 4 <= kKeyStages * kTile * kDim, "their sums fit the ring of keys");
constexpr int kWaitLimit = 1 << 17;      // tries of a wait before it is given up,
constexpr uint32_t kWaitNs = 20000;      // each of which may sleep this long: 2.6 s in all

// A scale that stands for a page outside the cache; every NaN scale of the cache gets other bits as it is read.
constexpr uint32_t kNoPage = 0x7fc00001u;
constexpr uint32_t kNan = 0x7fffffffu;

__device__ __forceinline__ uint32_t scale_bits(uint32_t v) { return (v & 0x7fffffffu) > 0x7f800000u ? kNan : v; }

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
  Divisor page_div;                // by page_size
  int32_t quads;                   // pages hold whole quads of keys: 1; and their scales are aligned 16-byte quads: 2
  int32_t queries, heads, group, groups;
  int32_t tiles, chunk;            // tiles of a row; tiles of an item
  int32_t tmem_shift, tmem_stride; // 2^tmem_shift stages of tmem_stride columns
  int32_t units, unit_queries;     // units of a tile (1 or 2); queries of a unit
  int32_t fail;                    // for tests: 1 as if a wait had run out, 2 as if shared memory were misaligned
};

struct Shared {
  alignas(1024) uint8_t keys[kKeyStages][kTile * kDim];
  alignas(1024) uint8_t queries[2][kMaxColumns * kDim];
  alignas(16) float scales[kMaxTmemStages][kTile];
  alignas(16) float weights[1024];  // a copy for each epilogue warp of its columns': no barrier among them
  int32_t lens[kEpilogueWarps][kMaxGroup];
  alignas(8) uint64_t key_full[kKeyStages], key_empty[kKeyStages];
  uint64_t query_full[2], query_empty[2];
  uint64_t tmem_full[kMaxTmemStages], tmem_empty[kMaxTmemStages];
  uint64_t drained;
  int32_t span_slice[2], span_tile[2];  // this CTA's span: where it begins, and where it ends
  int32_t warp_sums[32];
  uint32_t tmem_base;
  int32_t aborted;
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void bar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_arrive(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* bar) { bar_arrive(smem_addr(bar)); }

__device__ __forceinline__ void bar_expect(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)),
               "r"(bytes)
               : "memory");
}

__device__ __forceinline__ bool bar_try(uint32_t addr, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\n"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n"
      "selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(addr), "r"(parity), "r"(kWaitNs)
      : "memory");
  return ok != 0u;
}

__device__ __forceinline__ bool bar_test(uint32_t addr, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\n"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(addr), "r"(parity)
      : "memory");
  return ok != 0u;
}

// Waits for the end of a barrier's phase. False when this wait or another of the CTA ran out.
__device__ __forceinline__ bool bar_wait_thread(Shared& s, uint32_t addr, uint32_t parity) {
  for (int i = 0; i < kWaitLimit; ++i) {
    if (bar_try(addr, parity)) return true;
    if (*const_cast<volatile int32_t*>(&s.aborted) != 0) return false;
  }
  if (atomicExch(&s.aborted, 1) == 0) atomicAdd(&g_guard_hits, 1u);
  return false;
}

// The same for a whole warp that issues copies or MMAs: it goes on, or leaves its loop, as one.
__device__ __forceinline__ bool bar_wait(Shared& s, uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, bar_wait_thread(s, smem_addr(bar), parity));
}

// At the end of a role, whatever ended it: until its copies or MMAs have landed, some milliseconds at most.
__device__ __forceinline__ void bar_drain(uint64_t* bar, uint32_t parity) {
  for (int i = 0; i < 256 && !bar_try(smem_addr(bar), parity); ++i) {
  }
  __syncwarp();
}

// A wait of the other roles, which go on in any case: after a wait that ran out they run through to their end
// with wrong numbers, in bounds, over which the epilogue then writes NaN (and the count is in g_guard_hits).
__device__ __forceinline__ void bar_pass(Shared& s, uint32_t addr, uint32_t parity) {
  bar_wait_thread(s, addr, parity);
  __syncwarp();
}

__device__ __forceinline__ void tma_load_3d(const CUtensorMap* map, void* dst, uint64_t* bar, int x, int y,
                                            int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
      ::"r"(smem_addr(dst)), "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Four rows of a map of single rows, at any places, into 512 bytes.
__device__ __forceinline__ void tma_gather4(const CUtensorMap* map, void* dst, uint64_t* bar, int r0, int r1, int r2,
                                            int r3) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(smem_addr(bar)), "r"(0), "r"(r0), "r"(r1), "r"(r2), "r"(r3)
      : "memory");
}

// Descriptors of K-major rows of 128 bytes, 128-byte swizzle: groups of 8 rows are 1024 bytes apart.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t matrix_desc(uint32_t addr) { return ((addr & 0x3ffffu) >> 4) | (1u << 16); }

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0u;
}

// The products of a tile's 128 dimensions, 32 at a time. a, b: low words of the operands' descriptors.
__device__ __forceinline__ void mma_tile(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
  asm volatile(
      "{\n.reg .pred p, q;\n.reg .b64 x, y;\n.reg .b32 u, v;\n"
      "setp.ne.b32 p, 0, 0;\nsetp.eq.b32 q, 0, 0;\n"
      "mov.b64 x, {%1, %4};\nmov.b64 y, {%2, %4};\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, p;\n"
      "add.u32 u, %1, 2;\nadd.u32 v, %2, 2;\nmov.b64 x, {u, %4};\nmov.b64 y, {v, %4};\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, q;\n"
      "add.u32 u, %1, 4;\nadd.u32 v, %2, 4;\nmov.b64 x, {u, %4};\nmov.b64 y, {v, %4};\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, q;\n"
      "add.u32 u, %1, 6;\nadd.u32 v, %2, 6;\nmov.b64 x, {u, %4};\nmov.b64 y, {v, %4};\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, q;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(kDescHigh)
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
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ uint32_t page_of(const ScoresParams& p, uint32_t row) { return quotient(p.page_div, row); }

// One item: `count` queries from `query` on (rows of seq_lens and out, all of sequence b)
// against tiles [first, end); tiles from `seen` on have no key that any of the queries sees.
struct Item {
  int64_t query;
  int32_t b, count, first, seen, end, longest, shortest;
  int32_t len;  // of this lane's query
};

// A slice is the tiles of one group of queries of a sequence.
struct Slice {
  int64_t query;
  int32_t b, count;
};

__device__ __forceinline__ Slice slice_at(const ScoresParams& p, int64_t slice) {
  Slice r;
  r.b = static_cast<int32_t>(slice / p.groups);
  const int g0 = static_cast<int>(slice - static_cast<int64_t>(r.b) * p.groups) * p.group;
  r.count = min(p.group, p.queries - g0);
  r.query = static_cast<int64_t>(r.b) * p.queries + g0;
  return r;
}

__device__ __forceinline__ int32_t clamped(const ScoresParams& p, int32_t len) {
  return static_cast<int32_t>(min(static_cast<int64_t>(max(len, 0)), p.row_len));
}

__device__ __forceinline__ int32_t tiles_of(int32_t len) {
  return static_cast<int32_t>((static_cast<uint32_t>(len) + kTile - 1) / kTile);
}

// The tiles of a slice that some query sees, by one thread.
__device__ __forceinline__ int32_t seen_tiles(const ScoresParams& p, const Slice& r) {
  int32_t longest = 0;
  for (int k = 0; k < r.count; k += 4) {  // four loads at once
    int32_t len[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) len[q] = k + q < r.count ? p.seq_lens[r.query + k + q] : 0;
    longest = max(max(max(longest, len[0]), max(len[1], len[2])), len[3]);
  }
  return tiles_of(clamped(p, longest));
}

// How a CTA walks over its work: items blockIdx.x, blockIdx.x + gridDim.x, ... of fixed chunks of tiles; or
// (kSpans) the slices that its span of the tiles touches. Every role walks alike.
template <bool kSpans> struct Walk;
template <> struct Walk<false> {
  int64_t at;
  __device__ __forceinline__ Walk(const Shared&) : at(blockIdx.x) {}
  __device__ __forceinline__ bool more(const ScoresParams& p) const { return at < p.items; }
  __device__ __forceinline__ void on() { at += gridDim.x; }
};
template <> struct Walk<true> {
  int32_t at, first, end, end_tile;  // slices; the next one's first tile, and the last one's end
  __device__ __forceinline__ Walk(const Shared& s)
      : at(s.span_slice[0]), first(s.span_tile[0]), end(s.span_slice[1]), end_tile(s.span_tile[1]) {}
  __device__ __forceinline__ bool more(const ScoresParams& p) const {
    return at < end || (at == end && first < end_tile);
  }
  __device__ __forceinline__ void on() {
    ++at;
    first = 0;
  }
};

// The place of the item at w, or the one after it. Items in turn are ordered with the chunk of tiles outermost,
// so that the CTAs work on the same tiles of a sequence at about the same time and find them in L2.
template <bool kSpans>
__device__ __forceinline__ Item place_at(const ScoresParams& p, const Walk<kSpans>& w, int ahead) {
  Item it = {};
  int64_t slice, c = 0;
  if constexpr (kSpans) {
    slice = w.at + ahead;
    if (slice > w.end || slice >= p.slices) return it;
  } else {
    const int64_t index = w.at + static_cast<int64_t>(ahead) * gridDim.x;
    if (index >= p.items) return it;
    c = index / p.slices;
    slice = index - c * p.slices;
  }
  const Slice r = slice_at(p, slice);
  it.b = r.b;
  it.count = r.count;
  it.query = r.query;
  it.first = static_cast<int32_t>(c) * p.chunk;
  it.end = min(it.first + p.chunk, p.tiles);
  return it;
}

// The same and the load of its lengths: asked for one item ahead.
template <bool kSpans>
__device__ __forceinline__ Item item_at(const ScoresParams& p, const Walk<kSpans>& w, int ahead) {
  Item it = place_at(p, w, ahead);
  const int lane = threadIdx.x & 31;
  if (lane < it.count) it.len = p.seq_lens[it.query + lane];
  return it;
}

// The lengths' part of an item. Whole warps call this.
template <bool kSpans>
__device__ __forceinline__ void item_ready(const ScoresParams& p, const Walk<kSpans>& w, Item& it) {
  it.len = clamped(p, it.len);
  it.longest = __reduce_max_sync(0xffffffffu, it.len);
  it.shortest = __reduce_min_sync(0xffffffffu, (threadIdx.x & 31) < it.count ? it.len : INT32_MAX);
  const int32_t tiles = tiles_of(it.longest);
  if constexpr (kSpans) {
    it.first = w.first;
    it.seen = it.end = max(it.first, w.at == w.end ? min(tiles, w.end_tile) : tiles);
  } else {
    it.seen = max(it.first, min(it.end, tiles));
  }
}

// This CTA's span: of all slices' tiles that are seen, in a row, with kItemCost more for each slice that has
// any, its equal share. Every CTA adds up the same lengths by itself. All threads call this; `scratch` is of
// p.slices numbers.
__device__ __forceinline__ void find_span(const ScoresParams& p, Shared& s, int32_t* scratch) {
  const int threads = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int slices = static_cast<int>(p.slices), per = (slices + threads - 1) / threads;
  for (int k = threadIdx.x; k < slices; k += threads) {
    const int32_t tiles = seen_tiles(p, slice_at(p, k));
    scratch[k] = tiles > 0 ? tiles + kItemCost : 0;
  }
  if (threadIdx.x < 2) s.span_slice[threadIdx.x] = s.span_tile[threadIdx.x] = 0;  // no tile at all
  __syncthreads();
  const int begin = min(static_cast<int>(threadIdx.x) * per, slices), end = min(begin + per, slices);
  int32_t mine = 0;
  for (int k = begin; k < end; ++k) mine += scratch[k];
  int32_t sum = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int32_t below = __shfl_up_sync(0xffffffffu, sum, d);
    if (lane >= d) sum += below;
  }
  if (lane == 31) s.warp_sums[warp] = sum;
  __syncthreads();
  int32_t before = sum - mine, total = 0;
  for (int k = 0; k < threads / 32; ++k) {
    const int32_t v = s.warp_sums[k];
    before += k < warp ? v : 0;
    total += v;
  }
  // where the span begins, and where the next one does; the last one ends with the last tile
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int32_t at = static_cast<int32_t>(static_cast<int64_t>(total) * (blockIdx.x + e) / gridDim.x);
    const int32_t look = at < total ? at : total - 1;
    if (look >= before && look < before + mine) {
      int k = begin;
      int32_t rest = look - before;
      while (rest >= scratch[k]) rest -= scratch[k++];
      s.span_slice[e] = k;
      s.span_tile[e] = at < total ? max(rest - kItemCost, 0) : scratch[k] - kItemCost;
    }
  }
  // the copies that reuse the scratch come after these reads
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
}

// With spans: -inf into the tiles that no query of a slice sees. The chip's epilogue warps take blocks of 64
// tiles in turn; a lane looks a block up, the warp fills it.
__device__ __forceinline__ void fill_rest(const ScoresParams& p, int64_t warp, int64_t warps) {
  constexpr int kBlock = 64;
  const int lane = threadIdx.x & 31;
  const float minus_inf = __int_as_float(0xff800000);
  const int64_t blocks = (p.tiles + kBlock - 1) / kBlock, all = p.slices * blocks;
  for (int64_t u0 = warp; u0 < all; u0 += 32 * warps) {
    const int64_t u = u0 + lane * warps;
    Slice r = {};
    int32_t from = 0, to = 0;  // tiles
    if (u < all) {
      const int64_t slice = u / blocks;
      r = slice_at(p, slice);
      const int32_t first = static_cast<int32_t>(u - slice * blocks) * kBlock;
      from = max(first, seen_tiles(p, r));
      to = min(first + kBlock, p.tiles);
    }
    for (uint32_t todo = __ballot_sync(0xffffffffu, from < to); todo != 0u; todo &= todo - 1) {
      const int k = __ffs(todo) - 1;
      const int64_t query = __shfl_sync(0xffffffffu, r.query, k);
      const int32_t count = __shfl_sync(0xffffffffu, r.count, k);
      const int64_t a = static_cast<int64_t>(__shfl_sync(0xffffffffu, from, k)) * kTile;
      const int64_t b = min(static_cast<int64_t>(__shfl_sync(0xffffffffu, to, k)) * kTile, p.row_len);
      for (int g = 0; g < count; ++g) {
        float* out = p.out + (query + g) * p.row_len;
        for (int64_t j = a + lane; j < b; j += 32) out[j] = minus_inf;
      }
    }
  }
}

// The copies of every kLoaders-th tile. kPieces: copies of a tile that a lane may have to issue; or the page
// ids of its one copy, where kGather says that a page is one row.
template <int kGroups, bool kSpans, int kPieces, bool kGather>
__device__ __forceinline__ void load_keys(const ScoresParams& p, Shared& s, const CUtensorMap* key_map,
                                          const CUtensorMap* query_map, int head_rows, int turn) {
  constexpr int kLoaders = Plan<kGroups>::kLoaders;
  static_assert(kKeyStages % kLoaders == 0, "a ring's place belongs to one warp");
  const int lane = threadIdx.x & 31;
  const int pieces = kTile / p.piece_rows;
  const uint32_t piece_bytes = static_cast<uint32_t>(p.piece_rows) * kDim;
  uint32_t tiles = 0, items = 0;  // so far
  uint32_t next_own = turn;       // the running number of this warp's next tile
  bool ok = true;
  Walk<kSpans> w(s);
  Item next_item = item_at(p, w, 0);
  for (; ok && w.more(p); w.on()) {
    Item it = next_item;
    item_ready(p, w, it);
    next_item = item_at(p, w, 1);
    if (it.seen <= it.first) continue;
    if (turn == 0) {
      const int at = items & 1;
      ok = bar_wait(s, &s.query_empty[at], (items >> 1 & 1u) ^ 1u);
      if (!ok) break;
      if (lane == 0) {
        bar_expect(&s.query_full[at], static_cast<uint32_t>(head_rows * p.group) * kDim);
        tma_load_3d(query_map, s.queries[at], &s.query_full[at], 0, 0, static_cast<int>(it.query));
      }
      ++items;
    }
    const int32_t* table = p.page_table + static_cast<int64_t>(it.b) * p.pt_stride;
    int32_t page[kPieces], off[kPieces], next_page[kPieces], next_off[kPieces];
    auto pages_of = [&](int t) {
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int piece = kGather ? kPieces * lane + k : lane + 32 * k;
        const uint32_t row = static_cast<uint32_t>(t) * kTile + piece * p.piece_rows;
        next_page[k] = -1;
        if (t < it.seen && piece < pieces && row < static_cast<uint32_t>(it.longest)) {
          const uint32_t slot = page_of(p, row);
          next_off[k] = static_cast<int32_t>(row - slot * p.page_size);
          next_page[k] = table[slot];
        }
      }
    };
    int t = it.first + static_cast<int>((turn - tiles) % kLoaders);
    pages_of(t);
    for (; t < it.seen; t += kLoaders) {
#pragma unroll
      for (int k = 0; k < kPieces; ++k) page[k] = next_page[k], off[k] = next_off[k];
      pages_of(t + kLoaders);
      uint32_t copies = 0;
#pragma unroll
      for (int k = 0; k < kPieces; ++k)
        copies += __popc(__ballot_sync(0xffffffffu, page[k] >= 0 && page[k] < p.num_pages));
      const uint32_t n = tiles + (t - it.first), at = n % kKeyStages;
      ok = bar_wait(s, &s.key_empty[at], (n / kKeyStages & 1u) ^ 1u);
      if (!ok) break;
      uint64_t* full = &s.key_full[at];
      next_own = n + kLoaders;
      // the phase ends with this arrival and all bytes, in whatever order they come
      if constexpr (kGather) {
        // a key that is past the length or on no page takes row 0, where the cache has one: its score is not used
        if (lane == 0) bar_expect(full, copies > 0 ? kTile * kDim : 0);
        if (copies > 0) {
          int r[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) r[k] = page[k] >= 0 && page[k] < p.num_pages ? page[k] : 0;
          tma_gather4(key_map, s.keys[at] + lane * 4 * kDim, full, r[0], r[1], r[2], r[3]);
        }
      } else {
        if (lane == 0) bar_expect(full, copies * piece_bytes);
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
          if (page[k] >= 0 && page[k] < p.num_pages)
            tma_load_3d(key_map, s.keys[at] + (lane + 32 * k) * piece_bytes, full, 0, off[k], page[k]);
        }
      }
    }
    tiles += it.seen - it.first;
  }
  // no copy outlives the CTA (a place that was never used has not ended a phase, which its other parity says it
  // has)
  for (uint32_t n = next_own; n < next_own + kKeyStages; n += kLoaders)
    bar_drain(&s.key_full[n % kKeyStages], (n / kKeyStages & 1u) ^ 1u);
  if (turn == 0)
    for (uint32_t n = items; n < items + 2; ++n) bar_drain(&s.query_full[n & 1], (n >> 1 & 1u) ^ 1u);
}

// The first tile of an item that is epilogue group `wg`'s, and the step to its next: with two groups every tile
// (two units a tile) or every second one of the launch (one unit a tile), with four every tile.
template <int kGroups>
__device__ __forceinline__ int first_tile(const ScoresParams& p, const Item& it, int wg, uint32_t tiles) {
  return it.first + (kGroups == 2 && p.units == 1 ? static_cast<int>((wg ^ tiles) & 1u) : 0);
}
template <int kGroups>
__device__ __forceinline__ int tile_step(const ScoresParams& p) { return kGroups == 2 ? 3 - p.units : 1; }

// The products of the units of epilogue group `wg` of two; of four groups, of all of them.
template <int kGroups, bool kSpans>
__device__ __forceinline__ void multiply(const ScoresParams& p, Shared& s, uint32_t tmem, int head_rows, int wg) {
  // the TMEM stages of this warp's units: of two, wg, wg + 2, ...
  constexpr uint32_t kStep = Plan<kGroups>::kMultipliers;
  const uint32_t stages = (1u << p.tmem_shift) / kStep, stage_shift = p.tmem_shift - (kStep - 1);
  uint32_t tiles = 0, items = 0, units = 0;  // so far; units: of this warp
  bool ok = true;
  Walk<kSpans> w(s);
  Item next_item = item_at(p, w, 0);
  for (; ok && w.more(p); w.on()) {
    Item it = next_item;
    item_ready(p, w, it);
    next_item = item_at(p, w, 1);
    if (it.seen <= it.first) continue;
    ok = bar_wait(s, &s.query_full[items & 1], items >> 1 & 1u);
    const int u = p.units == 2 ? wg : 0;
    const int queries_here = min(it.count - u * p.unit_queries, p.unit_queries);  // none in the rest of a short group
    // fp32 accumulators, e4m3 operands, both K-major, M = 128
    const uint32_t idesc = (1u << 4) | ((static_cast<uint32_t>(queries_here * head_rows) >> 3) << 17) | ((kTile >> 4) << 24);
    const uint32_t b = matrix_desc(smem_addr(s.queries[items & 1])) + u * (Plan<kGroups>::kColumns * kDim / 16);
    for (int t = first_tile<kGroups>(p, it, wg, tiles); ok && t < it.seen; t += tile_step<kGroups>(p), ++units) {
      const uint32_t n = tiles + (t - it.first), key = n % kKeyStages;
      const uint32_t stage = wg + kStep * (units & (stages - 1)), phase = (units >> stage_shift) & 1u;
      // both barriers at once while neither has to be waited for
      const bool keys_here = bar_try(smem_addr(&s.key_full[key]), n / kKeyStages & 1u);
      const bool stage_free = bar_try(smem_addr(&s.tmem_empty[stage]), phase ^ 1u);
      if (!__all_sync(0xffffffffu, keys_here && stage_free))
        ok = bar_wait(s, &s.key_full[key], n / kKeyStages & 1u) && bar_wait(s, &s.tmem_empty[stage], phase ^ 1u);
      if (!ok) break;
      tmem_fence_after();
      const uint32_t a = matrix_desc(smem_addr(s.keys[key]));
      if (elect_one()) {
        if (queries_here > 0) mma_tile(tmem + stage * p.tmem_stride, a, b, idesc);
        mma_commit(&s.tmem_full[stage]);
        mma_commit(&s.key_empty[key]);
        if (kStep == 2 && p.units == 1) bar_arrive(&s.key_empty[key]);  // for the other warp, which has no unit here
      }
      __syncwarp();
    }
    if (ok && elect_one()) mma_commit(&s.query_empty[items & 1]);
    __syncwarp();
    ++items;
    tiles += it.seen - it.first;
  }
  // no MMA outlives the CTA
  if (elect_one()) mma_commit(&s.drained);
  __syncwarp();
  bar_drain(&s.drained, 0u);
}

// The scales of every kScalers-th unit, kScaleBatch of them at once: the page ids of all of them, then the
// scales, so that each latency is met once in a batch. They go where their unit's products go, to a
// place for each TMEM stage, and share its barriers. A lane brings four neighbouring keys;
// kQuads: they lie on one page.
template <int kGroups, bool kSpans, bool kQuads>
__device__ __forceinline__ void load_scales(const ScoresParams& p, Shared& s, int turn) {
  constexpr int kScalers = Plan<kGroups>::kScalers;
  constexpr int kPages = kQuads ? 1 : 4;
  const int lane = threadIdx.x & 31;
  const int step = kScalers / p.units;                  // tiles from one unit of this warp to its next
  const uint32_t place = p.units == 1 ? turn : turn / 2;  // of this warp's tiles among `step`
  uint32_t tiles = 0;
  Walk<kSpans> w(s);
  Item next_item = item_at(p, w, 0);
  for (; w.more(p); w.on()) {
    Item it = next_item;
    item_ready(p, w, it);
    next_item = item_at(p, w, 1);
    const int32_t* table = p.page_table + static_cast<int64_t>(it.b) * p.pt_stride;
    for (int t = it.first + static_cast<int>((place - tiles) & (step - 1)); t < it.seen; t += kScaleBatch * step) {
      int32_t page[kScaleBatch][kPages];
      uint32_t off[kScaleBatch][kPages];
#pragma unroll
      for (int u = 0; u < kScaleBatch; ++u) {
#pragma unroll
        for (int k = 0; k < kPages; ++k) {
          const int tile = t + u * step;
          const uint32_t j = static_cast<uint32_t>(tile) * kTile + 4 * lane + k;
          off[u][k] = 0xffffffffu;  // past the longest query: never used
          if (tile < it.seen && j < static_cast<uint32_t>(it.longest)) {
            const uint32_t slot = page_of(p, j);
            off[u][k] = j - slot * p.page_size;
            page[u][k] = table[slot];
          }
        }
      }
      uint32_t got[kScaleBatch][4];
#pragma unroll
      for (int u = 0; u < kScaleBatch; ++u) {
#pragma unroll
        for (int k = 0; k < kPages; ++k) {
          const bool inside = off[u][k] != 0xffffffffu && page[u][k] >= 0 && page[u][k] < p.num_pages;
          const float* src = p.scales + (inside ? page[u][k] * p.scale_ps + off[u][k] * p.scale_ts : 0);
          if constexpr (kQuads) {
#pragma unroll
            for (int q = 0; q < 4; ++q) got[u][q] = kNoPage;
            if (inside && p.quads == 2) {
              const uint4 v = *reinterpret_cast<const uint4*>(src);
              got[u][0] = scale_bits(v.x), got[u][1] = scale_bits(v.y), got[u][2] = scale_bits(v.z), got[u][3] = scale_bits(v.w);
            } else if (inside) {
#pragma unroll
              for (int q = 0; q < 4; ++q) got[u][q] = scale_bits(__float_as_uint(src[q * p.scale_ts]));
            }
          } else {
            got[u][k] = kNoPage;
            if (inside) got[u][k] = scale_bits(__float_as_uint(*src));
          }
          if (!inside && off[u][k] != 0xffffffffu) atomicAdd(&g_guard_hits, 1u);
        }
      }
#pragma unroll
      for (int u = 0; u < kScaleBatch; ++u) {
        const int tile = t + u * step;
        if (tile >= it.seen) break;
        const uint32_t unit = (tiles + (tile - it.first)) * p.units + (p.units == 1 ? 0 : turn & 1);
        const uint32_t at = unit & ((1u << p.tmem_shift) - 1);
        bar_pass(s, smem_addr(&s.tmem_empty[at]), (unit >> p.tmem_shift & 1u) ^ 1u);
        *reinterpret_cast<uint4*>(&s.scales[at][4 * lane]) = make_uint4(got[u][0], got[u][1], got[u][2], got[u][3]);
        __syncwarp();
        if (lane == 0) bar_arrive(&s.tmem_full[at]);
      }
    }
    tiles += it.seen - it.first;
  }
}

// What an epilogue warp knows of the tile it works on.
struct Lane {
  float* out;            // this key's score of the warp's first query
  const int32_t* lens;   // of the warp's queries
  uint32_t tmem_empty, next_full, next_phase;  // barriers: to be told that the tile is read; of the next unit
  uint32_t tmem;
  float scale;
  int32_t j, columns;
  bool no_page;          // this key is on none
};

// Columns from C * kLoad on, which are on their way to r. With registers for it (two epilogue groups) the next
// load is sent off before they are summed: 64 or 128 heads 4% faster; of four groups, whose warps hide it from
// one another, after. Whether the next unit is there already: asked before the last sums, for use after them.
template <int kHeads, int kLoad, bool kWhole, int C, int kPairs>
__device__ __forceinline__ bool columns_from(const ScoresParams& p, const Lane& l, const uint64_t (&w)[kPairs],
                                             float (&r)[kLoad], uint64_t acc0, uint64_t acc1) {
  constexpr int kColumns = 2 * kPairs;
  tmem_wait<kLoad>(r);
  auto add = [&]() {
#pragma unroll
    for (int h = 0; h < kLoad / 4; ++h) {
      constexpr int at = C * kLoad / 2;
      acc0 = fma2(pack2(fmaxf(r[4 * h], 0.0f), fmaxf(r[4 * h + 1], 0.0f)), w[at + 2 * h], acc0);
      acc1 = fma2(pack2(fmaxf(r[4 * h + 2], 0.0f), fmaxf(r[4 * h + 3], 0.0f)), w[at + 2 * h + 1], acc1);
    }
    if constexpr ((C + 1) * kLoad % kHeads == 0) {
      constexpr int g = C * kLoad / kHeads;
      const float2 a = unpack2(add2(acc0, acc1));
      const float y = (a.x + a.y) * l.scale;
      float* const out = l.out + g * p.row_len;
      if constexpr (kWhole) {
        *out = l.no_page ? __int_as_float(0xff800000) : y;
      } else if (l.j < p.row_len) {
        *out = l.no_page || l.j >= l.lens[g] ? __int_as_float(0xff800000) : y;
      }
      acc0 = acc1 = 0;
    }
  };
  if constexpr ((C + 1) * kLoad < kColumns) {
    if ((kWhole && kColumns == 64) || (C + 1) * kLoad < l.columns) {
      float next[kLoad];
      if constexpr (kColumns == 64) add();
      tmem_load<kLoad>(l.tmem + (C + 1) * kLoad, next);
      if constexpr (kColumns != 64) add();
      return columns_from<kHeads, kLoad, kWhole, C + 1>(p, l, w, next, acc0, acc1);
    }
  }
  // every column of the tile is in registers: its stage is free
  tmem_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) bar_arrive(l.tmem_empty);
  const bool ready = bar_test(l.next_full, l.next_phase);
  add();
  return ready;
}

// One epilogue warp: relu, weights and the sum over heads of its 32 lanes (keys), for its group's units or columns.
// kHeads: columns of a query.
template <int kGroups, bool kSpans, int kHeads>
__device__ __forceinline__ void reduce(const ScoresParams& p, Shared& s, uint32_t tmem, int wg) {
  constexpr int kLoad = 16;                         // columns of a load
  constexpr int kColumns = Plan<kGroups>::kColumns;
  constexpr int kQueries = kColumns / kHeads;       // queries of a group's columns at most
  constexpr int kBring = kColumns / 32;             // weights that a lane brings
  const int tid = threadIdx.x & 127, lane = tid & 31, warp = threadIdx.x / 32 - kFirstWarp<kGroups>;
  float* const weights = s.weights + warp * kColumns;
  const float minus_inf = __int_as_float(0xff800000);
  const int first = kGroups == 4 || p.units == 2 ? wg * kQueries : 0;  // of this warp's queries in a group of queries
  float bring[kBring];
  auto weights_of = [&](const Item& it) {
    const float* src = p.weights + (it.query + first) * p.heads;
#pragma unroll
    for (int k = 0; k < kBring; ++k) {
      const int g = (lane + 32 * k) / kHeads, h = (lane + 32 * k) % kHeads;
      bring[k] = first + g < it.count && h < p.heads ? src[g * p.heads + h] : 0.0f;
    }
  };
  Lane l;
  const uint32_t tmem_lane = tmem + (static_cast<uint32_t>(tid & ~31) << 16) + (kGroups == 4 ? wg * kColumns : 0);
  // the group's TMEM stages: of two groups wg, wg + 2, ..., of four all of them
  constexpr uint32_t kStep = kGroups == 2 ? 2 : 1;
  const uint32_t stages = 1u << p.tmem_shift, first_stage = kGroups == 2 ? wg : 0;
  const uint32_t full_base = smem_addr(s.tmem_full), empty_base = smem_addr(s.tmem_empty);
  uint32_t tiles = 0, stage = first_stage, phase = 0;
  bool ready = false;
  Walk<kSpans> walk(s);
  int32_t next_len;  // the rest of the next item's place is worked out again: registers are short while tiles go by
  {
    const Item it = item_at(p, walk, 0);
    next_len = it.len;
    weights_of(it);
  }
  for (; walk.more(p); walk.on()) {
    Item it = place_at(p, walk, 0);
    it.len = next_len;
    item_ready(p, walk, it);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kBring; ++k) weights[lane + 32 * k] = bring[k];
    if (lane < it.count) s.lens[warp][lane] = it.len;
    __syncwarp();
    uint64_t w[kColumns / 2];  // in pairs
#pragma unroll
    for (int k = 0; k < kColumns / 4; ++k) {
      const ulonglong2 f = reinterpret_cast<const ulonglong2*>(weights)[k];
      w[2 * k] = f.x, w[2 * k + 1] = f.y;
    }
    const int count = min(max(it.count - first, 0), kQueries);
    l.columns = count * kHeads;
    // every query of the group sees every key of the tiles that start here or before; of four groups, if all
    // its columns are in use: no look at their number at each load (2048 queries of 16 heads 4% faster)
    const int whole = kGroups == 4 && count < kQueries ? -1 : it.shortest - kTile;
    l.lens = s.lens[warp] + first;
    const Item next_item = item_at(p, walk, 1);
    next_len = next_item.len;
    weights_of(next_item);  // on their way while this item is worked on
    // The output's place goes on from tile to tile: worked out at each from a row's start, 2048 queries took 7%
    // longer.
    const int step = tile_step<kGroups>(p), t0 = first_tile<kGroups>(p, it, wg, tiles);
    l.out = p.out + (it.query + first) * p.row_len + static_cast<int64_t>(t0) * kTile + tid;
    for (int t = t0; t < it.seen; t += step, l.out += step * kTile) {
      const uint32_t at = stage, full = full_base + 8 * stage;
      l.tmem_empty = empty_base + 8 * stage;
      if (!ready) bar_pass(s, full, phase);
      tmem_fence_after();
      stage += kStep;
      if (stage >= stages) {
        stage = first_stage;
        phase ^= 1u;
      }
      ready = false;
      if (count == 0) {
        if (lane == 0) bar_arrive(l.tmem_empty);
        continue;
      }
      l.tmem = tmem_lane + at * p.tmem_stride;
      float r[kLoad];
      tmem_load<kLoad>(l.tmem, r);
      l.scale = s.scales[at][tid];
      l.j = t * kTile + tid;
      l.no_page = __float_as_uint(l.scale) == kNoPage;
      l.next_full = full_base + 8 * stage;
      l.next_phase = phase;
      const bool next = t * kTile <= whole ? columns_from<kHeads, kLoad, true, 0>(p, l, w, r, 0, 0)
                                           : columns_from<kHeads, kLoad, false, 0>(p, l, w, r, 0, 0);
      ready = __all_sync(0xffffffffu, next);
    }
    tiles += it.seen - it.first;
    if constexpr (kSpans) continue;  // fill_rest's
    // tiles that no query of the group sees
    const bool in_turn = kGroups == 2 && p.units == 1;
    float* const out = p.out + (it.query + first) * p.row_len;
    for (int t = it.seen + (in_turn ? wg : 0); t < it.end; t += in_turn ? 2 : 1) {
      const int64_t j = static_cast<int64_t>(t) * kTile + tid;
      if (j < p.row_len)
        for (int g = 0; g < count; ++g) out[g * p.row_len + j] = minus_inf;
    }
  }
}

// After a wait that ran out: NaN in place of every score that this epilogue warp has written. What is wrong
// among them was read after the wait's end was noted. Out of line, as no sound call comes here: inline, one
// decode row's kernel took 3.95 us instead of 3.73.
template <int kGroups, bool kSpans>
__device__ __noinline__ void give_up(const ScoresParams& p, const Shared& s, int head_rows, int wg) {
  const int tid = threadIdx.x & 127, queries = Plan<kGroups>::kColumns / head_rows;
  const int first = kGroups == 4 || p.units == 2 ? wg * queries : 0;
  uint32_t tiles = 0;
  if (p.fail != 0 && tid == 0) atomicAdd(&g_guard_hits, 1u);
  for (Walk<kSpans> walk(s); walk.more(p); walk.on()) {
    Item it = item_at(p, walk, 0);
    item_ready(p, walk, it);
    const int64_t query = it.query + first;
    for (int g = 0; g < min(it.count - first, queries); ++g) {
      const int32_t len = clamped(p, p.seq_lens[query + g]);
      for (int t = first_tile<kGroups>(p, it, wg, tiles); t < it.seen; t += tile_step<kGroups>(p)) {
        const int32_t j = t * kTile + tid;
        if (j < len) p.out[(query + g) * p.row_len + j] = __uint_as_float(kNan);
      }
    }
    tiles += it.seen - it.first;
  }
}

template <int kRegisters>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegisters));
}
template <int kRegisters>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegisters));
}

// NaN in place of every score of a launch that cannot start; out of line too.
__device__ __noinline__ void spoil(const ScoresParams& p) {
  begin_after_prior_grids();
  const int64_t all = p.slices / p.groups * p.queries * p.row_len, step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < all; i += step)
    p.out[i] = __uint_as_float(kNan);
}

// Whether the dynamic shared memory starts where its declared alignment says, which the swizzled tiles rely on.
// Without a rounding of its address every place in it is a constant, and the registers that held addresses are
// the epilogue's (2048 queries over 32768 keys, 64 heads: 548 -> 512 us). If it ever starts elsewhere, all
// scores are NaN, and counted.
__device__ __forceinline__ bool aligned_base(const ScoresParams& p, const Shared& s) {
  uint32_t base = smem_addr(&s);
  asm volatile("" : "+r"(base));
  if (__builtin_expect(base % 1024 == 0 && p.fail != 2, 1)) return true;
  if (threadIdx.x == 0) atomicAdd(&g_guard_hits, 1u);
  spoil(p);
  return false;
}

// kHeads: heads rounded up to 16, 32, 64 or 128. The rounding's rows of B are zeros (beyond the
// tensor map's heads) and their weights are 0.
template <int kGroups, bool kSpans, int kHeads>
__global__ void __launch_bounds__(kThreads<kGroups>, 1)
    scores_kernel(const __grid_constant__ ScoresParams p, const __grid_constant__ CUtensorMap key_map,
                  const __grid_constant__ CUtensorMap query_map) {
  using P = Plan<kGroups>;
  extern __shared__ __align__(1024) uint8_t raw[];
  Shared& s = *reinterpret_cast<Shared*>(raw);
  if (!aligned_base(p, s)) return;
  const int warp = threadIdx.x / 32;
  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&key_map) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&query_map) : "memory");
    for (int i = 0; i < kKeyStages; ++i) {
      bar_init(&s.key_full[i], 1);
      bar_init(&s.key_empty[i], P::kMultipliers);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&s.query_full[i], 1);
      bar_init(&s.query_empty[i], P::kMultipliers);
    }
    for (int i = 0; i < kMaxTmemStages; ++i) {
      bar_init(&s.tmem_full[i], 2);  // the products and the scales
      bar_init(&s.tmem_empty[i], kGroups == 2 ? 4 : 16);  // the warps that read it
    }
    bar_init(&s.drained, P::kMultipliers);
    s.aborted = p.fail;
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
  if constexpr (kSpans) find_span(p, s, reinterpret_cast<int32_t*>(s.keys));

  if (warp < kFirstWarp<kGroups>) {
    fewer_registers<P::kFewRegisters>();
    if (warp < P::kLoaders && p.page_size == 1)
      load_keys<kGroups, kSpans, 4, true>(p, s, &key_map, &query_map, kHeads, warp);
    else if (warp < P::kLoaders && p.piece_rows >= 4)
      load_keys<kGroups, kSpans, 1, false>(p, s, &key_map, &query_map, kHeads, warp);
    else if (warp < P::kLoaders)
      load_keys<kGroups, kSpans, 4, false>(p, s, &key_map, &query_map, kHeads, warp);
    else if (warp < P::kLoaders + P::kMultipliers)
      multiply<kGroups, kSpans>(p, s, tmem, kHeads, warp - P::kLoaders);
    else if (p.quads != 0)
      load_scales<kGroups, kSpans, true>(p, s, warp - P::kLoaders - P::kMultipliers);
    else
      load_scales<kGroups, kSpans, false>(p, s, warp - P::kLoaders - P::kMultipliers);
  } else {
    more_registers<P::kManyRegisters>();
    if constexpr (kSpans)  // while the first tiles are on their way
      fill_rest(p, static_cast<int64_t>(warp - kFirstWarp<kGroups>) * gridDim.x + blockIdx.x, 4 * kGroups * static_cast<int64_t>(gridDim.x));
    reduce<kGroups, kSpans, kHeads>(p, s, tmem, (warp - kFirstWarp<kGroups>) / 4);
    if (__builtin_expect(*const_cast<volatile int32_t*>(&s.aborted) != 0, 0))
      give_up<kGroups, kSpans>(p, s, kHeads, (warp - kFirstWarp<kGroups>) / 4);
  }

  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemColumns));
}

constexpr size_t kSmemBytes = sizeof(Shared);

std::atomic<int> g_fail{0};

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

// A map of rows of 128 bytes on one or two outer axes (`axes`), copied `box1` by `box2` rows at once.
cudaError_t row_map(EncodeTiled encode, CUtensorMap* map, int axes, const uint8_t* base, int64_t n1, int64_t stride1,
                    int64_t n2, int64_t stride2, int box1, int box2) {
  const cuuint64_t dims[3] = {kDim, static_cast<cuuint64_t>(n1), static_cast<cuuint64_t>(n2)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(stride1), static_cast<cuuint64_t>(stride2)};
  const cuuint32_t box[3] = {kDim, static_cast<cuuint32_t>(box1), static_cast<cuuint32_t>(box2)};
  const cuuint32_t steps[3] = {1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1 + axes, const_cast<uint8_t*>(base), dims, strides, box, steps,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int kGroups, bool kSpans, int kHeads>
cudaError_t launch_scores(ScoresParams p, const CUtensorMap& key_map, const CUtensorMap& query_map, unsigned grid,
                          cudaStream_t stream) {
  // set once for each device and kernel: the attribute belongs to the function on that device
  static std::atomic<uint64_t> prepared{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev > 63 || (prepared.load(std::memory_order_acquire) >> dev & 1u) == 0) {
    e = cudaFuncSetAttribute(scores_kernel<kGroups, kSpans, kHeads>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmemBytes));
    if (e != cudaSuccess) return e;
    if (dev <= 63) prepared.fetch_or(uint64_t(1) << dev, std::memory_order_release);
  }
  return launch(scores_kernel<kGroups, kSpans, kHeads>, grid, kThreads<kGroups>, kSmemBytes, stream, p, key_map, query_map);
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
  p.page_div = divisor(p.page_size);
  p.quads = p.page_size % 4 != 0 ? 0
            : p.scale_ts == 1 && p.scale_ps % 4 == 0 && (reinterpret_cast<uintptr_t>(p.scales) & 15u) == 0 ? 2 : 1;
  p.queries = queries;
  p.heads = heads;
  p.fail = g_fail.load(std::memory_order_relaxed);
  const int head_rows = heads <= 16 ? 16 : heads <= 32 ? 32 : heads <= 64 ? 64 : 128;
  p.group = kMaxColumns / head_rows < queries ? kMaxColumns / head_rows : queries;
  p.groups = (queries + p.group - 1) / p.group;
  p.tiles = static_cast<int32_t>((row_len + kTile - 1) / kTile);
  // Groups of queries of more than 128 columns, in columns of 16, 32 or 64 a query: four epilogue groups, a
  // quarter of a tile's columns each, and one unit a tile; otherwise two, and units of up to 128 columns. (2048
  // queries over 32768 keys, 64 heads: 511 us with four, 540 with two; 64 rows of 4 queries: 83.2 against 83.8.)
  const int columns = p.group * head_rows;
  const int epilogues = columns > 128 && head_rows <= 64 ? 4 : 2;
  p.unit_queries = epilogues == 4 ? p.group : Plan<2>::kColumns / head_rows;
  p.units = p.group > p.unit_queries ? 2 : 1;
  // TMEM stages of 32 columns or a larger power of two: 2 of 256, or 4 or 8
  p.tmem_stride = 32;
  while (p.tmem_stride < columns / p.units) p.tmem_stride *= 2;
  p.tmem_shift = p.tmem_stride == 256 ? 1 : p.tmem_stride == 128 ? 2 : 3;
  // Tiles of an item: what takes the SM with the most items the least time when every row is full, an
  // item's start counted as kItemCost tiles.
  p.slices = static_cast<int64_t>(batch) * p.groups;
  int64_t best = INT64_MAX;
  for (int32_t chunk = 1; chunk <= kMaxChunk && chunk <= p.tiles; ++chunk) {
    const int64_t items = p.slices * ((p.tiles + chunk - 1) / chunk), cost = (items + sms - 1) / sms * (chunk + kItemCost);
    if (cost < best) best = cost, p.chunk = chunk;
  }
  p.items = p.slices * ((p.tiles + p.chunk - 1) / p.chunk);
  // Equal spans of the tiles that are seen, whatever the lengths, instead of items in turn: adding the lengths
  // up costs 1.7 us, so from 32 tiles an SM on, were all rows full, and from more with more slices than a CTA's
  // threads read at once. Lengths even over the range: 64 rows of up to 32768 keys 31 against 39 us, 256 rows 103
  // against 137, 8 of up to 262144 22 against 33 (48 of up to 8192, 20 tiles an SM, which take items in turn:
  // 11.2 against 10.7). Prompts, whose later queries see more, gain too: 2048 queries 512 against 529. Full rows
  // lose: 64 of 32768 keys 52.7 against 50.9, 4 of 262144 31.4 against 28.7; 256 of 32768 are even at 178.
  const bool spans = p.slices <= kMaxSpanSlices && p.slices * (p.tiles + kItemCost) <= INT32_MAX &&
                     p.slices * p.tiles >= int64_t(sms) * (32 + p.slices / 64);

  CUtensorMap key_map, query_map;
  // a cache of no pages has none that passes the kernel's check: its map is never used
  if (cache->num_pages == 0) e = row_map(encode, &key_map, 2, q, 1, kDim, 1, kDim, 1, 1);
  else if (cache->page_size == 1) e = row_map(encode, &key_map, 1, cache->codes, cache->num_pages, code_ps, 1, kDim, 1, 1);
  else e = row_map(encode, &key_map, 2, cache->codes, cache->page_size, code_ts, cache->num_pages, code_ps, p.piece_rows, 1);
  if (e == cudaSuccess)
    e = row_map(encode, &query_map, 2, q, heads, kDim, static_cast<int64_t>(batch) * queries,
                static_cast<int64_t>(heads) * kDim, head_rows, p.group);
  if (e != cudaSuccess) return status_of(e);
  const unsigned grid = static_cast<unsigned>(!spans && p.items < sms ? p.items : sms);
  auto run = [&](auto plan, auto rows) {
    constexpr int kGroups = decltype(plan)::value, kHeads = decltype(rows)::value;
    return spans ? launch_scores<kGroups, true, kHeads>(p, key_map, query_map, grid, stream)
                 : launch_scores<kGroups, false, kHeads>(p, key_map, query_map, grid, stream);
  };
  using std::integral_constant;
  if (epilogues == 4) {
    constexpr integral_constant<int, 4> plan;
    e = head_rows == 16   ? run(plan, integral_constant<int, 16>())
        : head_rows == 32 ? run(plan, integral_constant<int, 32>())
                          : run(plan, integral_constant<int, 64>());
  } else {
    constexpr integral_constant<int, 2> plan;
    e = head_rows == 16   ? run(plan, integral_constant<int, 16>())
        : head_rows == 32 ? run(plan, integral_constant<int, 32>())
        : head_rows == 64 ? run(plan, integral_constant<int, 64>())
                          : run(plan, integral_constant<int, 128>());
  }
  return status_of(e);
}

extern "C" int indexer_set_scores_failure(int mode) {
  return indexer_gb300::g_fail.exchange(mode == 1 || mode == 2 ? mode : 0, std::memory_order_relaxed);
}
