// Attention over a block-scaled cache for more query rows on the same keys than one warp's registers take (prompts,
// drafted tokens, many query heads on one head of keys); the mathematics is that of indexer_attention.cu.
//
// Both products run on tcgen05 with query rows as the 128 lanes of TMEM:
// - q . k: the keys' codes are an operand as they are (kind::f8f6f4). A query row, scaled by a power of two that brings its
//   largest value to [2^7, 2^8), is the sum of two (bf16) or three (fp16) e4m3 numbers: all bits of values down to 2^-9 (bf16) or
//   2^-6 (fp16) of 2^7, where e4m3's last step, 2^-9, is their own last bit, and to within 2^-17 of the largest value below. Sums
//   are in fp32; the products of the parts add up in TMEM.
// - weights . v: the weights are fp16, in TMEM over the logits that they come from; the values' codes become fp16 in
//   shared memory, as many bits as they have. The tensor cores would take their codes too, but weights of 4 bits lose what many
//   small ones add up to.
// A CTA, one an SM, has
//   8 softmax warps    two streams of 128 rows, each with logits, weights and sums in TMEM; a thread owns a row
//   8 loader warps     a quarter of every second tile of keys each: their places, copies of the keys' codes, values
//                      converted; and the queries of the next tile of rows. None of them waits for another.
//   2 multipliers      tcgen05.mma, one for each stream
// A tile of 128 keys is worked on in two halves: while a stream's weights of one half are made, the other half's
// products run. Logits and weights of a half share their columns of TMEM, of which none are left.
// With more than 128 rows the streams are two tiles of rows on the same keys. With fewer they are one tile on every
// second tile of 128 keys each, and are joined at the tile's end. Of 64 rows and fewer each has two of a stream's lanes, with
// 32 keys of a half each and weights of zero for the other's (64 sequences of up to 8192 keys, 64 query heads on each of 8: 289 us
// when it was taken, 324 with one lane and half of the softmax threads without work; 278 now).
// What bounds it: a prompt's chunk (1024 queries behind 15360 keys, 8 heads, 4 query heads on each; 140 us of products at the
// measured rate) takes 359 us. No pipe is full: of a smaller chunk 37% of the issue slots are taken, the tensor pipe is busy 24%
// of the time, ALU 27%, exponentials 12%. Eight softmax warps, two a scheduler, each wait for their own logits from TMEM, compute,
// store weights and wait for the store, 32 logits at a time, with nothing of the next ones under way. Few rows wait for the loaders
// too, 8 warps that send copies, wait, and convert: 16 sequences of up to 16384 keys, 35 rows on each of 4 heads, 68 us. Copies
// sent a tile ahead held up the softmax's own loads behind them in the queue (100 us), with values' codes in registers or by way
// of shared memory.
// Every wait has a limit (2.6 s in all); after it the roles run through to their end, in bounds, and give NaN.

#include <algorithm>
#include <atomic>

#include "indexer_attention.cuh"

namespace indexer_gb300 {
namespace {

constexpr int kDim = 128;            // columns of a row: the cache's, and zeros
constexpr int kTile = 128;           // keys of a tile; rows of a stream
constexpr int kHalf = kTile / 2;     // keys whose logits are made, and held, at once
constexpr int kSoftmaxWarps = 8, kLoaderWarps = 8;
constexpr int kThreads = 32 * (kSoftmaxWarps + kLoaderWarps + 4);  // 2 multipliers, 2 that only give their registers
constexpr int kSoftmaxThreads = 32 * kSoftmaxWarps;
constexpr int kQuarter = kTile / 4;  // keys of a loader's part
constexpr int kValueStages = 2;
constexpr int kTmemColumns = 512;
constexpr int kWaitLimit = 1 << 17;      // tries of a wait before it is given up,
constexpr uint32_t kWaitNs = 20000;      // each of which may sleep this long: 2.6 s in all
// Registers of a thread: of the 640 * 96 of a launch, 256 * 120 + 256 * 96 + 128 * 40 = 60416; the loaders keep theirs (a
// prompt's chunk 353 us when they were taken; with 136 and 80 365, with 104 and 112 363).
constexpr int kSoftmaxRegisters = 120, kOtherRegisters = 40;

constexpr int kJoinWidth = 36;           // eight lanes' pieces on different banks
// Pages and slots outside the cache that were met, and waits that ran out (see indexer_guard_hits).
__device__ unsigned int g_guard_hits;

// kParts: e4m3 numbers of a query value. kTileRows: query rows of a tile of the work.
template <int kParts, int kTileRows> struct Plan {
  static constexpr int kRows = kTileRows;
  static constexpr bool kPair = kRows == 2 * kTile;                  // the streams are two tiles of 128 rows
  static constexpr int kSpread = kTile / kRows > 1 ? 2 : 1;          // lanes of a row in a stream, each with its part of the keys
  static_assert(kRows == kTile / 2 || kRows == kTile || kRows == 2 * kTile, "rows of a tile");
  static constexpr int kOwn = kHalf / kSpread;                       // keys of a half that a softmax thread has
  static constexpr int kKeys = kPair ? kTile : 2 * kTile;            // keys of a step of it
  static constexpr int kQueryBuffers = kPair || kParts == 3 ? 1 : 2;
  static constexpr int kQueryTiles = kPair ? 2 : 1;
  static constexpr int kKeyStages = kPair && kParts == 3 ? 2 : 4;    // what shared memory holds, an even number
  static constexpr int64_t kPartial = static_cast<int64_t>(kRows) * (kDim + 2);
};

// Where the n-th tile of keys of a stream lies, and which use of its places that is. A barrier's parity tells a phase from
// the next one alone, so whoever waits for a barrier has to wait for each of its phases: streams on the same tiles
// share both rings, streams on tiles of their own have a half of each.
template <typename P> struct Ring {
  uint32_t key, key_use, value, value_use;
  __device__ __forceinline__ Ring(int stream, uint32_t n) {
    if constexpr (P::kPair) {
      key = n % P::kKeyStages, key_use = n / P::kKeyStages;
      value = n % kValueStages, value_use = n / kValueStages;
    } else {
      constexpr uint32_t kOwn = P::kKeyStages / 2;
      key = stream * kOwn + n % kOwn, key_use = n / kOwn;
      value = stream, value_use = n;
    }
  }
};

template <int kParts, int kTileRows> struct Shared {
  using P = Plan<kParts, kTileRows>;
  alignas(1024) uint8_t queries[P::kQueryBuffers][P::kQueryTiles][kParts][kTile * kDim];
  alignas(1024) uint8_t keys[P::kKeyStages][kTile * kDim];
  alignas(1024) uint8_t values[kValueStages][2][kTile * 128];  // fp16, 64 columns each
  alignas(16) float key_scales[kValueStages][kTile], logs[kValueStages][kTile], inverses[kValueStages][kTile];
  alignas(16) uint32_t present[kValueStages][4];
  uint32_t uniform[kValueStages][4];                           // 32 keys there and with the same scales
  uint32_t clean[kValueStages][4];                             // keys there without a NaN among their value's codes
  alignas(16) uint32_t nan_columns[2][kTile][4];               // of rows that see such a key: see mark_columns
  float factors[4][2 * kTile];  // of four items: read until an item's last weights are made
  float2 stats[2][2][kTile];
  float joined[P::kSpread > 1 ? kTile : 1][kJoinWidth];        // 32 columns of the sums that make a row
  uint64_t key_full[P::kKeyStages], key_empty[P::kKeyStages], value_full[kValueStages], value_empty[kValueStages];
  uint64_t query_full[2], query_empty[2];
  uint64_t logits_full[2][2], weights_full[2][2], sums_full[2][2];  // of a stream's halves of a tile
  uint64_t sums_empty[2];
  uint64_t drained[2];
  Spans span;
  int64_t span_sums[kThreads / 32];
  uint32_t tmem_base;
  int32_t aborted;
};

__device__ __forceinline__ void bar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\n"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n"
      "selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity & 1u), "r"(kWaitNs)
      : "memory");
  return ok != 0u;
}

// Waits for the end of the phase with this parity. After a wait of the CTA ran out every wait returns at once, false.
__device__ __forceinline__ bool bar_wait(int32_t* aborted, uint64_t* bar, uint32_t parity) {
  for (int i = 0; i < kWaitLimit; ++i) {
    if (bar_try(bar, parity)) return true;
    if (*const_cast<volatile int32_t*>(aborted) != 0) return false;
  }
  if (atomicExch(aborted, 1) == 0) atomicAdd(&g_guard_hits, 1u);
  return false;
}

template <int kThreadsThere>
__device__ __forceinline__ void named_barrier(int id) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(kThreadsThere) : "memory");
}

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0u;
}

__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Descriptors of 128-byte swizzled rows of 128 bytes, groups of 8 rows 1024 bytes apart: the high word, and the low one with
// `next`, the bytes from one block of 64 columns to the next, where the columns are not what is summed over.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t matrix_desc(uint32_t addr, uint32_t next) { return ((addr & 0x3ffffu) >> 4) | (next >> 4) << 16; }

// d (+)= a b over 32 columns of codes; a, b: low words of descriptors.
__device__ __forceinline__ void mma_codes(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 x, y;\nsetp.ne.u32 p, %4, 0;\nmov.b64 x, {%1, %5};\nmov.b64 y, {%2, %5};\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(add), "r"(kDescHigh)
      : "memory");
}
// d (+)= a b over 16 keys; a: TMEM.
__device__ __forceinline__ void mma_halves(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 y;\nsetp.ne.u32 p, %4, 0;\nmov.b64 y, {%2, %5};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(add), "r"(kDescHigh)
      : "memory");
}

// 32 consecutive columns of this thread's lane; tmem_wait completes the loads before their values may be used.
__device__ __forceinline__ void tmem_load(uint32_t addr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]), "=f"(r[17]),
        "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]), "=f"(r[25]), "=f"(r[26]),
        "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(addr));
}
template <int N>
__device__ __forceinline__ void tmem_wait(float (&r)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(r[i]));
}
__device__ __forceinline__ void tmem_store(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr), "r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ uint32_t codes_of(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The tiles of keys of one tile of rows and head that lie in this CTA's span.
struct Item {
  int32_t slice, list, head, r0;       // r0: its first row of the list's
  int32_t first, tiles, longest;       // of keys
  int32_t steps_here, steps;
  bool from_start, to_end;
};

// Every role walks over the same items.
template <typename P> struct Walk {
  Cursor c;
  __device__ __forceinline__ void enter(const AttendParams& p) {
    c.list = c.slice / p.tiles;
    c.longest = p.seq_lens == nullptr
                    ? p.row_len
                    : max(__reduce_max_sync(0xffffffffu, longest_of(p, c.slice, P::kRows, threadIdx.x & 31, 32)), 0);
    c.steps = steps_of(c.longest, P::kKeys);
  }
  __device__ __forceinline__ Walk(const AttendParams& p, const Spans& s) {
    c.left = s.at[1] - s.at[0];
    c.slice = s.slice[0];
    enter(p);
    c.head = static_cast<int32_t>(s.rest[0] / c.steps);
    c.step = static_cast<int32_t>(s.rest[0] - static_cast<int64_t>(c.head) * c.steps);
  }
  __device__ __forceinline__ bool more() const { return c.left > 0; }
  // The next item; the walk goes on behind it.
  __device__ __forceinline__ Item take(const AttendParams& p) {
    Item it;
    it.slice = c.slice, it.list = c.list, it.head = c.head, it.longest = c.longest, it.steps = c.steps;
    it.r0 = (c.slice - c.list * p.tiles) * P::kRows;
    it.steps_here = static_cast<int32_t>(min(static_cast<int64_t>(c.steps - c.step), c.left));
    it.from_start = c.step == 0;
    it.to_end = c.step + it.steps_here == c.steps;
    constexpr int kPer = P::kKeys / kTile;
    it.first = c.step * kPer;
    it.tiles = min(it.first + it.steps_here * kPer, steps_of(c.longest, kTile)) - it.first;
    c.left -= it.steps_here;
    c.step += it.steps_here;
    if (c.step == c.steps && c.left > 0) {
      c.step = 0;
      if (++c.head == p.kv_heads) {
        c.head = 0;
        ++c.slice;
        enter(p);
      }
    }
    return it;
  }
};

// ---------------------------------------------------------------- the multipliers

template <int kParts, int kTileRows>
__device__ __forceinline__ void multiply(const AttendParams& p, Shared<kParts, kTileRows>& s, uint32_t tmem, int st) {
  using P = Plan<kParts, kTileRows>;
  // fp32 sums, M = 128: e4m3 operands with the columns summed over in a row, N = 64 keys; fp16 with the rows of B summed
  // over, N = 128 columns
  constexpr uint32_t kSums = 1u << 4 | (kTile / 16) << 24;
  constexpr uint32_t kCodes = kSums | (kHalf / 8) << 17, kHalves = kSums | 1u << 16 | (kDim / 8) << 17;
  const uint32_t logits = tmem + st * kTile, sums = tmem + (2 + st) * kTile;
  uint32_t items = 0, units = 0;  // so far; units: tiles of this stream
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) { ok = ok && __all_sync(0xffffffffu, bar_wait(&s.aborted, bar, parity)); };
  constexpr bool kPair = P::kPair;
  constexpr int kStep = kPair ? 1 : 2;
  const int first = kPair ? 0 : st;
  Walk<P> walk(p, s.span);
  for (; ok && walk.more(); ++items) {
    const Item it = walk.take(p);
    const uint32_t buffer = items % P::kQueryBuffers;
    const uint32_t a = matrix_desc(smem_addr(s.queries[buffer][kPair ? st : 0][0]), 16);
    wait(&s.query_full[buffer], items / P::kQueryBuffers);
    if (first >= it.tiles) {  // nothing for this stream
      if (elect_one()) mma_commit(&s.query_empty[buffer]);
      __syncwarp();
      if (items > 0) wait(&s.sums_empty[st], items - 1);
    }
    // the logits of half h of tile t, the stream's n-th
    auto ask = [&](int t, uint32_t n, int h) {
      const Ring<P> ring(st, n);
      const uint32_t key = ring.key;
      if (h == 0) wait(&s.key_full[key], ring.key_use);
      if (n > 0) wait(&s.sums_full[st][h], n - 1);  // the weights that the logits go over have been used
      if (!ok) return;
      tmem_fence_after();
      if (elect_one()) {
        const uint32_t b = matrix_desc(smem_addr(s.keys[key]) + h * kHalf * kDim, 16);
#pragma unroll
        for (int part = 0; part < kParts; ++part)
#pragma unroll
          for (int k = 0; k < kDim / 32; ++k)
            mma_codes(logits + h * kHalf, a + part * (kTile * kDim / 16) + 2 * k, b + 2 * k, kCodes, part > 0 || k > 0 ? 1u : 0u);
        mma_commit(&s.logits_full[st][h]);
        if (h == 0) bar_arrive(&s.logits_full[st][h]);  // the queries' barrier is behind it
        if (h == 1) {
          mma_commit(&s.key_empty[key]);
          if (t + kStep >= it.tiles) mma_commit(&s.query_empty[buffer]);
        }
      }
      __syncwarp();
    };
    if (first < it.tiles) {
      ask(first, units, 0);
      ask(first, units, 1);
    }
    for (int t = first; ok && t < it.tiles; t += kStep) {
      const Ring<P> ring(st, units);
      const uint32_t stage = ring.value;
      ++units;
#pragma unroll 1
      for (int h = 0; ok && h < 2; ++h) {
        if (h == 0) {
          wait(&s.value_full[stage], ring.value_use);
          if (t == first && items > 0) wait(&s.sums_empty[st], items - 1);
        }
        wait(&s.weights_full[st][h], units - 1);
        if (!ok) break;
        tmem_fence_after();
        if (elect_one()) {
          const uint32_t b = matrix_desc(smem_addr(s.values[stage]) + h * kHalf * 128, kTile * 128);
#pragma unroll
          for (int k = 0; k < kHalf / 16; ++k)
            mma_halves(sums, logits + h * kHalf + 8 * k, b + k * (16 * 128 / 16), kHalves, k > 0 || h > 0 || t > first ? 1u : 0u);
          mma_commit(&s.sums_full[st][h]);
          if (h == 1) mma_commit(&s.value_empty[stage]);
        }
        __syncwarp();
        if (t + kStep < it.tiles) ask(t + kStep, units, h);
      }
    }
  }
  // no MMA outlives the CTA
  if (elect_one()) mma_commit(&s.drained[st]);
  __syncwarp();
  for (int i = 0; i < 256 && !bar_try(&s.drained[st], 0); ++i) {
  }
  __syncwarp();
}

// ---------------------------------------------------------------- the loaders

// The fp16 number that stands for a NaN code among the values: the largest one, no code's. A row that does not see the key adds it
// with a weight of 0; of a row that does, the column becomes NaN at the item's end.
constexpr uint32_t kNanMark = 0x7bffu;
// Two values that were codes, with the mark for each NaN (all bits below the sign).
__device__ __forceinline__ uint32_t marked(uint32_t two) {
  const uint32_t nan = ((two & 0x7fff7fffu) + 0x00010001u) & 0x80008000u;
  return two & ~(nan | nan >> 5);
}

// 16 bytes that leave no line in L1, of which shared memory leaves little (a prompt's chunk 374 -> 360 us).
__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

// Rows [first, first + 4 * step) of an item's queries, `step` apart, by a warp: each as kParts e4m3 numbers a value.
template <int kParts, int kTileRows>
__device__ __forceinline__ void put_queries(const AttendParams& p, Shared<kParts, kTileRows>& s, const Item& it, uint32_t item, int first,
                                            int step) {
  using P = Plan<kParts, kTileRows>;
  constexpr int kBatch = 4;
  constexpr int kSpread = P::kSpread;
  const int lane = threadIdx.x & 31;
  const int32_t group = static_cast<int32_t>(p.group.d), rows_of_list = p.list_queries * group;
  uint2 got[kBatch];
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    const int32_t r = it.r0 + first + i * step;
    got[i] = make_uint2(0, 0);
    if (first + i * step < P::kRows && r < rows_of_list && 4 * lane < p.dim) {
      const int32_t n = quotient(p.group, r);
      const int64_t row = (static_cast<int64_t>(it.list) * p.list_queries + n) * p.heads + it.head * group + (r - n * group);
      got[i] = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.q) + row * p.dim)[lane];
    }
  }
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    const int r = first + i * step;
    if (r >= P::kRows) break;
    float v[4];
    if constexpr (kParts == 3) {
      __half2 h2[2];
      memcpy(h2, &got[i], 8);
      const float2 a = __half22float2(h2[0]), b = __half22float2(h2[1]);
      v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
    } else {
      v[0] = __uint_as_float(got[i].x << 16), v[1] = __uint_as_float(got[i].x & 0xffff0000u);
      v[2] = __uint_as_float(got[i].y << 16), v[3] = __uint_as_float(got[i].y & 0xffff0000u);
    }
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) top = max(top, __float_as_uint(v[k]) & 0x7fffffffu);
    top = __reduce_max_sync(0xffffffffu, top);
    const int e = max(static_cast<int>(top >> 23) - 127, -112);  // 2^e the largest value's power
    const float up = __uint_as_float(static_cast<uint32_t>(127 + 7 - min(e, 127)) << 23);
    const float down = __uint_as_float(static_cast<uint32_t>(max(e - 7 + 127, 1)) << 23);
    if (lane == 0) s.factors[item & 3][r] = top >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : p.scale * down;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] *= up;
    const int tile = r / kTile, m = r % kTile;
#pragma unroll
    for (int part = 0; part < kParts; ++part) {
      const uint32_t lo = codes_of(v[0], v[1]), hi = codes_of(v[2], v[3]);
      if (part + 1 < kParts) {
        const uint32_t ha = halves_of(lo), hb = halves_of(hi);
        __half2 h2;
        memcpy(&h2, &ha, 4);
        const float2 a = __half22float2(h2);
        memcpy(&h2, &hb, 4);
        const float2 b = __half22float2(h2);
        v[0] -= a.x, v[1] -= a.y, v[2] -= b.x, v[3] -= b.y;
      }
#pragma unroll
      for (int k = 0; k < kSpread; ++k)  // (rows of a tile are a multiple of 8)
        *reinterpret_cast<uint32_t*>(
            &s.queries[item % P::kQueryBuffers][tile][part][(m + k * P::kRows) * kDim + ((lane / 4) ^ (m & 7)) * 16 + (lane & 3) * 4]) = lo | hi << 16;
    }
  }
}

template <int kParts, int kTileRows>
__device__ __forceinline__ void load(const AttendParams& p, Shared<kParts, kTileRows>& s) {
  using P = Plan<kParts, kTileRows>;
  const int lane = threadIdx.x & 31, loader = threadIdx.x / 32 - kSoftmaxWarps;
  constexpr bool kPair = P::kPair;
  const int turn = loader / 4, key0 = loader % 4 * kQuarter;  // of every second tile (of its stream's) it has 32 keys
  const bool listed = p.seq_lens == nullptr;
  const int row0 = lane / 8, chunk = lane % 8;  // of the codes that this lane copies: rows row0, row0 + 4, ... of the 32
  const bool chunk_in = chunk * 16 < p.dim;
  auto wait = [&](uint64_t* bar, uint32_t parity) { bar_wait(&s.aborted, bar, parity); };
  auto arrive = [&](uint64_t* bar) {  // what the whole warp has written is there for the tensor cores
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) bar_arrive(bar);
  };
  uint32_t tiles = 0, items = 0, own = 0;  // so far; own: of this loader's tiles
  for (Walk<P> walk(p, s.span); walk.more(); ++items) {
    const Item it = walk.take(p);
    const int32_t* const entries = p.index + static_cast<int64_t>(it.list) * p.index_stride;
    int t = kPair ? static_cast<int>((turn - tiles) & 1u) : turn;
    auto look_up = [&]() {
      const int32_t j = (it.first + t) * kTile + key0 + lane;
      return t < it.tiles && j < it.longest ? entries[listed ? j : static_cast<int32_t>(quotient(p.page_size, j))] : -1;
    };
    int32_t id = look_up();
    if (items >= P::kQueryBuffers) wait(&s.query_empty[items % P::kQueryBuffers], items / P::kQueryBuffers - 1);
    for (int r = loader; r < P::kRows; r += 4 * kLoaderWarps) put_queries(p, s, it, items, r, kLoaderWarps);
    arrive(&s.query_full[items % P::kQueryBuffers]);
    for (; t < it.tiles; t += 2) {
      const Ring<P> ring(turn, kPair ? tiles + t : own);
      const uint32_t key = ring.key, stage = ring.value;
      ++own;
      // ---- places of the keys
      const int32_t j = (it.first + t) * kTile + key0 + lane;
      const bool in = j < it.longest;
      const bool there = in && static_cast<int64_t>(static_cast<uint32_t>(id)) < (listed ? p.capacity : p.num_pages);
      if (in && !there && (!listed || id != -1)) atomicAdd(&g_guard_hits, 1u);
      const uint32_t of = there ? (listed ? id : j) : 0u, entry = quotient(p.page_size, of);
      const uint32_t page = !there ? 0u : listed ? entry : static_cast<uint32_t>(id), off = of - entry * p.page_size.d;
      unsigned long long places[2];
      float scales[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const Side& side = p.side[k];
        places[k] = reinterpret_cast<unsigned long long>(
            side.codes + it.head * side.code_hs + 16 * (static_cast<uint64_t>(page) * side.code_ps + static_cast<uint64_t>(off) * side.code_ts));
        scales[k] = 1.0f;
        if (there)
          scales[k] = side.scales[it.head * side.scale_hs + static_cast<uint64_t>(page) * side.scale_ps +
                                  static_cast<uint64_t>(quotient(side.block, off)) * side.scale_bs];
      }
      const uint32_t present = __ballot_sync(0xffffffffu, there);
      // ---- codes on their way: keys that are not there take a row that is, if any is
      if (ring.key_use > 0) wait(&s.key_empty[key], ring.key_use - 1);
      uint4 codes[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) codes[k] = make_uint4(0, 0, 0, 0);
      if (present != 0u) {
        const uint32_t to = smem_addr(s.keys[key]) + key0 * kDim;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int row = row0 + 4 * k;
          const unsigned long long from = __shfl_sync(0xffffffffu, places[1], row), keys = __shfl_sync(0xffffffffu, places[0], row);
          if (chunk_in) {
            codes[k] = load_once(reinterpret_cast<const uint8_t*>(from) + chunk * 16);
            copy16(to + row * kDim + ((chunk ^ (row & 7)) * 16), reinterpret_cast<const uint8_t*>(keys) + chunk * 16);
          }
        }
      }
      {
        const int now = t;
        t += 2;
        id = look_up();
        t = now;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      arrive(&s.key_full[key]);
      // ---- values become fp16
      if (ring.value_use > 0) wait(&s.value_empty[stage], ring.value_use - 1);
      uint32_t bad = 0;  // rows with a NaN code: it becomes kNanMark, which is no code's value and adds 0 where the key is not seen
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        uint32_t x[4] = {codes[k].x, codes[k].y, codes[k].z, codes[k].w};
        const bool nan = ((nan_codes(x[0]) | nan_codes(x[1])) | (nan_codes(x[2]) | nan_codes(x[3]))) != 0u;
        const uint32_t lanes = __ballot_sync(0xffffffffu, nan);
        uint4 first = make_uint4(halves_of(x[0]), halves_of(x[0] >> 16), halves_of(x[1]), halves_of(x[1] >> 16));
        uint4 second = make_uint4(halves_of(x[2]), halves_of(x[2] >> 16), halves_of(x[3]), halves_of(x[3] >> 16));
        if (lanes != 0u) {
#pragma unroll
          for (int w = 0; w < 4; ++w)
            if ((lanes >> (8 * w) & 0xffu) != 0u) bad |= 1u << (4 * k + w);
          first = make_uint4(marked(first.x), marked(first.y), marked(first.z), marked(first.w));
          second = make_uint4(marked(second.x), marked(second.y), marked(second.z), marked(second.w));
        }
        // eight lanes store eight pieces of different banks: the lanes of the other block begin with their second piece
        const int row = key0 + row0 + 4 * k, odd = chunk >> 2, at = 2 * (chunk & 3);
        uint8_t* const to = s.values[stage][chunk >> 2] + row * 128;
        *reinterpret_cast<uint4*>(to + (((at + odd) ^ (row & 7)) * 16)) = odd ? second : first;
        *reinterpret_cast<uint4*>(to + (((at + 1 - odd) ^ (row & 7)) * 16)) = odd ? first : second;
      }
      const float scale = max_or_nan(scales[1], 0x1p-100f);  // no logarithm of zero
      s.key_scales[stage][key0 + lane] = scales[0];
      s.logs[stage][key0 + lane] = log2_fast(scale);
      s.inverses[stage][key0 + lane] = inverse_fast(scale);
      int same_keys, same_values;
      __match_all_sync(0xffffffffu, __float_as_uint(scales[0]), &same_keys);
      __match_all_sync(0xffffffffu, __float_as_uint(scales[1]), &same_values);
      if (lane == 0) {
        s.present[stage][key0 / 32] = present;
        s.clean[stage][key0 / 32] = present & ~bad;
        s.uniform[stage][key0 / 32] = same_keys != 0 && same_values != 0 && present == 0xffffffffu ? 1u : 0u;
      }
      arrive(&s.value_full[stage]);
    }
    tiles += it.tiles;
  }
}

// ---------------------------------------------------------------- the softmax

// Adds to `columns` (128 bits of this thread's row) those of its value that a NaN code has, for each of 32 keys (key0 on, of the
// tile) that `bad` names and the row sees: the first `seen` of them. All of a warp's threads read the same values. A call, out of the
// loop's way (64 sequences of up to 8192 keys, 64 query heads on each of 8: 287 us in the loop, 281 so).
__device__ __noinline__ void mark_columns(uint32_t* columns, const uint8_t* values, uint32_t bad, int key0, int32_t seen) {
#pragma unroll 1
  for (; bad != 0u; bad &= bad - 1u) {
    const int key = __ffs(bad) - 1, row = key0 + key;
#pragma unroll 1
    for (int word = 0; word < kDim / 32; ++word) {
      uint32_t bits = 0;
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {  // 8 columns
        const int piece = 4 * (word & 1) + k;
        const uint4 v = *reinterpret_cast<const uint4*>(values + (word >> 1) * (kTile * 128) + row * 128 + ((piece ^ (row & 7)) * 16));
        const uint32_t two[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          bits |= (two[i] & 0xffffu) == kNanMark ? 1u << (8 * k + 2 * i) : 0u;
          bits |= two[i] >> 16 == kNanMark ? 1u << (8 * k + 2 * i + 1) : 0u;
        }
      }
      if (bits != 0u && key < seen) atomicOr(columns + word, bits);  // (both streams' threads of a row, or its two lanes)
    }
  }
  __syncwarp();
}

// N values of a row of the output, from column `col` on.
template <int N>
__device__ __forceinline__ void put_values(const AttendParams& p, int64_t row, int col, const float (&v)[N], float f) {
#pragma unroll
  for (int k = 0; k < N; k += 16) {
    if (col + k >= p.dim) break;
    uint32_t y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = v[k + 2 * i] * f, b = v[k + 2 * i + 1] * f;
      if (p.fp16) {
        const __half2 h = __floats2half2_rn(a, b);
        memcpy(&y[i], &h, 4);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        memcpy(&y[i], &h, 4);
      }
    }
    uint4* const to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row * p.dim + col + k);
    to[0] = make_uint4(y[0], y[1], y[2], y[3]);
    to[1] = make_uint4(y[4], y[5], y[6], y[7]);
  }
}

template <int kParts, int kTileRows>
__device__ __forceinline__ void softmax(const AttendParams& p, Shared<kParts, kTileRows>& s, uint32_t tmem) {
  using P = Plan<kParts, kTileRows>;
  constexpr bool kPair = P::kPair;
  constexpr int kSpread = P::kSpread, kOwn = P::kOwn, kPieces = kOwn / 32;
  const float none = __uint_as_float(0xff800000u);
  const int st = threadIdx.x / kTile, m = threadIdx.x % kTile;
  const int r = kPair ? threadIdx.x : m % P::kRows;  // its row of the tile of the work
  const int share = kSpread > 1 ? m / P::kRows : 0, own = share * kOwn;  // its part of a half's keys
  const int32_t group = static_cast<int32_t>(p.group.d), rows_of_list = p.list_queries * group;
  const uint32_t lanes = static_cast<uint32_t>(m & ~31) << 16;
  const uint32_t logits = tmem + lanes + st * kTile, sums = tmem + lanes + (2 + st) * kTile;
  auto wait = [&](uint64_t* bar, uint32_t parity) { bar_wait(&s.aborted, bar, parity); };
  uint32_t items = 0, units[2] = {0, 0};  // so far; units: tiles of both streams
  Walk<P> walk(p, s.span);
  for (; walk.more(); ++items) {
    const Item it = walk.take(p);
    const int32_t row_in_list = it.r0 + r;
    const bool used = row_in_list < rows_of_list;
    const bool warp_used = __any_sync(0xffffffffu, used);
    const int32_t n_query = quotient(p.group, used ? row_in_list : 0);
    const int64_t query = static_cast<int64_t>(it.list) * p.list_queries + n_query;
    const int64_t out_row = query * p.heads + it.head * group + ((used ? row_in_list : 0) - n_query * group);
    const int32_t len = p.seq_lens == nullptr || !used ? INT32_MAX : p.seq_lens[query];
    float bound = none;
    uint64_t sum2 = 0;
    for (int t = kPair ? 0 : st; t < it.tiles; t += kPair ? 1 : 2) {
      const uint32_t unit = units[st]++;
      const Ring<P> ring(st, unit);
      const uint32_t stage = ring.value;
      wait(&s.value_full[stage], ring.value_use);
      float factor = 0.0f;
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        wait(&s.logits_full[st][half], unit);
        if (half == 0) factor = s.factors[items & 3][r];
        tmem_fence_after();
        if (warp_used) {
          const uint32_t weights = logits + half * kHalf;
          // 32 keys at a time, in a loop: unrolled to 64 the code does not stay in the instruction cache (a prompt's chunk 375 us
          // against 365)
#pragma unroll 1
          for (int c = 0; c < kPieces; ++c) {
            const int at = half * kHalf + own + 32 * c;  // of the tile's keys
            const int32_t j0 = (it.first + t) * kTile + at;
            float x[32];
            tmem_load(logits + at, x);
            const uint32_t clean = s.clean[stage][at / 32];
            const bool uniform = s.uniform[stage][at / 32] != 0u;  // all with the same scales: what they add is worked out once
            bool whole = __all_sync(0xffffffffu, clean == 0xffffffffu && j0 + 32 <= len);
            const float base = bound == none ? 0.0f : bound - kShift;
            const float4* const ks = reinterpret_cast<const float4*>(&s.key_scales[stage][at]);
            const float4* const lg = reinterpret_cast<const float4*>(&s.logs[stage][at]);
            const float4* const iv = reinterpret_cast<const float4*>(&s.inverses[stage][at]);
            tmem_wait(x);
            // ---- logits, in log2, with the values' scales, from the base on
            if (uniform) {
              const float a = ks[0].x * factor, b = lg[0].x - base;
              const uint64_t a2 = pack2(a, a), c2 = pack2(b, b);
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                const float2 y = unpack2(fma2(pack2(x[k], x[k + 1]), a2, c2));
                x[k] = y.x, x[k + 1] = y.y;
              }
            } else {
              const uint64_t f2 = pack2(factor, factor), b2 = pack2(-base, -base);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float4 a = ks[k], b = lg[k];
                const float2 y = unpack2(fma2(pack2(x[4 * k], x[4 * k + 1]), mul2(pack2(a.x, a.y), f2), add2(pack2(b.x, b.y), b2)));
                const float2 z = unpack2(fma2(pack2(x[4 * k + 2], x[4 * k + 3]), mul2(pack2(a.z, a.w), f2), add2(pack2(b.z, b.w), b2)));
                x[4 * k] = y.x, x[4 * k + 1] = y.y, x[4 * k + 2] = z.x, x[4 * k + 3] = z.y;
              }
            }
            if (!whole) {
              const uint32_t present = s.present[stage][at / 32];
              if (present != clean) {
                mark_columns(s.nan_columns[kPair ? st : items & 1][kPair ? m : r], s.values[stage][0], present & ~clean, at,
                             used ? len - j0 : 0);
                whole = __all_sync(0xffffffffu, present == 0xffffffffu && j0 + 32 <= len);  // the sums' order goes by what is seen
              }
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if ((present >> k & 1u) == 0u || j0 + k >= len) x[k] = none;
            }
            float top = none;
#pragma unroll
            for (int k = 0; k < 32; k += 2) top = fmaxf(top, fmaxf(x[k], x[k + 1]));
            // ---- a bound that is left too far below. All of a warp's rows move theirs at once: each by itself would hold the
            // others up more often (a prompt's chunk 367 -> 415 us).
            const bool above = bound == none ? top > none : top > kShift + kSlack;
            if (__any_sync(0xffffffffu, above)) {
              const float now = fmaxf(bound, top + base), now_base = now == none ? 0.0f : now - kShift, down = now_base - base;
              const float f = bound == none || now == none ? 1.0f : exp2_fast(bound - now);
              bound = now;
#pragma unroll
              for (int k = 0; k < 32; ++k) x[k] -= down;
              sum2 = mul2(sum2, pack2(f, f));
              if (c > 0) {  // the half's weights so far, which are no part of the sums yet: rounded to 11 bits once more
                tmem_stored();
                float y[32];  // (the second 16 columns are logits, and stay)
                tmem_load(weights, y);
                tmem_wait(y);
                uint32_t w[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                  __half2 h;
                  memcpy(&h, &y[k], 4);
                  const float2 v = __half22float2(h);
                  h = __floats2half2_rn(v.x * f, v.y * f);
                  memcpy(&w[k], &h, 4);
                }
                tmem_store(weights, w);
              }
              if (half == 1 || t >= (kPair ? 1 : 2)) {  // there are sums already: of the half before, when it is done
                if (half == 1) wait(&s.sums_full[st][0], unit);
                else wait(&s.sums_full[st][1], unit - 1);
                tmem_fence_after();
#pragma unroll 1
                for (int k = 0; k < kDim; k += 32) {
                  float o[32];
                  tmem_load(sums + k, o);
                  tmem_wait(o);
                  uint32_t v[32];
#pragma unroll
                  for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(o[i] * f);
                  tmem_store(sums + k, v);
                  tmem_store(sums + k + 16, v + 16);
                }
              }
            }
            // ---- weights, over their logits
            uint32_t w[16];
            if (whole) {
              float4 i4 = iv[0];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                if (!uniform) i4 = iv[k];
                const float* const y = x + 4 * k;
                const float e0 = exp2_fast(y[0]), e1 = exp2_fast(y[1]), e2 = exp2_fast(y[2]), e3 = exp2_fast(y[3]);
                sum2 = fma2(pack2(e0, e1), pack2(i4.x, i4.y), sum2);
                sum2 = fma2(pack2(e2, e3), pack2(i4.z, i4.w), sum2);
                const __half2 a = __floats2half2_rn(e0, e1), b = __floats2half2_rn(e2, e3);
                memcpy(&w[2 * k], &a, 4);
                memcpy(&w[2 * k + 1], &b, 4);
              }
            } else {
              const float* const inverses = &s.inverses[stage][at];
              float part = 0.0f;
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                const float e0 = exp2_fast(x[k]), e1 = exp2_fast(x[k + 1]);
                // a hidden key's scale may be anything
                if (x[k] != none) part = fmaf(e0, inverses[k], part);
                if (x[k + 1] != none) part = fmaf(e1, inverses[k + 1], part);
                const __half2 a = __floats2half2_rn(e0, e1);
                memcpy(&w[k / 2], &a, 4);
              }
              sum2 = add2(sum2, pack2(part, 0.0f));
            }
            tmem_store(weights + own / 2 + 16 * c, w);
          }
          if constexpr (kSpread == 2) {  // the other lane's keys
            const uint32_t zeros[16] = {};
            tmem_store(weights + (kOwn - own) / 2, zeros);
          }
          tmem_stored();
        }
        tmem_fence_before();
        bar_arrive(&s.weights_full[st][half]);
      }
    }
    // units of the other stream, for its barriers
    if constexpr (kPair) units[st ^ 1] += it.tiles;
    else units[st ^ 1] += (it.tiles + (st == 1 ? 1 : 0)) / 2;

    // ---- the end of the item
    const float2 both = unpack2(sum2);
    float sum = both.x + both.y;
    const bool aborted_now = *const_cast<volatile int32_t*>(&s.aborted) != 0;
    if (p.fail != 0 && threadIdx.x == 0) atomicAdd(&g_guard_hits, 1u);
    const float nan = __uint_as_float(0x7fffffffu);
    float* const piece = p.partial + (2 * static_cast<int64_t>(blockIdx.x) + (it.from_start ? 1 : 0)) * P::kPartial;
    const bool alone = it.from_start && it.to_end;
    if (!alone && it.from_start && threadIdx.x == 0) {
      // the last span that has steps of this tile
      const int64_t end = s.span.at[1] - it.steps_here + it.steps, spans = gridDim.x;
      const int64_t last = min((end * spans + s.span.total - 1) / s.span.total - 1, spans - 1);
      p.cuts[blockIdx.x] = Cut{s.span.total, it.slice, it.head, static_cast<int32_t>(last), 1};
    }
    auto put_row = [&](int k, const auto& v, float f) {  // columns from k on
      if (!used) return;
      if (alone) {
        put_values(p, out_row, k, v, f);
      } else {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(v) / sizeof(float)); i += 4)
          *reinterpret_cast<float4*>(piece + static_cast<int64_t>(r) * kDim + k + i) = make_float4(v[i] * f, v[i + 1] * f, v[i + 2] * f, v[i + 3] * f);
      }
    };
    auto spoil = [&](auto& v, uint32_t columns) {
      if (columns == 0u) return;
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(v) / sizeof(float)); ++i)
        if ((columns >> i & 1u) != 0u) v[i] = nan;
    };
    auto put_stats = [&](float top, float total) {
      if (!used) return;
      if (!alone) *reinterpret_cast<float2*>(piece + P::kRows * kDim + 2 * r) = make_float2(top, total);
      else if (p.lse != nullptr) p.lse[out_row] = log_sum(top, total);
    };
    if constexpr (kPair) {
      wait(&s.sums_full[st][1], units[st] - 1);
      tmem_fence_after();
      const bool failed = aborted_now || *const_cast<volatile int32_t*>(&s.aborted) != 0;
      if (failed) sum = nan;
      put_stats(bound, sum);
      const float f = failed ? nan : !alone ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
      if (warp_used) {
#pragma unroll 1
        for (int k = 0; k < kDim; k += 32) {
          float o[32];
          tmem_load(sums + k, o);
          tmem_wait(o);
          spoil(o, s.nan_columns[st][m][k / 32]);
          put_row(k, o, f);
        }
      }
      *reinterpret_cast<uint4*>(s.nan_columns[st][m]) = make_uint4(0, 0, 0, 0);
      tmem_fence_before();
      bar_arrive(&s.sums_empty[st]);
    } else if constexpr (kSpread > 1) {
      s.stats[items & 1][st][m] = make_float2(bound, sum);
      named_barrier<kSoftmaxThreads>(3);
      if (st == 0) {
        wait(&s.sums_full[0][1], units[0] - 1);
        if (it.tiles > 1) wait(&s.sums_full[1][1], units[1] - 1);
        tmem_fence_after();
        const bool failed = aborted_now || *const_cast<volatile int32_t*>(&s.aborted) != 0;
        // all that there is of this row
        float top = none, total = 0.0f;
#pragma unroll
        for (int k = 0; k < 2 * kSpread; ++k) top = fmaxf(top, s.stats[items & 1][k / kSpread][k % kSpread * P::kRows + r].x);
#pragma unroll
        for (int k = 0; k < 2 * kSpread; ++k) {
          const float2 v = s.stats[items & 1][k / kSpread][k % kSpread * P::kRows + r];
          total = fmaf(v.y, v.x == none ? 1.0f : exp2_fast(v.x - top), total);
        }
        const float other = s.stats[items & 1][1][m].x;
        const float f0 = bound == none ? 1.0f : exp2_fast(bound - top), f1 = other == none ? 1.0f : exp2_fast(other - top);
        if (failed) total = nan;
        if (share == 0) put_stats(top, total);
        const float out = failed ? nan : !alone ? 1.0f : total == 0.0f ? 0.0f : 1.0f / total;
        constexpr int kColumns = 32 / kSpread;
#pragma unroll 1
        for (int k = 0; k < kDim; k += 32) {
          float a[32];
          tmem_load(sums + k, a);
          tmem_wait(a);
#pragma unroll
          for (int i = 0; i < 32; ++i) a[i] *= f0;
          if (it.tiles > 1) {
            float b[32];
            tmem_load(sums + kTile + k, b);
            tmem_wait(b);
#pragma unroll
            for (int i = 0; i < 32; ++i) a[i] = fmaf(b[i], f1, a[i]);
          }
          if (k > 0) named_barrier<kTile>(4);
#pragma unroll
          for (int i = 0; i < 32; i += 4) *reinterpret_cast<float4*>(&s.joined[m][i]) = make_float4(a[i], a[i + 1], a[i + 2], a[i + 3]);
          named_barrier<kTile>(4);
          float y[kColumns];
#pragma unroll
          for (int i = 0; i < kColumns; ++i) y[i] = 0.0f;
#pragma unroll
          for (int from = 0; from < kSpread; ++from)
#pragma unroll
            for (int i = 0; i < kColumns; i += 4) {
              const float4 v = *reinterpret_cast<const float4*>(&s.joined[from * P::kRows + r][share * kColumns + i]);
              y[i] += v.x, y[i + 1] += v.y, y[i + 2] += v.z, y[i + 3] += v.w;
            }
          spoil(y, s.nan_columns[items & 1][r][k / 32] >> (share * kColumns));
          put_row(k + share * kColumns, y, out);
        }
        named_barrier<kTile>(4);
        if (share == 0) *reinterpret_cast<uint4*>(s.nan_columns[items & 1][r]) = make_uint4(0, 0, 0, 0);
        tmem_fence_before();
        bar_arrive(&s.sums_empty[0]);
        bar_arrive(&s.sums_empty[1]);
      }
    } else {
      s.stats[items & 1][st][m] = make_float2(bound, sum);
      named_barrier<kSoftmaxThreads>(3);
      if (st == 0) {
        wait(&s.sums_full[0][1], units[0] - 1);
        if (it.tiles > 1) wait(&s.sums_full[1][1], units[1] - 1);
        tmem_fence_after();
        const bool failed = aborted_now || *const_cast<volatile int32_t*>(&s.aborted) != 0;
        // both streams' of this row
        const float2 other = s.stats[items & 1][1][m];
        const float top = fmaxf(bound, other.x);
        // a stream whose keys are all hidden from a row has no bound; its sum is 0, or NaN
        const float f0 = bound == none ? 1.0f : exp2_fast(bound - top), f1 = other.x == none ? 1.0f : exp2_fast(other.x - top);
        const float total = failed ? nan : fmaf(sum, f0, other.y * f1);
        put_stats(top, total);
        const float out = failed ? nan : !alone ? 1.0f : total == 0.0f ? 0.0f : 1.0f / total;
        if (warp_used) {
#pragma unroll 1
          for (int k = 0; k < kDim; k += 32) {
            float a[32];
            tmem_load(sums + k, a);
            tmem_wait(a);
#pragma unroll
            for (int i = 0; i < 32; ++i) a[i] *= f0;
            if (it.tiles > 1) {
              float b[32];
              tmem_load(sums + kTile + k, b);
              tmem_wait(b);
#pragma unroll
              for (int i = 0; i < 32; ++i) a[i] = fmaf(b[i], f1, a[i]);
            }
            spoil(a, s.nan_columns[items & 1][r][k / 32]);
            put_row(k, a, out);
          }
        }
        *reinterpret_cast<uint4*>(s.nan_columns[items & 1][r]) = make_uint4(0, 0, 0, 0);  // for the item after the next one
        tmem_fence_before();
        bar_arrive(&s.sums_empty[0]);
        bar_arrive(&s.sums_empty[1]);
      }
    }
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

template <int kParts, int kTileRows>
__global__ void __launch_bounds__(kThreads, 1) wide_kernel(const __grid_constant__ AttendParams p) {
  using P = Plan<kParts, kTileRows>;
  using S = Shared<kParts, kTileRows>;
  constexpr bool kPair = P::kPair;
  extern __shared__ __align__(1024) uint8_t raw[];
  S& s = *reinterpret_cast<S*>(raw + (1024u - smem_addr(raw) % 1024u) % 1024u);
  const int warp = threadIdx.x / 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < P::kKeyStages; ++i) bar_init(&s.key_full[i], 4), bar_init(&s.key_empty[i], kPair ? 2 : 1);
    for (int i = 0; i < kValueStages; ++i) bar_init(&s.value_full[i], 4), bar_init(&s.value_empty[i], kPair ? 2 : 1);
    for (int i = 0; i < 2; ++i) {
      bar_init(&s.query_full[i], kLoaderWarps);
      bar_init(&s.query_empty[i], 2);
      bar_init(&s.drained[i], 1);
      for (int h = 0; h < 2; ++h) {
        bar_init(&s.logits_full[i][h], h == 0 ? 2 : 1);  // the products and, with the first ones, the rows' factors
        bar_init(&s.weights_full[i][h], kTile);
        bar_init(&s.sums_full[i][h], 1);
      }
      bar_init(&s.sums_empty[i], kTile);
    }
    s.aborted = p.fail;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (threadIdx.x < 2 * kTile) *reinterpret_cast<uint4*>(s.nan_columns[threadIdx.x / kTile][threadIdx.x % kTile]) = make_uint4(0, 0, 0, 0);
  // columns that the cache does not have are zeros, which no copy touches
  if (p.dim < kDim)
    for (int i = threadIdx.x; i < P::kKeyStages * kTile * kDim / 16; i += kThreads) reinterpret_cast<uint4*>(s.keys)[i] = make_uint4(0, 0, 0, 0);
  begin_after_prior_grids();
  find_span<P::kRows, P::kKeys>(p, s.span_sums, s.span);
  if (threadIdx.x == 0) p.cuts[blockIdx.x] = Cut{s.span.total, 0, 0, 0, 0};
  if (s.span.at[0] >= s.span.at[1]) return;
  if (warp == kSoftmaxWarps + kLoaderWarps) {
    // one CTA an SM (its shared memory sees to that), so the columns are free
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s.tmem_base)),
                 "r"(kTmemColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    tmem_fence_before();
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = s.tmem_base;
  if (warp < kSoftmaxWarps) {
    more_registers<kSoftmaxRegisters>();
    softmax<kParts, kTileRows>(p, s, tmem);
  } else if (warp < kSoftmaxWarps + kLoaderWarps) {
    load<kParts, kTileRows>(p, s);
  } else {
    fewer_registers<kOtherRegisters>();
    const int st = warp - kSoftmaxWarps - kLoaderWarps;
    if (st < 2) multiply<kParts, kTileRows>(p, s, tmem, st);
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == kSoftmaxWarps + kLoaderWarps)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemColumns));
}

struct InOrder {
  static __device__ __forceinline__ int column(int at) { return at; }
};

template <int kParts, int kTileRows>
cudaError_t launch_plan(AttendParams p, int sms, cudaStream_t stream) {
  using P = Plan<kParts, kTileRows>;
  constexpr int kBytes = static_cast<int>(sizeof(Shared<kParts, kTileRows>)) + 1024;
  static_assert(kBytes <= 227 * 1024, "shared memory of a CTA");
  const int64_t tiles = (static_cast<int64_t>(p.list_queries) * p.group.d + P::kRows - 1) / P::kRows;
  if (tiles * p.lists > INT32_MAX / 2) return cudaErrorInvalidValue;
  p.tiles = static_cast<int32_t>(tiles);
  p.slices = static_cast<int32_t>(tiles * p.lists);
  // no more spans than there can be steps
  const int64_t most = static_cast<int64_t>(p.slices) * p.kv_heads * ((static_cast<int64_t>(p.row_len) + P::kKeys) / P::kKeys);
  const int spans = static_cast<int>(std::min<int64_t>(sms, most));
  static thread_local int known = -1;  // the device whose kernel may use so much shared memory
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess && known != device) {
    e = cudaFuncSetAttribute(wide_kernel<kParts, kTileRows>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e == cudaSuccess) known = device;
  }
  if (e == cudaSuccess) e = launch(wide_kernel<kParts, kTileRows>, spans, kThreads, kBytes, stream, p);
  if (e != cudaSuccess || spans == 1) return e;
  return launch_join<kDim, InOrder>(p, spans, P::kRows, stream);
}

template <int kParts>
cudaError_t launch_parts(const AttendParams& p, int sms, cudaStream_t stream) {
  switch (wide_rows(static_cast<int64_t>(p.list_queries) * p.group.d)) {
    case kTile / 2: return launch_plan<kParts, kTile / 2>(p, sms, stream);
    case kTile: return launch_plan<kParts, kTile>(p, sms, stream);
    default: return launch_plan<kParts, 2 * kTile>(p, sms, stream);
  }
}

std::atomic<int> g_fail{0};

}  // namespace

int wide_rows(int64_t rows) { return rows <= kTile / 2 ? kTile / 2 : rows <= kTile ? kTile : 2 * kTile; }

cudaError_t launch_wide_attention(AttendParams p, int sms, cudaStream_t stream) {
  p.fail = g_fail.load(std::memory_order_relaxed);
  return p.fp16 ? launch_parts<3>(p, sms, stream) : launch_parts<2>(p, sms, stream);
}

cudaError_t wide_attention_guard_hits(unsigned int* hits) {
  return cudaMemcpyFromSymbol(hits, g_guard_hits, sizeof(unsigned int));
}

cudaError_t reset_wide_attention_guard_hits() {
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_guard_hits, &zero, sizeof(unsigned int));
}

}  // namespace indexer_gb300

extern "C" int indexer_set_attention_failure(int mode) {
  return indexer_gb300::g_fail.exchange(mode == 1 ? 1 : 0, std::memory_order_relaxed);
}
