// Weight-streaming engine of the few-token kernels (at most 32 tokens: few_layer.cu,
// adapter_few.cu).  With so few tokens every product is bound by reading its weights once
// from HBM, so the kernels are built around the stream, not around the MMA:
//
//   * One CTA per SM, all resident (cooperative launch).  Every phase cuts its output rows
//     (weight rows) evenly over the CTAs, at single-row granularity, whatever the expert.
//   * Warps 8.. produce: the CTA's rows are cut into tiles of up to 32 weight rows and the
//     contraction into chunks of 1 KB per row (2 or 4 KB in thin tiles, chunk_vecs); a slot of
//     the ring holds one chunk of a tile's weight rows and of its token rows, copied with one
//     bulk copy per row.  Slots are sized by the rows they hold, so thin tiles (a phase that
//     leaves a CTA 7 rows) still keep the whole ring in flight; the stream does not stop between
//     tiles or phases.
//     One warp issues a bulk copy about every 28 to 45 ns, which would cap the stream at half
//     of HBM's rate (Mixtral-shaped T=16: 890 us with one producer), so slot i belongs to
//     producer team i mod kTeams, one lane per row; every producer follows the same
//     sequence of slots and places them by the same arithmetic.  The rate is the ring's bytes
//     over a slot's time in it (4 us; the copies alone, in a ring a third as long, reach
//     6.6 TB/s), not HBM's latency: weights that are in L2 already stream as fast.
//   * Warps 0-7 consume, two or four warps to a slot, several slots at a time: a slot costs a warp
//     a fixed latency (its barrier, descriptor, first loads) that eight warps sharing every
//     slot all paid (Granite-shaped T=16: 0.7 us per 11-row slot), now paid in parallel.
//     bf16: mma.sync m16n8k16 with the weight rows on M and the tokens on N, fed by 16-byte
//     shared loads: thread q of a quad takes 8 consecutive k of its row, for weights and
//     tokens alike, which only permutes the k index inside a 32-wide block.  At 8 tokens
//     the pipe needs 2 * 8 FLOP per weight (about 53 TFLOP/s at the full HBM rate), far
//     below even the warp-level MMA rate, and there is no tensor-memory round trip at the
//     end of a 7-row tile; that is why this is not tcgen05, whose M is at least 64 rows.
//     fp32: FMA, a weight row per lane.
//   * The 8 partial sums per output meet in shared memory in warp order (which slots a warp
//     takes depends on the shape alone, so runs give the same bits); the caller's epilogue
//     consumes a tile's total while the next tile's slots are already being consumed.  Where a
//     tile has few slots, one group takes it whole, epilogue and all (solo_tiles).
//
// The MMA reads whole 16-row and 8-token fragments; rows past a tile's last one are clamped
// to it.  A garbage row or token column only reaches its own outputs, which are not stored.
#pragma once

#include "common.cuh"
#include "grid_sync.cuh"
#include "internal.h"

namespace moe {
namespace few {

constexpr int kMaxTokens = kFewTokens;  // one token-mask word
constexpr int kConsumerWarps = 8;
constexpr int kConsumers = 32 * kConsumerWarps;
// Warps that share a slot: more of them where token rows leave the ring few slots, which are then
// to be released sooner.  us with 2 / 4: 16+1 experts T=32 643 / 606, T=16 467 / 472,
// Granite-shaped T=16 38.9 / 40.0; fp32, 12+1 experts T=16 373 / 342.
template <bool F32, int NT> constexpr int kGroupWarps = NT == 1 || (NT == 2 && !F32) ? 2 : 4;
template <bool F32, int NT> constexpr int kGroups = kConsumerWarps / kGroupWarps<F32, NT>;
// Producers: teams of warps, a slot's copies dealt over the warps of its team.  A slot takes one warp
// 0.4 us plus 28 ns per copy, 1.5 us for 36 rows, which is a third of its time in the ring.
// Measured, us with 4 x 1 / 4 x 2 / 2 x 4 / 8 x 1 warps: Mixtral-shaped T=16 363 / 338 / 357 / 353,
// T=8 341 / 325 / 340 / 334, 16+1 experts T=16 508 / 474 / 507 / 484.  fp32 and more than 16 tokens
// need more than the 128 registers a thread of 8 producer warps (fp32 T=16: 312 / 465).
constexpr int kTeams = 4;
template <bool F32, int NT> constexpr int kTeamWarps = F32 || NT == 4 ? 1 : 2;
template <bool F32, int NT>
constexpr int kThreads = kConsumers + 32 * kTeams * kTeamWarps<F32, NT>;
constexpr int kSlots = 64;           // slot descriptors and barriers
constexpr int kChunkBytes = 1024;    // contraction bytes per row of the smallest chunk
constexpr int kChunkVecs = kChunkBytes / 16;
constexpr int kMaxChunkVecs = 4 * kChunkVecs;
constexpr int kThinSlot = 24 * 1024;  // limit of chunk_vecs
constexpr uint32_t kSmemBytes = 227 * 1024;
constexpr int kTileRows = 32;        // weight rows per tile at most (two MMA row blocks)
constexpr int kRedStride = 36;       // floats per token column of the partial sums: the MMA
                                     // fragment's stores and the row-wise reads hit 32 banks

// Row pitch of a slot.  bf16 fragments read 64 bytes of two rows per 8-lane phase (pitch
// 64 mod 128), fp32 lanes read 16 bytes of 8 rows (pitch 16 mod 128).
template <bool F32>
__host__ __device__ constexpr uint32_t pitch_of(int chunk_vecs) {
  return chunk_vecs * 16 + (F32 ? 16 : 64);
}
// 16-byte vectors along the contraction of a phase's chunks, for tiles of at most `rows` rows
// (token rows too) of `vecs` vectors.  A slot costs its warps a fixed latency whatever it holds,
// so thin tiles take longer chunks, while the slot stays within `limit` (of a ring of about 190 KB).
__device__ __forceinline__ int chunk_vecs(int rows, int vecs, int limit) {
  int v = kChunkVecs;
  while (v < kMaxChunkVecs && v < vecs && rows * (2 * v * 16 + 64) <= limit) v *= 2;
  return v;
}

// One slot of the ring, written by the producer before the slot's barrier completes.
struct alignas(16) SlotDesc {
  uint32_t off;    // byte offset in the ring
  int16_t r0, r1;  // weight rows of the first and second row block (the second follows the
                   // first in the slot; in a pair tile they are the gate and the up rows)
  int16_t kvec;    // valid 16-byte vectors along the contraction
  int16_t pitch;   // bytes between rows
  int8_t last;     // last chunk of the tile
  int8_t kind;     // caller's: which phase
  int8_t scatter;  // 1: the token of mask bit t is column t; 0: columns are 0..popc(mask)-1
  int8_t unused;
  uint32_t mask;   // tokens whose rows the slot holds, ascending
  int32_t seg;     // caller's: what the tile belongs to
  int32_t row;     // caller's: first output row of the tile
  int32_t kv;      // caller's: first vector of the chunk along the contraction
};

struct Shared {
  uint64_t* full;
  uint64_t* empty;
  SlotDesc* desc;
  uint64_t* sums;   // [2] a tile's partial sums are complete
  uint64_t* freed;  // a tile's epilogue is done (one buffer of partial sums)
  uint64_t* passed; // this CTA knows that all CTAs have arrived
  SlotDesc* tile;   // [2] its last slot's descriptor
  volatile int* abort_flag;
  uint8_t* ring;
  float* red;       // [kRedBufs][8 warps][8 NT][kRedStride]
  uint8_t* zeros;   // a chunk of zeros: the row of a token that a slot does not hold
  uint32_t ring_bytes;
};

constexpr int kCtlBytes = 2 * kSlots * 8 + kSlots * 32 + 2 * 32 + 64 + kChunkBytes;
static_assert(sizeof(SlotDesc) == 32, "descriptor size");
static_assert(kSlots % kGroups<false, 1> == 0 && kSlots % kGroups<true, 4> == 0,
              "a slot's barriers belong to one group");
template <int NT> constexpr int kRedFloats = kConsumerWarps * 8 * NT * kRedStride;
// Buffers of partial sums: two for up to 8 tokens; with more tokens one (and a barrier for its
// release), because the ring needs the room: a slot of 32 tokens takes 68 KB.
template <int NT> constexpr int kRedBufs = NT == 1 ? 2 : 1;
// The largest slot: a full tile and 32 token rows.
constexpr uint32_t kMaxSlotBytes = (kTileRows + kMaxTokens) * (kChunkBytes + 64);

// Control words, partial sums, the caller's tables (table_bytes), then the ring.
template <int NT>
__device__ __forceinline__ Shared carve(uint8_t* smem, uint32_t table_bytes, uint32_t total) {
  Shared s;
  s.full = reinterpret_cast<uint64_t*>(smem);
  s.empty = s.full + kSlots;
  s.desc = reinterpret_cast<SlotDesc*>(s.empty + kSlots);
  s.tile = s.desc + kSlots;
  s.sums = reinterpret_cast<uint64_t*>(s.tile + 2);
  s.freed = s.sums + 2;
  s.passed = s.freed + 1;
  s.abort_flag = reinterpret_cast<volatile int*>(s.passed + 1);
  s.red = reinterpret_cast<float*>(smem + kCtlBytes);
  s.zeros = smem + kCtlBytes - kChunkBytes;
  const uint32_t at = kCtlBytes + kRedBufs<NT> * kRedFloats<NT> * 4 + table_bytes;
  s.ring = smem + at;
  s.ring_bytes = (total - at) & ~15u;
  return s;
}

template <bool F32, int NT>
__device__ __forceinline__ void init_shared(const Shared& s) {
  for (int i = threadIdx.x; i < kChunkVecs; i += kThreads<F32, NT>)
    reinterpret_cast<uint4*>(s.zeros)[i] = make_uint4(0, 0, 0, 0);
  // one slot's barriers per thread: 128 initialisations in a row took 0.5 us
  if (threadIdx.x < kSlots) {
    mbar_init(&s.full[threadIdx.x], kTeamWarps<F32, NT>);
    mbar_init(&s.empty[threadIdx.x], kGroupWarps<F32, NT>);
  } else if (threadIdx.x == kSlots) {
    mbar_init(&s.sums[0], kConsumerWarps);
    mbar_init(&s.sums[1], kConsumerWarps);
    mbar_init(s.freed, kConsumerWarps);
    mbar_init(s.passed, 1);
    *s.abort_flag = 0;
  }
  if (threadIdx.x <= kSlots) fence_mbar_init();
}

// The engine's waits: one inlined try, the bounded loop out of line.  These kernels run once per
// layer from a cold instruction cache, where code size is latency: inlined everywhere the
// kernels were 175 KB.
static __device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity,
                                              volatile int* abort_flag, int32_t* status) {
  return mbar_wait_bounded(bar, parity, abort_flag, kWaitLimitNs, status);
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                     int32_t* status) {
  return mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort_flag, status);
}

__device__ __forceinline__ void consumer_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory");
}
// The same barrier; returns whether `v` held on every consumer thread.
__device__ __forceinline__ bool consumer_all(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v)), "n"(kConsumers)
      : "memory");
  return r != 0;
}

// The barrier of one group's warps; returns whether `v` held on all of its threads.
template <bool F32, int NT>
__device__ __forceinline__ bool group_all(uint32_t group, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v)), "r"(2 + group), "n"(32 * kGroupWarps<F32, NT>)
      : "memory");
  return r != 0;
}

// Where CTA i's share of n rows begins.
static __device__ __noinline__ int64_t share_begin(int64_t n, uint32_t i) {
  return n * i / gridDim.x;
}

// The same by several whole warps of a CTA, once per launch: one lane of the `poller` warp polls,
// the others wait in shared memory (polls of all warps would crowd the arrivals).
__device__ __forceinline__ bool grid_wait_warps(const GridSync& g, unsigned int target,
                                                bool poller, uint64_t* passed,
                                                volatile int* abort_flag, int32_t* status) {
  if (poller && (threadIdx.x & 31) == 0 && grid_wait(g, target, abort_flag, status))
    mbar_arrive(passed);
  return __all_sync(0xffffffffu, wait(passed, 0, abort_flag, status));
}
// Make this thread's global writes visible to bulk copies issued by other threads after a
// barrier (generic proxy -> async proxy), and the reader's counterpart.
__device__ __forceinline__ void fence_proxy_async_all() {
  asm volatile("fence.proxy.async;" ::: "memory");
}

// ---------------------------------------------------------------------------------
// Producer: a FIFO byte ring, run by whole producer warps.  Slot i starts at byte
// `at` of an endless line that skips the ring's end where the slot would not fit; its place
// is `at` modulo the ring.  The line depends on the slots' sizes only, so every producer
// computes the same places, and a slot may be written once the oldest slot still in use
// starts less than a ring's length before its end.  A producer waits for the slots' releases
// in order and keeps fewer than kInFlight of them unreleased when it fills one.
//   Slot i belongs to team i mod kTeams; warp j of a team of TW copies the slot's rows j, j + TW,
// ... and arrives at the slot's barrier for their bytes.
//   A producer must not fall behind by two uses of a slot, whose barrier parity would be
// ambiguous: while it waits, with its own slot j not filled, for the release of `tail`, no slot from
// tail + kSlots on may be released.  The other teams pass slot j only by being ahead, and fill
// slots below j + kInFlight at most; its own slots are kTeams apart, so
// j - tail < kInFlight + kTeams.  Hence 2 kInFlight + kTeams <= kSlots + 1.
// ---------------------------------------------------------------------------------
constexpr uint32_t kInFlight = (kSlots + 1 - kTeams) / 2;
template <int TW>
struct Producer {
  Shared s;
  int32_t* status;
  uint32_t start[kSlots / 32] = {};  // line positions of the last slots, slot i's in lane i % 32
  uint32_t me;         // this producer's index
  uint32_t line = 0;   // line position of the next slot
  uint32_t head = 0;   // the same modulo the ring
  uint32_t it = 0;     // slots passed
  uint32_t tail = 0;   // slots known to be released

  __device__ __forceinline__ Producer(const Shared& sh, int32_t* st)
      : s(sh), status(st), me((threadIdx.x >> 5) - kConsumerWarps) {}
  __device__ __forceinline__ uint32_t team() const { return me / TW; }
  __device__ __forceinline__ bool mine() const { return it % kTeams == team(); }
  // Whether this warp copies row r of its team's slots.
  __device__ __forceinline__ bool copies(uint32_t r) const {
    return r % TW == me % TW;
  }

  // Take the place of the next slot; `pass` moves on to the one after it.
  __device__ __forceinline__ void reserve(uint32_t bytes) {
    if (s.ring_bytes - head < bytes) {
      line += s.ring_bytes - head;
      head = 0;
    }
#pragma unroll
    for (int i = 0; i < kSlots / 32; ++i)
      if (it % kSlots == 32 * i + (threadIdx.x & 31)) start[i] = line;
  }
  __device__ __forceinline__ uint32_t start_of(uint32_t slot) const {
    uint32_t v = start[0];
#pragma unroll
    for (int i = 1; i < kSlots / 32; ++i)
      if (slot % kSlots >= 32 * i) v = start[i];
    return __shfl_sync(0xffffffffu, v, slot % 32);
  }
  __device__ __forceinline__ void pass(uint32_t bytes) {
    line += bytes;
    head += bytes;
    ++it;
  }
  // Wait until the reserved slot may be written: 1, or 0 if that takes the release of slot
  // `stop` or a later one, or -1 on abort.
  __device__ __forceinline__ int ready(uint32_t bytes, uint32_t stop) {
    while (tail != it &&  // warp-uniform: every lane sees the same state
           (it - tail >= kInFlight || line + bytes - start_of(tail) > s.ring_bytes)) {
      if (tail >= stop) return 0;
      if (!__all_sync(0xffffffffu, wait(&s.empty[tail % kSlots], (tail / kSlots) & 1u,
                                        s.abort_flag, status)))
        return -1;
      ++tail;
    }
    return 1;
  }
  // Publish the slot's descriptor (all warps of the team write the same) and arm its barrier for
  // this warp's part of `rows` rows of `bytes` bytes; then come its copies.
  __device__ __forceinline__ void open(SlotDesc d, uint32_t rows, uint32_t bytes) {
    d.off = head;
    if ((threadIdx.x & 31) == 0) {
      s.desc[it % kSlots] = d;
      mbar_arrive_expect_tx(&s.full[it % kSlots],
                            (rows + TW - 1 - me % TW) / TW * bytes);
    }
    __syncwarp();
  }
  // This warp's part of the weight rows of slot `it`: n0 (at most 32) from w0, then n1 from w1.
  __device__ __forceinline__ void copy_weights(uint32_t pitch, const uint8_t* w0, int n0,
                                               const uint8_t* w1, int n1, size_t stride,
                                               uint32_t bytes) {
    const int r = (threadIdx.x & 31) * TW + me % TW;  // a tile has at most 32 rows
    if (r < n0 + n1)
      bulk_load(s.ring + head + static_cast<uint32_t>(r) * pitch,
                r < n0 ? w0 + r * stride : w1 + (r - n0) * stride, bytes, &s.full[it % kSlots]);
    __syncwarp();
  }
  // This warp's part of `n` (at most 32) rows behind the `row` weight rows of the slot at `off`.
  __device__ __forceinline__ void copy_rows(uint32_t slot, uint32_t off, uint32_t pitch, int row,
                                            const uint8_t* src, size_t stride, int n,
                                            uint32_t bytes) {
    const int r = threadIdx.x & 31;
    if (r < n && copies(row + r))
      bulk_load(s.ring + off + static_cast<uint32_t>(row + r) * pitch, src + r * stride,
                bytes, &s.full[slot % kSlots]);
    __syncwarp();
  }
  // The same for the rows of a token mask.
  __device__ __forceinline__ void copy_tokens(uint32_t pitch, int row, const uint8_t* src,
                                              size_t stride, uint32_t mask, uint32_t bytes) {
    const int t = threadIdx.x & 31;
    const int r = row + __popc(mask & ((1u << t) - 1u));
    if (((mask >> t) & 1u) && copies(r))
      bulk_load(s.ring + head + static_cast<uint32_t>(r) * pitch, src + t * stride, bytes,
                &s.full[it % kSlots]);
    __syncwarp();
  }
  // Before leaving early: every copy of this producer has landed, or has had the wait's
  // limit to.
  __device__ __forceinline__ void drain() {
    for (uint32_t i = it - min(it, static_cast<uint32_t>(kSlots)); i < it; ++i)
      if (i % kTeams == team() &&
          !wait_slow(&s.full[i % kSlots], (i / kSlots) & 1u, nullptr, status))
        break;
  }
};

// ---------------------------------------------------------------------------------
// Consumers
// ---------------------------------------------------------------------------------
__device__ __forceinline__ uint4 lds_vec(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// bf16 pair tiles of at most 8 rows of each matrix take one 16-row block: the first matrix's rows
// are its rows 0-7, the second's its rows 8-15.
__device__ __forceinline__ bool pair_fold(const SlotDesc& d) { return d.r1 > 0 && d.r0 <= 8; }

// Accumulators of one tile: bf16 fragments [row block][token block][4], or fp32 [token].
template <bool F32, int NT> struct Acc;
template <int NT> struct Acc<false, NT> {
  float c[2][NT][4];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[m][n][i] = 0.f;
  }
  // One 32-wide block: two k-steps.  The k-step is the outer loop so that consecutive MMAs
  // have different accumulators (an MMA's result is 21 cycles away, its issue slot 8).
  template <bool TWO, int NB>
  __device__ __forceinline__ static void block(float (&c)[2][NT][4], const uint4 (&w)[4],
                                               const uint4 (&x)[NB]) {
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      mma_bf16(c[0][n], w[0].x, w[1].x, w[0].y, w[1].y, x[n].x, x[n].y);
      if (TWO) mma_bf16(c[1][n], w[2].x, w[3].x, w[2].y, w[3].y, x[n].x, x[n].y);
    }
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      mma_bf16(c[0][n], w[0].z, w[1].z, w[0].w, w[1].w, x[n].z, x[n].w);
      if (TWO) mma_bf16(c[1][n], w[2].z, w[3].z, w[2].w, w[3].w, x[n].z, x[n].w);
    }
  }
  // The chunk for NB token blocks, with a second row block or without.  Compile-time: a
  // branch around each MMA costs more than the MMA (T=16 slots: 3000 cycles instead of 1000).
  template <bool TWO, int NB>
  __device__ __forceinline__ void chunk_of(const SlotDesc& d, const Shared& s, int part,
                                           int lane) {
    const int P = d.pitch;
    const uint32_t base = smem_u32(s.ring) + d.off;
    const int g = lane >> 2, q = lane & 3;
    const uint32_t at = (part * 4 + q) * 16;
    // 16-row blocks: rows past a block's last one are clamped to it
    // (a pair tile of up to 8 rows each: one block, see pair_fold)
    const int up = d.r0 + min(g, d.r1 - 1);
    uint32_t a[4] = {base + min(g, d.r0 - 1) * P + at,
                     base + (pair_fold(d) ? up : min(g + 8, d.r0 - 1)) * P + at, base + up * P + at,
                     base + (d.r0 + min(g + 8, d.r1 - 1)) * P + at};
    const int nb = __popc(d.mask);
    uint32_t b[NB], step[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int t = 8 * n + g;
      int row = t < nb ? t : -1;  // the token row of this lane's column, or none
      if (d.scatter) row = ((d.mask >> t) & 1u) ? __popc(d.mask & ((1u << t) - 1u)) : -1;
      b[n] = row >= 0 ? base + (d.r0 + d.r1 + row) * P + at : smem_u32(s.zeros) + at;
      step[n] = row >= 0 ? kChunkBytes : 0;
    }
    float part_c[2][NT][4] = {};
    constexpr int kStep = kGroupWarps<false, NT> * 64;         // bytes between a warp's blocks
    constexpr int kBlocks = kChunkBytes / kStep;
    constexpr int HB = NB == 4 ? 2 : 4;  // blocks loaded together, so that latencies overlap
#pragma unroll 1
    for (int left = d.kvec;; left -= kChunkVecs) {  // 1 KB of every row at a time
      if (left >= kChunkVecs) {
#pragma unroll
        for (int i = 0; i < kBlocks; i += HB) {
          uint4 w[HB][4], x[HB][NB];
#pragma unroll
          for (int h = 0; h < HB; ++h) {
            const int o = (i + h) * kStep;
#pragma unroll
            for (int j = 0; j < (TWO ? 4 : 2); ++j) w[h][j] = lds_vec(a[j] + o);
#pragma unroll
            for (int n = 0; n < NB; ++n) x[h][n] = lds_vec(b[n] + o);
          }
#pragma unroll
          for (int h = 0; h < HB; ++h) block<TWO, NB>(part_c, w[h], x[h]);
        }
      } else {
#pragma unroll 1
        for (int o = 0; (part * 4 + o / 16) < left; o += kStep) {
          const bool in = part * 4 + q + o / 16 < left;  // the end inside a block: zeros
          const uint4 z = make_uint4(0, 0, 0, 0);
          uint4 w[4], x[NB];
#pragma unroll
          for (int j = 0; j < (TWO ? 4 : 2); ++j) w[j] = in ? lds_vec(a[j] + o) : z;
#pragma unroll
          for (int n = 0; n < NB; ++n) x[n] = in ? lds_vec(b[n] + o) : z;
          block<TWO, NB>(part_c, w, x);
        }
      }
      if (left <= kChunkVecs) break;
#pragma unroll
      for (int j = 0; j < 4; ++j) a[j] += kChunkBytes;
#pragma unroll
      for (int n = 0; n < NB; ++n) b[n] += step[n];
    }
    // A token column that the slot does not hold stays as it is, whatever zero times the
    // weights gave (infinities and NaNs of an expert's weights reach its own tokens only).
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const uint32_t keep = d.scatter ? d.mask >> (8 * n + 2 * q) : 3u;
#pragma unroll
      for (int m = 0; m < (TWO ? 2 : 1); ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if ((keep >> (i & 1)) & 1u) c[m][n][i] += part_c[m][n][i];
    }
  }
  template <int NB>
  __device__ __forceinline__ void chunk_n(const SlotDesc& d, const Shared& s, int part,
                                          int lane) {
    if (d.r1 > 0 && !pair_fold(d)) chunk_of<true, NB>(d, s, part, lane);
    else chunk_of<false, NB>(d, s, part, lane);
  }
  __device__ __forceinline__ void chunk(const SlotDesc& d, const Shared& s, int part, int lane) {
    // columns in use: up to the last token, or one per token
    const int cols = d.scatter ? 32 - __clz(d.mask) : __popc(d.mask);
    if (NT == 1 || cols <= 8) chunk_n<1>(d, s, part, lane);
    else if (NT == 2 || cols <= 16) chunk_n<(NT < 2 ? 1 : 2)>(d, s, part, lane);
    else chunk_n<NT>(d, s, part, lane);
  }
  __device__ __forceinline__ void store(float* red, int warp, int lane) const {
    const int g = lane >> 2, q = lane & 3;
    float* w = red + warp * (8 * NT * kRedStride);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float* p = w + (8 * n + 2 * q) * kRedStride + g;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        p[16 * m] = c[m][n][0];
        p[16 * m + kRedStride] = c[m][n][1];
        p[16 * m + 8] = c[m][n][2];
        p[16 * m + 8 + kRedStride] = c[m][n][3];
      }
    }
  }
};
// fp32: lane = row, and where the tile has fewer than 32 rows the lanes behind the rows (a power
// of two) take other parts of the contraction: with one row per lane alone, a 5-row tile left 27
// lanes to repeat it and the FMAs bound it.
template <int NT> struct Acc<true, NT> {
  float c[8 * NT];
  int rows, r0;  // lanes per part of the contraction; rows of the first row block
  __device__ __forceinline__ void zero() {
    rows = 32;
    r0 = 16;
#pragma unroll
    for (int n = 0; n < 8 * NT; ++n) c[n] = 0.f;
  }
  __device__ __forceinline__ void chunk(const SlotDesc& d, const Shared& s, int part, int lane) {
    const int P = d.pitch;
    // Vectors of the row held together.  The loop over tokens is unrolled, and its code is what bounds
    // many tokens (12 experts, d=776, F=4812, T=24: 582 us with 8 and a second loop for whole chunks,
    // 349 with this one, 307 with 4; T=12: 140 with 8, 178 with 4): blocks of 8 tokens that the slot
    // does not hold are passed over at once.
    constexpr int V = NT == 4 ? 4 : 8;
    const int n_rows = d.r0 + d.r1;
    rows = n_rows > 16 ? 32 : n_rows > 8 ? 16 : n_rows > 4 ? 8 : 4;
    r0 = d.r0;
    const int ks = 32 / rows, k = lane / rows;  // parts of the contraction, this lane's
    const uint32_t base = smem_u32(s.ring) + d.off;
    const int nb = __popc(d.mask);
    const uint32_t a = base + min(lane & (rows - 1), n_rows - 1) * P + k * 16;
    const uint32_t b = base + n_rows * P + k * 16;
#pragma unroll 1
    for (int v0 = part * V * ks; v0 < d.kvec; v0 += V * ks * kGroupWarps<true, NT>) {
      const int left = d.kvec - v0 - k;  // this lane's vectors: 0, ks, 2 ks, ...
      float w[V][4];
#pragma unroll
      for (int i = 0; i < V; ++i)
        Vec<float>::to_f32(i * ks < left ? lds_vec(a + (v0 + i * ks) * 16) : make_uint4(0, 0, 0, 0),
                           w[i]);
      bool held = true;
#pragma unroll
      for (int n = 0; n < 8 * NT; ++n) {
        if (n % 8 == 0) held = d.scatter ? ((d.mask >> n) & 0xffu) != 0 : n < nb;
        if (!held) continue;
        int slot = n;
        if (d.scatter) {
          if (!((d.mask >> n) & 1u)) continue;
          slot = __popc(d.mask & ((1u << n) - 1u));
        } else if (n >= nb) {
          continue;
        }
        const uint32_t xb = b + slot * P + v0 * 16;
        float s4[4] = {0.f, 0.f, 0.f, 0.f};
        float x[V][4];
#pragma unroll
        for (int i = 0; i < V; ++i)
          Vec<float>::to_f32(i * ks < left ? lds_vec(xb + i * ks * 16) : make_uint4(0, 0, 0, 0),
                             x[i]);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) s4[j] = fmaf(w[i][j], x[i][j], s4[j]);
        c[n] += (s4[0] + s4[1]) + (s4[2] + s4[3]);
      }
    }
  }
  __device__ __forceinline__ void store(float* red, int warp, int lane) const {
    float* w = red + warp * (8 * NT * kRedStride);
    const int at = lane < r0 ? lane : 16 + lane - r0;  // the second row block begins at 16
#pragma unroll
    for (int n = 0; n < 8 * NT; ++n) {
      float v = c[n];
      for (int o = rows; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane < rows && at < 32) w[n * kRedStride + at] = v;
    }
  }
};

// The total of output (row block m, row i of it, column n): the partial sums of `warps` warps (of
// a group, or all) in order.
template <int NT>
__device__ __forceinline__ float red_sum(const float* red, int warps, int m, int i, int n) {
  float v = 0.f;
  const float* p = red + n * kRedStride + 16 * m + i;
#pragma unroll
  for (int w = 0; w < kConsumerWarps; ++w)
    if (w < warps) v += p[w * (8 * NT * kRedStride)];
  return v;
}

// The total of row i of a pair tile's second matrix.
template <bool F32, int NT>
__device__ __forceinline__ float red_sum_second(const SlotDesc& d, const float* red, int warps,
                                                int i, int n) {
  const bool fold = !F32 && pair_fold(d);
  return red_sum<NT>(red, warps, fold ? 0 : 1, fold ? 8 + i : i, n);
}

// Who runs a tile's epilogue: `count` threads, this one the `index`-th of them, on the partial
// sums of `warps` warps.
struct Crew {
  int index, count, warps;
};

// A phase whose tiles have few slots gives a tile to one group, which sums up and finishes it by
// itself while the others are at other tiles: shared by all groups, a tile of two slots costs the
// latency of both barriers and of the epilogue each time (32 experts, d=512, F=4096 T=16: 144 us
// shared, 121 us by one group; Granite-shaped T=16 42.9 and 41.9).  Not in fp32, whose FMAs take
// longer than those barriers (12+1 experts T=4: 80 us shared, 98 us by one group).  With more
// slots to a tile the ring would hold slots of one group's tile only.
//   No group waits for use n + 1 of a slot's barrier before use n has completed: when it
// waits for slots of its next tile, at most kGroups tiles on, the slots up to kInFlight before
// the tile it finished have been filled.
constexpr int kSoloChunks = 4;
static_assert(kGroups<false, 1> * kSoloChunks + kInFlight <= kSlots,
              "no parity of a slot is ambiguous");
template <bool F32, int NT>
__device__ __forceinline__ bool solo_tiles(int tiles, int chunks) {
  return !F32 && chunks <= kSoloChunks && tiles >= kGroups<F32, NT>;
}

// Consume the tiles of two phases: tiles[0] of chunks[0] slots each, then `between`, then
// tiles[1] of chunks[1].  epilogue(desc, red, crew) runs once per tile, with the descriptor of
// its last slot and the partial sums.  `solo`: the first phase's tiles go to one group each (see
// solo_tiles).  Else all consumer threads run it: after the next tile's slots are
// consumed, or, for the last tile of a phase, at once.  A buffer of partial sums is written again
// only after its tile's epilogue: with two buffers because each warp arrives for a tile after its
// own epilogue of the tile before, and waits for all arrivals of that one first; with one buffer
// because it waits for all epilogues of the tile before.
//   between(ok) holds barriers of the consumer threads: every warp calls it once, also one that
// gives up before (every wait is bounded); it returns whether all are well.
// One loop for both phases on purpose: its code is there once.
template <bool F32, int NT, typename Epi, typename Between>
__device__ __forceinline__ void consume(const Shared& s, const int (&tiles)[2],
                                        const int (&chunks)[2], bool solo, int32_t* status,
                                        Epi&& epilogue, Between&& between) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t group = warp / kGroupWarps<F32, NT>;
  const int part = warp % kGroupWarps<F32, NT>;
  const int total = tiles[0] + tiles[1];
  constexpr int kWarpFloats = 8 * NT * kRedStride;
  uint32_t it = 0;       // slots passed
  int tile = solo ? group : 0;
  uint32_t n = 0;        // tiles of all groups stored
  bool pending = false;  // tile n - 1 of them awaits its epilogue
  bool crossed = false, ok = true;
  Acc<F32, NT> acc;
#pragma unroll 1
  for (;;) {
    const bool flush = pending && ((tile == tiles[0] && !crossed) || tile == total);
    bool last = false;
    SlotDesc d;
    if (!flush) {
      if (tile >= tiles[0] && !crossed) {
        crossed = true;
        if (!between(ok)) return;
        if (solo) {
          solo = false;
          tile = tiles[0];
          it = tiles[0] * chunks[0];
        }
      }
      if (tile == total) return;
      acc.zero();
      if (solo) it = tile * chunks[0];
      const uint32_t end = it + chunks[crossed ? 1 : 0], step = solo ? 1 : kGroups<F32, NT>;
#pragma unroll 1
      for (it += solo ? 0 : (group - it) % kGroups<F32, NT>; it < end; it += step) {
        const uint32_t slot = it % kSlots;
        ok = __all_sync(0xffffffffu,
                        wait(&s.full[slot], (it / kSlots) & 1u, s.abort_flag, status));
        if (!ok) break;
        d = s.desc[slot];
        acc.chunk(d, s, part, lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.empty[slot]);
        last = d.last != 0;
      }
      it = end;
      if (solo) {
        ok = group_all<F32, NT>(group, ok);  // and the tile before is finished
        acc.store(s.red, warp, lane);
        ok = group_all<F32, NT>(group, ok);
        if (!ok) {
          between(false);
          return;
        }
        constexpr int kCrew = 32 * kGroupWarps<F32, NT>;
        epilogue(d, s.red + group * kGroupWarps<F32, NT> * kWarpFloats,
                 Crew{static_cast<int>(threadIdx.x) % kCrew, kCrew, kGroupWarps<F32, NT>});
        tile += kGroups<F32, NT>;
        continue;
      }
    }
    if (pending && ok) {
      const uint32_t t = n - 1;
      ok = __all_sync(0xffffffffu, wait(&s.sums[t & 1u], (t >> 1) & 1u, s.abort_flag, status));
      if (ok)
        epilogue(s.tile[t & 1u], s.red + (t % kRedBufs<NT>) * kRedFloats<NT>,
                 Crew{static_cast<int>(threadIdx.x), kConsumers, kConsumerWarps});
      if (kRedBufs<NT> == 1) {
        __syncwarp();
        if (lane == 0) mbar_arrive(s.freed);
      }
    }
    pending = false;
    if (!ok) {
      if (!crossed) between(false);
      return;
    }
    if (!flush) {
      if (kRedBufs<NT> == 1 && n > 0 &&
          !__all_sync(0xffffffffu, wait(s.freed, (n - 1) & 1u, s.abort_flag, status))) {
        if (!crossed) between(false);
        return;
      }
      acc.store(s.red + (n % kRedBufs<NT>) * kRedFloats<NT>, warp, lane);
      if (last && part == 0 && lane == 0) s.tile[n & 1] = d;
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.sums[n & 1]);
      ++n;
      ++tile;
      pending = true;
    }
  }
}

}  // namespace few
}  // namespace moe
