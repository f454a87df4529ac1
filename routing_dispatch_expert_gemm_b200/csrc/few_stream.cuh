// Weight-streaming engine of the few-token kernels (at most 32 tokens: few_layer.cu,
// adapter_few.cu).  With so few tokens every product is bound by reading its weights once
// from HBM, so the kernels are built around the stream, not around the MMA:
//
//   * One CTA per SM, all resident (cooperative launch).  Every phase cuts its output rows
//     (weight rows) evenly over the CTAs, at single-row granularity, whatever the expert.
//   * Warp 8 is the producer: it cuts the CTA's rows into tiles of up to 32 weight rows and
//     the contraction into chunks of 1 KB per row, and copies each chunk's weight rows and
//     token rows to shared memory with one bulk copy per row.  Slots of a byte ring are
//     sized by the rows they hold, so thin tiles (a phase that leaves a CTA 7 rows) still
//     keep the whole ring in flight; the stream does not stop between tiles or phases.
//   * Warps 0-7 consume: each takes 1/8 of the chunk's contraction for all rows and tokens.
//     bf16: mma.sync m16n8k16 with the weight rows on M and the tokens on N, fed by 16-byte
//     shared loads: thread q of a quad takes 8 consecutive k of its row, for weights and
//     tokens alike, which only permutes the k index inside a 32-wide block.  At 8 tokens
//     the pipe needs 2 * 8 FLOP per weight (about 53 TFLOP/s at the full HBM rate), far
//     below even the warp-level MMA rate, and there is no tensor-memory round trip at the
//     end of a 7-row tile; that is why this is not tcgen05, whose M is at least 64 rows.
//     fp32: FMA, one weight row per lane.
//   * The 8 partial sums per output meet in shared memory in warp order (fixed order: the
//     same bits every run) and the caller's epilogue consumes the total.
//
// The MMA reads whole 16-row and 8-token fragments; rows past a tile's last one are clamped
// to it.  A garbage row or token column only reaches its own outputs, which are not stored.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace few {

constexpr int kMaxTokens = 32;       // one token-mask word
constexpr int kConsumerWarps = 8;
constexpr int kConsumers = 32 * kConsumerWarps;
constexpr int kThreads = kConsumers + 32;
constexpr int kSlots = 16;           // slots in flight at most
constexpr int kChunkBytes = 1024;    // contraction bytes per row and chunk
constexpr int kChunkVecs = kChunkBytes / 16;
constexpr uint32_t kSmemBytes = 227 * 1024;
constexpr int kTileRows = 32;        // weight rows per tile at most (two MMA row blocks)
constexpr int kRedStride = 36;       // floats per token column of the partial sums: the MMA
                                     // fragment's stores and the row-wise reads hit 32 banks

// Row pitch of a slot.  bf16 fragments read 64 bytes of two rows per 8-lane phase (pitch
// 64 mod 128), fp32 lanes read 16 bytes of 8 rows (pitch 16 mod 128).
template <bool F32> constexpr int kPitch = F32 ? kChunkBytes + 16 : kChunkBytes + 64;

// One slot of the ring, written by the producer before the slot's barrier completes.
struct alignas(16) SlotDesc {
  uint32_t off;    // byte offset in the ring
  int16_t r0, r1;  // weight rows of the first and second row block (the second follows the
                   // first in the slot; in a pair tile they are the gate and the up rows)
  int16_t kvec;    // valid 16-byte vectors along the contraction
  int8_t first, last;  // first / last chunk of the tile
  uint32_t mask;   // tokens whose rows the slot holds, ascending
  int32_t scatter; // 1: the token of mask bit t is column t; 0: columns are 0..popc(mask)-1
  int32_t seg;     // caller's: what the tile belongs to
  int32_t row;     // caller's: first output row of the tile
};

struct Shared {
  uint64_t* full;
  uint64_t* empty;
  SlotDesc* desc;
  volatile int* abort_flag;
  uint8_t* ring;
  float* red;      // [2][8 warps][8 NT][kRedStride]
  uint32_t ring_bytes;
};

constexpr int kCtlBytes = 2 * kSlots * 8 + kSlots * 32 + 64;
static_assert(sizeof(SlotDesc) == 32, "descriptor size");
template <int NT> constexpr int kRedFloats = kConsumerWarps * 8 * NT * kRedStride;
// The largest slot: a full tile and 32 token rows.
constexpr uint32_t kMaxSlotBytes = (kTileRows + kMaxTokens) * (kChunkBytes + 64);

// Control words, partial sums, the caller's tables (table_bytes), then the ring.
template <int NT>
__device__ __forceinline__ Shared carve(uint8_t* smem, uint32_t table_bytes, uint32_t total) {
  Shared s;
  s.full = reinterpret_cast<uint64_t*>(smem);
  s.empty = s.full + kSlots;
  s.desc = reinterpret_cast<SlotDesc*>(s.empty + kSlots);
  s.abort_flag = reinterpret_cast<volatile int*>(s.desc + kSlots);
  s.red = reinterpret_cast<float*>(smem + kCtlBytes);
  const uint32_t at = kCtlBytes + 2 * kRedFloats<NT> * 4 + table_bytes;
  s.ring = smem + at;
  s.ring_bytes = (total - at) & ~15u;
  return s;
}

__device__ __forceinline__ void init_shared(const Shared& s) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], kConsumerWarps);
    }
    *s.abort_flag = 0;
    fence_mbar_init();
  }
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

// ---------------------------------------------------------------------------------
// Grid barrier: counts arrivals in the workspace header (all CTAs are resident).  Both
// words are zero between launches: the last CTA to leave clears them.
// ---------------------------------------------------------------------------------
struct GridSync {
  unsigned int* count;  // arrivals so far in this launch
  unsigned int* left;   // CTAs that have left
};

__device__ __forceinline__ void grid_arrive(const GridSync& g) {  // one thread, after a barrier
  __threadfence();
  atomicAdd(g.count, 1u);
}
// Bounded: returns false (and records MOE_ERR_TIMEOUT) when the arrivals do not come.
__device__ __forceinline__ bool grid_wait(const GridSync& g, unsigned int target,
                                          volatile int* abort_flag, int32_t* status) {
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    unsigned int v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(g.count) : "memory");
    if (v >= target) return true;
    if ((it & 63u) == 0) {
      if (*abort_flag != 0) return false;
      if (static_cast<int64_t>(global_timer_ns() - t0) > kWaitLimitNs) {
        *abort_flag = 1;
        record_status(status, MOE_ERR_TIMEOUT);
        return false;
      }
    }
  }
}
__device__ __forceinline__ void grid_leave(const GridSync& g) {  // one thread, waits all passed
  __threadfence();
  if (atomicAdd(g.left, 1u) == gridDim.x - 1) {
    *g.count = 0;
    *g.left = 0;
  }
}
// Make this thread's global writes visible to bulk copies issued by other threads after a
// barrier (generic proxy -> async proxy), and the reader's counterpart.
__device__ __forceinline__ void fence_proxy_async_all() {
  asm volatile("fence.proxy.async;" ::: "memory");
}

// ---------------------------------------------------------------------------------
// Producer: a FIFO byte ring (warp-uniform state; every lane runs it)
// ---------------------------------------------------------------------------------
template <bool F32>
struct Producer {
  Shared s;
  int32_t* status;
  uint32_t head = 0;   // next free byte
  uint32_t it = 0;     // slots issued
  uint32_t tail = 0;   // slots known to be released

  __device__ __forceinline__ bool wait_tail() {  // the oldest live slot is released
    const uint32_t slot = tail % kSlots;
    if (!mbar_wait_bounded(&s.empty[slot], (tail / kSlots) & 1u, s.abort_flag, kWaitLimitNs,
                           status))
      return false;
    ++tail;
    return true;
  }

  // Place `bytes` in the ring without waiting for any slot >= `barrier_it`; *off is the
  // offset.  Returns 1 when placed, 0 when it would have to wait for such a slot, -1 on abort.
  __device__ __forceinline__ int place(uint32_t bytes, uint32_t barrier_it, uint32_t* off) {
    for (;;) {
      const uint32_t live = it - tail;
      if (live == 0) {
        head = bytes;
        *off = 0;
        return 1;
      }
      if (live < kSlots) {
        const uint32_t toff = s.desc[tail % kSlots].off;
        if (head > toff) {
          if (s.ring_bytes - head >= bytes) { *off = head; head += bytes; return 1; }
          if (toff > bytes) { *off = 0; head = bytes; return 1; }
        } else if (toff - head > bytes) {
          *off = head;
          head += bytes;
          return 1;
        }
      }
      if (tail >= barrier_it) return 0;
      if (!wait_tail()) return -1;
    }
  }

  // Open the slot: descriptor, then the barrier's expected bytes.
  __device__ __forceinline__ void open(const SlotDesc& d, uint32_t bytes) {
    const uint32_t slot = it % kSlots;
    if ((threadIdx.x & 31) == 0) {
      s.desc[slot] = d;
      mbar_arrive_expect_tx(&s.full[slot], bytes);
    }
    __syncwarp();
  }
  __device__ __forceinline__ uint8_t* row_ptr(uint32_t off, int row) const {
    return s.ring + off + static_cast<uint32_t>(row) * kPitch<F32>;
  }
  // Before leaving early: every copy in flight has landed.
  __device__ __forceinline__ void drain() {
    const uint32_t n = min(it, static_cast<uint32_t>(kSlots));
    for (uint32_t i = it - n; i < it; ++i)
      mbar_wait_bounded(&s.full[i % kSlots], (i / kSlots) & 1u, nullptr, kWaitLimitNs, status);
  }
};

// ---------------------------------------------------------------------------------
// Consumers
// ---------------------------------------------------------------------------------
__device__ __forceinline__ uint4 lds_vec(const uint8_t* p) {
  return *reinterpret_cast<const uint4*>(p);
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

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
  __device__ __forceinline__ void chunk(const SlotDesc& d, const uint8_t* base, int warp,
                                        int lane) {
    constexpr int P = kPitch<false>;
    const int g = lane >> 2, q = lane & 3;
    const int nb = __popc(d.mask);
    // 16-row blocks: rows past a block's last one are clamped to it
    const uint8_t* a00 = base + min(g, d.r0 - 1) * P;
    const uint8_t* a01 = base + min(g + 8, d.r0 - 1) * P;
    const uint8_t* a10 = base + (d.r0 + min(g, max(d.r1 - 1, 0))) * P;
    const uint8_t* a11 = base + (d.r0 + min(g + 8, max(d.r1 - 1, 0))) * P;
    const uint8_t* b = base + (d.r0 + d.r1) * P;
    const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int h = 0; h < kChunkVecs / 4 / kConsumerWarps; ++h) {
      const int kb = warp + h * kConsumerWarps;  // 32-wide block of the contraction
      if (kb * 4 >= d.kvec) break;
      const int v = kb * 4 + q;
      const bool in = v < d.kvec;  // a ragged contraction ends inside a block: zeros
      const int o = v * 16;
      const uint4 w00 = in ? lds_vec(a00 + o) : z, w01 = in ? lds_vec(a01 + o) : z;
      uint4 w10 = z, w11 = z;
      if (d.r1 > 0 && in) { w10 = lds_vec(a10 + o); w11 = lds_vec(a11 + o); }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint4 x = z;
        if (d.scatter) {  // column = token: zeros for the tokens the slot does not hold
          if (((d.mask >> (8 * n)) & 0xffu) == 0) continue;
          const int t = 8 * n + g;
          const int slot = __popc(d.mask & ((1u << t) - 1u));
          if (in && ((d.mask >> t) & 1u)) x = lds_vec(b + slot * P + o);
        } else {
          if (8 * n >= nb) continue;
          if (in) x = lds_vec(b + min(8 * n + g, nb - 1) * P + o);
        }
        mma_bf16(c[0][n], w00.x, w01.x, w00.y, w01.y, x.x, x.y);
        mma_bf16(c[0][n], w00.z, w01.z, w00.w, w01.w, x.z, x.w);
        if (d.r1 > 0) {
          mma_bf16(c[1][n], w10.x, w11.x, w10.y, w11.y, x.x, x.y);
          mma_bf16(c[1][n], w10.z, w11.z, w10.w, w11.w, x.z, x.w);
        }
      }
    }
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
template <int NT> struct Acc<true, NT> {
  float c[8 * NT];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int n = 0; n < 8 * NT; ++n) c[n] = 0.f;
  }
  __device__ __forceinline__ void chunk(const SlotDesc& d, const uint8_t* base, int warp,
                                        int lane) {
    constexpr int P = kPitch<true>;
    const int nb = __popc(d.mask);
    const int row = lane < 16 ? min(lane, d.r0 - 1) : d.r0 + min(lane - 16, max(d.r1 - 1, 0));
    const uint8_t* a = base + (lane >= 16 && d.r1 == 0 ? 0 : row) * P;
    const uint8_t* b = base + (d.r0 + d.r1) * P;
    constexpr int V = kChunkVecs / kConsumerWarps;
#pragma unroll 2
    for (int i = 0; i < V; ++i) {
      const int v = warp * V + i;
      if (v >= d.kvec) break;
      const uint4 wv = lds_vec(a + v * 16);
      float w[4];
      Vec<float>::to_f32(wv, w);
#pragma unroll
      for (int n = 0; n < 8 * NT; ++n) {
        int slot = n;
        if (d.scatter) {
          if (!((d.mask >> n) & 1u)) continue;
          slot = __popc(d.mask & ((1u << n) - 1u));
        } else if (n >= nb) {
          continue;
        }
        float x[4];
        Vec<float>::to_f32(lds_vec(b + slot * P + v * 16), x);
#pragma unroll
        for (int j = 0; j < 4; ++j) c[n] = fmaf(w[j], x[j], c[n]);
      }
    }
  }
  __device__ __forceinline__ void store(float* red, int warp, int lane) const {
    float* w = red + warp * (8 * NT * kRedStride);
#pragma unroll
    for (int n = 0; n < 8 * NT; ++n) w[n * kRedStride + lane] = c[n];
  }
};

// The total of output (row block m, row i of it, column n): the 8 warps in order.
template <int NT>
__device__ __forceinline__ float red_sum(const float* red, int m, int i, int n) {
  float v = 0.f;
  const float* p = red + n * kRedStride + 16 * m + i;
#pragma unroll
  for (int w = 0; w < kConsumerWarps; ++w) v += p[w * (8 * NT * kRedStride)];
  return v;
}

// Consume slots until `tiles` tiles are done.  epilogue(desc, red) runs on all consumer
// threads once per tile with the 8 warps' partial sums.  Returns false on abort; a warp that
// gives up still passes the remaining barriers, so none of the others waits for it forever.
template <bool F32, int NT, typename Epi>
__device__ __forceinline__ bool consume(const Shared& s, uint32_t& it, uint32_t& tile,
                                        int tiles, int32_t* status, Epi&& epilogue) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Acc<F32, NT> acc;
  for (int done = 0; done < tiles;) {
    const uint32_t slot = it % kSlots;
    const bool ok = mbar_wait_bounded(&s.full[slot], (it / kSlots) & 1u, s.abort_flag,
                                      kWaitLimitNs, status);
    if (!__all_sync(0xffffffffu, ok)) {
      for (; done < tiles; ++done) consumer_sync();
      return false;
    }
    const SlotDesc d = s.desc[slot];
    if (d.first) acc.zero();
    acc.chunk(d, s.ring + d.off, warp, lane);
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.empty[slot]);
    ++it;
    if (d.last) {
      // double-buffered: a buffer's readers passed the other buffer's barrier
      float* red = s.red + (tile & 1u) * kRedFloats<NT>;
      acc.store(red, warp, lane);
      consumer_sync();
      epilogue(d, red);
      ++tile;
      ++done;
    }
  }
  return true;
}

}  // namespace few
}  // namespace moe
