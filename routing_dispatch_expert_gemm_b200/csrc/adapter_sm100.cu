// Projections with per-token low-rank adapters for larger batches (bf16, moe_adapter_linear and
// moe_adapter_gate_up where the few-token kernel does not run):
//   p[t] = W x_t + s_a B_a (A_a x_t),  a = adapter of token t (-1: none)
//   linear   y[t] = p[t] (+ addend[t])         gate_up  h[t] = SiLU(p_gate[t]) * p_up[t]
//
// Two launches, the second starting under the first (programmatic dependent launch); few tokens
// beside few tiles take one, in which the GEMM's epilogue warps shrink while W streams:
//   adapter_shrink_kernel  u[t] = s_a A_a x_t, summed in fp32, kept as two bf16 halves.  A CTA takes
//       16 consecutive tokens and runs warp-level MMAs (tokens on M, ranks on N) once per adapter
//       in use among them (dealt over CTAs when there are few), its 8 warps splitting the
//       contraction.
//       A and x are read straight into MMA fragments (16-byte loads; the k permutation inside
//       a 32-wide block is the same on both sides).  2 T rank d_in FLOP and the bytes of x and
//       the A matrices: small beside W's product, and overlapped with its start.
//   adapter_gemm_kernel    W x on tcgen05: 128 rows of W on M, up to 256 tokens on N (128 with
//       a second projection beside it), fp32 accumulators in TMEM, both operands by TMA.
//       B u is a few more K blocks of the same product: with u split into two bf16 halves
//       (16 bits in all), a block holds 8 units of 8 ranks, [B_a | B_a] against the high and
//       low halves of the tokens of adapter a and zeros for the others.  A block costs what 64
//       columns of W cost; prompts of a few requests need one or two (fp32 FMA in the epilogue
//       instead: T=4099, rank 16: 165 us; rank 32 gate/up T=1531: 560 us).
//       Token blocks with more adapters than pay this (kAdapterTokens: 16 at most), and the split
//       form below, add B_a u in the epilogue, in fp32 FMA: a thread holds one row of W for 8
//       tokens.
// With enough tiles the GEMM is persistent, the epilogue of a tile overlapping the next tile's
// MMAs (two accumulator sets).  With few tiles (a decode batch on a small projection) a cluster
// of 2..8 CTAs splits the contraction of one tile; the partial tiles meet in distributed
// shared memory, where each CTA finishes its share of the tokens in rank order (no float atomics,
// the same bits every run).
#include <algorithm>

#include "adapter_gemm.cuh"
#include "gemm_common.cuh"
#include "grid_sync.cuh"
#include "internal.h"

namespace moe {
namespace {

using gemm::BK;

// ------------------------------------------------------------------------------ shrink
constexpr int kShrinkWarps = 8;
constexpr int kShrinkTokens = 16;  // MMA rows
constexpr int kShrinkRanks = 32;   // ranks per pass: 4 MMA column blocks
constexpr int kMaxParts = 8;         // pieces of the contraction, in the split form
// Tokens times pieces beyond one.  A launch of its own has two CTAs per SM and at least two per 16
// tokens, so on 148 SMs its pieces end at 148 * 16 / T anyway.
constexpr int64_t kPartTokens = 2560;

struct ShrinkParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* a[2];
  const float* scale;
  const int32_t* ids;
  const int32_t* n_tokens;
  uint4* u;         // [2, T, rank / 8]: 8 ranks as 8 high and 8 low bf16 halves (2 vectors)
  float* u_parts;   // else [parts, 2, T, rank]: fp32 sums of `parts` pieces of the contraction
  int turns, parts; // a token tile's work is dealt over turns x parts CTAs (see shrink_tile)
  int32_t* blocks;  // [token blocks][1 + kMaxBlockAdapters]: adapters of each GEMM token block,
                    // without u_parts
  uint8_t* broken;  // [2, T], with u: of tokens that have an adapter, whether a half is not finite
  int32_t* status;
  int T, d_in, n, rank, block_tokens;
};

// Adapters of token block `tb`, by the whole CTA: their number, then the adapters in the order
// of their first token; or kMaxBlockAdapters + 1 when the epilogue is to expand them (the rule
// beside kAdapterTokens).
__device__ __forceinline__ void list_block_adapters(const ShrinkParams& p, int tb, int live) {
  __shared__ int s_ids[32 * kShrinkWarps], s_count[kShrinkWarps];
  const int tid = threadIdx.x, t = tb * p.block_tokens + tid;
  int id = tid < p.block_tokens && t < live ? __ldg(p.ids + t) : -1;
  if (id < 0 || id >= p.n) id = -1;
  s_ids[tid] = id;
  __syncthreads();
  bool first = id >= 0;
#pragma unroll 8
  for (int i = 0; i < tid; ++i) first = first && s_ids[i] != id;
  const uint32_t mask = __ballot_sync(0xffffffffu, first);
  if ((tid & 31) == 0) s_count[tid >> 5] = __popc(mask);
  __syncthreads();
  int before = __popc(mask & ((1u << (tid & 31)) - 1u)), all = 0;
  for (int w = 0; w < kShrinkWarps; ++w) {
    if (w < (tid >> 5)) before += s_count[w];
    all += s_count[w];
  }
  int32_t* out = p.blocks + static_cast<size_t>(tb) * (1 + kMaxBlockAdapters);
  const bool few =
      all * kAdapterTokens <= min(p.block_tokens, live - tb * p.block_tokens) ||
      all * (p.rank / 8) * 2 <= kSmallBlocks * 8;
  if (tid == 0) out[0] = few || all == 0 ? all : kMaxBlockAdapters + 1;
  if (first && before < kMaxBlockAdapters) out[1 + before] = id;
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Partial product of one warp: its share of vectors v_lo .. dv - 1 of the contraction of 16
// tokens with 8 NB ranks.
// U 32-wide blocks are loaded before the first MMA (one at a time the loads' latency bounds).
template <int NB>
__device__ __forceinline__ void shrink_partial(float (&c)[4][4], const __nv_bfloat16* x0,
                                               const __nv_bfloat16* x1, const __nv_bfloat16* ar,
                                               int d_in, int v_lo, int dv, int warp, int q) {
  constexpr int U = NB == 4 ? 2 : 4;
  constexpr int kStep = 4 * kShrinkWarps;  // vectors between a warp's blocks
  const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll 1
  for (int v0 = v_lo + warp * 4; v0 < dv; v0 += U * kStep) {
    uint4 a[U][2], b[U][NB];
#pragma unroll
    for (int h = 0; h < U; ++h) {
      const int v = v0 + h * kStep + q;
      const bool in = v < dv;
      a[h][0] = in ? ld_vec(x0 + v * 8) : z;
      a[h][1] = in ? ld_vec(x1 + v * 8) : z;
#pragma unroll
      for (int n = 0; n < NB; ++n)
        b[h][n] = in ? ld_vec(ar + static_cast<size_t>(n) * 8 * d_in + v * 8) : z;
    }
#pragma unroll
    for (int h = 0; h < U; ++h) {
#pragma unroll
      for (int n = 0; n < NB; ++n)
        mma_16816(c[n], a[h][0].x, a[h][1].x, a[h][0].y, a[h][1].y, b[h][n].x, b[h][n].y);
#pragma unroll
      for (int n = 0; n < NB; ++n)
        mma_16816(c[n], a[h][0].z, a[h][1].z, a[h][0].w, a[h][1].w, b[h][n].z, b[h][n].w);
    }
  }
}

// Barrier of the 256 threads that shrink.
__device__ __forceinline__ void shrink_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kShrinkWarps) : "memory");
}
using ShrinkSums = float[kShrinkWarps][kShrinkTokens][kShrinkRanks + 1];

// Projection m of the 16 tokens of `tile` by 256 threads: every turns-th adapter of theirs from
// `turn` on, piece `part` of the contraction.  PARTS: fp32 pieces, else u.
template <bool PARTS>
__device__ __forceinline__ void shrink_tile(const ShrinkParams& p, ShrinkSums& red, int tile,
                                            int turn, int m, int part, int live) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int parts = PARTS ? p.parts : 1;
  const int t0 = tile * kShrinkTokens;
  const int dv = p.d_in / 8, blocks = (dv + 3) / 4;  // whole 32-wide blocks to a part
  const int v_lo = blocks * part / parts * 4, v_hi = min(dv, blocks * (part + 1) / parts * 4);
  const int nt = min(kShrinkTokens, live - t0);
  int id = lane < nt ? __ldg(p.ids + t0 + lane) : -1;
  if (id < -1 || id >= p.n) {
    if (turn == 0 && m == 0 && part == 0 && warp == 0)
      record_status(p.status, MOE_ERR_BAD_ADAPTER_ID);
    id = -1;
  }
  const uint32_t same = __match_any_sync(0xffffffffu, id);
  uint32_t leaders = __ballot_sync(0xffffffffu, id >= 0 && __ffs(same) - 1 == lane);
  // x rows of this lane's fragment rows (rows past the last token: the last one's, unused)
  const __nv_bfloat16* x0 = p.x + static_cast<size_t>(t0 + min(g, nt - 1)) * p.d_in;
  const __nv_bfloat16* x1 = p.x + static_cast<size_t>(t0 + min(g + 8, nt - 1)) * p.d_in;

  for (int i = 0; leaders != 0; leaders &= leaders - 1, ++i) {
    if (i % p.turns != turn) continue;  // the same for every warp
    const int lead = __ffs(leaders) - 1;
    const int a_id = __shfl_sync(0xffffffffu, id, lead);
    const uint32_t tokens = __shfl_sync(0xffffffffu, same, lead);
    const __nv_bfloat16* A =  // (an index into p.a would put p on the stack)
        (m == 0 ? p.a[0] : p.a[1]) + static_cast<size_t>(a_id) * p.rank * p.d_in;
    const float sc = p.scale != nullptr ? __ldg(p.scale + a_id) : 1.f;
    const int t = threadIdx.x / (kShrinkRanks / 2);  // this thread's token of the sums
    bool broken = false;
    for (int j0 = 0; j0 < p.rank; j0 += kShrinkRanks) {
      const int nb = min(4, (p.rank - j0) / 8);  // rank is a multiple of 8
      const __nv_bfloat16* ar = A + static_cast<size_t>(j0 + g) * p.d_in;
      float c[4][4] = {};
      if (nb == 1) shrink_partial<1>(c, x0, x1, ar, p.d_in, v_lo, v_hi, warp, q);
      else if (nb == 2) shrink_partial<2>(c, x0, x1, ar, p.d_in, v_lo, v_hi, warp, q);
      else if (nb == 3) shrink_partial<3>(c, x0, x1, ar, p.d_in, v_lo, v_hi, warp, q);
      else shrink_partial<4>(c, x0, x1, ar, p.d_in, v_lo, v_hi, warp, q);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        red[warp][g][8 * n + 2 * q] = c[n][0];
        red[warp][g][8 * n + 2 * q + 1] = c[n][1];
        red[warp][g + 8][8 * n + 2 * q] = c[n][2];
        red[warp][g + 8][8 * n + 2 * q + 1] = c[n][3];
      }
      shrink_sync();
      // a thread: two neighbouring ranks of a token
      const int j = threadIdx.x % (kShrinkRanks / 2) * 2;
      if (((tokens >> t) & 1u) && j0 + j < p.rank) {
        float v[2] = {0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kShrinkWarps; ++w) {
          v[0] += red[w][t][j];
          v[1] += red[w][t][j + 1];
        }
        v[0] *= sc;
        v[1] *= sc;
        if constexpr (PARTS) {
          *reinterpret_cast<float2*>(
              p.u_parts + ((static_cast<size_t>(part) * 2 + m) * p.T + t0 + t) * p.rank + j0 + j) =
              make_float2(v[0], v[1]);
        } else {
          const uint32_t hi = gemm::pack_bf16(v[0], v[1]);
          // an infinity has no low half (inf - inf is NaN)
          const float h0 = __uint_as_float(hi << 16), h1 = __uint_as_float(hi & 0xffff0000u);
          const uint32_t lo = gemm::pack_bf16(isfinite(h0) ? v[0] - h0 : 0.f,
                                              isfinite(h1) ? v[1] - h1 : 0.f);
          broken |= !isfinite(h0) || !isfinite(h1);
          uint32_t* u = reinterpret_cast<uint32_t*>(
              p.u + ((static_cast<size_t>(m) * p.T + t0 + t) * p.rank + j0) / 4) + (j / 8) * 8 +
              (j % 8) / 2;
          u[0] = hi;
          u[4] = lo;
        }
      }
      shrink_sync();
    }
    if constexpr (!PARTS) {  // a half warp holds a token
      const uint32_t any = __ballot_sync(0xffffffffu, broken) >> (lane & 16);
      if ((lane & 15) == 0 && ((tokens >> t) & 1u))
        p.broken[static_cast<size_t>(m) * p.T + t0 + t] = (any & 0xffffu) != 0;
    }
  }
}

template <bool PARTS>
__global__ void __launch_bounds__(32 * kShrinkWarps, 2) adapter_shrink_kernel(const ShrinkParams p) {
  __shared__ ShrinkSums red;
  pdl_trigger();  // the GEMM may start; it waits for this grid before it reads u
  const int live = live_tokens(p.n_tokens, p.T);
  const int tiles = (p.T + kShrinkTokens - 1) / kShrinkTokens;
  const int tile = blockIdx.x;
  if (!PARTS && tile >= tiles) {  // the CTAs behind the token tiles list the blocks' adapters
    const int tb = tile - tiles;
    if (blockIdx.y == 0 && blockIdx.z == 0 && tb * p.block_tokens < live)
      list_block_adapters(p, tb, live);
    return;
  }
  const int parts = PARTS ? p.parts : 1;
  if (tile * kShrinkTokens < live)
    shrink_tile<PARTS>(p, red, tile, blockIdx.y, blockIdx.z / parts, blockIdx.z % parts, live);
}

// ------------------------------------------------------------------------------ GEMM
constexpr int BW = 128;               // rows of W per tile and projection (MMA M)
constexpr int kTokBox = 64;           // token rows per TMA box
constexpr int kEpiWarps = 8;
constexpr int kProducerWarp = kEpiWarps;
constexpr int kMmaWarp = kEpiWarps + 1;
constexpr int kExtWarp0 = kEpiWarps + 2;  // two warps fill the adapters' K blocks
constexpr int kGemmThreads = 32 * (kEpiWarps + 2) + kExtThreads;
constexpr int W_BYTES = BW * BK * 2;
constexpr int kBoxBytes = kTokBox * BK * 2;
constexpr int kMaxStages = 8;
constexpr int kFlags = 16;
constexpr int kRingBytes = 192 * 1024;
// Tokens an epilogue thread finishes together.  Small on purpose: the loops over tokens stay
// rolled, and a launch that runs this code once reads it from a cold instruction cache (with 32
// tokens unrolled, a one-token gate/up call took 50 us instead of 20).
constexpr int kChunk = 8;
constexpr int kMaxRank = 128;
constexpr int kUBytes = kChunk * kMaxRank * 4;  // per epilogue warp
constexpr int kGemmSmem = 1024 + kRingBytes + kEpiWarps * kUBytes + 512 + 256 * 4;

template <bool PAIR> constexpr int kTileTokens = PAIR ? 128 : 256;  // MMA N at most

struct GemmMaps {
  CUtensorMap x;     // [T, d_in], 64-row boxes
  CUtensorMap w[2];  // [d_out, d_in], 128-row boxes
};

struct GemmParams {
  const __nv_bfloat16* b[2];
  const uint4* u;
  const float* u_parts;  // with `parts` > 0 instead of u
  int parts;
  const int32_t* blocks;
  const uint8_t* broken;
  const int32_t* ids;
  const __nv_bfloat16* addend;
  __nv_bfloat16* y;
  const int32_t* n_tokens;
  int32_t* status;
  int T, d_in, d_out, n, rank;
  int row_blocks, tok_blocks, boxes, stages, split;  // split: CTAs of a cluster per tile
  ShrinkParams shrink;  // with the shrink in this kernel
  GridSync sync;
};

// What of s B u the epilogue adds: nothing, all of it, or the products with a non-finite factor,
// which the adapters' K blocks leave out.  There a non-finite element of B would reach the zeros that
// stand for the other adapters' tokens, and one of u the zero that stands for such an element.
enum Expand { kExpandNone, kExpandAll, kExpandNonFinite };

// Finishes and stores `cnt` tokens from t0 on (row c of each projection).  v[m][i]: row c of
// projection m for token t0 + i.  One warp; su: its shared memory.
template <bool PAIR>
__device__ __forceinline__ void finish_tokens(const GemmParams& p, float (&v)[PAIR ? 2 : 1][kChunk],
                                              int t0, int cnt, int c, Expand expand, float* su) {
  constexpr int M = PAIR ? 2 : 1;
  const int lane = threadIdx.x & 31;
  const int row = min(c, p.d_out - 1);  // lanes past the last row compute it again
  int id = expand != kExpandNone && lane < cnt ? __ldg(p.ids + t0 + lane) : -1;
  if (id < 0 || id >= p.n) id = -1;
  const uint32_t with = __ballot_sync(0xffffffffu, id >= 0);
  if (!PAIR && p.addend != nullptr) {
    const __nv_bfloat16* ad = p.addend + static_cast<size_t>(t0) * p.d_out + row;
    __nv_bfloat16 a[kChunk];
#pragma unroll
    for (int i = 0; i < kChunk; ++i) a[i] = ad[static_cast<size_t>(min(i, cnt - 1)) * p.d_out];
#pragma unroll
    for (int i = 0; i < kChunk; ++i) v[0][i] += __bfloat162float(a[i]);
  }
  if (with != 0) {
    // tokens without an adapter run along with the first one that has one, and add nothing
    const int some = __shfl_sync(0xffffffffu, id, __ffs(with) - 1);
    const int eights = p.rank / 8;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const uint4* u = p.u + (static_cast<size_t>(m) * p.T + t0) * eights * 2;
      __syncwarp();
      for (int at = lane; at < kChunk * eights; at += 32) {
        const int t = at / eights;
        float h[8] = {}, l[8] = {};
        if (((with >> t) & 1u) && p.parts > 0) {
          const float4* f = reinterpret_cast<const float4*>(
              p.u_parts + (static_cast<size_t>(m) * p.T + t0) * p.rank) + 2 * at;
#pragma unroll 4
          for (int k = 0; k < p.parts; ++k, f += static_cast<size_t>(p.T) * p.rank / 2) {
            const float4 a = __ldcg(f), b = __ldcg(f + 1);
            h[0] += a.x; h[1] += a.y; h[2] += a.z; h[3] += a.w;
            h[4] += b.x; h[5] += b.y; h[6] += b.z; h[7] += b.w;
          }
        } else if ((with >> t) & 1u) {
          Vec<__nv_bfloat16>::to_f32(__ldcg(u + 2 * at), h);
          Vec<__nv_bfloat16>::to_f32(__ldcg(u + 2 * at + 1), l);
        }
        float* o = su + t * kMaxRank + at % eights * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = h[i] + l[i];
      }
      __syncwarp();
      if (expand == kExpandNonFinite) {  // rare, and rolled: see kChunk
#pragma unroll 1
        for (int i = 0; i < cnt; ++i) {
          if (!((with >> i) & 1u)) continue;
          const int e = __shfl_sync(0xffffffffu, id, i);
          const __nv_bfloat16* b = p.b[m] + (static_cast<size_t>(e) * p.d_out + row) * p.rank;
          float s = 0.f;
#pragma unroll 1
          for (int j = 0; j < p.rank; ++j) {
            const float f = __bfloat162float(b[j]), w = su[i * kMaxRank + j];
            if (!isfinite(f) || !isfinite(w)) s = fmaf(f, w, s);
          }
#pragma unroll
          for (int q = 0; q < kChunk; ++q)
            if (q == i) v[m][q] += s;
        }
        continue;
      }
      const __nv_bfloat16* brow[kChunk];
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        const int e = ((with >> i) & 1u) ? __shfl_sync(0xffffffffu, id, i) : some;
        brow[i] = p.b[m] + (static_cast<size_t>(e) * p.d_out + row) * p.rank;
      }
#pragma unroll 1
      for (int j0 = 0; j0 < p.rank; j0 += 8) {  // rank is a multiple of 8
        uint4 b[kChunk];
#pragma unroll
        for (int i = 0; i < kChunk; ++i) b[i] = ld_vec(brow[i] + j0);
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
          float bf[8];
          Vec<__nv_bfloat16>::to_f32(b[i], bf);
          const float4* uv = reinterpret_cast<const float4*>(su + i * kMaxRank + j0);
          const float4 w0 = uv[0], w1 = uv[1];
          float s = fmaf(bf[0], w0.x, fmaf(bf[1], w0.y, fmaf(bf[2], w0.z, bf[3] * w0.w)));
          s = fmaf(bf[4], w1.x, fmaf(bf[5], w1.y, fmaf(bf[6], w1.z, fmaf(bf[7], w1.w, s))));
          if ((with >> i) & 1u) v[m][i] += s;
        }
      }
    }
  }
  if (c < p.d_out) {
    __nv_bfloat16* y = p.y + static_cast<size_t>(t0) * p.d_out + c;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      float o = v[0][i];
      if constexpr (PAIR) o = gemm::silu_f(o) * v[M - 1][i];
      if (i < cnt) y[static_cast<size_t>(i) * p.d_out] = __float2bfloat16_rn(o);
    }
  }
}

// Totals of `cnt` tokens of one weight row over the cluster's S partial tiles, in rank order,
// all loads in flight together.
template <int S>
__device__ __forceinline__ void gather_partials(const float* part, int cnt, float (&v)[kChunk]) {
  float r[S][kChunk];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const uint32_t peer = cluster_map(part, s);
#pragma unroll
    for (int i = 0; i < kChunk; ++i) r[s][i] = ld_cluster_f32(peer + min(i, cnt - 1) * (BW * 4));
  }
#pragma unroll
  for (int i = 0; i < kChunk; ++i) {
    v[i] = r[0][i];
#pragma unroll
    for (int s = 1; s < S; ++s) v[i] += r[s][i];
  }
}

// SPLIT: a cluster per tile.  FUSED: the shrink is in this kernel.  Template arguments for the
// code's size: see kChunk.
template <bool PAIR, bool SPLIT, bool FUSED>
__global__ void __launch_bounds__(kGemmThreads, 1)
    adapter_gemm_kernel(const __grid_constant__ GemmMaps maps, const GemmParams p) {
  constexpr int M = PAIR ? 2 : 1;
  constexpr int NT = kTileTokens<PAIR>;
  constexpr int ACC_COLS = M * NT;  // 256 columns of TMEM per accumulator set
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* ring = base;
  float* su_all = reinterpret_cast<float*>(base + kRingBytes);
  uint8_t* ctl = base + kRingBytes + kEpiWarps * kUBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(ctl);
  uint64_t* empty = full + kMaxStages;
  uint64_t* tfull = empty + kMaxStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* ext_go = tempty + 2;  // a stage is the ext warps' to fill
  uint64_t* drain = ext_go + kMaxStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // per tile of this CTA, modulo kFlags: its K blocks of adapters met a non-finite element
  // (the ext warps run at most kMaxStages tiles ahead of the epilogue's two)
  volatile int* nonfinite = abort_flag + 1;
  volatile int* ticket = nonfinite + kFlags;  // [2] FUSED: this CTA's pieces of the shrink
  int* s_ids = reinterpret_cast<int*>(ctl + 512);  // the ext warps': adapters of their tile's tokens

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = SPLIT ? p.split : 1;
  const int rank = SPLIT ? static_cast<int>(cluster_rank()) : 0;
  const int first_tile = blockIdx.x / split, tile_step = gridDim.x / split;
  const int stages = p.stages;
  const int stage_bytes = M * W_BYTES + p.boxes * kBoxBytes;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&ext_go[s], 1);
    }
    for (int b = 0; b < 2; ++b) { mbar_init(&tfull[b], 1); mbar_init(&tempty[b], kEpiWarps); }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    if constexpr (FUSED) ticket[0] = static_cast<int>(atomicAdd(p.sync.ticket, 1u));
  }
  if (warp == kProducerWarp && lane == 0) {
    tma_prefetch_desc(&maps.x);
    tma_prefetch_desc(&maps.w[0]);
    if (PAIR) tma_prefetch_desc(&maps.w[1]);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, 2 * ACC_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // x, W, the ids and the token count were written before the shrink kernel started; only u
  // (and y's former readers) need pdl_wait, in the epilogue
  const int live = live_tokens(p.n_tokens, p.T);
  const int tok_blocks = (live + NT - 1) / NT;
  const int total = p.row_blocks * tok_blocks;
  const int k_all = (p.d_in + BK - 1) / BK;
  const int k_lo = k_all * rank / split, k_hi = k_all * (rank + 1) / split;
  const int shrink_items = FUSED ? (live + kShrinkTokens - 1) / kShrinkTokens *
                                       (p.shrink.turns * M * p.shrink.parts) : 0;
  // K blocks that the adapters of a token block add per projection; 0: the epilogue adds them,
  // or there are none (then it has nothing to add).  Written by the shrink kernel: after pdl_wait
  // only.
  const int units_per = p.rank / 8 * 2;  // 8-rank units of an adapter, high and low
  auto ext_blocks = [&](int tb) {
    if (SPLIT) return 0;
    const int n = __ldcg(p.blocks + static_cast<size_t>(tb) * (1 + kMaxBlockAdapters));
    return n > kMaxBlockAdapters ? 0 : (n * units_per + 7) / 8;
  };

  if (warp == kProducerWarp && lane == 0) {
    // ------------------------------------------------------------ TMA producer
    int stage = 0;
    uint32_t phase = 0;
    bool wrapped = false, ok = true;
    for (int tile = first_tile; tile < total && ok; tile += tile_step) {
      const int rb = tile / tok_blocks, tb = tile - rb * tok_blocks;
      const int boxes = (min(NT, live - tb * NT) + kTokBox - 1) / kTokBox;
      for (int kb = k_lo; kb < k_hi; ++kb) {
        if (!mbar_wait_bounded(&empty[stage], phase ^ 1u, abort_flag, kWaitLimitNs, p.status)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&full[stage], M * W_BYTES + boxes * kBoxBytes);
        uint8_t* dst = ring + stage * stage_bytes;
#pragma unroll
        for (int m = 0; m < M; ++m)
          tma_load_2d(dst + m * W_BYTES, &maps.w[m], &full[stage], kb * BK, rb * BW);
        for (int i = 0; i < boxes; ++i)
          tma_load_2d(dst + M * W_BYTES + i * kBoxBytes, &maps.x, &full[stage], kb * BK,
                      tb * NT + i * kTokBox);
        if (++stage == stages) { stage = 0; phase ^= 1u; wrapped = true; }
      }
      if (!ok) break;
      pdl_wait();
      for (int e = M * ext_blocks(tb); e > 0; --e) {  // the ext warps fill these stages
        if (!mbar_wait_bounded(&empty[stage], phase ^ 1u, abort_flag, kWaitLimitNs, p.status)) {
          ok = false;
          break;
        }
        mbar_arrive(&ext_go[stage]);
        if (++stage == stages) { stage = 0; phase ^= 1u; wrapped = true; }
      }
    }
    if (!ok) {  // drain our own copies in flight before the CTA leaves
      for (int s = 0; s < stages; ++s) {
        if (!wrapped && s >= stage) continue;
        mbar_wait_bounded(&full[s], (s < stage) ? phase : (phase ^ 1u), nullptr, kWaitLimitNs,
                          p.status);
      }
    }
  } else if (warp == kMmaWarp && lane == 0) {
    // ------------------------------------------------------------ MMA issuer
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    for (int tile = first_tile; tile < total && ok; tile += tile_step) {
      const int tb = tile % tok_blocks;
      const int cols = (min(NT, live - tb * NT) + 15) / 16 * 16;
      const uint32_t idesc = idesc_bf16_f32(BW, cols);
      if (!mbar_wait_bounded(&tempty[acc], acc_phase ^ 1u, abort_flag, kWaitLimitNs, p.status)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * ACC_COLS);
      for (int kb = k_lo; kb < k_hi; ++kb) {
        if (!mbar_wait_bounded(&full[stage], phase, abort_flag, kWaitLimitNs, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint8_t* src = ring + stage * stage_bytes;
        const uint64_t xd = smem_desc_k_sw128(src + M * W_BYTES);
#pragma unroll
        for (int m = 0; m < M; ++m) {
          const uint64_t wd = smem_desc_k_sw128(src + m * W_BYTES);
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)  // 16 elements = 32 bytes along K
            tc_mma_bf16(d_tmem + m * NT, wd + 2 * kk, xd + 2 * kk, idesc,
                        (kb > k_lo || kk > 0) ? 1u : 0u);
        }
        tc_commit(&empty[stage]);
        if (++stage == stages) { stage = 0; phase ^= 1u; }
      }
      if (ok) pdl_wait();
      for (int e = 0, n = ok ? ext_blocks(tb) : 0; e < M * n; ++e) {
        if (!mbar_wait_bounded(&full[stage], phase, abort_flag, kWaitLimitNs, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint8_t* src = ring + stage * stage_bytes;
        const uint64_t wd = smem_desc_k_sw128(src), xd = smem_desc_k_sw128(src + M * W_BYTES);
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          tc_mma_bf16(d_tmem + (e >= n ? NT : 0), wd + 2 * kk, xd + 2 * kk, idesc, 1u);
        tc_commit(&empty[stage]);
        if (++stage == stages) { stage = 0; phase ^= 1u; }
      }
      if (!ok) break;
      tc_commit(&tfull[acc]);
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
    if (!ok) {  // wait for every MMA this thread issued before the memory goes away
      tc_commit(drain);
      mbar_wait_bounded(drain, 0, nullptr, kWaitLimitNs, p.status);
    }
  } else if (!SPLIT && warp >= kExtWarp0) {
    // ------------------------------------------------------------ the adapters' K blocks
    const int et = threadIdx.x - kExtWarp0 * 32;
    // The TMA producer, which follows every use of a stage, hands a stage over (ext_go): these
    // warps skip the others' uses and could not tell a stage's phases apart by parity.
    int stage = 0;
    uint32_t go_phase = 0;  // bit s: parity of the next hand-over of stage s
    bool ok = true;
    pdl_wait();
    for (int tile = first_tile, iter = 0; tile < total && ok; tile += tile_step, ++iter) {
      const int rb = tile / tok_blocks, tb = tile - rb * tok_blocks;
      const int n = ext_blocks(tb);
      bool found = false;
      stage = (stage + k_hi - k_lo) % stages;
      if (n == 0) continue;
      const int32_t* list = p.blocks + static_cast<size_t>(tb) * (1 + kMaxBlockAdapters);
      const int units = __ldcg(list) * units_per;
      const int ntok = min(NT, live - tb * NT), rows = (ntok + 15) / 16 * 16;
      // the barrier at the end of the last block has passed: the table is free
      bool broken = false;
      for (int i = et; i < rows; i += kExtThreads) {
        const int id = i < ntok ? __ldg(p.ids + tb * NT + i) : -1;
        s_ids[i] = id;
        if (i < ntok) broken |= broken_token<M>(p.broken, p.T, tb * NT + i, id);
      }
      broken = !ext_all(!broken);
      for (int e = 0; e < M * n; ++e) {
        const int m = e >= n ? 1 : 0;
        ok = ext_all(mbar_wait_bounded(&ext_go[stage], (go_phase >> stage) & 1u, abort_flag,
                                       kWaitLimitNs, p.status));
        if (!ok) break;
        go_phase ^= 1u << stage;
        uint8_t* dst = ring + stage * stage_bytes;
        // this thread's 16-byte chunk of every row: unit q, in rows et / 8, et / 8 + 8, ...
        const int j = et & 7, q = (m == 0 ? e : e - n) * 8 + j;
        const int id = q < units ? __ldcg(list + 1 + q / units_per) : -1;
        const int g8 = q % units_per / 2;
        const __nv_bfloat16* b = p.b[m] + (static_cast<size_t>(max(id, 0)) * p.d_out) * p.rank +
                                 g8 * 8;
#pragma unroll 4
        for (int r = et >> 3; r < BW; r += 8) {
          const int c = rb * BW + r;
          cp_async_16_zfill(dst + r * 128 + ((j ^ (r & 7)) << 4),
                            b + static_cast<size_t>(min(c, p.d_out - 1)) * p.rank,
                            id >= 0 && c < p.d_out);
        }
        const uint4* u = p.u + (static_cast<size_t>(m) * p.T * (p.rank / 8) + g8) * 2 + (q & 1);
        uint8_t* xdst = dst + M * W_BYTES;
#pragma unroll 4
        for (int r = et >> 3; r < rows; r += 8) {
          const int t = tb * NT + min(r, ntok - 1);
          cp_async_16_zfill(xdst + r * 128 + ((j ^ (r & 7)) << 4),
                            u + static_cast<size_t>(t) * (p.rank / 8) * 2,
                            id >= 0 && s_ids[r] == id);
        }
        cp_async_wait_all();
#pragma unroll 4
        for (int r = et >> 3; r < BW; r += 8)  // this thread's own copies
          found |= zero_nonfinite(dst + r * 128 + ((j ^ (r & 7)) << 4));
        if (broken && id >= 0)
          for (int r = et >> 3; r < rows; r += 8)
            found |= zero_nonfinite(xdst + r * 128 + ((j ^ (r & 7)) << 4));
        fence_proxy_async_smem();  // for the tensor core
        found = !ext_all(!found);
        if (et == 0) {
          nonfinite[iter % kFlags] = found;
          mbar_arrive(&full[stage]);
        }
        if (++stage == stages) stage = 0;
      }
    }
  } else if (warp < kEpiWarps) {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3, half = warp >> 2;
    int acc = 0;
    uint32_t acc_phase = 0;
    if (SPLIT && first_tile < total) {
      // bring the rows of B that this CTA's share of the tokens needs into L2 meanwhile
      const int rb = first_tile / tok_blocks, tb = first_tile - rb * tok_blocks;
      const int ntok = min(NT, live - tb * NT), c = rb * BW + quarter * 32 + lane;
      const int lo = ntok * rank / p.split, hi = ntok * (rank + 1) / p.split;
      for (int t = tb * NT + lo + half; t < tb * NT + hi && c < p.d_out; t += 2) {
        const int id = __ldg(p.ids + t);
        if (id < 0 || id >= p.n) continue;
#pragma unroll
        for (int m = 0; m < M; ++m) {
          const __nv_bfloat16* b = p.b[m] + (static_cast<size_t>(id) * p.d_out + c) * p.rank;
          for (int j = 0; j < p.rank; j += 64)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(b + j));
        }
      }
    }
    if constexpr (FUSED) {
      // the shrink, over all CTAs that run, while W streams
      ShrinkSums& red = *reinterpret_cast<ShrinkSums*>(su_all);
      const int turns = p.shrink.turns, parts = p.shrink.parts;
      int done = 0;
#pragma unroll 1
      for (int i = ticket[0]; i < shrink_items; i = ticket[done & 1]) {
        int next = 0;  // its latency passes under the piece's work
        if (threadIdx.x == 0) next = static_cast<int>(atomicAdd(p.sync.ticket, 1u));
        const int part = i % parts, m = i / parts % M, turn = i / (parts * M) % turns;
        shrink_tile<true>(p.shrink, red, i / (parts * M * turns), turn, m, part, live);
        ++done;
        if (threadIdx.x == 0) ticket[done & 1] = next;
        shrink_sync();
      }
      if (threadIdx.x == 0 && done > 0) grid_arrive(p.sync, done);
    }
    pdl_wait();  // u is complete; what read y before this call is done
    for (int tile = first_tile, iter = 0; tile < total; tile += tile_step, ++iter) {
      const int rb = tile / tok_blocks, tb = tile - rb * tok_blocks;
      const int ntok = min(NT, live - tb * NT);
      int ok = 1;
      if (lane == 0)
        ok = mbar_wait_bounded(&tfull[acc], acc_phase, abort_flag, kWaitLimitNs, p.status);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      // the token block's adapters are in K blocks, or all of them are left to the epilogue
      const Expand expand = ext_blocks(tb) == 0 ? kExpandAll
                            : nonfinite[iter % kFlags] ? kExpandNonFinite : kExpandNone;
      const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                              static_cast<uint32_t>(acc * ACC_COLS);
#pragma unroll 1
      for (int c0 = half * kChunk; c0 < ntok; c0 += 2 * kChunk) {
        float v[M][kChunk];
#pragma unroll
        for (int m = 0; m < M; ++m) {
          uint32_t r[kChunk];
          tmem_ld_32x32b_x8(t_lane + m * NT + c0, r);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < kChunk; ++i) v[m][i] = __uint_as_float(r[i]);
        }
        if constexpr (!SPLIT) {
          finish_tokens<PAIR>(p, v, tb * NT + c0, min(kChunk, ntok - c0),
                              rb * BW + quarter * 32 + lane, expand, su_all + warp * (kUBytes / 4));
        } else {  // this CTA's partial tile, token-major, over the drained ring
          float* part = reinterpret_cast<float*>(ring);
#pragma unroll
          for (int m = 0; m < M; ++m)
#pragma unroll
            for (int i = 0; i < kChunk; ++i)
              part[(m * NT + c0 + i) * BW + quarter * 32 + lane] = v[m][i];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[acc]);
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
  }
  if constexpr (SPLIT) {  // one tile per cluster
    if (FUSED && threadIdx.x == 0 && first_tile < total)  // u is complete
      grid_wait(p.sync, shrink_items, abort_flag, p.status);
    __syncwarp();
    cluster_sync_all();
    if (warp < kEpiWarps && first_tile < total && *abort_flag == 0) {
      const int quarter = warp & 3, half = warp >> 2;
      const int rb = first_tile / tok_blocks, tb = first_tile - rb * tok_blocks;
      const int ntok = min(NT, live - tb * NT);
      const int lo = ntok * rank / p.split, hi = ntok * (rank + 1) / p.split;
      const int mid = (lo + hi + 1) / 2;  // the two warps of a row quarter share the tokens
      const int from = half == 0 ? lo : mid, to = half == 0 ? mid : hi;
      const float* part = reinterpret_cast<const float*>(ring) + quarter * 32 + lane;
#pragma unroll 1
      for (int c0 = from; c0 < to; c0 += kChunk) {
        const int cnt = min(kChunk, to - c0);
        float v[M][kChunk];
#pragma unroll
        for (int m = 0; m < M; ++m) {
          const float* at = part + (m * NT + c0) * BW;
          if (p.split == 2) gather_partials<2>(at, cnt, v[m]);
          else if (p.split == 4) gather_partials<4>(at, cnt, v[m]);
          else gather_partials<8>(at, cnt, v[m]);
        }
        finish_tokens<PAIR>(p, v, tb * NT + c0, cnt, rb * BW + quarter * 32 + lane,
                            kExpandAll, su_all + warp * (kUBytes / 4));
      }
    }
    __syncwarp();
    cluster_sync_all();  // no CTA leaves while another reads its partial tile
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem_base, 2 * ACC_COLS);
  if (FUSED && threadIdx.x == 0 && *abort_flag == 0) grid_leave(p.sync);
}

// Clusters of `size` CTAs of the GEMM that the current device holds at once: fewer than its SMs
// suggest, since a cluster stays within one GPC (B200: 74 of 2, 33 of 4, 15 of 8).  A second wave
// of clusters doubled a 2048x2048 call.
template <bool PAIR>
int resident_clusters(int size) {
  static std::atomic<int> known[64][4];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::atomic<int>& slot = known[dev][size == 2 ? 1 : size == 4 ? 2 : 3];
  int n = slot.load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(size);
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = kGemmSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, adapter_gemm_kernel<PAIR, true, true>, &cfg) != cudaSuccess)
      n = -1;
    slot.store(n > 0 ? n : -1, std::memory_order_relaxed);
  }
  return n;
}

template <bool PAIR, bool SPLIT, bool FUSED>
cudaError_t set_up_gemm() {
  static DeviceOnce once;
  return once.run([] {
    cudaError_t r = cudaFuncSetAttribute(adapter_gemm_kernel<PAIR, SPLIT, FUSED>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kGemmSmem);
    return r != cudaSuccess ? r : prefer_max_shared(adapter_gemm_kernel<PAIR, SPLIT, FUSED>);
  });
}

template <bool PAIR>
cudaError_t set_up_gemms() {
  cudaError_t e = set_up_gemm<PAIR, true, true>();
  if (e == cudaSuccess) e = set_up_gemm<PAIR, true, false>();
  return e == cudaSuccess ? set_up_gemm<PAIR, false, false>() : e;
}

template <bool PAIR>
cudaError_t launch_gemm(const GemmMaps& maps, GemmParams p, bool fused, int ctas,
                        cudaStream_t s) {
  constexpr int NT = kTileTokens<PAIR>;
  const int sms = sm_count();
  p.row_blocks = (p.d_out + BW - 1) / BW;
  p.tok_blocks = (p.T + NT - 1) / NT;
  p.boxes = std::min(NT / kTokBox, (p.T + kTokBox - 1) / kTokBox);
  p.stages = std::min(kMaxStages, kRingBytes / ((PAIR ? 2 : 1) * W_BYTES + p.boxes * kBoxBytes));
  const int64_t tiles = static_cast<int64_t>(p.row_blocks) * p.tok_blocks;
  const dim3 block(kGemmThreads);
  const unsigned split = static_cast<unsigned>(p.split);
  if (split == 1)
    return launch_pdl(adapter_gemm_kernel<PAIR, false, false>,
                      dim3(static_cast<unsigned>(std::min<int64_t>(tiles, sms))), block, kGemmSmem,
                      s, maps, p);
  if (!fused)
    return launch_pdl_cluster(adapter_gemm_kernel<PAIR, true, false>,
                              dim3(static_cast<unsigned>(tiles) * split), block, kGemmSmem, split, s,
                              maps, p);
  return launch_cluster(adapter_gemm_kernel<PAIR, true, true>, dim3(ctas), block, kGemmSmem,
                        split, s, maps, p);
}

}  // namespace

// CTAs that may split the contraction of a tile.  Few tiles: a cluster per tile, as many CTAs as
// fit the SMs, each with a K block at least.  (The launch takes fewer where the clusters would not
// all be resident at once.)
static int gemm_split(const moe_adapter_config& c, bool pair, int sms) {
  const int nt = pair ? kTileTokens<true> : kTileTokens<false>;
  const int64_t tiles =
      static_cast<int64_t>((c.d_out + BW - 1) / BW) * ((static_cast<int64_t>(c.T) + nt - 1) / nt);
  const int k_blocks = (c.d_in + BK - 1) / BK;
  int split = 1;
  while (split < 8 && tiles * split * 2 <= sms && split * 2 <= k_blocks) split *= 2;
  return split;
}

bool adapter_splits(const moe_adapter_config& c, bool pair) {
  return gemm_split(c, pair, sm_count()) > 1;
}

size_t adapter_u_bytes(const moe_adapter_config& c) {
  // T tokens once, or in the pieces of the split form, for either projection count.  From T and the
  // rank alone, and never falling: one workspace serves all smaller calls, on any device.
  const int64_t rows = std::max<int64_t>(c.T, std::min(int64_t{kMaxParts} * c.T, kPartTokens));
  return 2 * static_cast<size_t>(rows) * c.rank * 4;
}

size_t adapter_block_table_bytes(int T) {
  const size_t blocks = (static_cast<size_t>(T) + kTileTokens<true> - 1) / kTileTokens<true>;
  return blocks * (1 + kMaxBlockAdapters) * 4;
}

cudaError_t launch_adapter_sm100(const moe_adapter_config& c, const AdapterArgs& a,
                                 const AdapterLayout& L, void* ws, cudaStream_t s) {
  using bf16 = __nv_bfloat16;
  uint8_t* w = static_cast<uint8_t*>(ws);
  uint4* u = reinterpret_cast<uint4*>(w + L.u);
  int32_t* blocks = reinterpret_cast<int32_t*>(w + L.blocks);
  uint8_t* broken = w + L.broken;
  int32_t* status = reinterpret_cast<int32_t*>(w);
  unsigned int* sync = reinterpret_cast<unsigned int*>(w + kWsGridSyncOffset);
  GemmMaps maps;
  bool ok = encode_2d_box(&maps.x, a.x, c.d_in, c.T, kTokBox) &&
            encode_2d_box(&maps.w[0], a.w[0], c.d_in, c.d_out, BW);
  if (a.pair) ok = ok && encode_2d_box(&maps.w[1], a.w[1], c.d_in, c.d_out, BW);
  else maps.w[1] = maps.w[0];
  if (!ok) return cudaErrorInvalidValue;

  const bool pairs = adapter_pair_fits(c, a.pair);
  const int sms = sm_count();
  const int tiles = (c.T + kShrinkTokens - 1) / kShrinkTokens, m = a.pair ? 2 : 1;
  cudaError_t e = a.pair ? set_up_gemms<true>() : set_up_gemms<false>();
  if (e != cudaSuccess) return e;
  // (a cluster per tile: all clusters resident at once).  The kernel over SM pairs reads u as bf16
  // halves, which only the shrink of the form that is not split writes: enough pair tiles for it and
  // few enough tiles to split can meet (one row block of W, T near 128 times the SMs).
  int split = pairs ? 1 : gemm_split(c, a.pair, sms), clusters = 0;
  const int nt = a.pair ? kTileTokens<true> : kTileTokens<false>;
  const int64_t gemm_tiles = static_cast<int64_t>((c.d_out + BW - 1) / BW) * ((c.T + nt - 1) / nt);
  for (; split > 1; split /= 2) {
    clusters = a.pair ? resident_clusters<true>(split) : resident_clusters<false>(split);
    if (gemm_tiles <= clusters) break;
  }
  // The split form's GEMM can shrink by itself, its epilogue warps being idle while W streams: worth
  // it while a CTA has one adapter of a tile to itself at most.  us in one launch / two:
  // 14336x4096 T=24 32.5 / 39.6, gate/up 4096x8192 T=16 35.8 / 42.6, T=64 46 / 54, but gate/up
  // 4096x4096 T=96 45.9 / 43.8 and 1024x512 T=200 28.7 / 25.2.
  const bool fused = split > 1 && tiles * m * kShrinkTokens <= clusters * split;
  // Deal a tile's adapters over `turns` CTAs until the grid covers the SMs (twice, in a launch of
  // its own), and at least over two: the tile where two requests meet would take twice as long as
  // the others.  In the split form, whose epilogue adds the pieces up, also cut the contraction
  // (blocks of 32 for every warp).
  const int ctas = fused ? clusters * split : 2 * sms;
  const int turns = std::max(2, std::min(kShrinkTokens, ctas / (tiles * m)));
  const int parts = split == 1 ? 0
                               : std::max(1, std::min({kMaxParts, ctas / (tiles * m * turns),
                                                       c.d_in / (32 * kShrinkWarps),
                                                       static_cast<int>(kPartTokens / c.T)}));
  const ShrinkParams sp{static_cast<const bf16*>(a.x),
                        {static_cast<const bf16*>(a.a[0]), static_cast<const bf16*>(a.a[1])},
                        a.scale, a.ids, a.n_tokens, u, reinterpret_cast<float*>(w + L.u), turns,
                        parts, blocks, broken, status, c.T, c.d_in, c.n_adapters, c.rank,
                        pairs ? kPairBlockTokens : nt};
  if (!fused) {
    static DeviceOnce once;
    e = once.run([] {
      const cudaError_t r = prefer_max_shared(adapter_shrink_kernel<false>);
      return r != cudaSuccess ? r : prefer_max_shared(adapter_shrink_kernel<true>);
    });
    if (e != cudaSuccess) return e;
    // token tiles, then (the split form does without) the token blocks whose adapters are listed
    const int lists = parts > 0 ? 0 : (c.T + sp.block_tokens - 1) / sp.block_tokens;
    const dim3 grid(tiles + lists, turns, m * std::max(parts, 1));
    if (parts > 0) adapter_shrink_kernel<true><<<grid, 32 * kShrinkWarps, 0, s>>>(sp);
    else adapter_shrink_kernel<false><<<grid, 32 * kShrinkWarps, 0, s>>>(sp);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }

  if (pairs) return launch_adapter_pair(c, a, u, blocks, broken, status, s);
  GemmParams p{{static_cast<const bf16*>(a.b[0]), static_cast<const bf16*>(a.b[1])}, u,
               reinterpret_cast<const float*>(w + L.u), parts, blocks, broken, a.ids,
               static_cast<const bf16*>(a.addend), static_cast<bf16*>(a.y), a.n_tokens, status,
               c.T, c.d_in, c.d_out, c.n_adapters, c.rank, 0, 0, 0, 0, split, sp,
               GridSync{sync, sync + 1, sync + 2}};
  return a.pair ? launch_gemm<true>(maps, p, fused, ctas, s)
                : launch_gemm<false>(maps, p, fused, ctas, s);
}

}  // namespace moe
