// Projections with per-token low-rank adapters for larger batches (bf16, moe_adapter_linear and
// moe_adapter_gate_up beyond the few-token kernel's range):
//   p[t] = W x_t + s_a B_a (A_a x_t),  a = adapter of token t (-1: none)
//   linear   y[t] = p[t] (+ addend[t])         gate_up  h[t] = SiLU(p_gate[t]) * p_up[t]
//
// Two launches, the second starting under the first (programmatic dependent launch):
//   adapter_shrink_kernel  u[t] = s_a A_a x_t in fp32.  A CTA takes 16 consecutive tokens and
//       runs warp-level MMAs (tokens on M, ranks on N) once per adapter in use among them
//       (dealt over grid.y when there are few CTAs), its 8 warps splitting the contraction.
//       A and x are read straight into MMA fragments (16-byte loads; the k permutation inside
//       a 32-wide block is the same on both sides).  2 T rank d_in FLOP and the bytes of x and
//       the A matrices: small beside W's product, and overlapped with its start.
//   adapter_gemm_kernel    W x on tcgen05: 128 rows of W on M, up to 256 tokens on N (128 with
//       a second projection beside it), fp32 accumulators in TMEM, both operands by TMA.
//       Only its epilogue waits for u.  The epilogue adds B_a u: a thread holds one row of W
//       for 32 tokens, the token's u comes from shared memory, and B's row stays in registers
//       while the adapter does (requests lie back to back), in fp32.
// With enough tiles the GEMM is persistent, the epilogue of a tile overlapping the next tile's
// MMAs (two accumulator sets).  With few tiles (a decode batch on a small projection) a cluster
// of 2..8 CTAs splits the contraction of one tile; the partial tiles meet in distributed
// shared memory, where each CTA finishes its share of the tokens in rank order (no atomics,
// the same bits every run).
#include <algorithm>

#include "gemm_common.cuh"
#include "internal.h"

namespace moe {
namespace {

using gemm::BK;

// ------------------------------------------------------------------------------ shrink
constexpr int kShrinkWarps = 8;
constexpr int kShrinkTokens = 16;  // MMA rows
constexpr int kShrinkRanks = 32;   // ranks per pass: 4 MMA column blocks

struct ShrinkParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* a[2];
  const float* scale;
  const int32_t* ids;
  const int32_t* n_tokens;
  float* u;  // [2, T, rank]
  int32_t* status;
  int T, d_in, n, rank;
};

__device__ __forceinline__ int live_tokens(const int32_t* n_tokens, int T) {
  return n_tokens != nullptr ? min(max(__ldg(n_tokens), 0), T) : T;
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__global__ void __launch_bounds__(32 * kShrinkWarps, 2) adapter_shrink_kernel(const ShrinkParams p) {
  __shared__ float red[kShrinkWarps][kShrinkTokens][kShrinkRanks + 1];
  pdl_trigger();  // the GEMM may start; it waits for this grid before it reads u
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int t0 = blockIdx.x * kShrinkTokens, m = blockIdx.z;
  const int live = live_tokens(p.n_tokens, p.T);
  if (t0 >= live) return;
  const int nt = min(kShrinkTokens, live - t0);
  int id = lane < nt ? __ldg(p.ids + t0 + lane) : -1;
  if (id < -1 || id >= p.n) {
    if (blockIdx.y == 0 && m == 0 && warp == 0) record_status(p.status, MOE_ERR_BAD_ADAPTER_ID);
    id = -1;
  }
  const uint32_t same = __match_any_sync(0xffffffffu, id);
  uint32_t leaders = __ballot_sync(0xffffffffu, id >= 0 && __ffs(same) - 1 == lane);
  const int dv = p.d_in / 8;
  // x rows of this lane's fragment rows (rows past the last token: the last one's, unused)
  const __nv_bfloat16* x0 = p.x + static_cast<size_t>(t0 + min(g, nt - 1)) * p.d_in;
  const __nv_bfloat16* x1 = p.x + static_cast<size_t>(t0 + min(g + 8, nt - 1)) * p.d_in;
  const uint4 z = make_uint4(0, 0, 0, 0);

  for (int i = 0; leaders != 0; leaders &= leaders - 1, ++i) {
    if (i % gridDim.y != blockIdx.y) continue;  // the same for every warp
    const int lead = __ffs(leaders) - 1;
    const int a_id = __shfl_sync(0xffffffffu, id, lead);
    const uint32_t tokens = __shfl_sync(0xffffffffu, same, lead);
    const __nv_bfloat16* A = p.a[m] + static_cast<size_t>(a_id) * p.rank * p.d_in;
    const float sc = p.scale != nullptr ? __ldg(p.scale + a_id) : 1.f;
    for (int j0 = 0; j0 < p.rank; j0 += kShrinkRanks) {
      const int nb = min(4, (p.rank - j0) / 8);  // rank is a multiple of 8
      const __nv_bfloat16* ar = A + static_cast<size_t>(j0 + g) * p.d_in;
      float c[4][4] = {};
#pragma unroll 2
      for (int v = warp * 4 + q; v - q < dv; v += 4 * kShrinkWarps) {
        const bool in = v < dv;
        const uint4 a0 = in ? ld_vec(x0 + v * 8) : z, a1 = in ? ld_vec(x1 + v * 8) : z;
        uint4 b[4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
          b[n] = in && n < nb ? ld_vec(ar + static_cast<size_t>(n) * 8 * p.d_in + v * 8) : z;
#pragma unroll
        for (int n = 0; n < 4; ++n) mma_16816(c[n], a0.x, a1.x, a0.y, a1.y, b[n].x, b[n].y);
#pragma unroll
        for (int n = 0; n < 4; ++n) mma_16816(c[n], a0.z, a1.z, a0.w, a1.w, b[n].z, b[n].w);
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        red[warp][g][8 * n + 2 * q] = c[n][0];
        red[warp][g][8 * n + 2 * q + 1] = c[n][1];
        red[warp][g + 8][8 * n + 2 * q] = c[n][2];
        red[warp][g + 8][8 * n + 2 * q + 1] = c[n][3];
      }
      __syncthreads();
      for (int o = threadIdx.x; o < kShrinkTokens * kShrinkRanks; o += 32 * kShrinkWarps) {
        const int t = o / kShrinkRanks, j = o % kShrinkRanks;
        if (((tokens >> t) & 1u) && j0 + j < p.rank) {
          float v = 0.f;
#pragma unroll
          for (int w = 0; w < kShrinkWarps; ++w) v += red[w][t][j];
          p.u[(static_cast<size_t>(m) * p.T + t0 + t) * p.rank + j0 + j] = sc * v;
        }
      }
      __syncthreads();
    }
  }
}

// ------------------------------------------------------------------------------ GEMM
constexpr int BW = 128;               // rows of W per tile and projection (MMA M)
constexpr int kTokBox = 64;           // token rows per TMA box
constexpr int kEpiWarps = 8;
constexpr int kProducerWarp = kEpiWarps;
constexpr int kMmaWarp = kEpiWarps + 1;
constexpr int kGemmThreads = 32 * (kEpiWarps + 2);
constexpr int W_BYTES = BW * BK * 2;
constexpr int kBoxBytes = kTokBox * BK * 2;
constexpr int kMaxStages = 8;
constexpr int kRingBytes = 192 * 1024;
constexpr int kChunk = 32;            // tokens an epilogue thread finishes together
constexpr int kRankStep = 16;         // ranks per pass of the epilogue
constexpr int kUBytes = kChunk * kRankStep * 4;  // per epilogue warp
constexpr int kGemmSmem = 1024 + kRingBytes + kEpiWarps * kUBytes + 512;

template <bool PAIR> constexpr int kTileTokens = PAIR ? 128 : 256;  // MMA N at most

struct GemmMaps {
  CUtensorMap x;     // [T, d_in], 64-row boxes
  CUtensorMap w[2];  // [d_out, d_in], 128-row boxes
};

struct GemmParams {
  const __nv_bfloat16* b[2];
  const float* u;
  const int32_t* ids;
  const __nv_bfloat16* addend;
  __nv_bfloat16* y;
  const int32_t* n_tokens;
  int32_t* status;
  int T, d_in, d_out, n, rank;
  int row_blocks, tok_blocks, boxes, stages, split;  // split: CTAs of a cluster per tile
};

// Adds s B u for `cnt` tokens from t0 on (row c of each projection), then finishes and stores
// them.  v[m][i]: row c of projection m for token t0 + i.  One warp; su: its shared memory.
template <bool PAIR>
__device__ __forceinline__ void finish_tokens(const GemmParams& p, float (&v)[PAIR ? 2 : 1][kChunk],
                                              int t0, int cnt, int c, float* su) {
  constexpr int M = PAIR ? 2 : 1;
  const int lane = threadIdx.x & 31;
  const bool row_ok = c < p.d_out;
  int id = lane < cnt ? __ldg(p.ids + t0 + lane) : -1;
  if (id < 0 || id >= p.n) id = -1;
  if (!PAIR && p.addend != nullptr && row_ok) {
    const __nv_bfloat16* ad = p.addend + static_cast<size_t>(t0) * p.d_out + c;
    __nv_bfloat16 a[kChunk];
#pragma unroll
    for (int i = 0; i < kChunk; ++i)
      a[i] = i < cnt ? ad[static_cast<size_t>(i) * p.d_out] : __nv_bfloat16(0.f);
#pragma unroll
    for (int i = 0; i < kChunk; ++i) v[0][i] += __bfloat162float(a[i]);
  }
  if (__ballot_sync(0xffffffffu, id >= 0) != 0) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const float* u = p.u + (static_cast<size_t>(m) * p.T + t0) * p.rank;
      const __nv_bfloat16* brow = p.b[m] + static_cast<size_t>(min(c, p.d_out - 1)) * p.rank;
      const size_t bstep = static_cast<size_t>(p.d_out) * p.rank;
      for (int j0 = 0; j0 < p.rank; j0 += kRankStep) {
        // u of the tokens into shared memory; ranks past the last one as zeros
#pragma unroll
        for (int k = 0; k < kChunk * kRankStep / 4 / 32; ++k) {
          const int at = lane + 32 * k, t = at >> 2, j = j0 + (at & 3) * 4;
          float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
          if (t < cnt && j < p.rank)
            w = __ldcg(reinterpret_cast<const float4*>(u + static_cast<size_t>(t) * p.rank + j));
          reinterpret_cast<float4*>(su)[at] = w;
        }
        __syncwarp();
        const bool second = j0 + 8 < p.rank;
        int cur = -1;
        uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
#pragma unroll
        for (int i0 = 0; i0 < kChunk; i0 += 4) {
          int e[4];
          uint4 bl[4], bh[4];
          // the four tokens' rows of B together, unless the adapter stays
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            e[k] = __shfl_sync(0xffffffffu, id, i0 + k);
            if (e[k] >= 0 && e[k] != cur) {
              const __nv_bfloat16* b = brow + e[k] * bstep + j0;
              bl[k] = ld_vec(b);
              bh[k] = second ? ld_vec(b + 8) : make_uint4(0, 0, 0, 0);
            } else {
              bl[k] = lo;
              bh[k] = hi;
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (e[k] < 0) continue;
            float bf[kRankStep];
            Vec<__nv_bfloat16>::to_f32(bl[k], bf);
            Vec<__nv_bfloat16>::to_f32(bh[k], bf + 8);
            const float4* uv = reinterpret_cast<const float4*>(su + (i0 + k) * kRankStep);
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < kRankStep / 4; ++j) {
              const float4 w = uv[j];
              s = fmaf(bf[4 * j], w.x, s);
              s = fmaf(bf[4 * j + 1], w.y, s);
              s = fmaf(bf[4 * j + 2], w.z, s);
              s = fmaf(bf[4 * j + 3], w.w, s);
            }
            v[m][i0 + k] += s;
          }
          if (e[3] >= 0) { cur = e[3]; lo = bl[3]; hi = bh[3]; }
        }
        __syncwarp();
      }
    }
  }
  if (row_ok) {
    __nv_bfloat16* y = p.y + static_cast<size_t>(t0) * p.d_out + c;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      float o = v[0][i];
      if constexpr (PAIR) o = o / (1.f + __expf(-o)) * v[M - 1][i];
      if (i < cnt) y[static_cast<size_t>(i) * p.d_out] = __float2bfloat16_rn(o);
    }
  }
}

// Totals of `cnt` tokens of one weight row over the cluster's S partial tiles, in rank order.
// Four tokens' loads are in flight at a time.
template <int S>
__device__ __forceinline__ void gather_partials(const float* part, int cnt, float (&v)[kChunk]) {
  uint32_t peer[S];
#pragma unroll
  for (int s = 0; s < S; ++s) peer[s] = cluster_map(part, s);
#pragma unroll
  for (int i0 = 0; i0 < kChunk; i0 += 4) {
    if (i0 < cnt) {
      float r[4][S];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int s = 0; s < S; ++s)
          r[i][s] = ld_cluster_f32(peer[s] + min(i0 + i, cnt - 1) * (BW * 4));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i0 + i] = r[i][0];
#pragma unroll
        for (int s = 1; s < S; ++s) v[i0 + i] += r[i][s];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i0 + i] = 0.f;
    }
  }
}

template <bool PAIR>
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
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = p.split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int first_tile = blockIdx.x / p.split, tile_step = gridDim.x / p.split;
  const int stages = p.stages;
  const int stage_bytes = M * W_BYTES + p.boxes * kBoxBytes;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int b = 0; b < 2; ++b) { mbar_init(&tfull[b], 1); mbar_init(&tempty[b], kEpiWarps); }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
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
  const int k_lo = k_all * rank / p.split, k_hi = k_all * (rank + 1) / p.split;

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
      if (!ok) break;
      tc_commit(&tfull[acc]);
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
    if (!ok) {  // wait for every MMA this thread issued before the memory goes away
      tc_commit(drain);
      mbar_wait_bounded(drain, 0, nullptr, kWaitLimitNs, p.status);
    }
  } else if (warp < kEpiWarps) {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3, half = warp >> 2;
    int acc = 0;
    uint32_t acc_phase = 0;
    pdl_wait();  // u is complete; what read y before this call is done
    for (int tile = first_tile; tile < total; tile += tile_step) {
      const int rb = tile / tok_blocks, tb = tile - rb * tok_blocks;
      const int ntok = min(NT, live - tb * NT);
      int ok = 1;
      if (lane == 0)
        ok = mbar_wait_bounded(&tfull[acc], acc_phase, abort_flag, kWaitLimitNs, p.status);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                              static_cast<uint32_t>(acc * ACC_COLS);
#pragma unroll 1
      for (int c0 = half * kChunk; c0 < ntok; c0 += 2 * kChunk) {
        float v[M][kChunk];
#pragma unroll
        for (int m = 0; m < M; ++m) {
          uint32_t r[kChunk];
          tmem_ld_32x32b_x32(t_lane + m * NT + c0, r);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < kChunk; ++i) v[m][i] = __uint_as_float(r[i]);
        }
        if (p.split == 1) {
          finish_tokens<PAIR>(p, v, tb * NT + c0, min(kChunk, ntok - c0),
                              rb * BW + quarter * 32 + lane, su_all + warp * (kUBytes / 4));
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
  if (p.split > 1) {  // one tile per cluster
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
                            su_all + warp * (kUBytes / 4));
      }
    }
    __syncwarp();
    cluster_sync_all();  // no CTA leaves while another reads its partial tile
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem_base, 2 * ACC_COLS);
}

template <bool PAIR>
cudaError_t launch_gemm(const GemmMaps& maps, GemmParams p, cudaStream_t s) {
  static DeviceOnce once;
  cudaError_t e = once.run([] {
    cudaError_t r = cudaFuncSetAttribute(adapter_gemm_kernel<PAIR>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kGemmSmem);
    return r != cudaSuccess ? r : prefer_max_shared(adapter_gemm_kernel<PAIR>);
  });
  if (e != cudaSuccess) return e;
  constexpr int NT = kTileTokens<PAIR>;
  const int sms = sm_count();
  p.row_blocks = (p.d_out + BW - 1) / BW;
  p.tok_blocks = (p.T + NT - 1) / NT;
  p.boxes = std::min(NT / kTokBox, (p.T + kTokBox - 1) / kTokBox);
  p.stages = std::min(kMaxStages, kRingBytes / ((PAIR ? 2 : 1) * W_BYTES + p.boxes * kBoxBytes));
  // Few tiles: a cluster per tile, as many CTAs as fit the SMs, each with a K block at least.
  const int64_t tiles = static_cast<int64_t>(p.row_blocks) * p.tok_blocks;
  const int k_blocks = (p.d_in + BK - 1) / BK;
  p.split = 1;
  while (p.split < 8 && tiles * p.split * 2 <= sms && p.split * 2 <= k_blocks) p.split *= 2;
  if (p.split == 1)
    return launch_pdl(adapter_gemm_kernel<PAIR>, dim3(static_cast<unsigned>(std::min<int64_t>(
                                                     tiles, sms))),
                      dim3(kGemmThreads), kGemmSmem, s, maps, p);
  return launch_pdl_cluster(adapter_gemm_kernel<PAIR>,
                            dim3(static_cast<unsigned>(tiles * p.split)), dim3(kGemmThreads),
                            kGemmSmem, static_cast<unsigned>(p.split), s, maps, p);
}

}  // namespace

cudaError_t launch_adapter_sm100(const moe_adapter_config& c, const AdapterArgs& a,
                                 const AdapterLayout& L, void* ws, cudaStream_t s) {
  using bf16 = __nv_bfloat16;
  uint8_t* w = static_cast<uint8_t*>(ws);
  float* u = reinterpret_cast<float*>(w + L.u);
  int32_t* status = reinterpret_cast<int32_t*>(w);
  GemmMaps maps;
  bool ok = encode_2d_box(&maps.x, a.x, c.d_in, c.T, kTokBox) &&
            encode_2d_box(&maps.w[0], a.w[0], c.d_in, c.d_out, BW);
  if (a.pair) ok = ok && encode_2d_box(&maps.w[1], a.w[1], c.d_in, c.d_out, BW);
  else maps.w[1] = maps.w[0];
  if (!ok) return cudaErrorInvalidValue;

  const int tiles = (c.T + kShrinkTokens - 1) / kShrinkTokens, m = a.pair ? 2 : 1;
  // deal a tile's adapters over grid.y until the grid covers the SMs twice
  const int deal = std::max(1, std::min(kShrinkTokens, 2 * sm_count() / (tiles * m)));
  const ShrinkParams sp{static_cast<const bf16*>(a.x),
                        {static_cast<const bf16*>(a.a[0]), static_cast<const bf16*>(a.a[1])},
                        a.scale, a.ids, a.n_tokens, u, status, c.T, c.d_in, c.n_adapters, c.rank};
  static DeviceOnce once;
  cudaError_t e = once.run([] { return prefer_max_shared(adapter_shrink_kernel); });
  if (e != cudaSuccess) return e;
  adapter_shrink_kernel<<<dim3(tiles, deal, m), 32 * kShrinkWarps, 0, s>>>(sp);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;

  GemmParams p{{static_cast<const bf16*>(a.b[0]), static_cast<const bf16*>(a.b[1])}, u, a.ids,
               static_cast<const bf16*>(a.addend), static_cast<bf16*>(a.y), a.n_tokens, status,
               c.T, c.d_in, c.d_out, c.n_adapters, c.rank, 0, 0, 0, 0, 1};
  return a.pair ? launch_gemm<true>(maps, p, s) : launch_gemm<false>(maps, p, s);
}

}  // namespace moe
