// Projections with per-token low-rank adapters for prompts (bf16): the product W x and the
// adapters' B u on tcgen05 over SM pairs (cta_group::2).  The first launch (adapter_shrink_kernel,
// adapter_sm100.cu) has written u and each token block's adapters.
//
// A pair tile is 256 tokens x 256 rows of W (gate/up: 128 rows of W_gate and the same 128 of
// W_up), one M = 256, N = 256 MMA per K step: each SM holds 128 tokens and half of the weight
// rows, 32 KB per 64-wide K block, and ends up with its tokens' accumulators over all 256
// columns.  Against one SM per 128 x 256 tile (adapter_sm100.cu) an MMA reads a third fewer
// shared-memory bytes, which bounded that kernel: T=4099, 4096x4096 without adapters 118 us.
//   warp 8     TMA producer (both SMs), five-stage ring
//   warp 9     MMA issuer (leader)
//   warps 10-11 the adapters' K blocks: 8 units of 8 ranks, the high or the low bf16 halves of u
//              on the token side (zeros for other adapters' tokens), B_a on the weight side.  They
//              have a buffer of their own and are spread over the tile's K steps, so that filling
//              one (about 1.5 us: L2 latency) hides behind the W blocks between them.  For
//              gate/up a block serves one projection: N = 128, into its columns.
//   warps 0-7  epilogue of one accumulator set while the next tile's MMAs fill the other: SwiGLU
//              or addend, bf16 through a padded shared-memory slice, 64-byte row segments.
// Token blocks that leave their adapters to the epilogue (too many of them), and the products with
// a non-finite element of B or u, which the K blocks leave out (times the zeros there they would be
// NaN), are added there in fp32, a token per thread.
// No TMA multicast is used.
#include <algorithm>

#include "adapter_gemm.cuh"
#include "gemm_common.cuh"

namespace moe {
namespace {

using gemm::BK;
using gemm::pack_bf16;

constexpr int BM = 128;                       // tokens per SM
constexpr int BN = 256;                       // accumulator columns
constexpr int kEpiWarps = 8;
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kExtWarp0 = 10;
constexpr int kThreads = 32 * kExtWarp0 + kExtThreads;
constexpr int kHalfBytes = 128 * BK * 2;      // one operand half: 16 KB
constexpr int kStages = 5;
constexpr int kFlags = 16;
constexpr int kStageRowBytes = 80;            // 32 bf16 of a token + 16 B pad
constexpr int kEpiStageBytes = 32 * kStageRowBytes;
constexpr int kSmem = 1024 + 2 * kHalfBytes * (kStages + 1) + kEpiWarps * kEpiStageBytes + 512 +
                      BM * 4;

struct PairMaps {
  CUtensorMap x;     // [T, d_in], 128-row boxes
  CUtensorMap w[2];  // [d_out, d_in], 128-row boxes
};

struct PairParams {
  const __nv_bfloat16* b[2];
  const uint4* u;
  const int32_t* blocks;
  const uint8_t* broken;
  const int32_t* ids;
  const __nv_bfloat16* addend;
  __nv_bfloat16* y;
  const int32_t* n_tokens;
  int32_t* status;
  int T, d_in, d_out, n, rank, col_blocks, y_aligned, ad_aligned;
};

__device__ __forceinline__ void arrive_cluster(uint32_t bar) {  // release at cluster scope
  mbar_arrive_remote(bar);
}
__device__ __forceinline__ void st_cluster_s32(uint32_t addr, int v) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Adds u_t B[c0 .. c0 + 31] of the lane's token to v; with `only_nonfinite` the products with a
// non-finite factor alone.
__device__ __forceinline__ void expand_row(const PairParams& p, int m, int t, int id, int c0,
                                           bool only_nonfinite, float (&v)[32]) {
  if (id < 0) return;
  const uint4* u = p.u + (static_cast<size_t>(m) * p.T + t) * (p.rank / 8) * 2;
#pragma unroll 1
  for (int g = 0; g < p.rank / 8; ++g) {
    float h[8], l[8];
    Vec<__nv_bfloat16>::to_f32(__ldcg(u + 2 * g), h);
    Vec<__nv_bfloat16>::to_f32(__ldcg(u + 2 * g + 1), l);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] += l[i];
    const __nv_bfloat16* b =
        p.b[m] + (static_cast<size_t>(id) * p.d_out + c0) * p.rank + g * 8;
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      if (c0 + c >= p.d_out) break;
      float f[8];
      Vec<__nv_bfloat16>::to_f32(ld_vec(b + static_cast<size_t>(c) * p.rank), f);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (!only_nonfinite || !isfinite(f[i]) || !isfinite(h[i])) v[c] = fmaf(f[i], h[i], v[c]);
    }
  }
}

template <bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    adapter_pair_kernel(const __grid_constant__ PairMaps maps, const PairParams p) {
  constexpr int M = PAIR ? 2 : 1;
  constexpr int OUT = BN / M;  // output columns of a pair tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sA = base;                               // [kStages][128 tokens x 64]
  uint8_t* sB = sA + kStages * kHalfBytes;          // [kStages][128 weight rows x 64]
  uint8_t* extA = sB + kStages * kHalfBytes;        // the adapters' K block
  uint8_t* extB = extA + kHalfBytes;
  uint8_t* sEpi = extB + kHalfBytes;
  uint8_t* ctl = sEpi + kEpiWarps * kEpiStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(ctl);  // the leader's are the ones used
  uint64_t* empty = full + 8;
  uint64_t* tfull = empty + 8;
  uint64_t* tempty = tfull + 2;                       // the leader's are the ones used
  uint64_t* ext_full = tempty + 2;                    // the leader's is the one used
  uint64_t* ext_empty = ext_full + 1;
  uint64_t* drain = ext_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // per tile of this pair that has K blocks of adapters, modulo kFlags: they met a non-finite
  // element, [SM].  Only such tiles count: the ext warps may pass any number of others, but
  // fill a block only after the last one's MMAs, which wait for the epilogue two tiles before.
  volatile int* nonfinite = abort_flag + 1;
  int* s_ids = reinterpret_cast<int*>(ctl + 512);     // the ext warps': adapters of their tokens

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int b = 0; b < 2; ++b) { mbar_init(&tfull[b], 1); mbar_init(&tempty[b], 2 * kEpiWarps); }
    mbar_init(ext_full, 2);  // both SMs' ext warps
    mbar_init(ext_empty, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x < 2 * kFlags) nonfinite[threadIdx.x] = 0;
  if (warp == kProducerWarp && lane == 0) {
    tma_prefetch_desc(&maps.x);
    tma_prefetch_desc(&maps.w[0]);
    if (PAIR) tma_prefetch_desc(&maps.w[1]);
  }
  if (warp == kMmaWarp) {
    tmem_alloc_pair(tmem_slot, 2 * BN);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both SMs' barriers are initialised before any remote use
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // x, W, the ids and the token count were written before the shrink kernel started; u, the
  // blocks' adapters and y need pdl_wait
  const int live = live_tokens(p.n_tokens, p.T);
  const int tok_blocks = (live + 2 * BM - 1) / (2 * BM);
  const int total = p.col_blocks * tok_blocks;
  const int k_blocks = (p.d_in + BK - 1) / BK;
  const int units_per = p.rank / 8 * 2;  // 8-rank units of an adapter, high and low
  // K blocks that the adapters of a token block add, per projection
  auto ext_blocks = [&](int tb) {
    const int n = __ldcg(p.blocks + static_cast<size_t>(tb) * (1 + kMaxBlockAdapters));
    return n > kMaxBlockAdapters ? 0 : (n * units_per + 7) / 8;
  };

  if (warp == kProducerWarp && lane == 0) {
    // ------------------------------------------------------------ TMA producer (both)
    int stage = 0;
    uint32_t phase = 0;
    bool wrapped = false, ok = true;
    const CUtensorMap* mw = PAIR ? (leader ? &maps.w[0] : &maps.w[1]) : &maps.w[0];
    for (int tile = pair; tile < total && ok; tile += npairs) {
      const int cb = tile / tok_blocks, tb = tile - cb * tok_blocks;
      const int a_row = tb * 2 * BM + static_cast<int>(rank) * BM;
      const int b_row = PAIR ? cb * OUT : cb * BN + static_cast<int>(rank) * (BN / 2);
      for (int kb = 0; kb < k_blocks; ++kb) {
        if (!mbar_wait_bounded(&empty[stage], phase ^ 1u, abort_flag, kWaitLimitNs, p.status)) {
          ok = false;
          break;
        }
        if (leader) mbar_arrive_expect_tx(&full[stage], 4 * kHalfBytes);  // both SMs' bytes
        const uint32_t bar = cluster_map(&full[stage], 0);
        tma_load_2d_pair(sA + stage * kHalfBytes, &maps.x, bar, kb * BK, a_row);
        tma_load_2d_pair(sB + stage * kHalfBytes, mw, bar, kb * BK, b_row);
        if (++stage == kStages) { stage = 0; phase ^= 1u; wrapped = true; }
      }
    }
    if (!ok && leader) {  // drain the copies the leader's barriers still count
      for (int s = 0; s < kStages; ++s) {
        if (!wrapped && s >= stage) continue;
        mbar_wait_bounded(&full[s], (s < stage) ? phase : (phase ^ 1u), nullptr, kWaitLimitNs,
                          p.status);
      }
    }
  } else if (warp == kMmaWarp && lane == 0 && leader) {
    // ------------------------------------------------------------ MMA issuer (leader)
    constexpr uint32_t idesc = idesc_bf16_f32(2 * BM, BN), idesc_ext = idesc_bf16_f32(2 * BM, OUT);
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0, ext_phase = 0;
    bool ok = true;
    pdl_wait();
    int next_ext = pair < total ? M * ext_blocks(pair % tok_blocks) : 0;
    for (int tile = pair; tile < total && ok; tile += npairs) {
      const int ext = next_ext;  // loaded a tile ahead
      if (tile + npairs < total) next_ext = M * ext_blocks((tile + npairs) % tok_blocks);
      if (!mbar_wait_bounded(&tempty[acc], acc_phase ^ 1u, abort_flag, kWaitLimitNs, p.status)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
      // The adapters' blocks follow evenly spread ones of W, as far apart as they go: filling one takes
      // about as long as four of W's (gate/up T=1531, 12 blocks among 64: every fourth 309 us, every
      // fifth 298).  Only a compare per K block: this
      // thread issues one every 512 cycles, and 64-bit products here cost 10 us at T=4099.
      int e = 0;
      const int ext_step = ext > 0 ? max(1, k_blocks / ext) : k_blocks;
      int ext_at = ext > 0 ? min(ext_step, k_blocks) : k_blocks;
      for (int kb = 0; kb < k_blocks && ok; ++kb) {
        if (!mbar_wait_bounded(&full[stage], phase, abort_flag, kWaitLimitNs, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t ad = smem_desc_k_sw128(sA + stage * kHalfBytes);
        const uint64_t bd = smem_desc_k_sw128(sB + stage * kHalfBytes);
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)  // advance 16 elements = 32 bytes along K
          tc_mma_bf16_pair(d_tmem, ad + 2 * kk, bd + 2 * kk, idesc, (kb | kk) != 0 ? 1u : 0u);
        tc_commit_pair_mc(&empty[stage], 0x3);  // frees the stage in both SMs
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
        if (kb + 1 != ext_at) continue;
        ext_at = min(ext_at + ext_step, k_blocks);
        // one block, after W's last block all that are left
        for (const int upto = kb + 1 == k_blocks ? ext : min(e + 1, ext); e < upto; ++e) {
          if (!mbar_wait_bounded(ext_full, ext_phase, abort_flag, kWaitLimitNs, p.status)) {
            ok = false;
            break;
          }
          ext_phase ^= 1u;
          tc_fence_after();
          const uint64_t ea = smem_desc_k_sw128(extA), eb = smem_desc_k_sw128(extB);
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            tc_mma_bf16_pair(d_tmem + (e * M >= ext ? (M - 1) * OUT : 0), ea + 2 * kk,
                             eb + 2 * kk, idesc_ext, 1u);
          tc_commit_pair_mc(ext_empty, 0x3);
        }
      }
      if (!ok) break;
      tc_commit_pair_mc(&tfull[acc], 0x3);  // the accumulator is ready in both SMs
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
    if (!ok) {  // every issued MMA has finished before the memory goes away
      tc_commit_pair_mc(drain, 0x1);
      mbar_wait_bounded(drain, 0, nullptr, kWaitLimitNs, p.status);
    }
  } else if (warp >= kExtWarp0) {
    // ------------------------------------------------------------ the adapters' K blocks (both)
    const int et = threadIdx.x - kExtWarp0 * 32;
    const uint32_t full0 = cluster_map(ext_full, 0);
    uint32_t uses = 0;  // blocks filled so far
    bool ok = true;
    pdl_wait();
    for (int tile = pair, iter = -1; tile < total && ok; tile += npairs) {
      const int cb = tile / tok_blocks, tb = tile - cb * tok_blocks;
      const int n = ext_blocks(tb);
      if (n == 0) continue;
      ++iter;
      const int32_t* list = p.blocks + static_cast<size_t>(tb) * (1 + kMaxBlockAdapters);
      const int units = __ldcg(list) * units_per;
      const int t0 = tb * 2 * BM + static_cast<int>(rank) * BM;
      bool found = false;
      bool broken = false;
      for (int i = et; i < BM; i += kExtThreads) {  // the last block's barrier has passed
        const int id = t0 + i < live ? __ldg(p.ids + t0 + i) : -1;
        s_ids[i] = id;
        if (t0 + i < live) broken |= broken_token<M>(p.broken, p.T, t0 + i, id);
      }
      broken = !ext_all(!broken);
      for (int e = 0; e < M * n; ++e, ++uses) {
        const int m = e >= n ? 1 : 0;
        ok = ext_all(uses == 0 || mbar_wait_bounded(ext_empty, (uses - 1) & 1u, abort_flag,
                                                    kWaitLimitNs, p.status));
        if (!ok) break;
        // this thread's 16-byte chunk of every row: unit q, in rows et / 8, et / 8 + 8, ...
        const int j = et & 7, q = (m == 0 ? e : e - n) * 8 + j;
        const int id = q < units ? __ldcg(list + 1 + q / units_per) : -1;
        const int g8 = q % units_per / 2;
        // the weight rows of this SM: half of the tile's of projection m
        const int row0 = cb * OUT + static_cast<int>(rank) * (OUT / 2);
        const __nv_bfloat16* b =
            (m == 0 ? p.b[0] : p.b[M - 1]) +
            static_cast<size_t>(max(id, 0)) * p.d_out * p.rank + g8 * 8;
#pragma unroll 4
        for (int r = et >> 3; r < OUT / 2; r += 8)
          cp_async_16_zfill(extB + r * 128 + ((j ^ (r & 7)) << 4),
                            b + static_cast<size_t>(min(row0 + r, p.d_out - 1)) * p.rank,
                            id >= 0 && row0 + r < p.d_out);
        const uint4* u = p.u + (static_cast<size_t>(m) * p.T * (p.rank / 8) + g8) * 2 + (q & 1);
#pragma unroll 4
        for (int r = et >> 3; r < BM; r += 8)
          cp_async_16_zfill(extA + r * 128 + ((j ^ (r & 7)) << 4),
                            u + static_cast<size_t>(min(t0 + r, p.T - 1)) * (p.rank / 8) * 2,
                            id >= 0 && s_ids[r] == id);
        cp_async_wait_all();
#pragma unroll 4
        for (int r = et >> 3; r < OUT / 2; r += 8)  // this thread's own copies
          found |= zero_nonfinite(extB + r * 128 + ((j ^ (r & 7)) << 4));
        if (broken && id >= 0)
          for (int r = et >> 3; r < BM; r += 8)
            found |= zero_nonfinite(extA + r * 128 + ((j ^ (r & 7)) << 4));
        fence_proxy_async_smem();  // for the tensor core
        found = !ext_all(!found);
        if (et == 0) {
          const uint32_t flag = static_cast<uint32_t>(2 * (iter % kFlags)) + rank;
          st_cluster_s32(cluster_map(const_cast<int*>(nonfinite + flag), 0), found);
          st_cluster_s32(cluster_map(const_cast<int*>(nonfinite + flag), 1), found);
          asm volatile("fence.acq_rel.cluster;" ::: "memory");
          arrive_cluster(full0);
        }
      }
    }
  } else if (warp < kEpiWarps) {
    // ------------------------------------------------------------ epilogue (both)
    const int quarter = warp & 3, half = warp >> 2;
    constexpr int COLS = OUT / 2;
    uint8_t* stage_mem = sEpi + warp * kEpiStageBytes;
    const uint32_t tempty0 = cluster_map(&tempty[0], 0);
    const uint32_t tempty1 = cluster_map(&tempty[1], 0);
    int acc = 0;
    uint32_t acc_phase = 0;
    pdl_wait();  // what read y before this call is done
    for (int tile = pair, iter = -1; tile < total; tile += npairs) {
      const int cb = tile / tok_blocks, tb = tile - cb * tok_blocks;
      const bool blocks = ext_blocks(tb) != 0;
      iter += blocks;
      int ok = 1;
      if (lane == 0)
        ok = mbar_wait_bounded(&tfull[acc], acc_phase, abort_flag, kWaitLimitNs, p.status);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                             static_cast<uint32_t>(acc * BN);
      const int t0 = tb * 2 * BM + static_cast<int>(rank) * BM + quarter * 32;
      const int valid = live - t0;  // tokens of this warp's 32 that exist
      const bool fix = blocks && (nonfinite[2 * (iter % kFlags)] | nonfinite[2 * (iter % kFlags) + 1]);
      int id = lane < valid && (!blocks || fix) ? __ldg(p.ids + t0 + lane) : -1;
      if (id >= p.n) id = -1;
      const bool expand = __ballot_sync(0xffffffffu, id >= 0) != 0;
#pragma unroll 1
      for (int c0 = 0; c0 < COLS && valid > 0; c0 += 32) {
        const int col = cb * OUT + half * COLS + c0;  // of the output
        if (col >= p.d_out) break;
        float v[M][32];
#pragma unroll
        for (int m = 0; m < M; ++m) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(t_row + m * OUT + half * COLS + c0, r);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) v[m][i] = __uint_as_float(r[i]);
        }
        if (expand) {
#pragma unroll
          for (int m = 0; m < M; ++m) expand_row(p, m, t0 + lane, id, col, fix, v[m]);
        }
        if (!PAIR && p.addend != nullptr && lane < valid) {
          const __nv_bfloat16* ad = p.addend + static_cast<size_t>(t0 + lane) * p.d_out + col;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (col + 8 * q >= p.d_out) break;
            float f[8];
            if (p.ad_aligned) {
              // plain load: the addend may be y itself
              Vec<__nv_bfloat16>::to_f32(*reinterpret_cast<const uint4*>(ad + 8 * q), f);
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) f[i] = __bfloat162float(ad[8 * q + i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) v[0][8 * q + i] += f[i];
          }
        }
        uint32_t o[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float a0 = v[0][2 * i], a1 = v[0][2 * i + 1];
          if constexpr (PAIR) {
            a0 = gemm::silu_f(a0) * v[M - 1][2 * i];
            a1 = gemm::silu_f(a1) * v[M - 1][2 * i + 1];
          }
          o[i] = pack_bf16(a0, a1);
        }
        uint4* srow = reinterpret_cast<uint4*>(stage_mem + lane * kStageRowBytes);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          srow[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        __syncwarp();
        // 4 lanes per token (64 bytes), 8 tokens per instruction
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = i * 8 + (lane >> 2), q = lane & 3;
          const uint4 w = *reinterpret_cast<const uint4*>(stage_mem + r * kStageRowBytes + q * 16);
          if (r < valid && col + q * 8 < p.d_out) {
            __nv_bfloat16* y = p.y + static_cast<size_t>(t0 + r) * p.d_out + col + q * 8;
            if (p.y_aligned) {
              *reinterpret_cast<uint4*>(y) = w;
            } else {  // only x and the weights are bound to 16-byte alignment
              const __nv_bfloat16* h = reinterpret_cast<const __nv_bfloat16*>(&w);
#pragma unroll
              for (int z = 0; z < 8; ++z) y[z] = h[z];
            }
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(acc == 0 ? tempty0 : tempty1);  // the leader's barrier
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no SM frees its memory while the pair's MMAs may read it
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc_pair(tmem_base, 2 * BN);
}

template <bool PAIR>
cudaError_t launch(const PairMaps& maps, PairParams p, cudaStream_t s) {
  static DeviceOnce once;
  cudaError_t e = once.run([] {
    cudaError_t r = cudaFuncSetAttribute(adapter_pair_kernel<PAIR>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    return r != cudaSuccess ? r : prefer_max_shared(adapter_pair_kernel<PAIR>);
  });
  if (e != cudaSuccess) return e;
  constexpr int OUT = PAIR ? BN / 2 : BN;
  p.col_blocks = (p.d_out + OUT - 1) / OUT;
  const int64_t tiles =
      static_cast<int64_t>(p.col_blocks) * ((static_cast<int64_t>(p.T) + 2 * BM - 1) / (2 * BM));
  const int pairs = static_cast<int>(std::min<int64_t>(tiles, sm_count() / 2));
  return launch_pdl_cluster(adapter_pair_kernel<PAIR>, dim3(2 * pairs), dim3(kThreads), kSmem, 2,
                            s, maps, p);
}

}  // namespace

// Worth it from a round of tiles on and where padding T to 256 costs less than the pairs gain.
bool adapter_pair_fits(const moe_adapter_config& c, bool pair) {
  const int out = pair ? BN / 2 : BN;
  const int64_t tok = (static_cast<int64_t>(c.T) + 2 * BM - 1) / (2 * BM);
  const int64_t tiles = tok * ((c.d_out + out - 1) / out);
  return tiles >= sm_count() / 2 && tok * 2 * BM * 4 <= static_cast<int64_t>(c.T) * 5;
}

cudaError_t launch_adapter_pair(const moe_adapter_config& c, const AdapterArgs& a, const uint4* u,
                                const int32_t* blocks, const uint8_t* broken, int32_t* status,
                                cudaStream_t s) {
  using bf16 = __nv_bfloat16;
  PairMaps maps;
  bool ok = encode_2d_box(&maps.x, a.x, c.d_in, c.T, BM) &&
            encode_2d_box(&maps.w[0], a.w[0], c.d_in, c.d_out, BN / 2);
  if (a.pair) ok = ok && encode_2d_box(&maps.w[1], a.w[1], c.d_in, c.d_out, BN / 2);
  else maps.w[1] = maps.w[0];
  if (!ok) return cudaErrorInvalidValue;
  const PairParams p{{static_cast<const bf16*>(a.b[0]), static_cast<const bf16*>(a.b[1])}, u,
                     blocks, broken, a.ids, static_cast<const bf16*>(a.addend),
                     static_cast<bf16*>(a.y),
                     a.n_tokens, status, c.T, c.d_in, c.d_out, c.n_adapters, c.rank, 0,
                     (reinterpret_cast<uintptr_t>(a.y) & 15) == 0,
                     (reinterpret_cast<uintptr_t>(a.addend) & 15) == 0};
  return a.pair ? launch<true>(maps, p, s) : launch<false>(maps, p, s);
}

}  // namespace moe
