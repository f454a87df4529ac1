// The whole MoE layer for at most 32 tokens in one kernel (moe_forward_few).
//
//   z = x W_r^T + bias; ids, g = top-k; H'[t,e] = g (SiLU(x_t Wg_e^T) * (x_t Wu_e^T));
//   y[t] = sum_e H'[t,e] Wd_e^T (+ shared expert) (+ x_t)
// Sources: "271,104 Routes: What I Missed About Mixture-of-Experts", sections 1-3 (the layer),
// section 5 (with small batches the cost is moving the weights); "MoE Inference Visualized",
// Expert Execution.
//
// With few tokens the layer is bound by reading each touched expert's 3 d F weights once.
// The five launches of moe_forward each pay a ramp and a tail there, and the padding of
// their tiles; here one cooperative kernel runs three phases over the streaming engine of
// few_stream.cuh, with two grid barriers between them:
//   router   one warp per (expert, up to 4 tokens) dot product, spread over all CTAs.
//   -- barrier --  every CTA selects the top-k for all tokens itself (T * k <= 1024 routes)
//                  and builds the same tables: per expert a 32-bit mask of its tokens.
//   gate/up  (touched experts x F) row pairs, cut over the CTAs at equal cost; a tile is up to 16 gate
//            rows with their 16 up rows (8 with few tokens), against the expert's own tokens only.
//   -- barrier --  meanwhile the producer already streams W_down into the ring; only the
//                  H rows of those slots wait for the barrier.
//   down     d output rows, cut evenly over the CTAs; each CTA runs all touched experts'
//            columns for its rows, so the k-way combine is the contraction itself: the gate
//            is folded into H before it is rounded to the storage type (one rounding, as for
//            H without the gate), the sum over experts stays in fp32 and there is no
//            combine pass and no atomics.
#include <climits>
#include <cmath>

#include "few_stream.cuh"
#include "gemm_common.cuh"

namespace moe {
namespace {

using namespace few;

constexpr int kMaxExperts = 256;

struct FewParams {
  const void* x;
  const void* w_router;
  const float* bias;
  const void* w_gate;
  const void* w_up;
  const void* w_down;
  const void* s_gate;  // null without a shared expert
  const void* s_up;
  const void* s_down;
  void* y;
  int32_t* ids_out;
  float* gates_out;
  int32_t* demand_out;
  int32_t* offsets_out;
  const int32_t* n_tokens;  // null: all T
  float* logits;            // [T, E] scratch
  void* h;                  // [T k (+ T), F] scratch
  int32_t* status;
  GridSync sync;
  int T, d, E, k, F, gate_mode, capacity, has_shared, residual;
  uint32_t smem_bytes;
};

// What every CTA knows after the top-k: touched experts in ascending order, the shared
// expert last (index E).  H row of (expert, its s-th token): hrow + s.
struct Tables {
  uint32_t mask[kMaxExperts + 1];  // tokens that each expert runs for
  uint32_t seg_mask[kMaxExperts + 1];
  int16_t seg_e[kMaxExperts + 2];
  int16_t seg_hrow[kMaxExperts + 2];
  int16_t row[kMaxExperts + 2];    // first H row of each expert
  float gate_of_row[kMaxTokens * 33];
  int32_t cost[kMaxExperts + 2];   // per hidden row, summed over the segments before
  int32_t lo, hi;                  // this CTA's (segment, hidden row) pairs of gate/up
  int32_t c0, c1;                  // and its output rows of down
  int32_t nseg;
  int32_t most;                    // tokens of the fullest segment
};
// Cost of a gate/up row pair with nb tokens: two weight rows and, per 16 pairs, nb token rows
// through the same copies and shared memory, and their MMAs.  Measured on skewed experts (T=32,
// 1 to 30 tokens each): at 32 + nb the CTAs of the fullest expert took 497 us, the others 305.
// In fp32 a token costs twice that (12+1 experts, d=776, F=4812, T=16: 290 us at 2, 258 at 4, 269
// at 8).
template <bool F32>
__device__ __forceinline__ int pair_cost(int nb) { return 32 + (F32 ? 4 : 2) * nb; }

constexpr uint32_t kTableBytes = (sizeof(Tables) + 15) & ~15u;
// Only while the tables are built: in the ring, which is still empty.
struct Choice {
  int32_t ids[kMaxTokens * 32];  // [T, k]
  float gates[kMaxTokens * 32];  // [T, k]
  // Tokens that chose the expert at a logit of -inf, because fewer than k others are open.  Their
  // gate is 0 and the route does not run (a closed expert's weights may hold anything: 0 * NaN),
  // but demand, capacity and offsets count it.  A NaN logit ranks as -inf and runs: NaN stays NaN.
  uint32_t closed[kMaxExperts];
};
static_assert(kCtlBytes + kRedFloats<4> * 4 + kTableBytes + 2 * kMaxSlotBytes <= kSmemBytes,
              "the ring holds two of the largest slots");

__device__ __forceinline__ float rank_key(float z) { return isnan(z) ? -INFINITY : z; }
// Larger logit, larger key; -0 ranks as +0.
__device__ __forceinline__ uint32_t order_key(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);
  return b ^ ((b & 0x80000000u) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int s = 16; s >= 1; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

// Router logits: item (expert, group of tokens) per warp, spread over the grid.
template <typename Tin>
__device__ __forceinline__ void router_logits(const FewParams& p, int live) {
  constexpr int VEC = Vec<Tin>::N, U = 4;  // vectors in flight per lane and operand
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int warps = gridDim.x * kConsumerWarps;
  const int per = (live * p.E <= warps) ? 1 : (live * p.E <= 2 * warps) ? 2 : 4;
  const int groups = (live + per - 1) / per;
  const int nv = p.d / VEC;
  // neighbouring items on different SMs
  for (int item = warp * gridDim.x + blockIdx.x; item < p.E * groups; item += warps) {
    const int e = item % p.E, t0 = (item / p.E) * per;
    const Tin* w = static_cast<const Tin*>(p.w_router) + static_cast<size_t>(e) * p.d;
    const float bias = p.bias != nullptr ? __ldg(p.bias + e) : 0.f;
#pragma unroll 1
    for (int t = t0; t < min(t0 + per, live); ++t) {  // W_r's row stays in L1
      const Tin* x = static_cast<const Tin*>(p.x) + static_cast<size_t>(t) * p.d;
      float acc = 0.f;
#pragma unroll 1
      for (int v0 = lane; v0 < nv; v0 += 32 * U) {
        uint4 wv[U], xv[U];
#pragma unroll
        for (int h = 0; h < U; ++h) {
          const int v = v0 + 32 * h;
          wv[h] = v < nv ? ld_vec(w + v * VEC) : make_uint4(0, 0, 0, 0);
          xv[h] = v < nv ? ld_vec(x + v * VEC) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int h = 0; h < U; ++h) {
          float wf[VEC], xf[VEC];
          Vec<Tin>::to_f32(wv[h], wf);
          Vec<Tin>::to_f32(xv[h], xf);
#pragma unroll
          for (int q = 0; q < VEC; ++q) acc = fmaf(xf[q], wf[q], acc);
        }
      }
      acc = warp_sum(acc);
      if (lane == 0) p.logits[t * p.E + e] = acc + bias;
    }
  }
}

// Top-k and gates of token t by one warp; lane l holds experts l, l + 32, ...  k rounds of
// (largest key, then lowest index).  (Ranking each expert against all others by 32 shuffles
// instead took 1.7 us a token: the shuffles' dependent instructions, not the rounds, bound.)
template <int NP>
__device__ __forceinline__ void select_token(const FewParams& p, Tables& tb, Choice& ch, int t,
                                             const float (&z)[NP]) {
  const int lane = threadIdx.x & 31;
  uint32_t key[NP], most = 0;
  int rank[NP];  // slot of each of the lane's experts, kMaxExperts: not chosen
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    key[i] = 32 * i + lane < p.E ? order_key(rank_key(z[i])) : 0;  // 0: below every logit's key
    rank[i] = kMaxExperts;
  }
#pragma unroll 1
  for (int j = 0; j < p.k; ++j) {
    uint32_t best = 0;
    int be = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (rank[i] == kMaxExperts && key[i] > best) { best = key[i]; be = 32 * i + lane; }
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    int e;
    if constexpr (NP == 1) e = __ffs(__ballot_sync(0xffffffffu, best == top)) - 1;
    else e = __reduce_min_sync(0xffffffffu, best == top ? be : 0x7fffffff);
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (32 * i + lane == e) rank[i] = j;
    if (j == 0) most = top;
  }
  const float m = key_value(most);
  const bool open = m > -INFINITY;  // else every expert is masked: the token takes nothing
  float ej[NP], local = 0.f;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    ej[i] = open && 32 * i + lane < p.E ? expf(key_value(key[i]) - m) : 0.f;
    // renormalising the full softmax over the selected experts cancels its denominator
    if (rank[i] < p.k || p.gate_mode == MOE_GATE_SOFTMAX_TOPK) local += ej[i];
  }
  const float denom = warp_sum(local);
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    if (rank[i] < p.k) {
      const int e = 32 * i + lane;
      ch.ids[t * p.k + rank[i]] = e;
      ch.gates[t * p.k + rank[i]] = open ? ej[i] / denom : 0.f;
      atomicOr(&tb.mask[e], 1u << t);
      if (z[i] == -INFINITY) atomicOr(&ch.closed[e], 1u << t);
    }
  }
}

// The tokens of this warp; a token's logits are loaded while the one before is selected.
template <int NP>
__device__ __forceinline__ void select_tokens(const FewParams& p, Tables& tb, Choice& ch, int live) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float z[NP], next[NP] = {};
  auto load = [&](int t) {
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (t < live && 32 * i + lane < p.E) next[i] = __ldcg(p.logits + t * p.E + 32 * i + lane);
  };
  load(warp);
#pragma unroll 1
  for (int t = warp; t < live; t += kConsumerWarps) {
#pragma unroll
    for (int i = 0; i < NP; ++i) z[i] = next[i];
    load(t + kConsumerWarps);
    select_token<NP>(p, tb, ch, t, z);
  }
}

// The tables, by the consumer threads.
template <bool F32>
__device__ __forceinline__ void build_tables(const FewParams& p, Tables& tb, Choice& ch, int live) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int e = tid; e <= p.E; e += kConsumers) {
    tb.mask[e] = 0;
    if (e < p.E) ch.closed[e] = 0;
  }
  consumer_sync();
  if (p.E <= 32) select_tokens<1>(p, tb, ch, live);
  else if (p.E <= 64) select_tokens<2>(p, tb, ch, live);
  else select_tokens<8>(p, tb, ch, live);
  consumer_sync();
  if (warp == 0) {
    int nseg = 0, rows = 0, cost = 0, most = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      uint32_t m = e < p.E ? tb.mask[e] : 0;
      if (blockIdx.x == 0 && e < p.E && p.demand_out != nullptr) p.demand_out[e] = __popc(m);
      if (p.capacity >= 0)  // arrival order is token order: the lowest C tokens stay
        while (__popc(m) > p.capacity) m &= ~(0x80000000u >> __clz(m));
      const int kept = __popc(m);
      if (e < p.E) m &= ~ch.closed[e];
      const int n = __popc(m), w = n > 0 ? pair_cost<F32>(n) : 0;
      int incl = kept, cincl = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        const int q = __shfl_up_sync(0xffffffffu, cincl, o);
        if (lane >= o) { incl += v; cincl += q; }
      }
      const uint32_t has = __ballot_sync(0xffffffffu, n > 0);
      const int row = rows + incl - kept;  // H rows are numbered by the kept routes
      if (e < p.E) {
        tb.mask[e] = m;
        tb.row[e] = static_cast<int16_t>(row);
        if (blockIdx.x == 0 && p.offsets_out != nullptr) p.offsets_out[e] = row;
      }
      if (n > 0) {
        const int i = nseg + __popc(has & ((1u << lane) - 1u));
        tb.seg_e[i] = static_cast<int16_t>(e);
        tb.seg_mask[i] = m;
        tb.seg_hrow[i] = static_cast<int16_t>(row);
        tb.cost[i] = cost + cincl - w;
      }
      most = max(most, __reduce_max_sync(0xffffffffu, n));
      nseg += __popc(has);
      rows += __shfl_sync(0xffffffffu, incl, 31);
      cost += __shfl_sync(0xffffffffu, cincl, 31);
    }
    const int total = rows + (p.has_shared ? live : 0);
    if (lane == 0) {
      if (p.has_shared && live > 0) {
        tb.seg_e[nseg] = static_cast<int16_t>(p.E);
        tb.seg_mask[nseg] = live == 32 ? 0xffffffffu : (1u << live) - 1u;
        tb.seg_hrow[nseg] = static_cast<int16_t>(rows);
        tb.cost[nseg] = cost;
        cost += pair_cost<F32>(live);
        most = live;
        ++nseg;
      }
      tb.nseg = nseg;
      tb.most = most;
      tb.cost[nseg] = cost;
      tb.lo = tb.hi = nseg * p.F;  // the end, unless a segment has it
      tb.c0 = static_cast<int>(share_begin(p.d, blockIdx.x));
      tb.c1 = static_cast<int>(share_begin(p.d, blockIdx.x + 1));
      if (blockIdx.x == 0 && p.offsets_out != nullptr) {
        p.offsets_out[p.E] = rows;
        p.offsets_out[p.E + 1] = total;
      }
    }
    for (int i = rows + lane; i < total; i += 32) tb.gate_of_row[i] = 1.f;  // shared expert
  }
  consumer_sync();
  // Equal cost for every CTA: where this one's share of the pairs begins (lanes of even threads)
  // and ends.  The share's bounds in cost, then in the segment that holds them.
  {
    const int end = tid & 1;
    const int64_t at = share_begin(static_cast<int64_t>(tb.cost[tb.nseg]) * p.F, blockIdx.x + end);
    for (int s = tid >> 1; s < tb.nseg; s += kConsumers / 2) {
      const int64_t a = static_cast<int64_t>(tb.cost[s]) * p.F;
      const int w = tb.cost[s + 1] - tb.cost[s];
      if (at >= a && at < a + static_cast<int64_t>(w) * p.F)  // F <= 2^24, w < 2^8
        (end ? tb.hi : tb.lo) = s * p.F + static_cast<int>(static_cast<uint32_t>(at - a) / w);
    }
  }
  // gate of each kept route's H row
#pragma unroll 1
  for (int i = tid; i < live * p.k; i += kConsumers) {
    const int t = i / p.k, e = ch.ids[i];
    const uint32_t m = tb.mask[e];
    if ((m >> t) & 1u) tb.gate_of_row[tb.row[e] + __popc(m & ((1u << t) - 1u))] = ch.gates[i];
  }
  if (blockIdx.x == 0)
#pragma unroll 1
    for (int i = tid; i < live * p.k; i += kConsumers) {
      if (p.ids_out != nullptr) p.ids_out[i] = ch.ids[i];
      if (p.gates_out != nullptr) p.gates_out[i] = ch.gates[i];
    }
}

// Position of the down phase: tiles of output rows, and per tile every (segment, chunk),
// starting at a different one in each CTA.  In one common order all CTAs would ask for the
// same few H rows at the same moment, and the L2 slices that hold them become the limit.
struct DownPos {
  int row, nrows, seg, kv;  // first row and rows of the tile, segment, first vector
  int left;                 // (segment, chunk) pairs of the tile still to come, this one too
};

template <typename Tin, int NT>
__global__ void __launch_bounds__(kThreads<sizeof(Tin) == 4, NT>, 1)
    few_layer_kernel(const FewParams p) {
  constexpr bool F32 = sizeof(Tin) == 4;
  constexpr int VEC = Vec<Tin>::N;
  extern __shared__ __align__(128) uint8_t smem[];
  const Shared s = carve<NT>(smem, kTableBytes, p.smem_bytes);
  Tables& tb = *reinterpret_cast<Tables*>(smem + kCtlBytes + kRedBufs<NT> * kRedFloats<NT> * 4);
  const int tid = threadIdx.x, warp = tid >> 5;
  const Tin* X = static_cast<const Tin*>(p.x);
  Tin* H = static_cast<Tin*>(p.h);

  init_shared<F32, NT>(s);
  const int live = p.n_tokens != nullptr ? min(max(__ldg(p.n_tokens), 0), p.T) : p.T;
  __syncthreads();

  // ---- router, top-k, tables ----
  bool ok = true;
  if (warp < kConsumerWarps) {
    router_logits<Tin>(p, live);
    consumer_sync();
    if (tid == 0) {
      grid_arrive(p.sync);
      grid_wait(p.sync, gridDim.x, s.abort_flag, p.status);
    }
    consumer_sync();
    ok = *s.abort_flag == 0;  // written before the barrier: the same for all
    if (ok) build_tables<F32>(p, tb, *reinterpret_cast<Choice*>(s.ring), live);
    else if (tid == 0) tb.nseg = tb.c0 = tb.c1 = 0;
    fence_proxy_async_smem();  // Choice lies where bulk copies now write
  }
  __syncthreads();
  const int nseg = tb.nseg;
  const int g0 = nseg > 0 ? tb.lo : 0, g1 = nseg > 0 ? tb.hi : 0;
  const int c0 = tb.c0, c1 = tb.c1;
  const int dv = p.d / VEC, fv = p.F / VEC;  // 16-byte vectors of a row
  // chunks of the two phases
  const int most = nseg > 0 ? tb.most : 0;
  // Row pairs of a gate/up tile.  With few tokens 8, and chunks twice as long: half the copies for
  // the same bytes, one MMA row block instead of two, but twice the token rows.  us with 8 / 16:
  // Granite-shaped T=1 18.5 / 19.2; Mixtral-shaped T=1 120 / 124, T=8 398 / 324.
  const int pairs = !F32 && most <= 4 && dv >= 2 * kChunkVecs ? 8 : 16;
  const int gu_vecs = chunk_vecs(2 * min(pairs, g1 - g0) + most, dv,
                                 pairs == 8 ? 44 * 1024 : kThinSlot);
  const int dn_vecs = chunk_vecs(min(kTileRows, c1 - c0) + most, fv, kThinSlot);

  if (warp >= kConsumerWarps) {
    // ------------------------------------------------------------------ producers
    const uint32_t P = pitch_of<F32>(gu_vecs);
    const size_t xs = static_cast<size_t>(p.d) * sizeof(Tin);  // bytes of a row of d
    const size_t hs = static_cast<size_t>(p.F) * sizeof(Tin);  // bytes of a row of F
    Producer<kTeamWarps<F32, NT>> pr(s, p.status);
    bool go = *s.abort_flag == 0;
    for (int at = g0; at < g1 && go;) {
      const int seg = at / p.F, f0 = at - seg * p.F;
      const int np = min(min(pairs, g1 - at), p.F - f0);
      const int e = tb.seg_e[seg];
      const uint32_t mask = tb.seg_mask[seg];
      const uint32_t rows = 2 * np + __popc(mask);
      const bool sh = e == p.E;
      const size_t base = ((sh ? 0 : static_cast<size_t>(e) * p.F) + f0) * xs;
      const uint8_t* wg = static_cast<const uint8_t*>(sh ? p.s_gate : p.w_gate) + base;
      const uint8_t* wu = static_cast<const uint8_t*>(sh ? p.s_up : p.w_up) + base;
      const uint8_t* xb = static_cast<const uint8_t*>(p.x);
      const int chunks = (dv + gu_vecs - 1) / gu_vecs;
      int c = blockIdx.x % chunks;  // see DownPos: not all CTAs read the same token chunk
      for (int i = 0; i < chunks; ++i, c = c + 1 == chunks ? 0 : c + 1) {
        const int kv = c * gu_vecs;
        pr.reserve(rows * P);
        if (pr.mine()) {
          if (pr.ready(rows * P, 0xffffffffu) != 1) { go = false; break; }
          const int n = min(gu_vecs, dv - kv);
          const uint32_t bytes = n * 16, o = kv * 16;
          pr.open(SlotDesc{0, static_cast<int16_t>(np), static_cast<int16_t>(np),
                           static_cast<int16_t>(n), static_cast<int16_t>(P), i + 1 == chunks, 0, 0, 0,
                           mask, seg, f0, kv},
                  rows, bytes);
          pr.copy_weights(P, wg + o, np, wu + o, np, xs, bytes);
          pr.copy_tokens(P, 2 * np, xb + o, xs, mask, bytes);
        }
        pr.pass(rows * P);
      }
      at += np;
    }
    // Down: the weight rows of the slots that fit come before the barrier, their H rows
    // after it.
    const uint32_t first = pr.it;
    const uint32_t PD = pitch_of<F32>(dn_vecs);
    const int fch = (fv + dn_vecs - 1) / dn_vecs, turns = fch * nseg;
    const int turn = static_cast<int>(static_cast<int64_t>(turns) * blockIdx.x / gridDim.x);
    DownPos w{c0, min(kTileRows, c1 - c0),
              turn / fch, turn % fch * dn_vecs, turns};
    auto next = [&](DownPos& q) {
      q.kv += dn_vecs;
      if (q.kv >= fv) {
        q.kv = 0;
        if (++q.seg == nseg) q.seg = 0;
      }
      if (--q.left > 0) return;
      q.left = turns;  // back at the turn: the next tile
      q.row += q.nrows;
      q.nrows = min(kTileRows, c1 - q.row);
    };
    auto load_h = [&](uint32_t it) {  // the H rows of slot `it`, one of this team's
      const SlotDesc& d = s.desc[it % kSlots];
      pr.copy_rows(it, d.off, d.pitch, d.r0 + d.r1,
                   reinterpret_cast<const uint8_t*>(H) + tb.seg_hrow[d.seg] * hs + d.kv * 16, hs,
                   __popc(d.mask), d.kvec * 16);
    };
    auto load_late_h = [&] {
      uint32_t it = first + (pr.team() - first) % kTeams;
#pragma unroll 1
      for (; it < pr.it; it += kTeams) load_h(it);
    };
    bool passed = false;
    auto pass_barrier = [&] {  // H is complete; bulk copies may read it
      go = grid_wait_warps(p.sync, 2 * gridDim.x, pr.me == 0, s.passed, s.abort_flag, p.status);
      passed = true;
      fence_proxy_async_all();
      load_late_h();
    };
    while (go && nseg > 0 && w.nrows > 0) {
      const int e = tb.seg_e[w.seg];
      const uint32_t mask = tb.seg_mask[w.seg];
      const uint32_t rows = w.nrows + __popc(mask);
      pr.reserve(rows * PD);
      if (pr.mine()) {
        int r = pr.ready(rows * PD, passed ? 0xffffffffu : first);
        if (r == 0) {  // the ring is full of slots that wait for H
          pass_barrier();
          r = go ? pr.ready(rows * PD, 0xffffffffu) : -1;
        }
        if (r < 0) { go = false; break; }
        const int n = min(dn_vecs, fv - w.kv);
        const bool sh = e == p.E;
        const uint8_t* wd = static_cast<const uint8_t*>(sh ? p.s_down : p.w_down) +
                            ((sh ? 0 : static_cast<size_t>(e) * p.d) + w.row) * hs + w.kv * 16;
        const int r0 = min(16, w.nrows);
        pr.open(SlotDesc{0, static_cast<int16_t>(r0), static_cast<int16_t>(w.nrows - r0),
                         static_cast<int16_t>(n), static_cast<int16_t>(PD), w.left == 1, 1, 1, 0, mask,
                         w.seg, w.row, w.kv},
                rows, n * 16);
        pr.copy_weights(PD, wd, w.nrows, wd, 0, hs, n * 16);
        if (passed) load_h(pr.it);
      }
      pr.pass(rows * PD);
      next(w);
    }
    if (go && !passed && pr.it > first) pass_barrier();  // everything fitted
    if (!go) {  // every slot's copies are issued (H rows of any content), then land
      if (!passed) load_late_h();
      pr.drain();
    }
  } else {
    // ------------------------------------------------------------------ consumers
    const int rows = c1 - c0;
    int gu_tiles = 0;
#pragma unroll 1
    for (int at = g0; at < g1; ++gu_tiles) at += min(min(pairs, g1 - at), p.F - at % p.F);
    const int tiles[2] = {ok ? gu_tiles : 0,
                          ok && nseg > 0 ? (rows + kTileRows - 1) / kTileRows : 0};
    const int chunks[2] = {(dv + gu_vecs - 1) / gu_vecs, (fv + dn_vecs - 1) / dn_vecs * nseg};
    auto put = [&](int t, int c, float v) {
      const size_t o = static_cast<size_t>(t) * p.d + c;
      Tin* yo = static_cast<Tin*>(p.y) + o;
      if constexpr (F32) {
        *yo = p.residual ? v + X[o] : v;
      } else {
        *yo = __float2bfloat16_rn(p.residual ? v + __bfloat162float(X[o]) : v);
      }
    };
    auto epilogue = [&](const SlotDesc& d, const float* red, const Crew& crew) {
      if (d.kind == 0) {
        const int nb = __popc(d.mask), hrow = tb.seg_hrow[d.seg];
#pragma unroll 1
        for (int i = crew.index; i < 16 * nb; i += crew.count) {
          const int r = i & 15, n = i >> 4;
          if (r >= d.r0) continue;
          const float g = red_sum<NT>(red, crew.warps, 0, r, n);
          const float u = red_sum_second<F32, NT>(d, red, crew.warps, r, n);
          const float v = g / (1.f + expf(-g)) * u * tb.gate_of_row[hrow + n];
          Tin* o = H + static_cast<size_t>(hrow + n) * p.F + d.row + r;
          if constexpr (F32) *o = v;
          else *o = __float2bfloat16_rn(v);
        }
      } else {
        const int nr = d.r0 + d.r1;
#pragma unroll 1
        for (int i = tid; i < kTileRows * live; i += kConsumers) {
          const int r = i & 31, t = i >> 5;
          if (r < nr) put(t, d.row + r, red_sum<NT>(red, kConsumerWarps, 0, r, t));
        }
      }
    };
    auto between = [&](bool well) {
      fence_proxy_async_all();  // H is read by bulk copies
      well = consumer_all(well);
      if (tid == 0) grid_arrive(p.sync);
      return well;
    };
    consume<F32, NT>(s, tiles, chunks, solo_tiles<F32, NT>(tiles[0], chunks[0]), p.status, epilogue,
                     between);
    if (nseg == 0 && ok) {  // no route runs and no shared expert: only the residual is left
#pragma unroll 1
      for (int i = tid; i < rows * live; i += kConsumers) put(i / rows, c0 + i % rows, 0.f);
    }
  }
  __syncthreads();
  if (tid == 0 && *s.abort_flag == 0) grid_leave(p.sync);
}

template <typename Tin, int NT>
cudaError_t launch_nt(FewParams p, cudaStream_t s) {
  static DeviceOnce once;
  cudaError_t e = once.run([] {
    cudaError_t r = cudaFuncSetAttribute(few_layer_kernel<Tin, NT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    return r != cudaSuccess ? r : prefer_max_shared(few_layer_kernel<Tin, NT>);
  });
  if (e != cudaSuccess) return e;
  p.smem_bytes = kSmemBytes;
  return launch_cooperative(few_layer_kernel<Tin, NT>, dim3(sm_count()),
                            dim3(kThreads<sizeof(Tin) == 4, NT>), kSmemBytes, s, p);
}

template <typename Tin>
cudaError_t launch_typed(const FewParams& p, cudaStream_t s) {
  if (p.T <= 8) return launch_nt<Tin, 1>(p, s);
  if (p.T <= 16) return launch_nt<Tin, 2>(p, s);
  return launch_nt<Tin, 4>(p, s);
}

}  // namespace

FewLayout few_layer_layout(const moe_config& c) {
  auto align = [](size_t v) { return (v + 255) & ~static_cast<size_t>(255); };
  const size_t esz = c.dtype == MOE_BF16 ? 2 : 4;
  FewLayout L{};
  L.logits = kWsHeaderBytes;
  L.h = L.logits + align(static_cast<size_t>(c.T) * c.E * 4);
  L.total = L.h + align(static_cast<size_t>(c.T) * (c.k + c.has_shared) * c.d_ff * esz);
  return L;
}

bool few_layer_supported(const moe_config& c) {
  return c.T <= kMaxTokens && c.d <= (1 << 24) && c.d_ff <= (1 << 24) &&
         (c.E + 1) * static_cast<int64_t>(c.d_ff) <= INT_MAX && !c.stats &&
         c.layout == MOE_LAYOUT_RAGGED &&
         c.overflow == MOE_OVERFLOW_DROP && c.fuse == MOE_FUSE_NONE;
}

cudaError_t launch_few_layer(const moe_config& c, const FewArgs& a, void* ws, cudaStream_t s) {
  const FewLayout L = few_layer_layout(c);
  uint8_t* w = static_cast<uint8_t*>(ws);
  unsigned int* sync = reinterpret_cast<unsigned int*>(w + kWsGridSyncOffset);
  FewParams p{a.x, a.w_router, a.bias, a.w_gate, a.w_up, a.w_down, a.s_gate, a.s_up, a.s_down,
              a.y, a.ids, a.gates, a.demand, a.offsets, a.n_tokens,
              reinterpret_cast<float*>(w + L.logits), w + L.h,
              reinterpret_cast<int32_t*>(w), GridSync{sync, sync + 1, sync + 2},
              c.T, c.d, c.E, c.k, c.d_ff, c.gate_mode, c.capacity, c.has_shared,
              c.add_residual, 0};
  return c.dtype == MOE_BF16 ? launch_typed<__nv_bfloat16>(p, s) : launch_typed<float>(p, s);
}

}  // namespace moe
