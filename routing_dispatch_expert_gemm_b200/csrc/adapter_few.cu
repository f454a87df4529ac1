// A projection shared by all tokens plus each token's own low-rank adapter, for at most 32
// tokens, 16 in fp32 (moe_adapter_linear, moe_adapter_gate_up; adapter_streams in api.cu chooses):
//   p[t] = W x_t + s_a B_a (A_a x_t),  a = adapter of token t (-1: none)
//   linear   y[t] = p[t] (+ addend[t])         gate_up  h[t] = SiLU(p_gate[t]) * p_up[t]
// Source: "Mixture-of-Experts: routing and capacity", Top-k and mixture (the shared expert,
// a dense projection every token passes); "MoE Inference Visualized", Expert Execution.
//
// Bound by reading W once, and the used adapters' A and B.  One cooperative kernel over the
// streaming engine of few_stream.cuh, two phases:
//   shrink   u[t] = s_a A_a x_t: the rows of the A matrices in use, cut evenly over the CTAs,
//            each against the tokens of its adapter only; fp32, written to the workspace.
//   W        the rows of W, cut evenly over the CTAs, against all tokens.  Its weights follow
//            the A rows through the ring without a pause; only the epilogue needs u, so the
//            grid barrier between the phases is hidden behind the stream of W.  The epilogue
//            adds B_a u in fp32 (rank FMAs per output; T * rank is far too small to bound).
#include "few_stream.cuh"
#include "gemm_common.cuh"

namespace moe {
namespace {

using namespace few;

struct AdapterFewParams {
  const void* x;
  const void* w[2];
  const void* a[2];
  const void* b[2];
  const float* scale;       // null: 1
  const int32_t* ids;       // [T]
  const void* addend;       // null: none
  void* y;
  const int32_t* n_tokens;  // null: all T
  float* u;                 // [2, T, rank] scratch
  int32_t* status;
  GridSync sync;
  int T, d_in, d_out, n, rank;
  uint32_t smem_bytes;
};

// The adapters in use, in the order of their first token.
struct AdapterTables {
  int32_t id[kMaxTokens];          // of each token; -1 none
  uint32_t seg_mask[kMaxTokens];   // tokens of each adapter in use
  int32_t seg_id[kMaxTokens];
  int32_t seg_tok[kMaxTokens];     // where its tokens begin in tok
  int32_t tok[kMaxTokens];         // tokens by adapter
  int32_t nseg;
};
constexpr uint32_t kAdapterTableBytes = (sizeof(AdapterTables) + 15) & ~15u;
static_assert(kCtlBytes + kRedFloats<4> * 4 + kAdapterTableBytes + 2 * kMaxSlotBytes <= kSmemBytes,
              "the ring holds two of the largest slots");

__device__ __forceinline__ void build_adapter_tables(const AdapterFewParams& p,
                                                     AdapterTables& tb, int live) {
  const int lane = threadIdx.x & 31;
  int id = lane < live ? __ldg(p.ids + lane) : -1;
  if (id < -1 || id >= p.n) {
    if (blockIdx.x == 0) record_status(p.status, MOE_ERR_BAD_ADAPTER_ID);
    id = -1;
  }
  const uint32_t same = __match_any_sync(0xffffffffu, id);
  const bool leads = id >= 0 && __ffs(same) - 1 == lane;
  const uint32_t leaders = __ballot_sync(0xffffffffu, leads);
  const int mine = leads ? __popc(same) : 0;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  const int begin = __shfl_sync(0xffffffffu, incl - mine, __ffs(same) - 1);  // of my adapter
  tb.id[lane] = id;
  if (id >= 0) tb.tok[begin + __popc(same & ((1u << lane) - 1u))] = lane;
  if (leads) {
    const int s = __popc(leaders & ((1u << lane) - 1u));
    tb.seg_mask[s] = same;
    tb.seg_id[s] = id;
    tb.seg_tok[s] = begin;
  }
  if (lane == 0) tb.nseg = __popc(leaders);
}

// sum_j u[j] B[row, j] in fp32, fixed order.
template <typename Tin>
__device__ __forceinline__ float expand(const Tin* b, const float* u, int rank) {
  constexpr int VEC = Vec<Tin>::N;
  float v = 0.f;
#pragma unroll 4
  for (int j = 0; j < rank; j += VEC) {
    float bf[VEC];
    Vec<Tin>::to_f32(ld_vec(b + j), bf);
#pragma unroll
    for (int q = 0; q < VEC; q += 4) {
      const float4 w = __ldcg(reinterpret_cast<const float4*>(u + j + q));
      v = fmaf(bf[q], w.x, v);
      v = fmaf(bf[q + 1], w.y, v);
      v = fmaf(bf[q + 2], w.z, v);
      v = fmaf(bf[q + 3], w.w, v);
    }
  }
  return v;
}

template <typename Tin, int NT, bool PAIR>
__global__ void __launch_bounds__(kThreads<sizeof(Tin) == 4, NT>, 1)
    adapter_few_kernel(const AdapterFewParams p) {
  constexpr bool F32 = sizeof(Tin) == 4;
  constexpr int VEC = Vec<Tin>::N;
  constexpr int M = PAIR ? 2 : 1;           // projections
  constexpr int TILE = kTileRows / M;       // output rows of a tile
  extern __shared__ __align__(128) uint8_t smem[];
  const Shared s = carve<NT>(smem, kAdapterTableBytes, p.smem_bytes);
  AdapterTables& tb = *reinterpret_cast<AdapterTables*>(smem + kCtlBytes +
                                                        kRedBufs<NT> * kRedFloats<NT> * 4);
  const int tid = threadIdx.x, warp = tid >> 5;

  init_shared<F32, NT>(s);
  const int live = p.n_tokens != nullptr ? min(max(__ldg(p.n_tokens), 0), p.T) : p.T;
  if (warp == 0) build_adapter_tables(p, tb, live);
  __syncthreads();
  const int nseg = tb.nseg;
  const uint32_t all = live == 32 ? 0xffffffffu : (1u << live) - 1u;
  // this CTA's rows: of the A matrices in use ((projection, adapter, rank) order), and of W
  const int rows_a = M * nseg * p.rank, rows_w = live > 0 ? p.d_out : 0;
  const int a0 = static_cast<int>(share_begin(rows_a, blockIdx.x));
  const int a1 = static_cast<int>(share_begin(rows_a, blockIdx.x + 1));
  const int c0 = static_cast<int>(share_begin(rows_w, blockIdx.x));
  const int c1 = static_cast<int>(share_begin(rows_w, blockIdx.x + 1));
  const int dv = p.d_in / VEC;
  // chunks of the two phases
  const int vecs[2] = {chunk_vecs(min(kTileRows, a1 - a0) + live, dv, kThinSlot),
                       chunk_vecs(M * min(TILE, c1 - c0) + live, dv, kThinSlot)};
  const int chunks[2] = {(dv + vecs[0] - 1) / vecs[0], (dv + vecs[1] - 1) / vecs[1]};
  auto shrink_rows = [&](int at) {  // rows of the shrink tile at `at`: within one matrix
    return min(min(kTileRows, a1 - at), p.rank - at % p.rank);
  };

  if (warp >= kConsumerWarps) {
    // ------------------------------------------------------------------ producers
    const size_t xs = static_cast<size_t>(p.d_in) * sizeof(Tin);
    const uint8_t* xb = static_cast<const uint8_t*>(p.x);
    Producer<kTeamWarps<F32, NT>> pr(s, p.status);
    bool go = true;
    // a tile: n0 rows from w0, then n1 rows from w1, against the tokens of `mask`
    auto tile = [&](const uint8_t* w0, int n0, const uint8_t* w1, int n1, uint32_t mask, int seg,
                    int row, int kind) {
      const uint32_t rows = n0 + n1 + __popc(mask);
      const int cv = kind == 0 ? vecs[0] : vecs[1], nc = kind == 0 ? chunks[0] : chunks[1];
      const uint32_t P = pitch_of<F32>(cv);
      int c = blockIdx.x % nc;  // not all CTAs read the same token chunk at once
      for (int i = 0; i < nc; ++i, c = c + 1 == nc ? 0 : c + 1) {
        const int kv = c * cv;
        pr.reserve(rows * P);
        if (pr.mine()) {
          if (pr.ready(rows * P, 0xffffffffu) != 1) { go = false; return; }
          const int n = min(cv, dv - kv);
          const uint32_t bytes = n * 16, o = kv * 16;
          pr.open(SlotDesc{0, static_cast<int16_t>(n0), static_cast<int16_t>(n1),
                           static_cast<int16_t>(n), static_cast<int16_t>(P), i + 1 == nc,
                           static_cast<int8_t>(kind), 0, 0, mask, seg, row, kv},
                  rows, bytes);
          pr.copy_weights(P, w0 + o, n0, w1 + o, n1, xs, bytes);
          pr.copy_tokens(P, n0 + n1, xb + o, xs, mask, bytes);
        }
        pr.pass(rows * P);
      }
    };
    // one loop over the tiles of both phases: the copies' code once
    const int w_tiles = (c1 - c0 + TILE - 1) / TILE;
#pragma unroll 1
    for (int at = a0, i = 0; (at < a1 || i < w_tiles) && go;) {
      const uint8_t *w0, *w1;
      int n0, n1, seg = 0, row, kind = 0;
      uint32_t mask = all;
      if (at < a1) {
        const int n = shrink_rows(at);
        seg = at / p.rank;
        row = at - seg * p.rank;
        const int m = PAIR && seg >= nseg ? 1 : 0;
        w0 = static_cast<const uint8_t*>(p.a[m]) +
             (static_cast<size_t>(tb.seg_id[seg - m * nseg]) * p.rank + row) * xs;
        w1 = w0 + 16 * xs;
        n0 = min(16, n);
        n1 = n - n0;
        mask = tb.seg_mask[seg - m * nseg];
        at += n;
      } else {
        row = c0 + i * TILE;
        const int n = min(TILE, c1 - row);
        w0 = static_cast<const uint8_t*>(p.w[0]) + static_cast<size_t>(row) * xs;
        n0 = PAIR ? n : min(16, n);
        n1 = PAIR ? n : n - n0;
        w1 = PAIR ? static_cast<const uint8_t*>(p.w[M - 1]) + static_cast<size_t>(row) * xs
                  : w0 + 16 * xs;
        kind = 1;
        ++i;
      }
      tile(w0, n0, w1, n1, mask, seg, row, kind);
    }
    if (!go) pr.drain();
  } else {
    // ------------------------------------------------------------------ consumers
    // bring this CTA's rows of the B matrices into L2 while A and W stream
    {
      const uint32_t bytes = static_cast<uint32_t>(c1 - c0) * p.rank * sizeof(Tin);
      const int lines = (bytes + 127) / 128;
#pragma unroll 1
      for (int i = tid; i < M * nseg * lines; i += kConsumers) {
        const int seg = i / lines, m = PAIR && seg >= nseg ? 1 : 0;
        const uint8_t* b =
            static_cast<const uint8_t*>(p.b[m]) +
            (static_cast<size_t>(tb.seg_id[seg - m * nseg]) * p.d_out + c0) * p.rank * sizeof(Tin);
        asm volatile("prefetch.global.L2 [%0];" ::"l"(b + min((i % lines) * 128u, bytes - 1)));
      }
    }
    int a_tiles = 0;
#pragma unroll 1
    for (int at = a0; at < a1; ++a_tiles) at += shrink_rows(at);
    const int tiles[2] = {a_tiles, (c1 - c0 + TILE - 1) / TILE};
    bool waited = nseg == 0;
    auto epilogue = [&](const SlotDesc& d, const float* red, const Crew&) {
      if (d.kind == 0) {
        const int m = PAIR && d.seg >= nseg ? 1 : 0, seg = d.seg - m * nseg;
        const int nr = d.r0 + d.r1, nb = __popc(d.mask);
        const float sc = p.scale != nullptr ? __ldg(p.scale + tb.seg_id[seg]) : 1.f;
#pragma unroll 1
        for (int i = tid; i < kTileRows * nb; i += kConsumers) {
          const int r = i & 31, n = i >> 5;
          if (r < nr)
            p.u[(static_cast<size_t>(m) * p.T + tb.tok[tb.seg_tok[seg] + n]) * p.rank + d.row +
                r] = sc * red_sum<NT>(red, kConsumerWarps, 0, r, n);
        }
        return;
      }
      if (!waited) {  // u is complete
        if (!grid_wait_warps(p.sync, gridDim.x, tid < 32, s.passed, s.abort_flag, p.status)) return;
        waited = true;
      }
      const int nr = PAIR ? d.r0 : d.r0 + d.r1;
#pragma unroll 1
      for (int i = tid; i < TILE * live; i += kConsumers) {
        const int r = i % TILE, t = i / TILE;
        if (r >= nr) continue;
        const int c = d.row + r, id = tb.id[t];
        float v[M];
#pragma unroll
        for (int m = 0; m < M; ++m) {
          v[m] = m == 0 ? red_sum<NT>(red, kConsumerWarps, 0, r, t)
                        : red_sum_second<F32, NT>(d, red, kConsumerWarps, r, t);
          if (id >= 0)
            v[m] += expand(static_cast<const Tin*>(p.b[m]) +
                               (static_cast<size_t>(id) * p.d_out + c) * p.rank,
                           p.u + (static_cast<size_t>(m) * p.T + t) * p.rank, p.rank);
        }
        const size_t o = static_cast<size_t>(t) * p.d_out + c;
        float out = v[0];
        if constexpr (PAIR) out = v[0] / (1.f + expf(-v[0])) * v[M - 1];
        if constexpr (F32) {
          if (!PAIR && p.addend != nullptr) out += static_cast<const float*>(p.addend)[o];
          static_cast<float*>(p.y)[o] = out;
        } else {
          if (!PAIR && p.addend != nullptr)
            out += __bfloat162float(static_cast<const __nv_bfloat16*>(p.addend)[o]);
          static_cast<__nv_bfloat16*>(p.y)[o] = __float2bfloat16_rn(out);
        }
      }
    };
    auto between = [&](bool well) {
      well = consumer_all(well);
      if (tid == 0) grid_arrive(p.sync);
      return well;
    };
    consume<F32, NT>(s, tiles, chunks, false, p.status, epilogue, between);
  }
  __syncthreads();
  if (tid == 0 && *s.abort_flag == 0) grid_leave(p.sync);
}

template <typename Tin, int NT, bool PAIR>
cudaError_t launch_pair(AdapterFewParams p, cudaStream_t s) {
  static DeviceOnce once;
  cudaError_t e = once.run([] {
    cudaError_t r = cudaFuncSetAttribute(adapter_few_kernel<Tin, NT, PAIR>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    return r != cudaSuccess ? r : prefer_max_shared(adapter_few_kernel<Tin, NT, PAIR>);
  });
  if (e != cudaSuccess) return e;
  p.smem_bytes = kSmemBytes;
  return launch_cooperative(adapter_few_kernel<Tin, NT, PAIR>, dim3(sm_count()),
                            dim3(kThreads<sizeof(Tin) == 4, NT>), kSmemBytes, s, p);
}

template <typename Tin>
cudaError_t launch_typed(const AdapterFewParams& p, bool pair, cudaStream_t s) {
  if (p.T <= 8) return pair ? launch_pair<Tin, 1, true>(p, s) : launch_pair<Tin, 1, false>(p, s);
  if (p.T <= 16) return pair ? launch_pair<Tin, 2, true>(p, s) : launch_pair<Tin, 2, false>(p, s);
  // (fp32 beyond 16 tokens is the CUDA-core GEMM's)
  if constexpr (sizeof(Tin) == 4) return cudaErrorInvalidValue;
  else return pair ? launch_pair<Tin, 4, true>(p, s) : launch_pair<Tin, 4, false>(p, s);
}

}  // namespace

cudaError_t launch_adapter_few(const moe_adapter_config& c, const AdapterArgs& a,
                               const AdapterLayout& L, void* ws, cudaStream_t s) {
  if (c.T > kMaxTokens) return cudaErrorInvalidValue;
  uint8_t* w = static_cast<uint8_t*>(ws);
  unsigned int* sync = reinterpret_cast<unsigned int*>(w + kWsGridSyncOffset);
  const AdapterFewParams p{a.x, {a.w[0], a.w[1]}, {a.a[0], a.a[1]}, {a.b[0], a.b[1]}, a.scale,
                           a.ids, a.addend, a.y, a.n_tokens,
                           reinterpret_cast<float*>(w + L.u), reinterpret_cast<int32_t*>(w),
                           GridSync{sync, sync + 1, sync + 2}, c.T, c.d_in, c.d_out, c.n_adapters, c.rank,
                           0};
  return c.dtype == MOE_BF16 ? launch_typed<__nv_bfloat16>(p, a.pair, s)
                             : launch_typed<float>(p, a.pair, s);
}

}  // namespace moe
