// Projections with per-token low-rank adapters in fp32, where the few-token kernel does not run
// (moe_adapter_linear, moe_adapter_gate_up):
//   p[t] = W x_t + s_a B_a (A_a x_t);  y[t] = p[t] (+ addend[t])  or  SiLU(p_gate) * p_up
// CUDA cores, as the fp32 expert FFN: tf32 cannot meet its tolerance.  Two launches:
//   shrink  u[t] = s_a A_a x_t, one warp per token and four ranks.
//   GEMM    with enough tiles for the SMs, tiles of 64 tokens x 64 rows of W staged 32 columns
//           at a time in shared memory, the next stage's loads in registers, 4 x 4 outputs per
//           thread (bound by FMA, 128 per SM and clock); else a warp per 4 tokens x 4 rows,
//           its lanes splitting the contraction, straight from L1 (T=77, 1000x516: 33 us with
//           small shared-memory tiles, whose latencies follow one another).  The epilogue adds
//           B_a u.
#include <algorithm>

#include "gemm_common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

struct SimtParams {
  const float* x;
  const float* w[2];
  const float* a[2];
  const float* b[2];
  const float* scale;
  const int32_t* ids;
  const float* addend;
  float* y;
  const int32_t* n_tokens;
  float* u;
  int32_t* status;
  int T, d_in, d_out, n, rank;
};

__device__ __forceinline__ int live_tokens(const SimtParams& p) {
  return p.n_tokens != nullptr ? min(max(__ldg(p.n_tokens), 0), p.T) : p.T;
}

__global__ void __launch_bounds__(kThreads) adapter_shrink_f32_kernel(const SimtParams p) {
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int quads = p.rank / 4;  // rank is a multiple of 4
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int t = static_cast<int>(item / quads), j0 = static_cast<int>(item % quads) * 4;
  const int m = blockIdx.y;
  if (t >= live_tokens(p)) return;
  const int id = __ldg(p.ids + t);
  if (id < 0 || id >= p.n) {
    if (id != -1 && lane == 0 && j0 == 0 && m == 0) record_status(p.status, MOE_ERR_BAD_ADAPTER_ID);
    return;
  }
  const float4* x = reinterpret_cast<const float4*>(p.x + static_cast<size_t>(t) * p.d_in);
  const float4* a = reinterpret_cast<const float4*>(
      p.a[m] + (static_cast<size_t>(id) * p.rank + j0) * p.d_in);
  const int dv = p.d_in / 4;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
  for (int v = lane; v < dv; v += 32) {
    const float4 xv = __ldg(x + v);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 av = __ldg(a + static_cast<size_t>(j) * dv + v);
      s[j] = fmaf(xv.x, av.x, fmaf(xv.y, av.y, fmaf(xv.z, av.z, fmaf(xv.w, av.w, s[j]))));
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) s[j] += __shfl_xor_sync(0xffffffffu, s[j], o);
  if (lane == 0) {
    const float sc = p.scale != nullptr ? __ldg(p.scale + id) : 1.f;
    *reinterpret_cast<float4*>(p.u + (static_cast<size_t>(m) * p.T + t) * p.rank + j0) =
        make_float4(sc * s[0], sc * s[1], sc * s[2], sc * s[3]);
  }
}

// Adds B_a u to output (t, c) of each projection, finishes and stores it.
template <bool PAIR>
__device__ __forceinline__ void finish_f32(const SimtParams& p, float (&v)[PAIR ? 2 : 1], int t,
                                           int c) {
  constexpr int M = PAIR ? 2 : 1;
  const int id = __ldg(p.ids + t);
  if (id >= 0 && id < p.n) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const float4* u =
          reinterpret_cast<const float4*>(p.u + (static_cast<size_t>(m) * p.T + t) * p.rank);
      const float4* b = reinterpret_cast<const float4*>(
          p.b[m] + (static_cast<size_t>(id) * p.d_out + c) * p.rank);
      float s = 0.f;
#pragma unroll 4
      for (int r = 0; r < p.rank / 4; ++r) {
        const float4 uv = __ldcg(u + r), bv = __ldg(b + r);
        s = fmaf(uv.x, bv.x, fmaf(uv.y, bv.y, fmaf(uv.z, bv.z, fmaf(uv.w, bv.w, s))));
      }
      v[m] += s;
    }
  }
  const size_t o = static_cast<size_t>(t) * p.d_out + c;
  float out = v[0];
  if constexpr (PAIR) out = out / (1.f + expf(-out)) * v[M - 1];
  else if (p.addend != nullptr) out += p.addend[o];
  p.y[o] = out;
}

template <bool PAIR, int BT, int BC, int RT, int RC, int BKF>
__global__ void __launch_bounds__(kThreads) adapter_gemm_f32_kernel(const SimtParams p) {
  constexpr int M = PAIR ? 2 : 1;
  constexpr int TX = BC / RC;                 // threads across the rows of W
  constexpr int ROWS = BT + M * BC;           // rows staged: tokens, then W's
  constexpr int LOADS = (ROWS * (BKF / 4) + kThreads - 1) / kThreads;
  static_assert(TX * (BT / RT) == kThreads, "one micro-tile per thread");
  // [column][row]: a thread's RT tokens and RC rows are consecutive
  __shared__ __align__(16) float s_x[BKF][BT + 4];
  __shared__ __align__(16) float s_w[M][BKF][BC + 4];
  const int live = live_tokens(p);
  const int t0 = blockIdx.x * BT, c0 = blockIdx.y * BC;
  if (t0 >= live) return;
  const int tid = threadIdx.x, tx = tid % TX, ty = tid / TX;

  float4 next[LOADS];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int at = tid + i * kThreads, row = at / (BKF / 4), k = k0 + at % (BKF / 4) * 4;
      const float* src = nullptr;
      if (row < BT) {
        if (t0 + row < live) src = p.x + static_cast<size_t>(t0 + row) * p.d_in;
      } else if (row < ROWS) {
        const int m = (row - BT) / BC, c = c0 + (row - BT) % BC;
        if (c < p.d_out) src = p.w[m] + static_cast<size_t>(c) * p.d_in;
      }
      next[i] = src != nullptr && k < p.d_in ? __ldg(reinterpret_cast<const float4*>(src + k))
                                             : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  auto stage = [&] {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int at = tid + i * kThreads, row = at / (BKF / 4), k = at % (BKF / 4) * 4;
      if (row >= ROWS) continue;
      const float v[4] = {next[i].x, next[i].y, next[i].z, next[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (row < BT) s_x[k + j][row] = v[j];
        else s_w[(row - BT) / BC][k + j][(row - BT) % BC] = v[j];
      }
    }
  };
  float acc[M][RT][RC] = {};
  fetch(0);
  for (int k0 = 0; k0 < p.d_in; k0 += BKF) {
    __syncthreads();
    stage();
    __syncthreads();
    if (k0 + BKF < p.d_in) fetch(k0 + BKF);
#pragma unroll 8
    for (int k = 0; k < BKF; ++k) {
      float xr[RT], wr[M][RC];
#pragma unroll
      for (int i = 0; i < RT; ++i) xr[i] = s_x[k][ty * RT + i];
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int j = 0; j < RC; ++j) wr[m][j] = s_w[m][k][tx * RC + j];
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int j = 0; j < RC; ++j) acc[m][i][j] = fmaf(xr[i], wr[m][j], acc[m][i][j]);
    }
  }
  pdl_wait();  // u is complete; what read y before this call is done
#pragma unroll 1
  for (int i = 0; i < RT; ++i) {
    const int t = t0 + ty * RT + i;
    if (t >= live) continue;
#pragma unroll
    for (int j = 0; j < RC; ++j) {
      float v[M];
#pragma unroll
      for (int m = 0; m < M; ++m) {
        v[m] = acc[m][0][j];
#pragma unroll
        for (int q = 1; q < RT; ++q) v[m] = i == q ? acc[m][q][j] : v[m];
      }
      if (c0 + tx * RC + j < p.d_out) finish_f32<PAIR>(p, v, t, c0 + tx * RC + j);
    }
  }
}

// A warp per kWT tokens x kWC rows of W.
constexpr int kWT = 4, kWC = 4;
template <bool PAIR>
__global__ void __launch_bounds__(kThreads) adapter_warp_f32_kernel(const SimtParams p) {
  constexpr int M = PAIR ? 2 : 1;
  const int live = live_tokens(p);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // 2 x 4 warps of a CTA share token and weight rows through L1
  const int t0 = (blockIdx.x * 2 + warp / 4) * kWT, c0 = (blockIdx.y * 4 + warp % 4) * kWC;
  if (t0 >= live || c0 >= p.d_out) return;
  const int dv = p.d_in / 4;
  const float4* x[kWT];
  const float4* w[M][kWC];
#pragma unroll
  for (int i = 0; i < kWT; ++i)  // rows past the last one: the last one's, not stored
    x[i] = reinterpret_cast<const float4*>(p.x + static_cast<size_t>(min(t0 + i, live - 1)) * p.d_in);
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int j = 0; j < kWC; ++j)
      w[m][j] = reinterpret_cast<const float4*>(
          p.w[m] + static_cast<size_t>(min(c0 + j, p.d_out - 1)) * p.d_in);
  float acc[M][kWT][kWC] = {};
#pragma unroll 2
  for (int v = lane; v < dv; v += 32) {
    float4 xv[kWT], wv[M][kWC];
#pragma unroll
    for (int i = 0; i < kWT; ++i) xv[i] = __ldg(x[i] + v);
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int j = 0; j < kWC; ++j) wv[m][j] = __ldg(w[m][j] + v);
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int i = 0; i < kWT; ++i)
#pragma unroll
        for (int j = 0; j < kWC; ++j) {
          float& s = acc[m][i][j];
          s = fmaf(xv[i].x, wv[m][j].x, s);
          s = fmaf(xv[i].y, wv[m][j].y, s);
          s = fmaf(xv[i].z, wv[m][j].z, s);
          s = fmaf(xv[i].w, wv[m][j].w, s);
        }
  }
  // lane l < 16 gets the total of output (l / 4, l % 4)
  float v[M];
#pragma unroll
  for (int m = 0; m < M; ++m) {
    v[m] = 0.f;
#pragma unroll
    for (int i = 0; i < kWT; ++i)
#pragma unroll
      for (int j = 0; j < kWC; ++j) {
        float s = acc[m][i][j];
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == i * kWC + j) v[m] = s;
      }
  }
  pdl_wait();  // u is complete; what read y before this call is done
  const int t = t0 + lane / kWC, c = c0 + lane % kWC;
  if (lane < kWT * kWC && t < live && c < p.d_out) finish_f32<PAIR>(p, v, t, c);
}

template <bool PAIR, int BT, int BC, int RT, int RC, int BKF>
cudaError_t launch_tile(const SimtParams& p, cudaStream_t s) {
  static DeviceOnce once;
  cudaError_t e =
      once.run([] { return prefer_max_shared(adapter_gemm_f32_kernel<PAIR, BT, BC, RT, RC, BKF>); });
  if (e != cudaSuccess) return e;
  // tokens on grid.x: grid.y ends at 65535 blocks
  const int rows = (p.d_out + BC - 1) / BC;
  if (rows > 65535) return cudaErrorInvalidValue;
  return launch_pdl(adapter_gemm_f32_kernel<PAIR, BT, BC, RT, RC, BKF>,
                    dim3((p.T + BT - 1) / BT, rows), dim3(kThreads), 0, s, p);
}

template <bool PAIR>
cudaError_t launch_gemm_f32(const SimtParams& p, cudaStream_t s) {
  const int64_t big = static_cast<int64_t>((p.d_out + 63) / 64) * ((p.T + 63) / 64);
  const int rows = (p.d_out + 4 * kWC - 1) / (4 * kWC);
  if (big * 2 >= sm_count() || rows > 65535) return launch_tile<PAIR, 64, 64, 4, 4, 32>(p, s);
  static DeviceOnce once;
  const cudaError_t e = once.run([] { return prefer_max_shared(adapter_warp_f32_kernel<PAIR>); });
  if (e != cudaSuccess) return e;
  return launch_pdl(adapter_warp_f32_kernel<PAIR>, dim3((p.T + 2 * kWT - 1) / (2 * kWT), rows),
                    dim3(kThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_adapter_simt(const moe_adapter_config& c, const AdapterArgs& a,
                                const AdapterLayout& L, void* ws, cudaStream_t s) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  auto f = [](const void* q) { return static_cast<const float*>(q); };
  const SimtParams p{f(a.x), {f(a.w[0]), f(a.w[1])}, {f(a.a[0]), f(a.a[1])},
                     {f(a.b[0]), f(a.b[1])}, a.scale, a.ids, f(a.addend),
                     static_cast<float*>(a.y), a.n_tokens, reinterpret_cast<float*>(w + L.u),
                     reinterpret_cast<int32_t*>(w), c.T, c.d_in, c.d_out, c.n_adapters, c.rank};
  static DeviceOnce once;
  cudaError_t e = once.run([] { return prefer_max_shared(adapter_shrink_f32_kernel); });
  if (e != cudaSuccess) return e;
  const int64_t items = static_cast<int64_t>(c.T) * (c.rank / 4);
  adapter_shrink_f32_kernel<<<dim3(static_cast<unsigned>((items + 7) / 8), a.pair ? 2 : 1),
                              kThreads, 0, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return a.pair ? launch_gemm_f32<true>(p, s) : launch_gemm_f32<false>(p, s);
}

}  // namespace moe
