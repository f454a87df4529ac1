// C ABI of libmoe.so: argument validation, workspace layout and launch sequencing.
// Every entry point is declared, with argument meaning, layout, ownership and error
// behaviour, in include/moe.h.
#include <algorithm>
#include <climits>
#include <cmath>
#include <initializer_list>

#include "common.cuh"
#include "internal.h"

using namespace moe;

namespace moe {

// Host-side checks shared by every entry point that takes a config (declared in
// internal.h).
moe_status validate_config(const moe_config* c) {
  if (c == nullptr) return MOE_ERR_INVALID;
  if (c->T < 1 || c->d < 1 || c->E < 1 || c->k < 1 || c->d_ff < 1) return MOE_ERR_INVALID;
  if (c->k > c->E) return MOE_ERR_INVALID;
  if (c->dtype != MOE_F32 && c->dtype != MOE_BF16) return MOE_ERR_INVALID;
  if (c->gate_mode < MOE_GATE_SOFTMAX_TOPK || c->gate_mode > MOE_GATE_TOPK_SOFTMAX)
    return MOE_ERR_INVALID;
  if ((c->has_shared != 0 && c->has_shared != 1) || (c->add_residual != 0 && c->add_residual != 1) ||
      (c->stats != 0 && c->stats != 1))
    return MOE_ERR_INVALID;
  if ((c->layout != MOE_LAYOUT_RAGGED && c->layout != MOE_LAYOUT_PADDED) ||
      (c->overflow != MOE_OVERFLOW_DROP && c->overflow != MOE_OVERFLOW_REROUTE))
    return MOE_ERR_INVALID;
  if (c->tiles < MOE_TILES_AUTO || c->tiles > MOE_TILES_ROW_PAIRS) return MOE_ERR_INVALID;
  if (c->fuse < 0 || c->fuse > (MOE_FUSE_GATHER | MOE_FUSE_COMBINE)) return MOE_ERR_INVALID;
  if (c->fuse != 0 && (c->tiles == MOE_TILES_ROWS || c->tiles == MOE_TILES_ROW_PAIRS))
    return MOE_ERR_INVALID;
  if (c->fuse != 0 && (c->dtype != MOE_BF16 || c->overflow != MOE_OVERFLOW_DROP))
    return MOE_ERR_UNSUPPORTED;
  if (c->layout == MOE_LAYOUT_PADDED && c->capacity < 0) return MOE_ERR_INVALID;  // C sizes it
  if (c->overflow == MOE_OVERFLOW_REROUTE && c->layout != MOE_LAYOUT_PADDED)
    return MOE_ERR_UNSUPPORTED;
  if (c->E > 256 || c->k > 32) return MOE_ERR_UNSUPPORTED;
  if (c->T > (1 << 24) || static_cast<int64_t>(c->T) * c->k > (INT_MAX / 2)) return MOE_ERR_UNSUPPORTED;
  if (c->layout == MOE_LAYOUT_PADDED && static_cast<int64_t>(c->E) * c->capacity > (INT_MAX / 2))
    return MOE_ERR_UNSUPPORTED;
  if (c->dtype == MOE_BF16) {
    if (c->d % 128 != 0 || c->d_ff % 128 != 0) return MOE_ERR_UNSUPPORTED;
  } else {
    if (c->d % 4 != 0 || c->d_ff % 4 != 0) return MOE_ERR_UNSUPPORTED;
  }
  return MOE_OK;
}

}  // namespace moe

namespace {

moe_status validate(const moe_config* c) { return validate_config(c); }

constexpr int32_t kAbiVersion = 5;

size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

int64_t max_rows(const moe_config& c) {
  if (c.layout == MOE_LAYOUT_PADDED)
    return std::max<int64_t>(static_cast<int64_t>(c.E) * c.capacity, 1);
  int64_t r = static_cast<int64_t>(c.T) * c.k;
  if (c.capacity >= 0) r = std::min<int64_t>(r, static_cast<int64_t>(c.E) * c.capacity);
  return std::max<int64_t>(r, 1);
}

bool padded(const moe_config& c) { return c.layout == MOE_LAYOUT_PADDED; }
bool reroute(const moe_config& c) { return c.overflow == MOE_OVERFLOW_REROUTE; }
// Entries of the segment table (offsets): starts, plus the filled-slot counts when padded.
size_t offsets_len(const moe_config& c) { return c.E + 2 + (padded(c) ? c.E : 0); }

struct Layout {
  size_t tile_hist, tile_psum, stats_partial, zkeys, rlist, need, counters;
  size_t ids, gates, route_row, row_token, offsets, demand;
  size_t x_packed, h, y_packed;
  size_t scratch_end, total;
  int64_t rmax, rows_h;
};

Layout layout_of(const moe_config& c) {
  Layout L{};
  size_t off = kWsHeaderBytes;
  auto take = [&off](size_t bytes) {
    const size_t o = off;
    off = align256(off + bytes);
    return o;
  };
  const size_t esz = (c.dtype == MOE_BF16) ? 2 : 4;
  const size_t Tk = static_cast<size_t>(c.T) * c.k;
  L.rmax = max_rows(c);
  L.rows_h = L.rmax + (c.has_shared ? c.T : 0);
  L.tile_hist = take(static_cast<size_t>(num_tiles_for(c.T, c.E)) * c.E * 4);
  // Routing statistics (only with cfg.stats): per-tile probability sums and fp64 partials.
  L.tile_psum = c.stats ? take(static_cast<size_t>(num_tiles_for(c.T, c.E)) * c.E * 4) : 0;
  L.stats_partial = c.stats ? take(static_cast<size_t>(kStatsMaxBlocks) * c.E * 8) : 0;
  // Reroute policy (only with it): the router's ranking keys and the placement's scratch.
  L.zkeys = reroute(c) ? take(static_cast<size_t>(c.T) * c.E * 4) : 0;
  L.rlist = reroute(c) ? take(reroute_scratch_bytes(c)) : 0;
  // Fused combine (MOE_FUSE_COMBINE): contributions per token, counters per 32 columns.
  L.need = (c.fuse & MOE_FUSE_COMBINE) ? take(static_cast<size_t>(c.T) * 4) : 0;
  L.counters = (c.fuse & MOE_FUSE_COMBINE) ? take(static_cast<size_t>(c.T) * ((c.d + 31) / 32) * 4)
                                           : 0;
  L.scratch_end = off;
  L.ids = take(Tk * 4);
  L.gates = take(Tk * 4);
  L.route_row = take(Tk * 4);
  L.row_token = take(static_cast<size_t>(L.rmax) * 4);
  L.offsets = take(offsets_len(c) * 4);
  L.demand = take(static_cast<size_t>(c.E) * 4);
  L.x_packed = take(static_cast<size_t>(L.rmax) * c.d * esz);
  L.h = take(static_cast<size_t>(L.rows_h) * c.d_ff * esz);
  L.y_packed = take(static_cast<size_t>(L.rows_h) * c.d * esz);
  L.total = off;
  return L;
}

moe_status check_ws(const void* ws) {
  if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255) != 0) return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

template <typename P>
uint8_t* at(P* base, size_t off) {
  return reinterpret_cast<uint8_t*>(const_cast<void*>(static_cast<const void*>(base))) + off;
}

// Rows read by 16-byte loads and bulk copies.
bool aligned16(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if ((reinterpret_cast<uintptr_t>(p) & 15) != 0) return false;
  return true;
}

// Whether a of `an` bytes and b of `bn` share any.
bool overlap(const void* a, int64_t an, const void* b, int64_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + static_cast<uintptr_t>(bn) && y < x + static_cast<uintptr_t>(an);
}

moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

#define MOE_TRY(expr)                 \
  do {                                \
    const moe_status st_ = (expr);    \
    if (st_ != MOE_OK) return st_;    \
  } while (0)

moe_status ffn(const moe_config& c, const FfnArgs& f, cudaStream_t s, cudaEvent_t mid = nullptr) {
  return cuda_status(c.dtype == MOE_BF16 ? launch_ffn_sm100(c, f, s, mid)
                                         : launch_ffn_simt(c, f, s, mid));
}

moe_status validate_adapter(const moe_adapter_config* c) {
  if (c == nullptr) return MOE_ERR_INVALID;
  if (c->T < 1 || c->d_in < 1 || c->d_out < 1 || c->n_adapters < 1 || c->rank < 1)
    return MOE_ERR_INVALID;
  if (c->dtype != MOE_F32 && c->dtype != MOE_BF16) return MOE_ERR_INVALID;
  const int unit = c->dtype == MOE_BF16 ? 8 : 4;
  if (c->d_in % unit != 0 || c->d_out % unit != 0 || c->rank % unit != 0 || c->rank > 128)
    return MOE_ERR_UNSUPPORTED;
  const int64_t limit = int64_t{1} << 40;
  if (c->T > (1 << 24) || static_cast<int64_t>(c->T) * c->d_in >= limit ||
      static_cast<int64_t>(c->T) * c->d_out >= limit ||
      static_cast<int64_t>(c->d_in) * c->d_out >= limit || c->d_out > (1 << 20) || c->d_in > (1 << 24))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Whether the streaming kernel runs a call of at most 32 tokens.  Measured, us streaming / other
// kernel (W from HBM, 16 adapters in use).
//   bf16: it reads the token rows once per CTA, so more than 8 tokens beside a large W are better off
// on tcgen05, and up to 8 a large pair whose GEMM splits the contraction and shrinks in the same
// launch; but tcgen05's shrink and expansion grow with the rank, which costs streaming little.
//   rank 16   linear 2048x2048 T=16 12 / 15, T=24 15 / 15, T=32 16 / 15; 4096x2048 T=12 14 / 16, T=16
//             17 / 16; 4096x4096 T=8 15 / 18, T=16 21 / 18; 14336x4096 T=8 31 / 31, T=12 43 / 31;
//             8192x28672 T=8 91 / 108, T=12 112 / 99; gate/up 2048x2816 T=16 18 / 19, 4096x4096
//             T=8 23 / 25, T=12 28 / 25, 4096x8192 T=4 35 / 34, T=8 40 / 35, 4096x14336 (not split)
//             T=8 61 / 69, T=12 70 / 53
//   rank 32   linear 4096x4096 T=16 19 / 19, T=24 25 / 20, 4096x8192 T=12 27 / 24; gate/up 4096x8192
//             T=8 40 / 40, T=12 46 / 40
//   rank 64   linear 4096x4096 T=16 22 / 30, T=32 32 / 34, 4096x8192 T=16 34 / 37, T=24 45 / 42,
//             14336x4096 T=12 51 / 47; gate/up 4096x8192 T=8 46 / 58
//   rank 128  linear 4096x4096 T=16 25 / 46, T=32 37 / 54, 14336x4096 T=16 57 / 74, T=32 91 / 91,
//             8192x28672 T=8 128 / 178; gate/up 4096x8192 T=24 105 / 127
//   fp32: the streaming loop loads a token's vector again for each row of W, the other kernel holds 4
// tokens by 4 rows, but its warp goes through all of d_in alone, in as many rounds as its tiles take,
// and beyond 4096 rows of W it is the one with 64-token tiles.
//   linear    512x512 T=1 10 / 4; 1024x1024 T=8 11 / 10, T=16 23 / 10; 2048x1024 T=8 13 / 16, T=9
//             21 / 14; 2048x2048 T=4 14 / 16, T=8 16 / 17, T=16 32 / 18; 2048x4096 T=8 24 / 18;
//             4096x1024 T=8 18 / 30, T=16 52 / 29; 4096x4096 T=4 29 / 32, T=8 40 / 33, T=12
//             57 / 60, T=16 73 / 61; 8192x8192 T=16 222 / 360, T=32 554 / 363
//   gate/up   1024x1024 T=1 11 / 12, T=8 13 / 13, T=16 23 / 13; 2048x2048 T=4 20 / 21, T=8 25 / 22,
//             T=9 33 / 38, T=16 44 / 40; 4096x4096 T=8 67 / 77, T=16 123 / 142, T=32 290 / 250
bool adapter_streams(const moe_adapter_config& c, bool pair) {
  if (c.T > 32) return false;
  const int64_t rows = static_cast<int64_t>(c.d_out) * (pair ? 2 : 1), weights = rows * c.d_in;
  if (c.dtype == MOE_F32) {
    if (rows > 4096) return c.T <= 16;
    return c.T <= 8 && c.d_in > 1024 && (c.T <= 4 || c.d_in > c.d_out);
  }
  if (c.T <= 4) return true;
  if (c.T <= 8 && (c.rank > 16 || !adapter_splits(c, pair))) return true;
  const int mi = c.T <= 8 ? 60 : c.T <= 16 ? 12 : 6;  // Mi weights, at rank 16
  return weights <= (int64_t{mi} << 20) * std::max(c.rank, 16) / 16 * (c.rank > 64 ? 2 : 1);
}

AdapterLayout adapter_layout(const moe_adapter_config& c) {
  AdapterLayout L{};
  L.u = kWsHeaderBytes;
  L.blocks = align256(L.u + adapter_u_bytes(c));
  L.broken = align256(L.blocks + adapter_block_table_bytes(c.T));
  L.total = align256(L.broken + 2 * static_cast<size_t>(c.T));
  return L;
}

moe_status adapter_impl(const moe_adapter_config* cfg, const AdapterArgs& a, void* ws,
                        cudaStream_t stream) {
  MOE_TRY(validate_adapter(cfg));
  MOE_TRY(check_ws(ws));
  if (!a.x || !a.w[0] || !a.a[0] || !a.b[0] || !a.ids || !a.y) return MOE_ERR_INVALID;
  if (a.pair && (!a.w[1] || !a.a[1] || !a.b[1])) return MOE_ERR_INVALID;
  if (!aligned16({a.x, a.w[0], a.w[1], a.a[0], a.a[1], a.b[0], a.b[1]})) return MOE_ERR_INVALID;
  // x is read for other rows and columns after y's first are written; the addend is read where y
  // is written
  const int64_t esz = cfg->dtype == MOE_BF16 ? 2 : 4, yb = int64_t{1} * cfg->T * cfg->d_out * esz;
  if (overlap(a.x, int64_t{1} * cfg->T * cfg->d_in * esz, a.y, yb)) return MOE_ERR_INVALID;
  if (a.addend != nullptr && a.addend != a.y && overlap(a.addend, yb, a.y, yb))
    return MOE_ERR_INVALID;
  const AdapterLayout L = adapter_layout(*cfg);
  if (adapter_streams(*cfg, a.pair))
    return cuda_status(launch_adapter_few(*cfg, a, L, ws, stream));
  return cuda_status(cfg->dtype == MOE_BF16 ? launch_adapter_sm100(*cfg, a, L, ws, stream)
                                            : launch_adapter_simt(*cfg, a, L, ws, stream));
}

moe_status record(void* const* events, int i, cudaStream_t s) {
  if (events == nullptr) return MOE_OK;
  return cuda_status(record_event(static_cast<cudaEvent_t>(events[i]), s));
}

moe_status forward_impl(const moe_config* cfg, const void* x, const void* w_router,
                        const float* logit_bias, const void* w_gate, const void* w_up,
                        const void* w_down, const void* shared_gate, const void* shared_up,
                        const void* shared_down, void* y, int32_t* ids_out, float* gates_out,
                        int32_t* demand_out, int32_t* offsets_out, void* const* ev, int n_ev,
                        void* ws,
                        cudaStream_t stream) {
  MOE_TRY(validate(cfg));
  MOE_TRY(check_ws(ws));
  if (!x || !w_router || !w_gate || !w_up || !w_down || !y) return MOE_ERR_INVALID;
  if (cfg->has_shared && (!shared_gate || !shared_up || !shared_down)) return MOE_ERR_INVALID;
  const moe_config& c = *cfg;
  const Layout L = layout_of(c);
  int32_t* status = static_cast<int32_t*>(ws);
  int32_t* hist = reinterpret_cast<int32_t*>(at(ws, L.tile_hist));
  const RouterExtras extra{c.stats ? reinterpret_cast<float*>(at(ws, L.tile_psum)) : nullptr,
                           reroute(c) ? reinterpret_cast<float*>(at(ws, L.zkeys)) : nullptr};
  int32_t* ids = ids_out ? ids_out : reinterpret_cast<int32_t*>(at(ws, L.ids));
  float* gates = gates_out ? gates_out : reinterpret_cast<float*>(at(ws, L.gates));
  int32_t* demand = demand_out ? demand_out : reinterpret_cast<int32_t*>(at(ws, L.demand));
  int32_t* offsets = offsets_out ? offsets_out : reinterpret_cast<int32_t*>(at(ws, L.offsets));
  int32_t* route_row = reinterpret_cast<int32_t*>(at(ws, L.route_row));
  int32_t* row_token = reinterpret_cast<int32_t*>(at(ws, L.row_token));
  void* x_packed = at(ws, L.x_packed);
  void* h = at(ws, L.h);
  void* y_packed = at(ws, L.y_packed);

  // The router's last tile also turns the histogram into prefixes and writes the segment
  // table, so the pack reads finished positions.
  const DispatchPrep prep = make_dispatch_prep(
      c, hist, offsets, demand, reinterpret_cast<unsigned int*>(at(ws, kWsPrepCounterOffset)));
  // events: 0 start, then after route, pack, [reroute, with 7 events], gate/up, down, combine
  const int rr_ev = (n_ev == 7) ? 1 : 0;
  MOE_TRY(record(ev, 0, stream));
  MOE_TRY(cuda_status(
      launch_router(c, x, w_router, logit_bias, ids, gates, hist, extra, prep, status, stream)));
  MOE_TRY(record(ev, 1, stream));
  const bool fuse_gather = (c.fuse & MOE_FUSE_GATHER) != 0;
  const bool fuse_combine = (c.fuse & MOE_FUSE_COMBINE) != 0;
  int32_t* need = fuse_combine ? reinterpret_cast<int32_t*>(at(ws, L.need)) : nullptr;
  int32_t* counters = fuse_combine ? reinterpret_cast<int32_t*>(at(ws, L.counters)) : nullptr;
  const void* resid = c.add_residual ? x : nullptr;
  const PackFusion pf{fuse_gather ? 0 : 1, need, counters, resid, fuse_combine ? y : nullptr,
                      c.has_shared};
  MOE_TRY(cuda_status(launch_dispatch_pack(c, x, ids, hist, offsets, x_packed, row_token,
                                           route_row, status, stream,
                                           c.fuse != 0 ? &pf : nullptr)));
  if (rr_ev) MOE_TRY(record(ev, 2, stream));
  if (reroute(c))
    MOE_TRY(cuda_status(launch_reroute(c, x, ids, extra.zkeys, gates, x_packed, row_token,
                                       route_row, offsets,
                                       reinterpret_cast<int32_t*>(at(ws, L.rlist)), status,
                                       stream)));
  MOE_TRY(record(ev, 2 + rr_ev, stream));
  const FusedCombine fc{route_row, gates, row_token, need, counters, resid, y, c.k, c.has_shared};
  FfnArgs f{x, x_packed, offsets, w_gate, w_up, w_down, shared_gate, shared_up, shared_down,
            h, y_packed, L.rmax, status, padded(c) ? offsets + c.E + 2 : nullptr,
            fuse_gather ? row_token : nullptr, fuse_combine ? &fc : nullptr};
  MOE_TRY(ffn(c, f, stream, ev ? static_cast<cudaEvent_t>(ev[3 + rr_ev]) : nullptr));
  MOE_TRY(record(ev, 4 + rr_ev, stream));
  if (!fuse_combine)
    MOE_TRY(cuda_status(launch_combine(c, y_packed, route_row, gates, offsets, x, y, stream)));
  return record(ev, 5 + rr_ev, stream);
}

}  // namespace

extern "C" {

int32_t moe_abi_version(void) { return kAbiVersion; }

const char* moe_status_string(moe_status s) {
  switch (s) {
    case MOE_OK: return "ok";
    case MOE_ERR_INVALID: return "invalid argument";
    case MOE_ERR_UNSUPPORTED: return "unsupported configuration";
    case MOE_ERR_WORKSPACE: return "workspace missing or misaligned";
    case MOE_ERR_CUDA: return "CUDA error";
    case MOE_ERR_BAD_EXPERT_ID: return "expert id out of range or repeated within a token";
    case MOE_ERR_TIMEOUT: return "a bounded device wait ran out";
    case MOE_ERR_BAD_ADAPTER_ID: return "adapter id out of range";
  }
  return "unknown status";
}

int32_t moe_capacity(int32_t T, int32_t k, int32_t E, int32_t phi_num, int32_t phi_den) {
  if (T < 0 || k < 0 || E <= 0 || phi_num < 0 || phi_den <= 0) return -1;
  const int64_t num = static_cast<int64_t>(phi_num) * T * k;
  const int64_t den = static_cast<int64_t>(phi_den) * E;
  const int64_t c = (num + den - 1) / den;
  return c > INT32_MAX ? -1 : static_cast<int32_t>(c);
}

int32_t moe_ffn_tile_shape(const moe_config* cfg) {
  if (validate(cfg) != MOE_OK) return 0;
  return ffn_tile_shape(*cfg);
}

int32_t moe_ffn_launches(const moe_config* cfg) {
  if (validate(cfg) != MOE_OK) return 0;
  return ffn_launches(*cfg);
}

int64_t moe_max_rows(const moe_config* cfg) {
  if (validate(cfg) != MOE_OK) return 0;
  return max_rows(*cfg);
}

size_t moe_workspace_bytes(const moe_config* cfg) {
  if (validate(cfg) != MOE_OK) return 0;
  const size_t total = layout_of(*cfg).total;
  // moe_forward_few's part also for more tokens than it takes: with a capacity it can be the larger
  // one, and a workspace for the largest T serves the calls of fewer tokens.  And whatever the
  // options that it does not take: an option only adds bytes.
  moe_config few = *cfg;
  few.T = std::min(few.T, kFewTokens);
  few.stats = 0;
  few.layout = MOE_LAYOUT_RAGGED;
  few.overflow = MOE_OVERFLOW_DROP;
  few.fuse = MOE_FUSE_NONE;
  return few_layer_supported(few) ? std::max(total, few_layer_layout(few).total) : total;
}

moe_status moe_workspace_init(void* ws, moe_stream_t stream) {
  MOE_TRY(check_ws(ws));
  return cuda_status(cudaMemsetAsync(ws, 0, kWsHeaderBytes, stream));
}

moe_status moe_route(const moe_config* cfg, const void* x, const void* w_router,
                     const float* logit_bias, int32_t* ids, float* gates, void* ws,
                     moe_stream_t stream) {
  MOE_TRY(validate(cfg));
  MOE_TRY(check_ws(ws));
  if (!x || !w_router || !ids || !gates) return MOE_ERR_INVALID;
  const Layout L = layout_of(*cfg);
  const RouterExtras extra{cfg->stats ? reinterpret_cast<float*>(at(ws, L.tile_psum)) : nullptr,
                           reroute(*cfg) ? reinterpret_cast<float*>(at(ws, L.zkeys)) : nullptr};
  const DispatchPrep no_prep{};  // moe_dispatch recounts from the ids it is given
  return cuda_status(launch_router(*cfg, x, w_router, logit_bias, ids, gates,
                                   reinterpret_cast<int32_t*>(at(ws, L.tile_hist)), extra,
                                   no_prep, static_cast<int32_t*>(ws), stream));
}

moe_status moe_dispatch(const moe_config* cfg, const void* x, const int32_t* ids,
                        float* gates, void* x_packed, int32_t* row_token, int32_t* route_row,
                        int32_t* offsets, int32_t* demand, void* ws, moe_stream_t stream) {
  MOE_TRY(validate(cfg));
  MOE_TRY(check_ws(ws));
  if (!x || !ids || !x_packed || !row_token || !route_row || !offsets || !demand)
    return MOE_ERR_INVALID;
  if (reroute(*cfg) && !gates) return MOE_ERR_INVALID;
  const Layout L = layout_of(*cfg);
  int32_t* hist = reinterpret_cast<int32_t*>(at(ws, L.tile_hist));
  int32_t* status = static_cast<int32_t*>(ws);
  const DispatchPrep prep = make_dispatch_prep(
      *cfg, hist, offsets, demand, reinterpret_cast<unsigned int*>(at(ws, kWsPrepCounterOffset)));
  MOE_TRY(cuda_status(launch_dispatch_hist(*cfg, ids, prep, status, stream)));
  MOE_TRY(cuda_status(launch_dispatch_pack(*cfg, x, ids, hist, offsets, x_packed, row_token,
                                           route_row, status, stream)));
  if (!reroute(*cfg)) return MOE_OK;
  return cuda_status(launch_reroute(*cfg, x, ids, reinterpret_cast<const float*>(at(ws, L.zkeys)),
                                    gates, x_packed, row_token, route_row, offsets,
                                    reinterpret_cast<int32_t*>(at(ws, L.rlist)), status, stream));
}

moe_status moe_expert_ffn(const moe_config* cfg, const void* x, const void* x_packed,
                          const int32_t* offsets, const void* w_gate, const void* w_up,
                          const void* w_down, const void* shared_gate, const void* shared_up,
                          const void* shared_down, void* h, void* y_packed, void* ws,
                          moe_stream_t stream) {
  MOE_TRY(validate(cfg));
  MOE_TRY(check_ws(ws));
  if (!x_packed || !offsets || !w_gate || !w_up || !w_down || !h || !y_packed)
    return MOE_ERR_INVALID;
  if (cfg->has_shared && (!x || !shared_gate || !shared_up || !shared_down)) return MOE_ERR_INVALID;
  FfnArgs f{x, x_packed, offsets, w_gate, w_up, w_down, shared_gate, shared_up, shared_down,
            h, y_packed, max_rows(*cfg), static_cast<int32_t*>(ws),
            padded(*cfg) ? offsets + cfg->E + 2 : nullptr};
  return ffn(*cfg, f, stream);
}

moe_status moe_combine(const moe_config* cfg, const void* y_packed, const int32_t* route_row,
                       const float* gates, const int32_t* offsets, const void* residual,
                       void* y, moe_stream_t stream) {
  MOE_TRY(validate(cfg));
  if (!y_packed || !route_row || !gates || !y) return MOE_ERR_INVALID;
  if (cfg->has_shared && !offsets) return MOE_ERR_INVALID;
  if (cfg->add_residual && !residual) return MOE_ERR_INVALID;
  return cuda_status(launch_combine(*cfg, y_packed, route_row, gates, offsets, residual, y, stream));
}

moe_status moe_forward(const moe_config* cfg, const void* x, const void* w_router,
                       const float* logit_bias, const void* w_gate, const void* w_up,
                       const void* w_down, const void* shared_gate, const void* shared_up,
                       const void* shared_down, void* y, int32_t* ids_out, float* gates_out,
                       int32_t* demand_out, int32_t* offsets_out, void* ws,
                       moe_stream_t stream) {
  return forward_impl(cfg, x, w_router, logit_bias, w_gate, w_up, w_down, shared_gate, shared_up,
                      shared_down, y, ids_out, gates_out, demand_out, offsets_out, nullptr, 0,
                      ws, stream);
}

moe_status moe_forward_few(const moe_config* cfg, const void* x, const void* w_router,
                           const float* logit_bias, const void* w_gate, const void* w_up,
                           const void* w_down, const void* shared_gate, const void* shared_up,
                           const void* shared_down, void* y, int32_t* ids_out, float* gates_out,
                           int32_t* demand_out, int32_t* offsets_out, const int32_t* n_tokens,
                           void* ws, moe_stream_t stream) {
  MOE_TRY(validate(cfg));
  MOE_TRY(check_ws(ws));
  if (!few_layer_supported(*cfg)) return MOE_ERR_UNSUPPORTED;
  if (!x || !w_router || !w_gate || !w_up || !w_down || !y) return MOE_ERR_INVALID;
  if (cfg->has_shared && (!shared_gate || !shared_up || !shared_down)) return MOE_ERR_INVALID;
  if (!aligned16({x, w_router, w_gate, w_up, w_down, shared_gate, shared_up, shared_down}))
    return MOE_ERR_INVALID;
  const int64_t bytes = int64_t{1} * cfg->T * cfg->d * (cfg->dtype == MOE_BF16 ? 2 : 4);
  if (y != x && overlap(x, bytes, y, bytes)) return MOE_ERR_INVALID;
  const FewArgs a{x, w_router, logit_bias, w_gate, w_up, w_down, shared_gate, shared_up,
                  shared_down, y, ids_out, gates_out, demand_out, offsets_out, n_tokens};
  return cuda_status(launch_few_layer(*cfg, a, ws, stream));
}

size_t moe_adapter_workspace_bytes(const moe_adapter_config* cfg) {
  if (validate_adapter(cfg) != MOE_OK) return 0;
  return adapter_layout(*cfg).total;
}

moe_status moe_adapter_linear(const moe_adapter_config* cfg, const void* x, const void* w,
                              const void* a, const void* b, const float* scale,
                              const int32_t* adapter_ids, const void* addend, void* y,
                              const int32_t* n_tokens, void* ws, moe_stream_t stream) {
  return adapter_impl(cfg,
                      AdapterArgs{x, {w, nullptr}, {a, nullptr}, {b, nullptr}, scale,
                                  adapter_ids, addend, y, n_tokens, false},
                      ws, stream);
}

moe_status moe_adapter_gate_up(const moe_adapter_config* cfg, const void* x, const void* w_gate,
                               const void* w_up, const void* a_gate, const void* b_gate,
                               const void* a_up, const void* b_up, const float* scale,
                               const int32_t* adapter_ids, void* h, const int32_t* n_tokens,
                               void* ws, moe_stream_t stream) {
  return adapter_impl(cfg,
                      AdapterArgs{x, {w_gate, w_up}, {a_gate, a_up}, {b_gate, b_up}, scale,
                                  adapter_ids, nullptr, h, n_tokens, true},
                      ws, stream);
}

moe_status moe_forward_profiled(const moe_config* cfg, const void* x, const void* w_router,
                                const float* logit_bias, const void* w_gate, const void* w_up,
                                const void* w_down, const void* shared_gate,
                                const void* shared_up, const void* shared_down, void* y,
                                int32_t* ids_out, float* gates_out, int32_t* demand_out,
                                int32_t* offsets_out, void* const* events, int32_t n_events,
                                void* ws, moe_stream_t stream) {
  if (events == nullptr || (n_events != 6 && n_events != 7)) return MOE_ERR_INVALID;
  for (int i = 0; i < n_events; ++i)
    if (events[i] == nullptr) return MOE_ERR_INVALID;
  return forward_impl(cfg, x, w_router, logit_bias, w_gate, w_up, w_down, shared_gate, shared_up,
                      shared_down, y, ids_out, gates_out, demand_out, offsets_out, events,
                      n_events, ws, stream);
}

moe_status moe_routing_stats(const moe_config* cfg, const int32_t* demand,
                             const int32_t* offsets, float alpha, float* f, float* P,
                             moe_routing_summary* summary, void* ws, moe_stream_t stream) {
  MOE_TRY(validate(cfg));
  MOE_TRY(check_ws(ws));
  if (!cfg->stats || summary == nullptr || !std::isfinite(alpha)) return MOE_ERR_INVALID;
  const Layout L = layout_of(*cfg);
  const int32_t* dem = demand ? demand : reinterpret_cast<const int32_t*>(at(ws, L.demand));
  const int32_t* off = offsets ? offsets : reinterpret_cast<const int32_t*>(at(ws, L.offsets));
  return cuda_status(launch_routing_stats(
      *cfg, reinterpret_cast<const float*>(at(ws, L.tile_psum)), dem, off, alpha,
      reinterpret_cast<double*>(at(ws, L.stats_partial)),
      reinterpret_cast<unsigned int*>(at(ws, kWsStatsCounterOffset)), f, P, summary, stream));
}

moe_status moe_get_device_status(void* ws, moe_stream_t stream, int32_t clear,
                                 int32_t* status_out) {
  MOE_TRY(check_ws(ws));
  if (status_out == nullptr) return MOE_ERR_INVALID;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return MOE_ERR_CUDA;
  int32_t v = 0;
  if (cudaMemcpy(&v, ws, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess) return MOE_ERR_CUDA;
  // After a timeout the header's tickets and barrier counts may stand anywhere: all start again.
  // Whatever the word says: it keeps the first error, and a timeout may have followed another.
  // On `stream`, and complete on return: cleared on another stream, the counts could be zeroed under
  // the next launch, which would wait for arrivals that were erased.
  if (clear && v != MOE_OK) {
    if (cudaMemsetAsync(ws, 0, kWsHeaderBytes, stream) != cudaSuccess) return MOE_ERR_CUDA;
    if (cudaStreamSynchronize(stream) != cudaSuccess) return MOE_ERR_CUDA;
  }
  *status_out = v;
  return MOE_OK;
}

moe_status moe_debug_bounded_wait(void* ws, int64_t limit_ns, moe_stream_t stream) {
  MOE_TRY(check_ws(ws));
  if (limit_ns < 1000 || limit_ns > 10000000000LL) return MOE_ERR_INVALID;
  return cuda_status(launch_debug_wait(static_cast<int32_t*>(ws), limit_ns, stream));
}

}  // extern "C"
