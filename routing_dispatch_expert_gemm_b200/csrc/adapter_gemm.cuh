// Pieces shared by the two tcgen05 kernels of the adapter projections (adapter_sm100.cu,
// adapter_pair_sm100.cu).
#pragma once

#include "common.cuh"
#include "internal.h"

namespace moe {

constexpr int kPairBlockTokens = 256;  // tokens of a token block over SM pairs, the largest
// A token block's adapters go through extra K blocks if they have this many tokens each on average,
// or fit into this many K blocks of 8 units (8 ranks, high or low half); else the epilogue expands
// them.  A K block costs up to 1.5 us to fill; the last tokens of a prompt, expanded, cost T=4099
// 28 us.
constexpr int kAdapterTokens = 16, kSmallBlocks = 4;
constexpr int kMaxBlockAdapters = 16;  // that the rule admits
static_assert(kPairBlockTokens / kAdapterTokens <= kMaxBlockAdapters &&
                  kSmallBlocks * 8 / 2 <= kMaxBlockAdapters,
              "an adapter has two units at least");
constexpr int kExtThreads = 64;  // threads that fill those K blocks

__device__ __forceinline__ int live_tokens(const int32_t* n_tokens, int T) {
  return n_tokens != nullptr ? min(max(__ldg(n_tokens), 0), T) : T;
}

// Whether u of token t, whose adapter is `id`, is not finite for one of M projections.
template <int M>
__device__ __forceinline__ bool broken_token(const uint8_t* broken, int T, int t, int id) {
  uint32_t b = __ldcg(broken + t);
  if (M == 2) b |= __ldcg(broken + T + t);
  return id >= 0 && b != 0;
}
// Barrier of the ext warps; whether `v` held on all of their threads.
__device__ __forceinline__ bool ext_all(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 2, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v)), "n"(kExtThreads)
      : "memory");
  return r != 0;
}
// Zeros the infinities and NaNs among 8 bf16 of shared memory; whether there were any.
__device__ __forceinline__ bool zero_nonfinite(uint8_t* p) {
  uint4 v = *reinterpret_cast<const uint4*>(p);
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((w[i] & 0x7f800000u) == 0x7f800000u) { w[i] &= 0x0000ffffu; any = true; }
    if ((w[i] & 0x7f80u) == 0x7f80u) { w[i] &= 0xffff0000u; any = true; }
  }
  if (any) *reinterpret_cast<uint4*>(p) = v;
  return any;
}

// The GEMM over SM pairs: kPairBlockTokens tokens per token block.  u and blocks come from the shrink kernel.
bool adapter_pair_fits(const moe_adapter_config& c, bool pair);
cudaError_t launch_adapter_pair(const moe_adapter_config& c, const AdapterArgs& a, const uint4* u,
                                const int32_t* blocks, const uint8_t* broken, int32_t* status,
                                cudaStream_t s);

}  // namespace moe
