// What the two kernels of the attention over a paged cache share.
#pragma once

#include "ops.h"
#include "ptx.cuh"

namespace skl {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kTileN = 128;  // keys per tile
// The softmax's reference of a row (log2 units) moves when a term would exceed
// 2^kTau of it, or a tile's sum of terms 2^kTau = kSumMax.
constexpr float kTau = 8.0f;
constexpr float kSumMax = 256.0f;

// A place in the ring of K and V stages and the parity of its turn.
struct RingPos {
  int stage;
  uint32_t phase;
  __device__ __forceinline__ void step(int stages) {
    if (++stage == stages) {
      stage = 0;
      phase ^= 1;
    }
  }
};

// A bounded wait of a whole warp: false for all lanes where any gave up, so
// that the warp stays together for its .aligned instructions.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const WaitCtx& wc) {
  return __all_sync(0xFFFFFFFFu, wait_bounded(bar, parity, wc));
}

// Two values rounded to the inputs' 16-bit type.
template <int TYPE>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return TYPE == kTypeBf16 ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
}

}  // namespace skl
