// What the two kernels of the attention over a paged cache share.
#pragma once

#include "ops.h"
#include "ptx.cuh"

namespace skl {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kTileN = 128;  // keys per tile
// The softmax's reference of a row (log2 units) is taken kBelow under the row's
// maximum and moves when a term would exceed 2^kTau of it, or a tile's sum of
// terms 2^kTau = kSumMax. bf16 has fp32's range, so its largest term may be 1.
// In fp16 terms below 2^-14 lose bits and those below 2^-25 are gone, while the
// fp32 sum keeps them: with 1 for the largest, 131,072 keys 17.7 nats below one
// lost 0.3 % of max |v|. At 2^6 a term loses at most 2^-31 of the largest
// (2^-14 over 131,072 keys, an eighth of the output's own half step), and the
// largest of all, 2^14, stays two binary places under fp16's end.
template <int TYPE>
constexpr float kBelow = TYPE == kTypeF16 ? 6.0f : 0.0f;
template <int TYPE>
constexpr float kTau = 8.0f + kBelow<TYPE>;
template <int TYPE>
constexpr float kSumMax = TYPE == kTypeF16 ? 16384.0f : 256.0f;

// How far over a row's reference a tile's maximum may be. From 2^24 on (log2
// units) the maximum and the reference are themselves rounded by 1 and more, and
// fp16 ends at 2^16: there less is allowed, from 2^26 on nothing, so that terms
// stay finite up to maxima of 2^28.
template <int TYPE>
__device__ __forceinline__ float rise_allowed(float top) {
  return TYPE == kTypeF16 ? fmaxf(0.0f, fmaf(fabsf(top), -0x1p-22f, kTau<TYPE>)) : kTau<TYPE>;
}

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
