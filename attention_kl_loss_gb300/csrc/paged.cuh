// What the kernels of the attention over a paged cache share.
#pragma once

#include "ops.h"
#include "ptx.cuh"

namespace skl {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kTileN = 128;  // keys per tile
constexpr int kMostCluster = 16;  // CTAs that share an item and join their parts
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

// The rows of a sequence without keys, by threads first, first + step, ..
template <int D>
__device__ __forceinline__ void empty_rows(const PagedAttnArgs& a, int tok0, int n, int first, int step) {
  for (long long e = first; e < static_cast<long long>(n) * a.HQ * (D / 8); e += step) {
    const int r = static_cast<int>(e / (D / 8)), i = static_cast<int>(e % (D / 8));
    const int token = tok0 + r / a.HQ, head = r % a.HQ;
    reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + token * a.o_sn + head * a.o_sh)[i] = make_uint4(0, 0, 0, 0);
    if (i == 0) a.lse[static_cast<long long>(token) * a.HQ + head] = -INFINITY;
  }
}

// Rows of an item whose parts lie in the shared memory of a cluster's CTAs, joined by
// their lse: O in fp32 [part_rows][D] from `part` on, a row's 16-byte pieces turned by
// its number (^ row & 7), then the rows' lse in log2 units. Warp `at` of `warps` takes
// kMostCluster / MOST rows at once (a lane D / 32 columns of each), of at most MOST parts.
template <int TYPE, int D, int MOST>
__device__ __forceinline__ void join_cluster(const PagedAttnArgs& a, uint32_t part, int part_rows, int parts, int at, int warps,
                                             int rows, int row0, int tok0, int hk) {
  constexpr int V = D / 32, ROWS = kMostCluster / MOST;
  const int lane = threadIdx.x & 31, G = a.HQ / a.HK;
  for (int r0 = at * ROWS; r0 < rows; r0 += warps * ROWS) {
    const int my_row = r0 + lane / MOST, my_part = lane % MOST;
    float lse = -INFINITY;
    if (lane < ROWS * MOST && my_row < rows && my_part < parts)
      lse = ld_cluster_f32(mapa_shared(part + (part_rows * D + my_row) * 4, my_part));
    float p[ROWS][MOST][V];
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
      const int r = r0 + u;
      const uint32_t mine = part + (r * (D / 4) + ((lane * V / 4) ^ (r & 7))) * 16 + lane * V % 4 * 4;
#pragma unroll
      for (int i = 0; i < MOST; ++i) {
#pragma unroll
        for (int x = 0; x < V; ++x) p[u][i][x] = 0.f;
        if (r < rows && i < parts) ld_cluster_f32(mapa_shared(mine, i), p[u][i]);
      }
    }
    float top = lse;
#pragma unroll
    for (int m = MOST / 2; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
    const float weight = ex2(lse - (top == -INFINITY ? 0.f : top));  // 0 past the last part
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
      float sum = 0.f, o[V] = {};
#pragma unroll
      for (int i = 0; i < MOST; ++i) {
        const float w = __shfl_sync(0xFFFFFFFFu, weight, u * MOST + i);
        sum += w;
#pragma unroll
        for (int x = 0; x < V; ++x) o[x] = fmaf(w, p[u][i][x], o[x]);
      }
      const float most = __shfl_sync(0xFFFFFFFFu, top, u * MOST);
      if (r0 + u >= rows) break;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const int row = row0 + r0 + u, tok = row / G, token = tok0 + tok, head = hk * G + row - tok * G;
      uint32_t* dst =
          reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + token * a.o_sn + head * a.o_sh + lane * V);
#pragma unroll
      for (int x = 0; x < V / 2; ++x) dst[x] = pack2<TYPE>(o[2 * x] * inv, o[2 * x + 1] * inv);
      if (lane == 0)
        a.lse[static_cast<long long>(token) * a.HQ + head] = sum == 0.f ? -INFINITY : (most + log2f(sum)) * kLn2;
    }
  }
}

// The keys of a tile that a row sees: the first `seen`, or with TREE those whose
// bit is set (`all`: every one of them).
template <bool TREE, int WORDS = kTileN / 32>
struct TileMask;
template <>
struct TileMask<false> {
  int seen;
  __device__ __forceinline__ TileMask(const PagedAttnArgs&, bool, int, int, int, int lim, int key0) : seen(lim - key0) {}
  __device__ __forceinline__ bool partial() const { return seen < kTileN; }
  __device__ __forceinline__ bool some() const { return seen > 0; }
  __device__ __forceinline__ bool hides(int k) const { return k >= seen; }
};
template <int WORDS>  // of 32 keys, from key0 on
struct TileMask<true, WORDS> {
  uint32_t bits[WORDS];
  bool all;  // (the same in all rows that are there)
  // Bit k of word q: key key0 + 32 q + k, which is drafted token t + k of the
  // sequence's n. Tokens before the drafted ones (t + k < 0) are seen by every row,
  // those from n on (past the sequence's end) by none.
  __device__ __forceinline__ TileMask(const TreeAttnArgs& a, bool live, int token, int n, int len, int, int key0) {
    const int t = key0 - (len - n);
    all = live && t + 32 * WORDS <= 0;
    if (t + 32 * WORDS <= 0) {
#pragma unroll
      for (int q = 0; q < WORDS; ++q) bits[q] = live ? ~0u : 0u;
      return;
    }
    const int* row = a.mask + token * a.mask_sn;
    const int first = t >> 5;  // (t may be negative)
    uint32_t w[WORDS + 1];
#pragma unroll
    for (int x = 0; x < WORDS + 1; ++x) {
      const int i = first + x, left = n - 32 * i;
      w[x] = i >= 0 && i < a.mask_words && left > 0 && live ? static_cast<uint32_t>(__ldg(row + i)) : i < 0 && live ? ~0u : 0u;
    }
#pragma unroll
    for (int x = 0; x < WORDS + 1; ++x) {
      const int left = n - 32 * (first + x);
      if (left < 32) w[x] &= left > 0 ? (1u << left) - 1 : 0u;
    }
#pragma unroll
    for (int q = 0; q < WORDS; ++q) bits[q] = __funnelshift_r(w[q], w[q + 1], t & 31);
  }
  __device__ __forceinline__ bool partial() const { return !all; }
  __device__ __forceinline__ bool some() const {
    uint32_t any = 0;
#pragma unroll
    for (int q = 0; q < WORDS; ++q) any |= bits[q];
    return any != 0;
  }
  __device__ __forceinline__ bool hides(int k) const { return !(bits[k >> 5] >> (k & 31) & 1); }
};

}  // namespace skl
