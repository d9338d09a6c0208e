// Norm and rotation of query and key heads, forward and backward, and the
// append of new keys and values to a paged cache, which rotates on the way.
//
// A row x of d elements (one token, one head) becomes
//     y = R(p) (w * x r),   r = 1 / sqrt(mean(x^2) + eps),
// where R(p) turns each pair (a, b) of the first `rot` elements into
// (a c - b s, b c + a s), c and s read from tables at position p; without w
// the norm is left out. Backward, with g = R^T dy (the inverse turn; summed
// first over the repeats of a shared key head):
//     dw = sum over rows of g x r,   u = g w,
//     dx = r (u - x r^2 mean(u x)).
// r is computed again from x, which has to be read anyway, so the forward
// saves nothing. All arithmetic is fp32, each result is rounded once.
//
// Every row is read and written once, so the bound is the HBM bandwidth. A
// row is held by d / 16 lanes, two chunks of 8 elements each: for a rotated
// lane the two chunks that hold both ends of its pairs (half-split pairs lie
// rot / 2 apart), so the turn needs no exchange between lanes and the mean
// needs log2(d / 16) shuffles. A warp takes 32 / (d / 16) consecutive tokens
// and a chunk of heads: its lanes keep their tokens' c and s in registers for
// all of them, and the loads of several heads are in flight together.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "ops.h"
#include "ptx.cuh"

namespace skl {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
// Copies in flight per warp of the backward, repeats of a head (64 KB of shared
// memory a block, two blocks per SM).
template <int TYPE>
constexpr int kBwdStages = TYPE == kTypeF32 ? 2 : 4;

// 8 consecutive elements of a row: raw, as loaded with 16-byte loads.
template <int TYPE>
struct Raw8 {
  uint4 v[TYPE == kTypeF32 ? 2 : 1];
};

template <int TYPE>
struct ElemSize {
  static constexpr int value = TYPE == kTypeF32 ? 4 : 2;
};

template <int TYPE>
__device__ __forceinline__ Raw8<TYPE> load8(const void* p, long long elem) {
  Raw8<TYPE> r;
  const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + elem * ElemSize<TYPE>::value);
#pragma unroll
  for (int i = 0; i < (TYPE == kTypeF32 ? 2 : 1); ++i) r.v[i] = __ldg(q + i);
  return r;
}

template <int TYPE>
__device__ __forceinline__ void unpack8(const Raw8<TYPE>& r, float (&f)[8]) {
  if constexpr (TYPE == kTypeF32) {
    const float* s = reinterpret_cast<const float*>(r.v);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = s[i];
  } else if constexpr (TYPE == kTypeBf16) {
    const uint32_t* s = reinterpret_cast<const uint32_t*>(r.v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // bf16 is the upper half of an fp32
      f[2 * i] = __uint_as_float(s[i] << 16);
      f[2 * i + 1] = __uint_as_float(s[i] & 0xFFFF0000u);
    }
  } else {
    const __half2* s = reinterpret_cast<const __half2*>(r.v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = __half22float2(s[i]);
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
}

template <int TYPE>
__device__ __forceinline__ Raw8<TYPE> pack8(const float (&f)[8]) {
  Raw8<TYPE> r;
  if constexpr (TYPE == kTypeF32) {
    float* s = reinterpret_cast<float*>(r.v);
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = f[i];
  } else {
    uint32_t* s = reinterpret_cast<uint32_t*>(r.v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (TYPE == kTypeBf16) {
        s[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
      } else {
        const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        s[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
  }
  return r;
}

template <int TYPE>
__device__ __forceinline__ void store8(void* p, long long elem, const Raw8<TYPE>& r) {
  uint4* q = reinterpret_cast<uint4*>(static_cast<char*>(p) + elem * ElemSize<TYPE>::value);
#pragma unroll
  for (int i = 0; i < (TYPE == kTypeF32 ? 2 : 1); ++i) q[i] = r.v[i];
}

__device__ __forceinline__ void load_f8(const float* p, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
  f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

// The two chunks (of 8 elements) of lane l of a row: a lane below rot / 16
// holds chunks l and l + rot / 16, which are rotated; the others share out the
// d - rot elements that are not.
struct LaneChunks {
  int c0, c1;
  bool turned;
};
__device__ __forceinline__ LaneChunks lane_chunks(int l, int rot) {
  const int half = rot >> 4;
  LaneChunks c;
  c.turned = l < half;
  c.c0 = c.turned ? l : 2 * l;  // rot / 8 + 2 (l - rot / 16)
  c.c1 = c.turned ? l + half : c.c0 + 1;
  return c;
}

// cos and sin of a lane's 8 pairs at position pos.
template <bool INTER>
__device__ __forceinline__ void load_angles(const float* cs, const float* sn, int pos, int rot,
                                            const LaneChunks& lc, float (&c)[8], float (&s)[8]) {
  const long long row = static_cast<long long>(pos) * (rot >> 1);
  // half-split: pairs (c0[e], c1[e]), angle 8 c0 + e; interleaved: pairs
  // inside each chunk, angles 4 chunk + j
  const long long a0 = row + (INTER ? 4 * lc.c0 : 8 * lc.c0);
  const long long a1 = INTER ? row + 4 * lc.c1 : a0 + 4;
  const float4 c0 = __ldg(reinterpret_cast<const float4*>(cs + a0));
  const float4 c1 = __ldg(reinterpret_cast<const float4*>(cs + a1));
  const float4 s0 = __ldg(reinterpret_cast<const float4*>(sn + a0));
  const float4 s1 = __ldg(reinterpret_cast<const float4*>(sn + a1));
  c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w;
  c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
  s[0] = s0.x, s[1] = s0.y, s[2] = s0.z, s[3] = s0.w;
  s[4] = s1.x, s[5] = s1.y, s[6] = s1.z, s[7] = s1.w;
}

// Turn a lane's pairs by its angles (BACK: by minus its angles).
template <bool INTER, bool BACK>
__device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], const float (&c)[8],
                                     const float (&s)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float sn = BACK ? -s[e] : s[e];
    float& x = INTER ? (e < 4 ? a[2 * (e & 3)] : b[2 * (e & 3)]) : a[e];
    float& y = INTER ? (e < 4 ? a[2 * (e & 3) + 1] : b[2 * (e & 3) + 1]) : b[e];
    const float u = x * c[e] - y * sn, v = y * c[e] + x * sn;
    x = u;
    y = v;
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int m = 1; m < LPR; m <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
  return v;
}

__device__ __forceinline__ float sum_sq(const float (&a)[8], const float (&b)[8]) {
  float t = 0.f, u = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    t = fmaf(a[e], a[e], t);
    u = fmaf(b[e], b[e], u);
  }
  return t + u;
}

// 16 bytes, global to shared, in this thread's current copy group.
__device__ __forceinline__ void copy16(uint32_t dst, const char* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but this thread's N newest copy groups have landed.
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A lane's chunk in shared memory: 16-byte pieces 512 bytes (32 lanes) apart.
template <int TYPE>
__device__ __forceinline__ void copy8(uint32_t dst, const void* p, long long elem) {
  const char* src = static_cast<const char*>(p) + elem * ElemSize<TYPE>::value;
#pragma unroll
  for (int i = 0; i < ElemSize<TYPE>::value / 2; ++i) copy16(dst + 512 * i, src + 16 * i);
}
template <int TYPE>
__device__ __forceinline__ void read8(uint32_t src, float (&f)[8]) {
  Raw8<TYPE> r;
#pragma unroll
  for (int i = 0; i < ElemSize<TYPE>::value / 2; ++i) ld_shared_v4(src + 512 * i, r.v[i].x, r.v[i].y, r.v[i].z, r.v[i].w);
  unpack8<TYPE>(r, f);
}
template <int TYPE>
constexpr int kChunkBytes = 512 * (ElemSize<TYPE>::value / 2);  // of a warp

// A warp's items of a side, from `item` on in strides of the grid's warps: a
// batch's token tile and a range of heads.
struct Item {
  int b, n, h0, h1;
  bool there;  // this lane's token exists
};
__device__ __forceinline__ Item decode_item(const RopeArgs& a, const RopeSide& s, uint32_t item, int tokens,
                                            int grp) {
  Item t;
  const uint32_t tile = item / static_cast<uint32_t>(s.hchunks);
  t.b = static_cast<int>(tile / static_cast<uint32_t>(s.tiles));
  t.n = static_cast<int>(tile - static_cast<uint32_t>(t.b) * s.tiles) * tokens + grp;
  t.h0 = static_cast<int>(item - tile * s.hchunks) * a.hc;
  t.h1 = min(s.H, t.h0 + a.hc);
  t.there = item < s.items && t.n < s.N;
  return t;
}
__device__ __forceinline__ int position(const RopeSide& s, const Item& t) {
  return !t.there ? 0 : s.pos != nullptr ? __ldg(s.pos + t.b * s.pos_sb + t.n) : s.pos0 + t.n;
}

// Angles one item early, positions two.
template <int D, bool INTER>
struct Angles {
  float c[8], s[8];
  bool ok;    // the token exists, its position lies inside the tables
};
template <int D, bool INTER>
__device__ __forceinline__ void fetch_angles(const RopeArgs& a, const Item& t, int pos, const LaneChunks& lc,
                                             Angles<D, INTER>& g) {
  g.ok = t.there;
  if (g.ok && (pos < 0 || pos >= a.table_len)) {  // reported, its rows left unwritten
    atomicCAS(a.dev_status, 0, kStatusInvalidArg);
    g.ok = false;
  }
  if (lc.turned && g.ok) load_angles<INTER>(a.cos, a.sin, pos, a.rot, lc, g.c, g.s);
}

// Forward: one item per warp, four heads' loads in flight at a time. (Copies
// through shared memory as in the backward gain nothing here: 238 us against
// 239 at 65,521 tokens x 40 heads.)
template <int TYPE, int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 2)
    streamkl_rope_fwd_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int LPR = D / 16;          // lanes of a row
  constexpr int TOKENS = 32 / LPR;     // tokens of a warp
  constexpr int UNROLL = 4;            // heads whose loads are in flight together
  const int lane = threadIdx.x & 31, grp = lane / LPR, l = lane % LPR;
  uint32_t item = blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
  const int k = item >= a.side[0].items;
  if (k) item -= static_cast<uint32_t>(a.side[0].items);
  const RopeSide& s = a.side[k];
  if (item >= s.items) return;
  const LaneChunks lc = lane_chunks(l, a.rot);
  const Item t = decode_item(a, s, item, TOKENS, grp);
  Angles<D, INTER> g;
  fetch_angles(a, t, position(s, t), lc, g);
  float w0[8], w1[8];
  const bool norm = s.w != nullptr;
  if (norm) {
    load_f8(s.w + 8 * lc.c0, w0);
    load_f8(s.w + 8 * lc.c1, w1);
  }
  const long long x0 = t.b * s.xs.sb + t.n * s.xs.sn;
  const long long y0 = t.b * s.ys.sb + t.n * s.ys.sn;
  for (int h = t.h0; h < t.h1; h += UNROLL) {
    Raw8<TYPE> r0[UNROLL], r1[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
      if (g.ok && h + u < t.h1) {
        r0[u] = load8<TYPE>(s.x, x0 + (h + u) * s.xs.sh + 8 * lc.c0);
        r1[u] = load8<TYPE>(s.x, x0 + (h + u) * s.xs.sh + 8 * lc.c1);
      } else {
        r0[u] = r1[u] = Raw8<TYPE>{};
      }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if (h + u >= t.h1) break;  // (uniform in the warp)
      float f0[8], f1[8];
      unpack8<TYPE>(r0[u], f0);
      unpack8<TYPE>(r1[u], f1);
      if (norm) {
        const float r = rsqrtf(row_sum<LPR>(sum_sq(f0, f1)) * (1.f / D) + a.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          f0[e] *= r * w0[e];
          f1[e] *= r * w1[e];
        }
      }
      if (lc.turned) turn<INTER, false>(f0, f1, g.c, g.s);
      if (!g.ok) continue;
      const Raw8<TYPE> o0 = pack8<TYPE>(f0), o1 = pack8<TYPE>(f1);
      for (int q = 0; q < s.rep; ++q) {
        const long long y = y0 + (static_cast<long long>(h + u) * s.rep + q) * s.ys.sh;
        store8<TYPE>(s.y_out, y + 8 * lc.c0, o0);
        store8<TYPE>(s.y_out, y + 8 * lc.c1, o1);
      }
    }
  }
}

// Backward, a persistent grid: each warp takes items with a fixed stride and keeps its
// lanes' part of dw in registers, so the partials are one row per block and
// their order of summation is the same in every run.
template <int TYPE, int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 2)
    streamkl_rope_bwd_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int LPR = D / 16;
  constexpr int TOKENS = 32 / LPR;
  constexpr int STAGES = kBwdStages<TYPE>;
  constexpr int SLOT = 4 * kChunkBytes<TYPE>;  // one repeat of a head: two chunks of dy, two of x with the first
  extern __shared__ __align__(16) uint8_t stage_mem[];
  __shared__ float red[2][kRopeWarps][D];
  __shared__ float4 weights[2][D / 4];  // (read as such)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, grp = lane / LPR, l = lane % LPR;
  const uint32_t mem = smem_u32(stage_mem) + warp * STAGES * SLOT + lane * 16;
  const LaneChunks lc = lane_chunks(l, a.rot);
  const uint32_t stride = gridDim.x * kRopeWarps;
  if (threadIdx.x < 2 * D) {
    const float* w = a.side[threadIdx.x / D].w;
    if (w != nullptr) reinterpret_cast<float*>(weights[threadIdx.x / D])[threadIdx.x % D] = __ldg(w + threadIdx.x % D);
  }
  __syncthreads();
  // (no barrier from one side to the other: a warp that has no row of the first
  // goes on to the second)
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    const RopeSide& s = a.side[k];
    if (s.x == nullptr) continue;
    const bool norm = s.w != nullptr;
    const float4* ws = weights[k];
    float dw0[8], dw1[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dw0[e] = dw1[e] = 0.f;
    uint32_t item = blockIdx.x * kRopeWarps + warp;
    if (k == 1) item = (item + stride - static_cast<uint32_t>(a.side[0].items % stride)) % stride;
    if (item < s.items) {
      // copies: the repeat that comes next
      uint32_t p_item = item;
      Item p = decode_item(a, s, p_item, TOKENS, grp);
      int p_h = p.h0, p_q = 0, p_slot = 0;
      long long p_x, p_y;
      auto start = [&]() {
        p_x = p.b * s.xs.sb + p.n * s.xs.sn + p.h0 * s.xs.sh;
        p_y = p.b * s.ys.sb + p.n * s.ys.sn + static_cast<long long>(p.h0) * s.rep * s.ys.sh;
      };
      start();
      auto issue = [&]() {
        if (p_item < s.items) {
          if (p.there) {
            const uint32_t dst = mem + p_slot * SLOT;
            copy8<TYPE>(dst, s.y_in, p_y + 8 * lc.c0);
            copy8<TYPE>(dst + kChunkBytes<TYPE>, s.y_in, p_y + 8 * lc.c1);
            if (norm && p_q == 0) {
              copy8<TYPE>(dst + 2 * kChunkBytes<TYPE>, s.x, p_x + 8 * lc.c0);
              copy8<TYPE>(dst + 3 * kChunkBytes<TYPE>, s.x, p_x + 8 * lc.c1);
            }
          }
          p_y += s.ys.sh;
          if (++p_q == s.rep) {
            p_q = 0;
            p_x += s.xs.sh;
            if (++p_h == p.h1) {
              p_item += stride;
              p = decode_item(a, s, p_item, TOKENS, grp);
              p_h = p.h0;
              start();
            }
          }
        }
        p_slot = p_slot + 1 == STAGES ? 0 : p_slot + 1;
        copies_commit();
      };
      Item t = decode_item(a, s, item, TOKENS, grp), t1 = decode_item(a, s, item + stride, TOKENS, grp);
      const int pos0 = position(s, t);
      int pos1 = position(s, t1);
#pragma unroll
      for (int i = 0; i < STAGES - 1; ++i) issue();
      Angles<D, INTER> now, next;
      fetch_angles(a, t, pos0, lc, now);
      int slot = 0;
      for (; item < s.items; item += stride) {
        fetch_angles(a, t1, pos1, lc, next);
        const Item t2 = decode_item(a, s, item + 2 * stride, TOKENS, grp);
        pos1 = position(s, t2);
        long long dx = t.b * s.dxs.sb + t.n * s.dxs.sn + t.h0 * s.dxs.sh;
        for (int h = t.h0; h < t.h1; ++h, dx += s.dxs.sh) {
          copies_wait<STAGES - 2>();
          float g0[8], g1[8], f0[8], f1[8];
          read8<TYPE>(mem + slot * SLOT, g0);
          read8<TYPE>(mem + slot * SLOT + kChunkBytes<TYPE>, g1);
          if (norm) {
            read8<TYPE>(mem + slot * SLOT + 2 * kChunkBytes<TYPE>, f0);
            read8<TYPE>(mem + slot * SLOT + 3 * kChunkBytes<TYPE>, f1);
          }
          slot = slot + 1 == STAGES ? 0 : slot + 1;
          issue();
          for (int q = 1; q < s.rep; ++q) {
            copies_wait<STAGES - 2>();
            float e0[8], e1[8];
            read8<TYPE>(mem + slot * SLOT, e0);
            read8<TYPE>(mem + slot * SLOT + kChunkBytes<TYPE>, e1);
            slot = slot + 1 == STAGES ? 0 : slot + 1;
            issue();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              g0[e] += e0[e];
              g1[e] += e1[e];
            }
          }
          if (lc.turned) turn<INTER, true>(g0, g1, now.c, now.s);
          if (norm) {
            const float r = rsqrtf(row_sum<LPR>(sum_sq(f0, f1)) * (1.f / D) + a.eps);
            if (now.ok) {  // (a row that is absent holds anything)
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                dw0[e] = fmaf(g0[e] * r, f0[e], dw0[e]);
                dw1[e] = fmaf(g1[e] * r, f1[e], dw1[e]);
              }
            }
            float w0[8], w1[8];
            *reinterpret_cast<float4*>(&w0[0]) = ws[2 * lc.c0];
            *reinterpret_cast<float4*>(&w0[4]) = ws[2 * lc.c0 + 1];
            *reinterpret_cast<float4*>(&w1[0]) = ws[2 * lc.c1];
            *reinterpret_cast<float4*>(&w1[4]) = ws[2 * lc.c1 + 1];
            float dot = 0.f, dot1 = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              g0[e] *= w0[e];
              g1[e] *= w1[e];
              dot = fmaf(g0[e], f0[e], dot);
              dot1 = fmaf(g1[e], f1[e], dot1);
            }
            const float m = row_sum<LPR>(dot + dot1) * (1.f / D) * r * r;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              g0[e] = r * (g0[e] - f0[e] * m);
              g1[e] = r * (g1[e] - f1[e] * m);
            }
          }
          if (now.ok) {
            store8<TYPE>(s.dx, dx + 8 * lc.c0, pack8<TYPE>(g0));
            store8<TYPE>(s.dx, dx + 8 * lc.c1, pack8<TYPE>(g1));
          }
        }
        t = t1;
        t1 = t2;
        now = next;
      }
      copies_wait<0>();
    }
    if (!norm) continue;  // (uniform in the grid)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int m = LPR; m < 32; m <<= 1) {
        dw0[e] += __shfl_xor_sync(0xFFFFFFFFu, dw0[e], m);
        dw1[e] += __shfl_xor_sync(0xFFFFFFFFu, dw1[e], m);
      }
      if (grp == 0) {
        red[k][warp][8 * lc.c0 + e] = dw0[e];
        red[k][warp][8 * lc.c1 + e] = dw1[e];
      }
    }
  }
  __syncthreads();
  if (threadIdx.x < 2 * D) {
    const int k = threadIdx.x / D, c = threadIdx.x % D;
    if (a.side[k].x != nullptr && a.side[k].w != nullptr) {
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < kRopeWarps; ++i) t += red[k][i][c];
      a.part[(static_cast<long long>(k) * gridDim.x + blockIdx.x) * D + c] = t;
    }
  }
  grid_launch_dependents();  // the sum of the partials may be launched
}

// Sum the partials [2][blocks][D] over the blocks; a block takes 32 columns
// of one side (blockIdx.y), 32 rows at a time.
__global__ void __launch_bounds__(1024)
    streamkl_rope_dw_kernel(const float* __restrict__ part, int blocks, int D, float* dw_q, float* dw_k) {
  __shared__ float red[32][33];
  grid_dependency_wait();  // launched while the backward ends
  float* out = blockIdx.y ? dw_k : dw_q;
  if (out == nullptr) return;
  const int col = threadIdx.x & 31, row = threadIdx.x >> 5;
  const float* p = part + static_cast<long long>(blockIdx.y) * blocks * D + blockIdx.x * 32 + col;
  float t = 0.f;
  for (int i = row; i < blocks; i += 32) t += p[static_cast<long long>(i) * D];
  red[row][col] = t;
  __syncthreads();
  t = red[col][row];  // thread (row, col) now holds partial row `col` of column `row`
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, m);
  if (col == 0) out[blockIdx.x * 32 + row] = t;
}

// New keys (normed and rotated) and values into their pages. A warp takes
// consecutive tokens and a chunk of heads of K or of V, as above; each token
// finds its sequence by a binary search of the offsets.
template <int TYPE, int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 2)
    streamkl_paged_append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int LPR = D / 16;
  constexpr int TOKENS = 32 / LPR;
  constexpr int UNROLL = 4;
  const int lane = threadIdx.x & 31, grp = lane / LPR, l = lane % LPR;
  const long long item = static_cast<long long>(blockIdx.x) * kRopeWarps + (threadIdx.x >> 5);
  const int tile = static_cast<int>(item / (2 * a.hchunks));
  const int part = static_cast<int>(item - static_cast<long long>(tile) * 2 * a.hchunks);
  const bool is_v = part >= a.hchunks;
  const int h0 = (is_v ? part - a.hchunks : part) * a.hc, h1 = min(a.H, h0 + a.hc);
  const int t = tile * TOKENS + grp;
  const bool there = t < a.T;
  const void* src = is_v ? a.v : a.k;
  const RowStrides& st = is_v ? a.vs : a.ks;
  const LaneChunks lc = lane_chunks(l, a.rot);
  Raw8<TYPE> r0[UNROLL], r1[UNROLL];
  auto fetch = [&](int h) {
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
      if (there && h + u < h1) {
        r0[u] = load8<TYPE>(src, t * st.sn + (h + u) * st.sh + 8 * lc.c0);
        r1[u] = load8<TYPE>(src, t * st.sn + (h + u) * st.sh + 8 * lc.c1);
      } else {
        r0[u] = r1[u] = Raw8<TYPE>{};
      }
  };
  fetch(h0);  // beside the search for its place, a chain of loads
  bool ok = there;
  int pos = 0;
  long long place = 0, head = 0;  // element of head 0's slot, head stride
  if (ok) {
    int b = t, first = t, next = t + 1;
    if (a.cu != nullptr) {
      int lo = 0, hi = a.B;  // the last b with cu[b] <= t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.cu + mid) <= t)
          lo = mid;
        else
          hi = mid;
      }
      b = lo;
      first = __ldg(a.cu + b);
      next = __ldg(a.cu + b + 1);
    }
    ok = t >= first && t < next;  // false: a row behind the last sequence
    if (ok) {
      const int len = __ldg(a.kv_lens + b);
      pos = len - next + t;
      const int pg = pos >> a.page_shift;
      bool good = first >= 0 && next <= a.T && len >= next - first && pos >= 0 && pg < a.max_pages &&
                  (a.cos == nullptr || pos < a.table_len);
      int page = 0;
      if (good) {
        page = __ldg(a.table + b * a.table_sb + pg);
        good = page >= 0 && page < a.num_pages;
      }
      if (!good) atomicCAS(a.dev_status, 0, kStatusInvalidArg);
      ok = good;
      const long long slot = pos & ((1 << a.page_shift) - 1);
      place = page * (is_v ? a.vc_sp : a.kc_sp) + slot * (is_v ? a.vc_ss : a.kc_ss);
      head = is_v ? a.vc_sh : a.kc_sh;
    }
  }
  const bool norm = !is_v && a.w != nullptr;
  const bool turned = !is_v && lc.turned && a.cos != nullptr;
  float c[8], sn[8], w0[8], w1[8];
  if (turned && ok) load_angles<INTER>(a.cos, a.sin, pos, a.rot, lc, c, sn);
  if (norm) {
    load_f8(a.w + 8 * lc.c0, w0);
    load_f8(a.w + 8 * lc.c1, w1);
  }
  void* dst = is_v ? a.vc : a.kc;
  for (int h = h0; h < h1; h += UNROLL) {
    if (h > h0) fetch(h);
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if (h + u >= h1) break;
      if (norm || turned || (!is_v && a.cos != nullptr)) {
        float f0[8], f1[8];
        unpack8<TYPE>(r0[u], f0);
        unpack8<TYPE>(r1[u], f1);
        if (norm) {
          const float r = rsqrtf(row_sum<LPR>(sum_sq(f0, f1)) * (1.f / D) + a.eps);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            f0[e] *= r * w0[e];
            f1[e] *= r * w1[e];
          }
        }
        if (turned) turn<INTER, false>(f0, f1, c, sn);
        if (norm || turned) {
          r0[u] = pack8<TYPE>(f0);
          r1[u] = pack8<TYPE>(f1);
        }
      }
      if (ok) {
        store8<TYPE>(dst, place + (h + u) * head + 8 * lc.c0, r0[u]);
        store8<TYPE>(dst, place + (h + u) * head + 8 * lc.c1, r1[u]);
      }
    }
  }
}

// Heads per item. Where the warps that are resident together (two blocks an SM)
// can have one item each, as few heads as leave it at that (forward, 2,048 tokens
// x 20 heads 7.0 -> 5.5 us, 8,000 x 8 of 64 7.5 -> 4.3, append of 10,000 tokens x 8
// of 64 12.0 -> 9.8, against items of which a warp gets two or three). Else up to
// 16 (the forward at 65,521 tokens x 40 heads takes 238 us, 255 with 8 and 299
// with 4: the angles are loaded less often), fewer when there are not `per_sm`
// items an SM to even out the last round.
template <typename F>
int head_chunk(F&& items, long long tiles, int heads, int per_sm, int sms) {
  int hc = 1;
  for (; hc <= 16; ++hc)
    if (items(hc) <= 2LL * kRopeWarps * sms) return hc;
  for (hc = 16; hc > 1 && tiles * ((heads + hc - 1) / hc) < static_cast<long long>(per_sm) * sms;) hc >>= 1;
  return std::min(hc, heads);
}

long long side_items(RopeSide& s, int B, int d, int hc) {
  if (s.x == nullptr) {
    s.tiles = s.hchunks = 1;
    s.items = 0;
    return 0;
  }
  const int tokens = 32 / (d / 16);
  s.tiles = (s.N + tokens - 1) / tokens;
  s.hchunks = (s.H + hc - 1) / hc;
  s.items = static_cast<long long>(B) * s.tiles * s.hchunks;
  return s.items;
}

int rope_head_chunk(int B, int NQ, int HQ, int NK, int HK, int d, int sms) {
  const int tokens = 32 / (d / 16);
  const long long tq = static_cast<long long>(B) * ((NQ + tokens - 1) / tokens);
  const long long tk = static_cast<long long>(B) * ((NK + tokens - 1) / tokens);
  auto items = [&](int hc) { return tq * ((HQ + hc - 1) / hc) + tk * ((HK + hc - 1) / hc); };
  // (the backward at 8,192 tokens x 32 heads with 16 items an SM 53.9 us, with 32 51.6)
  return head_chunk(items, std::max(tq, tk), HQ + HK, 32, sms);
}

template <int TYPE, int D>
cudaError_t rope_fwd_t(const RopeArgs& a, unsigned blocks, cudaStream_t stream) {
  if (a.interleaved)
    streamkl_rope_fwd_kernel<TYPE, D, true><<<blocks, kRopeThreads, 0, stream>>>(a);
  else
    streamkl_rope_fwd_kernel<TYPE, D, false><<<blocks, kRopeThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int TYPE, int D>
cudaError_t rope_bwd_t(const RopeArgs& a, unsigned blocks, cudaStream_t stream) {
  constexpr int bytes = kRopeWarps * kBwdStages<TYPE> * 4 * kChunkBytes<TYPE>;
  auto kern = a.interleaved ? streamkl_rope_bwd_kernel<TYPE, D, true> : streamkl_rope_bwd_kernel<TYPE, D, false>;
  // the shared-memory attribute, once per device
  static std::atomic<unsigned long long> done[2];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (!(done[a.interleaved].load() & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    done[a.interleaved].fetch_or(bit);
  }
  kern<<<blocks, kRopeThreads, bytes, stream>>>(a);
  return cudaGetLastError();
}

template <int TYPE, int D>
cudaError_t append_t(const AppendArgs& a, unsigned blocks, cudaStream_t stream) {
  if (a.interleaved)
    streamkl_paged_append_kernel<TYPE, D, true><<<blocks, kRopeThreads, 0, stream>>>(a);
  else
    streamkl_paged_append_kernel<TYPE, D, false><<<blocks, kRopeThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

int rope_bwd_blocks(int B, int NQ, int HQ, int NK, int HK, int d, int sms) {
  const int tokens = 32 / (d / 16);
  const int hc = rope_head_chunk(B, NQ, HQ, NK, HK, d, sms);
  const long long iq = static_cast<long long>(B) * ((NQ + tokens - 1) / tokens) * ((HQ + hc - 1) / hc);
  const long long ik = static_cast<long long>(B) * ((NK + tokens - 1) / tokens) * ((HK + hc - 1) / hc);
  const long long want = (iq + ik + kRopeWarps - 1) / kRopeWarps;
  return static_cast<int>(std::max(1LL, std::min<long long>(want, 2LL * sms)));
}

cudaError_t launch_rope_fwd(RopeArgs& a, int sms, cudaStream_t stream) {
  const RopeSide &q = a.side[0], &k = a.side[1];
  a.hc = rope_head_chunk(a.B, q.x ? q.N : 0, q.x ? q.H : 0, k.x ? k.N : 0, k.x ? k.H : 0, a.d, sms);
  long long items = 0;
  for (RopeSide& s : a.side) items += side_items(s, a.B, a.d, a.hc);
  const unsigned blocks = static_cast<unsigned>((items + kRopeWarps - 1) / kRopeWarps);
  if (a.d == 128)
    return a.type == kTypeBf16  ? rope_fwd_t<kTypeBf16, 128>(a, blocks, stream)
           : a.type == kTypeF16 ? rope_fwd_t<kTypeF16, 128>(a, blocks, stream)
                                : rope_fwd_t<kTypeF32, 128>(a, blocks, stream);
  return a.type == kTypeBf16  ? rope_fwd_t<kTypeBf16, 64>(a, blocks, stream)
         : a.type == kTypeF16 ? rope_fwd_t<kTypeF16, 64>(a, blocks, stream)
                              : rope_fwd_t<kTypeF32, 64>(a, blocks, stream);
}

cudaError_t launch_rope_bwd(RopeArgs& a, int blocks, int sms, float* dw_q, float* dw_k, cudaStream_t stream) {
  const RopeSide &q = a.side[0], &k = a.side[1];
  a.hc = rope_head_chunk(a.B, q.x ? q.N : 0, q.x ? q.H : 0, k.x ? k.N : 0, k.x ? k.H : 0, a.d, sms);
  for (RopeSide& s : a.side) side_items(s, a.B, a.d, a.hc);
  const unsigned n = static_cast<unsigned>(blocks);
  cudaError_t e;
  if (a.d == 128)
    e = a.type == kTypeBf16  ? rope_bwd_t<kTypeBf16, 128>(a, n, stream)
        : a.type == kTypeF16 ? rope_bwd_t<kTypeF16, 128>(a, n, stream)
                             : rope_bwd_t<kTypeF32, 128>(a, n, stream);
  else
    e = a.type == kTypeBf16  ? rope_bwd_t<kTypeBf16, 64>(a, n, stream)
        : a.type == kTypeF16 ? rope_bwd_t<kTypeF16, 64>(a, n, stream)
                             : rope_bwd_t<kTypeF32, 64>(a, n, stream);
  if (e != cudaSuccess || (dw_q == nullptr && dw_k == nullptr)) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.d / 32, 2);
  cfg.blockDim = dim3(1024);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const float* part = a.part;
  return cudaLaunchKernelEx(&cfg, streamkl_rope_dw_kernel, part, blocks, a.d, dw_q, dw_k);
}

cudaError_t launch_append(AppendArgs& a, int sms, cudaStream_t stream) {
  const int tokens = 32 / (a.d / 16);
  const long long tiles = (a.T + tokens - 1) / tokens;
  auto items_of = [&](int hc) { return 2 * tiles * ((a.H + hc - 1) / hc); };
  a.hc = head_chunk(items_of, tiles, 2 * a.H, 16, sms);  // (with 32: 10,000 tokens x 8 heads 24.6 us, with 16 22.5)
  a.hc = std::min(a.hc, a.H);
  a.hchunks = (a.H + a.hc - 1) / a.hc;
  const long long items = tiles * 2 * a.hchunks;
  const unsigned blocks = static_cast<unsigned>((items + kRopeWarps - 1) / kRopeWarps);
  if (a.d == 128)
    return a.type == kTypeBf16 ? append_t<kTypeBf16, 128>(a, blocks, stream) : append_t<kTypeF16, 128>(a, blocks, stream);
  return a.type == kTypeBf16 ? append_t<kTypeBf16, 64>(a, blocks, stream) : append_t<kTypeF16, 64>(a, blocks, stream);
}

}  // namespace skl
