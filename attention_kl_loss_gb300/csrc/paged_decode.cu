// Attention over a paged cache for few rows: at most 32 (token, head of the
// group) rows per sequence and key head, as with one new token a sequence.
// The formulas are paged_attn.cu's; here reading the keys and values once is
// the whole cost, so the kernel is built to keep the loads running:
//   - A persistent grid of two CTAs per SM. The key tiles (128 keys) of all
//     (sequence, key head) items, in order, are one line of W tiles; each CTA
//     takes an equal stretch of it, whatever the sequences' lengths. A stretch
//     cuts at most its first and its last item; a combine kernel joins those
//     parts by their lse, whole items are written directly. Where sequences are
//     short each CTA takes whole items instead, and there is nothing to join.
//   - A CTA's loads run on through its items: Q of the next item is fetched by
//     a warp of its own while the current one is worked on, and the ring of K
//     and V stages never empties between items. Two CTAs per SM cover each
//     other's chain S -> P -> O (about 2,400 cycles a tile; an SM's share of
//     the HBM bandwidth brings a tile of K and V at d = 128 in 2,700).
//   - Only 32 rows of Q are kept (4 KB per 64 columns): the MMA reads 128 rows,
//     the ones past the 32nd from whatever lies behind, and its result rows
//     past the 32nd are never looked at.
// 64 sequences of 4,096 to 16,384 keys, 32 heads over 8 key heads of 128: 0.39 ms
// for 2.6 GB, 6.7 TB/s (one CTA per (sequence, key head) and key split: 0.54 ms).
// CTA: warp 0 softmax and output (thread = row, TMEM lanes 0..31), warp 1 loads
// of K and V, warp 2 MMAs, warp 3 Q and the items' numbers.
#include <algorithm>
#include <atomic>

#include "ops.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace skl {

namespace {

constexpr int kRows = kDecodeRows;
constexpr int kThreads = 128;

template <int D>
struct DecodeLayout {
  static constexpr int KB = D / 64;
  static constexpr int BOX = kTileN * 128;
  static constexpr int TILE = kTileN * D * 2;
  static constexpr int QBOX = kRows * 128;
  static constexpr int QBUF = KB * QBOX;
  static constexpr int STAGES = D == 128 ? 3 : 6;
  // Q (two buffers) lies before the ring: the MMA reads 128 rows from the start
  // of a 32-row box, the rest of them out of the boxes and stages behind it
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = 2 * QBUF;
  static_assert(OFF_KV % 1024 == 0 && STAGES * TILE >= kTileN * 128, "swizzle atoms; the rows read past Q exist");
  // kv_full[S], kv_empty[S], q_full[2], q_empty[2], s_full, p_full, o_full, drain
  static constexpr int NBAR = 2 * STAGES + 8;
  static constexpr int OFF_BAR = OFF_KV + STAGES * TILE;
  static constexpr int OFF_SEG = OFF_BAR + NBAR * 8;  // two items' numbers
  static constexpr int OFF_MISC = OFF_SEG + 2 * 32;
  static constexpr int BYTES = OFF_MISC + 64;
  static_assert(2 * (BYTES + 1024) <= 233472, "two CTAs per SM");
};

// One CTA's part of an item: tiles [t0, t0 + n_iter) of the keys of (b, hk).
struct Segment {
  int b, hk, t0, n_iter;
  int tok0, n, len;
  int slot;  // partial slot, or -1: the whole item
};

// A CTA's stretch of the line of tiles, from its next tile on; with whole items,
// its next one of them.
struct Stretch {
  int b, hk, tile;
  int left;  // tiles
  int item;
};

struct Seq {
  int tok0, n, len, tiles;
  bool ok;
};

__device__ __forceinline__ Seq load_seq(const PagedAttnArgs& a, int b) {
  Seq s;
  const int c0 = a.cu != nullptr ? __ldg(a.cu + b) : b;
  const int c1 = a.cu != nullptr ? __ldg(a.cu + b + 1) : b + 1;
  s.len = __ldg(a.kv_lens + b);
  s.tok0 = c0;
  s.n = c1 - c0;
  s.ok = c0 >= 0 && c1 >= c0 && c1 <= a.T && s.n <= a.max_q && s.len >= 0 && s.len <= a.max_kv;
  if (!s.ok) s.n = 0;
  // (the last row sees every key, so no tile is without work)
  s.tiles = s.n > 0 ? (s.len + kTileN - 1) / kTileN : 0;
  return s;
}

// The whole block finds its way in the line of tiles: each thread sums a run of
// consecutive sequences, a scan adds them up. The thread in whose run tile
// place(chunk) lies writes where that is to *at (left alone past the line's
// end). Returns the tiles of a CTA's stretch. Two barriers; *at is there after
// the next one.
struct Place {
  int b, hk, tile;
};
template <typename F, typename V>
__device__ __forceinline__ int locate(const PagedAttnArgs& a, int ctas, long long* scratch, volatile Place* at,
                                      long long* total, F&& place, V&& visit) {
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(a.B, static_cast<int>(threadIdx.x) * per), b1 = min(a.B, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const Seq s = load_seq(a, b);
    mine += s.tiles;
    visit(b, s);
  }
  mine *= a.HK;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long upto = mine;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long up = __shfl_up_sync(0xFFFFFFFFu, upto, m);
    if (lane >= m) upto += up;
  }
  if (lane == 31) scratch[warp] = upto;
  __syncthreads();
  long long base = 0, sum = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) base += scratch[i];
    sum += scratch[i];
  }
  const int chunk = static_cast<int>(max((sum + ctas - 1) / ctas, static_cast<long long>(a.split_tiles)));
  const long long x = place(chunk);
  long long first = base + upto - mine;
  if (first <= x && x < first + mine)
    for (int b = b0; b < b1; ++b) {
      const long long tiles = load_seq(a, b).tiles;
      if (first <= x && x < first + tiles * a.HK) {
        at->b = b;
        at->hk = static_cast<int>((x - first) / tiles);
        at->tile = static_cast<int>((x - first) % tiles);
      }
      first += tiles * a.HK;
    }
  *total = sum;
  return chunk;
}

// The next part of a CTA's stretch; false at its end.
__device__ __forceinline__ bool next_segment(const PagedAttnArgs& a, Stretch& st, Segment& sg, bool first) {
  if (st.left <= 0) return false;
  if (a.whole) {
    for (; st.item < a.B * a.HK; st.item += gridDim.x) {
      const int b = st.item / a.HK;
      const Seq s = load_seq(a, b);
      if (s.tiles == 0) continue;
      sg = {b, st.item - b * a.HK, 0, s.tiles, s.tok0, s.n, s.len, -1};
      st.item += gridDim.x;
      return true;
    }
    return false;
  }
  Seq s = load_seq(a, st.b);
  while (s.tiles == 0) {  // (b < B: tiles are left)
    ++st.b;
    s = load_seq(a, st.b);
  }
  sg.b = st.b;
  sg.hk = st.hk;
  sg.t0 = st.tile;
  sg.n_iter = min(st.left, s.tiles - st.tile);
  sg.tok0 = s.tok0;
  sg.n = s.n;
  sg.len = s.len;
  sg.slot = sg.n_iter == s.tiles ? -1 : 2 * static_cast<int>(blockIdx.x) + (first ? 0 : 1);
  st.left -= sg.n_iter;
  st.tile += sg.n_iter;
  if (st.tile == s.tiles) {
    st.tile = 0;
    if (++st.hk == a.HK) {
      st.hk = 0;
      ++st.b;
    }
  }
  return true;
}

template <int TYPE, int D>
__global__ void __launch_bounds__(kThreads, 2)
    streamkl_paged_decode_kernel(const __grid_constant__ CUtensorMap tm_k,
                                 const __grid_constant__ CUtensorMap tm_v,
                                 const __grid_constant__ PagedAttnArgs a) {
  using L = DecodeLayout<D>;
  extern __shared__ __align__(1024) uint8_t gb[];
  const uint32_t sb = smem_u32(gb);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.HQ / a.HK;
  const uint32_t bar0 = sb + L::OFF_BAR;
  auto kv_full = [&](int s) { return bar0 + 8u * s; };
  auto kv_empty = [&](int s) { return bar0 + 8u * (L::STAGES + s); };
  auto q_full = [&](int k) { return bar0 + 8u * (2 * L::STAGES + k); };
  auto q_empty = [&](int k) { return bar0 + 8u * (2 * L::STAGES + 2 + k); };
  const uint32_t s_full = bar0 + 8u * (2 * L::STAGES + 4), p_full = s_full + 8, o_full = s_full + 16,
                 drain = s_full + 24;
  static_assert(2 * L::STAGES + 8 == L::NBAR, "barrier region holds every barrier");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gb + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gb + L::OFF_MISC + 4);
  volatile int* skip_flag = reinterpret_cast<volatile int*>(gb + L::OFF_MISC + 8);
  long long* scratch = reinterpret_cast<long long*>(gb + L::OFF_MISC + 16);
  volatile Segment* segs = reinterpret_cast<volatile Segment*>(gb + L::OFF_SEG);
  volatile Place* start = reinterpret_cast<volatile Place*>(gb + L::OFF_SEG);  // (before the items)

  CheckCtx ck{sb, sb + L::OFF_BAR, sb + L::OFF_BAR, sb + L::OFF_BAR + L::NBAR * 8, 0, 0,
              abort_flag, a.dev_status};
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    bool lay_ok = (sb & 1023u) == 0;  // the swizzled tiles' alignment
    if (!lay_ok) atomicCAS(a.dev_status, 0, kStatusDeviceCheck);
    if (kDeviceChecks)
      for (int i = 0; i < L::NBAR; ++i) lay_ok = lay_ok && check_bar(ck, bar0 + 8u * i, __LINE__);
    if (lay_ok) {
      for (int s = 0; s < L::STAGES; ++s) {
        mbar_init(kv_full(s), 1);
        mbar_init(kv_empty(s), 1);
      }
      for (int k = 0; k < 2; ++k) {
        mbar_init(q_full(k), 1);
        mbar_init(q_empty(k), 1);
      }
      mbar_init(s_full, 1);
      mbar_init(p_full, 1);
      mbar_init(o_full, 1);
      mbar_init(drain, 1);
    }
    // a failure recorded earlier, or a failed layout check, skips the work; not a
    // bad number of some sequence, which may come from this very call
    const int before = *reinterpret_cast<volatile int*>(a.dev_status);
    *skip_flag = !lay_ok || (before != 0 && before != kStatusInvalidArg);
    fence_mbar_init();
  }
  if (warp == 1 && lane == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(tmem_slot), 256);
    tmem_relinquish();
  }
  // a sequence's numbers; its rows, where it has no key
  auto visit = [&](int b, const Seq& s, bool report, bool mine) {
    if (report && !s.ok) atomicCAS(a.dev_status, 0, kStatusInvalidArg);
    if (s.n == 0 || s.tiles > 0 || !mine) return;
    for (int r = 0; r < s.n * a.HQ; ++r) {
      const int token = s.tok0 + r / a.HQ, head = r % a.HQ;
      uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + token * a.o_sn + head * a.o_sh);
      for (int i = 0; i < D / 8; ++i) o[i] = make_uint4(0, 0, 0, 0);
      a.lse[static_cast<long long>(token) * a.HQ + head] = -INFINITY;
    }
  };
  Stretch st;
  if (a.whole) {  // every gridDim-th item
    st.item = static_cast<int>(blockIdx.x);
    st.left = 1;
    for (int i = st.item + static_cast<int>(threadIdx.x) * gridDim.x; i < a.B * a.HK; i += kThreads * gridDim.x)
      if (i % a.HK == 0) visit(i / a.HK, load_seq(a, i / a.HK), true, true);
  } else {  // this CTA's stretch of the line of tiles
    long long total;
    const int chunk = locate(
        a, gridDim.x, scratch, start, &total, [&](int per_cta) { return static_cast<long long>(blockIdx.x) * per_cta; },
        [&](int b, const Seq& s) { visit(b, s, blockIdx.x == 0, b % gridDim.x == blockIdx.x); });
    st.left = static_cast<int>(
        max(0LL, min(total - static_cast<long long>(blockIdx.x) * chunk, static_cast<long long>(chunk))));
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);  // (the same in every lane)
  if (!a.whole) {
    st.b = start->b;
    st.hk = start->hk;
    st.tile = start->tile;
  }
  if (*skip_flag) st.left = 0;
  __syncthreads();  // (the items are written there from here on)
  ck.tmem = tmem;
  ck.tmem_cols = 256;
  const WaitCtx wc{abort_flag, a.dev_status, a.timeout_ns};
  constexpr int COL_O = 128;  // S, and P over it, in [0, 128)

  if (warp == 3) {
    // ------------------------------------------------------------ Q, items
    Segment sg;
    bool first = true;
    for (int i = 0;; ++i) {
      const bool more = next_segment(a, st, sg, first);
      first = false;
      const int k = i & 1;
      if (!warp_wait(q_empty(k), ((i >> 1) & 1) ^ 1, wc)) break;
      if (lane == 0) {
        segs[k].b = sg.b;
        segs[k].hk = sg.hk;
        segs[k].t0 = sg.t0;
        segs[k].n_iter = more ? sg.n_iter : 0;
        segs[k].tok0 = sg.tok0;
        segs[k].n = sg.n;
        segs[k].len = sg.len;
        segs[k].slot = sg.slot;
      }
      if (more) {
        // rows as TMA would place them (128-byte swizzle); 16 bytes a lane
        const int rows = sg.n * G;
        const uint32_t dst = sb + L::OFF_Q + k * L::QBUF;
        for (int e = lane; e < rows * (D / 8); e += 32) {
          const int r = e / (D / 8), c = e % (D / 8);
          const int tok = r / G;
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                               (sg.tok0 + tok) * a.q_sn +
                                                               (sg.hk * G + r - tok * G) * a.q_sh) + c);
          st_shared_v4(dst + (c >> 3) * L::QBOX + r * 128 + (((c & 7) ^ (r & 7)) << 4), v.x, v.y, v.z, v.w);
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full(k));
      if (!more) break;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ K, V
    const int page = 1 << a.page_shift;
    const int box_rows = min(page, kTileN);
    Segment sg;
    RingPos ring{0, 0};
    bool ok = true, first = true;
    int issued = 0;
    while (ok && next_segment(a, st, sg, first)) {
      first = false;
      const int* table = a.table + static_cast<long long>(sg.b) * a.table_sb;
      // the page this lane loads of tile j; a number that is none is reported
      // and page 0 read in its place
      auto page_of = [&](int j) {
        const int key = (sg.t0 + j) * kTileN + lane * box_rows;
        if (j >= sg.n_iter || lane * box_rows >= kTileN || key >= sg.len) return -1;
        int p = __ldg(table + (key >> a.page_shift));
        if (p < 0 || p >= a.num_pages) {
          atomicCAS(a.dev_status, 0, kStatusInvalidArg);
          p = 0;
        }
        return p;
      };
      auto load = [&](const CUtensorMap* map, int j, int pg) {
        const int s = ring.stage;
        if (!warp_wait(kv_empty(s), ring.phase ^ 1, wc)) return false;
        const int key0 = (sg.t0 + j) * kTileN;
        const int pages = (min(kTileN, sg.len - key0) + box_rows - 1) / box_rows;
        const uint32_t dst = sb + L::OFF_KV + s * L::TILE + lane * box_rows * 128;
        if (lane == 0) mbar_arrive_expect_tx(kv_full(s), static_cast<uint32_t>(pages * box_rows * D * 2));
        __syncwarp();
        if (lane < pages) {
          const int slot = key0 & (page - 1);  // 0 below 128-slot pages
#pragma unroll
          for (int kb = 0; kb < L::KB; ++kb)
            if (check_tma(ck, dst + kb * L::BOX, box_rows * 128, kv_full(s), kb * 64, D, slot, page, 0, sg.hk,
                          a.HK, __LINE__))
              tma_load_4d(dst + kb * L::BOX, map, kv_full(s), kb * 64, slot, sg.hk, pg);
        }
        ring.step(L::STAGES);
        ++issued;
        return true;
      };
      int pg = page_of(0);
      for (int j = 0; ok && j < sg.n_iter; ++j) {
        const int pg_next = page_of(j + 1);
        ok = load(&tm_k, j, pg) && load(&tm_v, j, pg);
        pg = pg_next;
      }
    }
    // let every copy land before the CTA can exit
    for (int i = max(0, issued - L::STAGES); i < issued; ++i)
      wait_drain(kv_full(i % L::STAGES), (i / L::STAGES) & 1, a.timeout_ns);
  } else if (warp == 2) {
    // ------------------------------------------------------------ MMAs
    if (elect_one()) {
      constexpr uint32_t id_s = TYPE == kTypeBf16 ? idesc_bf16(128, kTileN, 0, 0) : idesc_f16(128, kTileN, 0, 0);
      constexpr uint32_t id_o = TYPE == kTypeBf16 ? idesc_bf16(128, D, 0, 1) : idesc_f16(128, D, 0, 1);
      const uint64_t q0 = smem_desc_sw128(sb + L::OFF_Q, 16, 1024);
      const uint64_t k0 = smem_desc_sw128(sb + L::OFF_KV, 16, 1024), v0 = smem_desc_sw128(sb + L::OFF_KV, L::BOX, 1024);
      RingPos ring{0, 0};
      uint32_t tiles = 0;  // so far
      bool ok = check_tmem(ck, tmem, 128, 256, __LINE__);
      auto landed = [&]() {
        const bool got = wait_bounded(kv_full(ring.stage), ring.phase, wc);
        tc_fence_after();
        return got;
      };
      for (int i = 0; ok; ++i) {
        const int k = i & 1;
        if (!(ok = wait_bounded(q_full(k), (i >> 1) & 1, wc))) break;
        const int n_iter = segs[k].n_iter;
        if (n_iter == 0) break;
        for (int j = 0; ok && j < n_iter; ++j, ++tiles) {
          if (!(ok = landed())) break;
          const uint32_t at = static_cast<uint32_t>(ring.stage) * (L::TILE >> 4);
#pragma unroll
          for (int e = 0; e < D / 16; ++e)
            mma_bf16(tmem, q0 + ((k * L::QBUF + (e >> 2) * L::QBOX + (e & 3) * 32) >> 4),
                     k0 + at + (((e >> 2) * L::BOX + (e & 3) * 32) >> 4), id_s, e > 0);
          mma_commit(s_full);
          mma_commit(kv_empty(ring.stage));
          ring.step(L::STAGES);
          // (P comes with V's rows past the last key cleared)
          if (!(ok = landed() && wait_bounded(p_full, tiles & 1, wc))) break;
          tc_fence_after();
          const uint32_t vt = static_cast<uint32_t>(ring.stage) * (L::TILE >> 4);
#pragma unroll
          for (int e = 0; e < kTileN / 16; ++e)
            mma_bf16_ts(tmem + COL_O, tmem + 8 * e, v0 + vt + e * (2048 >> 4), id_o, j > 0 || e > 0);
          mma_commit(kv_empty(ring.stage));
          ring.step(L::STAGES);
        }
        if (ok) mma_commit(o_full);
      }
      mma_commit(drain);
      wait_drain(drain, 0, a.timeout_ns);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const float c = a.scale * kLog2e;
    RingPos ring{1, 0};  // V's stage
    uint32_t tiles = 0;  // so far
    bool ok = true;
    for (int i = 0; ok; ++i) {
      const int k = i & 1;
      if (!(ok = warp_wait(q_full(k), (i >> 1) & 1, wc))) break;
      const int n_iter = segs[k].n_iter;
      if (n_iter == 0) break;
      const int len = segs[k].len, n = segs[k].n, t0 = segs[k].t0, slot = segs[k].slot;
      const bool live = lane < n * G;
      const int tok = live ? lane / G : 0;
      const int token = segs[k].tok0 + tok, head = segs[k].hk * G + (live ? lane - tok * G : 0);
      // keys < lim are seen by this row
      const int lim = !live ? 0 : a.causal ? min(len, len - n + tok + 1) : len;
      float ref = -INFINITY, l = 0.f;
      for (int j = 0; j < n_iter; ++j, ++tiles) {
        if (!(ok = warp_wait(s_full, tiles & 1, wc))) break;
        tc_fence_after();
        if (!(ok = check_tmem(ck, tmem, 32, 128, __LINE__))) break;
        float s[128];
        const int seen = lim - (t0 + j) * kTileN;  // of this tile's keys
        auto load_s = [&]() {
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32(tmem + 32 * q, *reinterpret_cast<float(*)[32]>(&s[32 * q]));
          tmem_wait_ld();
          if (seen < kTileN) {
#pragma unroll
            for (int e = 0; e < 128; ++e)
              if (e >= seen) s[e] = -INFINITY;
          }
        };
        uint32_t p[64];
        auto terms = [&]() {  // P against ref, in the inputs' type; its fp32 sum
          const float r0 = ref == -INFINITY ? 0.f : ref;
          const float2 c2 = make_float2(c, c), nr = make_float2(-r0, -r0);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int e = 0; e < 64; ++e) {
            const float2 x = __ffma2_rn(make_float2(s[2 * e], s[2 * e + 1]), c2, nr);
            const float2 y = make_float2(ex2(x.x), ex2(x.y));
            sum[e & 1] = __fadd2_rn(sum[e & 1], y);
            p[e] = pack2<TYPE>(y.x, y.y);
          }
          const float2 f = __fadd2_rn(sum[0], sum[1]);
          return f.x + f.y;
        };
        load_s();
        float f = 0.f;
        // as in paged_attn.cu: the reference stays while the sum is within kSumMax
        bool again = __any_sync(0xFFFFFFFFu, ref == -INFINITY && seen > 0);
        if (!again) {
          f = terms();
          again = __any_sync(0xFFFFFFFFu, !(f <= kSumMax<TYPE>));
          if (again) load_s();
        }
        if (again) {
          float m[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int e = 4; e < 124; e += 8) {
#pragma unroll
            for (int q = 0; q < 4; ++q) m[q] = max3(m[q], s[e + 2 * q], s[e + 2 * q + 1]);
          }
          const float top = max3(max3(m[0], m[1], m[2]), max3(m[3], s[124], s[125]), fmaxf(s[126], s[127])) * c;
          // (by its own maximum, whichever row of the warp asked: the others' sums may not have been looked at)
          const bool move = top > ref + rise_allowed<TYPE>(top) || (ref == -INFINITY && top > -INFINITY);
          const float alpha = move ? ex2(ref - (top - kBelow<TYPE>)) : 1.f;
          if (move) {
            ref = top - kBelow<TYPE>;
            l *= alpha;
          }
          if (j > 0) {  // O holds the tiles before this one, all done before this S
#pragma unroll
            for (int q = 0; q < D / 16; ++q) {
              float o[16];
              tmem_ld16(tmem + COL_O + 16 * q, o);
              tmem_wait_ld();
              uint32_t r[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(o[e] * alpha);
              tmem_st16(tmem + COL_O + 16 * q, r);
            }
          }
          f = terms();
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_st16(tmem + 16 * q, &p[16 * q]);
        l += f;
        // V's rows past the last key (the slots there hold anything, and
        // 0 x NaN is NaN): cleared once it has landed
        const int valid = len - (t0 + j) * kTileN;
        if (valid < kTileN) {
          if (!(ok = warp_wait(kv_full(ring.stage), ring.phase, wc))) break;
          uint8_t* v = gb + L::OFF_KV + ring.stage * L::TILE;
          for (int e = valid * 8 + lane; e < kTileN * 8; e += 32)  // 16 bytes each
#pragma unroll
            for (int kb = 0; kb < L::KB; ++kb)
              *reinterpret_cast<uint4*>(v + kb * L::BOX + e * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
        }
        ring.step(L::STAGES);
        ring.step(L::STAGES);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
      }
      // ---------------------------------------------------------- output
      if (!ok || !(ok = warp_wait(o_full, i & 1, wc))) break;
      tc_fence_after();
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;  // (NaN stays NaN)
      const bool none = l == 0.f;
      const long long e = static_cast<long long>(token) * a.HQ + head;
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        float o[32];
        tmem_ld32(tmem + COL_O + 32 * q, o);
        tmem_wait_ld();
#pragma unroll
        for (int x = 0; x < 32; ++x) o[x] = none ? 0.f : o[x] * inv;
        if (live) {
          if (slot >= 0) {
            float4* dst = reinterpret_cast<float4*>(a.part_o + (static_cast<long long>(slot) * kRows + lane) * D + 32 * q);
#pragma unroll
            for (int x = 0; x < 8; ++x) dst[x] = make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
          } else {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + token * a.o_sn + head * a.o_sh + 32 * q);
#pragma unroll
            for (int x = 0; x < 4; ++x)
              dst[x] = make_uint4(pack2<TYPE>(o[8 * x], o[8 * x + 1]), pack2<TYPE>(o[8 * x + 2], o[8 * x + 3]),
                                  pack2<TYPE>(o[8 * x + 4], o[8 * x + 5]), pack2<TYPE>(o[8 * x + 6], o[8 * x + 7]));
          }
        }
      }
      if (live) {
        const float lse2 = none ? -INFINITY : ref + log2f(l);
        if (slot >= 0)
          a.part_lse[slot * kRows + lane] = lse2;
        else
          a.lse[e] = lse2 * kLn2;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(q_empty(k));
    }
  }

  grid_launch_dependents();  // the combine kernel may be launched
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// Join the parts of the items that the CTAs' stretches cut: block c takes the
// item that starts in CTA c's stretch and goes on in the next, its warps the
// rows in turn; the parts of a row lie in the slots of consecutive CTAs.
template <int TYPE, int D>
__global__ void __launch_bounds__(kThreads)
    streamkl_paged_join_kernel(const __grid_constant__ PagedAttnArgs a) {
  constexpr int V = D / 32;  // columns of a lane
  __shared__ long long scratch[kThreads / 32];
  __shared__ Place where;
  long long total;
  const int c0 = static_cast<int>(blockIdx.x);
  const int chunk = locate(
      a, gridDim.x, scratch, &where, &total, [&](int per_cta) { return (c0 + 1LL) * per_cta; },
      [](int, const Seq&) {});
  __syncthreads();
  const long long cut = (c0 + 1LL) * chunk;  // the first tile of the next stretch
  // nothing after it, or an item that starts there, or before this stretch
  const bool none = cut >= total || where.tile == 0 || where.tile > chunk;
  const Seq s = load_seq(a, none ? 0 : where.b);
  const int hk = where.hk;
  const int inside = where.tile < chunk ? 1 : 0;  // the item starts inside this stretch: its last part
  const int parts = 1 + (s.tiles - where.tile + chunk - 1) / chunk;
  auto slot = [&](int i) { return 2 * (c0 + i) + (i == 0 ? inside : 0); };
  // launched while the decode kernel ends; every block waits for its end, since
  // what comes after this kernel counts on both
  grid_dependency_wait();
  if (none) return;
  const int G = a.HQ / a.HK, lane = threadIdx.x & 31;
  for (int r = threadIdx.x >> 5; r < s.n * G; r += kThreads / 32) {
    // parts whose loads are in flight, the first ones beside the lse's (one token
    // over 4,096 keys, both kernels: 12.2 us, 12.5 with 8, 13.9 with 8 after the lse)
    constexpr int RUN = 16;
    float p[RUN][V];
    auto fetch = [&](int i0) {
#pragma unroll
      for (int i = 0; i < RUN; ++i) {
        const float* src = a.part_o + (static_cast<long long>(slot(i0 + i)) * kRows + r) * D + lane * V;
#pragma unroll
        for (int x = 0; x < V; ++x) p[i][x] = 0.f;
        if (i0 + i < parts) {
          if constexpr (V == 4)
            *reinterpret_cast<float4*>(p[i]) = *reinterpret_cast<const float4*>(src);
          else
            *reinterpret_cast<float2*>(p[i]) = *reinterpret_cast<const float2*>(src);
        }
      }
    };
    fetch(0);
    float top = -INFINITY;
    for (int i = lane; i < parts; i += 32) top = fmaxf(top, a.part_lse[slot(i) * kRows + r]);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
    const float t0 = top == -INFINITY ? 0.f : top;
    float sum = 0.f, o[V] = {};
    for (int i0 = 0; i0 < parts; i0 += RUN) {
      if (i0 > 0) fetch(i0);
      const float mine = lane < RUN && i0 + lane < parts ? ex2(a.part_lse[slot(i0 + lane) * kRows + r] - t0) : 0.f;
#pragma unroll
      for (int i = 0; i < RUN; ++i) {
        const float w = __shfl_sync(0xFFFFFFFFu, mine, i);  // 0 past the last part
        sum += w;
#pragma unroll
        for (int x = 0; x < V; ++x) o[x] = fmaf(w, p[i][x], o[x]);
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int token = s.tok0 + r / G, head = hk * G + r % G;
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + token * a.o_sn + head * a.o_sh + lane * V);
#pragma unroll
    for (int x = 0; x < V / 2; ++x) dst[x] = pack2<TYPE>(o[2 * x] * inv, o[2 * x + 1] * inv);
    if (lane == 0) a.lse[static_cast<long long>(token) * a.HQ + head] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
  }
}

template <int TYPE, int D>
cudaError_t decode_t(const PagedAttnArgs& a, int ctas, cudaStream_t stream) {
  using L = DecodeLayout<D>;
  auto kern = streamkl_paged_decode_kernel<TYPE, D>;
  // the shared-memory attribute, once per device
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (!(done.load() & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit);
  }
  kern<<<ctas, kThreads, L::BYTES, stream>>>(*a.tm_k, *a.tm_v, a);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.whole) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, streamkl_paged_join_kernel<TYPE, D>, a);
}

}  // namespace

cudaError_t launch_paged_decode(const PagedAttnArgs& a, int ctas, cudaStream_t stream) {
  if (a.type == kTypeBf16)
    return a.d == 128 ? decode_t<kTypeBf16, 128>(a, ctas, stream) : decode_t<kTypeBf16, 64>(a, ctas, stream);
  return a.d == 128 ? decode_t<kTypeF16, 128>(a, ctas, stream) : decode_t<kTypeF16, 64>(a, ctas, stream);
}

}  // namespace skl
