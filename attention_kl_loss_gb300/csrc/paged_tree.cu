// Attention of drafted tokens over a paged cache (the tokens of a tree, or any that
// see all keys before the drafted ones and some of these): o_i = sum_j p_ij v_j with
// p = softmax(scale q K^T) over the keys j < len - n and the drafted tokens whose
// bits row i's mask has, and lse_i. For more than 32 (token, head of the group) rows
// per sequence and key head; fewer go to paged_decode.cu.
//
// The arithmetic is paged_attn.cu's: 128-row tiles of (token, head) rows, 128-key
// tiles, S = Q K^T and O += P V as tcgen05 MMAs, P = 2^(c s - ref) in the inputs'
// type (8 or 11 bits, the size of the output's own rounding), ref, sum and O in
// fp32, the reference moved only when terms would exceed 2^8 (2^14, fp16) of it.
//
// What differs is how the work is dealt out. A batch of drafts is many sequences of
// very different lengths with one or a few row tiles each, so the key tiles of all
// items (a sequence, a key head, a block of rows) form one line that persistent CTAs
// share evenly, as in paged_decode.cu: one CTA an SM, of NT row tiles that share each
// K and V tile (two CTAs, where one tile of d = 64 is all). A CTA's stretch cuts at
// most its first and its last item; a join kernel adds those parts by their lse.
// Where that is near an equal share each CTA takes whole items instead, and nothing
// is joined; where items are few, short and large enough for it a cluster takes each,
// its CTAs the tiles in turn, and joins their parts out of shared memory (CLUSTER: no
// search, no second kernel, first page numbers loaded beside the length). Loads run on
// from item to item (a warp publishes the coming items' numbers), so HBM is kept busy
// while an item's output leaves; the next item's rows of Q are copied into a second
// place of theirs meanwhile, or held in registers where there is only one.
//
// The mask is looked at only in tiles that hold drafted keys: four words of a row's
// bits, shifted into place, before that tile's S is there.
//
// What bounds it (one GB300, both kernels; a turn is one key tile of a CTA):
//   d = 128, one row tile: HBM. 64 sequences of up to 16,384 keys, 16 drafted tokens,
//     32 heads over 8: 456 us, 6.5 TB/s; 1.48 us a turn, some 20 us start, end and join.
//   d = 128, two: the chain S, P, O of a row tile, 1.8 us a turn for 1.3 of products.
//     4 sequences of up to 16,384 keys with 256 drafted tokens 131 us, 1.1 PFLOP/s.
//   d = 64: the softmax, 0.80 us a turn of one row tile (two CTAs an SM), 1.35 of two.
//     24 sequences of up to 5,000 keys, up to 61 tokens, 8 heads 48 us, 3.2 TB/s. With
//     two it is farthest from its bytes: 56 sequences of up to 1,023 keys, up to 339
//     tokens, 10 heads 96 us for 18 at a plain copy's rate.
// No faster, each measured: softmax by two halves of the columns at d = 64 with two
// row tiles (125 us for 104), barriers per row tile there (no change), two CTAs of one
// row tile for more than 128 rows of d = 64 in large calls (200 for 189; small ones do
// that), the output's loops rolled.
#include <algorithm>
#include <atomic>
#include <climits>
#include <type_traits>

#include "ops.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace skl {

namespace {

constexpr int kTileM = 128;  // rows per tile
constexpr int kFirst = 96;   // keys of a tile whose P is handed over first (P in S's place)
constexpr int kSegs = 4;     // items whose numbers are known ahead
constexpr int kJoinWarps = 8;  // rows of a block of the join kernel

// A CTA's part of an item: key tiles [t0, t0 + n_iter) of rows from rb * 128 NT on.
struct Seg {
  int b, hk, rb, t0, n_iter;  // n_iter 0: no more
  int tok0, n, len;
  int slot;  // partial slot, or -1: the whole item
};

template <int D, int NT>
struct TreeLayout {
  static constexpr int KB = D / 64;          // 64-column (128-byte) boxes per row
  static constexpr int BOX = kTileN * 128;   // 128 rows of one box
  static constexpr int TILE = kTileN * D * 2;
  // CTAs of an SM: two where shared memory and half of TMEM hold what one needs
  static constexpr int PER_SM = D == 64 && NT == 1 ? 2 : 1;
  static constexpr int STAGES = D == 64 && NT == 2 ? 10 : 5;
  static constexpr int TMEM = 512 / PER_SM;
  // Q of the next item beside this one's, where there is room for it
  static constexpr int QBUFS = D == 128 && NT == 2 ? 1 : 2;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = QBUFS * NT * TILE;
  static constexpr int OFF_BAR = OFF_KV + STAGES * TILE;
  // P in columns of its own, where TMEM has room for them; else in S's place
  static constexpr bool OWN_P = D == 64 || NT == 1;
  // Softmax warpgroups of a row tile, each with half of a key tile's columns where
  // there are two: one warp of a scheduler waits for its own instructions most of
  // the time
  static constexpr int HALVES = D == 128 && NT == 1 ? 2 : 1;
  static constexpr int CW = kTileN / HALVES;      // columns of S of a thread
  static constexpr int WARPS = 4 * NT * HALVES;   // of the softmax
  // q_full[2], kv_full[S], kv_empty[S], s_full[2], p_full[2], o_full[2], s_read, p_read,
  // drain, p_first[2], o_first[2], seg_full[kSegs], seg_empty[kSegs], pair[4]
  static constexpr int NBAR = 2 + 2 * STAGES + 13 + 2 * kSegs + 4;
  static constexpr int OFF_SEG = OFF_BAR + NBAR * 8;
  static constexpr int OFF_MISC = (OFF_SEG + kSegs * static_cast<int>(sizeof(Seg)) + 15) / 16 * 16;
  static constexpr int THREADS = 128 + 32 * WARPS;
  static constexpr int OFF_PAIR = OFF_MISC + 32 + THREADS / 32 * 8;  // [2][halves][rows] floats
  static constexpr int BYTES = OFF_PAIR + (HALVES == 2 ? 2 * 2 * kTileM * 4 : 0);
  static_assert(PER_SM == 1 ? BYTES <= 232448 : 2 * (BYTES + 1024) <= 233472, "shared memory budget");
  static constexpr int col_s(int t) { return 128 * t; }
  static constexpr int col_p(int t) { return OWN_P ? 128 * NT + 64 * t : 128 * t; }
  static constexpr int col_o(int t) { return (OWN_P ? 192 : 128) * NT + D * t; }
  static_assert(col_o(NT - 1) + D <= TMEM, "TMEM columns");
};

// What is known of a sequence.
struct Seq {
  int tok0, n, len, tiles, blocks;
  bool ok;
};

__device__ __forceinline__ Seq load_seq(const PagedAttnArgs& a, int b, int rows_block) {
  Seq s;
  const int c0 = a.cu != nullptr ? __ldg(a.cu + b) : b;
  const int c1 = a.cu != nullptr ? __ldg(a.cu + b + 1) : b + 1;
  s.len = __ldg(a.kv_lens + b);
  s.tok0 = c0;
  s.n = c1 - c0;
  s.ok = c0 >= 0 && c1 >= c0 && c1 <= a.T && s.n <= a.max_q && s.len >= 0 && s.len <= a.max_kv;
  if (!s.ok) s.n = 0;
  s.blocks = (s.n * (a.HQ / a.HK) + rows_block - 1) / rows_block;
  s.tiles = s.n > 0 ? (s.len + kTileN - 1) / kTileN : 0;
  return s;
}

// The whole block finds its way in the line of tiles: each thread sums a run of
// consecutive sequences, a scan adds them up; the thread in whose run this CTA's
// first tile lies writes where that is to *at (left alone past the line's end).
// Returns the tiles of a CTA's stretch. One barrier; *at is there after the next.
struct Place {
  int b, hk, rb, tile;
};
template <int THREADS, typename V>
__device__ __forceinline__ long long locate(const PagedAttnArgs& a, int rows_block, long long* scratch,
                                            volatile Place* at, long long* total, V&& visit) {
  const int per = (a.B + THREADS - 1) / THREADS;
  const int b0 = min(a.B, static_cast<int>(threadIdx.x) * per), b1 = min(a.B, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const Seq s = load_seq(a, b, rows_block);
    mine += static_cast<long long>(s.tiles) * s.blocks;
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
  for (int i = 0; i < THREADS / 32; ++i) {
    if (i < warp) base += scratch[i];
    sum += scratch[i];
  }
  const long long chunk = max((sum + gridDim.x - 1) / gridDim.x, static_cast<long long>(a.split_tiles));
  const long long x = blockIdx.x * chunk;
  long long first = base + upto - mine;
  if (first <= x && x < first + mine)
    for (int b = b0; b < b1; ++b) {
      const Seq s = load_seq(a, b, rows_block);
      const long long all = static_cast<long long>(s.tiles) * s.blocks * a.HK;
      if (first <= x && x < first + all) {
        const long long item = (x - first) / s.tiles;
        at->b = b;
        at->hk = static_cast<int>(item / s.blocks);
        at->rb = static_cast<int>(item % s.blocks);
        at->tile = static_cast<int>((x - first) % s.tiles);
      }
      first += all;
    }
  *total = sum;
  return chunk;
}

// 16 bytes from global to shared memory, past the registers; and the wait for all
// of this thread's.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void st_shared_f32(uint32_t at, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}
__device__ __forceinline__ float ld_shared_f32(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

// Lane `from`'s pointer.
template <typename T>
__device__ __forceinline__ T* shfl_ptr(T* p, int from) {
  return reinterpret_cast<T*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(p), from));
}

template <int TYPE, int D, int NT, bool CLUSTER>
__global__ void __launch_bounds__(TreeLayout<D, NT>::THREADS, TreeLayout<D, NT>::PER_SM)
    streamkl_paged_tree_kernel(const __grid_constant__ CUtensorMap tm_k,
                               const __grid_constant__ CUtensorMap tm_v,
                               const __grid_constant__ TreeAttnArgs a) {
  using L = TreeLayout<D, NT>;
  constexpr int kRows = kTileM * NT;
  extern __shared__ __align__(1024) uint8_t gb[];
  const uint32_t sb = smem_u32(gb);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.HQ / a.HK;
  const uint32_t bar0 = sb + L::OFF_BAR;
  auto q_full = [&](int it) { return bar0 + 8u * (it % L::QBUFS); };
  auto kv_full = [&](int s) { return bar0 + 8u * (2 + s); };
  auto kv_empty = [&](int s) { return bar0 + 8u * (2 + L::STAGES + s); };
  const uint32_t rest = bar0 + 8u * (2 + 2 * L::STAGES);
  auto s_full = [&](int k) { return rest + 8u * k; };
  auto p_full = [&](int k) { return rest + 8u * (2 + k); };
  auto o_full = [&](int k) { return rest + 8u * (4 + k); };
  const uint32_t s_read = rest + 48, p_read = rest + 56, drain = rest + 64;
  auto p_first = [&](int k) { return rest + 8u * (9 + k); };
  auto o_first = [&](int k) { return rest + 8u * (11 + k); };
  auto seg_full = [&](int k) { return rest + 8u * (13 + k); };
  auto seg_empty = [&](int k) { return rest + 8u * (13 + kSegs + k); };
  auto pair = [&](int k) { return rest + 8u * (13 + 2 * kSegs + k); };
  static_assert(2 + 2 * L::STAGES + 13 + 2 * kSegs + 4 == L::NBAR, "barrier region holds every barrier");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gb + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gb + L::OFF_MISC + 4);
  volatile int* skip_flag = reinterpret_cast<volatile int*>(gb + L::OFF_MISC + 8);
  long long* scratch = reinterpret_cast<long long*>(gb + L::OFF_MISC + 32);
  volatile Seg* segs = reinterpret_cast<volatile Seg*>(gb + L::OFF_SEG);
  volatile Place* start = reinterpret_cast<volatile Place*>(gb + L::OFF_MISC + 16);

  CheckCtx ck{sb, sb + L::OFF_BAR, sb + L::OFF_BAR, sb + L::OFF_BAR + L::NBAR * 8, 0, 0,
              abort_flag, a.dev_status};
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    bool lay_ok = (sb & 1023u) == 0;  // the swizzled tiles' alignment
    if (!lay_ok) atomicCAS(a.dev_status, 0, kStatusDeviceCheck);
    if (kDeviceChecks)
      for (int i = 0; i < L::NBAR; ++i) lay_ok = lay_ok && check_bar(ck, bar0 + 8u * i, __LINE__);
    if (lay_ok) {
      for (int k = 0; k < 2; ++k) mbar_init(bar0 + 8u * k, L::WARPS);  // q_full: one arrival per softmax warp
      for (int s = 0; s < L::STAGES; ++s) {
        mbar_init(kv_full(s), 1);
        mbar_init(kv_empty(s), NT);
      }
      for (int k = 0; k < 2; ++k) {
        mbar_init(s_full(k), 1);
        mbar_init(p_full(k), L::OWN_P ? L::WARPS : 4);
        mbar_init(o_full(k), 1);
        mbar_init(p_first(k), 4);
        mbar_init(o_first(k), 1);
      }
      mbar_init(s_read, L::WARPS);
      mbar_init(p_read, 1);
      mbar_init(drain, 1);
      for (int k = 0; k < 4; ++k) mbar_init(pair(k), 2);
      for (int k = 0; k < kSegs; ++k) {
        mbar_init(seg_full(k), 1);
        mbar_init(seg_empty(k), 3 + L::WARPS);  // loads of K and of V, MMAs, softmax warps
      }
    }
    // a failure recorded earlier, or a failed layout check, skips the work; not a
    // bad number of some sequence, which may come from this very call
    const int before = *reinterpret_cast<volatile int*>(a.dev_status);
    *skip_flag = !lay_ok || (before != 0 && before != kStatusInvalidArg);
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), L::TMEM);
    tmem_relinquish();
  }
  // this CTA's stretch of the line of tiles, or whole items; sequences without a key on
  // the way (those of a resize that found no pages, too)
  bool empty = false;
  auto visit = [&](int b, const Seq& s) {
    if (blockIdx.x == 0 && !s.ok) atomicCAS(a.dev_status, 0, kStatusInvalidArg);
    empty = empty || (s.n > 0 && s.tiles == 0 && b % gridDim.x == blockIdx.x);
  };
  long long total = 0, chunk = 0;
  // With CLUSTER the CTAs of a cluster take the key tiles of one item in turn
  int ranks = 1, rank = 0, one_b = 0, one_hk = 0, one_rb = 0, page0 = -1;
  if constexpr (CLUSTER) {
    ranks = a.cluster;
    rank = static_cast<int>(cluster_ctarank());
    const int item = static_cast<int>(blockIdx.x) / ranks;
    one_rb = item / (a.B * a.HK), one_b = item / a.HK - one_rb * a.B, one_hk = item % a.HK;
    if (warp == 0 || warp == 2) {  // the first tile's pages, before the length is known
      const int box_rows = min(1 << a.page_shift, kTileN);
      const long long at = (static_cast<long long>(rank) * kTileN + lane * box_rows) >> a.page_shift;
      if (at < a.max_pages) page0 = __ldg(a.table + one_b * a.table_sb + at);
    }
  }
  if (a.whole) {
    for (int b = threadIdx.x; b < a.B; b += L::THREADS)
      if (blockIdx.x == 0 || b % gridDim.x == blockIdx.x) visit(b, load_seq(a, b, kRows));
  } else {
    chunk = locate<L::THREADS>(a, kRows, scratch, start, &total, visit);
  }
  tc_fence_before();
  // Empty rows by the whole CTA (4 sequences of 256 tokens, 32 heads, up to 16,384 keys,
  // one of them empty: 122 us; by the thread that met it 880)
  if (__syncthreads_or(empty) && !*skip_flag)
    for (int b = static_cast<int>(blockIdx.x); b < a.B; b += static_cast<int>(gridDim.x)) {
      const Seq s = load_seq(a, b, kRows);
      if (s.tiles == 0) empty_rows<D>(a, s.tok0, s.n, static_cast<int>(threadIdx.x), L::THREADS);
    }
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);  // (the same in every lane)
  ck.tmem = tmem;
  ck.tmem_cols = L::TMEM;
  const WaitCtx wc{abort_flag, a.dev_status, a.timeout_ns};

  // Place of key tile j's K and V among an item's 2 n loads, in the order in which the
  // MMAs use them: K0 V0 K1 V1 .., with P in columns of its own K0 K1 V0 K2 V1 ..
  auto idx_k = [](int j) { return !L::OWN_P ? 2 * j : (j == 0 ? 0 : 2 * j - 1); };
  auto idx_v = [](int j, int n) { return !L::OWN_P ? 2 * j + 1 : (j + 1 < n ? 2 * j + 2 : 2 * j + 1); };
  // an item's numbers, handed back as soon as they are in registers (by the whole
  // warp; the issuing thread of the MMAs comes alone)
  auto take_seg = [&](int it, Seg& s, bool alone) {
    const int k = it % kSegs;
    const uint32_t parity = (it / kSegs) & 1;
    if (!(alone ? wait_bounded(seg_full(k), parity, wc) : warp_wait(seg_full(k), parity, wc))) return false;
    s.b = segs[k].b;
    s.hk = segs[k].hk;
    s.rb = segs[k].rb;
    s.t0 = segs[k].t0;
    s.n_iter = segs[k].n_iter;
    s.tok0 = segs[k].tok0;
    s.n = segs[k].n;
    s.len = segs[k].len;
    s.slot = segs[k].slot;
    if (!alone) __syncwarp();
    if (alone || lane == 0) mbar_arrive(seg_empty(k));
    return true;
  };

  if (warp < 4) {
  // A softmax thread holds a row of S (128, or half of one). 128 threads with 88
  // registers and 256 with 208 make up the launch's 384 x 168; two CTAs an SM: 128
  // with 48 and 128 with 208 its 256 x 128
  if (L::WARPS == 8) regs_dec<88>();
  if (L::PER_SM == 2) regs_dec<48>();
  if (warp == 3) {
    // ------------------------------------------------------------ items
    long long left = *skip_flag ? 0 : max(0LL, min(total - blockIdx.x * chunk, chunk));
    int b = 0, hk = 0, rb = 0, tile = 0;
    int item = *skip_flag ? INT_MAX : static_cast<int>(blockIdx.x);  // with whole items, every gridDim.x-th
    TreeCut cut{};  // the item that goes on in the next stretch
    if (left > 0) b = start->b, hk = start->hk, rb = start->rb, tile = start->tile;
    for (int it = 0;; ++it) {
      Seg sg{};
      if constexpr (CLUSTER) {
        if (it == 0) {
          const Seq s = load_seq(a, one_b, kRows);
          const bool mine = !*skip_flag && one_rb < s.blocks && rank < s.tiles;
          sg = {one_b,  one_hk, one_rb, rank, mine ? (s.tiles - rank + ranks - 1) / ranks : 0,
                s.tok0, s.n,    s.len,  s.tiles == 1 ? -1 : 0};
        }
      } else if (a.whole) {
        for (; item < a.B * a.HK * a.q_tiles && sg.n_iter == 0; item += gridDim.x) {
          // (all first blocks of rows, then the second ones that there are, ..)
          rb = item / (a.B * a.HK), b = item / a.HK - rb * a.B, hk = item % a.HK;
          const Seq s = load_seq(a, b, kRows);
          if (rb < s.blocks) sg = {b, hk, rb, 0, s.tiles, s.tok0, s.n, s.len, -1};
        }
      } else if (left > 0) {
        Seq s = load_seq(a, b, kRows);
        while (s.tiles == 0) s = load_seq(a, ++b, kRows);  // (b < B: tiles are left)
        sg = {b, hk, rb, tile, static_cast<int>(min(left, static_cast<long long>(s.tiles - tile))), s.tok0, s.n, s.len, 0};
        sg.slot = sg.n_iter == s.tiles ? -1 : 2 * static_cast<int>(blockIdx.x) + (it > 0);
        // (an item that began before this stretch is not its to join)
        if (tile + sg.n_iter < s.tiles && tile == 0)
          cut = {s.tok0, hk, rb * kRows, min(kRows, s.n * G - rb * kRows),
                 1 + static_cast<int>((s.tiles - sg.n_iter + chunk - 1) / chunk), it > 0};
        left -= sg.n_iter;
        tile += sg.n_iter;
        if (tile == s.tiles) {
          tile = 0;
          if (++rb == s.blocks) {
            rb = 0;
            if (++hk == a.HK) {
              hk = 0;
              ++b;
            }
          }
        }
      }
      const int k = it % kSegs;
      if (!warp_wait(seg_empty(k), ((it / kSegs) & 1) ^ 1, wc)) break;
      if (lane == 0) {
        segs[k].b = sg.b;
        segs[k].hk = sg.hk;
        segs[k].rb = sg.rb;
        segs[k].t0 = sg.t0;
        segs[k].n_iter = sg.n_iter;
        segs[k].tok0 = sg.tok0;
        segs[k].n = sg.n;
        segs[k].len = sg.len;
        segs[k].slot = sg.slot;
        mbar_arrive(seg_full(k));
      }
      __syncwarp();
      if (sg.n_iter == 0) break;
    }
    if (!a.whole && lane == 0) a.cuts[blockIdx.x] = cut;
  } else if (warp != 1) {
    // ------------------------------------------------------ loads of K or V
    const bool is_v = warp == 2;
    const CUtensorMap* map = is_v ? &tm_v : &tm_k;
    const int page = 1 << a.page_shift;
    const int box_rows = min(page, kTileN);
    int base = 0;                    // loads of the items before
    int recent[4] = {-1, -1, -1, -1};  // this warp's last ones
    bool ok = true;
    for (int it = 0; ok; ++it) {
      Seg sg;
      if (!(ok = take_seg(it, sg, false)) || sg.n_iter == 0) break;
      const int* table = a.table + static_cast<long long>(sg.b) * a.table_sb;
      // the page this lane loads of tile j; a number that is none is reported
      // and page 0 read in its place
      auto page_of = [&](int j) {
        const int key = (sg.t0 + j * ranks) * kTileN + lane * box_rows;
        if (j >= sg.n_iter || lane * box_rows >= kTileN || key >= sg.len) return -1;
        int p = CLUSTER && j == 0 ? page0 : __ldg(table + (key >> a.page_shift));
        if (p < 0 || p >= a.num_pages) {
          atomicCAS(a.dev_status, 0, kStatusInvalidArg);
          p = 0;
        }
        return p;
      };
      int pg = page_of(0), pg_next = page_of(1);
      for (int j = 0; j < sg.n_iter; ++j) {
        // The stage's barrier cannot be two phases behind what is waited for: loads
        // are used in their order but for neighbours, this warp's one before this
        // lies at most three back, and the ring is longer than that by two
        const int i = base + (is_v ? idx_v(j, sg.n_iter) : idx_k(j)), s = i % L::STAGES;
        if (!(ok = warp_wait(kv_empty(s), ((i / L::STAGES) & 1) ^ 1, wc))) break;
        const int key0 = (sg.t0 + j * ranks) * kTileN;
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
#pragma unroll
        for (int x = 3; x > 0; --x) recent[x] = recent[x - 1];
        recent[0] = i;
        pg = pg_next;
        pg_next = page_of(j + 2);
      }
      if (ok) base += 2 * sg.n_iter;
    }
    // Let every copy land before the CTA can exit: this warp's last in the ring (a
    // stage that was used again, its copy had landed; after a failure some of these
    // waits may be for a phase that is over, and end by their limit)
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (recent[x] >= 0 && (!ok || recent[x] >= base - L::STAGES))
        wait_drain(kv_full(recent[x] % L::STAGES), (recent[x] / L::STAGES) & 1, a.timeout_ns);
  } else if (elect_one()) {
    // ------------------------------------------------------------ MMAs
    // One thread issues every product; it waits for P and S only (with them come the
    // loads), but for an item's first K. As in paged_attn.cu.
    constexpr uint32_t id_s = TYPE == kTypeBf16 ? idesc_bf16(kTileM, kTileN, 0, 0) : idesc_f16(kTileM, kTileN, 0, 0);
    constexpr uint32_t id_o = TYPE == kTypeBf16 ? idesc_bf16(kTileM, D, 0, 1) : idesc_f16(kTileM, D, 0, 1);
    const uint64_t q0 = smem_desc_sw128(sb + L::OFF_Q, 16, 1024);
    const uint64_t k0 = smem_desc_sw128(sb + L::OFF_KV, 16, 1024), v0 = smem_desc_sw128(sb + L::OFF_KV, L::BOX, 1024);
    const uint32_t hi = static_cast<uint32_t>(k0 >> 32);  // the same in all three
    const uint32_t q_lo = static_cast<uint32_t>(q0), k_lo = static_cast<uint32_t>(k0), v_lo = static_cast<uint32_t>(v0);
    auto desc = [&](uint32_t lo) { return static_cast<uint64_t>(hi) << 32 | lo; };
    RingPos ring{0, 0};  // next stage to be used
    auto next = [&]() {  // its offset in descriptor units
      const uint32_t at = static_cast<uint32_t>(ring.stage) * (L::TILE >> 4);
      ring.step(L::STAGES);
      return at;
    };
    auto mma_s = [&](int t, uint32_t q_at, uint32_t k_at) {  // S = Q_t K_j^T
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint32_t off = ((i >> 2) * L::BOX + (i & 3) * 32) >> 4;
        mma_bf16(tmem + L::col_s(t), desc(q_at + t * (L::TILE >> 4) + off), desc(k_lo + k_at + off), id_s, i > 0);
      }
    };
    auto mma_o = [&](int t, int from, int to, uint32_t v_at, uint32_t add) {  // O_t += P V_j, of keys [from, to)
#pragma unroll
      for (int k = from / 16; k < to / 16; ++k)
        mma_bf16_ts(tmem + L::col_o(t), tmem + L::col_p(t) + 8 * k, desc(v_lo + v_at + k * (2048 >> 4)), id_o,
                    k > 0 ? 1 : add);
    };
    bool ok = check_tmem(ck, tmem, 128, L::TMEM, __LINE__);
    uint32_t tiles = 0;  // so far
    for (int it = 0; ok; ++it) {
      Seg sg;
      if (!(ok = take_seg(it, sg, true)) || sg.n_iter == 0) break;
      if (!(ok = wait_bounded(q_full(it), (it / L::QBUFS) & 1, wc) && wait_bounded(kv_full(ring.stage), ring.phase, wc)))
        break;
      // (with Q there early, the last item's S may still be read)
      if (L::QBUFS == 2 && it > 0 && !(ok = wait_bounded(s_read, (tiles - 1) & 1, wc))) break;
      tc_fence_after();
      const uint32_t q_at = q_lo + it % L::QBUFS * (NT * L::TILE >> 4);
      uint32_t k_at = next();
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        mma_s(t, q_at, k_at);
        if (!L::OWN_P || t == NT - 1) mma_commit(s_full(L::OWN_P ? 0 : t));
      }
#pragma unroll 1
      for (int j = 0; ok && j < sg.n_iter; ++j, ++tiles) {
        const bool more = j + 1 < sg.n_iter;
        if (!L::OWN_P) {
          // P of row tile 0 comes with V of this tile and K of the next
          const uint32_t v_at = next();
          if (more) k_at = next();
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            if (!(ok = wait_bounded(p_first(t), tiles & 1, wc))) break;
            tc_fence_after();
            mma_o(t, 0, kFirst, v_at, j > 0);
            mma_commit(o_first(t));
            if (!(ok = wait_bounded(p_full(t), tiles & 1, wc))) break;
            tc_fence_after();
            mma_o(t, kFirst, kTileN, v_at, 1);
            if (more) mma_s(t, q_at, k_at);
            mma_commit(more ? s_full(t) : o_full(t));
          }
          if (!ok) break;
        } else {
          // S comes back with K of the next tile, P with V of this one
          if (more) {
            k_at = next();
            if (!(ok = wait_bounded(s_read, tiles & 1, wc))) break;
            tc_fence_after();
#pragma unroll
            for (int t = 0; t < NT; ++t) mma_s(t, q_at, k_at);
            mma_commit(s_full(0));
          }
          const uint32_t v_at = next();
          if (!(ok = wait_bounded(p_full(0), tiles & 1, wc))) break;
          tc_fence_after();
#pragma unroll
          for (int t = 0; t < NT; ++t) mma_o(t, 0, kTileN, v_at, j > 0);
          mma_commit(more ? p_read : o_full(0));
        }
      }
    }
    mma_commit(drain);
    wait_drain(drain, 0, a.timeout_ns);
  }
  if constexpr (CLUSTER) {  // (the parts are there; they have been read)
    __syncwarp();
    cluster_sync();
    cluster_sync();
  }
  } else {
    // ------------------------------------------------------------ softmax
    if (L::WARPS == 8 || L::PER_SM == 2) regs_inc<208>();
    const int t = L::HALVES == 1 ? (warp - 4) >> 2 : 0;     // row tile
    const int half = L::HALVES == 2 ? (warp - 4) >> 2 : 0;  // of its columns
    const int r_tile = (warp & 3) * 32 + lane;   // TMEM lane
    const float c = a.scale * kLog2e;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + L::col_s(t) + L::CW * half + lanes, tp = tmem + L::col_p(t) + L::CW / 2 * half + lanes,
                   to = tmem + L::col_o(t) + D / L::HALVES * half + lanes;
    // the other half's number of the same row
    uint32_t swaps = 0;  // so far
    auto swap = [&](float mine, float* other) {
      const uint32_t at = sb + L::OFF_PAIR + ((swaps & 1) * 2 * kTileM + r_tile) * 4;
      st_shared_f32(at + half * kTileM * 4, mine);
      __syncwarp();
      if (lane == 0) mbar_arrive(pair(warp & 3));
      if (!warp_wait(pair(warp & 3), swaps & 1, wc)) return false;
      *other = ld_shared_f32(at + (1 - half) * kTileM * 4);
      ++swaps;
      return true;
    };
    // this warp's rows of Q, its half's columns of them (the part of Q's place that it
    // stages its output in, too), 128-byte swizzled as TMA would place them; rows that
    // are not there are zero
    constexpr int LPR = D / L::HALVES / 8, RPI = 32 / LPR;  // lanes of a row, rows at once
    static_assert(L::HALVES == 1 || D / L::HALVES == 64, "a half is one box");
    auto row_of_q = [&](const Seg& s) -> const uint16_t* {  // this thread's, null where there is none
      const int row = s.rb * kRows + t * kTileM + r_tile, tok = row / G;
      return s.n_iter > 0 && row < s.n * G ? static_cast<const uint16_t*>(a.q) + (s.tok0 + tok) * a.q_sn +
                                                 (s.hk * G + row - tok * G) * a.q_sh
                                           : nullptr;
    };
    const int cq = half * LPR + lane % LPR;
    auto place_q = [&](int i, int it) {  // of this lane's chunk of the warp's rows i * RPI ..
      const int r = (warp & 3) * 32 + i * RPI + lane / LPR;
      return sb + L::OFF_Q + (it % L::QBUFS * NT + t) * L::TILE + (cq >> 3) * L::BOX + r * 128 + (((cq & 7) ^ (r & 7)) << 4);
    };
    // into registers and from there, or past them where Q has two places
    auto fetch_q = [&](const Seg& s, uint4 (&v)[LPR]) {
      const uint16_t* mine = row_of_q(s);
#pragma unroll
      for (int i = 0; i < LPR; ++i) {
        const uint16_t* row_q = shfl_ptr(mine, i * RPI + lane / LPR);
        v[i] = make_uint4(0, 0, 0, 0);
        if (row_q != nullptr) v[i] = __ldg(reinterpret_cast<const uint4*>(row_q) + cq);
      }
    };
    auto give_q = [&](int it) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full(it));
    };
    auto put_q = [&](const uint4 (&v)[LPR], int it) {
#pragma unroll
      for (int i = 0; i < LPR; ++i) st_shared_v4(place_q(i, it), v[i].x, v[i].y, v[i].z, v[i].w);
      give_q(it);
    };
    auto copy_q = [&](const Seg& s, int it) {
      const uint16_t* mine = row_of_q(s);
#pragma unroll
      for (int i = 0; i < LPR; ++i) {
        const uint16_t* row_q = shfl_ptr(mine, i * RPI + lane / LPR);
        if (row_q != nullptr)
          copy16_async(place_q(i, it), row_q + 8 * cq);
        else
          st_shared_v4(place_q(i, it), 0, 0, 0, 0);
      }
    };
    int base = 0;        // loads of the items before
    uint32_t tiles = 0;  // of the items before
    uint32_t reads = 0;  // of P, commits so far
    Seg sg;
    bool ok = take_seg(0, sg, false);
    const int one_tok0 = sg.tok0, one_rows = ok ? min(kRows, sg.n * G - sg.rb * kRows) : 0, one_tiles = (sg.len + kTileN - 1) / kTileN;
    if (ok && sg.n_iter > 0) {
      uint4 v[LPR];
      fetch_q(sg, v);
      put_q(v, 0);
    }
    for (int it = 0; ok && sg.n_iter > 0; ++it) {
      const int n_iter = sg.n_iter, rows = sg.n * G;
      const int row = sg.rb * kRows + t * kTileM + r_tile;  // row of the sequence
      const bool live = row < rows;
      const int tok = live ? row / G : 0;
      const int token = sg.tok0 + tok, head = sg.hk * G + (live ? row - tok * G : 0);
      const bool warp_live = sg.rb * kRows + t * kTileM + (warp & 3) * 32 < rows;
      // keys of the last tile that are there; the rest of its V rows are cleared
      const int last_valid = min(kTileN, sg.len - (sg.t0 + (n_iter - 1) * ranks) * kTileN);
      float ref = -INFINITY, l = 0.f;
      Seg after{};  // the next item
      if (L::QBUFS == 2) {
        if (!(ok = take_seg(it + 1, after, false))) break;
        if (after.n_iter > 0) copy_q(after, it + 1);
      }
      auto landed_k = [&](int j) {
        const int i = base + idx_k(j);
        return warp_wait(kv_full(i % L::STAGES), (i / L::STAGES) & 1, wc);
      };
      // S has been read; K of the next tile comes with it, landed as warp 6 has seen: the
      // thread of the MMAs waits for nothing else of that tile, so the arrival releases
      auto hand_back_s = [&](int j) {
        const bool got = warp != 6 || j + 1 == n_iter || landed_k(j + 1);
        tc_fence_before();
        __syncwarp();
        if (got && lane == 0) mbar_arrive(s_read);
        return got;
      };
      // V of tile j (by warp 5, whose P comes with it); the slots past the last key
      // hold anything, and 0 x NaN is NaN
      auto landed_v = [&](int j) {
        const int i = base + idx_v(j, n_iter), s = i % L::STAGES;
        if (!warp_wait(kv_full(s), (i / L::STAGES) & 1, wc)) return false;
        if (j + 1 == n_iter && last_valid < kTileN) {
          uint8_t* v = gb + L::OFF_KV + s * L::TILE;
          for (int e = last_valid * 8 + lane; e < kTileN * 8; e += 32)  // 16 bytes each
#pragma unroll
            for (int kb = 0; kb < L::KB; ++kb)
              *reinterpret_cast<uint4*>(v + kb * L::BOX + e * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
        }
        return true;
      };
      auto hand_first = [&](int j) {  // P of the first keys, with V
        const bool got = warp != 5 || landed_v(j);
        tc_fence_before();
        __syncwarp();
        if (got && lane == 0) mbar_arrive(p_first(t));
        return got;
      };
      for (int j = 0; j < n_iter; ++j) {
        const uint32_t parity = (tiles + j) & 1;
        bool handed = false;  // P of the first keys
        const TileMask<true, L::CW / 32> mask(a, live, token, sg.n, sg.len, 0,
                                                 (sg.t0 + j * ranks) * kTileN + L::CW * half);
        if (!(ok = warp_wait(s_full(L::OWN_P ? 0 : t), parity, wc))) break;
        tc_fence_after();
        if (warp_live) {
          if (!(ok = check_tmem(ck, ts, 32, 128, __LINE__) && check_tmem(ck, tp, 32, 64, __LINE__))) break;
          constexpr int CW = L::CW;
          float s[CW];
          auto load_s = [&]() {
#pragma unroll
            for (int q = 0; q < CW / 32; ++q) tmem_ld32(ts + 32 * q, *reinterpret_cast<float(*)[32]>(&s[32 * q]));
            tmem_wait_ld();
            if (mask.partial()) {
#pragma unroll
              for (int k = 0; k < CW; ++k)
                if (mask.hides(k)) s[k] = -INFINITY;
            }
          };
          uint32_t p[CW / 2];
          auto terms_of = [&](auto first, auto last) {  // P against ref, in the inputs' type; its fp32 sum
            const float r0 = ref == -INFINITY ? 0.f : ref;
            const float2 c2 = make_float2(c, c), nr = make_float2(-r0, -r0);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int k = first; k < last; ++k) {
              const float2 x = __ffma2_rn(make_float2(s[2 * k], s[2 * k + 1]), c2, nr);
              const float2 e = make_float2(ex2(x.x), ex2(x.y));
              sum[k & 1] = __fadd2_rn(sum[k & 1], e);
              p[k] = pack2<TYPE>(e.x, e.y);
            }
            const float2 f = __fadd2_rn(sum[0], sum[1]);
            return f.x + f.y;
          };
          using std::integral_constant;
          auto terms = [&]() { return terms_of(integral_constant<int, 0>{}, integral_constant<int, CW / 2>{}); };
          // the maximum of the tile moves the reference if it exceeds it by more
          // than is allowed; by how much O and the sum scale then
          auto move_ref = [&](bool may, float* alpha) {
            float m[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int k = 4; k < CW - 4; k += 8) {
#pragma unroll
              for (int i = 0; i < 4; ++i) m[i] = max3(m[i], s[k + 2 * i], s[k + 2 * i + 1]);
            }
            float most = max3(max3(m[0], m[1], m[2]), max3(m[3], s[CW - 4], s[CW - 3]), fmaxf(s[CW - 2], s[CW - 1]));
            if constexpr (L::HALVES == 2) {
              float other;
              if (!swap(most, &other)) return false;
              most = fmaxf(most, other);
            }
            const float top = most * c;
            const bool move = may && (top > ref + rise_allowed<TYPE>(top) || (ref == -INFINITY && top > -INFINITY));
            *alpha = move ? ex2(ref - (top - kBelow<TYPE>)) : 1.f;
            if (move) {
              ref = top - kBelow<TYPE>;
              l *= *alpha;
            }
            return true;
          };
          auto scale_o = [&](float alpha) {  // (all of its products so far have ended)
#pragma unroll
            for (int q = 0; q < D / L::HALVES / 16; ++q) {
              float o[16];
              tmem_ld16(to + 16 * q, o);
              tmem_wait_ld();
              uint32_t r[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) r[k] = __float_as_uint(o[k] * alpha);
              tmem_st16(to + 16 * q, r);
            }
          };
          float f, alpha;
          load_s();
          if constexpr (L::OWN_P) {
            // S is in registers: the next tile's may come. P's columns and O are
            // touched once the product of the tile before has ended
            if (!(ok = hand_back_s(j) && move_ref(true, &alpha))) break;
            f = terms();
            if (j > 0) {
              if (!(ok = warp_wait(p_read, (reads + j - 1) & 1, wc))) break;
              tc_fence_after();
              if (__any_sync(0xFFFFFFFFu, alpha != 1.f)) scale_o(alpha);
            }
          } else {
            // Terms against the reference as it is, while their sum stays within
            // kSumMax; else (and in a row's first tile) the maximum is taken. The
            // products of the tiles before ended before this S. P of the first
            // keys is handed over while the others' is made
            f = terms_of(integral_constant<int, 0>{}, integral_constant<int, kFirst / 2>{});
            bool again = !(f <= kSumMax<TYPE>) || (ref == -INFINITY && mask.some());
            if (__any_sync(0xFFFFFFFFu, again)) {
              load_s();
              move_ref(true, &alpha);
              if (j > 0) scale_o(alpha);
              f = terms();
            } else {
#pragma unroll
              for (int q = 0; q < kFirst / 32; ++q) tmem_st16(tp + 16 * q, &p[16 * q]);
              tmem_wait_st();
              if (!hand_first(j)) {
                ok = false;
                break;
              }
              handed = true;
              float f2 = terms_of(integral_constant<int, kFirst / 2>{}, integral_constant<int, 64>{});
              again = !(f2 <= kSumMax<TYPE>);
              if (__any_sync(0xFFFFFFFFu, again)) {  // the others' maximum; the first keys are in O by then
                if (!(ok = warp_wait(o_first(t), parity, wc))) break;
                tc_fence_after();
#pragma unroll
                for (int q = kFirst / 32; q < 4; ++q) tmem_ld32(ts + 32 * q, *reinterpret_cast<float(*)[32]>(&s[32 * q]));
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 128; ++k)
                  if (k < kFirst || mask.hides(k)) s[k] = -INFINITY;
                l += f;
                f = 0.f;
                move_ref(again, &alpha);
                scale_o(alpha);
                f2 = terms_of(integral_constant<int, kFirst / 2>{}, integral_constant<int, 64>{});
              }
              f += f2;
            }
          }
          constexpr int kLate = L::OWN_P ? 0 : kFirst / 32;  // handed over with the rest
          if (!handed) {
#pragma unroll
            for (int q = 0; q < kLate; ++q) tmem_st16(tp + 16 * q, &p[16 * q]);
          }
#pragma unroll
          for (int q = kLate; q < CW / 32; ++q) tmem_st16(tp + 16 * q, &p[16 * q]);
          l += f;
          tmem_wait_st();
        } else if (L::OWN_P) {
          // a warp without rows keeps step: it must not arrive for this tile's P
          // while the others still owe the last one's
          if (!(ok = hand_back_s(j) && (j == 0 || warp_wait(p_read, (reads + j - 1) & 1, wc)))) break;
        }
        // P is handed over together with the loads that its products need, V of
        // this tile and (if S was not) K of the next
        if (!L::OWN_P && !handed) {
          if (!(ok = hand_first(j))) break;
        }
        if (warp == 5) {
          ok = L::OWN_P ? landed_v(j) : j + 1 == n_iter || landed_k(j + 1);
          if (!ok) break;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(p_full(L::OWN_P ? 0 : t));
          // S of this tile came from K's stage, the product of the V before it
          // has ended: both are free
          if ((warp & 3) == 0 && half == 0) {
            if (j > 0) mbar_arrive(kv_empty((base + idx_v(j - 1, n_iter)) % L::STAGES));
            mbar_arrive(kv_empty((base + idx_k(j)) % L::STAGES));
          }
        }
        if (L::QBUFS == 2 && j == 0 && after.n_iter > 0) {
          copy_async_wait();
          give_q(it + 1);
        }
      }
      if (!ok) break;
      // ---------------------------------------------------------- output
      // With one place for Q the next item's rows are on their way meanwhile
      uint4 next_q[LPR];
      if (L::QBUFS == 1) {
        if (!(ok = take_seg(it + 1, after, false))) break;
        fetch_q(after, next_q);
      }
      if (!(ok = warp_wait(o_full(L::OWN_P ? 0 : t), it & 1, wc))) break;
      if (CLUSTER && !L::OWN_P && NT == 2 && !(ok = warp_wait(o_full(1 - t), it & 1, wc))) break;  // (the ring is free)
      tc_fence_after();
      if ((warp & 3) == 0 && half == 0 && lane == 0) mbar_arrive(kv_empty((base + idx_v(n_iter - 1, n_iter)) % L::STAGES));
      if (warp_live) {
        if constexpr (L::HALVES == 2) {
          float other;
          if (!(ok = swap(l, &other))) break;
          l += other;
        }
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;  // (NaN stays NaN)
        const bool none = l == 0.f;
        const long long e = static_cast<long long>(token) * a.HQ + head;
        const long long part = static_cast<long long>(sg.slot) * kRows + t * kTileM + r_tile;
        // The rows go out through shared memory (this warp's part of Q's tile,
        // which no product reads any more), 128 bytes of each at a time, so that
        // eight lanes write a row's line together
        const uint32_t stage =
            sb + L::OFF_Q + (it % L::QBUFS * NT + t) * L::TILE + half * L::BOX + (warp & 3) * 32 * 128;
        const bool parts = sg.slot >= 0;
        uint8_t* mine = !live  ? nullptr
                        : parts ? reinterpret_cast<uint8_t*>(a.part_o + part * D)
                                : reinterpret_cast<uint8_t*>(static_cast<uint16_t*>(a.o) + token * a.o_sn + head * a.o_sh);
        uint8_t* row_out[8];  // of the rows that this lane writes a piece of
#pragma unroll
        for (int i = 0; i < 8; ++i) row_out[i] = shfl_ptr(mine, 4 * i + (lane >> 3));
        auto write_out = [&](int byte) {  // 128 bytes of each row from this one on
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 3);
            uint4 v;
            ld_shared_v4(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4), v.x, v.y, v.z, v.w);
            if (row_out[i] != nullptr) *reinterpret_cast<uint4*>(row_out[i] + byte + (lane & 7) * 16) = v;
          }
          __syncwarp();
        };
        // (a row that saw no key holds 0 times whatever V's rows are)
        const bool any_none = __any_sync(0xFFFFFFFFu, none);
        const float2 inv2 = make_float2(inv, inv);
#pragma unroll
        for (int q = 0; q < D / L::HALVES / 32; ++q) {
          float o[32];
          tmem_ld32(to + 32 * q, o);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            const float2 x = __fmul2_rn(make_float2(o[k], o[k + 1]), inv2);
            o[k] = x.x, o[k + 1] = x.y;
          }
          if (any_none) {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = none ? 0.f : o[k];
          }
          if (CLUSTER && parts) {
            // over the ring, which nothing uses any more: a row's 16-byte pieces turned
            // by its number
            const int piece = (D / L::HALVES * half + 32 * q) / 4;
            if (live) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                st_shared_v4(sb + L::OFF_KV + ((t * kTileM + r_tile) * (D / 4) + ((piece + k) ^ (lane & 7))) * 16,
                             __float_as_uint(o[4 * k]), __float_as_uint(o[4 * k + 1]), __float_as_uint(o[4 * k + 2]),
                             __float_as_uint(o[4 * k + 3]));
            }
          } else if (parts) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              st_shared_v4(stage + lane * 128 + ((k ^ (lane & 7)) << 4), __float_as_uint(o[4 * k]),
                           __float_as_uint(o[4 * k + 1]), __float_as_uint(o[4 * k + 2]), __float_as_uint(o[4 * k + 3]));
            write_out(D / L::HALVES * 4 * half + 128 * q);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              st_shared_v4(stage + lane * 128 + (((4 * (q & 1) + k) ^ (lane & 7)) << 4),
                           pack2<TYPE>(o[8 * k], o[8 * k + 1]), pack2<TYPE>(o[8 * k + 2], o[8 * k + 3]),
                           pack2<TYPE>(o[8 * k + 4], o[8 * k + 5]), pack2<TYPE>(o[8 * k + 6], o[8 * k + 7]));
            if (q & 1) write_out(D / L::HALVES * 2 * half + 64 * (q - 1));
          }
        }
        if (live && half == 0) {
          const float lse2 = none ? -INFINITY : ref + log2f(l);
          if (CLUSTER && parts)
            st_shared_f32(sb + L::OFF_KV + (kRows * D + t * kTileM + r_tile) * 4, lse2);
          else if (parts)
            a.part_lse[part] = lse2;
          else
            a.lse[e] = lse2 * kLn2;
        }
      }
      if (L::QBUFS == 1 && after.n_iter > 0) put_q(next_q, it + 1);
      base += 2 * n_iter;
      tiles += n_iter;
      reads += n_iter - 1;
      sg = after;
    }
    if constexpr (CLUSTER) {
      static_assert(kRows * (D + 1) * 4 <= L::STAGES * L::TILE, "parts lie in the ring");
      const int parts = min(ranks, one_tiles), at = rank * L::WARPS + warp - 4;
      cluster_sync();
      if (parts > 1 && !*skip_flag) {
        if (parts <= 4)
          join_cluster<TYPE, D, 4>(a, sb + L::OFF_KV, kRows, parts, at, ranks * L::WARPS, one_rows, one_rb * kRows, one_tok0, one_hk);
        else
          join_cluster<TYPE, D, 16>(a, sb + L::OFF_KV, kRows, parts, at, ranks * L::WARPS, one_rows, one_rb * kRows, one_tok0, one_hk);
      }
      cluster_sync();  // (this CTA's part may still be read)
    }
  }

  grid_launch_dependents();  // the join kernel may be launched
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::TMEM);
  }
}

// Join the parts of an item that the CTAs' stretches cut, one warp a row: blocks
// (c, ..) take the item that starts in CTA c's stretch and goes on in the next, as
// that CTA has written it down; the parts lie in the slots of consecutive CTAs.
template <int TYPE, int D, int NT>
__global__ void __launch_bounds__(32 * kJoinWarps)
    streamkl_paged_tree_join_kernel(const __grid_constant__ TreeAttnArgs a) {
  constexpr int V = D / 32;  // columns of a lane
  constexpr int kRows = kTileM * NT;
  grid_dependency_wait();  // launched while the tree kernel ends
  const int c0 = static_cast<int>(blockIdx.x);
  const TreeCut cut = a.cuts[c0];
  const int lane = threadIdx.x & 31, r = static_cast<int>(blockIdx.y) * kJoinWarps + static_cast<int>(threadIdx.x >> 5);
  if (r >= cut.rows) return;
  auto slot = [&](int i) { return static_cast<long long>(2 * (c0 + i) + (i == 0 ? cut.inside : 0)) * kRows + r; };
  constexpr int RUN = 8;  // parts whose loads are in flight, the first ones beside the lse's
  float p[RUN][V];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
#pragma unroll
      for (int x = 0; x < V; ++x) p[i][x] = 0.f;
      if (i0 + i < cut.parts) {
        const float* src = a.part_o + slot(i0 + i) * D + lane * V;
        if constexpr (V == 4)
          *reinterpret_cast<float4*>(p[i]) = *reinterpret_cast<const float4*>(src);
        else
          *reinterpret_cast<float2*>(p[i]) = *reinterpret_cast<const float2*>(src);
      }
    }
  };
  fetch(0);
  float top = -INFINITY;
  for (int i = lane; i < cut.parts; i += 32) top = fmaxf(top, a.part_lse[slot(i)]);
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
  const float t0 = top == -INFINITY ? 0.f : top;
  float sum = 0.f, o[V] = {};
  for (int i0 = 0; i0 < cut.parts; i0 += RUN) {
    if (i0 > 0) fetch(i0);
    const float mine = lane < RUN && i0 + lane < cut.parts ? ex2(a.part_lse[slot(i0 + lane)] - t0) : 0.f;
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
      const float w = __shfl_sync(0xFFFFFFFFu, mine, i);  // 0 past the last part
      sum += w;
#pragma unroll
      for (int x = 0; x < V; ++x) o[x] = fmaf(w, p[i][x], o[x]);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int G = a.HQ / a.HK, row = cut.row0 + r, token = cut.tok0 + row / G, head = cut.hk * G + row % G;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + token * a.o_sn + head * a.o_sh + lane * V);
#pragma unroll
  for (int x = 0; x < V / 2; ++x) dst[x] = pack2<TYPE>(o[2 * x] * inv, o[2 * x + 1] * inv);
  if (lane == 0) a.lse[static_cast<long long>(token) * a.HQ + head] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

template <int TYPE, int D, int NT, bool CLUSTER>
cudaError_t tree_t(const TreeAttnArgs& a, int ctas, cudaStream_t stream) {
  using L = TreeLayout<D, NT>;
  auto kern = streamkl_paged_tree_kernel<TYPE, D, NT, CLUSTER>;
  // the shared-memory attribute, once per device
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (!(done.load() & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
    if (e != cudaSuccess) return e;
    if (CLUSTER && (e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
      return e;
    done.fetch_or(bit);
  }
  if constexpr (CLUSTER) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(L::THREADS);
    cfg.dynamicSmemBytes = L::BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(a.cluster);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, *a.tm_k, *a.tm_v, a);
  }
  kern<<<ctas, L::THREADS, L::BYTES, stream>>>(*a.tm_k, *a.tm_v, a);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.whole) return e;
  const long long most = std::min<long long>(static_cast<long long>(a.max_q) * (a.HQ / a.HK), kTileM * NT);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), static_cast<unsigned>((most + kJoinWarps - 1) / kJoinWarps));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, streamkl_paged_tree_join_kernel<TYPE, D, NT>, a);
}

template <int TYPE, int D>
cudaError_t tree_d(const TreeAttnArgs& a, int ctas, cudaStream_t stream) {
  if (a.cluster > 0)
    return a.row_tiles == 2 ? tree_t<TYPE, D, 2, true>(a, ctas, stream) : tree_t<TYPE, D, 1, true>(a, ctas, stream);
  return a.row_tiles == 2 ? tree_t<TYPE, D, 2, false>(a, ctas, stream) : tree_t<TYPE, D, 1, false>(a, ctas, stream);
}

}  // namespace

cudaError_t launch_tree(const TreeAttnArgs& a, int ctas, cudaStream_t stream) {
  if (a.type == kTypeBf16)
    return a.d == 128 ? tree_d<kTypeBf16, 128>(a, ctas, stream) : tree_d<kTypeBf16, 64>(a, ctas, stream);
  return a.d == 128 ? tree_d<kTypeF16, 128>(a, ctas, stream) : tree_d<kTypeF16, 64>(a, ctas, stream);
}

}  // namespace skl
