// Attention of new tokens over a paged cache: for query row i of a sequence
// (its last n tokens), o_i = sum_j p_ij v_j with p = softmax(scale q K^T) over
// the keys j it sees (causal: j <= len - n + i), and lse_i for merging.
//
// Rows. The G = HQ / HK query heads of a key head read the same keys, so a row
// tile packs (token, head of the group) pairs, row r = token r / G, head r % G:
// a single new token of a grouped model is G rows of one tile and the keys are
// read once for all of them.
//
// One pass over the key tiles (128 keys) with the running reference and sum
// of the softmax, S = Q K^T and O += P V as tcgen05 MMAs:
//   S (fp32, TMEM) -> registers -> P = 2^(c s - ref) in the inputs' type (TMEM,
//   the PV product's A operand).
// P has 8 (bf16) or 11 (fp16) bits: its rounding is the size of the output's
// own (fp16's small terms: kBelow). ref, the sum (of unrounded terms) and O are
// fp32. The reference moves only when terms would exceed 2^8 of it (2^14, fp16),
// so that O need not be rescaled at every rise; the results do not depend on it.
// (At d = 128 with two row tiles, and in paged_decode.cu, where a tile's sum
// exceeds that but no term does, its terms are made twice and the reference
// stays: scores 3 to 4 nats higher from the second tile on take every tile that
// way, 813 us for the 689 of level ones at the 131,072 keys below.)
//
// CTA: warp 0 loads (at d = 128 K, and warp 2 V; each lane one page's box of a
// tile; pages are found through the block table), warp 1 issues MMAs, warps 4..
// are one softmax warpgroup per row tile, thread = row. Two row tiles (NT = 2)
// share each K and V tile. At d = 128 their O fill half of TMEM and P has to take
// S's place: the tiles alternate, the tensor pipe works on one while the other's
// softmax runs. At d = 64, or with one row tile, P has columns of its own and the next
// S is made while this one's terms are.
//
// At d = 128 512 rows x 32 heads against 131,072 keys take 0.68 ms, 1.62 PFLOP/s,
// one call alone (0.73 ms, 1.5 PFLOP/s, call after call under the power cap):
// about 2,800 cycles a turn (a key tile for both row tiles), of which the 32
// products take 2,048 back to back, as the 256 KB of operands and loads at 128
// bytes a cycle do; a row tile's own chain, S, terms, P, PV, is what is left. P of
// the first 96 keys is handed over before the others' terms are made (685 us with
// 64, 704 whole).
// Tried and not faster: two softmax warpgroups per row tile (936 us), an issuing
// thread per row tile (765 us), L2 prefetches (738 us). At d = 64 the terms are
// half of a turn: 2,700 cycles, the exponentials alone 1,024, the products 1,050.
//
// With few query tiles the keys are split over CTAs and a combine kernel joins
// the splits by their lse.
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
constexpr int kFirst = 96;   // keys of a tile whose P is handed over first (d = 128, two row tiles)

template <int D, int NT>
struct AttnLayout {
  static constexpr int KB = D / 64;               // 64-column (128-byte) boxes per row
  static constexpr int BOX = kTileN * 128;        // 128 rows of one box
  static constexpr int TILE = kTileN * D * 2;
  static constexpr int STAGES = D == 128 ? (NT == 2 ? 5 : 6) : (NT == 2 ? 10 : 12);
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = NT * TILE;
  static constexpr int OFF_BAR = OFF_KV + STAGES * TILE;
  // P in columns of its own, where TMEM has room for them
  static constexpr bool OWN_P = D == 64 || NT == 1;
  // Warps that load. Each box is an instruction of its own: with 16-slot pages one
  // warp takes longer over K and V of 128 columns than the rest takes (16 tokens x
  // 4 heads over 4,096 keys in one CTA a key head 56 us, 39 with one warp for each;
  // 64 tokens 61 and 56; at d = 64 50.1 and 51.6, a warp's share of the issue slots)
  static constexpr int LOADERS = D == 128 ? 2 : 1;
  // q_full, v_fixed, kv_full[S], kv_empty[S], s_full[2], p_full[2], o_full[2],
  // s_read, p_read, drain, p_first[2], o_first[2]
  static constexpr int NBAR = 2 + 2 * STAGES + 13;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int BYTES = OFF_MISC + 16;
  static_assert(BYTES <= 232448, "shared memory budget");
  static constexpr int THREADS = 128 + 128 * NT;
  static constexpr int col_s(int t) { return 128 * t; }
  static constexpr int col_p(int t) { return OWN_P ? 128 * NT + 64 * t : 128 * t; }
  static constexpr int col_o(int t) { return (OWN_P ? 192 : 128) * NT + D * t; }
  static_assert(col_o(NT - 1) + D <= 512, "TMEM columns");
};

// What a CTA works on: one sequence's rows of one key head, a range of keys.
struct Work {
  int n, len;          // new tokens, length
  int tok0;            // first token of the sequence
  int rows;            // rows of the sequence: n * G
  int row0;            // first row of this CTA
  int t0, n_iter;      // key tiles [t0, t0 + n_iter)
  int klim;            // keys any row of this CTA sees: [0, klim)
  bool ok;             // the sequence's numbers are sound
};

__device__ __forceinline__ Work find_work(const PagedAttnArgs& a, int b, int G, int rows_cta) {
  Work w;
  const int c0 = a.cu != nullptr ? __ldg(a.cu + b) : b;
  const int c1 = a.cu != nullptr ? __ldg(a.cu + b + 1) : b + 1;
  w.len = __ldg(a.kv_lens + b);
  w.n = c1 - c0;
  w.tok0 = c0;
  w.ok = c0 >= 0 && c1 >= c0 && c1 <= a.T && w.n <= a.max_q && w.len >= 0 && w.len <= a.max_kv;
  w.rows = w.ok ? w.n * G : 0;
  // the last rows see the most keys: their tiles first
  const int tiles = (w.rows + rows_cta - 1) / rows_cta;
  const int x = a.causal ? tiles - 1 - static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x);
  w.row0 = x >= 0 && x < tiles ? x * rows_cta : w.rows;  // no rows: nothing to do
  const int last = min(w.rows, w.row0 + rows_cta) - 1;
  w.klim = a.causal && w.rows > 0 ? min(w.len, w.len - w.n + last / G + 1) : w.len;
  const int n_tiles = (max(0, w.klim) + kTileN - 1) / kTileN;
  w.t0 = min(n_tiles, static_cast<int>(blockIdx.y) * a.split_tiles);
  w.n_iter = min(n_tiles, w.t0 + a.split_tiles) - w.t0;
  return w;
}

// Lane `from`'s pointer.
template <typename T>
__device__ __forceinline__ T* shfl_ptr(T* p, int from) {
  return reinterpret_cast<T*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(p), from));
}

// One row of the output: finished (o, lse) or a split's partial.
template <int TYPE, int D>
__device__ __forceinline__ void store_empty_row(const PagedAttnArgs& a, int token, int head) {
  const long long e = static_cast<long long>(token) * a.HQ + head;
  if (a.splits > 1) {
    a.part_lse[static_cast<long long>(blockIdx.y) * a.T * a.HQ + e] = -INFINITY;
    return;
  }
  uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + token * a.o_sn + head * a.o_sh);
#pragma unroll
  for (int i = 0; i < D / 8; ++i) o[i] = make_uint4(0, 0, 0, 0);
  a.lse[e] = -INFINITY;
}

template <int TYPE, int D, int NT>
__global__ void __launch_bounds__(AttnLayout<D, NT>::THREADS, 1)
    streamkl_paged_attn_kernel(const __grid_constant__ CUtensorMap tm_k,
                               const __grid_constant__ CUtensorMap tm_v,
                               const __grid_constant__ PagedAttnArgs a) {
  using L = AttnLayout<D, NT>;
  extern __shared__ __align__(1024) uint8_t gb[];
  const uint32_t sb = smem_u32(gb);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.HQ / a.HK;
  int b = static_cast<int>(blockIdx.z) / a.HK;
  const int hk = static_cast<int>(blockIdx.z) - b * a.HK;
  if (a.by_length) {  // (at most 32 sequences) the b-th longest
    const int len = lane < a.B ? __ldg(a.kv_lens + lane) : INT_MIN;
    int rank = 0;
#pragma unroll 8
    for (int i = 0; i < 32; ++i) {
      const int other = __shfl_sync(0xFFFFFFFFu, len, i);
      rank += other > len || (other == len && i < lane);
    }
    b = __ffs(__ballot_sync(0xFFFFFFFFu, rank == b)) - 1;
  }
  const Work w = find_work(a, b, G, kTileM * NT);
  if (!w.ok && threadIdx.x == 0) atomicCAS(a.dev_status, 0, kStatusInvalidArg);
  if (w.row0 >= w.rows) return;
  if (w.n_iter == 0) {  // no key in this range is seen
    for (int r = w.row0 + threadIdx.x; r < min(w.rows, w.row0 + kTileM * NT); r += blockDim.x)
      store_empty_row<TYPE, D>(a, w.tok0 + r / G, hk * G + r % G);
    return;
  }

  // row tiles of this CTA that have rows
  const int nt = (NT == 2 && w.rows - w.row0 > kTileM) ? 2 : 1;
  const uint32_t bar0 = sb + L::OFF_BAR;
  const uint32_t q_full = bar0, v_fixed = bar0 + 8;
  auto kv_full = [&](int s) { return bar0 + 8u * (2 + s); };
  auto kv_empty = [&](int s) { return bar0 + 8u * (2 + L::STAGES + s); };
  auto s_full = [&](int k) { return bar0 + 8u * (2 + 2 * L::STAGES + k); };
  auto p_full = [&](int k) { return bar0 + 8u * (4 + 2 * L::STAGES + k); };
  auto o_full = [&](int k) { return bar0 + 8u * (6 + 2 * L::STAGES + k); };
  const uint32_t s_read = bar0 + 8u * (8 + 2 * L::STAGES), p_read = s_read + 8, drain = s_read + 16;
  auto p_first = [&](int k) { return bar0 + 8u * (11 + 2 * L::STAGES + k); };
  auto o_first = [&](int k) { return bar0 + 8u * (13 + 2 * L::STAGES + k); };
  static_assert(15 + 2 * L::STAGES == L::NBAR, "barrier region holds every barrier");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gb + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gb + L::OFF_MISC + 4);
  volatile int* skip_flag = reinterpret_cast<volatile int*>(gb + L::OFF_MISC + 8);

  CheckCtx ck{sb, sb + L::OFF_BAR, sb + L::OFF_BAR, sb + L::OFF_BAR + L::NBAR * 8, 0, 0,
              abort_flag, a.dev_status};
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    bool lay_ok = (sb & 1023u) == 0;  // the swizzled tiles' alignment
    if (!lay_ok) atomicCAS(a.dev_status, 0, kStatusDeviceCheck);
    if (kDeviceChecks)
      for (int i = 0; i < L::NBAR; ++i) lay_ok = lay_ok && check_bar(ck, bar0 + 8u * i, __LINE__);
    if (lay_ok) {
      mbar_init(q_full, 4 * NT);  // one arrival per softmax warp
      mbar_init(v_fixed, 1);
      for (int s = 0; s < L::STAGES; ++s) {
        mbar_init(kv_full(s), 1);
        mbar_init(kv_empty(s), nt);
      }
      for (int k = 0; k < 2; ++k) {
        mbar_init(s_full(k), 1);
        mbar_init(p_full(k), L::OWN_P ? 4 * nt : 4);
        mbar_init(o_full(k), 1);
        mbar_init(p_first(k), 4);
        mbar_init(o_first(k), 1);
      }
      mbar_init(s_read, 4 * nt);
      mbar_init(p_read, 1);
      mbar_init(drain, 1);
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
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);  // (the same in every lane)
  ck.tmem = tmem;
  ck.tmem_cols = 512;
  const WaitCtx wc{abort_flag, a.dev_status, a.timeout_ns};
  const int n_iter = *skip_flag ? 0 : w.n_iter;
  // keys of the last tile that are there; the rest of its V rows are cleared
  const int last_valid = min(kTileN, w.klim - (w.t0 + w.n_iter - 1) * kTileN);

  // Place of key tile j's K and V among the loads, in the order in which the
  // MMAs use them: K0 V0 K1 V1 .., with P in columns of its own K0 K1 V0 K2 V1 ..
  auto idx_k = [&](int j) { return !L::OWN_P ? 2 * j : (j == 0 ? 0 : 2 * j - 1); };
  auto idx_v = [&](int j) { return !L::OWN_P ? 2 * j + 1 : (j + 1 < w.n_iter ? 2 * j + 2 : 2 * j + 1); };

  if (warp < 4) {
  // NT = 2: 128 threads with 88 registers and 256 with 208 make up the launch's
  // 384 x 168; a softmax thread holds a row of S (128)
  if (NT == 2) regs_dec<88>();
  if (warp == 0 || (L::LOADERS == 2 && warp == 2)) {
    // ------------------------------------------------- loads, of K, V or both
    const int page = 1 << a.page_shift;
    const int box_rows = min(page, kTileN);
    const int* table = a.table + static_cast<long long>(b) * a.table_sb;
    const bool has_v = L::LOADERS == 1 || warp == 2;
    int loads = 0;  // issued
    bool ok = true;
    // the page this lane loads of tile j; a number that is none is reported
    // and page 0 read in its place
    auto page_of = [&](int j) {
      const int key = (w.t0 + j) * kTileN + lane * box_rows;
      if (j >= n_iter || lane * box_rows >= kTileN || key >= w.klim) return -1;
      int p = __ldg(table + (key >> a.page_shift));
      if (p < 0 || p >= a.num_pages) {
        atomicCAS(a.dev_status, 0, kStatusInvalidArg);
        p = 0;
      }
      return p;
    };
    auto load = [&](const CUtensorMap* map, int i, int j, int pg) {
      // The stage's barrier cannot be two phases behind what is waited for: loads
      // are used in their order, so when this warp's one before this had its
      // stage, all that lie a ring and more back from there had been used
      const int s = i % L::STAGES;
      if (!warp_wait(kv_empty(s), ((i / L::STAGES) & 1) ^ 1, wc)) return false;
      const int key0 = (w.t0 + j) * kTileN;
      const int pages = (min(kTileN, w.klim - key0) + box_rows - 1) / box_rows;
      const uint32_t dst = sb + L::OFF_KV + s * L::TILE + lane * box_rows * 128;
      if (lane == 0) mbar_arrive_expect_tx(kv_full(s), static_cast<uint32_t>(pages * box_rows * D * 2));
      __syncwarp();
      if (lane < pages) {
        const int slot = key0 & (page - 1);  // 0 below 128-slot pages
#pragma unroll
        for (int kb = 0; kb < L::KB; ++kb)
          if (check_tma(ck, dst + kb * L::BOX, box_rows * 128, kv_full(s), kb * 64, D, slot, page, 0, hk,
                        a.HK, __LINE__))
            tma_load_4d(dst + kb * L::BOX, map, kv_full(s), kb * 64, slot, hk, pg);
      }
      ++loads;
      return true;
    };
    int pg = page_of(0), pg_next = page_of(1);
    if (L::LOADERS == 1) {
      static_assert(L::LOADERS == 2 || L::OWN_P, "K0 K1 V0 K2 V1 ..");
      if (n_iter > 0) ok = load(&tm_k, 0, 0, pg);
      for (int j = 0; ok && j < n_iter; ++j) {
        if (j + 1 < n_iter) ok = load(&tm_k, idx_k(j + 1), j + 1, pg_next);
        if (ok) ok = load(&tm_v, idx_v(j), j, pg);
        pg = pg_next;
        pg_next = page_of(j + 2);
      }
    } else {
      for (int j = 0; ok && j < n_iter; ++j) {
        ok = has_v ? load(&tm_v, idx_v(j), j, pg) : load(&tm_k, idx_k(j), j, pg);
        pg = pg_next;
        pg_next = page_of(j + 2);
      }
    }
    // the last tile's V: clear its rows past the last key (the slots there hold
    // anything, and 0 x NaN is NaN)
    if (has_v && ok && n_iter > 0 && last_valid < kTileN) {
      const int i = idx_v(n_iter - 1);
      if (warp_wait(kv_full(i % L::STAGES), (i / L::STAGES) & 1, wc)) {
        uint8_t* v = gb + L::OFF_KV + (i % L::STAGES) * L::TILE;
        for (int e = last_valid * 8 + lane; e < kTileN * 8; e += 32)  // 16 bytes each
#pragma unroll
          for (int kb = 0; kb < L::KB; ++kb)
            *reinterpret_cast<uint4*>(v + kb * L::BOX + e * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_fixed);
      }
    }
    // let every copy land before the CTA can exit: this warp's last in the ring
    // (a stage that was used again, its copy had landed)
    for (int j = max(0, loads - (L::STAGES + L::LOADERS - 1) / L::LOADERS); j < loads; ++j) {
      const int i = L::LOADERS == 1 ? j : has_v ? idx_v(j) : idx_k(j);
      if (!ok || i >= 2 * n_iter - L::STAGES) wait_drain(kv_full(i % L::STAGES), (i / L::STAGES) & 1, a.timeout_ns);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs
    // One thread issues every product, so its own instructions count: it waits
    // for P and S only (with them come the loads), the stages are released by
    // the softmax warps, and its branch is taken under elect.sync (729 -> 710 us
    // at the 131,072 keys above).
    if (n_iter > 0 && elect_one()) {
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
      auto landed = [&]() {
        const bool got = wait_bounded(kv_full(ring.stage), ring.phase, wc);
        tc_fence_after();
        return got;
      };
      auto mma_s = [&](uint32_t q, uint32_t k, uint32_t col) {  // S = Q_t K_j^T
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint32_t off = ((i >> 2) * L::BOX + (i & 3) * 32) >> 4;
          mma_bf16(tmem + col, desc(q + off), desc(k + off), id_s, i > 0);
        }
      };
      auto mma_o = [&](uint32_t v, uint32_t col_p, uint32_t col_o, uint32_t add) {  // O_t += P V_j
#pragma unroll
        for (int i = 0; i < kTileN / 16; ++i)
          mma_bf16_ts(tmem + col_o, tmem + col_p + 8 * i, desc(v + i * (2048 >> 4)), id_o, i > 0 ? 1 : add);
      };
      // of the first keys, or of the others
      auto mma_o_part = [&](int part, uint32_t v, uint32_t col_p, uint32_t col_o, uint32_t add) {
#pragma unroll
        for (int k = part ? kFirst / 16 : 0; k < (part ? kTileN : kFirst) / 16; ++k)
          mma_bf16_ts(tmem + col_o, tmem + col_p + 8 * k, desc(v + k * (2048 >> 4)), id_o, k > 0 ? 1 : add);
      };
      bool ok = check_tmem(ck, tmem, 128, 512, __LINE__) && wait_bounded(q_full, 0, wc) && landed();
      uint32_t k_at = next();
      auto both_s = [&]() {
        mma_s(q_lo, k_lo + k_at, L::col_s(0));
        if (!L::OWN_P && nt == 2) mma_commit(s_full(0));
        if (nt == 2) mma_s(q_lo + (L::TILE >> 4), k_lo + k_at, L::col_s(1));
        mma_commit(s_full(L::OWN_P ? 0 : nt - 1));
      };
      if (ok) both_s();
#pragma unroll 1
      for (int j = 0; ok && j < n_iter; ++j) {
        const bool more = j + 1 < n_iter;
        if (!L::OWN_P) {
          // P of row tile 0 comes with V of this tile and K of the next
          const uint32_t v_at = next();
          if (more) k_at = next();
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            if (t == nt) break;
            if (!(ok = wait_bounded(p_first(t), j & 1, wc))) break;
            tc_fence_after();
            mma_o_part(0, v_lo + v_at, L::col_p(t), L::col_o(t), j > 0);
            mma_commit(o_first(t));
            if (!(ok = wait_bounded(p_full(t), j & 1, wc))) break;
            tc_fence_after();
            mma_o_part(1, v_lo + v_at, L::col_p(t), L::col_o(t), 1);
            if (more) mma_s(q_lo + t * (L::TILE >> 4), k_lo + k_at, L::col_s(t));
            mma_commit(more ? s_full(t) : o_full(t));
          }
          if (!ok) break;
        } else {
          // S comes back with K of the next tile, P with V of this one
          if (more) {
            k_at = next();
            if (!(ok = wait_bounded(s_read, j & 1, wc))) break;
            tc_fence_after();
            both_s();
          }
          const uint32_t v_at = next();
          if (!(ok = wait_bounded(p_full(0), j & 1, wc))) break;
          tc_fence_after();
          mma_o(v_lo + v_at, L::col_p(0), L::col_o(0), j > 0);
          if (nt == 2) mma_o(v_lo + v_at, L::col_p(1), L::col_o(1), j > 0);
          mma_commit(more ? p_read : o_full(0));
        }
      }
      mma_commit(drain);
      wait_drain(drain, 0, a.timeout_ns);
    }
  }
  } else {
    // ------------------------------------------------------------ softmax
    if (NT == 2) regs_inc<208>();
    const int t = (warp - 4) >> 2;                    // row tile
    const int r_tile = (warp & 3) * 32 + lane;        // TMEM lane
    const int row = w.row0 + t * kTileM + r_tile;     // row of the sequence
    const bool live = row < w.rows;
    const int tok = live ? row / G : 0;
    const int token = w.tok0 + tok, head = hk * G + (live ? row - tok * G : 0);
    if (n_iter > 0) {
      // this warp's rows of Q, D / 8 lanes a row, 128-byte swizzled as TMA would
      // place them; rows that are not there are zero
      constexpr int LPR = D / 8, RPI = 32 / LPR;
      const int cq = lane % LPR;
      const uint16_t* mine = live ? static_cast<const uint16_t*>(a.q) + token * a.q_sn + head * a.q_sh : nullptr;
      uint4 v[LPR];
#pragma unroll
      for (int i = 0; i < LPR; ++i) {
        const uint16_t* row_q = shfl_ptr(mine, i * RPI + lane / LPR);
        v[i] = make_uint4(0, 0, 0, 0);
        if (row_q != nullptr) v[i] = __ldg(reinterpret_cast<const uint4*>(row_q) + cq);
      }
#pragma unroll
      for (int i = 0; i < LPR; ++i) {
        const int r = (warp & 3) * 32 + i * RPI + lane / LPR;
        st_shared_v4(sb + L::OFF_Q + t * L::TILE + (cq >> 3) * L::BOX + r * 128 + (((cq & 7) ^ (r & 7)) << 4), v[i].x,
                     v[i].y, v[i].z, v[i].w);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    const float c = a.scale * kLog2e;
    // keys < lim are seen by this row
    const int lim = !live ? 0 : a.causal ? min(w.len, w.len - w.n + tok + 1) : w.len;
    const bool warp_live = w.row0 + t * kTileM + (warp & 3) * 32 < w.rows;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t to = tmem + L::col_o(t) + lanes;
    float ref = -INFINITY, l = 0.f;
    bool ok = true;
    auto landed_k = [&](int j) {
      const int i = idx_k(j);
      return warp_wait(kv_full(i % L::STAGES), (i / L::STAGES) & 1, wc);
    };
    auto hand_back_s = [&](int j) {  // S has been read; K of the next tile comes with it
      const bool got = warp != 6 || j + 1 == n_iter || landed_k(j + 1);
      tc_fence_before();
      __syncwarp();
      if (got && lane == 0) mbar_arrive(s_read);
      return got;
    };
    auto landed_v = [&](int j) {
      const int i = idx_v(j);
      return warp_wait(kv_full(i % L::STAGES), (i / L::STAGES) & 1, wc) &&
             // (the last tile's rows past the last key are cleared first)
             (j + 1 < n_iter || last_valid == kTileN || warp_wait(v_fixed, 0, wc));
    };
    auto hand_first = [&](int j) {  // P of the first keys, with V
      const bool got = warp != 5 || landed_v(j);
      tc_fence_before();
      __syncwarp();
      if (got && lane == 0) mbar_arrive(p_first(t));
      return got;
    };
    for (int j = 0; t < nt && j < n_iter; ++j) {
      bool handed = false;  // P of the first keys
      if (!(ok = warp_wait(s_full(L::OWN_P ? 0 : t), j & 1, wc))) break;
      tc_fence_after();
      if (warp_live) {
        const uint32_t ts = tmem + L::col_s(t) + lanes, tp = tmem + L::col_p(t) + lanes;
        if (!(ok = check_tmem(ck, ts, 32, 128, __LINE__) && check_tmem(ck, tp, 32, 64, __LINE__))) break;
        float s[128];
        const int seen = lim - (w.t0 + j) * kTileN;  // of this tile's keys
        auto load_s = [&]() {
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32(ts + 32 * q, *reinterpret_cast<float(*)[32]>(&s[32 * q]));
          tmem_wait_ld();
          if (seen < kTileN) {
#pragma unroll
            for (int k = 0; k < 128; ++k)
              if (k >= seen) s[k] = -INFINITY;
          }
        };
        uint32_t p[64];
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
        auto terms = [&]() { return terms_of(integral_constant<int, 0>{}, integral_constant<int, 64>{}); };
        // the maximum of the tile moves the reference if it exceeds it by more
        // than 2^kTau, in the rows that may; by how much O and the sum scale then
        auto move_ref = [&](bool may) {
          float m[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int k = 4; k < 124; k += 8) {
#pragma unroll
            for (int i = 0; i < 4; ++i) m[i] = max3(m[i], s[k + 2 * i], s[k + 2 * i + 1]);
          }
          const float top = max3(max3(m[0], m[1], m[2]), max3(m[3], s[124], s[125]), fmaxf(s[126], s[127])) * c;
          const bool move = may && (top > ref + rise_allowed<TYPE>(top) || (ref == -INFINITY && top > -INFINITY));
          const float alpha = move ? ex2(ref - (top - kBelow<TYPE>)) : 1.f;
          if (move) {
            ref = top - kBelow<TYPE>;
            l *= alpha;
          }
          return alpha;
        };
        auto scale_o = [&](float alpha) {  // (all of its products so far have ended)
#pragma unroll
          for (int q = 0; q < D / 16; ++q) {
            float o[16];
            tmem_ld16(to + 16 * q, o);
            tmem_wait_ld();
            uint32_t r[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) r[k] = __float_as_uint(o[k] * alpha);
            tmem_st16(to + 16 * q, r);
          }
        };
        float f;
        load_s();
        if (L::OWN_P) {
          // S is in registers: the next tile's may come. P's columns and O are
          // touched once the product of the tile before has ended
          if (!(ok = hand_back_s(j))) break;
          const float alpha = move_ref(true);
          f = terms();
          if (j > 0) {
            if (!(ok = warp_wait(p_read, (j - 1) & 1, wc))) break;
            tc_fence_after();
            if (__any_sync(0xFFFFFFFFu, alpha != 1.f)) scale_o(alpha);
          }
        } else {
          // Terms against the reference as it is, while their sum stays within
          // kSumMax; else (and in a row's first tile) the maximum is taken. The
          // products of the tiles before ended before this S. P of the first
          // keys is handed over while the others' is made
          f = terms_of(integral_constant<int, 0>{}, integral_constant<int, kFirst / 2>{});
          bool again = !(f <= kSumMax<TYPE>) || (ref == -INFINITY && seen > 0);
          if (__any_sync(0xFFFFFFFFu, again)) {
            load_s();
            // (every row, whichever one asked: none has been asked about the other keys)
            const float alpha = move_ref(true);
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
              if (!(ok = warp_wait(o_first(t), j & 1, wc))) break;
              tc_fence_after();
#pragma unroll
              for (int q = kFirst / 32; q < 4; ++q) tmem_ld32(ts + 32 * q, *reinterpret_cast<float(*)[32]>(&s[32 * q]));
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 128; ++k)
                if (k < kFirst || k >= seen) s[k] = -INFINITY;
              l += f;
              f = 0.f;
              // (the others' sums were within: 729 us, all rows by their maximum 739)
              const float alpha = move_ref(again);
              scale_o(alpha);
              f2 = terms_of(integral_constant<int, kFirst / 2>{}, integral_constant<int, 64>{});
            }
            f += f2;
          }
        }
        if (!handed) {
#pragma unroll
          for (int q = 0; q < kFirst / 32; ++q) tmem_st16(tp + 16 * q, &p[16 * q]);
        }
#pragma unroll
        for (int q = kFirst / 32; q < 4; ++q) tmem_st16(tp + 16 * q, &p[16 * q]);
        l += f;
        tmem_wait_st();
      } else if (L::OWN_P) {
        // a warp without rows keeps step: it must not arrive for this tile's P
        // while the others still owe the last one's
        if (!(ok = hand_back_s(j) && (j == 0 || warp_wait(p_read, (j - 1) & 1, wc)))) break;
      }
      // P is handed over together with the loads that its products need, V of
      // this tile and (if S was not) K of the next: the waits are these warps'
      // to spend (a wait takes the issuer 100 cycles between products, with the
      // data there)
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
        if ((warp & 3) == 0) {
          if (j > 0) mbar_arrive(kv_empty(idx_v(j - 1) % L::STAGES));
          mbar_arrive(kv_empty(idx_k(j) % L::STAGES));
        }
      }
    }
    // ------------------------------------------------------------ output
    if (t < nt && n_iter > 0 && ok && warp_wait(o_full(L::OWN_P ? 0 : t), 0, wc) && warp_live) {
      tc_fence_after();
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;  // (NaN stays NaN)
      const bool none = l == 0.f;
      const long long e = static_cast<long long>(token) * a.HQ + head;
      const long long plane = static_cast<long long>(blockIdx.y) * a.T * a.HQ;
      // The rows go out through shared memory (this warp's part of Q's tile,
      // which no product reads any more), 128 bytes of each at a time, so that
      // eight lanes write a row's line together
      const uint32_t stage = sb + L::OFF_Q + t * L::TILE + (warp & 3) * 32 * 128;
      const bool parts = a.splits > 1;
      uint8_t* mine = !live  ? nullptr
                      : parts ? reinterpret_cast<uint8_t*>(a.part_o + (plane + e) * D)
                              : reinterpret_cast<uint8_t*>(static_cast<uint16_t*>(a.o) + token * a.o_sn + head * a.o_sh);
      auto write_out = [&](int byte) {  // 128 bytes of each row from this one on
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const int r = i + (lane >> 3);
          uint8_t* row_out = shfl_ptr(mine, r);
          uint4 v;
          ld_shared_v4(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4), v.x, v.y, v.z, v.w);
          if (row_out != nullptr) *reinterpret_cast<uint4*>(row_out + byte + (lane & 7) * 16) = v;
        }
        __syncwarp();
      };
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        float o[32];
        tmem_ld32(to + 32 * q, o);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = none ? 0.f : o[k] * inv;
        if (parts) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            st_shared_v4(stage + lane * 128 + ((k ^ (lane & 7)) << 4), __float_as_uint(o[4 * k]),
                         __float_as_uint(o[4 * k + 1]), __float_as_uint(o[4 * k + 2]), __float_as_uint(o[4 * k + 3]));
          write_out(128 * q);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            st_shared_v4(stage + lane * 128 + (((4 * (q & 1) + k) ^ (lane & 7)) << 4), pack2<TYPE>(o[8 * k], o[8 * k + 1]),
                         pack2<TYPE>(o[8 * k + 2], o[8 * k + 3]), pack2<TYPE>(o[8 * k + 4], o[8 * k + 5]),
                         pack2<TYPE>(o[8 * k + 6], o[8 * k + 7]));
          if (q & 1) write_out(64 * (q - 1));
        }
      }
      if (live) {
        const float lse2 = none ? -INFINITY : ref + log2f(l);
        if (a.splits > 1)
          a.part_lse[plane + e] = lse2;
        else
          a.lse[e] = lse2 * kLn2;
      }
    }
  }

  if (a.splits > 1) grid_launch_dependents();  // the combine kernel may be launched
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Join the splits of a row (token, head), one warp a row: with weights
// 2^(lse_s - lse), o = sum_s w_s o_s.
// RUN: splits whose loads are in flight, the first ones beside the lse's (16
// tokens x 4 heads over 4,096 keys in 16 splits, both kernels: 12.5 us, 15.3 after
// the lse); few where there are few, for more warps (512 tokens x 32 heads in two
// splits, both kernels: 112.5 us, 114.2 with 8).
template <int TYPE, int D, int RUN>
__global__ void __launch_bounds__(256) streamkl_paged_combine_kernel(const __grid_constant__ PagedAttnArgs a) {
  constexpr int V = D / 32;  // columns of a lane
  grid_dependency_wait();  // launched while the attention kernel ends
  const int lane = threadIdx.x & 31;
  const long long e = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const long long rows = static_cast<long long>(a.T) * a.HQ;
  // tokens in front of the first sequence and behind the last one stay
  const int begin = a.cu != nullptr ? __ldg(a.cu) : 0, end = a.cu != nullptr ? __ldg(a.cu + a.B) : a.B;
  const int token = static_cast<int>(e / a.HQ), head = static_cast<int>(e - static_cast<long long>(token) * a.HQ);
  if (e >= rows || token < begin || token >= end) return;
  float p[RUN][V];
  auto fetch = [&](int s0) {
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
      if (s0 + i >= a.splits) break;
      const float* src = a.part_o + ((s0 + i) * rows + e) * D + lane * V;
      if constexpr (V == 4)
        *reinterpret_cast<float4*>(p[i]) = *reinterpret_cast<const float4*>(src);
      else
        *reinterpret_cast<float2*>(p[i]) = *reinterpret_cast<const float2*>(src);
    }
  };
  fetch(0);
  float top = -INFINITY;
  for (int s = lane; s < a.splits; s += 32) top = fmaxf(top, a.part_lse[s * rows + e]);
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
  const float t0 = top == -INFINITY ? 0.f : top;
  float total = 0.f, o[V] = {};
  for (int s0 = 0; s0 < a.splits; s0 += RUN) {
    if (s0 > 0) fetch(s0);
    const float mine = lane < RUN && s0 + lane < a.splits ? ex2(a.part_lse[(s0 + lane) * rows + e] - t0) : 0.f;
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
      if (s0 + i >= a.splits) break;
      const float w = __shfl_sync(0xFFFFFFFFu, mine, i);
      total += w;
#pragma unroll
      for (int k = 0; k < V; ++k)  // (the partial of an empty range is not written)
        if (w != 0.f) o[k] = fmaf(w, p[i][k], o[k]);
    }
  }
  const float inv = total == 0.f ? 0.f : 1.f / total;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + token * a.o_sn + head * a.o_sh + lane * V);
#pragma unroll
  for (int k = 0; k < V / 2; ++k) dst[k] = pack2<TYPE>(o[2 * k] * inv, o[2 * k + 1] * inv);
  if (lane == 0) a.lse[e] = total == 0.f ? -INFINITY : (top + log2f(total)) * kLn2;
}

template <int TYPE, int D, int NT>
cudaError_t attn_t(const PagedAttnArgs& a, cudaStream_t stream) {
  using L = AttnLayout<D, NT>;
  auto kern = streamkl_paged_attn_kernel<TYPE, D, NT>;
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
  kern<<<dim3(a.q_tiles, a.splits, a.B * a.HK), L::THREADS, L::BYTES, stream>>>(*a.tm_k, *a.tm_v, a);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.splits == 1) return e;
  const long long rows = static_cast<long long>(a.T) * a.HQ;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((rows + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto combine = a.splits <= 2   ? streamkl_paged_combine_kernel<TYPE, D, 2>
                 : a.splits <= 4 ? streamkl_paged_combine_kernel<TYPE, D, 4>
                                 : streamkl_paged_combine_kernel<TYPE, D, 8>;
  return cudaLaunchKernelEx(&cfg, combine, a);
}

template <int TYPE, int D>
cudaError_t attn_d(const PagedAttnArgs& a, cudaStream_t stream) {
  return a.row_tiles == 2 ? attn_t<TYPE, D, 2>(a, stream) : attn_t<TYPE, D, 1>(a, stream);
}

}  // namespace

cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t stream) {
  if (a.type == kTypeBf16) return a.d == 128 ? attn_d<kTypeBf16, 128>(a, stream) : attn_d<kTypeBf16, 64>(a, stream);
  return a.d == 128 ? attn_d<kTypeF16, 128>(a, stream) : attn_d<kTypeF16, 64>(a, stream);
}

}  // namespace skl
