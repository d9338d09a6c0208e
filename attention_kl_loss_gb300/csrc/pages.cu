// What a serving step does with the pages of a cache beside attention: drafted
// tokens that were accepted move to the front (compact), pages are copied (copy),
// sequences go on from others' pages (fork), take pages and give them back (resize).
//
// Rows and pages are moved 16 bytes a lane; tables and counts are whole numbers, so
// results do not depend on the order of the atomics.
#include <algorithm>
#include <atomic>
#include <cooperative_groups.h>

#include "ops.h"
#include "ptx.cuh"

namespace skl {

namespace {

// ------------------------------------------------------------------ copy
// Page `dst` of both caches becomes page `src`, for each pair. A block moves
// kCopyVectors vectors of one pair and cache: every lane has its 8 loads in flight
// before the first store. Bound by HBM: 1,000 pages of 256 KB in each cache 152 us,
// 6.9 TB/s; 16 of 32 KB 2.9 us, which is the launch.
constexpr int kCopyThreads = 256, kCopyRun = 8, kCopyVectors = kCopyThreads * kCopyRun;

__global__ void __launch_bounds__(kCopyThreads) streamkl_page_copy_kernel(const __grid_constant__ PageCopyArgs a) {
  const int pair = static_cast<int>(blockIdx.x / a.chunks), chunk = static_cast<int>(blockIdx.x - pair * a.chunks);
  const int src = __ldg(a.pairs + 2LL * pair), dst = __ldg(a.pairs + 2LL * pair + 1);
  if (src < 0 && dst < 0) return;
  if (src < 0 || dst < 0 || src >= a.num_pages || dst >= a.num_pages) {
    if (chunk == 0 && blockIdx.y == 0 && threadIdx.x == 0) atomicCAS(a.dev_status, 0, kStatusInvalidArg);
    return;
  }
  if (src == dst) return;
  const CacheRows& c = a.cache[blockIdx.y];
  const uint4* from = static_cast<const uint4*>(c.data) + src * c.sp;
  uint4* to = static_cast<uint4*>(c.data) + dst * c.sp;
  const int page = 1 << a.page_shift, total = (a.H << a.page_shift) << a.vshift;
  uint4 v[kCopyRun];
  long long at[kCopyRun];
#pragma unroll
  for (int i = 0; i < kCopyRun; ++i) {
    const int e = chunk * kCopyVectors + i * kCopyThreads + static_cast<int>(threadIdx.x);
    const int row = e >> a.vshift;
    at[i] = e < total ? (row >> a.page_shift) * c.sh + (row & (page - 1)) * c.ss + (e & ((1 << a.vshift) - 1)) : -1;
    if (at[i] >= 0) v[i] = from[at[i]];
  }
#pragma unroll
  for (int i = 0; i < kCopyRun; ++i)
    if (at[i] >= 0) to[at[i]] = v[i];
}

// --------------------------------------------------------------- compact
// Row kept[i] of a sequence's last n becomes row i of them, i rising, in place. The
// kept rows rise too, so row i is at most kept[i]: what a batch of rows writes lies
// before all that later batches read, and within a batch every load comes before
// the first store. Columns do not meet, so an item is one (sequence, cache, head). 64
// sequences' up to 6 rows x 8 heads of 256 bytes: 3.3 us, the launch and the chain of
// offsets, list, page and row.
constexpr int kCompactRun = 8;

struct CompactSeq {
  int n, first, count;  // last tokens, position of the first of them, kept ones
  bool ok;
};

__device__ __forceinline__ CompactSeq compact_seq(const CompactArgs& a, int b) {
  const int c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1), len = __ldg(a.kv_lens + b);
  CompactSeq s;
  s.n = c1 - c0;
  s.first = len - s.n;
  s.count = __ldg(a.num_kept + b);
  s.ok = c0 >= 0 && c1 >= c0 && s.first >= 0 && s.count >= 0 && s.count <= s.n && s.count <= a.max_kept &&
         len <= (static_cast<long long>(a.max_pages) << a.page_shift);
  return s;
}

// THREADS threads an item: a warp each where few rows are kept, else a block for
// 32 bytes of its columns (whole sequences are pruned, and the longest one decides: 8
// sequences of up to 4,100 kept rows, 8 heads of 128 take 27 us, 30 by 64 bytes, 73
// by whole rows and 512 threads). The next rows' numbers are loaded beside the rows.
template <int THREADS>
__global__ void __launch_bounds__(THREADS == 32 ? 128 : THREADS, THREADS == 32 ? 1 : 3)
    streamkl_paged_compact_kernel(const __grid_constant__ CompactArgs a) {
  constexpr bool WARP = THREADS == 32;
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int split = WARP ? 0 : a.vshift - 1, vshift = a.vshift - split;  // column groups; vectors a row in one
  const long long item = WARP ? blockIdx.x * 4LL + (threadIdx.x >> 5) : blockIdx.x >> split;
  if (item >= 2LL * a.B * a.H) return;
  auto together = [](bool p) { return WARP ? __all_sync(0xFFFFFFFFu, p) != 0 : __syncthreads_and(p) != 0; };
  const int b = static_cast<int>(item / (2 * a.H)), rest = static_cast<int>(item - b * 2LL * a.H);
  const int h = rest >> 1;
  const CacheRows& c = a.cache[rest & 1];
  const CompactSeq s = compact_seq(a, b);
  const int* kept = a.kept + b * a.kept_sb;
  bool good = s.ok;
  // the list, before anything moves (eight numbers in flight: a block of its own
  // columns looks at all of it)
  for (int i0 = tid; good && i0 < s.count; i0 += THREADS * 8) {
    int now[8], before[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + u * THREADS;
      now[u] = i < s.count ? __ldg(kept + i) : 0;
      before[u] = i < s.count && i > 0 ? __ldg(kept + i - 1) : -1;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (i0 + u * THREADS < s.count) good = good && now[u] < s.n && now[u] > before[u] && now[u] >= 0;
  }
  if (!together(good)) {
    if (tid == 0 && rest == 0) atomicCAS(a.dev_status, 0, kStatusInvalidArg);
    return;
  }
  const int* table = a.table + b * a.table_sb;
  const int page = 1 << a.page_shift;
  const int column = (tid & ((1 << vshift) - 1)) + (WARP ? 0 : (blockIdx.x & ((1 << split) - 1)) << vshift);
  uint4* data = static_cast<uint4*>(c.data) + h * c.sh + column;
  auto place = [&](int i) -> uint4* {  // row i of the last n
    const int pos = s.first + i;
    const int p = __ldg(table + (pos >> a.page_shift));
    if (p < 0 || p >= a.num_pages) {
      atomicCAS(a.dev_status, 0, kStatusInvalidArg);
      return nullptr;
    }
    return data + p * c.sp + (pos & (page - 1)) * c.ss;
  };
  const int per = THREADS >> vshift, mine = tid >> vshift;  // rows at once
  int k[kCompactRun];
  auto numbers = [&](int i0) {
#pragma unroll
    for (int u = 0; u < kCompactRun; ++u) {
      const int i = i0 + u * per + mine;
      k[u] = i < s.count ? __ldg(kept + i) : i;  // (which moves nothing)
    }
  };
  numbers(0);
  for (int i0 = 0; i0 < s.count; i0 += per * kCompactRun) {
    uint4 v[kCompactRun];
    uint4* to[kCompactRun];
#pragma unroll
    for (int u = 0; u < kCompactRun; ++u) {
      const int i = i0 + u * per + mine;
      to[u] = nullptr;
      if (k[u] != i) {
        const uint4* from = place(k[u]);
        if (from != nullptr) {
          v[u] = *from;
          to[u] = place(i);
        }
      }
    }
    numbers(i0 + per * kCompactRun);
    if (WARP)
      __syncwarp();
    else
      __syncthreads();
#pragma unroll
    for (int u = 0; u < kCompactRun; ++u)
      if (to[u] != nullptr) *to[u] = v[u];
  }
}

// ------------------------------------------------------------------ fork
// table[b] = table[source[b]] for all b at once. A block takes a slab of columns of
// every row: all of it is read before any is written, and other slabs do not meet
// it. A page of the row b is afterwards held by as many rows more as there are
// sequences that go on from b, less the row b itself: one atomic an entry, which is
// what bounds a large call (512 sequences of up to 4,096 pages, 11.0 us for about a
// million of them; 64 of 256 pages 3.1 us, the launch).
constexpr int kForkThreads = 256, kForkRun = 8;  // entries whose loads are in flight

__global__ void __launch_bounds__(kForkThreads) streamkl_paged_fork_kernel(const __grid_constant__ ForkArgs a) {
  extern __shared__ int sm[];
  int *source = sm, *more = sm + a.B, *old = more + a.B;  // old: [B][columns], block 0 first uses it for the lengths
  for (int b = threadIdx.x; b < a.B; b += kForkThreads) more[b] = -1;
  __syncthreads();
  for (int b = threadIdx.x; b < a.B; b += kForkThreads) {
    int s = __ldg(a.source + b);
    if (s < 0 || s >= a.B) {
      if (blockIdx.x == 0) atomicCAS(a.dev_status, 0, kStatusInvalidArg);
      s = b;  // it stays
    }
    source[b] = s;
    atomicAdd(&more[s], 1);
    if (blockIdx.x == 0) old[b] = a.kv_lens[b];
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b < a.B; b += kForkThreads)
      if (source[b] != b) a.kv_lens[b] = old[source[b]];
    __syncthreads();
  }
  const int j0 = static_cast<int>(blockIdx.x) << a.cols, cols = min(1 << a.cols, a.max_pages - j0);
  const int entries = a.B << a.cols;
  for (int e0 = threadIdx.x; e0 < entries; e0 += kForkThreads * kForkRun) {
    int p[kForkRun];
#pragma unroll
    for (int u = 0; u < kForkRun; ++u) {
      const int e = e0 + u * kForkThreads, b = e >> a.cols, j = e & ((1 << a.cols) - 1);
      p[u] = -1;
      // (nothing to do where nobody takes it and it stays)
      if (e < entries && j < cols && (source[b] != b || more[b] != 0)) p[u] = a.table[b * a.table_sb + j0 + j];
    }
#pragma unroll
    for (int u = 0; u < kForkRun; ++u) {
      const int e = e0 + u * kForkThreads;
      if (e >= entries) break;
      old[e] = p[u];
      const int change = more[e >> a.cols];
      if (change != 0 && p[u] != -1) {
        if (p[u] < 0 || p[u] >= a.num_pages)
          atomicCAS(a.dev_status, 0, kStatusInvalidArg);
        else
          atomicAdd(a.refs + p[u], change);
      }
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < entries; e += kForkThreads) {
    const int b = e >> a.cols, j = e & ((1 << a.cols) - 1);
    if (j < cols && source[b] != b) a.table[b * a.table_sb + j0 + j] = old[(source[b] << a.cols) + j];
  }
}

// ---------------------------------------------------------------- resize
// One cluster: what is asked of a sequence hangs on those before it, and which page
// it gets on all pages before that one, so the whole call is two prefix sums, over
// the sequences (every block makes them for itself) and over the free pages (the
// blocks share them, one bit each, and exchange their counts). Between them lies what
// has to be in that order: pages given back, the counts of last pages, free pages.
// A step of 64 sequences takes 6.6 us, a chain of loads and barriers; 667,000 pages
// given back and 608,000 given out of two million 38 us: 9 give back, 7 look for free
// pages and some 20 write them down, at what sixteen SMs store (a page's count and its
// entry, in other lines for every warp).
//
// 1,024 threads a block, or one block of 256 where tables and pages are few: barriers,
// scans and looks of warps that have nothing to do are most of such a call.
constexpr int kResizeBlocks = 16;  // most of a cluster
constexpr int kResizeRounds = kMaxPages / (1024 * 32 * kResizeBlocks);  // a bit a page and thread, 32 in each
static_assert(kMaxPages % (1024 * 32 * kResizeBlocks) == 0);

// Exclusive sums of value(b) over b < B into out[0 .. B]; returns the total. All
// threads; two barriers, and one before the next use of `sums` [32].
template <int THREADS, typename F>
__device__ __forceinline__ int scan_sequences(int B, int* out, int* sums, F&& value) {
  const int per = (B + THREADS - 1) / THREADS;
  const int b0 = min(B, static_cast<int>(threadIdx.x) * per), b1 = min(B, b0 + per);
  int mine = 0;
  for (int b = b0; b < b1; ++b) mine += value(b);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int upto = mine;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int up = __shfl_up_sync(0xFFFFFFFFu, upto, m);
    if (lane >= m) upto += up;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  const int w = lane < THREADS / 32 ? sums[lane] : 0;
  const int before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? w : 0), total = __reduce_add_sync(0xFFFFFFFFu, w);
  int at = before + upto - mine;
  for (int b = b0; b < b1; ++b) {
    const int v = value(b);  // (it may lie in out)
    out[b] = at;
    at += v;
  }
  if (threadIdx.x == 0) out[B] = total;
  __syncthreads();
  return total;
}

// The sequence of lo .. hi in whose part of the exclusive sums x lies.
__device__ __forceinline__ int find_sequence(const int* sums, int lo, int hi, int x) {
  while (lo < hi) {  // sums[lo] <= x < sums[hi + 1]
    const int mid = (lo + hi + 1) >> 1;
    if (sums[mid] <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// What a sequence's numbers ask for; false where they do not fit.
__device__ __forceinline__ bool lengths_fit(const ResizeArgs& a, int from, int to) {
  const long long most = static_cast<long long>(a.max_pages) << a.page_shift;
  return from >= 0 && from <= most && to >= 0 && to <= most;
}

__device__ __forceinline__ void take_back(const ResizeArgs& a, int p) {
  if (p >= 0 && p < a.num_pages)
    atomicSub(a.refs + p, 1);
  else
    atomicCAS(a.dev_status, 0, kStatusInvalidArg);
}

// Entries first(b) + i, i below the sums' differences, of all sequences: a lane each
// where that is enough, else runs of 128 a warp, most of which lie in one sequence.
template <typename F>
__device__ __forceinline__ void give_back(const ResizeArgs& a, const int* sums, int total, int warp, int warps, F&& first) {
  const int lane = threadIdx.x & 31;
  if (total <= warps * 32) {
    const int i = warp * 32 + lane;
    if (i >= total) return;
    const int b = find_sequence(sums, 0, a.B - 1, i);
    int* entry = a.table + b * a.table_sb + first(b) + (i - sums[b]);
    const int p = *entry;
    *entry = -1;
    take_back(a, p);
    return;
  }
  for (int i0 = warp * 128; i0 < total; i0 += warps * 128) {
    const int lo = find_sequence(sums, 0, a.B - 1, i0);
    const int hi = find_sequence(sums, lo, a.B - 1, min(total, i0 + 128) - 1);
    int p[4];
    int* entry[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + 32 * u + lane;
      if (i >= total) continue;
      const int b = find_sequence(sums, lo, hi, i);
      entry[u] = a.table + b * a.table_sb + first(b) + (i - sums[b]);
      p[u] = *entry[u];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {  // (a store behind its load, before the others: 35 us for 9)
      if (i0 + 32 * u + lane >= total) continue;
      *entry[u] = -1;
      take_back(a, p[u]);
    }
  }
}

// Large tables: what is given back, by blocks on every SM before the cluster (scattered
// atomics: 667,000 of them take 9 us so, and 25 on the cluster's sixteen SMs).
constexpr int kReleaseThreads = 256;
constexpr long long kReleaseEntries = 1 << 18;  // of the tables, from which on

__global__ void __launch_bounds__(kReleaseThreads) streamkl_paged_release_kernel(const __grid_constant__ ResizeArgs a) {
  extern __shared__ int sm[];
  __shared__ int scratch[32];
  int *sums = sm, *first = sm + a.B + 1;
  grid_launch_dependents();
  const int page = 1 << a.page_shift;
  for (int b = threadIdx.x; b < a.B; b += kReleaseThreads) {
    const int from = a.kv_lens[b], to = __ldg(a.new_lens + b);
    const bool fits = lengths_fit(a, from, to);
    first[b] = fits ? (to + page - 1) >> a.page_shift : 0;
    sums[b] = fits ? max(0, ((from + page - 1) >> a.page_shift) - first[b]) : 0;
  }
  __syncthreads();
  const int total = scan_sequences<kReleaseThreads>(a.B, sums, scratch, [&](int b) { return sums[b]; });
  give_back(a, sums, total, static_cast<int>(blockIdx.x * (kReleaseThreads / 32) + (threadIdx.x >> 5)),
            static_cast<int>(gridDim.x * (kReleaseThreads / 32)), [&](int b) { return first[b]; });
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1) streamkl_paged_resize_kernel(const __grid_constant__ ResizeArgs a) {
  namespace cg = cooperative_groups;
  constexpr int kWarps = THREADS / 32, kBlockPages = THREADS * 32;  // (a block's of a round)
  cg::cluster_group cluster = cg::this_cluster();
  const int blocks = static_cast<int>(cluster.num_blocks()), me = static_cast<int>(cluster.block_rank());
  extern __shared__ int sm[];
  int* sums = sm;              // [B + 1]
  int* from = sums + a.B + 1;  // lengths; a sequence whose numbers do not fit stays
  int* to = from + a.B;
  int* last = to + a.B;        // a last page to be copied; kNone, kKeeps: the last of those that hold it
  uint16_t* list = reinterpret_cast<uint16_t*>(last + a.B);  // [block's pages]: free ones of a round, in their order
  uint32_t* bits = reinterpret_cast<uint32_t*>(list + kBlockPages);  // [rounds][threads]: free pages
  constexpr int kNone = -1, kKeeps = -2;
  constexpr int kShort = 4;  // entries given back that a sequence's own thread takes
  __shared__ int scratch[kWarps];
  __shared__ int counts[2][kResizeBlocks];  // free pages of the blocks, by the round's parity
  __shared__ int ranks[kResizeRounds + 1];  // of a round's first free page in this block
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int page = 1 << a.page_shift;
  auto pages_of = [&](int length) { return (length + page - 1) >> a.page_shift; };
  auto back_of = [&](int b) { return max(0, pages_of(from[b]) - pages_of(to[b])); };
  bool many = false;  // entries of some sequence to be given back
  for (int b = tid; b < a.B; b += THREADS) {
    int f = a.kv_lens[b], t = __ldg(a.new_lens + b), p = kNone;
    int* row = a.table + b * a.table_sb;
    if (!lengths_fit(a, f, t)) {
      if (me == 0) atomicCAS(a.dev_status, 0, kStatusInvalidArg);
      f = t = 0;
    } else if (t > f && (f & (page - 1)) != 0) {  // it grows into its last page
      p = row[f >> a.page_shift];
      if (p < 0 || p >= a.num_pages) {
        if (me == 0) atomicCAS(a.dev_status, 0, kStatusInvalidArg);
        p = kNone;
      }
    } else if (!a.released) {
      const int n = pages_of(f) - pages_of(t);
      many = many || n > kShort;
      if (n > 0 && n <= kShort && me == 0) {
        int old[kShort];
        row += pages_of(t);
#pragma unroll
        for (int i = 0; i < kShort; ++i)
          if (i < n) old[i] = row[i];
#pragma unroll
        for (int i = 0; i < kShort; ++i)
          if (i < n) {
            row[i] = -1;
            take_back(a, old[i]);
          }
      }
    }
    from[b] = f;
    to[b] = t;
    last[b] = p;
  }
  if (__syncthreads_or(many)) {
    const int back = scan_sequences<THREADS>(a.B, sums, scratch, [&](int b) {
      const int n = back_of(b);
      return n > kShort ? n : 0;
    });
    give_back(a, sums, back, me * kWarps + warp, blocks * kWarps, [&](int b) { return pages_of(to[b]); });
  }
  if (a.released) grid_dependency_wait();  // the other kernel has given back
  cluster.sync();
  // ---- free pages: bit 4 i + e of a thread: page base + 128 i + 4 lane + e of its warp's 1,024
  auto look = [&](int round) {
    const int base = (round * blocks + me) * kBlockPages + warp * 1024;
    uint32_t free = 0;
    if (base < a.num_pages) {
      const int* refs = a.refs + base + lane * 4;
      int4 v[8];
      if (base + 1024 <= a.num_pages) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __ldcg(reinterpret_cast<const int4*>(refs + 128 * i));
      } else {
        const int left = a.num_pages - base - lane * 4;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i].x = 128 * i < left ? __ldcg(refs + 128 * i) : 1;
          v[i].y = 128 * i + 1 < left ? __ldcg(refs + 128 * i + 1) : 1;
          v[i].z = 128 * i + 2 < left ? __ldcg(refs + 128 * i + 2) : 1;
          v[i].w = 128 * i + 3 < left ? __ldcg(refs + 128 * i + 3) : 1;
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        free |= static_cast<uint32_t>((v[i].x == 0) | (v[i].y == 0) << 1 | (v[i].z == 0) << 2 | (v[i].w == 0) << 3)
                << (4 * i);
    }
    bits[round * THREADS + tid] = free;
    return __popc(free);
  };
  // ---- last pages that others hold too (beside the first look at the counts)
  const int held = tid < a.B && last[tid] >= 0 ? __ldcg(a.refs + last[tid]) : 0;
  int seen = look(0);
  bool any = false;
  for (int b = tid; b < a.B; b += THREADS) {
    if (last[b] < 0) continue;
    const bool shared = (b == tid ? held : __ldcg(a.refs + last[b])) > 1;
    any = any || shared;
    if (!shared) last[b] = kNone;
  }
  if (__syncthreads_or(any)) {
    // in their order, each takes a copy while another holds the page
    for (int b0 = 0; b0 < a.B; b0 += THREADS) {  // (from the back, so that those before are as they were)
      const int b = a.B - 1 - b0 - tid;
      bool keeps = false;
      if (b >= 0 && last[b] >= 0) {
        const int p = last[b];
        int before = 0;
#pragma unroll 8
        for (int i = 0; i < b; ++i) before += last[i] == p;
        keeps = __ldcg(a.refs + p) - before <= 1;
      }
      __syncthreads();
      if (keeps) last[b] = kKeeps;
    }
    __syncthreads();
  }
  const int asked = scan_sequences<THREADS>(a.B, sums, scratch, [&](int b) {
    return max(0, pages_of(to[b]) - pages_of(from[b])) + (last[b] >= 0);
  });
  // ---- enough of the free pages, lowest numbers first
  const int rounds = static_cast<int>((a.num_pages + static_cast<long long>(blocks) * kBlockPages - 1) /
                                      (static_cast<long long>(blocks) * kBlockPages));
  int found = 0, round = 0;
  for (; round < rounds && found < asked; ++round) {
    if (round > 0) seen = look(round);
    const int mine = __reduce_add_sync(0xFFFFFFFFu, seen);
    if (lane == 0) scratch[warp] = mine;
    __syncthreads();
    const int block = __reduce_add_sync(0xFFFFFFFFu, lane < kWarps ? scratch[lane] : 0);
    if (tid < blocks) *cluster.map_shared_rank(&counts[round & 1][me], tid) = block;
    cluster.sync();  // (and `scratch` may be used again)
    int before = found, total = found;
    for (int i = 0; i < blocks; ++i) {
      if (i < me) before += counts[round & 1][i];
      total += counts[round & 1][i];
    }
    if (tid == 0) ranks[round] = before;
    found = total;
  }
  // ---- who is served: all that is asked up to a sequence has to be there
  auto served = [&](int b) { return (sums[b + 1] == sums[b] && last[b] != kKeeps) || sums[b + 1] <= found; };
  int limit = asked;
  if (found < asked) {  // (the sums do not fall: the largest that is there)
    int lo = 0, hi = a.B;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sums[mid] <= found)
        lo = mid;
      else
        hi = mid - 1;
    }
    limit = sums[lo];
  }
  // ---- pages to their places
  __syncthreads();  // (ranks)
  for (int r = 0; r < round; ++r) {
    if (ranks[r] >= limit) break;
    // in a list first, so that all threads take one page each, whichever they found
    const uint32_t free = bits[r * THREADS + tid];
    const int mine = __reduce_add_sync(0xFFFFFFFFu, __popc(free));
    __syncthreads();  // (the list of the round before has been read)
    if (lane == 0) scratch[warp] = mine;
    __syncthreads();
    const int count = lane < kWarps ? scratch[lane] : 0;
    const int all = __reduce_add_sync(0xFFFFFFFFu, count);
    int at = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? count : 0);  // of this warp's first free page
    const int n = min(all, limit - ranks[r]);
    if (mine > 0 && at < n) {
      // counts of the eight groups of 128 pages, a byte each, summed over the lanes together
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        uint32_t ones = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) ones |= __popc(free >> (16 * w + 4 * i) & 15) << (8 * i);
        uint32_t upto = ones;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
          const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, upto, m);
          if (lane >= m) upto += up;
        }
        const uint32_t sums_of = __shfl_sync(0xFFFFFFFFu, upto, 31), before = upto - ones;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t four = free >> (16 * w + 4 * i) & 15;
          int to_place = at + static_cast<int>(before >> (8 * i) & 255);
          const int number = warp * 1024 + 128 * (4 * w + i) + 4 * lane;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (four >> e & 1) list[to_place++] = static_cast<uint16_t>(number + e);
          at += static_cast<int>(sums_of >> (8 * i) & 255);
        }
      }
    }
    __syncthreads();
    const int base = (r * blocks + me) * kBlockPages;
    auto give = [&](int slot, int p, int b) {
      int* entry = a.table + b * a.table_sb + pages_of(from[b]) + (slot - sums[b]);
      a.refs[p] = 1;
      if (last[b] >= 0) {
        --entry;  // the copy comes first, in the last page's place
        if (slot == sums[b]) {
          a.copies[b] = make_int2(last[b], p);
          atomicSub(a.refs + last[b], 1);
        }
      }
      *entry = p;
    };
    if (n <= 2 * THREADS) {
      for (int x = tid; x < n; x += THREADS)
        give(ranks[r] + x, base + list[x], find_sequence(sums, 0, a.B - 1, ranks[r] + x));
      continue;
    }
    // runs of 128 a warp, most of which lie in one sequence: no search, no branch
    int hi = 0;
    for (int x0 = warp * 128; x0 < n; x0 += kWarps * 128) {
      const int x1 = min(n, x0 + 128) - 1, slot = ranks[r] + x0 + lane;
      const int lo = find_sequence(sums, hi, a.B - 1, ranks[r] + x0);
      hi = find_sequence(sums, lo, a.B - 1, ranks[r] + x1);
      if (lo == hi && last[lo] < 0) {
        int* entry = a.table + lo * a.table_sb + pages_of(from[lo]) + (slot - sums[lo]);
        int p[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) p[u] = base + list[min(x1, x0 + 32 * u + lane)];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (x0 + 32 * u + lane <= x1) {
            a.refs[p[u]] = 1;
            entry[32 * u] = p[u];
          }
      } else {
        for (int x = x0 + lane; x <= x1; x += 32)
          give(ranks[r] + x, base + list[x], find_sequence(sums, lo, hi, ranks[r] + x));
      }
    }
  }
  // ---- lengths (which every block has read, before the barriers above)
  if (me == 0) {
    for (int b = tid; b < a.B; b += THREADS) {
      const bool is_served = served(b);
      if (last[b] < 0 || !is_served) a.copies[b] = make_int2(-1, -1);
      if (is_served && from[b] != to[b]) a.kv_lens[b] = to[b];
      if (a.step_lens != nullptr) a.step_lens[b] = is_served ? to[b] : 0;
      if (!is_served) atomicCAS(a.dev_status, 0, kStatusNoPages);
    }
  }
}

int resize_shared(int B, int rounds, int threads) {
  return (4 * B + 1 + (rounds + 16) * threads) * static_cast<int>(sizeof(int));  // (the list: two bytes a page)
}

template <typename F>
cudaError_t once_per_device(std::atomic<unsigned long long>& done, F&& set) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (done.load() & bit) return cudaSuccess;
  e = set();
  if (e == cudaSuccess) done.fetch_or(bit);
  return e;
}

template <typename K>
cudaError_t allow_shared(K kern, std::atomic<unsigned long long>& done, int bytes) {
  return once_per_device(done, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  });
}

}  // namespace

cudaError_t launch_page_copy(PageCopyArgs& a, cudaStream_t stream) {
  const long long vectors = (static_cast<long long>(a.H) << a.page_shift) << a.vshift;
  a.chunks = static_cast<int>((vectors + kCopyVectors - 1) / kCopyVectors);
  const dim3 grid(static_cast<unsigned>(static_cast<long long>(a.n) * a.chunks), 2);
  streamkl_page_copy_kernel<<<grid, kCopyThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_compact(const CompactArgs& a, cudaStream_t stream) {
  const long long items = 2LL * a.B * a.H;
  // a warp moves 16 rows of 256 bytes at once; longer lists get a block
  if (a.max_kept <= 2 * kCompactRun * (32 >> a.vshift))
    streamkl_paged_compact_kernel<32><<<static_cast<unsigned>((items + 3) / 4), 128, 0, stream>>>(a);
  else
    streamkl_paged_compact_kernel<256><<<static_cast<unsigned>(items << (a.vshift - 1)), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_fork(ForkArgs& a, int sms, cudaStream_t stream) {
  static std::atomic<unsigned long long> done{0};
  constexpr int kMost = (kMaxTableRows * 6) * static_cast<int>(sizeof(int));
  cudaError_t e = allow_shared(streamkl_paged_fork_kernel, done, kMost);
  if (e != cudaSuccess) return e;
  // 32 columns (a line of each row), fewer for more blocks or where the slab would not fit
  a.cols = 5;
  while (a.cols > 2 && (a.max_pages >> a.cols < 2 * sms || a.B * ((1 << a.cols) + 2) > kMaxTableRows * 6)) --a.cols;
  const int cols = 1 << a.cols, bytes = a.B * (cols + 2) * static_cast<int>(sizeof(int));
  streamkl_paged_fork_kernel<<<(a.max_pages + cols - 1) / cols, kForkThreads, bytes, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_resize(ResizeArgs& a, int sms, cudaStream_t stream) {
  static std::atomic<unsigned long long> done{0}, wide{0};
  cudaError_t e = allow_shared(streamkl_paged_resize_kernel<1024>, done, resize_shared(kMaxTableRows, kResizeRounds, 1024));
  if (e != cudaSuccess) return e;
  // 256 threads as long as they look at all pages in one round
  const int threads = a.num_pages <= 256 * 32 && a.B <= 256 ? 256 : 1024;
  // as many blocks as look at all pages in one round; sixteen of a cluster have to be asked for
  const long long block_pages = threads * 32;
  int blocks = 1;
  while (blocks < kResizeBlocks && blocks * block_pages < a.num_pages) blocks *= 2;
  if (blocks > 8 && (e = once_per_device(wide, [] {
                       return cudaFuncSetAttribute(streamkl_paged_resize_kernel<1024>,
                                                   cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
                     })) != cudaSuccess)
    return e;
  const int rounds = static_cast<int>((a.num_pages + blocks * block_pages - 1) / (blocks * block_pages));
  a.released = static_cast<long long>(a.B) * a.max_pages > kReleaseEntries && a.num_pages > kReleaseEntries / 4;
  if (a.released) {
    const size_t bytes = (2 * static_cast<size_t>(a.B) + 1) * sizeof(int);
    streamkl_paged_release_kernel<<<2 * sms, kReleaseThreads, bytes, stream>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(resize_shared(a.B, rounds, threads));
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(blocks);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.released ? 2 : 1;
  return threads == 256 ? cudaLaunchKernelEx(&cfg, streamkl_paged_resize_kernel<256>, a)
                        : cudaLaunchKernelEx(&cfg, streamkl_paged_resize_kernel<1024>, a);
}

}  // namespace skl
