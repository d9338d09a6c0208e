// Internal launch interface of the operators around the attention-KL call:
// norm and rotation of queries and keys, the paged cache's append and the
// attention over it.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace skl {

// Element types of the rows (== STREAMKL_BF16 and so on).
constexpr int kTypeBf16 = 0, kTypeF16 = 1, kTypeF32 = 2;

// Where rows of d elements lie: row (b, n, h) starts at element
// b * sb + n * sn + h * sh.
struct RowStrides {
  long long sb, sn, sh;
};

// One of the two tensors (queries or keys) of a norm + rotation call.
struct RopeSide {
  const void* x;       // B x N x H rows; null: this side is absent
  RowStrides xs;
  const int* pos;      // position of token (b, n) at pos[b * pos_sb + n]; null: pos0 + n
  long long pos_sb;
  int pos0;
  const float* w;      // norm weights [d]; null: rotation only
  int N, H, rep;       // tokens, heads; each head stands rep times on the outer side
  const void* y_in;    // backward: gradient of the outer rows (head h * rep + r)
  void* y_out;         // forward: the outer rows
  RowStrides ys;
  void* dx;            // backward: gradient of x
  RowStrides dxs;
  // set by the launcher: warp items = batches x token tiles x head chunks
  int tiles, hchunks;
  long long items;
};

struct RopeArgs {
  RopeSide side[2];
  int B, d, rot, type, interleaved;
  int table_len;       // rows of cos, sin [table_len, rot / 2]
  const float* cos;
  const float* sin;
  float eps;
  int hc;              // heads of a warp item (set by the launcher)
  float* part;         // backward: weight-gradient partials [2][blocks][d]; null without norm
  int* dev_status;
};

struct AppendArgs {
  const void* k;
  const void* v;
  RowStrides ks, vs;   // sb unused
  void* kc;
  void* vc;
  long long kc_sp, kc_sh, kc_ss, vc_sp, vc_sh, vc_ss;  // page, head and slot strides, elements
  const int* table;    // [B][max_pages], rows table_sb apart
  long long table_sb;
  const int* kv_lens;
  const int* cu;       // [B + 1]; null: token b belongs to sequence b
  int B, T, H, d, rot, type, interleaved, page_shift, num_pages, max_pages, table_len;
  const float* cos;    // null: no rotation
  const float* sin;
  const float* w;
  float eps;
  int hc, hchunks;     // set by the launcher
  int* dev_status;
};

struct PagedAttnArgs {
  const CUtensorMap* tm_k;
  const CUtensorMap* tm_v;
  const void* q;
  long long q_sn, q_sh;      // elements
  void* o;
  long long o_sn, o_sh;
  float* lse;                // [T][HQ]
  const int* table;
  long long table_sb;
  const int* kv_lens;
  const int* cu;             // null: one token a sequence
  int B, T, HQ, HK, d, type, causal;
  int page_shift, num_pages, max_pages;
  int max_q, max_kv;
  float scale;
  int q_tiles;               // query tiles of a (sequence, key head)
  int row_tiles;             // 128-row tiles of a CTA (1 or 2)
  int splits, split_tiles;   // key splits and key tiles of one
  int by_length;             // the longest sequences' CTAs first (at most 32 sequences)
  int whole;                 // few rows: each CTA takes whole (sequence, key head) pairs, no parts
  float* part_o;             // [splits][T][HQ][d]; null without splits
  float* part_lse;           // [splits][T][HQ], log2 units
  int* dev_status;
  uint64_t timeout_ns;
};

// Blocks of the backward's persistent grid (its partials' row count).
int rope_bwd_blocks(int B, int NQ, int HQ, int NK, int HK, int d, int sms);

cudaError_t launch_rope_fwd(RopeArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_rope_bwd(RopeArgs& a, int blocks, int sms, float* dw_q, float* dw_k, cudaStream_t stream);
cudaError_t launch_append(AppendArgs& a, int sms, cudaStream_t stream);
// At most kDecodeRows rows (token, head of the group) per sequence and key
// head: `ctas` persistent CTAs share the key tiles evenly, at least split_tiles
// each; part_o [2 ctas][kDecodeRows][d] and part_lse hold the parts of items
// that they share.
constexpr int kDecodeRows = 32;
cudaError_t launch_paged_decode(const PagedAttnArgs& a, int ctas, cudaStream_t stream);
cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t stream);

}  // namespace skl
