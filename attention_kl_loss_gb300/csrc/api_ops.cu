// C-ABI layer of the operators around the attention-KL call: argument checks,
// tensor maps of the paged cache, key-split choice, launches. Like api.cu: no
// allocation, no synchronisation, everything on the caller's stream.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "streamkl.h"
#include "host.h"
#include "ops.h"

namespace {

using namespace skl::host;

static_assert(STREAMKL_BF16 == skl::kTypeBf16 && STREAMKL_FP16 == skl::kTypeF16 &&
                  STREAMKL_FP32 == skl::kTypeF32,
              "element types of the header and the kernels agree");

constexpr long long kMaxRows = 1LL << 30;  // rows (tokens x heads) of one tensor

size_t elem_size(int dtype) { return dtype == STREAMKL_FP32 ? 4 : 2; }

// The struct of a call, copied; false (with the error set) for another size.
template <typename A>
bool take_args(A* to, const A* from) {
  clear_error();
  if (from && from->struct_size == sizeof(A)) {
    *to = *from;
    return true;
  }
  fail(STREAMKL_ERR_INVALID_ARG, "struct_size is %zu, expected %zu", from ? from->struct_size : 0, sizeof(A));
  return false;
}

// Rows of d contiguous elements in dimensions of the sizes given (0: not
// used). The stride of a dimension of size 1 says nothing and becomes d.
// `own_rows`: the rows must be apart (outputs, caches), so each stride spans all
// that the smaller ones reach; inputs may repeat rows (stride 0).
streamkl_status check_rows(const char* name, streamkl_rows* r, int s0, int s1, int s2, int d, int dtype,
                           bool own_rows) {
  if (!r->data) return fail(STREAMKL_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned16(r->data)) return fail(STREAMKL_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  const int sizes[3] = {s0, s1, s2};
  for (int i = 0; i < 3; ++i) {
    long long& s = r->stride[i];
    if (sizes[i] <= 1) s = d;
    if (s < 0 || s * static_cast<long long>(elem_size(dtype)) % 16)
      return fail(STREAMKL_ERR_INVALID_ARG, "%s: stride %lld is not a multiple of 16 bytes", name, s);
    if (own_rows && s < d) return fail(STREAMKL_ERR_INVALID_ARG, "%s: stride %lld below one row of %d", name, s, d);
  }
  if (own_rows) {
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int x, int y) { return r->stride[x] < r->stride[y]; });
    double reach = d;  // (elements; in a double, since a stride can be anything)
    for (int i : order) {
      if (sizes[i] <= 1) continue;
      if (static_cast<double>(r->stride[i]) < reach)
        return fail(STREAMKL_ERR_INVALID_ARG, "%s: its rows overlap (stride %lld, %.0f elements within)", name,
                    r->stride[i], reach);
      reach += static_cast<double>(r->stride[i]) * (sizes[i] - 1);
    }
  }
  return STREAMKL_OK;
}

streamkl_status check_rope(int d, int rot, const float* cos, const float* sin, int table_len, float eps,
                           int interleaved) {
  if (d != 64 && d != 128) return fail(STREAMKL_ERR_UNSUPPORTED, "head dim d=%d (supported: 64, 128)", d);
  if (rot < 16 || rot > d || rot % 16)
    return fail(STREAMKL_ERR_UNSUPPORTED, "rotated elements %d (supported: multiples of 16 up to d)", rot);
  if (!cos || !sin) return fail(STREAMKL_ERR_INVALID_ARG, "cos and sin must be non-NULL");
  if (!aligned16(cos) || !aligned16(sin))
    return fail(STREAMKL_ERR_INVALID_ARG, "cos and sin must be 16-byte aligned");
  if (table_len < 1) return fail(STREAMKL_ERR_INVALID_ARG, "cos and sin need at least one row");
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(STREAMKL_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (interleaved != 0 && interleaved != 1) return fail(STREAMKL_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  return STREAMKL_OK;
}

skl::RowStrides row_strides(const streamkl_rows& r) { return skl::RowStrides{r.stride[0], r.stride[1], r.stride[2]}; }

// The part of a norm + rotation call that both directions share: the
// arguments' checks and the kernels' arguments without gradients.
streamkl_status rope_common(skl::RopeArgs* a, streamkl_rope_args* u, bool backward) {
  const bool q = u->q.data, k = u->k.data;
  if (!q && !k) return fail(STREAMKL_ERR_INVALID_ARG, "q and k are both NULL");
  if (u->dtype != STREAMKL_BF16 && u->dtype != STREAMKL_FP16 && u->dtype != STREAMKL_FP32)
    return fail(STREAMKL_ERR_UNSUPPORTED, "element type %d", u->dtype);
  streamkl_status st = check_rope(u->d, u->rot, u->cos, u->sin, u->table_len, u->eps, u->interleaved);
  if (st != STREAMKL_OK) return st;
  if (u->B < 1 || (q && (u->NQ < 1 || u->HQ < 1)) || (k && (u->NK < 1 || u->HK < 1)) || u->k_repeat < 1)
    return fail(STREAMKL_ERR_INVALID_ARG, "sizes must be >= 1 (B=%d NQ=%d HQ=%d NK=%d HK=%d k_repeat=%d)", u->B,
                u->NQ, u->HQ, u->NK, u->HK, u->k_repeat);
  if (!q) u->NQ = u->HQ = 0;
  if (!k) u->NK = u->HK = 0;
  if (static_cast<long long>(u->NQ) * u->HQ > kMaxRows / u->B ||
      static_cast<long long>(u->NK) * u->HK > kMaxRows / u->B / u->k_repeat)
    return fail(STREAMKL_ERR_UNSUPPORTED, "tokens x heads above 2^30");
  if (q && k && !u->q_positions && u->NQ > u->NK)
    return fail(STREAMKL_ERR_INVALID_ARG, "more queries than keys (%d > %d) need q_positions", u->NQ, u->NK);
  if (!u->dev_status) return fail(STREAMKL_ERR_INVALID_ARG, "dev_status must be non-NULL");
  *a = skl::RopeArgs{};
  for (int i = 0; i < 2; ++i) {
    streamkl_rows &in = i ? u->k : u->q, &outer = i ? u->k_out : u->q_out, &grad = i ? u->dk : u->dq;
    if (!in.data) continue;
    skl::RopeSide& s = a->side[i];
    s.N = i ? u->NK : u->NQ;
    s.H = i ? u->HK : u->HQ;
    s.rep = i ? u->k_repeat : 1;
    s.w = i ? u->k_weight : u->q_weight;
    s.pos = i ? u->k_positions : u->q_positions;
    s.pos_sb = i ? u->k_pos_stride : u->q_pos_stride;
    s.pos0 = i || !k ? 0 : std::max(u->NK - u->NQ, 0);
    if ((st = check_rows(i ? "k" : "q", &in, u->B, s.N, s.H, u->d, u->dtype, false)) != STREAMKL_OK) return st;
    if ((st = check_rows(i ? "k_out" : "q_out", &outer, u->B, s.N, s.H * s.rep, u->d, u->dtype, !backward)) !=
        STREAMKL_OK)
      return st;
    if (backward && (st = check_rows(i ? "dk" : "dq", &grad, u->B, s.N, s.H, u->d, u->dtype, true)) != STREAMKL_OK)
      return st;
    if (s.w && !aligned16(s.w))
      return fail(STREAMKL_ERR_INVALID_ARG, "%s is not 16-byte aligned", i ? "k_weight" : "q_weight");
    s.x = in.data;
    s.xs = row_strides(in);
    s.y_in = s.y_out = outer.data;
    s.ys = row_strides(outer);
    s.dx = grad.data;
    s.dxs = row_strides(grad);
  }
  a->B = u->B;
  a->d = u->d;
  a->rot = u->rot;
  a->type = u->dtype;
  a->interleaved = u->interleaved;
  a->table_len = u->table_len;
  a->cos = u->cos;
  a->sin = u->sin;
  a->eps = u->eps;
  a->dev_status = u->dev_status;
  return STREAMKL_OK;
}

streamkl_status check_cache(streamkl_rows* kc, streamkl_rows* vc, const int* table, long long table_stride,
                            const int* kv_lens, const int* cu_seqlens, int dtype, int B, int T, int HK, int d,
                            int page_size, int num_pages, int max_pages) {
  if (dtype != STREAMKL_BF16 && dtype != STREAMKL_FP16)
    return fail(STREAMKL_ERR_UNSUPPORTED, "cache element type %d (supported: bf16, fp16)", dtype);
  if (d != 64 && d != 128) return fail(STREAMKL_ERR_UNSUPPORTED, "head dim d=%d (supported: 64, 128)", d);
  if (B < 1 || T < 1 || HK < 1 || num_pages < 1 || max_pages < 1)
    return fail(STREAMKL_ERR_INVALID_ARG, "sizes must be >= 1 (B=%d T=%d HK=%d num_pages=%d max_pages=%d)", B, T,
                HK, num_pages, max_pages);
  if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)))
    return fail(STREAMKL_ERR_UNSUPPORTED, "page size %d (supported: powers of two from 16 to 1024)", page_size);
  if (static_cast<long long>(max_pages) * page_size > (1LL << 30))
    return fail(STREAMKL_ERR_UNSUPPORTED, "sequence length above 2^30");
  if (!table || !kv_lens) return fail(STREAMKL_ERR_INVALID_ARG, "block_table and kv_lens must be non-NULL");
  if (table_stride < 0) return fail(STREAMKL_ERR_INVALID_ARG, "block_table stride %lld", table_stride);
  if (!cu_seqlens && T != B)
    return fail(STREAMKL_ERR_INVALID_ARG, "without cu_seqlens each sequence has one token (T=%d B=%d)", T, B);
  streamkl_status st = check_rows("k_cache", kc, num_pages, HK, page_size, d, dtype, true);
  return st != STREAMKL_OK ? st : check_rows("v_cache", vc, num_pages, HK, page_size, d, dtype, true);
}

// How the attention over the cache is cut into CTAs. Few rows (decode) go to
// the persistent kernel, which deals the key tiles out evenly by itself, or a
// short (sequence, key head) to each CTA. With
// more, the keys of few query tiles against long sequences are cut into
// `splits` ranges of split_tiles 128-key tiles (counted from a sequence's
// start, so a short one uses fewer ranges).
struct AttnPlan {
  int decode_ctas;  // 0: not the persistent kernel
  bool whole;       // there: each CTA takes whole (sequence, key head) pairs
  int row_tiles, q_tiles, splits, split_tiles;
};

AttnPlan attn_plan(int B, int T, int HQ, int HK, int d, int max_q, int max_kv, int requested) {
  AttnPlan p{};
  const long long rows = static_cast<long long>(max_q) * (HQ / HK);
  if (requested == 0 && rows <= skl::kDecodeRows) {
    const long long ctas = 2LL * num_sms(), items = static_cast<long long>(B) * HK;
    const long long tiles = std::max(1, (max_kv + 127) / 128), all = items * tiles;
    // Whole items, without a search and without parts to join, where the longest
    // row of them is four tiles or one more than an equal share (8 key heads of
    // 128, one sequence of 128 keys 10.1 -> 6.7 us, of 512 level, of 768 10.9 -> 14.3
    // the other way; 64 sequences of up to 256 keys, two a CTA, 19.1 -> 16.7, 100 of
    // up to 512 34.8 -> 32.3, of 1,024 50.8 -> 52.5 the other way)
    p.split_tiles = 2;  // (one tile each is level: one sequence of 4,096 keys 18.7 us against 18.4)
    p.whole = (items + ctas - 1) / ctas * tiles <= std::max<long long>(4, (all + ctas - 1) / ctas + 1);
    p.decode_ctas = static_cast<int>(std::min(p.whole ? items : all, ctas));
    return p;
  }
  p.row_tiles = rows > 128 ? 2 : 1;
  p.q_tiles = static_cast<int>((rows + 128 * p.row_tiles - 1) / (128 * p.row_tiles));
  const int tiles = std::max(1, (max_kv + 127) / 128);
  int s = requested;
  if (s <= 0) {
    // A tile's time, a CTA's own, and the joining of partials. One sequence's CTAs
    // come in whole waves; of several sequences, which are seldom all of the largest
    // size, 3/4 of the CTAs have work and one follows another as it ends. The
    // constants are those that come nearest to the best split of 48 shapes (1 to
    // 100 sequences, 16 to 2,048 new tokens, 300 to 131,072 keys): 1.4 % from it, 22 %
    // at worst (five chunks of up to 400 rows over up to 3,000 keys: 43 us whole, 31
    // in two splits, 26 in three).
    const int sms = num_sms();
    const double ctas = static_cast<double>(p.q_tiles) * B * HK * (B > 1 ? 0.75 : 1.0);
    const double tile_us = d == 128 ? 1.5 : 1.1, cta_us = 5.0, join_us = 5.0, whole = B > 1 ? 0.1 : 1.0;
    const double part_us = static_cast<double>(T) * HQ * (d + 1) * 8.0 / 6.0e12 * 1e6;
    auto cost = [&](int n) {
      const int per = (tiles + n - 1) / n;
      const double waves = ctas * ((tiles + per - 1) / per) / sms;
      const double turns = std::max(1.0, whole * std::ceil(waves - 1e-9) + (1.0 - whole) * waves);
      return turns * (per * tile_us + cta_us) + (n > 1 ? join_us + n * part_us : 0.0);
    };
    s = 1;
    double best = cost(1);
    for (int n = 2; n <= std::min(64, tiles); ++n)
      if (cost(n) < best) {
        best = cost(n);
        s = n;
      }
  }
  s = std::max(1, std::min(s, tiles));
  p.split_tiles = (tiles + s - 1) / s;
  p.splits = (tiles + p.split_tiles - 1) / p.split_tiles;
  return p;
}

// Rows of the partial results.
size_t attn_part_rows(const AttnPlan& p, int T, int HQ) {
  if (p.whole) return 0;
  if (p.decode_ctas > 0) return static_cast<size_t>(2) * p.decode_ctas * skl::kDecodeRows;
  return p.splits > 1 ? static_cast<size_t>(p.splits) * T * HQ : 0;
}

size_t attn_part_bytes(const AttnPlan& p, int T, int HQ, int d) {
  return (attn_part_rows(p, T, HQ) * (d + 1) * sizeof(float) + 255) & ~static_cast<size_t>(255);
}

// 4-D map {d, page size, HK, pages} of a cache, 64-column boxes of one page's
// slots (at most one key tile of them), 128-byte swizzle.
streamkl_status make_map_cache(CUtensorMap* m, const streamkl_rows& cache, int dtype, int d, int page_size, int HK,
                               int num_pages, const char* name) {
  auto enc = encode_fn();
  if (!enc) return fail(STREAMKL_ERR_CUDA, "cuTensorMapEncodeTiled unavailable from the driver");
  const cuuint64_t gdim[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(page_size),
                              static_cast<cuuint64_t>(HK), static_cast<cuuint64_t>(num_pages)};
  const cuuint64_t gstride[3] = {static_cast<cuuint64_t>(cache.stride[2]) * 2, static_cast<cuuint64_t>(cache.stride[1]) * 2,
                                 static_cast<cuuint64_t>(cache.stride[0]) * 2};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(std::min(page_size, 128)), 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUtensorMapDataType type =
      dtype == STREAMKL_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUresult r = enc(m, type, 4, cache.data, gdim, gstride, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(STREAMKL_ERR_CUDA, "tensor map for %s failed (CUresult %d)", name, static_cast<int>(r));
  return STREAMKL_OK;
}

streamkl_status check_attn_sizes(int B, int T, int HQ, int HK, int d, int max_q, int max_kv) {
  if (B < 1 || T < 1 || HQ < 1 || HK < 1 || max_q < 1 || max_kv < 0)
    return fail(STREAMKL_ERR_INVALID_ARG, "sizes must be >= 1 (B=%d T=%d HQ=%d HK=%d max_seqlen_q=%d max_kv_len=%d)",
                B, T, HQ, HK, max_q, max_kv);
  if (HQ % HK) return fail(STREAMKL_ERR_INVALID_ARG, "query heads %d are not a multiple of key heads %d", HQ, HK);
  if (d != 64 && d != 128) return fail(STREAMKL_ERR_UNSUPPORTED, "head dim d=%d (supported: 64, 128)", d);
  if (static_cast<long long>(B) * HK > 65535)
    return fail(STREAMKL_ERR_UNSUPPORTED, "B*HK=%lld exceeds 65535", static_cast<long long>(B) * HK);
  if (max_q > T) return fail(STREAMKL_ERR_INVALID_ARG, "max_seqlen_q %d above the %d tokens", max_q, T);
  if (static_cast<long long>(T) * HQ > (1LL << 30) || max_kv > (1 << 30))
    return fail(STREAMKL_ERR_UNSUPPORTED, "more than 2^30 rows or keys");
  return STREAMKL_OK;
}

}  // namespace

extern "C" {

streamkl_status streamkl_qk_norm_rope_fwd(const streamkl_rope_args* args, void* stream) {
  streamkl_rope_args u;
  if (!take_args(&u, args)) return STREAMKL_ERR_INVALID_ARG;
  skl::RopeArgs a;
  streamkl_status st = rope_common(&a, &u, false);
  if (st != STREAMKL_OK) return st;
  cudaError_t e = skl::launch_rope_fwd(a, num_sms(), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? STREAMKL_OK : cuda_fail(e, "norm + rotation launch");
}

size_t streamkl_qk_norm_rope_bwd_workspace_size(int B, int NQ, int NK, int HQ, int HK, int d) {
  if (B < 1 || NQ < 0 || NK < 0 || HQ < 0 || HK < 0 || (d != 64 && d != 128)) return 0;
  return static_cast<size_t>(2) * skl::rope_bwd_blocks(B, NQ, HQ, NK, HK, d, num_sms()) * d * sizeof(float);
}

streamkl_status streamkl_qk_norm_rope_bwd(const streamkl_rope_args* args, void* stream) {
  streamkl_rope_args u;
  if (!take_args(&u, args)) return STREAMKL_ERR_INVALID_ARG;
  skl::RopeArgs a;
  streamkl_status st = rope_common(&a, &u, true);
  if (st != STREAMKL_OK) return st;
  float* dwq = u.q.data && u.q_weight ? u.dq_weight : nullptr;
  float* dwk = u.k.data && u.k_weight ? u.dk_weight : nullptr;
  if ((u.q.data && u.q_weight && !dwq) || (u.k.data && u.k_weight && !dwk))
    return fail(STREAMKL_ERR_INVALID_ARG, "a norm weight needs its gradient's buffer");
  const int blocks = skl::rope_bwd_blocks(u.B, u.NQ, u.HQ, u.NK, u.HK, u.d, num_sms());
  const size_t need = dwq || dwk ? static_cast<size_t>(2) * blocks * u.d * sizeof(float) : 0;
  if (need && (!u.workspace || u.ws_bytes < need))
    return fail(STREAMKL_ERR_INVALID_ARG, "workspace of %zu bytes, need %zu", u.workspace ? u.ws_bytes : 0, need);
  if (need && !aligned16(u.workspace)) return fail(STREAMKL_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
  a.part = static_cast<float*>(u.workspace);
  cudaError_t e = skl::launch_rope_bwd(a, blocks, num_sms(), dwq, dwk, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? STREAMKL_OK : cuda_fail(e, "norm + rotation backward launch");
}

streamkl_status streamkl_paged_append(const streamkl_append_args* args, void* stream) {
  streamkl_append_args u;
  if (!take_args(&u, args)) return STREAMKL_ERR_INVALID_ARG;
  if (static_cast<long long>(u.T) * u.HK > kMaxRows) return fail(STREAMKL_ERR_UNSUPPORTED, "tokens x heads above 2^30");
  streamkl_status st = check_cache(&u.k_cache, &u.v_cache, u.block_table, u.table_stride, u.kv_lens, u.cu_seqlens,
                                   u.dtype, u.B, u.T, u.HK, u.d, u.page_size, u.num_pages, u.max_pages);
  if (st != STREAMKL_OK) return st;
  if (u.table_stride < u.max_pages && u.B > 1)  // (to read them the sequences may share a row)
    return fail(STREAMKL_ERR_INVALID_ARG, "block_table rows overlap (stride %lld, %d pages)", u.table_stride,
                u.max_pages);
  if ((st = check_rows("k", &u.k, 0, u.T, u.HK, u.d, u.dtype, false)) != STREAMKL_OK) return st;
  if ((st = check_rows("v", &u.v, 0, u.T, u.HK, u.d, u.dtype, false)) != STREAMKL_OK) return st;
  if ((u.cos == nullptr) != (u.sin == nullptr))
    return fail(STREAMKL_ERR_INVALID_ARG, "cos and sin must be both NULL or both non-NULL");
  if (u.cos && (st = check_rope(u.d, u.rot, u.cos, u.sin, u.table_len, u.eps, u.interleaved)) != STREAMKL_OK) return st;
  if (!(u.eps >= 0.f) || !std::isfinite(u.eps)) return fail(STREAMKL_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (u.k_weight && !aligned16(u.k_weight)) return fail(STREAMKL_ERR_INVALID_ARG, "k_weight is not 16-byte aligned");
  if (!u.dev_status) return fail(STREAMKL_ERR_INVALID_ARG, "dev_status must be non-NULL");
  skl::AppendArgs a{};
  a.k = u.k.data;
  a.v = u.v.data;
  a.ks = row_strides(u.k);
  a.vs = row_strides(u.v);
  a.kc = u.k_cache.data;
  a.vc = u.v_cache.data;
  a.kc_sp = u.k_cache.stride[0], a.kc_sh = u.k_cache.stride[1], a.kc_ss = u.k_cache.stride[2];
  a.vc_sp = u.v_cache.stride[0], a.vc_sh = u.v_cache.stride[1], a.vc_ss = u.v_cache.stride[2];
  a.table = u.block_table;
  a.table_sb = u.table_stride;
  a.kv_lens = u.kv_lens;
  a.cu = u.cu_seqlens;
  a.B = u.B;
  a.T = u.T;
  a.H = u.HK;
  a.d = u.d;
  a.rot = u.cos ? u.rot : u.d;
  a.type = u.dtype;
  a.interleaved = u.cos ? u.interleaved : 0;
  a.page_shift = __builtin_ctz(static_cast<unsigned>(u.page_size));
  a.num_pages = u.num_pages;
  a.max_pages = u.max_pages;
  a.table_len = u.table_len;
  a.cos = u.cos;
  a.sin = u.sin;
  a.w = u.k_weight;
  a.eps = u.eps;
  a.dev_status = u.dev_status;
  cudaError_t e = skl::launch_append(a, num_sms(), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? STREAMKL_OK : cuda_fail(e, "append launch");
}

int streamkl_paged_attn_splits(int B, int T, int HQ, int HK, int d, int max_seqlen_q, int max_kv_len) {
  if (check_attn_sizes(B, T, HQ, HK, d, max_seqlen_q, max_kv_len) != STREAMKL_OK) return -1;
  return attn_plan(B, T, HQ, HK, d, max_seqlen_q, max_kv_len, 0).splits;
}

size_t streamkl_paged_attn_workspace_size(int B, int T, int HQ, int HK, int d, int max_seqlen_q, int max_kv_len,
                                          int num_splits) {
  if (check_attn_sizes(B, T, HQ, HK, d, max_seqlen_q, max_kv_len) != STREAMKL_OK || num_splits < 0) return 0;
  return attn_part_bytes(attn_plan(B, T, HQ, HK, d, max_seqlen_q, max_kv_len, num_splits), T, HQ, d);
}

streamkl_status streamkl_paged_attn(const streamkl_paged_attn_args* args, void* stream) {
  streamkl_paged_attn_args u;
  if (!take_args(&u, args)) return STREAMKL_ERR_INVALID_ARG;
  streamkl_status st = check_cache(&u.k_cache, &u.v_cache, u.block_table, u.table_stride, u.kv_lens, u.cu_seqlens,
                                   u.dtype, u.B, u.T, u.HK, u.d, u.page_size, u.num_pages, u.max_pages);
  if (st != STREAMKL_OK) return st;
  if ((st = check_attn_sizes(u.B, u.T, u.HQ, u.HK, u.d, u.max_seqlen_q, u.max_kv_len)) != STREAMKL_OK) return st;
  if (u.max_kv_len > static_cast<long long>(u.max_pages) * u.page_size)
    return fail(STREAMKL_ERR_INVALID_ARG, "max_kv_len %d above %d pages of %d", u.max_kv_len, u.max_pages, u.page_size);
  if ((st = check_rows("q", &u.q, 0, u.T, u.HQ, u.d, u.dtype, false)) != STREAMKL_OK) return st;
  if ((st = check_rows("out", &u.out, 0, u.T, u.HQ, u.d, u.dtype, true)) != STREAMKL_OK) return st;
  if (!u.lse) return fail(STREAMKL_ERR_INVALID_ARG, "lse must be non-NULL");
  if (u.causal != 0 && u.causal != 1) return fail(STREAMKL_ERR_INVALID_ARG, "causal must be 0 or 1");
  if (u.num_splits < 0) return fail(STREAMKL_ERR_INVALID_ARG, "num_splits must be >= 0");
  if (!(u.scale > 0.f) || !std::isfinite(u.scale))
    return fail(STREAMKL_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (!u.dev_status) return fail(STREAMKL_ERR_INVALID_ARG, "dev_status must be non-NULL");
  const AttnPlan p = attn_plan(u.B, u.T, u.HQ, u.HK, u.d, u.max_seqlen_q, u.max_kv_len, u.num_splits);
  if (p.splits > 65535) return fail(STREAMKL_ERR_UNSUPPORTED, "%d key splits (at most 65535)", p.splits);
  const size_t need = attn_part_bytes(p, u.T, u.HQ, u.d);
  if (need && (!u.workspace || u.ws_bytes < need))
    return fail(STREAMKL_ERR_INVALID_ARG, "workspace of %zu bytes, need %zu", u.workspace ? u.ws_bytes : 0, need);
  if (need && !aligned16(u.workspace)) return fail(STREAMKL_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
  CUtensorMap mk, mv;
  if ((st = make_map_cache(&mk, u.k_cache, u.dtype, u.d, u.page_size, u.HK, u.num_pages, "k_cache")) != STREAMKL_OK)
    return st;
  if ((st = make_map_cache(&mv, u.v_cache, u.dtype, u.d, u.page_size, u.HK, u.num_pages, "v_cache")) != STREAMKL_OK)
    return st;
  skl::PagedAttnArgs a{};
  a.tm_k = &mk;
  a.tm_v = &mv;
  a.q = u.q.data;
  a.q_sn = u.q.stride[1], a.q_sh = u.q.stride[2];
  a.o = u.out.data;
  a.o_sn = u.out.stride[1], a.o_sh = u.out.stride[2];
  a.lse = u.lse;
  a.table = u.block_table;
  a.table_sb = u.table_stride;
  a.kv_lens = u.kv_lens;
  a.cu = u.cu_seqlens;
  a.B = u.B;
  a.T = u.T;
  a.HQ = u.HQ;
  a.HK = u.HK;
  a.d = u.d;
  a.type = u.dtype;
  a.causal = u.causal;
  a.page_shift = __builtin_ctz(static_cast<unsigned>(u.page_size));
  a.num_pages = u.num_pages;
  a.max_pages = u.max_pages;
  a.max_q = u.max_seqlen_q;
  a.max_kv = u.max_kv_len;
  a.scale = u.scale;
  a.q_tiles = p.q_tiles;
  a.row_tiles = p.row_tiles;
  a.splits = p.splits;
  a.split_tiles = p.split_tiles;
  a.whole = p.whole;
  // more than one CTA per SM one after the other: long ones first, so that the
  // last to start are short (four ragged chunks of up to 2,048 rows over 16,384
  // keys, d = 64: 250 us against 258)
  a.by_length = u.B > 1 && u.B <= 32 && static_cast<long long>(p.q_tiles) * u.B * u.HK > num_sms();
  a.part_o = static_cast<float*>(u.workspace);
  a.part_lse = a.part_o ? a.part_o + attn_part_rows(p, u.T, u.HQ) * u.d : nullptr;
  a.dev_status = u.dev_status;
  a.timeout_ns = wait_timeout_ns();
  cudaError_t e = p.decode_ctas > 0 ? skl::launch_paged_decode(a, p.decode_ctas, static_cast<cudaStream_t>(stream))
                                    : skl::launch_paged_attn(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? STREAMKL_OK : cuda_fail(e, "paged attention launch");
}

}  // extern "C"
