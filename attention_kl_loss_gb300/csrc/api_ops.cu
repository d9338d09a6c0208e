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

constexpr long long kMaxRows = 1LL << 31;  // rows (tokens x heads) of one tensor

size_t elem_size(int dtype) { return dtype == STREAMKL_FP32 ? 4 : 2; }

// A tensor of n strided dimensions over rows of d contiguous elements. The
// stride of a dimension of size 1 says nothing and becomes d. `own_rows`: the
// rows must be apart (outputs, caches); inputs may repeat rows (stride 0).
streamkl_status check_tensor(const char* name, const void* p, long long* strides, const int* sizes, int n, int d,
                             int dtype, bool own_rows) {
  if (!p) return fail(STREAMKL_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned16(p)) return fail(STREAMKL_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  for (int i = 0; i < n; ++i) {
    if (sizes[i] == 1) strides[i] = d;
    if (strides[i] < 0 || strides[i] * static_cast<long long>(elem_size(dtype)) % 16)
      return fail(STREAMKL_ERR_INVALID_ARG, "%s: stride %lld is not a multiple of 16 bytes", name, strides[i]);
    if (own_rows && strides[i] < d)
      return fail(STREAMKL_ERR_INVALID_ARG, "%s: stride %lld below one row of %d", name, strides[i], d);
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

skl::RowStrides row_strides(const long long* s) { return skl::RowStrides{s[0], s[1], s[2]}; }

// The part of a norm + rotation call that both directions share: the
// arguments' checks and a's sides without their outer rows.
streamkl_status rope_common(skl::RopeArgs* a, const void* q, const void* k, int dtype, int B, int NQ, int NK,
                            int HQ, int HK, int d, int rot, long long* strides, const float* cos,
                            const float* sin, int table_len, const int* q_pos, long long q_pos_stride,
                            const int* k_pos, long long k_pos_stride, const float* q_weight,
                            const float* k_weight, float eps, int interleaved, int k_repeat, int* dev_status) {
  if (!q && !k) return fail(STREAMKL_ERR_INVALID_ARG, "q and k are both NULL");
  if (dtype != STREAMKL_BF16 && dtype != STREAMKL_FP16 && dtype != STREAMKL_FP32)
    return fail(STREAMKL_ERR_UNSUPPORTED, "element type %d", dtype);
  streamkl_status st = check_rope(d, rot, cos, sin, table_len, eps, interleaved);
  if (st != STREAMKL_OK) return st;
  if (B < 1 || (q && (NQ < 1 || HQ < 1)) || (k && (NK < 1 || HK < 1)) || k_repeat < 1)
    return fail(STREAMKL_ERR_INVALID_ARG, "sizes must be >= 1 (B=%d NQ=%d HQ=%d NK=%d HK=%d k_repeat=%d)", B,
                NQ, HQ, NK, HK, k_repeat);
  if ((q && static_cast<long long>(NQ) * HQ > kMaxRows / B) ||
      (k && static_cast<long long>(NK) * HK > kMaxRows / B / k_repeat))
    return fail(STREAMKL_ERR_UNSUPPORTED, "rows x heads above 2^31");
  if (q && k && !q_pos && NQ > NK)
    return fail(STREAMKL_ERR_INVALID_ARG, "more queries than keys (%d > %d) need q_positions", NQ, NK);
  if (!dev_status) return fail(STREAMKL_ERR_INVALID_ARG, "dev_status must be non-NULL");
  const int sq[3] = {B, NQ, HQ}, sk[3] = {B, NK, HK};
  if (q && (st = check_tensor("q", q, strides, sq, 3, d, dtype, false)) != STREAMKL_OK) return st;
  if (k && (st = check_tensor("k", k, strides + 3, sk, 3, d, dtype, false)) != STREAMKL_OK) return st;
  *a = skl::RopeArgs{};
  a->side[0].x = q;
  a->side[0].xs = row_strides(strides);
  a->side[0].pos = q_pos;
  a->side[0].pos_sb = q_pos_stride;
  a->side[0].pos0 = (k && NK > NQ) ? NK - NQ : 0;
  a->side[0].w = q_weight;
  a->side[0].N = NQ;
  a->side[0].H = HQ;
  a->side[0].rep = 1;
  a->side[1].x = k;
  a->side[1].xs = row_strides(strides + 3);
  a->side[1].pos = k_pos;
  a->side[1].pos_sb = k_pos_stride;
  a->side[1].w = k_weight;
  a->side[1].N = NK;
  a->side[1].H = HK;
  a->side[1].rep = k_repeat;
  for (int i = 0; i < 2; ++i) {
    a->side[i].ys = skl::RowStrides{0, 0, 0};
    a->side[i].dxs = skl::RowStrides{0, 0, 0};
  }
  a->B = B;
  a->d = d;
  a->rot = rot;
  a->type = dtype;
  a->interleaved = interleaved;
  a->table_len = table_len;
  a->cos = cos;
  a->sin = sin;
  a->eps = eps;
  a->dev_status = dev_status;
  return STREAMKL_OK;
}

streamkl_status check_cache(const void* kc, const void* vc, const int* table, long long table_stride,
                            const int* kv_lens, int dtype, int B, int T, int HK, int d, int page_size,
                            int num_pages, int max_pages, long long* strides) {
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
  if (table_stride < max_pages && B > 1)
    return fail(STREAMKL_ERR_INVALID_ARG, "block_table rows overlap (stride %lld, %d pages)", table_stride, max_pages);
  const int sizes[3] = {num_pages, HK, page_size};
  streamkl_status st = check_tensor("k_cache", kc, strides, sizes, 3, d, dtype, true);
  if (st != STREAMKL_OK) return st;
  return check_tensor("v_cache", vc, strides + 3, sizes, 3, d, dtype, true);
}

// Key split of the attention over the cache: with few query tiles against
// long sequences the keys are cut into `splits` ranges of split_tiles 128-key
// tiles (counted from a sequence's start, so a short one uses fewer ranges).
struct AttnPlan {
  int row_tiles, q_tiles, splits, split_tiles;
};

AttnPlan attn_plan(int B, int T, int HQ, int HK, int d, int max_q, int max_kv, int requested) {
  AttnPlan p;
  const long long rows = static_cast<long long>(max_q) * (HQ / HK);
  p.row_tiles = rows > 128 ? 2 : 1;
  p.q_tiles = static_cast<int>((rows + 128 * p.row_tiles - 1) / (128 * p.row_tiles));
  const int tiles = std::max(1, (max_kv + 127) / 128);
  int s = requested;
  if (s <= 0) {
    const int sms = num_sms();
    const long long ctas = static_cast<long long>(p.q_tiles) * B * HK;
    const double tile_us = (p.row_tiles == 2 ? 1.2 : 0.7) * (d == 128 ? 1.0 : 0.6), cta_us = 4.0;
    const double part_us = static_cast<double>(T) * HQ * (d + 1) * 8.0 / 4.0e12 * 1e6;
    auto cost = [&](int n) {
      const long long waves = (ctas * n + sms - 1) / sms;
      const int per = (tiles + n - 1) / n;
      return waves * (per * tile_us + cta_us) + (n > 1 ? 3.0 + n * part_us : 0.0);
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

size_t attn_part_bytes(int splits, int T, int HQ, int d) {
  if (splits <= 1) return 0;
  const size_t rows = static_cast<size_t>(splits) * T * HQ;
  return (rows * (d + 1) * sizeof(float) + 255) & ~static_cast<size_t>(255);
}

// 4-D map {d, page size, HK, pages} of a cache, 64-column boxes of one page's
// slots (at most one key tile of them), 128-byte swizzle.
streamkl_status make_map_cache(CUtensorMap* m, const void* ptr, int dtype, int d, int page_size, int HK,
                               int num_pages, const long long* strides, const char* name) {
  auto enc = encode_fn();
  if (!enc) return fail(STREAMKL_ERR_CUDA, "cuTensorMapEncodeTiled unavailable from the driver");
  const cuuint64_t gdim[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(page_size),
                              static_cast<cuuint64_t>(HK), static_cast<cuuint64_t>(num_pages)};
  const cuuint64_t gstride[3] = {static_cast<cuuint64_t>(strides[2]) * 2, static_cast<cuuint64_t>(strides[1]) * 2,
                                 static_cast<cuuint64_t>(strides[0]) * 2};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(std::min(page_size, 128)), 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUtensorMapDataType type =
      dtype == STREAMKL_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUresult r = enc(m, type, 4, const_cast<void*>(ptr), gdim, gstride, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
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

streamkl_status streamkl_qk_norm_rope_fwd(const void* q, const void* k, int dtype, int B, int NQ, int NK, int HQ,
                                          int HK, int d, int rot, const long long* strides, const float* cos,
                                          const float* sin, int table_len, const int* q_positions,
                                          long long q_pos_stride, const int* k_positions, long long k_pos_stride,
                                          const float* q_weight, const float* k_weight, float eps, int interleaved,
                                          int k_repeat, void* q_out, void* k_out, int* dev_status, void* stream) {
  clear_error();
  if (!strides) return fail(STREAMKL_ERR_INVALID_ARG, "strides is NULL");
  long long s[12];
  std::copy(strides, strides + 12, s);
  skl::RopeArgs a;
  streamkl_status st = rope_common(&a, q, k, dtype, B, NQ, NK, HQ, HK, d, rot, s, cos, sin, table_len,
                                   q_positions, q_pos_stride, k_positions, k_pos_stride, q_weight, k_weight, eps,
                                   interleaved, k_repeat, dev_status);
  if (st != STREAMKL_OK) return st;
  const int oq[3] = {B, NQ, HQ}, ok[3] = {B, NK, HK * k_repeat};
  if (q && (st = check_tensor("q_out", q_out, s + 6, oq, 3, d, dtype, true)) != STREAMKL_OK) return st;
  if (k && (st = check_tensor("k_out", k_out, s + 9, ok, 3, d, dtype, true)) != STREAMKL_OK) return st;
  a.side[0].y_out = q_out;
  a.side[1].y_out = k_out;
  a.side[0].ys = row_strides(s + 6);
  a.side[1].ys = row_strides(s + 9);
  cudaError_t e = skl::launch_rope_fwd(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? STREAMKL_OK : cuda_fail(e, "norm + rotation launch");
}

size_t streamkl_qk_norm_rope_bwd_workspace_size(int B, int NQ, int NK, int HQ, int HK, int d) {
  if (B < 1 || NQ < 0 || NK < 0 || HQ < 0 || HK < 0 || (d != 64 && d != 128)) return 0;
  return static_cast<size_t>(2) * skl::rope_bwd_blocks(B, NQ, HQ, NK, HK, d, num_sms()) * d * sizeof(float);
}

streamkl_status streamkl_qk_norm_rope_bwd(const void* q, const void* k, const void* dq_out, const void* dk_out,
                                          int dtype, int B, int NQ, int NK, int HQ, int HK, int d, int rot,
                                          const long long* strides, const float* cos, const float* sin,
                                          int table_len, const int* q_positions, long long q_pos_stride,
                                          const int* k_positions, long long k_pos_stride, const float* q_weight,
                                          const float* k_weight, float eps, int interleaved, int k_repeat, void* dq,
                                          void* dk, float* dq_weight, float* dk_weight, void* workspace,
                                          size_t ws_bytes, int* dev_status, void* stream) {
  clear_error();
  if (!strides) return fail(STREAMKL_ERR_INVALID_ARG, "strides is NULL");
  long long s[18];
  std::copy(strides, strides + 18, s);
  skl::RopeArgs a;
  streamkl_status st = rope_common(&a, q, k, dtype, B, NQ, NK, HQ, HK, d, rot, s, cos, sin, table_len,
                                   q_positions, q_pos_stride, k_positions, k_pos_stride, q_weight, k_weight, eps,
                                   interleaved, k_repeat, dev_status);
  if (st != STREAMKL_OK) return st;
  const int sq[3] = {B, NQ, HQ}, sk[3] = {B, NK, HK}, ok[3] = {B, NK, HK * k_repeat};
  if (q && (st = check_tensor("dq_out", dq_out, s + 6, sq, 3, d, dtype, false)) != STREAMKL_OK) return st;
  if (k && (st = check_tensor("dk_out", dk_out, s + 9, ok, 3, d, dtype, false)) != STREAMKL_OK) return st;
  if (q && (st = check_tensor("dq", dq, s + 12, sq, 3, d, dtype, true)) != STREAMKL_OK) return st;
  if (k && (st = check_tensor("dk", dk, s + 15, sk, 3, d, dtype, true)) != STREAMKL_OK) return st;
  const bool nq = q && q_weight, nk = k && k_weight;
  if ((nq && !dq_weight) || (nk && !dk_weight))
    return fail(STREAMKL_ERR_INVALID_ARG, "a norm weight needs its gradient's buffer");
  const int blocks = skl::rope_bwd_blocks(B, q ? NQ : 0, q ? HQ : 0, k ? NK : 0, k ? HK : 0, d, num_sms());
  const size_t need = nq || nk ? static_cast<size_t>(2) * blocks * d * sizeof(float) : 0;
  if (need && (!workspace || ws_bytes < need))
    return fail(STREAMKL_ERR_INVALID_ARG, "workspace of %zu bytes, need %zu", workspace ? ws_bytes : 0, need);
  if (need && !aligned16(workspace)) return fail(STREAMKL_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
  a.side[0].y_in = dq_out;
  a.side[0].dx = dq;
  a.side[0].ys = row_strides(s + 6);
  a.side[0].dxs = row_strides(s + 12);
  a.side[1].y_in = dk_out;
  a.side[1].dx = dk;
  a.side[1].ys = row_strides(s + 9);
  a.side[1].dxs = row_strides(s + 15);
  a.part = static_cast<float*>(workspace);
  cudaError_t e = skl::launch_rope_bwd(a, blocks, nq ? dq_weight : nullptr, nk ? dk_weight : nullptr,
                                       static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? STREAMKL_OK : cuda_fail(e, "norm + rotation backward launch");
}

streamkl_status streamkl_paged_append(const void* k, const void* v, void* k_cache, void* v_cache,
                                      const int* block_table, long long table_stride, const int* kv_lens,
                                      const int* cu_seqlens, int dtype, int B, int T, int HK, int d, int page_size,
                                      int num_pages, int max_pages, const long long* strides, int rot,
                                      const float* cos, const float* sin, int table_len, const float* k_weight,
                                      float eps, int interleaved, int* dev_status, void* stream) {
  clear_error();
  if (!strides) return fail(STREAMKL_ERR_INVALID_ARG, "strides is NULL");
  long long s[10];
  std::copy(strides, strides + 10, s);
  streamkl_status st = check_cache(k_cache, v_cache, block_table, table_stride, kv_lens, dtype, B, T, HK, d,
                                   page_size, num_pages, max_pages, s);
  if (st != STREAMKL_OK) return st;
  if (!cu_seqlens && T != B)
    return fail(STREAMKL_ERR_INVALID_ARG, "without cu_seqlens each sequence has one token (T=%d B=%d)", T, B);
  if (static_cast<long long>(T) * HK > kMaxRows) return fail(STREAMKL_ERR_UNSUPPORTED, "rows x heads above 2^31");
  const int sizes[2] = {T, HK};
  if ((st = check_tensor("k", k, s + 6, sizes, 2, d, dtype, false)) != STREAMKL_OK) return st;
  if ((st = check_tensor("v", v, s + 8, sizes, 2, d, dtype, false)) != STREAMKL_OK) return st;
  if ((cos == nullptr) != (sin == nullptr))
    return fail(STREAMKL_ERR_INVALID_ARG, "cos and sin must be both NULL or both non-NULL");
  if (cos && (st = check_rope(d, rot, cos, sin, table_len, eps, interleaved)) != STREAMKL_OK) return st;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(STREAMKL_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (!dev_status) return fail(STREAMKL_ERR_INVALID_ARG, "dev_status must be non-NULL");
  skl::AppendArgs a{};
  a.k = k;
  a.v = v;
  a.ks = skl::RowStrides{0, s[6], s[7]};
  a.vs = skl::RowStrides{0, s[8], s[9]};
  a.kc = k_cache;
  a.vc = v_cache;
  a.kc_sp = s[0], a.kc_sh = s[1], a.kc_ss = s[2];
  a.vc_sp = s[3], a.vc_sh = s[4], a.vc_ss = s[5];
  a.table = block_table;
  a.table_sb = table_stride;
  a.kv_lens = kv_lens;
  a.cu = cu_seqlens;
  a.B = B;
  a.T = T;
  a.H = HK;
  a.d = d;
  a.rot = cos ? rot : d;
  a.type = dtype;
  a.interleaved = cos ? interleaved : 0;
  a.page_shift = __builtin_ctz(static_cast<unsigned>(page_size));
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.table_len = table_len;
  a.cos = cos;
  a.sin = sin;
  a.w = k_weight;
  a.eps = eps;
  a.dev_status = dev_status;
  cudaError_t e = skl::launch_append(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? STREAMKL_OK : cuda_fail(e, "append launch");
}

int streamkl_paged_attn_splits(int B, int T, int HQ, int HK, int d, int max_seqlen_q, int max_kv_len) {
  if (check_attn_sizes(B, T, HQ, HK, d, max_seqlen_q, max_kv_len) != STREAMKL_OK) return 0;
  return attn_plan(B, T, HQ, HK, d, max_seqlen_q, max_kv_len, 0).splits;
}

size_t streamkl_paged_attn_workspace_size(int B, int T, int HQ, int HK, int d, int max_seqlen_q, int max_kv_len,
                                          int num_splits) {
  if (check_attn_sizes(B, T, HQ, HK, d, max_seqlen_q, max_kv_len) != STREAMKL_OK || num_splits < 0) return 0;
  return attn_part_bytes(attn_plan(B, T, HQ, HK, d, max_seqlen_q, max_kv_len, num_splits).splits, T, HQ, d);
}

streamkl_status streamkl_paged_attn(const void* q, const void* k_cache, const void* v_cache, const int* block_table,
                                    long long table_stride, const int* kv_lens, const int* cu_seqlens, int dtype,
                                    int B, int T, int HQ, int HK, int d, int page_size, int num_pages, int max_pages,
                                    const long long* strides, int max_seqlen_q, int max_kv_len, float scale,
                                    int causal, int num_splits, void* out, float* lse, void* workspace,
                                    size_t ws_bytes, int* dev_status, void* stream) {
  clear_error();
  if (!strides) return fail(STREAMKL_ERR_INVALID_ARG, "strides is NULL");
  long long s[10];
  std::copy(strides, strides + 10, s);
  streamkl_status st = check_cache(k_cache, v_cache, block_table, table_stride, kv_lens, dtype, B, T, HK, d,
                                   page_size, num_pages, max_pages, s);
  if (st != STREAMKL_OK) return st;
  if ((st = check_attn_sizes(B, T, HQ, HK, d, max_seqlen_q, max_kv_len)) != STREAMKL_OK) return st;
  if (!cu_seqlens && T != B)
    return fail(STREAMKL_ERR_INVALID_ARG, "without cu_seqlens each sequence has one token (T=%d B=%d)", T, B);
  if (max_kv_len > static_cast<long long>(max_pages) * page_size)
    return fail(STREAMKL_ERR_INVALID_ARG, "max_kv_len %d above %d pages of %d", max_kv_len, max_pages, page_size);
  const int sizes[2] = {T, HQ};
  if ((st = check_tensor("q", q, s + 6, sizes, 2, d, dtype, false)) != STREAMKL_OK) return st;
  if ((st = check_tensor("out", out, s + 8, sizes, 2, d, dtype, true)) != STREAMKL_OK) return st;
  if (!lse) return fail(STREAMKL_ERR_INVALID_ARG, "lse must be non-NULL");
  if (causal != 0 && causal != 1) return fail(STREAMKL_ERR_INVALID_ARG, "causal must be 0 or 1");
  if (num_splits < 0) return fail(STREAMKL_ERR_INVALID_ARG, "num_splits must be >= 0");
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(STREAMKL_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (!dev_status) return fail(STREAMKL_ERR_INVALID_ARG, "dev_status must be non-NULL");
  const AttnPlan p = attn_plan(B, T, HQ, HK, d, max_seqlen_q, max_kv_len, num_splits);
  if (p.splits > 65535) return fail(STREAMKL_ERR_UNSUPPORTED, "%d key splits (at most 65535)", p.splits);
  const size_t need = attn_part_bytes(p.splits, T, HQ, d);
  if (need && (!workspace || ws_bytes < need))
    return fail(STREAMKL_ERR_INVALID_ARG, "workspace of %zu bytes, need %zu", workspace ? ws_bytes : 0, need);
  if (need && !aligned16(workspace)) return fail(STREAMKL_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
  CUtensorMap mk, mv;
  if ((st = make_map_cache(&mk, k_cache, dtype, d, page_size, HK, num_pages, s, "k_cache")) != STREAMKL_OK)
    return st;
  if ((st = make_map_cache(&mv, v_cache, dtype, d, page_size, HK, num_pages, s + 3, "v_cache")) != STREAMKL_OK)
    return st;
  skl::PagedAttnArgs a{};
  a.tm_k = &mk;
  a.tm_v = &mv;
  a.q = q;
  a.q_sn = s[6], a.q_sh = s[7];
  a.o = out;
  a.o_sn = s[8], a.o_sh = s[9];
  a.lse = lse;
  a.table = block_table;
  a.table_sb = table_stride;
  a.kv_lens = kv_lens;
  a.cu = cu_seqlens;
  a.B = B;
  a.T = T;
  a.HQ = HQ;
  a.HK = HK;
  a.d = d;
  a.type = dtype;
  a.causal = causal;
  a.page_shift = __builtin_ctz(static_cast<unsigned>(page_size));
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.max_q = max_seqlen_q;
  a.max_kv = max_kv_len;
  a.scale = scale;
  a.q_tiles = p.q_tiles;
  a.row_tiles = p.row_tiles;
  a.splits = p.splits;
  a.split_tiles = p.split_tiles;
  a.part_o = static_cast<float*>(workspace);
  a.part_lse = a.part_o ? a.part_o + static_cast<size_t>(p.splits) * T * HQ * d : nullptr;
  a.dev_status = dev_status;
  a.timeout_ns = wait_timeout_ns();
  cudaError_t e = skl::launch_paged_attn(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? STREAMKL_OK : cuda_fail(e, "paged attention launch");
}

}  // extern "C"
