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

streamkl_status check_tensor(const char* name, const void* p, const long long* strides, int n, int dtype) {
  if (!p) return fail(STREAMKL_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned16(p)) return fail(STREAMKL_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  for (int i = 0; i < n; ++i)
    if (strides[i] < 0 || strides[i] * static_cast<long long>(elem_size(dtype)) % 16)
      return fail(STREAMKL_ERR_INVALID_ARG, "%s: stride %lld is not a multiple of 16 bytes", name, strides[i]);
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
                            int HQ, int HK, int d, int rot, const long long* strides, const float* cos,
                            const float* sin, int table_len, const int* q_pos, long long q_pos_stride,
                            const int* k_pos, long long k_pos_stride, const float* q_weight,
                            const float* k_weight, float eps, int interleaved, int k_repeat, int* dev_status) {
  clear_error();
  if (!q && !k) return fail(STREAMKL_ERR_INVALID_ARG, "q and k are both NULL");
  if (!strides) return fail(STREAMKL_ERR_INVALID_ARG, "strides is NULL");
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
  if (q && (st = check_tensor("q", q, strides, 3, dtype)) != STREAMKL_OK) return st;
  if (k && (st = check_tensor("k", k, strides + 3, 3, dtype)) != STREAMKL_OK) return st;
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
    a->side[i].ys = row_strides(strides + 6 + 3 * i);
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
                            int num_pages, int max_pages, const long long* strides) {
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
  streamkl_status st = check_tensor("k_cache", kc, strides, 3, dtype);
  if (st != STREAMKL_OK) return st;
  if ((st = check_tensor("v_cache", vc, strides + 3, 3, dtype)) != STREAMKL_OK) return st;
  for (int i = 0; i < 6; ++i)
    if (strides[i] < d)
      return fail(STREAMKL_ERR_INVALID_ARG, "cache stride %lld below one row of %d", strides[i], d);
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
  skl::RopeArgs a;
  streamkl_status st = rope_common(&a, q, k, dtype, B, NQ, NK, HQ, HK, d, rot, strides, cos, sin, table_len,
                                   q_positions, q_pos_stride, k_positions, k_pos_stride, q_weight, k_weight, eps,
                                   interleaved, k_repeat, dev_status);
  if (st != STREAMKL_OK) return st;
  if (q && (st = check_tensor("q_out", q_out, strides + 6, 3, dtype)) != STREAMKL_OK) return st;
  if (k && (st = check_tensor("k_out", k_out, strides + 9, 3, dtype)) != STREAMKL_OK) return st;
  a.side[0].y_out = q_out;
  a.side[1].y_out = k_out;
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
  skl::RopeArgs a;
  streamkl_status st = rope_common(&a, q, k, dtype, B, NQ, NK, HQ, HK, d, rot, strides, cos, sin, table_len,
                                   q_positions, q_pos_stride, k_positions, k_pos_stride, q_weight, k_weight, eps,
                                   interleaved, k_repeat, dev_status);
  if (st != STREAMKL_OK) return st;
  if (q && (st = check_tensor("dq_out", dq_out, strides + 6, 3, dtype)) != STREAMKL_OK) return st;
  if (k && (st = check_tensor("dk_out", dk_out, strides + 9, 3, dtype)) != STREAMKL_OK) return st;
  if (q && (st = check_tensor("dq", dq, strides + 12, 3, dtype)) != STREAMKL_OK) return st;
  if (k && (st = check_tensor("dk", dk, strides + 15, 3, dtype)) != STREAMKL_OK) return st;
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
  a.side[0].dxs = row_strides(strides + 12);
  a.side[1].y_in = dk_out;
  a.side[1].dx = dk;
  a.side[1].dxs = row_strides(strides + 15);
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
  streamkl_status st = check_cache(k_cache, v_cache, block_table, table_stride, kv_lens, dtype, B, T, HK, d,
                                   page_size, num_pages, max_pages, strides);
  if (st != STREAMKL_OK) return st;
  if (!cu_seqlens && T != B)
    return fail(STREAMKL_ERR_INVALID_ARG, "without cu_seqlens each sequence has one token (T=%d B=%d)", T, B);
  if (static_cast<long long>(T) * HK > kMaxRows) return fail(STREAMKL_ERR_UNSUPPORTED, "rows x heads above 2^31");
  if ((st = check_tensor("k", k, strides + 6, 2, dtype)) != STREAMKL_OK) return st;
  if ((st = check_tensor("v", v, strides + 8, 2, dtype)) != STREAMKL_OK) return st;
  if ((cos == nullptr) != (sin == nullptr))
    return fail(STREAMKL_ERR_INVALID_ARG, "cos and sin must be both NULL or both non-NULL");
  if (cos && (st = check_rope(d, rot, cos, sin, table_len, eps, interleaved)) != STREAMKL_OK) return st;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(STREAMKL_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (!dev_status) return fail(STREAMKL_ERR_INVALID_ARG, "dev_status must be non-NULL");
  skl::AppendArgs a{};
  a.k = k;
  a.v = v;
  a.ks = skl::RowStrides{0, strides[6], strides[7]};
  a.vs = skl::RowStrides{0, strides[8], strides[9]};
  a.kc = k_cache;
  a.vc = v_cache;
  a.kc_sp = strides[0], a.kc_sh = strides[1], a.kc_ss = strides[2];
  a.vc_sp = strides[3], a.vc_sh = strides[4], a.vc_ss = strides[5];
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

}  // extern "C"
