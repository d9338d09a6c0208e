/*
 * streamkl.h -- C ABI of the GB300 (sm_103a) attention-KL primitive.
 *
 * The operation ("StreamKL: Fast and Memory-Efficient KL Divergence for
 * Boosting Attention Distillation", abstract and gist.science technical
 * summary): for every batch b, head h and query row i,
 *
 *     S_t = scale * Q_t K_t^T (+ causal mask),  P_t = softmax(S_t),  t = 1, 2
 *     KL[b,h,i] = sum_j P1[i,j] * log(P1[i,j] / P2[i,j])
 *
 * with P1 the teacher and P2 the student, computed without ever writing the
 * N_Q x N_K matrices S1, S2, P1, P2 to device memory.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Q1, Q2 are [B, H, N_Q, d] and K1, K2 are [B, H, N_K, d], bf16, dense,
 *   row-major (d contiguous), 16-byte aligned device pointers. d is 64 or 128.
 * - Per-row vectors (kl, lse1, lse2, dkl) are [B, H, N_Q] fp32, dense.
 * - Causal masking is bottom-right aligned: key j is visible to query i iff
 *   j <= i + (N_K - N_Q) (j <= i when N_Q == N_K); it needs N_Q <= N_K.
 * - All pointers are device pointers owned by the caller. The library
 *   allocates no memory, never synchronises, and enqueues all work on
 *   `stream` (a cudaStream_t; NULL means the legacy default stream), so the
 *   calls can be captured into a CUDA graph once their kernels have run
 *   eagerly (the first call sets their shared-memory attributes).
 * - Synchronous argument errors return STREAMKL_ERR_INVALID_ARG or
 *   STREAMKL_ERR_UNSUPPORTED before anything is enqueued; a failed launch
 *   returns STREAMKL_ERR_CUDA. streamkl_last_error() gives the detail.
 * - dev_status is a caller-owned device int the kernels write when a bounded
 *   wait inside them gives up (STREAMKL_ERR_TIMEOUT), when packed sequence
 *   offsets are malformed (STREAMKL_ERR_INVALID_ARG) or, in the debug build,
 *   when a range check fails (STREAMKL_ERR_DEVICE_CHECK); they never clear it.
 *   Clear it before use and read it after synchronising the stream. Results
 *   of a call that set it are undefined.
 */
#ifndef STREAMKL_H_
#define STREAMKL_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  STREAMKL_OK = 0,
  STREAMKL_ERR_INVALID_ARG = 1,
  STREAMKL_ERR_UNSUPPORTED = 2,
  STREAMKL_ERR_CUDA = 3,
  STREAMKL_ERR_TIMEOUT = 4,
  /* Written to dev_status only by the debug build (libstreamkl_debug.so,
   * compiled with STREAMKL_DEVICE_CHECKS): a kernel found an operand of a
   * TMA copy, TMEM access or mbarrier outside its layout, skipped that access
   * and stopped (the first failing source line is printed from the device).
   * The release build never writes it. */
  STREAMKL_ERR_DEVICE_CHECK = 5,
  /* Written to dev_status by streamkl_paged_resize: free pages did not suffice
   * for every sequence (those that got none keep their lengths). */
  STREAMKL_ERR_NO_PAGES = 6
} streamkl_status;

/* Human-readable name of a status code (static string). */
const char* streamkl_status_string(streamkl_status s);

/* Detail message of the last failing call on this host thread ("" if none). */
const char* streamkl_last_error(void);

/*
 * Split count the forward pass uses when num_splits == 0 (split-K over the
 * key dimension; gist.science technical summary, section 3 "Variante
 * Split-K": keys are partitioned across thread blocks so that few query rows
 * still fill the GPU). Returns >= 1; 0 on invalid sizes.
 */
int streamkl_choose_splits(int B, int H, int NQ, int NK, int d, int causal);

/*
 * Workspace bytes the forward pass needs with `num_splits` splits (0 = the
 * automatic choice). The split partial states are five fp32 per (split, b, h,
 * row): running maxima, exponential sums and the weighted-logit-difference
 * accumulator. 0 when no split is used.
 */
size_t streamkl_fwd_workspace_size(int B, int H, int NQ, int NK, int d, int causal,
                                   int num_splits);

/*
 * Whether the forward runs as CTA pairs for these sizes: 1 = two CTAs of a
 * thread-block cluster take two query blocks of one (batch, head) slice and
 * compute their score tiles as one tcgen05 MMA with M = 256 (cta_group::2),
 * each CTA loading its own query tile and half of every key tile; 0 = one
 * CTA per query block. Pairs need dense batches without a key split
 * (num_splits as for streamkl_fwd; 0 = automatic) and an even number of
 * 128-row query blocks, and are off unless streamkl_set_fwd_pairs(1) was
 * called (on GB300 they match the one-CTA forward at the 64K causal
 * workload and are slower on smaller ones). Same results either way up to
 * fp32 rounding. Returns -1 on invalid sizes. The paper has no counterpart
 * (it is a scheduling choice of this implementation).
 */
int streamkl_fwd_pairs(int B, int H, int NQ, int NK, int d, int causal, int num_splits);

/*
 * CTA pairs in the forward for the process: 0 = never (default), 1 = when
 * the sizes allow. Returns 0, or -1 for another value.
 */
int streamkl_set_fwd_pairs(int mode);

/*
 * Backward algorithm used for these sizes (gist.science technical summary,
 * section 2, kernel fusion paragraph: a fused kernel with atomic dQ updates,
 * or separate kernels when the atomics contend too much):
 *   0 = separate dK and dQ kernels: each keeps its accumulators on chip for
 *       its whole sweep; no atomics; a workspace only for the dQ kernel's
 *       key split (below);
 *   1 = fused: every (query, key) pair visited once, dK on chip, dQ summed
 *       into an fp32 workspace, then converted to bf16. At most 64 query
 *       rows at d = 128: a persistent kernel over (batch-head, key tile)
 *       items keeping dQ on chip per batch-head; otherwise one CTA per key
 *       tile adding each query block's dQ with TMA bulk reductions (128-row
 *       blocks at d = 64, 64-row steps at d = 128).
 * The automatic choice (from the fused-vs-separate sweep on GB300) is 1 for
 * at most 64 query rows at d = 128; with one gradient set (want_grad1 = 0)
 * for at least 512 query rows at d = 64, and at d = 128 for at least 512
 * query rows without the mask or 1,024 with causal = 1; 0 otherwise.
 * Configuration 2 alone runs 0 except at most 64 query rows at d = 128.
 * Returns -1 on invalid sizes.
 */
int streamkl_bwd_algorithm(int B, int H, int NQ, int NK, int d, int causal, int want_grad1);

/*
 * Process-wide override of that choice: -1 = automatic, 0 = separate,
 * 1 = fused. Its initial value comes from the environment variable
 * STREAMKL_BWD_ALGO=separate|fused (automatic when unset). The workspace
 * size queries follow it; change it only while no other host thread is
 * between a size query and the matching streamkl_bwd call. Returns 0, or -1
 * for an invalid value.
 */
int streamkl_set_bwd_algorithm(int algo);

/*
 * Key split of the separate algorithm's dQ kernel. With few query blocks
 * against many keys (B H ceil(N_Q/128) below 8 per SM) the dQ kernel's
 * key range is cut into splits of 64-key steps, like the forward's split-K
 * (gist.science technical summary, section 3 "Variante Split-K": keys
 * partitioned across thread blocks); each split writes an fp32 partial dQ
 * into the workspace and a
 * combine kernel sums them into the bf16 output. Dense batches only (varlen
 * batches never split).
 *   streamkl_bwd_dq_splits: the split count streamkl_bwd will use for these
 *        sizes (want_grad1 != 0: both gradient sets); -1 on invalid sizes.
 *   streamkl_set_bwd_dq_splits: process-wide override, 0 = automatic, n >= 1
 *        forces n splits (clamped to the number of 64-key steps); same
 *        threading caveat as streamkl_set_bwd_algorithm. Returns 0, or -1
 *        for a negative value.
 */
int streamkl_bwd_dq_splits(int B, int H, int NQ, int NK, int d, int causal, int want_grad1);
int streamkl_set_bwd_dq_splits(int splits);

/*
 * Persistent dK kernel of the separate algorithm for short query sweeps
 * (N_Q <= 384, dense batches, more (key block, batch-head) items than SMs):
 * one CTA per SM takes the items in turn, heavy key blocks first, and loads
 * the next item's key block while the current one finishes, instead of one
 * CTA per key block paying its start and end each time. No counterpart in
 * the paper; same results.
 *   streamkl_bwd_dk_persist: the number of persistent CTAs streamkl_bwd will
 *        launch for these sizes (0: one CTA per key block); -1 on invalid sizes.
 *   streamkl_set_bwd_dk_persist: process-wide override, 0 = automatic,
 *        -1 = never, n >= 1 = always, with n CTAs; same threading caveat as
 *        streamkl_set_bwd_algorithm. Returns 0, or -1 below -1.
 */
int streamkl_bwd_dk_persist(int B, int H, int NQ, int NK, int d, int causal);
int streamkl_set_bwd_dk_persist(int ctas);

/*
 * Workspace bytes the backward pass needs, for one gradient set or, with
 * want_grad1 != 0, both (an upper bound for configuration 2 alone): for the
 * separate-kernel algorithm the fp32 partials of the dQ kernel's key split
 * (0 without a split); for the fused one, one fp32 [B, H, N_Q, d] dQ
 * accumulator per requested gradient set (with want_grad1 = 0 also enough
 * for configuration 2 alone where that runs the separate kernels).
 */
size_t streamkl_bwd_workspace_size(int B, int H, int NQ, int NK, int d, int causal,
                                   int want_grad1);

/* max(forward with automatic splits, backward): one buffer serves both. */
size_t streamkl_workspace_size(int B, int H, int NQ, int NK, int d, int causal,
                               int want_grad1);

/*
 * Forward pass (gist.science technical summary, "Metodologia" section 1:
 * online formulation; section 2 "Estado Guardado": only KL and the two
 * log-sum-exps are saved).
 *   in : q1, k1, q2, k2 (bf16, layout above); scale > 0; causal 0/1;
 *        num_splits: 0 = automatic, >= 1 forces that many key splits
 *        (clamped to the number of key tiles).
 *   out: kl[b,h,i] = KL(P1 || P2) of row i (nats), lse1/lse2[b,h,i] =
 *        log sum_j exp(S_t[i,j]) over the visible keys (fp32).
 *   workspace: device buffer of ws_bytes >= streamkl_fwd_workspace_size(...)
 *        (may be NULL when that is 0); contents need no initialisation.
 */
streamkl_status streamkl_fwd(const void* q1, const void* k1, const void* q2, const void* k2,
                             int B, int H, int NQ, int NK, int d, float scale, int causal,
                             int num_splits, float* kl, float* lse1, float* lse2,
                             void* workspace, size_t ws_bytes, int* dev_status, void* stream);

/*
 * Forward pass that allocates nothing and takes no workspace. The paper has
 * no counterpart; this entry point exists for callers that only hold the
 * input and output buffers handed to them and cannot obtain device memory of
 * their own: a plug-in operator inside another runtime that offers no
 * workspace, or code whose device memory is owned by a host framework's pool,
 * where a cudaMalloc would fail, fragment that pool or stall the device.
 *
 * Same arguments, results and errors as streamkl_fwd, minus the workspace.
 * The split partial states go to a scratch array built into the library:
 * 16 MiB (16777216 bytes) of device memory that every GPU which loads the
 * library keeps until the process exits. A call whose split plan needs more
 * than that (5 floats per split, batch, head and query row, rounded up to 256
 * bytes; see streamkl_fwd_workspace_size) returns STREAMKL_ERR_INVALID_ARG
 * with the sizes in streamkl_last_error(); pass fewer splits or use
 * streamkl_fwd. Calls without splits do not touch the scratch.
 *
 * The first call that uses the scratch on a device looks up its device
 * address (with that device current) and caches it together with the current
 * driver context; make that first call before any stream capture. A call
 * made in another context than the cached one (after cudaDeviceReset, which
 * drops the library's module and the array with it, or with a non-primary
 * context current) looks the address up again, so the first such call should
 * also come before any capture. All calls on a device share the one array and
 * each leaves its partial states in it; nothing there needs clearing because
 * every call writes all the states it reads, but calls whose kernels may
 * overlap on the GPU (different streams, other host threads) race on it and
 * must be ordered by the caller.
 */
streamkl_status streamkl_fwd_noalloc(const void* q1, const void* k1, const void* q2,
                                     const void* k2, int B, int H, int NQ, int NK, int d,
                                     float scale, int causal, int num_splits, float* kl,
                                     float* lse1, float* lse2, int* dev_status, void* stream);

/*
 * Backward pass of L = sum_{b,h,i} dkl[b,h,i] * KL[b,h,i] (gist.science
 * technical summary, section 2: probabilities regenerated tile by tile as
 * P_t = exp(S_t - LSE_t); "Configuracion 1": P1 fixed, gradients to Q2, K2;
 * "Configuracion 2": P2 fixed, gradients to Q1, K1; section 3 "Estabilidad
 * Numerica": log(P1/P2) from logits and saved LSEs).
 *   in : q1, k1, q2, k2, sizes, scale, causal exactly as given to streamkl_fwd;
 *        kl, lse1, lse2 as produced by streamkl_fwd; dkl = upstream gradient
 *        per row (fp32 [B, H, N_Q]).
 *   out: dq2 [B,H,N_Q,d], dk2 [B,H,N_K,d] (bf16) for configuration 1;
 *        dq1, dk1 likewise for configuration 2. Either pair may be NULL to
 *        skip that configuration (both of a pair NULL or neither; at least one
 *        pair is required). Configuration 2 alone runs the separate dK/dQ
 *        kernels, or the fused algorithm's short-sweep kernel where that is
 *        the algorithm chosen (at most 64 query rows at d = 128).
 *   workspace: ws_bytes >= streamkl_bwd_workspace_size(..., want_grad1) (may be
 *        NULL when that is 0); the call clears the part it uses (stream-ordered).
 */
streamkl_status streamkl_bwd(const void* q1, const void* k1, const void* q2, const void* k2,
                             int B, int H, int NQ, int NK, int d, float scale, int causal,
                             const float* kl, const float* lse1, const float* lse2,
                             const float* dkl, void* dq2, void* dk2, void* dq1, void* dk1,
                             void* workspace, size_t ws_bytes, int* dev_status, void* stream);

/*
 * Reverse direction, KL(P2 || P1) per row. The pages define the
 * teacher-first direction KL(P1 || P2) only (gist.science technical summary,
 * "Declaracion del Problema"); the reverse one is the same computation with
 * the two distributions exchanged, so these two calls run the kernels above
 * with the argument slots swapped and add nothing else.
 *   streamkl_fwd_reverse: arguments as for streamkl_fwd; out: kl[b,h,i] =
 *        KL(P2 || P1) of row i, lse1 / lse2 the log-partition of S1 / S2
 *        exactly as from streamkl_fwd.
 *   streamkl_bwd_reverse: gradients of L = sum dkl * KL(P2 || P1), with kl,
 *        lse1, lse2 from streamkl_fwd_reverse. dq2, dk2 get the student's
 *        gradients (P1 fixed), dq1, dk1 the teacher's (P2 fixed); either pair
 *        may be NULL to skip it (at least one pair). ws_bytes >=
 *        streamkl_bwd_workspace_size(..., want_grad1 = both pairs requested).
 * Errors as for streamkl_fwd / streamkl_bwd; a message about a tensor names
 * it by its slot in the exchanged call (q1 for the q2 given here, and so on).
 */
streamkl_status streamkl_fwd_reverse(const void* q1, const void* k1, const void* q2,
                                     const void* k2, int B, int H, int NQ, int NK, int d,
                                     float scale, int causal, int num_splits, float* kl,
                                     float* lse1, float* lse2, void* workspace, size_t ws_bytes,
                                     int* dev_status, void* stream);
streamkl_status streamkl_bwd_reverse(const void* q1, const void* k1, const void* q2,
                                     const void* k2, int B, int H, int NQ, int NK, int d,
                                     float scale, int causal, const float* kl, const float* lse1,
                                     const float* lse2, const float* dkl, void* dq2, void* dk2,
                                     void* dq1, void* dk1, void* workspace, size_t ws_bytes,
                                     int* dev_status, void* stream);

/*
 * Variable-length batches (packed, token-major). The same forward as
 * streamkl_fwd for B independent sequences of different lengths, each with
 * H heads (gist.science technical summary, section 1: the streaming pass is
 * per (batch, head) row and never needs the other sequences' keys).
 *   in : q1, q2 bf16 [total_q, H, d]; k1, k2 bf16 [total_k, H, d] (16-byte
 *        aligned, d contiguous, heads next, then tokens); cu_seqlens_q,
 *        cu_seqlens_k: DEVICE int32 arrays of B+1 offsets, 0 = cu[0] <= cu[1]
 *        <= ... <= cu[B] = total: sequence b owns query rows cu_seqlens_q[b]
 *        .. cu_seqlens_q[b+1] and key rows cu_seqlens_k[b] .. cu_seqlens_k[b+1];
 *        max_seqlen_q / max_seqlen_k: upper bounds on the per-sequence lengths
 *        (they size the grid); causal: per sequence, bottom-right aligned.
 *   out: kl, lse1, lse2 fp32 [total_q, H].
 * No split-K and no workspace. Host-side errors as for streamkl_fwd; the
 * offsets live on the device, so the kernels check them and write
 * STREAMKL_ERR_INVALID_ARG into *dev_status for offsets outside [0, total],
 * a length above its max_seqlen, a sequence with query rows but no key (a
 * softmax over no key is undefined), or a causal sequence with more query
 * rows than keys (its rows of that sequence are then left unwritten). A
 * sequence without query rows contributes nothing.
 */
streamkl_status streamkl_fwd_varlen(const void* q1, const void* k1, const void* q2, const void* k2,
                                    const int* cu_seqlens_q, const int* cu_seqlens_k, int B, int H,
                                    int total_q, int total_k, int max_seqlen_q, int max_seqlen_k,
                                    int d, float scale, int causal, float* kl, float* lse1,
                                    float* lse2, int* dev_status, void* stream);

/*
 * Backward of L = sum dkl * KL for a packed variable-length batch: inputs
 * and sequence offsets as for streamkl_fwd_varlen; kl, lse1, lse2, dkl fp32
 * [total_q, H]; gradients bf16 [total_q, H, d] (dq2, dq1) and [total_k, H, d]
 * (dk2, dk1), either pair NULL to skip that configuration (at least one
 * pair). Always the separate dK/dQ kernels; no workspace. Errors as for
 * streamkl_bwd and streamkl_fwd_varlen. The dK rows of a sequence without
 * query rows are zero (no query sees those keys).
 */
streamkl_status streamkl_bwd_varlen(const void* q1, const void* k1, const void* q2, const void* k2,
                                    const int* cu_seqlens_q, const int* cu_seqlens_k, int B, int H,
                                    int total_q, int total_k, int max_seqlen_q, int max_seqlen_k,
                                    int d, float scale, int causal, const float* kl,
                                    const float* lse1, const float* lse2, const float* dkl,
                                    void* dq2, void* dk2, void* dq1, void* dk1, int* dev_status,
                                    void* stream);

/*
 * ---------------------------------------------------------------------------
 * Operators around the KL: what a model computes before the call (norm and
 * rotation of its queries and keys, with the way back for the gradients) and
 * what a trained student is run with (a paged key/value cache, its append and
 * the attention of new tokens over it). The paper has no counterpart. The
 * conventions above hold, with these additions:
 * - Arguments come in one struct that lives on the host for the length of the
 *   call; struct_size is its sizeof (a call with another size is refused).
 * - dtype is the element type of q, k, v, caches and outputs; sums, norms,
 *   softmax statistics and weights are fp32.
 * - A tensor of rows of d contiguous elements is its address and the element
 *   strides of its other dimensions, address and strides multiples of 16
 *   bytes (the stride of a dimension of one element is ignored).
 * - Outputs must not overlap inputs, nor their own rows each other.
 * - Values that only the device knows (positions, lengths, page numbers) are
 *   checked by the kernels: a bad one sets STREAMKL_ERR_INVALID_ARG in
 *   *dev_status and is never used as an address.
 */
typedef enum { STREAMKL_BF16 = 0, STREAMKL_FP16 = 1, STREAMKL_FP32 = 2 } streamkl_dtype;

typedef struct {
  void* data; /* not written through for an input */
  long long stride[3];
} streamkl_rows;

/*
 * Norm and rotation of queries and keys, one pass over both. Each row x (one
 * token, one head, d elements) becomes R(p) (w * x / sqrt(mean(x^2) + eps)):
 * R(p) turns the pairs of the first `rot` elements by the angles of position
 * p, (a, b) -> (a cos - b sin, b cos + a sin); pairs are (i, i + rot / 2), or
 * (2i, 2i + 1) with interleaved = 1.
 *   q [B, NQ, HQ, d], k [B, NK, HK, d] -> q_out [B, HQ, NQ, d],
 *   k_out [B, HK * k_repeat, NK, d]: head h of k stands k_repeat times, from
 *   h * k_repeat on, so that grouped heads give streamkl_fwd its equal head
 *   counts. Strides of all: batch, token, head. A packed batch [total, H, d]
 *   is B = 1. A row whose position lies outside the tables is reported and
 *   not written. dtype: any; d is 64 or 128.
 * Backward: q_out, k_out are the gradients of the outputs (those of a key
 * head's repeats are summed), dq, dk and dq_weight, dk_weight are written.
 * workspace: ws_bytes >= streamkl_qk_norm_rope_bwd_workspace_size(...) (sizes
 * of an absent side 0; may be NULL without weights); no initialisation; calls
 * that may overlap need one each. The
 * weight gradients are summed in a fixed order: the same in every run. Rows
 * that the forward does not write get no gradient and add none.
 */
typedef struct {
  size_t struct_size;
  streamkl_rows q, k;         /* data NULL skips q or k */
  streamkl_rows q_out, k_out; /* forward: outputs; backward: their gradients */
  streamkl_rows dq, dk;       /* backward only */
  const float *cos, *sin;     /* [table_len, rot / 2] */
  const int* q_positions;     /* device; token (b, n) at [b * q_pos_stride + n] (0: the same for each b);
                                 NULL: query n at position n + max(NK - NQ, 0) (needs NQ <= NK) */
  long long q_pos_stride;
  const int* k_positions;     /* likewise; NULL: key n at position n */
  long long k_pos_stride;
  const float *q_weight, *k_weight; /* [d], 16-byte aligned; NULL: rotation without norm */
  float *dq_weight, *dk_weight;     /* backward: [d], needed where the weight is given */
  void* workspace;                  /* backward */
  size_t ws_bytes;
  int* dev_status;
  int dtype, B, NQ, NK, HQ, HK, d;
  int rot; /* a multiple of 16 up to d */
  int table_len, interleaved, k_repeat;
  float eps;
} streamkl_rope_args;

streamkl_status streamkl_qk_norm_rope_fwd(const streamkl_rope_args* args, void* stream);
size_t streamkl_qk_norm_rope_bwd_workspace_size(int B, int NQ, int NK, int HQ, int HK, int d);
streamkl_status streamkl_qk_norm_rope_bwd(const streamkl_rope_args* args, void* stream);

/*
 * Append new keys and values to a paged cache, the keys normed (k_weight) and
 * rotated (cos, sin) on the way as above; NULL leaves either out.
 *   k, v [T, HK, d]: the new tokens of B sequences packed one after the other;
 *   those from cu_seqlens[B] on (or before cu_seqlens[0]) are padding and ignored. Position p of
 *   sequence b lies in slot p % page_size of page block_table[b][p / page_size]
 *   of k_cache, v_cache [num_pages, HK, page_size, d]. Only the new tokens'
 *   slots are written. Two tokens of one call must not share a slot (one of
 *   them would be left there, no more is said). A token with a bad position
 *   or page is reported and not written. dtype: STREAMKL_BF16 or STREAMKL_FP16.
 */
typedef struct {
  size_t struct_size;
  streamkl_rows k, v;             /* strides: (unused), token, head */
  streamkl_rows k_cache, v_cache; /* strides: page, head, slot */
  const int* block_table;         /* device [B, max_pages], rows table_stride apart */
  long long table_stride;
  const int* kv_lens;             /* device [B]: length of each sequence with its new tokens, which end it */
  const int* cu_seqlens;          /* device [B + 1]: first token of each sequence; NULL: T = B, one token each */
  const float *cos, *sin;
  const float* k_weight;
  int* dev_status;
  int dtype, B, T, HK, d;
  int page_size; /* a power of two from 16 to 1024 */
  int num_pages, max_pages, rot, table_len, interleaved;
  float eps;
} streamkl_append_args;

streamkl_status streamkl_paged_append(const streamkl_append_args* args, void* stream);

/*
 * Attention of new tokens over a paged cache: row i of a sequence's n new
 * tokens gives o = softmax(scale q K^T) V over the keys it sees, all of the
 * sequence, or with causal = 1 those up to its own position (bottom-right
 * aligned as above: key j <= i + length - n).
 *   q [T, HQ, d] packed as k of streamkl_paged_append; caches, block_table,
 *   kv_lens, cu_seqlens as there; query head h reads key head h / (HQ / HK).
 *   out [T, HQ, d] and lse [T, HQ] (fp32, contiguous, the log of the softmax's
 *   sum, as streamkl_fwd's). A row that sees no key (length 0, or causal with
 *   more new tokens than keys) gets zeros and -inf. Rows behind the last
 *   sequence, or in front of the first, are left as they were.
 * workspace: ws_bytes >= streamkl_paged_attn_workspace_size(...) of the same
 * sizes and num_splits (may be NULL when that is 0); contents need no
 * initialisation; calls that may overlap need one each.
 * Slots past a sequence's length and page numbers past its last page are
 * never used, whatever they hold. A value of V that is not finite reaches
 * every row whose key tile it lies in. Offsets or lengths out of range or
 * above their bounds, and bad page numbers, are reported in *dev_status; the
 * rows of such a sequence mean nothing, those of the others are computed.
 * Results are the same in every run for the same sizes. Scores (times log2 e) of
 * fp16 inputs may reach 2^28, of which fp32 keeps steps of 16. B * HK is at most
 * 65535.
 */
typedef struct {
  size_t struct_size;
  streamkl_rows q, out;           /* strides: (unused), token, head */
  streamkl_rows k_cache, v_cache; /* strides: page, head, slot */
  const int* block_table;
  long long table_stride;
  const int *kv_lens, *cu_seqlens;
  float* lse;
  void* workspace;
  size_t ws_bytes;
  int* dev_status;
  int dtype, B, T, HQ, HK, d, page_size, num_pages, max_pages;
  int max_seqlen_q, max_kv_len; /* upper bounds of the sequences' new tokens and lengths (grid, key split) */
  int causal;
  int num_splits; /* 0: automatic; >= 1: that many key splits (clamped to the 128-key tiles) */
  float scale;
} streamkl_paged_attn_args;

/* Key splits that num_splits = 0 takes for these sizes; 0: few rows (at most 32
 * (token, head of a group) rows per sequence and key head), where persistent
 * CTAs share all key tiles evenly instead, or take short sequences whole; -1 on
 * invalid sizes. */
int streamkl_paged_attn_splits(int B, int T, int HQ, int HK, int d, int max_seqlen_q, int max_kv_len);
size_t streamkl_paged_attn_workspace_size(int B, int T, int HQ, int HK, int d, int max_seqlen_q, int max_kv_len,
                                          int num_splits);
streamkl_status streamkl_paged_attn(const streamkl_paged_attn_args* args, void* stream);

/*
 * Attention of drafted tokens: as streamkl_paged_attn, but the n new tokens of a
 * sequence are a tree (or any set) of guesses, and a row sees all keys before
 * them (j < length - n) and those of them whose bit its mask has: bit t % 32 of
 * word t / 32 for the sequence's drafted token t, its own and its ancestors' in a
 * tree. Bits from n on say nothing. A row that sees no key gets zeros and -inf.
 * With fewer keys than drafted tokens the first of these have no key. A hidden token's
 * key may hold anything; a value of V that is not finite reaches every row whose key
 * tile (128 keys from a multiple of 128 on) it lies in, those that it is hidden from
 * too, as 0 x infinity in the product. The keys are cached as they are to be seen,
 * rotated by their depth: streamkl_paged_append rotates by place.
 *   attn: the arguments of streamkl_paged_attn, struct_size and all; causal and
 *   num_splits must be 0. mask: device words [T, mask_words], rows mask_stride words apart, for
 *   the tokens in q's order; max_seqlen_q is at most 32 mask_words.
 *   workspace as there, of streamkl_paged_tree_attn_workspace_size(...) bytes.
 */
typedef struct {
  size_t struct_size;
  streamkl_paged_attn_args attn;
  const int* mask;
  long long mask_stride;
  int mask_words;
} streamkl_paged_tree_attn_args;

size_t streamkl_paged_tree_attn_workspace_size(int B, int T, int HQ, int HK, int d, int max_seqlen_q, int max_kv_len);
streamkl_status streamkl_paged_tree_attn(const streamkl_paged_tree_attn_args* args, void* stream);

/*
 * Keep some of the last tokens of each sequence: of its n = cu_seqlens[b + 1] -
 * cu_seqlens[b] last ones, token kept[b][i] (of 0 .. n - 1) moves to the place of
 * token i, for i < num_kept[b], in both caches and in place. kept[b] rises; places
 * from num_kept[b] on are left as they are. The lengths are not changed, so that a
 * call for each layer can follow (streamkl_paged_resize then gives the rest back).
 * Pages that other sequences hold change for these too, and no two sequences of a
 * call may have last tokens in the same page (streamkl_paged_resize, by which they
 * came, sees to that). A list that does not rise or leaves 0 .. n - 1 and numbers
 * that do not fit are reported, and that sequence is left as it was; a row whose
 * page number is none is reported and not moved. B * HK is at most 2^26.
 */
typedef struct {
  size_t struct_size;
  streamkl_rows k_cache, v_cache; /* strides: page, head, slot */
  const int* block_table;
  long long table_stride;
  const int *kv_lens, *cu_seqlens; /* lengths with these tokens; [B + 1] */
  const int* kept;                 /* device [B, max_kept], rows kept_stride apart */
  long long kept_stride;
  const int* num_kept; /* device [B] */
  int* dev_status;
  int dtype, B, HK, d, page_size, num_pages, max_pages, max_kept;
} streamkl_compact_args;

streamkl_status streamkl_paged_compact(const streamkl_compact_args* args, void* stream);

/*
 * Copy pages of both caches: pairs [n, 2] of (source, destination), device,
 * 8-byte aligned. A pair of negative numbers copies nothing. No page may be the
 * destination of two pairs, or of one and the source of another. Any other pair with
 * a number that is no page is reported and not copied. At most 2^30 pairs and 2^36
 * rows (pairs, heads and slots of a page).
 */
typedef struct {
  size_t struct_size;
  streamkl_rows k_cache, v_cache; /* strides: page, head, slot */
  const int* pairs;
  int* dev_status;
  int dtype, n, HK, d, page_size, num_pages;
} streamkl_page_copy_args;

streamkl_status streamkl_paged_copy(const streamkl_page_copy_args* args, void* stream);

/*
 * Sequences that share pages. page_refs[p] is the number of entries of
 * block_table [B, max_pages] that hold page p (0: free); entries that hold none
 * are -1, and a sequence's pages are its first ceil(length / page_size) entries.
 * The two calls below keep that so; a table is filled by streamkl_paged_resize
 * from lengths of 0, counts of 0 and entries of -1. Both change their arguments
 * in place; a call that sets STREAMKL_ERR_INVALID_ARG has found numbers that do
 * not fit, left those out and done the rest. After STREAMKL_ERR_CUDA part of a
 * call may have run, and the tables mean nothing. B is at most 4096, num_pages 2^23,
 * B * max_pages 2^30.
 *
 * streamkl_paged_fork: every sequence b becomes a copy of what source[b] was, for
 * all b at once (source[b] = b: it stays): entries, length and the pages' counts.
 */
typedef struct {
  size_t struct_size;
  int* page_refs;   /* device [num_pages] */
  int* block_table; /* device [B, max_pages], rows table_stride apart */
  long long table_stride;
  int* kv_lens;      /* device [B] */
  const int* source; /* device [B]; a number that is no sequence is reported, that sequence stays */
  int* dev_status;
  int B, num_pages, max_pages;
} streamkl_fork_args;

streamkl_status streamkl_paged_fork(const streamkl_fork_args* args, void* stream);

/*
 * streamkl_paged_resize: lengths become new_lens. A shorter sequence gives the
 * pages past its new end back. Then, in the order of the sequences, a longer one
 * gets the free pages of the lowest numbers: first, where its last page is partly
 * filled and others hold it too, one in that page's place (the last of those that
 * grow in one call keeps it if no other is left), then those that it lacks.
 *   copies [B, 2]: (old, new) of the page so replaced, whose slots
 *   streamkl_paged_copy has to copy in every layer before new tokens are written;
 *   (-1, -1) for the others.
 * Where free pages do not suffice, a sequence is served if all that is asked up to
 * and with it is there, or it asks for none (and grows into no shared page); the
 * others keep length and pages, and STREAMKL_ERR_NO_PAGES is set (in a word of its
 * own where the step goes on: attention that is given a word with a failure in it
 * does nothing). They have no places for new tokens: appended at their lengths
 * all the same, these would be written over their last ones, in pages that others
 * may hold.
 *   step_lens [B], or NULL: the lengths for the calls of the step that follows, the
 *   new ones; 0 for the sequences that were not served (and those whose numbers do
 *   not fit). A sequence of length 0 that is given tokens is left alone by these
 *   calls: append and compact report it and write nothing, attention gives its rows
 *   zeros and -inf, so a captured step stays right whether pages suffice or not.
 *   Memory of its own: not kv_lens, not new_lens.
 * page_refs and copies are 16 and 8-byte aligned. The struct may end before
 * step_lens (struct_size says so).
 */
typedef struct {
  size_t struct_size;
  int* page_refs;
  int* block_table;
  long long table_stride;
  int* kv_lens;
  const int* new_lens; /* device [B], 0 .. max_pages * page_size */
  int* copies;
  int* dev_status;
  int B, num_pages, max_pages, page_size;
  int* step_lens;
} streamkl_resize_args;

streamkl_status streamkl_paged_resize(const streamkl_resize_args* args, void* stream);

/*
 * Self-test of the bounded-wait path: launches one tiny kernel that waits on
 * a barrier nothing arrives on, for timeout_us microseconds, then records
 * STREAMKL_ERR_TIMEOUT in *dev_status and returns. No other state is touched.
 * The paper has no counterpart; it exists so that the failure path of the
 * kernels' waits can be tested without hanging a GPU.
 */
streamkl_status streamkl_selftest_wait_timeout(int* dev_status, unsigned timeout_us,
                                               void* stream);

/*
 * Self-test of the debug build's range checks: launches one tiny kernel that
 * checks a TMEM column range lying past any allocation (no TMEM is allocated
 * and nothing is accessed). In the debug build (libstreamkl_debug.so) the
 * check fails and records STREAMKL_ERR_DEVICE_CHECK in *dev_status; in the
 * release build the checks are compiled out and *dev_status is left as it
 * was. The paper has no counterpart; it exists so that the report path of
 * the checks can be tested without a faulty access.
 */
streamkl_status streamkl_selftest_device_check(int* dev_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* STREAMKL_H_ */
