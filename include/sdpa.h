/*
 * sdpa.h — C ABI of the GB300 (sm_103a) fused scaled-dot-product attention library.
 *
 * What it computes.  For every batch b and query head hq (KV head hk = hq / (h_q / h_kv)):
 *
 *     S   = attn_scale * Q K^T                  (scores, then the scale)
 *     S  += bias                                 (optional: ALiBi, or a bias tensor)
 *     S  += mask   (causal: -inf where key j > query i, top-left or bottom-right aligned;
 *                   variable lengths: -inf on padded keys; otherwise no mask)
 *     P   = softmax(S) over each row
 *     O   = (P * keep / (1 - p)) V               (optional dropout; O has Q's shape)
 *     LSE = log(sum_j exp(S_ij))                 (natural log, per query row)
 *
 * [attention codelab "Speeding up attention on GPU with cuDNN and TransformerEngine",
 *  §1 "How attention works" (the four steps) and §7 "Adding a causal mask";
 *  cuDNN 9 blog "Accelerating Transformers with NVIDIA cuDNN 9", "SDPA as a cuDNN
 *  graph", Fig. 4 (BMM1 -> scale -> causal mask -> softmax -> BMM2); the SDPA node's
 *  second output "stats" is the per-row statistic kept for training, read here as the
 *  log-sum-exp; the walkthrough's options bias, use_alibi_mask, use_padding_mask with
 *  seq_len_q / seq_len_kv, and dropout; the codelab's §10 FP8 recipe.]  The backward pass
 *  returns dQ, dK, dV (and, on request, the bias gradient) for an incoming dO, using the LSE
 *  kept by the forward pass (the blog's "fprop + bprop" figure; the pages give no formula,
 *  the derivative is the analytic one).
 *
 * Conventions shared by every entry point
 *  - All tensors are *logical* BHSD [b][h][s][d] views over caller memory described by
 *    four element strides (sdpa_strides_t).  The innermost stride must be 1.  A BSHD
 *    buffer is passed with strides (s*h*d, d, h*d, 1) — no copy is made [cuDNN-in-Python
 *    post: the GPT-2-like example views a BSHD buffer as BHSD with as_strided].
 *  - Pointers are DEVICE pointers on the current CUDA device; bases must be 16-byte
 *    aligned and every non-unit stride, in bytes, a multiple of 16 (they are handed to
 *    the tensor-memory-accelerator (TMA) unit as is).
 *  - Ownership: the caller owns every buffer.  The library allocates no device memory,
 *    frees nothing, does not synchronise the stream and keeps no pointer after return.
 *  - Work is enqueued asynchronously on `stream` (0 = legacy default stream).
 *  - Errors: arguments are validated on the host before anything is launched; a non-OK
 *    status comes with a message from sdpa_last_error_string().  Unsupported inputs are an
 *    error, never a silent fallback.  Launch failures return SDPA_ERR_CUDA.
 *  - Thread safety: re-entrant.  Concurrent calls must not share a workspace.
 */
#ifndef SDPA_GB300_H
#define SDPA_GB300_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define SDPA_API __attribute__((visibility("default")))
#else
#define SDPA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SDPA_OK = 0,
  SDPA_ERR_INVALID_ARG = 1,   /* null pointer, non-positive size, h_q % h_kv != 0, ... */
  SDPA_ERR_UNSUPPORTED = 2,   /* valid request this library does not implement (e.g. d=96) */
  SDPA_ERR_LAYOUT = 3,        /* stride / alignment not expressible to the TMA unit */
  SDPA_ERR_WORKSPACE = 4,     /* workspace missing or smaller than sdpa_workspace_size() */
  SDPA_ERR_CUDA = 5,          /* a CUDA runtime/driver call failed (message has the code) */
  SDPA_ERR_TIMEOUT = 6        /* a bounded device wait gave up (see sdpa_device_error) */
} sdpa_status_t;

typedef enum {
  SDPA_DTYPE_F16 = 0,         /* IEEE binary16 */
  SDPA_DTYPE_BF16 = 1,        /* bfloat16 */
  SDPA_DTYPE_E4M3 = 2,        /* OCP FP8 E4M3 (finite max 448): Q, K, V (forward and backward) */
  SDPA_DTYPE_E5M2 = 3,        /* OCP FP8 E5M2 (max 57344): dO of an FP8 backward pass only */
  SDPA_DTYPE_F32 = 4          /* IEEE binary32: probabilities of sdpa_verify only */
} sdpa_dtype_t;

/* Element strides of a logical [b][h][s][d] view.  d must be 1. */
typedef struct {
  int64_t b, h, s, d;
} sdpa_strides_t;

/* One attention problem.  Fields not used by a call are ignored. */
typedef struct {
  int32_t b;           /* batch, >= 1 */
  int32_t h_q;         /* query heads, >= 1 */
  int32_t h_kv;        /* key/value heads, >= 1, h_q % h_kv == 0 (MHA: ==, GQA: <, MQA: 1);
                          query head hq reads KV head hq / (h_q / h_kv) [codelab §9] */
  int32_t s_q;         /* query rows, >= 1 */
  int32_t s_kv;        /* key/value rows, >= 1 */
  int32_t d;           /* head dim of Q, K and V: 64, 128 or 256 */
  int32_t in_dtype;    /* sdpa_dtype_t of Q, K, V (and of dO for the backward pass) */
  int32_t out_dtype;   /* sdpa_dtype_t of O (and dQ/dK/dV): == in_dtype for F16/BF16;
                          BF16 or F16 for E4M3 inputs */
  float attn_scale;    /* multiplies Q K^T before the mask and softmax; any finite value
                          (usually 1/sqrt(d)) [cuDNN 9 blog, Fig. 4: scale node after BMM1] */
  int32_t causal;      /* 0: no mask.  1: top-left causal, key j visible to query i iff j <= i
                          (row 0 sees only key 0) [codelab §7].  2: bottom-right causal, key j
                          visible to query i iff j <= i + len_kv - len_q (the last query sees
                          every key, as when decoding against a KV cache) */
  sdpa_strides_t q, k, v, o;         /* forward and backward */
  sdpa_strides_t dout, dq, dk, dv;   /* backward only (dout = incoming gradient dO) */
  const float* descale_q;  /* E4M3 only: DEVICE pointers to one fp32 each; the real value of */
  const float* descale_k;  /* a stored code x is decode(x) * descale (per-tensor scaling of    */
  const float* descale_v;  /* the delayed-scaling FP8 recipe, codelab §10).  NULL otherwise.   */
  /* Variable lengths (the SDPA node's padding mask with per-batch sequence lengths, cuDNN 9
   * blog walkthrough).  Optional DEVICE pointers to b int32 values; NULL = every row valid.
   * For batch b only query rows i < len_q[b] and keys j < len_kv[b] take part (values are
   * clamped to [0, s_q] and [0, s_kv]).  Rows with no visible key — padded rows, or early rows
   * of a bottom-right mask with len_kv < len_q — give O = 0 and LSE = -inf, and padded rows of
   * dQ, dK and dV are 0. */
  const int32_t* seq_lens_q;
  const int32_t* seq_lens_kv;
  /* ALiBi (the SDPA node's ALiBi-mask option, cuDNN 9 blog walkthrough; the pages name it but
   * do not define it, and this is the linear-bias reading).  0 = off.  1 = the scaled score of
   * (i, j) gains m_hq * (j - i - off) before the mask and softmax, off = len_kv - len_q under
   * bottom-right causal alignment and 0 otherwise: zero on the aligned diagonal, a penalty
   * growing linearly with the distance to earlier keys.  ALiBi needs a causal mask (causal 1
   * or 2: every visible key is then at or before the aligned diagonal); with causal = 0 it is
   * refused with SDPA_ERR_UNSUPPORTED.  m_hq = alibi_slopes[hq] (a DEVICE
   * pointer to h_q finite fp32 values >= 0; a negative slope counts as 0), or, when
   * alibi_slopes is NULL, the geometric slopes 2^(-8 (hq + 1) / h_q).  F16 and BF16 inputs
   * only; the bias has no gradient. */
  int32_t alibi;
  const float* alibi_slopes;
  /* Dropout (the SDPA node's dropout option, cuDNN 9 blog walkthrough; named, not defined by
   * the pages).  dropout_p in [0, 1); 0 = off.  With p > 0 each softmax probability P_ij is
   * kept where its keep bit is set and scaled by 1/(1 - p), so O = (P * keep) V / (1 - p); the
   * LSE is that of the undropped softmax.  The keep bits come from sdpa_dropout_mask: the
   * forward pass reads `dropout_mask` (row-major), the backward pass `dropout_mask_t` (the
   * same bits transposed); both DEVICE pointers, 16-byte aligned.  F16/BF16 inputs only. */
  float dropout_p;
  const uint32_t* dropout_mask;
  const uint32_t* dropout_mask_t;
  /* FP8 backward (the HYBRID recipe of the codelab's TransformerEngine section: E4M3 in the
   * forward pass, E5M2 for gradients).  Read only when in_dtype is E4M3 and the call is
   * sdpa_bwd: dO has dout_dtype (E5M2 or E4M3) with the per-tensor descale *descale_do
   * (DEVICE pointer); Q, K, V are E4M3 with descale_q/k/v; O and dQ, dK, dV have out_dtype
   * (BF16 or F16).  The codes are widened exactly to out_dtype in the workspace and the
   * descales folded into the kernels' scale factors; the MMAs run at 16-bit precision. */
  int32_t dout_dtype;
  const float* descale_do;
  /* Additive bias (the SDPA node's bias input, cuDNN 9 blog walkthrough).  NULL = none; else
   * a DEVICE pointer to a logical [b][h_q][s_q][s_kv] tensor of in_dtype (F16/BF16) whose
   * element strides are bias_strides (b, h, s, and d = the key stride, which must be 1); a
   * zero b or h stride broadcasts one slice over the batch or the heads.  The bias is added
   * to the scaled scores before the mask and softmax and is treated as a constant (no
   * gradient is produced).  Base 16-byte aligned; non-zero b/h/s strides multiples of 8.
   * Not combined with alibi (fold ALiBi into the tensor instead).  A backward pass with a
   * bias needs workspace for a transposed copy (sdpa_workspace_size accounts for it); its
   * gradient is available through dbias. */
  const void* bias;
  sdpa_strides_t bias_strides;
  /* Bias gradient (sdpa_bwd only; needs `bias`): NULL = not wanted; else a DEVICE pointer to
   * a tensor of the bias's shape and dtype, strides dbias_strides (zero b/h strides exactly
   * where bias_strides has them), overwritten with dL/dbias = dS — the gradient of the
   * scaled scores — summed over the broadcast dimensions.  Same alignment rules as bias.
   * The workspace then also holds an fp32 accumulator (sdpa_workspace_size accounts for it). */
  void* dbias;
  sdpa_strides_t dbias_strides;
} sdpa_problem_t;

/*
 * Workspace bytes that sdpa_fwd (is_backward = 0) or sdpa_bwd (is_backward = 1) needs for
 * `p`.  Writes *bytes; never launches anything.  The forward pass needs 0 bytes; the
 * backward pass needs fp32 scratch for dQ accumulation and the per-row Delta term
 * (4*b*h_q*round_up(s_q,128)*(d+1) bytes plus alignment).
 * [cuDNN-in-Python post: the workspace size is queried, then allocated by the caller.]
 */
SDPA_API sdpa_status_t sdpa_workspace_size(const sdpa_problem_t* p, int is_backward, size_t* bytes);

/*
 * Forward pass: O (and, when lse != NULL, the per-row log-sum-exp) from Q, K, V.
 *   q:   [b][h_q][s_q][d]   in_dtype, strides p->q
 *   k,v: [b][h_kv][s_kv][d] in_dtype, strides p->k, p->v
 *   o:   [b][h_q][s_q][d]   out_dtype, strides p->o; overwritten
 *   lse: NULL (inference: no statistics written) or fp32 [b][h_q][s_q] dense row-major;
 *        lse[(b*h_q + hq)*s_q + i] = ln sum_j exp(S_ij) over the visible keys; overwritten.
 *        The SDPA node's "stats" output, kept for training [cuDNN 9 blog, SDPA walkthrough;
 *        cuDNN-in-Python post].
 *   workspace / workspace_bytes: may be NULL / 0 (the forward pass needs none).
 * E4M3 inputs require descale_q/k/v and give a BF16 or F16 O.
 */
SDPA_API sdpa_status_t sdpa_fwd(const sdpa_problem_t* p, const void* q, const void* k, const void* v,
                       void* o, float* lse, void* workspace, size_t workspace_bytes,
                       void* stream /* cudaStream_t */);

/*
 * Backward pass: dQ, dK, dV of O for the incoming gradient dO, recomputing P from the LSE
 * written by sdpa_fwd on the same inputs.
 *   q, k, v, o: as in sdpa_fwd (o is the forward output); dout: [b][h_q][s_q][d], in_dtype
 *   lse: fp32 [b][h_q][s_q] from sdpa_fwd (required)
 *   dq: Q's shape, dk/dv: K's/V's shape, all out_dtype (== in_dtype); overwritten.  dK and
 *       dV hold the sum over the query heads of each KV group (GQA/MQA).
 *   workspace: >= sdpa_workspace_size(p, 1) bytes, 256-byte aligned; its contents on entry
 *       do not matter and are clobbered.
 * F16/BF16, or E4M3 Q/K/V with E5M2 or E4M3 dO (see dout_dtype).
 */
SDPA_API sdpa_status_t sdpa_bwd(const sdpa_problem_t* p, const void* q, const void* k, const void* v,
                       const void* o, const void* dout, const float* lse, void* dq, void* dk,
                       void* dv, void* workspace, size_t workspace_bytes,
                       void* stream /* cudaStream_t */);

/*
 * Size of the built-in scratch that sdpa_bwd_noalloc uses: 32 MiB of device memory, held by
 * every GPU on which the library's kernels are loaded, until the process exits.
 */
#define SDPA_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)

/*
 * sdpa_bwd_noalloc: the backward pass of sdpa_bwd for callers that cannot allocate device
 * memory — for example a plugin running inside a host framework that owns all device
 * memory and offers no allocator, or a latency-critical loop that must not call cudaMalloc
 * (which can synchronise the device).  Arguments and results are those of sdpa_bwd minus
 * the workspace: the scratch comes from a fixed array inside the library
 * (SDPA_NOALLOC_SCRATCH_BYTES), so nothing is allocated or freed.  The pages have no
 * counterpart of this entry point.
 *   - Problems whose workspace (sdpa_workspace_size(p, 1)) exceeds the array are rejected
 *     with SDPA_ERR_UNSUPPORTED and a message giving both sizes; use sdpa_bwd then.
 *   - The first call on a device looks up the array's device address (with that device
 *     current); make that first call before any stream capture.  The address is kept for
 *     the life of the process, so do not call this entry point again on a device after
 *     cudaDeviceReset() there (the reset unloads the module that holds the array).
 *   - Every call shares the one array (whatever it held is overwritten; each call clears
 *     what must start at zero), so calls whose executions overlap on the GPU — on different
 *     streams, or from different threads — race and give wrong results.  Serialise them.
 */
SDPA_API sdpa_status_t sdpa_bwd_noalloc(const sdpa_problem_t* p, const void* q, const void* k,
                                        const void* v, const void* o, const void* dout,
                                        const float* lse, void* dq, void* dk, void* dv,
                                        void* stream /* cudaStream_t */);

/*
 * Byte sizes of the two dropout keep-mask arrays of `p` (b, h_q, s_q, s_kv are read):
 *   mask:   uint32 [b*h_q][s_q][ceil(s_kv/128)*4]   (key j of row i at bit 16*(j%2) + (j%32)/2
 *           of word j/32: the two keys of an even/odd pair sit 16 bits apart)
 *   mask_t: uint32 [b*h_q][s_kv][ceil(s_q/128)*4]   (row i of key j at bit 16*(i%2) + (i%32)/2
 *           of word i/32: the two rows of an even/odd pair sit 16 bits apart)
 */
SDPA_API sdpa_status_t sdpa_dropout_mask_size(const sdpa_problem_t* p, size_t* bytes, size_t* bytes_t);

/*
 * Draws the dropout keep bits for p->dropout_p (in [0, 1)) with the counter-based generator
 * Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel Random Numbers: As Easy as 1, 2, 3",
 * SC'11).  Element n of the row-major grid [b*h_q][s_q][ceil(s_kv/128)*128] takes the 16-bit
 * half n%2 (0 = low) of 32-bit word (n%8)/2 of the block for the 128-bit counter (n/8, offset)
 * and the 64-bit key seed (each as 32-bit words, low word first), and is kept iff that value
 * is >= round(dropout_p * 65536).  The same (seed, offset) gives the same bits on every run
 * and device; advance `offset` between steps for fresh draws.
 *   mask, mask_t: DEVICE arrays of sdpa_dropout_mask_size bytes, 16-byte aligned; either may
 *   be NULL (not written).  Bits of padded positions (keys >= s_kv in `mask`, rows >= s_q in
 *   `mask_t`) are written too and are not used.  When p->causal is 1 or 2 and no seq_lens
 *   are given, 128x128 tiles that lie wholly above the causal diagonal are not written (the
 *   attention kernels never use them); pass causal = 0 for the full grid.
 */
SDPA_API sdpa_status_t sdpa_dropout_mask(const sdpa_problem_t* p, uint64_t seed, uint64_t offset,
                                         uint32_t* mask, uint32_t* mask_t, void* stream /* cudaStream_t */);

/* ------------------------------------------------------------------------------------------
 * Serving: rotary positions, a paged key/value cache, attention of new tokens over it.
 *
 * The conventions above hold for these entry points too: device pointers, logical
 * [b][h][s][d] views with a unit d stride, 16-byte aligned bases and strides, caller-owned
 * memory, asynchronous execution, validation on the host before any launch.
 * ------------------------------------------------------------------------------------------ */

/* Frequencies of the rotary positions (Su et al., "RoFormer", 2021): pair i of rot/2 turns by
 * f_i = base^(-2 i / rot) radians per position.  Scaled for contexts longer than the one a
 * model was trained on (original_context), by `factor` >= 1:
 *   0  none
 *   1  linear: every f_i / factor (position interpolation, Chen et al., 2023)
 *   2  NTK-aware: base * factor^(rot / (rot - 2)) instead of base
 *   3  by parts (YaRN, Peng et al., 2023): with r_i = original_context * f_i / (2 pi), the turns
 *      pair i makes over the original context, and g = clamp((r_i - beta_slow) /
 *      (beta_fast - beta_slow), 0, 1): f_i * g + f_i / factor * (1 - g); the factor on the
 *      rotated values is 0.1 ln(factor) + 1. */
typedef struct {
  int32_t rot;              /* rotated elements of a head: even, >= 2 */
  int32_t scaling;          /* 0..3 as above */
  double base;              /* > 0, usually 10000 */
  double factor;            /* scalings 1..3: >= 1 */
  double original_context;  /* scaling 3: > 0, tokens */
  double beta_fast, beta_slow;  /* scaling 3: beta_fast > beta_slow, usually 32 and 1 */
  const double* inv_freq;   /* NULL, or HOST pointer to rot/2 frequencies (radians per position)
                               that replace all of the above; the factor is then 1 */
} sdpa_rope_table_t;

/* Fills table[0 .. rot/2) (HOST memory; the caller copies it to the device) with the turns per
 * position of each pair as 64-bit binary fractions, table[i] = f_i / (2 pi) * 2^64 mod 2^64, and
 * *attn_factor (may be NULL) with the factor on the rotated values.  A position times such a
 * fraction, modulo 2^64, is the angle as a fraction of a turn with nothing lost to its size; what the entry
 * itself lacks (computed in fp64: within 2^-51 of it) counts as often as the position says, 5e-7
 * radians at 2^30 radians. */
SDPA_API sdpa_status_t sdpa_rope_table(const sdpa_rope_table_t* cfg, int64_t* table, float* attn_factor);

/* Rotary positions of Q and K in one call. */
typedef struct {
  int32_t b, h_q, h_k;      /* h_k = 0: Q alone */
  int32_t s;                /* rows (tokens) of each batch */
  int32_t d;                /* head dim: a multiple of 8, 8..512 */
  int32_t rot;              /* rotated elements, even, 2..d: the first `rot` of each head; the others
                               are copied */
  int32_t dtype;            /* F16 or BF16 */
  int32_t interleaved;      /* pairs: 0 = elements (i, i + rot/2), 1 = elements (2i, 2i + 1) */
  float attn_factor;        /* multiplies the rotated elements (1 = none) */
  const int64_t* table;     /* DEVICE, rot/2 entries of sdpa_rope_table */
  const int32_t* positions; /* DEVICE [b][s], or NULL: row i of every batch is at position i */
  int64_t positions_stride; /* elements between two batches of positions (0: one row for all) */
  sdpa_strides_t q, k;           /* inputs */
  sdpa_strides_t q_out, k_out;   /* outputs */
} sdpa_rope_t;

/* y = factor * R(position) x for Q and K: pair (a, b) at angle t becomes
 * (a cos t - b sin t, a sin t + b cos t), computed in fp32 and rounded once.
 *   q_out may be q (with the same strides) and k_out may be k; otherwise outputs overlap no input. */
SDPA_API sdpa_status_t sdpa_rope_fwd(const sdpa_rope_t* p, const void* q, const void* k, void* q_out,
                                     void* k_out, void* stream);

/* The gradient of sdpa_rope_fwd: dx = factor * R(position)^T dy.  dq_out/dk_out (the incoming
 * gradients) have the views p->q/p->k, dq/dk the views p->q_out/p->k_out. */
SDPA_API sdpa_status_t sdpa_rope_bwd(const sdpa_rope_t* p, const void* dq_out, const void* dk_out, void* dq,
                                     void* dk, void* stream);

/* Positions with several axes (time, row and column of an image's or a clip's tokens, say): pair i of a head turns by the
 * position on its own axis, t = positions[axis[i]] * f_i; the table holds f_i pair by pair, as ever (for axes with
 * frequencies of their own, one axis's table behind the other's). */
typedef struct {
  int32_t axes;             /* 1..4 */
  uint8_t axis[256];        /* the axis of each of the rot/2 pairs, below `axes` */
  int64_t axis_stride;      /* elements between two axes of positions */
} sdpa_rope_axes_t;

/* sdpa_rope_fwd and sdpa_rope_bwd with p->positions DEVICE [axes][b][s] (not NULL; positions_stride between batches, 0:
 * one row for all). */
SDPA_API sdpa_status_t sdpa_rope_axes_fwd(const sdpa_rope_t* p, const sdpa_rope_axes_t* a, const void* q, const void* k,
                                          void* q_out, void* k_out, void* stream);
SDPA_API sdpa_status_t sdpa_rope_axes_bwd(const sdpa_rope_t* p, const sdpa_rope_axes_t* a, const void* dq_out,
                                          const void* dk_out, void* dq, void* dk, void* stream);

/* A paged key/value cache.  Position j of sequence i lives in page page_table[i][j / page_size],
 * slot j % page_size.  Keys and values are logical [num_pages][h_kv][page_size][d] views (the
 * fields b, h, s, d of the strides are page, head, slot, element), so a page may be stored
 * head-major or slot-major.  E4M3 caches have an fp32 scale >= 0 for each token and head:
 * value = code * scale; any such scale will do, zero and subnormal ones included. */
typedef struct {
  int32_t num_pages;        /* >= 1 */
  int32_t page_size;        /* tokens of a page: a multiple of 16 */
  int32_t h_kv;             /* >= 1 */
  int32_t d;                /* 64, 128 or 256 */
  int32_t dtype;            /* F16, BF16 or E4M3 */
  int32_t b;                /* sequences */
  int32_t max_pages;        /* columns of the page table.  sdpa_decode splits its work by them, since lengths are
                               on the device: a view narrowed to the batch's longest sequence (the stride stays)
                               spares short sequences a launch and a large workspace */
  void* k;
  void* v;
  sdpa_strides_t k_strides, v_strides;
  float* k_scale;           /* E4M3: DEVICE [num_pages][h_kv][page_size] dense, 16-byte aligned; else NULL */
  float* v_scale;
  const int32_t* page_table;   /* DEVICE [b][max_pages]; columns a sequence does not reach are not read.
                                  Positions whose page is outside [0, num_pages) hold no key: they are
                                  not written, read back as zeros and hidden from every query */
  int64_t page_table_stride;   /* elements between two sequences */
  const int32_t* seq_lens_kv;  /* DEVICE [b]: tokens of each sequence, those of this call included
                                  (clamped to [0, max_pages * page_size], and to 2^30) */
} sdpa_cache_t;

/* New rows for the cache (sdpa_cache_write), or dense rows read from it (sdpa_cache_read). */
typedef struct {
  int32_t s;                   /* rows of each sequence */
  int32_t dtype;               /* F16 or BF16; the cache's own dtype unless that is E4M3 */
  sdpa_strides_t k, v;         /* [b][h_kv][s][d] */
  const int32_t* seq_lens_q;   /* write: DEVICE [b] new rows of each sequence (clamped to [0, s]), or NULL: s */
  const sdpa_rope_t* rope;     /* write: NULL, or K is rotated first: rot, interleaved, attn_factor, table,
                                  positions and positions_stride are read (positions NULL: each row's
                                  position in its sequence) */
} sdpa_cache_rows_t;

/* Writes row i < len_q of each sequence to position len_kv - len_q + i (rows before position 0
 * are not written).  16-bit caches take the (rotated) values rounded once; E4M3 caches take
 * scale = max(amax, 2^-60) / 448 over the d elements of each row, and code = x * (1 / scale)
 * rounded to the nearest E4M3 value (K: rotated in fp32, with no rounding in between).  A row that
 * holds an infinity or a NaN reads back as NaN.  Two rows of one call must not map to the same
 * slot.  Other slots are left as they are. */
SDPA_API sdpa_status_t sdpa_cache_write(const sdpa_cache_t* c, const sdpa_cache_rows_t* r, const void* k,
                                        const void* v, void* stream);

/* sdpa_cache_write with r->rope (not NULL) and its positions DEVICE [axes][b][s] (not NULL). */
SDPA_API sdpa_status_t sdpa_cache_write_axes(const sdpa_cache_t* c, const sdpa_cache_rows_t* r, const sdpa_rope_axes_t* a,
                                             const void* k, const void* v, void* stream);

/* Reads positions 0 .. s-1 of each sequence into dense rows, code * scale rounded once; rows at
 * len_kv and behind are zeros (as sdpa_fwd with seq_lens_kv wants its padding). */
SDPA_API sdpa_status_t sdpa_cache_read(const sdpa_cache_t* c, const sdpa_cache_rows_t* r, void* k, void* v,
                                       void* stream);

/* Attention of the newest tokens over the cache. */
typedef struct {
  int32_t h_q;                 /* h_q % h_kv == 0 */
  int32_t s_q;                 /* rows (new tokens) of each sequence, >= 1 */
  int32_t dtype;               /* F16 or BF16, of Q and O; the cache's own dtype unless that is E4M3 */
  int32_t causal;              /* 0: every row sees the whole sequence.  2: bottom-right causal, row i sees
                                  keys j <= i + len_kv - len_q */
  float attn_scale;
  sdpa_strides_t q, o;         /* [b][h_q][s_q][d] */
  const int32_t* seq_lens_q;   /* DEVICE [b] rows that take part (clamped to [0, s_q]), or NULL: s_q */
  const uint32_t* tree_mask;   /* NULL, or DEVICE [b][s_q][ceil(s_q/32)]: the rows are drafted tokens, already
                                  in the cache as its last len_q positions; row i sees every earlier
                                  position, and of the drafted ones those j with bit j%32 of word j/32
                                  set.  causal must be 0 */
  int64_t tree_mask_stride;    /* 32-bit words between two sequences' masks (0: one tree for all) */
} sdpa_decode_t;

/* Workspace bytes of sdpa_decode (a function of the sizes alone, not of the lengths). */
SDPA_API sdpa_status_t sdpa_decode_workspace_size(const sdpa_cache_t* c, const sdpa_decode_t* p, size_t* bytes);

/* O (and LSE when lse != NULL: fp32 [b][h_q][s_q] dense, natural log) of the new tokens over the
 * cache.  Rows with no visible key, and rows >= len_q, give O = 0 and LSE = -inf.  Values at
 * hidden positions may hold anything, NaN included.  LSE depends on Q and K alone, whatever V and its scales are.
 * Weights are rounded once to the cache's 16-bit type (E4M3: F16), or kept to twice its bits where at most 8 rows
 * share a KV head and results keep as many.  Over an E4M3 cache a key adds to O within 2^-19 of the largest
 * V scale that the row sees times its largest weight, however small its own: far below that scale's own rounding.
 * Scores keep their fractions up to 2^24 (fp32); as in sdpa_fwd, rows with scores of 10^7 (F16, E4M3) or 10^9 (BF16)
 * and more may come out as NaN where more than 16 rows share a KV head (E4M3: 32).
 *   workspace: >= sdpa_decode_workspace_size bytes, 256-byte aligned; contents on entry do not matter. */
SDPA_API sdpa_status_t sdpa_decode(const sdpa_cache_t* c, const sdpa_decode_t* p, const void* q, void* o,
                                   float* lse, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------------------------
 * Pages: who owns which page of a cache, and pages and rows moved inside it.
 *
 * Every page has a count of its owners: the rows of page tables that reach it, and what else the caller counts
 * (a prefix that it keeps for later, say).  A page is free iff its count is 0.  The calls below change
 * counts and page tables on the device, without a copy to the host; they touch no keys and values, since the layers
 * of a model share a page table: where pages have to be copied they list them, and sdpa_cache_copy is
 * called for each layer's cache.
 *
 * A sequence of n tokens reaches columns 0 .. ceil(n / page_size) - 1 of its row; other columns are neither read nor
 * counted.  Lengths are clamped as in sdpa_cache_t.  Entries outside [0, num_pages) are missing pages: they have
 * no count.  Counts must be at least the number of reaching entries.  What a call writes lies apart from what it reads and from
 * what else it writes, but for a table or counts that are changed in place; anything else is refused.  Calls that
 * change the same counts or the same table must not run at the same time.
 * ------------------------------------------------------------------------------------------ */
typedef struct {
  int32_t num_pages;            /* 1..2^30 */
  int32_t page_size;            /* a multiple of 16 */
  int32_t b;                    /* rows of page_table: sequences, 1..2^24 */
  int32_t max_pages;            /* columns, 1..2^30 */
  const int32_t* page_table;    /* DEVICE [b][max_pages] */
  int64_t page_table_stride;
  const int32_t* seq_lens;      /* DEVICE [b]: tokens of each sequence */
  const int32_t* ref_counts;    /* DEVICE [num_pages] */
  int32_t* page_table_out;      /* DEVICE: may be page_table with its stride, otherwise apart from it (sdpa_cache_fork: always) */
  int64_t page_table_out_stride;
  int32_t* ref_counts_out;      /* DEVICE [num_pages]: may be ref_counts, otherwise apart from it */
} sdpa_pages_t;

/* Row i < b_out of the new table takes over sequence parents[i] with its pages (shared, none copied): parents DEVICE [b_out],
 * a value outside [0, b) gives an empty sequence.  Columns not reached are -1.  seq_lens_out: DEVICE [b_out].  The old
 * rows' ownership ends: sequences that nobody takes over are freed.  (A sequence that goes on beside its copies
 * is one of its own parents.)  Outputs lie apart from page_table and seq_lens. */
SDPA_API sdpa_status_t sdpa_cache_fork(const sdpa_pages_t* p, const int32_t* parents, int32_t b_out, int32_t* seq_lens_out,
                                       void* stream);

/* Room for sequences to grow from seq_lens to new_lens (DEVICE [b]; a shorter one changes nothing).  Every column that
 * new_lens reaches and seq_lens does not gets a free page, lowest first in the order of rows and columns.  A
 * partly filled page that others own too is replaced as well, by all of the rows that grow in it but the last owner: the free page takes its
 * column's place in that order, and (src[i], dst[i]) is the copy that row i needs before it is written
 * (DEVICE [b] each; -1, -1: none).  All or nothing: *missing (DEVICE) is 0, or the number of pages that
 * lacked, and nothing is changed then (outputs that lie apart are copies).  What follows must take *missing into account: a
 * program that does not wait for it gives the calls behind this one the old lengths and 0 new rows (seq_lens_q) where it is not
 * 0, as new rows would go into pages that sequences still share.  At most 4096 rows. */
SDPA_API sdpa_status_t sdpa_cache_grow(const sdpa_pages_t* p, const int32_t* new_lens, int32_t* src, int32_t* dst,
                                       int32_t* missing, void* stream);

/* Gives back the columns that seq_lens reaches and keep_lens (DEVICE [b], clamped to [0, seq_lens]) does not: their entries
 * become -1, their pages lose an owner. */
SDPA_API sdpa_status_t sdpa_cache_free(const sdpa_pages_t* p, const int32_t* keep_lens, void* stream);

/* Moves pages together, so that n pages in use are pages 0 .. n-1: the k-th page in use at or behind n becomes the k-th free
 * one before it, at most `pairs` of them in one call.  src and dst (DEVICE [pairs], src ascending, -1 behind the
 * last) list the copies to make before the pages are read again; src pages are free from then on.  Owners that are not in
 * this page table find their pages' new names in the lists. */
SDPA_API sdpa_status_t sdpa_cache_compact(const sdpa_pages_t* p, int32_t* src, int32_t* dst, int32_t pairs, void* stream);

/* Copies pages src[i] to dst[i] of K, V and their scales (DEVICE [pairs] each).  Pairs with an entry outside
 * [0, num_pages) are passed over.  No page may be the target of two pairs, nor target of one and source of another.
 * Of c the page table, b, max_pages and seq_lens_kv are not read. */
SDPA_API sdpa_status_t sdpa_cache_copy(const sdpa_cache_t* c, const int32_t* src, const int32_t* dst, int32_t pairs, void* stream);

/* Keeps some of the newest tokens: of the last len_q positions of each sequence (seq_lens_q DEVICE [b], clamped to [0, s], or
 * NULL: s), row path[i][j] moves to row j for all j < accepted[i].  path: DEVICE [b][s], ascending in the
 * part that is read (as sdpa_verify gives it); entries outside [0, len_q) move nothing.  accepted: DEVICE [b].  Lengths are the
 * caller's: seq_lens_kv - len_q + accepted afterwards; rows behind that are left as they come.  K, V and their scales.  The pages
 * of those positions are to be the sequence's own, as sdpa_cache_grow leaves them. */
SDPA_API sdpa_status_t sdpa_cache_keep(const sdpa_cache_t* c, const int32_t* path, const int32_t* accepted, int32_t s,
                                       const int32_t* seq_lens_q, void* stream);

/* Drafted tokens verified against the target's probabilities (speculative sampling: Leviathan et al., Chen et al., 2023; without
 * draft_probs a tree of candidates as in Miao et al., 2023).  accepted, path and new_tokens lie apart from each other and from all
 * that is read: a sequence's rows are read by several CTAs, and one of them writes. */
typedef struct {
  int32_t b;                    /* sequences */
  int32_t s;                    /* rows of each, 1..1024: row 0 the newest token that is decided, the others drafted */
  int32_t vocab;                /* 1..2^20 */
  int32_t dtype;                /* F16, BF16 or F32, of probs and draft_probs */
  const int32_t* tokens;        /* DEVICE [b][s]; row 0's is not read.  A token outside [0, vocab) is refused */
  const int32_t* parents;       /* DEVICE [b][s]: the row that row i > 0 follows, below i (rows with any other value, and rows
                                   behind those, are never accepted); row 0's is not read.  NULL: a chain, i - 1 */
  const int32_t* seq_lens_q;    /* DEVICE [b] rows that take part (clamped to [0, s]; 0: nothing is accepted and no token drawn), or NULL: s */
  const float* uniform;         /* DEVICE [b][s]: random numbers in [0, 1): row 0's draws the new token, the others test their rows */
  const void* probs;            /* DEVICE [b][s][vocab], strides below (elements; vocab: 1): the target's distribution behind each row */
  int64_t probs_b, probs_s;
  const void* draft_probs;      /* DEVICE [b][s][vocab], or NULL: the distribution that row i > 0 was drawn from.  Chains only */
  int64_t draft_b, draft_s;
  int32_t* accepted;            /* DEVICE [b]: accepted rows, row 0 among them */
  int32_t* path;                /* DEVICE [b][s]: those rows in order, -1 behind them */
  int32_t* new_tokens;          /* DEVICE [b][s]: the tokens of rows path[1..], and the new one: `accepted` tokens, -1 behind them */
} sdpa_verify_t;

/* Children of an accepted row n are tried in ascending order.  Child i with token x is accepted iff
 *   uniform[i] * draft_probs[i][x] < probs[n][x]                                    with draft_probs, or
 *   uniform[i] * max(0, 1 - sum of probs[n][x'] of refused siblings) < probs[n][x]  without (in the whole numbers below; a token
 *                                                                                   that an earlier sibling has too is refused).
 * The new token is drawn behind the last accepted row n: from max(probs[n] - draft_probs[i], 0) where a chain's row i was refused,
 * from probs[n] without its children's tokens where there are no draft_probs; from probs[n] where that leaves nothing.
 * Tokens so chosen are distributed as the target's own; without draft_probs as far as its rows sum to one, since the tests take
 * the total for one and the draw goes by the sum that is there (rows in 16 bits are off by what their roundings add up to).
 * Differences of probabilities are rounded to fp32.  In sums and draws a probability counts as a whole number of 2^-42
 * (values outside [0, 1] as the nearer end, NaN as 0; 2^-43 and less is nothing): the new token is the first whose running sum exceeds
 * floor(uniform[0] * 2^31) / 2^31 of the total, whatever the order of the sums.  Where the total is 0 it is -1. */
SDPA_API sdpa_status_t sdpa_verify(const sdpa_verify_t* p, void* stream);

/* sizeof of the structs above as compiled into the library: which = 0 sdpa_rope_table_t,
 * 1 sdpa_rope_t, 2 sdpa_cache_t, 3 sdpa_cache_rows_t, 4 sdpa_decode_t, 5 sdpa_rope_axes_t, 6 sdpa_pages_t,
 * 7 sdpa_verify_t (0 for any other). */
SDPA_API size_t sdpa_serving_struct_size(int which);

/* Message for the last non-OK status returned on the calling thread ("" if none).  The
 * pointer stays valid until the next library call on this thread [cuDNN 9 blog: errors
 * come with a retrievable last-error string]. */
SDPA_API const char* sdpa_last_error_string(void);

/*
 * Device-side error word of the current device: bit 0 = a bounded wait inside a kernel
 * gave up (the kernel then skipped its remaining work and returned without faulting);
 * bit 1 = shared memory was not 1024-byte aligned (the kernel did nothing).
 * Synchronises the device, writes the word to *flags and clears it.  Returns SDPA_OK, or
 * SDPA_ERR_CUDA if the synchronisation or copy failed.
 */
SDPA_API sdpa_status_t sdpa_device_error(uint32_t* flags);

/* Library version as major*10000 + minor*100 + patch. */
SDPA_API int sdpa_version(void);

/* sizeof(sdpa_problem_t) as compiled into the library, so that bindings built from this
 * header can check their copy of the struct layout. */
SDPA_API size_t sdpa_problem_struct_size(void);

#ifdef __cplusplus
}
#endif

#endif /* SDPA_GB300_H */
