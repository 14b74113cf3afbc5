/*
 * mtp.h -- C ABI of libmtp: the data-parallel hot path of DeepSeek-V3-style
 * sequential multi-token prediction on NVIDIA GB300 (sm_103a).
 *
 * Sources ("the pages"):
 *   [M7.6] "M7.6 - DeepSeek MTP: Sequential Modules, Teacher Forcing, and
 *          Speculative Runtime" (transformer-system.numinens.com)
 *   [M7.4] "M7.4 - Multi-Token Prediction Foundations" (same site)
 *   [SD]   speculative-decoding page, ailearn.mscapital.top ("投机解码")
 *
 * Conventions shared by every entry point:
 *   - Every tensor pointer is a DEVICE pointer (cudaMalloc / torch CUDA
 *     memory) unless the argument says "host".  Tensors are dense,
 *     row-major, 16-byte aligned.  The caller owns all memory; the library
 *     allocates nothing and keeps no state besides one device error word per
 *     translation unit (read with mtp_check_errors) and the tensor-map
 *     encoder entry point resolved on first use.
 *   - Calls are asynchronous on `stream`.  Inside one call, a GEMM or a kernel of
 *     an attention may be launched as a programmatic dependent of the call's
 *     previous kernel (its setup overlaps that kernel, or it runs beside it; it
 *     reads nothing that the kernel writes before it completes); the
 *     first kernel of every call is an ordinary launch, so a call is ordered
 *     after all earlier work on `stream`.  Argument errors are detected on the
 *     host, return a status and launch nothing.  Data-dependent errors (token
 *     id out of range, a kernel wait that ran out of time) set bits of the
 *     device error word (MTP_DEVERR_*) and never trap; spec_verify reports
 *     per-request statuses instead.
 *   - bf16 means IEEE bfloat16 storage with fp32 accumulation.  f32 means
 *     fp32 storage and arithmetic.
 */
#ifndef MTP_H
#define MTP_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MTP_ABI_VERSION 1

typedef enum mtp_status {
  MTP_OK = 0,
  MTP_ERR_INVALID_ARG = 1,  /* null pointer, negative size, bad enum        */
  MTP_ERR_SHAPE = 2,        /* inconsistent dimensions                      */
  MTP_ERR_ALIGNMENT = 3,    /* pointer not 16-byte aligned                  */
  MTP_ERR_WORKSPACE = 4,    /* workspace smaller than the query returned     */
  MTP_ERR_CUDA = 5,         /* a CUDA runtime/driver call failed             */
  MTP_ERR_DEVICE = 6,       /* a kernel set the device error word           */
  MTP_ERR_UNSUPPORTED = 7   /* a shape/dtype combination not implemented  */
} mtp_status;

/* MTP_E4M3: 8-bit codes of a paged cache (mtp_paged_cache) only. */
typedef enum mtp_dtype { MTP_F32 = 0, MTP_BF16 = 1, MTP_E4M3 = 2 } mtp_dtype;

/* Denominator policy of each loss term ([M7.6] §0x05).
 * FIXED: every term (main and each depth) divided by B*T, the paper's fixed
 *        denominator for a batch of B packed rows of T positions.
 * MASKED_MEAN: each term divided by its own count of supervised rows; an
 *        empty term is 0 and stays in the D-depth mean ([M7.6] §0x06A). */
/* How the per-depth loss sums S_k (k = 0 main, 1..D depths) and counts N_k
 * become the reported terms L^(k) ("M7.4 - Multi-Token Prediction
 * Foundations" §0x02C names the last four):
 *   FIXED          L^(k) = S_k / n_positions (the paper's 1/T, batch form)
 *   MASKED_MEAN    L^(k) = S_k / N_k          (head mean)
 *   SUM            L^(k) = S_k
 *   GLOBAL         L^(k) = S_k / sum_j N_j    (depths only)
 *   WEIGHTED_PAIR  L^(k) = S_k / sum_j w_j N_j (depths only)
 * and total = L_main + sum_k w_k L^(k), w_k the per-depth weights (lambda/D
 * unless given).  L_main is S_0 / n_positions (FIXED), S_0 (SUM), else
 * S_0 / N_0.  A zero denominator gives 0. */
typedef enum mtp_den {
  MTP_DEN_FIXED = 0,
  MTP_DEN_MASKED_MEAN = 1,
  MTP_DEN_SUM = 2,
  MTP_DEN_GLOBAL = 3,
  MTP_DEN_WEIGHTED_PAIR = 4
} mtp_den;

/* Per-request status written by spec_verify. */
enum {
  MTP_VERIFY_OK = 0,
  MTP_VERIFY_INVALID_DRAFT = 1,   /* draft id outside [0,V) or q_j[y_j] <= 0  */
  MTP_VERIFY_ZERO_RESIDUAL = 2,   /* rejection (or bonus row) with no mass     */
  MTP_VERIFY_INVALID_PROBS = 3,   /* NaN/Inf/negative entry in a row it read   */
  MTP_VERIFY_INVALID_BUDGET = 4,  /* remaining < 1                             */
  MTP_VERIFY_DEVICE_TIMEOUT = 5   /* a bounded wait gave up (also sets the
                                     device error word's MTP_DEVERR_TIMEOUT)  */
};

/* Per-row status written by mtp_logits_probs (rows that are not OK are all zero). */
enum {
  MTP_LOGITS_OK = 0,
  MTP_LOGITS_EMPTY = 1,        /* no allowed token has a logit above -inf      */
  MTP_LOGITS_INVALID = 2,      /* an allowed token's logit is NaN or +inf      */
  MTP_LOGITS_INVALID_PARAM = 3 /* temperature < 0, repetition <= 0, or one of
                                  the request's parameters is not finite       */
};

/* Bits of the device error word. */
enum {
  MTP_DEVERR_TOKEN_RANGE = 1u,  /* a token id outside [0, V) was read (clamped) */
  MTP_DEVERR_TIMEOUT = 2u,      /* a bounded pipeline wait gave up             */
  MTP_DEVERR_SEGMENTS = 4u,     /* a segment id re-appears after another one   */
  MTP_DEVERR_PAGE_RANGE = 8u,   /* a page outside [0, n_pages) or a row outside a
                                   request's pages was named (passed over)       */
  /* set beside the condition bits above: which kernel family raised them */
  MTP_DEVERR_FROM_CHAIN = 1u << 8,   /* prologue, norms, segment scan, CE reduce */
  MTP_DEVERR_FROM_GEMM = 1u << 9,    /* tcgen05 GEMM core                        */
  MTP_DEVERR_FROM_ATTN = 1u << 10,   /* chain attention                           */
  MTP_DEVERR_FROM_VERIFY = 1u << 11, /* spec_verify                               */
  MTP_DEVERR_FROM_DRAFT = 1u << 12,  /* draft-step kernels                        */
  MTP_DEVERR_FROM_FP8 = 1u << 13,    /* FP8 block-scaled weight GEMM              */
  MTP_DEVERR_FROM_DGEMM = 1u << 14,  /* bf16 decode-shaped GEMM                   */
  MTP_DEVERR_FROM_PREFIX = 1u << 15, /* shared-prefix attention                    */
  MTP_DEVERR_FROM_PAGED = 1u << 16,  /* rows of a paged cache                      */
  MTP_DEVERR_FROM_PAGED_ATTN = 1u << 17 /* attention over a paged cache            */
};

/* Problem sizes of one chain call.
 * B packed rows of T positions; model width d = n_heads * head_dim; SwiGLU
 * width ffn; shared vocabulary V; D sequential MTP depths.  eps is the RMSNorm
 * epsilon (the pages leave it open; 1e-6 recommended).  rope_base > 0 applies
 * rotate-half rotary embedding with that base to q and k at the given
 * positions; 0 disables it.  dtype is an mtp_dtype.
 * bf16 requires d % 128 == 0, head_dim in {64, 128}, ffn % 8 == 0; f32
 * requires head_dim <= 128 and T <= 12800. */
typedef struct mtp_dims {
  int B, T, d, n_heads, head_dim, ffn, V, D;
  float eps;
  float rope_base;
  int dtype;
} mtp_dims;

/* Weights of the chain ([M7.6] §0x03, §0x04B).  Shared by the main head and
 * every depth (passed once): embed [V,d], head [V,d], out_norm [d].
 * Per depth k = 0..D-1, each field below is a HOST array of D device
 * pointers: hnorm, enorm, attn_norm, ffn_norm [d]; eh_proj [d, 2d] whose
 * first d columns multiply the normalised hidden state and last d columns
 * the normalised embedding ("he" order, [M7.6] §0x03, §0x07B); wq, wk, wv,
 * wo [d, d]; w_gate, w_up [ffn, d]; w_down [d, ffn].  Every linear map is
 * y = x W^T (row-major [out, in]).  Element type = dims.dtype. */
typedef struct mtp_weights {
  const void* embed;
  const void* head;
  const void* out_norm;
  const void* const* hnorm;
  const void* const* enorm;
  const void* const* eh_proj;
  const void* const* attn_norm;
  const void* const* wq;
  const void* const* wk;
  const void* const* wv;
  const void* const* wo;
  const void* const* ffn_norm;
  const void* const* w_gate;
  const void* const* w_up;
  const void* const* w_down;
} mtp_weights;

/* Bytes of device workspace mtp_chain_forward / mtp_chain_loss need for
 * these sizes (0 if the sizes are invalid). */
size_t mtp_chain_workspace_bytes(const mtp_dims* dims);

/* Teacher-forced MTP chain, depths 1..D ([M7.6] §0x02-§0x04C, §0x06A).
 * For depth k and position t of packed row b:
 *   h̄ = RMSNorm_{h,k}(h^{k-1}_t), ē = RMSNorm_{e,k}(E[x_{t+k}]),
 *   u = M_k [h̄; ē], a = u + Attn_k(RMSNorm_{a,k}(u)), h^k_t = a + FFN_k(RMSNorm_{f,k}(a))
 * where attention is causal within the segment of t and FFN is SwiGLU.
 * Row t has a state at depth k iff t, ..., t+k are active and in one
 * segment ([M7.6] §0x04C); rows without a state are computed on clamped
 * inputs but their values are undefined.
 *   tokens [B,T] int32 in [0,V) (others set MTP_DEVERR_TOKEN_RANGE and are
 *   clamped); seg [B,T] int32 segment ids, -1 = padding; within a packed row
 *   the ids of successive segments strictly increase (a repeated id sets
 *   MTP_DEVERR_SEGMENTS); pos [B,T] int32 RoPE positions in [0,T), typically
 *   the index within the segment; h0 [B,T,d] main-model hidden states.
 *   h_out [D,B,T,d] receives h^1..h^D (pre-final-norm states).
 *   ws: workspace of at least mtp_chain_workspace_bytes(dims) bytes. */
mtp_status mtp_chain_forward(const mtp_dims* dims, const mtp_weights* w,
                             const int32_t* tokens, const int32_t* seg, const int32_t* pos,
                             const void* h0, void* h_out,
                             void* ws, size_t ws_bytes, cudaStream_t stream);

/* Chain forward plus the shared head and masked cross-entropy
 * ([M7.6] §0x03, §0x05; [M7.4] §0x06F), without materialising logits:
 *   ℓ_t = log Σ_v exp(z_v) - z_label, z = W_U RMSNorm_out(h_t).
 * Term 0 (main) uses h0 with label x_{t+1}, supervised where t+1 is active
 * and in the segment of t; term k uses h^k with label x_{t+k+1}, supervised
 * where t..t+k+1 are active and in one segment.  Then
 *   L = L_main + (lambda / D) Σ_k L^(k), each term reduced by `den`.
 *   sums_counts [2*(D+1)] double: (Σℓ, count) for main, then depths 1..D.
 *   losses [D+2] float: L, L_main, L^(1)..L^(D).
 *   row_loss [(D+1),B,T] float, nullable: ℓ per term and row, NaN where the
 *   row is not supervised.  h_out nullable, as in mtp_chain_forward.
 *   with_main = 0 skips the main term (L_main = 0, its sum/count = 0). */
mtp_status mtp_chain_loss(const mtp_dims* dims, const mtp_weights* w,
                          const int32_t* tokens, const int32_t* seg, const int32_t* pos,
                          const void* h0, float lambda, int den, int with_main,
                          double* sums_counts, float* losses, float* row_loss, void* h_out,
                          void* ws, size_t ws_bytes, cudaStream_t stream);

/* Allocation-free variant of mtp_chain_loss.  The pages have no counterpart:
 * this is an integration entry point.  It is for callers that cannot call
 * cudaMalloc or own device memory for a workspace -- plugin hosts whose
 * allocator belongs to someone else, runtimes that forbid allocation on their
 * hot path, code that must not touch the allocator in the middle of a
 * stream.  Same arguments and results as mtp_chain_loss, without ws/ws_bytes:
 * the workspace is a static device array of MTP_NOALLOC_SCRATCH_BYTES inside
 * the library, held on every GPU that loads the library until the process
 * exits.  Returns MTP_ERR_WORKSPACE, launching nothing, when
 * mtp_chain_workspace_bytes(dims) exceeds that size (small shapes only).  The
 * first call on a device looks up the array's device address with that device
 * current; make that first call before any stream capture.  The address is
 * kept for the life of the process: after cudaDeviceReset of a device, do not
 * call this entry point on that device again.  Calls share the
 * one array: calls that overlap on the GPU race, so serialise them (one
 * stream, or events).  It allocates nothing itself. */
#define MTP_NOALLOC_SCRATCH_BYTES (32u * 1024u * 1024u)
mtp_status mtp_chain_loss_noalloc(const mtp_dims* dims, const mtp_weights* w,
                                  const int32_t* tokens, const int32_t* seg, const int32_t* pos,
                                  const void* h0, float lambda, int den, int with_main,
                                  double* sums_counts, float* losses, float* row_loss, void* h_out,
                                  cudaStream_t stream);

/* Loss assembly from per-term (sum, count) pairs ([M7.6] §0x05, §0x06A):
 * L = L_main + (lambda / D) Σ_k L^(k) with each term reduced by `den`
 * (FIXED divides by n_positions).  A data-parallel caller all-reduces the
 * sums_counts of mtp_chain_loss across ranks first -- numerators and
 * denominators are reduced before dividing -- and passes the global
 * n_positions.  sums_counts [2*(D+1)] double, losses [D+2] float (device). */
mtp_status mtp_loss_assemble(int D, const double* sums_counts, double n_positions, float lambda,
                             int den, int with_main, float* losses, cudaStream_t stream);

/* mtp_loss_assemble with per-depth weights: depth_weights is a HOST array of
 * D floats copied at the call (NULL = lambda/D each; D <= 32 when given). */
mtp_status mtp_loss_assemble_weighted(int D, const double* sums_counts, double n_positions,
                                      const float* depth_weights, float lambda, int den, int with_main,
                                      float* losses, cudaStream_t stream);

/* Exact speculative verification of R requests with gamma drafts each
 * ([M7.6] §0x09 one-proposal selector, generalised to gamma by the
 * left-to-right rule of [SD]).  For j = 0..gamma-1: accept y_j iff
 * u_j < min(1, p_j[y_j] / q_j[y_j]) (evaluated exactly as u_j q_j[y_j] <
 * p_j[y_j]); the first rejection emits a
 * correction drawn from (p_j - q_j)+ / Σ(p_j - q_j)+ and ends the round; an
 * accepted y_j that equals eos, or that fills `remaining`, ends the round
 * with no further token; if all gamma are accepted a bonus is drawn from
 * p_gamma / Σ p_gamma.  A draw from weights w with uniform u' is the smallest
 * index whose running sum exceeds u' Σ w.
 *   p [R, gamma+1, V] f32 target rows; q [R, gamma, V] f32 draft rows;
 *   draft [R, gamma] int32.  Uniforms: Philox4x32-10 with key (seed lo, hi)
 *   and counter (j, r, offset lo, offset hi); word 0 -> accept uniform of
 *   position j, word 1 -> correction/bonus uniform (j = gamma for the bonus);
 *   u = (word >> 8) * 2^-24.
 *   eos [R] nullable (-1 = none); remaining [R] nullable (default gamma+1).
 *   Outputs [R] int32: accepted = number of drafts accepted, next_token =
 *   correction or bonus (-1 if the round ended without one), n_emit =
 *   accepted + (next_token >= 0), status = MTP_VERIFY_*.
 * Reads only p_j[y_j], q_j[y_j] up to the decision and the one row pair (or
 * bonus row) it samples from; those rows are checked for NaN/negatives. */
mtp_status spec_verify(int R, int gamma, int V, const float* p, const float* q,
                       const int32_t* draft, uint64_t seed, uint64_t offset,
                       const int32_t* eos, const int32_t* remaining,
                       int32_t* accepted, int32_t* next_token, int32_t* n_emit,
                       int32_t* status, cudaStream_t stream);

/* What shapes a request's distribution besides its logits; every pointer is a
 * nullable DEVICE pointer, 4-byte aligned.  Per request r (float [R]):
 *   temperature (default 1; 0 = greedy), repetition (default 1), frequency and
 *   presence (default 0).
 *   hist [R, hist_cap] int32: the request's tokens, of which the first
 *   hist_len[r] count (default hist_cap; clamped to [0, hist_cap]) and of those
 *   the first prompt_len[r] are the prompt (default 0).  Ids outside [0, V) are
 *   passed over.
 *   draft [R, L-1] int32: tokens that precede row (r, j): draft[r, 0..j-1].
 *   bias_ids [R, n_bias] int32, bias [R, n_bias] float: added to the logits of
 *   those ids (ids outside [0, V) are passed over; of entries with the same id
 *   the last one holds).
 *   mask [R, L, ceil(V/32)] uint32: bit v % 32 of word v / 32 allows token v.
 * hist_cap <= 262144, n_bias <= 4095. */
typedef struct mtp_logits_params {
  const float* temperature;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const int32_t* hist;
  const int32_t* hist_len;
  const int32_t* prompt_len;
  const int32_t* draft;
  const int32_t* bias_ids;
  const float* bias;
  const uint32_t* mask;
  int hist_cap;
  int n_bias;
} mtp_logits_params;

/* Logits to probability rows: the p (or q) that spec_verify takes, under each
 * request's sampling parameters and grammar.  Row (r, j), j = 0..L-1, is the
 * position after the request's tokens and draft[r, 0..j-1] (L = gamma + 1 for
 * verification).  With n(v) the occurrences of v among the generated tokens
 * (hist from prompt_len on, and the row's drafts), and seen(v) whether v occurs
 * among them or in the prompt:
 *   z(v) = seen(v) ? (x(v) > 0 ? x(v) / repetition : x(v) * repetition) : x(v)
 *   z(v) -= frequency * n(v) + presence * [n(v) > 0];  z(v) += bias(v)
 *   z(v) = -inf where the mask does not allow v
 *   p = softmax(z / temperature), or at temperature 0 the one-hot row of the
 *   lowest index of the maximum.
 * Masked logits may hold anything; an allowed -inf is a probability of 0.
 *   logits: R * L rows of V elements (dtype MTP_F32 or MTP_BF16), ld elements
 *   apart (V <= ld <= 2^33); p [R, L, V] float (p may be the logits' own buffer when
 *   dtype is MTP_F32 and ld == V, and must not overlap them otherwise);
 *   status [R, L] int32 nullable = MTP_LOGITS_*; a row that is not OK is zero,
 *   which spec_verify reports as MTP_VERIFY_ZERO_RESIDUAL where it draws from
 *   it.  prm nullable (a plain softmax).  V <= 524288, L <= 65536.
 * p is fp32: values below 2^-126 are 0.  A row is written once and read twice where
 * it is longer than its CTAs hold (4096 values each); no workspace. */
mtp_status mtp_logits_probs(int R, int L, int V, int dtype, const void* logits, long long ld,
                            const mtp_logits_params* prm, float* p, int32_t* status, cudaStream_t stream);

/* Gradient buffers of the training step (fp32, device, same shapes as the
 * corresponding weights; the step ADDS into them, so the caller zeroes them
 * or accumulates across calls).  Per-depth members are host arrays of D
 * device pointers.  NULL members are not computed. */
typedef struct mtp_grads {
  float* embed;     /* [V, d] */
  float* head;      /* [V, d] */
  float* out_norm;  /* [d] */
  float* h0;        /* [B, T, d]: gradient with respect to the main model's hidden states */
  float* const* hnorm;
  float* const* enorm;
  float* const* eh_proj;
  float* const* attn_norm;
  float* const* wq;
  float* const* wk;
  float* const* wv;
  float* const* wo;
  float* const* ffn_norm;
  float* const* w_gate;
  float* const* w_up;
  float* const* w_down;
} mtp_grads;

/* Bytes of device workspace mtp_chain_loss_grad needs (0 if unsupported). */
size_t mtp_chain_grad_workspace_bytes(const mtp_dims* dims);

/* Training step of the chain: mtp_chain_loss's forward (same arguments and
 * outputs, with optional per-depth weights as in mtp_loss_assemble_weighted)
 * followed by the gradients of the assembled loss, added into `grads`
 * ([M7.6] §0x05: the shared head receives the main term's and every depth's
 * gradient).  The head backward recomputes the logits per vocabulary chunk
 * (as [tokens, chunk] for dz = (softmax - onehot) dL/dl and as [chunk,
 * tokens] for dz^T) and never stores them whole.  The module backward then
 * runs depth D down to 1 on activations the forward saved: GEMMs for the
 * weight gradients (on transposed activations) and the input gradients (on
 * transposed weights), SwiGLU from recomputed gate/up pre-activations,
 * segment-causal attention (scores recomputed), RoPE, the norms, and the
 * prologue's two RMSNorms -- the state's into depth k-1, the embedding rows'
 * scattered into grads->embed.  Gradients flow through the bf16 rounding
 * points unchanged.  bf16 only. */
mtp_status mtp_chain_loss_grad(const mtp_dims* dims, const mtp_weights* w, const int32_t* tokens,
                               const int32_t* seg, const int32_t* pos, const void* h0, float lambda, int den,
                               int with_main, const float* depth_weights, double* sums_counts, float* losses,
                               const mtp_grads* grads, void* ws, size_t ws_bytes, cudaStream_t stream);

/* Bytes of device workspace mtp_draft_step needs (0 if the sizes are invalid). */
size_t mtp_draft_workspace_bytes(const mtp_dims* dims);

/* Decode-shaped MTP draft step: one proposal per request ([M7.6] §0x09: a
 * carried-frontier round proposes y from the saved parent hidden state and
 * E(f) and keeps q for verification; §0x09A: the MTP block attends over its
 * own K/V cache).  For request r:
 *   c = [RMSNorm_h(parent_hidden_r); RMSNorm_e(E[frontier_r])], u = M c,
 *   a = u + Attn(RMSNorm_a u) over cached rows [0, ctx_len_r) and the new row
 *   (RoPE at pos_r for its q and k; cached keys are used as stored),
 *   h = a + SwiGLU(RMSNorm_f a), q_r = softmax(W_U RMSNorm_out(h)),
 *   y_r = smallest v with Σ_{i<=v} q_r[i] > u Σ q_r, u = (word 2 >> 8) * 2^-24
 *   of Philox4x32-10 with key (seed lo, hi) and counter (0, r, offset lo, hi).
 * dims: B = R requests (<= 32), T = cache capacity, D = 1, dtype MTP_BF16,
 * d % 64 == 0, head_dim in {64, 128}, ffn % 8 == 0; weights as for the chain
 * (depth arrays of length 1).
 *   parent_hidden [R, d]; frontier [R] int32; pos [R] int32 in [0, T];
 *   kv_k, kv_v [R, T, d] bf16 cached keys/values; ctx_len [R] int32 in [0, T].
 *   q_out [R, V] float receives q; y_out [R] int32 the draws; h_out [R, d]
 *   nullable receives the pre-final-norm state of the new row.
 * Streams the block's weights, the head and the cache once: it is
 * HBM-bandwidth bound. */
mtp_status mtp_draft_step(const mtp_dims* dims, const mtp_weights* w, const void* parent_hidden,
                          const int32_t* frontier, const int32_t* pos, const void* kv_k,
                          const void* kv_v, const int32_t* ctx_len, uint64_t seed, uint64_t offset,
                          float* q_out, int32_t* y_out, void* h_out, void* ws, size_t ws_bytes,
                          cudaStream_t stream);

/* Bytes of device workspace mtp_draft_round needs for `gamma` steps (0 if the
 * sizes are invalid or gamma is outside [1, 31]). */
size_t mtp_draft_round_workspace_bytes(const mtp_dims* dims, int gamma);

/* gamma recurrent draft steps by reuse of one MTP module ([M7.6] §0x09: the
 * retained depth proposes the next token from its own output state).  Step s
 * (0-based) is mtp_draft_step's computation with
 *   parent = h of step s-1 (step 0: parent_hidden), frontier = y of step s-1
 *   (step 0: frontier), position pos_r + s, keys = the cached rows
 *   [0, ctx_len_r), the rows of steps 0..s-1 (their rotated keys and values,
 *   staged in the workspace) and the row itself,
 * and its draw uses word 2 of Philox4x32-10 at counter (s, r, offset lo, hi).
 * The staged rows are not written back to the cache.
 *   q_out [R, gamma, V] float: q of every step (the draft distributions that
 *   spec_verify takes); y_out [R, gamma] int32: the draws (spec_verify's
 *   draft tokens); h_out [R, gamma, d] bf16 nullable: every step's state.
 * gamma in [1, 31]; other arguments as for mtp_draft_step, whose call equals
 * this one with gamma = 1.  The block's weights, the head and the cache are
 * streamed once per step. */
mtp_status mtp_draft_round(const mtp_dims* dims, const mtp_weights* w, const void* parent_hidden,
                           const int32_t* frontier, const int32_t* pos, const void* kv_k, const void* kv_v,
                           const int32_t* ctx_len, int gamma, uint64_t seed, uint64_t offset, float* q_out,
                           int32_t* y_out, void* h_out, void* ws, size_t ws_bytes, cudaStream_t stream);

/* Sizes and layouts of mtp_prefix_attention: R requests with L new tokens each,
 * n_heads query heads of which n_heads / n_kv_heads consecutive ones share a
 * key head, head_dim 64 or 128, P rows of shared prefix (0: none), T rows of
 * capacity in each request's own cache (0: none).  scale 0 means
 * 1/sqrt(head_dim).  Strides count elements, must be multiples of 8, and are
 * those of dense tensors where 0: q [R, L, n_heads, head_dim], prefix_k and
 * prefix_v [P, n_kv_heads, head_dim], kv_k and kv_v [R, T, n_kv_heads, head_dim]
 * (head_dim is dense; any order of the others will do).
 * R <= 65535, n_heads / n_kv_heads <= 128, R * L * n_heads <= 2^24,
 * P + T <= 2^31 - 256. */
typedef struct mtp_prefix_dims {
  int R, L, n_heads, n_kv_heads, head_dim, P, T, causal;
  float scale;
  long long q_stride_r, q_stride_t, q_stride_h;
  long long prefix_stride_t, prefix_stride_h;
  long long kv_stride_r, kv_stride_t, kv_stride_h;
} mtp_prefix_dims;

/* Bytes of device workspace mtp_prefix_attention needs on the current device
 * (0 if the sizes are invalid). */
size_t mtp_prefix_attention_workspace_bytes(const mtp_prefix_dims* dims);

/* Attention of a batch whose requests share a prefix ([M7.6] §0x09A: the module
 * serves attention from its own K/V cache; here the rows of a common prompt are
 * kept, and read, once for the batch).  For request r, new token i and head h
 *   out = softmax(scale q [Kp; Kr]^T) [Vp; Vr]
 * over all P prefix rows and the rows j of the request's own cache with
 *   j < ctx_len[r] - (L - 1 - i)   if causal (the last L rows are the new
 *                                  tokens' own: each sees itself and what precedes it),
 *   j < ctx_len[r]                 otherwise.
 * Rows that a token does not see (from ctx_len[r] on; of later tokens) may hold
 * anything, padding and NaN among it.  Keys are used as stored.  A token that sees no row gets zeros (and lse = -inf).
 *   q, prefix_k, prefix_v, kv_k, kv_v: bf16, 16-byte aligned; ctx_len [R]
 *   int32, nullable (T), clamped to [0, T]; out [R, L, n_heads, head_dim] bf16;
 *   lse [R, L, n_heads] float, nullable: the natural logarithm of the softmax's
 *   denominator with the maximum put back in.
 *   ws: mtp_prefix_attention_workspace_bytes(dims) bytes, 16-byte aligned; calls
 *   that may overlap need workspaces of their own.
 * Scores, softmax statistics and outputs are fp32; the softmax weights enter
 * the product with the values as two bf16 parts (2^-15 of a weight). */
mtp_status mtp_prefix_attention(const mtp_prefix_dims* dims, const void* q, const void* prefix_k, const void* prefix_v,
                                const void* kv_k, const void* kv_v, const int32_t* ctx_len, void* out, float* lse,
                                void* ws, size_t ws_bytes, cudaStream_t stream);

/* Rotary positions.  Pair p of a head's first `rot` elements, p < rot / 2, is
 * elements (p, p + rot / 2), or (2p, 2p + 1) if interleaved; at position n it turns by
 * n * inv_freq[p]:
 *   (a, b) -> mscale * (a cos - b sin, b cos + a sin);
 * elements from rot on are left as they are.  inv_freq [rot / 2] double (device): any
 * scaling for long contexts is a choice of these numbers (mtp_rope_frequencies).  Angles
 * are taken modulo a turn in 64 bits, at any position. */
typedef struct mtp_rotation {
  const double* inv_freq; /* null: no rotation */
  int rot;                /* even, 2..head_dim */
  int interleaved;
  float mscale;
} mtp_rotation;

/* Frequencies of the rot / 2 pairs (HOST array out) and the factor on the rotated
 * values (nullable) for a base and a scaling of the positions:
 *   NONE    base^(-2p/rot);
 *   LINEAR  that / factor;
 *   YARN    pairs that turn less than beta_slow times within `original` positions
 *           / factor, those that turn more than beta_fast times as they are, linear in
 *           the pair's index between; mscale = 0.1 ln(factor) + 1.  The index that turns so
 *           many times, rot ln(original / (2 pi turns)) / (2 ln base), is rounded down for
 *           beta_fast and up for beta_slow, and kept within 0 and rot - 1;
 *   BANDS   pairs whose wavelength is above original / low / factor, those below
 *           original / high as they are, linear in original / wavelength between
 *           (beta_slow = low, beta_fast = high). */
typedef enum mtp_rope_scaling { MTP_ROPE_NONE = 0, MTP_ROPE_LINEAR = 1, MTP_ROPE_YARN = 2, MTP_ROPE_BANDS = 3 } mtp_rope_scaling;
mtp_status mtp_rope_frequencies(int rot, double base, int scaling, double factor, double original, double beta_slow,
                                double beta_fast, double* out, float* mscale);

/* Rows x [N, H, head_dim] at positions pos [N] turned into out (backward = 0), or
 * gradients of the turned rows into gradients of the rows (backward = 1: the angles
 * negated).  dtype MTP_F32 or MTP_BF16; head_dim even, up to 1024; strides count elements,
 * 0 are those of dense rows; out may be x itself (with the same strides) and must not
 * overlap it otherwise, nor may out's rows overlap one another.  pos may be negative.  Arithmetic in fp32. */
mtp_status mtp_rope(long long N, int H, int head_dim, int dtype, const mtp_rotation* rotation, const int32_t* pos,
                    int backward, const void* x, long long x_stride_n, long long x_stride_h, void* out,
                    long long out_stride_n, long long out_stride_h, cudaStream_t stream);

/* A cache of keys and values in pages.  k, v [n_pages, n_kv_heads, page, head_dim]:
 * the rows of one head lie together within a page.  Row j of request r is slot
 * j % page of page page_table[r, j / page].  page: 16, 32, .. 1024; head_dim 64 or 128.
 *   dtype MTP_BF16: bf16 rows; k_scale and v_scale are not read.
 *   dtype MTP_E4M3: codes as in mtp_fp8_matrix, and for every 16 rows of a page and
 *   head one power of two: k_scale, v_scale [n_pages, n_kv_heads, page / 16] bytes b,
 *   1..254 (others are taken as the nearest), for 2^(b - 127); a value is code * 2^(b - 127), exactly.  mtp_paged_attention
 *   takes v_scale within 27..227, as mtp_kv_append makes it of values up to 2^108.
 * page_table [R, table_len] int32.  Tensors are 16-byte aligned, the scales and the
 * table 4-byte aligned.  A page may stand in several requests' tables (a shared prompt).
 * n_pages * n_kv_heads <= 2^31 - 1; table_len * page <= 2^31 - 256. */
typedef struct mtp_paged_cache {
  void *k, *v;
  uint8_t *k_scale, *v_scale;
  const int32_t* page_table;
  int n_pages, page, table_len, n_kv_heads, head_dim, dtype;
} mtp_paged_cache;

/* A step's rows for a paged cache: k, v (and q) [R, L, heads, head_dim] bf16 with
 * strides in elements (0: those of dense tensors; multiples of 8, the last dimension
 * dense; k and v share theirs).  q and q_out are null, or the queries and where they go
 * turned, [R, L, n_heads, head_dim] dense (q_out may be a dense q; it must not lie within
 * what q, k and v span otherwise).
 *   ctx_len [R]: rows of request r once the step's are in; n_new [R] (nullable: L): how
 *   many those are, clamped to [0, L]: row i < n_new[r] goes to ctx_len[r] - n_new[r] + i.
 *   pos [R, L] (nullable: that index): positions for the rotation. */
typedef struct mtp_kv_rows {
  int R, L, n_heads;
  const void *k, *v, *q;
  void* q_out;
  long long kv_stride_r, kv_stride_t, kv_stride_h, q_stride_r, q_stride_t, q_stride_h;
  const int32_t *ctx_len, *n_new, *pos;
} mtp_kv_rows;

/* Appends the rows to the cache, keys turned on the way (rotation nullable: as they
 * are), and turns the queries.  Rotation in fp32, one rounding to the cache's type (q_out:
 * bf16).
 *   MTP_E4M3: per 16 rows of a page and head that get rows, with a = the largest finite
 *   magnitude among those of this call and 2^E the smallest power of two, E >= -90, with
 *   a <= 448 * 2^E: where the first of the 16 is a row of this call, the scale is 2^E;
 *   otherwise it is the larger of that and the one that was there, and where it grows the
 *   codes that were there are rounded again to the new scale.  code = RNE_e4m3(x / scale);
 *   what is not finite becomes NaN.  So a cache that is cut back (drafts that were turned
 *   down) is continued by the next call with the right ctx_len, with a scale at least the
 *   one that it had.
 * Rows past n_new are not read (their q is: q_out holds all L rows); slots that get no
 * row stay as they are.  Rows outside [0, table_len * page) and pages outside
 * [0, n_pages) are passed over and set MTP_DEVERR_PAGE_RANGE.  The 16-row blocks that a
 * call writes must stand once in the tables: where rows of two requests, or of two places
 * of one, are written to the same block, its contents are undefined. */
mtp_status mtp_kv_append(const mtp_paged_cache* cache, const mtp_kv_rows* rows, const mtp_rotation* rotation,
                         cudaStream_t stream);

/* The first T rows of every request as dense bf16 caches k_out, v_out [R, T, n_kv_heads,
 * head_dim], as mtp_prefix_attention and the draft step take them: rows from ctx_len[r] on
 * (and of pages outside [0, n_pages), which set MTP_DEVERR_PAGE_RANGE) are zero.  T <= table_len * page. */
mtp_status mtp_kv_gather(const mtp_paged_cache* cache, int R, int T, const int32_t* ctx_len, void* k_out, void* v_out,
                         cudaStream_t stream);

/* Sizes of mtp_paged_attention: R requests with up to L new tokens each, n_heads query
 * heads of which n_heads / n_kv_heads consecutive ones share a key head.  scale 0 means
 * 1/sqrt(head_dim).  Strides of q [R, L, n_heads, head_dim] count elements, must be
 * multiples of 8, and are those of a dense tensor where 0 (head_dim is dense).
 * R <= 65535, n_heads / n_kv_heads <= 128, R * L * n_heads <= 2^24. */
typedef struct mtp_paged_dims {
  int R, L, n_heads, causal;
  float scale;
  long long q_stride_r, q_stride_t, q_stride_h;
} mtp_paged_dims;

/* Bytes of device workspace mtp_paged_attention needs on the current device (0 if the
 * sizes are invalid, and where it needs none: short tables and few heads and requests; the
 * cache's pointers are not looked at). */
size_t mtp_paged_attention_workspace_bytes(const mtp_paged_dims* dims, const mtp_paged_cache* cache);

/* Attention of a batch's new tokens over a paged cache that already holds their rows
 * (mtp_kv_append): out = softmax(scale q K^T) V for token i < n_new[r] over the rows j of
 * request r with
 *   j < ctx_len[r] - (n_new[r] - 1 - i)  if causal (a token sees itself and what precedes it),
 *   j < ctx_len[r]                       otherwise.
 *   ctx_len [R] clamped to [0, table_len * page]; n_new [R] nullable (L), clamped to
 *   [0, L].  Tokens from n_new[r] on and tokens that see no row get zeros (lse = -inf).
 *   Rows that a token does not see may hold anything, NaN among it.  A value that is not
 *   finite, in a row that a token sees, makes its outputs of that dimension not finite.
 *   Pages outside [0, n_pages) set MTP_DEVERR_PAGE_RANGE and are not read; the outputs of
 *   requests that name them are of no use.  Pages behind ctx_len[r], and those of a request with
 *   n_new[r] = 0, are not looked up.
 *   q bf16, 16-byte aligned; out [R, L, n_heads, head_dim] bf16, apart from q; lse [R, L, n_heads]
 *   float, nullable: natural logarithm of the softmax's denominator, maximum included.
 *   ws: mtp_paged_attention_workspace_bytes bytes (null if 0), 16-byte aligned; calls that may
 *   overlap need workspaces of their own.
 * Scores, statistics, sums and outputs are fp32.  MTP_E4M3: the cache's codes enter the
 * products as they are; q is two codes and a power of two per row (exact above 2^-9 of
 * the row's largest element, off by 2^-17 of it below); a softmax weight is rounded to
 * fp16 (2^-11) and is three codes, off by 2^-26 of the largest p 2^E among
 * the keys that a part of the kernel takes one after another, at the most: weights below that leave the outputs (not
 * the sums), n of them less than n 2^-26 of the largest.  MTP_BF16, and both where no workspace is needed or L * n_heads / n_kv_heads is 64 or more (and a copy
 * of the rows as bf16 in the workspace at most 4 GB): q, keys and values as they are, a softmax
 * weight as two bf16 parts (2^-15).  Which kernel a call takes follows from the sizes alone, table_len
 * among them, not from the lengths: a call repeated gives the same bits, one with a wider table may differ within these bounds. */
mtp_status mtp_paged_attention(const mtp_paged_dims* dims, const mtp_paged_cache* cache, const void* q,
                               const int32_t* ctx_len, const int32_t* n_new, void* out, float* lse, void* ws,
                               size_t ws_bytes, cudaStream_t stream);

/* One FP8 block-scaled weight matrix W [n, K] ([M7.6] §0x03C: released
 * weights are FP8 with block scales; the runtime chooses the compute
 * representation).  q: e4m3 codes (OCP FP8 E4M3: sign, 4 exponent bits with
 * bias 7, 3 mantissa bits, subnormals, no infinities, 0x7F/0xFF = NaN),
 * row-major with row stride K bytes, 16-byte aligned; scale: fp32
 * [ceil(n/128), ceil(K/128)] row-major, one factor per 128 x 128 block.
 * The represented weight is W[m][k] = e4m3(q[m][k]) * scale[m/128][k/128],
 * used exactly.  The activations meet it on the tensor cores as e4m3 in two
 * terms: per token and 128-wide k-tile, x~ = 2^E (hi + lo) with 2^E the
 * smallest power of two such that max|x| <= 448 * 2^E, hi = RNE_e4m3(x/2^E),
 * lo = RNE_e4m3(x/2^E - hi); x~ = x for every element of magnitude >=
 * 2^(E-2) and |x~ - x| <= 2^(E-10) otherwise.  Products are summed in fp32,
 * one fp32 partial per 128-wide k-block scaled by its block factors. */
typedef struct mtp_fp8_matrix {
  const void* q;
  const float* scale;
} mtp_fp8_matrix;

/* The linear maps of one MTP module in FP8 (shapes as in mtp_weights:
 * eh_proj [d, 2d], wq/wk/wv/wo [d, d], w_gate/w_up [ffn, d], w_down [d, ffn]). */
typedef struct mtp_block_fp8 {
  mtp_fp8_matrix eh_proj, wq, wk, wv, wo, w_gate, w_up, w_down;
} mtp_block_fp8;

/* mtp_draft_round with the module's linear maps in FP8 block-scaled form
 * ([M7.6] §0x03C; it halves the decode step's weight bytes).
 * w supplies the bf16 embedding, head and norm gains (its linear-map fields
 * are not read and may be null: the output head and norms stay in bf16, as
 * the pages keep them in higher precision); f8 the eight linear maps.
 * Requires ffn % 16 == 0.  Everything else, including the outputs and the
 * random stream, is as for mtp_draft_round. */
mtp_status mtp_draft_round_fp8(const mtp_dims* dims, const mtp_weights* w, const mtp_block_fp8* f8,
                               const void* parent_hidden, const int32_t* frontier, const int32_t* pos,
                               const void* kv_k, const void* kv_v, const int32_t* ctx_len, int gamma,
                               uint64_t seed, uint64_t offset, float* q_out, int32_t* y_out, void* h_out,
                               void* ws, size_t ws_bytes, cudaStream_t stream);

/* One 4-bit weight matrix W [n, K] with group scales:
 *   W[m][k] = (code[m][k] - zero[m][k/group]) * scale[m][k/group], taken exactly.
 * q: [n, K/2] bytes, row-major, 16-byte aligned; byte j of a row holds code 2j
 * in its low and code 2j+1 in its high half, 0..15.  scale: bf16
 * [n, ceil(K/group)] row-major (the last group of a row may be short).  zero:
 * bytes of the same shape, of which the low four bits count, or null: 8
 * everywhere (symmetric codes). */
typedef struct mtp_int4_matrix {
  const void* q;
  const void* scale;
  const void* zero;
} mtp_int4_matrix;

/* The linear maps of one MTP module in 4 bits (shapes as in mtp_weights), all
 * with the same group size: 32, 64 or 128. */
typedef struct mtp_block_int4 {
  mtp_int4_matrix eh_proj, wq, wk, wv, wo, w_gate, w_up, w_down;
  int group;
} mtp_block_int4;

/* What a draft round may have besides mtp_draft_round's arguments; zero
 * members leave it as it is.
 *   fp8, int4 (at most one): the module's linear maps in that form; w's are not
 *   read then and may be null.  int4 requires ffn % 32 == 0.
 *   prefix_k, prefix_v [prefix_len, d] bf16, 16-byte aligned: keys and values, as
 *   the cache holds them, of rows that precede every request's own cache (a
 *   prompt that the batch shares).  They are kept and read once for the batch;
 *   the result is that of caches which begin with these rows, to 2^-15 of the
 *   prefix's softmax weights.  pos may reach T + prefix_len, which is at
 *   most 2^31 - 256. */
typedef struct mtp_draft_ext {
  const mtp_block_fp8* fp8;
  const mtp_block_int4* int4;
  const void* prefix_k;
  const void* prefix_v;
  int prefix_len;
} mtp_draft_ext;

/* Bytes of device workspace mtp_draft_round_ext needs on the current device (0
 * if the sizes are invalid). */
size_t mtp_draft_round_ext_workspace_bytes(const mtp_dims* dims, int gamma, int prefix_len);

/* mtp_draft_round with `ext` (nullable).  Everything else, including the
 * outputs and the random stream, is as for mtp_draft_round. */
mtp_status mtp_draft_round_ext(const mtp_dims* dims, const mtp_weights* w, const mtp_draft_ext* ext,
                               const void* parent_hidden, const int32_t* frontier, const int32_t* pos,
                               const void* kv_k, const void* kv_v, const int32_t* ctx_len, int gamma,
                               uint64_t seed, uint64_t offset, float* q_out, int32_t* y_out, void* h_out,
                               void* ws, size_t ws_bytes, cudaStream_t stream);

/* Bytes of device workspace mtp_draft_round_paged needs on the current device (0 if the
 * sizes are invalid; the cache's pointers are not looked at). */
size_t mtp_draft_round_paged_workspace_bytes(const mtp_dims* dims, int gamma, int prefix_len, const mtp_paged_cache* cache);

/* mtp_draft_round_ext over a paged cache of the module's keys and values (bf16 or 8 bits)
 * in the place of kv_k and kv_v: n_kv_heads = n_heads, head_dim the module's, and
 * dims->T = table_len * page.  Request r attends to its first ctx_len[r] rows there
 * (mtp_paged_attention's precision), the round's own rows and the prefix, if any.
 * The step turns its own q and k as the chain does: whole heads in halves, frequencies
 * rope_base^(-2p/head_dim), factor 1 (rope_base = 0: not at all).  The cache's keys must have been
 * turned in that way (mtp_rope_frequencies NONE with rot = head_dim, not interleaved): with keys
 * that were turned by scaled frequencies, as neighbours or in part the scores are wrong, and nothing
 * reports it.
 *   rows_k, rows_v [R, gamma, d] bf16, nullable (both or none), 16-byte aligned: receive the
 *   round's rotated keys and values; those of the drafts that verification keeps go into the
 *   cache by mtp_kv_append without a rotation (n_new: how many). */
mtp_status mtp_draft_round_paged(const mtp_dims* dims, const mtp_weights* w, const mtp_draft_ext* ext,
                                 const mtp_paged_cache* cache, const void* parent_hidden, const int32_t* frontier,
                                 const int32_t* pos, const int32_t* ctx_len, int gamma, uint64_t seed, uint64_t offset,
                                 float* q_out, int32_t* y_out, void* h_out, void* rows_k, void* rows_v, void* ws,
                                 size_t ws_bytes, cudaStream_t stream);

/* Bytes of device workspace mtp_gemm_fp8w needs for reduction length K. */
size_t mtp_gemm_fp8w_workspace_bytes(int K);

/* Diagnostic FP8 weight GEMM (the kernel the FP8 draft step uses):
 * out[R, N] (fp32, row stride N) += x~[R, K] · W^T with W the FP8
 * block-scaled matrix (wq [N, K] e4m3, scale [ceil(N/128), ceil(K/128)]) and
 * x~ the two-term e4m3 form of x (bf16) described at mtp_fp8_matrix.
 * R in [1, 32], K % 16 == 0, x and wq 16-byte aligned; ws: at least
 * mtp_gemm_fp8w_workspace_bytes(K) bytes of device memory, 16-byte aligned. */
mtp_status mtp_gemm_fp8w(int R, int N, int K, const void* x, const void* wq, const float* scale, float* out,
                         void* ws, size_t ws_bytes, cudaStream_t stream);

/* Product of 1..32 tokens with a 4-bit weight matrix (the kernel the draft
 * step uses with 4-bit weights): out[R, N] (fp32, row stride N) = x[R, K] · W^T,
 * added to what out holds if `accumulate`.  x bf16; group 32, 64 or 128;
 * K % 32 == 0; N, K <= 2^30; x and w->q 16-byte aligned.  Products are exact in fp32, sums
 * and scales fp32, in an order fixed by the sizes: the result is the same every
 * time.  No workspace. */
mtp_status mtp_gemm_int4w(int R, int N, int K, int group, const void* x, const mtp_int4_matrix* w, float* out,
                          int accumulate, cudaStream_t stream);

/* Diagnostic GEMM on the same tcgen05 core the chain uses:
 * C[M,N] (bf16) = A[M,K] (bf16) · B[N,K]^T (bf16), fp32 accumulation.
 * K % 8 == 0; A, B, C 16-byte aligned. */
mtp_status mtp_gemm_bf16(int M, int N, int K, const void* A, const void* B, void* C,
                         cudaStream_t stream);

/* Diagnostic bf16 decode-shaped GEMM (the draft step's linear maps):
 * out[R, N] (fp32, row stride N) += x[R, K] · W^T with x bf16 [R, K] (R in
 * [1, 32]) and W bf16 [N, K]; K % 8 == 0, x and W 16-byte aligned. */
mtp_status mtp_gemm_decode_bf16(int R, int N, int K, const void* x, const void* w, float* out,
                                cudaStream_t stream);

/* Diagnostic fp32-accumulating GEMM on the same core (the training step's
 * gradient GEMMs): out[M,N] (fp32, row stride ldo) += A · B^T, bf16 operands.
 * a_mn = 0: A is row-major [M, K] (row stride lda); a_mn = 1: A is stored as
 * [K, M] (row stride lda), i.e. the product reads the transpose of a
 * row-major [K, M] matrix.  b_mn likewise for B ([N, K] or [K, N]).  K is
 * split into `splits` ranges (1..ceil(K/64)) whose partial tiles are added
 * with fp32 atomics.  Leading dimensions % 8 == 0; pointers 16-byte aligned. */
mtp_status mtp_gemm_f32acc(int M, int N, int K, const void* A, int lda, int a_mn, const void* B, int ldb, int b_mn,
                           float* out, int ldo, int splits, cudaStream_t stream);

/* Failure-path diagnostic of spec_verify's bounded waits (the method has no
 * counterpart; it exercises the failure detection every pipeline wait of
 * this library relies on).  Runs spec_verify's bulk-copy kernel with the same
 * arguments (no EOS, no budget) except that its producer issues no copy, so
 * each request that reaches the row sweep (a rejection or a bonus draw)
 * waits on a ring stage nothing will fill; that wait gives up after
 * `wait_limit_cycles` SM clock cycles (1 .. the library's limit of 3e9,
 * ~1.5 s) with no copy in flight.  Such requests end with status
 * MTP_VERIFY_DEVICE_TIMEOUT, accepted = the accept prefix, next_token = -1,
 * and the device error word gets MTP_DEVERR_TIMEOUT | MTP_DEVERR_FROM_VERIFY
 * (read and cleared by mtp_check_errors); requests that end in the accept
 * phase (invalid draft) report as spec_verify would.  The kernel returns
 * normally and the stream stays usable.  Requires V % 4 == 0 and 16-byte
 * aligned p and q (else MTP_ERR_UNSUPPORTED); other argument errors as
 * spec_verify, plus MTP_ERR_INVALID_ARG for a limit out of range. */
mtp_status mtp_diag_verify_starved(int R, int gamma, int V, const float* p, const float* q,
                                   const int32_t* draft, uint64_t seed, uint64_t offset,
                                   int32_t* accepted, int32_t* next_token, int32_t* n_emit,
                                   int32_t* status, long long wait_limit_cycles, cudaStream_t stream);

/* Kernel classes for mtp_profile_kernel. */
enum {
  MTP_KC_HEAD_CE_GEMM = 0,  /* shared head GEMM with the online max/sum-exp epilogue */
  MTP_KC_GATE_UP_GEMM = 1,  /* gate/up GEMM with the SwiGLU epilogue                 */
  MTP_KC_DOWN_GEMM = 2,     /* down-projection GEMM with the residual epilogue      */
  MTP_KC_QKV_GEMM = 3,      /* QKV GEMM with the RoPE epilogue                      */
  MTP_KC_O_GEMM = 4,        /* attention output GEMM with the residual epilogue     */
  MTP_KC_PROJ_GEMM = 5,     /* eh_proj fusion GEMM                                  */
  MTP_KC_ATTENTION = 6,     /* segment-causal attention                             */
  MTP_KC_SPEC_VERIFY = 7,   /* spec_verify                                          */
  MTP_KC_PROLOGUE = 8,      /* embedding gather + dual RMSNorm + concat of a depth  */
  MTP_KC_COUNT = 9
};

/* Measurement hook (not thread-safe; for benchmarks).  Each kernel class
 * has its own slot.  While a slot is armed, every launch of that class issued
 * by this library records events[2*i] on its stream just before and
 * events[2*i+1] just after the launch, i = 0, 1, ... up to n_pairs;
 * *recorded (host) counts the pairs used.  Events are created by the caller
 * (timing enabled).  A null `events` disarms the slot.  Returns
 * MTP_ERR_INVALID_ARG on a bad class. */
mtp_status mtp_profile_kernel(int kernel_class, cudaEvent_t* events, int n_pairs, int* recorded);

/* Number of kernel launches this library has issued since it was loaded
 * (host-side counter). */
unsigned long long mtp_kernel_launches(void);

/* Synchronises `stream`, ORs the device error words of every kernel file
 * into *flags (host, nullable) and clears them.  Returns MTP_ERR_DEVICE if
 * any bit was set, MTP_ERR_CUDA if the synchronisation failed. */
mtp_status mtp_check_errors(cudaStream_t stream, unsigned int* flags);

/* Static string for a status code. */
const char* mtp_status_string(int status);

/* MTP_ABI_VERSION of the loaded library. */
int mtp_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MTP_H */
