/*
 * libgdn.h -- C ABI of the MI355X (gfx950) gated delta rule library.
 *
 * The method (statement of "Gated DeltaNet State Update", first display):
 *     S_t = gamma_t (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T
 *     y_t = scale * q_t^T S_t            (read out after the update)
 * taken independently per value head; value head h reads query/key head
 * h * hq / hv ("com.microsoft.GatedDeltaNet", Description).
 *
 * Conventions shared by every call
 *  - All data pointers are DEVICE pointers (hipMalloc / torch CUDA memory) and
 *    are owned by the caller.  The library never allocates, frees or keeps a
 *    pointer after a call returns.  Inputs are never written.
 *  - `stream` is a hipStream_t passed as void* (NULL = the null stream).  Work
 *    is enqueued asynchronously; calls read no device memory on the host and
 *    never synchronise, so every call is hipGraph-capturable.
 *  - Recurrent states are fp32 and V-major: one head's state is a [dv][dk]
 *    array, row j holding value index j across all dk keys (the ONNX card's
 *    (batch, Hv, Dv, Dk) state; the FlashInfer pool's "K-last" layout).
 *  - Argument errors visible on the host (NULL required pointer, bad sizes,
 *    unsupported head sizes, misalignment, forbidden combinations) return a
 *    status other than GDN_OK before anything is enqueued; gdn_last_error()
 *    then returns a description (thread-local, valid until the next call on
 *    that thread).  Data-dependent conditions are never errors: out-of-range
 *    cu_seqlens become empty requests, out-of-range or negative slots mean
 *    "skip" (see each call).
 *  - Supported head sizes: dk and dv in {16, 32, 64, 128}.
 *  - Calls that overlap on one device race only where they write the same
 *    memory; two rows of one decode call that name the same pool slot (for
 *    reading by one and writing by another) are undefined behaviour.
 */
#ifndef LIBGDN_H
#define LIBGDN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  GDN_OK = 0,
  GDN_ERR_NULL = 1,        /* a required pointer is NULL                          */
  GDN_ERR_SHAPE = 2,       /* a size is <= 0, inconsistent, or hv % hq != 0        */
  GDN_ERR_DTYPE = 3,       /* unknown dtype or decay kind                          */
  GDN_ERR_LAYOUT = 4,      /* misaligned pointer / stride, or a partial overlap    */
  GDN_ERR_UNSUPPORTED = 5, /* valid request the library does not implement           */
  GDN_ERR_HIP = 6          /* a HIP launch failed; gdn_last_error() has the text   */
} gdn_status;

/* GDN_E4M3 (OCP 8-bit float, largest value 448) and GDN_I8 (whole numbers of
 * -127 to 127) are types of key-value caches only. */
typedef enum { GDN_F32 = 0, GDN_BF16 = 1, GDN_E4M3 = 2, GDN_I8 = 3 } gdn_dtype;

/* update_rule of "com.microsoft.GatedDeltaNet" (Attributes): which terms of
 *   S_t = exp(g_t) S_{t-1} + k_t (beta_t (v_t - exp(g_t) S_{t-1}^T k_t))^T
 * survive.  Rules without the decay use g = 0, rules without beta use 1 in
 * the write, and linear / gated drop the retrieval S^T k. */
typedef enum {
  GDN_RULE_GATED_DELTA = 0, /* decay and delta retrieval (the default)         */
  GDN_RULE_GATED = 1,       /* decay only:     S = exp(g) S + k v^T            */
  GDN_RULE_DELTA = 2,       /* retrieval only: S = S + k (beta (v - S^T k))^T  */
  GDN_RULE_LINEAR = 3       /* neither:        S = S + k v^T                   */
} gdn_update_rule;

/* Meaning of the prefill decay input. */
typedef enum {
  GDN_DECAY_LOG = 0,   /* log-space decay g, gamma = exp(g); -inf means gamma = 0 */
  GDN_DECAY_GAMMA = 1  /* gamma itself, in [0, 1]                                 */
} gdn_decay_kind;

/* Text describing the last non-OK status returned on the calling thread. */
const char* gdn_last_error(void);

/* Library version as "major.minor.patch". */
const char* gdn_version(void);

/* Digest of this header, comments aside, as the library was built from it:
 * argument structs grow between versions, and a program whose own build took
 * another header must not call the library. */
const char* gdn_header_digest(void);

/* gdn_wait_timeouts -- health check of the in-kernel waits.
 *
 * The bf16 pair prefill kernel (and the scan's passes, which run it) hands
 * each chunk from its preparing waves to its state waves through counters
 * in workgroup memory; every wait on such a counter is bounded (2^22 polls,
 * far beyond any working schedule).  A wait that runs out adds 1 to a
 * per-device word and the kernel finishes normally, with results that are
 * then not to be trusted.  This call stores the current device's word in
 * *count (0 in every correct run) and sets it back to 0 when clear != 0.
 * Synchronous: it waits for all work on the current device.  Returns
 * GDN_ERR_NULL for a NULL count, GDN_ERR_HIP when the copy fails.
 */
gdn_status gdn_wait_timeouts(uint32_t* count, int32_t clear);

/* ----------------------------------------------------------------------------
 * gdn_gate -- fused gates, elementwise over n_tokens rows of hv heads.
 *
 * Follows the "qwen" gate_activation of "com.microsoft.GatedDeltaNet"
 * (Attributes) and the fused gate of "flashinfer.cake_gdp.
 * cake_gated_delta_product_mtp" (description; softplus threshold 20):
 *     log_decay[i,h] = -exp(A_log[h]) * softplus(a[i,h] + dt_bias[h])
 *     gamma[i,h]     = exp(log_decay[i,h])
 *     beta[i,h]      = sigmoid(b[i,h])
 * with softplus(x) = x for x > 20, log1p(exp(x)) otherwise.  Arithmetic fp32.
 *
 *   A_log, dt_bias   [hv] fp32                     (required when a != NULL)
 *   a, b             [n_tokens, hv] dense, ab_dtype; either may be NULL
 *   log_decay_out, gamma_out   [n_tokens, hv] fp32, nullable; need a
 *   beta_out                   [n_tokens, hv] fp32, nullable; needs b
 * n_tokens == 0 is a no-op.  An output requested without its input is
 * GDN_ERR_NULL.
 * ------------------------------------------------------------------------- */
gdn_status gdn_gate(const float* A_log, const float* dt_bias,
                    const void* a, const void* b, int32_t ab_dtype,
                    int64_t n_tokens, int32_t hv,
                    float* log_decay_out, float* gamma_out, float* beta_out,
                    void* stream);

/* ----------------------------------------------------------------------------
 * gdn_prefill -- chunked prefill over packed or ragged requests.
 *
 * Contract of "com.microsoft.GatedDeltaNet" (Inputs, Outputs, Attributes) with
 * the update_rule the update_rule field names (gated_delta when zero), the
 * gates either as given (gate_activation and beta_activation none: they come
 * from gdn_gate or the caller) or fused (gate_activation qwen and
 * beta_activation sigmoid, from the gate_a / gate_b fields), and qk_l2_norm
 * as the qk_l2norm field says (off: keys arrive normalised, as "Gated DeltaNet
 * State Update" Constraints require):
 *  - request r covers tokens [cu_seqlens[r], cu_seqlens[r+1]), both offsets
 *    clamped to [0, total_tokens]; a decreasing pair is an empty request.
 *    cu_seqlens == NULL means uniform packing, request r = [r*seq_len,
 *    (r+1)*seq_len), and then n_seqs * seq_len must equal total_tokens.
 *  - the state of (request r, value head h) starts from initial_state[r,h]
 *    (zeros when initial_state == NULL) and ends in final_state[r,h]; an
 *    empty request copies its incoming state.
 *  - out[t,h,:] = scale * S_t^T q[t, h*hq/hv] for every token t of a request;
 *    rows of tokens no request covers are not written.
 *  - chunk_size is a scheduling hint (0 = 64; accepted 16, 32, 64): it never
 *    changes which result is computed, only the rounding order.
 *
 * Layouts (strides in elements; the last dimension is always dense):
 *   q, k   [total_tokens, hq, dk] io_dtype, strides {token, head}
 *   v      [total_tokens, hv, dv] io_dtype, strides {token, head}
 *   out    [total_tokens, hv, dv] io_dtype, strides {token, head}
 *   decay  [total_tokens, hv] fp32 dense  (decay_kind says log or gamma)
 *   beta   [total_tokens, hv] fp32 dense  (already activated)
 *   cu_seqlens   [n_seqs + 1] int32, or NULL
 *   initial_state, final_state  [n_seqs, hv, dv, dk] fp32 dense, V-major;
 *                final_state may be the same buffer as initial_state (each
 *                state slice is read completely before it is written) but
 *                must not partially overlap it.
 * Gate inputs per update_rule, as the card has them "present exactly" for the
 * rules that use them: the decay source (decay, or gate_a with A_log and
 * dt_bias) is required for gated_delta and gated and must be absent for delta
 * and linear; the beta source (beta, or gate_b) is required for gated_delta
 * and delta and must be absent for gated and linear.  Each source is given
 * or fused on its own, as the card's gate_activation and beta_activation are
 * separate attributes: a fused decay with a given beta, or a given decay with
 * a fused beta, is accepted (it runs on the general kernel, which picks the
 * form per input).
 * Requirements: pointers 16-byte aligned; head and token strides multiples of
 * 8 elements and below 2^23 (in-chunk offsets are 32-bit); total_tokens * hv below 2^31; io_dtype in
 * {GDN_F32, GDN_BF16}.  total_tokens == 0 still writes final_state (copies /
 * zeros).  n_seqs == 0 is a no-op.
 * ------------------------------------------------------------------------- */
typedef struct {
  int32_t n_seqs;
  int32_t seq_len;         /* used iff cu_seqlens == NULL                     */
  int64_t total_tokens;
  int32_t hq, hv, dk, dv;
  int32_t io_dtype;        /* gdn_dtype of q, k, v and out                     */
  int32_t decay_kind;      /* gdn_decay_kind                                   */
  int32_t chunk_size;      /* 0 = default 64                                   */
  float scale;             /* applied as given                                 */
  const void* q;  int64_t q_stride_token, q_stride_head;
  const void* k;  int64_t k_stride_token, k_stride_head;
  const void* v;  int64_t v_stride_token, v_stride_head;
  void* out;      int64_t out_stride_token, out_stride_head;
  const float* decay;
  const float* beta;
  const int32_t* cu_seqlens;
  const float* initial_state;
  float* final_state;
  /* Optional, zero = off (appended; a zero-filled struct keeps the behaviour
   * above).  qk_l2_norm of the ONNX card: with qk_l2norm != 0 every q and k
   * head vector x is used as x / sqrt(sum(x^2) + qk_l2norm_eps) (the card's
   * epsilon is 1e-12); the inputs are not modified. */
  int32_t qk_l2norm;
  float qk_l2norm_eps;     /* >= 0 and finite                                  */
  /* Fused gate: the gates are computed in the kernel as gdn_gate computes
   * them -- log-decay -exp(A_log[h]) softplus(a + dt_bias[h]) (threshold 20)
   * from gate_a, beta = sigmoid(b) from gate_b; decay and beta must then be
   * NULL and decay_kind is ignored.  A_log, dt_bias [hv] fp32 (with gate_a);
   * gate_a, gate_b [total_tokens, hv] io_dtype, dense. */
  const float* A_log;
  const float* dt_bias;
  const void* gate_a;
  const void* gate_b;
  int32_t update_rule;     /* gdn_update_rule; 0 = gated_delta                 */
  /* State pool (optional; appended).  With state_pool != NULL the states live
   * in a slot-indexed pool laid out as gdn_decode's pool (slot s, head h at
   * state_pool + s*pool_slot_stride + h*pool_head_stride, a dense [dv][dk]
   * fp32 block), and initial_state and final_state must be NULL.  Request r
   * starts from slot read_slot[r] (zeros when read_slot is NULL or the entry
   * is < 0 or >= pool_size) and its final state is stored to slot
   * write_slot[r] (read_slot[r] when write_slot is NULL; nothing when the
   * entry is < 0 or >= pool_size).  A request may read and write one slot; a
   * slot that one request writes and another reads or writes is undefined
   * behaviour.  Same alignment and stride rules as gdn_decode's pool.  With
   * the fused gate and one request per batch row this is a multi-token
   * (chunked) decode over the decode's pool. */
  float* state_pool;
  int32_t pool_size;
  int64_t pool_slot_stride, pool_head_stride;
  const int32_t* read_slot;  /* [n_seqs] or NULL                             */
  const int32_t* write_slot; /* [n_seqs] or NULL                             */
  /* Caller-provided device scratch (appended), 256-byte aligned.  With
   * workspace_bytes >= gdn_prefill_workspace_size(args) > 0 the call runs as
   * a scan over the affine maps of request segments (three launches; see
   * gdn_prefill_workspace_size); otherwise, and whenever that size is 0, the
   * workspace is ignored and every (request, head) is one serial walk over
   * its chunks (for many short bf16 requests one workgroup walks a run of
   * consecutive requests, each from its own initial state).  All compute the
   * same result up to rounding order.  The
   * library neither allocates nor keeps the workspace; calls that share one
   * workspace on overlapping streams race. */
  void* workspace;
  size_t workspace_bytes;
  /* Per-key decay (appended): with decay_per_key != 0, decay is
   * [total_tokens, hv, dk] fp32 dense, one decay per key dimension (the ONNX
   * card's per-key-dimension spelling, in decay_kind's meaning), read in the
   * card's recurrence: each token first scales key column i of the V-major
   * state by its own factor.  Needs a given decay (not gate_a), a given
   * beta or a fused one (gate_b), and an update_rule with a decay (gated_delta or gated; others
   * return GDN_ERR_SHAPE); runs a separate 16-token-chunk MFMA kernel,
   * slower than the scalar-decay kernels. */
  int32_t decay_per_key;
} gdn_prefill_args;

/* Device scratch bytes a gdn_prefill call with these arguments can use; 0
 * when it needs none (args may be NULL: 0).
 *
 * Over any run of tokens the recurrence maps the state entering the run to
 * the state leaving it by an affine map S_out = P S_in + R ("Gated DeltaNet
 * State Update", statement: every step is affine in S), and the chunk is a
 * scheduling choice ("com.microsoft.GatedDeltaNet", Attributes, chunk_size).
 * A call with few (request, value head) units and long requests -- bf16,
 * dk and dv in {64, 128}, the default chunk, scalar decay, gates not mixed,
 * and a serial walk that would fill at most 64 workgroups -- is cut into
 * nseg segments per request (nseg between 4 and 64, chosen from the sizes
 * alone: about 512 workgroups in the first launch, segments of 16 chunks or
 * more on average).  The size is
 *     n_seqs * nseg * hv * dk * (2 dv + dk) * 4 bytes
 * (each segment's map, then each segment's incoming state), at most about
 * 25 MiB for such calls.  Sizes only decide it: the same arguments give the
 * same size on every device. */
size_t gdn_prefill_workspace_size(const gdn_prefill_args* args);

gdn_status gdn_prefill(const gdn_prefill_args* args, void* stream);

/* ----------------------------------------------------------------------------
 * gdn_prefill_noalloc -- gdn_prefill for callers that cannot allocate device
 * memory: code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc.
 *
 * Runs exactly what gdn_prefill runs with a workspace of
 * gdn_prefill_workspace_size(args) bytes, taking that workspace from a static
 * device array of GDN_NOALLOC_SCRATCH_BYTES (32 MiB) that the library holds on
 * every device it runs on until the process ends; args->workspace and
 * args->workspace_bytes are ignored.  It allocates and frees nothing.  A call
 * whose workspace size exceeds the array returns GDN_ERR_UNSUPPORTED (the
 * segment choice keeps every call within about 25 MiB).  Argument errors and
 * results are those of gdn_prefill.
 * Every call on one device shares that device's array, which keeps the last
 * call's contents: calls that overlap on one device (other streams, other
 * threads) race and must be serialised by the caller.  The array needs no
 * clearing -- each call writes every scratch byte it reads.
 * ------------------------------------------------------------------------- */
#define GDN_NOALLOC_SCRATCH_BYTES (32u << 20)
gdn_status gdn_prefill_noalloc(const gdn_prefill_args* args, void* stream);

/* ----------------------------------------------------------------------------
 * gdn_decode -- one fused launch over a slot-indexed fp32 state pool.
 *
 * Contract of "flashinfer.cake_gdp.cake_gated_delta_product_mtp" (parameters
 * and notes), generalised to grouped value heads (hv a multiple of hq) and to
 * dk, dv in {16, 32, 64, 128}; q/k arrive normalised unless qk_l2norm asks
 * for the in-kernel L2 norm (use_qk_l2norm).
 * For every batch row b and value head h:
 *  - rd = read_idx[b]; rd < 0 or rd >= pool_size skips the row entirely: no
 *    pool read, no output store, no write-back, no scatter.
 *  - S = pool[rd, h].  For each token t: gamma_t from the fused gate (as in
 *    gdn_gate, on a[b,t,h]); S <- gamma_t S; then for each sub-step
 *    j < n_householder: beta = sigmoid(b[b,t,j,h]) and
 *    S <- (I - beta k k^T) S + beta k v^T with k = k[b,t,j,h*hq/hv],
 *    v = v[b,t,j,h]; then out[b,t,h] = scale * S^T q[b,t,h*hq/hv].
 *  - scatter_idx != NULL: after every token, S is stored to
 *    pool[scatter_idx[b,t], h] unless that entry is < 0 or >= pool_size; no
 *    end-of-row write-back happens.  Requires disable_state_update == 0.
 *  - otherwise, unless disable_state_update != 0: after the last token S is
 *    stored to pool[wr, h] with wr = write_idx ? write_idx[b] : rd, unless
 *    wr < 0 or wr >= pool_size (the output is still stored).
 *
 * Layouts (dense, row-major):
 *   q [batch, T, hq, dk]; k [batch, T, n_householder, hq, dk];
 *   v [batch, T, n_householder, hv, dv]; a [batch, T, hv];
 *   b [batch, T, n_householder, hv]  -- all io_dtype
 *   A_log, dt_bias [hv] fp32
 *   pool: slot s, head h starts at pool + s*pool_slot_stride +
 *         h*pool_head_stride and holds a dense [dv][dk] fp32 array
 *         (padding between heads or slots is allowed)
 *   read_idx [batch] int32; write_idx [batch] int32 or NULL;
 *   scatter_idx [batch, T] int32 or NULL
 *   out [batch, T, hv, dv] io_dtype; rows of skipped batch rows keep their
 *       previous contents
 * Requirements: pool pointer 16-byte aligned and both pool strides multiples
 * of 4 elements; q, k, v, out 8-byte aligned; 1 <= T <= 64;
 * 1 <= n_householder <= 4; hv <= 65536 (GDN_ERR_UNSUPPORTED above);
 * batch == 0 is a no-op.
 * With T >= 16, n_householder == 1, no scatter_idx and q, k, v, out 16-byte
 * aligned, the call runs the chunked form of the same recurrence (the
 * prefill kernels over the pool, one request per row; the per-key prefill
 * kernel when decay_per_key is given): same results up to rounding order,
 * same skip / write / disable rules.
 * ------------------------------------------------------------------------- */
typedef struct {
  int32_t batch, T, n_householder;
  int32_t hq, hv, dk, dv;
  int32_t io_dtype;
  int32_t disable_state_update;
  float scale;                     /* applied as given (0.0 included)          */
  const void* q;
  const void* k;
  const void* v;
  const float* A_log;
  const float* dt_bias;
  const void* a;
  const void* b;
  float* pool;
  int32_t pool_size;
  int64_t pool_slot_stride, pool_head_stride;
  const int32_t* read_idx;
  const int32_t* write_idx;
  const int32_t* scatter_idx;
  void* out;
  /* Optional, zero = off (appended).  use_qk_l2norm of the FlashInfer page:
   * with qk_l2norm != 0 every q and k head vector x is used as
   * x / sqrt(sum(x^2) + qk_l2norm_eps) (the page's epsilon is 1e-6). */
  int32_t qk_l2norm;
  float qk_l2norm_eps;     /* >= 0 and finite                                  */
  /* Per-key decay (optional, appended): [batch, T, hv, dk] fp32 log-decay,
   * one per key dimension (the ONNX card's per-key-dimension decay spelling).
   * When given it replaces the fused gate's decay -- each token first scales
   * key column i of the V-major state by exp(decay_per_key[b,t,h,i]) -- and a,
   * A_log, dt_bias are not read (may be NULL); beta still comes from b.
   * 16-byte aligned. */
  const float* decay_per_key;
} gdn_decode_args;

gdn_status gdn_decode(const gdn_decode_args* args, void* stream);

/* ----------------------------------------------------------------------------
 * gdn_conv1d -- causal depthwise conv1d over a ragged batch, reading and
 * updating a slot-indexed conv-state pool in place.
 *
 * Contract of "gated_delta_conv1d_fwd" (parameters and example).  Sequence b
 * covers rows [row_offsets[b], row_offsets[b+1]) of x (offsets clamped to
 * total_tokens; a decreasing pair is an empty sequence).  For every channel c
 * the window is the slot's kernel_size-1 saved inputs, oldest first, followed
 * by the sequence's inputs:
 *     win = conv_state[slot_idx[b], c, :] ++ x[row_offsets[b] .., c]
 *     out[row_offsets[b] + t, c] = sum_{j < K} weight[c, j] * win[t + j]
 * so weight[c, K-1] multiplies the current input; products are summed in
 * fp32 and rounded once to io_dtype.  With write_state != 0 the slot then
 * holds the last K-1 entries of win (an empty sequence leaves it unchanged);
 * with write_state == 0 the pool is only read.  A slot_idx entry >= max_slots
 * reads zeros as its saved inputs and is never written.  Rows of x that no
 * sequence covers leave their out rows untouched.
 *
 * Layouts (row-major):
 *   x    [total_tokens, conv_dim] io_dtype, row stride x_stride_token
 *   out  [total_tokens, conv_dim] io_dtype, row stride out_stride_token
 *   weight     [conv_dim, kernel_size] io_dtype, dense
 *   conv_state [max_slots, conv_dim, kernel_size - 1] io_dtype, dense
 *   slot_idx [n_seqs] uint32; row_offsets [n_seqs + 1] uint32, non-decreasing
 *       (rows that several sequences cover get an unspecified one's output)
 * Requirements: 1 <= kernel_size <= 8; conv_dim a multiple of 16 bytes of
 * io_dtype (8 bf16 / 4 fp32 elements); x, out and conv_state 16-byte aligned;
 * row strides of x and out at least conv_dim and multiples of that same
 * count; out must not overlap x.  conv_state may be NULL only when
 * kernel_size == 1.
 * n_seqs == 0 or total_tokens == 0 is a no-op (every sequence is empty).  Two
 * sequences of one call that name the same valid slot are undefined
 * behaviour.  Two launches: the outputs, then the state write-back, in stream
 * order.
 * ------------------------------------------------------------------------- */
typedef struct {
  int64_t total_tokens;
  int32_t conv_dim;
  int32_t kernel_size;
  int32_t n_seqs;
  int32_t io_dtype;
  int32_t write_state;
  int32_t max_slots;
  const void* x;        int64_t x_stride_token;
  const void* weight;
  void* conv_state;
  const uint32_t* slot_idx;
  const uint32_t* row_offsets;
  void* out;            int64_t out_stride_token;
} gdn_conv1d_args;

gdn_status gdn_conv1d(const gdn_conv1d_args* args, void* stream);

/* ============================================================================
 * Paged key-value caches: the softmax-attention layers of a model that also
 * has gated-delta-rule layers, served beside gdn_decode's state pool.
 *
 * A cache is an array of n_pages pages of page_size tokens, each token hkv
 * heads of d elements: element (page, slot, head, i) lies at
 *     cache + page*stride_page + slot*stride_token + head*stride_head + i
 * (elements; tokens before heads or heads before tokens).  A batch row's
 * tokens are found through its page table row: position j is slot
 * j % page_size of page page_table[b][j / page_size], and lens[b] (clamped to
 * [0, max_pages*page_size]) is how many positions it holds.  Table entries
 * outside [0, n_pages) hold nothing: they are never read through or written
 * through.  One table serves every layer whose caches have its page count.
 *
 *   page_table  [batch, max_pages] int32, rows page_table_stride apart
 *   lens        [batch] int32
 *   k_scale, v_scale  [hkv] fp32: the factor of each head's stored values,
 *               given for GDN_E4M3 caches without block scales and NULL for
 *               the others
 * An 8-bit cache (GDN_E4M3, and GDN_I8 always) may instead have a scale for
 * each block of scale_block tokens of a page and head; scale_block divides
 * page_size and is at most 65536, and 0 means that there are no block scales:
 *   k_block_scale, v_block_scale  [n_pages, hkv, page_size / scale_block] fp32,
 *               dense: slot i of a page lies in block i / scale_block.  A page's
 *               scales are one dense block, for gdn_pages_copy beside its codes.
 * gdn_kv_append sets them from what it writes; a stored value is its code
 * times its block's scale.
 * Common requirements: page_size and max_pages * page_size at most 2^30; d in
 * {32, 64, 128, 256}; hq a multiple of hkv (query head h reads key-value head
 * h*hkv/hq); a cache has io_dtype's type or an 8-bit one; caches, q, k, v and out
 * 16-byte aligned, their strides non-negative multiples of 16 bytes; a cache's
 * token strides in [d, 2^23) and its head strides in [d, 2^40) elements, its rows
 * apart and its page stride not smaller than a page.
 * ========================================================================= */

/* ----------------------------------------------------------------------------
 * gdn_attn_decode -- attention of each row's newest T tokens over the cache.
 *
 * The cache already holds the new tokens (gdn_kv_append): token t of row b is
 * position lens[b] - T + t, and sees the positions up to and with its own:
 *     s_j = scale * k_scale[g] * <q[b,t,h], K[b,j,g]>,   g = h*hkv/hq
 *     out[b,t,h] = v_scale[g] * sum_j e^{s_j} V[b,j,g] / sum_j e^{s_j}
 *     lse[b,t,h] = log sum_j e^{s_j}
 * With block scales k_scale[g] is that of key j's block, and v_scale[g] stands
 * inside the sum; scales of blocks that hold no token of the row are not read.
 * A token that sees nothing (a row of no tokens, a position below 0, only
 * invalid pages), or whose scores are all -inf, gets zeros and lse -inf.  A NaN
 * in a token's query or in a key that it sees makes its result and lse NaN.
 * Values at positions that a token does not see never reach its result,
 * infinities and NaN included.  Sums and the softmax are fp32; bf16 weights
 * enter the product as two bf16 terms.
 *
 *   q    [batch, T, hq, d] io_dtype, strides {row, token, head}
 *   out  [batch, T, hq, d] io_dtype, dense
 *   lse  [batch, T, hq] fp32 or NULL
 * 1 <= T <= 64, hq <= 65536; batch * hq * T below 2^31, batch * (max_pages *
 * page_size / 16 + 1) below 2^31 and at most 2^23 groups (row, key-value head,
 * 16 of its T*hq/hkv query rows), GDN_ERR_UNSUPPORTED above.  batch == 0 is a
 * no-op.  Rows of the batch are independent: tables may share pages.
 *
 * out must not overlap q.  With a workspace of at least
 * gdn_attn_decode_workspace_size(args) bytes (device memory, 256-byte aligned;
 * 0 when none is of use) the rows' keys are dealt evenly to the waves of one
 * launch and the parts of a row joined by a second; with less, one wave walks
 * each row and key-value head: the same result up to rounding order.  The size
 * depends on sizes alone, not on lens, and is 0 for sizes that the call refuses.
 * The library keeps nothing in the workspace between calls; calls that share one
 * must not overlap.
 * ------------------------------------------------------------------------- */
typedef struct {
  int32_t batch, T, hq, hkv, d;
  int32_t io_dtype, cache_dtype;
  float scale;              /* applied as given */
  const void* q;
  int64_t q_stride_row, q_stride_token, q_stride_head;
  const void* k_cache;
  int64_t k_stride_page, k_stride_token, k_stride_head;
  const void* v_cache;
  int64_t v_stride_page, v_stride_token, v_stride_head;
  int32_t n_pages, page_size, max_pages;
  const int32_t* page_table;
  int64_t page_table_stride;
  const int32_t* lens;
  const float* k_scale;
  const float* v_scale;
  void* out;
  float* lse;
  void* workspace;
  size_t workspace_bytes;
  int32_t scale_block;      /* appended; 0: no block scales */
  const float* k_block_scale;
  const float* v_block_scale;
} gdn_attn_decode_args;

size_t gdn_attn_decode_workspace_size(const gdn_attn_decode_args* args);
gdn_status gdn_attn_decode(const gdn_attn_decode_args* args, void* stream);

/* ----------------------------------------------------------------------------
 * gdn_kv_append -- new tokens' keys and values into their pages.
 *
 * lens already counts the new tokens: row b's n_b tokens go to positions
 * lens[b] - n_b .. lens[b] - 1, in order.  Tokens whose position is negative
 * or past the table, or whose page entry is invalid, are not written.  An
 * e4m3 cache stores x / scale of the head, rounded to nearest even, clamped
 * to +-448 (NaN stays NaN); others store x as it is.
 *
 * With block scales the call sets the scale of every block that it writes to,
 * for each head, from the largest finite |x| of the block's new tokens, a:
 *     GDN_E4M3:  need = the smallest power of two with a <= 448 need
 *     GDN_I8:    need = a * (1 / 127), both fp32
 *     s = max(need, 2^-126, and, where the row has older tokens in the block,
 *             its scale until now)
 * and stores x / s rounded to nearest even, clamped to +-448 or +-127.  Where
 * the scale of a block with older tokens changes, their codes c become
 * c * s_old / s (fp32), rounded and clamped alike.  A power of two costs an 8-bit
 * float no precision, and a step from one to a larger one keeps the older
 * values, but for those that fall below the type's smallest normal number;
 * whole numbers take the closest scale and round again.  A block's first new
 * token at the block's first slot starts it anew: what its scale and codes held
 * does not matter.  NaN is a code of GDN_E4M3; GDN_I8 has none, so NaN in a
 * token makes its block's scale NaN.  A scale that is NaN stays so.
 * total_tokens / scale_block + 2 * batch is below 2^29, and K and V have
 * caches and block scales of their own (one start for both: GDN_ERR_LAYOUT).
 *
 *   k, v  [total_tokens, hkv, d] io_dtype, strides {token, head}
 *   cu_seqlens  [batch + 1] int32, non-decreasing: row b's tokens are
 *         cu_seqlens[b] .. cu_seqlens[b+1] - 1, offsets clamped to [0,
 *         total_tokens]; tokens of no row are not written.  NULL: total_tokens /
 *         batch tokens each (a whole number).  Where offsets decrease, tokens
 *         may be left out; none goes anywhere but to its place in a row whose
 *         range holds it
 * Rows whose new tokens fall into one page slot race, with block scales into one
 * block (rows share full pages only: see gdn_pages_fork).  total_tokens is at most 2^28.  batch == 0 or
 * total_tokens == 0 is a no-op.
 * ------------------------------------------------------------------------- */
typedef struct {
  int64_t total_tokens;
  int32_t batch, hkv, d;
  int32_t io_dtype, cache_dtype;
  const void* k;
  int64_t k_stride_token, k_stride_head;
  const void* v;
  int64_t v_stride_token, v_stride_head;
  const int32_t* cu_seqlens;
  void* k_cache;
  int64_t kc_stride_page, kc_stride_token, kc_stride_head;
  void* v_cache;
  int64_t vc_stride_page, vc_stride_token, vc_stride_head;
  int32_t n_pages, page_size, max_pages;
  const int32_t* page_table;
  int64_t page_table_stride;
  const int32_t* lens;
  const float* k_scale;
  const float* v_scale;
  int32_t scale_block;      /* appended; 0: no block scales */
  float* k_block_scale;
  float* v_block_scale;
} gdn_kv_append_args;

gdn_status gdn_kv_append(const gdn_kv_append_args* args, void* stream);

/* ----------------------------------------------------------------------------
 * gdn_kv_read -- tokens read back out of their pages, the way that
 * gdn_kv_append put them in.
 *
 * Row b's n_b tokens are those of positions lens[b] - n_b .. lens[b] - 1, in
 * order, of any type of cache: k and v get the stored values (the code times
 * its scale for 8-bit caches), rounded once to io_dtype.  Tokens at positions
 * that hold nothing (negative, past the table, an invalid page entry) get zeros.
 *
 *   k, v  [total_tokens, hkv, d] io_dtype, strides {token, head}; written;
 *         rows that overlap are GDN_ERR_LAYOUT
 *   cu_seqlens  as for gdn_kv_append; tokens of no row are left as they were,
 *         or get zeros with zero_rest != 0
 * k and v must not overlap each other or the caches (not checked).  cache_dtype
 * is io_dtype's type or an 8-bit one.  total_tokens is at most 2^28.  batch == 0
 * or total_tokens == 0 is a no-op.
 * ------------------------------------------------------------------------- */
typedef struct {
  int64_t total_tokens;
  int32_t batch, hkv, d;
  int32_t io_dtype, cache_dtype;
  void* k;
  int64_t k_stride_token, k_stride_head;
  void* v;
  int64_t v_stride_token, v_stride_head;
  const int32_t* cu_seqlens;
  const void* k_cache;
  int64_t kc_stride_page, kc_stride_token, kc_stride_head;
  const void* v_cache;
  int64_t vc_stride_page, vc_stride_token, vc_stride_head;
  int32_t n_pages, page_size, max_pages;
  const int32_t* page_table;
  int64_t page_table_stride;
  const int32_t* lens;
  const float* k_scale;
  const float* v_scale;
  int32_t scale_block;
  const float* k_block_scale;
  const float* v_block_scale;
  int32_t zero_rest;
} gdn_kv_read_args;

gdn_status gdn_kv_read(const gdn_kv_read_args* args, void* stream);

/* ----------------------------------------------------------------------------
 * gdn_rope -- rotary positions of queries and keys, before gdn_kv_append and
 * gdn_attn_decode.
 *
 * Of each head vector the first rot dimensions are turned in pairs (x1, x2) by
 * the angle pos * inv_freq[i], the others are copied:
 *     y1 = factor * (x1 cos - x2 sin),   y2 = factor * (x1 sin + x2 cos)
 * Pair i < rot / 2 is dimensions (i, i + rot / 2), with interleaved != 0 (2i,
 * 2i + 1).  Angles are formed in fp64 (so that far positions keep theirs), sines
 * and products in fp32; one rounding to io_dtype.
 *
 * A token's position is positions[token] where given, else it follows from lens
 * as in gdn_kv_append: token i of row b's n_b is lens[b] - n_b + i.
 *
 *   q, q_out  [total_tokens, hq, d] io_dtype, strides {token, head}
 *   k, k_out  [total_tokens, hkv, d] likewise; k NULL: queries only (hkv 0)
 *   inv_freq  [rot / 2] fp64, in radians a position
 *   positions [total_tokens] int32, or int64 with positions_i64 != 0, or NULL
 *   lens [batch] int32, cu_seqlens [batch + 1] int32 or NULL: as for
 *             gdn_kv_append (read where positions is NULL); tokens of no row
 *             are left as they were in the outputs, or get zeros with
 *             zero_rest != 0
 * An output may be its input (equal pointer and strides), or a slice of the same
 * buffer (one token stride, its heads between those of the input's tokens); other
 * overlaps, rows of an output over each other among them, are GDN_ERR_LAYOUT, and
 * so are rows dealt out in turn in other ways.  rot is even,
 * 2 <= rot <= d <= 1024; hq + hkv at most 65536; total_tokens at most 2^24;
 * pointers aligned to their element.  q_out starts neither at k nor at k_out,
 * and k_out not at q (GDN_ERR_LAYOUT); rows of q_out must not overlap those of
 * k and k_out, nor k_out's those of q (not checked: they may be slices of one
 * buffer).  total_tokens == 0 is a no-op, and so is batch == 0 without
 * positions.
 * ------------------------------------------------------------------------- */
typedef struct {
  int64_t total_tokens;
  int32_t batch, hq, hkv, d, rot;
  int32_t io_dtype, interleaved;
  float factor;
  const void* q;
  int64_t q_stride_token, q_stride_head;
  const void* k;
  int64_t k_stride_token, k_stride_head;
  void* q_out;
  int64_t qo_stride_token, qo_stride_head;
  void* k_out;
  int64_t ko_stride_token, ko_stride_head;
  const double* inv_freq;
  const void* positions;
  int32_t positions_i64;
  const int32_t* lens;
  const int32_t* cu_seqlens;
  int32_t zero_rest;
} gdn_rope_args;

gdn_status gdn_rope(const gdn_rope_args* args, void* stream);

/* ----------------------------------------------------------------------------
 * gdn_pages_copy -- contents of pages (or of state-pool and conv-state slots)
 * copied inside one pool: page dst[i] becomes page src[i] for i < n.
 *
 * page_bytes bytes at pool + page*page_stride (bytes, any alignment).  Pairs
 * with an entry outside [0, n_pages), or equal entries, are skipped.  A page
 * that one pair writes and another reads or writes is undefined behaviour.
 * n == 0 is a no-op.
 * ------------------------------------------------------------------------- */
gdn_status gdn_pages_copy(void* pool, int64_t page_bytes, int64_t page_stride, int32_t n_pages,
                          const int32_t* src, const int32_t* dst, int64_t n, void* stream);

/* ----------------------------------------------------------------------------
 * Page tables on the device.  refs[p] is how many holders page p has (table
 * rows, and whatever else the caller counts); 0 means free.  A row's pages
 * are its first ceil(lens / page_size) entries.  Free pages are taken lowest
 * first in row order, so results are determined by the inputs; nothing is
 * read on the host, and the calls can be captured.
 *
 * Inputs page_table, lens, refs; outputs page_table_out, lens_out, refs_out,
 * which extend, free and compact also take as the inputs themselves (equal
 * pointers and strides; partial overlaps are not checked); fork reads rows
 * while it writes others and needs page_table_out and lens_out apart.
 * workspace: gdn_pages_workspace_size(rows, n_pages) bytes (256-byte aligned;
 * pages_free needs none); calls that share one must not overlap.
 * Requirements: n_pages in [1, 2^22], rows at most 2^20, max_pages >= 1, page_size >= 1,
 * max_pages * page_size at most 2^30, row strides at least max_pages.
 *
 *  extend   Row r grows by add[r] tokens (below 0: by none).  A row is served,
 *           ok[r] = 1, if the new length fits its table row and the pages that
 *           it and the rows before it need (those that fit their tables) are
 *           free; a row that needs no page is always served.  Others stay as
 *           they are, ok[r] = 0.
 *  fork     Row r becomes what row parent[r] was on entry: its length and
 *           pages, shared; parent[r] == r keeps it, an entry outside
 *           [0, rows) leaves it empty and releases its pages.  A part-filled
 *           last page that others hold too gets its own copy, so that rows
 *           may append: dst[r] is the fresh page and src[r] the shared one,
 *           for gdn_pages_copy on each cache (-1 where there is none).  Where
 *           every holder has the page as its part-filled last one, the lowest
 *           such row keeps it.  A row for which no page is left ends empty
 *           (length 0) with its pages released.  Entries past a row's pages
 *           become -1.
 *  free     Rows with mask[r] != 0 release their pages and end empty.
 *  compact  The pages in use (refs > 0; n_live of them) move to the lowest
 *           page numbers: the i-th page in use at or above n_live moves to
 *           the i-th free page below it, in every table entry and in refs.
 *           src[i], dst[i] for i < n_pages / 2 are the moves, for
 *           gdn_pages_copy (no page is both; -1 past the last).  lens is not
 *           read and lens_out not written.
 * ------------------------------------------------------------------------- */
typedef struct {
  int32_t rows, max_pages, n_pages, page_size;
  const int32_t* page_table;
  int64_t page_table_stride;
  const int32_t* lens;
  const int32_t* refs;      /* [n_pages] */
  int32_t* page_table_out;
  int64_t page_table_out_stride;
  int32_t* lens_out;
  int32_t* refs_out;
  void* workspace;
  size_t workspace_bytes;
} gdn_pages_args;

size_t gdn_pages_workspace_size(int32_t rows, int32_t n_pages);
gdn_status gdn_pages_extend(const gdn_pages_args* args, const int32_t* add, int32_t* ok, void* stream);
gdn_status gdn_pages_fork(const gdn_pages_args* args, const int32_t* parent, int32_t* src, int32_t* dst,
                          void* stream);
gdn_status gdn_pages_free(const gdn_pages_args* args, const uint8_t* mask, void* stream);
gdn_status gdn_pages_compact(const gdn_pages_args* args, int32_t* src, int32_t* dst, int32_t* n_live,
                             void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBGDN_H */
