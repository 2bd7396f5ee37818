/*
 * moeffn.h - C ABI of the routed MoE-FFN step on GB300 (sm_103a).
 *
 * The step, for each token t (diskformer engine modules, as shown by diffend.io):
 *   logit_e = sum_h Wr[e][h] x[t][h]                      router, F32 "ffn_gate_inp"
 *                                                          (lfm2_moe_ssd.js, initBuffers: router binding)
 *   p_e = 1 / (1 + exp(-logit_e)); s_e = p_e + bias_e      bias only selects
 *                                                          (lfm2_moe_ssd.js, TOPK_SIG_BODY and its comment)
 *   groups (n_groups > 1): group score = the two largest s of the group summed;
 *   keep the groups_used best groups, lowest group on ties  (ling_moe_ssd.js, routeLing)
 *   picks: top_k rounds of argmax over the kept s, lowest index on ties, in
 *   selection order                                         (TOPK_SIG_BODY)
 *   w_j = p_pick_j / max(sum_j p_pick_j, norm_min) * weights_scale   (TOPK_SIG_BODY, routeLing)
 *   expert: [g; u] = W_gu x (gate rows then up rows), y = W_down (silu(g) * u), or with a
 *   clamp limit L > 0, y = W_down (min(silu(g), L) * clamp(u, -L, L))
 *                                                          (ling_moe_ssd.js, swiglu;
 *                                                           flint_moe_ssd.js, planLayoutFlint record)
 *   shared expert: the same SwiGLU with weight 1, no gate  (flint_moe_ssd.js, file header)
 *   out[t] = sum_j w_j y_j + shared                         (ling_moe_ssd.js, moeAccum)
 * Weights are ggml 4-bit blocks of 32 values (flint_moe_ssd.js, WGSL section,
 * comment above Q41DOT): Q4_1 = f16 d, f16 m, 16 nibble bytes, value d*q + m;
 * Q4_0 = f16 d, 16 nibble bytes, value d*(q - 8). In a block the low nibble of
 * byte i is value i and its high nibble is value 16 + i.
 * K-quant super-blocks of 256 values, the types the Ling store keeps (ling_moe_ssd.js,
 * file header and planLayoutLing: Q4_K gate/up rows, Q6_K or Q4_K down rows); the pages
 * name these types without their layouts, which are ggml's:
 *   Q4_K, 144 bytes: f16 d, f16 dmin, 12 bytes of packed 6-bit scales sc_j and mins mn_j
 *     of the eight 32-value sub-blocks, then four runs of 32 nibble bytes (run c: values
 *     64c .. in the low nibbles, 64c + 32 .. in the high nibbles); value = d sc_j q - dmin mn_j.
 *   Q6_K, 210 bytes: 128 bytes of low nibbles, 64 bytes of 2-bit high parts, 16 int8
 *     scales (one per 16 values), f16 d; value = d * scale * (q - 32).
 *
 * Layouts (all row-major, little-endian):
 *   x, out         [n_tokens][hidden] f32
 *   router_w       [n_experts][hidden] f32 (row e = expert e)
 *   router_bias    [n_experts] f32, or NULL for no selection bias
 *   expert_blocks  n_experts records back to back; record = gate [expert_ff rows of hidden
 *                  values], up [expert_ff rows], both in qtype, then down [hidden rows of
 *                  expert_ff values] in the down type (qtype_down, or qtype when it is 0);
 *                  a row of n values takes n/32 blocks (Q4_0 18, Q4_1 20 bytes) or n/256
 *                  super-blocks (Q4_K 144, Q6_K 210 bytes)
 *   shared_blocks  one record of the same form with shared_ff, or NULL when shared_ff == 0
 *   topk_ids       [n_tokens][top_k] int32 picks in selection order (optional output)
 *   topk_w         [n_tokens][top_k] f32 weights (optional output)
 *
 * Ownership: the caller owns every buffer; the library never frees caller memory.
 * Device pointers unless MOE_HOST_IO is set. Weights must not change while a call
 * that reads them is in flight: calls read weights before the previous kernel on
 * the stream has finished (programmatic dependent launch) unless MOE_NO_PDL is set.
 * x and out must not overlap.
 *
 * Errors: every entry point returns MOE_OK (0) or a negative MOE_ERR_* code and
 * sets a thread-local message (moe_last_error). Configurations and pointers are
 * checked on the host before anything is launched. Kernels never trap: a device
 * wait that runs out of time sets a status word in the workspace, which
 * moe_workspace_status reports as MOE_ERR_TIMEOUT.
 */
#ifndef MOEFFN_H
#define MOEFFN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ggml block type ids (flint_moe_ssd.js: GGML_Q4_1 = 3). */
#define MOE_Q4_0 2
#define MOE_Q4_1 3
#define MOE_Q4_K 12
#define MOE_Q6_K 14

/* Activation types of the operators next to the step (ggml type ids). */
#define MOE_F32 0
#define MOE_F16 1
#define MOE_BF16 30
/* 4-bit rows held as separate planes, for moe_q4_matvec (not a ggml type). */
#define MOE_Q4_PLANES 64
/* Codes of the 8-bit key/value cache: int8 (ggml type id), e4m3 (not a ggml type). */
#define MOE_I8 24
#define MOE_E4M3 65

/* moe_cfg.flags */
#define MOE_ACCUMULATE 1u /* out = out + contribution (the pages' x += ...)          */
#define MOE_RESIDUAL 2u   /* out = x + contribution                                 */
#define MOE_HOST_IO 4u    /* x, out, topk_ids, topk_w are host pointers: x is copied in;
                           * outputs in page-locked memory mapped into the device's address
                           * space are written in place, other outputs are staged */
#define MOE_NO_PDL 8u     /* launch without programmatic dependent launch             */
#define MOE_TRACE 16u     /* record a per-CTA timeline in the workspace (see below)   */
#define MOE_BATCHED 32u   /* take the batched path whatever the token count           */
#define MOE_F32_ACT 64u   /* decode chain: f32 activations in the block dots (the pages'
                           * arithmetic) instead of 16-bit block fixed point (see below) */
#define MOE_GRAPH 128u    /* replay a captured CUDA graph for an argument set seen before
                           * (see moe_ffn_forward_ex)                                  */

enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_CFG = -1,
  MOE_ERR_NULL_PTR = -2,
  MOE_ERR_ALIGNMENT = -3,
  MOE_ERR_UNSUPPORTED = -4,
  MOE_ERR_CUDA = -5,
  MOE_ERR_TIMEOUT = -6,
  MOE_ERR_WORKSPACE = -7
};

/* One MoE layer and one batch of tokens. The knobs are the layer's GGUF keys
 * (expert_count, expert_used_count, expert_feed_forward_length,
 * expert_shared_feed_forward_length, expert_group_count, expert_group_used_count,
 * expert_weights_scale; flint_moe_ssd.js configFromGgufFlint, ling_moe_ssd.js
 * configFromGgufLing). Limits checked by every entry point:
 *   hidden, expert_ff, shared_ff multiples of 32 (shared_ff may be 0), at most 3072;
 *   1 <= top_k <= min(n_experts, 32); n_experts <= 1024;
 *   n_groups divides n_experts; n_groups > 1 needs n_experts / n_groups >= 2,
 *   n_groups <= 64, 1 <= groups_used <= n_groups, top_k <= groups_used * n_experts / n_groups;
 *   n_tokens >= 0 (0: nothing is launched); qtype MOE_Q4_0, MOE_Q4_1 or MOE_Q4_K;
 *   qtype_down 0 (the same as qtype), MOE_Q4_0, MOE_Q4_1, MOE_Q4_K or MOE_Q6_K;
 *   K-quant gate/up rows need hidden % 256 == 0, K-quant down rows expert_ff and
 *   shared_ff multiples of 256;
 *   norm_min >= 0 (the pages use 2^-14 = 6.103515625e-5). */
typedef struct moe_cfg {
  int32_t hidden;
  int32_t n_experts;
  int32_t top_k;
  int32_t expert_ff;
  int32_t shared_ff;
  int32_t n_groups;    /* 1 = plain top-k */
  int32_t groups_used; /* ignored when n_groups == 1 */
  int32_t n_tokens;
  int32_t qtype;
  float weights_scale; /* 1.0 unless the layer says otherwise */
  float norm_min;      /* clamp on the sum of the picked sigmoids */
  uint32_t flags;      /* MOE_* flags above */
  /* SwiGLU clamp limits L, >= 0 (ling_moe_ssd.js, the swiglu kernel and its comment:
   * act = min(silu(g), L) * clamp(u, -L, L); L = 0 means no clamp). The routed experts
   * and the shared expert take separate per-layer limits, as the page's
   * swiglu_clamp_exp / swiglu_clamp_shexp arrays do. */
  float swiglu_limit;
  float swiglu_limit_shared;
  /* Optional layer prologue: with ffn_norm (a device vector [hidden] f32, 16-byte
   * aligned) the step's input is rms_norm(x) * ffn_norm, rms_norm(x) = x /
   * sqrt(mean(x^2) + rms_eps) (flint_moe_ssd.js / lfm2_moe_ssd.js headers: x +=
   * ffn(rms_norm(x) * ffn_norm)); MOE_RESIDUAL then adds the raw x, giving the whole
   * FFN block. NULL: x enters as is. */
  float rms_eps;
  const float* ffn_norm;
  /* Block type of the down rows (routed and shared), or 0 for qtype: the Ling store
   * types its down rows per layer, apart from the gate/up rows (ling_moe_ssd.js,
   * planLayoutLing). */
  int32_t qtype_down;
} moe_cfg;

/* Two execution paths, chosen by n_tokens (both are exact restatements of the step
 * above; they differ in arithmetic only):
 *   n_tokens < 44  the decode chain, up to 16 tokens per launch: a router kernel,
 *                  (with several tokens) a selection kernel, a gate/up kernel and a
 *                  down kernel with the weighted sum. The router is an f32 dot. By
 *                  default the 4-bit blocks meet activations held in 16-bit block
 *                  fixed point (a power-of-two scale per 16 values, error at most
 *                  2^-15 of the largest magnitude among those 16), so each block dot is an
 *                  exact int32 sum (dp4a), scaled and accumulated in f32. With
 *                  MOE_F32_ACT the activations stay f32 and each block contributes
 *                  d * sum(q x) + m * sum(x) by f32 fused multiply-adds (the pages'
 *                  arithmetic); it runs about 12% slower on the Flint-shaped layer.
 *   n_tokens >= 44 (or MOE_BATCHED) the batched path, in passes of at most 512
 *                  tokens. A router contraction accumulated in f32 (on the tile pipeline
 *                  from f16 hi + lo parts of the f32 rows and tokens, in up to four K
 *                  slices summed in order); one warp per token for the selection; a stable
 *                  counting sort of the (token, pick) pairs by expert; grouped
 *                  contractions on the tensor cores. The 4-bit blocks are dequantised
 *                  exactly to f16 before a single rounding; K-quant values on the tile
 *                  pipeline below take their f16-rounded scale and offset (up to three
 *                  roundings of 2^-11). x enters as an f16 hi + lo pair (22 bits). The
 *                  SwiGLU activations are rounded once to f16. Products accumulate in
 *                  f32. Requires |x| and every activation to stay below 65504 (the f16
 *                  range).
 *   The batched contractions run as warp-specialised TMA/TMEM pipelines for layers whose
 *   three matrices are all Q4_1 (or all Q4_0) with hidden, expert_ff and shared_ff whole
 *   multiples of 128 (Q4_1) or 256 (Q4_0), and for Q4_K gate/up rows with Q4_K or Q6_K down
 *   rows with all three multiples of 256 (Q6_K down rows of at most 768 values); other
 *   layers run a general form of the same contractions.
 * Both paths give the same picks; outputs agree to the tolerance of their arithmetic
 * (relative L2 well under 2e-3 against a float64 evaluation). */

/* The step on the default stream with a library-owned workspace (one per
 * device, grown on demand, freed by moe_shutdown). Blocks until the step is
 * done and returns device-side errors directly. Pointer alignment: x, out,
 * router_w, expert_blocks, shared_blocks 16 bytes; router_bias 4 bytes. */
int moe_ffn_forward(const float* x, const float* router_w, const float* router_bias,
                    const void* expert_blocks, const void* shared_blocks, const moe_cfg* cfg,
                    float* out);

/* The step enqueued on `stream` (a cudaStream_t, NULL = legacy default stream)
 * with a caller-owned device workspace of at least moe_workspace_size(cfg) bytes,
 * 256-byte aligned. A workspace must be zero-filled before its first use and then
 * only touched by this library: its first 512 bytes are control words (the
 * status word that moe_workspace_status reads). Calls sharing one workspace must
 * be ordered (same stream, or synchronised); calls with different configurations
 * may share one.
 * Asynchronous: device-side errors surface through moe_workspace_status.
 * topk_ids / topk_w may be NULL.
 * With MOE_GRAPH the library remembers the 64 argument sets (every pointer, the sizes and
 * the cfg) used most recently in the process. The second call with a set captures all of
 * its work into a CUDA graph on a library-owned stream, and every later call with that set
 * is one launch of the graph on `stream`: the same kernels and arguments, so the same
 * results, with less host time per call. The buffers of a remembered set must stay
 * allocated, and host buffers page-locked, until moe_shutdown or until 64 other sets have
 * been used since. A call made while `stream` is being captured, a MOE_TRACE call, and a
 * set whose capture fails run directly. */
int moe_ffn_forward_ex(const float* x, const float* router_w, const float* router_bias,
                       const void* expert_blocks, const void* shared_blocks, const moe_cfg* cfg,
                       float* out, void* workspace, size_t workspace_bytes, void* stream,
                       int32_t* topk_ids, float* topk_w);

/* Workspace bytes a call with this configuration needs (0 for an invalid cfg). */
size_t moe_workspace_size(const moe_cfg* cfg);

/* Byte offset of the MOE_TRACE timeline in the workspace (0 when cfg is invalid or
 * has no MOE_TRACE). The timeline holds 24 u64 words for each of the first
 * n_SM CTA indices: %globaltimer readings in nanoseconds, written by thread 0 of
 * the CTA with that index in each of the three decode kernels of the last token:
 * router kernel 0 start, 1 x ready (previous kernel done), 2 logits written;
 * gate/up kernel 4 start, 5 x quantised, 6 logits ready, 7 picks made, 8 the CTA's
 * first rows in shared memory, 9 activation block written, and within its selection
 * (single-token calls) 3 keys made, 19 candidates gathered, 22 picks ranked; down kernel 12 start,
 * 13 picks made, 14 row copies issued, 15 activation blocks ready, 16 activation
 * blocks staged, 17 rows in shared memory, 18 output rows written. Unused words
 * stay 0. */
size_t moe_trace_offset(const moe_cfg* cfg);

/* Waits for `stream`, then reads and clears the workspace's status word:
 * MOE_OK, or MOE_ERR_TIMEOUT when a device-side wait ran out of time, or
 * MOE_ERR_INVALID_CFG when offsets left sequences without room (moe_linattn_prefill); the
 * workspace's control block is zeroed again so it can be reused. */
int moe_workspace_status(void* workspace, void* stream);

/* Exercises the error path above without a fault: one kernel waits on an mbarrier that
 * nothing completes, through the same bounded wait the step's kernels use, gives up after
 * its time limit (0.5 s) and sets the timeout bit in the workspace's status word, as a
 * stalled copy would. A following moe_workspace_status reports MOE_ERR_TIMEOUT and clears
 * it; the context stays usable. `workspace` is any workspace of at least 512 bytes;
 * asynchronous on `stream`. Returns MOE_OK or MOE_ERR_NULL_PTR / MOE_ERR_CUDA. */
int moe_selftest_timeout(void* workspace, void* stream);

/* The step for callers that cannot allocate memory: the call makes no cudaMalloc,
 * cudaFree or other allocating call, on the device or on the host. Such callers include
 * code that runs where an allocator may not be entered (inside another allocator's hooks,
 * in a real-time or signal context, under a memory budget that has already been handed
 * out) or that has no allocator of its own to lend a workspace. The pages have no
 * counterpart: their engines own every buffer.
 * The scratch lives in a fixed device array of 512 KiB compiled into the library; every
 * device that loads the library holds it until the process exits, and every call on a
 * device shares it, so calls whose work overlaps on the GPU (other streams, other
 * threads) race and must not be made. Each call looks the array's device address up
 * afresh. CUDA loads the library's kernels and this array onto a device on first use,
 * and that loading may itself allocate device memory: make the first call on each device
 * before the stretch in which nothing may be allocated, and before any stream capture.
 * Up to 16 tokens are decoded per launch, as many as the array holds the scratch of
 * (control block, logits and SwiGLU activations); one token of the largest layer the
 * configuration checks admit needs about 401 KiB, so every admitted layer runs, and a
 * layer that needed more would be rejected with MOE_ERR_UNSUPPORTED. Device buffers
 * only: MOE_HOST_IO and MOE_TRACE are rejected. Blocking: returns after the step has
 * finished on `stream` (a cudaStream_t, NULL = legacy default stream), with device-side
 * errors reported directly. Arguments otherwise as moe_ffn_forward. */
int moe_ffn_forward_noalloc(const float* x, const float* router_w, const float* router_bias,
                            const void* expert_blocks, const void* shared_blocks, const moe_cfg* cfg,
                            float* out, void* stream);

/* ---------------------------------------------------------------------------------------
 * Operators next to the step: the projections of a layer whose matrices are 4-bit blocks,
 * and linear attention with a decay for each head (one number a head and token; no decay
 * for each key channel and no delta rule). With the step they make a whole recurrent layer
 * of that kind: projection, moe_linattn_prefill or moe_linattn_step, projection added
 * into the residual stream, moe_ffn_forward_ex with the norm prologue and MOE_RESIDUAL
 * (examples/linear_layer.py).
 * ------------------------------------------------------------------------------------- */

/* moe_linattn_cfg.flags (besides MOE_NO_PDL) */
#define MOE_FRESH_STATE 256u /* sequences start from a zero state: the pool is only written */
#define MOE_TOKEN_DECAY 512u /* log_decay has a row for each token                          */

/* A matrix W [rows][cols] and the vectors it multiplies.
 *   qtype MOE_Q4_0, MOE_Q4_1, MOE_Q4_K: rows of blocks as in the expert records above
 *     (cols a multiple of 32, of 256 for MOE_Q4_K), group 0.
 *   qtype MOE_Q4_PLANES: `weights` is [rows][cols / 2] nibble bytes, 16 bytes for every 32
 *     values in the blocks' order (byte i: value i low, value 16 + i high); `scales` is
 *     [rows][cols / group] f16 and `mins` the same or NULL, group 32, 64 or 128, dividing
 *     cols; value = scale q + min, without mins scale (q - 8).
 * Limits: 1 <= rows; 32 <= cols <= 16384; 0 <= n_vec <= 65535 (0: nothing is launched). */
typedef struct moe_matvec_cfg {
  int32_t rows;
  int32_t cols;
  int32_t n_vec;
  int32_t qtype;
  int32_t group;
  int32_t x_type;   /* MOE_F32, MOE_F16 or MOE_BF16 */
  int32_t y_type;
  uint32_t flags;   /* MOE_ACCUMULATE (y = y + ...), MOE_NO_PDL */
  int64_t x_stride; /* values from one vector to the next; 0: cols */
  int64_t y_stride; /* 0: rows */
} moe_matvec_cfg;

/* y_t = W x_t (+ bias) (+ y_t) for n_vec vectors, enqueued on `stream`. `bias` is [rows] f32
 * or NULL; scales and mins are NULL unless qtype is MOE_Q4_PLANES. No workspace. Weights
 * enter as they are. x enters in 22 bits (two f16 parts) of each value down to 2^-15 of the
 * largest of its block of 32, fewer below (f16 and bf16 values as they are down to 2^-27).
 * Sums are f32, y is rounded once, and repeat calls agree bit for bit. Each vector's result
 * does not depend on the others of the call (their number picks the order of the sums). A
 * vector that holds an infinity or a NaN gives rows that are not finite.
 * A call reads the matrix once for up to 16 vectors (fewer where rows are long) and again for
 * every further 16, so it is not the form for long prompts: with torch, dequantising
 * 8192 x 2560 and one library product take less time from about 350 bf16 vectors (600 f32
 * ones) on, and where the dequantised matrix is kept from a handful (70 f32 ones) on.
 * The matrix is read before the previous kernel on the stream has finished, as the step
 * reads its weights, unless MOE_NO_PDL is set. Alignment: weights, scales, mins, x and every
 * vector of x (x_stride) 16 bytes; y and bias their element. x and y must not overlap. */
int moe_q4_matvec(const void* x, const void* weights, const void* scales, const void* mins, const float* bias,
                  const moe_matvec_cfg* cfg, void* y, void* stream);

/* Linear attention with a decay for each head. For each sequence and each of n_heads heads
 * the state S is key_dim x value_dim, and token t does
 *   S = exp(g_t) S + k_t v_t^T,   o_t = scale * S^T q_t
 * (the token's own k and v included). Layouts, all row-major:
 *   q, k       [n_tokens][n_qk_heads][key_dim]; head h reads q/k head h / (n_heads / n_qk_heads)
 *   v, o       [n_tokens][n_heads][value_dim]
 *   log_decay  g, f32: [n_heads], or [n_tokens][n_heads] with MOE_TOKEN_DECAY. -infinity
 *              is a factor of 0: it forgets the finite state before the token (an infinity or a
 *              NaN stays one as a NaN; MOE_FRESH_STATE takes no notice of either).
 *   state      [n_states][n_heads][key_dim][value_dim] f32, updated in place
 *   slots      [n_seq] int32, the state of each sequence, or NULL for sequence b in state b.
 *              A sequence whose slot is outside 0 .. n_states - 1 is inactive: its rows of o
 *              become 0 and no state is touched. Two sequences must not share a slot.
 * q, k, v and o have one type; tokens may be strided (views of one projected buffer).
 * Limits: key_dim and value_dim multiples of 8 from 8 to 128; n_qk_heads divides n_heads,
 * n_heads <= 1024; n_seq <= 65535; n_seq and n_tokens >= 0; scale finite. Alignment: q, k,
 * v, o, state and every token row (strides) 16 bytes, the others 4. o must not overlap
 * q, k or v. */
typedef struct moe_linattn_cfg {
  int32_t n_seq;
  int32_t n_tokens;  /* of all sequences together; a step has n_tokens == n_seq */
  int32_t n_heads;
  int32_t n_qk_heads;
  int32_t key_dim;
  int32_t value_dim;
  int32_t n_states;
  int32_t type;      /* of q, k, v, o: MOE_F32, MOE_F16 or MOE_BF16 */
  float scale;
  uint32_t flags;    /* MOE_FRESH_STATE, MOE_TOKEN_DECAY, MOE_NO_PDL */
  int64_t q_stride;  /* values from one token to the next; 0: packed */
  int64_t k_stride;
  int64_t v_stride;
  int64_t o_stride;
} moe_linattn_cfg;

/* Whole prompts: sequence b is the tokens offsets[b] .. offsets[b + 1] - 1 (device int32,
 * n_seq + 1 values, ascending; bounds outside 0 .. n_tokens are clamped to it and a
 * descending pair is an empty sequence; where they then rise again, sequences share tokens:
 * what their common rows of o hold is open, and long sequences for which the call has no units
 * keep their state and rows, which moe_workspace_status reports as MOE_ERR_INVALID_CFG).
 * offsets NULL: n_seq sequences of n_tokens / n_seq
 * tokens. An empty sequence keeps its state (or gets a zero one with MOE_FRESH_STATE).
 * Rows of o that no sequence covers are not written. `workspace` as for
 * moe_ffn_forward_ex (zero-filled before its first use, then this library's), of at
 * least moe_linattn_workspace_size(cfg) bytes; a wait that gave up surfaces through
 * moe_workspace_status.
 * Bits: sums, decays and states are f32, o is rounded once. Short prompts multiply in f32.
 * Longer ones multiply on the tensor cores: f32 values, scores and states as they are (24
 * bits each, whatever stands beside them); f16 and bf16 q, k, v as they are, with bf16's
 * scores and states in 16 bits and its decayed keys in 24, and f16's scores, states and
 * decayed keys in 22 bits down to 2^-15 of the largest beside them, fewer below (of a token's
 * scores, of a value channel's state, of the decayed keys of 64 tokens).
 * A value that is not finite reaches what the formula gives it and no earlier token, no other
 * sequence and no other head. Chunks of 64 tokens with such an output are redone token by
 * token, so a head whose state holds one takes several times as long from there on. */
int moe_linattn_prefill(const void* q, const void* k, const void* v, const float* log_decay,
                        const int32_t* offsets, const int32_t* slots, const moe_linattn_cfg* cfg, float* state,
                        void* o, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes of a moe_linattn_prefill call (0 for an invalid cfg); fewer tokens of the
 * same heads and type need no more. */
size_t moe_linattn_workspace_size(const moe_linattn_cfg* cfg);

/* One token for each sequence (row b of q, k, v, o and of a per-token log_decay is
 * sequence b). No workspace. */
int moe_linattn_step(const void* q, const void* k, const void* v, const float* log_decay, const int32_t* slots,
                     const moe_linattn_cfg* cfg, float* state, void* o, void* stream);

/* ---------------------------------------------------------------------------------------
 * The 8-bit key/value cache and the attention that reads it: what a layer with softmax attention
 * needs next to the projections and the step. A layer's turn is projection, moe_kv8_write of the
 * new tokens' keys and values, moe_kv8_attn_step or moe_kv8_attn_prefill, projection, step
 * (examples/attention_layer.py).
 * ------------------------------------------------------------------------------------- */

/* A cache is n_pages records of moe_kv8_page_bytes(cfg) bytes back to back (`cache`, 16-byte
 * aligned). A page holds page_tokens tokens of every key/value head:
 *   for each head: codes of K [page_tokens][head_dim], codes of V [page_tokens][head_dim];
 *   then for each head: scale bytes of K [page_tokens / block_tokens], of V the same;
 *   padded to a multiple of 128 bytes.
 * A code is an int8 (-127 .. 127; MOE_I8) or an e4m3 number (finite; MOE_E4M3). A scale byte s
 * stands for 2^(s - 127), 255 for NaN: a value is code * 2^(s - 127).
 * `pages` [n_seq][max_pages] (device int32) is the page table: position p of sequence b is place
 * p % page_tokens of page pages[b][p / page_tokens]. A page outside 0 .. n_pages - 1 is not held,
 * and neither are positions outside 0 .. max_pages * page_tokens - 1: nothing is written there, reads
 * give 0, and attention does not see them. Sequences may share pages that nobody writes.
 * Every call has n_tokens token rows; sequence b is the rows offsets[b] .. offsets[b + 1] - 1 (device
 * int32, n_seq + 1 values, ascending, clamped to 0 .. n_tokens; a descending pair is an empty
 * sequence; NULL: n_seq sequences of n_tokens / n_seq rows), and its row i has position past[b] + i
 * (device int32 [n_seq]; NULL: zeros). Rows that no sequence covers are not written. Where offsets
 * fall and rise again, which sequence a shared row belongs to is open.
 * Limits: n_seq <= 65535; n_tokens <= 2^28; n_kv_heads divides n_heads <= 1024; n_tokens * n_heads <
 * 2^31; head_dim a multiple of 16 from 16 to 256; page_tokens a power of two from 16 to 256; block_tokens a power of two from 1 to 64,
 * at most page_tokens; max_pages * page_tokens <= 2^30; the pool less than 2^38 bytes; window >= 0; scale finite. k, v, q and o
 * have one type; tokens may be strided (views of one projected buffer). Alignment: q, k, v, o, cache and
 * every token row (strides) 16 bytes, the others 4. Nothing that a call writes may overlap what it
 * reads. */
typedef struct moe_kv8_cfg {
  int32_t n_seq;
  int32_t n_tokens;   /* of all sequences together; a step has n_tokens == n_seq */
  int32_t n_heads;    /* query heads (attention) */
  int32_t n_kv_heads; /* head h reads key/value head h / (n_heads / n_kv_heads) */
  int32_t head_dim;
  int32_t page_tokens;
  int32_t block_tokens; /* tokens that share a scale */
  int32_t n_pages;
  int32_t max_pages;  /* entries of a row of the page table */
  int32_t code;       /* MOE_I8 or MOE_E4M3 */
  int32_t type;       /* of q, k, v, o: MOE_F32, MOE_F16 or MOE_BF16 */
  int32_t window;     /* attention: a token sees itself and the window - 1 before it; 0: all */
  float scale;        /* of the scores */
  uint32_t flags;     /* MOE_NO_PDL */
  int64_t q_stride;   /* values from one token to the next; 0: packed */
  int64_t k_stride;
  int64_t v_stride;
  int64_t o_stride;
} moe_kv8_cfg;

/* Bytes of a page (0 for an invalid cfg). */
size_t moe_kv8_page_bytes(const moe_kv8_cfg* cfg);

/* Quantises k, v [n_tokens][n_kv_heads][head_dim] into the cache. For each block that the call
 * touches, head, and K and V apart: amax is the largest magnitude of the call's values, e the smallest
 * integer, at least -127, with amax <= 127 * 2^e (448 * 2^e for e4m3), and a code is x / 2^e rounded to
 * nearest even. Tokens of the block at positions before the call's first one stay: the scale is then the
 * larger of theirs and e, and where it grew their codes are rounded again to it (all such roundings
 * of a value together lose less than one step of the scale it ends with for int8). Tokens behind the
 * call's last one mean nothing any more. A call that starts at a block's first position takes no notice
 * of what the block held, so pages need no clearing. A block with an infinity or a NaN gets the
 * NaN scale, which makes all of its values NaN until its first position is written again.
 * Two sequences must not write to one block, nor one sequence twice to a block of a page that its table has twice. */
int moe_kv8_write(const void* k, const void* v, const int32_t* offsets, const int32_t* past, const int32_t* pages,
                  const moe_kv8_cfg* cfg, void* cache, void* stream);

/* The values of positions past[b] .. of each sequence as k, v [n_tokens][n_kv_heads][head_dim], each rounded
 * once to the type (int8 and e4m3 values are bf16 numbers: they come back as they are). */
int moe_kv8_read(const void* cache, const int32_t* offsets, const int32_t* past, const int32_t* pages,
                 const moe_kv8_cfg* cfg, void* k, void* v, void* stream);

/* Attention of the rows of q [n_tokens][n_heads][head_dim] over the cache, which holds their own keys and
 * values already (moe_kv8_write before). Row i of sequence b, at position p = past[b] + i, sees the held
 * positions j <= p (with a window, j > p - window), the prompt's own earlier tokens among them:
 *   s_j = scale * q . k_j,   o = sum_j exp(s_j) v_j / (sum_j exp(s_j) + exp(sinks[h]))
 * The sinks [n_heads] f32 are logits that take weight and add no value (NULL: none; flint_moe_ssd.js,
 * SOFTMAX_SINK). A row that sees nothing becomes 0. `workspace` as for moe_ffn_forward_ex, of at
 * least moe_kv8_workspace_size(cfg) bytes.
 * Bits: scores, softmax statistics and sums are f32, o is rounded once. As operands the weights have 16 bits (bf16, and
 * f16 sequences of more than 48 rows: tokens x heads that share a key/value head) or 24 (the others), each by its own size,
 * however small it is beside the row's largest. V is exact; in sequences of more than 48 rows of 16-bit types and heads of up
 * to 128 while no V scale among a tile's tokens is above 2^49, else for scales down to 2^-170 of the largest. Weights below
 * 2^-110 of the row's largest, or of its sink's, may be 0. (Scores beyond f32's range are infinities
 * and what their rows become is open.) A row of q that holds an infinity or a
 * NaN gives a row that is not finite, and so does a NaN block that a row sees; neither reaches other
 * rows. */
int moe_kv8_attn_prefill(const void* q, const void* cache, const int32_t* offsets, const int32_t* past,
                         const int32_t* pages, const float* sinks, const moe_kv8_cfg* cfg, void* o, void* workspace,
                         size_t workspace_bytes, void* stream);

/* The same for one token of each sequence: row b is sequence b's, at position past[b]. */
int moe_kv8_attn_step(const void* q, const void* cache, const int32_t* past, const int32_t* pages,
                      const float* sinks, const moe_kv8_cfg* cfg, void* o, void* workspace, size_t workspace_bytes,
                      void* stream);

/* Workspace bytes of an attention call (0 for an invalid cfg); fewer tokens or sequences need no more. */
size_t moe_kv8_workspace_size(const moe_kv8_cfg* cfg);

/* Text of the last error on the calling thread ("" if none). */
const char* moe_last_error(void);

/* Frees the library-owned workspaces. Returns MOE_OK or MOE_ERR_CUDA. */
int moe_shutdown(void);

#ifdef __cplusplus
}
#endif

#endif /* MOEFFN_H */
