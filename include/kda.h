/*
 * kda.h -- C ABI of libkda.so, the MI355X (gfx950) implementation of the Kimi Delta Attention
 * (KDA) forward pass: the forget gate, chunked prefill and the single-token decode step; and of its
 * siblings: linear attention with one decay per head (prefill, gradients, decode step), the selective state
 * space scan with its short convolution (the same three), an 8-bit cache of recurrent states and the
 * management of their slots.
 *
 * Pages the operations come from (titles as published):
 *   [bagrov] "Архитектура Kimi K3: как открытая модель с миллионным контекстом конкурирует с
 *            лидерами рынка" (bagrov.by)
 *   [habr]   "Как устроена Kimi K3: 2,8 трлн параметров, линейное внимание и агенты на миллион
 *            токенов" (savepearlharbor.com)
 *
 * The recurrence, per (sequence, head), with a fixed d_k x d_v state S (key channel = row):
 *     S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T,   o_t = scale * S_t^T q_t,
 *     alpha_t = exp(g_t) (one factor per key channel).
 * The state has a fixed size, each token partly erases what is stored along its key and writes
 * its value there, with write strength beta and forget factor alpha ([bagrov, § Как архитектура
 * Kimi K3 удерживает миллион токенов контекста]); the forget is per channel and acts before
 * the write ([habr, § Последовательность: три KDA на один глобальный MLA]).
 *
 * Conventions shared by every entry point
 *   - All tensor pointers are DEVICE memory owned by the caller; the library keeps no pointer
 *     after returning and allocates no device memory.
 *   - Tensors are contiguous, row-major:
 *       q, k, g, z : [B, T, H, d_k]          v, o : [B, T, H, d_v]          beta : [B, T, H]
 *       state      : [N, H, d_k, d_v] fp32 (row = key channel, d_v contiguous)
 *     Packed variable-length batches use B = 1, T = total tokens and device cu_seqlens[N+1].
 *     The decode step drops T.
 *   - Work is enqueued asynchronously on `stream` (a hipStream_t passed as void*; NULL = the
 *     default stream).  There is no host synchronisation and the host never reads device data.
 *     Buffers must stay alive until the stream has passed the work.  Segmented 16-bit prefills
 *     at d_k = d_v = 128 also run half of the heads on a second stream the library keeps per
 *     device (created on first use, never destroyed).  That stream starts after the work already
 *     on `stream` and `stream` waits for it before its next work, so the call's ordering on
 *     `stream` is as for a single stream.  kda_chunk_fwd_gated_noalloc never uses it.
 *   - Every call returns a kda_status; nothing is printed and nothing aborts.  Host-checkable
 *     argument errors are reported before any device work is enqueued.  Device-resident
 *     preconditions (g in [-5, 0], well-formed cu_seqlens) are the caller's contract and are not
 *     checked; violating them gives unspecified results but no out-of-bounds access: the
 *     kernels clamp every offset to 0 <= cu_seqlens[n] <= cu_seqlens[n+1] <= T before using it.
 *   - Debug check: with the environment variable KDA_DEBUG_VALIDATE set (to anything but "" or
 *     "0"), kda_chunk_fwd, kda_chunk_fwd_checkpointed and the three decode calls first test those
 *     preconditions on the device (kda_chunk_fwd_gated tests cu_seqlens only: its g is in range
 *     by construction; the linear-attention calls test g <= 0 and cu_seqlens, those of the selective
 *     scan A <= 0 and cu_seqlens, the convolution's cu_seqlens), wait for the answer
 *     on `stream` and return KDA_ERR_INVALID_ARGUMENT, with nothing else enqueued, on a violation.
 *     This synchronises the host, shares one word of library-owned device memory between all calls
 *     on a device (overlapping checked calls race on it) and must not be used under stream capture.
 *   - Calls are stateless and reentrant (the debug check aside).
 */
#ifndef KDA_H
#define KDA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { KDA_F32 = 0, KDA_BF16 = 1 } kda_dtype;

typedef enum {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARGUMENT = 1, /* null pointer, non-positive size, bad dtype, aliasing     */
    KDA_ERR_UNSUPPORTED = 2,      /* valid but not implemented: d_k/d_v not in {64,128}, ... */
    KDA_ERR_WORKSPACE = 3,        /* workspace smaller than kda_chunk_fwd_workspace_size()   */
    KDA_ERR_HIP = 4               /* a HIP runtime call or kernel launch failed              */
} kda_status;

/* Human-readable name of a status code (static storage; never NULL). */
const char *kda_status_string(int status);

/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
int kda_version(void);

/*
 * kda_gate -- forget-gate log-decay, [habr, § Последовательность]:
 *     g[t,h,c] = g_min * sigmoid(exp(A[h,c]) * z[t,h,c]),   sigmoid(x) = 1 / (1 + exp(-x)),
 * so alpha = exp(g) lies in [e^g_min, 1].  The pages fix g_min = -5; this bound is what keeps
 * every causal 16-token block of the chunked prefill inside the bf16/fp32 exponent range.
 *   A       : [H, d_k] fp32, device.
 *   z       : [n_tokens, H, d_k] in z_dtype (KDA_F32 or KDA_BF16), device.
 *   g       : [n_tokens, H, d_k] in g_dtype (KDA_F32 or KDA_BF16, round-to-nearest-even), device;
 *             must not overlap z or A.
 *   n_tokens: >= 0 (0 is a no-op); H, d_k >= 1.
 *   g_min   : must lie in [-5, 0); other values return KDA_ERR_UNSUPPORTED.
 * Precision (fp32 g): within 1.5 ulp of the exact value wherever |exp(A) z| <= 126 ln 2 (the
 * hardware exp2 of the rounded argument, 1 ulp, and a corrected quotient, 0.5 ulp; the argument's
 * rounding error is carried separately); beyond that g is g_min or below 2^-123 in magnitude.
 * z = 0 gives g_min / 2 exactly.  bf16 g is the fp32 value rounded.
 */
int kda_gate(const float *A, const void *z, int z_dtype, void *g, int g_dtype, int64_t n_tokens,
             int32_t H, int32_t dk, float g_min, void *stream);

/*
 * Workspace bytes kda_chunk_fwd needs for a batch of n_seqs sequences holding total_tokens tokens
 * (B*T for fixed-length batches) with inputs in in_dtype.  The prefill runs in two kernels: the
 * first computes, for every (head, 32-token record; 16 tokens for fp32 inputs), everything that
 * does not depend on the state and writes it to the workspace; the second passes the state
 * along each sequence reading it.  At d_k = 128 a record is 27.5 KiB for bf16 inputs (880 bytes
 * per token and head) and 26.5 KiB for fp32 inputs (16 tokens).  Long sequences with few
 * (sequence, head) units also need per-segment state buffers.  Batches of bf16 inputs at
 * d_k = d_v = 128 with n_seqs * H >= 256 run one fused kernel that builds the records on chip:
 * their size is 0 (a NULL workspace is accepted).
 * Never fails; returns 0 for invalid sizes (kda_chunk_fwd then reports the error).  The size is that of
 * these very numbers: fewer sequences may need more.
 */
size_t kda_chunk_fwd_workspace_size(int32_t n_seqs, int64_t total_tokens, int32_t H, int32_t dk,
                                    int32_t dv, int32_t chunk, int in_dtype);

/*
 * kda_chunk_fwd -- chunked prefill of the recurrence above over whole sequences.
 * Tokens inside a chunk are handled together and the state is carried from chunk to chunk
 * ([bagrov, § Уровень чипа: специализированное ядро FlashKDA]); with g >= -5 every causal
 * 16-token block, diagonal ones included, is a dense matrix product
 * ([habr, § Последовательность]).
 *   q, k, v, beta : inputs in in_dtype (KDA_F32 or KDA_BF16), layouts above.
 *   g             : [B, T, H, d_k] log-decay in g_dtype (KDA_F32 recommended; KDA_BF16 allowed),
 *                   values must lie in [-5, 0] (caller contract).
 *   initial_state : [N, H, d_k, d_v] fp32 or NULL (= zeros); never written unless it is also
 *                   final_state.
 *   final_state   : [N, H, d_k, d_v] fp32 or NULL; may equal initial_state (in-place update)
 *                   but must not partially overlap it.
 *   cu_seqlens    : NULL for B fixed-length sequences of T tokens (then n_seqs must equal B), or
 *                   device int32 [n_seqs + 1] offsets of a packed batch (then B must be 1,
 *                   cu_seqlens[0] = 0, non-decreasing, cu_seqlens[n_seqs] = T; caller contract).
 *                   Empty sequences are allowed: their final state is their initial state.
 *   o             : [B, T, H, d_v] in o_dtype (KDA_F32 or KDA_BF16); must not overlap any input.
 *   T             : >= 0 (T = 0 only copies initial_state to final_state, or zeroes it).
 *   dk, dv        : 64 or 128 each.  chunk: must be 64.  scale: any finite value (1 = none).
 *   workspace     : device buffer of at least kda_chunk_fwd_workspace_size(...) bytes, owned
 *                   by the caller; its contents on entry do not matter and on return are
 *                   unspecified.  It must not overlap any other argument.  Calls that share
 *                   a workspace must not overlap in time.
 * Results match the token-by-token definition up to rounding: the kernels evaluate the chunked
 * form with fp32 accumulation and split-precision matrix products.  Any finite input values are
 * accepted (beta included: the pages give it no range).  For bf16 inputs the state-pass operands
 * are staged in fp16, whose largest value is 65504: the results hold their tolerance while the
 * state, initial_state, v, scale * |q| * |k| and the entries of each 16-token block's UT
 * transform stay well inside that range.  The usual KDA inputs (q, k L2-normalised, beta in
 * [0, 1], the gate's decay) keep them below 10; the tests also cover beta in [-0.5, 1.5],
 * |q| = |k| = 3 with scale 4 and |v| about 30 (states to about 1000).  Keys with
 * beta * |k|^2 > 2 make the recurrence itself expansive along k (the transition scales that
 * direction by 1 - beta |k|^2 alpha), so long sequences of such inputs overflow any precision.
 * fp32 inputs use bf16 hi/lo splits throughout and have the fp32 range.
 */
int kda_chunk_fwd(const void *q, const void *k, const void *v, const void *beta, int in_dtype,
                  const void *g, int g_dtype, const float *initial_state, float *final_state,
                  const int32_t *cu_seqlens, void *o, int o_dtype, int32_t B, int64_t T,
                  int32_t n_seqs, int32_t H, int32_t dk, int32_t dv, int32_t chunk, float scale,
                  void *workspace, size_t workspace_bytes, void *stream);

/*
 * kda_chunk_fwd_gated -- kda_chunk_fwd with the forget gate fused in: takes the gate's inputs
 * A [H, d_k] fp32 and z [B, T, H, d_k] (z_dtype KDA_F32 or KDA_BF16) instead of g, and computes
 * g = g_min * sigmoid(exp(A) * z) on the fly ([habr, § Последовательность]) with the same
 * arithmetic as kda_gate, so that g never travels through memory.  The results equal
 * kda_gate followed by kda_chunk_fwd on an fp32 g bit for bit.  g_min must lie in [-5, 0)
 * (KDA_ERR_UNSUPPORTED otherwise); A and z must not overlap o, final_state or the workspace.
 * Every other argument, the workspace size and the error behaviour are those of kda_chunk_fwd.
 */
int kda_chunk_fwd_gated(const void *q, const void *k, const void *v, const void *beta,
                        int in_dtype, const float *A, const void *z, int z_dtype, float g_min,
                        const float *initial_state, float *final_state, const int32_t *cu_seqlens,
                        void *o, int o_dtype, int32_t B, int64_t T, int32_t n_seqs, int32_t H,
                        int32_t dk, int32_t dv, int32_t chunk, float scale, void *workspace,
                        size_t workspace_bytes, void *stream);

/*
 * kda_chunk_fwd_gated_noalloc -- kda_chunk_fwd_gated for callers that cannot allocate device
 * memory: code under HIP graph capture, tight serving loops, harnesses that forbid allocation.
 * It takes no workspace argument; the prefill's workspace is a static device array of
 * KDA_NOALLOC_SCRATCH_BYTES inside the library, which each GPU holds from the first call on it
 * until the process ends.  The call itself allocates nothing.
 *   Sizes: the call is refused with KDA_ERR_WORKSPACE, before any device work, when
 *   kda_chunk_fwd_workspace_size(n_seqs, B*T, H, dk, dv, 64, in_dtype) exceeds
 *   KDA_NOALLOC_SCRATCH_BYTES (256 MiB: e.g. 16-bit inputs with d_k = 128 up to about 290 K
 *   token-heads, such as 4 x 4096 tokens x 16 heads).
 *   Sharing: every call on one GPU uses that GPU's array.  Nothing in it has to start at zero and
 *   it keeps the last call's contents; calls that overlap in time on one GPU (another stream,
 *   another thread) race on it and must be serialised by the caller.
 *   Device: the array of the device `stream` belongs to (the current device for NULL) is used.
 * Every other argument, the results (equal to kda_chunk_fwd_gated's bit for bit) and the error
 * behaviour are those of kda_chunk_fwd_gated.
 */
#define KDA_NOALLOC_SCRATCH_BYTES ((size_t)256 << 20)
int kda_chunk_fwd_gated_noalloc(const void *q, const void *k, const void *v, const void *beta,
                                int in_dtype, const float *A, const void *z, int z_dtype,
                                float g_min, const float *initial_state, float *final_state,
                                const int32_t *cu_seqlens, void *o, int o_dtype, int32_t B,
                                int64_t T, int32_t n_seqs, int32_t H, int32_t dk, int32_t dv,
                                int32_t chunk, float scale, void *stream);

/*
 * kda_chunk_fwd_checkpointed -- the chunked prefill that also stores the state at fixed token
 * boundaries, for prefix caching: a later request that shares a prefix resumes from the stored
 * state (copy it, then continue) instead of recomputing the prefix ([habr, § Как обслуживать
 * два разных кеша]: the recurrent state is what such a cache keeps).
 *   A, g_or_z, gz_dtype, g_min : A non-NULL fuses the gate as kda_chunk_fwd_gated does (g_or_z
 *                   is z, g_min as there); A NULL makes g_or_z the log-decay g of kda_chunk_fwd
 *                   (g_min is then ignored).
 *   checkpoints   : fp32 device buffer [max_checkpoints, H, d_k, d_v] owned by the caller.
 *                   Checkpoint j >= 1 of sequence n is its state after its first
 *                   j * checkpoint_every tokens, for every j with j * checkpoint_every <= len_n
 *                   (the last one equals the final state when the length is a multiple); it goes
 *                   to slot base(n) + j - 1 with base(n) = n * floor(T / checkpoint_every) for
 *                   fixed-length batches and floor(cu_seqlens[n] / checkpoint_every) + n for
 *                   packed ones.  Slots no checkpoint maps to are left untouched.
 *   checkpoint_every : tokens between checkpoints, a positive multiple of 64 (the chunk).
 *   max_checkpoints  : slots in `checkpoints`; at least B * floor(T / checkpoint_every) for
 *                   fixed-length batches and floor(T / checkpoint_every) + n_seqs for packed ones.
 * A NULL buffer, a checkpoint_every that is not a positive multiple of 64, too few slots, or a
 * buffer that overlaps any other argument return KDA_ERR_INVALID_ARGUMENT.  Every other argument,
 * the workspace size and the error behaviour are those of kda_chunk_fwd; o and final_state equal
 * kda_chunk_fwd's (or kda_chunk_fwd_gated's) bit for bit.
 */
int kda_chunk_fwd_checkpointed(const void *q, const void *k, const void *v, const void *beta,
                               int in_dtype, const float *A, const void *g_or_z, int gz_dtype,
                               float g_min, const float *initial_state, float *final_state,
                               const int32_t *cu_seqlens, void *o, int o_dtype, int32_t B,
                               int64_t T, int32_t n_seqs, int32_t H, int32_t dk, int32_t dv,
                               int32_t chunk, float scale, float *checkpoints,
                               int32_t checkpoint_every, int64_t max_checkpoints, void *workspace,
                               size_t workspace_bytes, void *stream);

/*
 * kda_decode_step -- one token of the recurrence for N independent sequences, updating each
 * state in place.  One pass reads S once and writes it once: reading the large recurrent
 * state is this step's cost ([habr, § Как обслуживать два разных кеша]).
 *   q, k, g : [N, H, d_k]; v : [N, H, d_v]; beta : [N, H]; q, k, v, beta in in_dtype, g in g_dtype
 *             (KDA_F32 or KDA_BF16 each); g must lie in [-5, 0] (caller contract).
 *   state   : [N, H, d_k, d_v] fp32, read and overwritten in place.
 *   o       : [N, H, d_v] in o_dtype; must not overlap any input or the state.
 *   N >= 0 (0 is a no-op); H >= 1; dk, dv: 64 or 128 each.
 */
int kda_decode_step(const void *q, const void *k, const void *v, const void *beta, int in_dtype,
                    const void *g, int g_dtype, float *state, void *o, int o_dtype, int32_t N,
                    int32_t H, int32_t dk, int32_t dv, float scale, void *stream);

/*
 * Speculative decoding ([habr, § Как обслуживать два разных кеша]: no copy of the state is kept
 * per draft token; the accepted stretch is recomputed on chip from the token inputs, which is
 * cheaper than reading the large state again and again).  A draft of K tokens per sequence is
 * laid out like a prefill batch: q, k, g [N, K, H, d_k]; v [N, K, H, d_v]; beta [N, K, H]
 * (token j of sequence n is row (n*K + j)*H + h).
 *
 * kda_decode_verify -- runs all K draft tokens of every sequence from `state` (read only, never
 * written) and writes each token's output o [N, K, H, d_v] (o_dtype): the outputs K calls of
 * kda_decode_step would give, with one read of the state instead of K reads and writes.  Drafts
 * of up to 8 tokens are evaluated together from one pass over the state (the state after token
 * j is S_0 under the cumulative decay plus j rank-one terms); the first token's output equals
 * kda_decode_step's bit for bit, the others equal it up to fp32 rounding.  Longer drafts run
 * token by token and equal the step outputs bit for bit.  o must not overlap any other argument.
 *
 * kda_decode_commit -- once the draft has been checked, advances each state in place by its
 * accepted tokens: accepted is a device int32 [N] array of counts (values outside [0, K] are
 * clamped; 0 leaves the state untouched).  The same inputs are passed again; no o is produced.  The new
 * state equals accepted[n] successive kda_decode_step calls bit for bit.  The state must not
 * overlap any input or `accepted`.
 *
 * Both: dtypes, dimensions (d_k, d_v in {64, 128}), N >= 0 (0 is a no-op), K >= 1, H >= 1 and the
 * error behaviour as in kda_decode_step; the caller owns every buffer; work is enqueued on
 * `stream`.
 */
int kda_decode_verify(const void *q, const void *k, const void *v, const void *beta, int in_dtype,
                      const void *g, int g_dtype, const float *state, void *o, int o_dtype,
                      int32_t N, int32_t K, int32_t H, int32_t dk, int32_t dv, float scale,
                      void *stream);

int kda_decode_commit(const void *q, const void *k, const void *v, const void *beta, int in_dtype,
                      const void *g, int g_dtype, float *state, const int32_t *accepted, int32_t N,
                      int32_t K, int32_t H, int32_t dk, int32_t dv, void *stream);

/*
 * ---- Linear attention with one decay per head ------------------------------------------------
 * The recurrent sibling of KDA: the same d_k x d_v state per (sequence, head), which each token only
 * decays and adds to (no erase along the key, no per-channel gate):
 *     S_t = e^g S_{t-1} + k_t v_t^T,   o_t = scale * S_t^T q_t,
 * with g = g[h] <= 0 one log-decay per head, a constant of the model (0 = plain linear attention,
 * -inf = each token sees itself alone).  Layouts, streams, workspaces and errors are those stated at
 * the top of this file; further, for these calls and those of the state cache:
 *   - every tensor pointer must be aligned to 16 bytes except g, cu_seqlens, slots, scales (4)
 *     (KDA_ERR_UNSUPPORTED);
 *   - the stream must belong to the current device;
 *   - g is device memory and its sign the caller's contract, tested by KDA_DEBUG_VALIDATE;
 *     positive values grow the state instead of failing;
 *   - sizes (KDA_ERR_UNSUPPORTED past them): H <= 32768 and n_seqs * H <= 2^21 in the prefill and the
 *     gradients; N * H < 2^24 in the decode step; N * H * d_k * d_v < 2^36 in the state cache.
 * Inputs are finite numbers: besides what the formulas give it, an infinity or a NaN in one token may reach
 * o and dq of its sequence's tokens up to 64 before it, and dk and dv of those up to 64 after it (never
 * another sequence's).
 *
 * kda_linear_chunk_workspace_size -- workspace bytes of kda_linear_chunk_fwd (backward = 0) or
 * kda_linear_chunk_bwd (backward != 0) for n_seqs sequences of total_tokens tokens (B*T).  May be
 * 0 (a NULL workspace is then accepted).  Never fails; 0 for invalid sizes.  The size is that of these very
 * numbers: fewer tokens or sequences may need more.
 */
size_t kda_linear_chunk_workspace_size(int32_t n_seqs, int64_t total_tokens, int32_t H, int32_t dk,
                                       int32_t dv, int in_dtype, int backward);

/*
 * kda_linear_chunk_fwd -- chunked prefill of the recurrence above.
 *   q, k, v       : inputs in in_dtype (KDA_F32 or KDA_BF16), layouts at the top of this file.
 *   g             : [H] fp32 log-decay.
 *   initial_state, final_state, cu_seqlens, o, o_dtype, B, T, n_seqs, dk, dv, scale, workspace :
 *                   as in kda_chunk_fwd (T = 0 and empty sequences pass the state through).
 *   workspace     : at least kda_linear_chunk_workspace_size(..., 0) bytes.
 * Sums and states are fp32; bf16 inputs enter the products exactly, and values formed on the way
 * (the states, the decayed scores) as two or more bf16 terms, so that o is the fp32 result rounded
 * once to o_dtype (error of an fp32 o: about 1e-5 of its size for bf16 inputs) and the final state
 * holds fp32 accuracy.
 */
int kda_linear_chunk_fwd(const void *q, const void *k, const void *v, int in_dtype, const float *g,
                         const float *initial_state, float *final_state, const int32_t *cu_seqlens,
                         void *o, int o_dtype, int32_t B, int64_t T, int32_t n_seqs, int32_t H,
                         int32_t dk, int32_t dv, float scale, void *workspace,
                         size_t workspace_bytes, void *stream);

/*
 * kda_linear_chunk_bwd -- gradients of kda_linear_chunk_fwd.  With G_t the gradient of S_t
 * (G_T = d_final_state + scale q_T do_T^T, G_t = e^g G_{t+1} + scale q_t do_t^T):
 *     dq_t = scale * S_t do_t,   dk_t = G_t v_t,   dv_t = G_t^T k_t,   d_initial_state = e^g G_1.
 * The states are recomputed from q, k, v; nothing has to be kept from the forward call.  The decays
 * are constants: no gradient of g is formed.
 *   d_o             : [B, T, H, d_v] in in_dtype.
 *   d_final_state   : [N, H, d_k, d_v] fp32 or NULL (= zeros).
 *   dq, dk_out, dv_out : gradients of q, k, v, same shapes, in in_dtype.
 *   d_initial_state : [N, H, d_k, d_v] fp32 or NULL (not wanted).
 * No output may overlap an input, the workspace or another output; initial_state may be NULL
 * (= zeros).  workspace: at least kda_linear_chunk_workspace_size(..., 1) bytes.
 */
int kda_linear_chunk_bwd(const void *q, const void *k, const void *v, int in_dtype, const float *g,
                         const float *initial_state, const int32_t *cu_seqlens, const void *d_o,
                         const float *d_final_state, void *dq, void *dk_out, void *dv_out,
                         float *d_initial_state, int32_t B, int64_t T, int32_t n_seqs, int32_t H,
                         int32_t dk, int32_t dv, float scale, void *workspace,
                         size_t workspace_bytes, void *stream);

/*
 * kda_linear_decode_step -- one token of the recurrence for N independent sequences, each state
 * updated in place (read once, written once).
 *   q, k : [N, H, d_k]; v : [N, H, d_v] in in_dtype; g : [H] fp32; state : [N, H, d_k, d_v] fp32;
 *   o    : [N, H, d_v] in o_dtype; must not overlap any input or the state.
 *   N >= 0 (0 is a no-op).
 */
int kda_linear_decode_step(const void *q, const void *k, const void *v, int in_dtype,
                           const float *g, float *state, void *o, int o_dtype, int32_t N, int32_t H,
                           int32_t dk, int32_t dv, float scale, void *stream);

/*
 * ---- 8-bit state cache -------------------------------------------------------------------------
 * A pool of n_slots slots, each holding one sequence's states [H, d_k, d_v] as 8-bit codes with one
 * fp32 scale per group of `group` neighbouring value channels of a state row.  It keeps the states
 * a recurrent layer's prefix cache or scheduler puts aside ([habr, § Как обслуживать два разных
 * кеша]) -- final states, or the checkpoints of kda_chunk_fwd_checkpointed -- in about a quarter of
 * their fp32 size; KDA and linear-attention states alike.
 *   codes  : [n_slots, H, d_k, d_v], one byte each: KDA_CODE_I8 (signed integers -127 .. 127) or
 *            KDA_CODE_E4M3 (8-bit floats of 4 exponent and 3 mantissa bits, largest 448, no
 *            infinities).
 *   scales : [n_slots, H, d_k, d_v / group] fp32.
 *   group  : 32, 64 or 128, at most d_v.
 *   slots  : device int32 [N], the slot of each of the N sequences, or NULL (sequence n in slot n;
 *            then N <= n_slots is required).
 *
 * kda_state_store -- writes states [N, H, d_k, d_v] fp32 into their slots:
 *     scale = max|x| * (1 / M) (M = 127 or 448) over the group, each operation rounded to fp32;
 *     code = x / scale rounded to the nearest code, ties to even (the exact quotient, rounded once),
 *     at most M.
 * A group of zeros gets scale 0 and codes 0; a group with an infinity or a NaN gets a NaN scale and
 * codes 0, and reads back as NaN.  Sequences whose slot is outside [0, n_slots) are not stored; of
 * several sequences with one slot the last is.  Other slots are left as they were.
 *
 * kda_state_load -- states[n] = code * scale of slots[n] (fp32, rounded once); a slot outside
 * [0, n_slots) gives zeros, the state of a sequence without a cached prefix.
 */
typedef enum { KDA_CODE_I8 = 0, KDA_CODE_E4M3 = 1 } kda_code;

int kda_state_store(const float *states, const int32_t *slots, void *codes, int code,
                    float *scales, int32_t N, int32_t n_slots, int32_t H, int32_t dk, int32_t dv,
                    int32_t group, void *stream);

int kda_state_load(const void *codes, int code, const float *scales, const int32_t *slots,
                   float *states, int32_t N, int32_t n_slots, int32_t H, int32_t dk, int32_t dv,
                   int32_t group, void *stream);

/*
 * ---- Selective state space scan, short convolution, slot pools ---------------------------------
 * The recurrent sibling of linear attention whose decay and write strength come from the token, with the short
 * causal convolution that such layers run before it, and the management of the slots their states live in.  For
 * the calls from here to the end of this file:
 *   - Rows of tokens may be parts of wider rows: ldx, ldb, .. are the elements from one token's row to the next
 *     (at least a row's own; token t of sequence n of a fixed-length batch is row n * T + t), so that x, B and C can
 *     be read where one convolution wrote them side by side, and their gradients written the same way.  A stride
 *     may be up to 2^24 bytes (KDA_ERR_UNSUPPORTED past it).  States and windows are contiguous.
 *   - Outputs must not overlap inputs or one another (rows of one stride side by side do not).
 *   - The stream must belong to the current device.
 *   - The workspace sizes never fail, are 0 for arguments out of range, and never fall as sequences, tokens or slots
 *     grow within it: with the same heads, channels and types, a workspace for the largest call serves every smaller one.
 *   - Pools: where a call takes `slots` (device int32 [N]), sequence n works on slot slots[n] of an array of
 *     n_slots, or on slot n with slots NULL (then N <= n_slots is required).  A sequence whose slot lies outside
 *     [0, n_slots) -- a padded row of a batch -- is skipped and gets zeros for its output; of several with one slot
 *     only the last is carried out, and the others get zeros.
 *   - Rows of a packed batch that belong to no sequence (cu_seqlens[n_seqs] < T: a padded buffer) are left as they were.
 *     The debug check asks for cu_seqlens[n_seqs] == T and refuses them.
 *   - Inputs are finite numbers: an infinity or a NaN in one token may reach, besides what the formulas give it,
 *     outputs and gradients of its sequence's tokens up to 63 before and behind it; never another sequence's (the sums
 *     over tokens, dA and the like, aside).
 *
 * kda_conv_fwd -- short causal convolution of every channel (W = 2, 3 or 4 taps):
 *     u_t = bias + sum_i weight[c, i] x_{t - W + 1 + i},   y_t = u_t / (1 + e^-u_t) with silu, else u_t.
 *   x, y          : [B, T, C] in dtype (KDA_F32 or KDA_BF16), strides ldx, ldy.  Any C; four channels an access
 *                   where C, the strides and the addresses allow it, else single elements.
 *   weight, bias  : [C, W] fp32; [C] fp32 or NULL (= zeros).
 *   initial_state : [N, W - 1, C] in dtype, the inputs before a sequence's first token, or NULL (= zeros).
 *   final_state   : [N, W - 1, C] in dtype or NULL: the last W - 1 inputs (initial ones where a sequence is
 *                   shorter); must not overlap initial_state.
 *   cu_seqlens, B, T, n_seqs : as in kda_chunk_fwd.
 * Sums are fp32, y is rounded once.
 */
int kda_conv_fwd(const void *x, int64_t ldx, int dtype, const float *weight, const float *bias,
                 const void *initial_state, void *final_state, const int32_t *cu_seqlens, void *y,
                 int64_t ldy, int32_t B, int64_t T, int32_t n_seqs, int32_t C, int32_t W, int silu,
                 void *stream);

/*
 * kda_conv_bwd -- gradients of kda_conv_fwd, u recomputed from x.
 *   dy, d_final_state : gradients of y and of final_state (dtype; the latter NULL = zeros).
 *   dx, d_initial_state : in dtype; the latter NULL where it is not wanted.
 *   d_weight, d_bias  : [C, W], [C] fp32, written (not added to); d_bias NULL where it is not wanted.  Their sums over
 *                       the tokens have a fixed order.
 *   workspace     : at least kda_conv_bwd_workspace_size(...) bytes, aligned to 16 (KDA_ERR_WORKSPACE).
 */
size_t kda_conv_bwd_workspace_size(int32_t n_seqs, int64_t total_tokens, int32_t C, int32_t W);

int kda_conv_bwd(const void *x, int64_t ldx, int dtype, const float *weight, const float *bias,
                 const void *initial_state, const int32_t *cu_seqlens, const void *dy, int64_t lddy,
                 const void *d_final_state, void *dx, int64_t lddx, float *d_weight, float *d_bias,
                 void *d_initial_state, int32_t B, int64_t T, int32_t n_seqs, int32_t C, int32_t W,
                 int silu, void *workspace, size_t workspace_bytes, void *stream);

/*
 * kda_conv_step -- one token of N sequences: x, y [N, C] (strides ldx, ldy), windows [n_slots, W - 1, C] in dtype,
 * moved on by the token in place; slots as above.  N >= 0 (0 is a no-op).
 */
int kda_conv_step(const void *x, int64_t ldx, int dtype, const float *weight, const float *bias,
                  void *windows, const int32_t *slots, void *y, int64_t ldy, int32_t N, int32_t n_slots,
                  int32_t C, int32_t W, int silu, void *stream);

/*
 * kda_ssm_chunk_fwd -- chunked prefill of the selective scan.  Per head, with
 *     delta_t = softplus(dt_t + dt_bias),   a_t = e^(delta_t A):
 *     S_t = a_t S_{t-1} + delta_t B_t x_t^T,   y_t = S_t^T C_t + D x_t,
 * the state S as everywhere [d_k, d_v] (row = channel of B and C); head h uses B and C of group h / (H / G).
 *   x             : [B, T, H, d_v];  dt : [B, T, H];  Bm, Cm : [B, T, G, d_k], all in in_dtype, strides ldx, lddt,
 *                   ldb, ldc.  x, Bm, Cm, y: addresses and strides in steps of 16 bytes (KDA_ERR_UNSUPPORTED).
 *   A, dt_bias, D : [H] fp32; A <= 0 (caller contract, tested by KDA_DEBUG_VALIDATE); dt_bias, D may be NULL (= 0).
 *   initial_state, final_state : [N, H, d_k, d_v] fp32 or NULL; may be the same buffer.
 *   cu_seqlens, B, T, n_seqs   : as in kda_chunk_fwd.
 *   y             : [B, T, H, d_v] in y_dtype, stride ldy.
 *   H, G, dk, dv  : G divides H; dk, dv 64 or 128 each.  Sizes (KDA_ERR_UNSUPPORTED past them): H <= 32768,
 *                   (B * T / 128 + n_seqs) * H <= 2^21, B * T * G * dk <= 2^33.
 *   workspace     : at least kda_ssm_chunk_workspace_size(..., 0) bytes, aligned to 16 (may be 0).
 * Sums and states are fp32.  Decays between tokens come from fp64 sums over up to 64 tokens: steps delta_t |A| of 2^29 and
 * more would drown small ones beside them.  bf16 inputs enter the products exactly.  With them y reads states and
 * weighted scores as two bf16 terms each (2^-17 a term, error of an fp32 y: about 1e-6 of its size; fp32 inputs: 2e-7),
 * and is rounded once to y_dtype; the final state holds fp32 accuracy.
 */
size_t kda_ssm_chunk_workspace_size(int32_t n_seqs, int64_t total_tokens, int32_t H, int32_t G, int32_t dk,
                                    int32_t dv, int in_dtype, int backward);

int kda_ssm_chunk_fwd(const void *x, int64_t ldx, const void *dt, int64_t lddt, const void *Bm, int64_t ldb,
                      const void *Cm, int64_t ldc, int in_dtype, const float *A, const float *dt_bias,
                      const float *D, const float *initial_state, float *final_state,
                      const int32_t *cu_seqlens, void *y, int64_t ldy, int y_dtype, int32_t B, int64_t T,
                      int32_t n_seqs, int32_t H, int32_t G, int32_t dk, int32_t dv, void *workspace,
                      size_t workspace_bytes, void *stream);

/*
 * kda_ssm_chunk_bwd -- gradients of kda_ssm_chunk_fwd; the states are recomputed, nothing has to be kept from the
 * forward call.  With G_t the gradient of S_t (G_t = a_{t+1} G_{t+1} + C_t dy_t^T, behind the last token
 * d_final_state):
 *     dC_t = sum over the group's heads of S_t dy_t,      dB_t = sum over them of delta_t G_t x_t,
 *     dx_t = delta_t G_t^T B_t + D dy_t,                  dg_t = a_t <G_t, S_{t-1}>  (of the log-decay delta_t A),
 *     ddt_t = (x_t . G_t^T B_t + A dg_t) / (1 + e^-(dt_t + dt_bias)),   d_dt_bias = sum ddt_t,
 *     dA = sum delta_t dg_t,   dD = sum x_t . dy_t,       d_initial_state = a_1 G_1.
 *   dy, dx, ddt, dBm, dCm : in in_dtype, shaped as y, x, dt, Bm, Cm, strides lddy, lddx, ldddt, lddb, lddc.
 *   d_final_state : [N, H, d_k, d_v] fp32 or NULL (= zeros).
 *   dA, dD, d_dt_bias : [H] fp32, written; dD, d_dt_bias NULL where they are not wanted.  Sums have a fixed order.
 *   d_initial_state : [N, H, d_k, d_v] fp32 or NULL where it is not wanted.
 *   Sizes         : those of kda_ssm_chunk_fwd, and (B * T / c + n_seqs) * H < 2^22 - 8 with chunks of c = 64 tokens in
 *                   KDA_BF16, 32 in KDA_F32 (KDA_ERR_UNSUPPORTED past it).
 *   workspace     : at least kda_ssm_chunk_workspace_size(..., 1) bytes, aligned to 16: the states before, and their
 *                   gradients behind, every chunk, 8 d_k d_v bytes a head and chunk, are most of it.
 */
int kda_ssm_chunk_bwd(const void *x, int64_t ldx, const void *dt, int64_t lddt, const void *Bm, int64_t ldb,
                      const void *Cm, int64_t ldc, int in_dtype, const float *A, const float *dt_bias,
                      const float *D, const float *initial_state, const int32_t *cu_seqlens, const void *dy,
                      int64_t lddy, const float *d_final_state, void *dx, int64_t lddx, void *ddt,
                      int64_t ldddt, void *dBm, int64_t lddb, void *dCm, int64_t lddc, float *dA, float *dD,
                      float *d_dt_bias, float *d_initial_state, int32_t B, int64_t T, int32_t n_seqs,
                      int32_t H, int32_t G, int32_t dk, int32_t dv, void *workspace, size_t workspace_bytes,
                      void *stream);

/*
 * kda_ssm_decode_step -- one token of N sequences on a pool of states [n_slots, H, d_k, d_v] fp32, each read once and
 * written once; slots as above.  x [N, H, d_v], dt [N, H], Bm, Cm [N, G, d_k] in in_dtype, y [N, H, d_v] in y_dtype,
 * strides and alignments as in kda_ssm_chunk_fwd.  N >= 0 (0 is a no-op).
 */
int kda_ssm_decode_step(const void *x, int64_t ldx, const void *dt, int64_t lddt, const void *Bm, int64_t ldb,
                        const void *Cm, int64_t ldc, int in_dtype, const float *A, const float *dt_bias,
                        const float *D, float *state, const int32_t *slots, void *y, int64_t ldy, int y_dtype,
                        int32_t N, int32_t n_slots, int32_t H, int32_t G, int32_t dk, int32_t dv,
                        void *stream);

/*
 * Slot pools.  A pool is n_planes (1 to 4) device arrays of n_slots slots each -- states, 8-bit codes and scales,
 * convolution windows -- given by host arrays of their addresses (aligned to 16 bytes) and of the bytes of a slot
 * (any number; 16-byte accesses where 16 divides it).  refs (device int32 [n_slots], n_slots <= 2^20) counts the
 * users of each slot, 0 or less: free.  The calls keep refs; the host never reads it.
 *
 * kda_slots_copy -- dst[dst_slots[n]] = src[src_slots[n]] for N pairs between two pools that do not overlap (a batch's
 * states into a pool, or back).  NULL lists: pair n has slot n.  A source outside [0, n_src) gives zeros, a
 * destination outside [0, n_dst) is skipped, and of several pairs with one destination the last is taken.
 *
 * kda_slots_retain, kda_slots_release -- one user more or less of each listed slot, a slot listed k times k users; free
 * slots and numbers outside [0, n_slots) are left alone, and no count falls below 0.
 *
 * kda_slots_fork -- children[n] = a free slot (the lowest ones, in order; -1 where none is left) that from now on has
 * one user and the contents of slot parents[n]; zeros where the parent is free, lies outside [0, n_slots) or
 * parents is NULL (a new sequence's state).  Parents keep their users.
 *
 * kda_slots_compact -- moves the used slots together: with U of them, those from U on go to the free ones before U,
 * both in order, with their users.  *used = U (device int32).  table: n_table slot numbers (device int32, or NULL with
 * n_table 0) rewritten to where the slots are now, -1 for what named no used slot.
 *
 * workspace     : at least kda_slots_workspace_size(n_slots, N) bytes (compact: N = 0), aligned to 16.
 */
size_t kda_slots_workspace_size(int32_t n_slots, int32_t N);

int kda_slots_copy(const void *const *src, void *const *dst, const int64_t *slot_bytes, int32_t n_planes,
                   const int32_t *src_slots, const int32_t *dst_slots, int32_t N, int32_t n_src,
                   int32_t n_dst, void *stream);

int kda_slots_retain(int32_t *refs, const int32_t *slots, int32_t N, int32_t n_slots, void *stream);

int kda_slots_release(int32_t *refs, const int32_t *slots, int32_t N, int32_t n_slots, void *stream);

int kda_slots_fork(void *const *planes, const int64_t *slot_bytes, int32_t n_planes, int32_t *refs,
                   const int32_t *parents, int32_t *children, int32_t N, int32_t n_slots, void *workspace,
                   size_t workspace_bytes, void *stream);

int kda_slots_compact(void *const *planes, const int64_t *slot_bytes, int32_t n_planes, int32_t *refs,
                      int32_t *table, int64_t n_table, int32_t *used, int32_t n_slots, void *workspace,
                      size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H */
