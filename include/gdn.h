/*
 * gdn.h -- C ABI of libgdn, the Gated DeltaNet token mixer on one GB300 GPU.
 *
 * The mixer is the linear-attention layer of the Qwen3.5 / Qwen3.8 hybrid
 * decoders.  Per sequence b, per value head h, per token t it computes
 *
 *   1. u = silu(causal depthwise conv, width 4) on the q|k|v channels
 *        page "Qwen3.8-27B" (docs.theformalera.com), node gdn.conv:
 *        y[t,c] = silu( sum_{j<4} w[c,j] * x[t+j-3, c] ); tokens before the
 *        first come from the carried conv window.
 *   2. q^ = q / sqrt(sum q^2 + eps_l2) * q_scale,  k^ = k / sqrt(sum k^2 + eps_l2)
 *        page "How Qwen3.5 works" (azmle112.github.io), section 9.4; value
 *        head h reads key head h / (Hv / Hk) (integer division).
 *   3. S_t = e^{g_t} S_{t-1} (I - beta_t k^_t k^_t^T) + beta_t v_t k^_t^T,
 *      o_t = S_t q^_t
 *        node gdn.core of the same spec (S is Dv x Dk, "value rows");
 *        "How Qwen3.5 works" section 9.6 gives the decay -> predict ->
 *        correct -> read order, section 9.11 the chunked form used by
 *        gdn_prefill.
 *   4. y_t = norm_w * o_t / sqrt(mean(o_t^2) + eps_norm) * silu(z_t), per head
 *        node gdn.norm; "How Qwen3.5 works" section 9.9.
 *
 * Layouts (row-major, innermost last; C = 2*Hk*Dk + Hv*Dv conv channels,
 * ordered q (Hk heads) | k (Hk heads) | v (Hv heads)):
 *   qkv_pre [B][T][C]       z, o [B][T][Hv*Dv]      g, beta [B][T][Hv] (fp32)
 *   conv_w  [C][4]          norm_w [Dv]             S [B][Hv][Dv][Dk] (fp32)
 *   conv window [B][3][C]   raw (pre-conv) rows of the three previous tokens,
 *                           oldest first
 * "io" tensors (qkv_pre, z, o, conv windows, conv_w, norm_w) all have the
 * dtype shape->io_dtype; g, beta and the state are always fp32.
 *
 * Ownership and execution: every pointer is a device pointer owned by the
 * caller; the library allocates no memory, keeps no state between calls
 * (apart from a per-device error word, see gdn_device_status), and enqueues
 * its kernels on `stream` (a cudaStream_t; NULL = the legacy default stream)
 * without synchronising.  Calls on different streams do not share buffers.
 *
 * Errors: arguments are checked on the host before anything is launched; a
 * non-zero status means nothing was enqueued, except GDN_ERR_CUDA from the
 * launch itself.  Values are not checked: g must be <= 0 (finite, or -inf
 * for a reset) and beta in [0, 1]; other values give unspecified results
 * but stay within the buffers.
 *
 * Numeric domain of the bf16-io prefill (the chunked tensor-core kernels).
 * The products run on the tensor cores with fp16 operands and fp32
 * accumulation; the state itself stays fp32.
 *   - g below -80 acts as -80: a decay of e^-80 (about 1.8e-35) stands in for
 *     any smaller one, the reset g = -inf included.  Decode and the fp32-io
 *     kernels use e^g as given (e^-inf = 0).
 *   - Overflow: the fp16 copy of the state that multiplies W and q^, the
 *     chunk's Delta = U - W S (and Delta scaled by decay ratios <= 1) and W
 *     are converted without a range clamp, so |S|, |Delta| and |W| must stay
 *     below 65504; entries beyond it become inf.  Inputs (v, S0, the inverse
 *     T) are saturated to +-65504 instead.  Normalised q^ and k^ are <= 1.
 *   - Underflow: entries below 6.1e-5 in magnitude are fp16 subnormals
 *     (absolute spacing 6.0e-8), so where the state's entries are of order
 *     1e-4 and smaller, the products S W^T and S q^ carry them with fewer
 *     significant bits (the fp32 state and its update keep full precision).
 *   Tested against the fp64 oracle within the tolerances: qkv_pre scaled by
 *   1e-3 and by 30, initial states of rms 1e-4 and 10, g = -inf anywhere in
 *   a chunk, g down to -1e4, runs of beta = 0 and beta = 1.
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_ABI_VERSION 7

typedef enum {
  GDN_OK = 0,
  GDN_ERR_INVALID_ARG = 1,       /* null pointer, B < 1, T < 1, bad dtype or eps */
  GDN_ERR_UNSUPPORTED_SHAPE = 2, /* Dk or Dv != 128, Hv % Hk != 0, too large */
  GDN_ERR_ALIGNMENT = 3,         /* a pointer not 16-byte aligned */
  GDN_ERR_ALIAS = 4,             /* two buffers overlap where that is forbidden */
  GDN_ERR_CUDA = 5,              /* a CUDA runtime call failed */
  GDN_ERR_TIMEOUT = 6,           /* a device-side wait gave up (see gdn_device_status) */
  GDN_ERR_NO_DEVICE = 7,         /* the current device is not an sm_103 GPU */
  GDN_ERR_BOUNDS = 8             /* a device bounds check failed (GDN_CHECKS builds only) */
} gdn_status;

typedef enum { GDN_F32 = 0, GDN_BF16 = 1 } gdn_dtype;

typedef struct {
  int B;          /* sequences */
  int T;          /* tokens per sequence in this call (decode: 1) */
  int Hk, Hv;     /* key heads, value heads; Hv % Hk == 0 */
  int Dk, Dv;     /* head widths; the GPU kernels take 128 only */
  int io_dtype;   /* gdn_dtype of the io tensors */
  float eps_l2;   /* epsilon inside the q/k L2 root (1e-6 in the models) */
  float eps_norm; /* epsilon of the gated RMSNorm (1e-6 in the models) */
  float q_scale;  /* query scale after normalising; 0 means 1/sqrt(Dk) */
} gdn_shape;

/* GDN_ABI_VERSION of the loaded library. */
int gdn_abi_version(void);

/* A static, human-readable name for a status code. */
const char *gdn_status_str(int status);

/*
 * Prefill: run T tokens of B sequences through the mixer, carrying the state.
 *
 *   qkv_pre, z, g, beta      this call's tokens, layouts above
 *   conv_w, norm_w           layer weights
 *   S0     [B][Hv][Dv][Dk]   incoming state, or NULL for zeros
 *   conv0  [B][3][C]         incoming conv window, or NULL for zeros
 *   o      [B][T][Hv*Dv]     out: the mixer output (after the gated norm)
 *   S_T    [B][Hv][Dv][Dk]   out: final state; may be exactly S0 (in place),
 *                            must not otherwise overlap any buffer
 *   conv_T [B][3][C]         out: the last three raw rows of conv0 ++ qkv_pre;
 *                            must not overlap conv0 or qkv_pre
 *   o must not overlap any input.  All pointers 16-byte aligned.
 *
 * The chunked form ("How Qwen3.5 works" section 9.11, chunk 64) is used:
 * it is the same recurrence reorganised, so results match the token loop up
 * to rounding.  Continuing a prefill from (S_T, conv_T) equals one longer
 * prefill; a decode step is a prefill of one token.
 */
gdn_status gdn_prefill(const gdn_shape *shape, const void *qkv_pre, const void *z,
                       const float *g, const float *beta, const void *conv_w,
                       const void *norm_w, const float *S0, const void *conv0, void *o,
                       float *S_T, void *conv_T, void *stream);

/*
 * Decode: one new token for each of B sequences ("How Qwen3.5 works"
 * section 13.3: each linear layer updates its conv window and does one
 * recurrent step on the cached state).  shape->T must be 1.
 *
 *   qkv_pre [B][C], z [B][Hv*Dv], g and beta [B][Hv]    the new token
 *   S       [B][Hv][Dv][Dk]   the cached state, updated in place
 *   conv_in [B][3][C]         the cached window
 *   conv_out[B][3][C]         out: the new window; must not overlap conv_in
 *                             (callers ping-pong two buffers)
 *   o       [B][Hv*Dv]        out: the mixer output for the token
 */
gdn_status gdn_decode_step(const gdn_shape *shape, const void *qkv_pre, const void *z,
                           const float *g, const float *beta, const void *conv_w,
                           const void *norm_w, float *S, const void *conv_in, void *conv_out,
                           void *o, void *stream);

/*
 * Raw gate projections ("How Qwen3.5 works" section 9.5): per token and
 * value head the library forms, in fp32,
 *   beta = sigmoid(b),   g = -exp(A_log[h]) * softplus(a + dt_bias[h]).
 *   a, b            [tokens][Hv], io dtype (the outputs of the a and b
 *                   projections, same token order as z)
 *   A_log, dt_bias  [Hv] fp32 layer parameters
 */
typedef struct {
  const void *a, *b;
  const float *A_log, *dt_bias;
} gdn_raw_gates;

/*
 * Arguments of gdn_prefill_ex.  Exactly one gate source: (g, beta) or
 * raw_gates.  "tokens" is B*T for fixed-length sequences and T for packed
 * ones (below).
 *   qkv_pre [tokens][C]   z, o [tokens][Hv*Dv]   g, beta [tokens][Hv]
 *   S0, S_T, conv0, conv_T per sequence, as for gdn_prefill
 *   cu_seqlens  device int32 [B+1] or NULL.  When given, the B sequences are
 *               packed back to back ("varlen"): sequence s owns tokens
 *               cu_seqlens[s] .. cu_seqlens[s+1]-1 and shape->T is the total
 *               token count.  Each sequence starts from its own S0[s] and
 *               conv0[s] (or zeros); nothing flows between sequences.  A
 *               sequence of length 0 copies its incoming state and window.
 *               The offsets are read on the device: offsets that decrease
 *               or leave [0, T] make the kernel skip that sequence (its
 *               outputs stay untouched) and record GDN_ERR_INVALID_ARG for
 *               gdn_device_status.
 *   S_snap      [tokens][Hv][Dv][Dk] fp32 or NULL: the state after every
 *               token (for rollback; costs one state write per token).
 *   workspace   device scratch, 256-byte aligned, overlapping no other
 *               argument, or NULL; workspace_bytes says how large it is.
 *               Owned by the caller; its contents are undefined after the
 *               call and it must not be shared by calls that may run
 *               concurrently.  The chunked prefill takes the fastest form
 *               the workspace holds:
 *                 >= gdn_prefill_workspace_bytes(), and B * Hv (sequences x
 *                    value heads) below twice the GPU's SM count: the
 *                    chunk-parallel form (with more units the staged form
 *                    below already fills every SM, and moves fewer bytes).
 *                    q^ and k^ are formed once per key head (first kernel);
 *                    everything of a chunk that does not depend on the
 *                    carried state (the inverse T, U, W, the decayed
 *                    Q K^T) is formed for every chunk at once (second
 *                    kernel); a third kernel walks the chunks of each
 *                    (sequence, value head) with the state in TMEM, doing
 *                    only the state-dependent products, the state update
 *                    and the gated norm ("How Qwen3.5 works" section 9.11
 *                    separates exactly these two parts).
 *                 >= gdn_prefill_staged_bytes(): q^ and k^ once per key head
 *                    into the workspace, then one kernel per (sequence,
 *                    value head) for the rest.
 *                 smaller: GDN_ERR_INVALID_ARG.
 *               NULL: one kernel per (sequence, value head) does everything.
 *               All forms compute the same chunked recurrence; they differ
 *               in rounding order only.
 * bf16 io without snapshots (fixed length or packed) runs the chunked
 * tensor-core kernels; fp32 io and snapshots run the token-serial kernel,
 * which ignores the workspace.
 */
typedef struct {
  const void *qkv_pre, *z;
  const float *g, *beta;
  const gdn_raw_gates *raw_gates;
  const void *conv_w, *norm_w;
  const float *S0;
  const void *conv0;
  void *o;
  float *S_T;
  void *conv_T;
  const int *cu_seqlens;
  float *S_snap;
  void *workspace;
  size_t workspace_bytes;
} gdn_prefill_io;

/* Bytes of workspace of the chunk-parallel prefill for this shape (packed:
 * the call passes cu_seqlens, so the token rows are shape->T, else B*T):
 * the staged q^ and k^ (gdn_prefill_staged_bytes, rounded up to 256) plus
 * 57,860 bytes per (chunk slot, value head) -- U^T fp32 and -W^T fp16
 * [128][64], M fp16 [64][64], two fp32 vectors of 64 and a ready flag (the
 * two parts may run in one launch) -- where the chunk
 * slots are B * ceil(T/64) for fixed-length sequences and T/64 + B + 2 for
 * packed ones.  Where the work items would exceed 2^24 it returns the staged
 * size.  0 when the shape is invalid or the call would not run the chunked
 * kernels (fp32 io). */
size_t gdn_prefill_workspace_bytes(const gdn_shape *shape, int packed);

/* Bytes of workspace of the staged form alone: the q^ and k^ of every token
 * row and key head, 3 fp16 values per element (q^, and k^ as a hi/lo
 * pair).  0 as above. */
size_t gdn_prefill_staged_bytes(const gdn_shape *shape, int packed);

/* Prefill with the options above; aliasing and alignment rules as for
 * gdn_prefill (raw gates, cu_seqlens and S_snap count as inputs / outputs). */
gdn_status gdn_prefill_ex(const gdn_shape *shape, const gdn_prefill_io *io, void *stream);

/*
 * gdn_prefill_ex with no caller workspace and no allocation: the call runs
 * in a device scratch array that the library owns, one per device,
 * GDN_STATIC_SCRATCH_BYTES large, as gdn_prefill_ex would with a workspace
 * of that size (the chunk-parallel form where it fits, else the staged
 * form).  The pages have no counterpart; this is a serving convenience of
 * the library.
 *   io->workspace must be NULL (GDN_ERR_INVALID_ARG otherwise).
 *   A call whose staged need (gdn_prefill_staged_bytes) exceeds the scratch
 *   returns GDN_ERR_UNSUPPORTED_SHAPE before any launch.
 *   Nothing in the scratch has to start at zero: every byte a kernel reads
 *   there is written first by an earlier kernel of the same call.
 *   The scratch is shared by every call on the device: calls that overlap in
 *   time (different streams, or unordered host threads) race on it and give
 *   undefined results.  Issue them on one stream, or order them.
 *   The array is device memory of the library's own module; with lazy
 *   module loading (the CUDA default) it is allocated at the first call.
 */
#define GDN_STATIC_SCRATCH_BYTES (512ull << 20)
gdn_status gdn_prefill_static(const gdn_shape *shape, const gdn_prefill_io *io, void *stream);

/*
 * Arguments of gdn_decode_ex: shape->T >= 1 new tokens for each of B
 * sequences from the cached state, e.g. the draft tokens of speculative
 * decoding being verified ("How Qwen3.5 works" section 13).
 *   qkv_pre [B][T][C]   z, o [B][T][Hv*Dv]   g, beta [B][T][Hv] (or raw_gates)
 *   S        [B][Hv][Dv][Dk]     the cached state, updated in place (final state)
 *   S_snap   [B][T][Hv][Dv][Dk]  or NULL: the state after each token, so that a
 *                                caller who accepts only the first m tokens can
 *                                restore snapshot m-1
 *   conv_in, conv_out [B][3][C]  cached window in; window after the T tokens out
 *                                (must not overlap)
 * T <= 16 runs the decode kernel of gdn_decode_step (the state streamed once
 * through registers for all T tokens); longer runs use the token-serial
 * prefill kernel with the state in place.
 */
typedef struct {
  const void *qkv_pre, *z;
  const float *g, *beta;
  const gdn_raw_gates *raw_gates;
  const void *conv_w, *norm_w;
  float *S;
  float *S_snap;
  const void *conv_in;
  void *conv_out;
  void *o;
} gdn_decode_io;

gdn_status gdn_decode_ex(const gdn_shape *shape, const gdn_decode_io *io, void *stream);

/*
 * The projections around the mixer, nodes gdn.in_proj (K=5120 -> N=16480)
 * and gdn.out_proj (K=6144 -> N=5120) of the page "Qwen3.8-27B":
 *   y[t, n] = sum_k x[t, k] w[n, k],   t < M, n < N, k < K
 * bf16 inputs, fp32 accumulation on the tensor cores, bf16 outputs.  The
 * pages give the formula; the column routing is this library's: columns
 * [col_begin, col_end) of y are written to ptr[t * ld + (n - col_begin)],
 * so the in_proj output can land directly in the mixer's qkv_pre, z, b and a
 * buffers (columns 0-10239, 10240-16383, 16384-16431, 16432-16479 at the 27B
 * shape).
 *   x   [M][ldx] bf16, ldx >= K       w [N][ldw] bf16 (nn.Linear layout), ldw >= K
 *   ldx, ldw multiples of 8 (16-byte rows); x, w 16-byte aligned
 *   out[0 .. n_out-1], 1 <= n_out <= 4: disjoint column ranges inside [0, N),
 *   ld >= col_end - col_begin; output rows must not overlap x, w or each other
 * Columns not covered by any range are computed and dropped.
 */
typedef struct {
  int col_begin, col_end;
  void *ptr;
  long long ld;
} gdn_linear_out;

gdn_status gdn_linear(int M, int N, int K, const void *x, long long ldx, const void *w, long long ldw,
                      int n_out, const gdn_linear_out *out, void *stream);

/*
 * gdn_linear with an epilogue, for the projections around a linear-attention
 * mixer and the gated feed-forward behind it:
 *   p[t, n] = sum_k x[t, k] w[n, k] + bias[n]
 *   y[t, n] = act(p[t, n]) + residual[t, n]                 t < M, n < N
 * or, gated != 0, with w [2N][K] and bias [2N] (gate rows first, up rows after):
 *   y[t, n] = act(p[t, n]) p[t, N + n] + residual[t, n]
 * bf16 tensors, fp32 accumulation on the tensor cores; bias, activation,
 * product and residual in fp32, rounded once.
 *   x, w, ldx, ldw   as for gdn_linear
 *   bias             16-byte aligned, or NULL
 *   out[0 .. n_out-1], 1 <= n_out <= 4: disjoint ranges of the N output
 *     columns; each has its own activation and, or NULL, its own residual
 *     [M][ldr] whose column 0 is col_begin.  A residual may be exactly the
 *     range's output (same pointer and stride: y is then added in place).
 *     Otherwise outputs and residuals must not overlap, except as disjoint
 *     column blocks of one buffer (the same stride).
 * Columns not covered by any range are computed and dropped.
 */
typedef enum {
  GDN_ACT_NONE = 0,
  GDN_ACT_SILU = 1,    /* x sigmoid(x) */
  GDN_ACT_GELU = 2,    /* x Phi(x), in the tails to 2^-16 of itself */
  GDN_ACT_SIGMOID = 3
} gdn_activation;

typedef struct {
  int col_begin, col_end;
  void *ptr;
  long long ld;
  int act;              /* gdn_activation */
  const void *residual; /* or NULL */
  long long ldr;
} gdn_linear_ex_out;

gdn_status gdn_linear_ex(int M, int N, int K, int gated, const void *x, long long ldx, const void *w,
                         long long ldw, const void *bias, int n_out, const gdn_linear_ex_out *out, void *stream);

/* Which of its kernels gdn_linear_ex takes for these sizes on the current
 * device (residual != 0: some range has one), for tests that mean one. */
typedef enum {
  GDN_LINEAR_EX_PAIR = 0, /* tiles by pairs of CTAs */
  GDN_LINEAR_EX_TILE = 1, /* tiles of one CTA */
  GDN_LINEAR_EX_FEW = 2   /* few tokens or columns: the contraction over a cluster */
} gdn_linear_ex_kernel;

typedef struct {
  int kernel;      /* gdn_linear_ex_kernel */
  int tile;        /* output columns of a tile; FEW: tokens */
  long long tiles;
  int rows_w;      /* FEW: rows of w per tile, else 0 */
  int split;       /* FEW: CTAs of a cluster, else 0 */
} gdn_linear_ex_form;

gdn_status gdn_selftest_linear_ex_form(int M, int N, int K, int gated, int residual, gdn_linear_ex_form *form);

/*
 * Linear attention with a decay for each head ("How Qwen3.5 works" section
 * 9.1 gives the ungated form, section 9.6 the decay):
 *   S_t = e^{g_t} S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t
 * per sequence and value head (value head h reads key head h / (Hv / Hk)).
 * shape gives B, T, Hk, Hv, Dk = Dv = 128 and io_dtype; q_scale is `scale`
 * (0 means 1/sqrt(Dk)); the eps fields are not used.
 *   q, k [tokens][ldq], [tokens][ldk]   Hk heads of 128, io dtype
 *   v, o [tokens][ldv], [tokens][ldo]   Hv heads of 128, io dtype
 *        Rows may be further apart than they are wide (views of one fused
 *        buffer): ld >= heads * 128 elements, rows 16-byte aligned.
 *   g         [tokens][Hv] fp32 log decay per token, or NULL
 *   log_decay [Hv] fp32 constant log decay of a head, or NULL; exactly one of
 *        the two.  Values are <= 0; -inf resets the state (in chunks to
 *        within the bounds below).
 *   S0, S_T, cu_seqlens as for gdn_prefill_ex: S_T may be exactly S0; packed
 *        sequences of any length from 0; o must not overlap any other tensor.
 *   workspace 256-byte aligned scratch of at least
 *        gdn_linattn_workspace_bytes(), or NULL.  With few sequences x value
 *        heads it lets a prompt be cut into segments that run side by side.
 *        Undefined after the call; not to be shared by calls that may overlap
 *        in time.
 *
 * bf16 io runs in chunks of 64 tokens on the tensor cores (the shortest
 * prompts, up to about a hundred tokens, token by token as fp32 io does): operands that are
 * not bf16 already enter as sums of bf16 pieces (24 bits of what feeds the
 * state, 16 bits of what feeds o only), the state itself is summed in fp32.
 * Log decays below -80 act as -80 there: of a state that a reset should have
 * emptied e^-80 is left.  An output sees at least 2^-58 of the state at the
 * start of its chunk, also behind decays or a reset that should leave less of
 * it.  An output's sums carry the inverse of what has decayed since the start
 * of the chunk, 2^58 at most: where it is that, o / scale must stay below 2^69
 * in size.  None of this holds for the token loop.  q, k and v are finite: a NaN or
 * infinity spreads over its chunk and into the state (never into another
 * sequence).  A NaN log decay makes the outputs of its head from its token on
 * and the head's state NaN, whichever way the call runs.  fp32 io runs token
 * by token in fp32.
 */
typedef struct {
  const void *q, *k, *v;
  long long ldq, ldk, ldv, ldo;
  const float *g, *log_decay;
  const float *S0;
  void *o;
  float *S_T;
  const int *cu_seqlens;
  void *workspace;
  size_t workspace_bytes;
} gdn_linattn_io;

gdn_status gdn_linattn_prefill(const gdn_shape *shape, const gdn_linattn_io *io, void *stream);

/* Bytes of workspace of gdn_linattn_prefill for this shape on the current
 * device (packed: shape->T is the total token count); 0 where the call uses
 * none or the shape is invalid. */
size_t gdn_linattn_workspace_bytes(const gdn_shape *shape, int packed);

/* shape->T >= 1 new tokens for each of B sequences from the cached state:
 * io->S_T is the state, updated in place; io->S0, cu_seqlens and workspace
 * are NULL.  The state is read and written once, whatever T is. */
gdn_status gdn_linattn_decode(const gdn_shape *shape, const gdn_linattn_io *io, void *stream);

/* How gdn_linattn_prefill runs a shape on the current device (packed as for
 * gdn_linattn_workspace_bytes; workspace != 0: the call has one), for tests
 * that mean one form. */
typedef struct {
  int chunked;  /* 1: in chunks on the tensor cores, 0: token by token */
  int segments; /* of a sequence, side by side */
  int parts;    /* of a segment, in the launch that forms the states between them */
} gdn_linattn_form;

gdn_status gdn_selftest_linattn_form(const gdn_shape *shape, int packed, int workspace, gdn_linattn_form *form);

/*
 * Softmax attention over a paged cache in 8 bits: the layer of the hybrid
 * decoders that stands between the linear ones (page "Qwen3.8-27B": pages of 16
 * tokens; "How Qwen3.5 works" sections 10 and 13), from the output of its
 * in-projection to the input of its out-projection.
 *
 * The cache of a layer: n_pages pages of `page` tokens (16, 32, 64 or 128)
 *   k, v       [n_pages][Hk][page][D] e4m3 (1 sign, 4 exponent and 3 fraction
 *              bits, bias 7): the value byte * scale
 *   k_scale, v_scale [n_pages][Hk] fp32: the scale of a page and head
 * and where the sequences lie in it
 *   block_table [B][table_ld] int32: token t of sequence b is row t % page of
 *              page block_table[b][t / page]; max_blocks entries of a row count
 *   kv_lens    [B] int32: the tokens of each sequence, those of the call included
 * D is 64, 128 or 256.  Pages may be shared by sequences that only read them.
 *
 * The new tokens of a call: fixed length, sequence b owns token rows b*T ..
 * b*T+T-1 and T tokens are new; packed, rows cu_seqlens[b] .. cu_seqlens[b+1]-1
 * of T rows (rows behind cu_seqlens[B] are neither read nor written).  They are
 * the last of the sequence: row i of n is at position kv_lens[b] - n + i.
 *   max_new   packed: no sequence has more new tokens (0: T)
 *   max_kv    no sequence has more tokens in all (0: max_blocks * page)
 * Lengths and tables are read on the device.  A sequence with more tokens than
 * max_new, max_kv or its table allow is skipped (its outputs stay untouched); with
 * offsets out of order or range all are; an entry of the table that is used and
 * is not a page of the cache is left out.  Each records GDN_ERR_INVALID_ARG for
 * gdn_device_status.
 * B <= 65536, 2^24 token rows, Hq <= 4096, 2^27 pages, max_blocks * page <= 2^30.
 */
typedef struct {
  int B, T;
  int Hq, Hk;     /* query heads, key heads; Hq % Hk == 0, at most 64 query heads to a key head, Hk <= 1024 */
  int D;
  int io_dtype;   /* gdn_dtype of q, k, v and o */
  int max_new, max_kv;
} gdn_attn_shape;

typedef struct {
  void *k, *v;
  float *k_scale, *v_scale;
  int n_pages, page;
  const int *block_table;
  long long table_ld;
  int max_blocks;
  const int *kv_lens;
} gdn_kv_cache;

/*
 * New keys and values into the cache: k, v [rows][ldk], [rows][ldv], Hk heads
 * of D, rows 16-byte aligned.  Hq is not used.
 *   The scale of a page and head is the smallest power of two s with |x| <= 448 s
 *   for the page's new tokens, at least 2^-120 and at most 2^7 (larger values
 *   are stored as +-57344), and never below the one it has where the page holds
 *   older tokens of the sequence; where it grows, those are rounded anew.  A
 *   byte is x / s rounded to nearest, ties to even.
 *   A NaN or infinity among a page's new tokens makes the scale of that page
 *   and head NaN (the new bytes are 0).
 *   Rows of a page behind the sequence's end keep what they hold.
 *   A page that is written belongs to one sequence, once: where the table gives
 *   it to two, or twice to one, what is written there is not specified.
 */
typedef struct {
  const void *k, *v;
  long long ldk, ldv;
  const int *cu_seqlens; /* or NULL: fixed length */
  gdn_kv_cache cache;
} gdn_kv_append_io;

gdn_status gdn_kv_append(const gdn_attn_shape *shape, const gdn_kv_append_io *io, void *stream);

/*
 * Attention of the new tokens over the cache (which holds their keys and values
 * already):  o_i = sum_j p_ij v_j,  p_ij = softmax over j of scale q_i . k_j,
 * query head h with key head h / (Hq / Hk).
 *   q, o [rows][ldq], [rows][ldo]   Hq heads of D, io dtype, 16-byte rows; o overlaps
 *     no input (but q as disjoint column blocks of one buffer: the same stride)
 *   causal != 0: row i at position p sees tokens 0 .. p; 0: it sees all
 *     kv_lens[b] (an encoder's states, say).  A row that sees none gives 0.
 *   scale   0 means 1/sqrt(D)
 *   workspace 256-byte aligned scratch of gdn_attn_workspace_bytes(), or NULL;
 *     with it the tokens of long sequences are spread over the GPU where there
 *     are few rows.  Undefined after the call; not to be shared by calls that
 *     may overlap in time.
 * What the cache holds behind a row's last token does not reach it, whatever it
 * is, but for its page's scales: a row that sees a token of a page whose k or
 * v scale is NaN gives NaN.  Scales are 0 <= s <= 2^7 (below 2^-126 they may count
 * as 0).  The bytes of a sequence's kv_lens tokens hold no NaN (0x7f, 0xff;
 * gdn_kv_append writes none): with one there, what its rows give, those before
 * that token too, is not specified.
 * bf16 io: products on the tensor cores, of the bytes themselves, of q (for many
 * rows to within 2^-17 of the largest of its row and head) and of p rounded to
 * fp16; scores, softmax and sums in fp32.  p has its page's value scale with it
 * there: 11 bits down to 2^-25 of the largest product of a weight and its scale that
 * the row has seen, and what is smaller to within 2^-36 of that.  Weights below
 * 2^-120 of the row's largest, and rows whose products are all below 2^-120 of it, may
 * count as 0.  fp32 io: fp32 throughout.  A NaN or infinity in a head of q makes
 * that row and head NaN.
 * max_new and max_kv choose how the call runs: a few rows (new tokens x Hq / Hk) of
 * each sequence and key head side by side, or tiles of 128 rows.  A batch of
 * prompts and of single tokens is faster as two calls.
 */
typedef struct {
  const void *q;
  void *o;
  long long ldq, ldo;
  const int *cu_seqlens; /* or NULL: fixed length */
  gdn_kv_cache cache;
  int causal;
  float scale;
  void *workspace;
  size_t workspace_bytes;
} gdn_attn_io;

gdn_status gdn_attn(const gdn_attn_shape *shape, const gdn_attn_io *io, void *stream);

/* Bytes of workspace that do for gdn_attn of this shape on the current device (packed
 * as for gdn_linattn_workspace_bytes), and for every call of the same heads, type and
 * form, packed or not, with no more sequences, tokens, new tokens (max_new) and tokens in
 * all (max_kv): sized for the largest batch it serves the smaller ones.  0 where the
 * shape is invalid or none of these calls uses any.  gdn_attn refuses a workspace that is
 * smaller than what the call at hand would use. */
size_t gdn_attn_workspace_bytes(const gdn_attn_shape *shape, int packed);

/* How gdn_attn runs a shape on the current device (packed as above; workspace !=
 * 0: the call has one; max_kv 0 stands for long sequences), for tests that mean one form. */
typedef enum {
  GDN_ATTN_ROWS = 0, /* fp32 arithmetic (fp32 io) */
  GDN_ATTN_FEW = 1,  /* bf16, few rows: work cut evenly over the GPU */
  GDN_ATTN_TILE = 2  /* bf16, tiles of 128 rows */
} gdn_attn_kernel;

typedef struct {
  int kernel; /* gdn_attn_kernel */
  int rows;   /* of a tile */
  int parts;  /* ranges of the tokens side by side (TILE: of the last blocks, or all); FEW: 0, they follow from the lengths */
} gdn_attn_form;

gdn_status gdn_selftest_attn_form(const gdn_attn_shape *shape, int packed, int workspace, gdn_attn_form *form);

/*
 * Rotary positions on the first `rot` elements of every head ("How Qwen3.5
 * works" section 10: 64 of 256).  The pair (a, b) of index i at position p
 * becomes m (a cos x - b sin x, b cos x + a sin x), x = p f_i.
 *   GDN_ROPE_HALF         the pair is elements i and i + rot/2
 *   GDN_ROPE_INTERLEAVED  elements 2i and 2i + 1
 * gdn_rope_plan_init fills a plan on the host (no GPU is needed):
 *   GDN_ROPE_PLAIN   f_i = base^(-2i/rot), m = 1
 *   GDN_ROPE_LINEAR  f_i / factor
 *   GDN_ROPE_NTK     base * factor^(rot/(rot-2)) in the place of base (rot > 2)
 *   GDN_ROPE_PARTS   pairs that turn more than `fast` times over the `original`
 *                    context keep f_i, those that turn less than `slow` times
 *                    take f_i / factor, a ramp over the pairs between lies
 *                    between the two: with c(n) = rot ln(original / (2 pi n)) /
 *                    (2 ln base) it goes from max(floor(c(fast)), 0) to
 *                    min(ceil(c(slow)), rot - 1), and m = 0.1 ln(factor) + 1.
 *                    (Peng et al., arXiv 2309.00071, sections 3.2 and 3.4)
 * Other frequencies: write turns and m into the plan.  turns[i] is f_i / (2 pi),
 * modulo 1, times 2^64: the angle of any 32-bit position is p * turns[i] modulo
 * 2^64, a product that rounds nothing.  gdn_rope_plan_init has f_i as a double, to
 * within a few 2^-53: times p that is below 2^-36 of a turn at p = 2^17, some 10^-7 at
 * 2^31.
 */
typedef enum { GDN_ROPE_HALF = 0, GDN_ROPE_INTERLEAVED = 1 } gdn_rope_layout;
typedef enum { GDN_ROPE_PLAIN = 0, GDN_ROPE_LINEAR = 1, GDN_ROPE_NTK = 2, GDN_ROPE_PARTS = 3 } gdn_rope_scaling;

#define GDN_ROPE_MAX_PAIRS 128
typedef struct {
  int rot;     /* even, 2 .. 256 */
  int layout;  /* gdn_rope_layout */
  float m;
  unsigned long long turns[GDN_ROPE_MAX_PAIRS];
} gdn_rope_plan;

typedef struct {
  int rot, layout, scaling;  /* scaling: gdn_rope_scaling */
  double base, factor;       /* base > 1, factor >= 1 */
  double original, fast, slow; /* GDN_ROPE_PARTS only: original > 0, fast > slow > 0 */
} gdn_rope_spec;

gdn_status gdn_rope_plan_init(const gdn_rope_spec *spec, gdn_rope_plan *plan);

/*
 *   positions  [tokens] int32, any values
 *   x[0 .. n_x-1], 1 <= n_x <= 4: q, k and the like, [tokens] rows of `heads`
 *     heads of D elements, ld* elements apart, io dtype.  y may be exactly x
 *     (the same pointer and stride: turned in place, the other D - rot elements
 *     of a head are not touched); otherwise it must not overlap any x or y
 *     (but as disjoint column blocks of one buffer: the same stride) and takes
 *     whole heads.
 *   D: rot .. 1024.  Elements are aligned to their own size only; heads of
 *     16-byte alignment run faster.
 *   inverse != 0: turns back (by -x), times m all the same: the gradient of
 *     the forward call.
 */
typedef struct {
  const void *x;
  void *y;
  long long ldx, ldy;
  int heads;
} gdn_rope_x;

gdn_status gdn_rope(int tokens, int D, int io_dtype, const gdn_rope_plan *plan, const int *positions, int n_x,
                    const gdn_rope_x *x, int inverse, void *stream);

/*
 * Block tables and slot maps, on the GPU: pages for the new tokens of B requests.
 *   kv_lens     [B] int32: tokens cached so far
 *   new_tokens  [B] int32: tokens to come, 0 or more
 *   free_pages  [n_free] int32: pages to hand out, the first free_used[0] are gone
 *   block_table [B][table_ld] int32, max_blocks entries of a row: of request b the
 *               entries from ceil(kv / page) to ceil((kv + new) / page) - 1 get
 *               the next free pages (in order: requests, then blocks); the others
 *               are not written
 *   kv_lens_out [B], free_used_out [1]: kv + new, and the count moved on; each may
 *               be exactly the buffer it comes from
 *   cu_seqlens  [B + 1]: out: the offsets of the requests' new tokens
 *   slots       [max_tokens] int64 or NULL: page * page size + row of each new
 *               token; -1 behind the last one
 *   positions   [max_tokens] int32 or NULL: its position; 0 behind the last one
 * All or nothing: where a count is negative, a request would need more than
 * max_blocks, the pages do not suffice or there are more than max_tokens new
 * tokens, the call records GDN_ERR_INVALID_ARG for gdn_device_status, hands out
 * nothing, and leaves cu_seqlens all 0, every slot -1, kv_lens_out and
 * free_used_out as if no token were new (the other calls then have nothing to do).
 * An entry of the table that is already there is not checked.
 * page: 16, 32, 64 or 128; n_free may be 0; B <= 16384, max_tokens <= 2^30.
 */
typedef struct {
  int B, page, max_blocks, n_free;
  long long table_ld, max_tokens;
  const int *kv_lens, *new_tokens, *free_pages, *free_used;
  int *block_table, *kv_lens_out, *free_used_out, *cu_seqlens;
  long long *slots;
  int *positions;
} gdn_kv_pages_io;

gdn_status gdn_kv_pages(const gdn_kv_pages_io *io, void *stream);

/*
 * Synchronise `stream` and report device-side failures recorded since the
 * last reset: GDN_ERR_TIMEOUT if a kernel's bounded wait gave up (the kernel
 * then returned early and its outputs are incomplete), GDN_ERR_BOUNDS if a
 * store failed its bounds check (only in a library built with GDN_CHECKS,
 * where every thread-issued global store of the prefill and decode kernels
 * is checked against its buffer and skipped when outside it),
 * GDN_ERR_INVALID_ARG if a kernel met packed-sequence offsets it could not
 * use, GDN_ERR_CUDA if the synchronisation itself failed, GDN_OK otherwise.  reset != 0 clears the
 * record afterwards.  The record is one word per device, shared by all
 * streams.
 */
gdn_status gdn_device_status(void *stream, int reset);

/*
 * Failure-detection self-test; the pages have no counterpart (they describe
 * no kernels).  Enqueues one CTA that takes the same steps as a prefill
 * kernel whose awaited work never completes: it allocates TMEM, waits on an
 * mbarrier that nothing arrives on with the bounded wait the prefill kernel
 * uses, here limited to `wait_us` microseconds (1 .. 1000000), records the
 * timeout in the device error word, frees its TMEM and returns.  Afterwards
 * gdn_device_status reports GDN_ERR_TIMEOUT and the context stays usable.
 * Nothing is allocated and no caller buffer is touched.
 * Errors: GDN_ERR_INVALID_ARG for wait_us out of range, GDN_ERR_NO_DEVICE,
 * GDN_ERR_CUDA from the launch.
 */
gdn_status gdn_selftest_wait_timeout(int wait_us, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H */
