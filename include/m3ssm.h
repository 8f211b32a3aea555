/*
 * m3ssm.h -- C ABI of the Mamba-3 SSM core for AMD Instinct MI355X (gfx950).
 *
 * The operation (sources are web pages on Mamba-3, cited by title/section):
 *   "Znakomstvo s Mamba-3" (chernovdev.ru), sec. 1, the displayed recurrence:
 *       h_t = alpha_t h_{t-1} + beta_t B_{t-1} x_{t-1}^T + gamma_t B_t x_t^T,
 *       alpha_t = exp(Delta_t A), beta_t = (1 - lambda_t) Delta_t alpha_t,
 *       gamma_t = lambda_t Delta_t;
 *   same page, sec. 2: complex dynamics as data-dependent cumulative RoPE on
 *       B and C (angles aggregated over all time steps);
 *   same page, sec. 3, and "La dualita: Mamba-2 e Mamba-3" (book.paithon.it),
 *       sec. "Mamba-3": rank-R MIMO, B_t, C_t in R^{N x R}, x_t in R^{P x R},
 *       the update is a sum of R outer products on an unchanged N x P state;
 *   "La dualita", sec. "State Space Duality" / "Perche conviene": the chunked
 *       evaluation (intra-chunk masked product, chunk states, inter-chunk
 *       recurrence, readout of the previous state).
 *
 * Conventions fixed by this library (the pages leave them open):
 *   - Rotation pairs are adjacent state entries (2j, 2j+1).  With the inclusive
 *     cumulative angle Phi_t = Phi_{-1} + sum_{s<=t} theta_s, the kernels use
 *     Btil = R(Phi)^T B and Ctil = R(Phi)^T C, R(phi) = [[cos,-sin],[sin,cos]].
 *   - y_t[r] = h_t^T Ctil_t[r] (state after the update, no skip term).
 *   - The carried previous-token term uses the previous token's rotated B.
 *   - The state h is the real state in the rotated frame, fp32, [N][P] per head.
 *
 * Layouts: every tensor is dense row-major (C order), innermost dimension
 * last, with the shapes given below.  Base pointers of x, B, C, y, xprev,
 * xprev_out, h0, h_final, h, Bprev_rot, Bprev_rot_out must be 16-byte
 * aligned; theta / phi pointers must be 16-byte aligned.
 * All pointers are device pointers (hipMalloc'd or equivalent) unless noted.
 * The caller owns every buffer, including the optional prefill workspace; the
 * library allocates nothing.  Between calls it keeps only per-device caches,
 * each safe under concurrent first calls from several host threads: the
 * compute-unit count (atomics), which kernels have had their dynamic-LDS
 * limit raised (an atomic bit mask per kernel) and the address of the
 * no-allocation scratch (under a mutex).  Calls on different streams are
 * independent given separate workspaces (m3_ssm_prefill_noalloc shares its
 * scratch per device).
 * `stream` is a hipStream_t (NULL = the null stream).  All calls are
 * asynchronous with respect to the host; results are visible after the
 * stream is synchronised.  Results are deterministic (no atomics).
 *
 * Errors: every entry point validates its arguments on the host before any
 * launch and returns a negative m3_status without touching the GPU when they
 * are invalid.  No exception crosses the ABI.
 */
#ifndef M3SSM_H
#define M3SSM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum m3_status {
  M3_OK = 0,
  M3_ERR_INVALID_ARG = -1, /* null required pointer, bad size, misalignment  */
  M3_ERR_UNSUPPORTED = -2, /* shape/dtype outside the compiled kernel tiles  */
  M3_ERR_HIP = -3,         /* a HIP launch or runtime error was reported     */
  M3_ERR_SCRATCH = -4      /* m3_ssm_prefill_noalloc: the call needs more
                              scratch than M3_NOALLOC_SCRATCH_BYTES          */
} m3_status;

typedef enum m3_dtype {
  M3_F32 = 0,  /* IEEE float32 */
  M3_BF16 = 1  /* bfloat16 stored as uint16 bit patterns */
} m3_dtype;

/* Order of the token and head axes of the prefill's x, B, C and y. */
typedef enum m3_layout {
  M3_TOKEN_MAJOR = 0, /* [Bt, L, H, R, .] (the default) */
  M3_HEAD_MAJOR = 1   /* [Bt, H, L, R, .]: each head's rows one contiguous run */
} m3_layout;

/*
 * Prefill (chunked, whole sequence per (batch, head)).
 *
 *   x       [Bt, L, H, R, P]  in_dtype   inputs x_t (R columns of length P)
 *   B, C    [Bt, L, H, R, N]  in_dtype   input / output projections
 *   dt      [Bt, L, H]        float32    Delta_t (> 0, already positive)
 *   lam     [Bt, L, H]        float32    lambda_t in [0, 1]
 *   A       [H]               float32    per-head scalar A (< 0); may be NULL
 *                                        when A_tok is given
 *   A_tok   [Bt, L, H]        float32    A per token (< 0), or NULL: the decay
 *                                        rate itself depending on the token
 *                                        ("La dualita", sec. "Mamba-3");
 *                                        alpha_t = exp(Delta_t A_tok_t)
 *   theta   [Bt, L, H, N/2]   float32    per-token rotation angles, or NULL
 *                                        for the real-valued SSM (no RoPE)
 *   omega   [Bt, L, N/2]      float32    alternative to theta: rotation
 *                                        rates per token and pair, shared by
 *                                        all heads; the angle
 *                                        is then theta_t = Delta_t * omega_t
 *                                        (the step times the rate, per head),
 *                                        formed on chip, which saves reading
 *                                        the per-head theta tensor.  Setting
 *                                        both theta and omega is
 *                                        M3_ERR_INVALID_ARG.
 *   Carry-in, each nullable (NULL = zeros, i.e. a fresh sequence):
 *   h0        [Bt, H, N, P]   float32    state before the first token
 *   Bprev_rot [Bt, H, R, N]   float32    rotated B of the token before
 *   xprev     [Bt, H, R, P]   in_dtype   x of the token before
 *   phi0      [Bt, H, N/2]    float32    cumulative angle before the first token
 *   Outputs:
 *   y         [Bt, L, H, R, P] in_dtype  required
 *   h_final   [Bt, H, N, P]   float32    state after token L-1 (nullable)
 *   Bprev_rot_out [Bt,H,R,N]  float32    rotated B_{L-1} (nullable)
 *   xprev_out [Bt, H, R, P]   in_dtype   x_{L-1} (nullable)
 *   phi_out   [Bt, H, N/2]    float32    Phi_{L-1} reduced modulo 2*pi into
 *                                        [-pi, pi] (nullable; needs theta or
 *                                        omega)
 * Sizes: Bt, L, H >= 1; N, P in {16, 32, 64, 128}; R a power of two <= 64;
 * combinations whose chunk tiles exceed the 160 KB LDS of a CU return
 * M3_ERR_UNSUPPORTED (fp32 with RoPE at N = 128, and fp32 at N = P = 128);
 * chunk = tokens per chunk Q of the chunked evaluation, 0 selects 64 / R.
 * A chunk tile holds 64 (token, rank) rows: the bf16 path takes only
 * Q = 64 / R; the fp32 path also any smaller power of two (the tile's rows
 * past Q R then stay empty).  Results do not depend on Q beyond rounding.
 * Outputs must not alias inputs.  Passing the carry-out of one call as the
 * carry-in of the next continues the sequence exactly.
 * workspace: optional, see m3_ssm_prefill_workspace_size; a non-NULL
 * workspace smaller than that size (or not 256-byte aligned) is
 * M3_ERR_INVALID_ARG.
 * layout: M3_TOKEN_MAJOR (0, the shapes above) or M3_HEAD_MAJOR (1): x, B, C
 * and y as [Bt, H, L, R, .] (dt, lam, A_tok, theta and omega keep the shapes
 * above).  The arithmetic is the same, so both layouts give identical bits;
 * head-major reads each (batch, head) walk as one contiguous run.  Other
 * values are M3_ERR_INVALID_ARG.
 * Prologue (optional steps fused in front of the core; all off when zero /
 * NULL), see m3_prologue below: the B and C given are then the raw
 * projections and dt the raw step.
 */
/*
 * The steps just before the SSM core, computed on chip ("Znakomstvo s
 * Mamba-3" (chernovdev.ru), sec. "Architecture and normalisation": RMS
 * normalisation of the B and C projections, by analogy with QK normalisation,
 * then learnable head-specific biases added to B and C after it; "Mamba-3:
 * un modello a spazio di stato progettato per l'inferenza" (cartesia.ai),
 * "Normalizzazioni" and "Addio convoluzione corta"):
 *   bc_norm      0 or 1: each (token, head, rank) row of B and of C, an
 *                N-vector, becomes row / sqrt(mean(row^2) + bc_eps) times the
 *                gain B_norm_w / C_norm_w [N] (NULL = 1); a row of zeros stays
 *                zero.  bc_eps >= 0.
 *   B_bias, C_bias  [H, R, N] float32 added after the normalisation (or to
 *                the raw B / C without it), or NULL.
 *   dt_softplus  0 or 1: Delta = softplus(dt + dt_bias[h]) (dt_bias [H] or
 *                NULL; needs dt_softplus), the step made positive on chip.
 * The rotation (RoPE) applies to the normalised and biased B and C, and the
 * carried B (Bprev_rot, Bprev_rot_out) is that rotated B.  Gains and biases
 * must be 4-byte aligned.  Other values are M3_ERR_INVALID_ARG.
 */
typedef struct m3_prologue {
  int32_t bc_norm;
  int32_t dt_softplus;
  float bc_eps;
  const float* B_norm_w;
  const float* C_norm_w;
  const float* B_bias;
  const float* C_bias;
  const float* dt_bias;
} m3_prologue;

typedef struct m3_prefill_args {
  int32_t Bt, L, H, P, N, R, chunk;
  int32_t in_dtype; /* m3_dtype */
  const void* x;
  const void* B;
  const void* C;
  const float* dt;
  const float* lam;
  const float* A;
  const float* theta;
  const float* h0;
  const float* Bprev_rot;
  const void* xprev;
  const float* phi0;
  void* y;
  float* h_final;
  float* Bprev_rot_out;
  void* xprev_out;
  float* phi_out;
  void* workspace;        /* device scratch of workspace_bytes (256-byte aligned), or NULL */
  size_t workspace_bytes;
  const float* omega;     /* [Bt, L, N/2] angular rates, or NULL (see above) */
  const float* A_tok;     /* [Bt, L, H] A per token, or NULL (see above) */
  int32_t layout;         /* m3_layout of x, B, C, y (see above) */
  m3_prologue pro;        /* steps fused in front of the core (zeros = none) */
} m3_prefill_args;

int m3_ssm_prefill(const m3_prefill_args* args, void* stream);

/* Device scratch that lets m3_ssm_prefill use more of the GPU; 0 when it
 * would not (fp32 inputs, or at least half as many (batch, head) units as the
 * device has compute units, or sequences shorter than 8 chunks).
 *   With fewer units than that, a bf16 prefill given a workspace of this size
 * first walks the first half of every sequence for its state only (the
 * chunked evaluation of "La dualita: Mamba-2 e Mamba-3", sec. "Perche
 * conviene", needs only the state to hand over), then computes both halves at
 * once, the second one starting from that state -- the same carry that
 * continues a sequence across calls.  When the first half has at least 8
 * chunks, its state walk itself runs as two parts at once, the second from a
 * zero state and zero angle, and a small kernel joins them (the recurrence is
 * linear in the state and the rotations compose).  Results agree with the
 * unsplit call to rounding (the handed-over carry is exact fp32, where the
 * unsplit walk passes the pending term through bf16).  With workspace == NULL
 * the call runs unsplit.
 * The workspace holds the state and carry of two segments
 * (Bt*H*2*(4NP + 4RN + 2RP + 2N) bytes, rounded); it is overwritten by every
 * call, so concurrent calls need their own.  Depends only on the shape
 * fields (and the current device), not on pointers. */
size_t m3_ssm_prefill_workspace_size(const m3_prefill_args* args);

/*
 * m3_ssm_prefill for callers that cannot allocate device memory: code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc.
 * Same arguments, results and kernels as m3_ssm_prefill, except that
 * `workspace` must be NULL and `workspace_bytes` 0: where the call would use
 * the optional workspace (m3_ssm_prefill_workspace_size > 0) it uses instead
 * a static device buffer of M3_NOALLOC_SCRATCH_BYTES that the library holds
 * on every device it runs on until the process ends.  Nothing is allocated
 * by the call (the buffer's address is looked up once per device, with the
 * device current, on the first call there).  A call whose workspace size
 * exceeds M3_NOALLOC_SCRATCH_BYTES (16 MiB) returns M3_ERR_SCRATCH without
 * launching: on a 256-CU device every split shape with N * P <= 128 * 64
 * fits (at most ~8.6 MB); at N = P = 128 calls with more than ~120 (batch,
 * head) units do not (they can use m3_ssm_prefill with a workspace).  The
 * buffer needs no clearing (each call writes what it reads), but every call
 * on one device shares it: calls that overlap in time on one device (two
 * streams, two host threads) race and give undefined results; serialise
 * them, or use m3_ssm_prefill with a workspace per stream.
 */
#define M3_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)
int m3_ssm_prefill_noalloc(const m3_prefill_args* args, void* stream);

/*
 * One decode token against a resident state (the same token update as the
 * prefill, "La dualita", sec. "Mamba-3": MIMO update on an unchanged state).
 *
 *   In/out (updated in place):
 *   h         [Bt, H, N, P]   float32    state
 *   phi       [Bt, H, N/2]    float32    cumulative angle (NULL iff neither
 *                                        theta nor omega is given);
 *                                        stored reduced modulo 2*pi
 *   Bprev_rot [Bt, H, R, N]   float32    rotated B of the previous token
 *   xprev     [Bt, H, R, P]   in_dtype   x of the previous token
 *   In:
 *   x [Bt,H,R,P], B, C [Bt,H,R,N] (in_dtype); dt, lam [Bt,H] float32;
 *   A [H] float32, or A_tok [Bt,H] float32 (A per (batch, head) for this
 *   token; then A may be NULL); theta [Bt,H,N/2] float32 or NULL, or instead
 *   omega [Bt,N/2] float32 (rates shared by the heads: theta = dt * omega).
 *   Out: y [Bt, H, R, P] in_dtype.
 * Sizes: N, P in {16, 32, 64, 128}; R in 1..16.  A fresh sequence starts with
 * h = 0 (or any state), Bprev_rot = 0, xprev = 0, phi = 0.
 * With bf16 inputs, N in {32, 64, 128} and P in {64, 128} the rank-2R update
 * and the readout run on the matrix cores ("Znakomstvo s Mamba-3", sec. 3: with
 * MIMO the update is a matrix product); other shapes and fp32 inputs on the
 * vector ALUs.  Both keep the state in fp32.
 * pro: the same prologue as the prefill's (B, C, dt raw), so that a decode
 * continues a prefill that used it.
 */
typedef struct m3_decode_args {
  int32_t Bt, H, P, N, R;
  int32_t in_dtype; /* m3_dtype */
  float* h;
  float* phi;
  float* Bprev_rot;
  void* xprev;
  const void* x;
  const void* B;
  const void* C;
  const float* dt;
  const float* lam;
  const float* A;
  const float* theta;
  void* y;
  const float* A_tok; /* [Bt, H] A of this token, or NULL */
  const float* omega; /* [Bt, N/2] rotation rates shared by the heads, or NULL */
  m3_prologue pro;    /* steps fused in front of the core (zeros = none) */
} m3_decode_args;

int m3_ssm_decode_step(const m3_decode_args* args, void* stream);

/*
 * Backward pass of the prefill: gradients of a loss that reaches the core
 * through y (upstream gradient dy) and the final state (dh_final), by reverse-
 * mode differentiation of the chunked evaluation ("La dualita: Mamba-2 e
 * Mamba-3", sec. "Perche conviene: i tensor core") of the recurrence
 * ("Znakomstvo s Mamba-3", sec. 1-3); the pages print no backward pass.  The
 * carry-out (rotated B, x, angle) is not differentiated.
 *
 *   Forward inputs (as given to m3_ssm_prefill, token-major): x, B, C [Bt, L,
 *   H, R, .] bf16; dt, lam [Bt, L, H]; A [H] or A_tok [Bt, L, H]; theta [Bt, L,
 *   H, N/2] or NULL; carry-in h0, Bprev_rot, xprev, phi0 (nullable).
 *   Upstream: dy [Bt, L, H, R, P] bf16; dh_final [Bt, H, N, P] float32 or NULL.
 *   Gradients (outputs): dx, dB, dC (bf16, shapes of x, B, C); ddt, dlam [Bt,
 *   L, H] float32; dA: [H] when A is given (summed over batch and tokens),
 *   [Bt, L, H] when A_tok is given; dtheta [Bt, L, H, N/2] (required iff
 *   theta); dh0 [Bt, H, N, P], dBprev_rot [Bt, H, R, N] (float32), dxprev
 *   [Bt, H, R, P] (bf16), dphi0 [Bt, H, N/2]: each nullable.
 *   workspace: required, m3_ssm_prefill_backward_workspace_size bytes,
 *   256-byte aligned (the shifted state, in bf16, and the angle entering
 *   every chunk of every (batch, head), written by the kernel's forward
 *   state walk; with at most half as many (batch, head) units as the
 *   device has compute units and at least 8 chunks the sequence is split in
 *   two walked at once, and the workspace also holds the values joined at
 *   the split: so its size depends on the current device).
 * Sizes: bf16 only (M3_ERR_UNSUPPORTED for float32); N, P in {16, 32, 64,
 * 128} whose tiles fit the LDS of a CU (N = P = 128 does not:
 * M3_ERR_UNSUPPORTED); R a power of two <= 8; chunks of 64 / R tokens.
 * Gradients are deterministic (no atomics).
 */
typedef struct m3_backward_args {
  int32_t Bt, L, H, P, N, R;
  int32_t in_dtype;       /* m3_dtype: M3_BF16 */
  const void* x;
  const void* B;
  const void* C;
  const float* dt;
  const float* lam;
  const float* A;
  const float* A_tok;
  const float* theta;
  const float* h0;
  const float* Bprev_rot;
  const void* xprev;
  const float* phi0;
  const void* dy;
  const float* dh_final;
  void* dx;
  void* dB;
  void* dC;
  float* ddt;
  float* dlam;
  float* dA;
  float* dtheta;
  float* dh0;
  float* dBprev_rot;
  void* dxprev;
  float* dphi0;
  void* workspace;
  size_t workspace_bytes;
} m3_backward_args;

size_t m3_ssm_prefill_backward_workspace_size(const m3_backward_args* args);
int m3_ssm_prefill_backward(const m3_backward_args* args, void* stream);

/*
 * Inclusive cumulative rotation angle ("Znakomstvo s Mamba-3", sec. 2: the
 * rotations are aggregated over all time steps):
 *   phi[b, t, h, j] = phi0[b, h, j] + sum_{s <= t} theta[b, s, h, j].
 * theta, phi: [Bt, L, H, npairs] float32; phi0: [Bt, H, npairs] or NULL.
 * H * npairs must be a multiple of 4.  phi is the plain fp32 running sum
 * (no modular reduction).  phi must not alias theta.
 */
int m3_rope_angles_cumsum(const float* theta, const float* phi0, float* phi,
                          int32_t Bt, int32_t L, int32_t H, int32_t npairs,
                          void* stream);

/*
 * ---------------------------------------------------------------- layer operators
 * The operators that stand around a selective state-space core in a layer: the
 * short causal convolution in front of it, the selective scan itself with a
 * decay per channel and state (the two-term recurrence of "La dualita:
 * Mamba-2 e Mamba-3", sec. "State Space Duality", with a diagonal A per
 * channel), the gated norm behind it and the residual norm in front of the
 * next block ("Mamba-3: un modello a spazio di stato progettato per
 * l'inferenza" (cartesia.ai), "Normalizzazioni" and "Addio convoluzione
 * corta", names them as the parts around the core).
 *
 * Common to all of them:
 *   - Types: in_dtype M3_BF16 or M3_F32 for the activations; parameters
 *     (taps, biases, A, D, gains, scales), states of the scan and the
 *     gradients of parameters are float32.  All arithmetic is fp32; an output
 *     is rounded once.
 *   - Strides: a tensor with a field `*_ld` may be a slice of wider rows: ld
 *     is the number of elements from one token (row) to the next, 0 meaning
 *     dense; rows of all batch items follow each other at that distance, and
 *     the elements within a row are dense.  Everything else is dense
 *     row-major.  Pointers need the alignment of their elements only (rows
 *     whose addresses allow it are read 16 bytes at a time).
 *   - lengths [Bt] int32 or NULL: item b holds lengths[b] tokens (taken
 *     into [0, L] on the device); what lies behind them is never used, whatever
 *     it holds.  Forward outputs behind them are left as they were, gradients
 *     of inputs behind them are set to zero, states end with the last token
 *     held (lengths[b] = 0: the state passes through).
 *   - Outputs do not alias inputs or each other, except where noted.
 *   - Sizes: Bt D and M below 2^31, 2^35 elements of one tensor, L and D up to
 *     2^28.  A launch has fewer than 2^32 work items, which bounds calls of
 *     millions of short sequences and of very wide rows further:
 *       scan and its backward  512 for each item, group and 64 channels of it (32
 *                              with N > 16, 16 with N > 32)
 *       its backward           2 N for each token and group; up to 64 D (N + 2)
 *       its token              N / 16 for each item and channel, N rounded up to a
 *                              power of two from 4
 *       convolution's backward 256 for each item, 256 channels and 512 tokens; up
 *                              to 64 (W + 1) D
 *       norms' backwards       up to 64 D for each parameter
 *     Larger calls are M3_ERR_UNSUPPORTED, before anything is launched.
 */

/* Short causal depthwise convolution over the token axis:
 *   y[b,t,d] = act(bias[d] + sum_{k<W} w[d,k] x[b, t-(W-1)+k, d]),
 * act = SiLU with silu = 1, identity with 0.
 *   x [Bt, L, D] (x_ld), w [D, W], bias [D] or NULL, y [Bt, L, D].
 *   state [Bt, W-1, D] in_dtype or NULL (zeros): the inputs before the first
 *   token, oldest first; state_out (nullable): the W-1 inputs that end with the
 *   last token, may be `state` itself.  W in {2, 3, 4}. */
typedef struct m3_conv_args {
  int32_t Bt, L, D, W;
  int32_t in_dtype; /* m3_dtype */
  int32_t silu;     /* 0 or 1 */
  const void* x;
  int64_t x_ld;
  const float* w;
  const float* bias;
  const int32_t* lengths;
  const void* state;
  void* y;
  void* state_out;
} m3_conv_args;
int m3_causal_conv(const m3_conv_args* args, void* stream);

/* One token of it: x [Bt, D] (x_ld between the batch rows), state [Bt, W-1, D]
 * updated in place, or read only when state_out is given (which may be `state`
 * too); y [Bt, D]. */
typedef struct m3_conv_step_args {
  int32_t Bt, D, W;
  int32_t in_dtype;
  int32_t silu;
  const void* x;
  int64_t x_ld;
  const float* w;
  const float* bias;
  void* state;
  void* state_out; /* NULL: state */
  void* y;
} m3_conv_step_args;
int m3_causal_conv_step(const m3_conv_step_args* args, void* stream);

/* Gradients of the convolution for dy [Bt, L, D] (dense): dx [Bt, L, D], dw
 * [D, W], dbias [D] (nullable), dstate [Bt, W-1, D] in_dtype (nullable;
 * gradient of the carry-in).  The carry-out is not differentiated.
 * workspace: m3_causal_conv_backward_workspace_size bytes, 256-byte aligned
 * (partial sums of dw and dbias, joined in a fixed order). */
typedef struct m3_conv_backward_args {
  int32_t Bt, L, D, W;
  int32_t in_dtype;
  int32_t silu;
  const void* x;
  int64_t x_ld;
  const float* w;
  const float* bias;
  const int32_t* lengths;
  const void* state;
  const void* dy;
  void* dx;
  float* dw;
  float* dbias;
  void* dstate;
  void* workspace;
  size_t workspace_bytes;
} m3_conv_backward_args;
size_t m3_causal_conv_backward_workspace_size(const m3_conv_backward_args* args);
int m3_causal_conv_backward(const m3_conv_backward_args* args, void* stream);

/* Selective scan, a diagonal state per channel:
 *   delta = softplus(dt + dt_bias[d]) with dt_softplus = 1 (dt_bias nullable),
 *           dt itself with 0 (dt_bias must then be NULL);
 *   h_t[d,n] = exp(delta_t[d] A[d,n]) h_{t-1}[d,n] + delta_t[d] x_t[d] B_t[g,n];
 *   o_t[d] = sum_n C_t[g,n] h_t[d,n] + D[d] x_t[d];
 *   y_t[d] = o_t[d] silu(z_t[d])   (z NULL: y = o),  g = d / (D / G).
 *   x, dt, z [Bt, L, D] (x_ld, dt_ld, z_ld), B, C [Bt, L, G, N] (B_ld, C_ld),
 *   A [D, N], D_skip [D] or NULL; h0 [Bt, D, N] or NULL (zeros); y [Bt, L, D];
 *   h_final [Bt, D, N] (nullable).
 * Sizes: N in 1..64, G divides D, row distances below 2^24 elements (for its
 * backward and its token too; others are M3_ERR_INVALID_ARG).
 * workspace: optional; with few (batch, channel) pairs the token axis is cut
 * into segments scanned at once, whose states are joined, when a workspace of
 * m3_selective_scan_workspace_size bytes (256-byte aligned; 0: not used) is
 * given.  It is overwritten by every call, so calls at once need their own; the
 * size depends on the sizes and on whether lengths is given. */
typedef struct m3_scan_args {
  int32_t Bt, L, D, N, G;
  int32_t in_dtype;
  int32_t dt_softplus;
  const void* x;
  int64_t x_ld;
  const void* dt;
  int64_t dt_ld;
  const float* A;
  const void* B;
  int64_t B_ld;
  const void* C;
  int64_t C_ld;
  const float* D_skip;
  const void* z;
  int64_t z_ld;
  const float* dt_bias;
  const float* h0;
  const int32_t* lengths;
  void* y;
  float* h_final;
  void* workspace;
  size_t workspace_bytes;
} m3_scan_args;
size_t m3_selective_scan_workspace_size(const m3_scan_args* args);
int m3_selective_scan(const m3_scan_args* args, void* stream);

/* One token of it: x, dt, z [Bt, D], B, C [Bt, G, N] (each `*_ld` between the
 * batch rows), h [Bt, D, N] updated in place, or read only when h_out is given
 * (which may be h too); y [Bt, D]. */
typedef struct m3_scan_step_args {
  int32_t Bt, D, N, G;
  int32_t in_dtype;
  int32_t dt_softplus;
  const void* x;
  int64_t x_ld;
  const void* dt;
  int64_t dt_ld;
  const float* A;
  const void* B;
  int64_t B_ld;
  const void* C;
  int64_t C_ld;
  const float* D_skip;
  const void* z;
  int64_t z_ld;
  const float* dt_bias;
  float* h;
  float* h_out; /* NULL: h */
  void* y;
} m3_scan_step_args;
int m3_selective_scan_step(const m3_scan_step_args* args, void* stream);

/* Gradients of the scan for dy [Bt, L, D] (dense) and dh_final [Bt, D, N]
 * (nullable).  Outputs: dx, ddt [Bt, L, D], dB, dC [Bt, L, G, N] in in_dtype;
 * dA [D, N]; dD [D] (required iff D_skip), dz [Bt, L, D] (required iff z),
 * ddt_bias [D] (required iff dt_bias), dh0 [Bt, D, N] (nullable).  ddt is the
 * gradient of dt as given (before the softplus).  workspace:
 * m3_selective_scan_backward_workspace_size bytes, 256-byte aligned. */
typedef struct m3_scan_backward_args {
  m3_scan_args fwd; /* the forward's inputs; y, h_final, workspace are not read */
  const void* dy;
  const float* dh_final;
  void* dx;
  void* ddt;
  float* dA;
  void* dB;
  void* dC;
  float* dD;
  void* dz;
  float* ddt_bias;
  float* dh0;
  void* workspace;
  size_t workspace_bytes;
} m3_scan_backward_args;
size_t m3_selective_scan_backward_workspace_size(const m3_scan_backward_args* args);
int m3_selective_scan_backward(const m3_scan_backward_args* args, void* stream);

/* Gated group RMS norm over rows of D = G groups (up to 2^20) of D / G:
 *   gate_first = 1: v = x silu(z),  y = v rsqrt(mean_group(v^2) + eps) w;
 *   gate_first = 0: y = x rsqrt(mean_group(x^2) + eps) w silu(z).
 * x, z [M, D] (x_ld, z_ld; z NULL: no gate), w [D] or NULL (ones), y [M, D]
 * (may be x or z themselves where those are dense).  eps >= 0; a group of zeros
 * with eps = 0 gives NaN. */
typedef struct m3_gated_norm_args {
  int64_t M;
  int32_t D, G;
  int32_t in_dtype;
  int32_t gate_first;
  float eps;
  const void* x;
  int64_t x_ld;
  const void* z;
  int64_t z_ld;
  const float* w;
  void* y;
} m3_gated_norm_args;
int m3_gated_norm(const m3_gated_norm_args* args, void* stream);

/* Its gradients for dy [M, D] (dense): dx, dz [M, D] (dz required iff z), dw [D]
 * (required iff w). */
typedef struct m3_gated_norm_backward_args {
  m3_gated_norm_args fwd; /* y is not read */
  const void* dy;
  void* dx;
  void* dz;
  float* dw;
  void* workspace;
  size_t workspace_bytes;
} m3_gated_norm_backward_args;
size_t m3_gated_norm_backward_workspace_size(const m3_gated_norm_backward_args* args);
int m3_gated_norm_backward(const m3_gated_norm_backward_args* args, void* stream);

/* Residual sum and RMS norm over rows of D:
 *   h = residual + scale x (residual NULL: 0; scale [D], NULL: 1),
 *   residual_out = h (nullable; may be `residual` itself),
 *   y = h rsqrt(mean(h^2) + eps) w   (w [D], NULL: ones; h unrounded).
 * x [M, D] (x_ld), y [M, D] in_dtype; residual, residual_out [M, D] res_dtype:
 * in_dtype or M3_F32. */
typedef struct m3_residual_norm_args {
  int64_t M;
  int32_t D;
  int32_t in_dtype;
  int32_t res_dtype;
  float eps;
  const void* x;
  int64_t x_ld;
  const void* residual;
  const float* scale;
  const float* w;
  void* y;
  void* residual_out;
} m3_residual_norm_args;
int m3_residual_norm(const m3_residual_norm_args* args, void* stream);

/* Its gradients at the stored sum h = residual_out [M, D] res_dtype, for dy
 * [M, D] in_dtype and dresidual_out [M, D] res_dtype (nullable: gradient that
 * reaches h along the residual stream):
 *   dh = dresidual_out + d(norm)/dh,  dresidual = dh (nullable),
 *   dx = scale dh (nullable, in_dtype), dw [D] (required iff w), dscale [D]
 *   (required iff scale) = sum_rows dh x.
 * x (x_ld) is read for dscale only.  dresidual may be dresidual_out itself. */
typedef struct m3_residual_norm_backward_args {
  int64_t M;
  int32_t D;
  int32_t in_dtype;
  int32_t res_dtype;
  float eps;
  const void* h;
  const void* x;
  int64_t x_ld;
  const float* scale;
  const float* w;
  const void* dy;
  const void* dresidual_out;
  void* dx;
  void* dresidual;
  float* dw;
  float* dscale;
  void* workspace;
  size_t workspace_bytes;
} m3_residual_norm_backward_args;
size_t m3_residual_norm_backward_workspace_size(const m3_residual_norm_backward_args* args);
int m3_residual_norm_backward(const m3_residual_norm_backward_args* args, void* stream);

/* Static description of a status code (never NULL). */
const char* m3_status_string(int status);

/* Library version, e.g. "0.1.0". */
const char* m3_version(void);

#ifdef __cplusplus
}
#endif

#endif /* M3SSM_H */
