/*
 * ssm_scan.h -- C ABI of the MI355X (gfx950) selective state-space scan library.
 *
 * Entry points, each a hand-written HIP kernel pipeline for CDNA4:
 *   ssm_scan_fwd     Mamba-1 selective scan over a whole sequence (prefill)
 *   ssm_scan_fwd_noalloc  the same on a fixed per-GPU scratch (no workspace argument)
 *   ssm_scan_fwd_ex  the same with exact zero-order hold and/or Delta = softplus(delta + bias)
 *   ssm_scan3_fwd    Mamba-3: complex transitions, exponential-trapezoidal rule
 *   ssm_step3        the Mamba-3 one-token decode step, complex state updated in place
 *   ssm_scan_bwd     the scan's gradient (training backward pass)
 *   ssm_ssd_fwd      Mamba-2 SSD: scalar decay per head, chunked decayed-attention form
 *   ssm_step         one-token recurrent decode step, state updated in place
 *   ssm_step_ex      the decode step with the options of ssm_scan_fwd_ex
 *   ssm_ssd_step     the same for the Mamba-2 form (scalar decay per head, (N, P) state)
 *   ssm_linattn_fwd  linear attention with a decay per head, queries and keys per head
 *                    or head group (prefill; padded batches)
 *   ssm_linattn_bwd  its gradient
 *   ssm_linattn_step its one-token decode step, optionally with the group norm and gate
 *   ssm_group_norm_fwd, ssm_group_norm_bwd
 *                    group norm, channels last, with activation and/or silu(z) gate
 *   ssm_glr_fwd      gated linear recurrence: a decay per token and channel, one state a
 *                    channel (prefill; padded batches)
 *   ssm_glr_bwd      its gradient
 *   ssm_glr_step     its one-token decode step
 *   ssm_add_norm_fwd, ssm_add_norm_bwd
 *                    residual add with dropout, then layer norm or RMS norm
 *   ssm_dropout      dropout from a counter, forward and gradient
 *
 * The operation (selective SSM of Gu & Dao, "Mamba: Linear-Time Sequence
 * Modeling with Selective State Spaces", 2023, and the SSD form of Dao & Gu,
 * "Transformers are SSMs", 2024 -- both in the ssm-bench README's references;
 * the variants as described by "Efficient Sequence Modeling: From S4 to
 * Mamba-3", section 03 System: mamba_minimal.py has input-dependent Delta, B, C
 * and an incremental step(); mamba2_minimal.py has a scalar A per head, chunked
 * decayed-attention matmuls and a carried (N, P) state):
 *
 *   per (batch b, channel d), state h in R^N, for t = 0 .. L-1:
 *     h_t = exp(Delta_t * A) (.) h_{t-1} + Delta_t * B_t * x_t      (exponential-Euler:
 *     y_t = (C_t . h_t + D * x_t) * silu(z_t),  silu(z) = z / (1 + e^-z)   section 04/09)
 *
 * Conventions shared by every entry point
 *  - Tensors are contiguous, row-major, last index fastest.
 *  - Every pointer is a DEVICE pointer owned by the caller. The library never
 *    allocates, frees or synchronises inside these calls and keeps no pointer
 *    after return, except for work in flight on `stream`.
 *  - `stream` is a hipStream_t (NULL = the default stream). All work is queued
 *    asynchronously on it; results are ready when the stream reaches that point.
 *  - `io` (ssm_dtype_t) is the storage type of x, delta, B, C, z and y.
 *    A, D, h0, h_final and the decode state are always fp32.
 *    Arithmetic is fp32 throughout (fp32 state and accumulation).
 *  - delta is used as given (already positive: no softplus inside).
 *  - A holds the actual (negative) decay rates, not log(-A).
 *  - B and C are one group shared by all channels (Mamba-1) or all heads (SSD).
 *  - Optional pointers may be NULL: Dskip (no skip term), z (no gate),
 *    h0 (zero initial state), h_final (not written).
 *  - Aliasing: y must not alias any input; h_final must not alias h0.
 *  - Errors: arguments are validated BEFORE any HIP call. A rejected call has
 *    queued nothing. Status codes are below; ssm_last_error() returns a
 *    human-readable detail of the calling thread's last failure.
 *    No C++ exception crosses this boundary.
 *  - Results are deterministic run to run (no floating-point atomics).
 *  - Thread-safe and reentrant: no mutable global state beyond a per-thread
 *    error message and cached device properties.
 */
#ifndef SSM_SCAN_H
#define SSM_SCAN_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SSM_ABI_VERSION 1

/* Storage type of the io tensors. The last enumerator only widens the type to a
 * full int, so any int a caller passes is a valid value (out-of-range values are
 * rejected with SSM_ERR_INVALID_ARG). */
typedef enum { SSM_F32 = 0, SSM_BF16 = 1, SSM_DTYPE_INT_RANGE_ = 0x7fffffff } ssm_dtype_t;

/* Discretisation of the continuous system dh/dt = A h + B x over one step Delta
 * (diagonal A). Exponential-Euler is what every entry point uses by default. */
typedef enum {
    SSM_DISC_EULER = 0, /* Abar = exp(Delta A), Bbar = Delta B */
    SSM_DISC_ZOH = 1,   /* Abar = exp(z), Bbar = Delta B (e^z - 1)/z, z = Delta A (exact zero-order hold) */
    SSM_DISC_INT_RANGE_ = 0x7fffffff
} ssm_disc_t;

typedef enum {
    SSM_OK = 0,
    SSM_ERR_INVALID_ARG = 1, /* null required pointer, bad dimension, misaligned pointer */
    SSM_ERR_UNSUPPORTED = 2, /* shape outside the compiled range (e.g. unsupported N or P) */
    SSM_ERR_WORKSPACE = 3,   /* workspace NULL or smaller than *_workspace_size() */
    SSM_ERR_HIP = 4          /* a HIP launch error (hipGetLastError after the launch) */
} ssm_status_t;

/* SSM_ABI_VERSION of the built library. */
int ssm_abi_version(void);

/* Static string naming a status code. */
const char* ssm_status_string(int status);

/* Detail of the calling thread's last non-OK status ("" if none). */
const char* ssm_last_error(void);

/* Kernel-level timing without a profiler (diagnostic; for benchmarks).
 * After ssm_profile_events(events, n) with n > 0, every kernel launched by an
 * entry point called from this thread takes the next two events (events[0] and
 * events[1] for the first kernel, and so on; each a hipEvent_t created by the
 * caller), which the HIP runtime stamps at that kernel's own start and end
 * (hipExtLaunchKernel), so hipEventElapsedTime of a pair is the kernel's
 * duration. Recording stops when fewer than two events remain.
 * ssm_profile_events(NULL, 0) switches recording off. Returns the number of
 * events used since the previous call (twice the number of kernels timed).
 * Per thread; the library never creates, synchronises or destroys the events. */
int ssm_profile_events(void* const* events, int n);

/* ---------------------------------------------------------------------------
 * ssm_scan_fwd -- Mamba-1 selective scan (prefill).
 *
 * Defined by "Efficient Sequence Modeling: From S4 to Mamba-3", section 03
 * System (mamba_minimal.py: input-dependent Delta, B, C and an explicit
 * time-loop selective scan), with the exponential-Euler discretisation the
 * same page names as the lambda = 1, theta = 0 limit (section 04, "Complex
 * transitions for state tracking"; section 09 Validation). Per (b, d), over
 * t = 0 .. L-1, from h = h0[b, d, :] (or zeros):
 *   h[n]      = exp(delta[b,t,d] * A[d,n]) * h[n] + delta[b,t,d] * Bm[b,t,n] * x[b,t,d]
 *   y[b,t,d]  = (sum_n Cm[b,t,n] * h[n] + Dskip[d] * x[b,t,d]) * silu(z[b,t,d])
 *   h_final[b, d, :] = h after the last step.
 * The work is cut along L into segments whose carried states compose as affine
 * maps; the result equals the sequential recurrence up to rounding.
 *
 *   x, delta, z, y : [B, L, D]  io dtype     (z may be NULL)
 *   A              : [D, N]     fp32, A < 0 as used in exp(delta * A)
 *   Bm, Cm         : [B, L, N]  io dtype, shared by all D channels
 *   Dskip          : [D]        fp32 or NULL
 *   h0             : [B, D, N]  fp32 or NULL (zeros)
 *   h_final        : [B, D, N]  fp32 out, or NULL
 *   workspace      : device scratch of at least ssm_scan_workspace_size(B, L, D, N)
 *                    bytes (NULL allowed when that size is 0); contents on entry
 *                    are ignored and on return are undefined.
 * Supported: N in {4, 8, 16, 32, 64, 128, 256}; B, D >= 1; L >= 0 (L = 0 writes
 * h_final = h0). N = 256 needs a workspace whenever L > 0 (it holds the C . h sums
 * of its two groups of state chunks).
 * Every pointer must be 16-byte aligned.
 * ------------------------------------------------------------------------- */
size_t ssm_scan_workspace_size(int B, int L, int D, int N);

int ssm_scan_fwd(int B, int L, int D, int N, ssm_dtype_t io,
                 const void* x, const void* delta, const float* A,
                 const void* Bm, const void* Cm, const float* Dskip,
                 const void* z, const float* h0,
                 void* y, float* h_final,
                 void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * ssm_scan_fwd_noalloc -- ssm_scan_fwd for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc): no workspace argument, and nothing is allocated or freed.
 *
 * The scan's carry workspace is a fixed device array inside the library,
 * SSM_NOALLOC_SCRATCH_BYTES (128 MiB) per GPU, held from the library's load until
 * the process ends. Its device address is looked up on the first call made for
 * a device (with that device made current for the lookup). Every other argument,
 * the result and the errors are those of ssm_scan_fwd; a shape whose
 * ssm_scan_workspace_size() exceeds SSM_NOALLOC_SCRATCH_BYTES returns
 * SSM_ERR_UNSUPPORTED (for instance B=8, L=32768, D=512, N=16 needs 99.5 MiB
 * and fits; N = 256 at B=1, L=4096, D=1536 needs 141.2 MiB and does not). The
 * kernels run on the device of `stream` (the current device when stream is NULL).
 *
 * Concurrency: all calls on one GPU share its scratch array and nothing clears
 * it between calls (the scan ignores its previous contents). Calls that can
 * overlap on one GPU -- on different streams, or from different threads without
 * ordering -- race on it and give undefined results; serialise them (one stream,
 * or events between streams).
 * ------------------------------------------------------------------------- */
#define SSM_NOALLOC_SCRATCH_BYTES ((size_t)128 << 20)

int ssm_scan_fwd_noalloc(int B, int L, int D, int N, ssm_dtype_t io,
                         const void* x, const void* delta, const float* A,
                         const void* Bm, const void* Cm, const float* Dskip,
                         const void* z, const float* h0,
                         void* y, float* h_final, void* stream);

/* ---------------------------------------------------------------------------
 * ssm_scan_fwd_ex -- ssm_scan_fwd with a choice of discretisation and the
 * Delta preprocessing done inside the kernels.
 *
 *   disc           SSM_DISC_EULER or SSM_DISC_ZOH. Exact zero-order hold is the
 *                  discretisation of "Efficient Sequence Modeling: From S4 to
 *                  Mamba-3" (section 03, s4_minimal.py; section 04 "Math-verified
 *                  discretization"; Q01): Bbar = Delta B (e^z - 1)/z, z = Delta A,
 *                  evaluated without the 0/0 at z = 0 (a series where |z| < 1/32).
 *   delta_bias     [D] fp32 or NULL: added to delta before everything else.
 *   delta_softplus nonzero: Delta = softplus(delta + delta_bias) = log(1 + e^(.)).
 * Every other argument, the workspace (ssm_scan_workspace_size) and the errors
 * are those of ssm_scan_fwd; with SSM_DISC_EULER, no bias and no softplus it is
 * ssm_scan_fwd. Every N of ssm_scan_fwd is supported (N >= 64 runs as chunks of
 * 16 states, as there). delta_bias must be 16-byte aligned.
 * ------------------------------------------------------------------------- */
int ssm_scan_fwd_ex(int B, int L, int D, int N, ssm_dtype_t io, ssm_disc_t disc,
                    const float* delta_bias, int delta_softplus,
                    const void* x, const void* delta, const float* A,
                    const void* Bm, const void* Cm, const float* Dskip,
                    const void* z, const float* h0,
                    void* y, float* h_final,
                    void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * ssm_scan3_fwd -- Mamba-3 selective scan: complex diagonal transitions and the
 * exponential-trapezoidal rule.
 *
 * "Efficient Sequence Modeling: From S4 to Mamba-3", section 03 System
 * (mamba3_minimal.py: complex diagonal transitions A = -exp(a) + i theta with a
 * data-dependent exponential-trapezoidal rule, reducing to Mamba-1/2 at lam = 1)
 * and section 04 "Complex transitions for state tracking" (the rotation phase
 * lets the state track parity; lam = 1, theta = 0 is exponential-Euler). The
 * pages do not write the rule out; the reading implemented is the trapezoidal
 * rule, weighted by lam, on the exact one-step integral of e^{A (Delta - s)} B x.
 * Per (b, d), complex state h[n], for t = 0 .. L-1:
 *   alpha   = exp(delta[b,t,d] * (Are[d,n] + i theta[d,n]))
 *   h[n]    = alpha h[n] + (1 - lam[b,t,d]) delta[b,t,d] alpha Bm[b,t-1,n] x[b,t-1,d]
 *                        + lam[b,t,d] delta[b,t,d] Bm[b,t,n] x[b,t,d]
 *   y[b,t,d] = (sum_n Cm[b,t,n] Re(h[n]) + Dskip[d] x[b,t,d]) * silu(z[b,t,d])
 * where the step before t = 0 is (x_prev[b,d], B_prev[b,:]) -- the last token of
 * a previous call, so that a sequence can be continued -- or zero when both are
 * NULL.
 *
 *   x, delta, lam, z, y : [B, L, D]  io dtype (z may be NULL); lam in [0, 1]
 *   Are, theta     : [D, N]     fp32 (Are < 0: the real part of A; theta in radians
 *                               per unit of delta)
 *   Bm, Cm         : [B, L, N]  io dtype
 *   Dskip          : [D]        fp32 or NULL
 *   h0, h_final    : [B, D, N, 2] fp32 complex (real, imaginary), or NULL
 *   x_prev, B_prev : [B, D], [B, N] io dtype, both given or both NULL
 *   workspace      : at least ssm_scan3_workspace_size(B, L, D, N) bytes
 * Supported: N in {4, 8, 16}; B <= 65535. Every pointer must be 16-byte aligned.
 * Errors as for ssm_scan_fwd.
 * ------------------------------------------------------------------------- */
size_t ssm_scan3_workspace_size(int B, int L, int D, int N);

int ssm_scan3_fwd(int B, int L, int D, int N, ssm_dtype_t io,
                  const void* x, const void* delta, const void* lam,
                  const float* Are, const float* theta,
                  const void* Bm, const void* Cm, const float* Dskip, const void* z,
                  const float* h0, const void* x_prev, const void* B_prev,
                  void* y, float* h_final,
                  void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * ssm_step3 -- Mamba-3 one-token decode step: the recurrence of ssm_scan3_fwd for
 * one time step, the complex state updated in place.
 *
 * "Efficient Sequence Modeling: From S4 to Mamba-3", section 03 System
 * (mamba3_minimal.py: the incremental form of the complex, exponential-trapezoidal
 * recurrence). Per (batch b, channel d) and state n:
 *   alpha = exp(delta (Are[d,n] + i theta[d,n]))
 *   h[n]  = alpha (h[n] + (1 - lam) delta B_prev[n] x_prev) + lam delta B[n] x
 *   y     = (sum_n C[n] Re h[n] + Dskip[d] x) * silu(z)
 * ssm_step3 on a state equals ssm_scan3_fwd over one token from that state with
 * the same (x_prev, B_prev); a decode loop passes the previous token's x and B
 * row as the next call's x_prev and B_prev.
 *
 *   state  : [B, D, N, 2] fp32 (real, imaginary), read and written in place
 *   x, delta, lam, z : [B, D] io dtype (z may be NULL: no gate)
 *   Are, theta       : [D, N] fp32, as for ssm_scan3_fwd
 *   Bm, Cm           : [B, N] io dtype
 *   Dskip            : [D] fp32 or NULL
 *   x_prev, B_prev   : [B, D] and [B, N] io dtype, both or neither (neither: the
 *                      previous token's term is zero, as at a sequence start)
 *   y                : [B, D] io dtype out
 * Supported: N in {4, 8, 16, 32, 64, 128}; B <= 65535; D * N < 2^31. Every pointer
 * must be 16-byte aligned. Errors: SSM_ERR_INVALID_ARG (a required pointer NULL,
 * x_prev without B_prev or the reverse, bad dims, misalignment), SSM_ERR_UNSUPPORTED
 * (N, B or D * N out of range), SSM_ERR_HIP.
 * ------------------------------------------------------------------------- */
int ssm_step3(int B, int D, int N, ssm_dtype_t io,
              float* state, const void* x, const void* delta, const void* lam,
              const float* Are, const float* theta, const void* Bm, const void* Cm,
              const float* Dskip, const void* z, const void* x_prev, const void* B_prev,
              void* y, void* stream);

/* ---------------------------------------------------------------------------
 * ssm_scan_bwd -- gradient of ssm_scan_fwd (training backward pass).
 *
 * Training Mamba models on GPUs is the workload of "Characterizing the Behavior
 * of Training Mamba-based State Space Models on GPUs" (abstract) and of the
 * training-step sweep in "Efficient Sequence Modeling: From S4 to Mamba-3",
 * section 05 Evaluation. The pages do not write the backward pass out: this is
 * the exact gradient of the forward recurrence above, by the chain rule. For
 * the loss  l = sum(dy * y) + sum(dh_final * h_final)  every output is dl/d(the
 * input of the same name):
 *
 *   inputs  : x, delta, A, Bm, Cm, Dskip, z, h0 exactly as given to ssm_scan_fwd
 *   dy      : [B, L, D]  io dtype, gradient of y (required)
 *   dh_final: [B, D, N]  fp32 gradient of h_final, or NULL (zero)
 *   dx, ddelta : [B, L, D] io dtype out
 *   dA      : [D, N]     fp32 out (summed over batch and time)
 *   dBm, dCm: [B, L, N]  io dtype out (summed over channels in fp32, then rounded)
 *   dDskip  : [D]        fp32 out; given exactly when Dskip is given
 *   dz      : [B, L, D]  io dtype out; given exactly when z is given
 *   dh0     : [B, D, N]  fp32 out, or NULL (not written); the gradient of the
 *                        initial state, also when h0 is NULL (zero state)
 *   workspace: device scratch of at least ssm_scan_bwd_workspace_size(B, L, D, N)
 *              bytes (0 only when L = 0); contents on entry are ignored.
 * The forward states are recomputed, not read from a forward call. Outputs must
 * not alias inputs or each other. Arithmetic is fp32 with fp32 accumulation;
 * reductions run in a fixed order (no atomics), so results are deterministic.
 * Supported: N in {4, 8, 16, 32, 64, 128, 256} (N >= 32 runs as chunks of 16
 * states whose partial sums over n are added in a fixed order: chunk order within
 * groups of up to four chunks, then the groups in order); B <= 65535; L >= 0
 * (L = 0 writes dh0 = dh_final, dA = 0, dDskip = 0). Every pointer must be
 * 16-byte aligned. Errors as for ssm_scan_fwd.
 * ------------------------------------------------------------------------- */
size_t ssm_scan_bwd_workspace_size(int B, int L, int D, int N);

int ssm_scan_bwd(int B, int L, int D, int N, ssm_dtype_t io,
                 const void* x, const void* delta, const float* A,
                 const void* Bm, const void* Cm, const float* Dskip,
                 const void* z, const float* h0,
                 const void* dy, const float* dh_final,
                 void* dx, void* ddelta, float* dA, void* dBm, void* dCm,
                 float* dDskip, void* dz, float* dh0,
                 void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * ssm_ssd_fwd -- Mamba-2 SSD chunked scan (prefill), scalar decay per head.
 *
 * Defined by "Efficient Sequence Modeling: From S4 to Mamba-3", section 03
 * System (mamba2_minimal.py: a scalar A per head reduces the recurrence to SSD,
 * computed as chunked decayed-attention matmuls with a carried (N, P) state)
 * and section 04 "Chunked SSD with a sequential reference" (the chunked form
 * equals the sequential recurrence). Per (b, h), from S = h0[b, h] (or zeros):
 *   S[n, p]    = exp(delta[b,t,h] * A[h]) * S[n, p] + delta[b,t,h] * Bm[b,t,n] * x[b,t,h,p]
 *   y[b,t,h,p] = (sum_n Cm[b,t,n] * S[n, p] + Dskip[h] * x[b,t,h,p]) * silu(z[b,t,h,p])
 *   h_final[b, h] = S after the last step.
 * Inside a chunk, with s_i the inclusive prefix of delta * A_h:
 *   y_i = sum_{j <= i} (C_i . B_j) exp(s_i - s_j) delta_j x_j + exp(s_i) C_i S_in (+ skip, gate);
 *   S_out = exp(s_last) S_in + sum_j exp(s_last - s_j) delta_j B_j^T x_j.
 *
 *   x, z, y : [B, L, H, P]  io dtype     (z may be NULL)
 *   delta   : [B, L, H]     io dtype
 *   A       : [H]           fp32, A_h < 0
 *   Bm, Cm  : [B, L, N]     io dtype, one group shared by all H heads
 *   Dskip   : [H]           fp32 or NULL
 *   h0      : [B, H, N, P]  fp32 or NULL (zeros)
 *   h_final : [B, H, N, P]  fp32 out, or NULL
 *   chunk   : chunk length Q >= 1 (0 = default 256). The last chunk is ragged
 *             when Q does not divide L. The result does not depend on Q beyond
 *             rounding; chunks above 256 steps run as 256-step chunks (one
 *             chunk's rows must fit a workgroup's LDS). The kernels tile a chunk
 *             by 32 rows, so a chunk that is not a multiple of 32 costs the work
 *             of the next multiple.
 * Supported: io = SSM_BF16; N in {64, 128}; P = 64; B, H <= 65535;
 * B * H < 2^23 (512 lanes each, in one grid dimension); L * H * P * 2 < 2^31.
 * ------------------------------------------------------------------------- */
size_t ssm_ssd_workspace_size(int B, int L, int H, int P, int N, int chunk);

int ssm_ssd_fwd(int B, int L, int H, int P, int N, int chunk, ssm_dtype_t io,
                const void* x, const void* delta, const float* A,
                const void* Bm, const void* Cm, const float* Dskip,
                const void* z, const float* h0,
                void* y, float* h_final,
                void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * ssm_step -- one-token recurrent decode step, state read and written in place.
 *
 * Defined by "Efficient Sequence Modeling: From S4 to Mamba-3", section 03
 * System (mamba_minimal.py's incremental step() for decoding) and section 09
 * Validation (step() equals a full forward): one iteration of the ssm_scan_fwd
 * recurrence above, per (b, d), on the state [b, d, :] held in place.
 *
 *   state  : [B, D, N]  fp32, updated in place
 *   x, delta, z, y : [B, D]  io dtype   (z may be NULL)
 *   A      : [D, N]  fp32
 *   Bm, Cm : [B, N]  io dtype
 *   Dskip  : [D]     fp32 or NULL
 * Supported: N in {4, 8, 16, 32, 64, 128, 256}; B <= 65535; D * N <= 2^32.
 * ------------------------------------------------------------------------- */
int ssm_step(int B, int D, int N, ssm_dtype_t io,
             float* state, const void* x, const void* delta, const float* A,
             const void* Bm, const void* Cm, const float* Dskip, const void* z,
             void* y, void* stream);

/* ssm_step_ex -- ssm_step with disc, delta_bias and delta_softplus as in
 * ssm_scan_fwd_ex (all N of ssm_step), so a sequence prefilled with
 * ssm_scan_fwd_ex continues token by token with the same options. */
int ssm_step_ex(int B, int D, int N, ssm_dtype_t io, ssm_disc_t disc,
                const float* delta_bias, int delta_softplus,
                float* state, const void* x, const void* delta, const float* A,
                const void* Bm, const void* Cm, const float* Dskip, const void* z,
                void* y, void* stream);

/* ---------------------------------------------------------------------------
 * ssm_ssd_step -- one-token decode step of the Mamba-2 form, state in place
 * (the incremental step of "Efficient Sequence Modeling: From S4 to Mamba-3",
 * section 03, applied to mamba2_minimal.py's per-head scalar decay and (N, P)
 * state). Per batch b and head h, with a = exp(delta[b,h] * A[h]):
 *   S[n, p] = a * S[n, p] + delta[b,h] * Bm[b,n] * x[b,h,p]
 *   y[b,h,p] = (sum_n Cm[b,n] * S[n, p] + Dskip[h] * x[b,h,p]) * silu(z[b,h,p])
 *
 *   state  : [B, H, N, P]  fp32, updated in place
 *   x, z, y : [B, H, P]    io dtype   (z may be NULL)
 *   delta  : [B, H]        io dtype
 *   A      : [H]           fp32
 *   Bm, Cm : [B, N]        io dtype, shared by all heads
 *   Dskip  : [H]           fp32 or NULL
 * Supported: P = 64; N in {16, 32, 64, 128, 256}; B * H <= 2^31 - 1.
 * Errors as for ssm_step; every pointer must be 16-byte aligned.
 * ------------------------------------------------------------------------- */
int ssm_ssd_step(int B, int H, int P, int N, ssm_dtype_t io,
                 float* state, const void* x, const void* delta, const float* A,
                 const void* Bm, const void* Cm, const float* Dskip, const void* z,
                 void* y, void* stream);

/* ---------------------------------------------------------------------------
 * ssm_linattn_fwd -- linear attention with a decay for each head (prefill).
 *
 * The SSD recurrence with a constant decay per head and queries and keys of
 * their own per head (or per group of heads, as B and C groups): per (b, h), with
 * lam = exp(log_decay[h]) and g = h / (H / G), from S = h0[b, h] (or zeros), for
 * t = 0 .. len_b - 1:
 *   S[i, j]   = lam * S[i, j] + k[b,t,g,i] * v[b,t,h,j]
 *   o[b,t,h,j] = scale * sum_i q[b,t,g,i] * S[i, j]
 *   h_final[b, h] = S after step len_b - 1.
 * Rows t >= len_b are padding: their q, k, v are not used and their o is 0.
 *
 *   q, k      : [B, L, G, K]  io dtype; G divides H
 *   v, o      : [B, L, H, V]  io dtype
 *   log_decay : [H]           fp32, <= 0 (0: no decay; -infinity: the current
 *                             token only)
 *   scale     : factor of o (usually 1 / sqrt(K))
 *   seqlens   : [B] int32 or NULL (every length L); a value outside [0, L] is
 *               taken as the nearest of the two
 *   h0        : [B, H, K, V]  fp32 or NULL (zeros)
 *   h_final   : [B, H, K, V]  fp32 out, or NULL
 *   norm      : NULL, or the group norm and gate that follow: o becomes
 *               ((o - mean) rstd weight + bias) silu(z) with the statistics of each
 *               head's V values of a token, exactly what ssm_group_norm_fwd gives
 *               on the stored o viewed as [B L, 1, H V] with H groups (padding
 *               rows: what that gives for a row of zeros)
 *   workspace : at least ssm_linattn_workspace_size(B, L, H, G, K, V, io) bytes
 * Arithmetic: fp32 state and accumulators. With io = SSM_BF16 the matrix cores take
 * the stored values exactly and what is formed in fp32 (the state, the decayed scores)
 * as pairs of bf16 numbers (about 17 significant bits, below the rounding of o); what
 * enters the state itself as triples (24 bits) where h_final is given, as pairs where
 * not, so o may differ in its last bit between the two. With io = SSM_F32 every product
 * is fp32.
 * A row that is not finite reaches the rows from its own on, and may reach the rows
 * before it in its chunk of 64 (a product with a zero weight); padding rows reach none.
 * Supported: K, V in {64, 128}; B, H <= 65535; B * H <= 2^22; L <= 2^30; with norm H * V
 * <= 65536 and B * L * H <= 2^30. Every pointer must be 16-byte aligned. Outputs must not
 * alias inputs or each other (the same address is refused). Errors as for ssm_scan_fwd.
 * ------------------------------------------------------------------------- */
typedef struct {
    const float* weight; /* [H * V] fp32 or NULL (ones) */
    const float* bias;   /* [H * V] fp32 or NULL (zeros) */
    const void* z;       /* gate, the shape and dtype of o, or NULL (no gate) */
    float eps;           /* > 0, added to the variance */
} ssm_linattn_norm_t;

size_t ssm_linattn_workspace_size(int B, int L, int H, int G, int K, int V, ssm_dtype_t io);

int ssm_linattn_fwd(int B, int L, int H, int G, int K, int V, ssm_dtype_t io,
                    const void* q, const void* k, const void* v, const float* log_decay,
                    float scale, const int* seqlens, const float* h0,
                    const ssm_linattn_norm_t* norm,
                    void* o, float* h_final,
                    void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * ssm_linattn_bwd -- gradient of ssm_linattn_fwd (without norm).
 *
 * For the loss  l = sum(dout * o) + sum(dh_final * h_final)  every output is dl/d(the
 * input of the same name), with n = len_b, T = dh_final:
 *   dq_i = scale (sum_{j<=i} lam^(i-j) (dout_i . v_j) k_j + lam^(i+1) h0 dout_i)
 *   dk_j = scale  sum_{i>=j} lam^(i-j) (dout_i . v_j) q_i + lam^(n-1-j) T v_j
 *   dv_j = scale  sum_{i>=j} lam^(i-j) (q_i . k_j) dout_i + lam^(n-1-j) T^t k_j
 *   dh0  = lam^n T + scale sum_i lam^(i+1) q_i (x) dout_i
 * dq and dk of a head group are the sums over its heads (fp32, in head order,
 * rounded once). The decay is a constant of the model and has no gradient here.
 *
 *   inputs   : q, k, v, log_decay, scale, seqlens, h0 exactly as given to ssm_linattn_fwd
 *   dout     : [B, L, H, V]  io dtype (rows t >= len_b are not used)
 *   dh_final : [B, H, K, V]  fp32 or NULL (zeros)
 *   dq, dk   : [B, L, G, K]  io dtype out (0 at padding)
 *   dv       : [B, L, H, V]  io dtype out (0 at padding)
 *   dh0      : [B, H, K, V]  fp32 out, or NULL (not written)
 *   workspace: at least ssm_linattn_bwd_workspace_size(B, L, H, G, K, V, io) bytes
 * States are recomputed, not read from a forward call; reductions run in a fixed
 * order. Arithmetic as in ssm_linattn_fwd (triples for dh0's state). Supported sizes,
 * alignment, aliasing and errors as for ssm_linattn_fwd.
 * ------------------------------------------------------------------------- */
size_t ssm_linattn_bwd_workspace_size(int B, int L, int H, int G, int K, int V, ssm_dtype_t io);

int ssm_linattn_bwd(int B, int L, int H, int G, int K, int V, ssm_dtype_t io,
                    const void* q, const void* k, const void* v, const float* log_decay,
                    float scale, const int* seqlens, const float* h0,
                    const void* dout, const float* dh_final,
                    void* dq, void* dk, void* dv, float* dh0,
                    void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * ssm_linattn_step -- one-token decode step of ssm_linattn_fwd, state in place.
 *
 *   state : [B, H, K, V]  fp32, updated in place
 *   q, k  : [B, G, K]     io dtype;  v, o : [B, H, V]  io dtype
 *   norm  : as for ssm_linattn_fwd (z: [B, H, V]); here the norm takes o before it
 *           is rounded to the io dtype
 * Supported: K, V in {64, 128}; B, H <= 65535; B * H <= 2^22. Every pointer must be
 * 16-byte aligned; o and state must not alias each other or another argument. Errors as
 * for ssm_step.
 * ------------------------------------------------------------------------- */
int ssm_linattn_step(int B, int H, int G, int K, int V, ssm_dtype_t io,
                     float* state, const void* q, const void* k, const void* v,
                     const float* log_decay, float scale, const ssm_linattn_norm_t* norm,
                     void* o, void* stream);

/* ---------------------------------------------------------------------------
 * ssm_group_norm_fwd -- group norm over channels-last data, with an activation
 * and / or a gate: the output stage of linear attention (S = 1, G = heads, gate z),
 * and the norm of the convolutional blocks around a scan (S positions, SiLU).
 *
 * Group g holds the channels c with c / (C / G) = g. Per sample m and group g,
 * over the S * (C / G) values of that sample and group:
 *   mean[m, g], var (biased), rstd[m, g] = 1 / sqrt(var + eps)
 *   u = (x[m,s,c] - mean) * rstd * weight[c] + bias[c]
 *   y[m,s,c] = act(u) * silu(z[m,s,c])
 *
 *   x, z, y      : [M, S, C]  io dtype (z may be NULL: no gate); y may be x
 *   weight, bias : [C]        fp32, each may be NULL (ones, zeros)
 *   mean, rstd   : [M, G]     fp32 out, both given or both NULL
 *   act          : SSM_ACT_NONE or SSM_ACT_SILU
 *   eps          : > 0
 *   workspace    : at least ssm_group_norm_workspace_size(M, S, C, G, io) bytes
 * Statistics are fp32, from squared distances to a mean (no difference of large
 * sums). Supported: C >= 1 a multiple of G, C <= 65536; M >= 0 and S >= 1 (M = 0 does
 * nothing); M * S * C <= 2^38, M * S <= 2^30, M * G <= 2^30. Every pointer must be
 * 16-byte aligned. But for y and x, outputs must not alias inputs or each other (the
 * same address is refused). Errors as for ssm_scan_fwd.
 * ------------------------------------------------------------------------- */
typedef enum { SSM_ACT_NONE = 0, SSM_ACT_SILU = 1, SSM_ACT_INT_RANGE_ = 0x7fffffff } ssm_act_t;

size_t ssm_group_norm_workspace_size(int M, int S, int C, int G, ssm_dtype_t io);

int ssm_group_norm_fwd(int M, int S, int C, int G, ssm_dtype_t io, ssm_act_t act,
                       const void* x, const float* weight, const float* bias, const void* z, float eps,
                       void* y, float* mean, float* rstd,
                       void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * ssm_group_norm_bwd -- gradient of ssm_group_norm_fwd.
 *
 *   x, weight, bias, z, act : as given to ssm_group_norm_fwd; mean, rstd: its outputs
 *   dy            : [M, S, C]  io dtype
 *   dx            : [M, S, C]  io dtype out
 *   dweight, dbias: [C]        fp32 out, each may be NULL (not written); given or not
 *                              whether weight and bias are
 *   dz            : [M, S, C]  io dtype out; given exactly when z is
 *   workspace     : at least ssm_group_norm_bwd_workspace_size(M, S, C, G, io) bytes
 * Outputs must not alias inputs or each other. Sums over samples and positions run
 * in a fixed order. M = 0 writes dweight = dbias = 0. Sizes and errors as for
 * ssm_group_norm_fwd.
 * ------------------------------------------------------------------------- */
size_t ssm_group_norm_bwd_workspace_size(int M, int S, int C, int G, ssm_dtype_t io);

int ssm_group_norm_bwd(int M, int S, int C, int G, ssm_dtype_t io, ssm_act_t act,
                       const void* x, const float* weight, const float* bias, const void* z,
                       const float* mean, const float* rstd, const void* dy,
                       void* dx, float* dweight, float* dbias, void* dz,
                       void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * ssm_glr_fwd -- gated linear recurrence (prefill): a state per channel whose decay
 * is gated by the input of every token. Per (b, d), from h = h0[b, d] (or 0), for
 * t = 0 .. len_b - 1, with sigma the logistic function:
 *   SSM_GLR_DECAY    a = exp(A[d] sigma(r[b,t,d])),  u = sqrt(1 - a^2) sigma(i[b,t,d]) x[b,t,d]
 *                    (the real-gated linear recurrent unit of De et al., arXiv
 *                    2402.19427, 2024; the factor keeps the state's variance that of the gated input)
 *   SSM_GLR_CONVEX   a = 1 - sigma(r[b,t,d]),        u = sigma(r[b,t,d]) x[b,t,d]
 *                    (the minimal gated unit of Feng et al., "Were RNNs all we needed?", 2024)
 *   h = a h + u
 *   y[b,t,d] = h * silu(z[b,t,d])
 *   h_final[b, d] = h after step len_b - 1.
 * Rows t >= len_b are padding: their inputs are not used, their y is 0.
 *
 *   x, r, i, z : [B, L, D]  io dtype, rows ld[0..3] elements apart (i: given exactly with
 *                SSM_GLR_DECAY; z may be NULL: no gate)
 *   A          : [D]        fp32, in [-2^100, 0] (SSM_GLR_DECAY; else NULL)
 *   ld         : HOST array of the row strides of x, r, i, z in elements (slices of one
 *                projection's rows; row t of batch b at (b L + t) ld), or NULL: D each. The
 *                entry of an absent tensor is not read.
 *   seqlens    : [B] int32 or NULL (every length L); a value outside [0, L] is taken as
 *                the nearest of the two
 *   h0         : [B, D]     fp32 or NULL (zeros)
 *   y          : [B, L, D]  io dtype out
 *   h_final    : [B, D]     fp32 out, or NULL
 *   states     : [B, ceil(L / SSM_GLR_STATE_STEPS), D] fp32 out, or NULL: the state entering
 *                every SSM_GLR_STATE_STEPS-th step, which ssm_glr_bwd takes
 *   workspace  : at least ssm_glr_workspace_size(B, L, D) bytes, for one call at a time
 * Arithmetic: fp32; 1 - a^2 by a series where a is close to 1. Order of the sums: fixed by the
 * sizes, io and whether x, r, i and z hold whole pairs of bf16 (D, every row stride and every
 * address in elements even). Calls alike in that give the same bits; a slice at an odd channel
 * gives those of another order.
 * A value that is not finite stays in its channel and sequence, from its own step on.
 * A sequence is one: its state is not reset inside (documents packed into one row need a call
 * each, or rows of a padded batch), and its first step is scaled by sqrt(1 - a^2) as the others.
 * Tiles of a sequence wait for one another within the launch. A wait that took some seconds would
 * give up: what depends on it becomes NaN (the call has returned and reports no status).
 * Supported: B <= 65535; L <= 2^30; D <= 2^18; ld in [D, 2^24]; B ceil(L / 128) ceil(D / 64)
 * <= 2^30. x, r, i and z must be aligned to their element, every other pointer to 16 bytes.
 * Outputs must not alias inputs or each other (the same address is refused). Errors as for
 * ssm_scan_fwd.
 * ------------------------------------------------------------------------- */
#define SSM_GLR_STATE_STEPS 128
typedef enum { SSM_GLR_DECAY = 0, SSM_GLR_CONVEX = 1, SSM_GLR_INT_RANGE_ = 0x7fffffff } ssm_glr_form_t;

size_t ssm_glr_workspace_size(int B, int L, int D);

int ssm_glr_fwd(int B, int L, int D, ssm_dtype_t io, ssm_glr_form_t form,
                const void* x, const void* r, const void* i, const float* A, const void* z,
                const int* ld, const int* seqlens, const float* h0,
                void* y, float* h_final, float* states,
                void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * ssm_glr_bwd -- gradient of ssm_glr_fwd.
 *
 * For the loss  l = sum(dy * y) + sum(dh_final * h_final)  every output is dl/d(the input of
 * the same name). With g_t the gradient of h_t (from the right: g_t = dy_t silu(z_t) +
 * a_{t+1} g_{t+1}, the last step's plus dh_final):
 *   SSM_GLR_DECAY    m = sqrt(1 - a^2), s = sigma(r), q = sigma(i):
 *                    dx = g m q,  di = g m x q (1 - q),  w = g (a h_{t-1} - a^2 q x / m),
 *                    dr = w A s (1 - s),  dA = sum over b, t of w s
 *                    (where m rounds to 0 the term with 1 / m is 0, its limit in dr)
 *   SSM_GLR_CONVEX   k = sigma(r):  dx = g k,  dr = g (x - h_{t-1}) k (1 - k)
 *   dz = dy h silu'(z),  dh0 = a_0 g_0.
 *
 *   inputs     : x, r, i, A, z, ld, seqlens as given to ssm_glr_fwd; states: its output
 *   dy         : [B, L, D]  io dtype (rows t >= len_b are not used)
 *   dh_final   : [B, D]     fp32 or NULL (zeros)
 *   dx, dr, di, dz : [B, L, D] io dtype out, 0 at padding; di is given exactly when i is, dz
 *                exactly when z is
 *   dA         : [D]        fp32 out; given exactly when A is
 *   dh0        : [B, D]     fp32 out, or NULL (not written)
 *   workspace  : at least ssm_glr_bwd_workspace_size(B, L, D) bytes, for one call at a time
 * Sums over b and t run in a fixed order; orders and waits as for ssm_glr_fwd, and so are sizes,
 * alignment, aliasing and errors. L = 0 writes dh0 = dh_final and dA = 0.
 * ------------------------------------------------------------------------- */
size_t ssm_glr_bwd_workspace_size(int B, int L, int D);

int ssm_glr_bwd(int B, int L, int D, ssm_dtype_t io, ssm_glr_form_t form,
                const void* x, const void* r, const void* i, const float* A, const void* z,
                const int* ld, const int* seqlens, const float* states,
                const void* dy, const float* dh_final,
                void* dx, void* dr, void* di, float* dA, void* dz, float* dh0,
                void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * ssm_glr_step -- one-token decode step of ssm_glr_fwd, state in place.
 *
 *   state      : [B, D]  fp32, updated in place
 *   x, r, i, z : [B, D]  io dtype, rows ld[0..3] elements apart (ld NULL: D each)
 *   y          : [B, D]  io dtype out
 * Supported: B * D <= 2^30; any ld >= D. Sizes, alignment and errors otherwise as for
 * ssm_glr_fwd; y and state must not alias each other or another argument.
 * ------------------------------------------------------------------------- */
int ssm_glr_step(int B, int D, ssm_dtype_t io, ssm_glr_form_t form,
                 float* state, const void* x, const void* r, const void* i, const float* A,
                 const void* z, const int* ld, void* y, void* stream);

/* ---------------------------------------------------------------------------
 * ssm_add_norm_fwd -- what stands between two layers of a residual network: the last
 * layer's output x is dropped out, added to the residual stream, and the sum normed for the
 * next layer. Per row m, over its C channels:
 *   s = residual + dropout(x)
 *   SSM_NORM_LAYER   y = (s - mean) * rstd * weight + bias,  rstd = 1 / sqrt(var + eps) (biased)
 *   SSM_NORM_RMS     y = s * rstd * weight + bias,           rstd = 1 / sqrt(mean of s^2 + eps)
 *
 *   x, y          : [M, C]  io dtype; y may be x
 *   residual, sum : [M, C]  res dtype (SSM_F32, or that of io); residual may be NULL (zero);
 *                   sum (s, rounded to res once; y is made from s before that) may be NULL
 *                   (not written) or residual
 *   weight, bias  : [C]     fp32, each may be NULL (ones, zeros)
 *   mean, rstd    : [M]     fp32 out, each may be NULL; mean must be NULL with SSM_NORM_RMS
 *   p, rng        : dropout probability and generator as for ssm_dropout (p = 0: none, rng
 *                   may be NULL)
 *   eps           : > 0
 * Statistics are fp32, the variance from squared distances to the mean. Supported: 1 <= C <=
 * 16384; M >= 0, M * C <= 2^38, M <= 2^30. Every pointer must be 16-byte aligned. But for y
 * and x, sum and residual, outputs must not alias inputs or each other (the same address is
 * refused). Errors as for ssm_scan_fwd.
 * ------------------------------------------------------------------------- */
typedef enum { SSM_NORM_LAYER = 0, SSM_NORM_RMS = 1, SSM_NORM_INT_RANGE_ = 0x7fffffff } ssm_norm_t;

int ssm_add_norm_fwd(int M, int C, ssm_dtype_t io, ssm_dtype_t res, ssm_norm_t norm,
                     const void* x, const void* residual, const float* weight, const float* bias,
                     float eps, double p, const unsigned long long* rng,
                     void* y, void* sum, float* mean, float* rstd, void* stream);

/* ---------------------------------------------------------------------------
 * ssm_add_norm_bwd -- gradient of ssm_add_norm_fwd.
 *
 *   sum, mean, rstd : its outputs (x with res = io where there was neither residual nor
 *                     dropout; mean NULL with SSM_NORM_RMS)
 *   weight, p, rng  : as given to it
 *   dy              : [M, C]  io dtype
 *   dsum            : [M, C]  res dtype, what else the sum's gradient holds (the residual
 *                     stream's from later layers), or NULL
 *   dresidual       : [M, C]  res dtype out, or NULL: the gradient of s; may be dsum
 *   dx              : [M, C]  io dtype out, or NULL: dropout of the gradient of s. One of the
 *                     two is given at least.
 *   dweight, dbias  : [C]     fp32 out, each may be NULL (not written); given or not whether
 *                     weight and bias were
 *   workspace       : at least ssm_add_norm_bwd_workspace_size(M, C, io, res) bytes, for one
 *                     call at a time; not used (NULL) without dweight and dbias
 * Sums over rows run in a fixed order. But for dresidual and dsum, outputs must not alias
 * inputs or each other. M = 0 writes dweight = dbias = 0. Sizes and errors as for
 * ssm_add_norm_fwd.
 * ------------------------------------------------------------------------- */
size_t ssm_add_norm_bwd_workspace_size(int M, int C, ssm_dtype_t io, ssm_dtype_t res);

int ssm_add_norm_bwd(int M, int C, ssm_dtype_t io, ssm_dtype_t res, ssm_norm_t norm,
                     const void* sum, const float* weight, const float* mean, const float* rstd,
                     const void* dy, const void* dsum, double p, const unsigned long long* rng,
                     void* dx, void* dresidual, float* dweight, float* dbias,
                     void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * ssm_dropout -- dropout whose mask is drawn from a counter and never stored. The same call
 * on dy with the same rng is its gradient.
 *   y[m,c] = x[m,c] * scale where the element is kept, else 0
 *
 *   p        : in [0, 1); least = p * 65536 rounded to the nearest whole number (ties to even)
 *              must be below 65536. An element is kept where its 16 bits are >= least, and
 *              scale = 65536 / (65536 - least): the mean is exact for the rounded p.
 *   rng      : DEVICE array {seed, offset}, read when the kernel runs, so that a captured graph
 *              draws anew when the caller advances it; may be NULL where least = 0
 *   The bits : row m's channels 8k .. 8k + 7 share block offset + m * ceil(C / 8) + k (mod 2^64),
 *              whose number (low word first, then two zero words) is encrypted by Philox-4x32-10
 *              (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3", 2011) under the
 *              seed's two words (low first); channel 8k + j takes half j % 2 (0: the low one) of
 *              word j / 2. A call uses ssm_dropout_blocks(M, C) = M * ceil(C / 8) blocks: the
 *              next offset is that much further.
 *   x, y     : [M, C]  io dtype; y may be x
 * Sizes as for ssm_add_norm_fwd but C <= 2^24; every pointer must be 16-byte aligned.
 * ------------------------------------------------------------------------- */
unsigned long long ssm_dropout_blocks(int M, int C);

int ssm_dropout(int M, int C, ssm_dtype_t io, const void* x, double p, const unsigned long long* rng,
                void* y, void* stream);

/* ---------------------------------------------------------------------------
 * Diagnostics for benchmarks (not part of the method; asynchronous on `stream`,
 * time them with events on that stream).
 *
 * ssm_diag_valu_rate: `blocks` workgroups of 256 lanes, each lane running 8
 *   independent chains for `iters` rounds of 4 dependent ops: mode 0 v_exp_f32
 *   only, mode 1 v_fma_f32 only, mode 2 one v_exp_f32 per three v_fma_f32, mode 3
 *   v_sin_f32 only, mode 4 v_cos_f32 only (so blocks * 256 * 32 * iters ops in
 *   all). out: blocks * 256 floats (a sum per lane, so nothing is optimised away).
 * ssm_diag_stream_scale: p[i] *= s for i < n, in place (n a multiple of 4): what a
 *   kernel that only reads and writes an array of the decode state's size reaches.
 * ssm_diag_copy: dst[i] = src[i] (n a multiple of 4): the byte reference that
 *   scales HBM byte counters.
 * ssm_diag_linattn_plan: how ssm_linattn_fwd (gradient = 0) or ssm_linattn_bwd
 *   (gradient = 1) cuts a sequence; no GPU call. plan[0] chunks of 64 steps,
 *   plan[1] super-chunks of plan[2] chunks each (one workgroup each), plan[3] pieces
 *   of plan[4] chunks each that what a super-chunk adds to the state is formed in,
 *   plan[5] heads that share a workgroup in dq and dk.
 * Pointers are device pointers (but for plan), 16-byte aligned. Errors as for the entry points.
 * ------------------------------------------------------------------------- */
int ssm_diag_valu_rate(int mode, int blocks, int iters, float* out, void* stream);
int ssm_diag_stream_scale(float* p, size_t n, float s, void* stream);
int ssm_diag_copy(const float* src, float* dst, size_t n, void* stream);
int ssm_diag_linattn_plan(int B, int L, int H, int G, int K, int V, ssm_dtype_t io, int gradient, int plan[6]);

#ifdef __cplusplus
}
#endif
#endif /* SSM_SCAN_H */
