/*
 * pn.h -- C interface of libpn, a GPU engine that evaluates nonlinear
 * recurrences s_t = f_t(s_{t-1}), t = 1..T, in parallel over time.
 *
 * Method: the web article "并行牛顿方法：加速非线性序列评估的计算革命" (a survey of
 * parallel Newton methods for nonlinear sequence evaluation; cited below as
 * [PN §x]).  The whole trajectory s = (s_1..s_T) is the unknown of a
 * fixed-point problem F(s) = 0 [PN §1.2] with
 *     F_t(s) = s_t - f_t(s_{t-1}),   s_0 given,
 * and is improved by s <- s - J~^{-1}(s) F(s), where J~ is I minus the
 * sub-diagonal of approximated state Jacobians A~_t ~ df_t/ds_{t-1}:
 *     Jacobi        A~_t = 0                      [PN §1.2]
 *     Picard        A~_t = I                      [PN §1.2, §2.2.3]
 *     quasi-Newton  A~_t = diag(df_t/ds_{t-1})    [PN §2.2.1]
 *     banded        A~_t = band_k(df_t/ds_{t-1})  [PN §2.2.2]
 *                   (entries with |i - j| <= k kept, the rest zero)
 *     Newton        A~_t = df_t/ds_{t-1} (dense)  [PN §1.2]
 * Applying J~^{-1} is the first-order linear recurrence
 *     s^_t = v_t + A~_t (s^_{t-1} - p_t),  p_t = s_{t-1},  v_t = f_t(p_t),
 * evaluated by an associative scan over affine maps [PN §2.1].
 *
 * Readings fixed by this library where the article is silent:
 *   - initial iterate s_t = s_0 for every t;
 *   - residual r = max over (b, t, d) of |F|, one stop rule for the batch;
 *   - stop at the first check with r non-finite (PN_NONFINITE), else with
 *     r <= tol (PN_OK), else when max_iter updates have been applied
 *     (PN_NOT_CONVERGED); the count reported is the number of updates;
 *   - damping lam in (0, 1] is step damping, s <- s + lam (s^ - s)
 *     [PN §4.3 suggests more damping when iterations stall];
 *   - windows [PN §1.3.1, §2.3]: consecutive blocks of W steps solved in
 *     order, window w starting from the last state of window w-1; or, with
 *     PN_WINDOW_ADVANCING, one window of W steps that slides past its
 *     converged prefix (below).
 *
 * Memory conventions (the solver and scan entries; the sequence-layer
 * operators state theirs where they are declared):
 *   - float pointers named params, x, s0, out, A, b are DEVICE pointers to
 *     C-contiguous float32 arrays owned by the caller; the library never
 *     frees them.
 *   - x is [B, T, m]; s0 is [B, D]; out is [B, T, D] and receives s_1..s_T.
 *   - pointers named *_hist, *_iters, iters_out, profile are HOST pointers.
 *   - calls block until the result is complete on the device.
 *   - on a negative (error) status the message is available from
 *     pn_last_error() on the calling thread.  Argument, size and workspace
 *     errors are found before any device work and leave out untouched; once
 *     kernels have been enqueued (PN_EHIP from a failed launch, copy or
 *     wait), out is unspecified.
 *   - out must not share a byte with x, s0 or params (PN_EINVAL otherwise).
 *   - thread-safe when concurrent calls use distinct streams and workspaces.
 */
#ifndef PN_H
#define PN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Transition maps f(p, x) (p = previous state, x = input at this step).
 *  PN_CELL_DIAG_TANH  f = tanh(a * p + x), channel-wise; params a[D];
 *                     input_dim must equal D.  Any D >= 1.
 *  PN_CELL_TANH_RNN   f = tanh(W p + U x + b); params W[D*D] | U[D*m] | b[D]
 *                     (row-major, W[i*D+k] multiplies p_k into output i).
 *                     1 <= D <= 64.
 *  PN_CELL_GRU        gated recurrent unit with torch.nn.GRU's equations and
 *                     gate order (r, z, n); params W_ih[3D*m] | W_hh[3D*D] |
 *                     b_ih[3D] | b_hh[3D].  1 <= D <= 64.
 *  PN_CELL_EULER_TANH f = p + h * (tanh(W p + U x + b) - p): one explicit
 *                     Euler step (per-channel step sizes h) of the
 *                     continuous-time RNN ds/dt = -s + tanh(W s + U x + b);
 *                     params W[D*D] | U[D*m] | b[D] | h[D].  1 <= D <= 64.
 * The RNN cells are the application the article names [PN §1.3.2]; the
 * Euler cell is the small-step regime of [PN §1.3.1, §2.2.3], where the
 * dynamics Jacobian is close to the identity. */
enum { PN_CELL_DIAG_TANH = 0, PN_CELL_TANH_RNN = 1, PN_CELL_GRU = 2, PN_CELL_EULER_TANH = 3 };

/* Jacobian approximations (see above).  Every cell supports every mode.
 * PN_BANDED takes its half-bandwidth k from pn_opts.bandwidth; band_0 is the
 * diagonal and band_{D-1} the whole matrix, so k = 0 runs as PN_QUASI_NEWTON
 * and k >= D-1 as PN_NEWTON (for the channel-wise cell every k runs as
 * PN_QUASI_NEWTON: its Jacobian is diagonal). */
enum { PN_JACOBI = 0, PN_PICARD = 1, PN_QUASI_NEWTON = 2, PN_NEWTON = 3, PN_BANDED = 4 };

/* Status codes. */
enum {
    PN_OK = 0,              /* converged: final r <= tol                       */
    PN_NOT_CONVERGED = 1,   /* max_iter updates applied; out = last iterate     */
    PN_NONFINITE = 2,       /* r became NaN/Inf; out = the offending iterate     */
    PN_EINVAL = -1,         /* bad argument (null pointer, negative size, ...)  */
    PN_EUNSUPPORTED = -2,   /* valid but unsupported shape (e.g. D > 64 RNN)    */
    PN_EHIP = -3,           /* a HIP runtime call failed                         */
    PN_EWORKSPACE = -4      /* workspace missing, misaligned or too small        */
};

typedef struct pn_cell {
    int32_t kind;        /* PN_CELL_*                                        */
    int32_t input_dim;   /* m, the width of x (>= 1; == D for DIAG_TANH)      */
} pn_cell;

/* Optional per-call measurements of the library's own kernels, taken with
 * HIP events on the call's stream.  They cover the steady-state launches of
 * the fused per-iteration "apply" kernel (cell + Jacobian + scan replay +
 * damping + residual + next chunk maps) for iterations i >= 1, including the
 * last launches, which find the loop stopped and exit at once; with
 * pn_opts.profile_stride n > 1, only every n-th of them (each event pair
 * adds stream work between launches).  Algorithmic bytes of a launch that
 * runs: read x and s^(i), write s^(i+1); 0 for a launch that exits. */
typedef struct pn_profile {
    double apply_ms;          /* summed device time of apply launches       */
    int32_t apply_launches;   /* timed launches, including early-exit ones    */
    double apply_bytes;       /* summed algorithmic bytes of those launches   */
    double apply_flops;       /* summed algorithmic flops: matrix-cell
                                 evaluations and, for Newton and the banded
                                 mode, the chunk-map compose with A~_t (a
                                 band of 2k+1 diagonals costs that fraction
                                 of the dense product; 0 for the
                                 channel-wise cell)                           */
    double total_ms;          /* first launch to last completion              */
} pn_profile;

typedef struct pn_opts {
    float damping;            /* (0, 1]; 1 = plain update                      */
    int32_t chunk;            /* timesteps per tile; 0 = library choice         */
    int64_t window;           /* 0 = whole horizon, else W >= 1                 */
    void* stream;             /* hipStream_t; NULL = the null stream            */
    void* workspace;          /* device memory, 256-byte aligned; NULL = the
                                 library allocates (stream-ordered) per call   */
    size_t workspace_bytes;
    float* resid_hist;        /* host; receives r_0..r_K of each window in
                                 order (truncated to resid_hist_len)           */
    int32_t resid_hist_len;
    int32_t* window_iters;    /* host; updates per window (truncated)          */
    int64_t window_iters_len;
    pn_profile* profile;      /* host; NULL = no event timing                   */
    int32_t flags;            /* PN_FLAG_* bits, 0 = defaults                    */
    int32_t bandwidth;        /* PN_BANDED half-bandwidth k >= 0 (default 1)    */
    int32_t window_mode;      /* PN_WINDOW_CONSECUTIVE (default) or
                                 PN_WINDOW_ADVANCING                            */
    int32_t* accepted;        /* host; advancing window: steps accepted at each
                                 check with a finite residual, in order
                                 (truncated to accepted_len)                   */
    int64_t accepted_len;
    int32_t switch_mode;      /* -1 (default): off; else the mode a window
                                 moves to when its residual stalls (below)     */
    float switch_ratio;       /* rho >= 0 of the stall test (default 0.5)      */
    int32_t* window_switch;   /* host; per window: the check that switched, or
                                 -1 (truncated to window_switch_len)           */
    int64_t window_switch_len;
    float switch_damping;     /* 0 (default): the damping stays `damping` after
                                 a switch; else, in (0, 1], the step damping of
                                 the updates after it (below)                  */
    int32_t profile_stride;   /* with profile: time every n-th steady apply
                                 launch (0 or 1: every one)                    */
} pn_opts;

/* Residual-driven switching [PN §5.3]: start each window on the coarse
 * approximation `mode` and move to `switch_mode` once the residual stalls.
 * At each check i >= 1 of a window still on `mode`, r_i > switch_ratio *
 * r_{i-1} switches it: update i (already under way) keeps `mode`, updates
 * i+1, ... use `switch_mode` (its chunk maps are rebuilt at s^(i+1) by one
 * extra sweep when it differs from `mode`) and, if switch_damping > 0, the
 * step damping switch_damping instead of `damping` -- the other remedy the
 * article gives for a stalling curve.  switch_mode == mode with
 * switch_damping set switches the damping alone.  Consecutive windows, float
 * storage (pn_eval_ex); PN_EUNSUPPORTED with the advancing window or
 * pn_eval_f16.  A typical use is quasi-Newton first, then the banded or full
 * Jacobian. */

/* pn_opts.window_mode.
 * PN_WINDOW_CONSECUTIVE: windows of W steps solved one after another, each
 *   to tol; max_iter caps the updates of each window; window_iters and
 *   resid_hist hold one entry / one run per window.
 * PN_WINDOW_ADVANCING (every cell; float storage; the sliding window of
 *   [PN §1.3.1]): steps [0, a) are accepted and never change again; the
 *   window is [a, min(T, a + W)).  Each round checks the current iterate on
 *   the window, r_t = max over (b, d) of |F_t|, and r = max_t r_t (stored in
 *   resid_hist); r not finite stops with PN_NONFINITE; otherwise a moves to
 *   the first t with r_t > tol (past the window if none), a = T stops with
 *   PN_OK, and after max_iter updates in total the solve stops with
 *   PN_NOT_CONVERGED.  The window then slides to [a, min(T, a + W)), steps
 *   entering it start from its last state, and one update of the chosen mode
 *   is applied to it.  *iters_out and window_iters[0] count the updates; on
 *   exit, steps the window never reached hold its last state.  Damping and
 *   every mode apply; PN_FLAG_PERSISTENT is ignored. */
enum { PN_WINDOW_CONSECUTIVE = 0, PN_WINDOW_ADVANCING = 1 };

/* pn_opts.flags.  PN_FLAG_PERSISTENT runs a solve of a matrix cell in a
 * diagonal mode as one cooperative launch (all windows and iterations, with
 * grid-wide barriers between the carry and apply phases), when the device
 * supports cooperative launches and the weights fit in LDS; otherwise, and by
 * default, each phase is its own launch.  Results meet the same bar; on
 * MI355X a grid barrier costs more than a launch boundary, so the default is
 * the faster one for the shapes measured here. */
enum { PN_FLAG_PERSISTENT = 1 };

/* pn_opts.flags.  By default the library runs some solves in one launch:
 *  - a matrix cell with D <= 8 whose windows hold at most 1024 (D <= 4) or
 *    512 (D <= 8) (b, t) pairs, in one workgroup, every window, iteration
 *    and check included (float storage, consecutive windows, no switching,
 *    chunk 0, max_iter <= 16384);
 *  - a matrix cell in a diagonal mode (Jacobi, Picard, quasi-Newton) with D
 *    padded to 16, 32 or 64, float storage and no switching, as one
 *    cooperative launch of workgroups that each keep a chunk on chip, when
 *    all chunks fit on the device at once: consecutive windows of at most
 *    128 chunks (max_iter <= 16384), or the advancing window, whose
 *    acceptance decisions and window moves are then taken on the device
 *    (max_iter below ceil(T / W) * (W + 1) and below 65536, the capacity of
 *    its residual history).
 * PN_FLAG_MULTI_LAUNCH keeps such a solve on the launch-per-phase driver
 * instead.  Results meet the same bar either way. */
enum { PN_FLAG_MULTI_LAUNCH = 2 };

/* Fill *o with the defaults: damping 1, chunk 0, window 0, bandwidth 1,
 * switch_mode -1, switch_ratio 0.5, switch_damping 0, profile_stride 1,
 * everything else NULL / 0. */
void pn_opts_init(pn_opts* o);

/* Solve the recurrence for all B sequences [PN §1.1, §1.2].
 *   cell      host struct, read during the call only.
 *   params    device, float32, layout per cell kind (above).
 *   x         device [B, T, m];  s0 device [B, D].
 *   mode      PN_JACOBI .. PN_BANDED (PN_BANDED needs opts->bandwidth >= 0;
 *             pn_eval without options uses k = 1).
 *   tol       stop when r <= tol (tol >= 0; 0 runs to max_iter unless r == 0).
 *   max_iter  cap on updates per window (>= 0).
 *   out       device [B, T, D].  iters_out host int32: total updates applied
 *             over all windows.
 * Returns a status code.  B, T or D equal to 0 is an empty problem: PN_OK
 * with *iters_out = 0 and nothing written. */
int pn_eval(const pn_cell* cell, const float* params, const float* x, const float* s0,
            int64_t B, int64_t T, int64_t D, int32_t mode, float tol, int32_t max_iter,
            float* out, int32_t* iters_out);

/* pn_eval with options (opts may be NULL = defaults). */
int pn_eval_ex(const pn_cell* cell, const float* params, const float* x, const float* s0,
               int64_t B, int64_t T, int64_t D, int32_t mode, float tol, int32_t max_iter,
               float* out, int32_t* iters_out, const pn_opts* opts);

/* pn_eval_ex for callers that cannot allocate device memory (serving loops
 * and harnesses that forbid allocation during a call): the same solve, with
 * the same arguments, options and results, run on a static device scratch
 * that the library holds on each GPU it runs on until the process ends
 * (32 MiB, enough for every workload in this repository's benchmarks).  The
 * call itself allocates nothing: no device or pinned memory, no events.
 * opts->workspace must be NULL and opts->profile NULL (PN_EINVAL otherwise);
 * a problem whose workspace (pn_workspace_bytes) exceeds the scratch less
 * 256 bytes of check records returns PN_EWORKSPACE before any device work.
 * The host reads each convergence check back with a copy after draining the
 * stream, so iterations do not overlap the host's reading as in pn_eval_ex.
 * Every call on a GPU shares that GPU's scratch, which keeps the contents
 * of the last call (the library clears what must start at zero): calls that
 * overlap on one GPU, from any threads or streams, race and must not be
 * made. */
int pn_eval_noalloc(const pn_cell* cell, const float* params, const float* x, const float* s0,
                    int64_t B, int64_t T, int64_t D, int32_t mode, float tol, int32_t max_iter,
                    float* out, int32_t* iters_out, const pn_opts* opts);

/* Bytes of workspace pn_eval_ex (and pn_eval_f16) needs for this problem
 * with these options (opts may be NULL).  The size depends on the window and
 * also on the chunk, the mode switch and the bandwidth, so the whole option
 * block is taken rather than the window alone.  Returns 0 and sets the last
 * error for invalid or unsupported arguments. */
size_t pn_workspace_bytes(const pn_cell* cell, int64_t B, int64_t T, int64_t D,
                          int32_t mode, const pn_opts* opts);

/* pn_eval_ex with reduced-precision storage [PN §2.3, §4.2]: x and out hold
 * IEEE binary16 values (device, same shapes and layouts as pn_eval); params
 * and s0 stay float32 and all arithmetic is float32.  Every stored state is
 * rounded to nearest-even binary16, and the iteration continues from the
 * stored (rounded) states, so tol must lie above the binary16 resolution of
 * the states (about 2.4e-4 for |s| < 1).  Supported for PN_CELL_DIAG_TANH,
 * solved as one window (opts->window 0 or >= T, consecutive mode);
 * PN_EUNSUPPORTED otherwise.  With D even, x and out must be 4-byte aligned
 * (two channels move per access).  pn_workspace_bytes covers this entry
 * too.  It moves 6 bytes per state element and iteration instead of 12. */
int pn_eval_f16(const pn_cell* cell, const float* params, const uint16_t* x, const float* s0,
                int64_t B, int64_t T, int64_t D, int32_t mode, float tol, int32_t max_iter,
                uint16_t* out, int32_t* iters_out, const pn_opts* opts);

/* The scan step alone [PN §2.1]: out_t = A_t out_{t-1} + b_t, out_0 = s0,
 * for t = 1..T.  A is device [B, T, D] (dense = 0: diagonal A_t) or
 * [B, T, D, D] (dense = 1, row-major, 1 <= D <= 64); b device [B, T, D];
 * s0 device [B, D]; out device [B, T, D], sharing no byte with the inputs.
 * Diagonal A runs in one pass with a decoupled look-back over 32-step
 * chunks (A and b read once, out written once); dense A composes chunk
 * maps, scans their carries and replays (opts->chunk steps per chunk, 0 =
 * 32).  Uses opts->stream and opts->workspace (NULL: allocated per call);
 * returns PN_OK or an error code. */
int pn_affine_scan(const float* A, const float* b, const float* s0, int64_t B, int64_t T,
                   int64_t D, int32_t dense, float* out, const pn_opts* opts);

/* Workspace bytes for pn_affine_scan. */
size_t pn_affine_scan_workspace_bytes(int64_t B, int64_t T, int64_t D, int32_t dense,
                                      const pn_opts* opts);

/* ------------------------------------------------------------------------
 * Sequence-layer operators: the linear recurrence with a matrix state
 * (linear attention with a decay per head), and what prepares its queries
 * and keys (rotation by position, norm per head).
 *
 * Conventions of this part:
 *   - every field of the argument blocks is 8 bytes wide (a double, an
 *     int64_t or a pointer); pointers are DEVICE pointers unless named host;
 *   - token tensors are [B, T, heads, channels] in one storage type (PN_F32,
 *     PN_BF16, PN_F16), channels adjacent, the other strides free and given
 *     in elements (0 broadcasts an input); outputs are C-contiguous;
 *   - states are C-contiguous float32 [B, H, dk, dv]; sums, norms and states
 *     are held in at least float32, with one rounding of the result at the
 *     end.  The matrix products of linear attention take their float32
 *     operands as sums of bfloat16 parts: three, 24 bits, for float32 storage
 *     and for states that are results; two, to 2^-16 of each operand, where
 *     only outputs in 16-bit storage come of them (their error against 64 bits
 *     is that of their last rounding either way).  float32 elements and states
 *     beyond 3.389e38, the largest bfloat16, count as infinite there;
 *   - calls ENQUEUE their kernels on `stream` (hipStream_t, NULL = the null
 *     stream) and return without waiting, so they can be captured into a
 *     graph; nothing is allocated: a workspace is given by the caller,
 *     256-byte aligned (PN_EWORKSPACE otherwise), and is free for reuse by
 *     later work of the same stream;
 *   - sizes, strides, pointers and overlaps are checked on the host before
 *     any launch (PN_EINVAL, PN_EUNSUPPORTED, the latter also for more
 *     sequences and heads than a launch holds: by their sizes, from 2.8 million
 *     in the attention's gradients, 2^24 in steps); a size of 0 is an empty
 *     problem (PN_OK; what has elements left is still written, as a state);
 *   - indices held in device memory (positions, lengths, slots) are bounded
 *     in the kernels as each entry states: no value of theirs reads or
 *     writes outside the arrays given. */
enum { PN_F32 = 0, PN_BF16 = 1, PN_F16 = 2 };

/* A token tensor [B, T, heads, channels]: strides in elements. */
typedef struct pn_tokens {
    void* p;
    int64_t sb, st, sh;
} pn_tokens;

/* table[p][i] = magnitude * (cos, sin)(p * freq[i]), computed in float64 and
 * rounded once: float32 [n_pos, n_freq, 2].  freq is a HOST array of n_freq
 * (1 .. 128) float64 angles per position. */
int pn_rotary_table(const double* freq_host, int64_t n_freq, int64_t n_pos, double magnitude,
                    float* table, void* stream);

/* Arguments of pn_rotary, pn_qk_norm_rotary and its backward.
 * Rotation: of the first R (even, 0 <= R <= D) of D (1 .. 256) channels,
 * channel pairs (i, i + R/2), or (2i, 2i + 1) if interleaved, turn by the
 * angle of table row p: (a, b) -> (a c - b s, b c + a s); the other channels
 * pass.  p = positions[b * pos_sb + t * pos_st] (int32, or int64 if pos64),
 * or offset + t if positions is NULL; a p outside [0, n_pos) gives NaN in the
 * rotated channels. */
typedef struct pn_rotary_args {
    int64_t dtype, B, T, D, R, interleaved;
    int64_t inverse;            /* pn_rotary: 1 turns back (the gradient)       */
    int64_t hq, hk;             /* heads of q and k; hk = 0: no k                */
    pn_tokens q, k;             /* inputs                                       */
    void *q_out, *k_out;        /* contiguous [B, T, hq | hk, D]                 */
    const float* table;         /* [n_pos, R/2, 2]                              */
    int64_t n_pos;
    const void* positions;
    int64_t pos64, pos_sb, pos_st, offset;
    double eps;                 /* norm entries: x / sqrt(mean x^2 + eps), the
                                   mean in float32: rows of elements past 1e18
                                   come out as 0                                */
    const float *qw, *kw;       /* norm weights, float32 [D] or [heads, D]; NULL = 1 */
    int64_t qw_sh, kw_sh;       /* 0: one [D] for all heads, D: one per head      */
    pn_tokens dq, dk;           /* backward: gradients of q_out and k_out         */
    float *dqw, *dkw;           /* backward: gradients of the weights, shaped as
                                   they are (written where qw / kw is given)     */
    void* workspace;
    int64_t workspace_bytes;
    void* stream;
} pn_rotary_args;

/* Rotation alone, of q and (hk > 0) k.  q_out may be q itself (in place, if
 * q is contiguous), likewise k_out; other overlaps are PN_EINVAL. */
int pn_rotary(const pn_rotary_args* a);
/* Norm of each head's channels, times its weight, then the rotation, in one
 * pass.  In place as above. */
int pn_qk_norm_rotary(const pn_rotary_args* a);
/* Gradients: dq, dk come in (of the outputs), q_out and k_out receive the
 * gradients of q and k, dqw and dkw those of the weights (sums in a fixed
 * order: the same bits on every run).  No output may overlap an input. */
int pn_qk_norm_rotary_backward(const pn_rotary_args* a);
/* Workspace bytes of pn_qk_norm_rotary_backward (the other two need none), a
 * function of sizes alone; 256 means that none is needed, 0 invalid
 * arguments, with the error set.  Pointers are not looked at. */
size_t pn_qk_norm_rotary_workspace_bytes(const pn_rotary_args* a);

/* Linear attention with a decay per head.  For each sequence and head,
 *     S_t = lam S_{t-1} + k_t^T v_t,   o_t = scale * q_t S_t,
 * lam = exp(log_decay[h]), S_0 = initial_state or 0.  log_decay <= 0 in use;
 * -inf is a state that holds the current token only, and growth is allowed as
 * far as lam^T is finite in float32.
 * q has H heads; k and v have HK heads, H a multiple of HK: head h uses key
 * and value head h / (H / HK).  1 <= dk, dv <= 256.
 * lengths (int32 [B], NULL = T each; values are clamped to [0, T]): tokens at
 * and after lengths[b] are padding: never read, their rows of the outputs 0,
 * and final_state is the state after lengths[b] tokens.  A NaN or infinity
 * in a token reaches the outputs from that token on, as NaN or infinity, and
 * may reach those of the up to 31 tokens before it (in the gradients of k and
 * v, which run backwards, after it).  An infinite element of a state stays
 * infinite (lam > 0), and the outputs of its channel are NaN or infinite. */
typedef struct pn_linattn_args {
    int64_t dtype, B, T, H, HK, dk, dv;
    double scale;
    const float* log_decay;     /* [H]                                          */
    const int32_t* lengths;     /* [B] or NULL                                  */
    pn_tokens q, k, v;
    const float* initial_state; /* [B, H, dk, dv] or NULL (zeros)                */
    void* o;                    /* forward: [B, T, H, dv]                        */
    float* final_state;         /* forward: [B, H, dk, dv] or NULL               */
    pn_tokens do_;              /* backward: gradient of o                       */
    const float* d_final_state; /* backward: gradient of final_state, or NULL    */
    void *dq, *dk_, *dv_;       /* backward: [B, T, H, dk], [B, T, HK, dk | dv]   */
    float* d_initial_state;     /* backward: [B, H, dk, dv] or NULL              */
    void* workspace;
    int64_t workspace_bytes;
    void* stream;
} pn_linattn_args;

/* All T tokens of every sequence (prompts, training). */
int pn_linear_attention(const pn_linattn_args* a);
/* Gradients of q, k, v (summed over the heads that share them) and of the
 * initial state; the decay is a constant of the layer. */
int pn_linear_attention_backward(const pn_linattn_args* a);
/* Workspace bytes of the two, a function of dtype and sizes alone; 256 means
 * that none is needed (workspace may be NULL), 0 invalid arguments, with the
 * error set.  Pointers are not looked at. */
size_t pn_linear_attention_workspace_bytes(const pn_linattn_args* a, int32_t backward);

/* One token for each of B sequences (serving): the state is updated in place
 * and o_t returned.  q, k, v: [B, heads, channels] (st is not used).  state
 * is a pool [n_slots, H, dk, dv]; sequence b owns slot slots[b] (int32), or
 * slot b if slots is NULL (then n_slots >= B).  A slot outside [0, n_slots)
 * marks an idle row: o is 0 there and no state is touched.  Two rows of one
 * call must not name the same slot. */
typedef struct pn_linattn_step_args {
    int64_t dtype, B, H, HK, dk, dv;
    double scale;
    const float* log_decay;     /* [H]                                          */
    pn_tokens q, k, v;
    float* state;
    const int32_t* slots;       /* [B] or NULL                                  */
    int64_t n_slots;
    void* o;                    /* [B, H, dv]                                   */
    void* stream;
} pn_linattn_step_args;

int pn_linear_attention_step(const pn_linattn_step_args* a);

/* ------------------------------------------------------------------------
 * State-space operators: the diagonal recurrence whose decay depends on the
 * token (a selective scan), the short causal convolution in front of it, and
 * the norms that join a block to its residual stream.  The conventions above
 * hold; tokens here are [B, T, D] (pn_tokens' sh is not used) unless stated.
 * lengths (int32 [B], NULL = T each; values are clamped to [0, T]): tokens at
 * and after lengths[b] are padding: never read, their rows of the outputs 0,
 * and final states those after lengths[b] tokens.  Sums over tokens or
 * channels run in a fixed order: the same bits on every run. */

/* Causal convolution of each channel with W (1 .. 8) taps,
 *     y_t = act(bias + sum_{k < W} weight[d][k] x_{t - W + 1 + k}),
 * act(v) = v / (1 + e^-v), or v if activation is 0.  Tokens before the first
 * come from initial_state [B, W - 1, D] (the storage type; the last row is
 * the newest), or are 0.  final_state holds the last W - 1 tokens, of the
 * initial state where the sequence is shorter. */
typedef struct pn_conv_args {
    int64_t dtype, B, T, D, W, activation;
    const float *weight, *bias; /* [D, W]; [D] or NULL                          */
    const int32_t* lengths;
    pn_tokens x;
    const void* initial_state;  /* [B, W - 1, D] or NULL                         */
    void *y, *final_state;      /* forward: [B, T, D]; [B, W - 1, D] or NULL      */
    pn_tokens dy;               /* backward: gradient of y                       */
    const void* d_final_state;  /* backward: [B, W - 1, D] or NULL                */
    void* dx;                   /* backward: [B, T, D]                           */
    float *dweight, *dbias;     /* backward: [D, W]; [D] or NULL                  */
    void* d_initial_state;      /* backward: [B, W - 1, D] or NULL                */
    void* workspace;
    int64_t workspace_bytes;
    void* stream;
} pn_conv_args;

int pn_short_conv(const pn_conv_args* a);
int pn_short_conv_backward(const pn_conv_args* a);
/* Workspace bytes of pn_short_conv_backward (the forward needs none), a
 * function of dtype and sizes alone; 256 means that none is needed, 0 invalid
 * arguments, with the error set.  Pointers are not looked at. */
size_t pn_short_conv_workspace_bytes(const pn_conv_args* a);

/* One token for each of B sequences: x and y [B, D]; state is a pool
 * [n_slots, W - 1, D] in the storage type, which drops its oldest token for
 * this one.  Slots as in pn_linear_attention_step. */
typedef struct pn_conv_step_args {
    int64_t dtype, B, D, W, activation;
    const float *weight, *bias;
    pn_tokens x;
    void* state;
    const int32_t* slots;       /* [B] or NULL                                  */
    int64_t n_slots;
    void* y;                    /* [B, D]                                       */
    void* stream;
} pn_conv_step_args;

int pn_short_conv_step(const pn_conv_step_args* a);

/* Selective scan.  For each channel d with N (1 .. 128) states,
 *     delta_t = softplus(dt_t + dt_bias[d])   (without softplus: the sum),
 *     h_t = exp(delta_t A[d]) h_{t-1} + delta_t x_t b_t,
 *     y_t = (c_t . h_t + skip[d] x_t) * gate_t / (1 + e^-gate_t),
 * h_0 = initial_state or 0; a NULL dt_bias is 0, a NULL skip leaves its term
 * out, a NULL gate.p the gate.  x, dt, gate [B, T, D]; b and c [B, T, G, N],
 * D a multiple of G: channel d reads group d / (D / G).  A is finite, < 0 in
 * use; growth is allowed as far as exp(A[d] sum delta) over the tokens is
 * finite in float32, and the gradient of delta_t as far as it is.  The token
 * strides of x, dt, gate, b, c and dy go up to
 * 2^26 elements, D up to 2^24.  Steps and decays are float32: exp(delta A) to
 * (2 |delta A| + 2) 2^-24 of itself, 0 below 2^-126.  A NaN or infinity in a
 * token reaches that token's outputs and those after it (in the gradients also
 * those before it), as NaN or infinity. */
typedef struct pn_ssm_args {
    int64_t dtype, B, T, D, N, G, softplus;
    const float *A, *skip, *dt_bias;    /* [D, N]; [D] or NULL; [D] or NULL       */
    const int32_t* lengths;
    pn_tokens x, dt, gate, b, c;
    const float* initial_state;         /* [B, D, N] or NULL (zeros)              */
    void* y;                            /* forward: [B, T, D]                    */
    float* final_state;                 /* forward: [B, D, N] or NULL             */
    pn_tokens dy;                       /* backward: gradient of y               */
    const float* d_final_state;         /* backward: of final_state, or NULL      */
    void *dx, *ddt, *dgate, *db, *dc;   /* backward: shaped as the inputs (dgate
                                           written where the gate is given)      */
    float *dA, *dskip, *ddt_bias;       /* backward: shaped as the inputs (the last
                                           two written where their input is given) */
    float* d_initial_state;             /* backward: [B, D, N] or NULL            */
    void* workspace;
    int64_t workspace_bytes;
    void* stream;
} pn_ssm_args;

int pn_ssm_scan(const pn_ssm_args* a);
int pn_ssm_scan_backward(const pn_ssm_args* a);
/* Workspace bytes of the two, a function of dtype and sizes alone; 256 means
 * that none is needed, 0 invalid arguments, with the error set.  Pointers are
 * not looked at.  The backward's holds the states of every eighth token and
 * shares of db and dc: 0.6 to 0.8 bytes for each state of each token (B T D N; N
 * counts as 4, 8 or a multiple of 16, the channels of a group as a multiple of
 * 32, or of 64 or 128 where that adds little), 0.7 GB for 8 x 4096 tokens of 2048
 * channels with 16 states, up to 2 bytes where tokens are few.  Sequences taken
 * in several calls need it for those of one call; their sums are then added by
 * the caller. */
size_t pn_ssm_scan_workspace_bytes(const pn_ssm_args* a, int32_t backward);

/* One token for each of B sequences: x, dt, gate, y [B, D], b and c
 * [B, G, N]; state is a pool float32 [n_slots, D, N], updated in place.  Slots
 * as in pn_linear_attention_step. */
typedef struct pn_ssm_step_args {
    int64_t dtype, B, D, N, G, softplus;
    const float *A, *skip, *dt_bias;
    pn_tokens x, dt, gate, b, c;
    float* state;
    const int32_t* slots;       /* [B] or NULL                                  */
    int64_t n_slots;
    void* y;                    /* [B, D]                                       */
    void* stream;
} pn_ssm_step_args;

int pn_ssm_step(const pn_ssm_step_args* a);

/* The norms around a block.  For each token of D (1 .. 8192) channels,
 *     u = x * gate / (1 + e^-gate)                 (x without a gate),
 *     p = post_weight * u / sqrt(mean u^2 + eps)   (u without post_weight),
 *     s = residual + scale * p                     (scale NULL: 1; residual.p NULL: 0),
 *     y = weight * s / sqrt(mean s^2 + eps)        (not computed without weight):
 * x is what a block gives, s the residual stream after it and y what the next
 * block takes.  x, gate, y and their gradients have the storage type, the
 * residual, s and theirs residual_dtype: the storage type or PN_F32.  Means
 * are float32 sums of squares: a row whose squares sum past 3.4e38 (elements
 * of u, or of s, past sqrt(3.4e38 / D): 4e17 with 2048 channels) comes out of
 * that norm as 0, and passes it no gradient.  eps is taken in float32, and
 * squares below 1e-38 are lost beside it: with an eps of 0, rows of elements
 * under 1e-19 come out too large, infinite or NaN.
 * The backward takes what the forward took, and forms s again. */
typedef struct pn_block_norm_args {
    int64_t dtype, residual_dtype, B, T, D;
    double eps;
    const float *weight, *post_weight, *scale;   /* float32 [D] or NULL            */
    pn_tokens x, gate, residual;                 /* [B, T, D]; p NULL: none         */
    void *y, *s;                /* forward: contiguous [B, T, D]; y where weight is given */
    pn_tokens dy, ds;           /* backward: gradients of y (where weight is given) and of
                                   s (p NULL: 0)                                 */
    void *dx, *dgate, *dresidual;   /* backward: [B, T, D]; dgate where the gate is given,
                                   dresidual or NULL                             */
    float *dweight, *dpost_weight, *dscale;      /* backward, where the input is given */
    void* workspace;
    int64_t workspace_bytes;
    void* stream;
} pn_block_norm_args;

int pn_block_norm(const pn_block_norm_args* a);
int pn_block_norm_backward(const pn_block_norm_args* a);
/* Workspace bytes of pn_block_norm_backward (the forward needs none), a
 * function of types and sizes alone, and of which of weight, post_weight and
 * scale are given; 256 means that none is needed, 0 invalid arguments, with
 * the error set. */
size_t pn_block_norm_workspace_bytes(const pn_block_norm_args* a);

/* Message of the last error on this thread ("" if none).  The pointer stays
 * valid until the next library call on the same thread. */
const char* pn_last_error(void);

/* Library version string, e.g. "pn 0.1.0 gfx950". */
const char* pn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PN_H */
