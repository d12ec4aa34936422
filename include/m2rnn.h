/*
 * m2rnn.h — C ABI of the MI355X (gfx950) M²RNN recurrence library (libm2rnn.so).
 *
 * The operation is the M²RNN matrix-state nonlinear recurrence of the reading notes
 * "M²RNN：矩阵状态非线性 RNN 的容量、表达力与系统代价" on arXiv:2603.14360v2 ("M²RNN notes"):
 * for every batch entry b and head n, independently, starting from H_0 (zeros, or a given state),
 *
 *     Z_t = tanh(H_{t-1} W_n + k_t v_t^T)          (§2.1, Eq. 10)
 *     H_t = f_t H_{t-1} + (1 - f_t) Z_t             (§2.1, Eq. 11)
 *     y_t = H_t^T q_t + w_r,n (.) v_t               (§2.1, Eq. 12)
 *
 * with H_t a K x V state, W_n a V x V matrix per head (right-multiplied, so it mixes the value
 * dimension only: (H W)[i][j] = sum_l H[i][l] W[l][j]), f_t a scalar per (batch, step, head),
 * and w_r,n a V-vector per head.  The backward is the chain-rule BPTT of §2.7.
 *
 * Conventions shared by every call
 * --------------------------------
 *  - Tensor layouts are contiguous row-major:
 *        q, k      [B, T, Nqk, K]   (dtype given by qkv_dtype; Nqk = N, or 1 when all value heads
 *                                    share one query/key, the notes' multi-value layout §2.4)
 *        v         [B, T, N, V]     (dtype given by qkv_dtype)
 *        f         [B, T, N]        fp32, expected in [0, 1] (not checked, computed as given)
 *        W         [N, V, V]        fp32
 *        w_r       [N, V]           fp32
 *        H0, H_T   [B, N, K, V]     fp32
 *        y, dy     [B, T, N, V]     fp32
 *    Gradients have the shape of their input and are fp32.
 *  - Every array pointer is a DEVICE pointer on the current HIP device, 16-byte aligned.  The
 *    caller owns all memory, including the workspace, and every stream: the library allocates no
 *    device memory and keeps no state that one call leaves for another (bar m2rnn_fwd_noalloc's
 *    fixed array, below; the host side caches only device and kernel attributes, under a lock),
 *    so calls on different streams may run concurrently.
 *  - Work is enqueued on `stream` (a hipStream_t; NULL = the null stream) and the call returns
 *    without synchronising.  Outputs are valid once the stream reaches that point.
 *  - Outputs are overwritten, never accumulated.  Outputs must not alias inputs or each other.
 *  - Arguments are validated on the host before anything is enqueued; an invalid call returns
 *    an error status and touches no memory.  M2RNN_EHIP reports a launch failure
 *    (m2rnn_last_hip_error() gives the hipError_t of the most recent one on this thread).
 *  - Supported sizes: V in {16, 32, 64, 128}; K a positive multiple of 16; B, T, N >= 0;
 *    Nqk in {0, 1, N}; one batch entry's slice of a tensor below 2 GiB (T N max(K, V) fp32 values),
 *    whatever the batch (whole tensors may exceed 4 GiB); B N K / 16 below 2^31.
 *    T = 0 is legal: y is empty and H_T = H0 (or zeros).
 */
#ifndef M2RNN_H_
#define M2RNN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct m2rnn_dims {
  int64_t B; /* batch */
  int64_t T; /* steps */
  int64_t N; /* heads */
  int64_t K; /* key size: rows of the state */
  int64_t V; /* value size: columns of the state, side of W */
  int64_t Nqk; /* heads of q and k: N (one query/key per head) or 1 (one query/key shared by all
                  N value heads, §2.4: N_q = N_k = 1); 0 means N.  With Nqk = 1, dq and dk are
                  the gradients of the shared q and k, summed over the heads (§2.7). */
} m2rnn_dims;

/* dtype of q, k, v.  E4M3 (OCP 8-bit: 1 sign, 4 exponent and 3 mantissa bits, largest number 448) is an output of
 * m2rnn_add_norm_fwd only. */
enum { M2RNN_DTYPE_F32 = 0, M2RNN_DTYPE_BF16 = 1, M2RNN_DTYPE_E4M3 = 2 };

/* How the per-step contraction H_{t-1} W runs on the matrix cores.  The state, the
 * accumulation and everything outside the contraction are fp32 in every mode.
 *   F32     fp32 MFMA (v_mfma_f32_16x16x4_f32).
 *   F16X3   split precision: H = H_hi + H_lo and W = W_hi + W_lo, all four fp16 (H_lo, W_lo the
 *           fp16 rounding remainders); H W ~ W_hi H_hi + W_lo H_hi + W_hi H_lo on fp16 MFMA with
 *           fp32 accumulation (about 22 significant bits per product).
 *   BF16X3  split precision with bf16 halves: W_hi H_hi + W_lo H_hi + W_hi H_lo.
 *   BF16    one bf16 pass: bf16(W) bf16(H) (coarse; meant for a 2e-2 error budget).
 *   AUTO    the forwards' default: BF16X3 (measured as fast as F16X3 at the 16K-token
 *           workload, with the full fp32 exponent range; about 3e-6 max-abs error on the state
 *           where F16X3 gives 3e-7, both far inside a 5e-4 budget).  The backward's own
 *           contraction is F16X3 (below).
 * Range of the split modes: the contraction takes 2 log2(e) W (so that tanh is one exp2) and the
 * state as 16-bit halves.  F16X3 needs |W| < 65504 / (2 log2 e) ~ 22700 elementwise and a state
 * below 65504 (with f in [0, 1] the state stays within max(|H0|, 1), Eq. 11); the fp16 remainder is
 * subnormal below about 6e-5, so its absolute rounding is about 3e-8 whatever the value's size,
 * which the state's [-1, 1] range makes small.  Outside these bounds the results are undefined
 * (inf or NaN); they are not checked. */
enum { M2RNN_MATH_AUTO = -1, M2RNN_MATH_F32 = 0, M2RNN_MATH_F16X3 = 1, M2RNN_MATH_BF16X3 = 2, M2RNN_MATH_BF16 = 3 };

/* Status codes. */
enum {
  M2RNN_OK = 0,
  M2RNN_EINVAL = -1,      /* null required pointer, negative size, misaligned pointer, bad enum */
  M2RNN_EUNSUPPORTED = -2, /* K or V outside the supported set, or a mode not built */
  M2RNN_EWORKSPACE = -3,   /* workspace missing or smaller than the *_workspace_size answer */
  M2RNN_EHIP = -4          /* a HIP launch or runtime call failed */
};

/* Library version, as MAJOR*10000 + MINOR*100 + PATCH.  The minor number changes with every
 * change of an entry point's arguments, the patch number when entry points are added; a caller
 * built against this header should check that m2rnn_version() == M2RNN_VERSION before calling
 * anything else. */
#define M2RNN_VERSION 402
int m2rnn_version(void);

/* Human-readable text for a status code (static storage). */
const char* m2rnn_status_string(int status);

/* hipError_t of the last HIP failure seen by this thread (0 if none). */
int m2rnn_last_hip_error(void);

/*
 * Overlap object: a side stream (default priority) and the events that fork work onto it from a
 * call's stream and join it back, on the device current at creation.  The forward calls below take
 * one to overlap the second pass of a long sequence with its scan (see m2rnn_fwd); NULL runs
 * everything on the call's stream.  The caller owns it: one object serves one call at a time, so
 * give each stream (or thread) that issues calls its own, and destroy it once its work is done.
 * Returns M2RNN_EHIP if the stream or an event cannot be made.
 */
typedef struct m2rnn_overlap_s* m2rnn_overlap;
int m2rnn_overlap_create(m2rnn_overlap* out);
int m2rnn_overlap_destroy(m2rnn_overlap overlap);

/*
 * Forward pass, Eq. (10)-(12).  One pass over all T steps for every (b, n).
 *
 *   row_blocks   0 = automatic (one, wherever that kernel keeps its state in registers);
 *                otherwise the number of 16-row blocks of the state that one workgroup carries
 *                (must divide K/16).  The K rows of a state evolve
 *                independently (W mixes only the value dimension, §1.2), so a (b, n) pair may be
 *                split over S = K/(16*row_blocks) workgroups; when S > 1 their partial readouts are
 *                summed by a second, deterministic pass.
 *   H0           initial state, or NULL for zeros.
 *   y            output [B,T,N,V] (may be NULL only when T == 0 or B*N == 0).
 *   H_T          final state [B,N,K,V], or NULL to skip it.
 *   workspace    device scratch of at least m2rnn_fwd_workspace_size() bytes (NULL if that is 0).
 *
 *   overlap      NULL, or an overlap object of the current device (see above).
 *
 * With split rows, T >= 4096 and an overlap object, m2rnn_fwd runs the sequence in two time
 * segments, the second starting from the state the first ended in, and the first segment's second
 * pass runs on the object's side stream while the second segment is scanned (the second segment is
 * sized to cover it); the call's stream waits for all of it before any later work.  This needs the
 * state buffer that m2rnn_fwd_workspace_size() adds for such shapes; with a smaller workspace (the
 * partial planes only), without an overlap object, or on a stream under graph capture, the single
 * pass runs instead.  The two ways of running give the same bits: H_t is a function of H_{t-1} and the
 * step's inputs only, and a scan started from a stored state computes exactly what a continuous
 * scan does.
 */
int m2rnn_fwd_workspace_size(const m2rnn_dims* dims, int qkv_dtype, int math, int row_blocks,
                             size_t* bytes);
int m2rnn_fwd(const m2rnn_dims* dims, int qkv_dtype, int math, int row_blocks, const void* q,
              const void* k, const void* v, const float* f, const float* W, const float* w_r,
              const float* H0, float* y, float* H_T, void* workspace, size_t workspace_bytes,
              void* stream, m2rnn_overlap overlap);

/*
 * m2rnn_fwd for callers that cannot allocate: code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc.  Same arguments as m2rnn_fwd without the workspace and the
 * overlap object; the same bits as m2rnn_fwd.  It allocates nothing: the partial readouts of split
 * rows and the states between time segments live in a fixed device array of the library
 * (m2rnn_fwd_noalloc_max_bytes() = 64 MiB; every device that runs the library holds one copy until
 * the process ends).  Long sequences run in time segments whose partial planes fit in it (each
 * segment's second pass on the call's stream).  Sizes whose two states and 16 steps of partial
 * planes do not fit return M2RNN_EUNSUPPORTED: 2 B N K V + 16 S B N V floats (S = partial planes,
 * K / 16 / row_blocks when the rows are split) at most.  When one workgroup carries all rows the
 * array is not used.  All calls on one device share the array: calls that overlap in time on one
 * device (on different streams, or from several threads) race, and must be ordered by the caller.
 */
int m2rnn_fwd_noalloc_max_bytes(size_t* bytes);
int m2rnn_fwd_noalloc(const m2rnn_dims* dims, int qkv_dtype, int math, int row_blocks, const void* q,
                      const void* k, const void* v, const float* f, const float* W, const float* w_r,
                      const float* H0, float* y, float* H_T, void* stream);

/*
 * The two launches of m2rnn_fwd's single pass, exposed so that a caller can time them apart.
 * Same arguments as m2rnn_fwd.  m2rnn_scan_fwd runs the recurrence over the whole sequence (it
 * writes y directly when one workgroup carries all K rows, else per-workgroup partial readouts
 * into the workspace); m2rnn_scan_fwd_finish then forms y = sum of partials + w_r (.) v, and is a
 * no-op when the scan already wrote y.  Calling both, in order, on one stream is exactly
 * m2rnn_fwd's single pass (see above for the time segments of long sequences).
 */
int m2rnn_scan_fwd(const m2rnn_dims* dims, int qkv_dtype, int math, int row_blocks, const void* q,
                   const void* k, const void* v, const float* f, const float* W, const float* w_r,
                   const float* H0, float* y, float* H_T, void* workspace, size_t workspace_bytes,
                   void* stream);
int m2rnn_scan_fwd_finish(const m2rnn_dims* dims, int qkv_dtype, int math, int row_blocks,
                          const void* q, const void* k, const void* v, const float* f,
                          const float* W, const float* w_r, const float* H0, float* y, float* H_T,
                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * Backward pass (BPTT of §2.7) for the loss L = sum_t <dy_t, y_t> + <dH_T, H_T>.
 *
 * The forward states are not taken from the caller: the library re-runs the recurrence and keeps
 * the state every I = m2rnn_checkpoint_interval() steps, then walks the `M2RNN_BWD_CHECKPOINT`-step
 * segments from last to first, recomputing each sub-segment's states from its checkpoint in
 * on-chip memory (the notes' §2.6 re-runs the recurrence at the start of the backward; here only
 * checkpoints are stored, not every state).
 *
 *   dH_T   upstream gradient of the final state, or NULL for zeros.
 *   grad_clip  0 for the exact gradient; > 0 clamps every element of the gradient that each step
 *          sends back to its input state, C_{t-1} = f_t R_t + D_t W^T, to [-grad_clip, grad_clip]
 *          before it is used (the per-step recurrent-gradient clipping of the notes' §2.3, read as
 *          an elementwise bound; dH0 is then the clamped C_0).  The readout gradient q_t u_t^T and
 *          dH_T enter unclamped.  Negative or NaN: M2RNN_EINVAL.
 *   dq, dk [B,T,Nqk,K]; dv [B,T,N,V]; df [B,T,N]; dW [N,V,V] and dw_r [N,V] summed over batch and
 *   time; dH0 [B,N,K,V] or NULL to skip it.  All fp32.
 *   math   M2RNN_MATH_F16X3 or M2RNN_MATH_AUTO (the other modes return M2RNN_EUNSUPPORTED).  The
 *          reverse scan recomputes the forward with F16X3 either way; the checkpoint pass that
 *          m2rnn_bwd runs first uses the forwards' default for AUTO and F16X3 for F16X3.
 *
 * Scale of dy.  Every gradient is linear in (dy, dH_T) jointly, and the walk holds the chain's
 * D_t = ((1 - f_t) R_t) (.) (1 - Z_t^2) in split fp16, whose accurate range is narrow.  So each
 * (b, n) pair runs at its own power-of-two scale: a first pass finds the largest |dy| and |dH_T|
 * of the pair, the walk takes 2^e dy and 2^e dH_T with the largest in [1, 2) (and the clip bound
 * 2^e grad_clip), and every gradient is multiplied by 2^-e before it is stored.  Both products
 * are exact, so the result for 2^k dy is exactly 2^k times the result for dy (over the whole
 * fp32 range of dy, bar fp32 underflow or overflow of the gradients themselves): training without
 * loss scaling, whose activation gradients are far below unit size, keeps the same accuracy.
 * W must satisfy |W| < 65504 elementwise (the chain multiplies by W^T in split fp16), and k
 * |k| < 65504 (dv = D^T k is formed on fp16 MFMA with k in one fp16 pass, a relative rounding of
 * 2^-12 per term, as dW's operands).
 */
#define M2RNN_BWD_CHECKPOINT 64
int m2rnn_bwd_workspace_size(const m2rnn_dims* dims, int qkv_dtype, int math, size_t* bytes);
int m2rnn_bwd(const m2rnn_dims* dims, int qkv_dtype, int math, const void* q, const void* k,
              const void* v, const float* f, const float* W, const float* w_r, const float* H0,
              const float* dy, const float* dH_T, float grad_clip, float* dq, float* dk, float* dv,
              float* df, float* dW, float* dw_r, float* dH0, void* workspace, size_t workspace_bytes,
              void* stream);

/*
 * Training pair: a forward that keeps the backward's checkpoints, and a backward that takes them
 * instead of re-running the recurrence.  The notes' §2.6 re-runs the recurrence at the start of the
 * backward so that the forward keeps no history; when a training step runs the forward anyway,
 * keeping only the states that enter every I-th step (an eighth to a sixty-fourth of the states)
 * lets the backward skip that re-run.
 *
 * m2rnn_fwd_ckpt     m2rnn_fwd (time segments included, with the same overlap argument and the
 *                    same bits) plus `ckpt` [B,N,ceil(T/I),K,V] fp32 with I = m2rnn_checkpoint_interval():
 *                    ckpt[b][n][s] is the state entering step I s (ckpt[b][n][0] = H0, or zeros).
 *                    Required when T > 0.
 * m2rnn_bwd_ckpt     m2rnn_bwd with `ckpt` from m2rnn_fwd_ckpt on the same inputs in place of H0
 *                    (H0 is ckpt[., ., 0]); its workspace (m2rnn_bwd_ckpt_workspace_size) excludes
 *                    the checkpoints.  Gradients equal m2rnn_bwd's when the forward used the
 *                    contraction of m2rnn_bwd's own checkpoint pass: the forwards' default for
 *                    math = AUTO, F16X3 for math = F16X3.  Checkpoints from another mode give
 *                    gradients that differ within that mode's error.
 */
/* Steps between checkpoints (I above): 8 for V <= 64, 64 for V = 128.  Smaller
 * intervals let the backward skip a forward pass over every segment; at V = 128 the state is large
 * and the backward runs that pass itself. */
int m2rnn_checkpoint_interval(const m2rnn_dims* dims, int64_t* steps);
int m2rnn_fwd_ckpt(const m2rnn_dims* dims, int qkv_dtype, int math, int row_blocks, const void* q,
                   const void* k, const void* v, const float* f, const float* W, const float* w_r,
                   const float* H0, float* y, float* H_T, float* ckpt, void* workspace,
                   size_t workspace_bytes, void* stream, m2rnn_overlap overlap);
int m2rnn_bwd_ckpt_workspace_size(const m2rnn_dims* dims, int qkv_dtype, int math, size_t* bytes);
int m2rnn_bwd_ckpt(const m2rnn_dims* dims, int qkv_dtype, int math, const void* q, const void* k,
                   const void* v, const float* f, const float* W, const float* w_r, const float* ckpt,
                   const float* dy, const float* dH_T, float grad_clip, float* dq, float* dk, float* dv,
                   float* df, float* dW, float* dw_r, float* dH0, void* workspace, size_t workspace_bytes,
                   void* stream);

/*
 * The launches of m2rnn_bwd_ckpt apart, so that a caller can time the reverse scan alone.  Same
 * arguments as m2rnn_bwd_ckpt.  m2rnn_scan_bwd runs the pass that finds each pair's scale (the
 * largest |dy|, |dH_T|) and the reverse scan, which writes dq, dk and dH0 (or per-head partials of
 * a shared q/k), and dv, df (or per-workgroup partials when a pair's rows are split) and per-
 * workgroup partials of dW, dw_r into the workspace; m2rnn_scan_bwd_finish sums those partials in a
 * fixed order.  Calling both, in order, on one stream with the same workspace is m2rnn_bwd_ckpt.
 */
int m2rnn_scan_bwd(const m2rnn_dims* dims, int qkv_dtype, int math, const void* q, const void* k,
                   const void* v, const float* f, const float* W, const float* w_r, const float* ckpt,
                   const float* dy, const float* dH_T, float grad_clip, float* dq, float* dk, float* dv,
                   float* df, float* dW, float* dw_r, float* dH0, void* workspace, size_t workspace_bytes,
                   void* stream);
int m2rnn_scan_bwd_finish(const m2rnn_dims* dims, int qkv_dtype, int math, const void* q, const void* k,
                          const void* v, const float* f, const float* W, const float* w_r,
                          const float* ckpt, const float* dy, const float* dH_T, float grad_clip, float* dq,
                          float* dk, float* dv, float* df, float* dW, float* dw_r, float* dH0,
                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * One step of Eq. (10)-(12) for every (b, n), with the state kept in device memory: the decode
 * (token-by-token inference) form of the layer.  The notes point out that inference carries a
 * fixed-size recurrent state (§2.6); this call reads it, advances it by one token and writes it
 * back, so its cost is the state traffic (about 8 K V bytes per (b, n)), not the contraction.
 *
 *   dims         T must be 1.  Layouts are those of m2rnn_fwd with T = 1:
 *                q, k [B,1,N,K]; v [B,1,N,V] (dtype qkv_dtype); f [B,1,N]; W [N,V,V]; w_r [N,V].
 *   H_in         the state before the step [B,N,K,V], or NULL for zeros.
 *   H_out        the state after the step [B,N,K,V].  H_out == H_in updates the state in place;
 *                any other overlap of the two is rejected (M2RNN_EINVAL).
 *   y            the readout of the step [B,1,N,V].
 *   math         M2RNN_MATH_F16X3 or M2RNN_MATH_AUTO (the other modes return M2RNN_EUNSUPPORTED).
 * No workspace.  Results equal m2rnn_fwd over one step with H0 = H_in, up to rounding order.
 */
int m2rnn_decode_step(const m2rnn_dims* dims, int qkv_dtype, int math, const void* q, const void* k,
                      const void* v, const float* f, const float* W, const float* w_r,
                      const float* H_in, float* H_out, float* y, void* stream);

/*
 * The steps on either side of the recurrence in the M²RNN block (§2.2, §2.3).  Each is an
 * HBM-bound stream with its backward; reductions over batch and time run in a fixed order.
 * Sizes are passed directly; every call enqueues on `stream` and validates arguments on the host
 * like the calls above.
 *
 * Gate (§2.2, Eq. 13/17): f = (1 + e^{a + beta})^{-alpha} = exp(-alpha softplus(a + beta)), with
 * a the gate pre-activation [B,T,N] (fp32) and alpha, beta [N] per head (alpha >= 0 keeps f in
 * [0, 1]; not checked).  f [B,T,N] fp32 is the recurrence's f.  The backward takes df (the
 * recurrence backward's gradient of f) and gives da [B,T,N] and dalpha, dbeta [N] (summed over
 * batch and time); its workspace holds B T N floats.  Pointers 4-byte aligned.
 */
int m2rnn_gate_fwd(int64_t B, int64_t T, int64_t N, const float* a, const float* alpha,
                   const float* beta, float* f, void* stream);
int m2rnn_gate_bwd_workspace_size(int64_t B, int64_t T, int64_t N, size_t* bytes);
int m2rnn_gate_bwd(int64_t B, int64_t T, int64_t N, const float* a, const float* alpha,
                   const float* beta, const float* df, float* da, float* dalpha, float* dbeta,
                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * Output gate + RMSNorm (§2.3, step 4; the norm's statistic and gradient as in Appendix C):
 *     x = y (.) SiLU(gz),   out = gamma (.) x / sqrt(mean_j x_j^2 + eps)
 * normalised over the D features of each of `rows` rows: y, out [rows, D] fp32 (for the layer's
 * y [B,T,N,V], rows = B T and D = N V, so the statistic spans all heads), gz the output gate's
 * pre-activation [rows, D] (gz_dtype fp32 or bf16), gamma [D] fp32.  The gate multiplies before
 * the norm.  eps >= 0 is the caller's (the notes leave it out).  D a multiple of 4, at most 8192.
 * The backward gives dy, dgz [rows, D] fp32 and dgamma [D] (summed over rows).  Pointers 16-byte
 * aligned.
 */
int m2rnn_out_norm_fwd(int64_t rows, int64_t D, const float* y, const void* gz, int gz_dtype,
                       const float* gamma, float eps, float* out, void* stream);
int m2rnn_out_norm_bwd_workspace_size(int64_t rows, int64_t D, size_t* bytes);
int m2rnn_out_norm_bwd(int64_t rows, int64_t D, const float* y, const void* gz, int gz_dtype,
                       const float* gamma, float eps, const float* dout, float* dy, float* dgz,
                       float* dgamma, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The block's forward from the gate pre-activation to the normalised output, for inference and
 * prefill (§2.2, §2.3 steps 2-4, Appendix C):
 *     f = exp(-alpha softplus(a + beta)),   y = M2RNN(q, k, v, f; W, w_r, H0)  (as m2rnn_fwd),
 *     out = gamma (.) x / sqrt(mean_j x_j^2 + eps),   x = y (.) SiLU(gz)  over the N V features of a token.
 * The gate goes into the workspace ([B,T,N], 1/V of y's size); then the scan, and one epilogue
 * pass per token that sums the scan's partial readouts, adds w_r (.) v and applies the output
 * gate and the norm, so y is never written to HBM (when one workgroup carries all K rows the scan
 * writes y to the workspace and the epilogue reads it once).  Long sequences run in time segments
 * as in m2rnn_fwd, each segment's epilogue on the overlap object's side stream (NULL: one pass).
 * out is bit-identical to
 * m2rnn_gate_fwd, m2rnn_fwd and m2rnn_out_norm_fwd in turn.  The backward needs y: a training
 * step takes those three calls instead.
 *   a            gate pre-activation [B,T,N] fp32; alpha, beta [N] fp32 (4-byte aligned).
 *   gz           output gate pre-activation [B,T,N,V] (gz_dtype fp32 or bf16); gamma [N V] fp32;
 *                eps >= 0.  N V at most 8192.
 *   out          [B,T,N,V] fp32.  The other arguments are m2rnn_fwd's.
 *   workspace    at least m2rnn_fwd_block_workspace_size() bytes.
 */
int m2rnn_fwd_block_workspace_size(const m2rnn_dims* dims, int qkv_dtype, int math, int row_blocks,
                                   size_t* bytes);
int m2rnn_fwd_block(const m2rnn_dims* dims, int qkv_dtype, int math, int row_blocks, const void* q,
                    const void* k, const void* v, const float* a, const float* alpha,
                    const float* beta, const float* W, const float* w_r, const float* H0,
                    const void* gz, int gz_dtype, const float* gamma, float eps, float* out,
                    float* H_T, void* workspace, size_t workspace_bytes, void* stream,
                    m2rnn_overlap overlap);

/*
 * Causal depthwise Conv1D of kernel size 4 + SiLU (§2.3, step 1), applied to each of q, k, v:
 *     u_t[c] = SiLU(sum_{i<4} w[c][i] x_{t-3+i}[c] + bias[c]),   x_t = 0 for t < 0
 * x, u [B,T,C] in `dtype` (fp32 or bf16; u is rounded to nearest even for bf16), w [C,4] fp32,
 * bias [C] fp32 or NULL (none).  C a multiple of 4.  The backward takes du [B,T,C] fp32 and gives
 * dx [B,T,C], dw [C,4] and dbias [C] (NULL to skip) fp32, summed over batch and time.  Pointers
 * 16-byte aligned.  T at most 2^31 - 257, B ceil(T/16) ceil(C/256) at most 2^31 - 1, and a launch holds fewer
 * than 2^32 threads (B ceil(T/64) ceil(C/256) at most 2^26 - 4, in the backward with T/128); larger sizes:
 * M2RNN_EUNSUPPORTED.
 */
int m2rnn_conv4_silu_fwd(int64_t B, int64_t T, int64_t C, int dtype, const void* x, const float* w,
                         const float* bias, void* u, void* stream);
int m2rnn_conv4_silu_bwd_workspace_size(int64_t B, int64_t T, int64_t C, size_t* bytes);
int m2rnn_conv4_silu_bwd(int64_t B, int64_t T, int64_t C, int dtype, const void* x, const float* w,
                         const float* bias, const float* du, float* dx, float* dw, float* dbias,
                         void* workspace, size_t workspace_bytes, void* stream);

/*
 * Selective state space scan: the linear recurrence with a scalar decay per head that hybrid stacks
 * place next to M²RNN blocks.  Per (b, n), from H_0 (zeros, or a given state),
 *
 *     D_t = softplus(a_t + beta),     f_t = exp(-alpha D_t)
 *     H_t = f_t H_{t-1} + D_t k_t v_t^T
 *     y_t = H_t^T q_t + w_r (.) v_t
 *
 * f_t is the M²RNN gate (m2rnn_gate_fwd) of the same a, alpha, beta; the step size D_t also scales
 * the write.  alpha >= 0 keeps f in [0, 1] (not checked, computed as given).
 *
 *   dims       as above, with K a multiple of 16 up to 128, and Nqk 0 (= N) or any divisor of N: query/key
 *              j serves the heads j N/Nqk .. (j + 1) N/Nqk - 1.  Tensors may exceed 4 GiB; B N (T / 32 + 64)
 *              must stay below 2^28, N at 2^20 at most, and in the backward, with c = B ceil(T / I) chunks (I: the
 *              checkpoint interval), c at 65535 * 64 at most and c Nqk (Nqk = 0: c N) below 2^24.
 *   a          gate pre-activation [B,T,N] fp32; alpha, beta [N] fp32; w_r [N,V] fp32 (a, alpha, beta
 *              and lens 4-byte aligned, everything else 16-byte).
 *   lens       [B] int32 device array or NULL: the steps of each batch entry, clamped to [0, T] (NULL:
 *              all T).  Steps at or past a sequence's end are not read (whatever they hold), their
 *              y is written as zeros, H_T is the state after the last step within, and their
 *              gradients are zeros.
 *   y          [B,T,N,V] fp32; H_T [B,N,K,V] fp32, or NULL to skip it.
 *   ckpt       m2rnn_ssm_fwd_ckpt also keeps the states that enter every I-th step for the backward,
 *              [B,N,ceil(T/I),K,V] fp32 with I = m2rnn_ssm_checkpoint_interval().
 *   workspace  at least the *_workspace_size() bytes (NULL if that is 0).  Long sequences with few heads
 *              run as time segments whose entering states are kept there.
 *
 * Products run on the bf16 MFMA with fp32 accumulation, every computed fp32 operand (decayed scores,
 * states, gradients) and fp32 input split into three bf16 planes (24 bits), so results are those
 * of fp32 arithmetic; the sums of log decays within a chunk are formed in fp64.  Values below 2^-110
 * may lose low bits.  a = -infinity masks a step (D = 0, f = 1).  Where any other value within a sequence is not
 * finite, the forward's outputs that depend on it (y from its step on, H_T, later checkpoints) are not finite
 * (an infinity may become NaN) and all others keep their bits; m2rnn_ssm_bwd expects finite values within the
 * sequences, a = -infinity apart (one that is not may reach every gradient of its chunk and the sums over it).
 * Two calls on the same inputs give the same bits, and need not equal another segmentation's.
 *
 * m2rnn_ssm_bwd gives the gradients of L = sum <dy, y> + <dH_T, H_T>: dq, dk [B,T,Nqk,K] (summed
 * over the heads that share them), dv [B,T,N,V], da [B,T,N], dalpha, dbeta [N], dw_r [N,V] and dH0
 * [B,N,K,V] (NULL to skip), all fp32, from m2rnn_ssm_fwd_ckpt's ckpt on the same inputs.
 */
int m2rnn_ssm_checkpoint_interval(int qkv_dtype, int64_t* steps);
int m2rnn_ssm_fwd_workspace_size(const m2rnn_dims* dims, int qkv_dtype, size_t* bytes);
int m2rnn_ssm_fwd(const m2rnn_dims* dims, int qkv_dtype, const void* q, const void* k, const void* v,
                  const float* a, const float* alpha, const float* beta, const float* w_r,
                  const int32_t* lens, const float* H0, float* y, float* H_T, void* workspace,
                  size_t workspace_bytes, void* stream);
int m2rnn_ssm_fwd_ckpt(const m2rnn_dims* dims, int qkv_dtype, const void* q, const void* k, const void* v,
                       const float* a, const float* alpha, const float* beta, const float* w_r,
                       const int32_t* lens, const float* H0, float* y, float* H_T, float* ckpt,
                       void* workspace, size_t workspace_bytes, void* stream);
int m2rnn_ssm_bwd_workspace_size(const m2rnn_dims* dims, int qkv_dtype, size_t* bytes);
int m2rnn_ssm_bwd(const m2rnn_dims* dims, int qkv_dtype, const void* q, const void* k, const void* v,
                  const float* a, const float* alpha, const float* beta, const float* w_r,
                  const int32_t* lens, const float* ckpt, const float* dy, const float* dH_T, float* dq,
                  float* dk, float* dv, float* da, float* dalpha, float* dbeta, float* dw_r, float* dH0,
                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * One step of the selective scan for every (b, n), the state in device memory (dims->T = 1; layouts
 * with T = 1).  H_in NULL: zeros.  H_out == H_in updates in place; any other overlap of the two is
 * rejected (M2RNN_EINVAL).  No workspace.  fp32 arithmetic.
 */
int m2rnn_ssm_step(const m2rnn_dims* dims, int qkv_dtype, const void* q, const void* k, const void* v,
                   const float* a, const float* alpha, const float* beta, const float* w_r,
                   const float* H_in, float* H_out, float* y, void* stream);

/*
 * The causal conv4 + SiLU for prompts and single tokens: m2rnn_conv4_silu_fwd with the three inputs
 * before the first step, and the three that the next call needs.
 *   win        [B,3,C] in `dtype`, oldest first: x_{-3}, x_{-2}, x_{-1}; NULL: zeros.
 *   win_out    [B,3,C]: the last three inputs of each sequence (of win and x together).
 *   lens       [B] int32 or NULL, as in m2rnn_ssm_fwd: x at or past a sequence's end is not read, its u is
 *              zeros.
 * In m2rnn_conv4_silu_fwd_state win and win_out must not overlap (M2RNN_EINVAL); T = 0 copies the
 * window.  m2rnn_conv4_silu_step takes x, u [B,C], and win_out may be win (any other overlap:
 * M2RNN_EINVAL).  x, u, win and win_out are aligned to four elements (8 bytes in bf16), w and bias to 16.
 * Sizes as in m2rnn_conv4_silu_fwd; in the step, B C at most 2^34 - 1024.
 */
int m2rnn_conv4_silu_fwd_state(int64_t B, int64_t T, int64_t C, int dtype, const void* x, const float* w,
                               const float* bias, const int32_t* lens, const void* win, void* u,
                               void* win_out, void* stream);
int m2rnn_conv4_silu_step(int64_t B, int64_t C, int dtype, const void* x, const float* w, const float* bias,
                          const void* win, void* u, void* win_out, void* stream);

/*
 * Norm of queries and keys per head, with the position rotation in the same pass (between the conv
 * and a scan or an attention):
 *     xn = gamma (.) x / sqrt(mean_j x_j^2 + eps) over the K features of each head, then the pairs
 *     p < R/2 of features (p, p + R/2), or (2p, 2p + 1) if `interleaved`, turned by pos * inv_freq[p]:
 *     (a, b) -> (a cos - b sin, b cos + a sin).  The last K - R features are not turned (R = 0: norm only).
 *   q [B,T,Nq,K], k [B,T,Nk,K] and q_out, k_out alike in `dtype` (fp32 or bf16); gamma_q, gamma_k
 *   [K] fp32; pos [B,T] int32 (any value, also negative); inv_freq [R/2] fp64, in radians per position.
 *   K a multiple of 16 up to 256, R a multiple of 8 up to K; Nq or Nk may be 0 (their pointers NULL).
 *   Angles are formed in fp64, so far positions keep their angle.  Pointers 16-byte aligned (pos 4).
 *   eps >= 0 (a head of zeros with eps = 0 is 0/0: NaN); the squares of a head are summed in fp32 and must
 *   stay within it (|x| below 1e18).
 * The backward takes the gradients of the outputs (fp32) and gives dq, dk (fp32) and dgamma_q, dgamma_k
 * [K], summed over batch, time and heads in a fixed order.
 */
int m2rnn_qk_norm_rope_fwd(int64_t B, int64_t T, int64_t Nq, int64_t Nk, int64_t K, int64_t R,
                           int interleaved, int dtype, const void* q, const void* k, const float* gamma_q,
                           const float* gamma_k, const int32_t* pos, const double* inv_freq, float eps,
                           void* q_out, void* k_out, void* stream);
int m2rnn_qk_norm_rope_bwd_workspace_size(int64_t B, int64_t T, int64_t Nq, int64_t Nk, int64_t K,
                                          size_t* bytes);
int m2rnn_qk_norm_rope_bwd(int64_t B, int64_t T, int64_t Nq, int64_t Nk, int64_t K, int64_t R,
                           int interleaved, int dtype, const void* q, const void* k, const float* gamma_q,
                           const float* gamma_k, const int32_t* pos, const double* inv_freq, float eps,
                           const float* dq_out, const float* dk_out, float* dq, float* dk, float* dgamma_q,
                           float* dgamma_k, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Global gradient norm and clipping over many tensors (a training step clips at a norm of 1).
 *     norm = sqrt(sum over all elements of all tensors of g^2)
 *     g <- g max_norm / norm where norm > max_norm, else unchanged
 * The list is a host array, read during the call only (a captured graph keeps its own copy).  A tensor
 * has any number of elements (also none), contiguous, aligned to its element, in fp32 or bf16.
 * Squares are summed in fp64 in a fixed order.
 *   norm       device fp32 scalar: m2rnn_grad_norm writes it, m2rnn_grad_clip reads it (in between a
 *              caller may combine the norms of several ranks).  No tensors: 0.  Not within a tensor of the
 *              list (M2RNN_EINVAL).
 *   out        NULL: in place.  Otherwise a host array of `count` device pointers (NULL entries: in place)
 *              of the tensors' own types and sizes.  An output that overlaps another output, another
 *              tensor, the norm, or a part of its own tensor is rejected (M2RNN_EINVAL).
 *   max_norm   >= 0 (negative or NaN: M2RNN_EINVAL).
 * A norm that is not finite leaves the gradients unchanged (out of place: copied): the caller finds it
 * in `norm` and skips the step.
 */
typedef struct m2rnn_tensor {
  void* data;    /* device pointer */
  int64_t numel; /* elements */
  int64_t dtype; /* M2RNN_DTYPE_F32 or M2RNN_DTYPE_BF16 */
} m2rnn_tensor;
int m2rnn_grad_norm_workspace_size(const m2rnn_tensor* grads, int64_t count, size_t* bytes);
int m2rnn_grad_norm(const m2rnn_tensor* grads, int64_t count, float* norm, void* workspace,
                    size_t workspace_bytes, void* stream);
int m2rnn_grad_clip(const m2rnn_tensor* grads, int64_t count, void* const* out, const float* norm,
                    float max_norm, void* stream);

/*
 * The entry of a layer (the pre-norm and the residual around a block): the residual stream takes a branch's
 * output and the sum is normalised for the next branch,
 *     h = res + x (rounded to the stream's type),   out = gamma (.) h / sqrt(mean_j h_j^2 + eps)
 * over the D features of each of `rows` rows.  The norm is of h as it is kept.
 *   x          [rows, D] in x_dtype; res [rows, D] in res_dtype (fp32 or bf16 each), or NULL: h = x, and h must
 *              be NULL (res_dtype is then not used, but must be one of the two).
 *   h          [rows, D] in res_dtype, or NULL to skip it.  May be res, or x of the same type (in place).
 *   out        [rows, D] in out_dtype: fp32, bf16 or E4M3.
 *   group      E4M3: the features that share a scale, 0 or D (one scale a row) or 128 (D a multiple of 128);
 *              0 for the other types.
 *   scale      E4M3: [rows, D / group] fp32, s = max(amax |.| / 448, 2^-126) over the group; out holds the
 *              norm's values over s, rounded to nearest even, so values are out times scale.
 *   D a multiple of 4 up to 16384; rows at most 2^31 - 1; eps >= 0.  Squares are summed in fp32 and must stay
 *   within it (|h| below 1e18, and above 1e-18 where eps is so small that they count).  A row with a value that is not finite is not finite: NaN where the value, or
 *   its group's scale, is.  Pointers 16-byte aligned (scale 4).  No output may overlap another array except as said.
 * The backward takes h as kept (x without a residual), dout (fp32) and dh, the gradient that reaches h down the
 * stream (fp32, or NULL: zeros), and gives dx [rows, D] fp32, which is the gradient of x and of res alike, and
 * dgamma [D], summed over the rows in a fixed order.  dx may be dout or dh.
 */
int m2rnn_add_norm_fwd(int64_t rows, int64_t D, int x_dtype, const void* x, int res_dtype, const void* res,
                       const float* gamma, float eps, void* h, int out_dtype, int64_t group, void* out, float* scale,
                       void* stream);
int m2rnn_add_norm_bwd_workspace_size(int64_t rows, int64_t D, size_t* bytes);
int m2rnn_add_norm_bwd(int64_t rows, int64_t D, int h_dtype, const void* h, const float* gamma, float eps,
                       const float* dout, const float* dh, float* dx, float* dgamma, void* workspace,
                       size_t workspace_bytes, void* stream);

/*
 * Gated linear recurrence of channels: the blend and the gate of the M²RNN recurrence on a vector state, without
 * the tanh, for the linear layers of a hybrid stack.  Per (b, d), from h_0 (zeros, or a given state),
 *     f_t = exp(-alpha softplus(a_t + beta)),   h_t = f_t h_{t-1} + (1 - f_t) v_t,   y_t = h_t
 *   v, a       [B,T,D] in `dtype` (fp32 or bf16); alpha, beta [D] fp32 (alpha >= 0 keeps f in [0, 1]; not checked,
 *              computed as given); h0, h_T [B,D] fp32 (NULL: zeros; not written); y [B,T,D] fp32.
 *   lens       [B] int32 device array or NULL, as in m2rnn_ssm_fwd: steps at or past a sequence's end change
 *              nothing, their y and gradients are zeros, whatever v and a hold there.  h_T is the state after the
 *              last step within (that step's y, bit for bit).  T = 0: h_T = h0.
 *   D a multiple of 4 up to 2^24, T at most 2^30, B D at most 2^35, and ceil(B D / 256) ceil(T / 32) below 2^23.
 *   Pointers 16-byte aligned (lens 4).
 * fp32 arithmetic; 1 - f is formed without cancellation (where alpha < 0: from the rounded f).  A step whose 1 - f is
 * zero (a = -infinity or the lowest number: masked through its gate; alpha = 0) holds the state, whatever v is.  Any
 * other value that is not finite reaches its own channel of its own sequence from its step on (an infinity may become
 * NaN), and nothing else.  Two calls on the same inputs give the same bits.  Where there are several chunks a workgroup
 * waits for those before its own, within the launch; a wait that is not served within seconds (a workspace that another
 * call writes at the same time) ends, and the outputs behind it are then NaN, with no other sign of it.
 *
 * m2rnn_gated_scan_bwd gives the gradients of L = sum <dy, y> + <dh_T, h_T> from the forward's inputs and its y:
 * dv, da [B,T,D], dalpha, dbeta [D] (summed over batch and time), dh0 [B,D] (NULL to skip), all fp32.  It expects
 * finite values within the sequences (masked steps apart: their a may be -infinity, their v anything).
 * m2rnn_gated_scan_step is one step for every sequence: v, a [B,D], the state h [B,D] (NULL: zeros) to
 * h_out [B,D] (which is the step's y too).  h_out may be h; any other overlap is rejected (M2RNN_EINVAL).
 */
int m2rnn_gated_scan_fwd_workspace_size(int64_t B, int64_t T, int64_t D, int dtype, size_t* bytes);
int m2rnn_gated_scan_fwd(int64_t B, int64_t T, int64_t D, int dtype, const void* v, const void* a, const float* alpha,
                         const float* beta, const int32_t* lens, const float* h0, float* y, float* h_T, void* workspace,
                         size_t workspace_bytes, void* stream);
int m2rnn_gated_scan_bwd_workspace_size(int64_t B, int64_t T, int64_t D, int dtype, size_t* bytes);
int m2rnn_gated_scan_bwd(int64_t B, int64_t T, int64_t D, int dtype, const void* v, const void* a, const float* alpha,
                         const float* beta, const int32_t* lens, const float* h0, const float* y, const float* dy,
                         const float* dh_T, float* dv, float* da, float* dalpha, float* dbeta, float* dh0,
                         void* workspace, size_t workspace_bytes, void* stream);
int m2rnn_gated_scan_step(int64_t B, int64_t D, int dtype, const void* v, const void* a, const float* alpha,
                          const float* beta, const float* h, float* h_out, void* stream);

/*
 * Orthogonalised update of matrices (W of all heads, projections), the step after the clipping for optimisers
 * that take a matrix's update at equal singular values.  For each m x n matrix of a batch,
 *     X = G / (||G||_F + eps),  then for each step, with A = X X^T over the shorter side (X transposed if m > n),
 *     X <- a X + (b A + c A A) X
 *   g, out     [batch, m, n] in `dtype` (fp32 or bf16); out may be g (any other overlap: M2RNN_EINVAL).
 *   coefs      host array of `steps` triples (a, b, c), read during the call only.  Singular values must stay below
 *              2 and |b s^2 + c s^4| below 24 for those that occur (products run on split fp16 values, which end
 *              there; the usual coefficients keep them below 1.21 and 2.9).  With a shorter side of 32 at most products
 *              are in fp32 and there is no such bound.  c = 0 (a cubic step) takes two products instead of three.
 *   steps      1 to 64; m, n up to 65536, batch up to 65535, and less than 2^36 elements in all, sides rounded up
 *              to 64.
 * The norm is summed in fp64, X is kept in fp32, and products are those of fp32 (with a shorter side above 32: fp16 values
 * in two parts, 22 bits, each row and column at a power of two of its own, three passes with fp32 accumulation): an
 * entry's error is relative to its row and its column, however much smaller than others these are.  A matrix of zeros
 * gives zeros (eps > 0); one with a value that is not finite is not finite; past the bound above a result is right or not
 * finite.  Two calls on the same inputs give the same bits.  Pointers 16-byte aligned.
 */
int m2rnn_orthogonalize_workspace_size(int64_t batch, int64_t m, int64_t n, int dtype, size_t* bytes);
int m2rnn_orthogonalize(int64_t batch, int64_t m, int64_t n, int dtype, const void* g, int64_t steps, const float* coefs,
                        float eps, void* out, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* M2RNN_H_ */
