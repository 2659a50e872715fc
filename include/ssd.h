/*
 * ssd.h -- C ABI of libssd, the Mamba-2 SSD selective scan for AMD MI355X
 * (gfx950).
 *
 * The operation ("Mamba-3 deep dive ch. 2, SSM foundations", 171host.com,
 * section 2.1.2, the discrete recurrence with forget gate alpha and input
 * gate gamma, and section 2.1.1 for the skip term D):
 *
 *     Delta_t = softplus(dt_t + dt_bias_h)
 *     h_t     = exp(Delta_t * A_h) * h_{t-1} + Delta_t * x_t B_t^T   (P x N)
 *     y_t     = h_t C_t + D_h * x_t                                    (P)
 *
 * for every batch row and head h independently; head h reads the B/C group
 * g = floor(h * G / H).  Section 2.2.1 of the same page shows the equal
 * matrix form Y = (L o C B^T) X; the library evaluates it chunk by chunk
 * ("Transformers are SSMs" summary, gongshangzheng.github.io, section 1.2:
 * the quadratic path inside short blocks, the recurrent path across them).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Tensors are described by ssd_tensor.  Every tensor must be dense and
 * row-major (strides, in elements, equal to the contiguous strides of its
 * shape) with a 16-byte aligned data pointer.  All data pointers must be
 * memory the current HIP device can address: its own device memory,
 * managed memory, or pinned host memory (read over the bus, slowly).
 * Pageable host memory and another device's memory are refused with
 * SSD_ERR_LAYOUT (checked with hipPointerGetAttributes after every other
 * argument check, before any launch).
 *
 * Ownership: the caller allocates every tensor and keeps it alive until the
 * work queued on `stream` has finished.  The library keeps no pointer to
 * caller memory after a call returns.
 *
 * Scratch: an algorithm that needs scratch space uses a device buffer the
 * library keeps, one per (device, stream) handle, reused by every call on
 * that stream in stream order and grown stream-ordered on `stream` when a
 * call needs more (an event recorded after each call orders the next use if
 * a handle is reused for another stream).  A request above 4 GiB is
 * allocated and freed stream-ordered on `stream` for that call alone.  At
 * most 16 buffers of at most 8 GiB in total are kept: a call that needs a
 * new buffer first frees the least recently used ones (after waiting for
 * their last use) until both limits hold.  Kept buffers live until
 * ssd_release_scratch(), eviction, or the end of the process.  Allocating
 * scratch per call would make the host wait for the stream's earlier work;
 * keeping it lets back-to-back calls queue ahead of the GPU.  Calls that take
 * scratch are serialised on the host while they queue their launches.
 *
 * Errors: every argument is validated on the host before any work is
 * queued; a failed validation returns a nonzero status and queues nothing.  A failed
 * kernel launch or allocation returns SSD_ERR_HIP / SSD_ERR_NOMEM.  Faults
 * inside kernels surface at the caller's next synchronisation.  The text of
 * the most recent error on the calling thread is returned by
 * ssd_last_error().  Calls are asynchronous with respect to the host and
 * ordered on `stream` (a hipStream_t; NULL is the default stream).  No call
 * prints or throws.
 */
#ifndef SSD_H
#define SSD_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SSD_VERSION 100 /* 1.0.0 */

/* Element types.  The integer types are taken by reset, lengths, positions,
 * page_table, start and tokens only. */
enum { SSD_F32 = 0, SSD_BF16 = 1, SSD_U8 = 2, SSD_I32 = 3, SSD_I64 = 4 };

/* Status codes. */
enum {
  SSD_OK = 0,
  SSD_ERR_NULL = 1,        /* a required tensor or data pointer is NULL      */
  SSD_ERR_SHAPE = 2,       /* shapes disagree, H % G != 0, b or L is zero    */
  SSD_ERR_DTYPE = 3,       /* unsupported or mismatched element type         */
  SSD_ERR_LAYOUT = 4,      /* not dense row-major, not 16B aligned, or not
                              memory the current device can address        */
  SSD_ERR_UNSUPPORTED = 5, /* P, N, chunk or size outside the supported set  */
  SSD_ERR_ALIAS = 6,       /* an output overlaps an input it may not alias   */
  SSD_ERR_NOMEM = 7,       /* scratch allocation failed                      */
  SSD_ERR_HIP = 8          /* a HIP runtime call or kernel launch failed     */
};

/* Algorithms for ssd_scan_fwd_algo (results agree to rounding). */
enum {
  SSD_ALGO_AUTO = 0,    /* choose by shape                                    */
  SSD_ALGO_FUSED = 1,   /* one kernel; each workgroup walks one (batch, head)
                           sequence in order with the state in registers      */
  SSD_ALGO_CHUNKED = 2, /* chunk-parallel: log-decay cumsum, chunk states,
                           inter-chunk state passing, fused intra+output      */
  SSD_ALGO_ROWS = 3,    /* bf16, N in {32, 64, 128}: C, B and the causal
                           C B^T scores of each (batch, group, 64-token
                           block) laid out once in matrix-core fragment
                           order and shared by the heads of the group; each
                           wave walks 16 state rows of one head            */
  SSD_ALGO_QUAD = 4     /* L <= 256: the whole-sequence quadratic form
                           Y = (L o C B^T) X (+ D x, + the decayed initial
                           state) with no state carried between blocks: one
                           workgroup per (batch, head, 64-token query
                           block), its key blocks spread over its waves;
                           P in {16,32,64} (128 for bf16)                   */
};

/* Dense tensor descriptor.  shape/strides beyond ndim are ignored; strides
 * are in elements. */
typedef struct ssd_tensor {
  void *data;
  int32_t dtype; /* SSD_F32 or SSD_BF16 */
  int32_t ndim;
  int64_t shape[4];
  int64_t strides[4];
} ssd_tensor;

/*
 * ssd_scan_fwd -- forward scan over whole sequences.
 *
 *   x          [b, L, H, P]  f32 or bf16                         required
 *   dt         [b, L, H]     f32, raw (before softplus)           required
 *   dt_bias    [H]           f32, added to dt before softplus     NULL => 0
 *   A          [H]           f32, the decay rate A_h (normally < 0) required
 *   B, C       [b, L, G, N]  dtype of x                           required
 *   D          [H]           f32, skip weight                     NULL => 0
 *   init_state [b, H, P, N]  f32, state before token 0            NULL => 0
 *   out        [b, L, H, P]  dtype of x, written                  required
 *   final_state[b, H, P, N]  f32, state after token L-1           NULL => skip
 *   chunk      a power of two in [64, 65536]: the segment length of the
 *              chunked algorithm, i.e. the granularity at which states are
 *              passed between segments.  A performance knob only: with
 *              SSD_ALGO_AUTO the library chooses the algorithm and segment
 *              length itself (see ssd_scan_plan) and chunk is not used.
 *   stream     hipStream_t
 *
 * The state is stored with N fastest: state[b][h][p][n] is the n-th state
 * entry of channel p (the transpose of the N x P product B x^T).
 * Supported sizes: P in {16, 32, 64, 128} (bf16) or {16, 32, 64} (fp32),
 * N in {16, 32, 64, 128}, H % G == 0, b >= 1, 1 <= L <= 2^24 (any L in
 * that range; the last chunk may be partial), H*P and G*N at most 2^22;
 * larger problems are refused with SSD_ERR_UNSUPPORTED.
 * Arithmetic: products on MFMA in the input dtype with fp32 accumulation,
 * the state and all decay factors in fp32.  final_state may be the same
 * tensor as init_state (updated in place); out may not overlap any input.
 */
int ssd_scan_fwd(const ssd_tensor *x, const ssd_tensor *dt,
                 const ssd_tensor *dt_bias, const ssd_tensor *A,
                 const ssd_tensor *B, const ssd_tensor *C, const ssd_tensor *D,
                 const ssd_tensor *init_state, ssd_tensor *out,
                 ssd_tensor *final_state, int chunk, void *stream);

/* ssd_scan_fwd with an explicit algorithm (SSD_ALGO_*). Same contract;
 * SSD_ALGO_CHUNKED uses `chunk` as its segment length; SSD_ALGO_ROWS
 * returns SSD_ERR_UNSUPPORTED for fp32 inputs or N outside {32, 64, 128}.
 * SSD_ALGO_ROWS and SSD_ALGO_CHUNKED use scratch (see Scratch above; ROWS:
 * b*G*ceil(L/64)*(N/4 + 6) KiB of operand records, 38 KiB per block at
 * N = 128, plus b*H*64*ceil(L/64)*4 bytes for a head-major copy of dt). */
int ssd_scan_fwd_algo(const ssd_tensor *x, const ssd_tensor *dt,
                      const ssd_tensor *dt_bias, const ssd_tensor *A,
                      const ssd_tensor *B, const ssd_tensor *C,
                      const ssd_tensor *D, const ssd_tensor *init_state,
                      ssd_tensor *out, ssd_tensor *final_state, int chunk,
                      int algo, void *stream);

/*
 * ssd_scan_fwd_noalloc -- ssd_scan_fwd for callers that cannot allocate
 * device memory: code under HIP graph capture, tight serving loops, and
 * harnesses that forbid allocation.  Same arguments, validation, plan
 * (SSD_ALGO_AUTO) and results as ssd_scan_fwd; the call makes no hipMalloc,
 * hipFree or other allocation.  Its scratch is a fixed array of
 * ssd_fixed_scratch_bytes() bytes (64 MiB) in the library's device memory,
 * one copy per device, held until the process ends; a call whose plan needs
 * more scratch than that returns SSD_ERR_NOMEM before queuing anything
 * (every scratch user writes its scratch before reading it, so nothing
 * needs clearing between calls).  Every ssd_scan_fwd_noalloc call on one
 * device shares that device's array: calls that overlap in time on one
 * device (on different streams, or from several host threads) race on it
 * and must be ordered by the caller.
 */
int ssd_scan_fwd_noalloc(const ssd_tensor *x, const ssd_tensor *dt,
                         const ssd_tensor *dt_bias, const ssd_tensor *A,
                         const ssd_tensor *B, const ssd_tensor *C,
                         const ssd_tensor *D, const ssd_tensor *init_state,
                         ssd_tensor *out, ssd_tensor *final_state, int chunk,
                         void *stream);

/* Size in bytes of the fixed scratch array of ssd_scan_fwd_noalloc. */
int64_t ssd_fixed_scratch_bytes(void);

/*
 * ssd_scan_fwd_gated -- the scan with the block's output gate fused into its
 * output step.  The Mamba block follows the selective SSM with a gate before
 * the output projection (Mamba paper-reading notes, sxlin0.github.io, the
 * section on the simplified block), and its main branch is a Linear+SiLU
 * ("Transformers are SSMs" summary, gongshangzheng.github.io, section 2.3,
 * the correspondence table); read as
 *
 *     out_t = y_t * silu(z_t),   silu(v) = v / (1 + e^{-v})
 *
 * elementwise, with y_t exactly as ssd_scan_fwd computes it (D term
 * included).  final_state is the same as ssd_scan_fwd's.
 *
 *   z   [b, L, H, P]  dtype of x, dense, 16-byte aligned     required
 *
 * Every other argument as ssd_scan_fwd_algo (any algorithm, any supported
 * size).  out and final_state may not overlap z.  Arithmetic: y is formed
 * as in ssd_scan_fwd and the gate in fp32; out is rounded once to the dtype
 * of x, except that SSD_ALGO_ROWS with more than four waves per workgroup
 * rounds y to bf16 before gating (a second rounding of the same size).
 */
int ssd_scan_fwd_gated(const ssd_tensor *x, const ssd_tensor *dt,
                       const ssd_tensor *dt_bias, const ssd_tensor *A,
                       const ssd_tensor *B, const ssd_tensor *C,
                       const ssd_tensor *D, const ssd_tensor *z,
                       const ssd_tensor *init_state, ssd_tensor *out,
                       ssd_tensor *final_state, int chunk, int algo,
                       void *stream);

/*
 * ssd_scan_fwd_rows -- ssd_scan_fwd with SSD_ALGO_ROWS and an explicit
 * workgroup size: `waves` in 1..8 waves per workgroup (16 state rows each),
 * 0 = the size SSD_ALGO_AUTO would take.  For tuning and tests; the result
 * does not depend on `waves` beyond rounding order (it does not at all:
 * every state row is computed by the same instruction sequence).  bf16
 * inputs and N in {32, 64, 128} only (else SSD_ERR_UNSUPPORTED).
 */
int ssd_scan_fwd_rows(const ssd_tensor *x, const ssd_tensor *dt,
                      const ssd_tensor *dt_bias, const ssd_tensor *A,
                      const ssd_tensor *B, const ssd_tensor *C,
                      const ssd_tensor *D, const ssd_tensor *init_state,
                      ssd_tensor *out, ssd_tensor *final_state, int waves,
                      void *stream);

/*
 * ssd_step -- one recurrent step for every (batch, head), state in place
 * ("From Transformer to Mamba", jsqmd.com, section 2.1: the single-step
 * update ssm_step(x_t, h_prev, A, B, C) -> (y_t, h_t); "Mamba-3 deep dive
 * ch. 2", section 2.2.2: recurrent mode with a constant-size cache).
 *
 *   state [b, H, P, N]  f32, read and overwritten with the new state
 *   x     [b, H, P]     f32 or bf16
 *   dt    [b, H]        f32, the step size Delta itself (already activated:
 *                       no bias and no softplus are applied here)
 *   A     [H]           f32                                     required
 *   B, C  [b, G, N]     dtype of x                              required
 *   D     [H]           f32                                     NULL => 0
 *   out   [b, H, P]     dtype of x, written
 *
 * Supported sizes: N in {16, 32, 64, 128, 256}, any P >= 1, H % G == 0.
 * All arithmetic in fp32; out is rounded to its dtype once.  out may not
 * overlap any input or the state.
 */
int ssd_step(ssd_tensor *state, const ssd_tensor *x, const ssd_tensor *dt,
             const ssd_tensor *A, const ssd_tensor *B, const ssd_tensor *C,
             const ssd_tensor *D, ssd_tensor *out, void *stream);

/*
 * ssd_selective_scan_fwd -- the selective scan with a per-channel step size
 * and a diagonal A per (channel, state index), the Mamba-1 selective SSM
 * (Mamba paper-reading notes, sxlin0.github.io, the selective-mechanism
 * section: B, C and Delta depend on the input, Delta per channel; "Transformers
 * are SSMs" summary, gongshangzheng.github.io, section 1.3 table: a small
 * state, N = 16).  For every batch row and channel d:
 *
 *     Delta_t = softplus(dt[t][d] + dt_bias[d])
 *     h_t[n]  = exp(Delta_t * A[d][n]) * h_{t-1}[n] + Delta_t * B_t[n] * x_t[d]
 *     y_t[d]  = sum_n C_t[n] * h_t[n] + D[d] * x_t[d]
 *
 *   x           [b, L, D]     f32 or bf16                        required
 *   dt          [b, L, D]     f32, raw (before bias and softplus) required
 *   dt_bias     [D]           f32                                NULL => 0
 *   A           [D, N]        f32, the values A[d][n]            required
 *   B, C        [b, L, G, N]  dtype of x; channel d reads group
 *                             floor(d * G / D)                   required
 *   D           [D]           f32 (the skip term)                NULL => 0
 *   init_state  [b, D, N]     f32, the state before token 0      NULL => 0
 *   out         [b, L, D]     dtype of x, written
 *   final_state [b, D, N]     f32, written; may be init_state    NULL => skip
 *   segments    the sequence is cut into this many segments walked in
 *               parallel (their entering states folded from a first
 *               state-only pass); 0 chooses from the device size.  Raised
 *               if needed so that one segment's x, dt or out stays under
 *               2 GiB, capped at 1024 and at one segment per 8 tokens.  The
 *               result does not depend on it beyond rounding order.
 *
 * Supported sizes: N in {4, 8, 16}, D/G a multiple of 64 (64 channels of
 * one group per wave), 1 <= L <= 2^24.  The state and all arithmetic in
 * fp32; out is rounded to its dtype once.  Scratch (segment end states,
 * b * segments * D * (N + 1) floats, plus b * D * N staged initial state)
 * is used when segments > 1 (see Scratch above).  out may not overlap any input; final_state may not
 * overlap any input other than (exactly) init_state.
 */
int ssd_selective_scan_fwd(const ssd_tensor *x, const ssd_tensor *dt,
                           const ssd_tensor *dt_bias, const ssd_tensor *A,
                           const ssd_tensor *B, const ssd_tensor *C,
                           const ssd_tensor *D, const ssd_tensor *init_state,
                           ssd_tensor *out, ssd_tensor *final_state,
                           int segments, void *stream);

/*
 * ssd_scan_bwd -- gradients of ssd_scan_fwd with respect to all its inputs.
 *
 * Training needs them.  The Mamba paper-reading notes (sxlin0.github.io, the
 * section on the hardware-aware selective scan) describe the backward pass
 * as recomputing the states it needs instead of storing them.  This call
 * recomputes the states at 64-token chunk boundaries from the inputs and
 * rebuilds everything inside a chunk on chip.  No forward-pass residue is
 * needed.
 *
 * The gradients are those of the scalar sum <dout, y> + <dfinal_state, h_last>,
 * where y and h_last are what ssd_scan_fwd computes from the same inputs.
 * dout is the gradient arriving at the output and dfinal_state the one
 * arriving at the final state.
 *
 * Inputs: x, dt, dt_bias, A, B, C, D and init_state exactly as for
 * ssd_scan_fwd (dt_bias, D, init_state may be NULL: zero).  dout
 * [b,L,H,P] has the dtype of x.  dfinal_state [b,H,P,N] f32 may be NULL
 * (zero).
 *
 * Outputs, all f32, written in full (nothing is accumulated into them):
 *   dx [b,L,H,P]         ddt [b,L,H] (gradient at the raw dt, before
 *                         dt_bias and softplus)
 *   dA [H]               dB, dC [b,L,G,N] (summed over the heads of a group)
 *   ddt_bias [H], dD [H], dinit_state [b,H,P,N]: each may be NULL (not
 *                         computed).
 *
 * Supported: P in {16, 32, 64}, N in {16, 32, 64, 128}, either input dtype,
 * the size limits of ssd_scan_fwd.  No output may overlap an input or another
 * output (SSD_ERR_ALIAS).  Arithmetic: fp32 inputs use fp32 matrix-core
 * products throughout.  bf16 inputs use bf16 matrix-core products with fp32
 * accumulation; where a product pairs a bf16 input with an fp32 quantity
 * (decayed scores, states, adjoints, weighted x or dout), the fp32 operand is
 * carried as a bf16 high part plus a bf16 remainder, so each such product is
 * two bf16 MFMAs with a relative error near 2^-17.  The state walks keep
 * their states in fp32.  Sums over heads, chunks and batch run
 * in a fixed order, so the result does not vary from run to run.  Scratch:
 * b*H*ceil(L/64)*(2*P*N + 3) floats (the states entering each 64-token chunk,
 * the gradients at each chunk's end, per-chunk partial sums; see Scratch
 * above: 1.34 GB at b=4, L=4096, H=80, P=64, N=128, kept between calls
 * like any scratch up to 4 GiB).
 */
int ssd_scan_bwd(const ssd_tensor *x, const ssd_tensor *dt,
                 const ssd_tensor *dt_bias, const ssd_tensor *A,
                 const ssd_tensor *B, const ssd_tensor *C, const ssd_tensor *D,
                 const ssd_tensor *init_state, const ssd_tensor *dout,
                 const ssd_tensor *dfinal_state, ssd_tensor *dx,
                 ssd_tensor *ddt, ssd_tensor *ddt_bias, ssd_tensor *dA,
                 ssd_tensor *dB, ssd_tensor *dC, ssd_tensor *dD,
                 ssd_tensor *dinit_state, void *stream);

/*
 * ssd_scan_bwd_gated -- gradients of ssd_scan_fwd_gated (out = y * silu(z),
 * y the scan output including the D term) for the objective
 * <dout, out> + <dfinal_state, h_last>.
 *
 * The gated output is the Mamba block's gate before its output projection
 * (Mamba paper-reading notes, sxlin0.github.io, the simplified-block section).
 * Arguments are as for ssd_scan_bwd, plus z [b,L,H,P] (dtype of x, an input)
 * and dz [b,L,H,P] f32 (an output, required).  The call recomputes y with the
 * forward scan, forms dy = dout * silu(z) (rounded to x's dtype) and
 * dz = dout * y * silu'(z), then runs ssd_scan_bwd on dy.  Scratch: two
 * tensors the size of x, plus what the forward scan and ssd_scan_bwd use.
 */
int ssd_scan_bwd_gated(const ssd_tensor *x, const ssd_tensor *dt,
                       const ssd_tensor *dt_bias, const ssd_tensor *A,
                       const ssd_tensor *B, const ssd_tensor *C,
                       const ssd_tensor *D, const ssd_tensor *z,
                       const ssd_tensor *init_state, const ssd_tensor *dout,
                       const ssd_tensor *dfinal_state, ssd_tensor *dx,
                       ssd_tensor *ddt, ssd_tensor *ddt_bias, ssd_tensor *dA,
                       ssd_tensor *dB, ssd_tensor *dC, ssd_tensor *dD,
                       ssd_tensor *dz, ssd_tensor *dinit_state, void *stream);

/*
 * Gated linear recurrence: ssd_glr_fwd, ssd_glr_bwd, ssd_glr_step
 * ----------------------------------------------------------------
 * One scalar state per channel, both gates computed from the input.  It is
 * the forget-gate / input-gate recurrence of "Mamba-3 deep dive ch. 2"
 * (171host.com, section 2.1.2) with a diagonal state and gates of its own:
 *
 *     s_t = sigmoid(r_t + r_bias)              recurrence gate
 *     a_t = exp(A * s_t)                       decay, A normally < 0
 *     h_t = a_t * h_{t-1} + sqrt(1 - a_t^2) * sigmoid(i_t + i_bias) * x_t
 *
 * for every batch row and channel; out_t = h_t.  The factor sqrt(1 - a^2)
 * keeps the variance of h at that of its input.  A is meant to be finite and at
 * most 0: where a > 1 the factor is taken as 0, and the decays of 128
 * successive tokens multiplied must stay within fp32's range.  An r of -infinity,
 * or of its type's lowest finite value, shuts its gate (a_t = 1, the factor 0)
 * whatever r_bias is.
 *
 * Packed and padded batches.  reset [b, L] marks (nonzero) the first token of
 * each document: it starts from a zero state (a_t = 0, so the factor is 1).
 * lengths [b] says how many tokens of each row exist (values outside [0, L]
 * count as the nearer end): the tokens behind are not read, their outputs are
 * left as they were, and the final state is the one after the last token that
 * exists (the initial state if there is none).  What the state held before a
 * reset, NaN and infinities among it, does not reach what follows.
 *
 * Layout: x, r, i and dout may be strided views (slices of a fused
 * projection, broadcast batches): the last dimension contiguous, other
 * strides >= 0, the token stride at most 2^22 elements.  All other tensors are
 * dense row-major.  Pointers need the alignment of their element; bf16
 * rows of odd width, stride or alignment are moved two bytes at a time.
 *
 * Workspace: these calls take no scratch of the library's.  The caller passes
 * `workspace`, 16-byte aligned device memory of at least
 * ssd_glr_workspace(...) bytes (NULL if that is 0), which the call may write
 * until its work on `stream` has finished; its contents need not be set and
 * are of no further use.  Calls that may run at the same time, and graphs that
 * may be replayed at the same time, need a workspace each.  The calls allocate
 * nothing and record no event, so they may be captured into a HIP graph.
 *
 * Arithmetic: everything in fp32; out and the gradients of x, r and i are
 * rounded once to the dtype of x.  Values below 2^-126 count as 0 (a gate
 * that nearly shut leaves a_t = 1 and the factor 0).  Results do not vary from
 * run to run.
 * Supported: any D in [1, 2^20], 1 <= L <= 2^24, up to 2^22 tiles of 64
 * channels by 128 tokens (64 for the gradients) over the batch.
 */

/* Tokens between the saved states of ssd_glr_fwd. */
#define SSD_GLR_SEGMENT 64

/* Workspace bytes of ssd_glr_fwd (backward = 0) or ssd_glr_bwd (1); -1 for a
 * shape those calls refuse.  Host only. */
int64_t ssd_glr_workspace(int64_t b, int64_t L, int64_t D, int backward);

/*
 * ssd_glr_fwd -- whole sequences.
 *
 *   x, r, i     [b, L, D]  f32 or bf16, one dtype; r and i before bias and
 *                          sigmoid                             required
 *   A           [D]        f32                                 required
 *   r_bias, i_bias [D]     f32                                 NULL => 0
 *   reset       [b, L]     u8                                  NULL => none
 *   lengths     [b]        i32                                 NULL => L
 *   init_state  [b, D]     f32                                 NULL => 0
 *   out         [b, L, D]  dtype of x, written                 required
 *   final_state [b, D]     f32, written; may be init_state     NULL => skip
 *   states      [b, ceil(L / SSD_GLR_SEGMENT), D]  f32, written: the state
 *                          entering every segment that holds a token (and
 *                          the first), for ssd_glr_bwd         NULL => skip
 * Other overlaps of an output with any argument are refused.
 */
int ssd_glr_fwd(const ssd_tensor *x, const ssd_tensor *r, const ssd_tensor *i,
                const ssd_tensor *A, const ssd_tensor *r_bias,
                const ssd_tensor *i_bias, const ssd_tensor *reset,
                const ssd_tensor *lengths, const ssd_tensor *init_state,
                ssd_tensor *out, ssd_tensor *final_state, ssd_tensor *states,
                void *workspace, int64_t workspace_bytes, void *stream);

/*
 * ssd_glr_bwd -- gradients of ssd_glr_fwd for <dout, out> +
 * <dfinal_state, final state>.  Inputs as for ssd_glr_fwd;
 * states is what ssd_glr_fwd wrote for the same inputs, or NULL: then they
 * are formed again from the inputs (one more pass over x, r and i).
 * dout [b, L, D] has the dtype of x or is f32 (as ssd_scan_bwd writes its
 * gradients); dfinal_state [b, D] f32 may be NULL.
 * Written in full: dx, dr, di [b, L, D] in the dtype of x (zero behind a
 * row's length); dA, dr_bias, di_bias [D] and dinit_state [b, D] f32, each of
 * these four may be NULL.  Where sqrt(1 - a^2) is 0 the gradient through it
 * is taken as 0.  No output may overlap any other argument.
 */
int ssd_glr_bwd(const ssd_tensor *x, const ssd_tensor *r, const ssd_tensor *i,
                const ssd_tensor *A, const ssd_tensor *r_bias,
                const ssd_tensor *i_bias, const ssd_tensor *reset,
                const ssd_tensor *lengths, const ssd_tensor *init_state,
                const ssd_tensor *states, const ssd_tensor *dout,
                const ssd_tensor *dfinal_state, ssd_tensor *dx, ssd_tensor *dr,
                ssd_tensor *di, ssd_tensor *dA, ssd_tensor *dr_bias,
                ssd_tensor *di_bias, ssd_tensor *dinit_state, void *workspace,
                int64_t workspace_bytes, void *stream);

/*
 * ssd_glr_step -- one token for every row (serving).  state [b, D] f32;
 * x, r, i [b, D]; reset [b] u8 or NULL (nonzero: the slot starts anew);
 * new_state [b, D] f32, written, may be `state`; out [b, D] dtype of x,
 * written.  b * ceil(D / 256) at most 2^22.
 */
int ssd_glr_step(const ssd_tensor *state, const ssd_tensor *x,
                 const ssd_tensor *r, const ssd_tensor *i, const ssd_tensor *A,
                 const ssd_tensor *r_bias, const ssd_tensor *i_bias,
                 const ssd_tensor *reset, ssd_tensor *new_state,
                 ssd_tensor *out, void *stream);

/*
 * Norm and rotation of queries and keys
 * -------------------------------------
 * In the dual (attention) form of the scan, C holds the queries and B the keys
 * ("Mamba-3 deep dive ch. 2", 171host.com, section 2.2.2, the linear-attention
 * view).  Turning both by an angle that grows with the position gives the
 * scalar decay of a head an imaginary part per pair of state indices; normed
 * queries and keys bound the scores.  For every token and head vector x of
 * q [b, L, Hq, N] or k [b, L, Hk, N]:
 *
 *     n = x / sqrt(mean(x^2) + eps),    y = R(position) (weight * n)
 *
 * R turns pair j by position * freqs[j] (radians): the pair (j, j + npair), or
 * with interleaved = 1 (2j, 2j + 1), of the first 2 * npair elements;
 * npair = the length of freqs (NULL: no rotation).  Hq and Hk are free of each
 * other (shared keys: Hk < Hq).
 *
 *   q, k         f32 or bf16, one dtype; views allowed: the last dimension
 *                contiguous, other strides >= 0                required
 *   q_weight, k_weight [N]  f32                               NULL => 1
 *   freqs        [npair]    f32                               NULL => none
 *   positions    [b, L]     i32 or i64, up to 2^53 either way NULL => 0..L-1
 *   q_out, k_out dtype and shape of q and k, dense, written
 *
 * Supported: N a multiple of 8 up to 256, npair a multiple of 4 up to N / 2,
 * L at most 2^24, b * L at most 2^25, Hq and Hk at most 2^16.
 * Arithmetic: fp32; angles are reduced to a turn in more than 64 bits, to fp32
 * accuracy at every such position; results are rounded once.  Elements up to
 * 2^59; values below 2^-126 count as 0, but not the squares of larger ones.  The
 * gradients' products (w dy x summed over a head) have to stay in fp32's range.
 * Results do not vary from run to run.  No output may overlap any other
 * argument.  Nothing is allocated; the calls may be captured into a HIP graph.
 */
int ssd_norm_rotate_fwd(const ssd_tensor *q, const ssd_tensor *k,
                        const ssd_tensor *q_weight, const ssd_tensor *k_weight,
                        const ssd_tensor *freqs, const ssd_tensor *positions,
                        ssd_tensor *q_out, ssd_tensor *k_out, float eps,
                        int interleaved, void *stream);

/* Workspace bytes of ssd_norm_rotate_bwd (see Workspace above); -1 for an N it
 * refuses.  Host only. */
int64_t ssd_norm_rotate_workspace(int64_t N);

/*
 * ssd_norm_rotate_bwd -- gradients for <dq_out, q_out> + <dk_out, k_out>.
 * dq_out, dk_out: shape of q and k, dtype of q or both f32 (as ssd_scan_bwd writes
 * its gradients), views allowed.  Written in full:
 * dq, dk (dtype of q, dense) and dq_weight, dk_weight [N] f32, each of these
 * two may be NULL (both: no workspace is needed).  Nothing of the forward is
 * needed but its inputs.
 */
int ssd_norm_rotate_bwd(const ssd_tensor *q, const ssd_tensor *k,
                        const ssd_tensor *q_weight, const ssd_tensor *k_weight,
                        const ssd_tensor *freqs, const ssd_tensor *positions,
                        const ssd_tensor *dq_out, const ssd_tensor *dk_out,
                        ssd_tensor *dq, ssd_tensor *dk, ssd_tensor *dq_weight,
                        ssd_tensor *dk_weight, float eps, int interleaved,
                        void *workspace, int64_t workspace_bytes, void *stream);

/*
 * Paged key-value cache and attention over it
 * -------------------------------------------
 * Models that mix states by scans and recurrences hold attention layers among
 * them.  Their cache lies in pages: k_cache and v_cache [pages, page_size, Hk, N]
 * hold the keys and values of all rows, page_table [b, width] i32 says which page
 * holds which part of a row: the key at position j of row i is
 * cache[page_table[i][j / page_size]][j mod page_size].  Any page_size >= 1;
 * multiples of 16 are faster.
 *
 *   start  [b]  i32: the position of the row's first new token, which is the number of
 *               tokens its cache held before                   required
 *   tokens [b]  i32: how many of the L tokens of the row there are (values
 *               outside [0, L] count as the nearer end); those behind are
 *               not read, their outputs are left as they were  NULL => L
 *
 * New token t of row i stands at position p = start[i] + t.  A call of the
 * append followed by one of the attention with the same start and tokens is a
 * layer's step; start then grows by tokens.
 *
 * What only the device holds is not checked by the host, and bounded there: an
 * entry of page_table outside [0, pages) (a page not dealt out, or taken back)
 * holds no keys, and nothing is stored to it; positions below 0 or from
 * width * page_size on have no place.  Such entries are otherwise allowed.  Rows
 * may share pages (a common prefix), but tokens that one call stores to the
 * same place leave any one of them, or a mixture, there.
 *
 * Caches may be views: the last dimension contiguous, data and the other strides
 * (>= 0, that of a page's tokens at most 2^24, of pages below 2^32) multiples of 16 bytes; for the append
 * no element may be two (strides that overlap), and k_cache and v_cache may lie
 * in each other's gaps, such as halves of one tensor [pages, 2, page_size, Hk, N].  page_table
 * may have a batch stride.  Offsets are 64 bits wide.
 * Supported: f32 or bf16, N a multiple of 8 up to 256, b, Hq and Hk at most 2^16, L at most
 * 2^24, b * L at most 2^25, width * page_size at most 2^30 and b times that at most
 * 2^36.  The calls allocate nothing and may be captured into a HIP graph.
 */

/*
 * ssd_kv_append -- keys and values of new tokens into the cache, keys and
 * queries turned by their positions on the way.
 *
 *   q         [b, L, Hq, N]  f32 or bf16                       NULL => keys only
 *   k, v      [b, L, Hk, N]  dtype of the caches               required
 *   freqs     [npair]        f32                               NULL => not turned
 *   q_out     [b, L, Hq, N]  dense, written                    with q
 *   k_cache, v_cache         written at the new tokens' places
 *
 *     k_cache[p] = R(p) k,   v_cache[p] = v,   q_out = R(p) q
 *
 * R, freqs, npair and interleaved as for ssd_norm_rotate_fwd, whose angles it
 * has (fp32, one rounding); values are moved as they are, and what is not
 * turned as well.  q, k and v may be views (the last dimension contiguous, other
 * strides >= 0).  q_out is written for tokens without a place in the cache too.
 * No output may overlap any other argument.
 */
int ssd_kv_append(const ssd_tensor *q, const ssd_tensor *k, const ssd_tensor *v,
                  const ssd_tensor *freqs, const ssd_tensor *page_table,
                  const ssd_tensor *start, const ssd_tensor *tokens,
                  ssd_tensor *q_out, ssd_tensor *k_cache, ssd_tensor *v_cache,
                  int interleaved, void *stream);

/* Workspace bytes of ssd_attn_fwd (and, with L = 1, of ssd_attn_step), see
 * Workspace above; 0 where none is needed, -1 for sizes they refuse.  Host only.
 * It does not depend on the cache or on the rows' lengths, and suffices for either
 * dtype.  At most about 220 MB. */
int64_t ssd_attn_workspace(int64_t b, int64_t L, int64_t Hq, int64_t Hk,
                           int64_t N);

/*
 * ssd_attn_fwd -- attention of new tokens over the cache, which holds them
 * already.  Head h reads the key head floor(h * Hk / Hq); Hq is a multiple of Hk.
 * The query at position p sees the keys at 0 .. p, with window > 0 the last
 * `window` of them (its own included):
 *
 *     s_j = scale * q . k_j,   lse = log sum_j e^{s_j},   out = sum_j e^{s_j - lse} v_j
 *
 *   q    [b, L, Hq, N]  f32 or bf16; views allowed as for ssd_kv_append
 *   out  [b, L, Hq, N]  dtype of q, dense, 16-byte aligned, written
 *   lse  [b, L, Hq]     f32, written                           NULL => skip
 *   scale               2^-126 to 1e30 in size (1 / sqrt(N) is usual); may be negative
 *   window              0 => all keys
 *
 * A query that sees no key, or only scores of -infinity, has out 0 and lse
 * -infinity.  Keys that a query does not see do not reach it, whatever they hold
 * (NaN and infinities among it).  One or several new tokens a row, prompts and pieces
 * of prompts: any L.  Rows of any lengths share the device evenly (below half a million
 * workgroups b * Hk * ceil(L * Hq / Hk / 16); above, a row is not spread over several).
 * Arithmetic: scores, maxima, sums and outputs in fp32; with bf16 inputs
 * the weights e^{s - m} are held to 1.25 2^-15 of each for the product with the values, and
 * to 2^-8 (one bf16) where a row has more than 16 query vectors L Hq / Hk of a key head; out
 * is rounded once.  The sums of weighted values, weights up to 4, have to
 * stay in fp32's range.  Results do not vary from run to run; a row's do depend, to
 * rounding, on the other rows' lengths, the table's width and the window (which say
 * where it is cut).  out and lse may not overlap any other argument.
 * b * Hk * ceil(L * Hq / Hk / 16) at most 2^23.
 */
int ssd_attn_fwd(const ssd_tensor *q, const ssd_tensor *k_cache,
                 const ssd_tensor *v_cache, const ssd_tensor *page_table,
                 const ssd_tensor *start, const ssd_tensor *tokens,
                 ssd_tensor *out, ssd_tensor *lse, float scale, int64_t window,
                 void *workspace, int64_t workspace_bytes, void *stream);

/* ssd_attn_step -- one new token for every row (serving): q and out [b, Hq, N],
 * lse [b, Hq] or NULL, otherwise as ssd_attn_fwd with L = 1. */
int ssd_attn_step(const ssd_tensor *q, const ssd_tensor *k_cache,
                  const ssd_tensor *v_cache, const ssd_tensor *page_table,
                  const ssd_tensor *start, ssd_tensor *out, ssd_tensor *lse,
                  float scale, int64_t window, void *workspace,
                  int64_t workspace_bytes, void *stream);

/*
 * ssd_scan_plan -- the plan SSD_ALGO_AUTO uses for a shape on a device with
 * `cus` compute units for inputs of element type `dtype` (SSD_BF16 or
 * SSD_F32), host only, no HIP call: *algo is SSD_ALGO_FUSED,
 * SSD_ALGO_CHUNKED or SSD_ALGO_ROWS and *seg_len the segment length (L for
 * the single-pass walks).
 * The choice trades the spread of (batch, head, segment) walks over the
 * compute units against the extra state-only pass and state traffic of
 * shorter segments.
 */
int ssd_scan_plan(int64_t b, int64_t L, int64_t H, int64_t P, int64_t G,
                  int64_t N, int dtype, int cus, int *algo, int *seg_len);

/* Static text for a status code. */
const char *ssd_status_string(int status);

/* Text of the most recent failure on the calling thread ("" if none). */
const char *ssd_last_error(void);

/* SSD_VERSION of the built library. */
int ssd_version(void);

/* Frees the scratch buffers the library keeps between calls (see Scratch
 * above), after waiting for the queued work that uses them; the next call
 * that needs scratch allocates it again.  Safe to call at any time from any
 * thread (calls that take scratch meanwhile wait for it); returns SSD_OK, or
 * SSD_ERR_HIP if a HIP call failed (the buffers are forgotten either way).
 * Makes no HIP call when no buffer is kept. */
int ssd_release_scratch(void);

/* Number of scratch buffers the library currently keeps and their total
 * bytes (see Scratch above).  Host only; returns SSD_ERR_NULL for a NULL
 * argument. */
int ssd_scratch_stats(int64_t *buffers, int64_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* SSD_H */
