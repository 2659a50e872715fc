// ssd_seq.h -- launch interface between the C ABI (ssd_seq_api.hip) and the
// kernels of the gated linear recurrence (ssd_glr.hip) and of the norm with
// rotation (ssd_normrot.hip).  Not installed; not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssd {

// The gated linear recurrence.  A workgroup of the forward takes kGlrChunk
// tokens, one of the backward kGlrSegment tokens (the spacing of the saved
// states), of 64 or 128 channels.
constexpr int kGlrChunk = 128;
constexpr int kGlrSegment = 64; // SSD_GLR_SEGMENT
struct GlrParams {
  const void *x, *r, *i, *dout;          // [b, L, D], last dim contiguous
  int dout_f32;                          // dout is fp32 whatever x is
  int64_t xb, rb_, ib_, db;              // batch strides, elements
  int xt, rt, it, dt;                    // token strides, elements
  const float *A, *rbias, *ibias;        // [D]; the biases may be null
  const uint8_t *reset;                  // [b, L] or null
  const int32_t *lengths;                // [b] or null
  const float *init;                     // [b, D] or null
  void *out;                             // [b, L, D] dense, or null (states only)
  float *fin;                            // [b, D] or null; may be init (inplace)
  float *states;                         // [b, ceil(L/kGlrSegment), D] or null
  const float *dfin;                     // [b, D] or null
  void *dx, *dr, *di;                    // [b, L, D] dense
  float *dinit;                          // [b, D] or null
  float *part;                           // [b, nchunk, 3, D], null: no parameter gradients
  uint64_t *words;                       // chain words [b, nchunk, wstride], null if nchunk == 1
  uint32_t *ticket;                      // behind the words
  int64_t wstride;
  int b, L, D, nchunk;
  int ntile; // set by the launch
  int inplace;
};
// Words of a chunk, bytes of the chain words and the ticket behind them.
inline int64_t glr_wstride(int64_t D) { return (D + 127) / 128 * 128; }
inline int64_t glr_chain_bytes(int64_t b, int64_t nchunk, int64_t D) { return b * nchunk * glr_wstride(D) * 8 + 16; }
// dtype 1 = bf16, 0 = fp32; vec: bf16 widths, strides and pointers allow 4-byte
// accesses (of an fp32 dout 8-byte ones).
hipError_t launch_glr(int dtype, bool vec, bool back, const GlrParams &p, hipStream_t stream);
// Sums n partial rows [3][D] into dA, d r_bias, d i_bias (each may be null).
hipError_t launch_glr_sum(const float *part, int n, int D, float *dA, float *drb, float *dib, hipStream_t stream);
struct GlrStepParams {
  const void *x, *r, *i;          // [b, D]
  int64_t xb, rb_, ib_;           // batch strides
  const float *A, *rbias, *ibias; // [D]
  const uint8_t *reset;           // [b] or null
  const float *state;             // [b, D]
  float *new_state;               // [b, D], may be state
  void *out;                      // [b, D]
  int b, D, nblk;                 // nblk is set by the launch
};
hipError_t launch_glr_step(int dtype, bool vec, const GlrStepParams &p, hipStream_t stream);

// Norm of queries and keys for each head with the position rotation.
constexpr int kNormRotGroups = 1024; // workgroups (and partial rows) of the backward
struct NormRotParams {
  const void *q, *k;                      // [b, L, Hq / Hk, N], last dim contiguous
  int64_t qb, qt, qh, kb, kt, kh;         // strides, elements
  const void *dyq, *dyk;                  // gradients at the outputs (backward)
  int64_t dqb, dqt, dqh, dkb, dkt, dkh;
  int dy_f32;                             // both are fp32 whatever q is
  const float *qw, *kw;                   // [N] or null
  const float *freqs;                     // [npair]
  const int32_t *pos32;                   // [b, L], or
  const int64_t *pos64;                   // [b, L], or both null: 0 .. L-1
  void *oq, *ok;                          // outputs or gradients, dense
  float *part;                            // [nwg, 2, N] (backward), null: no weight gradients
  float *dqw, *dkw;                       // [N] or null
  float eps;
  int L, Hq, Hk, N, npair, interleaved;
  int64_t ntok;
  // set by norm_rotate_plan
  int64_t nitem;
  int hg_log, per, split, nwg;
};
// N a multiple of 8 up to 256, npair a multiple of 4 up to N/2.
void norm_rotate_plan(NormRotParams *p);
// dtype 1 = bf16, 0 = fp32; vec: strides and pointers allow 4-element accesses.
hipError_t launch_norm_rotate(int dtype, bool vec, bool back, const NormRotParams &p, hipStream_t stream);
} // namespace ssd
