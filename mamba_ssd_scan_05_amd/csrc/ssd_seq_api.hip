// ssd_seq_api.hip -- the C ABI of the gated linear recurrence and of the
// norm with rotation: argument validation, workspace layout and launches.  Declarations and the contract
// are in include/ssd.h.  As in ssd_api.hip every check runs on the host
// before the first launch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssd.h"
#include "ssd_check.h"
#include "ssd_seq.h"

using namespace ssd;

static_assert(kGlrSegment == SSD_GLR_SEGMENT, "the saved states' spacing");

namespace {

constexpr int64_t kMaxTokens = (int64_t)1 << 24;
constexpr int64_t kMaxWidth = (int64_t)1 << 20;  // channels of the recurrence
constexpr int64_t kMaxStride = (int64_t)1 << 22; // token stride of the recurrence: 128 fp32 rows within 2^31 bytes
constexpr int64_t kMaxOuter = (int64_t)1 << 36;  // other strides
constexpr int64_t kMaxHeads = (int64_t)1 << 16;
constexpr int64_t kMaxBatchTokens = (int64_t)1 << 25; // tokens of the norm: at most as many waves in one launch
constexpr int64_t kMaxTiles = (int64_t)1 << 22;  // workgroups of 512 threads in one launch

const char *dtype_name(int d) {
  switch (d) {
  case SSD_F32: return "f32";
  case SSD_BF16: return "bf16";
  case SSD_U8: return "u8";
  case SSD_I32: return "i32";
  case SSD_I64: return "i64";
  }
  return "unknown";
}

// Memory from the first element's first byte to the last one's last.
Range span_of(const ssd_tensor *t) {
  Range r;
  if (!t || !t->data) return r;
  int64_t last = 0;
  for (int i = 0; i < t->ndim; ++i) last += (t->shape[i] - 1) * t->strides[i];
  r.lo = (uintptr_t)t->data;
  r.hi = r.lo + (uintptr_t)((last + 1) * elem_size(t->dtype));
  return r;
}

// Presence, dtype, rank, shape, and the alignment of one element; dense
// row-major, or (view) a contiguous last dimension with other strides >= 0,
// those behind the batch at most max_stride.
int check_arg(const ssd_tensor *t, const char *name, int dtype, int ndim, const int64_t *shape, bool view = false,
              int64_t max_stride = kMaxOuter) {
  if (!t) return fail(SSD_ERR_NULL, "%s: descriptor is NULL", name);
  if (!t->data) return fail(SSD_ERR_NULL, "%s: data pointer is NULL", name);
  if (t->dtype != dtype)
    return fail(SSD_ERR_DTYPE, "%s: dtype %s, expected %s", name, dtype_name(t->dtype), dtype_name(dtype));
  if (t->ndim != ndim) return fail(SSD_ERR_SHAPE, "%s: rank %d, expected %d", name, t->ndim, ndim);
  for (int i = 0; i < ndim; ++i)
    if (t->shape[i] != shape[i])
      return fail(SSD_ERR_SHAPE, "%s: dim %d is %lld, expected %lld", name, i, (long long)t->shape[i],
                  (long long)shape[i]);
  int64_t dense = 1;
  for (int i = ndim - 1; i >= 0; --i) {
    const int64_t st = t->strides[i];
    if (t->shape[i] != 1) {
      if ((!view || i == ndim - 1) && st != dense)
        return fail(SSD_ERR_LAYOUT, "%s: stride of dim %d is %lld, expected %lld", name, i, (long long)st,
                    (long long)dense);
      if (view && (st < 0 || st > (i == 0 ? kMaxOuter : max_stride)))
        return fail(st < 0 ? SSD_ERR_LAYOUT : SSD_ERR_UNSUPPORTED, "%s: stride of dim %d is %lld", name, i,
                    (long long)st);
    }
    dense *= t->shape[i];
  }
  if ((uintptr_t)t->data % (uintptr_t)elem_size(dtype) != 0)
    return fail(SSD_ERR_LAYOUT, "%s: data pointer is not aligned to its element", name);
  return SSD_OK;
}

int act_dtype(const ssd_tensor *t, const char *name) {
  if (t->dtype != SSD_F32 && t->dtype != SSD_BF16)
    return fail(SSD_ERR_DTYPE, "%s: dtype %s, expected f32 or bf16", name, dtype_name(t->dtype));
  return SSD_OK;
}

// The type asked of an output's gradient: f32 or that of x.
int grad_dtype(const ssd_tensor *t, const ssd_tensor *x) { return t && t->dtype == SSD_F32 ? SSD_F32 : x->dtype; }

// A call's tensors, for the checks over all of them.
struct Args {
  static constexpr int kMax = 24;
  const ssd_tensor *t[kMax];
  const char *name[kMax];
  bool out[kMax];
  int n = 0;
  void add(const ssd_tensor *q, const char *nm, bool is_out) {
    if (!q) return;
    t[n] = q;
    name[n] = nm;
    out[n] = is_out;
    ++n;
  }
  // No output overlaps another argument; `same_out` may be exactly `same_in`.
  int overlaps(const ssd_tensor *same_out, const ssd_tensor *same_in) const {
    for (int i = 0; i < n; ++i) {
      if (!out[i]) continue;
      const Range ri = span_of(t[i]);
      for (int j = 0; j < n; ++j) {
        if (j == i || (out[j] && j < i)) continue;
        if (t[i] == same_out && t[j] == same_in && t[i]->data == t[j]->data) continue;
        if (overlap(ri, span_of(t[j]))) return fail(SSD_ERR_ALIAS, "%s overlaps %s", name[i], name[j]);
      }
    }
    return SSD_OK;
  }
  int workspace(const void *ws, int64_t have, int64_t need) const {
    if (need == 0) return SSD_OK;
    if (!ws) return fail(SSD_ERR_NULL, "workspace: NULL, %lld bytes needed", (long long)need);
    if (have < need)
      return fail(SSD_ERR_NOMEM, "workspace: %lld bytes, %lld needed", (long long)have, (long long)need);
    if ((uintptr_t)ws % 16 != 0) return fail(SSD_ERR_LAYOUT, "workspace: not 16-byte aligned");
    Range w;
    w.lo = (uintptr_t)ws;
    w.hi = w.lo + (uintptr_t)need;
    for (int i = 0; i < n; ++i)
      if (overlap(w, span_of(t[i]))) return fail(SSD_ERR_ALIAS, "workspace overlaps %s", name[i]);
    return SSD_OK;
  }
  int addressable(const void *ws) const {
    SSD_CHECK(check_addressable(t, name, n));
    if (!ws) return SSD_OK;
    ssd_tensor w{};
    w.data = const_cast<void *>(ws);
    const ssd_tensor *wt[1] = {&w};
    const char *wn[1] = {"workspace"};
    return check_addressable(wt, wn, 1);
  }
};

// ---------------------------------------------------------------------------
// the gated linear recurrence
// ---------------------------------------------------------------------------
int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

struct GlrPlan {
  int64_t ntile, nfwd, nseg;             // channel tiles, forward chunks, segments
  int64_t chain_f, chain_b, part, state; // bytes
};
bool glr_plan(int64_t b, int64_t L, int64_t D, bool back, GlrPlan *q) {
  if (b < 1 || L < 1 || D < 1 || L > kMaxTokens || D > kMaxWidth || b > kMaxTiles) return false;
  q->ntile = (D + 63) / 64; // of the narrower tiles
  q->nfwd = (L + kGlrChunk - 1) / kGlrChunk;
  q->nseg = (L + kGlrSegment - 1) / kGlrSegment;
  if (b * q->ntile > kMaxTiles || b * q->ntile * (back ? q->nseg : q->nfwd) > kMaxTiles) return false;
  q->chain_f = q->nfwd > 1 ? glr_chain_bytes(b, q->nfwd, D) : 0;
  q->chain_b = q->nseg > 1 ? glr_chain_bytes(b, q->nseg, D) : 0;
  q->part = b * q->nseg * 3 * D * 4;
  q->state = b * q->nseg * D * 4;
  return true;
}
// backward workspace: the chain (the larger one, the states' own pass uses it
// first), the partial sums, the states
int64_t glr_back_bytes(const GlrPlan &q) {
  return up256(q.chain_f > q.chain_b ? q.chain_f : q.chain_b) + up256(q.part) + up256(q.state);
}

int validate_glr(const ssd_tensor *x, const ssd_tensor *r, const ssd_tensor *i, const ssd_tensor *A,
                 const ssd_tensor *r_bias, const ssd_tensor *i_bias, const ssd_tensor *reset,
                 const ssd_tensor *lengths, const ssd_tensor *init_state, bool back, GlrPlan *plan, Args *args) {
  if (!x) return fail(SSD_ERR_NULL, "x: descriptor is NULL");
  if (x->ndim != 3) return fail(SSD_ERR_SHAPE, "x: rank %d, expected 3 [b,L,D]", x->ndim);
  const int64_t b = x->shape[0], L = x->shape[1], D = x->shape[2];
  if (b < 1 || L < 1 || D < 1)
    return fail(SSD_ERR_SHAPE, "empty problem: b=%lld L=%lld D=%lld", (long long)b, (long long)L, (long long)D);
  if (!glr_plan(b, L, D, back, plan))
    return fail(SSD_ERR_UNSUPPORTED, "problem too large: b=%lld L=%lld D=%lld", (long long)b, (long long)L,
                (long long)D);
  SSD_CHECK(act_dtype(x, "x"));
  const int64_t sx[3] = {b, L, D}, sd[1] = {D}, sr[2] = {b, L}, sl[1] = {b}, ss[2] = {b, D};
  SSD_CHECK(check_arg(x, "x", x->dtype, 3, sx, true, kMaxStride));
  SSD_CHECK(check_arg(r, "r", x->dtype, 3, sx, true, kMaxStride));
  SSD_CHECK(check_arg(i, "i", x->dtype, 3, sx, true, kMaxStride));
  SSD_CHECK(check_arg(A, "A", SSD_F32, 1, sd));
  if (r_bias) SSD_CHECK(check_arg(r_bias, "r_bias", SSD_F32, 1, sd));
  if (i_bias) SSD_CHECK(check_arg(i_bias, "i_bias", SSD_F32, 1, sd));
  if (reset) SSD_CHECK(check_arg(reset, "reset", SSD_U8, 2, sr));
  if (lengths) SSD_CHECK(check_arg(lengths, "lengths", SSD_I32, 1, sl));
  if (init_state) SSD_CHECK(check_arg(init_state, "init_state", SSD_F32, 2, ss));
  args->add(x, "x", false);
  args->add(r, "r", false);
  args->add(i, "i", false);
  args->add(A, "A", false);
  args->add(r_bias, "r_bias", false);
  args->add(i_bias, "i_bias", false);
  args->add(reset, "reset", false);
  args->add(lengths, "lengths", false);
  args->add(init_state, "init_state", false);
  return SSD_OK;
}

const float *fptr(const ssd_tensor *t) { return t ? (const float *)t->data : nullptr; }
float *fptr_out(ssd_tensor *t) { return t ? (float *)t->data : nullptr; }

GlrParams glr_params(const ssd_tensor *x, const ssd_tensor *r, const ssd_tensor *i, const ssd_tensor *A,
                     const ssd_tensor *r_bias, const ssd_tensor *i_bias, const ssd_tensor *reset,
                     const ssd_tensor *lengths, const ssd_tensor *init_state, const GlrPlan &plan) {
  GlrParams p{};
  p.x = x->data; p.r = r->data; p.i = i->data;
  p.xb = x->strides[0]; p.rb_ = r->strides[0]; p.ib_ = i->strides[0];
  // the stride of a dimension of one element means nothing
  const bool one = x->shape[1] == 1;
  p.xt = one ? 0 : (int)x->strides[1];
  p.rt = one ? 0 : (int)r->strides[1];
  p.it = one ? 0 : (int)i->strides[1];
  if (x->shape[0] == 1) p.xb = p.rb_ = p.ib_ = 0;
  p.A = fptr(A); p.rbias = fptr(r_bias); p.ibias = fptr(i_bias);
  p.reset = reset ? (const uint8_t *)reset->data : nullptr;
  p.lengths = lengths ? (const int32_t *)lengths->data : nullptr;
  p.init = fptr(init_state);
  p.b = (int)x->shape[0]; p.L = (int)x->shape[1]; p.D = (int)x->shape[2];
  p.wstride = glr_wstride(p.D);
  return p;
}

// Rows in pieces of `bytes`: the width, the strides that are used and the
// pointers are multiples of them.
bool rows_of(const ssd_tensor *t, int bytes) {
  const int V = bytes / elem_size(t->dtype), n = t->ndim;
  if ((uintptr_t)t->data % (uintptr_t)bytes != 0 || t->shape[n - 1] % V != 0) return false;
  for (int i = 0; i < n - 1; ++i)
    if (t->shape[i] != 1 && t->strides[i] % V != 0) return false;
  return true;
}
bool rows4b(const ssd_tensor *t) { return rows_of(t, 4); }
bool rows16(const ssd_tensor *t) { return rows_of(t, 16); }

void set_chain(GlrParams *p, int64_t nchunk, void *ws) {
  p->nchunk = (int)nchunk;
  p->words = nchunk > 1 ? (uint64_t *)ws : nullptr;
  p->ticket = nchunk > 1 ? (uint32_t *)((char *)ws + glr_chain_bytes(p->b, nchunk, p->D) - 16) : nullptr;
}

// ---------------------------------------------------------------------------
// norm and rotation of queries and keys
// ---------------------------------------------------------------------------
// Element groups of four at 8 (bf16) or 16 bytes (f32).
bool rows4(const ssd_tensor *t) {
  if (!t) return true;
  if ((uintptr_t)t->data % (uintptr_t)(4 * elem_size(t->dtype)) != 0) return false;
  for (int i = 0; i < t->ndim - 1; ++i)
    if (t->shape[i] != 1 && t->strides[i] % 4 != 0) return false;
  return true;
}

int64_t norm_rotate_bytes(int64_t N) { return (int64_t)kNormRotGroups * 2 * N * 4; }

int validate_norm_rotate(const ssd_tensor *q, const ssd_tensor *k, const ssd_tensor *q_weight,
                         const ssd_tensor *k_weight, const ssd_tensor *freqs, const ssd_tensor *positions, float eps,
                         int interleaved, NormRotParams *p, Args *args) {
  if (!q) return fail(SSD_ERR_NULL, "q: descriptor is NULL");
  if (!k) return fail(SSD_ERR_NULL, "k: descriptor is NULL");
  if (q->ndim != 4) return fail(SSD_ERR_SHAPE, "q: rank %d, expected 4 [b,L,Hq,N]", q->ndim);
  if (k->ndim != 4) return fail(SSD_ERR_SHAPE, "k: rank %d, expected 4 [b,L,Hk,N]", k->ndim);
  const int64_t b = q->shape[0], L = q->shape[1], Hq = q->shape[2], N = q->shape[3], Hk = k->shape[2];
  if (b < 1 || L < 1 || Hq < 1 || Hk < 1 || N < 1)
    return fail(SSD_ERR_SHAPE, "empty problem: b=%lld L=%lld Hq=%lld Hk=%lld N=%lld", (long long)b, (long long)L,
                (long long)Hq, (long long)Hk, (long long)N);
  if (N % 8 != 0 || N > 256)
    return fail(SSD_ERR_UNSUPPORTED, "N=%lld is not a multiple of 8 up to 256", (long long)N);
  if (L > kMaxTokens || b > kMaxTokens || b * L > kMaxBatchTokens || Hq > kMaxHeads || Hk > kMaxHeads)
    return fail(SSD_ERR_UNSUPPORTED, "problem too large: b=%lld L=%lld Hq=%lld Hk=%lld", (long long)b, (long long)L,
                (long long)Hq, (long long)Hk);
  if (!(eps >= 0.f) || eps > 1e30f) return fail(SSD_ERR_UNSUPPORTED, "eps=%g is not a finite number >= 0", (double)eps);
  if (interleaved != 0 && interleaved != 1)
    return fail(SSD_ERR_UNSUPPORTED, "interleaved=%d is not 0 or 1", interleaved);
  SSD_CHECK(act_dtype(q, "q"));
  const int64_t sq[4] = {b, L, Hq, N}, sk[4] = {b, L, Hk, N}, sw[1] = {N}, sp[2] = {b, L};
  SSD_CHECK(check_arg(q, "q", q->dtype, 4, sq, true));
  SSD_CHECK(check_arg(k, "k", q->dtype, 4, sk, true));
  if (q_weight) SSD_CHECK(check_arg(q_weight, "q_weight", SSD_F32, 1, sw));
  if (k_weight) SSD_CHECK(check_arg(k_weight, "k_weight", SSD_F32, 1, sw));
  int64_t npair = 0;
  if (freqs) {
    if (freqs->ndim != 1) return fail(SSD_ERR_SHAPE, "freqs: rank %d, expected 1", freqs->ndim);
    npair = freqs->shape[0];
    if (npair < 1 || 2 * npair > N)
      return fail(SSD_ERR_SHAPE, "freqs: %lld pairs do not fit in N=%lld", (long long)npair, (long long)N);
    if (npair % 4 != 0)
      return fail(SSD_ERR_UNSUPPORTED, "freqs: %lld pairs, not a multiple of 4", (long long)npair);
    SSD_CHECK(check_arg(freqs, "freqs", SSD_F32, 1, &npair));
  }
  if (positions) {
    if (positions->dtype != SSD_I32 && positions->dtype != SSD_I64)
      return fail(SSD_ERR_DTYPE, "positions: dtype %s, expected i32 or i64", dtype_name(positions->dtype));
    SSD_CHECK(check_arg(positions, "positions", positions->dtype, 2, sp));
  }
  args->add(q, "q", false);
  args->add(k, "k", false);
  args->add(q_weight, "q_weight", false);
  args->add(k_weight, "k_weight", false);
  args->add(freqs, "freqs", false);
  args->add(positions, "positions", false);
  p->q = q->data;
  p->k = k->data;
  p->qb = q->strides[0]; p->qt = q->strides[1]; p->qh = q->strides[2];
  p->kb = k->strides[0]; p->kt = k->strides[1]; p->kh = k->strides[2];
  p->qw = fptr(q_weight);
  p->kw = fptr(k_weight);
  p->freqs = fptr(freqs);
  p->pos32 = positions && positions->dtype == SSD_I32 ? (const int32_t *)positions->data : nullptr;
  p->pos64 = positions && positions->dtype == SSD_I64 ? (const int64_t *)positions->data : nullptr;
  p->eps = eps;
  p->L = (int)L; p->Hq = (int)Hq; p->Hk = (int)Hk; p->N = (int)N;
  p->npair = (int)npair;
  p->interleaved = interleaved;
  p->ntok = b * L;
  norm_rotate_plan(p);
  return SSD_OK;
}

} // namespace

extern "C" {

int64_t ssd_glr_workspace(int64_t b, int64_t L, int64_t D, int backward) {
  GlrPlan q;
  if (!glr_plan(b, L, D, backward != 0, &q)) return -1;
  return backward ? glr_back_bytes(q) : q.chain_f;
}

int ssd_glr_fwd(const ssd_tensor *x, const ssd_tensor *r, const ssd_tensor *i, const ssd_tensor *A,
                const ssd_tensor *r_bias, const ssd_tensor *i_bias, const ssd_tensor *reset,
                const ssd_tensor *lengths, const ssd_tensor *init_state, ssd_tensor *out, ssd_tensor *final_state,
                ssd_tensor *states, void *workspace, int64_t workspace_bytes, void *stream) {
  clear_error();
  GlrPlan plan;
  Args args;
  SSD_CHECK(validate_glr(x, r, i, A, r_bias, i_bias, reset, lengths, init_state, false, &plan, &args));
  const int64_t b = x->shape[0], L = x->shape[1], D = x->shape[2];
  const int64_t so[3] = {b, L, D}, sf[2] = {b, D}, ss[3] = {b, plan.nseg, D};
  SSD_CHECK(check_arg(out, "out", x->dtype, 3, so));
  if (final_state) SSD_CHECK(check_arg(final_state, "final_state", SSD_F32, 2, sf));
  if (states) SSD_CHECK(check_arg(states, "states", SSD_F32, 3, ss));
  args.add(out, "out", true);
  args.add(final_state, "final_state", true);
  args.add(states, "states", true);
  SSD_CHECK(args.overlaps(final_state, init_state));
  SSD_CHECK(args.workspace(workspace, workspace_bytes, plan.chain_f));
  SSD_CHECK(args.addressable(plan.chain_f ? workspace : nullptr));
  GlrParams p = glr_params(x, r, i, A, r_bias, i_bias, reset, lengths, init_state, plan);
  p.out = out->data;
  p.fin = fptr_out(final_state);
  p.states = fptr_out(states);
  p.inplace = final_state && init_state && final_state->data == init_state->data;
  set_chain(&p, plan.nfwd, workspace);
  const bool vec = rows4b(x) && rows4b(r) && rows4b(i) && rows4b(out);
  const hipError_t e = launch_glr(x->dtype, vec, false, p, (hipStream_t)stream);
  return e == hipSuccess ? SSD_OK : hip_fail(e, "gated recurrence launch");
}

int ssd_glr_bwd(const ssd_tensor *x, const ssd_tensor *r, const ssd_tensor *i, const ssd_tensor *A,
                const ssd_tensor *r_bias, const ssd_tensor *i_bias, const ssd_tensor *reset,
                const ssd_tensor *lengths, const ssd_tensor *init_state, const ssd_tensor *states,
                const ssd_tensor *dout, const ssd_tensor *dfinal_state, ssd_tensor *dx, ssd_tensor *dr,
                ssd_tensor *di, ssd_tensor *dA, ssd_tensor *dr_bias, ssd_tensor *di_bias, ssd_tensor *dinit_state,
                void *workspace, int64_t workspace_bytes, void *stream) {
  clear_error();
  GlrPlan plan;
  Args args;
  SSD_CHECK(validate_glr(x, r, i, A, r_bias, i_bias, reset, lengths, init_state, true, &plan, &args));
  const int64_t b = x->shape[0], L = x->shape[1], D = x->shape[2];
  const int64_t so[3] = {b, L, D}, sf[2] = {b, D}, ss[3] = {b, plan.nseg, D}, sd[1] = {D};
  if (states) SSD_CHECK(check_arg(states, "states", SSD_F32, 3, ss));
  SSD_CHECK(check_arg(dout, "dout", grad_dtype(dout, x), 3, so, true, kMaxStride));
  if (dfinal_state) SSD_CHECK(check_arg(dfinal_state, "dfinal_state", SSD_F32, 2, sf));
  SSD_CHECK(check_arg(dx, "dx", x->dtype, 3, so));
  SSD_CHECK(check_arg(dr, "dr", x->dtype, 3, so));
  SSD_CHECK(check_arg(di, "di", x->dtype, 3, so));
  if (dA) SSD_CHECK(check_arg(dA, "dA", SSD_F32, 1, sd));
  if (dr_bias) SSD_CHECK(check_arg(dr_bias, "dr_bias", SSD_F32, 1, sd));
  if (di_bias) SSD_CHECK(check_arg(di_bias, "di_bias", SSD_F32, 1, sd));
  if (dinit_state) SSD_CHECK(check_arg(dinit_state, "dinit_state", SSD_F32, 2, sf));
  args.add(states, "states", false);
  args.add(dout, "dout", false);
  args.add(dfinal_state, "dfinal_state", false);
  args.add(dx, "dx", true);
  args.add(dr, "dr", true);
  args.add(di, "di", true);
  args.add(dA, "dA", true);
  args.add(dr_bias, "dr_bias", true);
  args.add(di_bias, "di_bias", true);
  args.add(dinit_state, "dinit_state", true);
  SSD_CHECK(args.overlaps(nullptr, nullptr));
  SSD_CHECK(args.workspace(workspace, workspace_bytes, glr_back_bytes(plan)));
  SSD_CHECK(args.addressable(workspace));
  GlrParams p = glr_params(x, r, i, A, r_bias, i_bias, reset, lengths, init_state, plan);
  char *ws = (char *)workspace;
  float *part = (float *)(ws + up256(plan.chain_f > plan.chain_b ? plan.chain_f : plan.chain_b));
  const bool sums = dA || dr_bias || di_bias;
  p.part = sums ? part : nullptr;
  hipStream_t st = (hipStream_t)stream;
  const bool vec = rows4b(x) && rows4b(r) && rows4b(i);
  hipError_t e;
  if (states) {
    p.states = (float *)states->data;
  } else {
    p.states = (float *)((char *)part + up256(plan.part));
    set_chain(&p, plan.nfwd, ws);
    e = launch_glr(x->dtype, vec, false, p, st);
    if (e != hipSuccess) return hip_fail(e, "gated recurrence states launch");
  }
  p.dout = dout->data;
  p.db = b == 1 ? 0 : dout->strides[0];
  p.dt = L == 1 ? 0 : (int)dout->strides[1];
  p.dout_f32 = dout->dtype == SSD_F32;
  p.dfin = fptr(dfinal_state);
  p.dx = dx->data; p.dr = dr->data; p.di = di->data;
  p.dinit = fptr_out(dinit_state);
  set_chain(&p, plan.nseg, ws);
  e = launch_glr(x->dtype, vec && rows_of(dout, 2 * elem_size(dout->dtype)) && rows4b(dx) && rows4b(dr) && rows4b(di), true, p, st);
  if (e != hipSuccess) return hip_fail(e, "gated recurrence backward launch");
  if (!sums) return SSD_OK;
  e = launch_glr_sum(part, (int)(b * plan.nseg), (int)D, fptr_out(dA), fptr_out(dr_bias), fptr_out(di_bias), st);
  return e == hipSuccess ? SSD_OK : hip_fail(e, "gated recurrence parameter sums launch");
}

int ssd_glr_step(const ssd_tensor *state, const ssd_tensor *x, const ssd_tensor *r, const ssd_tensor *i,
                 const ssd_tensor *A, const ssd_tensor *r_bias, const ssd_tensor *i_bias, const ssd_tensor *reset,
                 ssd_tensor *new_state, ssd_tensor *out, void *stream) {
  clear_error();
  if (!x) return fail(SSD_ERR_NULL, "x: descriptor is NULL");
  if (x->ndim != 2) return fail(SSD_ERR_SHAPE, "x: rank %d, expected 2 [b,D]", x->ndim);
  const int64_t b = x->shape[0], D = x->shape[1];
  if (b < 1 || D < 1) return fail(SSD_ERR_SHAPE, "empty problem: b=%lld D=%lld", (long long)b, (long long)D);
  if (D > kMaxWidth || b > kMaxTiles || b * ((D + 255) / 256) > kMaxTiles)
    return fail(SSD_ERR_UNSUPPORTED, "problem too large: b=%lld D=%lld", (long long)b, (long long)D);
  SSD_CHECK(act_dtype(x, "x"));
  const int64_t sx[2] = {b, D}, sd[1] = {D}, sb[1] = {b};
  SSD_CHECK(check_arg(state, "state", SSD_F32, 2, sx));
  SSD_CHECK(check_arg(x, "x", x->dtype, 2, sx, true));
  SSD_CHECK(check_arg(r, "r", x->dtype, 2, sx, true));
  SSD_CHECK(check_arg(i, "i", x->dtype, 2, sx, true));
  SSD_CHECK(check_arg(A, "A", SSD_F32, 1, sd));
  if (r_bias) SSD_CHECK(check_arg(r_bias, "r_bias", SSD_F32, 1, sd));
  if (i_bias) SSD_CHECK(check_arg(i_bias, "i_bias", SSD_F32, 1, sd));
  if (reset) SSD_CHECK(check_arg(reset, "reset", SSD_U8, 1, sb));
  SSD_CHECK(check_arg(new_state, "new_state", SSD_F32, 2, sx));
  SSD_CHECK(check_arg(out, "out", x->dtype, 2, sx));
  Args args;
  args.add(state, "state", false);
  args.add(x, "x", false);
  args.add(r, "r", false);
  args.add(i, "i", false);
  args.add(A, "A", false);
  args.add(r_bias, "r_bias", false);
  args.add(i_bias, "i_bias", false);
  args.add(reset, "reset", false);
  args.add(new_state, "new_state", true);
  args.add(out, "out", true);
  SSD_CHECK(args.overlaps(new_state, state));
  SSD_CHECK(args.addressable(nullptr));
  GlrStepParams p{};
  p.x = x->data; p.r = r->data; p.i = i->data;
  p.xb = b == 1 ? 0 : x->strides[0];
  p.rb_ = b == 1 ? 0 : r->strides[0];
  p.ib_ = b == 1 ? 0 : i->strides[0];
  p.A = fptr(A); p.rbias = fptr(r_bias); p.ibias = fptr(i_bias);
  p.reset = reset ? (const uint8_t *)reset->data : nullptr;
  p.state = fptr(state);
  p.new_state = fptr_out(new_state);
  p.out = out->data;
  p.b = (int)b; p.D = (int)D;
  const bool vec = rows16(x) && rows16(r) && rows16(i) && rows16(out) && rows16(state) && rows16(new_state) &&
                   rows16(A) && (!r_bias || rows16(r_bias)) && (!i_bias || rows16(i_bias));
  const hipError_t e = launch_glr_step(x->dtype, vec, p, (hipStream_t)stream);
  return e == hipSuccess ? SSD_OK : hip_fail(e, "gated recurrence step launch");
}

int64_t ssd_norm_rotate_workspace(int64_t N) { return N >= 8 && N <= 256 && N % 8 == 0 ? norm_rotate_bytes(N) : -1; }

int ssd_norm_rotate_fwd(const ssd_tensor *q, const ssd_tensor *k, const ssd_tensor *q_weight,
                        const ssd_tensor *k_weight, const ssd_tensor *freqs, const ssd_tensor *positions,
                        ssd_tensor *q_out, ssd_tensor *k_out, float eps, int interleaved, void *stream) {
  clear_error();
  NormRotParams p{};
  Args args;
  SSD_CHECK(validate_norm_rotate(q, k, q_weight, k_weight, freqs, positions, eps, interleaved, &p, &args));
  SSD_CHECK(check_arg(q_out, "q_out", q->dtype, 4, q->shape));
  SSD_CHECK(check_arg(k_out, "k_out", q->dtype, 4, k->shape));
  args.add(q_out, "q_out", true);
  args.add(k_out, "k_out", true);
  SSD_CHECK(args.overlaps(nullptr, nullptr));
  SSD_CHECK(args.addressable(nullptr));
  p.oq = q_out->data;
  p.ok = k_out->data;
  const bool vec = rows4(q) && rows4(k) && rows4(q_weight) && rows4(k_weight) && rows4(q_out) && rows4(k_out);
  const hipError_t e = launch_norm_rotate(q->dtype, vec, false, p, (hipStream_t)stream);
  return e == hipSuccess ? SSD_OK : hip_fail(e, "norm and rotation launch");
}

int ssd_norm_rotate_bwd(const ssd_tensor *q, const ssd_tensor *k, const ssd_tensor *q_weight,
                        const ssd_tensor *k_weight, const ssd_tensor *freqs, const ssd_tensor *positions,
                        const ssd_tensor *dq_out, const ssd_tensor *dk_out, ssd_tensor *dq, ssd_tensor *dk,
                        ssd_tensor *dq_weight, ssd_tensor *dk_weight, float eps, int interleaved, void *workspace,
                        int64_t workspace_bytes, void *stream) {
  clear_error();
  NormRotParams p{};
  Args args;
  SSD_CHECK(validate_norm_rotate(q, k, q_weight, k_weight, freqs, positions, eps, interleaved, &p, &args));
  SSD_CHECK(check_arg(dq_out, "dq_out", grad_dtype(dq_out, q), 4, q->shape, true));
  SSD_CHECK(check_arg(dk_out, "dk_out", dq_out->dtype, 4, k->shape, true));
  SSD_CHECK(check_arg(dq, "dq", q->dtype, 4, q->shape));
  SSD_CHECK(check_arg(dk, "dk", q->dtype, 4, k->shape));
  const int64_t sw[1] = {q->shape[3]};
  if (dq_weight) SSD_CHECK(check_arg(dq_weight, "dq_weight", SSD_F32, 1, sw));
  if (dk_weight) SSD_CHECK(check_arg(dk_weight, "dk_weight", SSD_F32, 1, sw));
  args.add(dq_out, "dq_out", false);
  args.add(dk_out, "dk_out", false);
  args.add(dq, "dq", true);
  args.add(dk, "dk", true);
  args.add(dq_weight, "dq_weight", true);
  args.add(dk_weight, "dk_weight", true);
  SSD_CHECK(args.overlaps(nullptr, nullptr));
  const int64_t need = dq_weight || dk_weight ? norm_rotate_bytes(q->shape[3]) : 0;
  SSD_CHECK(args.workspace(workspace, workspace_bytes, need));
  SSD_CHECK(args.addressable(need ? workspace : nullptr));
  p.dyq = dq_out->data;
  p.dyk = dk_out->data;
  p.dy_f32 = dq_out->dtype == SSD_F32;
  p.dqb = dq_out->strides[0]; p.dqt = dq_out->strides[1]; p.dqh = dq_out->strides[2];
  p.dkb = dk_out->strides[0]; p.dkt = dk_out->strides[1]; p.dkh = dk_out->strides[2];
  p.oq = dq->data;
  p.ok = dk->data;
  p.dqw = fptr_out(dq_weight);
  p.dkw = fptr_out(dk_weight);
  p.part = need ? (float *)workspace : nullptr;
  const bool vec = rows4(q) && rows4(k) && rows4(q_weight) && rows4(k_weight) && rows4(dq_out) && rows4(dk_out) &&
                   rows4(dq) && rows4(dk);
  const hipError_t e = launch_norm_rotate(q->dtype, vec, true, p, (hipStream_t)stream);
  return e == hipSuccess ? SSD_OK : hip_fail(e, "norm and rotation backward launch");
}

} // extern "C"
