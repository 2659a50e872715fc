// ssd_cache_api.hip -- the C ABI of the paged key-value cache and of the
// attention over it: argument validation, workspace layout and launches.
// Declarations and the contract are in include/ssd.h.  Every check runs on the
// host before the first launch; what only the device knows (start, tokens, the
// page table's entries) is bounded in the kernels.
#include <hip/hip_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "ssd.h"
#include "ssd_args.h"
#include "ssd_cache.h"

using namespace ssd;

namespace {

constexpr int64_t kMaxTokens = (int64_t)1 << 24;
constexpr int64_t kMaxBatch = (int64_t)1 << 16;
constexpr int64_t kMaxBatchTokens = (int64_t)1 << 25; // at most as many waves in one launch
constexpr int64_t kMaxHeads = (int64_t)1 << 16;
constexpr int64_t kMaxSlot = (int64_t)1 << 24;        // token stride of a page: 16 fp32 rows within 2^31 bytes
constexpr int64_t kMaxPage = ((int64_t)1 << 32) - 1;   // page stride
constexpr int64_t kMaxCapacity = (int64_t)1 << 30;    // tokens of a row
constexpr int64_t kMaxWindow = (int64_t)1 << 33;      // positions stay below 2^31 + 2^24
constexpr int64_t kMaxUnits = (int64_t)1 << 30;       // of all rows together

// A cache [pages, page_size, Hk, N]: a view with rows of 16-byte pieces, no
// element of which is two.
int check_cache(const ssd_tensor *t, const char *name, int dtype, const int64_t *shape, bool written) {
  SSD_CHECK(check_arg(t, name, dtype, 4, shape, true));
  if (!rows_of(t, 16)) return fail(SSD_ERR_LAYOUT, "%s: rows are not in 16-byte pieces", name);
  for (int d = 0; d < 2; ++d)
    if (t->shape[d] != 1 && t->strides[d] > (d == 0 ? kMaxPage : kMaxSlot))
      return fail(SSD_ERR_UNSUPPORTED, "%s: stride of dim %d is %lld", name, d, (long long)t->strides[d]);
  if (written) {
    // strides from the largest: each holds all of what the smaller ones reach
    int dim[3] = {0, 1, 2};
    for (int i = 0; i < 2; ++i)
      for (int j = i + 1; j < 3; ++j)
        if (t->strides[dim[j]] > t->strides[dim[i]]) { const int x = dim[i]; dim[i] = dim[j]; dim[j] = x; }
    int64_t inner = t->shape[3];
    for (int i = 2; i >= 0; --i) {
      const int d = dim[i];
      if (t->shape[d] == 1) continue;
      if (t->strides[d] < inner) return fail(SSD_ERR_LAYOUT, "%s: its own rows overlap (stride of dim %d)", name, d);
      inner += (t->shape[d] - 1) * t->strides[d];
    }
  }
  return SSD_OK;
}

// Two caches of one shape that lie in each other's gaps, as the halves of one
// tensor [pages, 2, page_size, Hk, N] or [pages, page_size, Hk, 2, N] do: with
// equal, nested strides, the distance between them must pass over all of what lies
// inside some stride, and with that still fit into it and into the larger ones.
bool woven_apart(const ssd_tensor *a, const ssd_tensor *b) {
  const int es = elem_size(a->dtype);
  uintptr_t x = (uintptr_t)a->data, y = (uintptr_t)b->data;
  const uintptr_t diff = x < y ? y - x : x - y;
  if (diff % es) return false;
  const int64_t delta = (int64_t)(diff / es);
  int dim[3], n = 0;
  for (int d = 0; d < 3; ++d) {
    if (a->shape[d] == 1) continue;
    if (a->strides[d] != b->strides[d]) return false;
    dim[n++] = d;
  }
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j)
      if (a->strides[dim[j]] > a->strides[dim[i]]) { const int t = dim[i]; dim[i] = dim[j]; dim[j] = t; }
  for (int i = 0; i <= n; ++i) {
    int64_t extent = a->shape[3];
    for (int j = i; j < n; ++j) extent += (a->shape[dim[j]] - 1) * a->strides[dim[j]];
    if (delta >= extent) return true;
    if (i < n) {
      int64_t inner = a->shape[3];
      for (int j = i + 1; j < n; ++j) inner += (a->shape[dim[j]] - 1) * a->strides[dim[j]];
      if (inner + delta > a->strides[dim[i]]) return false;
    }
  }
  return false;
}

int64_t stride(const ssd_tensor *t, int d) { return t->shape[d] == 1 ? 0 : t->strides[d]; }

// The caches and the rows' places: b rows of at most L new tokens.
int validate_cache(const ssd_tensor *k_cache, const ssd_tensor *v_cache, const ssd_tensor *page_table,
                   const ssd_tensor *start, const ssd_tensor *tokens, int dtype, int64_t b, int64_t Hk, int64_t N,
                   bool written, CacheParams *c, Args *args) {
  if (!k_cache) return fail(SSD_ERR_NULL, "k_cache: descriptor is NULL");
  if (k_cache->ndim != 4)
    return fail(SSD_ERR_SHAPE, "k_cache: rank %d, expected 4 [pages,page_size,Hk,N]", k_cache->ndim);
  const int64_t pages = k_cache->shape[0], size = k_cache->shape[1];
  if (pages < 1 || size < 1)
    return fail(SSD_ERR_SHAPE, "empty cache: pages=%lld page_size=%lld", (long long)pages, (long long)size);
  if (pages > INT32_MAX) return fail(SSD_ERR_UNSUPPORTED, "k_cache: %lld pages", (long long)pages);
  const int64_t sc[4] = {pages, size, Hk, N}, sb[1] = {b};
  SSD_CHECK(check_cache(k_cache, "k_cache", dtype, sc, written));
  SSD_CHECK(check_cache(v_cache, "v_cache", dtype, sc, written));
  if (!page_table) return fail(SSD_ERR_NULL, "page_table: descriptor is NULL");
  if (page_table->ndim != 2) return fail(SSD_ERR_SHAPE, "page_table: rank %d, expected 2 [b,width]", page_table->ndim);
  const int64_t width = page_table->shape[1];
  if (width < 1) return fail(SSD_ERR_SHAPE, "page_table: no columns");
  const int64_t st[2] = {b, width};
  SSD_CHECK(check_arg(page_table, "page_table", SSD_I32, 2, st, true));
  SSD_CHECK(check_arg(start, "start", SSD_I32, 1, sb));
  if (tokens) SSD_CHECK(check_arg(tokens, "tokens", SSD_I32, 1, sb));
  if (width > kMaxCapacity || size > kMaxCapacity || width * size > kMaxCapacity ||
      b * ((width * size + kAttnUnit - 1) / kAttnUnit) > kMaxUnits)
    return fail(SSD_ERR_UNSUPPORTED, "page_table: %lld rows of %lld pages of %lld tokens are too many", (long long)b,
                (long long)width, (long long)size);
  args->add(k_cache, "k_cache", written);
  args->add(v_cache, "v_cache", written);
  args->add(page_table, "page_table", false);
  args->add(start, "start", false);
  args->add(tokens, "tokens", false);
  c->kc = k_cache->data;
  c->vc = v_cache->data;
  c->kp = stride(k_cache, 0); c->ks = stride(k_cache, 1); c->kh = stride(k_cache, 2);
  c->vp = stride(v_cache, 0); c->vs = stride(v_cache, 1); c->vh = stride(v_cache, 2);
  c->table = (const int32_t *)page_table->data;
  c->tb = stride(page_table, 0);
  c->start = (const int32_t *)start->data;
  c->tokens = tokens ? (const int32_t *)tokens->data : nullptr;
  c->page = fast_div((uint32_t)size);
  c->pages = (int)pages;
  c->width = (int)width;
  c->capacity = (int)(width * size);
  return SSD_OK;
}

int check_heads(int64_t N) {
  if (N % 8 != 0 || N > 256 || N < 8)
    return fail(SSD_ERR_UNSUPPORTED, "N=%lld is not a multiple of 8 up to 256", (long long)N);
  return SSD_OK;
}

// The attention's sizes; false if the call is refused for them.
bool attn_sizes(int64_t b, int64_t L, int64_t Hq, int64_t Hk, int64_t N) {
  return b >= 1 && L >= 1 && Hq >= 1 && Hk >= 1 && b <= kMaxBatch && L <= kMaxTokens && b * L <= kMaxBatchTokens &&
         Hq <= kMaxHeads && Hk <= kMaxHeads && Hq % Hk == 0 && b * L * Hq <= (int64_t)1 << 30 && N >= 8 && N <= 256 &&
         N % 8 == 0;
}
int64_t attn_setup(AttnParams *p, int dtype, int64_t b, int64_t L, int64_t Hq, int64_t Hk, int64_t N) {
  p->b = (int)b; p->L = (int)L; p->Hq = (int)Hq; p->Hk = (int)Hk; p->N = (int)N;
  p->G = (int)(Hq / Hk);
  p->group = fast_div((uint32_t)p->G);
  return attn_plan(p, dtype);
}
// Workspace that suffices for either type, -1 if the sizes are refused.
int64_t attn_bytes(int64_t b, int64_t L, int64_t Hq, int64_t Hk, int64_t N) {
  if (!attn_sizes(b, L, Hq, Hk, N)) return -1;
  AttnParams p{};
  const int64_t f = attn_setup(&p, SSD_F32, b, L, Hq, Hk, N), h = attn_setup(&p, SSD_BF16, b, L, Hq, Hk, N);
  return f < 0 || h < 0 ? -1 : f > h ? f : h;
}

// q and out [b, Hq, N] (step) or [b, L, Hq, N].
int attn(const ssd_tensor *q, const ssd_tensor *k_cache, const ssd_tensor *v_cache, const ssd_tensor *page_table,
         const ssd_tensor *start, const ssd_tensor *tokens, ssd_tensor *out, ssd_tensor *lse, float scale,
         int64_t window, void *workspace, int64_t workspace_bytes, bool step, void *stream) {
  clear_error();
  if (!q) return fail(SSD_ERR_NULL, "q: descriptor is NULL");
  const int nd = step ? 3 : 4;
  if (q->ndim != nd) return fail(SSD_ERR_SHAPE, "q: rank %d, expected %s", q->ndim, step ? "3 [b,Hq,N]" : "4 [b,L,Hq,N]");
  const int64_t b = q->shape[0], L = step ? 1 : q->shape[1], Hq = q->shape[nd - 2], N = q->shape[nd - 1];
  if (!k_cache) return fail(SSD_ERR_NULL, "k_cache: descriptor is NULL");
  if (k_cache->ndim != 4)
    return fail(SSD_ERR_SHAPE, "k_cache: rank %d, expected 4 [pages,page_size,Hk,N]", k_cache->ndim);
  const int64_t Hk = k_cache->shape[2];
  if (b < 1 || L < 1 || Hq < 1 || Hk < 1 || N < 1)
    return fail(SSD_ERR_SHAPE, "empty problem: b=%lld L=%lld Hq=%lld Hk=%lld N=%lld", (long long)b, (long long)L,
                (long long)Hq, (long long)Hk, (long long)N);
  SSD_CHECK(check_heads(N));
  if (Hq % Hk != 0) return fail(SSD_ERR_SHAPE, "Hq=%lld is not a multiple of Hk=%lld", (long long)Hq, (long long)Hk);
  if (attn_bytes(b, L, Hq, Hk, N) < 0)
    return fail(SSD_ERR_UNSUPPORTED, "problem too large: b=%lld L=%lld Hq=%lld", (long long)b, (long long)L,
                (long long)Hq);
  if (!(fabsf(scale) >= FLT_MIN && fabsf(scale) <= 1e30f))
    return fail(SSD_ERR_UNSUPPORTED, "scale=%g is not in size between 2^-126 and 1e30", (double)scale);
  if (window < 0) return fail(SSD_ERR_UNSUPPORTED, "window=%lld is negative", (long long)window);
  SSD_CHECK(act_dtype(q, "q"));
  AttnParams p{};
  const int64_t need = attn_setup(&p, q->dtype, b, L, Hq, Hk, N);
  Args args;
  SSD_CHECK(check_arg(q, "q", q->dtype, nd, q->shape, true));
  args.add(q, "q", false);
  SSD_CHECK(validate_cache(k_cache, v_cache, page_table, start, tokens, q->dtype, b, Hk, N, false, &p.c, &args));
  SSD_CHECK(check_arg(out, "out", q->dtype, nd, q->shape));
  if ((uintptr_t)out->data % 16) return fail(SSD_ERR_LAYOUT, "out: data pointer is not 16-byte aligned");
  const int64_t sl[3] = {b, step ? Hq : L, Hq};
  if (lse) SSD_CHECK(check_arg(lse, "lse", SSD_F32, nd - 1, sl));
  args.add(out, "out", true);
  args.add(lse, "lse", true);
  SSD_CHECK(args.overlaps(nullptr, nullptr));
  SSD_CHECK(args.workspace(workspace, workspace_bytes, need));
  SSD_CHECK(args.addressable(need ? workspace : nullptr));
  p.q = q->data;
  p.qb = stride(q, 0);
  p.qt = step ? 0 : stride(q, 1);
  p.qh = stride(q, nd - 2);
  p.qvec = rows_of(q, 16);
  p.out = out->data;
  p.lse = fptr_out(lse);
  p.scale = fabsf(scale) * 1.4426950408889634f;
  p.negate = scale < 0.f;
  p.window = window < kMaxWindow ? window : 0; // one that reaches past every position is none
  attn_slots(&p);
  if (need) attn_workspace(&p, workspace);
  const hipError_t e = launch_attn(q->dtype, p, (hipStream_t)stream);
  return e == hipSuccess ? SSD_OK : hip_fail(e, "attention launch");
}

} // namespace

extern "C" {

int ssd_kv_append(const ssd_tensor *q, const ssd_tensor *k, const ssd_tensor *v, const ssd_tensor *freqs,
                  const ssd_tensor *page_table, const ssd_tensor *start, const ssd_tensor *tokens, ssd_tensor *q_out,
                  ssd_tensor *k_cache, ssd_tensor *v_cache, int interleaved, void *stream) {
  clear_error();
  if (!k) return fail(SSD_ERR_NULL, "k: descriptor is NULL");
  if (k->ndim != 4) return fail(SSD_ERR_SHAPE, "k: rank %d, expected 4 [b,L,Hk,N]", k->ndim);
  const int64_t b = k->shape[0], L = k->shape[1], Hk = k->shape[2], N = k->shape[3];
  int64_t Hq = 0;
  if (q) {
    if (q->ndim != 4) return fail(SSD_ERR_SHAPE, "q: rank %d, expected 4 [b,L,Hq,N]", q->ndim);
    Hq = q->shape[2];
  } else if (q_out) {
    return fail(SSD_ERR_NULL, "q: descriptor is NULL, but q_out is there");
  }
  if (b < 1 || L < 1 || Hk < 1 || N < 1 || (q && Hq < 1))
    return fail(SSD_ERR_SHAPE, "empty problem: b=%lld L=%lld Hq=%lld Hk=%lld N=%lld", (long long)b, (long long)L,
                (long long)Hq, (long long)Hk, (long long)N);
  SSD_CHECK(check_heads(N));
  if (b > kMaxBatch || L > kMaxTokens || b * L > kMaxBatchTokens || Hq > kMaxHeads || Hk > kMaxHeads)
    return fail(SSD_ERR_UNSUPPORTED, "problem too large: b=%lld L=%lld Hq=%lld Hk=%lld", (long long)b, (long long)L,
                (long long)Hq, (long long)Hk);
  if (interleaved != 0 && interleaved != 1)
    return fail(SSD_ERR_UNSUPPORTED, "interleaved=%d is not 0 or 1", interleaved);
  SSD_CHECK(act_dtype(k, "k"));
  const int64_t sq[4] = {b, L, Hq, N}, sk[4] = {b, L, Hk, N};
  Args args;
  AppendParams p{};
  SSD_CHECK(check_arg(k, "k", k->dtype, 4, sk, true));
  SSD_CHECK(check_arg(v, "v", k->dtype, 4, sk, true));
  if (q) {
    SSD_CHECK(check_arg(q, "q", k->dtype, 4, sq, true));
    SSD_CHECK(check_arg(q_out, "q_out", k->dtype, 4, sq));
  }
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
  SSD_CHECK(validate_cache(k_cache, v_cache, page_table, start, tokens, k->dtype, b, Hk, N, true, &p.c, &args));
  args.add(q, "q", false);
  args.add(k, "k", false);
  args.add(v, "v", false);
  args.add(freqs, "freqs", false);
  args.add(q_out, "q_out", true);
  if (woven_apart(k_cache, v_cache)) args.apart[0] = k_cache, args.apart[1] = v_cache;
  SSD_CHECK(args.overlaps(nullptr, nullptr));
  SSD_CHECK(args.addressable(nullptr));
  p.k = k->data; p.v = v->data;
  p.kb = k->strides[0]; p.kt = k->strides[1]; p.kh = k->strides[2];
  p.vb = v->strides[0]; p.vt = v->strides[1]; p.vh = v->strides[2];
  if (q) {
    p.q = q->data;
    p.qb = q->strides[0]; p.qt = q->strides[1]; p.qh = q->strides[2];
    p.q_out = q_out->data;
  }
  p.freqs = fptr(freqs);
  p.L = (int)L; p.Hq = (int)Hq; p.Hk = (int)Hk; p.N = (int)N;
  p.npair = (int)npair;
  p.interleaved = interleaved;
  p.ntok = b * L;
  append_plan(&p);
  const bool vec = rows4(q) && rows4(k) && rows4(v) && rows4(q_out);
  const hipError_t e = launch_append(k->dtype, vec, p, (hipStream_t)stream);
  return e == hipSuccess ? SSD_OK : hip_fail(e, "cache append launch");
}

int64_t ssd_attn_workspace(int64_t b, int64_t L, int64_t Hq, int64_t Hk, int64_t N) {
  return attn_bytes(b, L, Hq, Hk, N);
}

int ssd_attn_fwd(const ssd_tensor *q, const ssd_tensor *k_cache, const ssd_tensor *v_cache,
                 const ssd_tensor *page_table, const ssd_tensor *start, const ssd_tensor *tokens, ssd_tensor *out,
                 ssd_tensor *lse, float scale, int64_t window, void *workspace, int64_t workspace_bytes,
                 void *stream) {
  return attn(q, k_cache, v_cache, page_table, start, tokens, out, lse, scale, window, workspace, workspace_bytes,
              false, stream);
}

int ssd_attn_step(const ssd_tensor *q, const ssd_tensor *k_cache, const ssd_tensor *v_cache,
                  const ssd_tensor *page_table, const ssd_tensor *start, ssd_tensor *out, ssd_tensor *lse, float scale,
                  int64_t window, void *workspace, int64_t workspace_bytes, void *stream) {
  return attn(q, k_cache, v_cache, page_table, start, nullptr, out, lse, scale, window, workspace, workspace_bytes,
              true, stream);
}

} // extern "C"
