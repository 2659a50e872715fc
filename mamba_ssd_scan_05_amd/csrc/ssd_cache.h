// ssd_cache.h -- launch interface between the C ABI (ssd_cache_api.hip) and the
// kernels of the paged key-value cache (ssd_append.hip) and of the attention
// over it (ssd_attn.hip).  Not installed; not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssd {

// n / d for 0 <= n < 2^31 and d >= 1 by a product: with 2^s >= d the least such
// power and m = floor(2^(31+s) / d) + 1, m d - 2^(31+s) is at most d <= 2^s, so
// n m / 2^(31+s) exceeds n / d by less than 1 / d.
struct FastDiv {
  uint32_t d, m;
  int s; // of the product's high 32 bits
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f{d, 0, 0};
  if (d == 1) return f; // m would need 33 bits
  int s = 1;
  while (((uint64_t)1 << s) < d) ++s;
  f.m = (uint32_t)((((uint64_t)1 << (31 + s)) / d) + 1);
  f.s = s - 1;
  return f;
}
__device__ __forceinline__ uint32_t div_by(uint32_t n, const FastDiv &f) {
  return f.d == 1 ? n : __umulhi(n, f.m) >> f.s;
}

// The cache and the rows' places in it.  Strides in elements.
struct CacheParams {
  void *kc, *vc;                    // [pages, page_size, Hk, N], last dim contiguous
  int64_t kp, ks, kh, vp, vs, vh;
  const int32_t *table;             // [b, width]
  int64_t tb;                       // its batch stride
  const int32_t *start;             // [b]
  const int32_t *tokens;            // [b] or null: L
  FastDiv page;                     // the page size
  int pages, width, capacity;       // capacity = width * page size < 2^31
};

struct AppendParams {
  CacheParams c;
  const void *q, *k, *v;            // [b, L, Hq / Hk, N], last dim contiguous; q may be null
  int64_t qb, qt, qh, kb, kt, kh, vb, vt, vh;
  void *q_out;                      // [b, L, Hq, N] dense
  const float *freqs;               // [npair]
  int L, Hq, Hk, N, npair, interleaved; // Hq = 0 without q
  int64_t ntok;
  // set by append_plan
  int64_t nitem;
  int hg_log, per, split;
};
void append_plan(AppendParams *p);
// dtype 1 = bf16, 0 = fp32; vec: strides and pointers of q, k and v allow
// 4-element accesses.
hipError_t launch_append(int dtype, bool vec, const AppendParams &p, hipStream_t stream);

// Attention of a row's new tokens over the cache.  A row's query vectors of one
// key head are the L G pairs (token, head of the group of G), tokens first.
constexpr int kAttnUnit = 64; // keys: the plan's unit of a row's length
struct AttnParams {
  CacheParams c;
  const void *q;                    // [b, L, Hq, N], last dim contiguous
  int64_t qb, qt, qh;
  int qvec;                         // strides and pointer of q allow 16-byte loads
  void *out;                        // [b, L, Hq, N] dense
  float *lse;                       // [b, L, Hq] or null
  float scale;                      // of the products, times log2(e), >= 0
  int negate;                       // the scale was negative
  int64_t window;                   // 0: none
  int b, L, Hq, Hk, G, N;
  FastDiv group;                    // G
  // set by attn_plan
  int workers;                      // pieces of all rows' lengths together, at most; 1: one piece a row
  int prefer, enough;               // as many, but no larger than `enough` units, if workers allows
  int slots;                        // pieces at most
  int stores, cuts;                 // pieces of rows that have more than one, and such rows, at most
  int rows, tiles;                  // query vectors of a tile, tiles of a row and key head
  int prow;                         // query vectors of a tile that may be there
  float *part;                      // [stores, Hk, tiles, prow, N], products' sums
  float2 *part_ml;                  // [stores, Hk, tiles, prow], maximum and sum
  int2 *pieces;                     // [b]: the place in part of a row's first piece, and how many it has
  int4 *list;                       // [slots]: row (-1: none), index, count, place; null: every workgroup
                                    // makes the plan for itself
  int4 *cut;                        // [cuts], with list: row (-1: none), first place, count
};
// Fills workers, slots, stores, cuts, rows and tiles; workspace bytes, -1 if the call is too large.
int64_t attn_plan(AttnParams *p, int dtype);
// Many query vectors of a row and key head, bf16 (ssd_attn_rows.hip); query vectors of its tile.
int attn_rows(int N);
hipError_t launch_attn_rows(const AttnParams &p, hipStream_t stream);
// Fewer slots where the cache (c, window) has no room for more pieces.
void attn_slots(AttnParams *p);
void attn_workspace(AttnParams *p, void *workspace);
hipError_t launch_attn(int dtype, const AttnParams &p, hipStream_t stream);
} // namespace ssd
