// ssd_append.hip -- keys and values of new tokens into a paged cache, the
// position rotation applied to the keys on the way and to the queries in the
// same pass.  Token t of row i stands at p = start[i] + t:
//
//   k_cache[slot(i, p)] = R(p) k,   v_cache[slot(i, p)] = v,   q_out = R(p) q
//
// with slot(i, p) = (page_table[i][p / page_size], p mod page_size) and R(p) as
// in the norm with rotation, whose decomposition this is: a lane owns eight
// elements of a head vector, four whole pairs, so the rotation needs no
// exchange; LH lanes make a head, and a wave walks over its token's heads, so the
// angles and the slot are formed once per token.  Heads are walked queries
// first, then keys, then values, which are moved as they are.  Bound by HBM
// (each input once in, once out), in a decode step by the launch and three
// loads one behind the other (start, page table, rows).
#include "ssd_cache.h"
#include "ssd_device.h"
#include "ssd_rotate.h"

namespace ssd {
namespace {

constexpr int kThreads = 256;

// A lane's eight elements moved as they are.
template <typename T, bool VEC> __device__ __forceinline__ void move8(T *lo, T *hi, const Raw<T, VEC> &r) {
  if constexpr (VEC && sizeof(T) == 2) {
    *reinterpret_cast<u32x2 *>(lo) = u32x2{r.d[0], r.d[1]};
    *reinterpret_cast<u32x2 *>(hi) = u32x2{r.d[2], r.d[3]};
  } else if constexpr (sizeof(T) == 2) {
    uint16_t *a = reinterpret_cast<uint16_t *>(lo), *b = reinterpret_cast<uint16_t *>(hi);
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e] = (uint16_t)(r.d[e] >> 16), b[e] = (uint16_t)(r.d[4 + e] >> 16);
  } else if constexpr (VEC) {
    *reinterpret_cast<u32x4 *>(lo) = u32x4{r.d[0], r.d[1], r.d[2], r.d[3]};
    *reinterpret_cast<u32x4 *>(hi) = u32x4{r.d[4], r.d[5], r.d[6], r.d[7]};
  } else {
    uint32_t *a = reinterpret_cast<uint32_t *>(lo), *b = reinterpret_cast<uint32_t *>(hi);
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e] = r.d[e], b[e] = r.d[4 + e];
  }
}

// Where the lane group stands: a token, its slot in the cache and the heads left.
struct Place {
  int64_t row, kslot, vslot; // kslot, vslot: elements from the caches' first, of head 0
  int t;
  bool stored; // the token has a slot
};

// The walk over a token's heads: kind 0 queries, 1 keys, 2 values.
template <typename T> struct HeadWalk {
  const T *src;
  T *dst;
  int h, kind;
  __device__ __forceinline__ void at(const AppendParams &p, const Place &pl, const Slot &sl) {
    kind = h < p.Hq ? 0 : h < p.Hq + p.Hk ? 1 : 2;
    if (kind == 0) {
      src = (const T *)p.q + pl.row * p.qb + pl.t * p.qt + h * p.qh;
      dst = (T *)p.q_out + ((pl.row * p.L + pl.t) * p.Hq + h) * p.N;
    } else if (kind == 1) {
      src = (const T *)p.k + pl.row * p.kb + pl.t * p.kt + (h - p.Hq) * p.kh;
      dst = (T *)p.c.kc + pl.kslot + (h - p.Hq) * p.c.kh;
    } else {
      src = (const T *)p.v + pl.row * p.vb + pl.t * p.vt + (h - p.Hq - p.Hk) * p.vh;
      dst = (T *)p.c.vc + pl.vslot + (h - p.Hq - p.Hk) * p.c.vh;
    }
    src += sl.lo, dst += sl.lo;
  }
  __device__ __forceinline__ void next(const AppendParams &p, const Place &pl, const Slot &sl, int step) {
    h += step;
    const int end = kind == 0 ? p.Hq : kind == 1 ? p.Hq + p.Hk : p.Hq + 2 * p.Hk;
    if (h >= end) {
      at(p, pl, sl);
    } else {
      src += step * (kind == 0 ? p.qh : kind == 1 ? p.kh : p.vh);
      dst += step * (kind == 0 ? (int64_t)p.N : kind == 1 ? p.c.kh : p.c.vh);
    }
  }
};

template <typename T, int LH, bool VEC, bool INTER, bool ONCE>
__global__ __launch_bounds__(kThreads) void append_kernel(AppendParams p) {
  constexpr int HPW = 64 / LH;
  const int lane = threadIdx.x & 63, g = lane / LH;
  const uint32_t item = __builtin_amdgcn_readfirstlane(blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6));
  const uint32_t group = item / (uint32_t)p.split;
  const int slice = (int)(item - group * (uint32_t)p.split);
  const uint32_t tok = group * (uint32_t)(HPW >> p.hg_log) + (uint32_t)(g >> p.hg_log);
  if (tok >= p.ntok) return;
  const int heads = p.Hq + 2 * p.Hk, hend = min(heads, (slice + 1) * p.per), step = 1 << p.hg_log;
  HeadWalk<T> cur;
  cur.h = slice * p.per + (g & (step - 1));
  if (cur.h >= hend) return;
  Place pl;
  pl.row = tok / (uint32_t)p.L;
  pl.t = (int)(tok - (uint32_t)pl.row * (uint32_t)p.L);
  if (p.c.tokens && pl.t >= p.c.tokens[pl.row]) return;
  const int64_t pos = (int64_t)p.c.start[pl.row] + pl.t;
  pl.stored = pos >= 0 && pos < p.c.capacity;
  pl.kslot = pl.vslot = 0;
  if (pl.stored) {
    const uint32_t entry = div_by((uint32_t)pos, p.c.page), slot = (uint32_t)pos - entry * p.c.page.d;
    const int id = p.c.table[pl.row * p.c.tb + entry];
    pl.stored = id >= 0 && id < p.c.pages;
    if (pl.stored) {
      pl.kslot = id * p.c.kp + slot * p.c.ks;
      pl.vslot = id * p.c.vp + slot * p.c.vs;
    }
  }
  const Slot sl = lane_slot<INTER>(p.N, p.npair, lane % LH);
  if (!sl.in) return;
  const int gap = sl.hi - sl.lo;
  cur.at(p, pl, sl);
  Raw<T, VEC> r{};
  r.template load<ONCE>(cur.src, cur.src + gap);
  const Turn an = sl.turns && cur.kind < 2 ? turn_at(p.freqs, sl, (double)pos) : no_turn();
  for (;;) {
    HeadWalk<T> nxt = cur;
    nxt.next(p, pl, sl, step);
    const bool more = nxt.h < hend;
    Raw<T, VEC> rn{};
    if (more) rn.template load<ONCE>(nxt.src, nxt.src + gap);
    if (cur.kind == 2 || !sl.turns) {
      if (cur.kind == 0 || pl.stored) move8<T, VEC>(cur.dst, cur.dst + gap, r);
    } else {
      float x[8], y[8];
      r.template pairs<INTER>(x);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[e] = fmaf(x[e], an.c[e], -(x[4 + e] * an.s[e]));
        y[4 + e] = fmaf(x[e], an.s[e], x[4 + e] * an.c[e]);
      }
      if (cur.kind == 0 || pl.stored) store8<T, VEC, INTER>(cur.dst, cur.dst + gap, y);
    }
    if (!more) break;
    cur = nxt;
    r = rn;
  }
}

constexpr int64_t kOnceBytes = (int64_t)128 << 20;

template <typename T, int LH, bool VEC> hipError_t launch_one(const AppendParams &p, hipStream_t st) {
  const uint32_t grid = (uint32_t)((p.nitem + 3) / 4);
  const bool once = VEC && p.ntok * (p.Hq + 2 * p.Hk) * p.N * (int64_t)sizeof(T) >= kOnceBytes;
  if (p.interleaved) {
    if (once) append_kernel<T, LH, VEC, true, VEC><<<grid, kThreads, 0, st>>>(p);
    else append_kernel<T, LH, VEC, true, false><<<grid, kThreads, 0, st>>>(p);
  } else {
    if (once) append_kernel<T, LH, VEC, false, VEC><<<grid, kThreads, 0, st>>>(p);
    else append_kernel<T, LH, VEC, false, false><<<grid, kThreads, 0, st>>>(p);
  }
  return hipGetLastError();
}
template <typename T, bool VEC> hipError_t launch_lh(const AppendParams &p, hipStream_t st) {
  if (p.N <= 16) return launch_one<T, 2, VEC>(p, st);
  if (p.N <= 32) return launch_one<T, 4, VEC>(p, st);
  if (p.N <= 64) return launch_one<T, 8, VEC>(p, st);
  if (p.N <= 128) return launch_one<T, 16, VEC>(p, st);
  return launch_one<T, 32, VEC>(p, st);
}

} // namespace

// Splits the tokens' heads into items: fewer than kEnough waves leave compute
// units idle, the heads of a token are then spread over several waves, each
// forming the angles again.
void append_plan(AppendParams *p) {
  constexpr int64_t kEnough = 4096;
  int lh = 2;
  while (8 * lh < p->N) lh *= 2;
  const int hpw = 64 / lh, H = p->Hq + 2 * p->Hk;
  p->hg_log = 0;
  while ((1 << p->hg_log) < hpw && (1 << p->hg_log) < H) ++p->hg_log;
  const int hg = 1 << p->hg_log, tpw = hpw / hg;
  const int64_t groups = (p->ntok + tpw - 1) / tpw;
  const int rounds = (H + hg - 1) / hg;
  const int64_t want = (kEnough + groups - 1) / groups;
  const int split0 = (int)(want < rounds ? want : rounds);
  const int per = (rounds + split0 - 1) / split0;
  p->per = per * hg;
  p->split = (rounds + per - 1) / per;
  p->nitem = groups * p->split;
}

hipError_t launch_append(int dtype, bool vec, const AppendParams &p, hipStream_t st) {
  if (dtype == 1) return vec ? launch_lh<__bf16, true>(p, st) : launch_lh<__bf16, false>(p, st);
  return vec ? launch_lh<float, true>(p, st) : launch_lh<float, false>(p, st);
}

} // namespace ssd
