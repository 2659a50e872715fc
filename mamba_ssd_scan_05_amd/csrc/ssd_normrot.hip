// ssd_normrot.hip -- norm of queries and keys for each head with the position
// rotation in the same pass, and its gradients.  Per head vector x of N
// elements at position p:
//
//   n = x * rstd,  rstd = 1 / sqrt(mean(x^2) + eps),   y = R(p) (w * n)
//
// R(p) turns pair j of the first 2*npair elements by the angle p * freqs[j];
// pairs are (j, j + npair) or, interleaved, (2j, 2j + 1).  Backwards, with
// v = R(p)^T dy:   dw = sum v * n,   dx = rstd * (w * v - n * mean(w * v * n)).
//
// Decomposition.  A lane owns eight elements of a head vector: four whole
// pairs, or eight elements that are not turned; so the rotation needs no
// exchange and the sums over the head are lane-group sums by DPP.  LH lanes
// make a head, a wave holds 64 / LH heads of one token (of several tokens
// where a token has fewer) and walks over the rest of the token's heads, so
// the angles are formed once per token and lane, exact to fp32 at any position
// (see turn_fraction).  Bound by HBM: x in, y out (backward: x and dy in, dx out).
#include <float.h>

#include "ssd_device.h"
#include "ssd_seq.h"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kFold = 64; // items of a wave summed in registers, backward

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// A lane's eight elements of a head vector as they lie in memory: four at lo
// and four at hi.  VEC: two accesses of four elements, otherwise eight.
template <typename T, bool VEC> struct Raw {
  static constexpr int W = sizeof(T) == 2 ? (VEC ? 4 : 8) : 8;
  uint32_t d[W];
  // ONCE: the row is marked as not read again
  template <bool ONCE = false> __device__ __forceinline__ void load(const T *lo, const T *hi) {
    if constexpr (!VEC) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(T) == 2) {
          d[e] = (uint32_t) reinterpret_cast<const uint16_t *>(lo)[e] << 16;
          d[4 + e] = (uint32_t) reinterpret_cast<const uint16_t *>(hi)[e] << 16;
        } else {
          d[e] = __builtin_bit_cast(uint32_t, lo[e]), d[4 + e] = __builtin_bit_cast(uint32_t, hi[e]);
        }
      }
    } else if constexpr (sizeof(T) == 2) {
      const u32x2 *pa = reinterpret_cast<const u32x2 *>(lo), *pb = reinterpret_cast<const u32x2 *>(hi);
      u32x2 a, b;
      if constexpr (ONCE) a = __builtin_nontemporal_load(pa), b = __builtin_nontemporal_load(pb);
      else a = *pa, b = *pb;
      d[0] = a.x, d[1] = a.y, d[2] = b.x, d[3] = b.y;
    } else {
      const u32x4 *pa = reinterpret_cast<const u32x4 *>(lo), *pb = reinterpret_cast<const u32x4 *>(hi);
      u32x4 a, b;
      if constexpr (ONCE) a = __builtin_nontemporal_load(pa), b = __builtin_nontemporal_load(pb);
      else a = *pa, b = *pb;
      d[0] = a.x, d[1] = a.y, d[2] = a.z, d[3] = a.w, d[4] = b.x, d[5] = b.y, d[6] = b.z, d[7] = b.w;
    }
  }
  // element k of the eight
  __device__ __forceinline__ float at(int k) const {
    if constexpr (W == 8) return __builtin_bit_cast(float, d[k]);
    else return __builtin_bit_cast(float, (k & 1) ? (d[k >> 1] & 0xFFFF0000u) : (d[k >> 1] << 16));
  }
  // as four pairs: v[e] turns with v[4 + e]
  template <bool INTER> __device__ __forceinline__ void pairs(float *v) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = at(INTER ? 2 * e : e), v[4 + e] = at(INTER ? 2 * e + 1 : 4 + e);
  }
};
template <typename T, bool VEC, bool INTER> __device__ __forceinline__ void store8(T *lo, T *hi, const float *v) {
  float o[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) o[INTER ? 2 * e : e] = v[e], o[INTER ? 2 * e + 1 : 4 + e] = v[4 + e];
  if constexpr (VEC) {
    st4<T>(lo, o[0], o[1], o[2], o[3]);
    st4<T>(hi, o[4], o[5], o[6], o[7]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) lo[e] = (T)o[e], hi[e] = (T)o[4 + e];
  }
}

// Adds a lane's eight sums, in pair order, to its place in LDS.
template <bool INTER> __device__ __forceinline__ void add8(float *lo, float *hi, const float *v) {
  float o[8];
  Raw<float, true> r;
  r.load(lo, hi);
  r.template pairs<INTER>(o);
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] += v[e];
  store8<float, true, INTER>(lo, hi, o);
}

// Sum over aligned groups of LH lanes; every lane gets it.
template <int LH> __device__ __forceinline__ float head_sum(float v) {
  if constexpr (LH == 2) return dpp_add<0xB1>(v);
  else if constexpr (LH <= 16) return lane_group_sum<LH>(v);
  else {
    v = lane_group_sum<16>(v);
    return v + __shfl_xor(v, 16);
  }
}

// 1 / sqrt(mean(x^2) + eps) from the lane's eight elements x and the head's sum
// of squares ss.  SMALL (an eps below kSmallEps, where a mean square may leave
// fp32's range): a head whose mean square does is summed again with x scaled by
// a power of two.
constexpr float kSmallEps = 0x1p-100f;
template <int LH, bool SMALL>
__device__ __forceinline__ float rstd_of(const float *x, float ss, float invn, float eps) {
  const float ms = fmaf(ss, invn, eps);
  float r = __builtin_amdgcn_rsqf(ms);
  if constexpr (SMALL) {
    const bool low = ms < kSmallEps, high = ms > FLT_MAX;
    if (__builtin_amdgcn_ballot_w64(low || high) != 0) {
      const float c = low ? 0x1p80f : high ? 0x1p-80f : 1.f;
      float d = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) d = fmaf(x[e] * c, x[e] * c, d);
      d = head_sum<LH>(d);
      r = __builtin_amdgcn_rsqf(fmaf(d, invn, eps * c * c)) * c;
    }
  }
  return r;
}

// A lane's place in a head: its eight elements are [lo, lo + 4) and
// [hi, hi + 4); `turns` says that they are four pairs, pair0 the first one.
struct Slot {
  int lo, hi, pair0;
  bool in, turns;
};
template <bool INTER> __device__ __forceinline__ Slot lane_slot(const NormRotParams &p, int l) {
  Slot s;
  s.in = 8 * l < p.N;
  s.turns = 4 * l < p.npair;
  s.pair0 = 4 * l;
  const bool apart = s.turns && !INTER;
  s.lo = apart ? 4 * l : 8 * l;
  s.hi = apart ? p.npair + 4 * l : 8 * l + 4;
  return s;
}

// The fraction of a turn, in [-1/2, 1/2], of pos * freq / 2 pi, with freq / 2 pi
// in twice 64 bits (c and the rest of it): whole turns drop out of the product
// without a rounding (fma).  c alone is off by about 2^-53 of itself, so by that
// share of the turns: nothing to fp32 at 2^24 turns, a sixth of a turn at position
// 2^53 with a freq of 1.  The rest costs nothing at large sizes, up to 3 % of small
// fp32 calls (b3 L1001 7 + 1 heads N80 7.7 -> 7.9 us), and counting it from 2^24
// turns on only the same.
__device__ __forceinline__ float turn_fraction(double pos, double freq) {
  constexpr double kTurn = 0x1.45f306dc9c883p-3, kTurnLow = -0x1.6b01ec5417056p-57; // 1 / 2 pi and the rest of it
  const double c = freq * kTurn, rest = fma(freq, kTurn, -c) + freq * kTurnLow;
  const double r = fma(pos, rest, fma(pos, c, -rint(pos * c)));
  return (float)(r - rint(r));
}

// cos and sin of the lane's four angles at a position (1 and 0 where it does
// not turn).
struct Turn {
  float c[4], s[4];
};
__device__ __forceinline__ Turn angles(const NormRotParams &p, const Slot &sl, int64_t tok, int t) {
  Turn a;
#pragma unroll
  for (int e = 0; e < 4; ++e) a.c[e] = 1.f, a.s[e] = 0.f;
  if (!sl.turns) return a;
  const double pos = p.pos32 ? (double)p.pos32[tok] : p.pos64 ? (double)p.pos64[tok] : (double)t;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float frac = turn_fraction(pos, (double)p.freqs[sl.pair0 + e]);
    sincospif(2.f * frac, &a.s[e], &a.c[e]);
  }
  return a;
}

// The lane's weights, in pair order.
template <bool VEC, bool INTER> __device__ __forceinline__ void load_weight(const float *w, const Slot &sl, float *v) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 1.f;
  if (!w || !sl.in) return;
  Raw<float, VEC> r;
  r.load(w + sl.lo, w + sl.hi);
  r.template pairs<INTER>(v);
}

// A wave's item: TPW tokens (a power of two, 64 / LH / HG) and a slice of
// their heads, taken HG at a time.
struct Item {
  int64_t tok;
  int t, row, head, hend;
  bool live;
};
template <int LH> __device__ __forceinline__ Item item_of(const NormRotParams &p, uint32_t item) {
  constexpr int HPW = 64 / LH;
  const int g = (threadIdx.x & 63) / LH;
  const int tpw = HPW >> p.hg_log;
  Item it;
  const uint32_t group = item / (uint32_t)p.split;
  const int slice = (int)(item - group * (uint32_t)p.split);
  const uint32_t tok = group * (uint32_t)tpw + (uint32_t)(g >> p.hg_log);
  it.tok = tok;
  it.live = it.tok < p.ntok;
  it.row = (int)(tok / (uint32_t)p.L);
  it.t = (int)(tok - (uint32_t)it.row * (uint32_t)p.L);
  it.head = slice * p.per + (g & ((1 << p.hg_log) - 1));
  it.hend = min(p.Hq + p.Hk, (slice + 1) * p.per);
  return it;
}

// The lane group's walk over its heads: queries first, then keys.  Where a
// head lies is formed at the first one of either kind and advanced from there.
// TD: the type of the outputs' gradients.
template <typename T, bool BACK, typename TD = T> struct Walk {
  const T *src;
  const TD *dy;
  T *dst;
  int h;
  bool isq;
  __device__ __forceinline__ void at(const NormRotParams &p, const Item &it, const Slot &sl) {
    isq = h < p.Hq;
    const int hk = h - p.Hq;
    src = isq ? (const T *)p.q + it.row * p.qb + it.t * p.qt + h * p.qh
              : (const T *)p.k + it.row * p.kb + it.t * p.kt + hk * p.kh;
    if constexpr (BACK)
      dy = isq ? (const TD *)p.dyq + it.row * p.dqb + it.t * p.dqt + h * p.dqh
               : (const TD *)p.dyk + it.row * p.dkb + it.t * p.dkt + hk * p.dkh;
    dst = isq ? (T *)p.oq + (it.tok * p.Hq + h) * p.N : (T *)p.ok + (it.tok * p.Hk + hk) * p.N;
    src += sl.lo, dst += sl.lo;
    if constexpr (BACK) dy += sl.lo;
  }
  __device__ __forceinline__ void next(const NormRotParams &p, const Item &it, const Slot &sl, int step) {
    h += step;
    if (isq && h >= p.Hq) {
      at(p, it, sl);
    } else {
      src += step * (isq ? p.qh : p.kh);
      if constexpr (BACK) dy += step * (isq ? p.dqh : p.dkh);
      dst += step * p.N;
    }
  }
};

// Forward.  The weights are multiplied into the turn's coefficients once per
// token and kind of head: y_i = n_i (w_i c) - n_j (w_j s), y_j = n_i (w_i s) +
// n_j (w_j c).  The next head is loaded while one is worked on.
// b4 L4096 32 + 8 heads N128 bf16: a call 59 us, the kernel alone 56 (6.0 TB/s,
// outputs left in the last-level cache); addresses, weights and pair order chosen
// anew for every head kept the vector ALU busy for 73.
template <typename T, int LH, bool VEC, bool INTER, bool ONCE, bool SMALL>
__global__ __launch_bounds__(kThreads) void norm_rotate_fwd_kernel(NormRotParams p) {
  const int lane = threadIdx.x & 63;
  const Item it = item_of<LH>(p, __builtin_amdgcn_readfirstlane(blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6)));
  if (!it.live || it.head >= it.hend) return;
  const Slot sl = lane_slot<INTER>(p, lane % LH);
  const int step = 1 << p.hg_log, gap = sl.hi - sl.lo;
  const float invn = 1.f / (float)p.N;
  Walk<T, false> cur;
  cur.h = it.head;
  cur.at(p, it, sl);
  Raw<T, VEC> r{};
  if (sl.in) r.template load<ONCE>(cur.src, cur.src + gap);
  const Turn an = angles(p, sl, it.tok, it.t);
  float ci[4], cj[4], si[4], sj[4];
  bool fresh = true;
  for (;;) {
    if (fresh) {
      float w[8];
      load_weight<VEC, INTER>(cur.isq ? p.qw : p.kw, sl, w);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ci[e] = an.c[e] * w[e], si[e] = an.s[e] * w[e];
        cj[e] = an.c[e] * w[4 + e], sj[e] = an.s[e] * w[4 + e];
      }
    }
    Walk<T, false> nxt = cur;
    nxt.next(p, it, sl, step);
    fresh = nxt.isq != cur.isq;
    const bool more = nxt.h < it.hend;
    Raw<T, VEC> rn{};
    if (more && sl.in) rn.template load<ONCE>(nxt.src, nxt.src + gap);
    float x[8];
    r.template pairs<INTER>(x);
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
    ss = head_sum<LH>(ss);
    const float rstd = rstd_of<LH, SMALL>(x, ss, invn, p.eps);
    float y[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float u = x[e] * rstd, v = x[4 + e] * rstd;
      y[e] = fmaf(u, ci[e], -(v * sj[e]));
      y[4 + e] = fmaf(u, si[e], v * cj[e]);
    }
    if (sl.in) store8<T, VEC, INTER>(cur.dst, cur.dst + gap, y);
    if (!more) break;
    cur = nxt;
    r = rn;
  }
}

// Backward, persistent: the waves stride over the items, each lane keeps its
// share of the weights' gradients in registers, and adds it to its place in LDS
// every kFold items (so that no sum grows by one small term after another
// however many tokens there are); one partial row per workgroup.
// Four waves a SIMD hide the loads: b4 L2048 32 + 8 heads N128 bf16 47 us (5.4
// TB/s); three and the next head loaded ahead, as in the forward, 64 us.  128
// registers do not hold every variant: the fp32 ones with pairs in halves keep six
// to eight in scratch, those moved element by element two to five, some others two
// or three.  TD is the type of the outputs' gradients: fp32 with bf16 inputs is
// what ssd_scan_bwd writes (the same case 67 us, with casts to bf16 before 92).
template <typename T, typename TD, int LH, bool VEC, bool INTER, bool SMALL>
__global__ __launch_bounds__(kThreads, 4) void norm_rotate_bwd_kernel(NormRotParams p) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Slot sl = lane_slot<INTER>(p, lane % LH);
  const int step = 1 << p.hg_log, gap = sl.hi - sl.lo;
  const float invn = 1.f / (float)p.N;
  __shared__ __align__(16) float part[kThreads / LH][2][8 * LH];
  float *const mine = part[threadIdx.x / LH][0];
  uint32_t item = blockIdx.x * (kThreads / 64) + wave;
  bool folded = false;
  do {
    float aq[8], ak[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) aq[e] = ak[e] = 0.f;
    for (int k = 0; k < kFold && item < (uint32_t)p.nitem; ++k, item += gridDim.x * (kThreads / 64)) {
      const Item it = item_of<LH>(p, item);
      if (!it.live || it.head >= it.hend) continue;
      Walk<T, true, TD> cur;
      cur.h = it.head;
      cur.at(p, it, sl);
      Raw<T, VEC> rx{};
      Raw<TD, VEC> rv{};
      if (sl.in) rx.load(cur.src, cur.src + gap), rv.load(cur.dy, cur.dy + gap);
      const Turn an = angles(p, sl, it.tok, it.t);
      float w[8], acc[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = 0.f;
      bool fresh = true;
      for (;;) {
        if (fresh) load_weight<VEC, INTER>(cur.isq ? p.qw : p.kw, sl, w);
        Walk<T, true, TD> nxt = cur;
        nxt.next(p, it, sl, step);
        fresh = nxt.isq != cur.isq;
        const bool more = nxt.h < it.hend;
        float x[8], dy[8], v[8], wv[8];
        rx.template pairs<INTER>(x);
        rv.template pairs<INTER>(dy);
        float ss = 0.f, sv = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = fmaf(dy[e], an.c[e], dy[4 + e] * an.s[e]);
          v[4 + e] = fmaf(dy[4 + e], an.c[e], -(dy[e] * an.s[e]));
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          wv[e] = v[e] * w[e];
          ss = fmaf(x[e], x[e], ss);
          sv = fmaf(wv[e], x[e], sv);
        }
        ss = head_sum<LH>(ss);
        sv = head_sum<LH>(sv);
        const float rstd = rstd_of<LH, SMALL>(x, ss, invn, p.eps);
        const float m = sv * rstd * invn; // mean(w v n)
        float d[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float n = x[e] * rstd;
          d[e] = rstd * fmaf(-n, m, wv[e]);
          acc[e] = fmaf(v[e], n, acc[e]);
        }
        if (sl.in) store8<T, VEC, INTER>(cur.dst, cur.dst + gap, d);
        if (fresh || !more) {
          // the sums of one kind of head
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            aq[e] += cur.isq ? acc[e] : 0.f;
            ak[e] += cur.isq ? 0.f : acc[e];
            acc[e] = 0.f;
          }
        }
        if (!more) break;
        cur = nxt;
        if (sl.in) rx.load(cur.src, cur.src + gap), rv.load(cur.dy, cur.dy + gap);
      }
    }
    if (sl.in) {
      if (folded) {
        add8<INTER>(mine + sl.lo, mine + sl.hi, aq);
        add8<INTER>(mine + 8 * LH + sl.lo, mine + 8 * LH + sl.hi, ak);
      } else {
        store8<float, true, INTER>(mine + sl.lo, mine + sl.hi, aq);
        store8<float, true, INTER>(mine + 8 * LH + sl.lo, mine + 8 * LH + sl.hi, ak);
      }
    }
    folded = true;
  } while (item < (uint32_t)p.nitem);
  if (!p.part) return;
  __syncthreads();
  // lane groups of the workgroup in a fixed order
  for (int c = threadIdx.x; c < 2 * p.N; c += kThreads) {
    const int which = c >= p.N, el = c - which * p.N;
    float s = 0.f;
    for (int k = 0; k < kThreads / LH; ++k) s += part[k][which][el];
    p.part[(int64_t)blockIdx.x * 2 * p.N + c] = s;
  }
}

// Sum of n partial rows [2][N] in a fixed order, in 64 bits: 16 columns by 64
// row shares per workgroup.
__global__ __launch_bounds__(1024) void norm_rotate_sum_kernel(const float *part, int n, int N, float *dqw, float *dkw) {
  __shared__ double acc[64][17];
  const int col = threadIdx.x & 15, row = threadIdx.x >> 4;
  const int c = (int)blockIdx.x * 16 + col; // 2N is a multiple of 16
  double s = 0.;
#pragma unroll 16
  for (int k = row; k < n; k += 64) s += part[(int64_t)k * 2 * N + c];
  acc[row][col] = s;
  __syncthreads();
  if (row == 0) {
#pragma unroll 8
    for (int k = 1; k < 64; ++k) s += acc[k][col];
    float *o = c < N ? dqw : dkw;
    if (o) o[c < N ? c : c - N] = (float)s;
  }
}

// A forward whose input takes half of the 256 MB last-level cache reads it past
// the caches, which leaves them to the outputs (b4 L4096 32 + 8 heads N128 bf16,
// 168 MB: 67.5 -> 59 us); a smaller one leaves its input there for the backward
// (b4 L2048 of the same, 84 MB, forward and backward: 85 us, past the caches 92).
constexpr int64_t kOnceBytes = (int64_t)128 << 20;

template <typename T, typename TD, int LH, bool VEC, bool INTER>
void launch_back(const NormRotParams &p, uint32_t nwg, hipStream_t st) {
  if (p.eps < kSmallEps) norm_rotate_bwd_kernel<T, TD, LH, VEC, INTER, true><<<nwg, kThreads, 0, st>>>(p);
  else norm_rotate_bwd_kernel<T, TD, LH, VEC, INTER, false><<<nwg, kThreads, 0, st>>>(p);
}
// A small eps takes kernels of its own: the branch of rstd_of in the forward's
// walk costs 5 % there (b4 L4096 32 + 8 heads N128 bf16 58.5 -> 61.7 us).
template <typename T, int LH, bool VEC, bool INTER>
void launch_pair(bool back, const NormRotParams &p, hipStream_t st) {
  const uint32_t grid = (uint32_t)((p.nitem + 3) / 4), nwg = (uint32_t)p.nwg;
  const bool once = VEC && p.ntok * (p.Hq + p.Hk) * p.N * (int64_t)sizeof(T) >= kOnceBytes;
  if (back) {
    if (p.dy_f32) launch_back<T, float, LH, VEC, INTER>(p, nwg, st);
    else launch_back<T, T, LH, VEC, INTER>(p, nwg, st);
  } else if (p.eps < kSmallEps) {
    norm_rotate_fwd_kernel<T, LH, VEC, INTER, false, true><<<grid, kThreads, 0, st>>>(p);
  } else {
    if (once) norm_rotate_fwd_kernel<T, LH, VEC, INTER, VEC, false><<<grid, kThreads, 0, st>>>(p);
    else norm_rotate_fwd_kernel<T, LH, VEC, INTER, false, false><<<grid, kThreads, 0, st>>>(p);
  }
}
template <typename T, int LH, bool VEC> hipError_t launch_one(bool back, const NormRotParams &p, hipStream_t st) {
  if (p.interleaved) launch_pair<T, LH, VEC, true>(back, p, st);
  else launch_pair<T, LH, VEC, false>(back, p, st);
  return hipGetLastError();
}
template <typename T, bool VEC> hipError_t launch_lh(bool back, const NormRotParams &p, hipStream_t st) {
  if (p.N <= 16) return launch_one<T, 2, VEC>(back, p, st);
  if (p.N <= 32) return launch_one<T, 4, VEC>(back, p, st);
  if (p.N <= 64) return launch_one<T, 8, VEC>(back, p, st);
  if (p.N <= 128) return launch_one<T, 16, VEC>(back, p, st);
  return launch_one<T, 32, VEC>(back, p, st);
}

} // namespace

// Splits the tokens' heads into items.  Fewer than kEnough waves leave compute
// units idle (a decode step): the heads of a token are then spread over
// several waves, each forming the angles again (b32 L1 32 + 8 heads N128 bf16
// forward in a graph: 3.1 us, one wave a token 6.6; b1 L1000 7.2 against 8.0;
// from L2000 on the two are the same).
void norm_rotate_plan(NormRotParams *p) {
  constexpr int64_t kEnough = 4096;
  int lh = 2;
  while (8 * lh < p->N) lh *= 2;
  const int hpw = 64 / lh, H = p->Hq + p->Hk;
  p->hg_log = 0;
  while ((1 << p->hg_log) < hpw && (1 << p->hg_log) < H) ++p->hg_log;
  const int hg = 1 << p->hg_log, tpw = hpw / hg;
  const int64_t groups = (p->ntok + tpw - 1) / tpw;
  const int rounds = (H + hg - 1) / hg; // of hg heads each
  const int64_t want = (kEnough + groups - 1) / groups;
  const int split0 = (int)(want < rounds ? want : rounds);
  const int per = (rounds + split0 - 1) / split0;
  p->per = per * hg;
  p->split = (rounds + per - 1) / per;
  p->nitem = groups * p->split;
  const int64_t wgs = (p->nitem + 3) / 4;
  p->nwg = (int)(wgs < kNormRotGroups ? wgs : kNormRotGroups);
}

hipError_t launch_norm_rotate(int dtype, bool vec, bool back, const NormRotParams &p, hipStream_t st) {
  hipError_t e;
  if (dtype == 1) e = vec ? launch_lh<__bf16, true>(back, p, st) : launch_lh<__bf16, false>(back, p, st);
  else e = vec ? launch_lh<float, true>(back, p, st) : launch_lh<float, false>(back, p, st);
  if (!back || e != hipSuccess || !p.part) return e;
  norm_rotate_sum_kernel<<<(uint32_t)(2 * p.N / 16), 1024, 0, st>>>(p.part, p.nwg, p.N, p.dqw, p.dkw);
  return hipGetLastError();
}

} // namespace ssd
