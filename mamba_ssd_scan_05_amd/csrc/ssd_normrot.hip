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
// the angles are formed once per token and lane.  An angle is p * freq / 2 pi
// in 64 bits, reduced to a fraction of a turn there: exact to fp32 at any
// position.  Bound by HBM: x in, y out (backward: x and dy in, dx out).
#include "ssd_device.h"
#include "ssd_internal.h"

namespace ssd {
namespace {

constexpr int kThreads = 256;

// Four elements at element offset `o` from p.
template <typename T, bool VEC> __device__ __forceinline__ void load4(const T *p, float *v) {
  if constexpr (!VEC) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = to_f(p[e]);
  } else if constexpr (sizeof(T) == 2) {
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    v[0] = __builtin_bit_cast(float, w.x << 16), v[1] = __builtin_bit_cast(float, w.x & 0xFFFF0000u);
    v[2] = __builtin_bit_cast(float, w.y << 16), v[3] = __builtin_bit_cast(float, w.y & 0xFFFF0000u);
  } else {
    const float4 w = *reinterpret_cast<const float4 *>(p);
    v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
  }
}
template <typename T, bool VEC> __device__ __forceinline__ void store4(T *p, const float *v) {
  if constexpr (VEC) {
    st4<T>(p, v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = (T)v[e];
  }
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

// A lane's place in a head: its eight elements are [lo, lo + 4) and
// [hi, hi + 4); `turns` says that they are four pairs, pair0 the first one.
struct Slot {
  int lo, hi, pair0;
  bool in, turns;
};
__device__ __forceinline__ Slot lane_slot(const NormRotParams &p, int l) {
  Slot s;
  s.in = 8 * l < p.N;
  s.turns = 4 * l < p.npair;
  s.pair0 = 4 * l;
  const bool apart = s.turns && !p.interleaved;
  s.lo = apart ? 4 * l : 8 * l;
  s.hi = apart ? p.npair + 4 * l : 8 * l + 4;
  return s;
}

// cos and sin of the lane's four angles at a position.
struct Turn {
  float c[4], s[4];
};
__device__ __forceinline__ Turn angles(const NormRotParams &p, const Slot &sl, int64_t tok, int t) {
  Turn a;
  double pos;
  if (p.pos32) pos = (double)p.pos32[tok];
  else if (p.pos64) pos = (double)p.pos64[tok];
  else pos = (double)t;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const double f = sl.turns ? (double)p.freqs[sl.pair0 + e] : 0.0;
    const double turns = pos * (f * 0.15915494309189533577);
    const float frac = (float)(turns - rint(turns));
    sincospif(2.f * frac, &a.s[e], &a.c[e]);
  }
  return a;
}

// y = R x on the lane's elements (back: R^T x).
__device__ __forceinline__ void turn8(float *v, const Turn &a, const Slot &sl, bool interleaved, bool back) {
  if (!sl.turns) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int i = interleaved ? 2 * e : e, j = interleaved ? 2 * e + 1 : e + 4;
    const float s = back ? -a.s[e] : a.s[e], u = v[i], w = v[j];
    v[i] = fmaf(u, a.c[e], -(w * s));
    v[j] = fmaf(u, s, w * a.c[e]);
  }
}

// A wave's item: TPW tokens (a power of two, 64 / LH / HG) and a slice of
// their heads, taken HG at a time.
struct Item {
  int64_t tok;
  int t, row, head, hend;
  bool live;
};
template <int LH> __device__ __forceinline__ Item item_of(const NormRotParams &p, int64_t item) {
  constexpr int HPW = 64 / LH;
  const int g = (threadIdx.x & 63) / LH;
  const int tpw = HPW >> p.hg_log;
  Item it;
  const int64_t group = item / p.split;
  const int slice = (int)(item - group * p.split);
  it.tok = group * tpw + (g >> p.hg_log);
  it.live = it.tok < p.ntok;
  it.row = (int)(it.tok / p.L);
  it.t = (int)(it.tok - (int64_t)it.row * p.L);
  it.head = slice * p.per + (g & ((1 << p.hg_log) - 1));
  it.hend = min(p.Hq + p.Hk, (slice + 1) * p.per);
  return it;
}

template <typename T, int LH, bool VEC>
__global__ __launch_bounds__(kThreads) void norm_rotate_fwd_kernel(NormRotParams p) {
  constexpr int U = 2; // rows in flight per lane group
  const int lane = threadIdx.x & 63;
  const Item it = item_of<LH>(p, (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6));
  if (!it.live) return;
  const Slot sl = lane_slot(p, lane % LH);
  const int step = 1 << p.hg_log;
  const float invn = 1.f / (float)p.N;
  Turn an;
  if (p.npair) an = angles(p, sl, it.tok, it.t);
  for (int h0 = it.head; h0 < it.hend; h0 += U * step) {
    float x[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * step;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[u][e] = 0.f;
      if (h < it.hend && sl.in) {
        const T *src = h < p.Hq ? (const T *)p.q + it.row * p.qb + it.t * p.qt + h * p.qh
                                : (const T *)p.k + it.row * p.kb + it.t * p.kt + (h - p.Hq) * p.kh;
        load4<T, VEC>(src + sl.lo, x[u]);
        load4<T, VEC>(src + sl.hi, x[u] + 4);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * step;
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[u][e], x[u][e], ss);
      ss = head_sum<LH>(ss);
      if (h >= it.hend || !sl.in) continue;
      const float rstd = __builtin_amdgcn_rsqf(fmaf(ss, invn, p.eps));
      const bool isq = h < p.Hq;
      const float *w = isq ? p.qw : p.kw;
      float y[8], wv[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) wv[e] = 1.f;
      if (w) load4<float, VEC>(w + sl.lo, wv), load4<float, VEC>(w + sl.hi, wv + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = x[u][e] * rstd * wv[e];
      turn8(y, an, sl, p.interleaved, false);
      T *dst = isq ? (T *)p.oq + (it.tok * p.Hq + h) * p.N : (T *)p.ok + (it.tok * p.Hk + (h - p.Hq)) * p.N;
      store4<T, VEC>(dst + sl.lo, y);
      store4<T, VEC>(dst + sl.hi, y + 4);
    }
  }
}

// Persistent: the waves stride over the items, each lane keeps its share of
// the weights' gradients in registers; one partial row per workgroup.
template <typename T, int LH, bool VEC>
__global__ __launch_bounds__(kThreads) void norm_rotate_bwd_kernel(NormRotParams p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Slot sl = lane_slot(p, lane % LH);
  const int step = 1 << p.hg_log;
  const float invn = 1.f / (float)p.N;
  float aq[8], ak[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) aq[e] = ak[e] = 0.f;
  for (int64_t item = (int64_t)blockIdx.x * (kThreads / 64) + wave; item < p.nitem;
       item += (int64_t)gridDim.x * (kThreads / 64)) {
    const Item it = item_of<LH>(p, item);
    if (!it.live) continue;
    Turn an;
    if (p.npair) an = angles(p, sl, it.tok, it.t);
    for (int h = it.head; h < it.hend; h += step) {
      const bool isq = h < p.Hq;
      const int hk = h - p.Hq;
      float x[8], v[8], wv[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = v[e] = 0.f, wv[e] = 1.f;
      if (sl.in) {
        const T *src = isq ? (const T *)p.q + it.row * p.qb + it.t * p.qt + h * p.qh
                           : (const T *)p.k + it.row * p.kb + it.t * p.kt + hk * p.kh;
        const T *dsrc = isq ? (const T *)p.dyq + it.row * p.dqb + it.t * p.dqt + h * p.dqh
                            : (const T *)p.dyk + it.row * p.dkb + it.t * p.dkt + hk * p.dkh;
        load4<T, VEC>(src + sl.lo, x);
        load4<T, VEC>(src + sl.hi, x + 4);
        load4<T, VEC>(dsrc + sl.lo, v);
        load4<T, VEC>(dsrc + sl.hi, v + 4);
        const float *w = isq ? p.qw : p.kw;
        if (w) load4<float, VEC>(w + sl.lo, wv), load4<float, VEC>(w + sl.hi, wv + 4);
      }
      turn8(v, an, sl, p.interleaved, true);
      float ss = 0.f, sv = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss = fmaf(x[e], x[e], ss);
        sv = fmaf(v[e] * wv[e], x[e], sv);
      }
      ss = head_sum<LH>(ss);
      sv = head_sum<LH>(sv);
      const float rstd = __builtin_amdgcn_rsqf(fmaf(ss, invn, p.eps));
      const float m = sv * rstd * invn; // mean(w v n)
      float d[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = x[e] * rstd;
        d[e] = rstd * fmaf(-n, m, wv[e] * v[e]);
        const float g = v[e] * n;
        aq[e] += isq ? g : 0.f;
        ak[e] += isq ? 0.f : g;
      }
      if (sl.in) {
        T *dst = isq ? (T *)p.oq + (it.tok * p.Hq + h) * p.N : (T *)p.ok + (it.tok * p.Hk + hk) * p.N;
        store4<T, VEC>(dst + sl.lo, d);
        store4<T, VEC>(dst + sl.hi, d + 4);
      }
    }
  }
  // lane groups of the workgroup in a fixed order
  __shared__ float part[kThreads / LH][2][8 * LH];
  const int g = threadIdx.x / LH;
  if (sl.in) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      part[g][0][sl.lo + e] = aq[e], part[g][0][sl.hi + e] = aq[e + 4];
      part[g][1][sl.lo + e] = ak[e], part[g][1][sl.hi + e] = ak[e + 4];
    }
  }
  __syncthreads();
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

template <typename T, int LH, bool VEC> hipError_t launch_one(bool back, const NormRotParams &p, hipStream_t st) {
  if (back) norm_rotate_bwd_kernel<T, LH, VEC><<<(uint32_t)p.nwg, kThreads, 0, st>>>(p);
  else norm_rotate_fwd_kernel<T, LH, VEC><<<(uint32_t)((p.nitem + 3) / 4), kThreads, 0, st>>>(p);
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
// several waves, each forming the angles again.
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
  if (!back || e != hipSuccess || (!p.dqw && !p.dkw)) return e;
  norm_rotate_sum_kernel<<<(uint32_t)(2 * p.N / 16), 1024, 0, st>>>(p.part, p.nwg, p.N, p.dqw, p.dkw);
  return hipGetLastError();
}

} // namespace ssd
