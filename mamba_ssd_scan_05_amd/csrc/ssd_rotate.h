// ssd_rotate.h -- head vectors as a lane of the norm with rotation and of the
// cache's append holds them: eight elements, four whole pairs of the position
// rotation, and the angles of a position.
#pragma once

#include "ssd_device.h"

namespace ssd {
namespace {

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

// A lane's place in a head: its eight elements are [lo, lo + 4) and
// [hi, hi + 4); `turns` says that they are four pairs, pair0 the first one.
struct Slot {
  int lo, hi, pair0;
  bool in, turns;
};
template <bool INTER> __device__ __forceinline__ Slot lane_slot(int N, int npair, int l) {
  Slot s;
  s.in = 8 * l < N;
  s.turns = 4 * l < npair;
  s.pair0 = 4 * l;
  const bool apart = s.turns && !INTER;
  s.lo = apart ? 4 * l : 8 * l;
  s.hi = apart ? npair + 4 * l : 8 * l + 4;
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
__device__ __forceinline__ Turn no_turn() {
  Turn a;
#pragma unroll
  for (int e = 0; e < 4; ++e) a.c[e] = 1.f, a.s[e] = 0.f;
  return a;
}
__device__ __forceinline__ Turn turn_at(const float *freqs, const Slot &sl, double pos) {
  Turn a;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float frac = turn_fraction(pos, (double)freqs[sl.pair0 + e]);
    sincospif(2.f * frac, &a.s[e], &a.c[e]);
  }
  return a;
}

} // namespace
} // namespace ssd
