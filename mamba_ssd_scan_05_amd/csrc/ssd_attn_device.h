// ssd_attn_device.h -- what the attention kernels share: the rows of the batch and
// the pieces their lengths are cut into, V tiles in LDS, odd values.
#pragma once

#include "ssd_cache.h"
#include "ssd_device.h"

namespace ssd {
namespace {

__device__ __forceinline__ int wave_incl_scan_i(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
  return v;
}
// Maximum over a wave of values from 0 on.
__device__ __forceinline__ int wave_max_i(int v) {
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false));
  return __builtin_amdgcn_readlane(v, 63);
}

// What workgroup `id` does: a tile of the query vectors of a key head of a piece.  The
// tiles of a piece and head read the same keys: they go to one XCD (workgroups are dealt to
// the eight in turn) where that gives each the same number of them (bf16 prompt b4 L4096
// 1320 -> 924 us at the time, its 8 MB of keys and values a head more than an L2 holds); the
// longest ones first.
__device__ __forceinline__ void place_of(const AttnParams &p, uint32_t id, int *tile, int *hk, int *slot) {
  const bool deal = p.tiles > 1 && (uint32_t)p.slots * (uint32_t)p.Hk % 8 == 0;
  const uint32_t n = deal ? id >> 3 : id, group = n / (uint32_t)p.tiles;
  *tile = p.tiles - 1 - (int)(n - group * (uint32_t)p.tiles);
  const uint32_t g = deal ? group * 8 + (id & 7) : group;
  *slot = (int)(g / (uint32_t)p.Hk);
  *hk = (int)(g - (uint32_t)*slot * (uint32_t)p.Hk);
}

// A row of the batch: how many new tokens it has, where the first one stands and
// the keys that any of them sees, [lo, hi).
struct Row {
  int n, lo, hi, start;
  // kAttnUnit-key units from lo, rounded down to a unit, to hi; a row with tokens
  // but no keys has one, in which nothing is seen
  __device__ __forceinline__ int units() const {
    if (n == 0) return 0;
    const int u = (hi + kAttnUnit - 1) / kAttnUnit - lo / kAttnUnit;
    return max(u, 1);
  }
};
__device__ __forceinline__ Row row_of(const AttnParams &p, int i) {
  Row r;
  r.start = p.c.start[i];
  r.n = p.c.tokens ? min(max(p.c.tokens[i], 0), p.L) : p.L;
  const int64_t cap = p.c.capacity;
  const int64_t hi = min(max((int64_t)r.start + r.n, (int64_t)0), cap);
  const int64_t lo = p.window ? min(max((int64_t)r.start + 1 - p.window, (int64_t)0), hi) : 0;
  r.lo = (int)lo, r.hi = (int)hi;
  return r;
}

// A piece: the `index`th of `count` of row i.
struct Piece {
  int i, index, count, place; // place: its own in p.part, if the row has more pieces
  Row row;
  // units of each of the row's pieces
  __device__ __forceinline__ int size() const { return count == 1 ? INT32_MAX : (row.units() + count - 1) / count; }
};
// The plan, the same in every workgroup: all rows' lengths together are cut into pieces of
// about equal size, so that a batch of one long row and many short ones keeps the device as
// busy as an even one.  Units of a piece, for all rows' `total`, which stays below 2^31
// (checked on the host).  Pieces of few rounds of workgroups are halved where rows are uneven, `longest`
// more than 1.25 times their mean: b100 0 to 2000 keys 32 + 8 heads N128 108 -> 94 us, b40 0 to
// 6000 keys 16 + 2 heads N256 62 -> 52; of even rows those would slow down, b64 4000 keys
// N256 fp32 109 and 121.
__device__ __forceinline__ int piece_units(const AttnParams &p, int total, int longest) {
  const int least = (total + p.workers - 1) / p.workers, one = (total + p.prefer - 1) / p.prefer;
  const bool halve = one < 2 * p.enough && (int64_t)longest * p.b > total + (int64_t)total / 4;
  return max(max(least, min(one, halve ? (p.enough + 1) / 2 : p.enough)), 2);
}
// Pieces of a row of u units: a rest of up to a quarter of a piece is spread over the others.
__device__ __forceinline__ int pieces_of(int u, int size) {
  return u == 0 ? 0 : max((u + size - 1 - size / 4) / size, 1);
}
// Places in p.part are given to rows of more than one piece only.  Such a row has more than 1.25
// sizes of units and, its rest spread, less than 0.75 more pieces than sizes: 1.6 times
// as many places as there are sizes in all the rows are enough, whatever the batch.
__device__ __forceinline__ int places_of(int cnt) { return cnt > 1 ? cnt : 0; }

// Piece `slot`; false behind the last.  ROWS: the rows up to which a workgroup makes the plan for
// itself, 64 or as many as threads; sh: 12 words of LDS for more than 64.  Counts of pieces and of places are
// added up in one word, 16 bits each (at most 4096 + 256 and 1.6 * 4096).
template <int ROWS>
__device__ __forceinline__ bool piece_of(const AttnParams &p, int slot, int *sh, Piece *pc) {
  if (p.workers == 1) {
    *pc = Piece{slot, 0, 1, slot, row_of(p, slot)}; // slots = b
    return true;
  }
  if (p.list) {
    const int4 e = p.list[slot];
    const int i = __builtin_amdgcn_readfirstlane(e.x);
    if (i < 0) return false;
    *pc = Piece{i, __builtin_amdgcn_readfirstlane(e.y), __builtin_amdgcn_readfirstlane(e.z),
                __builtin_amdgcn_readfirstlane(e.w), row_of(p, i)};
    return true;
  }
  const int tid = threadIdx.x, lane = tid & 63;
  if (p.b <= 64) { // every wave by itself, a row a lane
    Row row{};
    if (lane < p.b) row = row_of(p, lane);
    const int u = row.units();
    const int total = __builtin_amdgcn_readlane(wave_incl_scan_i(u), 63);
    const int size = piece_units(p, total, wave_max_i(u));
    const int cnt = pieces_of(u, size), end = wave_incl_scan_i(cnt | places_of(cnt) << 16);
    const uint64_t m = __builtin_amdgcn_ballot_w64((end & 0xFFFF) > slot);
    if (m == 0) return false;
    const int i = (int)__builtin_ctzll(m);
    const int c = __builtin_amdgcn_readlane(cnt, i), e = __builtin_amdgcn_readlane(end, i);
    const int index = slot - ((e & 0xFFFF) - c);
    *pc = Piece{i, index, c, (e >> 16) - places_of(c) + index, row};
    pc->row.n = __builtin_amdgcn_readlane(row.n, i);
    pc->row.lo = __builtin_amdgcn_readlane(row.lo, i);
    pc->row.hi = __builtin_amdgcn_readlane(row.hi, i);
    pc->row.start = __builtin_amdgcn_readlane(row.start, i);
    return true;
  }
  if constexpr (ROWS <= 64) return false; // not reached, more rows have the list
  // a row a thread
  constexpr int kW = ROWS / 64;
  static_assert(ROWS % 64 == 0 && kW <= 4, "waves of a workgroup of ROWS threads");
  Row row{};
  if (tid < p.b) row = row_of(p, tid);
  const int u = row.units(), sum = wave_incl_scan_i(u);
  int longest = wave_max_i(u);
  if (lane == 63) sh[tid >> 6] = sum, sh[4 + (tid >> 6)] = longest;
  __syncthreads();
  int total = 0;
  for (int w = 0; w < kW; ++w) total += sh[w], longest = max(longest, sh[4 + w]);
  __syncthreads();
  const int size = piece_units(p, total, longest), cnt = pieces_of(u, size);
  int end = wave_incl_scan_i(cnt | places_of(cnt) << 16);
  if (lane == 63) sh[tid >> 6] = end;
  if (tid == 0) sh[8] = -1;
  __syncthreads();
  for (int w = 0; w < (tid >> 6); ++w) end += sh[w];
  const int before = (end & 0xFFFF) - cnt;
  if (slot >= before && slot < before + cnt)
    sh[8] = tid, sh[9] = before, sh[10] = cnt, sh[11] = (end >> 16) - places_of(cnt);
  __syncthreads();
  const int i = __builtin_amdgcn_readfirstlane(sh[8]), f = __builtin_amdgcn_readfirstlane(sh[9]),
            c = __builtin_amdgcn_readfirstlane(sh[10]), at = __builtin_amdgcn_readfirstlane(sh[11]);
  __syncthreads();
  if (i < 0) return false;
  *pc = Piece{i, slot - f, c, at + slot - f, row_of(p, i)};
  return true;
}

// A V tile of a wave in LDS: 16-byte pieces of its rows as they come, but the
// 16-column units of a row exchanged by its number, so that the rows a transposed
// read touches at once lie on different banks.
template <typename T, int NP> struct Swizzle {
  static constexpr int UB = 16 * sizeof(T), NU = NP / 16; // bytes of a unit, units of a row
  static constexpr int kAll = 256 / UB;                   // units of all banks: 8 (bf16), 4 (fp32)
  static constexpr int pow2(int n) { return n % 2 ? 1 : 2 * pow2(n / 2); }
  static constexpr int U2 = pow2(NU) < kAll ? pow2(NU) : kAll;
  __device__ static __forceinline__ int at(int row, int unit) { // first element of the unit
    const int x = sizeof(T) == 2 ? row / (kAll / U2) : row / 4;
    return row * NP + (unit ^ (x & (U2 - 1))) * 16;
  }
};

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ bool odd_values(u32x4 v, __bf16) { // an infinity or a NaN among them
  bool b = false;
#pragma unroll
  for (int e = 0; e < 4; ++e) b |= (v[e] & 0x7F80u) == 0x7F80u || (v[e] & 0x7F800000u) == 0x7F800000u;
  return b;
}
__device__ __forceinline__ bool odd_values(u32x4 v, float) {
  bool b = false;
#pragma unroll
  for (int e = 0; e < 4; ++e) b |= (v[e] & 0x7F800000u) == 0x7F800000u;
  return b;
}

__device__ __forceinline__ void load_frag(FragBF &f, const __bf16 *p) { f.v = *reinterpret_cast<const bf16x8 *>(p); }
__device__ __forceinline__ void load_frag(FragF32 &f, const float *p) {
  const f32x4 a = *reinterpret_cast<const f32x4 *>(p), b = *reinterpret_cast<const f32x4 *>(p + 4);
#pragma unroll
  for (int e = 0; e < 4; ++e) f.v[e] = a[e], f.v[4 + e] = b[e];
}

} // namespace
} // namespace ssd
