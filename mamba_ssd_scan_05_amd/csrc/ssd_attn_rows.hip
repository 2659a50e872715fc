// ssd_attn_rows.hip -- attention of more than 16 query vectors of a row and key head
// (prompts, pieces of them, drafted tokens) over the paged cache, bf16.  The products and
// the orientation are those of ssd_attn.hip, S^T = K Q^T and O^T = V^T P^T, with 32 x 32
// tiles: a lane holds the scores of one query (its column), 16 keys of 32 with those of the
// lane 32 further, and eight of them are the B operand of 16 keys of the second product
// as they stand.  A wave owns 32 query vectors for all keys; W waves share tiles of 64 keys
// in LDS.
//
// A pass of the loop works on a tile whose scores lie in registers: between the products of the next
// tile's scores and those of its own sums its weights are formed, so that the matrix cores
// and the vector ALU run at the same time, and the next tile's maximum is taken.  K of the
// tile after the next and V of the next are on their way to registers meanwhile.  The
// running maximum that the weights refer to moves only when one would pass 4, which mostly
// spares the sums' scaling.  (Where it always moves, the largest weight is 1 and rounds to
// itself: error against 64 bits 0.0019 of the output's norm, 656 us for the prompt below
// when this took 647 with 0.0019 to 0.0020; moved past 2^8: 0.0022, 638 us.  The output's
// rounding alone is 0.0016.)
//
// Measured, 32 + 8 heads N128 (bf16): prompt b4 L4096 636 to 666 us (826 to 865 TFLOP/s counted
// on the pairs that are seen; a large product reaches 1358), 512 tokens behind 32000 289 to 328 us
// (825 to 936) with their join, by the clock.
// Of a pass's 5000 cycles the matrix cores work 37 %, the vector ALU 44 (32 exponentials a
// lane are 512 of its 1000 cycles a wave); LDS reads have no conflicts.  Without the loads,
// stores and barrier of a pass the second case took 249 of 314 us, without exponentials
// 300.  Steps that did not pay: four waves a workgroup and two of them a compute unit (788
// against 775), one barrier for two tiles (777 against 737), reads three or four products
// ahead (648 and 654 against 650), the stores between the products (661 against 621).
// 96 registers hold O and Q and 64 two tiles' scores, so eight waves are all a compute unit
// takes.  Wide heads (N > 128): four waves with the whole register file, tiles of 32 keys;
// b4 L2048 10 + 1 heads N256 208 us, 413 TFLOP/s.
#include <type_traits>

#include "ssd_attn_device.h"

namespace ssd {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

// Keys of a tile: with 32 the wide heads' tiles and weights leave room for their sums.
constexpr int tile_keys(int NP) { return NP <= 128 ? 64 : 32; }

// 16-byte pieces of a K row, exchanged by the row's number so that eight rows
// read at once lie on different banks.
template <int NP> struct KSwizzle {
  static constexpr int pow2(int n) { return n % 2 ? 1 : 2 * pow2(n / 2); }
  // a period of 8 rows for the widest heads, of which a thread's pieces lie 8 rows apart
  static constexpr int kMost = NP == 256 ? 8 : 16;
  static constexpr int C2 = pow2(NP / 8) < kMost ? pow2(NP / 8) : kMost;
  __device__ static __forceinline__ int at(int row, int piece) {
    return row * NP + (piece ^ (row / (kMost / C2) & (C2 - 1))) * 8;
  }
};

// V rows: units of 16 columns two by two, exchanged so that the four rows and two units
// that half of a wave reads at once lie on different banks.
template <int NP> struct VSwizzle {
  static constexpr int pow2(int n) { return n % 2 ? 1 : 2 * pow2(n / 2); }
  static constexpr int P2 = pow2(NP / 32) < 4 ? pow2(NP / 32) : 4;
  __device__ static __forceinline__ int at(int row, int unit) { // first element of the unit
    return row * NP + (unit ^ 2 * (row / (4 / P2) & (P2 - 1))) * 16;
  }
};

// Bits [a, b) of 64, the ends anywhere.
__device__ __forceinline__ uint64_t bits(int a, int b) {
  const uint64_t lo = a <= 0 ? ~0ull : a >= 64 ? 0ull : ~0ull << a;
  const uint64_t hi = b >= 64 ? ~0ull : b <= 0 ? 0ull : ~(~0ull << b);
  return lo & hi;
}

// UNI: the page size is a multiple of 16; the 64 pieces a wave loads at once lie in
// 16 rows of one page then, one behind the other.
template <int NP, int W, bool UNI> __global__ __launch_bounds__(64 * W, NP <= 128 ? 2 : 1) void attn_rows_kernel(AttnParams p) {
  constexpr int kTK = tile_keys(NP), KG = kTK / 32;       // groups of 32 keys
  constexpr uint64_t kAll = kTK == 64 ? ~0ull : 0xFFFFFFFFull;
  constexpr int KS = NP / 16, DT = NP / 32;               // steps of 16 dims, tiles of 32 dims
  constexpr int PC = NP / 8, CH = (kTK * PC + 64 * W - 1) / (64 * W); // pieces of a row, of a thread
  constexpr int kRows = 32 * W;
  constexpr int AHEAD = 2; // reads from LDS ahead of their products
  using KW = KSwizzle<NP>;
  using VW = VSwizzle<NP>;
  __shared__ __align__(16) __bf16 ktile[2][kTK * NP], vtile[3][kTK * NP]; // vtile[2]: zeros

  const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int tile, hk, slot;
  place_of(p, blockIdx.x, &tile, &hk, &slot);
  Piece pc;
  if (!piece_of<64>(p, slot, nullptr, &pc)) return;
  const Row row = pc.row;
  if (p.workers > 1 && !p.list && pc.index == 0 && hk == 0 && tile == 0 && threadIdx.x == 0)
    p.pieces[pc.i] = make_int2(pc.place, pc.count);
  const int nrows = row.n * p.G, r0 = tile * kRows;
  if (r0 >= nrows) return;

  const int64_t cap = p.c.capacity;
  auto token = [&](int r) { return (int)div_by((uint32_t)r, p.group); };
  auto last_key = [&](int t) { return (int)min(max((int64_t)row.start + t + 1, (int64_t)0), cap); };
  auto first_key = [&](int t) { return p.window ? (int)min(max((int64_t)row.start + t + 1 - p.window, (int64_t)0), cap) : 0; };
  const int64_t base_key = (int64_t)(row.lo / kAttnUnit) * kAttnUnit, size = (int64_t)pc.size() * kAttnUnit;
  const int64_t piece0 = base_key + pc.index * size, piece1 = piece0 + size;
  auto from = [&](int t) { return (int)max((int64_t)first_key(t), piece0); };
  auto to = [&](int t) { return (int)min((int64_t)last_key(t), piece1); };
  // keys that any query of the workgroup, and of the wave, sees; and those that all of them see
  const int t_first = token(r0), t_last = token(min(r0 + kRows, nrows) - 1);
  const int k0 = from(t_first), k1 = to(t_last), all0 = from(t_last), all1 = to(t_first);
  const int rw = r0 + 32 * wave;
  const bool busy = rw < nrows;
  const int wt_first = token(busy ? rw : r0), wt_last = token(busy ? min(rw + 32, nrows) - 1 : r0);
  const int w0 = from(wt_first), w1 = busy ? to(wt_last) : 0, wall0 = from(wt_last), wall1 = to(wt_first);

  // this lane's query
  const int r = rw + col;
  const bool live = r < nrows;
  const int t = token(live ? r : r0), h = hk * p.G + (live ? r : r0) - t * p.G;
  const int q0 = from(t), q1 = to(t);
  bf16x8 qf[KS];
  {
    const __bf16 *src = (const __bf16 *)p.q + pc.i * p.qb + t * p.qt + h * p.qh;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const int d = 16 * k + 8 * half;
#pragma unroll
      for (int e = 0; e < 8; ++e) qf[k][e] = (__bf16)0.f;
      if (live && d < p.N) {
        if (p.qvec) {
          qf[k] = *reinterpret_cast<const bf16x8 *>(src + d);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) qf[k][e] = src[d + e];
        }
        if (p.negate) {
#pragma unroll
          for (int e = 0; e < 8; ++e) qf[k][e] = -qf[k][e];
        }
      }
    }
  }

  const __bf16 *const kc = (const __bf16 *)p.c.kc + hk * p.c.kh, *const vc = (const __bf16 *)p.c.vc + hk * p.c.vh;
  const int32_t *const table = p.c.table + pc.i * p.c.tb;
  // the thread's pieces of a tile: row and element, places in the LDS tiles, offsets in
  // bytes from the first of 16 rows
  u32x4 kr[CH], vr[CH];
  // Where pieces of one thread lie whole periods of the exchanges apart, one register holds
  // each of these for all of them.
  constexpr int RW = 64 * W / PC;
  constexpr bool kEven = 64 * W % PC == 0 && RW % KW::kMost == 0;
  constexpr int CA = kEven ? 1 : CH;
  int krow_[CA], kat_[CA], vat_[CA];
  uint32_t koff_[CA], voff_[CA];
  bool none_[CA]; // behind N: zero for K (nothing is taken there for V)
#pragma unroll
  for (int c = 0; c < CA; ++c) {
    const int x = c * 64 * W + (int)threadIdx.x, piece = x % PC;
    krow_[c] = min(x / PC, kTK - 1);
    kat_[c] = KW::at(krow_[c], piece);
    vat_[c] = VW::at(krow_[c], piece / 2) + piece % 2 * 8;
    none_[c] = 8 * piece >= p.N;
    const int d = none_[c] ? 0 : 8 * piece;
    koff_[c] = (uint32_t)(((UNI ? krow_[c] % 16 * p.c.ks : 0) + d) * 2);
    voff_[c] = (uint32_t)(((UNI ? krow_[c] % 16 * p.c.vs : 0) + d) * 2);
  }
  auto krow = [&](int c) { return kEven ? krow_[0] + c * RW : krow_[c]; };
  auto kat = [&](int c) { return kEven ? kat_[0] + c * RW * NP : kat_[c]; };
  auto vat = [&](int c) { return kEven ? vat_[0] + c * RW * NP : vat_[c]; };
  // (of rows 8 apart those of a group's second half lie further on)
  auto koff = [&](int c) { return kEven ? koff_[0] + (UNI ? (uint32_t)(c * RW % 16 * p.c.ks * 2) : 0) : koff_[c]; };
  auto voff = [&](int c) { return kEven ? voff_[0] + (UNI ? (uint32_t)(c * RW % 16 * p.c.vs * 2) : 0) : voff_[c]; };
  auto none = [&](int c) { return none_[kEven ? 0 : c]; };
  // Where the rows of a tile lie.  UNI: lane l keeps the page and the places of the l-th 16 keys
  // of a batch of 16 or 32 tiles, found once for the batch; a wave's loads read their group's
  // from its lane.  Otherwise lane l finds the page of the tile's l-th key, and each row's
  // place is formed by the lanes that load it.  Strides of pages and tokens are below 2^32.
  const int kstart = k0 & ~(kTK - 1);
  constexpr int kBatch = 64 * 16; // keys
  uint64_t gk = 0, gv = 0, gok = 0;
  int page_k = -1, entry = -1; // entry: the table's, of the batch (tile) to come
  auto entry_of = [&](int kb) {
    return table[div_by((uint32_t)min(kb + (UNI ? 16 : 1) * lane, p.c.capacity - 1), p.c.page)];
  };
  auto page_of = [&](int kb, int entry) { // of the lane's key
    return kb + lane < p.c.capacity && lane < kTK && entry < p.c.pages ? max(entry, -1) : -1;
  };
  // Before the loads of the tile at kb: its places, and which of its keys lie on a page.
  auto locate = [&](int kb) {
    if constexpr (UNI) {
      if ((kb - kstart) % kBatch == 0) {
        const uint32_t key = (uint32_t)(kb + 16 * lane), at = key - div_by(key, p.c.page) * p.c.page.d;
        const bool ok = (int)key < p.c.capacity && entry >= 0 && entry < p.c.pages;
        gk = ok ? (uint64_t)(uint32_t)entry * (uint32_t)p.c.kp + (uint64_t)at * (uint32_t)p.c.ks : 0;
        gv = ok ? (uint64_t)(uint32_t)entry * (uint32_t)p.c.vp + (uint64_t)at * (uint32_t)p.c.vs : 0;
        gok = __builtin_amdgcn_ballot_w64(ok);
        if (kb + kBatch < k1) entry = entry_of(kb + kBatch);
      }
      const uint32_t b = (uint32_t)(gok >> ((kb - kstart) / 16 % 64)) & ((1u << (kTK / 16)) - 1);
      if (b == (1u << (kTK / 16)) - 1) return kAll;
      uint64_t have = 0;
#pragma unroll
      for (int g = 0; g < kTK / 16; ++g) have |= b >> g & 1 ? 0xFFFFull << (16 * g) : 0;
      return have;
    } else {
      page_k = page_of(kb, entry);
      entry = entry_of(kb + kTK);
      return (uint64_t)__builtin_amdgcn_ballot_w64(page_k >= 0);
    }
  };
  auto row_at = [&](int kb, int c, uint64_t group, int pages, uint32_t ps, uint32_t ts) {
    if constexpr (UNI) {
      const int f = (kb - kstart) / 16 % 64 + __builtin_amdgcn_readfirstlane(krow(c)) / 16;
      return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(group >> 32), f) << 32 |
             (uint32_t)__builtin_amdgcn_readlane((int)group, f);
    } else {
      const int f = krow(c), pg = __shfl(pages, f);
      const uint32_t key = (uint32_t)(kb + f), at = pg < 0 ? 0 : key - div_by(key, p.c.page) * p.c.page.d;
      return (uint64_t)(uint32_t)max(pg, 0) * ps + (uint64_t)at * ts;
    }
  };
  auto load_k = [&](int kb) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
      kr[c] = *reinterpret_cast<const u32x4 *>(
          (const char *)(kc + row_at(kb, c, gk, page_k, (uint32_t)p.c.kp, (uint32_t)p.c.ks)) + koff(c));
  };
  auto load_v = [&](int kb, int pages) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
      vr[c] = *reinterpret_cast<const u32x4 *>(
          (const char *)(vc + row_at(kb, c, gv, pages, (uint32_t)p.c.vp, (uint32_t)p.c.vs)) + voff(c));
  };
  constexpr bool kRagged = kTK * PC % (64 * W) != 0; // some threads have no last piece
  auto store = [&](int c, __bf16 *tile, int at, u32x4 v) {
    if (!kRagged || c * 64 * W + (int)threadIdx.x < kTK * PC) *reinterpret_cast<u32x4 *>(tile + at) = v;
  };
  auto store_k = [&](int c, __bf16 *tile) { store(c, tile, kat(c), none(c) ? u32x4{0, 0, 0, 0} : kr[c]); };
  auto store_v = [&](int c, __bf16 *tile) { store(c, tile, vat(c), vr[c]); };
  // An edge tile: rows of V that no query of the workgroup sees are zero in LDS, whatever
  // they held.  True if another row holds an infinity or a NaN.
  auto clean_v = [&](__bf16 *tile, uint64_t seen) {
    bool odd = false;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (kRagged && c * 64 * W + (int)threadIdx.x >= kTK * PC) continue;
      if (seen >> krow(c) & 1) odd |= odd_values(vr[c], __bf16());
      else store(c, tile, vat(c), u32x4{0, 0, 0, 0});
    }
    return odd;
  };
  // Where the lane reads in a tile: the exchanges have a period of 16 rows (K) and 4 (V) at
  // most.  The step's place is formed at each read from the first one's: a register for
  // each would leave none for reads ahead.  Rows of a power of two: one exclusive or, for the
  // row's own place has no bits there.
  constexpr bool kPow2 = (NP & (NP - 1)) == 0;
  const int krow0 = col * NP, vrow0 = (4 * half + (lane >> 2 & 3)) * NP;
  const int kfirst = KW::at(col, half) - (kPow2 ? 0 : krow0);
  const int vfirst = VW::at(4 * half + (lane >> 2 & 3), lane >> 4 & 1) + 4 * (lane & 3) - (kPow2 ? 0 : vrow0);
  auto k_at = [&](int first, int step) { return kPow2 ? first ^ 16 * step : (first ^ 16 * step) + krow0; };
  auto v_at = [&](int first, int d) { return kPow2 ? first ^ 32 * d : (first ^ 32 * d) + vrow0; };

  f32x16 o[DT], s0[KG], s1[KG];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[d][e] = 0.f;
  float m = -INFINITY, l = 0.f, top = -INFINITY; // top: the lane's largest score of the tile
  int odd = 0, odd_ever = 0;
  auto highest_of = [&](const f32x16 *s) {
    float x = -INFINITY;
#pragma unroll
    for (int g = 0; g < KG; ++g)
#pragma unroll
      for (int e = 0; e < 16; ++e) x = fmaxf(x, s[g][e]);
    return x;
  };
  // S^T = K Q^T: the operand of product i, keys 32 (i % KG) and on, step i / KG
  auto key_frag = [&](const __bf16 *tile, int kf, int i) {
    return *reinterpret_cast<const bf16x8 *>(tile + 32 * (i % KG) * NP + k_at(kf, i / KG));
  };
  f32x16 zero;
#pragma unroll
  for (int e = 0; e < 16; ++e) zero[e] = 0.f;
  // Tile t's V and tile t + 1's K lie in LDS, tile t's scores in registers.  While t's
  // weights are formed, the scores of t + 1 run on the matrix cores.
  int kb = kstart;
  uint64_t have0 = 0, have1 = 0; // keys of this tile and of the next that lie on a page
  // behind the stores of a tile
  auto publish = [&](int tile_kb, uint64_t have, __bf16 *tile) {
    if (have == kAll && tile_kb >= all0 && tile_kb + kTK <= all1) {
      odd = 0;
      __syncthreads();
    } else {
      odd = __syncthreads_or(clean_v(tile, have & bits(k0 - tile_kb, k1 - tile_kb)));
      odd_ever |= odd;
    }
  };
  for (int x = threadIdx.x; x < kTK * PC; x += 64 * W)
    *reinterpret_cast<u32x4 *>(&vtile[2][8 * x]) = u32x4{0, 0, 0, 0};
  if (kb < k1) {
    entry = entry_of(kb);
    have0 = locate(kb);
    load_k(kb);
    load_v(kb, page_k);
    // The queries are there from here on: as loads still on their way they would be waited for
    // at the first product of every tile, and with them the loads of the tile to come.
#pragma unroll
    for (int k = 0; k < KS; ++k) __asm__ volatile("" : "+v"(qf[k]));
#pragma unroll
    for (int c = 0; c < CH; ++c) store_k(c, ktile[0]), store_v(c, vtile[0]);
    publish(kb, have0, vtile[0]);
    have1 = locate(kb + kTK);
    load_k(kb + kTK);
#pragma unroll
    for (int c = 0; c < CH; ++c) store_k(c, ktile[1]);
    if (busy) {
#pragma unroll
      for (int i = 0; i < KS * KG; ++i)
        s0[i % KG] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(key_frag(ktile[0], kfirst, i), qf[i / KG],
                                                             i < KG ? zero : s0[i % KG], 0, 0, 0);
      top = highest_of(s0);
    }
    __syncthreads(); // its place is written again
  }
  auto body = [&](auto par, f32x16 *s, f32x16 *sn) {
    constexpr int P = decltype(par)::value;
    const int next = kb + kTK, ahead = kb + 2 * kTK;
    const uint64_t here = have0;
    have0 = have1;
    if (next < k1) {
      load_v(next, page_k);
      have1 = locate(ahead);
      load_k(ahead);
    }
    if (busy) {
      const bool full = here == kAll && kb >= wall0 && next <= wall1;
      if (!full) {
        const uint64_t mine = here & bits(q0 - kb, q1 - kb);
#pragma unroll
        for (int g = 0; g < KG; ++g) {
          const uint32_t mg = (uint32_t)(mine >> (32 * g)) >> (4 * half);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (!(mg & 1u << (e % 4 + 8 * (e / 4)))) s[g][e] = -INFINITY;
        }
        top = highest_of(s);
      }
      const Both tops = swap32(top);
      const float highest = fmaxf(tops.a, tops.b) * p.scale;
      // the weights' reference moves only when some weight would pass 4
      if (__builtin_amdgcn_ballot_w64(highest > m + 2.f) != 0) {
        const float mn = fmaxf(m, highest), a = hw_exp2(m - (mn == -INFINITY ? 0.f : mn));
        l *= a;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] *= a;
        m = mn;
      }
      const float base = m == -INFINITY ? 0.f : m;
      // The order is fixed here, step by step: reads from LDS AHEAD of the product that takes
      // them, and between two products of the next tile's scores some of this tile's weights
      // (the compiler's own order reads, waits and multiplies in turn).  Then
      // O^T += V^T P^T, 16 keys at a time: eight weights of a lane against the same keys of V.
      // Behind the last tile the scores are of whatever lies there, and not used.
      const __bf16 *const vt = vtile[full || !odd ? P : 2];
      int kf = kfirst, vf = vfirst;
      __asm__ volatile("" : "+v"(kf), "+v"(vf));
      auto kfrag = [&](int i) { return key_frag(ktile[1 - P], kf, i); };
      auto vfrag = [&](int j) {
        const __bf16 *const at = vt + 16 * (j / DT) * NP + v_at(vf, j % DT);
        const auto tr = [&](int row) {
          return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
              (__attribute__((address_space(3))) lds_bf16x4 *)(at + row * NP)));
        };
        return __builtin_shufflevector(tr(0), tr(8), 0, 1, 2, 3, 4, 5, 6, 7);
      };
      // products of either kind, weights of a lane; of these the first E1 between the scores'
      // products, the rest between those of the sums, before any that takes them
      constexpr int NK = KS * KG, NV = 2 * KG * DT, E = 16 * KG, E1 = E * 5 / 8, NE = NV - DT;
      bf16x8 ka[AHEAD], va[AHEAD], pf[2 * KG];
      float part[4] = {l, 0.f, 0.f, 0.f};
      auto weights = [&](int from, int to) {
#pragma unroll
        for (int x = from; x < to; ++x) {
          const float w = hw_exp2(fmaf(s[x / 16][x % 16], p.scale, -base));
          part[x % 4] += w;
          // rounded to bf16 for the product (half a step, 2^-8 of each).  A second part, as in
          // attn_kernel: prompt b4 L4096 644 -> 810 us, 512 tokens behind 32000 294 -> 386, wide heads
          // b4 L4096 638 -> 719, 8 tokens behind 8000 41.5 -> 45.2
          pf[x / 8][x % 8] = (__bf16)w;
        }
      };
      // one of a SIMD's two waves goes first, so that the other's vector work falls between
      // its products (prompt b4 L4096 660 -> 651 us; all waves alike 665 -> 660)
      if (W == 8 && (wave & 4)) __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) ka[i] = kfrag(i);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        sn[i % KG] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ka[i % AHEAD], qf[i / KG], i < KG ? zero : sn[i % KG], 0, 0, 0);
        if (i + AHEAD < NK) ka[i % AHEAD] = kfrag(i + AHEAD);
        else va[i + AHEAD - NK] = vfrag(i + AHEAD - NK);
        weights(i * E1 / NK, (i + 1) * E1 / NK);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        o[j % DT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(va[j % AHEAD], pf[j / DT], o[j % DT], 0, 0, 0);
        if (j + AHEAD < NV) va[j % AHEAD] = vfrag(j + AHEAD);
        if (j < NE) weights(E1 + j * (E - E1) / NE, E1 + (j + 1) * (E - E1) / NE);
        if (j == NV / 2 - 1) top = -INFINITY;
        if (j >= NV / 2) // the largest score of the next tile, if all of it is seen
#pragma unroll
          for (int x = (j - NV / 2) * E / (NV / 2); x < (j + 1 - NV / 2) * E / (NV / 2); ++x) top = fmaxf(top, sn[x / 16][x % 16]);
        __builtin_amdgcn_sched_barrier(0);
      }
      l = (part[0] + part[1]) + (part[2] + part[3]);
      if constexpr (W == 8) __builtin_amdgcn_s_setprio(0);
    }
    if (next < k1) {
#pragma unroll
      for (int c = 0; c < CH; ++c) store_k(c, ktile[P]), store_v(c, vtile[1 - P]);
      publish(next, have0, vtile[1 - P]);
    }
    kb = next;
  };
  while (kb < k1) {
    body(std::integral_constant<int, 0>(), s0, s1);
    if (kb >= k1) break;
    body(std::integral_constant<int, 1>(), s1, s0);
  }

  // The edge tiles with an infinity or a NaN in a value that some queries see and others
  // may not: a product would have carried it to all.  Key by key, from the cache.
  if (odd_ever && busy) {
#pragma unroll 1
    for (kb = kstart; kb < k1; kb += kTK) {
      const int pages = page_of(kb, table[div_by((uint32_t)min(kb + lane, p.c.capacity - 1), p.c.page)]);
      const uint64_t have = __builtin_amdgcn_ballot_w64(pages >= 0);
      const uint64_t any = have & bits(k0 - kb, k1 - kb), seen = have & bits(w0 - kb, w1 - kb);
      if (seen == 0 || (any == kAll && kb >= all0 && kb + kTK <= all1)) continue;
      if (seen == kAll && kb >= wall0 && kb + kTK <= wall1) continue;
      auto value_row = [&](int j, int pg) {
        const uint32_t key = (uint32_t)(kb + j);
        return vc + pg * p.c.vp + (int64_t)(key - div_by(key, p.c.page) * p.c.page.d) * p.c.vs;
      };
      bool o1 = false;
#pragma unroll 1
      for (int x = lane; x < kTK * PC; x += 64) {
        const int j = x / PC, d = x % PC * 8, pg = __shfl(pages, j);
        if (d < p.N && (any >> j & 1)) o1 |= odd_values(*reinterpret_cast<const u32x4 *>(value_row(j, pg) + d), __bf16());
      }
      if (__builtin_amdgcn_ballot_w64(o1) == 0) continue;
      const uint64_t mine = seen & bits(q0 - kb, q1 - kb);
      const float base = m == -INFINITY ? 0.f : m;
#pragma unroll 1
      for (uint64_t left = seen; left; left &= left - 1) {
        const int j = (int)__builtin_ctzll(left), pg = __builtin_amdgcn_readlane(pages, j);
        const uint32_t key = (uint32_t)(kb + j);
        const __bf16 *kr1 = kc + pg * p.c.kp + (int64_t)(key - div_by(key, p.c.page) * p.c.page.d) * p.c.ks;
        const __bf16 *vr1 = value_row(j, pg);
        float sj = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          if (16 * k + 8 * half >= p.N) continue;
          const bf16x8 a = *reinterpret_cast<const bf16x8 *>(kr1 + 16 * k + 8 * half);
#pragma unroll
          for (int e = 0; e < 8; ++e) sj = fmaf((float)a[e], (float)qf[k][e], sj);
        }
        sj += __shfl_xor(sj, 32);
        const float pj = hw_exp2(fmaf(sj, p.scale, -base));
        if (!(mine >> j & 1)) continue;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int dim = 32 * d + 8 * e + 4 * half;
            if (dim >= p.N) continue;
            const bf16x4 v = *reinterpret_cast<const bf16x4 *>(vr1 + dim);
#pragma unroll
            for (int x = 0; x < 4; ++x) o[d][4 * e + x] = fmaf(pj, (float)v[x], o[d][4 * e + x]);
          }
      }
    }
  }

  if (!live) return;
  l += __shfl_xor(l, 32);
  if (pc.count == 1) {
    const int64_t at = ((int64_t)pc.i * p.L + t) * p.Hq + h;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (l == 0.f) // no key, or weights of 0 only, whatever V holds (0 times an infinity)
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[d][e] = 0.f;
    __bf16 *const dst = (__bf16 *)p.out + at * p.N;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int dim = 32 * d + 8 * e + 4 * half;
        if (dim < p.N)
          st4<__bf16>(dst + dim, o[d][4 * e] * inv, o[d][4 * e + 1] * inv, o[d][4 * e + 2] * inv, o[d][4 * e + 3] * inv);
      }
    if (p.lse && half == 0) p.lse[at] = l == 0.f ? -INFINITY : (m + hw_log2(l)) * kLn2;
  } else {
    const int64_t pr = (((int64_t)pc.place * p.Hk + hk) * p.tiles + tile) * p.prow + r - r0;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int dim = 32 * d + 8 * e + 4 * half;
        if (dim < p.N)
          *reinterpret_cast<f32x4 *>(p.part + pr * p.N + dim) =
              f32x4{o[d][4 * e], o[d][4 * e + 1], o[d][4 * e + 2], o[d][4 * e + 3]};
      }
    if (half == 0) p.part_ml[pr] = make_float2(m, l);
  }
}

} // namespace

int attn_rows(int N) { return N <= 128 ? 256 : 128; }

template <int NP, int W> static void launch_np(const AttnParams &p, hipStream_t st) {
  const uint32_t grid = (uint32_t)((int64_t)p.slots * p.Hk * p.tiles);
  if (p.c.page.d % 16 == 0) attn_rows_kernel<NP, W, true><<<grid, 64 * W, 0, st>>>(p);
  else attn_rows_kernel<NP, W, false><<<grid, 64 * W, 0, st>>>(p);
}
hipError_t launch_attn_rows(const AttnParams &p, hipStream_t st) {
  if (p.N <= 32) launch_np<32, 8>(p, st);
  else if (p.N <= 64) launch_np<64, 8>(p, st);
  else if (p.N <= 96) launch_np<96, 8>(p, st);
  else if (p.N <= 128) launch_np<128, 8>(p, st);
  else if (p.N <= 192) launch_np<192, 4>(p, st);
  else launch_np<256, 4>(p, st);
  return hipGetLastError();
}

} // namespace ssd
