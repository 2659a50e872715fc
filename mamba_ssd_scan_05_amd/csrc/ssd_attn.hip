// ssd_attn.hip -- attention of new tokens over a paged key-value cache.  For
// query vector q of a token at position p, over the keys j in (p - window, p]
// that the cache holds:
//
//   s_j = scale q . k_j,   out = sum_j e^{s_j - m} v_j / l,   l = sum_j e^{s_j - m}
//
// in one pass with the running maximum m.  All exponents are base 2 (the scale
// carries log2 e).
//
// Decomposition.  The G query heads that share a key head are rows of one
// product, so K and V are read once for all of them: 16 rows (token, head) a
// workgroup, as columns of the products S^T = K Q^T and O^T = V^T P^T.  In that
// orientation a lane holds scores of one query only (its column), its four
// accumulator rows are keys, and they are the B operand of the second product
// as they stand (keys {4g..4g+3, 16+4g..16+4g+3} of lane group g): P does not
// leave the registers.  The four waves of a workgroup take every fourth tile of
// keys, each with its own m, l and O, and are joined in LDS at the end.
// K rows go to registers as A operands; V tiles pass through LDS, a wave's own
// part of it, written as rows and read transposed (ds_read_b64_tr_b16).  The next
// tile's K and V are on their way while one is worked on.
//
// Long caches are cut into pieces (see piece_of); attn_join_kernel joins them.
//
// Bound by HBM: b128 rows of up to 16384 keys, 32 + 8 heads N128 bf16 780 us (5.5 TB/s;
// a large copy reaches 4.9, reading and writing), one row of 262143 keys 200 us (5.4), b32
// 2047 keys 48 us (5.6).  Small calls by their chain of waits (start, page table, keys,
// join): b1 1000 keys 10.5 us in a graph, of which 3.5 are two launches that do
// nothing and 3.6 the join.  fp32 with many queries by the matrix cores and the reads of K
// and V for every 16 rows: b1 L2048 32 + 8 heads N128 430 us, 80 TFLOP/s of the 154 that a
// large product reaches.
#include "ssd_attn_device.h"

namespace ssd {
namespace {

constexpr int kThreads = 256, kWaves = 4, kRows = 16;

// Groups of 16 keys in a tile: the K of the second product's matrix instruction (bf16 32,
// fp32 four times 4).
template <typename T> constexpr int kKT = sizeof(T) == 2 ? 2 : 1;

// Maximum over the four lane groups of a column.
__device__ __forceinline__ float col_max(float v) {
  const Both x = swap16(v);
  const Both y = swap32(fmaxf(x.a, x.b));
  return fmaxf(y.a, y.b);
}
__device__ __forceinline__ float col_sum(float v) {
  const Both x = swap16(v);
  const Both y = swap32(x.a + x.b);
  return y.a + y.b;
}

template <typename T> __device__ __forceinline__ typename FragOf<T>::type zero_frag() {
  const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  return pack8<T>(z);
}

// A use of the fragments that costs nothing but the wait for them.
template <int K> __device__ __forceinline__ void arrived(FragBF (&f)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k) __asm__ volatile("" : "+v"(f[k].v));
}
template <int K> __device__ __forceinline__ void arrived(FragF32 (&f)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) __asm__ volatile("" : "+v"(f[k].v[e]));
}

// UNI: the page size is a multiple of 16, so that 16 keys from a multiple of 16 on lie in
// one page, one behind the other (see locate).  Wide heads hold so much of a tile that one
// workgroup to a compute unit is all there is room for (two, with 91 registers in scratch:
// b64, a window of 2048 keys, 10 + 1 heads N256 104 us, one 48).
template <typename T, int NP, bool UNI>
__global__ __launch_bounds__(kThreads, NP <= 128 ? 2 : 1) void attn_kernel(AttnParams p) {
  constexpr int KT = kKT<T>, TK = 16 * KT, ES = sizeof(T);
  constexpr int KK = NP / 32, ND = NP / 16;    // steps of 32 dims, tiles of 16 dims
  constexpr int PC = NP * ES / 16, PI = PC / 4; // 16-byte pieces of a row, loads of 16 rows
  constexpr int LO = NP + 4;                   // row stride of the join's tile
  using Frag = typename FragOf<T>::type;
  using SW = Swizzle<T, NP>;
  constexpr int kTile = TK * NP * ES, kJoin = 16 * LO * 4;
  __shared__ __align__(16) char lds[kWaves * (kTile > kJoin ? kTile : kJoin)];
  __shared__ float2 ml[kWaves][16];
  __shared__ int sh[12];

  const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int tile, hk, slot;
  place_of(p, blockIdx.x, &tile, &hk, &slot);
  Piece pc;
  if (!piece_of<kThreads>(p, slot, sh, &pc)) return;
  const Row row = pc.row;
  if (p.workers > 1 && !p.list && pc.index == 0 && hk == 0 && tile == 0 && threadIdx.x == 0)
    p.pieces[pc.i] = make_int2(pc.place, pc.count);
  const int nrows = row.n * p.G, r0 = tile * kRows;
  if (r0 >= nrows) return;

  // the tile's tokens and the keys that any and all of its queries see
  const int t_first = (int)div_by((uint32_t)r0, p.group);
  const int t_last = (int)div_by((uint32_t)(min(r0 + kRows, nrows) - 1), p.group);
  const int64_t cap = p.c.capacity;
  auto last_key = [&](int t) { return (int)min(max((int64_t)row.start + t + 1, (int64_t)0), cap); };
  auto first_key = [&](int t) { return p.window ? (int)min(max((int64_t)row.start + t + 1 - p.window, (int64_t)0), cap) : 0; };
  int k0 = first_key(t_first), k1 = last_key(t_last);
  const int all0 = first_key(t_last), all1 = last_key(t_first); // seen by every query: [all0, all1)
  {
    const int64_t base = (int64_t)(row.lo / kAttnUnit) * kAttnUnit, size = (int64_t)pc.size() * kAttnUnit;
    const int64_t a = base + pc.index * size;
    k0 = (int)max((int64_t)k0, a);
    k1 = (int)min((int64_t)k1, a + size);
  }
  // this lane's query
  const int r = r0 + li;
  const bool live = r < nrows;
  const int t = (int)div_by((uint32_t)(live ? r : r0), p.group), h = hk * p.G + (live ? r : r0) - t * p.G;
  const int q0 = first_key(t), q1 = last_key(t);
  Frag qf[KK];
  {
    const T *src = (const T *)p.q + pc.i * p.qb + t * p.qt + h * p.qh;
#pragma unroll
    for (int k = 0; k < KK; ++k) {
      const int d = 32 * k + 8 * lg;
      qf[k] = zero_frag<T>();
      if (live && d < p.N) {
        if (p.qvec) {
          load_frag(qf[k], src + d);
        } else {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = to_f(src[d + e]);
          qf[k] = pack8<T>(v);
        }
        if (p.negate) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = -elem(qf[k], e);
          qf[k] = pack8<T>(v);
        }
      }
    }
  }

  // the loads of a tile of keys
  const T *const kc = (const T *)p.c.kc + hk * p.c.kh, *const vc = (const T *)p.c.vc + hk * p.c.vh;
  const int32_t *const table = p.c.table + pc.i * p.c.tb;
  // page of a key that may lie outside the cache or on no page (then 0, *ok = false)
  auto lookup = [&](int key, bool *ok, int *at) {
    const uint32_t kk = (uint32_t)min(key, p.c.capacity - 1), e = div_by(kk, p.c.page);
    const int pg = table[e];
    *ok = key < p.c.capacity && pg >= 0 && pg < p.c.pages;
    *at = *ok ? (int)(kk - e * p.c.page.d) : 0;
    return *ok ? pg : 0;
  };
  int vrow[PI], vcol[PI]; // of the lane's pieces of 16 rows of V
  uint32_t voff[PI], koff = (uint32_t)((UNI ? li * p.c.ks : 0) * ES); // offsets from a group's first row, bytes
#pragma unroll
  for (int i = 0; i < PI; ++i) {
    const int x = i * 64 + lane;
    vrow[i] = x / PC, vcol[i] = x % PC * (16 / ES);
    voff[i] = (uint32_t)(((UNI ? vrow[i] * p.c.vs : 0) + (vcol[i] < p.N ? vcol[i] : 0)) * ES);
  }
  // Where the keys lie.  UNI: lane l keeps the places of the l-th 16 keys of a batch of 1024,
  // found once for the batch.  Otherwise lane l keeps those of the tile's l-th key.  The
  // table's entries for the next batch or tile are on their way.
  const int kstart = k0 & ~(kWaves * TK - 1);
  constexpr int kBatch = 64 * 16;
  uint64_t gk = 0, gv = 0, gok = 0; // gok: the lanes whose key is on a page
  int entry = -1;
  auto entry_of = [&](int kb) {
    return table[div_by((uint32_t)min(kb + (UNI ? 16 : 1) * lane, p.c.capacity - 1), p.c.page)];
  };
  auto locate = [&](int kb, int next) { // the batch or tile at kb; the one behind it
    const uint32_t key = (uint32_t)(kb + (UNI ? 16 : 1) * lane), at = key - div_by(key, p.c.page) * p.c.page.d;
    const bool ok = (int)key < p.c.capacity && entry >= 0 && entry < p.c.pages;
    gk = ok ? (uint64_t)(uint32_t)entry * (uint32_t)p.c.kp + (uint64_t)at * (uint32_t)p.c.ks : 0;
    gv = ok ? (uint64_t)(uint32_t)entry * (uint32_t)p.c.vp + (uint64_t)at * (uint32_t)p.c.vs : 0;
    gok = __builtin_amdgcn_ballot_w64(ok);
    if (next < k1) entry = entry_of(next);
  };
  auto of_lane = [](uint64_t x, int f) {
    if constexpr (UNI)
      return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(x >> 32), f) << 32 |
             (uint32_t)__builtin_amdgcn_readlane((int)x, f);
    else
      return (uint64_t)(uint32_t)__shfl((int)(x >> 32), f) << 32 | (uint32_t)__shfl((int)x, f);
  };
  Frag kf[KT][KK];
  u32x4 vr[KT * PI];
  uint32_t have_k = 0, have_v = 0; // keys of the tile that lie on a page, one bit each
  auto load_k = [&](int kb) {
    const int f = (kb - kstart) / 16 % 64; // the tile's first group
    if constexpr (UNI) {
      if (f < kWaves * KT) locate(kb - 16 * f, kb - 16 * f + kBatch);
      have_k = 0;
#pragma unroll
      for (int g = 0; g < KT; ++g) have_k |= gok >> (f + g) & 1 ? 0xFFFFu << (16 * g) : 0;
    } else {
      locate(kb, kb + kWaves * TK);
      have_k = (uint32_t)gok & (TK == 32 ? ~0u : 0xFFFFu);
    }
#pragma unroll
    for (int g = 0; g < KT; ++g) {
      const T *src = kc + of_lane(gk, UNI ? f + g : 16 * g + li);
#pragma unroll
      for (int k = 0; k < KK; ++k) {
        const int d = 32 * k + 8 * lg;
        if (d < p.N) load_frag(kf[g][k], (const T *)((const char *)src + koff) + d);
        else kf[g][k] = zero_frag<T>();
      }
    }
  };
  auto load_v = [&](int kb) {
#pragma unroll
    for (int g = 0; g < KT; ++g)
#pragma unroll
      for (int i = 0; i < PI; ++i) {
        const uint64_t base = of_lane(gv, UNI ? (kb - kstart) / 16 % 64 + g : 16 * g + vrow[i]);
        vr[g * PI + i] = *reinterpret_cast<const u32x4 *>((const char *)(vc + base) + voff[i]);
      }
  };

  f32x4 o[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d) o[d] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;
  bool left_out = false; // this wave left products out
  T *const vt = reinterpret_cast<T *>(lds + wave * kTile);
  int kb = kstart + wave * TK;
  if (kb < k1) {
    entry = entry_of(UNI ? kstart : kb);
    load_k(kb);
    load_v(kb);
  }
  // The queries are there from here on: as loads still on their way they would be waited
  // for in every pass of the loop, and with them the next tile's.
  arrived(qf);
  for (; kb < k1; kb += kWaves * TK) {
    const int next = kb + kWaves * TK;
    // S^T = K Q^T
    f32x4 s[KT];
#pragma unroll
    for (int g = 0; g < KT; ++g) {
      s[g] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < KK; ++k) s[g] = mma(kf[g][k], qf[k], s[g]);
    }
    have_v = have_k;
    if (next < k1) load_k(next);
    // the keys of the tile that any query of the workgroup sees, and whether all see them all
    const uint32_t lo_bits = k0 - kb >= 32 ? 0u : k0 > kb ? ~0u << (k0 - kb) : ~0u;
    const uint32_t hi_bits = k1 - kb < 32 ? (1u << (k1 - kb)) - 1 : ~0u;
    const uint32_t seen = have_v & lo_bits & hi_bits;
    const bool full = seen == (TK == 32 ? ~0u : 0xFFFFu) && kb >= all0 && kb + TK <= all1;
    if (!full) {
#pragma unroll
      for (int g = 0; g < KT; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 16 * g + 4 * lg + e;
          if (!(seen >> j & 1) || kb + j < q0 || kb + j >= q1) s[g][e] = -INFINITY;
        }
    }
    float top = -INFINITY;
#pragma unroll
    for (int g = 0; g < KT; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e) top = fmaxf(top, s[g][e]);
    const float mn = fmaxf(m, col_max(top) * p.scale);
    const float base = mn == -INFINITY ? 0.f : mn; // nothing seen yet: every weight 0
    if (__builtin_amdgcn_ballot_w64(mn != m) != 0) {
      const float a = hw_exp2(m - base);
      l *= a;
#pragma unroll
      for (int d = 0; d < ND; ++d) o[d] *= a;
      m = mn;
    }
    float w[8];
#pragma unroll
    for (int g = 0; g < KT; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[4 * g + e] = hw_exp2(fmaf(s[g][e], p.scale, -base));
        l += w[4 * g + e];
      }
    // V through LDS; rows that no query sees are zero there, whatever they held
    bool odd = false;
#pragma unroll
    for (int g = 0; g < KT; ++g)
#pragma unroll
      for (int i = 0; i < PI; ++i) {
        u32x4 v = vr[g * PI + i];
        if (!full) {
          if (!(seen >> (16 * g + vrow[i]) & 1)) v = u32x4{0, 0, 0, 0};
          odd |= odd_values(v, T());
        }
        const int unit = vcol[i] / 16;
        *reinterpret_cast<u32x4 *>(vt + SW::at(16 * g + vrow[i], unit) + vcol[i] % 16) = v;
      }
    if (next < k1) load_v(next);
    if (!full && __builtin_amdgcn_ballot_w64(odd) != 0) {
      left_out = true; // added behind the loop
    } else if constexpr (ES == 2) {
      // O^T += V^T P^T, P as the sum of two bf16 parts: off by 1.25 2^-15 of each weight (one
      // rounded part: 2^-8, which the output's rounding does not hide: error against 64 bits
      // 0.0017 of the output's norm, two 0.0016).  HBM bounds these calls, so the second
      // product costs little: b128 rows of up to 16384 keys 779 us, by one part 778, b8 2047
      // keys 18.7 and 18.5, b64 a window of 2048 keys 10 + 1 heads N256 31.5 and 31.1.
      // The first part is w cut off a quarter of bf16's last place below it, so that what is
      // left is above 0 where w is, and takes an infinity in V to the same side.
      float w1[8], w2[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t u = __builtin_elementwise_sub_sat(__builtin_bit_cast(uint32_t, w[e]), 0x4000u) & 0xFFFF0000u;
        w1[e] = __builtin_bit_cast(float, u);
        w2[e] = w[e] - w1[e];
      }
      const FragBF pf = pack8<__bf16>(w1), pr = pack8<__bf16>(w2);
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        FragBF vf;
        const auto tr = [&](int row0) {
          const __bf16 *a = reinterpret_cast<const __bf16 *>(vt) + SW::at(row0 + 4 * lg + (li >> 2), d) + 4 * (li & 3);
          return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                                                (__attribute__((address_space(3))) lds_bf16x4 *)(a)));
        };
        vf.v = __builtin_shufflevector(tr(0), tr(16), 0, 1, 2, 3, 4, 5, 6, 7);
        o[d] = mma(vf, pr, mma(vf, pf, o[d]));
      }
    } else {
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[d] = __builtin_amdgcn_mfma_f32_16x16x4f32(to_f(vt[SW::at(4 * lg + e, d) + li]), w[e], o[d], 0, 0, 0);
    }
  }

  // The tiles with an infinity or a NaN in a value that some queries see and others may not:
  // a product would have carried it to all.  Key by key, from the cache.
  if (left_out) {
#pragma unroll 1
    for (kb = kstart + wave * TK; kb < k1; kb += kWaves * TK) {
      bool ok;
      int at;
      const int pg = lookup(kb + lane, &ok, &at);
      const uint32_t seen = (uint32_t)__builtin_amdgcn_ballot_w64(ok && kb + lane >= k0 && kb + lane < k1 && lane < TK);
      if (seen == (TK == 32 ? ~0u : 0xFFFFu) && kb >= all0 && kb + TK <= all1) continue;
      const uint64_t krow = (uint64_t)pg * p.c.kp + (uint64_t)at * p.c.ks, vrow1 = (uint64_t)pg * p.c.vp + (uint64_t)at * p.c.vs;
      auto at_lane = [&](uint64_t x, int j) {
        return (uint64_t)(uint32_t)__shfl((int)(x >> 32), j) << 32 | (uint32_t)__shfl((int)x, j);
      };
      bool odd = false;
#pragma unroll 1
      for (int x = lane; x < TK * PC; x += 64) {
        const int j = x / PC, d = x % PC * (16 / ES);
        const T *v = vc + at_lane(vrow1, j) + d;
        if (d < p.N && (seen >> j & 1)) odd |= odd_values(*reinterpret_cast<const u32x4 *>(v), T());
      }
      if (__builtin_amdgcn_ballot_w64(odd) == 0) continue;
      const float base = m == -INFINITY ? 0.f : m;
#pragma unroll 1
      for (uint32_t left = seen; left; left &= left - 1) {
        const int j = __builtin_ctz(left);
        const T *ks = kc + at_lane(krow, j), *vs = vc + at_lane(vrow1, j);
        float sj = 0.f;
#pragma unroll
        for (int k = 0; k < KK; ++k) {
          const int d = 32 * k + 8 * lg;
          if (d >= p.N) continue;
          Frag a;
          load_frag(a, ks + d);
#pragma unroll
          for (int e = 0; e < 8; ++e) sj = fmaf(elem(a, e), elem(qf[k], e), sj);
        }
        const float w = hw_exp2(fmaf(col_sum(sj), p.scale, -base));
        if (kb + j < q0 || kb + j >= q1) continue;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (16 * d + 4 * lg < p.N) o[d][e] = fmaf(w, to_f(vs[16 * d + 4 * lg + e]), o[d][e]);
      }
    }
  }

  // join the waves
  l = col_sum(l);
  __syncthreads();
  float *const oj = reinterpret_cast<float *>(lds) + wave * 16 * LO;
#pragma unroll
  for (int d = 0; d < ND; ++d) *reinterpret_cast<f32x4 *>(oj + li * LO + 16 * d + 4 * lg) = o[d];
  if (lg == 0) ml[wave][li] = make_float2(m, l);
  __syncthreads();
  const bool whole = pc.count == 1;
  const int64_t pr = (((int64_t)pc.place * p.Hk + hk) * p.tiles + tile) * p.prow;
  for (int x = threadIdx.x; x < 16 * (NP / 4); x += kThreads) {
    const int q = x / (NP / 4), c = x % (NP / 4) * 4;
    if (r0 + q >= nrows || c >= p.N) continue;
    float2 e[kWaves];
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) e[w] = ml[w][q], top = fmaxf(top, e[w].x);
    const float base = top == -INFINITY ? 0.f : top;
    f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float a = hw_exp2(e[w].x - base);
      sum = fmaf(a, e[w].y, sum);
      acc += a * *reinterpret_cast<const f32x4 *>(reinterpret_cast<float *>(lds) + (w * 16 + q) * LO + c);
    }
    if (whole) {
      const int tq = (int)div_by((uint32_t)(r0 + q), p.group), hq = hk * p.G + r0 + q - tq * p.G;
      const int64_t at = ((int64_t)pc.i * p.L + tq) * p.Hq + hq;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      if (sum == 0.f) acc = f32x4{0.f, 0.f, 0.f, 0.f}; // (0 times an infinity in V among them)
      st4<T>((T *)p.out + at * p.N + c, acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
      if (p.lse && c == 0) p.lse[at] = sum == 0.f ? -INFINITY : (top + hw_log2(sum)) * kLn2;
    } else {
      *reinterpret_cast<f32x4 *>(p.part + (pr + q) * p.N + c) = acc;
      if (c == 0) p.part_ml[pr + q] = make_float2(top, sum);
    }
  }
}

// The plan of a batch of many rows, by one workgroup: p.list and p.cut.  Every workgroup for
// itself would read all rows (b60000 of 200 keys, one head N64: 27 ms, so 0.52; b1024 8 heads 138 us and 91).
constexpr int kPlanThreads = 1024, kPlanRows = 4; // rows of a thread at once
__global__ __launch_bounds__(kPlanThreads) void attn_plan_kernel(AttnParams p) {
  constexpr int kW = kPlanThreads / 64;
  __shared__ int sh[2][kW];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int total = 0, longest = 0;
#pragma unroll 4
  for (int i = tid; i < p.b; i += kPlanThreads) {
    const int u = row_of(p, i).units();
    total += u, longest = max(longest, u);
  }
  total = wave_incl_scan_i(total), longest = wave_max_i(longest);
  if (lane == 63) sh[0][wave] = total, sh[1][wave] = longest;
  __syncthreads();
  total = 0;
  for (int w = 0; w < kW; ++w) total += sh[0][w], longest = max(longest, sh[1][w]);
  const int size = piece_units(p, total, longest);
  // Pieces before a row, and in one word of 16 bits each the places and the cut rows before it
  int pieces = 0, stored = 0;
  for (int i0 = 0; i0 < p.b; i0 += kPlanThreads * kPlanRows) {
    int cnt[kPlanRows], c = 0, s = 0;
#pragma unroll
    for (int k = 0; k < kPlanRows; ++k) {
      const int i = i0 + tid * kPlanRows + k;
      cnt[k] = i < p.b ? pieces_of(row_of(p, i).units(), size) : 0;
      c += cnt[k], s += places_of(cnt[k]) | (cnt[k] > 1) << 16;
    }
    const int ce = wave_incl_scan_i(c), se = wave_incl_scan_i(s);
    __syncthreads();
    if (lane == 63) sh[0][wave] = ce, sh[1][wave] = se;
    __syncthreads();
    int at = pieces + ce - c, st = stored + se - s;
    for (int w = 0; w < kW; ++w) {
      if (w < wave) at += sh[0][w], st += sh[1][w];
      pieces += sh[0][w], stored += sh[1][w];
    }
#pragma unroll
    for (int k = 0; k < kPlanRows; ++k) {
      const int i = i0 + tid * kPlanRows + k;
      for (int x = 0; x < cnt[k]; ++x) p.list[at++] = make_int4(i, x, cnt[k], (st & 0xFFFF) + x);
      if (cnt[k] > 1) p.cut[st >> 16] = make_int4(i, st & 0xFFFF, cnt[k], 0), st += cnt[k] | 1 << 16;
    }
  }
  for (int x = pieces + tid; x < p.slots; x += kPlanThreads) p.list[x] = make_int4(-1, 0, 0, 0);
  for (int x = (stored >> 16) + tid; x < p.cuts; x += kPlanThreads) p.cut[x] = make_int4(-1, 0, 0, 0);
}

// Joins the pieces of the rows that have more than one: WPV waves an output vector, N / 4
// threads a piece, as many pieces at once as that leaves, each group of threads with its
// own running maximum (a maximum over all pieces first would be one more wait for memory).
// LIST: of the rows in p.cut, otherwise of all rows.
template <typename T, int WPV, bool LIST> __global__ __launch_bounds__(kThreads) void attn_join_kernel(AttnParams p) {
  __shared__ float acc_sh[kThreads][4];
  __shared__ float2 ml_sh[kThreads];
  constexpr int TPV = 64 * WPV; // threads of a vector
  const int tid = threadIdx.x % TPV, first_tid = threadIdx.x - tid;
  const uint32_t vec = blockIdx.x * (kThreads / TPV) + threadIdx.x / TPV;
  const uint32_t vt = vec / (uint32_t)p.Hq;
  const int h = (int)(vec - vt * (uint32_t)p.Hq);
  int i = (int)(vt / (uint32_t)p.L);
  const int t = (int)(vt - (uint32_t)i * (uint32_t)p.L);
  int2 pc = make_int2(0, 0);
  if constexpr (LIST) {
    const int4 e = i < p.cuts ? p.cut[i] : make_int4(-1, 0, 0, 0);
    i = e.x;
    if (i >= 0 && (!p.c.tokens || t < p.c.tokens[i])) pc = make_int2(e.y, e.z);
  } else {
    if (i < p.b && (!p.c.tokens || t < p.c.tokens[i])) pc = p.pieces[i];
  }
  const bool mine = pc.y > 1;
  const int hk = (int)div_by((uint32_t)h, p.group), r = t * p.G + h - hk * p.G;
  const int tile = r / p.rows;
  const int64_t step = (int64_t)p.Hk * p.tiles * p.prow;
  const int64_t first = (((int64_t)pc.x * p.Hk + hk) * p.tiles + tile) * p.prow + r - tile * p.rows;
  const int nv = p.N / 4, groups = TPV / nv;
  const int g = tid / nv, c4 = (tid - g * nv) * 4;
  f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, sum = 0.f;
  if (mine && g < groups) {
#pragma unroll 4
    for (int c = g; c < pc.y; c += groups) {
      const float2 e = p.part_ml[first + c * step];
      const f32x4 v = *reinterpret_cast<const f32x4 *>(p.part + (first + c * step) * p.N + c4);
      const float mn = fmaxf(m, e.x), base = mn == -INFINITY ? 0.f : mn;
      const float a = hw_exp2(m - base), w = hw_exp2(e.x - base);
      sum = fmaf(sum, a, w * e.y);
      acc = acc * a + w * v;
      m = mn;
    }
  }
  *reinterpret_cast<f32x4 *>(acc_sh[threadIdx.x]) = acc;
  ml_sh[threadIdx.x] = make_float2(m, sum);
  __syncthreads();
  if (!mine || tid >= nv) return;
  float top = -INFINITY;
  for (int k = 0; k < groups; ++k) top = fmaxf(top, ml_sh[first_tid + k * nv].x);
  const float base = top == -INFINITY ? 0.f : top;
  acc = f32x4{0.f, 0.f, 0.f, 0.f};
  sum = 0.f;
  for (int k = 0; k < groups; ++k) {
    const float2 e = ml_sh[first_tid + k * nv];
    const float w = hw_exp2(e.x - base);
    sum = fmaf(w, e.y, sum);
    acc += w * *reinterpret_cast<const f32x4 *>(acc_sh[first_tid + k * nv + tid]);
  }
  const int64_t at = ((int64_t)i * p.L + t) * p.Hq + h;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (sum == 0.f) acc = f32x4{0.f, 0.f, 0.f, 0.f};
  st4<T>((T *)p.out + at * p.N + c4, acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
  if (p.lse && tid == 0) p.lse[at] = sum == 0.f ? -INFINITY : (top + hw_log2(sum)) * kLn2;
}

template <typename T, int NP> void launch_np(const AttnParams &p, hipStream_t st) {
  const uint32_t grid = (uint32_t)((int64_t)p.slots * p.Hk * p.tiles);
  if (p.c.page.d % 16 == 0) attn_kernel<T, NP, true><<<grid, kThreads, 0, st>>>(p);
  else attn_kernel<T, NP, false><<<grid, kThreads, 0, st>>>(p);
}
template <typename T, bool LIST> hipError_t launch_join(const AttnParams &p, hipStream_t st) {
  const int64_t vecs = (int64_t)(LIST ? p.cuts : p.b) * p.L * p.Hq;
  // a wave each where they fill the device: b3 L777 5 heads N96 fp32 43.8 us, four 49.2; fewer
  // vectors wait longer for their pieces: b1 262143 keys 32 heads 203 us, with four waves 197
  if (vecs >= 4096) attn_join_kernel<T, 1, LIST><<<(uint32_t)((vecs + 3) / 4), kThreads, 0, st>>>(p);
  else attn_join_kernel<T, 4, LIST><<<(uint32_t)vecs, kThreads, 0, st>>>(p);
  return hipGetLastError();
}
template <typename T> hipError_t launch_t(const AttnParams &p, hipStream_t st) {
  if (p.list) {
    attn_plan_kernel<<<1, kPlanThreads, 0, st>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (p.rows != kRows) {
    const hipError_t e = launch_attn_rows(p, st);
    if (e != hipSuccess) return e;
  } else if (p.N <= 32) launch_np<T, 32>(p, st);
  else if (p.N <= 64) launch_np<T, 64>(p, st);
  else if (p.N <= 96) launch_np<T, 96>(p, st);
  else if (p.N <= 128) launch_np<T, 128>(p, st);
  else if (p.N <= 192) launch_np<T, 192>(p, st);
  else launch_np<T, 256>(p, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.workers == 1) return e;
  return p.list ? launch_join<T, true>(p, st) : launch_join<T, false>(p, st);
}

int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }
constexpr int64_t kMaxGroups = (int64_t)1 << 23; // workgroups of one launch
constexpr int64_t kMaxCut = (int64_t)1 << 19;    // without pieces, from which on there are none

// n sizes of units in all rows together, at most: the pieces, their places and the cut rows.
void set_pieces(AttnParams *p, int64_t n) {
  const int64_t places = 8 * n / 5;
  p->slots = (int)n + p->b;
  p->stores = places < p->slots ? (int)places : p->slots;
  p->cuts = p->stores / 2 < p->b ? p->stores / 2 : p->b;
}
void uncut(AttnParams *p) { p->workers = 1, p->slots = p->b, p->stores = p->cuts = 0; }

} // namespace

// More than one tile of query vectors in bf16 goes to attn_rows_kernel, which reads K and V
// once for 256 (128) of them: b4, 8 new tokens behind 8000, 32 + 8 heads N128 41 us, by two
// tiles of 16 here 47; 16 tokens 44 and 86.
//
// Pieces: as many as run at once (512 workgroups, 256 of wide heads; with twice as many b8
// 2047 keys 20.6 us, so 18.3), but none larger than a MB of keys and values while there are
// fewer than 4096 workgroups (b128 rows of 0 to 16384 keys: 1024 929 us, 2048 844, 4096 796;
// with one row of 262143 keys 199, 211 and 232, since a workgroup costs 8 us before its
// first key).  Only cut rows' pieces have sums, at most 1.6 times as many as that and the heads once
// more: 100 to 220 MB, whatever the batch (as many as pieces and rows b127 L512 32 heads N128 had
// 1.1 GB).  From half a million workgroups on, 1000 rounds of the device, rows are not cut.
int64_t attn_plan(AttnParams *p, int dtype) {
  const int64_t vecs = (int64_t)p->L * p->G;
  const bool wide = dtype == 1 && vecs > kRows;
  p->rows = wide ? attn_rows(p->N) : kRows;
  const int64_t tiles = (vecs + p->rows - 1) / p->rows, heads = p->Hk * tiles;
  p->tiles = (int)tiles;
  const int64_t prefer = wide ? 512 : p->N <= 128 ? 512 : 256, most = wide ? 512 : 4096;
  p->workers = heads * p->b >= kMaxCut ? 1 : (int)((most + heads - 1) / heads);
  p->prefer = (int)((prefer + heads - 1) / heads);
  p->enough = (int)((1 << 20) / (2 * kAttnUnit * p->N * (dtype == 1 ? 2 : 4)));
  if (p->enough < 2) p->enough = 2;
  p->prow = (int)(vecs < p->rows ? vecs : p->rows);
  if (heads * p->b > kMaxGroups) return -1;
  if (p->workers == 1) {
    uncut(p);
    return 0;
  }
  set_pieces(p, p->workers);
  const int64_t rows = p->stores * heads * p->prow;
  return up256(rows * p->N * 4) + up256(rows * 8) +
         up256((int64_t)p->slots * 16) + up256((int64_t)p->cuts * 16); // (or 8 b)
}

// Pieces that there can be with this table and window: a row has no more units than its
// table or its window and new tokens, and a piece no fewer than piece_units gives it.
// (Workgroups without a piece cost their launch, behind all others: 3700 of them 12 us.)
//
// No pieces where every row has several tiles, the workgroups fill the device without them
// and even the longest that the table allows takes little of the whole: fp32 b3 L777
// window 500 29.6 us, with pieces 35.5; bf16 b16 L1024 behind up to 4000 keys 847 and 910.
// Where the table is wide one row may be all the work: b32 L128, one row behind 131000 keys
// and 31 behind 1000, 32 + 8 heads N128 4540 us without and 545 with pieces (all 32 behind
// 8000: 643 and 661); b8 L512 behind 0 to 30000 1610 and 1370.  Of one tile a row, 8192
// workgroups of up to 4096 keys: b1024, one row of 16000 keys and the others of 200, 8 heads
// N64 204 us without and 113 with pieces; b256, 32000 and 500, 32 heads N128 647 and 478; even
// rows of 5000 or 0 to 8000 keys the same within 2 %.
void attn_slots(AttnParams *p) {
  if (p->workers == 1) return;
  int64_t keys = p->c.capacity;
  if (p->window && p->window + p->L < keys) keys = p->window + p->L;
  const int64_t groups = (int64_t)p->Hk * p->tiles * p->b;
  if (p->tiles > 1 ? groups >= 512 && keys <= 4 * (groups / 512) * p->L : groups >= 8192 && keys <= 4096)
    return uncut(p);
  const int64_t total = (int64_t)p->b * ((keys + kAttnUnit - 1) / kAttnUnit + 1);
  // of the largest pieces, or twice as many (below 4 * prefer) where uneven rows halve them
  int64_t n = (total + p->enough - 1) / p->enough;
  const int64_t halved = 2 * n < 4 * (int64_t)p->prefer ? 2 * n : 4 * (int64_t)p->prefer;
  if (n < halved) n = halved;
  if (n < p->prefer) n = p->prefer;
  if (n > (total + 1) / 2) n = (total + 1) / 2;
  if (n > p->workers) n = p->workers;
  if (n == 1) return uncut(p);
  set_pieces(p, n);
}

void attn_workspace(AttnParams *p, void *workspace) {
  if (p->workers == 1) return;
  const int64_t rows = (int64_t)p->stores * p->Hk * p->tiles * p->prow;
  char *w = (char *)workspace;
  p->part = (float *)w;
  w += up256(rows * p->N * 4);
  p->part_ml = (float2 *)w;
  w += up256(rows * 8);
  // The plan by a kernel of its own (3 us) for more rows than a workgroup has threads for (b300 0 to 200
  // keys 16 + 4 heads N128 31 us, by every workgroup for itself 37; b128 1000 keys 8 + 2 heads N64 23.4
  // and 19.4), among several tokens, whose workgroups are few and long, than a wave has lanes (b128 L8 0 to
  // 2000 keys 32 + 8 heads N128 182 us and 185).  Also where few of the rows can be cut, of so many vectors that
  // it costs less than to start the join for all (fp32 b256 L20 0 to 2000 keys 1195 us and 1228).
  if (p->b > (p->rows == kRows ? kThreads : 64) ||
      (2 * p->cuts <= p->b && (int64_t)p->b * p->L * p->Hq >= 65536)) {
    p->list = (int4 *)w;
    p->cut = (int4 *)(w + up256((int64_t)p->slots * 16));
  } else {
    p->pieces = (int2 *)w;
  }
}

hipError_t launch_attn(int dtype, const AttnParams &p, hipStream_t st) {
  return dtype == 1 ? launch_t<__bf16>(p, st) : launch_t<float>(p, st);
}

} // namespace ssd
