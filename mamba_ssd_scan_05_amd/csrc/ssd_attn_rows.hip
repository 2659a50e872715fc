// ssd_attn_rows.hip -- attention of many new tokens of a row (prompts and pieces of
// them) over the paged cache, bf16.  The products and the orientation are those of
// ssd_attn.hip, S^T = K Q^T and O^T = V^T P^T, but with 32 x 32 tiles: a wave owns 32
// query vectors for all keys, W waves share the K and V tiles of 64 keys in LDS, two
// buffers of them, the next tile's rows on their way to registers while one is
// worked on.  Bound by the matrix cores together with the exponentials.
#include "ssd_attn_device.h"

namespace ssd {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kTK = 64; // keys of a tile

// 16-byte pieces of a K row, exchanged by the row's number so that eight rows
// read at once lie on different banks.
template <int NP> struct KSwizzle {
  static constexpr int pow2(int n) { return n % 2 ? 1 : 2 * pow2(n / 2); }
  static constexpr int C2 = pow2(NP / 8) < 16 ? pow2(NP / 8) : 16;
  __device__ static __forceinline__ int at(int row, int piece) {
    return row * NP + (piece ^ (row / (16 / C2) & (C2 - 1))) * 8;
  }
};

// Bits [a, b) of 64, the ends anywhere.
__device__ __forceinline__ uint64_t bits(int a, int b) {
  const uint64_t lo = a <= 0 ? ~0ull : a >= 64 ? 0ull : ~0ull << a;
  const uint64_t hi = b >= 64 ? ~0ull : b <= 0 ? 0ull : ~(~0ull << b);
  return lo & hi;
}

template <int NP, int W> __global__ __launch_bounds__(64 * W) void attn_rows_kernel(AttnParams p) {
  constexpr int KS = NP / 16, DT = NP / 32;               // steps of 16 dims, tiles of 32 dims
  constexpr int PC = NP / 8, CH = (kTK * PC + 64 * W - 1) / (64 * W); // pieces of a row, of a thread
  constexpr int kRows = 32 * W;
  using KW = KSwizzle<NP>;
  using VW = Swizzle<__bf16, NP>;
  __shared__ __align__(16) __bf16 ktile[2][kTK * NP], vtile[2][kTK * NP];
  __shared__ int sh[11];

  const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint32_t id = blockIdx.x;
  const int tile = p.tiles - 1 - (int)(id % (uint32_t)p.tiles); // the longest ones first
  id /= (uint32_t)p.tiles;
  const int hk = (int)(id % (uint32_t)p.Hk), slot = (int)(id / (uint32_t)p.Hk);
  Piece pc;
  if (!piece_of<64 * W>(p, slot, sh, &pc)) return;
  pc.i = __builtin_amdgcn_readfirstlane(pc.i);
  pc.index = __builtin_amdgcn_readfirstlane(pc.index);
  pc.size = __builtin_amdgcn_readfirstlane(pc.size);
  const Row row = row_of(p, pc.i);
  if (p.workers > 1 && pc.index == 0 && hk == 0 && tile == 0 && threadIdx.x == 0)
    p.pieces[pc.i] = make_int2(pc.first, pc.count);
  const int nrows = row.n * p.G, r0 = tile * kRows;
  if (r0 >= nrows) return;

  const int64_t cap = p.c.capacity;
  auto token = [&](int r) { return (int)div_by((uint32_t)r, p.group); };
  auto last_key = [&](int t) { return (int)min(max(row.start + t + 1, (int64_t)0), cap); };
  auto first_key = [&](int t) { return p.window ? (int)min(max(row.start + t + 1 - p.window, (int64_t)0), cap) : 0; };
  const int64_t base_key = (int64_t)(row.lo / kAttnUnit) * kAttnUnit, size = (int64_t)pc.size * kAttnUnit;
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
  // lane l: the page of key kb + l, -1 for none
  auto page_of = [&](int kb) {
    const int key = kb + lane;
    const int pg = table[div_by((uint32_t)min(key, p.c.capacity - 1), p.c.page)];
    return key < p.c.capacity && pg < p.c.pages ? max(pg, -1) : -1;
  };
  u32x4 kr[CH], vr[CH];
  auto load = [&](int kb, int pages) { // the thread's pieces of a tile
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int x = c * 64 * W + (int)threadIdx.x, krow = min(x / PC, kTK - 1), piece = x % PC;
      const int pg = __shfl(pages, krow);
      const uint32_t key = (uint32_t)(kb + krow);
      const int64_t at = pg < 0 ? 0 : key - div_by(key, p.c.page) * p.c.page.d, page = max(pg, 0);
      const int d = 8 * piece < p.N ? 8 * piece : 0;
      kr[c] = *reinterpret_cast<const u32x4 *>(kc + page * p.c.kp + at * p.c.ks + d);
      vr[c] = *reinterpret_cast<const u32x4 *>(vc + page * p.c.vp + at * p.c.vs + d);
      if (8 * piece >= p.N) kr[c] = u32x4{0, 0, 0, 0};
    }
  };
  // to LDS; rows of V that no query of the workgroup sees are zero there, whatever they
  // held.  An edge tile: true if another row holds an infinity or a NaN.
  auto store = [&](int buf, uint64_t seen, bool edge) {
    bool odd = false;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int x = c * 64 * W + (int)threadIdx.x, krow = x / PC, piece = x % PC;
      if (kTK * PC % (64 * W) != 0 && krow >= kTK) continue;
      u32x4 v = vr[c];
      if (edge) {
        if (!(seen >> krow & 1)) v = u32x4{0, 0, 0, 0};
        odd |= odd_values(v, __bf16());
      }
      *reinterpret_cast<u32x4 *>(&ktile[buf][KW::at(krow, piece)]) = kr[c];
      *reinterpret_cast<u32x4 *>(&vtile[buf][VW::at(krow, piece / 2) + piece % 2 * 8]) = v;
    }
    return odd;
  };

  f32x16 o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[d][e] = 0.f;
  float m = -INFINITY, l = 0.f;

  int kb = k0 & ~(kTK - 1), buf = 0;
  uint64_t have = 0;
  int odd = 0, pages = -1;
  // a tile's rows to LDS and the barrier behind them
  auto publish = [&](int tile_kb, int b) {
    const uint64_t seen = have & bits(k0 - tile_kb, k1 - tile_kb);
    const bool edge = seen != ~0ull || tile_kb < all0 || tile_kb + kTK > all1;
    const bool o1 = store(b, seen, edge);
    if (edge) {
      odd = __syncthreads_or(o1);
    } else {
      odd = 0;
      __syncthreads();
    }
  };
  if (kb < k1) {
    const int first = page_of(kb);
    have = __builtin_amdgcn_ballot_w64(first >= 0);
    load(kb, first);
    if (kb + kTK < k1) pages = page_of(kb + kTK);
    publish(kb, 0);
  }
  for (; kb < k1; kb += kTK, buf ^= 1) {
    const int next = kb + kTK;
    const uint64_t here = have;
    if (next < k1) {
      have = __builtin_amdgcn_ballot_w64(pages >= 0);
      load(next, pages);
      if (next + kTK < k1) pages = page_of(next + kTK);
    }
    if (kb < w1 && next > w0) {
      // S^T = K Q^T
      f32x16 s[2];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
#pragma unroll
        for (int e = 0; e < 16; ++e) s[g][e] = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const bf16x8 a = *reinterpret_cast<const bf16x8 *>(&ktile[buf][KW::at(32 * g + col, 2 * k + half)]);
          s[g] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, qf[k], s[g], 0, 0, 0);
        }
      }
      const uint64_t seen = here & bits(w0 - kb, w1 - kb);
      const bool full = seen == ~0ull && kb >= wall0 && next <= wall1;
      if (!full) {
        const uint64_t mine = seen & bits(q0 - kb, q1 - kb);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const uint32_t mg = (uint32_t)(mine >> (32 * g)) >> (4 * half);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (!(mg & 1u << (e % 4 + 8 * (e / 4)))) s[g][e] = -INFINITY;
        }
      }
      float top = -INFINITY;
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int e = 0; e < 16; ++e) top = fmaxf(top, s[g][e]);
      top = fmaxf(top, __shfl_xor(top, 32)) * p.scale;
      // the weights' reference moves only when some weight would pass 2^8
      if (__builtin_amdgcn_ballot_w64(top > m + 8.f) != 0) {
        const float mn = fmaxf(m, top), a = hw_exp2(m - (mn == -INFINITY ? 0.f : mn));
        l *= a;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] *= a;
        m = mn;
      }
      const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          s[g][e] = hw_exp2(fmaf(s[g][e], p.scale, -base));
          l += s[g][e];
        }
      if (!full && odd) {
        // an infinity or a NaN in a value that some queries see and others may not: key by key
        const uint64_t mine = seen & bits(q0 - kb, q1 - kb);
        for (int j = 0; j < kTK; ++j) {
          const int jj = j & 31, src = col + 32 * (jj >> 2 & 1), reg = (jj & 3) + 4 * (jj >> 3);
          float pj = 0.f;
#pragma unroll
          for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float x = __shfl(s[g][e], src);
              if (j / 32 == g && reg == e) pj = x;
            }
          if (mine >> j & 1) {
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const int dim = 32 * d + 8 * (e / 4) + 4 * half + e % 4;
                o[d][e] = fmaf(pj, (float)vtile[buf][VW::at(j, dim / 16) + dim % 16], o[d][e]);
              }
          }
        }
      } else {
        // O^T += V^T P^T, 16 keys at a time: eight weights of a lane, rounded to bf16
        // (half a step, 2^-8 of each), against the same keys of V
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            bf16x8 pf;
#pragma unroll
            for (int e = 0; e < 8; ++e) pf[e] = (__bf16)s[g][8 * u + e];
            const int row0 = 32 * g + 16 * u + 4 * half + (lane >> 2 & 3);
#pragma unroll
            for (int d = 0; d < DT; ++d) {
              const int unit = 2 * d + (lane >> 4 & 1);
              const auto tr = [&](int rr) {
                return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                    (__attribute__((address_space(3))) lds_bf16x4 *)(&vtile[buf][VW::at(rr, unit) + 4 * (lane & 3)])));
              };
              const bf16x8 vf = __builtin_shufflevector(tr(row0), tr(row0 + 8), 0, 1, 2, 3, 4, 5, 6, 7);
              o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pf, o[d], 0, 0, 0);
            }
          }
      }
    }
    if (next < k1) publish(next, buf ^ 1);
  }

  if (!live) return;
  l += __shfl_xor(l, 32);
  if (pc.count == 1) {
    const int64_t at = ((int64_t)pc.i * p.L + t) * p.Hq + h;
    const float inv = l == 0.f ? 0.f : 1.f / l;
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
    const int64_t pr = (((int64_t)slot * p.Hk + hk) * p.tiles + tile) * kRows + r - r0;
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

hipError_t launch_attn_rows(const AttnParams &p, hipStream_t st) {
  const uint32_t grid = (uint32_t)((int64_t)p.slots * p.Hk * p.tiles);
  if (p.N <= 32) attn_rows_kernel<32, 8><<<grid, 512, 0, st>>>(p);
  else if (p.N <= 64) attn_rows_kernel<64, 8><<<grid, 512, 0, st>>>(p);
  else if (p.N <= 96) attn_rows_kernel<96, 8><<<grid, 512, 0, st>>>(p);
  else if (p.N <= 128) attn_rows_kernel<128, 8><<<grid, 512, 0, st>>>(p);
  else if (p.N <= 192) attn_rows_kernel<192, 4><<<grid, 256, 0, st>>>(p);
  else attn_rows_kernel<256, 4><<<grid, 256, 0, st>>>(p);
  return hipGetLastError();
}

} // namespace ssd
