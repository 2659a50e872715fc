// ssd_glr.hip -- the gated linear recurrence: forward scan, gradients and
// single-token step.  Per channel
//
//   s_t = sigmoid(r_t + rb),  a_t = exp(A s_t),  beta_t = sqrt(1 - a_t^2)
//   h_t = a_t h_{t-1} + beta_t sigmoid(i_t + ib) x_t
//
// and backwards, with g_t the gradient at h_t and c_t = a_t g_t the one at
// h_{t-1}:   c_t = a_t (dout_t + c_{t+1}).
// Both are chains of affine maps v -> A v + w, which compose associatively:
// (A2, w2) after (A1, w1) is (A2 A1, A2 w1 + w2).
//
// Decomposition.  A workgroup owns 256 bytes of channels of one batch row over
// one chunk of tokens.  A lane owns one or two channels, a wave a run of
// successive tokens, read once into registers: the walk over them needs no
// exchange between lanes, and what is per token (its existence, a reset, its
// address) is per wave.  (Measured before: 16 bytes a lane with the token groups
// of a wave composed by shuffles, b4 L4096 D5120 bf16 forward 265 us against
// 147.)  The waves' maps are composed through LDS, and the chunks' through
// one 64-bit word per (chunk, channel) in the workspace: a chunk publishes its
// own map as soon as it is known and the finished state once its
// predecessor's is; a later chunk looks back over several words at a time.  So
// the data crosses HBM once in each direction however the time axis is
// split.  The fold over words always runs forward from a finished state with
// one fma per chunk, the same operations that produced the words in between,
// so results do not depend on timing.
//
// Workgroups take their chunk from a ticket counter, chunks in time order:
// a workgroup waits only for lower tickets, which were handed to workgroups
// that already run, so every wait ends.
#include <float.h>

#include "ssd_device.h"
#include "ssd_seq.h"

namespace ssd {
namespace {

// Tokens of a wave, forward and backward, and the tokens whose decays are
// formed together (two branches, of which a wave takes one; more at a time need
// more registers than two workgroups a compute unit leave).
constexpr int kFwdTokens = 16, kBwdTokens = 8;
constexpr int kTogether = 2;
// A workgroup has eight waves; rows that fewer cover take four or two.
constexpr int kWaves = 8;
static_assert(kGlrChunk == kWaves * kFwdTokens && kGlrSegment == kWaves * kBwdTokens, "tokens of a chunk");

// Words read at a time in a look back, and how far back it goes: as long as it
// finds maps, up to kWindow words.
constexpr int kRead = 4, kWindow = 16;

// Words of the chunk chain: {A (high half), value (low half)}.  A is a
// product of values in [0, inf) or a canonical NaN, so two other NaN
// patterns mark the two remaining states.
constexpr uint32_t kNotYet = 0xFFFFFFFFu;   // the fill value
constexpr uint32_t kFinished = 0xFFFFFFFEu; // the value is the carried state itself

__device__ __forceinline__ uint64_t make_word(uint32_t hi, float v) {
  return ((uint64_t)hi << 32) | __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ uint32_t decay_bits(float A) {
  return A == A ? __builtin_bit_cast(uint32_t, A) : 0x7FC00000u;
}
__device__ __forceinline__ void publish(uint64_t *w, uint64_t v) {
  __hip_atomic_store(w, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Carried value entering a chunk: `prev` points at the word of the chunk
// right before it in chain order, `step` (in words) leads to earlier ones and
// `n` of them exist (n >= 1; the first one only ever holds kFinished).
// `stash` is this thread's column of kWindow rows of `ld` words in LDS: maps
// behind the first four wait there, registers are short here.
__device__ __forceinline__ float look_back(const uint64_t *prev, int64_t step, int n, uint64_t *stash, int ld) {
  for (;;) {
#pragma unroll 1
    for (int k0 = 0; k0 < kWindow; k0 += kRead) {
      uint64_t w[kRead];
      int kp = -1;
      bool open = true;
#pragma unroll
      for (int k = 0; k < kRead; ++k)
        w[k] = __hip_atomic_load(prev + step * (k0 + k < n ? k0 + k : n - 1), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
      for (int k = 0; k < kRead; ++k) {
        const uint32_t hi = (uint32_t)(w[k] >> 32);
        if (open && hi == kFinished) kp = k;
        open = open && hi < kFinished;
      }
      if (kp >= 0) {
        float v = 0.f;
#pragma unroll
        for (int k = kRead - 1; k >= 0; --k) {
          const float val = __builtin_bit_cast(float, (uint32_t)w[k]);
          const float A = __builtin_bit_cast(float, (uint32_t)(w[k] >> 32));
          v = k == kp ? val : k < kp ? fmaf(A, v, val) : v;
        }
#pragma unroll 1
        for (int k = k0 - 1; k >= 0; --k) {
          const uint64_t q = stash[k * ld];
          v = fmaf(__builtin_bit_cast(float, (uint32_t)(q >> 32)), v, __builtin_bit_cast(float, (uint32_t)q));
        }
        return v;
      }
      if (!open) break;
#pragma unroll
      for (int k = 0; k < kRead; ++k) stash[(k0 + k) * ld] = w[k];
    }
    __builtin_amdgcn_s_sleep(2);
  }
}

// V elements of one row at byte offset off (per lane) + so (per wave), in one
// access of 2, 4, 8 or 16 bytes.  A lane without channels passes kNowhere: its
// reads give zero and its stores are dropped.  AUX: the cache policy (0 or
// kNonTemporal).
constexpr uint32_t kNowhere = 0xFFFFFF00u; // past every range
template <typename T, int V, int AUX> struct Row {
  static constexpr int kBytes = V * (int)sizeof(T);
  static constexpr int W = kBytes < 4 ? 1 : kBytes / 4; // 32-bit words held
  static_assert(kBytes == 2 || kBytes == 4 || kBytes == 8 || kBytes == 16, "one access");
  uint32_t d[W];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int e = 0; e < W; ++e) d[e] = 0;
  }
  // A gate of -infinity: s = 0 whatever the bias is (see chan_of), so a = 1 and
  // beta = 0 for every finite A; a token that does not exist passes the state on.
  __device__ __forceinline__ void shut() {
#pragma unroll
    for (int e = 0; e < W; ++e) d[e] = sizeof(T) == 4 ? 0xFF800000u : V == 1 ? 0xFF80u : 0xFF80FF80u;
  }
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off, int so) {
    if constexpr (W == 4) {
      const i32x4 v = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, so, AUX));
      d[0] = (uint32_t)v[0], d[1] = (uint32_t)v[1], d[2] = (uint32_t)v[2], d[3] = (uint32_t)v[3];
    } else if constexpr (W == 2) {
      const i32x2 v = __builtin_bit_cast(i32x2, __builtin_amdgcn_raw_buffer_load_b64(r, (int)off, so, AUX));
      d[0] = (uint32_t)v[0], d[1] = (uint32_t)v[1];
    } else if constexpr (kBytes == 4) {
      d[0] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, (int)off, so, AUX);
    } else {
      d[0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)off, so, AUX);
    }
  }
  // Makes the value opaque here, so that nothing computed from it is moved
  // above: the compiler otherwise unpacks every row early and runs out of
  // registers.
  __device__ __forceinline__ void pin() {
#pragma unroll
    for (int e = 0; e < W; ++e) __asm__ volatile("" : "+v"(d[e]));
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (sizeof(T) == 4) return __builtin_bit_cast(float, d[e]);
    else return __builtin_bit_cast(float, (e & 1) ? (d[e >> 1] & 0xFFFF0000u) : (d[e >> 1] << 16));
  }
};

// Stores V values, rounded once to T.
template <typename T, int V, int AUX>
__device__ __forceinline__ void store_row(__amdgpu_buffer_rsrc_t r, uint32_t off, int so, const float *v) {
  constexpr int W = Row<T, V, AUX>::W;
  if constexpr (Row<T, V, AUX>::kBytes == 2) {
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(short, (__bf16)v[0]), r, (int)off, so, AUX);
  } else {
    int d[W];
#pragma unroll
    for (int k = 0; k < W; ++k) {
      if constexpr (sizeof(T) == 2) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        bf16x2 t;
        t[0] = (__bf16)v[2 * k], t[1] = (__bf16)v[2 * k + 1];
        d[k] = __builtin_bit_cast(int, t);
      } else {
        d[k] = __builtin_bit_cast(int, v[k]);
      }
    }
    if constexpr (W == 4) {
      const i32x4 t = {d[0], d[1], d[2], d[3]};
      __builtin_amdgcn_raw_buffer_store_b128(t, r, (int)off, so, AUX);
    } else {
      __builtin_amdgcn_raw_buffer_store_b32(d[0], r, (int)off, so, AUX);
    }
  }
}

// sigmoid(v + bias) from v and nb = -bias * log2(e).
__device__ __forceinline__ float sigmoid1(float v, float nb) {
  return __builtin_amdgcn_rcpf(1.f + hw_exp2(fmaf(v, -kLog2e, nb)));
}

// beta = sqrt(1 - a^2) from l = log2(a) and a.  Near a = 1 the subtraction
// cancels: with y = 2 ln(a) in (-1/4, 0], 1 - a^2 = -y (1 + y/2 + y^2/6 + ...) to
// y^6/720 (remainder below 5e-8 of the sum); elsewhere 1 - a^2 itself is good to
// 4e-7.  Its root halves both.  For A > 0 it is 0.
__device__ __forceinline__ float beta_any(float l, float a) {
  const float y = l * (2.f * kLn2);
  float p = fmaf(y, 1.f / 720.f, 1.f / 120.f);
  p = fmaf(p, y, 1.f / 24.f);
  p = fmaf(p, y, 1.f / 6.f);
  p = fmaf(p, y, 0.5f);
  p = fmaf(p, y, 1.f);
  const float q = y > -0.25f ? -y * p : fmaf(-a, a, 1.f);
  return __builtin_amdgcn_sqrtf(q < 0.f ? 0.f : q);
}

// One token's gates of one channel.  SMALL: |A| <= 1/2, so y = 2 A s > -1 and
// beta = sqrt(-2 A) sqrt(s) g(l) with g = sqrt((1 - e^y) / -y), a fifth-degree
// minimax polynomial in l = y / 2 ln 2 (off by 2.4e-9, evaluated to 2^-24 * 1.3);
// sqrt(s) = 1 / sqrt(1 + e^-v) then costs no root of its own: five
// transcendentals a token instead of six, and no selection.
struct Chan {
  float A2, K, nrb, nib; // A log2 e, sqrt(-2 A), -bias * log2 e
};
struct Gate {
  float s, a, beta;
};
template <bool SMALL> __device__ __forceinline__ Gate gate_of(const Chan &c, float r) {
  Gate g;
  const float e1 = 1.f + hw_exp2(fmaf(r, -kLog2e, c.nrb));
  if constexpr (SMALL) {
    const float t = __builtin_amdgcn_rsqf(e1);
    g.s = t * t;
    const float l = c.A2 * g.s;
    g.a = hw_exp2(l);
    float p = fmaf(l, 0x1.391178p-12f, 0x1.972de2p-9f);
    p = fmaf(p, l, 0x1.54a87ep-6f);
    p = fmaf(p, l, 0x1.99f8aep-4f);
    p = fmaf(p, l, 0x1.62e42p-2f);
    p = fmaf(p, l, 1.f);
    g.beta = c.K * t * p;
  } else {
    g.s = __builtin_amdgcn_rcpf(e1);
    const float l = c.A2 * g.s;
    g.a = hw_exp2(l);
    g.beta = beta_any(l, g.a);
  }
  return g;
}
// An r_bias of +infinity counts as one of 2.4e38: the gate is open for every r
// above -2^127, and an r of -infinity leaves it shut, where inf - inf would be NaN
// (a NaN bias stays one): a token that does not exist has such an r.  Choosing a =
// 1, beta = 0 for those tokens instead costs 2 to 4 % of the bf16 backward (b4
// L2048 D5120 158 to 161 us against 154).
__device__ __forceinline__ Chan chan_of(float A, float rbias, float ibias) {
  Chan k;
  k.A2 = A * kLog2e;
  k.K = __builtin_amdgcn_sqrtf(fmaxf(-2.f * A, 0.f));
  k.nrb = __builtin_elementwise_maximum(-kLog2e * rbias, -FLT_MAX);
  k.nib = -kLog2e * ibias;
  return k;
}
__device__ __forceinline__ bool small_decay(float A2) { return fabsf(A2) <= 0.5f * kLog2e; }

// Where this workgroup is: chunk, batch row, channel tile.
struct Place {
  int chunk, row, tile;
};
__device__ __forceinline__ Place take_place(const GlrParams &p, bool back) {
  uint32_t t = blockIdx.x;
  if (p.words) {
    __shared__ uint32_t ticket;
    // the counter starts at the fill value, one before 0
    if (threadIdx.x == 0) ticket = atomicAdd(p.ticket, 1u) + 1u;
    __syncthreads();
    t = ticket;
  }
  t = __builtin_amdgcn_readfirstlane(t);
  const uint32_t per = (uint32_t)p.b * (uint32_t)p.ntile;
  const uint32_t j = t / per, q = t - j * per;
  Place pl;
  pl.chunk = back ? p.nchunk - 1 - (int)j : (int)j;
  pl.row = (int)(q / (uint32_t)p.ntile);
  pl.tile = (int)(q - (uint32_t)pl.row * (uint32_t)p.ntile);
  return pl;
}

__device__ __forceinline__ int row_length(const GlrParams &p, int row) {
  if (!p.lengths) return p.L;
  const int n = p.lengths[row];
  return n < 0 ? 0 : n > p.L ? p.L : n;
}

// Byte range of `nt` rows of a strided tensor, from the first one's start to
// the last one's end.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const void *base, int64_t first, int64_t stride, int nt,
                                                            int D, int es) {
  const char *q = (const char *)base + first * es;
  return make_rsrc(q, nt > 0 ? (uint32_t)(((int64_t)(nt - 1) * stride + D) * es) : 0u);
}

// ---------------------------------------------------------------------------
// Forward.  A wave takes TT successive tokens of the tile's channels, a lane V
// of them.  31 vector instructions an element, 5 of them transcendental (two
// issue slots each).  b4 L4096 D5120 bf16, 671 MB: a call with its fill takes 147
// us (4.6 TB/s; in a loop over three sets of inputs 155; the kernel alone, under
// the profiler, 154, at best 144), where a large copy reaches 5.1 TB/s.  HBM moves
// 1.04 times the inputs and outputs (the rest are chain words), the vector ALU is
// busy 53 % of the time.  The same kernel without gates, look back and ticket
// takes 138 of the 147: what is left is the wait at the two barriers and the tail
// of the chain.
// ---------------------------------------------------------------------------
template <typename T, int V, int NW, bool CUT, int AUX>
__global__ __launch_bounds__(64 * NW) void glr_fwd_kernel(GlrParams p) {
  constexpr int kTile = 64 * V, TT = kFwdTokens, kChunk = NW * TT, ES = (int)sizeof(T);
  __shared__ float aggA[NW][kTile], aggw[NW][kTile], carry[NW][kTile];
  __shared__ int aggcut[NW];
  __shared__ uint64_t stash[kWindow][kTile];
  const Place pl = take_place(p, false);
  const int len = row_length(p, pl.row);
  const int t0 = pl.chunk * kChunk;
  if (pl.chunk > 0 && t0 >= len) return; // nothing here, and nothing after it
  const int nt = min(kChunk, len - t0);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c0 = pl.tile * kTile + lane * V; // V divides D: all of a lane's channels exist or none
  const int lt0 = wave * TT, ntw = max(0, min(TT, nt - lt0)); // the wave's first token, its tokens that exist
  const uint32_t off = c0 < p.D ? (uint32_t)(c0 * ES) : kNowhere;

  const __amdgpu_buffer_rsrc_t rx = rows_rsrc(p.x, pl.row * p.xb + (int64_t)t0 * p.xt, p.xt, nt, p.D, ES);
  const __amdgpu_buffer_rsrc_t rr = rows_rsrc(p.r, pl.row * p.rb_ + (int64_t)t0 * p.rt, p.rt, nt, p.D, ES);
  const __amdgpu_buffer_rsrc_t ri = rows_rsrc(p.i, pl.row * p.ib_ + (int64_t)t0 * p.it, p.it, nt, p.D, ES);
  Row<T, V, AUX> vx[TT], vr[TT], vi[TT];
  if (ntw == TT) {
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      vr[j].load(rr, off, (lt0 + j) * p.rt * ES);
      vi[j].load(ri, off, (lt0 + j) * p.it * ES);
      vx[j].load(rx, off, (lt0 + j) * p.xt * ES);
    }
  } else {
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      if (j < ntw) {
        vr[j].load(rr, off, (lt0 + j) * p.rt * ES);
        vi[j].load(ri, off, (lt0 + j) * p.it * ES);
        vx[j].load(rx, off, (lt0 + j) * p.xt * ES);
      } else {
        vr[j].shut(), vi[j].zero(), vx[j].zero();
      }
    }
  }
  // bit j: the wave's token j is a reset
  uint64_t resets = 0;
  if constexpr (CUT)
    resets = __ballot(lane < ntw && p.reset[(int64_t)pl.row * p.L + t0 + lt0 + (lane < ntw ? lane : 0)] != 0);
  Chan ch[V];
  bool sm = true;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const int c = min(c0 + e, p.D - 1);
    ch[e] = chan_of(p.A[c], p.rbias ? p.rbias[c] : 0.f, p.ibias ? p.ibias[c] : 0.f);
    sm = sm && small_decay(ch[e].A2);
  }

  const bool small = __all(sm); // the same for every wave: they share the tile's channels

  // the wave's own map
  float a[TT][V], b[TT][V], A[V], w[V];
#pragma unroll
  for (int e = 0; e < V; ++e) A[e] = 1.f, w[e] = 0.f;
  constexpr int GR = TT < kTogether ? TT : kTogether;
#pragma unroll
  for (int j0 = 0; j0 < TT; j0 += GR) {
    if (j0 >= ntw) continue;
    float beta[GR][V];
#pragma unroll
    for (int j = j0; j < j0 + GR; ++j) vr[j].pin(), vi[j].pin(), vx[j].pin();
    if (small) {
#pragma unroll
      for (int j = 0; j < GR; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const Gate g = gate_of<true>(ch[e], vr[j0 + j].get(e));
          a[j0 + j][e] = g.a, beta[j][e] = g.beta;
        }
    } else {
#pragma unroll
      for (int j = 0; j < GR; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const Gate g = gate_of<false>(ch[e], vr[j0 + j].get(e));
          a[j0 + j][e] = g.a, beta[j][e] = g.beta;
        }
    }
#pragma unroll
    for (int j = j0; j < j0 + GR; ++j) {
      const bool rs = CUT && ((resets >> j) & 1);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float u = sigmoid1(vi[j].get(e), ch[e].nib) * vx[j].get(e);
        a[j][e] = rs ? 0.f : a[j][e];
        b[j][e] = rs ? u : beta[j - j0][e] * u;
        A[e] *= a[j][e];
        w[e] = rs ? u : fmaf(a[j][e], w[e], b[j][e]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < V; ++e) aggA[wave][lane * V + e] = A[e], aggw[wave][lane * V + e] = w[e];
  if (CUT && lane == 0) aggcut[wave] = resets != 0;
  __syncthreads();

  // between waves and chunks: one thread per channel of the tile
  if (tid < kTile) {
    const int c = pl.tile * kTile + tid;
    const bool live = c < p.D;
    float cA = 1.f, cw = 0.f;
    bool ccut = false;
#pragma unroll
    for (int v = 0; v < NW; ++v) {
      const bool k = CUT && aggcut[v];
      cw = k ? aggw[v][tid] : fmaf(aggA[v][tid], cw, aggw[v][tid]);
      cA *= aggA[v][tid];
      ccut = ccut || k;
    }
    const int last = len > 0 ? (len - 1) / kChunk : 0;
    float h = 0.f;
    if (live) {
      uint64_t *word = nullptr;
      if (p.words) word = p.words + ((int64_t)pl.row * p.nchunk + pl.chunk) * p.wstride + c;
      const bool more = pl.chunk < last;
      // A chunk with a reset hands on a finished state at once, unless the
      // final state overwrites the initial one: then "finished" also says
      // that chunk 0 has read it.
      const bool early = ccut && !p.inplace;
      if (pl.chunk == 0) {
        h = p.init ? p.init[(int64_t)pl.row * p.D + c] : 0.f;
      } else {
        if (more && early) publish(word, make_word(kFinished, cw));
        else if (more && !ccut) publish(word, make_word(decay_bits(cA), cw));
        h = look_back(word - p.wstride, -p.wstride, pl.chunk, &stash[0][tid], kTile);
      }
      // the initial state has been read before anything is published
      if (p.inplace) __asm__ volatile("" ::"v"(h) : "memory");
      const float hend = ccut ? cw : fmaf(cA, h, cw);
      if (more && !(early && pl.chunk > 0)) publish(word, make_word(kFinished, hend));
      if (p.fin && pl.chunk == last) p.fin[(int64_t)pl.row * p.D + c] = hend;
    }
#pragma unroll
    for (int v = 0; v < NW; ++v) {
      carry[v][tid] = h;
      h = CUT && aggcut[v] ? aggw[v][tid] : fmaf(aggA[v][tid], h, aggw[v][tid]);
    }
  }
  __syncthreads();

  // the states, from the one entering the wave's tokens
  float h[V];
#pragma unroll
  for (int e = 0; e < V; ++e) h[e] = carry[wave][lane * V + e];
  if (p.states && (t0 + lt0) % kGlrSegment == 0 && (ntw > 0 || t0 + lt0 == 0)) {
    const int64_t nseg = (p.L + kGlrSegment - 1) / kGlrSegment;
    float *s = p.states + ((int64_t)pl.row * nseg + (t0 + lt0) / kGlrSegment) * p.D + c0;
    if (c0 < p.D) {
#pragma unroll
      for (int e = 0; e < V; ++e) s[e] = h[e];
    }
  }
  if (!p.out) return;
  const __amdgpu_buffer_rsrc_t ro = rows_rsrc(p.out, ((int64_t)pl.row * p.L + t0) * p.D, p.D, nt, p.D, ES);
#pragma unroll
  for (int j = 0; j < TT; ++j)
    if (j < ntw) {
      const bool rs = CUT && ((resets >> j) & 1);
#pragma unroll
      for (int e = 0; e < V; ++e) h[e] = rs ? b[j][e] : fmaf(a[j][e], h[e], b[j][e]);
      store_row<T, V, AUX>(ro, off, (lt0 + j) * p.D * ES, h);
    }
}

// ---------------------------------------------------------------------------
// Backward.  Chunks of kGlrSegment tokens, entering state given; the chain runs
// from the last chunk to the first.  4 tensors read, 3 written.  Only the decay,
// beta and the state before each token are kept per element; the gates are formed
// once more for the gradients, which costs less than the registers to keep them
// (two workgroups a compute unit instead of one: b4 L2048 D5120 bf16 150 us
// against 227).  587 MB at 3.9 TB/s; the vector ALU is busy 61 % of the time
// (74 instructions an element).  TD is the type of dout: with bf16 inputs also
// the fp32 of ssd_scan_bwd's gradients.  That takes eight registers more; held to
// four waves a SIMD it keeps four to seven in scratch (the same case 178 us, not
// held 224, with a cast to bf16 before 185).
// ---------------------------------------------------------------------------
template <typename T, typename TD, int V, int NW, bool CUT, int AUX>
__global__ __launch_bounds__(64 * NW, sizeof(TD) > sizeof(T) ? 4 : 1) void glr_bwd_kernel(GlrParams p) {
  constexpr int kTile = 64 * V, TT = kBwdTokens, kChunk = NW * TT, ES = (int)sizeof(T), ESD = (int)sizeof(TD);
  __shared__ float fA[NW][kTile], fw[NW][kTile], bA[NW][kTile], bw[NW][kTile];
  __shared__ float fcarry[NW][kTile], bcarry[NW][kTile];
  __shared__ int aggcut[NW];
  __shared__ uint64_t stash[kWindow][kTile];
  const Place pl = take_place(p, true);
  const int len = row_length(p, pl.row);
  const int t0 = pl.chunk * kChunk;
  const int last = len > 0 ? (len - 1) / kChunk : 0;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lt0 = wave * TT;
  const int nt = max(0, min(kChunk, len - t0)); // rows that exist
  const int ntw = max(0, min(TT, nt - lt0));
  const int ntp = min(kChunk, p.L - t0), ntpw = max(0, min(TT, ntp - lt0)); // rows of the gradients
  const int c0 = pl.tile * kTile + lane * V; // V divides D: all of a lane's channels exist or none
  const uint32_t off = c0 < p.D ? (uint32_t)(c0 * ES) : kNowhere;
  const uint32_t offd = c0 < p.D ? (uint32_t)(c0 * ESD) : kNowhere;
  const int64_t prow = ((int64_t)pl.row * p.nchunk + pl.chunk) * 3 * p.D; // row of the partial sums
  const int64_t g0 = ((int64_t)pl.row * p.L + t0) * p.D;
  const __amdgpu_buffer_rsrc_t odx = rows_rsrc(p.dx, g0, p.D, ntp, p.D, ES);
  const __amdgpu_buffer_rsrc_t odr = rows_rsrc(p.dr, g0, p.D, ntp, p.D, ES);
  const __amdgpu_buffer_rsrc_t odi = rows_rsrc(p.di, g0, p.D, ntp, p.D, ES);
  float zero[V];
#pragma unroll
  for (int e = 0; e < V; ++e) zero[e] = 0.f;

  // behind the row's length: zero gradients
  for (int j = ntw; j < ntpw; ++j) {
    store_row<T, V, AUX>(odx, off, (lt0 + j) * p.D * ES, zero);
    store_row<T, V, AUX>(odr, off, (lt0 + j) * p.D * ES, zero);
    store_row<T, V, AUX>(odi, off, (lt0 + j) * p.D * ES, zero);
  }
  if (pl.chunk > last) {
    for (int k = tid; k < 3 * kTile && p.part; k += 64 * NW) {
      const int c = pl.tile * kTile + k % kTile;
      if (c < p.D) p.part[prow + (int64_t)(k / kTile) * p.D + c] = 0.f;
    }
    return;
  }

  const __amdgpu_buffer_rsrc_t rx = rows_rsrc(p.x, pl.row * p.xb + (int64_t)t0 * p.xt, p.xt, nt, p.D, ES);
  const __amdgpu_buffer_rsrc_t rr = rows_rsrc(p.r, pl.row * p.rb_ + (int64_t)t0 * p.rt, p.rt, nt, p.D, ES);
  const __amdgpu_buffer_rsrc_t ri = rows_rsrc(p.i, pl.row * p.ib_ + (int64_t)t0 * p.it, p.it, nt, p.D, ES);
  const __amdgpu_buffer_rsrc_t rd = rows_rsrc(p.dout, pl.row * p.db + (int64_t)t0 * p.dt, p.dt, nt, p.D, ESD);
  Row<T, V, AUX> vx[TT], vr[TT], vi[TT];
  Row<TD, V, AUX> vd[TT];
  if (ntw == TT) {
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      vr[j].load(rr, off, (lt0 + j) * p.rt * ES);
      vi[j].load(ri, off, (lt0 + j) * p.it * ES);
      vx[j].load(rx, off, (lt0 + j) * p.xt * ES);
      vd[j].load(rd, offd, (lt0 + j) * p.dt * ESD);
    }
  } else {
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      if (j < ntw) {
        vr[j].load(rr, off, (lt0 + j) * p.rt * ES);
        vi[j].load(ri, off, (lt0 + j) * p.it * ES);
        vx[j].load(rx, off, (lt0 + j) * p.xt * ES);
        vd[j].load(rd, offd, (lt0 + j) * p.dt * ESD);
      } else {
        vr[j].shut(), vi[j].zero(), vx[j].zero(), vd[j].zero();
      }
    }
  }
  uint64_t resets = 0;
  if constexpr (CUT)
    resets = __ballot(lane < ntw && p.reset[(int64_t)pl.row * p.L + t0 + lt0 + (lane < ntw ? lane : 0)] != 0);
  Chan ch[V];
  bool sm = true;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const int c = min(c0 + e, p.D - 1);
    ch[e] = chan_of(p.A[c], p.rbias ? p.rbias[c] : 0.f, p.ibias ? p.ibias[c] : 0.f);
    sm = sm && small_decay(ch[e].A2);
  }

  const bool small = __all(sm); // the same for every wave: they share the tile's channels

  // decay, factor and input of every token; the wave's map
  float a[TT][V], be[TT][V], b[TT][V], A[V], w[V], wb[V];
#pragma unroll
  for (int e = 0; e < V; ++e) A[e] = 1.f, w[e] = 0.f, wb[e] = 0.f;
  constexpr int GR = TT < kTogether ? TT : kTogether;
#pragma unroll
  for (int j0 = 0; j0 < TT; j0 += GR) {
    if (j0 >= ntw) { // these tokens pass both walks on
#pragma unroll
      for (int j = j0; j < j0 + GR; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) a[j][e] = 1.f, be[j][e] = b[j][e] = 0.f;
      continue;
    }
#pragma unroll
    for (int j = j0; j < j0 + GR; ++j) vr[j].pin(), vi[j].pin(), vx[j].pin();
    if (small) {
#pragma unroll
      for (int j = j0; j < j0 + GR; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const Gate g = gate_of<true>(ch[e], vr[j].get(e));
          a[j][e] = g.a, be[j][e] = g.beta;
        }
    } else {
#pragma unroll
      for (int j = j0; j < j0 + GR; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const Gate g = gate_of<false>(ch[e], vr[j].get(e));
          a[j][e] = g.a, be[j][e] = g.beta;
        }
    }
#pragma unroll
    for (int j = j0; j < j0 + GR; ++j) {
      const bool rs = CUT && ((resets >> j) & 1);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (rs) a[j][e] = 0.f, be[j][e] = 1.f;
        b[j][e] = be[j][e] * (sigmoid1(vi[j].get(e), ch[e].nib) * vx[j].get(e));
        A[e] *= a[j][e];
        w[e] = rs ? b[j][e] : fmaf(a[j][e], w[e], b[j][e]);
      }
    }
  }
#pragma unroll
  for (int j = TT - 1; j >= 0; --j) {
    const bool rs = CUT && ((resets >> j) & 1);
#pragma unroll
    for (int e = 0; e < V; ++e) wb[e] = rs ? 0.f : a[j][e] * (vd[j].get(e) + wb[e]);
  }
#pragma unroll
  for (int e = 0; e < V; ++e) {
    fA[wave][lane * V + e] = A[e], fw[wave][lane * V + e] = w[e];
    bw[wave][lane * V + e] = wb[e];
  }
  if (CUT && lane == 0) aggcut[wave] = resets != 0;
  __syncthreads();

  if (tid < kTile) {
    const int c = pl.tile * kTile + tid;
    const bool live = c < p.D;
    float cA = 1.f, cw = 0.f;
    bool ccut = false;
#pragma unroll
    for (int v = NW - 1; v >= 0; --v) {
      const bool k = CUT && aggcut[v];
      cw = k ? bw[v][tid] : fmaf(fA[v][tid], cw, bw[v][tid]);
      cA *= fA[v][tid];
      ccut = ccut || k;
    }
    float cin = 0.f, h = 0.f;
    if (live) {
      uint64_t *word = nullptr;
      if (p.words) word = p.words + ((int64_t)pl.row * p.nchunk + pl.chunk) * p.wstride + c;
      const bool more = pl.chunk > 0;
      h = p.states[((int64_t)pl.row * p.nchunk + pl.chunk) * p.D + c];
      if (pl.chunk == last) {
        cin = p.dfin ? p.dfin[(int64_t)pl.row * p.D + c] : 0.f;
      } else {
        if (more) publish(word, ccut ? make_word(kFinished, cw) : make_word(decay_bits(cA), cw));
        cin = look_back(word + p.wstride, p.wstride, last - pl.chunk, &stash[0][tid], kTile);
      }
      const float cend = ccut ? cw : fmaf(cA, cin, cw);
      if (more && !(ccut && pl.chunk != last)) publish(word, make_word(kFinished, cend));
      if (p.dinit && pl.chunk == 0) p.dinit[(int64_t)pl.row * p.D + c] = cend;
    }
#pragma unroll
    for (int v = NW - 1; v >= 0; --v) {
      bcarry[v][tid] = cin;
      cin = CUT && aggcut[v] ? bw[v][tid] : fmaf(fA[v][tid], cin, bw[v][tid]);
    }
#pragma unroll
    for (int v = 0; v < NW; ++v) {
      fcarry[v][tid] = h;
      h = CUT && aggcut[v] ? fw[v][tid] : fmaf(fA[v][tid], h, fw[v][tid]);
    }
  }
  __syncthreads();

  // the states before each token, in the place of the inputs
  float c[V], sA[V], sr[V], si[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    float h = fcarry[wave][lane * V + e];
    c[e] = bcarry[wave][lane * V + e];
    sA[e] = sr[e] = si[e] = 0.f;
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      const float n = CUT && ((resets >> j) & 1) ? b[j][e] : fmaf(a[j][e], h, b[j][e]);
      b[j][e] = h;
      h = n;
    }
  }
  // the gates once more: less than it costs to keep them
#pragma unroll
  for (int j = TT - 1; j >= 0; --j) {
    if (j >= ntw) continue; // passes c on and adds nothing to the sums
    float ox[V], orr[V], oi[V];
    const bool rs = CUT && ((resets >> j) & 1);
    vr[j].pin(), vi[j].pin(), vx[j].pin(), vd[j].pin();
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float g = vd[j].get(e) + c[e];
      // capped, so that 1 - s = e s and 1 - gi = e gi stay finite (a NaN stays one)
      const float er = __builtin_elementwise_minimum(hw_exp2(fmaf(vr[j].get(e), -kLog2e, ch[e].nrb)), 0x1p120f);
      const float ei = __builtin_elementwise_minimum(hw_exp2(fmaf(vi[j].get(e), -kLog2e, ch[e].nib)), 0x1p120f);
      const float sg = __builtin_amdgcn_rcpf(1.f + er), gi = __builtin_amdgcn_rcpf(1.f + ei);
      const float x = vx[j].get(e), ak = a[j][e], beta = be[j][e];
      const float rb = beta > 0.f ? __builtin_amdgcn_rcpf(beta) : 0.f;
      const float ag = ak * g;
      const float dl = ag * fmaf(-ak * (gi * x), rb, b[j][e]); // at log a
      ox[e] = g * beta * gi;
      oi[e] = ox[e] * x * (ei * gi);
      float ds = dl * sg;
      orr[e] = ds * (er * sg) * (ch[e].A2 * kLn2);
      c[e] = ag;
      if (CUT && rs) orr[e] = ds = c[e] = 0.f;
      sA[e] += ds;
      sr[e] += orr[e];
      si[e] += oi[e];
    }
    store_row<T, V, AUX>(odx, off, (lt0 + j) * p.D * ES, ox);
    store_row<T, V, AUX>(odr, off, (lt0 + j) * p.D * ES, orr);
    store_row<T, V, AUX>(odi, off, (lt0 + j) * p.D * ES, oi);
  }
  // parameter gradients: the waves' sums in a fixed order (fA, fw and bA are
  // read no more once every wave has its carries)
  if (!p.part) return;
  __syncthreads();
#pragma unroll
  for (int e = 0; e < V; ++e) {
    fA[wave][lane * V + e] = sA[e];
    fw[wave][lane * V + e] = sr[e];
    bA[wave][lane * V + e] = si[e];
  }
  __syncthreads();
  for (int k = tid; k < 3 * kTile; k += 64 * NW) {
    const int cl = k % kTile, what = k / kTile;
    const float (*src)[kTile] = what == 0 ? fA : what == 1 ? fw : bA;
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < NW; ++v) s += src[v][cl];
    if (pl.tile * kTile + cl < p.D) p.part[prow + (int64_t)what * p.D + pl.tile * kTile + cl] = s;
  }
}

// Sum of the chunks' partial rows [n][3][D] in a fixed order, in 64 bits.
constexpr int kSumRows = 16;
__global__ __launch_bounds__(64 * kSumRows) void glr_sum_kernel(const float *part, int n, int D, float *dA, float *drb,
                                                                float *dib) {
  __shared__ double acc[kSumRows][64];
  const int lane = threadIdx.x & 63, row = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 64 + lane, width = 3 * (int64_t)D;
  double s = 0.;
  if (col < width)
    for (int k = row; k < n; k += kSumRows) s += part[k * width + col];
  acc[row][lane] = s;
  __syncthreads();
  if (row == 0 && col < width) {
#pragma unroll
    for (int k = 1; k < kSumRows; ++k) s += acc[k][lane];
    const int what = (int)(col / D), c = (int)(col - (int64_t)what * D);
    float *o = what == 0 ? dA : what == 1 ? drb : dib;
    if (o) o[c] = (float)s;
  }
}

// Workspace words to kNotYet and the ticket to one before 0 (one kernel, so
// that a captured call replays).
__global__ __launch_bounds__(256) void glr_fill_kernel(uint4 *p, int64_t n) {
  const uint4 v = make_uint4(kNotYet, kNotYet, kNotYet, kNotYet);
  for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < n; k += (int64_t)gridDim.x * 256) p[k] = v;
}

// V floats, 16 bytes at a time.
template <int V> __device__ __forceinline__ void load_f32(const float *p, float *v) {
  if constexpr (V == 1) {
    v[0] = p[0];
  } else {
#pragma unroll
    for (int e = 0; e < V; e += 4) {
      const float4 q = *reinterpret_cast<const float4 *>(p + e);
      v[e] = q.x, v[e + 1] = q.y, v[e + 2] = q.z, v[e + 3] = q.w;
    }
  }
}

// One token: V channels per lane; bound by the launch at small batches (b1 D2048:
// 2.4 us) and by latency and HBM (the fp32 state in and out) at large ones (b256
// D5120 bf16, 21 MB: 6.5 us).
template <typename T, int V> __global__ __launch_bounds__(256) void glr_step_kernel(GlrStepParams p) {
  constexpr int ES = (int)sizeof(T);
  const int row = (int)(blockIdx.x / (uint32_t)p.nblk);
  const int c0 = ((int)(blockIdx.x - (uint32_t)row * (uint32_t)p.nblk) * 256 + (int)threadIdx.x) * V;
  if (c0 >= p.D) return;
  Row<T, V, 0> vr, vi, vx;
  vr.load(rows_rsrc(p.r, row * p.rb_, 0, 1, p.D, ES), (uint32_t)(c0 * ES), 0);
  vi.load(rows_rsrc(p.i, row * p.ib_, 0, 1, p.D, ES), (uint32_t)(c0 * ES), 0);
  vx.load(rows_rsrc(p.x, row * p.xb, 0, 1, p.D, ES), (uint32_t)(c0 * ES), 0);
  const bool rs = p.reset && p.reset[row] != 0;
  const float *st = p.state + (int64_t)row * p.D + c0;
  float *ns = p.new_state + (int64_t)row * p.D + c0;
  float h[V], A[V], rb[V], ib[V];
  load_f32<V>(st, h);
  load_f32<V>(p.A + c0, A);
#pragma unroll
  for (int e = 0; e < V; ++e) rb[e] = ib[e] = 0.f;
  if (p.rbias) load_f32<V>(p.rbias + c0, rb);
  if (p.ibias) load_f32<V>(p.ibias + c0, ib);
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const Chan ch = chan_of(A[e], rb[e], ib[e]);
    const Gate g = gate_of<false>(ch, vr.get(e));
    const float u = sigmoid1(vi.get(e), ch.nib) * vx.get(e);
    h[e] = rs ? u : fmaf(g.a, h[e], g.beta * u);
  }
  if constexpr (V > 1) {
#pragma unroll
    for (int e = 0; e < V; e += 4) *reinterpret_cast<float4 *>(ns + e) = make_float4(h[e], h[e + 1], h[e + 2], h[e + 3]);
  } else {
    ns[0] = h[0];
  }
  store_row<T, V, 0>(rows_rsrc(p.out, (int64_t)row * p.D, 0, 1, p.D, ES), (uint32_t)(c0 * ES), 0, h);
}

template <typename T, typename TD, int V, int NW, int AUX> void launch_waves(bool back, const GlrParams &p, hipStream_t st) {
  const dim3 grid((uint32_t)p.b * (uint32_t)p.ntile * (uint32_t)p.nchunk);
  if (back) {
    if (p.reset) glr_bwd_kernel<T, TD, V, NW, true, AUX><<<grid, 64 * NW, 0, st>>>(p);
    else glr_bwd_kernel<T, TD, V, NW, false, AUX><<<grid, 64 * NW, 0, st>>>(p);
  } else {
    if (p.reset) glr_fwd_kernel<T, V, NW, true, AUX><<<grid, 64 * NW, 0, st>>>(p);
    else glr_fwd_kernel<T, V, NW, false, AUX><<<grid, 64 * NW, 0, st>>>(p);
  }
}
// x, r and i that take half of the 256 MB last-level cache pass it by; smaller
// ones find themselves there again.  In a loop over three sets of inputs, kept
// in the caches and passed by: b4 L4096 D5120 bf16 forward 159 and 155 us, b4 L2048
// forward and backward 247 and 239, b5 L1009 D1100 f32 forward 25.5 and 28.6.
constexpr int64_t kOnceBytes = (int64_t)128 << 20;

// As many waves as the rows need (b256 L32 D5120 bf16 forward: eight 119 us, four
// 88, two 84; b64 L17: eight 27, two 16; a workgroup has a thread for each of
// its 128 or 64 channels, so two at least).
template <typename T, typename TD, int V> hipError_t scan_launch(bool back, const GlrParams &p, hipStream_t st) {
  const int need = (p.L + (back ? kBwdTokens : kFwdTokens) - 1) / (back ? kBwdTokens : kFwdTokens);
  if (need <= 2) launch_waves<T, TD, V, 2, 0>(back, p, st);
  else if (need <= 4) launch_waves<T, TD, V, 4, 0>(back, p, st);
  else if ((int64_t)p.b * p.L * p.D * 3 * (int64_t)sizeof(T) < kOnceBytes) launch_waves<T, TD, V, kWaves, 0>(back, p, st);
  else launch_waves<T, TD, V, kWaves, kNonTemporal>(back, p, st);
  return hipGetLastError();
}

} // namespace

// Four bytes a lane (256 of a row per workgroup) where bf16 rows allow it;
// two where the width, a stride or a pointer is odd.
hipError_t launch_glr(int dtype, bool vec, bool back, const GlrParams &p0, hipStream_t st) {
  GlrParams p = p0;
  const int V = dtype == 1 && vec ? 2 : 1;
  p.ntile = (p.D + 64 * V - 1) / (64 * V);
  if (p.words) {
    // words and the ticket behind them, in 16-byte pieces
    const int64_t n = glr_chain_bytes(p.b, p.nchunk, p.D) / 16;
    const int64_t blocks = (n + 255) / 256;
    glr_fill_kernel<<<(uint32_t)(blocks < 2048 ? blocks : 2048), 256, 0, st>>>((uint4 *)p.words, n);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (dtype != 1) return scan_launch<float, float, 1>(back, p, st);
  if (back && p.dout_f32) return vec ? scan_launch<__bf16, float, 2>(back, p, st) : scan_launch<__bf16, float, 1>(back, p, st);
  return vec ? scan_launch<__bf16, __bf16, 2>(back, p, st) : scan_launch<__bf16, __bf16, 1>(back, p, st);
}

hipError_t launch_glr_sum(const float *part, int n, int D, float *dA, float *drb, float *dib, hipStream_t st) {
  glr_sum_kernel<<<(uint32_t)((3 * (int64_t)D + 63) / 64), 64 * kSumRows, 0, st>>>(part, n, D, dA, drb, dib);
  return hipGetLastError();
}

hipError_t launch_glr_step(int dtype, bool vec, const GlrStepParams &p0, hipStream_t st) {
  const int V = !vec ? 1 : dtype == 1 ? 8 : 4;
  GlrStepParams p = p0;
  p.nblk = (p.D + 256 * V - 1) / (256 * V);
  const uint32_t grid = (uint32_t)p.nblk * (uint32_t)p.b;
  if (dtype == 1) {
    if (vec) glr_step_kernel<__bf16, 8><<<grid, 256, 0, st>>>(p);
    else glr_step_kernel<__bf16, 1><<<grid, 256, 0, st>>>(p);
  } else {
    if (vec) glr_step_kernel<float, 4><<<grid, 256, 0, st>>>(p);
    else glr_step_kernel<float, 1><<<grid, 256, 0, st>>>(p);
  }
  return hipGetLastError();
}

} // namespace ssd
