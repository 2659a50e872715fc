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
// Decomposition.  A workgroup owns 64 channels (128 B of a bf16 row) of one
// batch row over one chunk of tokens.  A lane owns V channels (16 B) and T
// successive tokens; its data is read once into registers.  The lanes' maps
// are composed inside the wave by lane shuffles, between the waves through
// LDS, and between the chunks through one 64-bit word per (chunk, channel)
// in the workspace: a chunk publishes its own map as soon as it is known and
// the finished state once its predecessor's is; a later chunk looks back over
// kLook words at a time.  So the data crosses HBM once in each direction
// however the time axis is split.  The fold over words always runs forward
// from a finished state with one fma per chunk, the same operations that
// produced the words in between, so results do not depend on timing.
//
// Workgroups take their chunk from a ticket counter, chunks in time order:
// a workgroup waits only for lower tickets, which were handed to workgroups
// that already run, so every wait ends.
#include "ssd_device.h"
#include "ssd_internal.h"

namespace ssd {
namespace {

constexpr int kTile = 64; // channels of a workgroup
constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kLook = 8; // words examined per look back

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
__device__ __forceinline__ float look_back(const uint64_t *prev, int64_t step, int n) {
  for (;;) {
    uint64_t w[kLook];
#pragma unroll
    for (int k = 0; k < kLook; ++k)
      w[k] = __hip_atomic_load(prev + step * (k < n ? k : n - 1), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    int kp = -1;
    bool open = true;
#pragma unroll
    for (int k = 0; k < kLook; ++k) {
      const uint32_t hi = (uint32_t)(w[k] >> 32);
      if (open && hi == kFinished) kp = k;
      open = open && hi < kFinished;
    }
    if (kp >= 0) {
      float v = 0.f;
#pragma unroll
      for (int k = kLook - 1; k >= 0; --k) {
        const float val = __builtin_bit_cast(float, (uint32_t)w[k]);
        const float A = __builtin_bit_cast(float, (uint32_t)(w[k] >> 32));
        v = k == kp ? val : k < kp ? fmaf(A, v, val) : v;
      }
      return v;
    }
    __builtin_amdgcn_s_sleep(2);
  }
}

template <typename T> struct Geo; // V channels per lane (16 bytes)
template <> struct Geo<__bf16> { static constexpr int V = 8; };
template <> struct Geo<float> { static constexpr int V = 4; };

// V elements of one row.  VEC: one 16-byte access; otherwise V single ones
// (odd widths or strides).  Reads past the resource's range give zero.
template <typename T, bool VEC> struct Row;
template <> struct Row<__bf16, true> {
  i32x4 d;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    d = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
  }
  __device__ __forceinline__ float get(int e) const {
    const uint32_t w = (uint32_t)d[e >> 1];
    return __builtin_bit_cast(float, (e & 1) ? (w & 0xFFFF0000u) : (w << 16));
  }
};
template <> struct Row<float, true> {
  i32x4 d;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    d = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
  }
  __device__ __forceinline__ float get(int e) const {
    const int w = d[e]; // a bit cast of the vector's element itself reads element 0
    return __builtin_bit_cast(float, w);
  }
};
template <> struct Row<__bf16, false> {
  uint16_t d[8];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
#pragma unroll
    for (int e = 0; e < 8; ++e) d[e] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)(off + 2 * e), 0, 0);
  }
  __device__ __forceinline__ float get(int e) const { return __builtin_bit_cast(float, (uint32_t)d[e] << 16); }
};
template <> struct Row<float, false> {
  int d[4];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = (int)__builtin_amdgcn_raw_buffer_load_b32(r, (int)(off + 4 * e), 0, 0);
  }
  __device__ __forceinline__ float get(int e) const { return __builtin_bit_cast(float, d[e]); }
};

// Stores V values, rounded once to T; the first `n` of them if !VEC.  A lane
// whose row or channels do not exist passes n = 0.
constexpr uint32_t kNowhere = 0xFFFFFF00u; // an offset past every range: the store is dropped
template <typename T, bool VEC>
__device__ __forceinline__ void store_row(__amdgpu_buffer_rsrc_t r, uint32_t off, const float *v, int n) {
  constexpr int V = Geo<T>::V;
  if constexpr (VEC) {
    i32x4 d;
    if constexpr (V == 8) {
      bf16x8 t;
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = (__bf16)v[e];
      d = __builtin_bit_cast(i32x4, t);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) d[e] = __builtin_bit_cast(int, v[e]);
    }
    __builtin_amdgcn_raw_buffer_store_b128(d, r, (int)(n ? off : kNowhere), 0, 0);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const uint32_t o = e < n ? off + (uint32_t)(e * sizeof(T)) : kNowhere;
      if constexpr (V == 8)
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(short, (__bf16)v[e]), r, (int)o, 0, 0);
      else
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(int, v[e]), r, (int)o, 0, 0);
    }
  }
}

// sigmoid(v + bias) from v and nb = -bias * log2(e).  e is capped so that
// e * s stays finite: the backward forms 1 - s = e * s without cancellation.
struct Sig {
  float s, e;
};
__device__ __forceinline__ Sig sigmoid2(float v, float nb) {
  Sig g;
  g.e = fminf(hw_exp2(fmaf(v, -kLog2e, nb)), 0x1p120f);
  g.s = __builtin_amdgcn_rcpf(1.f + g.e);
  return g;
}
__device__ __forceinline__ float sigmoid1(float v, float nb) {
  return __builtin_amdgcn_rcpf(1.f + hw_exp2(fmaf(v, -kLog2e, nb)));
}

// 1 - a^2 from l = log2(a) <= 0 and a.  Near a = 1 the subtraction cancels:
// with y = 2 ln(a) in (-1/4, 0], -expm1(y) = -y (1 + y/2 + y^2/6 + ...) to
// y^6/720 (remainder below 5e-8 of the sum); elsewhere 1 - a^2 itself is good to
// 4e-7.  Its root halves both.  For A > 0 the result is clamped at 0.
__device__ __forceinline__ float one_minus_sq(float l, float a) {
  const float y = l * (2.f * kLn2);
  float p = fmaf(y, 1.f / 720.f, 1.f / 120.f);
  p = fmaf(p, y, 1.f / 24.f);
  p = fmaf(p, y, 1.f / 6.f);
  p = fmaf(p, y, 0.5f);
  p = fmaf(p, y, 1.f);
  const float q = y > -0.25f ? -y * p : fmaf(-a, a, 1.f);
  return fmaxf(q, 0.f);
}

// Exclusive composition of the lanes' maps over the TG token groups of a
// wave (lane = channel group + LPR * token group).  In: each lane's own map;
// out: the composed map of the earlier groups (identity for the first) and, in
// inc*, the inclusive one.  BACK runs over later groups instead.  cut: this
// lane's tokens hold a reset, so nothing passes through it.
template <int V, bool BACK, bool CUT>
__device__ __forceinline__ void wave_compose(float *A, float *w, bool &cut, float *exA, float *exw, bool &excut) {
  constexpr int LPR = 64 / V, TG = V;
  const int lane = threadIdx.x & 63, tg = lane / LPR;
#pragma unroll
  for (int k = 1; k < TG; k *= 2) {
    const bool take = BACK ? tg + k < TG : tg >= k;
    const int src = BACK ? lane + k * LPR : lane - k * LPR;
    bool c2 = false;
    if constexpr (CUT) c2 = __shfl((int)cut, src & 63) != 0;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float A1 = __shfl(A[e], src & 63), w1 = __shfl(w[e], src & 63);
      if (take && (!CUT || !cut)) {
        w[e] = fmaf(A[e], w1, w[e]);
        A[e] *= A1;
      }
    }
    if constexpr (CUT) cut = cut || (take && c2);
  }
  const bool first = BACK ? tg == TG - 1 : tg == 0;
  const int src = (BACK ? lane + LPR : lane - LPR) & 63;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float a1 = __shfl(A[e], src), w1 = __shfl(w[e], src);
    exA[e] = first ? 1.f : a1;
    exw[e] = first ? 0.f : w1;
  }
  excut = false;
  if constexpr (CUT) {
    const bool c1 = __shfl((int)cut, src) != 0;
    excut = !first && c1;
  }
}

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
// Forward.  Chunk of 256 tokens; T tokens per lane.  Bound by HBM (3 tensors
// read, 1 written) with the vector ALU close behind: about 50 full-rate slots
// an element, 24 of them in its six transcendentals.
// ---------------------------------------------------------------------------
template <typename T, bool VEC, bool CUT>
__global__ __launch_bounds__(kThreads) void glr_fwd_kernel(GlrParams p) {
  constexpr int V = Geo<T>::V, LPR = 64 / V, TG = V, TT = kGlrChunk / (kWaves * TG), ES = (int)sizeof(T);
  __shared__ float aggA[kWaves][kTile], aggw[kWaves][kTile], carry[kWaves][kTile];
  __shared__ int aggcut[kWaves];
  const Place pl = take_place(p, false);
  const int len = row_length(p, pl.row);
  const int t0 = pl.chunk * kGlrChunk;
  if (pl.chunk > 0 && t0 >= len) return; // nothing here, and nothing after it
  const int nt = min(kGlrChunk, len - t0);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int tg = lane / LPR, c0 = pl.tile * kTile + (lane % LPR) * V;
  const int nch = max(0, min(V, p.D - c0));
  const int lt0 = (wave * TG + tg) * TT; // this lane's first token in the chunk

  const __amdgpu_buffer_rsrc_t rx = rows_rsrc(p.x, pl.row * p.xb + (int64_t)t0 * p.xt, p.xt, nt, p.D, ES);
  const __amdgpu_buffer_rsrc_t rr = rows_rsrc(p.r, pl.row * p.rb_ + (int64_t)t0 * p.rt, p.rt, nt, p.D, ES);
  const __amdgpu_buffer_rsrc_t ri = rows_rsrc(p.i, pl.row * p.ib_ + (int64_t)t0 * p.it, p.it, nt, p.D, ES);
  Row<T, VEC> dx[TT], dr[TT], di[TT];
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    dr[j].load(rr, (uint32_t)(((lt0 + j) * p.rt + c0) * ES));
    di[j].load(ri, (uint32_t)(((lt0 + j) * p.it + c0) * ES));
    dx[j].load(rx, (uint32_t)(((lt0 + j) * p.xt + c0) * ES));
  }
  bool rs[TT];
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    rs[j] = false;
    if constexpr (CUT)
      if (lt0 + j < nt) rs[j] = p.reset[(int64_t)pl.row * p.L + t0 + lt0 + j] != 0;
  }
  float A2[V], nrb[V], nib[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const int c = min(c0 + e, p.D - 1);
    A2[e] = p.A[c] * kLog2e;
    nrb[e] = p.rbias ? -kLog2e * p.rbias[c] : 0.f;
    nib[e] = p.ibias ? -kLog2e * p.ibias[c] : 0.f;
  }

  // the lane's own maps
  float a[TT][V], b[TT][V], A[V], w[V];
#pragma unroll
  for (int e = 0; e < V; ++e) A[e] = 1.f, w[e] = 0.f;
  bool cut = false;
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    const bool gone = lt0 + j >= nt;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float l = A2[e] * sigmoid1(dr[j].get(e), nrb[e]);
      const float al = hw_exp2(l);
      const float q = CUT && rs[j] ? 1.f : one_minus_sq(l, al);
      const float u = sigmoid1(di[j].get(e), nib[e]) * dx[j].get(e);
      b[j][e] = gone ? 0.f : __builtin_amdgcn_sqrtf(q) * u;
      a[j][e] = gone ? 1.f : al;
      if (CUT && rs[j]) {
        a[j][e] = 0.f;
        A[e] = 0.f;
        w[e] = b[j][e];
      } else {
        A[e] *= a[j][e];
        w[e] = fmaf(a[j][e], w[e], b[j][e]);
      }
    }
    cut = cut || rs[j];
  }
  float exA[V], exw[V];
  bool excut;
  wave_compose<V, false, CUT>(A, w, cut, exA, exw, excut);
  if (tg == TG - 1) {
    const int cl = (lane % LPR) * V;
#pragma unroll
    for (int e = 0; e < V; ++e) aggA[wave][cl + e] = A[e], aggw[wave][cl + e] = w[e];
    if (CUT && lane == 63) aggcut[wave] = cut;
  }
  __syncthreads();

  // between waves and chunks: lane = channel of the tile
  if (wave == 0) {
    const int c = pl.tile * kTile + lane;
    const bool live = c < p.D;
    float cA = 1.f, cw = 0.f;
    bool ccut = false;
#pragma unroll
    for (int v = 0; v < kWaves; ++v) {
      const bool k = CUT && aggcut[v];
      cw = k ? aggw[v][lane] : fmaf(aggA[v][lane], cw, aggw[v][lane]);
      cA *= aggA[v][lane];
      ccut = ccut || k;
    }
    const int last = len > 0 ? (len - 1) / kGlrChunk : 0;
    float h = 0.f;
    if (live) {
      uint64_t *word = nullptr;
      const int64_t step = (int64_t)p.ntile * kTile;
      if (p.words) word = p.words + ((int64_t)pl.row * p.nchunk + pl.chunk) * step + c;
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
        h = look_back(word - step, -step, pl.chunk);
      }
      // the initial state has been read before anything is published
      if (p.inplace) __asm__ volatile("" ::"v"(h) : "memory");
      const float hend = ccut ? cw : fmaf(cA, h, cw);
      if (more && !(early && pl.chunk > 0)) publish(word, make_word(kFinished, hend));
      if (p.fin && pl.chunk == last) p.fin[(int64_t)pl.row * p.D + c] = hend;
    }
#pragma unroll
    for (int v = 0; v < kWaves; ++v) {
      carry[v][lane] = h;
      h = CUT && aggcut[v] ? aggw[v][lane] : fmaf(aggA[v][lane], h, aggw[v][lane]);
    }
  }
  __syncthreads();

  // the states, from the one entering the lane's tokens
  float h[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float hc = carry[wave][(lane % LPR) * V + e];
    h[e] = CUT && excut ? exw[e] : fmaf(exA[e], hc, exw[e]);
  }
  if (p.states && lt0 % kGlrSegment == 0 && (lt0 < nt || t0 + lt0 == 0)) {
    const int64_t nseg = (p.L + kGlrSegment - 1) / kGlrSegment;
    float *s = p.states + ((int64_t)pl.row * nseg + (t0 + lt0) / kGlrSegment) * p.D + c0;
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (e < nch) s[e] = h[e];
  }
  if (!p.out) return;
  const __amdgpu_buffer_rsrc_t ro = rows_rsrc(p.out, ((int64_t)pl.row * p.L + t0) * p.D, p.D, nt, p.D, ES);
#pragma unroll
  for (int j = 0; j < TT; ++j) {
#pragma unroll
    for (int e = 0; e < V; ++e) h[e] = CUT && rs[j] ? b[j][e] : fmaf(a[j][e], h[e], b[j][e]);
    store_row<T, VEC>(ro, (uint32_t)(((lt0 + j) * p.D + c0) * ES), h, lt0 + j < nt ? nch : 0);
  }
}

// ---------------------------------------------------------------------------
// Backward.  Chunk of 128 tokens, entering state given; the chain runs from
// the last chunk to the first.  4 tensors read, 3 written.
// ---------------------------------------------------------------------------
template <typename T, bool VEC, bool CUT>
__global__ __launch_bounds__(kThreads) void glr_bwd_kernel(GlrParams p) {
  constexpr int V = Geo<T>::V, LPR = 64 / V, TG = V, TT = kGlrSegment / (kWaves * TG), ES = (int)sizeof(T);
  __shared__ float fA[kWaves][kTile], fw[kWaves][kTile], bA[kWaves][kTile], bw[kWaves][kTile];
  __shared__ float fcarry[kWaves][kTile], bcarry[kWaves][kTile];
  __shared__ int aggcut[kWaves];
  __shared__ float psum[kWaves * TG / 2][3][kTile];
  const Place pl = take_place(p, true);
  const int len = row_length(p, pl.row);
  const int t0 = pl.chunk * kGlrSegment;
  const int last = len > 0 ? (len - 1) / kGlrSegment : 0;
  const int ntp = min(kGlrSegment, p.L - t0);        // rows of the gradients
  const int nt = max(0, min(kGlrSegment, len - t0)); // rows that exist
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int tg = lane / LPR, cl = (lane % LPR) * V, c0 = pl.tile * kTile + cl;
  const int nch = max(0, min(V, p.D - c0));
  const int lt0 = (wave * TG + tg) * TT;
  const int64_t prow = ((int64_t)pl.row * p.nchunk + pl.chunk) * 3 * p.D; // row of the partial sums
  const int64_t g0 = ((int64_t)pl.row * p.L + t0) * p.D;
  const __amdgpu_buffer_rsrc_t odx = rows_rsrc(p.dx, g0, p.D, ntp, p.D, ES);
  const __amdgpu_buffer_rsrc_t odr = rows_rsrc(p.dr, g0, p.D, ntp, p.D, ES);
  const __amdgpu_buffer_rsrc_t odi = rows_rsrc(p.di, g0, p.D, ntp, p.D, ES);

  if (pl.chunk > last) { // behind the row's length: zero gradients
    float z[V];
#pragma unroll
    for (int e = 0; e < V; ++e) z[e] = 0.f;
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      const uint32_t off = (uint32_t)(((lt0 + j) * p.D + c0) * ES);
      const int n = lt0 + j < ntp ? nch : 0;
      store_row<T, VEC>(odx, off, z, n);
      store_row<T, VEC>(odr, off, z, n);
      store_row<T, VEC>(odi, off, z, n);
    }
    if (tid < 3 * kTile) {
      const int c = pl.tile * kTile + tid % kTile;
      if (c < p.D) p.part[prow + (int64_t)(tid / kTile) * p.D + c] = 0.f;
    }
    return;
  }

  const __amdgpu_buffer_rsrc_t rx = rows_rsrc(p.x, pl.row * p.xb + (int64_t)t0 * p.xt, p.xt, nt, p.D, ES);
  const __amdgpu_buffer_rsrc_t rr = rows_rsrc(p.r, pl.row * p.rb_ + (int64_t)t0 * p.rt, p.rt, nt, p.D, ES);
  const __amdgpu_buffer_rsrc_t ri = rows_rsrc(p.i, pl.row * p.ib_ + (int64_t)t0 * p.it, p.it, nt, p.D, ES);
  const __amdgpu_buffer_rsrc_t rd = rows_rsrc(p.dout, pl.row * p.db + (int64_t)t0 * p.dt, p.dt, nt, p.D, ES);
  Row<T, VEC> vx[TT], vr[TT], vi[TT], vd[TT];
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    vr[j].load(rr, (uint32_t)(((lt0 + j) * p.rt + c0) * ES));
    vi[j].load(ri, (uint32_t)(((lt0 + j) * p.it + c0) * ES));
    vx[j].load(rx, (uint32_t)(((lt0 + j) * p.xt + c0) * ES));
    // zero behind the row's length (a token stride of 0 stays in range there)
    vd[j].load(rd, lt0 + j < nt ? (uint32_t)(((lt0 + j) * p.dt + c0) * ES) : kNowhere);
  }
  bool rs[TT];
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    rs[j] = false;
    if constexpr (CUT)
      if (lt0 + j < nt) rs[j] = p.reset[(int64_t)pl.row * p.L + t0 + lt0 + j] != 0;
  }
  float Ac[V], nrb[V], nib[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const int c = min(c0 + e, p.D - 1);
    Ac[e] = p.A[c];
    nrb[e] = p.rbias ? -kLog2e * p.rbias[c] : 0.f;
    nib[e] = p.ibias ? -kLog2e * p.ibias[c] : 0.f;
  }

  // ir = 1 / beta (0 where beta is 0), so beta = q ir
  float a[TT][V], q[TT][V], ir[TT][V];
  float A[V], w[V], Ab[V], wb[V];
#pragma unroll
  for (int e = 0; e < V; ++e) A[e] = 1.f, w[e] = 0.f, wb[e] = 0.f;
  bool cut = false;
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    const bool gone = lt0 + j >= nt;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float l = Ac[e] * kLog2e * sigmoid1(vr[j].get(e), nrb[e]);
      const float al = hw_exp2(l);
      q[j][e] = CUT && rs[j] ? 1.f : one_minus_sq(l, al);
      if (gone) q[j][e] = 0.f;
      ir[j][e] = q[j][e] > 0.f ? __builtin_amdgcn_rsqf(q[j][e]) : 0.f;
      a[j][e] = gone ? 1.f : al;
      const float b = q[j][e] * ir[j][e] * sigmoid1(vi[j].get(e), nib[e]) * vx[j].get(e);
      if (CUT && rs[j]) {
        a[j][e] = 0.f;
        A[e] = 0.f;
        w[e] = b;
      } else {
        A[e] *= a[j][e];
        w[e] = fmaf(a[j][e], w[e], b);
      }
    }
    cut = cut || rs[j];
  }
#pragma unroll
  for (int j = TT - 1; j >= 0; --j)
#pragma unroll
    for (int e = 0; e < V; ++e) wb[e] = CUT && rs[j] ? 0.f : a[j][e] * (vd[j].get(e) + wb[e]);
#pragma unroll
  for (int e = 0; e < V; ++e) Ab[e] = A[e];
  float fexA[V], fexw[V], bexA[V], bexw[V];
  bool fexcut, bexcut, cutb = cut;
  wave_compose<V, false, CUT>(A, w, cut, fexA, fexw, fexcut);
  wave_compose<V, true, CUT>(Ab, wb, cutb, bexA, bexw, bexcut);
  if (tg == TG - 1) {
#pragma unroll
    for (int e = 0; e < V; ++e) fA[wave][cl + e] = A[e], fw[wave][cl + e] = w[e];
    if (CUT && lane == 63) aggcut[wave] = cut;
  }
  if (tg == 0) {
#pragma unroll
    for (int e = 0; e < V; ++e) bA[wave][cl + e] = Ab[e], bw[wave][cl + e] = wb[e];
  }
  __syncthreads();

  if (wave == 0) {
    const int c = pl.tile * kTile + lane;
    const bool live = c < p.D;
    float cA = 1.f, cw = 0.f;
    bool ccut = false;
#pragma unroll
    for (int v = kWaves - 1; v >= 0; --v) {
      const bool k = CUT && aggcut[v];
      cw = k ? bw[v][lane] : fmaf(bA[v][lane], cw, bw[v][lane]);
      cA *= bA[v][lane];
      ccut = ccut || k;
    }
    float cin = 0.f, h = 0.f;
    if (live) {
      const int64_t nseg = (p.L + kGlrSegment - 1) / kGlrSegment;
      uint64_t *word = nullptr;
      const int64_t step = (int64_t)p.ntile * kTile;
      if (p.words) word = p.words + ((int64_t)pl.row * p.nchunk + pl.chunk) * step + c;
      const bool more = pl.chunk > 0;
      if (pl.chunk == last) {
        cin = p.dfin ? p.dfin[(int64_t)pl.row * p.D + c] : 0.f;
      } else {
        if (more) publish(word, ccut ? make_word(kFinished, cw) : make_word(decay_bits(cA), cw));
        cin = look_back(word + step, step, last - pl.chunk);
      }
      const float cend = ccut ? cw : fmaf(cA, cin, cw);
      if (more && !(ccut && pl.chunk != last)) publish(word, make_word(kFinished, cend));
      if (p.dinit && pl.chunk == 0) p.dinit[(int64_t)pl.row * p.D + c] = cend;
      h = p.states[((int64_t)pl.row * nseg + pl.chunk) * p.D + c];
    }
#pragma unroll
    for (int v = kWaves - 1; v >= 0; --v) {
      bcarry[v][lane] = cin;
      cin = CUT && aggcut[v] ? bw[v][lane] : fmaf(bA[v][lane], cin, bw[v][lane]);
    }
#pragma unroll
    for (int v = 0; v < kWaves; ++v) {
      fcarry[v][lane] = h;
      h = CUT && aggcut[v] ? fw[v][lane] : fmaf(fA[v][lane], h, fw[v][lane]);
    }
  }
  __syncthreads();

  float hp[TT][V], c[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float hc = fcarry[wave][cl + e], cc = bcarry[wave][cl + e];
    float h = CUT && fexcut ? fexw[e] : fmaf(fexA[e], hc, fexw[e]);
    c[e] = CUT && bexcut ? bexw[e] : fmaf(bexA[e], cc, bexw[e]);
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      hp[j][e] = h;
      if (j + 1 < TT) {
        const float b = q[j][e] * ir[j][e] * sigmoid1(vi[j].get(e), nib[e]) * vx[j].get(e);
        h = CUT && rs[j] ? b : fmaf(a[j][e], h, b);
      }
    }
  }
  float sA[V], sr[V], si[V];
#pragma unroll
  for (int e = 0; e < V; ++e) sA[e] = sr[e] = si[e] = 0.f;
#pragma unroll
  for (int j = TT - 1; j >= 0; --j) {
    float ox[V], orr[V], oi[V];
    const bool gone = lt0 + j >= nt;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float g = vd[j].get(e) + c[e];
      const Sig s = sigmoid2(vr[j].get(e), nrb[e]), gi = sigmoid2(vi[j].get(e), nib[e]);
      const float x = vx[j].get(e), ak = a[j][e];
      const float beta = q[j][e] * ir[j][e];
      const float gb = g * beta * gi.s;                 // dx
      const float dl = g * ak * (hp[j][e] - ak * (gi.s * x) * ir[j][e]); // at log a
      ox[e] = gb;
      oi[e] = gb * x * (gi.e * gi.s);
      orr[e] = dl * Ac[e] * s.s * (s.e * s.s);
      float da = dl * s.s;
      c[e] = ak * g;
      if (CUT && rs[j]) orr[e] = 0.f, da = 0.f, c[e] = 0.f;
      if (gone) {
        ox[e] = orr[e] = oi[e] = da = 0.f;
        c[e] = g;
      }
      sA[e] += da;
      sr[e] += orr[e];
      si[e] += oi[e];
    }
    const uint32_t off = (uint32_t)(((lt0 + j) * p.D + c0) * ES);
    const int n = lt0 + j < ntp ? nch : 0;
    store_row<T, VEC>(odx, off, ox, n);
    store_row<T, VEC>(odr, off, orr, n);
    store_row<T, VEC>(odi, off, oi, n);
  }
  // parameter gradients: pairs of token groups by shuffle, the rest in LDS
  // in a fixed order
#pragma unroll
  for (int e = 0; e < V; ++e) {
    sA[e] += __shfl_xor(sA[e], LPR);
    sr[e] += __shfl_xor(sr[e], LPR);
    si[e] += __shfl_xor(si[e], LPR);
    if ((tg & 1) == 0) {
      const int k = wave * (TG / 2) + tg / 2;
      psum[k][0][cl + e] = sA[e];
      psum[k][1][cl + e] = sr[e];
      psum[k][2][cl + e] = si[e];
    }
  }
  __syncthreads();
  if (tid < 3 * kTile) {
    const int ch = tid % kTile, what = tid / kTile;
    float s = 0.f;
#pragma unroll 8
    for (int k = 0; k < kWaves * TG / 2; ++k) s += psum[k][what][ch];
    if (pl.tile * kTile + ch < p.D) p.part[prow + (int64_t)what * p.D + pl.tile * kTile + ch] = s;
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

// One token: V channels per lane; bound by the launch at small batches and by
// HBM (the fp32 state in and out) at large ones.
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void glr_step_kernel(GlrStepParams p) {
  constexpr int V = Geo<T>::V, ES = (int)sizeof(T);
  const int row = (int)(blockIdx.x / (uint32_t)p.nblk);
  const int c0 = ((int)(blockIdx.x - (uint32_t)row * (uint32_t)p.nblk) * 256 + (int)threadIdx.x) * V;
  if (c0 >= p.D) return;
  const int nch = min(V, p.D - c0);
  Row<T, VEC> vr, vi, vx;
  vr.load(rows_rsrc(p.r, row * p.rb_, 0, 1, p.D, ES), (uint32_t)(c0 * ES));
  vi.load(rows_rsrc(p.i, row * p.ib_, 0, 1, p.D, ES), (uint32_t)(c0 * ES));
  vx.load(rows_rsrc(p.x, row * p.xb, 0, 1, p.D, ES), (uint32_t)(c0 * ES));
  const bool rs = p.reset && p.reset[row] != 0;
  const float *st = p.state + (int64_t)row * p.D + c0;
  float *ns = p.new_state + (int64_t)row * p.D + c0;
  float h[V];
  if constexpr (VEC) {
#pragma unroll
    for (int e = 0; e < V; e += 4) {
      const float4 v = *reinterpret_cast<const float4 *>(st + e);
      h[e] = v.x, h[e + 1] = v.y, h[e + 2] = v.z, h[e + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) h[e] = e < nch ? st[e] : 0.f;
  }
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const int c = min(c0 + e, p.D - 1);
    const float l = p.A[c] * kLog2e * sigmoid1(vr.get(e), p.rbias ? -kLog2e * p.rbias[c] : 0.f);
    const float a = hw_exp2(l);
    const float u = sigmoid1(vi.get(e), p.ibias ? -kLog2e * p.ibias[c] : 0.f) * vx.get(e);
    h[e] = rs ? u : fmaf(a, h[e], __builtin_amdgcn_sqrtf(one_minus_sq(l, a)) * u);
  }
  if constexpr (VEC) {
#pragma unroll
    for (int e = 0; e < V; e += 4) *reinterpret_cast<float4 *>(ns + e) = make_float4(h[e], h[e + 1], h[e + 2], h[e + 3]);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (e < nch) ns[e] = h[e];
  }
  store_row<T, VEC>(rows_rsrc(p.out, (int64_t)row * p.D, 0, 1, p.D, ES), (uint32_t)(c0 * ES), h, nch);
}

template <typename T, bool VEC, bool CUT>
hipError_t scan_launch(bool back, const GlrParams &p, hipStream_t st) {
  const dim3 grid((uint32_t)p.b * (uint32_t)p.ntile * (uint32_t)p.nchunk);
  if (back) glr_bwd_kernel<T, VEC, CUT><<<grid, kThreads, 0, st>>>(p);
  else glr_fwd_kernel<T, VEC, CUT><<<grid, kThreads, 0, st>>>(p);
  return hipGetLastError();
}

} // namespace

hipError_t launch_glr(int dtype, bool vec, bool back, const GlrParams &p, hipStream_t st) {
  if (p.words) {
    // words and the ticket behind them, in 16-byte pieces
    const int64_t n = glr_chain_bytes(p.b, p.nchunk, p.ntile) / 16;
    const int64_t blocks = (n + 255) / 256;
    glr_fill_kernel<<<(uint32_t)(blocks < 2048 ? blocks : 2048), 256, 0, st>>>((uint4 *)p.words, n);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const bool cut = p.reset != nullptr;
#define SSD_GLR(T, VEC) (cut ? scan_launch<T, VEC, true>(back, p, st) : scan_launch<T, VEC, false>(back, p, st))
  if (dtype == 1) return vec ? SSD_GLR(__bf16, true) : SSD_GLR(__bf16, false);
  return vec ? SSD_GLR(float, true) : SSD_GLR(float, false);
#undef SSD_GLR
}

hipError_t launch_glr_sum(const float *part, int n, int D, float *dA, float *drb, float *dib, hipStream_t st) {
  glr_sum_kernel<<<(uint32_t)((3 * (int64_t)D + 63) / 64), 64 * kSumRows, 0, st>>>(part, n, D, dA, drb, dib);
  return hipGetLastError();
}

hipError_t launch_glr_step(int dtype, bool vec, const GlrStepParams &p0, hipStream_t st) {
  const int V = dtype == 1 ? 8 : 4;
  GlrStepParams p = p0;
  p.nblk = (p.D + 256 * V - 1) / (256 * V);
  const dim3 grid((uint32_t)p.nblk * (uint32_t)p.b);
  if (dtype == 1) {
    if (vec) glr_step_kernel<__bf16, true><<<grid, 256, 0, st>>>(p);
    else glr_step_kernel<__bf16, false><<<grid, 256, 0, st>>>(p);
  } else {
    if (vec) glr_step_kernel<float, true><<<grid, 256, 0, st>>>(p);
    else glr_step_kernel<float, false><<<grid, 256, 0, st>>>(p);
  }
  return hipGetLastError();
}

} // namespace ssd
