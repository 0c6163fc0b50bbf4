// Elementwise gated linear recurrence over a sequence and its gradient.  Per
// batch row and channel, in fp32:
//   h_t = a_t h_{t-1} + b_t,  y_t = h_t
//   form LRU : la = A sigma(r), a = e^la, b = sqrt(1 - a^2) sigma(i) x
//   form UNIT: a = sigma(r),              b = (1 - a) x
// and a = 0 where the token's reset flag is set.
//
// The map of a run of tokens on the state is affine, h -> P h + H with P the
// product of its decays, and two runs compose to (P2 P1, P2 H1 + H2).  A
// workgroup takes a group of channels and walks the sequence in tiles.  Within
// a tile each lane takes V channels of K consecutive tokens, forms (P, H) of
// its run in registers, the runs of a wave are combined by shuffles, those of
// the waves through LDS, and each lane then replays its run from its true
// starting state.  The gradient runs the tiles from the last to the first: it
// rebuilds h in the tile from the state stored at the tile's start, and scans
// the adjoint mu_t = a_t (dout_t + mu_{t+1}) the other way with the same P.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "device_common.h"
#include "ssm_internal.h"

namespace ssm {
namespace {

constexpr int kWaves = 8;              // waves of a workgroup
constexpr int kThreads = 64 * kWaves;
constexpr float kLog2e = 1.4426950408889634f;
// Products of decays are kept from underflowing, so that P == 0 says that the
// run holds a reset, after which nothing of before (not even a NaN) is left.
constexpr float kTinyP = 1e-37f;

// V consecutive values of one token as they lie in memory.
template <bool BF16, int V>
struct Raw;
template <>
struct Raw<true, 2> {
  unsigned u;
  __device__ __forceinline__ float get(int v) const {
    return __builtin_bit_cast(float, v == 0 ? u << 16 : u & 0xffff0000u);
  }
  static __device__ __forceinline__ Raw make(const float (&f)[2]) {
    const unsigned lo = __builtin_bit_cast(unsigned short, (__bf16)f[0]);
    const unsigned hi = __builtin_bit_cast(unsigned short, (__bf16)f[1]);
    return {lo | (hi << 16)};
  }
};
template <>
struct Raw<true, 1> {
  unsigned short u;
  __device__ __forceinline__ float get(int) const { return __builtin_bit_cast(float, (unsigned)u << 16); }
  static __device__ __forceinline__ Raw make(const float (&f)[1]) {
    return {__builtin_bit_cast(unsigned short, (__bf16)f[0])};
  }
};
template <>
struct Raw<false, 2> {
  float2 u;
  __device__ __forceinline__ float get(int v) const { return v == 0 ? u.x : u.y; }
  static __device__ __forceinline__ Raw make(const float (&f)[2]) { return {make_float2(f[0], f[1])}; }
};
template <>
struct Raw<false, 1> {
  float u;
  __device__ __forceinline__ float get(int) const { return u; }
  static __device__ __forceinline__ Raw make(const float (&f)[1]) { return {f[0]}; }
};

__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-v * kLog2e));
}

// The gates of one element.
struct Gate {
  float a;    // decay
  float s;    // factor of sigma(i) x (LRU) or of x (UNIT)
  float rs;   // LRU: 1 / s, 0 where s is 0
  float g;    // LRU: sigma(r)
};

// LRU decay.  a is near 1 and enters a product over thousands of tokens, so it
// is rounded once from m = 1 - a = -expm1(la), which below |la| = 1/4 is the
// series of e^la (the first term left out is under 2^-25 of m); the same m gives
// 1 - a^2 = m (1 + a) without cancellation.
__device__ __forceinline__ Gate lru_gate(float r, float A) {
  Gate q;
  q.g = sigmoid(r);
  const float la = A * q.g;
  const float e = __builtin_amdgcn_exp2f(la * kLog2e);
  float p = fmaf(la, 1.f / 720.f, 1.f / 120.f);
  p = fmaf(p, la, 1.f / 24.f);
  p = fmaf(p, la, 1.f / 6.f);
  p = fmaf(p, la, 0.5f);
  p = fmaf(p, la, 1.f);
  const bool near1 = la > -0.25f;
  const float m = near1 ? -la * p : 1.f - e;
  q.a = near1 ? 1.f - m : e;
  const float w = m * (1.f + q.a);
  q.rs = w == 0.f ? 0.f : __builtin_amdgcn_rsqf(w);
  q.s = w * q.rs;
  return q;
}
__device__ __forceinline__ Gate unit_gate(float r) {
  Gate q;
  q.a = sigmoid(r);
  q.s = sigmoid(-r);   // 1 - a without cancellation
  q.rs = 0.f;
  q.g = q.a;
  return q;
}
template <int FORM>
__device__ __forceinline__ Gate gate_of(float r, float A) {
  if constexpr (FORM == kGatedLru) return lru_gate(r, A);
  else return unit_gate(r);
}

// (P, H) of an earlier run followed by a later one, into the later one's place.
template <bool RESET>
__device__ __forceinline__ void then(float p1, float h1, float& p2, float& h2) {
  if (RESET) {
    h2 = p2 == 0.f ? h2 : fmaf(p2, h1, h2);
    p2 = p1 == 0.f || p2 == 0.f ? 0.f : fmaxf(p1 * p2, kTinyP);
  } else {
    h2 = fmaf(p2, h1, h2);
    p2 = fmaxf(p1 * p2, kTinyP);
  }
}
// The state after a run.
template <bool RESET>
__device__ __forceinline__ float after(float p, float h, float state) {
  return RESET && p == 0.f ? h : fmaf(p, state, h);
}

// Where a workgroup and a lane stand.  Workgroups of neighbouring channel
// groups run on one XCD (workgroup ids go round the 8 XCDs), so that the lines
// they share are read into one L2.
struct Place {
  int col, row, wave, lane;
  int64_t b, c0, chunk, t_begin, t_end;
  bool active;
};
template <int V>
__device__ __forceinline__ Place place(const GatedArgs& a) {
  Place p;
  const unsigned n = gridDim.x, q = n / 8, rest = n % 8, xcd = blockIdx.x % 8;
  const unsigned id = xcd * q + (xcd < rest ? xcd : rest) + blockIdx.x / 8;
  const int64_t cw = (int64_t)a.cols * V;
  const unsigned groups = (unsigned)((a.dim + cw - 1) / cw);
  const unsigned rest2 = id / groups;
  p.lane = threadIdx.x & 63;
  p.wave = threadIdx.x >> 6;
  p.col = p.lane & (a.cols - 1);
  p.row = p.wave * (64 / a.cols) + p.lane / a.cols;
  p.b = rest2 % (unsigned)a.batch;
  p.chunk = rest2 / (unsigned)a.batch;
  p.c0 = (int64_t)(id % groups) * cw + p.col * V;
  p.active = p.c0 < a.dim;
  p.t_begin = p.chunk * a.chunk_len;
  p.t_end = min(a.seqlen, p.t_begin + a.chunk_len);
  return p;
}

// K tokens of one lane, from a uniform address and the lane's byte offset; the
// tokens from nv on are left as they are.
template <bool BF16, int V, int K>
__device__ __forceinline__ void load_run(const void* src, int64_t first, int64_t dim, unsigned off, int nv,
                                         Raw<BF16, V> (&out)[K]) {
  const char* base = (const char*)src + first * (BF16 ? 2 : 4);
  const int64_t step = dim * (BF16 ? 2 : 4);
  if (nv == K) {
#pragma unroll
    for (int j = 0; j < K; ++j) out[j] = *reinterpret_cast<const Raw<BF16, V>*>(base + j * step + off);
  } else {
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (j < nv) out[j] = *reinterpret_cast<const Raw<BF16, V>*>(base + j * step + off);
  }
}

// Reset flags of a lane's run as a bit mask.
template <int K>
__device__ __forceinline__ unsigned load_resets(const unsigned char* reset, int64_t at, int nv) {
  unsigned m = 0;
  if (reset == nullptr) return 0;
#pragma unroll
  for (int j = 0; j < K; ++j)
    if (j < nv) m |= (reset[at + j] != 0 ? 1u : 0u) << j;
  return m;
}

// Combines the runs of a wave, the earlier row first (DIR 1) or the later row
// first (DIR -1): on return (pe, he) is the map of the wave's rows before
// (DIR 1) or after (DIR -1) the lane's own, and (p, h) that of all of them up to
// and including it.
template <bool RESET, int DIR, int V>
__device__ __forceinline__ void wave_scan(int lane, int cols, float (&p)[V], float (&h)[V], float (&pe)[V],
                                          float (&he)[V]) {
  for (int sh = cols; sh < 64; sh <<= 1) {
    const bool has = DIR > 0 ? lane >= sh : lane + sh < 64;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float p1 = DIR > 0 ? __shfl_up(p[v], sh) : __shfl_down(p[v], sh);
      const float h1 = DIR > 0 ? __shfl_up(h[v], sh) : __shfl_down(h[v], sh);
      float p2 = p[v], h2 = h[v];
      then<RESET>(p1, h1, p2, h2);
      p[v] = has ? p2 : p[v];
      h[v] = has ? h2 : h[v];
    }
  }
  const bool has = DIR > 0 ? lane >= cols : lane + cols < 64;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float p1 = DIR > 0 ? __shfl_up(p[v], cols) : __shfl_down(p[v], cols);
    const float h1 = DIR > 0 ? __shfl_up(h[v], cols) : __shfl_down(h[v], cols);
    pe[v] = has ? p1 : 1.f;
    he[v] = has ? h1 : 0.f;
  }
}

// Forward.  AGG: only the map of each time chunk, (ws_p, ws_h), for chunks that
// run in parallel; else y, the states entering every kGatedSave-th token and
// the final state, from the maps of the chunks before.
template <bool BF16, int V, int FORM, bool RESET, int K, bool AGG>
__global__ __launch_bounds__(kThreads) void gated_fwd_kernel(GatedArgs a) {
  __shared__ float2 tot[2][kWaves][kGatedMaxCols][V];
  const Place q = place<V>(a);
  const int R = 64 / a.cols;
  const int T = kWaves * R * K;
  const int64_t L = a.seqlen, dim = a.dim;
  const int64_t plane = a.batch * dim;
  const int64_t state_at = q.b * dim + q.c0;   // (b, c0)
  const unsigned es = BF16 ? 2 : 4;
  const int64_t c_ld = q.active ? q.c0 : 0;
  const unsigned off = (unsigned)(((int64_t)q.row * K * dim + c_ld) * es);

  float A[V], carry[V], pall[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A[v] = FORM == kGatedLru ? a.A[c_ld + v] : 0.f;
    carry[v] = 0.f;
    pall[v] = 1.f;
    if (!AGG && q.active) {
      if (a.nchunks > 1) {   // the state entering the first chunk, then the chunks before this one
        carry[v] = a.ws_h0[state_at + v];
        for (int64_t k = 0; k < q.chunk; ++k)
          carry[v] = after<RESET>(a.ws_p[k * plane + state_at + v], a.ws_h[k * plane + state_at + v], carry[v]);
      } else if (a.h0 != nullptr) {
        carry[v] = a.h0[state_at + v];
      }
    }
  }
  if (AGG && q.chunk == 0 && q.active && q.row == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) a.ws_h0[state_at + v] = a.h0 != nullptr ? a.h0[state_at + v] : 0.f;
  }

  int buf = 0;
  for (int64_t t0 = q.t_begin; t0 < q.t_end; t0 += T, buf ^= 1) {
    const int64_t tl = t0 + q.row * K;
    const int nv = (int)max((int64_t)0, min((int64_t)K, q.t_end - tl));
    const int64_t first = (q.b * L + t0) * dim;
    Raw<BF16, V> rr[K] = {}, ri[K] = {}, rx[K] = {};
    load_run<BF16, V, K>(a.r, first, dim, off, nv, rr);
    if (FORM == kGatedLru) load_run<BF16, V, K>(a.i, first, dim, off, nv, ri);
    load_run<BF16, V, K>(a.x, first, dim, off, nv, rx);
    const unsigned rm = RESET ? load_resets<K>(a.reset, q.b * L + tl, nv) : 0u;

    float da[K][V], db[K][V], p[V], h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) { p[v] = 1.f; h[v] = 0.f; }
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const bool rs = RESET && ((rm >> j) & 1u);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        Gate w = gate_of<FORM>(rr[j].get(v), A[v]);
        if (RESET) { w.a = rs ? 0.f : w.a; w.s = rs ? 1.f : w.s; }
        float u = rx[j].get(v);
        if (FORM == kGatedLru) u *= sigmoid(ri[j].get(v));
        const bool in = j < nv;
        da[j][v] = in ? w.a : 1.f;
        db[j][v] = in ? w.s * u : 0.f;
        h[v] = rs ? db[j][v] : fmaf(da[j][v], h[v], db[j][v]);
        p[v] *= da[j][v];
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = RESET && rm != 0 ? 0.f : fmaxf(p[v], kTinyP);

    float pe[V], he[V];
    wave_scan<RESET, 1, V>(q.lane, a.cols, p, h, pe, he);
    if (q.lane >= 64 - a.cols) {
#pragma unroll
      for (int v = 0; v < V; ++v) tot[buf][q.wave][q.col][v] = make_float2(p[v], h[v]);
    }
    lds_sync();
    float st[V];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float2 ph = tot[buf][w][q.col][v];
        if (w == q.wave) st[v] = carry[v];
        carry[v] = after<RESET>(ph.x, ph.y, carry[v]);
        if (AGG) pall[v] = RESET && (pall[v] == 0.f || ph.x == 0.f) ? 0.f : fmaxf(pall[v] * ph.x, kTinyP);
      }
    }
    if (!AGG) {
#pragma unroll
      for (int v = 0; v < V; ++v) st[v] = after<RESET>(pe[v], he[v], st[v]);
      if (a.states != nullptr && (q.row * K) % kGatedSave == 0 && nv > 0 && q.active) {
#pragma unroll
        for (int v = 0; v < V; ++v) a.states[(tl / kGatedSave) * plane + state_at + v] = st[v];
      }
      char* yb = (char*)a.y + first * es;
#pragma unroll
      for (int j = 0; j < K; ++j) {
        const bool rs = RESET && ((rm >> j) & 1u);
#pragma unroll
        for (int v = 0; v < V; ++v) st[v] = rs ? db[j][v] : fmaf(da[j][v], st[v], db[j][v]);
        if (a.y != nullptr && j < nv && q.active)
          *reinterpret_cast<Raw<BF16, V>*>(yb + j * dim * es + off) = Raw<BF16, V>::make(st);
      }
    }
  }
  if (AGG) {
    if (q.active && q.row == 0) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        a.ws_p[q.chunk * plane + state_at + v] = pall[v];
        a.ws_h[q.chunk * plane + state_at + v] = carry[v];
      }
    }
  } else if (a.h_final != nullptr && q.chunk == a.nchunks - 1) {
    __syncthreads();   // with no token, every wave has read h0, which h_final may be
    if (q.active && q.row == 0) {
#pragma unroll
      for (int v = 0; v < V; ++v) a.h_final[state_at + v] = carry[v];
    }
  }
}

// Backward of a time chunk from what later chunks hand back: the map of mu
// over the chunk, for chunks that run in parallel.
template <bool BF16, int V, int FORM, bool RESET, int K>
__global__ __launch_bounds__(kThreads) void gated_bwd_agg_kernel(GatedArgs a) {
  __shared__ float2 tot[2][kWaves][kGatedMaxCols][V];
  const Place q = place<V>(a);
  const int T = kWaves * (64 / a.cols) * K;
  const int64_t L = a.seqlen, dim = a.dim;
  const int64_t plane = a.batch * dim;
  const int64_t state_at = q.b * dim + q.c0;
  const unsigned es = BF16 ? 2 : 4;
  const int64_t c_ld = q.active ? q.c0 : 0;
  const unsigned off = (unsigned)(((int64_t)q.row * K * dim + c_ld) * es);
  float A[V], carry[V], pall[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A[v] = FORM == kGatedLru ? a.A[c_ld + v] : 0.f;
    carry[v] = 0.f;
    pall[v] = 1.f;
  }
  int buf = 0;
  const int64_t ntiles = (q.t_end - q.t_begin + T - 1) / T;
  for (int64_t it = ntiles - 1; it >= 0; --it, buf ^= 1) {
    const int64_t t0 = q.t_begin + it * T, tl = t0 + q.row * K;
    const int nv = (int)max((int64_t)0, min((int64_t)K, q.t_end - tl));
    const int64_t first = (q.b * L + t0) * dim;
    Raw<BF16, V> rr[K] = {}, rd[K] = {};
    load_run<BF16, V, K>(a.r, first, dim, off, nv, rr);
    load_run<BF16, V, K>(a.dout, first, dim, off, nv, rd);
    const unsigned rm = RESET ? load_resets<K>(a.reset, q.b * L + tl, nv) : 0u;
    float p[V], m[V];
#pragma unroll
    for (int v = 0; v < V; ++v) { p[v] = 1.f; m[v] = 0.f; }
#pragma unroll
    for (int j = K - 1; j >= 0; --j) {
      const bool rs = RESET && ((rm >> j) & 1u);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Gate w = gate_of<FORM>(rr[j].get(v), A[v]);
        const bool in = j < nv;
        const float lam = m[v] + (in ? rd[j].get(v) : 0.f);
        m[v] = rs ? 0.f : (in ? w.a * lam : lam);
        p[v] *= in ? w.a : 1.f;
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = RESET && rm != 0 ? 0.f : fmaxf(p[v], kTinyP);
    float pe[V], me[V];
    wave_scan<RESET, -1, V>(q.lane, a.cols, p, m, pe, me);
    if (q.lane < a.cols) {
#pragma unroll
      for (int v = 0; v < V; ++v) tot[buf][q.wave][q.col][v] = make_float2(p[v], m[v]);
    }
    lds_sync();
#pragma unroll
    for (int w = kWaves - 1; w >= 0; --w) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float2 ph = tot[buf][w][q.col][v];
        carry[v] = after<RESET>(ph.x, ph.y, carry[v]);
        pall[v] = RESET && (pall[v] == 0.f || ph.x == 0.f) ? 0.f : fmaxf(pall[v] * ph.x, kTinyP);
      }
    }
  }
  if (q.active && q.row == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      a.ws_p[q.chunk * plane + state_at + v] = pall[v];
      a.ws_h[q.chunk * plane + state_at + v] = carry[v];
    }
  }
}

// Backward: dx, dr, di, dh0 and the workgroup's share of dA.
template <bool BF16, int V, int FORM, bool RESET, int K>
__global__ __launch_bounds__(kThreads) void gated_bwd_kernel(GatedArgs a) {
  __shared__ float2 tot[2][kWaves][kGatedMaxCols][V];   // (P, H) of the waves' runs
  __shared__ float tom[2][kWaves][kGatedMaxCols][V];    // M of the waves' runs
  const Place q = place<V>(a);
  const int T = kWaves * (64 / a.cols) * K;
  const int64_t L = a.seqlen, dim = a.dim;
  const int64_t plane = a.batch * dim;
  const int64_t state_at = q.b * dim + q.c0;
  const unsigned es = BF16 ? 2 : 4;
  const int64_t c_ld = q.active ? q.c0 : 0;
  const unsigned off = (unsigned)(((int64_t)q.row * K * dim + c_ld) * es);
  float A[V], mu[V], accA[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A[v] = FORM == kGatedLru ? a.A[c_ld + v] : 0.f;
    mu[v] = a.dh_final != nullptr && q.active ? a.dh_final[state_at + v] : 0.f;
    accA[v] = 0.f;
    if (q.active)
      for (int64_t k = a.nchunks - 1; k > q.chunk; --k)
        mu[v] = after<RESET>(a.ws_p[k * plane + state_at + v], a.ws_h[k * plane + state_at + v], mu[v]);
  }
  int buf = 0;
  const int64_t ntiles = (q.t_end - q.t_begin + T - 1) / T;
  for (int64_t it = ntiles - 1; it >= 0; --it, buf ^= 1) {
    const int64_t t0 = q.t_begin + it * T, tl = t0 + q.row * K;
    const int nv = (int)max((int64_t)0, min((int64_t)K, q.t_end - tl));
    const int64_t first = (q.b * L + t0) * dim;
    Raw<BF16, V> rr[K] = {}, ri[K] = {}, rx[K] = {}, rd[K] = {};
    load_run<BF16, V, K>(a.r, first, dim, off, nv, rr);
    if (FORM == kGatedLru) load_run<BF16, V, K>(a.i, first, dim, off, nv, ri);
    load_run<BF16, V, K>(a.x, first, dim, off, nv, rx);
    load_run<BF16, V, K>(a.dout, first, dim, off, nv, rd);
    const unsigned rm = RESET ? load_resets<K>(a.reset, q.b * L + tl, nv) : 0u;
    float hst[V];   // the state entering the tile
#pragma unroll
    for (int v = 0; v < V; ++v) hst[v] = q.active ? a.saved[(t0 / kGatedSave) * plane + state_at + v] : 0.f;

    float da[K][V], hp[K][V], p[V], h[V], m[V], pr[V];
#pragma unroll
    for (int v = 0; v < V; ++v) { p[v] = 1.f; h[v] = 0.f; m[v] = 0.f; }
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const bool rs = RESET && ((rm >> j) & 1u);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        Gate w = gate_of<FORM>(rr[j].get(v), A[v]);
        if (RESET) { w.a = rs ? 0.f : w.a; w.s = rs ? 1.f : w.s; }
        float u = rx[j].get(v);
        if (FORM == kGatedLru) u *= sigmoid(ri[j].get(v));
        const bool in = j < nv;
        da[j][v] = in ? w.a : 1.f;
        hp[j][v] = in ? w.s * u : 0.f;   // b, replaced by h_{t-1} below
        h[v] = rs ? hp[j][v] : fmaf(da[j][v], h[v], hp[j][v]);
        p[v] *= da[j][v];
      }
    }
#pragma unroll
    for (int j = K - 1; j >= 0; --j) {
      const bool rs = RESET && ((rm >> j) & 1u);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float lam = m[v] + (j < nv ? rd[j].get(v) : 0.f);
        m[v] = rs ? 0.f : da[j][v] * lam;
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      p[v] = RESET && rm != 0 ? 0.f : fmaxf(p[v], kTinyP);
      pr[v] = p[v];
    }
    float pe[V], he[V], qe[V], me[V];
    wave_scan<RESET, 1, V>(q.lane, a.cols, p, h, pe, he);
    wave_scan<RESET, -1, V>(q.lane, a.cols, pr, m, qe, me);
    if (q.lane >= 64 - a.cols) {
#pragma unroll
      for (int v = 0; v < V; ++v) tot[buf][q.wave][q.col][v] = make_float2(p[v], h[v]);
    }
    if (q.lane < a.cols) {
#pragma unroll
      for (int v = 0; v < V; ++v) tom[buf][q.wave][q.col][v] = m[v];
    }
    lds_sync();
    float st[V], ms[V];
#pragma unroll
    for (int v = 0; v < V; ++v) { st[v] = hst[v]; ms[v] = mu[v]; }
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float2 f = tot[buf][w][q.col][v];
        if (w < q.wave) st[v] = after<RESET>(f.x, f.y, st[v]);
        const int w2 = kWaves - 1 - w;
        const float2 f2 = tot[buf][w2][q.col][v];
        if (w2 == q.wave) ms[v] = mu[v];
        mu[v] = after<RESET>(f2.x, tom[buf][w2][q.col][v], mu[v]);
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      st[v] = after<RESET>(pe[v], he[v], st[v]);
      ms[v] = after<RESET>(qe[v], me[v], ms[v]);
    }
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const bool rs = RESET && ((rm >> j) & 1u);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float b = hp[j][v];
        hp[j][v] = st[v];
        st[v] = rs ? b : fmaf(da[j][v], st[v], b);
      }
    }
    char* xb = (char*)a.dx + first * es;
    char* gb = (char*)a.dr + first * es;
    char* ib = (char*)a.di + first * es;
#pragma unroll
    for (int j = K - 1; j >= 0; --j) {
      const bool rs = RESET && ((rm >> j) & 1u);
      float ox[V], og[V], oi[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const bool in = j < nv;
        const float lam = ms[v] + (in ? rd[j].get(v) : 0.f);
        const float x = rx[j].get(v);
        Gate w = gate_of<FORM>(rr[j].get(v), A[v]);
        if (RESET) w.s = rs ? 1.f : w.s;
        if constexpr (FORM == kGatedLru) {
          const float gi = sigmoid(ri[j].get(v));
          const float u = gi * x, ls = lam * w.s;
          float dla = lam * w.a * fmaf(-u * w.a, w.rs, hp[j][v]);
          if (RESET) dla = rs ? 0.f : dla;
          const float dag = dla * w.g;
          accA[v] += in ? dag : 0.f;
          og[v] = dag * A[v] * (1.f - w.g);
          ox[v] = ls * gi;
          oi[v] = ls * u * (1.f - gi);
        } else {
          ox[v] = lam * w.s;
          og[v] = rs ? 0.f : ox[v] * w.a * (hp[j][v] - x);
          oi[v] = 0.f;
        }
        ms[v] = rs ? 0.f : da[j][v] * lam;
      }
      if (j < nv && q.active) {
        *reinterpret_cast<Raw<BF16, V>*>(xb + j * dim * es + off) = Raw<BF16, V>::make(ox);
        *reinterpret_cast<Raw<BF16, V>*>(gb + j * dim * es + off) = Raw<BF16, V>::make(og);
        if (FORM == kGatedLru)
          *reinterpret_cast<Raw<BF16, V>*>(ib + j * dim * es + off) = Raw<BF16, V>::make(oi);
      }
    }
  }
  if (a.dh0 != nullptr && q.chunk == 0 && q.active && q.row == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) a.dh0[state_at + v] = mu[v];
  }
  if (FORM == kGatedLru) {
    // rows of the wave, then the waves, in a fixed order
    for (int sh = a.cols; sh < 64; sh <<= 1)
#pragma unroll
      for (int v = 0; v < V; ++v) accA[v] += __shfl_xor(accA[v], sh);
    __syncthreads();
    if (q.lane < a.cols) {
#pragma unroll
      for (int v = 0; v < V; ++v) tom[0][q.wave][q.col][v] = accA[v];
    }
    lds_sync();
    if (q.active && q.row == 0) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float s = 0.f;
        for (int w = 0; w < kWaves; ++w) s += tom[0][w][q.col][v];
        a.ws_da[q.chunk * plane + state_at + v] = s;
      }
    }
  }
}

// dA[d] = sum of the parts (chunk, batch) of channel d, in a fixed order.
__global__ __launch_bounds__(256) void gated_da_kernel(const float* parts, float* dA, int64_t n, int64_t dim) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= dim) return;
  float s = 0.f;
  for (int64_t k = 0; k < n; ++k) s += parts[k * dim + c];
  dA[c] = s;
}

// One token of every (batch, channel), the state updated in place.
template <bool BF16, int V, int FORM>
__global__ __launch_bounds__(256) void gated_step_kernel(GatedArgs a) {
  const int64_t k = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V;
  if (k >= a.batch * a.dim) return;
  const int64_t c = k % a.dim;
  const unsigned es = BF16 ? 2 : 4;
  using R = Raw<BF16, V>;
  const R rr = *reinterpret_cast<const R*>((const char*)a.r + k * es);
  const R rx = *reinterpret_cast<const R*>((const char*)a.x + k * es);
  R ri = {};
  if (FORM == kGatedLru) ri = *reinterpret_cast<const R*>((const char*)a.i + k * es);
  float st[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const Gate w = gate_of<FORM>(rr.get(v), FORM == kGatedLru ? a.A[c + v] : 0.f);
    float u = rx.get(v);
    if (FORM == kGatedLru) u *= sigmoid(ri.get(v));
    st[v] = fmaf(w.a, a.states[k + v], w.s * u);
    a.states[k + v] = st[v];
  }
  *reinterpret_cast<R*>((char*)a.y + k * es) = R::make(st);
}

constexpr int run_len(bool bf16) { return bf16 ? 16 : 8; }   // tokens of a lane's run

template <bool BF16, int V, int FORM, bool RESET>
void launch_fwd(const GatedArgs& a, unsigned grid, hipStream_t st) {
  constexpr int K = run_len(BF16);
  if (a.nchunks > 1) gated_fwd_kernel<BF16, V, FORM, RESET, K, true><<<grid, kThreads, 0, st>>>(a);
  gated_fwd_kernel<BF16, V, FORM, RESET, K, false><<<grid, kThreads, 0, st>>>(a);
}

template <bool BF16, int V, int FORM, bool RESET>
void launch_bwd(const GatedArgs& a, unsigned grid, hipStream_t st) {
  constexpr int K = 8;
  if (a.nchunks > 1) gated_bwd_agg_kernel<BF16, V, FORM, RESET, K><<<grid, kThreads, 0, st>>>(a);
  gated_bwd_kernel<BF16, V, FORM, RESET, K><<<grid, kThreads, 0, st>>>(a);
}

// Instances: V = 2 where the rows allow it, with and without resets; the
// one-channel kernels always look for them.
template <bool BF16, int FORM>
void pick(const GatedArgs& a, unsigned grid, bool bwd, hipStream_t st) {
  if (a.vec) {
    if (a.reset != nullptr) bwd ? launch_bwd<BF16, 2, FORM, true>(a, grid, st) : launch_fwd<BF16, 2, FORM, true>(a, grid, st);
    else bwd ? launch_bwd<BF16, 2, FORM, false>(a, grid, st) : launch_fwd<BF16, 2, FORM, false>(a, grid, st);
  } else {
    bwd ? launch_bwd<BF16, 1, FORM, true>(a, grid, st) : launch_fwd<BF16, 1, FORM, true>(a, grid, st);
  }
}

void pick(const GatedArgs& a, unsigned grid, bool bwd, hipStream_t st) {
  if (a.act_bf16) {
    a.form == kGatedLru ? pick<true, kGatedLru>(a, grid, bwd, st) : pick<true, kGatedUnit>(a, grid, bwd, st);
  } else {
    a.form == kGatedLru ? pick<false, kGatedLru>(a, grid, bwd, st) : pick<false, kGatedUnit>(a, grid, bwd, st);
  }
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

GatedPlan plan_gated(int64_t batch, int64_t seqlen, int64_t dim, bool bf16, int num_cus) {
  GatedPlan p{kGatedMaxCols, 1, 1, 0, 0, 0};
  if (batch == 0 || dim == 0) return p;
  const int V = dim % 2 == 0 ? 2 : 1;
  auto groups = [&](int cols) { return batch * ((dim + (int64_t)cols * V - 1) / ((int64_t)cols * V)); };
  while (p.cols > 4 && groups(p.cols) < 2 * num_cus) p.cols /= 2;
  // the forward and the backward share the plan, so a chunk is whole tiles of both
  const int64_t T = (int64_t)kWaves * (64 / p.cols) * std::max(run_len(bf16), 8);
  const int64_t tiles = (seqlen + T - 1) / T;
  if (groups(p.cols) < num_cus && tiles > 1) {
    p.nchunks = std::min<int64_t>(std::min<int64_t>((num_cus + groups(p.cols) - 1) / groups(p.cols), tiles), 64);
  }
  const int64_t per = std::max<int64_t>(1, (tiles + p.nchunks - 1) / p.nchunks);
  p.chunk_len = per * T;
  p.nchunks = std::max<int64_t>(1, (tiles + per - 1) / per);
  const size_t plane = (size_t)(batch * dim) * sizeof(float);
  p.maps_bytes = p.nchunks > 1 ? up256(plane) + 2 * up256(p.nchunks * plane) : 0;
  p.da_bytes = up256(p.nchunks * plane);
  p.states_bytes = (size_t)((seqlen + kGatedSave - 1) / kGatedSave) * plane;
  return p;
}

static void set_maps(GatedArgs& a, const GatedPlan& p, char* ws) {
  const size_t plane = up256((size_t)(a.batch * a.dim) * sizeof(float));
  const size_t planes = up256((size_t)p.nchunks * (size_t)(a.batch * a.dim) * sizeof(float));
  a.ws_h0 = (float*)ws;
  a.ws_p = (float*)(ws + plane);
  a.ws_h = (float*)(ws + plane + planes);
}

static int grid_of(const GatedArgs& a, const GatedPlan& p, unsigned* grid) {
  const int V = a.vec ? 2 : 1;
  const int64_t cw = (int64_t)p.cols * V;
  const int64_t n = ((a.dim + cw - 1) / cw) * a.batch * p.nchunks;
  // a lane's byte offset in a tile is held in 32 bits
  const int64_t tile = (int64_t)kWaves * (64 / p.cols) * 16 * (a.act_bf16 ? 2 : 4);
  if (n > 0x7fffffffLL || a.dim > 0x7fffffffLL / tile) return fail(4, "batch or dim too large");
  *grid = (unsigned)n;
  return 0;
}

int launch_gated_fwd(GatedArgs a, const GatedPlan& p, void* ws, void* stream) {
  unsigned grid = 0;
  const int rc = grid_of(a, p, &grid);
  if (rc != 0) return rc;
  a.cols = p.cols; a.nchunks = p.nchunks; a.chunk_len = p.chunk_len;
  if (p.nchunks > 1) set_maps(a, p, (char*)ws);
  pick(a, grid, false, (hipStream_t)stream);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? 0 : fail(6, std::string("gated scan launch: ") + hipGetErrorString(e));
}

// Workspace: the chunk maps, the dA parts and, without the forward's states, the states.
int launch_gated_bwd(GatedArgs a, const GatedPlan& p, void* ws, void* stream) {
  unsigned grid = 0;
  const int rc = grid_of(a, p, &grid);
  if (rc != 0) return rc;
  hipStream_t st = (hipStream_t)stream;
  if (a.batch == 0) {   // dA of no rows
    if (a.form == kGatedLru) gated_da_kernel<<<(unsigned)((a.dim + 255) / 256), 256, 0, st>>>(nullptr, a.dA, 0, a.dim);
    const hipError_t e0 = hipGetLastError();
    return e0 == hipSuccess ? 0 : fail(6, std::string("gated scan backward launch: ") + hipGetErrorString(e0));
  }
  a.cols = p.cols; a.nchunks = p.nchunks; a.chunk_len = p.chunk_len;
  if (p.nchunks > 1) set_maps(a, p, (char*)ws);
  a.ws_da = (float*)((char*)ws + p.maps_bytes);
  if (a.saved == nullptr) {
    a.states = (float*)((char*)ws + p.maps_bytes + p.da_bytes);
    pick(a, grid, false, st);   // y and h_final are null: the states only
    a.saved = a.states;
  }
  pick(a, grid, true, st);
  if (a.form == kGatedLru)
    gated_da_kernel<<<(unsigned)((a.dim + 255) / 256), 256, 0, st>>>(a.ws_da, a.dA, p.nchunks * a.batch, a.dim);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? 0 : fail(6, std::string("gated scan backward launch: ") + hipGetErrorString(e));
}

int launch_gated_step(const GatedArgs& a, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  const int V = a.vec ? 2 : 1;
  const int64_t n = (a.batch * a.dim / V + 255) / 256;
  if (n > 0x7fffffffLL) return fail(4, "batch or dim too large");
  const unsigned grid = (unsigned)n;
  const bool lru = a.form == kGatedLru;
  if (a.act_bf16) {
    if (a.vec) lru ? gated_step_kernel<true, 2, kGatedLru><<<grid, 256, 0, st>>>(a) : gated_step_kernel<true, 2, kGatedUnit><<<grid, 256, 0, st>>>(a);
    else lru ? gated_step_kernel<true, 1, kGatedLru><<<grid, 256, 0, st>>>(a) : gated_step_kernel<true, 1, kGatedUnit><<<grid, 256, 0, st>>>(a);
  } else {
    if (a.vec) lru ? gated_step_kernel<false, 2, kGatedLru><<<grid, 256, 0, st>>>(a) : gated_step_kernel<false, 2, kGatedUnit><<<grid, 256, 0, st>>>(a);
    else lru ? gated_step_kernel<false, 1, kGatedLru><<<grid, 256, 0, st>>>(a) : gated_step_kernel<false, 1, kGatedUnit><<<grid, 256, 0, st>>>(a);
  }
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? 0 : fail(6, std::string("gated step launch: ") + hipGetErrorString(e));
}

}  // namespace ssm
