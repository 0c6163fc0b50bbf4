// Gradient of the causal depthwise conv1d + SiLU.  With xx the inputs, the W-1
// carried ones in front,
//   pre_t  = bias + sum_k w[k] xx[t-(W-1)+k],   dpre_t = dout_t silu'(pre_t)
//   dxx[p] = sum_j w[W-1-j] dpre_{p+j}  (p + j inside the segment)
//            + the gradient of the carried-out state where p is one of the last W-1 inputs
//   dw[k]  = sum_{b,t} dpre_t xx[t-(W-1)+k],    dbias = sum_{b,t} dpre_t.
//
// Bound by HBM: x and dout read once, dx written once (pre is recomputed).  A
// thread takes V channels of a run of tokens and slides two windows of W
// along it, the inputs and dpre; it starts W-1 inputs early and runs W-1 tokens
// late, rows that its neighbours read too and that come from the caches.  dw and
// dbias are summed in registers over the run, over a workgroup's runs by
// shuffles and LDS, and over the workgroups by a second kernel, all in a fixed
// order.  About 24 vector instructions an element (W = 4, SiLU), four tokens a
// step with the next step's loads ahead, two channels a thread: 109 registers,
// four waves a SIMD.  bf16 b8 x 2048 x 1536, W = 4: 33 us and 4 us for the sums
// (29 at a copy's rate; four channels a thread and no loads ahead: 40 and 9);
// b1 x 131072 x 2048: 347 us (309).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "ssm_internal.h"
#include "vec_io.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;
constexpr int kVec = 2;       // channels of a thread where the rows allow it
constexpr int kMaxParts = 64;  // workgroups that share a channel group

// V channels of one token as they lie in memory.
template <bool BF16, int V>
struct Tok;
template <>
struct Tok<true, 2> {
  unsigned u;
  __device__ __forceinline__ float get(int c) const { return c == 0 ? bf16_lo(u) : bf16_hi(u); }
  static __device__ __forceinline__ Tok make(const float (&v)[2]) { return {pack_bf16(v[0], v[1])}; }
};
template <>
struct Tok<false, 2> {
  f32x2 u;
  __device__ __forceinline__ float get(int c) const { return u[c]; }
  static __device__ __forceinline__ Tok make(const float (&v)[2]) { return {f32x2{v[0], v[1]}}; }
};
template <>
struct Tok<true, 1> {
  unsigned short u;
  __device__ __forceinline__ float get(int) const { return bf16_lo(u); }
  static __device__ __forceinline__ Tok make(const float (&v)[1]) { return {__builtin_bit_cast(unsigned short, (__bf16)v[0])}; }
};
template <>
struct Tok<false, 1> {
  float u;
  __device__ __forceinline__ float get(int) const { return u; }
  static __device__ __forceinline__ Tok make(const float (&v)[1]) { return {v[0]}; }
};

// A workgroup is COLS threads of V channels by ROWS runs.
template <int V>
struct Shape {
  static constexpr int COLS = V == 1 ? 32 : 64 / V;
  static constexpr int ROWS = kThreads / COLS;
};

template <int W, bool BF16, int V, bool SILU>
__global__ __launch_bounds__(kThreads, W <= 4 ? 4 : 2) void conv_bwd_kernel(ConvBwdArgs a, unsigned groups, int64_t blocks_per_row) {
  constexpr int COLS = Shape<V>::COLS, ROWS = Shape<V>::ROWS;
  __shared__ float red[4][(W + 1) * V][COLS];
  const int64_t L = a.seqlen, dim = a.dim;
  const int col = threadIdx.x % COLS, run = threadIdx.x / COLS;
  const unsigned part = blockIdx.x / groups;
  const int64_t c0 = ((int64_t)(blockIdx.x % groups) * COLS + col) * V;
  const bool active = c0 < dim;
  using T = Tok<BF16, V>;
  constexpr int64_t es = BF16 ? 2 : 4;

  float wt[W][V], bs[V], dw[W][V], db[V];
#pragma unroll
  for (int c = 0; c < V; ++c) {
#pragma unroll
    for (int k = 0; k < W; ++k) {
      wt[k][c] = active ? a.w[(c0 + c) * W + k] : 0.f;
      dw[k][c] = 0.f;
    }
    bs[c] = active && a.bias != nullptr ? a.bias[c0 + c] : 0.f;
    db[c] = 0.f;
  }

  constexpr int U = 4;   // tokens of a step
  const int64_t nblk = a.batch * blocks_per_row;
  for (int64_t blk = part; blk < nblk; blk += a.nparts) {
    const int64_t b = blk / blocks_per_row;
    const int64_t tb = (blk % blocks_per_row) * ROWS * a.run, t0 = tb + run * a.run;
    if (!active || t0 >= L) continue;
    const int64_t t1 = min(L, t0 + a.run), last = min(L, t1 + W - 1);   // own tokens, tokens read
    const int64_t row0 = b * L;
    const int64_t srow = (b * dim + c0) * (W - 1);
    // the workgroup's block in scalar registers, the thread's place in it in 32 bits (x, dout and dx share it)
    const int64_t from = (row0 + tb) * dim * es;
    const char *const x = (const char*)a.x + from, *const dy = (const char*)a.dout + from;
    char* const dx = (char*)a.dx + from;
    const unsigned stride = (unsigned)(dim * es);
    unsigned off = (unsigned)((run * (int64_t)a.run * dim + c0) * es);   // of token t
    // the inputs and dpre of a step's tokens and of the W-1 before them: xs[j] is xx[t-(W-1)+j], ds[j] dpre there
    float xs[W - 1 + U][V], ds[W - 1 + U][V];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int64_t pos = t0 - (W - 1) + j;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        xs[j][c] = ds[j][c] = 0.f;
        if (pos < 0 && a.state_in != nullptr) xs[j][c] = load1<BF16>(a.state_in, srow + c * (W - 1) + (W - 1) + pos);
      }
      if (pos >= 0) {
        const T v = *(const T*)(x + (off + (pos - t0) * (int64_t)stride));
#pragma unroll
        for (int c = 0; c < V; ++c) xs[j][c] = v.get(c);
      }
    }
    T nx[U], nd[U];   // the next step's tokens
    auto fetch = [&](int64_t t, unsigned off) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        nx[u] = {};
        nd[u] = {};
        if (t + u < last) {
          nx[u] = *(const T*)(x + (off + u * stride));
          nd[u] = *(const T*)(dy + (off + u * stride));
        }
      }
    };
    // EDGE: the step reaches out of the run's own tokens
    auto step = [&](int64_t t, auto edge) {
      constexpr bool EDGE = decltype(edge)::value;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int c = 0; c < V; ++c) {
          xs[W - 1 + u][c] = nx[u].get(c);
          ds[W - 1 + u][c] = nd[u].get(c);   // zeros behind the last token
        }
      if (EDGE || t + 2 * U > last) {
        fetch(t + U, off + U * stride);
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          nx[u] = *(const T*)(x + (off + (U + u) * stride));
          nd[u] = *(const T*)(dy + (off + (U + u) * stride));
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool own = !EDGE || t + u < t1;
        if (EDGE && t + u >= last) {
#pragma unroll
          for (int c = 0; c < V; ++c) ds[W - 1 + u][c] = 0.f;
        }
#pragma unroll
        for (int c = 0; c < V; ++c) {
          float& d = ds[W - 1 + u][c];
          if constexpr (SILU) {
            float pre = bs[c];
#pragma unroll
            for (int k = 0; k < W; ++k) pre = fmaf(wt[k][c], xs[u + k][c], pre);
            const float s = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-pre * 1.4426950408889634f));
            d *= s * fmaf(pre, 1.f - s, 1.f);
          }
          if (own) {
            db[c] += d;
#pragma unroll
            for (int k = 0; k < W; ++k) dw[k][c] = fmaf(d, xs[u + k][c], dw[k][c]);
          }
        }
        const int64_t p = t + u - (W - 1);
        if (EDGE && (p >= t1 || (p < t0 && t0 > 0))) continue;   // another run's
        float o[V];
#pragma unroll
        for (int c = 0; c < V; ++c) {
          o[c] = 0.f;
#pragma unroll
          for (int j = 0; j < W; ++j) o[c] = fmaf(wt[W - 1 - j][c], ds[u + j][c], o[c]);
        }
        if (EDGE && a.dstate_out != nullptr && p - L + (W - 1) >= 0) {   // one of the segment's last inputs
#pragma unroll
          for (int c = 0; c < V; ++c) o[c] += load1<BF16>(a.dstate_out, srow + c * (W - 1) + p - L + (W - 1));
        }
        if (!EDGE || p >= 0) {
          *(T*)(dx + (EDGE ? off + (u - (W - 1)) * (int64_t)stride : off + (u - (W - 1)) * stride)) = T::make(o);
        } else if (a.dstate_in != nullptr) {
#pragma unroll
          for (int c = 0; c < V; ++c) store1<BF16>(a.dstate_in, srow + c * (W - 1) + (W - 1) + p, o[c]);
        }
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int c = 0; c < V; ++c) { xs[j][c] = xs[j + U][c]; ds[j][c] = ds[j + U][c]; }
      off += U * stride;
    };
    fetch(t0, off);
    int64_t t = t0;
    for (; t < t0 + W - 1; t += U) step(t, std::true_type{});
    for (; t + U <= t1; t += U) step(t, std::false_type{});
    for (; t < t1 + W - 1; t += U) step(t, std::true_type{});
  }

  // runs of the wave, then the waves
  constexpr int N = (W + 1) * V;
  float acc[N];
#pragma unroll
  for (int c = 0; c < V; ++c) {
#pragma unroll
    for (int k = 0; k < W; ++k) acc[k * V + c] = dw[k][c];
    acc[W * V + c] = db[c];
  }
#pragma unroll
  for (int n = 0; n < N; ++n) {
#pragma unroll
    for (int sh = COLS; sh < 64; sh <<= 1) acc[n] += __shfl_xor(acc[n], sh);
    if ((threadIdx.x & 63) < COLS) red[threadIdx.x >> 6][n][col] = acc[n];
  }
  lds_sync();
  for (int k = threadIdx.x; k < N * COLS; k += kThreads) {
    const int n = k / COLS, cc = k % COLS;
    const int64_t c = ((int64_t)(blockIdx.x % groups) * COLS + cc) * V + n % V;
    if (c < dim)
      a.ws[((int64_t)part * (W + 1) + n / V) * dim + c] = red[0][n][cc] + red[1][n][cc] + red[2][n][cc] + red[3][n][cc];
  }
}

// dweight and dbias from the workgroups' parts, in a fixed order: 64 sums by 4 slices of the parts.
__global__ __launch_bounds__(256) void conv_bwd_sum_kernel(const float* ws, float* dweight, float* dbias, int64_t nparts,
                                                           int64_t dim, int width) {
  __shared__ float red[4][64];
  const int lane = threadIdx.x & 63, slice = threadIdx.x >> 6;
  const int64_t n = dim * (width + 1), i = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.f;
  if (i < n) {
#pragma unroll 8
    for (int64_t p = slice; p < nparts; p += 4) s += ws[p * n + i];
  }
  red[slice][lane] = s;
  lds_sync();
  if (slice != 0 || i >= n) return;
  s = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
  const int64_t k = i / dim, c = i % dim;
  if (k < width) dweight[c * width + k] = s;
  else if (dbias != nullptr) dbias[c] = s;
}

// A segment without tokens hands its state through.
template <bool BF16>
__global__ __launch_bounds__(256) void conv_bwd_state_kernel(const void* dstate_out, void* dstate_in, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) store1<BF16>(dstate_in, i, dstate_out != nullptr ? load1<BF16>(dstate_out, i) : 0.f);
}

int64_t groups_of(int64_t dim, int V) {
  const int64_t cw = V == 1 ? Shape<1>::COLS : Shape<kVec>::COLS * kVec;
  return (dim + cw - 1) / cw;
}
int64_t blocks_of(int64_t seqlen, int V, int run) {
  const int rows = V == 1 ? Shape<1>::ROWS : Shape<kVec>::ROWS;
  return (seqlen + (int64_t)rows * run - 1) / ((int64_t)rows * run);
}
// Tokens of a run: 32 (the W-1 tokens read twice are then a tenth), fewer while that leaves compute units
// without a workgroup.
int run_of(int64_t batch, int64_t seqlen, int64_t dim, int V, int num_cus) {
  int run = 32;
  while (run > 8 && batch * blocks_of(seqlen, V, run) * groups_of(dim, V) < num_cus) run /= 2;
  return run;
}
// Workgroups that share a channel group: about four a compute unit in all, each with as many blocks as the
// others (64 blocks by 43 workgroups left a third of them idle half the time: 36.6 us against 33 by 32), and few
// enough to keep the sum of the parts short.
int64_t parts_of(int64_t batch, int64_t seqlen, int64_t dim, int V, int num_cus) {
  const int64_t want = std::min<int64_t>(kMaxParts, std::max<int64_t>(1, 4 * (int64_t)num_cus / groups_of(dim, V)));
  const int64_t blocks = batch * blocks_of(seqlen, V, run_of(batch, seqlen, dim, V, num_cus));
  const int64_t each = std::max<int64_t>(1, (blocks + want - 1) / want);
  return (blocks + each - 1) / each;
}

template <int W, bool BF16, int V>
void launch(const ConvBwdArgs& a, unsigned grid, unsigned groups, int64_t blocks, hipStream_t st) {
  if (a.silu) conv_bwd_kernel<W, BF16, V, true><<<grid, kThreads, 0, st>>>(a, groups, blocks);
  else conv_bwd_kernel<W, BF16, V, false><<<grid, kThreads, 0, st>>>(a, groups, blocks);
}
template <int W>
void launch_w(const ConvBwdArgs& a, unsigned grid, unsigned groups, int64_t blocks, hipStream_t st) {
  if (a.vec) a.act_bf16 ? launch<W, true, kVec>(a, grid, groups, blocks, st) : launch<W, false, kVec>(a, grid, groups, blocks, st);
  else a.act_bf16 ? launch<W, true, 1>(a, grid, groups, blocks, st) : launch<W, false, 1>(a, grid, groups, blocks, st);
}

}  // namespace

size_t conv_bwd_ws_bytes(int64_t batch, int64_t seqlen, int64_t dim, int64_t width, int num_cus) {
  const int64_t parts = std::max(parts_of(batch, seqlen, dim, 1, num_cus), parts_of(batch, seqlen, dim, kVec, num_cus));
  return (size_t)parts * (size_t)(width + 1) * (size_t)dim * sizeof(float);
}

int launch_conv_bwd(ConvBwdArgs a, int num_cus, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  const int V = a.vec ? kVec : 1;
  a.nparts = 0;
  if (a.seqlen > 0 && a.batch > 0) {
    a.run = run_of(a.batch, a.seqlen, a.dim, V, num_cus);
    const int64_t blocks = blocks_of(a.seqlen, V, a.run), groups = groups_of(a.dim, V);
    a.nparts = parts_of(a.batch, a.seqlen, a.dim, V, num_cus);
    // (a thread's place in its workgroup's block is held in 32 bits)
    if (groups * a.nparts > 0x7fffffffLL || a.dim > 0x7fffffffLL / (4 * 1024)) return fail(4, "dim too large");
    const unsigned grid = (unsigned)(groups * a.nparts);
    switch (a.width) {
      case 1: launch_w<1>(a, grid, (unsigned)groups, blocks, st); break;
      case 2: launch_w<2>(a, grid, (unsigned)groups, blocks, st); break;
      case 3: launch_w<3>(a, grid, (unsigned)groups, blocks, st); break;
      case 4: launch_w<4>(a, grid, (unsigned)groups, blocks, st); break;
      case 5: launch_w<5>(a, grid, (unsigned)groups, blocks, st); break;
      case 6: launch_w<6>(a, grid, (unsigned)groups, blocks, st); break;
      case 7: launch_w<7>(a, grid, (unsigned)groups, blocks, st); break;
      case 8: launch_w<8>(a, grid, (unsigned)groups, blocks, st); break;
      default: return fail(4, "conv width must be 1..8");
    }
  } else if (a.dstate_in != nullptr && a.batch * (a.width - 1) > 0) {
    const int64_t n = a.batch * a.dim * (a.width - 1), grid = (n + 255) / 256;
    if (grid > 0x7fffffffLL) return fail(4, "batch or dim too large");
    if (a.act_bf16) conv_bwd_state_kernel<true><<<(unsigned)grid, 256, 0, st>>>(a.dstate_out, a.dstate_in, n);
    else conv_bwd_state_kernel<false><<<(unsigned)grid, 256, 0, st>>>(a.dstate_out, a.dstate_in, n);
  }
  const int64_t sums = (a.dim * (a.width + 1) + 63) / 64;
  if (sums > 0x7fffffffLL) return fail(4, "dim too large");
  conv_bwd_sum_kernel<<<(unsigned)sums, 256, 0, st>>>(a.ws, a.dweight, a.dbias, a.nparts, a.dim, (int)a.width);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? 0 : fail(6, std::string("conv1d backward launch: ") + hipGetErrorString(e));
}

}  // namespace ssm
