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
// order.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "device_common.h"
#include "ssm_internal.h"
#include "vec_io.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxParts = 64;  // workgroups that share a channel group

template <bool BF16, int V>
__device__ __forceinline__ void load_v(const void* p, int64_t i, float (&v)[V]) {
  if constexpr (V == 4) load4<BF16>(p, i, v);
  else v[0] = load1<BF16>(p, i);
}
template <bool BF16, int V>
__device__ __forceinline__ void store_v(void* p, int64_t i, const float (&v)[V]) {
  if constexpr (V == 4) store4<BF16>(p, i, v);
  else store1<BF16>(p, i, v[0]);
}

// A workgroup is COLS threads of V channels by ROWS runs.
template <int V>
struct Shape {
  static constexpr int COLS = V == 4 ? 16 : 32;
  static constexpr int ROWS = kThreads / COLS;
};

template <int W, bool BF16, int V>
__global__ __launch_bounds__(kThreads) void conv_bwd_kernel(ConvBwdArgs a, unsigned groups, int64_t blocks_per_row) {
  constexpr int COLS = Shape<V>::COLS, ROWS = Shape<V>::ROWS;
  __shared__ float red[4][(W + 1) * V][COLS];
  const int64_t L = a.seqlen, dim = a.dim;
  const int col = threadIdx.x % COLS, run = threadIdx.x / COLS;
  const unsigned part = blockIdx.x / groups;
  const int64_t c0 = ((int64_t)(blockIdx.x % groups) * COLS + col) * V;
  const bool active = c0 < dim;

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

  const int64_t nblk = a.batch * blocks_per_row;
  for (int64_t blk = part; blk < nblk; blk += a.nparts) {
    const int64_t b = blk / blocks_per_row;
    const int64_t t0 = ((blk % blocks_per_row) * ROWS + run) * a.run;
    if (!active || t0 >= L) continue;
    const int64_t t1 = min(L, t0 + a.run);
    const int64_t row0 = b * L;
    const int64_t srow = (b * dim + c0) * (W - 1);
    float xw[W][V], dp[W][V];   // xx[t-(W-1)+k]; dpre at p+j, p = t-(W-1)
#pragma unroll
    for (int k = 0; k < W; ++k) {
#pragma unroll
      for (int c = 0; c < V; ++c) { xw[k][c] = 0.f; dp[k][c] = 0.f; }
      const int64_t pos = t0 - (W - 1) + k;
      if (k < W - 1) {
        if (pos >= 0) {
          load_v<BF16, V>(a.x, (row0 + pos) * dim + c0, xw[k]);
        } else if (a.state_in != nullptr) {
#pragma unroll
          for (int c = 0; c < V; ++c) xw[k][c] = load1<BF16>(a.state_in, srow + c * (W - 1) + (W - 1) + pos);
        }
      }
    }
#pragma unroll 4
    for (int64_t t = t0; t < t1 + W - 1; ++t) {
      float d[V];
#pragma unroll
      for (int c = 0; c < V; ++c) d[c] = 0.f;
      if (t < L) {
        load_v<BF16, V>(a.x, (row0 + t) * dim + c0, xw[W - 1]);
        load_v<BF16, V>(a.dout, (row0 + t) * dim + c0, d);
        if (a.silu) {
#pragma unroll
          for (int c = 0; c < V; ++c) {
            float pre = bs[c];
#pragma unroll
            for (int k = 0; k < W; ++k) pre = fmaf(wt[k][c], xw[k][c], pre);
            const float s = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-pre * 1.4426950408889634f));
            d[c] *= s * fmaf(pre, 1.f - s, 1.f);
          }
        }
        if (t < t1) {
#pragma unroll
          for (int c = 0; c < V; ++c) {
            db[c] += d[c];
#pragma unroll
            for (int k = 0; k < W; ++k) dw[k][c] = fmaf(d[c], xw[k][c], dw[k][c]);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int c = 0; c < V; ++c) { dp[j][c] = dp[j + 1][c]; xw[j][c] = xw[j + 1][c]; }
#pragma unroll
      for (int c = 0; c < V; ++c) dp[W - 1][c] = d[c];
      const int64_t p = t - (W - 1);
      if (p >= t0 || t0 == 0) {
        float o[V];
#pragma unroll
        for (int c = 0; c < V; ++c) {
          o[c] = 0.f;
#pragma unroll
          for (int j = 0; j < W; ++j) o[c] = fmaf(wt[W - 1 - j][c], dp[j][c], o[c]);
        }
        const int64_t q = p - L + (W - 1);   // place in the carried-out state
        if (a.dstate_out != nullptr && q >= 0) {
#pragma unroll
          for (int c = 0; c < V; ++c) o[c] += load1<BF16>(a.dstate_out, srow + c * (W - 1) + q);
        }
        if (p >= 0) {
          store_v<BF16, V>(a.dx, (row0 + p) * dim + c0, o);
        } else if (a.dstate_in != nullptr) {
#pragma unroll
          for (int c = 0; c < V; ++c) store1<BF16>(a.dstate_in, srow + c * (W - 1) + (W - 1) + p, o[c]);
        }
      }
    }
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
  const int64_t cw = V == 4 ? Shape<4>::COLS * 4 : Shape<1>::COLS;
  return (dim + cw - 1) / cw;
}
int64_t blocks_of(int64_t seqlen, int V, int run) {
  const int rows = V == 4 ? Shape<4>::ROWS : Shape<1>::ROWS;
  return (seqlen + (int64_t)rows * run - 1) / ((int64_t)rows * run);
}
// Tokens of a run: 32 (the W-1 tokens read twice are then a tenth), fewer while that leaves compute units
// without a workgroup.
int run_of(int64_t batch, int64_t seqlen, int64_t dim, int V, int num_cus) {
  int run = 32;
  while (run > 8 && batch * blocks_of(seqlen, V, run) * groups_of(dim, V) < num_cus) run /= 2;
  return run;
}
// Enough workgroups for four a compute unit, as many parts at most as keep the sum of the parts short.
int64_t parts_of(int64_t batch, int64_t seqlen, int64_t dim, int V, int num_cus) {
  const int64_t want = (4 * (int64_t)num_cus + groups_of(dim, V) - 1) / groups_of(dim, V);
  const int64_t blocks = batch * blocks_of(seqlen, V, run_of(batch, seqlen, dim, V, num_cus));
  return std::min<int64_t>(std::min<int64_t>(blocks, kMaxParts), std::max<int64_t>(want, 1));
}

template <int W>
void launch_w(const ConvBwdArgs& a, unsigned grid, unsigned groups, int64_t blocks, hipStream_t st) {
  if (a.vec) {
    if (a.act_bf16) conv_bwd_kernel<W, true, 4><<<grid, kThreads, 0, st>>>(a, groups, blocks);
    else conv_bwd_kernel<W, false, 4><<<grid, kThreads, 0, st>>>(a, groups, blocks);
  } else {
    if (a.act_bf16) conv_bwd_kernel<W, true, 1><<<grid, kThreads, 0, st>>>(a, groups, blocks);
    else conv_bwd_kernel<W, false, 1><<<grid, kThreads, 0, st>>>(a, groups, blocks);
  }
}

}  // namespace

size_t conv_bwd_ws_bytes(int64_t batch, int64_t seqlen, int64_t dim, int64_t width, int num_cus) {
  const int64_t parts = std::max(parts_of(batch, seqlen, dim, 1, num_cus), parts_of(batch, seqlen, dim, 4, num_cus));
  return (size_t)parts * (size_t)(width + 1) * (size_t)dim * sizeof(float);
}

int launch_conv_bwd(ConvBwdArgs a, int num_cus, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  const int V = a.vec ? 4 : 1;
  a.nparts = 0;
  if (a.seqlen > 0 && a.batch > 0) {
    a.run = run_of(a.batch, a.seqlen, a.dim, V, num_cus);
    const int64_t blocks = blocks_of(a.seqlen, V, a.run), groups = groups_of(a.dim, V);
    a.nparts = parts_of(a.batch, a.seqlen, a.dim, V, num_cus);
    if (groups * a.nparts > 0x7fffffffLL) return fail(4, "dim too large");
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
