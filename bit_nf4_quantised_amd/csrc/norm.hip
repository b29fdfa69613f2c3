// Root-mean-square norm with the residual's addition, forward and backward (gfx950).
//
// Forward, per row of K values:  h = x + res,  rstd = (mean(h^2) + eps)^(-1/2),  y = h rstd w.
// Backward, n = h rstd:  dx = dh + rstd (w dy - n mean(w dy n)),  dw = sum over rows of dy n,
// dx the gradient of x and of the residual alike, dh what flows into h from elsewhere.
// All arithmetic is fp32, h enters the statistics and y before its rounding to bf16; the outputs are
// rounded once. With an 8-bit checkpoint, the codes are of the rounded y (act8.h).
//
// Both are bound by memory: 8 bytes per value forward (two bf16 in, two out; 9.03 with the codes) and
// 8 backward (dy, h, dh in, dx out). A row is read once and kept in registers, V 16-byte vectors a
// thread: by one wave up to 2048 columns (four rows a workgroup, no barrier), by a workgroup above.
// Measured: 4096 x 8192 forward 51 us (5.3 TB/s), backward with dw 45 + 5 us (6 TB/s for the first; its
// inputs are partly in the memory-side cache); 2048 x 4096 with the checkpoint 14 us (5.4 TB/s). A copy of
// 4 GiB reaches 4.7 TB/s.
#include "act8.h"
#include "launch.h"

namespace nf4 {

__device__ __forceinline__ void unpack8(const u32x4& p, float (&f)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = __uint_as_float(p[k] << 16);
    f[2 * k + 1] = __uint_as_float(p[k] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ u32x4 pack8f(const float (&f)[8]) {
  u32x4 p;
#pragma unroll
  for (int k = 0; k < 4; ++k) p[k] = pack_bf16x2(f[2 * k], f[2 * k + 1]);
  return p;
}

// sum over the wave, in all lanes
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_f<0xB1>(v);
  v += dpp_f<0x4E>(v);
  v += dpp_f<0x141>(v);
  v += dpp_f<0x140>(v);
  const float r0 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 0));
  const float r1 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 16));
  const float r2 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 32));
  const float r3 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 48));
  return (r0 + r1) + (r2 + r3);
}

// sum over the W waves that share a row; `slot` alternates between calls, so one barrier is enough
template <int W>
__device__ __forceinline__ float row_sum(float v, float* slot) {
  v = wave_sum(v);
  if (W == 1) return v;
  if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < W; ++w) s += slot[w];
  return s;
}

// W waves per row, R rows per workgroup, V vectors of 8 columns per thread.
template <int W, int R, int V>
__global__ __launch_bounds__(W * R * 64) void rmsnorm_fwd_kernel(const NormFwdArgs a) {
  __shared__ float slot[W];
  const int t = threadIdx.x % (W * 64), vecs = (int)(a.K / 8);
  const int64_t row = (int64_t)blockIdx.x * R + threadIdx.x / (W * 64);
  if (row >= a.M) return;   // whole waves, and only where a wave has its row alone
  const int64_t base = row * a.K;
  float h[V][8];
  u32x4 px[V], pr[V], pw[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = v * W * 64 + t;
    px[v] = pr[v] = pw[v] = u32x4{0u, 0u, 0u, 0u};
    if (i < vecs) {
      px[v] = *reinterpret_cast<const u32x4*>(a.x + base + 8 * i);
      if (a.res) pr[v] = *reinterpret_cast<const u32x4*>(a.res + base + 8 * i);
      pw[v] = *reinterpret_cast<const u32x4*>(a.w + 8 * i);
    }
  }
  float sq = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float r[8];
    unpack8(px[v], h[v]);
    unpack8(pr[v], r);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[v][e] += r[e];
      sq = __fmaf_rn(h[v][e], h[v][e], sq);
    }
  }
  const float mean = row_sum<W>(sq, slot) / (float)a.K;
  const float rstd = 1.f / sqrtf(mean + a.eps);
  if (a.rstd && t == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = v * W * 64 + t;
    float w[8], y[8];
    unpack8(pw[v], w);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = h[v][e] * rstd * w[e];
    const u32x4 py = pack8f(y);
    // all lanes take part: vecs is a multiple of 8 where codes are asked for
    const uint32_t am = a.codes ? act8_absmax(py) : 0u;
    if (i < vecs) {
      if (a.h) *reinterpret_cast<u32x4*>(a.h + base + 8 * i) = pack8f(h[v]);
      *reinterpret_cast<u32x4*>(a.y + base + 8 * i) = py;
      if (a.codes) {
        *reinterpret_cast<u32x2*>(a.codes + base + 8 * i) = act8_codes(py, am);
        if ((i & 7) == 0) a.absmax[(base + 8 * i) / 64] = (uint16_t)am;
      }
    }
  }
}

// A workgroup takes rows b, b + grid, ... (R at a time) and keeps its sums of dw in registers; they go
// to part[workgroup][K], and rmsnorm_dw_kernel adds them in workgroup order.
template <int W, int R, int V, bool DW>
__global__ __launch_bounds__(W * R * 64) void rmsnorm_bwd_kernel(const NormBwdArgs a, float* part) {
  __shared__ float slot[2][W];
  __shared__ float join[DW && R > 1 ? R : 1][DW && R > 1 ? V * W * 512 : 1];
  const int t = threadIdx.x % (W * 64), sub = threadIdx.x / (W * 64), vecs = (int)(a.K / 8);
  u32x4 pw[V];
  float dw[DW ? V : 1][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = v * W * 64 + t;
    pw[v] = u32x4{0u, 0u, 0u, 0u};
    if (i < vecs) pw[v] = *reinterpret_cast<const u32x4*>(a.w + 8 * i);
    if (DW)
#pragma unroll
      for (int e = 0; e < 8; ++e) dw[v][e] = 0.f;
  }
  int flip = 0;
  for (int64_t row = (int64_t)blockIdx.x * R + sub; row < a.M; row += (int64_t)gridDim.x * R) {
    const int64_t base = row * a.K;
    const float rstd = a.rstd[row];
    u32x4 pd[V], ph[V], pg[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = v * W * 64 + t;
      pd[v] = ph[v] = pg[v] = u32x4{0u, 0u, 0u, 0u};
      if (i < vecs) {
        pd[v] = *reinterpret_cast<const u32x4*>(a.dy + base + 8 * i);
        ph[v] = *reinterpret_cast<const u32x4*>(a.h + base + 8 * i);
        if (a.dh) pg[v] = *reinterpret_cast<const u32x4*>(a.dh + base + 8 * i);
      }
    }
    float dot = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float d[8], h[8], w[8];
      unpack8(pd[v], d);
      unpack8(ph[v], h);
      unpack8(pw[v], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = h[e] * rstd;
        dot = __fmaf_rn(d[e] * w[e], n, dot);
        if (DW) dw[v][e] = __fmaf_rn(d[e], n, dw[v][e]);
      }
    }
    const float mean = row_sum<W>(dot, slot[flip]) / (float)a.K;
    flip ^= 1;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = v * W * 64 + t;
      float d[8], h[8], w[8], g[8];
      unpack8(pd[v], d);
      unpack8(ph[v], h);
      unpack8(pw[v], w);
      unpack8(pg[v], g);
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = __fmaf_rn(rstd, d[e] * w[e] - h[e] * rstd * mean, g[e]);
      if (i < vecs) *reinterpret_cast<u32x4*>(a.dx + base + 8 * i) = pack8f(g);
    }
  }
  if (DW) {
    // the rows' sums of one workgroup, added in row order
    if (R > 1) {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) join[sub][(v * 8 + e) * W * 64 + t] = dw[v][e];
      __syncthreads();
      if (sub) return;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          for (int r = 1; r < R; ++r) dw[v][e] += join[r][(v * 8 + e) * W * 64 + t];
    }
    float* dst = part + (int64_t)blockIdx.x * a.K;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = v * W * 64 + t;
      if (i < vecs) {
        *reinterpret_cast<f32x4*>(dst + 8 * i) = f32x4{dw[v][0], dw[v][1], dw[v][2], dw[v][3]};
        *reinterpret_cast<f32x4*>(dst + 8 * i + 4) = f32x4{dw[v][4], dw[v][5], dw[v][6], dw[v][7]};
      }
    }
  }
}

// dw[k] = (dw[k] +) sum over p of part[p][k]: 64 columns a workgroup, 16 waves take every 16th part,
// and their sums are added in wave order.
__global__ __launch_bounds__(1024) void rmsnorm_dw_kernel(const float* __restrict__ part, int parts, int64_t K, float* dw,
                                                          int accumulate) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t k = min((int64_t)blockIdx.x * 64 + lane, K - 1);
  float s = 0.f;
#pragma unroll 4
  for (int p = wave; p < parts; p += 16) s += part[(int64_t)p * K + k];
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && (int64_t)blockIdx.x * 64 + lane < K) {
    s = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) s += red[w][lane];
    dw[k] = accumulate ? dw[k] + s : s;
  }
}

// Calls f with the shape (waves per row, rows per workgroup, vectors per thread) for K columns.
template <int W, int R, int V>
struct NormShape {
  static constexpr int kW = W, kR = R, kV = V;
};
template <typename F>
static void norm_shape(int64_t K, F f) {
  if (K <= 512) f(NormShape<1, 4, 1>{});
  else if (K <= 1024) f(NormShape<1, 4, 2>{});
  else if (K <= 2048) f(NormShape<1, 4, 4>{});
  else if (K <= 4096) f(NormShape<4, 1, 2>{});
  else if (K <= 8192) f(NormShape<4, 1, 4>{});
  else f(NormShape<8, 1, 4>{});   // K <= 16384
}

// workgroups of the backward: 512 keep the GPU busy, and the sums of dw short
static int norm_bwd_groups(int64_t M, int64_t K) {
  const int64_t rows = K <= 2048 ? (M + 3) / 4 : M;
  return (int)(rows < 512 ? rows : 512);
}
size_t norm_bwd_ws_floats(int64_t M, int64_t K) { return (size_t)norm_bwd_groups(M, K) * (size_t)K; }

// A workgroup has its R rows to itself; more rows than one launch holds threads for take several.
hipError_t launch_rmsnorm_fwd(const NormFwdArgs& args, hipStream_t stream) {
  norm_shape(args.K, [&](auto s) {
    using S = decltype(s);
    constexpr int threads = S::kW * S::kR * 64;
    constexpr int64_t most = kMaxThreads / threads * S::kR;
    for (int64_t row = 0; row < args.M; row += most) {
      NormFwdArgs a = args;
      const int64_t at = row * a.K;
      a.M = args.M - row < most ? args.M - row : most;
      a.x += at;
      if (a.res) a.res += at;
      if (a.h) a.h += at;
      a.y += at;
      if (a.rstd) a.rstd += row;
      if (a.codes) {
        a.codes += at;
        a.absmax += at / 64;
      }
      hipLaunchKernelGGL((rmsnorm_fwd_kernel<S::kW, S::kR, S::kV>), dim3((unsigned)((a.M + S::kR - 1) / S::kR)), dim3(threads), 0,
                         stream, a);
    }
  });
  return hipGetLastError();
}

hipError_t launch_rmsnorm_bwd(const NormBwdArgs& a, float* dw, int accumulate, float* ws, hipStream_t stream) {
  const int groups = norm_bwd_groups(a.M, a.K);
  norm_shape(a.K, [&](auto s) {
    using S = decltype(s);
    const dim3 grid((unsigned)groups), block(S::kW * S::kR * 64);
    if (dw) hipLaunchKernelGGL((rmsnorm_bwd_kernel<S::kW, S::kR, S::kV, true>), grid, block, 0, stream, a, ws);
    else hipLaunchKernelGGL((rmsnorm_bwd_kernel<S::kW, S::kR, S::kV, false>), grid, block, 0, stream, a, ws);
  });
  if (dw)
    hipLaunchKernelGGL(rmsnorm_dw_kernel, dim3((unsigned)((a.K + 63) / 64)), dim3(1024), 0, stream, ws, groups, a.K, dw,
                       accumulate);
  return hipGetLastError();
}

}  // namespace nf4
