// Rotary positions of query and key heads, with the heads' norms in the same pass, and the backward (gfx950).
//
// One row x of d values per token and head; with a weight w it is normed first: n = x rstd, z = n w,
// rstd = (mean(x^2) + eps)^(-1/2); without one z = x. Its first `rot` features are rotated in pairs (a, b) by the
// angle t_i = position * inv_freq[i] of the pair i:
//   y_a = f (z_a cos t_i - z_b sin t_i)    y_b = f (z_b cos t_i + z_a sin t_i)    (f: the config's factor)
// and the others stay. Backward: g = the pairs of dy rotated back (the transpose, times f), then
//   dx = rstd (w g - n mean(w g n)),  dw = sum over tokens and heads of g n    (without a weight dx = g).
//
// Angles are held in turns, as 64-bit fractions: a position times the frequency in units of 2^-64 turns, modulo
// 2^64, is the angle's fraction of a turn, however far the position, to 2^-64 a position. Its top 32 bits go, as
// a signed fraction, to the hardware's sine and cosine, which take turns (within 1.3e-7 of the exact ones over
// half a turn either way).
//
// Bound by memory: a value is read once and written once (backward with a weight: dy and x read). A row is
// held by L = 8 (d <= 64) or 16 lanes, 8 values a lane, 4 on either side of the pairs' middle, so that a pair never
// leaves its lane. A workgroup works on queries or on keys alone, so that strides and weights are the same for
// all its lanes; a group of L lanes takes heads of one token, four at a time, whose loads are all on their way
// together and which share the lane's four sines and cosines. All sums are fp32; outputs are rounded once.
// 4096 tokens of 64 and 8 heads, d 128, normed: forward 25 us (151 MB, 6.0 TB/s), backward 42 (226 MB, 5.4 TB/s) and
// 4.4 for the weights' sums; 32 and 56 with queries and keys in one workgroup and sines by polynomials. 2048 tokens of 32 and 8
// heads, not normed: 9.4 either way (42 MB, 4.5 TB/s). One token: 3.3, the latency of its arguments and loads.
#include "common.h"
#include "rope_plan.h"

namespace nf4 {

struct CosSin {
  float c, s;
};

// sum over the L lanes of a row, in all of them
template <int L>
__device__ __forceinline__ float row_total(float v) {
  v += dpp_f<0xB1>(v);
  v += dpp_f<0x4E>(v);
  v += dpp_f<0x141>(v);
  if (L == 16) v += dpp_f<0x140>(v);
  return v;
}

__device__ __forceinline__ void unpack4(const u32x2& p, float* f) {
  f[0] = __uint_as_float(p[0] << 16);
  f[1] = __uint_as_float(p[0] & 0xFFFF0000u);
  f[2] = __uint_as_float(p[1] << 16);
  f[3] = __uint_as_float(p[1] & 0xFFFF0000u);
}
__device__ __forceinline__ u32x2 pack4(const float* f) { return u32x2{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])}; }

// pair p of the lane's 8 values: neighbours, or the same place on either side
template <bool INTER>
__device__ __forceinline__ void rotate(float (&x)[8], const CosSin (&cs)[4]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int a = INTER ? 2 * p : p, b = INTER ? 2 * p + 1 : p + 4;
    const float xa = x[a], xb = x[b];
    x[a] = __fmaf_rn(xa, cs[p].c, -xb * cs[p].s);
    x[b] = __fmaf_rn(xb, cs[p].c, xa * cs[p].s);
  }
}

// What a workgroup and a lane of it work on: the queries or the keys, and where the lane's 8 values start (4 each).
template <int L, bool INTER>
struct RopeWork {
  static constexpr int GROUPS = 256 / L;
  bool key, in, turns;
  int heads, chunks, first, count, j, at0, at1;   // workgroups first .. first + count - 1 share the work
  int64_t items;
  uint64_t turn[4];
  __device__ __forceinline__ explicit RopeWork(const RopeArgs& a) {
    key = (int)blockIdx.x >= a.q_groups;
    heads = key ? a.kv_heads : a.heads;
    first = key ? a.q_groups : 0;
    count = key ? (int)gridDim.x - a.q_groups : a.q_groups;
    chunks = (heads + a.per - 1) / a.per;
    items = a.tokens * chunks;
    j = (int)threadIdx.x % L;
    in = 8 * j < a.d;
    turns = 8 * j < a.rot;
    at0 = !INTER && turns ? 4 * j : 8 * j;
    at1 = !INTER && turns ? a.rot / 2 + 4 * j : 8 * j + 4;
#pragma unroll
    for (int p = 0; p < 4; ++p) turn[p] = turns ? a.turn[4 * j + p] : 0;
  }
  __device__ __forceinline__ void weight(float (&w)[8], const uint16_t* p) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 1.f;
    if (!in) return;
    unpack4(*reinterpret_cast<const u32x2*>(p + at0), w);
    unpack4(*reinterpret_cast<const u32x2*>(p + at1), w + 4);
  }
  // the item's token and first head
  __device__ __forceinline__ void item(int64_t i, int per, int64_t& token, int& head) const {
    if ((uint64_t)items >> 32 == 0) {   // without a 64-bit division
      const uint32_t t = (uint32_t)i / (uint32_t)chunks;
      token = t;
      head = (int)((uint32_t)i - t * (uint32_t)chunks) * per;
    } else {
      token = i / chunks;
      head = (int)(i - token * chunks) * per;
    }
  }
  // sines and cosines of the lane's four pairs; sign -1 turns back
  __device__ __forceinline__ void angles(CosSin (&cs)[4], int64_t position, float factor, float sign) const {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float x = (float)(int32_t)((uint64_t)position * turn[p] >> 32) * 0x1p-32f;
      cs[p].c = __builtin_amdgcn_cosf(x) * factor;
      cs[p].s = __builtin_amdgcn_sinf(x) * (factor * sign);
    }
  }
};

template <int L, bool INTER, bool NORM>
__global__ __launch_bounds__(256) void rope_fwd_kernel(const RopeArgs a) {
  typedef RopeWork<L, INTER> Work;
  const Work w(a);
  const AttnTensor& in = w.key ? a.k : a.q;
  const AttnTensor& out = w.key ? a.ko : a.qo;
  const uint16_t* weight = w.key ? a.kw : a.qw;
  const bool normed = NORM && weight;
  float wt[8];
  if (normed) w.weight(wt, weight);
  const float per = 1.f / (float)a.d;
  // groups of a wave run on together to the last one's end: the row sums need all lanes
  for (int64_t i0 = (int64_t)((int)blockIdx.x - w.first) * Work::GROUPS; i0 < w.items; i0 += (int64_t)w.count * Work::GROUPS) {
    const int64_t item = i0 + threadIdx.x / L;
    int64_t token;
    int head0;
    w.item(item < w.items ? item : w.items - 1, a.per, token, head0);
    const bool live = item < w.items && w.in;
    const uint16_t* x0 = in.p + token * in.token + (int64_t)head0 * in.head;
    uint16_t* y0 = out.p + token * out.token + (int64_t)head0 * out.head;
    CosSin cs[4];
    if (a.rot) w.angles(cs, a.pos[token], a.factor, 1.f);
    for (int b = 0; b < a.per; b += kRopeHeads) {
      u32x2 p0[kRopeHeads], p1[kRopeHeads];
#pragma unroll
      for (int h = 0; h < kRopeHeads; ++h) {
        p0[h] = p1[h] = u32x2{0u, 0u};
        if (live && head0 + b + h < w.heads) {
          const uint16_t* x = x0 + (int64_t)(b + h) * in.head;
          p0[h] = *reinterpret_cast<const u32x2*>(x + w.at0);
          p1[h] = *reinterpret_cast<const u32x2*>(x + w.at1);
        }
      }
#pragma unroll
      for (int h = 0; h < kRopeHeads; ++h) {
        float x[8];
        unpack4(p0[h], x);
        unpack4(p1[h], x + 4);
        if (normed) {
          float sq = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) sq = __fmaf_rn(x[e], x[e], sq);
          const float rstd = __builtin_amdgcn_rsqf(__fmaf_rn(row_total<L>(sq), per, a.eps));
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= rstd * wt[e];
        }
        if (w.turns) rotate<INTER>(x, cs);
        if (live && head0 + b + h < w.heads) {
          uint16_t* y = y0 + (int64_t)(b + h) * out.head;
          *reinterpret_cast<u32x2*>(y + w.at0) = pack4(x);
          *reinterpret_cast<u32x2*>(y + w.at1) = pack4(x + 4);
        }
      }
    }
  }
}

// Backward: q, k are the forward's inputs (with a weight), qo, ko the gradients of its outputs, dq, dk what is
// asked for. Sums of dw are kept per lane, added over the workgroup's groups in order and left in
// part[workgroup][128]; rope_dw_kernel adds the workgroups', in order.
template <int L, bool INTER, bool NORM, bool DW>
__global__ __launch_bounds__(256) void rope_bwd_kernel(const RopeArgs a, float* part) {
  typedef RopeWork<L, INTER> Work;
  const Work w(a);
  const AttnTensor& grad = w.key ? a.ko : a.qo;
  const AttnTensor& in = w.key ? a.k : a.q;
  const AttnTensor& out = w.key ? a.dk : a.dq;
  const uint16_t* weight = w.key ? a.kw : a.qw;
  const bool normed = NORM && weight;
  float wt[8], sum[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.f;
  if (normed) w.weight(wt, weight);
  const float per = 1.f / (float)a.d;
  for (int64_t i0 = (int64_t)((int)blockIdx.x - w.first) * Work::GROUPS; i0 < w.items; i0 += (int64_t)w.count * Work::GROUPS) {
    const int64_t item = i0 + threadIdx.x / L;
    int64_t token;
    int head0;
    w.item(item < w.items ? item : w.items - 1, a.per, token, head0);
    const bool live = item < w.items && w.in;
    const uint16_t* gp = grad.p + token * grad.token + (int64_t)head0 * grad.head;
    const uint16_t* xp = in.p + token * in.token + (int64_t)head0 * in.head;
    uint16_t* yp = out.p + token * out.token + (int64_t)head0 * out.head;
    CosSin cs[4];
    if (a.rot) w.angles(cs, a.pos[token], a.factor, -1.f);
    for (int b = 0; b < a.per; b += kRopeHeads) {
      u32x2 g0[kRopeHeads], g1[kRopeHeads], x0[kRopeHeads], x1[kRopeHeads];
#pragma unroll
      for (int h = 0; h < kRopeHeads; ++h) {
        g0[h] = g1[h] = x0[h] = x1[h] = u32x2{0u, 0u};
        if (live && head0 + b + h < w.heads) {
          const uint16_t* g = gp + (int64_t)(b + h) * grad.head;
          g0[h] = *reinterpret_cast<const u32x2*>(g + w.at0);
          g1[h] = *reinterpret_cast<const u32x2*>(g + w.at1);
          if (normed) {
            const uint16_t* x = xp + (int64_t)(b + h) * in.head;
            x0[h] = *reinterpret_cast<const u32x2*>(x + w.at0);
            x1[h] = *reinterpret_cast<const u32x2*>(x + w.at1);
          }
        }
      }
#pragma unroll
      for (int h = 0; h < kRopeHeads; ++h) {
        const bool valid = live && head0 + b + h < w.heads;
        float g[8];
        unpack4(g0[h], g);
        unpack4(g1[h], g + 4);
        if (w.turns) rotate<INTER>(g, cs);
        if (normed) {
          float n[8], wg[8], sq = 0.f, wgn = 0.f;
          unpack4(x0[h], n);
          unpack4(x1[h], n + 4);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            sq = __fmaf_rn(n[e], n[e], sq);
            wg[e] = g[e] * wt[e];
            wgn = __fmaf_rn(wg[e], n[e], wgn);
          }
          const float rstd = __builtin_amdgcn_rsqf(__fmaf_rn(row_total<L>(sq), per, a.eps));
          // mean(w g n) and n itself are those of x times rstd
          const float mean = row_total<L>(wgn) * per * rstd;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            n[e] *= rstd;
            if (DW && valid) sum[e] = __fmaf_rn(g[e], n[e], sum[e]);
            g[e] = rstd * __fmaf_rn(-n[e], mean, wg[e]);
          }
        }
        if (valid) {
          uint16_t* y = yp + (int64_t)(b + h) * out.head;
          *reinterpret_cast<u32x2*>(y + w.at0) = pack4(g);
          *reinterpret_cast<u32x2*>(y + w.at1) = pack4(g + 4);
        }
      }
    }
  }
  if constexpr (DW) {
    __shared__ float sums[Work::GROUPS][L * 8];
    if (w.in) {
#pragma unroll
      for (int e = 0; e < 8; ++e) sums[threadIdx.x / L][(e < 4 ? w.at0 : w.at1) + (e & 3)] = sum[e];
    }
    __syncthreads();
    const int c = (int)threadIdx.x;
    if (c < a.d) {
      float v = 0.f;
#pragma unroll
      for (int g = 0; g < Work::GROUPS; ++g) v += sums[g][c];
      part[(int64_t)blockIdx.x * 128 + c] = v;
    }
  }
}

// dw from the workgroups' sums: workgroup (x, y) takes columns 8 x .. 8 x + 7 of the queries' (y = 0) or the keys' weight;
// thread (slice, column) adds every 128th workgroup's sums, and the slices are added in order, by sixteens.
__global__ __launch_bounds__(1024) void rope_dw_kernel(const float* part, int q_groups, int groups, int d, float* dqw, float* dkw,
                                                      int accumulate) {
  __shared__ float s[128][9];
  const int x = (int)threadIdx.x & 7, slice = (int)threadIdx.x >> 3, c = (int)blockIdx.x * 8 + x;
  float* out = blockIdx.y ? dkw : dqw;
  if (!out) return;   // the whole workgroup
  const int from = blockIdx.y ? q_groups : 0, to = blockIdx.y ? groups : q_groups;
  float v = 0.f;
  for (int w = from + slice; w < to; w += 128 * 16) {   // sixteen on their way; past the end the last again, not added
    float p[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) p[k] = part[(int64_t)min(w + 128 * k, to - 1) * 128 + c];
#pragma unroll
    for (int k = 0; k < 16; ++k) v += w + 128 * k < to ? p[k] : 0.f;
  }
  s[slice][x] = v;
  __syncthreads();
  if (slice >= 8) return;
  v = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) v += s[16 * slice + k][x];
  s[16 * slice][x] = v;
  wave_lds_order();   // the first wave alone is left
  if (slice) return;
  v = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) v += s[16 * k][x];
  out[c] = accumulate ? out[c] + v : v;
}

// ------------------------------------------------------------------------------------------
// Host side
size_t rope_bwd_ws_floats(RopeArgs a) { return (size_t)rope_plan(a, true) * 128; }

template <bool INTER, bool NORM>
static void rope_fwd(RopeArgs a, hipStream_t stream) {
  const dim3 grid((unsigned)rope_plan(a, false));
  if (a.d <= 64) hipLaunchKernelGGL((rope_fwd_kernel<8, INTER, NORM>), grid, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((rope_fwd_kernel<16, INTER, NORM>), grid, dim3(256), 0, stream, a);
}

hipError_t launch_rope_fwd(const RopeArgs& a, hipStream_t stream) {
  const bool norm = a.qw || a.kw;
  if (a.interleaved) norm ? rope_fwd<true, true>(a, stream) : rope_fwd<true, false>(a, stream);
  else norm ? rope_fwd<false, true>(a, stream) : rope_fwd<false, false>(a, stream);
  return hipGetLastError();
}

template <bool INTER, bool NORM, bool DW>
static void rope_bwd(RopeArgs a, float* part, hipStream_t stream) {
  const dim3 grid((unsigned)rope_plan(a, DW));
  if (a.d <= 64) hipLaunchKernelGGL((rope_bwd_kernel<8, INTER, NORM, DW>), grid, dim3(256), 0, stream, a, part);
  else hipLaunchKernelGGL((rope_bwd_kernel<16, INTER, NORM, DW>), grid, dim3(256), 0, stream, a, part);
}

static hipError_t rope_dw(const float* part, int q_groups, int groups, int d, float* dqw, float* dkw, int accumulate, hipStream_t stream) {
  hipLaunchKernelGGL(rope_dw_kernel, dim3((unsigned)(d / 8), 2), dim3(1024), 0, stream, part, q_groups, groups, d, dqw, dkw, accumulate);
  return hipGetLastError();
}

hipError_t launch_rope_no_dw(int d, float* dqw, float* dkw, hipStream_t stream) { return rope_dw(nullptr, 0, 0, d, dqw, dkw, 0, stream); }

hipError_t launch_rope_bwd(const RopeArgs& args, float* dqw, float* dkw, int accumulate, float* part, hipStream_t stream) {
  const RopeArgs& a = args;
  const bool norm = a.qw || a.kw, dw = dqw || dkw;
  if (a.interleaved) {
    if (dw) rope_bwd<true, true, true>(a, part, stream);
    else if (norm) rope_bwd<true, true, false>(a, part, stream);
    else rope_bwd<true, false, false>(a, part, stream);
  } else {
    if (dw) rope_bwd<false, true, true>(a, part, stream);
    else if (norm) rope_bwd<false, true, false>(a, part, stream);
    else rope_bwd<false, false, false>(a, part, stream);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !dw) return e;
  RopeArgs p = a;
  const int groups = rope_plan(p, true);
  return rope_dw(part, p.q_groups, groups, a.d, dqw, dkw, accumulate, stream);
}

}  // namespace nf4
