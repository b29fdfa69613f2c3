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
// 2^64, is the angle's fraction of a turn, however far the position, to 2^-64 per position. Its top 32 bits
// are reduced to a quadrant and an angle of at most an eighth of a turn by integer operations, and the Taylor
// sums of sine and cosine there (to r^9 and r^10) are within an ulp or two of fp32.
//
// Bound by memory: a value is read once and written once (backward with a weight: dy and x read). A row is
// held by L = 8 (d <= 64) or 16 lanes, 8 values a lane, 4 on either side of the pairs' middle, so that a pair
// never leaves its lane; a lane takes four heads of a token, whose loads are all on their way together and which
// share its four sines and cosines. All sums are fp32; outputs are rounded once.
#include "common.h"
#include "launch.h"

#include <algorithm>

namespace nf4 {

constexpr int kRopeHeads = 4;      // heads of a token that a group of lanes takes at a time
constexpr int kRopeGrid = 2048;    // workgroups at most: they go on to further tokens
constexpr int kRopeSums = 512;     // the same where each leaves partial sums of dw

struct CosSin {
  float c, s;
};
// cosine and sine of a fraction of a turn in units of 2^-32
__device__ __forceinline__ CosSin cos_sin(uint32_t turn) {
  const uint32_t quadrant = (turn + 0x20000000u) >> 30;
  const float r = (float)(int32_t)(turn - (quadrant << 30)) * 1.4629180792671596e-09f;   // 2 pi / 2^32
  const float q = r * r;
  float s = __fmaf_rn(q, 2.7557319e-06f, -1.9841270e-04f);    // 1/9!, 1/7!
  s = __fmaf_rn(q, s, 8.3333333e-03f);                        // 1/5!
  s = __fmaf_rn(q, s, -1.6666667e-01f);                       // 1/3!
  s = __fmaf_rn(r * q, s, r);
  float c = __fmaf_rn(q, -2.7557319e-07f, 2.4801587e-05f);    // 1/10!, 1/8!
  c = __fmaf_rn(q, c, -1.3888889e-03f);                       // 1/6!
  c = __fmaf_rn(q, c, 4.1666667e-02f);                        // 1/4!
  c = __fmaf_rn(q, c, -0.5f);
  c = __fmaf_rn(q, c, 1.f);
  const bool odd = quadrant & 1u;
  const float a = odd ? s : c, b = odd ? c : s;
  CosSin o;
  o.c = (quadrant + 1u) & 2u ? -a : a;
  o.s = quadrant & 2u ? -b : b;
  return o;
}

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

// A lane's place: its 8 values start at columns at0 and at1 (4 each), and whether its pairs are rotated.
struct RopeLane {
  int j, at0, at1;
  bool in, turns;
  template <bool INTER>
  __device__ __forceinline__ void init(int lane, int d, int rot) {
    j = lane;
    in = 8 * j < d;
    turns = 8 * j < rot;
    at0 = !INTER && turns ? 4 * j : 8 * j;
    at1 = !INTER && turns ? rot / 2 + 4 * j : 8 * j + 4;
  }
};

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

// the lane's four angles at a position; sign -1 turns back
template <bool INTER>
__device__ __forceinline__ void angles(CosSin (&cs)[4], const RopeArgs& a, const RopeLane& l, int64_t position, float sign) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    cs[p] = CosSin{1.f, 0.f};
    if (l.turns) {
      cs[p] = cos_sin((uint32_t)(((uint64_t)position * a.turn[4 * l.j + p]) >> 32));
      cs[p].c *= a.factor;
      cs[p].s *= a.factor * sign;
    }
  }
}

// Item: a token's heads 4 c .. 4 c + 3, the query heads first, then the key heads.
struct RopeItem {
  int64_t token;
  int head;
};
__device__ __forceinline__ RopeItem rope_item(int64_t item, int chunks) {
  RopeItem r;
  if ((uint64_t)item >> 31 == 0) {   // the common case without a 64-bit division
    const uint32_t t = (uint32_t)item / (uint32_t)chunks;
    r.token = t;
    r.head = ((uint32_t)item - t * (uint32_t)chunks) * kRopeHeads;
  } else {
    r.token = item / chunks;
    r.head = (int)(item - r.token * chunks) * kRopeHeads;
  }
  return r;
}

__device__ __forceinline__ int64_t row_at(const AttnTensor& q, const AttnTensor& k, int heads, int64_t token, int head, bool key) {
  return key ? token * k.token + (int64_t)(head - heads) * k.head : token * q.token + (int64_t)head * q.head;
}

template <int L, bool INTER, bool NORM>
__global__ __launch_bounds__(256) void rope_fwd_kernel(const RopeArgs a) {
  constexpr int GROUPS = 256 / L;
  RopeLane l;
  l.init<INTER>((int)threadIdx.x % L, a.d, a.rot);
  const int all = a.heads + a.kv_heads, chunks = (all + kRopeHeads - 1) / kRopeHeads;
  const int64_t items = a.tokens * chunks;
  float wq[8], wk[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) wq[e] = wk[e] = 1.f;
  if (NORM && l.in) {
    if (a.qw) {
      unpack4(*reinterpret_cast<const u32x2*>(a.qw + l.at0), wq);
      unpack4(*reinterpret_cast<const u32x2*>(a.qw + l.at1), wq + 4);
    }
    if (a.kw) {
      unpack4(*reinterpret_cast<const u32x2*>(a.kw + l.at0), wk);
      unpack4(*reinterpret_cast<const u32x2*>(a.kw + l.at1), wk + 4);
    }
  }
  const float per = 1.f / (float)a.d;
  // groups of a wave run on together to the last one's end: the row sums need all lanes
  for (int64_t i0 = (int64_t)blockIdx.x * GROUPS; i0 < items; i0 += (int64_t)gridDim.x * GROUPS) {
    const int64_t item = i0 + threadIdx.x / L;
    const RopeItem it = rope_item(item < items ? item : items - 1, chunks);
    const bool live = item < items && l.in;
    u32x2 p0[kRopeHeads], p1[kRopeHeads];
#pragma unroll
    for (int h = 0; h < kRopeHeads; ++h) {
      const int head = it.head + h;
      p0[h] = p1[h] = u32x2{0u, 0u};
      if (live && head < all) {
        const bool key = head >= a.heads;
        const uint16_t* x = (key ? a.k.p : a.q.p) + row_at(a.q, a.k, a.heads, it.token, head, key);
        p0[h] = *reinterpret_cast<const u32x2*>(x + l.at0);
        p1[h] = *reinterpret_cast<const u32x2*>(x + l.at1);
      }
    }
    CosSin cs[4];
    if (a.rot) angles<INTER>(cs, a, l, a.pos[it.token], 1.f);
#pragma unroll
    for (int h = 0; h < kRopeHeads; ++h) {
      const int head = it.head + h;
      const bool key = head >= a.heads;
      float x[8];
      unpack4(p0[h], x);
      unpack4(p1[h], x + 4);
      if (NORM) {
        float sq = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sq = __fmaf_rn(x[e], x[e], sq);
        const float rstd = 1.f / sqrtf(row_total<L>(sq) * per + a.eps);
        if (key ? a.kw != nullptr : a.qw != nullptr) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= rstd * (key ? wk[e] : wq[e]);
        }
      }
      if (l.turns) rotate<INTER>(x, cs);
      if (live && head < all) {
        uint16_t* y = (key ? a.ko.p : a.qo.p) + row_at(a.qo, a.ko, a.heads, it.token, head, key);
        *reinterpret_cast<u32x2*>(y + l.at0) = pack4(x);
        *reinterpret_cast<u32x2*>(y + l.at1) = pack4(x + 4);
      }
    }
  }
}

// Backward: q, k are the forward's inputs (with a weight), qo, ko the gradients of its outputs, dq, dk what is
// asked for. Sums of dw are kept per lane, added over the workgroup's groups in order and left in
// part[workgroup][query, key][128]; rope_dw_kernel adds the workgroups', in order.
template <int L, bool INTER, bool NORM, bool DW>
__global__ __launch_bounds__(256) void rope_bwd_kernel(const RopeArgs a, float* part) {
  constexpr int GROUPS = 256 / L;
  RopeLane l;
  l.init<INTER>((int)threadIdx.x % L, a.d, a.rot);
  const int all = a.heads + a.kv_heads, chunks = (all + kRopeHeads - 1) / kRopeHeads;
  const int64_t items = a.tokens * chunks;
  float wq[8], wk[8], sq_[8], sk_[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    wq[e] = wk[e] = 1.f;
    sq_[e] = sk_[e] = 0.f;
  }
  if (NORM && l.in) {
    if (a.qw) {
      unpack4(*reinterpret_cast<const u32x2*>(a.qw + l.at0), wq);
      unpack4(*reinterpret_cast<const u32x2*>(a.qw + l.at1), wq + 4);
    }
    if (a.kw) {
      unpack4(*reinterpret_cast<const u32x2*>(a.kw + l.at0), wk);
      unpack4(*reinterpret_cast<const u32x2*>(a.kw + l.at1), wk + 4);
    }
  }
  const float per = 1.f / (float)a.d;
  for (int64_t i0 = (int64_t)blockIdx.x * GROUPS; i0 < items; i0 += (int64_t)gridDim.x * GROUPS) {
    const int64_t item = i0 + threadIdx.x / L;
    const RopeItem it = rope_item(item < items ? item : items - 1, chunks);
    const bool live = item < items && l.in;
    u32x2 g0[kRopeHeads], g1[kRopeHeads], x0[kRopeHeads], x1[kRopeHeads];
#pragma unroll
    for (int h = 0; h < kRopeHeads; ++h) {
      const int head = it.head + h;
      g0[h] = g1[h] = x0[h] = x1[h] = u32x2{0u, 0u};
      if (live && head < all) {
        const bool key = head >= a.heads;
        const uint16_t* g = (key ? a.ko.p : a.qo.p) + row_at(a.qo, a.ko, a.heads, it.token, head, key);
        g0[h] = *reinterpret_cast<const u32x2*>(g + l.at0);
        g1[h] = *reinterpret_cast<const u32x2*>(g + l.at1);
        if (NORM && (key ? a.kw != nullptr : a.qw != nullptr)) {
          const uint16_t* x = (key ? a.k.p : a.q.p) + row_at(a.q, a.k, a.heads, it.token, head, key);
          x0[h] = *reinterpret_cast<const u32x2*>(x + l.at0);
          x1[h] = *reinterpret_cast<const u32x2*>(x + l.at1);
        }
      }
    }
    CosSin cs[4];
    if (a.rot) angles<INTER>(cs, a, l, a.pos[it.token], -1.f);
#pragma unroll
    for (int h = 0; h < kRopeHeads; ++h) {
      const int head = it.head + h;
      const bool key = head >= a.heads;
      float g[8];
      unpack4(g0[h], g);
      unpack4(g1[h], g + 4);
      if (l.turns) rotate<INTER>(g, cs);
      if (NORM) {
        float n[8], sq = 0.f, wgn = 0.f;
        unpack4(x0[h], n);
        unpack4(x1[h], n + 4);
#pragma unroll
        for (int e = 0; e < 8; ++e) sq = __fmaf_rn(n[e], n[e], sq);
        const float rstd = 1.f / sqrtf(row_total<L>(sq) * per + a.eps);
        const bool normed = key ? a.kw != nullptr : a.qw != nullptr;
        float wg[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          n[e] *= rstd;
          wg[e] = g[e] * (key ? wk[e] : wq[e]);
          wgn = __fmaf_rn(wg[e], n[e], wgn);
        }
        const float mean = row_total<L>(wgn) * per;
        if (normed && live && head < all) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (DW) {
              const float t = g[e] * n[e];
              sq_[e] += key ? 0.f : t;
              sk_[e] += key ? t : 0.f;
            }
            g[e] = rstd * __fmaf_rn(-n[e], mean, wg[e]);
          }
        }
      }
      if (live && head < all) {
        uint16_t* y = (key ? a.dk.p : a.dq.p) + row_at(a.dq, a.dk, a.heads, it.token, head, key);
        *reinterpret_cast<u32x2*>(y + l.at0) = pack4(g);
        *reinterpret_cast<u32x2*>(y + l.at1) = pack4(g + 4);
      }
    }
  }
  if constexpr (DW) {
    __shared__ float sums[GROUPS][2][L * 8];
    if (l.in) {
      float* s = sums[threadIdx.x / L][0];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = (e < 4 ? l.at0 : l.at1) + (e & 3);
        s[c] = sq_[e];
        s[L * 8 + c] = sk_[e];
      }
    }
    __syncthreads();
    const int c = (int)threadIdx.x & 127, which = (int)threadIdx.x >> 7;
    if (c < a.d) {
      float v = 0.f;
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) v += sums[g][which][c];
      part[(int64_t)blockIdx.x * 256 + threadIdx.x] = v;
    }
  }
}

// dw from the workgroups' sums: 16 columns a workgroup, thread (slice, column) adds every 16th workgroup's, and
// the slices are added in order
__global__ __launch_bounds__(256) void rope_dw_kernel(const float* part, int workgroups, int d, float* dqw, float* dkw,
                                                      int accumulate) {
  __shared__ float s[16][17];
  const int x = (int)threadIdx.x & 15, slice = (int)threadIdx.x >> 4;
  const int col = (int)blockIdx.x * 16 + x;   // of 256: query columns, then key columns
  float v = 0.f;
  for (int w = slice; w < workgroups; w += 16) v += part[(int64_t)w * 256 + col];
  s[slice][x] = v;
  __syncthreads();
  if (slice) return;
  float* out = col < 128 ? dqw : dkw;
  const int c = col & 127;
  if (c >= d || !out) return;
  v = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) v += s[k][x];
  out[c] = accumulate ? out[c] + v : v;
}

// ------------------------------------------------------------------------------------------
// Host side
static int64_t rope_workgroups(const RopeArgs& a, int64_t most) {
  const int64_t chunks = (a.heads + a.kv_heads + kRopeHeads - 1) / kRopeHeads;
  const int64_t groups = a.d <= 64 ? 32 : 16;
  return std::min<int64_t>(most, (a.tokens * chunks + groups - 1) / groups);
}

size_t rope_bwd_ws_floats(const RopeArgs& a) { return (size_t)rope_workgroups(a, kRopeSums) * 256; }

template <bool INTER, bool NORM>
static void rope_fwd(const RopeArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)rope_workgroups(a, kRopeGrid));
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
static void rope_bwd(const RopeArgs& a, float* part, hipStream_t stream) {
  const dim3 grid((unsigned)rope_workgroups(a, DW ? kRopeSums : kRopeGrid));
  if (a.d <= 64) hipLaunchKernelGGL((rope_bwd_kernel<8, INTER, NORM, DW>), grid, dim3(256), 0, stream, a, part);
  else hipLaunchKernelGGL((rope_bwd_kernel<16, INTER, NORM, DW>), grid, dim3(256), 0, stream, a, part);
}

hipError_t launch_rope_bwd(const RopeArgs& a, float* dqw, float* dkw, int accumulate, float* part, hipStream_t stream) {
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
  hipLaunchKernelGGL(rope_dw_kernel, dim3(16), dim3(256), 0, stream, part, (int)rope_workgroups(a, kRopeSums), a.d, dqw, dkw,
                     accumulate);
  return hipGetLastError();
}

}  // namespace nf4
