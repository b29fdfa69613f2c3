// Keys and values to and from a 4-bit cache (gfx950; format in kv4.h).
//
// The new tokens of every sequence go behind the others it holds: token i of a sequence with nq new ones, nk in
// all, goes to the cache's token k0 + nk - nq + i; reading goes the other way. Two lanes hold a block of a key and of
// its value, 16 values a lane. A workgroup takes 256 / (2 B) rows (B blocks a row, 1, 2 or 4, the last of them perhaps
// empty): neighbouring tokens of one head, so that stores to a cache whose heads come first run on, or, where the
// sequences are shorter than that, tokens of several heads. Where a lane stands takes shifts alone: with divisions that
// took three times the instructions of the codes, and 8191 tokens of 8 heads, d 128, FP4, 20 us to write and 14.6 to read.
//
// The nearest code to x is decided exactly, ties to the lower code, by an approximate quotient (2^-22, relative): x and
// absmax have 8 significant bits, and a quotient of two such numbers is a tie or well away from one.
//   NF4   no quotient is within 2.1e-7 of a midpoint, and the comparison is good to 1.3e-7 there (the midpoint 0.0398);
//         none is within 2.9e-7 of another, where it is good to 2.3e-7 (the test suite checks all of them):
//         y = 16 x / absmax + 16, whose whole part is a bin of width 1/16 that holds one midpoint at most; a table in LDS
//         gives the number of midpoints below the bin and the one in it.
//   INT4  ceil(7 x / absmax - 1/2 - 1e-5), which a tie passes downwards: other quotients are 1e-4 away from one.
//   FP4   the hardware's conversion of 6 x / absmax, of which 1e-5 of its magnitude is taken away first, so that a
//         tie falls to the lower code; other quotients are 1e-4 away, relative. -0 becomes 0.
// Bound by memory: 2 bytes a value on one side, 0.5625 on the other. Those 8191 tokens are written in 10 us and read in 10.4
// (43 MB, 4.3 and 4.1 TB/s); 6007 of them in NF4 are read in 8.8 us (3.6 TB/s), 1024 written in 4.4, 16 written in 3.7 and
// read in 2.9 (the latency of arguments and loads, and of the bins).
#include "kv4.h"

#include <string.h>

#include "attn.h"

namespace nf4 {

// Codes of a block's values. Blocks of very small or large values are scaled by a power of two, so that the reciprocal and
// the products stay in range (values that this flushes to zero are nearest to the zero code either way).
struct Kv4Bin {
  float mid;       // the midpoint in the bin, or infinity
  uint32_t base;   // midpoints below the bin
};
template <int BOOK>
struct Kv4Codes {
  float mul, rcp;
  __device__ __forceinline__ explicit Kv4Codes(uint32_t absmax) {
    const float a = __uint_as_float(absmax << 16);
    mul = a < 0x1p-60f ? 0x1p100f : a > 0x1p100f ? 0x1p-100f : 1.f;
    const float den = a > 0.f ? a * mul : 1.f;
    rcp = (BOOK == 0 ? 16.f : BOOK == 1 ? 6.f : 7.f) * __builtin_amdgcn_rcpf(den);
  }
  // two neighbours, x in the high half, into byte j of `codes`
  __device__ __forceinline__ void two(uint32_t& codes, int j, float x, float y, const Kv4Bin* bins) const {
    const float n = x * mul, m = y * mul;
    if (BOOK == 1) {
      const float u = n * rcp, v = m * rcp;
      const float a = __fmaf_rn(fabsf(v), -1e-5f, v), b = __fmaf_rn(fabsf(u), -1e-5f, u);
      if (j == 0) codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, a, b, 1.f, 0);
      if (j == 1) codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, a, b, 1.f, 1);
      if (j == 2) codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, a, b, 1.f, 2);
      if (j == 3) codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, a, b, 1.f, 3);
      return;
    }
    codes |= (code(n, bins) << 4 | code(m, bins)) << (8 * j);
  }
  __device__ __forceinline__ uint32_t code(float n, const Kv4Bin* bins) const {
    if (BOOK == 2) return (uint32_t)ceilf(__fmaf_rn(n, rcp, 6.49999f));
    const float y = __fmaf_rn(n, rcp, 16.f);
    const Kv4Bin b = bins[min((uint32_t)fmaxf(y, 0.f), 32u)];
    return b.base + (y > b.mid ? 1u : 0u);
  }
  static __device__ __forceinline__ uint32_t finish(uint32_t codes) {
    if (BOOK != 1) return codes;
    const uint32_t some = (codes & 0x77777777u) + 0x77777777u;   // bit 3 of a nibble: its magnitude is not zero
    return codes & (0x77777777u | some);
  }
  static constexpr uint32_t zero = BOOK == 1 ? 0u : 0x77777777u;
};

// What a lane works on: 16 values of a row's block.
struct Kv4Place {
  bool in, first, second;   // the block is the sequence's; its half's first and last 8 values are the row's (not filling)
  int64_t token, at;        // of k and v; of the cache
  int head, block, half, column;
};
template <int B>
__device__ __forceinline__ Kv4Place kv4_place(const AttnSeqs& sq, const Kv4Args& a) {
  constexpr int ROWS = 128 / B;
  const Found f = find_seq(sq, (int)blockIdx.x);
  const int tokens = 1 << a.log_tokens, heads = ROWS >> a.log_tokens;   // of a workgroup
  const int across = (a.kv_heads + heads - 1) / heads, tile = (int)blockIdx.x - f.first;
  const int t = (int)threadIdx.x % (2 * B), row = (int)threadIdx.x / (2 * B);
  Kv4Place p;
  const int i = tile / across * tokens + (row & (tokens - 1));
  p.head = tile % across * heads + (row >> a.log_tokens);
  p.block = t >> 1;
  p.half = t & 1;
  p.column = 16 * t;
  p.in = i < f.seq.nq && p.head < a.kv_heads && p.block < a.nb;
  p.first = p.in && p.column < a.d;
  p.second = p.in && p.column + 8 < a.d;
  p.token = f.seq.q0 + i;
  p.at = f.seq.k0 + (f.seq.nk - f.seq.nq) + i;
  return p;
}

template <int BOOK, int B>
__global__ __launch_bounds__(256) void kv4_write_kernel(const Kv4Args a, const AttnSeqs sq) {
  __shared__ Kv4Bin bins[33];
  if (BOOK == 0 && threadIdx.x < 33) {
    Kv4Bin b{__builtin_inff(), 0u};
#pragma unroll
    for (int i = 0; i < 15; ++i) {
      const double m = 8.0 * ((double)code_value(i) + (double)code_value(i + 1)) + 16.0;
      if (m < (double)threadIdx.x) ++b.base;
      else if (m < (double)threadIdx.x + 1.0) b.mid = (float)m;
    }
    bins[threadIdx.x] = b;
  }
  const Kv4Place p = kv4_place<B>(sq, a);
  u32x4 x[2][2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const AttnTensor& src = w ? a.v : a.k;
    const uint16_t* from = src.p + p.token * src.token + (int64_t)p.head * src.head + p.column;
    x[w][0] = x[w][1] = u32x4{0u, 0u, 0u, 0u};
    if (p.first) x[w][0] = *reinterpret_cast<const u32x4*>(from);
    if (p.second) x[w][1] = *reinterpret_cast<const u32x4*>(from + 8);
  }
  if (BOOK == 0) __syncthreads();
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    uint32_t m = 0, h = 0;   // largest magnitudes, of the low and high halves
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      m = max(m, x[w][k / 4][k % 4] & 0x7FFFu);
      h = max(h, x[w][k / 4][k % 4] & 0x7FFF0000u);
    }
    m = max(m, h >> 16);
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));   // the block's other lane
    const Kv4Codes<BOOK> c(m);
    u32x2 o = u32x2{0u, 0u};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t e = o[k / 4];
      c.two(e, k % 4, __uint_as_float(x[w][k / 4][k % 4] << 16), __uint_as_float(x[w][k / 4][k % 4] & 0xFFFF0000u), bins);
      o[k / 4] = e;
    }
    o[0] = m >= kBf16Infinity ? c.zero : c.finish(o[0]);
    o[1] = m >= kBf16Infinity ? c.zero : c.finish(o[1]);
    if (p.in) {
      const Kv4Tensor& dst = w ? a.v4 : a.k4;
      const int64_t at = p.at * dst.token + (int64_t)p.head * dst.head + p.block;
      *reinterpret_cast<u32x2*>(dst.codes + 16 * at + 8 * p.half) = o;
      if (p.half == 0) dst.absmax[at] = (uint16_t)m;
    }
  }
}

template <class Deq, int B>
__global__ __launch_bounds__(256) void kv4_read_kernel(const Kv4Args a, const AttnSeqs sq) {
  const Kv4Place p = kv4_place<B>(sq, a);
  if (!p.first) return;
  u32x2 codes[2];
  uint32_t m[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const Kv4Tensor& src = w ? a.v4 : a.k4;
    const int64_t at = p.at * src.token + (int64_t)p.head * src.head + p.block;
    codes[w] = *reinterpret_cast<const u32x2*>(src.codes + 16 * at + 8 * p.half);
    m[w] = src.absmax[at];
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const AttnTensor& dst = w ? a.v : a.k;
    uint16_t* to = dst.p + p.token * dst.token + (int64_t)p.head * dst.head + p.column;
    const Deq q(a.t, kv4_step(m[w] >= kBf16Infinity ? kBf16Nan : m[w], a.unit));   // infinity stands for NaN with every code
    *reinterpret_cast<u32x4*>(to) = q.in_order(codes[w][0]);
    if (p.second) *reinterpret_cast<u32x4*>(to + 8) = q.in_order(codes[w][1]);
  }
}

// ------------------------------------------------------------------------------------------
// Host side
bool kv4_codes(int book, Codes& t, float* unit) {
  static constexpr uint32_t nf4[16] = {NF4_CODE_BITS};
  static constexpr float e2m1[8] = {0.f, 0.5f, 1.f, 1.5f, 2.f, 3.f, 4.f, 6.f};
  for (int i = 0; i < 16; ++i) {
    switch (book) {
      case 0: memcpy(&t.v[i], &nf4[i], 4); break;
      case 1: t.v[i] = i < 8 ? e2m1[i] : -e2m1[i - 8]; break;
      case 2: t.v[i] = (float)std::min(i - 7, 7); break;
      default: return false;
    }
  }
  *unit = book == 0 ? 1.f : book == 1 ? 1.f / 6.f : 1.f / 7.f;
  return true;
}

// 1, 2 or 4 blocks a row; as many tokens a workgroup as it has rows, or the power of two that holds the longest sequence's
template <int B>
static void kv4_rows(Kv4Args a, int book, bool write, const std::vector<AttnSeq>& v, hipStream_t stream) {
  constexpr int kRows = 128 / B;
  int longest = 1;
  for (const AttnSeq& s : v) longest = std::max(longest, s.nq);
  a.log_tokens = 0;
  while ((1 << a.log_tokens) < std::min(longest, kRows)) ++a.log_tokens;
  const int64_t across = ceil64(a.kv_heads, kRows >> a.log_tokens);
  for (size_t from = 0; from < v.size();) {
    const AttnSeqs q = pack_seqs(v, from, 1, [&](const AttnSeq& s) { return ceil64(s.nq, 1 << a.log_tokens) * across; });
    from += (size_t)q.count;
    const dim3 grid((unsigned)q.first[q.count]), wg(256);
    if (!write && book == 1) hipLaunchKernelGGL((kv4_read_kernel<Kv4E2m1, B>), grid, wg, 0, stream, a, q);
    else if (!write) hipLaunchKernelGGL((kv4_read_kernel<Kv4Table, B>), grid, wg, 0, stream, a, q);
    else if (book == 0) hipLaunchKernelGGL((kv4_write_kernel<0, B>), grid, wg, 0, stream, a, q);
    else if (book == 1) hipLaunchKernelGGL((kv4_write_kernel<1, B>), grid, wg, 0, stream, a, q);
    else hipLaunchKernelGGL((kv4_write_kernel<2, B>), grid, wg, 0, stream, a, q);
  }
}

hipError_t launch_kv4(const Kv4Args& a, int book, bool write, const AttnSeq* seqs, int64_t count, hipStream_t stream) {
  const std::vector<AttnSeq> v = by_work(seqs, count, false);
  if (v.empty()) return hipSuccess;
  if (a.nb == 1) kv4_rows<1>(a, book, write, v, stream);
  else if (a.nb == 2) kv4_rows<2>(a, book, write, v, stream);
  else kv4_rows<4>(a, book, write, v, stream);
  return hipGetLastError();
}

}  // namespace nf4
