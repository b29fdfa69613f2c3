// Keys and values to and from a 4-bit cache (gfx950; format in kv4.h).
//
// The new tokens of every sequence go behind the others it holds: token i of a sequence with nq new ones, nk in
// all, goes to the cache's token k0 + nk - nq + i; reading goes the other way. A quad of lanes holds a block,
// 8 values a lane; quads run over the blocks of a row, rows over the tokens of a head, then over the heads, so
// that stores to a cache whose heads come first run on. Keys and values are the launch's two rows of workgroups.
//
// The nearest code to x is decided exactly, ties to the lower code:
//   NF4   x / absmax is computed to 2^-22 and compared with the codes' midpoints. That decides as the exact quotient:
//         x and absmax have 8 significant bits, and no quotient of two such numbers is within 1.4e-6 of a
//         midpoint, relative to it (checked over all of them; the test suite repeats it);
//   INT4  the code k near 7 x / absmax, put right by comparing 14 x with (2 k +- 1) absmax, which fp32 holds exactly;
//   FP4   6 |x| against absmax times the seven midpoints of E2M1, exact in fp32 too.
// Bound by memory: 2 bytes a value on one side, 0.5625 on the other.
#include "kv4.h"

#include <string.h>

#include "attn.h"

namespace nf4 {

// largest of the quad's values, as integers
__device__ __forceinline__ uint32_t umax4(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
}

// Codes of a block's values. Blocks of very small or large values are scaled by a power of two, so that the reciprocal and
// the products stay in range (values that this flushes to zero are nearest to the zero code either way).
template <int BOOK>
struct Kv4Codes {
  float den, rcp, mul;
  __device__ __forceinline__ explicit Kv4Codes(float a) {
    mul = a < 0x1p-60f ? 0x1p100f : a > 0x1p100f ? 0x1p-100f : 1.f;
    den = a > 0.f ? a * mul : 1.f;
    rcp = __builtin_amdgcn_rcpf(den);
  }
  __device__ __forceinline__ uint32_t code(float x) const {
    const float n = x * mul;
    if (BOOK == 0) {
      const float q = n * rcp;
      uint32_t idx = 0;
#pragma unroll
      for (int i = 0; i < 15; ++i) idx += q > 0.5f * (code_value(i) + code_value(i + 1)) ? 1u : 0u;
      return idx;
    }
    if (BOOK == 2) {
      float k = fminf(fmaxf(ceilf(__fmaf_rn(7.f * n, rcp, -0.5f)), -7.f), 7.f);
      const float l = 14.f * n;
      if (k < 7.f && l > __fmaf_rn(2.f * k, den, den)) k += 1.f;
      else if (k > -7.f && l <= __fmaf_rn(2.f * k, den, -den)) k -= 1.f;
      return (uint32_t)(int)(k + 7.f);
    }
    // |x| past a midpoint, or on it where x is negative (the lower code is then the larger magnitude)
    constexpr float mid[7] = {0.25f, 0.75f, 1.25f, 1.75f, 2.5f, 3.5f, 5.f};
    const uint32_t neg = __float_as_uint(x) >> 31, m = __float_as_uint(6.f * fabsf(n)) + neg;
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 7; ++i) c += m > __float_as_uint(mid[i] * den) ? 1u : 0u;
    return c ? c | neg << 3 : 0u;
  }
  static constexpr uint32_t zero = BOOK == 1 ? 0u : 7u;
};

// What a lane works on: values 8 e .. 8 e + 7 of the block, the row's token and head.
struct Kv4Place {
  bool in, values;    // a block of the sequence; its 8 values are the row's (not filling)
  int64_t token, at;  // of k and v; of the cache
  int head, block, e;
};
__device__ __forceinline__ Kv4Place kv4_place(const AttnSeqs& sq, int tile, int kv_heads, int nb, int d) {
  const Found f = find_seq(sq, tile);
  const int u = (tile - f.first) * 256 + (int)threadIdx.x;   // quads of all blocks of the sequence in turn
  const int blocks = f.seq.nq * kv_heads * nb;
  Kv4Place p;
  const int blk = min(u >> 2, blocks - 1);
  p.in = (u >> 2) < blocks;
  const int row = blk / nb, t = row % f.seq.nq;
  p.block = blk % nb;
  p.head = row / f.seq.nq;
  p.token = f.seq.q0 + t;
  p.at = f.seq.k0 + (f.seq.nk - f.seq.nq) + t;
  p.e = u & 3;
  p.values = p.in && 32 * p.block + 8 * p.e < d;
  return p;
}

template <int BOOK>
__global__ __launch_bounds__(256) void kv4_write_kernel(const Kv4Args a, const AttnSeqs sq) {
  const Kv4Place p = kv4_place(sq, (int)blockIdx.x, a.kv_heads, a.nb, a.d);
  const AttnTensor& src = blockIdx.y ? a.v : a.k;
  const Kv4Tensor& dst = blockIdx.y ? a.v4 : a.k4;
  u32x4 x = u32x4{0u, 0u, 0u, 0u};
  if (p.values)
    x = *reinterpret_cast<const u32x4*>(src.p + p.token * src.token + (int64_t)p.head * src.head + 32 * p.block + 8 * p.e);
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) m = max(m, max(x[k] & 0x7FFFu, x[k] >> 16 & 0x7FFFu));
  m = umax4(m);
  const Kv4Codes<BOOK> c(__uint_as_float(m << 16));
  uint32_t o = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t lo = c.code(__uint_as_float(x[k] << 16)), hi = c.code(__uint_as_float(x[k] & 0xFFFF0000u));
    o |= (lo << 4 | hi) << (8 * k);
  }
  if (m >= kBf16Infinity) o = 0x11111111u * Kv4Codes<BOOK>::zero;
  if (p.in) {
    const int64_t at = p.at * dst.token + (int64_t)p.head * dst.head + p.block;
    *reinterpret_cast<uint32_t*>(dst.codes + 16 * at + 4 * p.e) = o;
    if (p.e == 0) dst.absmax[at] = (uint16_t)m;
  }
}

__global__ __launch_bounds__(256) void kv4_read_kernel(const Kv4Args a, const AttnSeqs sq) {
  const Kv4Place p = kv4_place(sq, (int)blockIdx.x, a.kv_heads, a.nb, a.d);
  if (!p.values) return;
  const AttnTensor& dst = blockIdx.y ? a.v : a.k;
  const Kv4Tensor& src = blockIdx.y ? a.v4 : a.k4;
  const int64_t at = p.at * src.token + (int64_t)p.head * src.head + p.block;
  const uint32_t codes = *reinterpret_cast<const uint32_t*>(src.codes + 16 * at + 4 * p.e);
  const uint32_t m = src.absmax[at];
  u32x4 o = Kv4Table(a.t, kv4_step(m, a.unit)).in_order(codes);
  // infinity stands for NaN with every code
  if (m >= kBf16Infinity) o = u32x4{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
  *reinterpret_cast<u32x4*>(dst.p + p.token * dst.token + (int64_t)p.head * dst.head + 32 * p.block + 8 * p.e) = o;
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

static int kv4_tiles(const AttnSeq& s, const Kv4Args& a) { return (int)ceil64((int64_t)s.nq * a.kv_heads * a.nb, 64); }

hipError_t launch_kv4(const Kv4Args& a, int book, bool write, const AttnSeq* seqs, int64_t count, hipStream_t stream) {
  const std::vector<AttnSeq> v = by_work(seqs, count, false);
  for (size_t from = 0; from < v.size();) {
    const AttnSeqs q = pack_seqs(v, from, 2, [&](const AttnSeq& s) { return kv4_tiles(s, a); });
    from += (size_t)q.count;
    const dim3 grid((unsigned)q.first[q.count], 2), wg(256);
    if (!write) hipLaunchKernelGGL(kv4_read_kernel, grid, wg, 0, stream, a, q);
    else if (book == 0) hipLaunchKernelGGL(kv4_write_kernel<0>, grid, wg, 0, stream, a, q);
    else if (book == 1) hipLaunchKernelGGL(kv4_write_kernel<1>, grid, wg, 0, stream, a, q);
    else hipLaunchKernelGGL(kv4_write_kernel<2>, grid, wg, 0, stream, a, q);
  }
  return hipGetLastError();
}

}  // namespace nf4
