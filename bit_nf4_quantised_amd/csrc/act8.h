// The 8-bit activation format, shared by the kernels that write it (gfx950).
//
// Blocks of 64 values along a row: absmax a (the largest |x| of the block, bf16, exact because x is
// bf16) and codes round(127 x / a) in -127..127, nearest integer of the exact quotient, ties to even;
// a block of zeros stores a = 0 and codes 0. The value a code stands for is code * a / 127.
// A block that holds a NaN or an infinity stores it as a (a NaN before an infinity) and codes 0: it stands
// for NaN throughout, so that what is lost in 8 bits cannot pass for numbers. Magnitudes are compared as
// integers, in which order NaN > infinity > numbers; a maximum of floats drops NaN.
#pragma once
#include "common.h"

namespace nf4 {

constexpr uint32_t kBf16Inf = 0x7F80u;

// The codes of a block's values: num(x) / den, with one Newton step after the hardware reciprocal.
// 127 x is exact in fp32 (15 significant bits), and a quotient of such numbers that is not a tie is
// further from one than the 2^-23 the step leaves; a tie is representable, and the step returns it
// exactly. Blocks whose maximum is very small or large are scaled by a power of two, so that the
// reciprocal and 127 x stay in range (values that this flushes round to code 0 either way).
struct Act8Block {
  float den, rcp, mul;
  __device__ __forceinline__ explicit Act8Block(float a) {
    const float s = a < 0x1p-60f ? 0x1p100f : a > 0x1p100f ? 0x1p-100f : 1.f;
    den = a > 0.f ? a * s : 1.f;
    mul = 127.f * s;
    rcp = __builtin_amdgcn_rcpf(den);
  }
  __device__ __forceinline__ int code(float x) const {
    const float n = x * mul;
    const float q = n * rcp;
    return (int)__builtin_rintf(__fmaf_rn(__fmaf_rn(-q, den, n), rcp, q));
  }
};

// Codes of 8 consecutive bf16 values (4 dwords) whose block maximum has the bf16 bits `absmax`, in byte order.
__device__ __forceinline__ u32x2 act8_codes(const u32x4& x, uint32_t absmax) {
  const Act8Block b(__uint_as_float(absmax << 16));
  u32x2 o;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t p = x[2 * k], q = x[2 * k + 1];
    const uint32_t c0 = (uint32_t)b.code(__uint_as_float(p << 16)), c1 = (uint32_t)b.code(__uint_as_float(p & 0xFFFF0000u));
    const uint32_t c2 = (uint32_t)b.code(__uint_as_float(q << 16)), c3 = (uint32_t)b.code(__uint_as_float(q & 0xFFFF0000u));
    const uint32_t lo = __builtin_amdgcn_perm(c1, c0, 0x0C0C0400u), hi = __builtin_amdgcn_perm(c3, c2, 0x0C0C0400u);
    o[k] = absmax < kBf16Inf ? lo | (hi << 16) : 0u;
  }
  return o;
}

// bf16 bits of the largest magnitude among the 8 values of each of 8 neighbouring lanes (a block), in all of them
__device__ __forceinline__ uint32_t act8_absmax(const u32x4& x) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  u16x2 m{0, 0};
#pragma unroll
  for (int k = 0; k < 4; ++k) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, x[k] & 0x7FFF7FFFu));
  return umax8(max((uint32_t)m.x, (uint32_t)m.y));
}

}  // namespace nf4
