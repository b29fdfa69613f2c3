// The 4-bit format of keys and values, shared by the kernels that write, read and attend to it (gfx950).
//
// A row (one token and key head, d values) is nb = ceil(d / 32) blocks of 32 values, the last one filled up with
// zeros. A block keeps its largest magnitude `absmax` (bf16 bits, exact as the values are bf16) and 32 codes
// of 4 bits in 16 bytes, byte j holding value 2 j in its high nibble. A code p stands for
//   bf16(fl32(t[p] * step)),  step = fl32(absmax * unit),
// t the 16 values that a nibble selects and unit one over the largest: NF4's codes and 1; -7 .. 7 for nibbles
// 0 .. 14 and 1/7 (INT4); the E2M1 bit patterns' values and 1/6 (FP4). A block that holds a NaN or an infinity
// keeps the largest magnitude's bits and the zero code: it stands for NaN throughout.
#pragma once
#include "common.h"

namespace nf4 {

constexpr uint32_t kBf16Infinity = 0x7F80u, kBf16Nan = 0x7FC0u;

__device__ __forceinline__ float kv4_step(uint32_t absmax, float unit) { return __fmul_rn(__uint_as_float(absmax << 16), unit); }

// A block's codes as bf16: eight() takes one packed dword (8 values) and gives them in the order 0 2 4 6 1 3 5 7,
// which costs no byte moves; in_order() in their own.
//
// Any 16 values whose nibble 7 is zero: a table of the block's 16 bf16 values, looked up with byte permutes (23
// instructions for 8 values). The table takes 32 instructions to make, for 32 values. But a maximum has 8 significant bits and
// a power of two scales the table's values, which leaves 256 tables up to the upper seven bits of the exponent, the
// low part of a value's high byte. A kernel of many blocks makes these 256 (Kv4Tables, in LDS) for maxima near 2^-119
// and reads the block's, 10 instructions to put its exponent right. Maxima below that, and from 2^127 on, infinity and NaN
// among them, take the long way, with their whole wave.
struct Kv4Tables {
  u32x4 lo[256], hi[256];
};
constexpr uint32_t kKv4Low = 4;   // upper seven bits of the tables' exponents
struct Kv4Table {
  typedef Kv4Tables Shared;
  BlockLut lut;
  __device__ __forceinline__ Kv4Table(const Codes& t, float step) : lut(make_lut(step, t.v)) {}
  // table i of `s`, by thread i
  static __device__ __forceinline__ void share(Shared& s, int i, const Codes& t, float unit) {
    if (i >= 256) return;
    const BlockLut l = make_lut(kv4_step(kKv4Low << 8 | (uint32_t)i, unit), t.v);
    s.lo[i] = u32x4{l.lo[0], l.lo[1], l.lo[2], l.lo[3]};
    s.hi[i] = u32x4{l.hi[0], l.hi[1], l.hi[2], l.hi[3]};
  }
  __device__ __forceinline__ Kv4Table(const Shared& s, const Codes& t, float unit, uint32_t absmax) {
    const uint32_t up = (absmax >> 8) - kKv4Low;
    if (__any(up > 0x7Eu - kKv4Low)) {
      lut = make_lut(kv4_step(absmax, unit), t.v);
      return;
    }
    const u32x4 lo = s.lo[absmax & 0xFFu], hi = s.hi[absmax & 0xFFu];
    const uint32_t all = __builtin_amdgcn_perm(up, up, 0u), but7 = __builtin_amdgcn_perm(up, up, 0x0C000000u);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      lut.lo[k] = lo[k];
      lut.hi[k] = hi[k] + (k == 1 ? but7 : all);   // within the bytes
    }
  }
  __device__ __forceinline__ u32x4 eight(uint32_t p) const {
    uint32_t a, b, c, d;
    lut4(lut, (p >> 4) & 0x0F0F0F0Fu, a, b);
    lut4(lut, p & 0x0F0F0F0Fu, c, d);
    return u32x4{a, b, c, d};
  }
  __device__ __forceinline__ u32x4 in_order(uint32_t p) const {
    uint32_t o[4];
    dequant8(lut, p, o);
    return u32x4{o[0], o[1], o[2], o[3]};
  }
};
// E2M1: converted by the hardware, two codes an instruction, then multiplied and rounded (16 instructions for 8 values)
struct Kv4E2m1 {
  struct Shared {};
  float step;
  __device__ __forceinline__ Kv4E2m1(const Codes&, float s) : step(s) {}
  static __device__ __forceinline__ void share(Shared&, int, const Codes&, float) {}
  __device__ __forceinline__ Kv4E2m1(const Shared&, const Codes&, float unit, uint32_t absmax) : step(kv4_step(absmax, unit)) {}
  __device__ __forceinline__ u32x4 eight(uint32_t p) const {
    const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(p, 1.f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(p, 1.f, 1),
               c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(p, 1.f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(p, 1.f, 3);
    return u32x4{pack_bf16x2(a[1] * step, b[1] * step), pack_bf16x2(c[1] * step, d[1] * step),
                 pack_bf16x2(a[0] * step, b[0] * step), pack_bf16x2(c[0] * step, d[0] * step)};
  }
  __device__ __forceinline__ u32x4 in_order(uint32_t p) const {
    const u32x4 e = eight(p);
    return u32x4{__builtin_amdgcn_perm(e[2], e[0], 0x05040100u), __builtin_amdgcn_perm(e[2], e[0], 0x07060302u),
                 __builtin_amdgcn_perm(e[3], e[1], 0x05040100u), __builtin_amdgcn_perm(e[3], e[1], 0x07060302u)};
  }
};
// 8 bf16 values in order to the order of eight()
__device__ __forceinline__ u32x4 kv4_order(const u32x4& x) {
  return u32x4{__builtin_amdgcn_perm(x[1], x[0], 0x05040100u), __builtin_amdgcn_perm(x[3], x[2], 0x05040100u),
               __builtin_amdgcn_perm(x[1], x[0], 0x07060302u), __builtin_amdgcn_perm(x[3], x[2], 0x07060302u)};
}
// where value e of 8 stands in that order
constexpr int kv4_place_of(int e) { return (e & 1) * 4 + e / 2; }

}  // namespace nf4
