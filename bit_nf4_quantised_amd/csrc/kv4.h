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

constexpr uint32_t kBf16Infinity = 0x7F80u;

__device__ __forceinline__ float kv4_step(uint32_t absmax, float unit) { return __fmul_rn(__uint_as_float(absmax << 16), unit); }

// One packed dword (8 values) as 4 bf16 pairs, from the block's table of values.
struct Kv4Table {
  BlockLut lut;
  __device__ __forceinline__ Kv4Table(const Codes& t, float step) : lut(make_lut(step, t.v)) {}
  __device__ __forceinline__ u32x4 eight(uint32_t p) const {
    uint32_t o[4];
    dequant8(lut, p, o);
    return u32x4{o[0], o[1], o[2], o[3]};
  }
};

}  // namespace nf4
