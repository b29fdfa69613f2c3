// 8-bit activation checkpoints (gfx950): packing, unpacking, and the adapter gradient that reads them.
//
// The adapted linear's backward needs its input x only for dA = s v^T x (v = dY B). With x kept as
// codes and block maxima (act8.h), x[m][c] = q[m][c] a[m][b] / 127 for the 64-column block b of c:
//   dA[j][c] = s sum_m (v[m][j] a[m][b] / 127) q[m][c],
// so the scale goes into the rank-sized operand once per row and block, and the streamed operand is
// the codes themselves, which bf16 holds exactly. The pass reads 1.03 bytes per value where the bf16
// input would take 2.
#include "act8.h"
#include "launch.h"

namespace nf4 {

// Packing: a lane takes 8 values, 8 lanes a block. Bound by memory: 2 bytes in and 1.03 out per value
// (2048 x 14336: 16 us, 5.5 TB/s).
__global__ __launch_bounds__(256) void act8_pack_kernel(const u32x4* __restrict__ x, int64_t vecs, u32x2* __restrict__ codes,
                                                        uint16_t* __restrict__ absmax) {
  constexpr int U = 4;   // loads in flight per lane
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x; i0 < vecs; i0 += U * step) {
    u32x4 v[U];
#pragma unroll
    for (int k = 0; k < U; ++k) v[k] = x[min(i0 + k * step, vecs - 1)];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t i = i0 + k * step;
      const uint32_t a = act8_absmax(v[k]);   // vecs is a multiple of 8: a block's lanes are in or out together
      if (i < vecs) {
        codes[i] = act8_codes(v[k], a);
        if ((i & 7) == 0) absmax[i >> 3] = (uint16_t)a;
      }
    }
  }
}

// Unpacking: a lane takes 8 values. Bound by memory: 1.03 bytes in and 2 out per value (2048 x 14336: 15 us,
// 6 TB/s).
__global__ __launch_bounds__(256) void act8_unpack_kernel(const u32x2* __restrict__ codes, const uint16_t* __restrict__ absmax,
                                                          int64_t vecs, u32x4* __restrict__ x) {
  constexpr int U = 4;
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x; i0 < vecs; i0 += U * step) {
    u32x2 q[U];
    uint32_t a[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t i = min(i0 + k * step, vecs - 1);
      q[k] = codes[i];
      a[k] = absmax[i >> 3];
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t i = i0 + k * step;
      if (i >= vecs) break;
      const float f = __uint_as_float(a[k] << 16) * (1.f / 127.f);
      u32x4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t w = q[k][e >> 1] >> (16 * (e & 1));
        o[e] = pack_bf16x2((float)(int8_t)w * f, (float)(int8_t)(w >> 8) * f);
      }
      x[i] = o;
    }
  }
}

static unsigned stream_grid(int64_t vecs) {
  const int64_t b = (vecs + 1023) / 1024;   // four vectors a thread
  return (unsigned)(b < 1 ? 1 : b > 8192 ? 8192 : b);
}

hipError_t launch_act8_pack(const uint16_t* x, int64_t numel, int8_t* codes, uint16_t* absmax, hipStream_t stream) {
  const int64_t vecs = numel / 8;
  hipLaunchKernelGGL(act8_pack_kernel, dim3(stream_grid(vecs)), dim3(256), 0, stream, reinterpret_cast<const u32x4*>(x),
                     vecs, reinterpret_cast<u32x2*>(codes), absmax);
  return hipGetLastError();
}

hipError_t launch_act8_unpack(const int8_t* codes, const uint16_t* absmax, int64_t numel, uint16_t* x, hipStream_t stream) {
  const int64_t vecs = numel / 8;
  hipLaunchKernelGGL(act8_unpack_kernel, dim3(stream_grid(vecs)), dim3(256), 0, stream,
                     reinterpret_cast<const u32x2*>(codes), absmax, vecs, reinterpret_cast<u32x4*>(x));
  return hipGetLastError();
}

// ------------------------------------------------------------------------------------------
// dA from the codes. A workgroup takes 128 columns (two blocks), a range of rows and up to RT tiles of
// 16 adapter ranks (of one linear or of several that share x); its 4 waves take 32-row chunks in turn.
// In v_mfma_f32_16x16x32_bf16 a lane's operand fragment is 8 rows of one column, so a lane loads one
// dword (4 columns) from each of 8 rows and keeps all four columns: column tile t is the columns
// 4 i + t of the block, and nothing is transposed. The rank operand is scaled in fp32 and split into a
// bf16 pair hi + lo, as the passes over bf16 inputs split theirs (relative error 2^-17). Bound by its reads:
// 2048 rows, K = 4096, two linears of rank 16 (8.7 MB of checkpoint) 11 us and 5 for the sums, most of it
// latency (512 workgroups whose waves take one chunk each); dX beside it takes 480.
struct Dx8Tile {
  const float* v;      // [M x r], at the tile's first column
  float* out;          // at the tile's first row: partial sums [row ranges][r][K], or dA [r][K] itself
};
constexpr int kDx8Tiles = 4 * 8;   // four linears of rank 128
struct Dx8Args {
  const int8_t* codes;
  const uint16_t* absmax;
  int64_t M, K;
  int64_t rows;        // rows per range (a multiple of 32)
  int r, tiles;        // rank; rank tiles in all
  int final_;          // one range: out is dA, scaled (and added to)
  int accumulate;
  float scale;
  Dx8Tile tile[kDx8Tiles];
};

template <int RT>
__global__ __launch_bounds__(256) void act8_grad_kernel(const Dx8Args a) {
  __shared__ f32x4 red[4][4][64];
  __shared__ __attribute__((aligned(16))) float out[16][68];   // 16 ranks x 64 columns
  const int tid = threadIdx.x, lane = tid & 63, grp = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t nb = a.K / 64, b0 = (int64_t)blockIdx.x * 2;
  const int blocks = (int)min((int64_t)2, nb - b0);
  const int64_t m_begin = (int64_t)blockIdx.y * a.rows, m_end = min(a.M, m_begin + a.rows);
  const int tile0 = (int)blockIdx.z * RT;
  f32x4 acc[RT][2][4];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[t][b][c] = f32x4{0.f, 0.f, 0.f, 0.f};

  for (int64_t m0 = m_begin + 32 * wave; m0 < m_end; m0 += 128) {
    uint32_t x[2][8];
    float s[2][8], v[RT][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t m = m0 + 8 * grp + e, mr = min(m, m_end - 1);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int64_t blk = b0 + min(b, blocks - 1);
        x[b][e] = *reinterpret_cast<const uint32_t*>(a.codes + mr * a.K + blk * 64 + 4 * col);
        s[b][e] = __uint_as_float((uint32_t)a.absmax[mr * nb + blk] << 16) * (1.f / 127.f);
      }
#pragma unroll
      for (int t = 0; t < RT; ++t) v[t][e] = m < m_end ? a.tile[min(tile0 + t, a.tiles - 1)].v[mr * a.r + col] : 0.f;
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      bf16x8 xf[4];
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) xf[c][e] = (__bf16)(float)(int8_t)(x[b][e] >> (8 * c));
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        bf16x8 hi, lo;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float p = v[t][e] * s[b][e];
          hi[e] = (__bf16)p;
          lo[e] = (__bf16)(p - (float)hi[e]);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          acc[t][b][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, xf[c], acc[t][b][c], 0, 0, 0);
          acc[t][b][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, xf[c], acc[t][b][c], 0, 0, 0);
        }
      }
    }
  }
  // the waves' sums, added in wave order (wave w finishes column tile w), then rows of 64 columns
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    if (tile0 + t >= a.tiles) break;
    float* dst = a.tile[tile0 + t].out + (int64_t)blockIdx.y * a.r * a.K;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if (b >= blocks) break;
#pragma unroll
      for (int c = 0; c < 4; ++c) red[wave][c][lane] = acc[t][b][c];
      __syncthreads();
      f32x4 v = red[0][wave][lane];
#pragma unroll
      for (int w = 1; w < 4; ++w) v += red[w][wave][lane];
#pragma unroll
      for (int e = 0; e < 4; ++e) out[4 * grp + e][4 * col + wave] = v[e];
      __syncthreads();
      const int j = tid >> 4;
      float* p = dst + j * a.K + (b0 + b) * 64 + 4 * (tid & 15);
      f32x4 o = *reinterpret_cast<const f32x4*>(&out[j][4 * (tid & 15)]);
      if (a.final_) {
        o *= a.scale;
        if (a.accumulate) o += *reinterpret_cast<const f32x4*>(p);
      }
      *reinterpret_cast<f32x4*>(p) = o;
    }
  }
}

// Rows per range: about 512 workgroups, 128 rows (one chunk a wave) at least.
static int64_t dx8_rows(int64_t M, int64_t K) {
  const int64_t groups = (K / 64 + 1) / 2;
  int64_t ranges = (512 + groups - 1) / groups;
  if (ranges > (M + 127) / 128) ranges = (M + 127) / 128;
  return ((M + ranges - 1) / ranges + 31) / 32 * 32;
}
static int64_t dx8_ranges(int64_t M, int64_t K) {
  const int64_t rows = dx8_rows(M, K);
  return (M + rows - 1) / rows;
}

// partial sums only where there are several ranges
size_t act8_grad_ws_floats(int count, int64_t M, int64_t K, int r) {
  const int64_t ranges = dx8_ranges(M, K);
  return ranges > 1 ? (size_t)count * (size_t)ranges * (size_t)K * r : 0;
}

hipError_t launch_act8_grad(int count, const int8_t* codes, const uint16_t* absmax, int64_t M, int64_t K,
                            const float* const* v, int r, float scale, int accumulate, float* ws, float* const* dA,
                            hipStream_t stream) {
  if (count < 1 || count > 4) return hipErrorInvalidValue;
  const int64_t ranges = dx8_ranges(M, K), groups = (K / 64 + 1) / 2;
  Dx8Args a{};
  a.codes = codes;
  a.absmax = absmax;
  a.M = M;
  a.K = K;
  a.rows = dx8_rows(M, K);
  a.r = r;
  a.final_ = ranges == 1;
  a.accumulate = accumulate;
  a.scale = scale;
  const float* part[4];
  for (int i = 0; i < count; ++i) {
    float* base = a.final_ ? dA[i] : ws + (size_t)i * ranges * K * r;
    part[i] = base;
    for (int t = 0; t < r / 16; ++t) a.tile[a.tiles++] = Dx8Tile{v[i] + 16 * t, base + (int64_t)16 * t * K};
  }
  // as many rank tiles to a workgroup (they share its reads of x) as leave 256 workgroups: at 77 rows,
  // K = 4096 and 12 tiles one tile each took 5 us where four took 24 in three launches
  int rt = 4;
  while (rt > 1 && groups * ranges * ((a.tiles + rt - 1) / rt) < 256) rt /= 2;
  const dim3 grid((unsigned)groups, (unsigned)ranges, (unsigned)((a.tiles + rt - 1) / rt)), block(256);
  if (rt == 4) hipLaunchKernelGGL(act8_grad_kernel<4>, grid, block, 0, stream, a);
  else if (rt == 2) hipLaunchKernelGGL(act8_grad_kernel<2>, grid, block, 0, stream, a);
  else hipLaunchKernelGGL(act8_grad_kernel<1>, grid, block, 0, stream, a);
  if (a.final_) return hipGetLastError();
  return launch_lora_sum(count, part, (int)ranges, K * r, scale, accumulate, dA, stream);
}

}  // namespace nf4
