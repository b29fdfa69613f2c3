// Attention of the layer around the quantised linears (gfx950): forward, few-row forward over a long
// cache, and the backward pass that recomputes the probabilities.
//
// For query row i of a sequence with nq queries and nk keys, standing at position p_i = nk - nq + i,
// over its visible keys j (j <= p_i when causal, j > p_i - window with a window):
//   z_ij = scale q_i.k_j    lse_i = ln sum_j exp(z_ij)    P_ij = exp(z_ij - lse_i)    o_i = sum_j P_ij v_j
//   delta_i = do_i.o_i      dS_ij = P_ij (do_i.v_j - delta_i)
//   dq_i = scale sum_j dS_ij k_j    dk_j = scale sum_i dS_ij q_i    dv_j = sum_i P_ij do_i
// (dk, dv also sum over the query heads that share the key head). Scores, softmax statistics and all
// sums are fp32; P and dS are rounded to bf16 where they enter the second product of each pair, as
// the matrix instructions take bf16 operands (relative error up to 2^-8 a term, independent over terms).
//
// Layout. Every product is taken with v_mfma_f32_32x32x16_bf16, whose result holds in lane l column
// l % 32 and rows 8 (i / 4) + 4 (l / 32) + i % 4 for i < 16. The scores are formed with the rows that
// the wave streams past as result rows and the rows that it owns as result columns, so a lane holds
// 16 consecutive-in-groups-of-4 streamed rows of one owned row: the softmax of a row is a reduction
// inside a lane plus one exchange between lane halves, and the rounded probabilities are already the
// second product's operand (its contraction runs over the streamed rows in the lane's own order; the
// other operand is read in the same order from LDS with transpose loads). Nothing goes through LDS
// between the two products.
#include "attn.h"

namespace nf4 {

// Two groups of 4 waves that hold sums of the same 32-row tiles exchange halves: group 0 keeps columns dt < H
// and group 1 the rest, and each gives the other's away, into a buffer of [wave][H][4][lane][4] floats.
template <int H>
constexpr size_t kHalf = 4 * H * 4 * 64 * 16;
template <int H>
__device__ __forceinline__ void give_half(void* to0, void* to1, const f32x16 (&v)[2 * H], int grp, int wave, int lane) {
  f32x4* p = reinterpret_cast<f32x4*>(grp ? to0 : to1) + wave * (H * 4 * 64) + lane;
#pragma unroll
  for (int dt = 0; dt < H; ++dt)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      f32x4 x;
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = grp ? v[dt][4 * g + k] : v[dt + H][4 * g + k];
      p[(dt * 4 + g) * 64] = x;
    }
}
template <int H>
__device__ __forceinline__ f32x16 taken_half(const void* to0, const void* to1, int dt, int grp, int wave, int lane) {
  const f32x4* p = reinterpret_cast<const f32x4*>(grp ? to1 : to0) + wave * (H * 4 * 64) + lane;
  f32x16 v;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const f32x4 x = p[(dt * 4 + g) * 64];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[4 * g + k] = x[k];
  }
  return v;
}

// ------------------------------------------------------------------------------------------
// Forward. 4 waves take 128 query rows of one head, 32 per wave; keys and values stream through LDS in
// tiles of 64, two tiles deep, by LDS-DMA. Bound by the matrix unit and, in launches that fill the GPU,
// by its power: 8192 tokens, 32 heads over 8, d 128, not causal, 962 us = 1143 TFLOP/s, where a plain
// product of 16384^3 reaches 1355 (d 64: 572 us = 961 TFLOP/s, d 80 and 96 take d 128's tiles: 873 and 906 us). A tile costs a workgroup that shares its compute unit with another
// 0.93 us, but 1.15 to 1.4 us alone, with one wave a SIMD that waits for its own reads and exponentials.
// So where the longest workgroups decide, a workgroup has GR = 2 groups of 4 waves, which take the tiles of
// the same rows in turn and are joined at the end; two_groups() says where. Measured, one group and two, us:
// 256 workgroups of up to 4096 keys 94 and 77; one causal sequence, 32 heads over 8, of 1536 tokens 31.7 and
// 27.8, of 2048 44.7 and 42.3; 3000 tokens, 16 heads over 4, 55.3 and 45.7. Where the work spreads evenly the
// other form is better, as two workgroups on a unit start and end at different times: four causal sequences
// of 512, 32 heads over 8, 20.8 and 23.6, 2048 tokens without a mask 68.7 and 70.8, 8192 causal ones 493 and
// 518, 2368 workgroups of packed sequences 109 and 137. At d = 64: 1536 tokens 22.8 and 19.1, 2048 31.5 and 29.3,
// 3000 37.3 and 30.0, four of 512 14.3 and 16.0, 2048 without a mask 43.4 and 44.2, 8192 293 and 322.
template <int DP, int GR>
__global__ __launch_bounds__(256 * GR, 2) void attn_fwd_kernel(const AttnFwdArgs a, const AttnSeqs sq) {
  constexpr int BN = 64, KS = DP / 16, DT = DP / 32;
  typedef Tile<DP> T;
  typedef KvStream<DP, BN, 4> Stream;
  // a variable per stage and code of its own for each (tile() twice in the loop): from one array, or through
  // a stage index, the compiler lets a tile's reads wait for the next tile's loads, which are on their way
  // (prefill chunk 68 -> 65 us)
  __shared__ __attribute__((aligned(16))) uint16_t Ks0[GR][BN * DP], Ks1[GR][BN * DP], Vs0[GR][BN * DP], Vs1[GR][BN * DP];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) & 3;
  const int grp = GR == 1 ? 0 : __builtin_amdgcn_readfirstlane(tid >> 8);
  const int G = a.heads / a.kv_heads;
  const Unit u = unit_of((int)blockIdx.x, a.kv_heads, G);
  const Found at_seq = find_seq(sq, u.tile);
  const AttnSeq s = at_seq.seq;
  // a sequence's tiles run from its last rows (the most keys when causal) to its first
  const int qt = at_seq.next - 1 - u.tile;
  const int head = u.kvh * G + u.sub;
  const int r0 = qt * 128, shift = s.nk - s.nq;   // row i stands at position i + shift

  const int row = r0 + wave * 32 + (lane & 31);
  bf16x8 qf[KS];
  load_rows<DP>(qf, row < s.nq ? a.q.p + (s.q0 + row) * a.q.token + (int64_t)head * a.q.head : nullptr, a.d, lane);

  // keys that some row of the workgroup (of this wave) sees; none before the first is read: with a window a
  // cache may hold anything there, and 0 times NaN is no zero
  const int r1 = min(s.nq, r0 + 128) - 1;
  const int k_lo = visible(r0 + shift, s.nk, a.causal, a.window).lo;
  const int k_hi = visible(r1 + shift, s.nk, a.causal, a.window).hi;
  const int w0 = r0 + wave * 32, w1 = min(s.nq - 1, w0 + 31);
  const Range wa = visible(w0 + shift, s.nk, a.causal, a.window), wb = visible(w1 + shift, s.nk, a.causal, a.window);
  const Range mine = visible(row + shift, s.nk, a.causal, a.window);
  const int nt = k_hi > k_lo ? (k_hi - k_lo + GR * BN - 1) / (GR * BN) : 0;   // of each group

  Stream kv;
  kv.init(a.k, a.v, s, u.kvh, a.d, wave, lane);

  Online<DT> acc;
  acc.init();
  const float slack = slack_of(a.c);
  const int j_g = k_lo + grp * BN;   // the group's first tile; its tiles are GR apart
  if (nt > 0) kv.load(Ks0[grp], Vs0[grp], j_g, wave);
  auto tile = [&](int t, const uint16_t* Kt, const uint16_t* Vt, uint16_t* kn, uint16_t* vn) __attribute__((always_inline)) {
    wait_vmcnt<0>();
    // the only barrier of a tile (a second one after its products cost 1 % of a full launch and 4 % of a
    // launch with one workgroup a compute unit): tile t is in, and every wave is done with tile t - 1
    lds_barrier();
    if (t + 1 < nt) kv.load(kn, vn, j_g + (t + 1) * GR * BN, wave);
    const int j0 = j_g + t * GR * BN;
    if (j0 < wb.hi && j0 + BN > wa.lo) {
      f32x16 sc[BN / 32];
      // KS operands are on their way from LDS at any time: each register takes its next contents as soon as its
      // product is issued, the first half of the values' operands before the exponentials (8192 tokens, not
      // causal, 1016 -> 987 us, 8 heads of 4096 tokens 60 -> 55; the compiler's own order keeps two)
      bf16x8 f[KS];
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) f[ks] = T::rows(Kt, 0, ks, lane);
      sc[0] = zero16();
      sc[1] = zero16();
      keep_order();
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        sc[0] = mfma(f[ks], qf[ks], sc[0]);
        f[ks] = T::rows(Kt, 32, ks, lane);
        keep_order();
      }
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        sc[1] = mfma(f[ks], qf[ks], sc[1]);
        f[ks] = T::cols(Vt, 16 * (ks / DT), ks % DT, lane);
        keep_order();
      }
      // some row of the wave does not see some key of the tile
      if (j0 + BN > wa.hi || j0 < wb.lo) {
#pragma unroll
        for (int kt = 0; kt < BN / 32; ++kt) hide(sc[kt], mine, j0 + 32 * kt, lane, -INFINITY);
      }
      acc.update(sc, a.c, slack);
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        acc.o[i % DT] = mfma(f[i], pack8(sc[0], i / DT), acc.o[i % DT]);
        f[i] = T::cols(Vt, 32 + 16 * (i / DT), i % DT, lane);
      }
#pragma unroll
      for (int i = 0; i < KS; ++i) acc.o[i % DT] = mfma(f[i], pack8(sc[1], i / DT), acc.o[i % DT]);
    }
  };
  for (int t = 0; t < nt; t += 2) {
    tile(t, Ks0[grp], Vs0[grp], Ks1[grp], Vs1[grp]);
    if (t + 1 < nt) tile(t + 1, Ks1[grp], Vs1[grp], Ks0[grp], Vs0[grp]);
  }

  float l = half_sum(acc.l);
  uint16_t* dst = row < s.nq ? a.o.p + (s.q0 + row) * a.o.token + (int64_t)head * a.o.head : nullptr;
  if constexpr (GR == 1) {
    const float inv = inverse_sum(l);
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) store_cols(dst, acc.o[dt], inv, dt, a.d, lane);
  } else {
    // join the groups: each keeps half of the columns and gets the other group's sums of them, through the
    // tiles' place in LDS
    lds_barrier();
    __shared__ float Ms[GR][128], Ls[GR][128];
    const int rl = wave * 32 + (lane & 31);
    if (lane < 32) {
      Ms[grp][rl] = acc.m;
      Ls[grp][rl] = l;
    }
    constexpr int H = DT / 2;
    give_half<H>(Ks0, Ks1, acc.o, grp, wave, lane);
    static_assert(kHalf<H> <= sizeof(Ks0), "a half fits");
    lds_barrier();
    const float mo = Ms[grp ^ 1][rl], lo = Ls[grp ^ 1][rl], m = fmaxf(acc.m, mo);
    const float mc = m == -INFINITY ? 0.f : m * a.c;
    const float fm = acc.m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(acc.mc - mc);
    const float fo = mo == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mo * a.c - mc);
    l = l * fm + lo * fo;
    acc.mc = mc;
    const float inv = inverse_sum(l);
#pragma unroll
    for (int dt = 0; dt < H; ++dt) {
      f32x16 v = taken_half<H>(Ks0, Ks1, dt, grp, wave, lane);
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] = (grp ? acc.o[dt + H][k] : acc.o[dt][k]) * fm + v[k] * fo;
      store_cols(dst, v, inv, grp * H + dt, a.d, lane);
    }
  }
  if (a.lse && grp == 0 && lane < 32 && row < s.nq)
    a.lse[(int64_t)head * a.lse_stride + s.q0 + row] = lse_of(acc.mc, l);
}

// ------------------------------------------------------------------------------------------
// Few query rows over many keys. The query heads that share a key head are packed with the tokens
// into rows (row = token * group + head in group), 32 rows a workgroup; its keys are one range of the
// sequence's, and its 4 waves take 32-key tiles of that range in turn, each through two LDS tiles of its
// own without barriers: a tile is read into registers whole and its place refilled before the
// arithmetic, so two tiles (32 KiB a wave at d = 128) are always on their way. The waves' results are
// joined in LDS; with several ranges they go to the workspace and attn_join_kernel joins them, in order.
// Bound by memory: the keys and values, once. One token each for sixteen sequences of 1 to 8191 keys, 64
// heads over 8, d 128: 42 us for 224 MB (5.3 TB/s) and 4 us for the join; with one tile in flight a wave and
// ranges for two workgroups a compute unit it took 58.
template <int DP>
struct SplitWave {
  static constexpr int BN = 32, KS = DP / 16, DT = DP / 32;
  typedef Tile<DP> T;
  typedef KvStream<DP, BN, 1> Stream;
  bf16x8 qf[KS];
  Online<DT> acc;
  Stream kv;
  Range mine, first, last;   // keys that the lane's row, the tile's first and its last row see
  float c, slack;
  int lane;
  // the tile in (kt, vt) with keys from j0; afterwards the tile from `next` (if below `end`) is on its way there
  __device__ __forceinline__ void tile(uint16_t* kt, uint16_t* vt, int j0, int next, int end) {
    bf16x8 kf[KS], vf[2 * DT];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) kf[ks] = T::rows(kt, 0, ks, lane);
#pragma unroll
    for (int i = 0; i < 2 * DT; ++i) vf[i] = T::cols(vt, 16 * (i / DT), i % DT, lane);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read out before it is refilled
    if (next < end) kv.load(kt, vt, next, 0);
    f32x16 sc[1];
    sc[0] = zero16();
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) sc[0] = mfma(kf[ks], qf[ks], sc[0]);
    // some row does not see some key (ranges end on tiles)
    if (j0 + BN > first.hi || j0 < last.lo) hide(sc[0], mine, j0, lane, -INFINITY);
    acc.update(sc, c, slack);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const bf16x8 p = pack8(sc[0], kk);
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) acc.o[dt] = mfma(vf[kk * DT + dt], p, acc.o[dt]);
    }
  }
};

template <int DP>
__global__ __launch_bounds__(256, DP == 128 ? 1 : 2) void attn_split_kernel(const AttnFwdArgs a, const AttnSeqs sq,
                                                                          const AttnSplit sp) {
  constexpr int BN = 32, DT = DP / 32;
  typedef SplitWave<DP> Wave;
  typedef typename Wave::Stream Stream;
  // [keys, values][wave]; a variable per tile in flight, so that reads of one wait only for its own loads
  __shared__ __attribute__((aligned(16))) uint16_t ring0[2][4][BN * DP];
  __shared__ __attribute__((aligned(16))) uint16_t ring1[2][4][BN * DP];
  __shared__ float Ms[4][32], Ls[4][32];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int G = a.heads / a.kv_heads;
  const Unit u = unit_of((int)blockIdx.x, a.kv_heads, 1);
  const Found at_seq = find_seq(sq, u.tile);
  const AttnSeq s = at_seq.seq;
  const int si = at_seq.index, local = u.tile - at_seq.first;
  const int ns = sp.nsplit[si], split = local % ns, rt = local / ns;
  const int shift = s.nk - s.nq, rows = s.nq * G;
  const int row = rt * 32 + (lane & 31);
  const int tok = min(row, rows - 1) / G, head = u.kvh * G + min(row, rows - 1) % G;
  const int t0 = rt * 32 / G, t1 = min(rows - 1, rt * 32 + 31) / G;   // tokens of the row tile
  Wave w;
  w.first = visible(t0 + shift, s.nk, a.causal, a.window);
  w.last = visible(t1 + shift, s.nk, a.causal, a.window);
  w.mine = visible(tok + shift, s.nk, a.causal, a.window);
  // tiles are counted from the first key that the sequence's first row sees (none before it is read)
  const int lo = sp.lo[si];
  const int k_lo = lo + max((w.first.lo - lo) & ~(BN - 1), split * sp.chunk);
  const int k_hi = min(w.last.hi, lo + (split + 1) * sp.chunk);
  const int j_w = k_lo + wave * BN;   // the wave's first tile; its tiles are 4 apart
  w.kv.init(a.k, a.v, s, u.kvh, a.d, 0, lane);
  if (j_w < k_hi) w.kv.load(ring0[0][wave], ring0[1][wave], j_w, 0);
  if (j_w + 4 * BN < k_hi) w.kv.load(ring1[0][wave], ring1[1][wave], j_w + 4 * BN, 0);
  load_rows<DP>(w.qf, row < rows ? a.q.p + (s.q0 + tok) * a.q.token + (int64_t)head * a.q.head : nullptr, a.d, lane);
  w.acc.init();
  w.c = a.c;
  w.slack = slack_of(a.c);
  w.lane = lane;
  for (int j = j_w; j < k_hi; j += 8 * BN) {
    if (j + 4 * BN < k_hi) wait_vmcnt<Stream::kLoads>();   // ring1's loads may be in flight
    else wait_vmcnt<0>();
    asm volatile("" ::: "memory");   // the tile's LDS reads stay after the wait
    w.tile(ring0[0][wave], ring0[1][wave], j, j + 8 * BN, k_hi);
    if (j + 4 * BN >= k_hi) break;
    if (j + 8 * BN < k_hi) wait_vmcnt<Stream::kLoads>();
    else wait_vmcnt<0>();
    asm volatile("" ::: "memory");
    w.tile(ring1[0][wave], ring1[1][wave], j + 4 * BN, j + 12 * BN, k_hi);
  }
  Online<DT>& acc = w.acc;

  // join the waves: the common maximum, then the scaled sums, added in wave order
  float l = half_sum(acc.l);
  if (lane < 32) {
    Ms[wave][lane] = acc.m;
    Ls[wave][lane] = l;
  }
  __syncthreads();
  const int col = lane & 31;
  float mx = -INFINITY;
#pragma unroll
  for (int k = 0; k < 4; ++k) mx = fmaxf(mx, Ms[k][col]);
  const float mxc = mx == -INFINITY ? 0.f : mx * a.c;
  l = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float w = Ms[k][col] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(Ms[k][col] * a.c - mxc);
    l += Ls[k][col] * w;   // 0 times NaN stays NaN
  }
  const float f = acc.m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(acc.mc - mxc);
  __syncthreads();
  // the waves' outputs as [wave][d][32 rows]
  constexpr int P = 33;
  // waves 0 and 1 in ring0, 2 and 3 in ring1
  static_assert(2 * DP * P * 4 <= sizeof(ring0), "two waves' outputs fit a ring");
  float* const out0 = reinterpret_cast<float*>(&ring0[0][0][0]);
  float* const out1 = reinterpret_cast<float*>(&ring1[0][0][0]);
  float* buf = (wave < 2 ? out0 : out1) + (wave & 1) * (DP * P);
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int i = 0; i < 16; ++i) buf[(32 * dt + acc_row(i, lane)) * P + col] = acc.o[dt][i] * f;
  __syncthreads();
  // thread: row tid / 8, columns 8 (tid % 8) + 64 k
  const int orow = tid >> 3, grow = rt * 32 + orow;
  const float rl = __shfl(l, orow), rm = __shfl(mxc, orow);   // the row's statistics, as lane `orow` holds them
  if (grow >= rows) return;
  const int otok = grow / G, ohead = u.kvh * G + grow % G;
#pragma unroll
  for (int k = 0; k < DP / 64; ++k) {
    const int c0 = 8 * (tid & 7) + 64 * k;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = 0.f;
#pragma unroll
      for (int k2 = 0; k2 < 4; ++k2) v[e] += (k2 < 2 ? out0 : out1)[(k2 & 1) * (DP * P) + (c0 + e) * P + orow];
    }
    if (c0 >= a.d) continue;
    if (ns == 1) {
      const float inv = inverse_sum(rl);
      u32x4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = pack_bf16x2(v[2 * e] * inv, v[2 * e + 1] * inv);
      *reinterpret_cast<u32x4*>(a.o.p + (s.q0 + otok) * a.o.token + (int64_t)ohead * a.o.head + c0) = o;
    } else {
      float* part = sp.part + (sp.row0[si] + ((int64_t)grow * a.kv_heads + u.kvh) * ns + split) * (int64_t)(a.d + 8);
      *reinterpret_cast<f32x4*>(part + c0) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(part + c0 + 4) = f32x4{v[4], v[5], v[6], v[7]};
    }
  }
  if ((tid & 7) == 0) {
    if (ns == 1) {
      if (a.lse) a.lse[(int64_t)ohead * a.lse_stride + s.q0 + otok] = lse_of(rm, rl);
    } else {
      float* part = sp.part + (sp.row0[si] + ((int64_t)grow * a.kv_heads + u.kvh) * ns + split) * (int64_t)(a.d + 8);
      part[a.d] = rl == 0.f ? -INFINITY : rm;   // finite (0 at least) where the sum is NaN: the join reads it
      part[a.d + 1] = rl;
    }
  }
}

// Joins the ranges of attn_split_kernel: one wave per query row and head, ranges in order.
__global__ __launch_bounds__(256) void attn_join_kernel(const AttnFwdArgs a, const AttnSeqs sq, const AttnSplit sp) {
  const int lane = threadIdx.x & 63;
  const int G = a.heads / a.kv_heads;
  const int item = (int)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);   // row of a joined sequence x key head
  // sequences with one range have no items
  const int f = lane < sq.count ? sp.join_first[lane] : 0x7FFFFFFF;
  const int si = __builtin_amdgcn_readfirstlane((int)__popcll(__ballot(f <= item)) - 1);
  if (item >= sp.join_first[sq.count]) return;
  const AttnSeq s = sq.seq[si];
  const int local = item - sp.join_first[si], ns = sp.nsplit[si];
  const int grow = local / a.kv_heads, kvh = local % a.kv_heads;
  const int tok = grow / G, head = kvh * G + grow % G;
  const float* part = sp.part + (sp.row0[si] + (int64_t)local * ns) * (int64_t)(a.d + 8);
  const int64_t step = a.d + 8;
  float mx = -INFINITY, l = 0.f, v0 = 0.f, v1 = 0.f;
  const int c = 2 * lane;
  for (int k0 = 0; k0 < ns; k0 += 64) {   // 64 ranges at a time: lane i holds the statistics of range k0 + i
    const int n = min(64, ns - k0);
    const float* p = part + (k0 + min(lane, n - 1)) * step + a.d;
    const float m = lane < n ? p[0] : -INFINITY, lk = lane < n ? p[1] : 0.f;
    const float top = fmaxf(mx, wave_max(m));
    if (top == -INFINITY) continue;
    const float f = __builtin_amdgcn_exp2f(mx - top);   // 0 while nothing was seen
    const float w = __builtin_amdgcn_exp2f(m - top), wl = w * lk;
    l *= f;
    v0 *= f;
    v1 *= f;
    mx = top;
    for (int k = 0; k < n; k += 4) {   // four ranges' loads at a time; those past the end have weight 0
      float2 x[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        x[q] = c < a.d ? *reinterpret_cast<const float2*>(part + (k0 + min(k + q, n - 1)) * step + c) : make_float2(0.f, 0.f);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int at = min(k + q, 63);
        const float wk = k + q < n ? __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w), at)) : 0.f;
        l += k + q < n ? __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wl), at)) : 0.f;
        v0 = __fmaf_rn(wk, x[q].x, v0);
        v1 = __fmaf_rn(wk, x[q].y, v1);
      }
    }
  }
  const float inv = inverse_sum(l);
  if (c < a.d)
    *reinterpret_cast<uint32_t*>(a.o.p + (s.q0 + tok) * a.o.token + (int64_t)head * a.o.head + c) =
        pack_bf16x2(v0 * inv, v1 * inv);
  if (a.lse && lane == 0)
    a.lse[(int64_t)head * a.lse_stride + s.q0 + tok] = lse_of(mx, l);
}

// ------------------------------------------------------------------------------------------
// Backward, first launch: delta (and, for the second launch, lse log2(e) and -delta) and dq. As the
// forward (128 query rows a workgroup, keys streamed), with the probabilities recomputed from lse: three
// products a tile instead of two, 8192 tokens, 32 heads over 8, d 128, not causal 1303 us = 1266 TFLOP/s.
// delta is formed from the forward's rounded o, as the call gets it: an error of up to 2^-8 |do||o| in every
// dS of a row, which with the rounding of dS itself puts dq and dk at 2.5e-3 of their norm from the exact
// ones (their own rounding to bf16 alone is 1.7e-3), and at 4e-3 where rows see few keys. -delta enters the
// products as their starting value, which saves a subtraction per score.
// GR as in the forward, one group and two, us for the whole backward: one causal sequence, 32 heads over 8, of
// 1536 tokens 110.5 and 107.2, of 2048 154.8 and 153.9, 3000 tokens, 16 heads over 4, 184 and 170; four causal
// sequences of 512 74.9 and 81.8, 8192 tokens 1706 and 1755. At d = 64: 78.6 and 75.5, 102.7 and 99.4, 131 and 120;
// 48.1 and 51.6, 935 and 983.
// One pass over the pairs could give dq, dk and dv together with five products instead of seven, but its
// sums of dq over key tiles would need atomics, in no fixed order, or a partial dq per key tile.
template <int DP, int GR>
__global__ __launch_bounds__(256 * GR, 2) void attn_dq_kernel(const AttnBwdArgs a, const AttnSeqs sq) {
  constexpr int BN = 64, KS = DP / 16, DT = DP / 32;
  typedef Tile<DP> T;
  typedef KvStream<DP, BN, 4> Stream;
  __shared__ __attribute__((aligned(16))) uint16_t Ks0[GR][BN * DP], Ks1[GR][BN * DP], Vs0[GR][BN * DP], Vs1[GR][BN * DP];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) & 3;
  const int grp = GR == 1 ? 0 : __builtin_amdgcn_readfirstlane(tid >> 8);
  const int G = a.heads / a.kv_heads;
  const Unit u = unit_of((int)blockIdx.x, a.kv_heads, G);
  const Found at_seq = find_seq(sq, u.tile);
  const AttnSeq s = at_seq.seq;
  const int qt = at_seq.next - 1 - u.tile;
  const int head = u.kvh * G + u.sub;
  const int r0 = qt * 128, shift = s.nk - s.nq;

  const int row = r0 + wave * 32 + (lane & 31);
  const bool own = row < s.nq;
  bf16x8 qf[KS], gf[KS];
  load_rows<DP>(qf, own ? a.q.p + (s.q0 + row) * a.q.token + (int64_t)head * a.q.head : nullptr, a.d, lane);
  load_rows<DP>(gf, own ? a.dout.p + (s.q0 + row) * a.dout.token + (int64_t)head * a.dout.head : nullptr, a.d, lane);
  float delta = 0.f, lse2 = 0.f;
  {
    bf16x8 of[KS];
    load_rows<DP>(of, own ? a.o.p + (s.q0 + row) * a.o.token + (int64_t)head * a.o.head : nullptr, a.d, lane);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int e = 0; e < 8; ++e) delta = __fmaf_rn((float)gf[ks][e], (float)of[ks][e], delta);
    delta = half_sum(delta);
  }
  const int64_t at = (int64_t)head * a.lse_stride + s.q0 + row;
  if (own) {
    lse2 = a.lse[at] * kLog2e;
    if (grp == 0 && lane < 32) {   // as the second launch takes them
      a.lse2[at] = lse2;
      a.less_delta[at] = -delta;
    }
  }
  f32x16 less_delta;
#pragma unroll
  for (int i = 0; i < 16; ++i) less_delta[i] = -delta;

  const int r1 = min(s.nq, r0 + 128) - 1;
  const int k_lo = visible(r0 + shift, s.nk, a.causal, a.window).lo;
  const int k_hi = visible(r1 + shift, s.nk, a.causal, a.window).hi;
  const int w0 = r0 + wave * 32, w1 = min(s.nq - 1, w0 + 31);
  const Range wa = visible(w0 + shift, s.nk, a.causal, a.window), wb = visible(w1 + shift, s.nk, a.causal, a.window);
  const Range mine = visible(row + shift, s.nk, a.causal, a.window);
  const int nt = k_hi > k_lo ? (k_hi - k_lo + GR * BN - 1) / (GR * BN) : 0;   // of each group

  Stream kv;
  kv.init(a.k, a.v, s, u.kvh, a.d, wave, lane);
  f32x16 dq[DT];
#pragma unroll
  for (int dt = 0; dt < DT; ++dt) dq[dt] = zero16();
  const int j_g = k_lo + grp * BN;   // the group's first tile; its tiles are GR apart
  if (nt > 0) kv.load(Ks0[grp], Vs0[grp], j_g, wave);
  auto tile = [&](int t, const uint16_t* Kt, const uint16_t* Vt, uint16_t* kn, uint16_t* vn) __attribute__((always_inline)) {
    wait_vmcnt<0>();
    lds_barrier();
    if (t + 1 < nt) kv.load(kn, vn, j_g + (t + 1) * GR * BN, wave);
#pragma unroll
    for (int kt = 0; kt < BN / 32; ++kt) {
      const int j0 = j_g + t * GR * BN + 32 * kt;
      if (j0 < wb.hi && j0 + 32 > wa.lo) {
        f32x16 sc = zero16(), dp = less_delta;   // do.v - delta comes out of the products
        constexpr int R = 2;   // operands on their way, as in the forward; more of them spill
        bf16x8 f[R];
        auto operand = [&](int n) __attribute__((always_inline)) {
          if (n < KS) return T::rows(Kt, 32 * kt, n, lane);
          if (n < 2 * KS) return T::rows(Vt, 32 * kt, n - KS, lane);
          return T::cols(Kt, 32 * kt + 16 * ((n - 2 * KS) / DT), n % DT, lane);
        };
#pragma unroll
        for (int n = 0; n < R; ++n) f[n] = operand(n);
        keep_order();
#pragma unroll
        for (int n = 0; n < 2 * KS; ++n) {
          if (n < KS) sc = mfma(f[n % R], qf[n % KS], sc);
          else dp = mfma(f[n % R], gf[n % KS], dp);
          f[n % R] = operand(n + R);
          keep_order();
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) dp[i] *= __builtin_amdgcn_exp2f(__fmaf_rn(sc[i], a.c, -lse2));
        // selected away, not multiplied: a row without keys has lse -inf
        if (j0 + 32 > wa.hi || j0 < wb.lo) hide(dp, mine, j0, lane, 0.f);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          const bf16x8 ds = pack8(dp, kk);
#pragma unroll
          for (int dt = 0; dt < DT; ++dt) {
            const int n = 2 * KS + kk * DT + dt;
            dq[dt] = mfma(f[n % R], ds, dq[dt]);
            if (n + R < 3 * KS) f[n % R] = operand(n + R);
          }
        }
      }
    }
  };
  for (int t = 0; t < nt; t += 2) {
    tile(t, Ks0[grp], Vs0[grp], Ks1[grp], Vs1[grp]);
    if (t + 1 < nt) tile(t + 1, Ks1[grp], Vs1[grp], Ks0[grp], Vs0[grp]);
  }
  uint16_t* dst = own ? a.dq.p + (s.q0 + row) * a.dq.token + (int64_t)head * a.dq.head : nullptr;
  if constexpr (GR == 1) {
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) store_cols(dst, dq[dt], a.scale, dt, a.d, lane);
  } else {
    // each group keeps half of the columns and adds the other group's sums of them
    constexpr int H = DT / 2;
    lds_barrier();
    give_half<H>(Ks0, Ks1, dq, grp, wave, lane);
    static_assert(kHalf<H> <= sizeof(Ks0), "a half fits");
    lds_barrier();
#pragma unroll
    for (int dt = 0; dt < H; ++dt) {
      f32x16 v = taken_half<H>(Ks0, Ks1, dt, grp, wave, lane);
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] += grp ? dq[dt + H][k] : dq[dt][k];
      store_cols(dst, v, a.scale, grp * H + dt, a.d, lane);
    }
  }
}

// ------------------------------------------------------------------------------------------
// Backward, second launch: dk and dv. A workgroup of 4 waves takes 128 keys of one key head, 32 per
// wave; the rows of q and do of its query heads stream through LDS, two tiles deep. The query heads of
// the group can be split over several workgroups (gper heads each): their fp32 results go to the
// workspace, and attn_dkv_sum_kernel adds them in order.
// WV = 1: the keys' and the values' operands stay in registers (of 512, one wave a SIMD) and tiles have 64
// rows, two blocks that overlap. WV = 2: the values' operands are read from LDS and tiles have 32 rows, which
// leaves room for two waves a SIMD. A workgroup of the first kind alone on a compute unit takes 1.9 us for 64
// rows of 128 keys at d = 128, of the second 2.25 us, and two of the second 3.9 us for both (kv_plan chooses):
// 32 heads over 8, one causal sequence of 2048 tokens 94 us and 97, four of 512 42 and 34, 8192 tokens, not
// causal, 2.06 ms and 1.94 (1130 TFLOP/s of the four products).
template <int DP, int ROWS, int NW>
struct RowStream {   // rows [lo, hi) of q, do, lse2 and less_delta, head after head, in tiles of ROWS <= 64
  typedef TileDma<DP, ROWS, NW> Dma;
  static constexpr int kLoads = 2 * Dma::kLoads + 2;   // per wave and tile
  Dma qd, gd;
  const AttnBwdArgs& a;
  int64_t q0;
  int nq, head, i, lo, hi;
  __device__ __forceinline__ RowStream(const AttnBwdArgs& args, const AttnSeq& s, int head0, int lo_, int hi_, int wave, int lane)
      : a(args), q0(s.q0), nq(s.nq), head(head0), i(lo_), lo(lo_), hi(hi_) {
    qd.init(wave, lane, a.d, (uint32_t)a.q.token);
    gd.init(wave, lane, a.d, (uint32_t)a.dout.token);
  }
  // the values of 32 keys from j, as an LDS tile
  static __device__ __forceinline__ void values(uint16_t* t, const AttnBwdArgs& a, const AttnSeq& s, int kvh, int j, int lane) {
    TileDma<DP, 32, 1> vd;
    vd.init(0, lane, a.d, (uint32_t)a.v.token);
    vd.load(t, a.v.p + (s.k0 + j) * a.v.token + (int64_t)kvh * a.v.head, s.nk - j, a.d, (uint32_t)a.v.token, 0);
  }
  // the next tile; lse2 and less_delta go to the wave's own copies. Rows past the sequence read 0: their q
  // and do are 0 too, so they add nothing.
  __device__ __forceinline__ void load(uint16_t* qt, uint16_t* gt, float* lt, float* dt, int wave, int lane) {
    const int64_t tok = q0 + i, at = (int64_t)head * a.lse_stride + tok;
    const int rows = nq - i, nrec = min(ROWS, rows) * 4;
    qd.load(qt, a.q.p + tok * a.q.token + (int64_t)head * a.q.head, rows, a.d, (uint32_t)a.q.token, wave);
    gd.load(gt, a.dout.p + tok * a.dout.token + (int64_t)head * a.dout.head, rows, a.d, (uint32_t)a.dout.token, wave);
    __amdgpu_buffer_rsrc_t rl = __builtin_amdgcn_make_buffer_rsrc((void*)(a.lse2 + at), (short)0, nrec, kRsrcFlags);
    __amdgpu_buffer_rsrc_t rd = __builtin_amdgcn_make_buffer_rsrc((void*)(a.less_delta + at), (short)0, nrec, kRsrcFlags);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rl, (lds_void*)lt, 4, (uint32_t)lane * 4u, 0, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rd, (lds_void*)dt, 4, (uint32_t)lane * 4u, 0, 0, 0);
    i += ROWS;
    if (i >= hi) {
      i = lo;
      ++head;
    }
  }
};

template <int DP, int WV>
__global__ __launch_bounds__(256, WV) void attn_dkv_kernel(const AttnBwdArgs a, const AttnSeqs sq, const AttnKvSplit sp) {
  constexpr int BM = WV == 1 ? 64 : 32, KS = DP / 16, DT = DP / 32;
  typedef Tile<DP> T;
  typedef RowStream<DP, BM, 4> Stream;
  // a variable per stage, as in the forward (dq and this kernel together: packed 70B batch 390 -> 362 us)
  __shared__ __attribute__((aligned(16))) uint16_t Qs0[BM * DP], Qs1[BM * DP], Gs0[BM * DP], Gs1[BM * DP];
  // lse log2(e) and -delta, a copy per wave
  __shared__ __attribute__((aligned(16))) float Ls0[4][64], Ls1[4][64], Ds0[4][64], Ds1[4][64];
  __shared__ __attribute__((aligned(16))) uint16_t Vs[WV == 1 ? 8 : 128 * DP];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int G = a.heads / a.kv_heads;
  const Unit u = unit_of((int)blockIdx.x, a.kv_heads, sp.splits, WV == 2);
  const Found at_seq = find_seq(sq, u.tile);
  const AttnSeq s = at_seq.seq;
  const int j0 = (u.tile - at_seq.first) * 128;     // first key of the workgroup
  const int shift = s.nk - s.nq;
  const int key = j0 + wave * 32 + (lane & 31);
  const bool own = key < s.nk;
  bf16x8 kf[KS], vf[WV == 1 ? KS : 1];
  load_rows<DP>(kf, own ? a.k.p + (s.k0 + key) * a.k.token + (int64_t)u.kvh * a.k.head : nullptr, a.d, lane);
  uint16_t* const vt = Vs + (WV == 1 ? 0 : wave * 32 * DP);
  if constexpr (WV == 1)
    load_rows<DP>(vf, own ? a.v.p + (s.k0 + key) * a.v.token + (int64_t)u.kvh * a.v.head : nullptr, a.d, lane);
  else
    Stream::values(vt, a, s, u.kvh, j0 + wave * 32, lane);

  // query rows [i_lo, i_hi) that see some key of the workgroup, from a multiple of BM on; but none that sees no
  // key at all (when causal the first nq - nk), whose q and dout may hold anything: 0 times NaN is no zero
  const int jl = min(s.nk, j0 + 128) - 1;
  const int i_lo = a.causal ? max(max(0, j0 - shift) & ~(BM - 1), -shift) : 0;
  const int i_hi = a.window ? (int)min((int64_t)s.nq, (int64_t)jl + a.window - shift) : s.nq;
  const int tiles = i_hi > i_lo ? (i_hi - i_lo + BM - 1) / BM : 0;
  const int g0 = u.sub * sp.gper, g1 = min(G, g0 + sp.gper);
  const int total = tiles * (g1 - g0);
  // rows that see the lane's key
  Range seen;
  seen.lo = a.causal ? max(0, key - shift) : 0;
  seen.hi = a.window ? (int)min((int64_t)key + a.window - shift, (int64_t)INT_MAX) : INT_MAX;
  // and of the wave's keys: rows in [all_lo, all_hi) see all, rows in [any_lo, any_hi) see some
  const int kw = j0 + wave * 32;
  const int any_lo = a.causal ? kw - shift : INT_MIN, all_lo = a.causal ? kw + 31 - shift : INT_MIN;
  const int all_hi = a.window ? (int)min((int64_t)kw + a.window - shift, (int64_t)INT_MAX) : INT_MAX;
  const int any_hi = a.window ? (int)min((int64_t)kw + 31 + a.window - shift, (int64_t)INT_MAX) : INT_MAX;

  Stream rows(a, s, u.kvh * G + g0, i_lo, i_hi, wave, lane);

  f32x16 dk[DT], dv[DT];
#pragma unroll
  for (int dt = 0; dt < DT; ++dt) {
    dk[dt] = zero16();
    dv[dt] = zero16();
  }
  if (total > 0) rows.load(Qs0, Gs0, Ls0[wave], Ds0[wave], wave, lane);
  int ci = i_lo;   // first row of the tile in work
  auto tile = [&](int t, const uint16_t* Qt, const uint16_t* Gt, const float* Lt, const float* Dt, uint16_t* qn, uint16_t* gn, float* ln,
                  float* dn) __attribute__((always_inline)) {
    wait_vmcnt<0>();
    lds_barrier();
    if (t + 1 < total) rows.load(qn, gn, ln, dn, wave, lane);
    if constexpr (WV == 1) {
      if (ci + BM - 1 >= any_lo && ci < any_hi) {
        // The wave is alone on its SIMD, so its two blocks of 32 rows overlap by program order: the second's
        // scores are formed between the first's exponentials, the first's sums between the second's. Each
        // operand register takes its next contents from LDS as soon as its product is issued.
        const bool masked = ci < all_lo || ci + BM - 1 >= all_hi;
        bf16x8 fa[KS], fb[KS];   // operands on their way
        f32x16 sc[2], dp[2], ls;
        bf16x8 p[2], ds[2];
        auto start = [&](int mt) __attribute__((always_inline)) {
          sc[mt] = zero16();
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(&Dt[32 * mt + 8 * g + 4 * (lane >> 5)]);
#pragma unroll
            for (int e = 0; e < 4; ++e) dp[mt][4 * g + e] = x[e];
          }
        };
        auto take_lse = [&](int mt) __attribute__((always_inline)) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(&Lt[32 * mt + 8 * g + 4 * (lane >> 5)]);
#pragma unroll
            for (int e = 0; e < 4; ++e) ls[4 * g + e] = x[e];
          }
        };
        auto finish = [&](int mt) __attribute__((always_inline)) {
          if (masked) {
            hide(sc[mt], seen, ci + 32 * mt, lane, 0.f);
            hide(dp[mt], seen, ci + 32 * mt, lane, 0.f);
          }
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) {
            p[kk] = pack8(sc[mt], kk);
            ds[kk] = pack8(dp[mt], kk);
          }
        };
#pragma unroll
        for (int k = 0; k < KS; ++k) fa[k] = T::rows(Qt, 0, k, lane);
        start(0);
#pragma unroll
        for (int k = 0; k < KS; ++k) fb[k] = T::rows(Gt, 0, k, lane);
        keep_order();
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          sc[0] = mfma(fa[k], kf[k], sc[0]);
          fa[k] = T::rows(Qt, 32, k, lane);
          keep_order();
        }
        take_lse(0);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          dp[0] = mfma(fb[k], vf[k], dp[0]);
          fb[k] = T::rows(Gt, 32, k, lane);
          keep_order();
        }
        start(1);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          sc[1] = mfma(fa[k], kf[k], sc[1]);
#pragma unroll
          for (int e = 16 / KS * k; e < 16 / KS * (k + 1); ++e) sc[0][e] = __builtin_amdgcn_exp2f(__fmaf_rn(sc[0][e], a.c, -ls[e]));
          fa[k] = T::cols(Gt, 16 * (k / DT), k % DT, lane);
          keep_order();
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          dp[1] = mfma(fb[k], vf[k], dp[1]);
#pragma unroll
          for (int e = 16 / KS * k; e < 16 / KS * (k + 1); ++e) dp[0][e] *= sc[0][e];
          fb[k] = T::cols(Qt, 16 * (k / DT), k % DT, lane);
          keep_order();
        }
        take_lse(1);
        finish(0);
        keep_order();
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          dv[k % DT] = mfma(fa[k], p[k / DT], dv[k % DT]);
#pragma unroll
          for (int e = 16 / KS * k; e < 16 / KS * (k + 1); ++e) sc[1][e] = __builtin_amdgcn_exp2f(__fmaf_rn(sc[1][e], a.c, -ls[e]));
          fa[k] = T::cols(Gt, 32 + 16 * (k / DT), k % DT, lane);
          keep_order();
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          dk[k % DT] = mfma(fb[k], ds[k / DT], dk[k % DT]);
#pragma unroll
          for (int e = 16 / KS * k; e < 16 / KS * (k + 1); ++e) dp[1][e] *= sc[1][e];
          fb[k] = T::cols(Qt, 32 + 16 * (k / DT), k % DT, lane);
          keep_order();
        }
        finish(1);
#pragma unroll
        for (int k = 0; k < KS; ++k) dv[k % DT] = mfma(fa[k], p[k / DT], dv[k % DT]);
#pragma unroll
        for (int k = 0; k < KS; ++k) dk[k % DT] = mfma(fb[k], ds[k / DT], dk[k % DT]);
      }
    } else {
      const int i0 = ci;
      if (i0 + 31 >= any_lo && i0 < any_hi) {
        f32x16 sc = zero16(), dp;   // do.v - delta comes out of the products
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x4 x = *reinterpret_cast<const f32x4*>(&Dt[8 * g + 4 * (lane >> 5)]);
#pragma unroll
          for (int e = 0; e < 4; ++e) dp[4 * g + e] = x[e];
        }
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) sc = mfma(T::rows(Qt, 0, ks, lane), kf[ks], sc);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
          dp = mfma(T::rows(Gt, 0, ks, lane), T::rows(vt, 0, ks, lane), dp);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x4 x = *reinterpret_cast<const f32x4*>(&Lt[8 * g + 4 * (lane >> 5)]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = 4 * g + e;
            sc[i] = __builtin_amdgcn_exp2f(__fmaf_rn(sc[i], a.c, -x[e]));
            dp[i] *= sc[i];
          }
        }
        // selected away, not multiplied: a row without keys has lse -inf
        if (i0 < all_lo || i0 + 31 >= all_hi) {
          hide(sc, seen, i0, lane, 0.f);
          hide(dp, seen, i0, lane, 0.f);
        }
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          const bf16x8 p = pack8(sc, kk), ds = pack8(dp, kk);
#pragma unroll
          for (int dt = 0; dt < DT; ++dt) dv[dt] = mfma(T::cols(Gt, 16 * kk, dt, lane), p, dv[dt]);
#pragma unroll
          for (int dt = 0; dt < DT; ++dt) dk[dt] = mfma(T::cols(Qt, 16 * kk, dt, lane), ds, dk[dt]);
        }
      }
    }
    ci += BM;
    if (ci >= i_hi) ci = i_lo;
  };
  if constexpr (WV == 1 || DP == 64) {
    for (int t = 0; t < total; t += 2) {
      tile(t, Qs0, Gs0, Ls0[wave], Ds0[wave], Qs1, Gs1, Ls1[wave], Ds1[wave]);
      if (t + 1 < total) tile(t + 1, Qs1, Gs1, Ls1[wave], Ds1[wave], Qs0, Gs0, Ls0[wave], Ds0[wave]);
    }
  } else {   // at d > 64 code for each stage does not leave registers enough for two waves
    for (int t = 0; t < total; ++t) {
      const bool o = t & 1;
      tile(t, o ? Qs1 : Qs0, o ? Gs1 : Gs0, o ? Ls1[wave] : Ls0[wave], o ? Ds1[wave] : Ds0[wave], o ? Qs0 : Qs1, o ? Gs0 : Gs1,
           o ? Ls0[wave] : Ls1[wave], o ? Ds0[wave] : Ds1[wave]);
    }
  }
  if (sp.splits == 1) {
    uint16_t* pk = own ? a.dk.p + (s.k0 + key) * a.dk.token + (int64_t)u.kvh * a.dk.head : nullptr;
    uint16_t* pv = own ? a.dv.p + (s.k0 + key) * a.dv.token + (int64_t)u.kvh * a.dv.head : nullptr;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) {
      store_cols(pk, dk[dt], a.scale, dt, a.d, lane);
      store_cols(pv, dv[dt], 1.f, dt, a.d, lane);
    }
  } else {
    // accumulators as they lie in the lanes: [tile][key head][split][wave][dk, dv][DT][4][lane][4]
    float* dst = sp.part + ((((int64_t)u.tile * a.kv_heads + u.kvh) * sp.splits + u.sub) * 4 + wave) * (2 * 32 * DP) + 4 * lane;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        f32x4 x, y;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = dk[dt][4 * g + e];
          y[e] = dv[dt][4 * g + e];
        }
        *reinterpret_cast<f32x4*>(dst + (dt * 4 + g) * 256) = x;
        *reinterpret_cast<f32x4*>(dst + 32 * DP + (dt * 4 + g) * 256) = y;
      }
  }
}

// Sums the split results of attn_dkv_kernel in split order: a workgroup per key tile, key head and one
// of dk, dv; a wave per 32 keys.
template <int DP>
__global__ __launch_bounds__(256) void attn_dkv_sum_kernel(const AttnBwdArgs a, const AttnSeqs sq, const AttnKvSplit sp) {
  constexpr int DT = DP / 32;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int which = (int)blockIdx.x & 1;
  const int kvh = ((int)blockIdx.x >> 1) % a.kv_heads, tile = ((int)blockIdx.x >> 1) / a.kv_heads;
  const Found at_seq = find_seq(sq, tile);
  const AttnSeq s = at_seq.seq;
  const int key = (tile - at_seq.first) * 128 + wave * 32 + (lane & 31);
  const float* src = sp.part + (((int64_t)tile * a.kv_heads + kvh) * sp.splits * 4 + wave) * (2 * 32 * DP) + which * 32 * DP + 4 * lane;
  f32x16 v[DT];
#pragma unroll
  for (int dt = 0; dt < DT; ++dt) v[dt] = zero16();
  for (int k = 0; k < sp.splits; ++k) {
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(src + (dt * 4 + g) * 256);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[dt][4 * g + e] += x[e];
      }
    src += 4 * (2 * 32 * DP);
  }
  const AttnTensor o = which ? a.dv : a.dk;
  uint16_t* dst = key < s.nk ? o.p + (s.k0 + key) * o.token + (int64_t)kvh * o.head : nullptr;
#pragma unroll
  for (int dt = 0; dt < DT; ++dt) store_cols(dst, v[dt], which ? 1.f : a.scale, dt, a.d, lane);
}

// ------------------------------------------------------------------------------------------
// Host side: plans and launches
static int q_tiles(const AttnSeq& s) { return (int)ceil64(s.nq, 128); }
static int k_tiles(const AttnSeq& s) { return (int)ceil64(s.nk, 128); }

// The forward's plan. Sequences of up to kFewRows query rows are work for attn_split_kernel; the others go
// to attn_fwd_kernel when its workgroups outnumber the compute units (256), or when its estimate, the
// longest workgroup at 0.94 us for 64 keys and 7 us around it, is below that of attn_split_kernel
// (split_chunk); all sequences of a launch of attn_split_kernel have one length of key range. Measured,
// forward and split, us: 512 tokens of 600 keys, 32 heads over 8, 15 and 19; four sequences of 300, 8 heads
// over 2, 10.5 and 14.5; 2000 tokens, 8 heads, 29 and 31; 1000 tokens, 8 heads over 2, 18 and 14; 128 tokens of
// 4096 keys, 32 heads over 8, 52 and 28. The estimate of attn_fwd_kernel is for d = 128 and not made smaller for
// d <= 64, where a tile costs a wave alone nearly as much: at d = 64 the same take 11.1 and 10.8, 10.5 and 10.6, 21
// and 16, 13 and 11, 37 and 20.5, and the split is chosen for all but the four sequences.
// Beside attn_fwd_kernel a launch of attn_split_kernel costs 4 us even for one token, so the short sequences
// stay with the others if that adds less work than 4 us and none is longer than the longest of these (a
// sequence of one token packed with 4095 others, 64 heads over 8: 106 us against 110).
constexpr int kFewRows = 16, kUnits = 256;
struct FwdPlan {
  std::vector<AttnSeq> many, few;
  int64_t chunk = 0;        // keys per range
  int64_t part_floats = 0;  // workspace of one launch (the largest)
};
static int split_count(const AttnSeq& s, int window, int64_t chunk) {
  return (int)std::max<int64_t>(1, ceil64(s.nk - first_key(s, window), chunk));
}
static int64_t row_tiles(const AttnSeq& s, int G) { return ceil64((int64_t)s.nq * G, 32); }

// A compute unit holds one workgroup of attn_split_kernel at a time, so the launch takes as many rounds
// as there are workgroups to a unit, each as long as a range and a fixed part of 5 us (start, first loads,
// joining the waves), and joining ranges costs another launch, 4 us. A key takes a workgroup 0.0064 us by
// the latency of its own loads, 0.0096 where all units read keys that others read too, and 0.022 where all
// read their own (d = 128; less in proportion for smaller tiles). The range length with the smallest sum
// wins. Sixteen sequences of 1 to 8191 keys, 64 heads over 8: 42 us, where ranges for two workgroups a unit on
// average took 52; one sequence of 601 keys, 32 heads over 8: one range 10.8 us, three and the join 13.8; of
// 2000 keys one range 19 and four 15; 128 tokens over 4096 keys: two ranges, 29 us measured and estimated.
static int64_t split_chunk(const std::vector<AttnSeq>& v, int G, int kv_heads, int d, int window, double* cost_us) {
  const double size = padded_d(d) / 128.0;
  int64_t longest = 1, best = 0;
  *cost_us = -1;
  for (const AttnSeq& s : v) longest = std::max(longest, s.nk - first_key(s, window));
  for (int64_t chunk = 256;; chunk += std::max<int64_t>(128, chunk / 8 / 128 * 128)) {
    int64_t wgs = 0, ranges = 0, most = 0;
    for (const AttnSeq& s : v) {
      const int64_t n = (int64_t)split_count(s, window, chunk) * kv_heads;
      ranges += n;
      wgs += row_tiles(s, G) * n;
      most = std::max(most, row_tiles(s, G) * n);
    }
    if (most > kAttnGroups && chunk < longest) continue;   // a sequence has to fit a launch
    const double key = size * std::max({0.0064, 0.0096 * std::min<int64_t>(wgs, kUnits) / kUnits,
                                        0.022 * std::min<int64_t>(ranges, kUnits) / kUnits});
    const double cost = ceil64(wgs, kUnits) * (5 + key * std::min(chunk, longest)) + (chunk < longest ? 4 : 0);
    if (*cost_us < 0 || cost < *cost_us) {
      *cost_us = cost;
      best = chunk;
    }
    if (chunk >= longest) return best;
  }
}
// the sequences of the attn_split_kernel launch from p.few[from] on
static AttnSeqs few_seqs(const FwdPlan& p, size_t from, int G, int kv_heads, int window) {
  return pack_seqs(p.few, from, kv_heads,
                   [&](const AttnSeq& s) { return row_tiles(s, G) * split_count(s, window, p.chunk); });
}
static FwdPlan fwd_plan(const std::vector<AttnSeq>& v, int heads, int kv_heads, int d, int window) {
  FwdPlan p;
  const int G = heads / kv_heads;
  // keys that a workgroup of 128 rows sees at most
  auto seen = [&](const AttnSeq& s) { return window ? std::min<int64_t>(s.nk, (int64_t)window + 128) : (int64_t)s.nk; };
  int64_t wgs = 0, keys = 0, few_keys = 0, few_tiles = 0;
  double cost;
  for (const AttnSeq& s : v) {
    if (s.nq > kFewRows) {
      p.many.push_back(s);
      wgs += (int64_t)q_tiles(s) * heads;
      keys = std::max(keys, seen(s));
    } else {
      p.few.push_back(s);
      few_keys = std::max(few_keys, seen(s));
      few_tiles += ceil64(seen(s), 64) * heads;
    }
  }
  if (!p.many.empty() && wgs <= kUnits) {
    split_chunk(p.many, G, kv_heads, d, window, &cost);
    if (7 + 0.94 / 64 * (double)keys > cost) p.many.clear();
  }
  if (p.many.empty()) {
    p.few = v;
  } else if (few_keys <= keys && 0.94 * (double)few_tiles < 4.0 * kUnits) {
    p.many = v;
    p.few.clear();
  }
  if (p.few.empty()) return p;
  p.chunk = split_chunk(p.few, G, kv_heads, d, window, &cost);
  for (size_t from = 0; from < p.few.size();) {
    const AttnSeqs q = few_seqs(p, from, G, kv_heads, window);
    int64_t f = 0;
    for (int i = 0; i < q.count; ++i) {
      const int ns = split_count(q.seq[i], window, p.chunk);
      if (ns > 1) f += (int64_t)q.seq[i].nq * heads * ns * (d + 8);
    }
    p.part_floats = std::max(p.part_floats, f);
    from += (size_t)q.count;
  }
  return p;
}

// Whether a launch over tiles of 128 query rows takes the form with two groups of waves (see
// attn_fwd_kernel): when its work, spread over the compute units, is at most 1.2 times that of its longest
// workgroup, in tiles of 64 keys (1.13 gains 15 % in the forward, 1.25 loses 14 %).
static bool two_groups(const AttnSeqs& q, int heads, int causal, int window) {
  if ((int64_t)q.first[q.count] * heads > kMaxThreads / 512) return false;
  int64_t longest = 0, total = 0;
  for (int i = 0; i < q.count; ++i) {
    const AttnSeq& s = q.seq[i];
    for (int64_t r = 0; r < s.nq; r += 128) {
      const int64_t p0 = (int64_t)s.nk - s.nq + r, p1 = (int64_t)s.nk - s.nq + std::min<int64_t>(s.nq, r + 128);
      const int64_t hi = causal ? std::max<int64_t>(0, p1) : s.nk;
      const int64_t lo = window ? std::max<int64_t>(0, p0 - window + 1) : 0;
      const int64_t n = hi > lo ? ceil64(hi - lo, 64) : 0;
      longest = std::max(longest, n);
      total += n;
    }
  }
  return (double)total * heads <= 1.2 * kUnits * (double)longest;
}

// 64-row tiles of queries that see some key of key tile t (as attn_dkv_kernel counts them)
static int64_t dkv_row_tiles(const AttnSeq& s, int t, int causal, int window) {
  const int64_t shift = (int64_t)s.nk - s.nq, j0 = 128 * (int64_t)t, jl = std::min<int64_t>(s.nk, j0 + 128) - 1;
  const int64_t lo = causal ? std::max(std::max<int64_t>(0, j0 - shift) & ~int64_t(63), -shift) : 0;
  const int64_t hi = window ? std::min<int64_t>(s.nq, jl + window - shift) : s.nq;
  return hi > lo ? ceil64(hi - lo, 64) : 0;
}

// Plan of the dk, dv launch: parts that the query heads of a group are split into, and waves per SIMD
// (see attn_dkv_kernel). Work is counted in tiles of 64 rows of 128 keys for one query head. The launch takes
// as long as its longest workgroup alone, or as the mean over the compute units with the starts and ends of
// the workgroups and, with a mask, the tiles on its edge of every key tile and head; the parts' fp32 results
// (written, read and added) cost 0.03 us for every tile of 128 keys and part. The coefficients (us) are
// fitted to d = 128. Estimated and measured, sums included: 32 heads over 8, one causal sequence of 2048, 4
// parts, one wave 109 and 109, two waves 113 and 111; four of 512, 4 parts, one wave 60 and 56, two 50 and 47;
// 64 heads over 8, packed sequences of 1500, 1031, 783, 700, 64, 17 and 1 tokens, one wave, 2 parts 232 and
// 234, two waves, 4 parts 230 and 219; 8 heads, one sequence of 4096, one wave 135 and 133, two 176 and 155; 8192
// tokens, not causal, 2113 and 2055, 2024 and 1941. At d <= 64 the times are smaller but the number of parts that
// they choose is still the best or within 1 % of it (d = 64, the whole backward with 1, 2, 4, 8 parts: 2048 tokens
// 235, 143, 99; four of 512 72, 54, 48; the packed batch 361, 232, 186, 204; 1000 tokens, 32 heads over 4, 220, 125,
// 77, 56, where 4, 4, 4 and 8 are chosen).
struct KvPlan {
  int splits, gper, waves;
};
static KvPlan kv_plan(const std::vector<AttnSeq>& v, int heads, int kv_heads, int d, int causal, int window) {
  const int G = heads / kv_heads;
  int64_t tiles = 0, longest = 0, total = 0;
  for (const AttnSeq& s : v) {
    tiles += k_tiles(s);
    if (tiles * kv_heads >= 16 * kUnits) return KvPlan{1, G, 2};   // workgroups enough
    for (int t = 0; t < k_tiles(s); ++t) {
      const int64_t n = dkv_row_tiles(s, t, causal, window);
      longest = std::max(longest, n);
      total += n;
    }
  }
  KvPlan best{1, G, 2};
  double best_cost = -1;
  for (int want = 1; want <= G; ++want) {
    if (G % want) continue;   // equal parts (packed batch as above: 3 parts 10 us slower than 4)
    if (want > 1 && tiles * kv_heads * want > kAttnGroups) break;
    const int gper = G / want;
    const double mean = (double)total * G * kv_heads / kUnits, most = (double)longest * gper;
    const double wgs = (double)tiles * kv_heads * want / kUnits;
    const double edges = causal || window ? (double)tiles * kv_heads * G / kUnits : 0;
    const double sums = want > 1 ? 4 + 0.03 * tiles * kv_heads * want : 0;
    const double one = std::max(1.95 * most + 10, 2.05 * mean + 7 * wgs + 3 * edges) + sums;
    const double two = std::max(2.6 * most + 10, 1.97 * mean + 3.5 * wgs + 1.5 * edges) + sums;
    for (int waves = d <= 64 ? 2 : 1; waves <= 2; ++waves) {   // the small tiles of d <= 64 leave room for two waves anyway
      const double cost = waves == 1 ? one : two;
      if (best_cost < 0 || cost < best_cost) {
        best = KvPlan{want, gper, waves};
        best_cost = cost;
      }
    }
  }
  return best;
}
static int64_t dkv_part_floats(const std::vector<AttnSeq>& v, int splits, int kv_heads, int dp) {
  if (splits == 1) return 0;   // with parts the workgroups of the whole call fit a launch: kAttnSeqs to each
  int64_t most = 0;
  for (size_t from = 0; from < v.size(); from += kAttnSeqs) {
    int64_t t = 0;
    for (size_t i = from; i < v.size() && i < from + kAttnSeqs; ++i) t += k_tiles(v[i]);
    most = std::max(most, t * kv_heads * splits * (128 * 2 * dp));
  }
  return most;
}
static int64_t round64(int64_t f) { return (f + 63) & ~int64_t(63); }

size_t attn_fwd_ws_floats(const AttnSeq* seqs, int64_t count, int heads, int kv_heads, int d, int window) {
  const std::vector<AttnSeq> v = by_work(seqs, count, false);
  return v.empty() ? 0 : (size_t)fwd_plan(v, heads, kv_heads, d, window).part_floats;
}
size_t attn_bwd_ws_floats(const AttnSeq* seqs, int64_t count, int heads, int kv_heads, int d, int causal, int window,
                          int64_t q_tokens) {
  const std::vector<AttnSeq> v = by_work(seqs, count, true);
  const KvPlan plan = kv_plan(v, heads, kv_heads, d, causal, window);
  return (size_t)(2 * round64(q_tokens * heads) + dkv_part_floats(v, plan.splits, kv_heads, padded_d(d)));
}

hipError_t launch_attn_fwd(const AttnFwdArgs& a, const AttnSeq* seqs, int64_t count, float* ws, hipStream_t stream) {
  const std::vector<AttnSeq> v = by_work(seqs, count, false);
  if (v.empty()) return hipSuccess;
  const int G = a.heads / a.kv_heads;
  const FwdPlan plan = fwd_plan(v, a.heads, a.kv_heads, a.d, a.window);
  for (size_t from = 0; from < plan.many.size();) {
    const AttnSeqs q = pack_seqs(plan.many, from, a.heads, q_tiles);
    from += (size_t)q.count;
    const dim3 grid((unsigned)(q.first[q.count] * a.heads));
    if (two_groups(q, a.heads, a.causal, a.window)) {
      if (a.d <= 64) hipLaunchKernelGGL((attn_fwd_kernel<64, 2>), grid, dim3(512), 0, stream, a, q);
      else hipLaunchKernelGGL((attn_fwd_kernel<128, 2>), grid, dim3(512), 0, stream, a, q);
    } else {
      if (a.d <= 64) hipLaunchKernelGGL((attn_fwd_kernel<64, 1>), grid, dim3(256), 0, stream, a, q);
      else hipLaunchKernelGGL((attn_fwd_kernel<128, 1>), grid, dim3(256), 0, stream, a, q);
    }
  }
  for (size_t from = 0; from < plan.few.size();) {
    const AttnSeqs q = few_seqs(plan, from, G, a.kv_heads, a.window);
    from += (size_t)q.count;
    AttnSplit sp{};
    sp.part = ws;
    sp.chunk = (int)plan.chunk;
    int64_t row0 = 0;
    for (int i = 0; i < q.count; ++i) {
      sp.lo[i] = (int)first_key(q.seq[i], a.window);
      sp.nsplit[i] = split_count(q.seq[i], a.window, plan.chunk);
      sp.row0[i] = row0;
      const int64_t items = sp.nsplit[i] > 1 ? (int64_t)q.seq[i].nq * a.heads : 0;
      row0 += items * sp.nsplit[i];
      sp.join_first[i + 1] = sp.join_first[i] + (int)items;
    }
    const dim3 grid((unsigned)(q.first[q.count] * a.kv_heads));
    if (a.d <= 64) hipLaunchKernelGGL(attn_split_kernel<64>, grid, dim3(256), 0, stream, a, q, sp);
    else hipLaunchKernelGGL(attn_split_kernel<128>, grid, dim3(256), 0, stream, a, q, sp);
    const int items = sp.join_first[q.count];
    if (items) hipLaunchKernelGGL(attn_join_kernel, dim3((unsigned)((items + 3) / 4)), dim3(256), 0, stream, a, q, sp);
  }
  return hipGetLastError();
}

hipError_t launch_attn_bwd(const AttnBwdArgs& args, const AttnSeq* seqs, int64_t count, int64_t q_tokens, float* ws,
                           hipStream_t stream) {
  AttnBwdArgs a = args;
  a.lse2 = ws;
  a.less_delta = ws + round64(q_tokens * a.heads);
  const std::vector<AttnSeq> vq = by_work(seqs, count, false), vk = by_work(seqs, count, true);
  for (size_t from = 0; from < vq.size();) {
    const AttnSeqs q = pack_seqs(vq, from, a.heads, q_tiles);
    from += (size_t)q.count;
    const dim3 grid((unsigned)(q.first[q.count] * a.heads));
    if (two_groups(q, a.heads, a.causal, a.window)) {
      if (a.d <= 64) hipLaunchKernelGGL((attn_dq_kernel<64, 2>), grid, dim3(512), 0, stream, a, q);
      else hipLaunchKernelGGL((attn_dq_kernel<128, 2>), grid, dim3(512), 0, stream, a, q);
    } else {
      if (a.d <= 64) hipLaunchKernelGGL((attn_dq_kernel<64, 1>), grid, dim3(256), 0, stream, a, q);
      else hipLaunchKernelGGL((attn_dq_kernel<128, 1>), grid, dim3(256), 0, stream, a, q);
    }
  }
  const KvPlan plan = kv_plan(vk, a.heads, a.kv_heads, a.d, a.causal, a.window);
  const AttnKvSplit sp{ws + 2 * round64(q_tokens * a.heads), plan.splits, plan.gper};
  for (size_t from = 0; from < vk.size();) {
    const AttnSeqs q = pack_seqs(vk, from, (int64_t)a.kv_heads * sp.splits, k_tiles);
    from += (size_t)q.count;
    const int units = q.first[q.count] * a.kv_heads;
    const dim3 grid((unsigned)(units * sp.splits)), sums((unsigned)(units * 2));
    if (a.d <= 64) {
      hipLaunchKernelGGL((attn_dkv_kernel<64, 2>), grid, dim3(256), 0, stream, a, q, sp);
      if (sp.splits > 1) hipLaunchKernelGGL(attn_dkv_sum_kernel<64>, sums, dim3(256), 0, stream, a, q, sp);
    } else {
      if (plan.waves == 1) hipLaunchKernelGGL((attn_dkv_kernel<128, 1>), grid, dim3(256), 0, stream, a, q, sp);
      else hipLaunchKernelGGL((attn_dkv_kernel<128, 2>), grid, dim3(256), 0, stream, a, q, sp);
      if (sp.splits > 1) hipLaunchKernelGGL(attn_dkv_sum_kernel<128>, sums, dim3(256), 0, stream, a, q, sp);
    }
  }
  return hipGetLastError();
}

}  // namespace nf4
