// Attention over a key/value cache in 4 bits (gfx950): as attention over the bf16 values that its blocks stand
// for (kv4.h), which exist only in registers and LDS.
//
// Scores, softmax and sums are those of attn.hip: 32 x 32 products, streamed keys as result rows and query rows as
// result columns, fp32 statistics, probabilities rounded to bf16 where they enter the second product (2^-8). The query
// heads that share a key head are packed with the tokens into rows (row = token * group + head in group), 32 rows
// a workgroup; its keys are one range of the sequence's, and its 4 waves take 32-key tiles of that range in turn.
//
// A lane holds one key of the tile and, of its row, the blocks 2 b + h (h the lane's half of the wave): 16 bytes of codes
// and a scale each, for the key and for the value. The keys' blocks, dequantised, are the first product's operand as
// they are (its contraction runs over d in that order, and the queries are loaded in the same); the values' go
// through an LDS tile of the wave's own, from which they are read across with transpose loads. The codes of the
// next tile are on their way while a tile is worked on; there are no barriers until the waves are joined.
//
// A value block that stands for NaN enters as zeros, and the same block of its key as NaN: a query that sees the
// key gets NaN through the score, and one that does not gets nothing of it (0 times NaN would be NaN).
#include "attn.h"
#include "kv4.h"

namespace nf4 {

// A lane's blocks of one tile, as they lie in the cache.
template <int NB>
struct Kv4Blocks {
  u32x4 k[NB], v[NB];
  uint32_t ka[NB], va[NB];
};

template <int DP>
struct Kv4Wave {
  static constexpr int BN = 32, KS = DP / 16, DT = DP / 32, NB = DP / 64;
  typedef Tile<DP> T;
  bf16x8 qf[KS];
  Online<DT> acc;
  Range mine, first, last;   // keys that the lane's row, the tile's first and its last row see
  float c, slack;
  int lane;

  // The tile of keys from j0; keys from `end` on repeat the last one (they are hidden), blocks past the
  // row's repeat its last (their queries are zero, and their columns of the output are not stored).
  __device__ __forceinline__ void load(Kv4Blocks<NB>& x, const AttnKv4Args& a, int64_t kbase, int64_t vbase, int j0, int end) const {
    const int key = min(lane & 31, end - 1 - j0), h = lane >> 5;
    const int64_t kt = kbase + (int64_t)j0 * a.k4.token, vt = vbase + (int64_t)j0 * a.v4.token;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint32_t at = (uint32_t)min(2 * b + h, a.nb - 1);
      const uint32_t ko = (uint32_t)key * (uint32_t)a.k4.token + at, vo = (uint32_t)key * (uint32_t)a.v4.token + at;
      x.k[b] = *reinterpret_cast<const u32x4*>(a.k4.codes + 16 * kt + 16u * ko);
      x.v[b] = *reinterpret_cast<const u32x4*>(a.v4.codes + 16 * vt + 16u * vo);
      x.ka[b] = a.k4.absmax[kt + ko];
      x.va[b] = a.v4.absmax[vt + vo];
    }
  }

  // x: the tile of keys from j0; vt: the wave's tile in LDS
  __device__ __forceinline__ void tile(const Kv4Blocks<NB>& x, const AttnKv4Args& a, uint16_t* vt, int j0) {
    f32x16 sc[1];
    sc[0] = zero16();
    const int h = lane >> 5;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const bool lost = x.va[b] >= kBf16Infinity;   // absmax has no sign
      const Kv4Table kt(a.t, kv4_step(lost ? 0x7FC0u : x.ka[b], a.unit)), vv(a.t, kv4_step(lost ? 0u : x.va[b], a.unit));
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        sc[0] = mfma(__builtin_bit_cast(bf16x8, kt.eight(x.k[b][t])), qf[4 * b + t], sc[0]);
        *reinterpret_cast<u32x4*>(vt + T::elem(lane & 31, 4 * (2 * b + h) + t)) = vv.eight(x.v[b][t]);
      }
    }
    // some row does not see some key
    if (j0 + BN > first.hi || j0 < last.lo) hide(sc[0], mine, j0, lane, -INFINITY);
    acc.update(sc, c, slack);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const bf16x8 p = pack8(sc[0], kk);
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) acc.o[dt] = mfma(T::cols(vt, 16 * kk, dt, lane), p, acc.o[dt]);
    }
  }
};

template <int DP>
__global__ __launch_bounds__(256, 2) void attn_kv4_kernel(const AttnKv4Args a, const AttnSeqs sq, const AttnSplit sp) {
  typedef Kv4Wave<DP> Wave;
  constexpr int BN = Wave::BN, DT = Wave::DT, KS = Wave::KS, P = 33;
  // the waves' tiles of values, later their outputs as [wave][d][32 rows]
  __shared__ __attribute__((aligned(16))) float lds[4 * DP * P];
  __shared__ float Ms[4][32], Ls[4][32];
  static_assert(4 * BN * DP * 2 <= (int)sizeof(lds), "the tiles fit");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int G = a.f.heads / a.f.kv_heads;
  const Unit u = unit_of((int)blockIdx.x, a.f.kv_heads, 1);
  const Found at_seq = find_seq(sq, u.tile);
  const AttnSeq s = at_seq.seq;
  const int si = at_seq.index, local = u.tile - at_seq.first;
  const int ns = sp.nsplit[si], split = local % ns, rt = local / ns;
  const int shift = s.nk - s.nq, rows = s.nq * G;
  const int row = rt * 32 + (lane & 31);
  const int tok = min(row, rows - 1) / G, head = u.kvh * G + min(row, rows - 1) % G;
  const int t0 = rt * 32 / G, t1 = min(rows - 1, rt * 32 + 31) / G;   // tokens of the row tile
  Wave w;
  w.first = visible(t0 + shift, s.nk, a.f.causal, a.f.window);
  w.last = visible(t1 + shift, s.nk, a.f.causal, a.f.window);
  w.mine = visible(tok + shift, s.nk, a.f.causal, a.f.window);
  w.lane = lane;
  // tiles are counted from the first key that the sequence's first row sees (none before it is read)
  const int lo = sp.lo[si];
  const int k_lo = lo + max((w.first.lo - lo) & ~(BN - 1), split * sp.chunk);
  const int k_hi = min(w.last.hi, lo + (split + 1) * sp.chunk);
  const int64_t kbase = s.k0 * a.k4.token + (int64_t)u.kvh * a.k4.head, vbase = s.k0 * a.v4.token + (int64_t)u.kvh * a.v4.head;
  const int j_w = k_lo + wave * BN;   // the wave's first tile; its tiles are 4 apart
  Kv4Blocks<Wave::NB> now, next;
  if (j_w < k_hi) w.load(now, a, kbase, vbase, j_w, k_hi);
  {
    const uint16_t* q = a.f.q.p + (s.q0 + tok) * a.f.q.token + (int64_t)head * a.f.q.head;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int col = 64 * (ks >> 2) + 32 * (lane >> 5) + 8 * (ks & 3);
      u32x4 v = u32x4{0u, 0u, 0u, 0u};
      if (row < rows && col < a.f.d) v = *reinterpret_cast<const u32x4*>(q + col);
      w.qf[ks] = __builtin_bit_cast(bf16x8, v);
    }
  }
  w.acc.init();
  w.c = a.f.c;
  w.slack = slack_of(a.f.c);
  uint16_t* const vt = reinterpret_cast<uint16_t*>(lds) + wave * BN * DP;
  for (int j = j_w; j < k_hi; j += 4 * BN) {
    if (j + 4 * BN < k_hi) w.load(next, a, kbase, vbase, j + 4 * BN, k_hi);
    w.tile(now, a, vt, j);
    now = next;
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
  const float mxc = mx == -INFINITY ? 0.f : mx * a.f.c;
  l = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float f = Ms[k][col] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(Ms[k][col] * a.f.c - mxc);
    l += Ls[k][col] * f;   // 0 times NaN stays NaN
  }
  const float f = acc.m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(acc.mc - mxc);
  float* const buf = lds + wave * (DP * P);
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
  float* const part = sp.part + (sp.row0[si] + ((int64_t)grow * a.f.kv_heads + u.kvh) * ns + split) * (int64_t)(a.f.d + 8);
#pragma unroll
  for (int k = 0; k < DP / 64; ++k) {
    const int c0 = 8 * (tid & 7) + 64 * k;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = 0.f;
#pragma unroll
      for (int k2 = 0; k2 < 4; ++k2) v[e] += lds[k2 * (DP * P) + (c0 + e) * P + orow];
    }
    if (c0 >= a.f.d) continue;
    if (ns == 1) {
      const float inv = inverse_sum(rl);
      u32x4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = pack_bf16x2(v[2 * e] * inv, v[2 * e + 1] * inv);
      *reinterpret_cast<u32x4*>(a.f.o.p + (s.q0 + otok) * a.f.o.token + (int64_t)ohead * a.f.o.head + c0) = o;
    } else {
      *reinterpret_cast<f32x4*>(part + c0) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(part + c0 + 4) = f32x4{v[4], v[5], v[6], v[7]};
    }
  }
  if ((tid & 7) == 0) {
    if (ns == 1) {
      if (a.f.lse) a.f.lse[(int64_t)ohead * a.f.lse_stride + s.q0 + otok] = lse_of(rm, rl);
    } else {
      part[a.f.d] = rl == 0.f ? -INFINITY : rm;   // finite (0 at least) where the sum is NaN: the join reads it
      part[a.f.d + 1] = rl;
    }
  }
}

// ------------------------------------------------------------------------------------------
// Host side: ranges of keys, launches
static int64_t kv4_row_tiles(const AttnSeq& s, int G) { return ceil64((int64_t)s.nq * G, 32); }
static int kv4_ranges(const AttnSeq& s, int window, int64_t chunk) {
  return (int)std::max<int64_t>(1, ceil64(s.nk - first_key(s, window), chunk));
}

// Keys per range, one length for all sequences of a launch: the smallest sum of rounds of workgroups (two on a
// compute unit) times a range and a fixed part, and of the launch that joins ranges.
static int64_t kv4_chunk(const std::vector<AttnSeq>& v, int G, int kv_heads, int d, int window) {
  const double key = 0.011 * padded_d(d) / 128.0;
  int64_t longest = 1, best = 0;
  double best_cost = -1;
  for (const AttnSeq& s : v) longest = std::max(longest, s.nk - first_key(s, window));
  for (int64_t chunk = 128;; chunk += std::max<int64_t>(128, chunk / 8 / 128 * 128)) {
    int64_t wgs = 0, most = 0;
    for (const AttnSeq& s : v) {
      const int64_t n = kv4_row_tiles(s, G) * kv4_ranges(s, window, chunk) * kv_heads;
      wgs += n;
      most = std::max(most, n);
    }
    if (most > kAttnGroups && chunk < longest) continue;   // a sequence has to fit a launch
    const double cost = ceil64(wgs, 512) * (5 + key * std::min(chunk, longest)) + (chunk < longest ? 4 : 0);
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      best = chunk;
    }
    if (chunk >= longest) return best;
  }
}

static AttnSeqs kv4_seqs(const std::vector<AttnSeq>& v, size_t from, int G, int kv_heads, int window, int64_t chunk) {
  return pack_seqs(v, from, kv_heads, [&](const AttnSeq& s) { return kv4_row_tiles(s, G) * kv4_ranges(s, window, chunk); });
}

size_t attn_kv4_ws_floats(const AttnSeq* seqs, int64_t count, int heads, int kv_heads, int d, int window) {
  const std::vector<AttnSeq> v = by_work(seqs, count, false);
  if (v.empty()) return 0;
  const int G = heads / kv_heads;
  const int64_t chunk = kv4_chunk(v, G, kv_heads, d, window);
  int64_t most = 0;
  for (size_t from = 0; from < v.size();) {
    const AttnSeqs q = kv4_seqs(v, from, G, kv_heads, window, chunk);
    int64_t f = 0;
    for (int i = 0; i < q.count; ++i) {
      const int ns = kv4_ranges(q.seq[i], window, chunk);
      if (ns > 1) f += (int64_t)q.seq[i].nq * heads * ns * (d + 8);
    }
    most = std::max(most, f);
    from += (size_t)q.count;
  }
  return (size_t)most;
}

hipError_t launch_attn_kv4(const AttnKv4Args& a, int book, const AttnSeq* seqs, int64_t count, float* ws, hipStream_t stream) {
  const std::vector<AttnSeq> v = by_work(seqs, count, false);
  if (v.empty()) return hipSuccess;
  const int G = a.f.heads / a.f.kv_heads;
  const int64_t chunk = kv4_chunk(v, G, a.f.kv_heads, a.f.d, a.f.window);
  for (size_t from = 0; from < v.size();) {
    const AttnSeqs q = kv4_seqs(v, from, G, a.f.kv_heads, a.f.window, chunk);
    from += (size_t)q.count;
    AttnSplit sp{};
    sp.part = ws;
    sp.chunk = (int)chunk;
    int64_t row0 = 0;
    for (int i = 0; i < q.count; ++i) {
      sp.lo[i] = (int)first_key(q.seq[i], a.f.window);
      sp.nsplit[i] = kv4_ranges(q.seq[i], a.f.window, chunk);
      sp.row0[i] = row0;
      const int64_t items = sp.nsplit[i] > 1 ? (int64_t)q.seq[i].nq * a.f.heads : 0;
      row0 += items * sp.nsplit[i];
      sp.join_first[i + 1] = sp.join_first[i] + (int)items;
    }
    const dim3 grid((unsigned)(q.first[q.count] * a.f.kv_heads));
    if (a.f.d <= 64) hipLaunchKernelGGL(attn_kv4_kernel<64>, grid, dim3(256), 0, stream, a, q, sp);
    else hipLaunchKernelGGL(attn_kv4_kernel<128>, grid, dim3(256), 0, stream, a, q, sp);
    launch_attn_join(a.f, q, sp, stream);
  }
  return hipGetLastError();
}

}  // namespace nf4
