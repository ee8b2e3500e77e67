// Attention of ragged chunks of new tokens over the paged cache on the
// 5th-generation tensor cores (what it computes: chunk_common.cuh).
//
// One CTA per SM stays and works through units: a row tile of one (sequence, KV
// head), up to 256 rows, a row being a new token and one of the KV head's query
// heads, over one split of the tile's visible keys, in key tiles of 128 (64
// where EARLY needs the columns).  A CTA starts with the unit of its own block
// index and then takes those of blocks that have not started (cluster launch
// control), so that unequal units even out, and loads and products of a unit
// begin under the softmax and the output of the one before.  The rows are two
// groups of 128 TMEM lanes, which share every K and V tile.  Roles:
//   0-7   softmax and output: thread t of group g is row 128 g + t
//   8, 11 issue the products of group 0 and of group 1:
//         S_g(k) = Q_g K(k)^T and O_g += P_g(k) V(k)
//   9     takes the units and loads K, 10 loads V and Q: TMA, a lane per box (a
//         block's rows of one 128-byte column half), K and V alternately in one
//         ring of 128 KB (E4M3 caches: 96 KB, and 48 KB for the codes)
//   12-15 (E4M3 and E2M1 caches) widen the codes to f16 tiles of the ring (E2M1:
//         times their groups' scales, which is exact), and Q to f16
// TMEM: S of both groups and O of both, 512 columns for 128-wide heads, so that
// P_g(k), 16-bit pairs, takes the first half of S_g's columns once the softmax
// has read them, and S_g(k+1) is issued behind PV_g(k), which reads P from its
// columns: one group's softmax runs under the other group's products, and
// S_g(k) having completed (sfull) means that PV_g(k-1) has, so the softmax may
// rescale O_g without a barrier of its own.  EARLY (capped or biased scores of
// bf16 caches, whose softmax is the longer part): P has columns of its own and
// S(k+1) is issued as soon as the softmax has read S(k); for plain scores it
// costs (128-wide heads 1175 us where the other takes 1015, 64-wide 175 / 164).
//
// A whole warp walks an issuing role and an elected lane's predicate issues the
// products: a branch on the lane costs 115 cycles per product.
//
// The running maximum is lazy: O is rescaled only when the maximum grows by
// more than 2^8, so P stays within 2^8 (f16 holds that) and most tiles rescale
// nothing.  Sums, maxima and O are binary32; P is rounded to 16 bits (bf16
// 2^-8, f16 2^-11 of a weight), next to the output's own 2^-8.
//
// Bound: 4 D flops per row and visible key on the tensor pipe, with the
// softmax's exponentials (8 a cycle and sub-partition) at half its time.  Two
// chunks of 4096 tokens over 4096, 64 + 8 heads of 128, bf16: 1010-1080 us
// with the clock (1.93 GHz under the power cap), 1530-1630 Tflop/s, 78-83 % of
// the measured library product; the tensor pipe is active 70 % of the time,
// the rest is the first and last tile of a unit and the softmax's two warps per
// sub-partition waiting for each other's issue slots.  Steps that did not pay:
// 16 softmax warps, half a row each (1410-1540 us: they spill); P handed over
// in halves (12 % slower) and S as two products of 64 keys (24 %); three ring
// slots instead of four (1290); 128 bytes of a row per output pass (1045).
// E4M3 caches: chunks of 512 tokens over 3584 take 616 us where bf16 takes 513:
// the softmax has 200 registers a thread instead of 224 (bf16 with 192: 570 us
// where it then took 521), and the widening is worth 30 us (586 with none); S from
// the codes themselves, with Q as two E4M3 planes, has half the widening but was
// no faster (633 us).
//
// Every wait is bounded; a time-out records the error and raises the CTA's abort
// flag, which ends every role's loop.  Each product issuer leaves after its
// products.  Once every role has left, so that nothing is issued any more, an
// aborted CTA waits (bounded again) for the last copy on every barrier, K, V, Q
// and the launch control's answer, before its shared memory goes to another CTA.

#pragma once

#include <type_traits>

#include "chunk_common.cuh"
#include "pkv_tc.cuh"

namespace pkv {
namespace {

// What a score is besides scale * q.k: nothing; capped; biased; both.
constexpr int kPlain = 0, kCapped = 1, kBiased = 2, kCappedBiased = 3;
constexpr int kFar = 4;  // added to the capped ones: a cap above kCapNear

// KV: type of the caches (kBF16KV, kE4M3, kE2M1).  WIDE: their tiles are widened
// to f16 before the products.
constexpr int kBF16KV = 0;

template <int D, int KV, int MODE>
struct TcShape {
  static constexpr bool WIDE = KV != kBF16KV;
  static constexpr int M = 128, GROUPS = 2, ROWS = M * GROUPS;
  // EARLY: P has TMEM columns of its own, so that S(k+1) is issued as soon as the
  // softmax has read S(k).  They are there for 64-wide heads; 128-wide ones need
  // 64-key tiles for it.
  static constexpr bool EARLY = chunk_tc_early(WIDE, MODE != kPlain);
  static constexpr int NK = chunk_tc_tile(D, WIDE, MODE != kPlain);
  static constexpr int HALVES = D / 64;            // 128-byte column halves of a 16-bit row
  static constexpr int QHALF = ROWS * 128;
  static constexpr int QBYTES = HALVES * QHALF;
  static constexpr int HALFB = NK * 128;
  static constexpr int TILE = HALVES * HALFB;      // a 16-bit K or V tile
  // a K or V tile as it lies in the cache; E2M1: rows of codes, then a kilobyte
  // for the rows of scales, whose boxes of 64 bytes or more start at multiples of 128
  static constexpr int RAWROW = KV == kE2M1 ? D / 2 : D;
  static constexpr int CODES = NK * RAWROW;
  static constexpr int RAW = CODES + (KV == kE2M1 ? 1024 : 0);
  static constexpr int NS = WIDE ? (D == 128 ? 3 : 6) : 131072 / TILE;
  static constexpr int NR = WIDE ? (D == 128 ? (KV == kE2M1 ? 4 : 3) : 6) : 0;
  static constexpr int SB = 64;                    // output staging of a softmax warp: SB bytes of its 32 rows
  static constexpr int STAGE = 32 * SB;
  static constexpr int RU = 4;                     // units in flight between the roles
  static constexpr int UNIT = 20;                  // words of one
  static constexpr int NBARS = 2 * NS + 2 * NR + 5 * GROUPS + 6 + 2 * RU + GROUPS;
  static constexpr int BYTES = QBYTES + NS * TILE + NR * RAW + 8 * STAGE + 16 + NBARS * 8 + RU * UNIT * 4 + 32 + 1024;
  static_assert(BYTES <= 232448, "shared memory per CTA");
  static constexpr int THREADS = WIDE ? 512 : 384;
  // registers: 384 x 168 or 512 x 128 at launch.  The softmax wants all it can
  // get (a row's 128 scores; bf16 caches at 192 instead of 224: 570 us where it
  // takes 521); with E4M3 caches 200 / 56 spill least for plain scores of
  // 128-wide heads (614 us, 192 / 64: 617), 192 / 64 for all others (capped 862
  // us, 200 / 56: 880); E2M1's widening has more to hold (12 chunks of 1-512: 200 /
  // 56 264 us, 192 / 64 259, 184 / 72 261, 176 / 80 268)
  static constexpr int REGS_SOFTMAX = !WIDE ? 224 : (D == 128 && MODE == kPlain && KV == kE4M3 ? 200 : 192);
  static constexpr int REGS_OTHER = WIDE && REGS_SOFTMAX == 192 ? 64 : 56;
  static_assert(256 * REGS_SOFTMAX + (THREADS - 256) * REGS_OTHER <= THREADS * (WIDE ? 128 : 168), "register file");
};

// One work unit as the roles read it from shared memory.
struct TcUnit {
  int b;            // sequence, -1: no unit is left
  int h;            // KV head
  int row0;         // first query token (row of q and out)
  int rows;         // rows of the tile: tokens x group
  int pos0;         // position of the first token
  int ctx, prefix, lo, hi, na, b0;
  int k0, ntile;    // tiles [k0, k0 + ntile) of the row tile's visible ones
  int split, nsplit;
  int k_bits, v_bits;  // scales of the sequence's head (binary32 words)
  __device__ __forceinline__ int tile(int k) const { return k0 + k < na ? k0 + k : b0 + (k0 + k - na); }
  __device__ __forceinline__ bool sees(int t0, int t1) const { return t0 < prefix || (t0 < hi && t1 > lo); }
  // rows of V's last tile past the sequence's end that share a block with its last token
  __device__ __forceinline__ int tail_first(int nk) const { return ctx - tile(ntile - 1) * nk; }
  __device__ __forceinline__ bool v_tail(int nk, int block_size) const {
    return ntile > 0 && tail_first(nk) < nk && tail_first(nk) % block_size != 0;
  }
};

// x := cap * tanh(x / cap) in log2 units for any x: a polynomial up to 0.35 of
// the cap, else 1 - 2 / (e^2y + 1), one reciprocal shared by four scores,
// 1 / a = b c d / (a b c d); 2y is held below 28 log2 units, where tanh is 1 to
// binary32 and the product of four cannot overflow.  What lies past the
// sequence's end may be NaN and must not reach its neighbours: scores that are
// not seen enter as 0.
template <int N, bool FAR>
__device__ __forceinline__ void cap_scores(float* x, float w_mult, float cap_log2, const CapPoly<FAR>& poly, bool masked,
                                           const uint32_t* see) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    float q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float v = masked && !((see[(i + j) / 32] >> ((i + j) % 32)) & 1u) ? 0.f : x[i + j];
      q[j] = fast_exp2(min_nan(v * w_mult, 28.f)) + 1.f;
    }
    const float2 pr = __fmul2_rn(make_float2(q[0], q[2]), make_float2(q[1], q[3]));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(pr.x * pr.y));
    const float2 rp = __fmul2_rn(make_float2(r, r), make_float2(pr.y, pr.x));  // 1 / (q0 q1), 1 / (q2 q3)
    const float2 m2c = make_float2(-2.f * cap_log2, -2.f * cap_log2), c = make_float2(cap_log2, cap_log2);
    const float2 a = __ffma2_rn(__fmul2_rn(make_float2(rp.x, rp.x), make_float2(q[1], q[0])), m2c, c);
    const float2 b = __ffma2_rn(__fmul2_rn(make_float2(rp.y, rp.y), make_float2(q[3], q[2])), m2c, c);
    const float z[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (FAR)
        x[i + j] = poly.far_holds(x[i + j]) ? poly.far(x[i + j], cap_log2) : z[j];
      else
        x[i + j] = poly.holds(fabsf(x[i + j])) ? poly.of(x[i + j]) : z[j];
    }
  }
}

// tanh(y) for |y| <= kMidLimit (kMidC0 ...).  Ten packed FMA-pipe operations for two
// weights' exponents, where the exponential form takes 2.25 special-function and
// about 15 other operations for each: E2M1 caches, whose scores the groups' largest
// channels bring past 0.35 of a cap, 3 chunks of 2000 over 1000 of 128-wide heads
// with cap 30 1383 -> 730 us.
__device__ __forceinline__ float2 mid_tanh(float2 x, float y_mult) {
  const float2 u = __fmul2_rn(x, make_float2(y_mult, y_mult)), t = __fmul2_rn(u, u);
  float2 q = make_float2(kMidC6, kMidC6);
  q = __ffma2_rn(q, t, make_float2(kMidC5, kMidC5));
  q = __ffma2_rn(q, t, make_float2(kMidC4, kMidC4));
  q = __ffma2_rn(q, t, make_float2(kMidC3, kMidC3));
  q = __ffma2_rn(q, t, make_float2(kMidC2, kMidC2));
  q = __ffma2_rn(q, t, make_float2(kMidC1, kMidC1));
  q = __ffma2_rn(q, t, make_float2(kMidC0, kMidC0));
  return __fmul2_rn(u, q);
}

// Largest of N magnitudes.
template <int N>
__device__ __forceinline__ float abs_max(const float* x) {
  float am[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < N; i += 8)
#pragma unroll
    for (int j = 0; j < 4; ++j) am[j] = max3f(am[j], fabsf(x[i + 2 * j]), fabsf(x[i + 2 * j + 1]));
  return fmaxf(max3f(am[0], am[1], am[2]), am[3]);
}

// Largest of N scores.
template <int N>
__device__ __forceinline__ float row_max(const float* x) {
  float mp[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    mp[j] = max3f(x[j], x[8 + j], x[16 + j]);
#pragma unroll
    for (int i = 24; i + 8 < N; i += 16) mp[j] = max3f(mp[j], x[i + j], x[i + 8 + j]);
    mp[j] = fmaxf(mp[j], x[N - 8 + j]);
  }
  return max3f(max3f(mp[0], mp[1], mp[2]), max3f(mp[3], mp[4], mp[5]), fmaxf(mp[6], mp[7]));
}

// x := -inf where the key is not seen; words that every lane sees whole are
// passed over.
template <int N>
__device__ __forceinline__ void mask_scores(float* x, const uint32_t* see) {
#pragma unroll
  for (int w = 0; w < N / 32; ++w)
    if (!__all_sync(kFull, see[w] == 0xFFFFFFFFu)) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (!((see[w] >> i) & 1u)) x[32 * w + i] = -CUDART_INF_F;
    }
}

// The unit that block index (x, y) stands for; false if it stands for none (a
// tile number no sequence uses, a split past the tile's keys).  A whole warp.
template <int NK, int KV>
__device__ __forceinline__ bool tc_unit(const ChunkParams& p, int x, int y, TcUnit& u) {
  u.h = x % p.num_kv_heads;
  const int t = x / p.num_kv_heads;
  ChunkSeq sq;
  int tile;
  if (p.batch <= 32) {
    // a lane per sequence: the sequences whose last tokens see most keys first
    // (equal ones in order), so that no long unit is left for the end (12 chunks
    // of 1-512 tokens over 0-3584: 250 us, in the order given 272); the tiles
    // before a sequence's are those of the sequences ahead of it.  More than a
    // warp's lanes come in the order they are given: 33 of 1-128 tokens 129 us
    // if that is longest first and 152-158 if not, 64 246 and 257-270; of 1-512
    // tokens less than 1 %.
    const int lane = threadIdx.x & 31;
    const ChunkSeq mine = chunk_seq(p, lane < p.batch ? lane : 0, lane < p.batch && y == 0 && u.h == 0);
    const int nt = lane < p.batch ? (mine.n + p.tile_q - 1) / p.tile_q : 0;
    const int most = nt > 0 ? chunk_range<NK>(p, mine, (nt - 1) * p.tile_q, mine.n - 1).n : 0;
    int base = 0;
#pragma unroll 1
    for (int j = 0; j < p.batch; ++j) {
      const int ahead = __shfl_sync(kFull, most, j), tiles = __shfl_sync(kFull, nt, j);
      if (ahead > most || (ahead == most && j < lane)) base += tiles;
    }
    const unsigned hit = __ballot_sync(kFull, t >= base && t - base < nt);
    if (hit == 0u) return false;
    u.b = __ffs(hit) - 1;
    sq.start = __shfl_sync(kFull, mine.start, u.b);
    sq.n = __shfl_sync(kFull, mine.n, u.b);
    sq.ctx = __shfl_sync(kFull, mine.ctx, u.b);
    sq.prefix = __shfl_sync(kFull, mine.prefix, u.b);
    tile = __shfl_sync(kFull, nt - 1 - (t - base), u.b);
  } else {
    u.b = warp_search(p.batch, t, [&](int i) { return chunk_tile_base(p, i); });
    sq = chunk_seq(p, u.b, (threadIdx.x & 31) == 0 && y == 0 && u.h == 0);
    const int ntq = (sq.n + p.tile_q - 1) / p.tile_q;
    tile = ntq - 1 - (t - chunk_tile_base(p, u.b));
    if (tile < 0 || tile >= ntq) return false;
  }
  // longest first within a sequence: its last tokens see the most keys
  const int i0 = tile * p.tile_q, i1 = min(sq.n, i0 + p.tile_q) - 1;
  const ChunkRange rg = chunk_range<NK>(p, sq, i0, i1);
  const ChunkSplit sp(rg.n, p.split_tokens / NK, y);
  u.nsplit = sp.nsplit;
  u.split = y;
  if (u.split >= u.nsplit) return false;
  u.row0 = sq.start + i0;
  u.rows = (i1 - i0 + 1) * p.group;
  u.pos0 = sq.ctx - sq.n + i0;
  u.ctx = sq.ctx;
  u.prefix = rg.prefix;
  u.lo = rg.lo;
  u.hi = rg.hi;
  u.na = rg.na;
  u.b0 = rg.b0;
  u.k0 = sp.k0;
  u.ntile = sp.ntile;
  u.k_bits = u.v_bits = __float_as_int(1.f);
  if (KV == kE4M3 || (KV == kE2M1 && p.k_scale != nullptr)) {
    u.k_bits = __float_as_int(p.k_scale[static_cast<int64_t>(u.b) * p.scale_stride + u.h]);
    u.v_bits = __float_as_int(p.v_scale[static_cast<int64_t>(u.b) * p.scale_stride + u.h]);
  }
  return true;
}

// Row t of an E4M3 tile (16 codes of a 16-byte chunk, swizzled as the TMA unit
// stores 128- and 64-byte rows) as f16 in the ring's tile: half hf of the row
// hf * half_bytes on, its 16-byte chunks swizzled.
template <int D>
__device__ __forceinline__ void widen_e4m3(const uint8_t* src, uint8_t* dst, int half_bytes, int t, bool live) {
  constexpr int CH = D / 16;                     // 16-byte chunks of a raw row
  const uint32_t rsw = D == 128 ? (t & 7) : ((t >> 1) & 3);
#pragma unroll
  for (int c0 = 0; c0 < CH; c0 += 4) {
    uint4 w[4];                                  // four loads before the first store
#pragma unroll
    for (int c = 0; c < 4; ++c) w[c] = *reinterpret_cast<const uint4*>(src + (((c0 + c) ^ rsw) << 4));
    if (!live) {
#pragma unroll
      for (int c = 0; c < 4; ++c) w[c] = make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint4 a, e;
      a.x = e4m3x2_to_f16x2(static_cast<uint16_t>(w[c].x & 0xFFFFu));
      a.y = e4m3x2_to_f16x2(static_cast<uint16_t>(w[c].x >> 16));
      a.z = e4m3x2_to_f16x2(static_cast<uint16_t>(w[c].y & 0xFFFFu));
      a.w = e4m3x2_to_f16x2(static_cast<uint16_t>(w[c].y >> 16));
      e.x = e4m3x2_to_f16x2(static_cast<uint16_t>(w[c].z & 0xFFFFu));
      e.y = e4m3x2_to_f16x2(static_cast<uint16_t>(w[c].z >> 16));
      e.z = e4m3x2_to_f16x2(static_cast<uint16_t>(w[c].w & 0xFFFFu));
      e.w = e4m3x2_to_f16x2(static_cast<uint16_t>(w[c].w >> 16));
      uint8_t* to = dst + (c0 / 4) * half_bytes;
      *reinterpret_cast<uint4*>(to + (((2 * c) ^ (t & 7)) << 4)) = a;
      *reinterpret_cast<uint4*>(to + (((2 * c + 1) ^ (t & 7)) << 4)) = e;
    }
  }
}

// The same of an E2M1 tile: 32 codes of a 16-byte chunk (64- and 32-byte rows)
// times the scales of their two groups, which is exact in f16.
template <int D>
__device__ __forceinline__ void widen_e2m1(const uint8_t* tile, uint8_t* dst, int half_bytes, int t, int block_size,
                                           bool live) {
  constexpr int CH = D / 32;                     // 16-byte chunks of a raw row
  const uint32_t rsw = D == 128 ? ((t >> 1) & 3) : ((t >> 2) & 1);
  const uint8_t* src = tile + t * (D / 2);
  const int per_box = block_size * (D / 16);
  const uint8_t* sc = tile + 128 * (D / 2) + (t / block_size) * (per_box < 128 ? 128 : per_box) +
                      (t % block_size) * (D / 16);
  uint4 w[CH];
  uint32_t g[D / 64];                            // four scale codes each
#pragma unroll
  for (int c = 0; c < CH; ++c) w[c] = *reinterpret_cast<const uint4*>(src + ((c ^ rsw) << 4));
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    g[i] = reinterpret_cast<const uint32_t*>(sc)[i];
    if (!live) g[i] = 0u;                        // codes are finite whatever they are: zeros
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const uint32_t q[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
    // chunk c's groups have scales 2 c and 2 c + 1
    const uint32_t s0 = e4m3x2_to_f16x2(static_cast<uint16_t>(prmt(g[c / 2], 0u, c % 2 ? 0x4422u : 0x4400u) & 0xFFFFu));
    const uint32_t s1 = e4m3x2_to_f16x2(static_cast<uint16_t>(prmt(g[c / 2], 0u, c % 2 ? 0x4433u : 0x4411u) & 0xFFFFu));
    uint8_t* to = dst + (c / 2) * half_bytes;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h[4];
      e2m1x8_to_f16x2(q[i], h);
      const uint32_t s = i < 2 ? s0 : s1;
      *reinterpret_cast<uint4*>(to + (((4 * (c % 2) + i) ^ (t & 7)) << 4)) =
          make_uint4(mul_f16x2(h[0], s), mul_f16x2(h[1], s), mul_f16x2(h[2], s), mul_f16x2(h[3], s));
    }
  }
}

// Tensor maps of the caches' rows of scales (E2M1; nothing for other caches).
template <int KV>
struct ScaleMaps {};
template <>
struct ScaleMaps<kE2M1> {
  CUtensorMap k, v;
};

template <int D, int KV, int MODE>
__global__ void __launch_bounds__(TcShape<D, KV, MODE>::THREADS, 1)
    chunk_tc_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                    const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ ScaleMaps<KV> tmap_s,
                    const ChunkParams p) {
  using C = TcShape<D, KV, MODE>;
  constexpr bool WIDE = C::WIDE;
  constexpr int M = C::M, NK = C::NK, NS = C::NS, NR = C::NR, GROUPS = C::GROUPS, RU = C::RU;
  constexpr bool EARLY = C::EARLY, FAR = (MODE & kFar) != 0;
  constexpr int SCORE = MODE & ~kFar;
  constexpr bool MID = KV == kE2M1 && !FAR;  // scores past the small ones' polynomial, up to kMidLimit caps
  constexpr bool PARTS = MID && SCORE == kCapped;
  static_assert(!(PARTS && EARLY), "scores in parts are read from S until the last P is written: S(k+1) may not come first");
  // + g * NK, + g * (EARLY ? NK / 2 : NK), + g * D
  constexpr uint32_t COL_S = 0, COL_P = EARLY ? GROUPS * NK : COL_S, COL_O = COL_P + GROUPS * (EARLY ? NK / 2 : NK);
  constexpr uint32_t P_STEP = EARLY ? NK / 2 : NK;
  constexpr uint32_t IDESC_S = WIDE ? idesc_f16(M, NK, false) : idesc_bf16(M, NK, false);
  constexpr uint32_t IDESC_PV = WIDE ? idesc_f16(M, D, true) : idesc_bf16(M, D, true);
  constexpr int kMma = 8, kLoadK = 9, kLoadV = 10, kMma1 = 11, kConv = 12;
  constexpr int READERS = 8 + 2 + 1 + (WIDE ? 4 : 0);  // warps that read a unit
  static_assert(COL_O + GROUPS * D <= 512, "TMEM columns");
  static_assert(sizeof(TcUnit) <= C::UNIT * 4, "unit slot");

  // the warp number as a broadcast: roles branch uniformly
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kFull, tid >> 5, 0);
  const int G = p.group, H_q = p.num_q_heads;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* q_sm = smem;                              // half hf, row r at hf * QHALF + r * 128
  uint8_t* ring = smem + C::QBYTES;                  // 16-bit K and V tiles, alternately
  uint8_t* raw = ring + NS * C::TILE;                // E4M3 K and V tiles, alternately
  uint8_t* s_stage = raw + NR * C::RAW;
  uint8_t* s_clc = s_stage + 8 * C::STAGE;           // 16 bytes
  uint64_t* full = reinterpret_cast<uint64_t*>(s_clc + 16);
  uint64_t* empty = full + NS;
  uint64_t* rfull = empty + NS;
  uint64_t* rempty = rfull + NR;
  uint64_t* sfull = rempty + NR;     // [GROUPS]: S_g of the next tile is in TMEM
  uint64_t* pfull = sfull + GROUPS;  // [GROUPS]: P_g is in TMEM
  uint64_t* sfree = pfull + GROUPS;  // [GROUPS]: the softmax has read S_g (EARLY)
  uint64_t* pfree = sfree + GROUPS;  // [GROUPS]: P_g's product has completed (EARLY)
  uint64_t* odone = pfree + GROUPS;  // [GROUPS]: O_g of the unit is complete
  uint64_t* qfull = odone + GROUPS;  // Q of the unit is in shared memory
  uint64_t* qready = qfull + 1;      // ... as f16 (E4M3 caches)
  uint64_t* qempty = qready + 1;     // every S of the unit has read it
  // [2]: the last V tile's rows past the end are zeros, of alternate units: the
  // loader may be one unit ahead of a product issuer that has yet to ask, and
  // two phases of one barrier cannot be told apart
  uint64_t* vfix = qempty + 1;
  uint64_t* clc = vfix + 2;          // the next unit's block index has arrived
  uint64_t* ufull = clc + 1;         // [RU]
  uint64_t* uempty = ufull + RU;     // [RU]
  uint64_t* done = uempty + RU;      // [GROUPS]
  uint32_t* s_unit = reinterpret_cast<uint32_t*>(done + GROUPS);
  uint32_t* s_tmem = s_unit + RU * C::UNIT;
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  int* s_issued = reinterpret_cast<int*>(s_tmem + 2);  // [4]: next K item, next V item, answers asked for, Qs loaded

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(smem_u32(full + s), WIDE ? 4 : 1);
      mbar_init(smem_u32(empty + s), GROUPS);
    }
    for (int s = 0; s < NR; ++s) {
      mbar_init(smem_u32(rfull + s), 1);
      mbar_init(smem_u32(rempty + s), 4);
    }
    for (int g = 0; g < GROUPS; ++g) {
      mbar_init(smem_u32(sfull + g), 1);
      mbar_init(smem_u32(pfull + g), 4);
      mbar_init(smem_u32(sfree + g), 4);
      mbar_init(smem_u32(pfree + g), 1);
      mbar_init(smem_u32(odone + g), 1);
      mbar_init(smem_u32(done + g), 1);
    }
    mbar_init(smem_u32(qfull), 1);
    mbar_init(smem_u32(qready), 4);
    mbar_init(smem_u32(qempty), GROUPS);
    mbar_init(smem_u32(vfix), 1);
    mbar_init(smem_u32(vfix + 1), 1);
    mbar_init(smem_u32(clc), 1);
    for (int i = 0; i < RU; ++i) {
      mbar_init(smem_u32(ufull + i), 1);
      mbar_init(smem_u32(uempty + i), READERS);
    }
    *s_abort = 0;
    fence_mbar_init();
    prefetch_tmap(&tmap_q);
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(s_tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = __shfl_sync(kFull, *s_tmem, 0);
  wait_prior_grid();

  auto wait = [&](uint64_t* bar, int phase) {  // a whole warp
    return __all_sync(kFull, wait_or_abort(smem_u32(bar), static_cast<uint32_t>(phase & 1), p.err, s_abort)) != 0;
  };
  // Unit number n of this CTA; false when none is left (or the CTA aborts).  A
  // whole warp; every value is the same in all its lanes.
  auto read_unit = [&](int n, TcUnit& u) {
    const int slot = n % RU;
    if (!wait(ufull + slot, n / RU)) return false;
    constexpr int W = sizeof(TcUnit) / 4;
    const uint32_t w = lane < W ? s_unit[slot * C::UNIT + lane] : 0u;
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(uempty + slot));
    uint32_t* to = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
    for (int i = 0; i < W; ++i) to[i] = __shfl_sync(kFull, w, i);
    return u.b >= 0;
  };

  if (warp >= kMma) {
    regs_dec<C::REGS_OTHER>();
    if (warp == kMma || warp == kMma1) {
      // ------------------------------------------------------------ products
      // The whole warp walks this role, one lane's products are issued: see
      // tc_mma_ss_if.
      const int g = warp == kMma ? 0 : 1;
      const uint32_t leader = elect_one();
      const uint32_t ring0 = __shfl_sync(kFull, smem_u32(ring), 0), q0 = __shfl_sync(kFull, smem_u32(q_sm), 0);
      const uint32_t c_s = tbase + COL_S + g * NK, c_p = tbase + COL_P + g * P_STEP, c_o = tbase + COL_O + g * D;
      const uint64_t a0 = smem_desc_sw128(q0 + g * M * 128, 0, 1024);
      int slot = 0, use = 0;  // ring slot of the next item, and its use number
      int pk = 0, tails = 0;  // this group's tiles so far; units with a zeroed tail so far
      bool ok = true;
      auto next_slot = [&]() {
        if (++slot == NS) {
          slot = 0;
          ++use;
        }
      };
      auto issue_s = [&]() {  // S of the K tile in `slot`, which then goes back to its loader
        const uint64_t b0 = smem_desc_sw128(ring0 + slot * C::TILE, 0, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)  // descriptor addresses are in 16-byte units
          tc_mma_ss_if(leader, c_s, a0 + ((kk / 4) * C::QHALF + (kk % 4) * 32) / 16,
                       b0 + ((kk / 4) * C::HALFB + (kk % 4) * 32) / 16, IDESC_S, kk > 0 ? 1u : 0u);
        tc_commit_if(leader, smem_u32(sfull + g));
        tc_commit_if(leader, smem_u32(empty + slot));
        next_slot();
      };
      auto fixed = [&]() {
        const int i = tails++;
        return wait(vfix + (i & 1), i >> 1);
      };
      TcUnit u;
      for (int n = 0; ok && read_unit(n, u); ++n) {
        const bool tail = !WIDE && u.v_tail(NK, p.block_size);
        if (g * M >= u.rows) {
          // no rows of this group: its arrivals keep the ring's phases
          ok = wait(WIDE ? qready : qfull, n);
          tc_commit_if(leader, smem_u32(qempty));
          for (int i = 0; i < 2 * u.ntile && ok; ++i) {
            ok = wait(full + slot, use);
            tc_commit_if(leader, smem_u32(empty + slot));
            next_slot();
          }
          if (tail && ok) ok = fixed();
          continue;
        }
        ok = wait(WIDE ? qready : qfull, n);
        if (ok && u.ntile > 0) {
          ok = wait(full + slot, use);
          if (EARLY && ok && pk > 0) ok = wait(sfree + g, pk - 1);
          if (!ok) break;
          tc_fence_after();
          issue_s();
        }
        if (u.ntile <= 1) tc_commit_if(leader, smem_u32(qempty));
        for (int k = 0; k < u.ntile && ok; ++k, ++pk) {
          const int vslot = slot, vuse = use;
          next_slot();
          const bool more = k + 1 < u.ntile;
          if (EARLY && more) {  // S(k+1), once the softmax has read S(k)
            ok = wait(full + slot, use) && wait(sfree + g, pk);
            if (!ok) break;
            tc_fence_after();
            issue_s();
            if (k + 2 == u.ntile) tc_commit_if(leader, smem_u32(qempty));  // the unit's last S
          }
          ok = wait(full + vslot, vuse);
          if (!ok) break;
          if (tail && k == u.ntile - 1) {  // its loader has zeroed the rows past the sequence's end
            ok = fixed();
            if (!ok) break;
          }
          if (!EARLY && more) ok = wait(full + slot, use);  // K(k+1), ahead of the wait for P
          const uint64_t v0 = smem_desc_sw128(ring0 + vslot * C::TILE, C::HALVES > 1 ? C::HALFB : 0, 1024);
          ok = ok && wait(pfull + g, pk);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < NK / 16; ++kk)  // MN-major V: 8-key groups 1024 B apart, column halves HALFB apart
            tc_mma_ts_if(leader, c_o, c_p + kk * 8, v0 + kk * (2048 / 16), IDESC_PV, (k > 0 || kk > 0) ? 1u : 0u);
          if (EARLY) tc_commit_if(leader, smem_u32(pfree + g));
          tc_commit_if(leader, smem_u32(empty + vslot));
          if (!EARLY && more) {
            issue_s();
            if (k + 2 == u.ntile) tc_commit_if(leader, smem_u32(qempty));  // the unit's last S
          }
          if (!more) tc_commit_if(leader, smem_u32(odone + g));
        }
      }
      // nothing of this warp's may still be running when TMEM is freed
      tc_commit_if(leader, smem_u32(done + g));
      mbar_wait(smem_u32(done + g), 0u, nullptr);
    } else if (warp == kLoadK || warp == kLoadV) {
      // ------------------------------------------------------------ loads
      // The K loader also hands out the units: its own block index first, then
      // those of CTAs that it keeps from starting.
      const int v = warp == kLoadV ? 1 : 0;
      constexpr int ROWB = WIDE ? C::RAWROW : 128;      // bytes of a box row
      constexpr int BYTES = WIDE ? C::RAW : C::TILE;
      constexpr int MOVED = KV == kE2M1 ? C::CODES + NK * (D / 16) : BYTES;
      constexpr int NRING = WIDE ? NR : NS;
      const uint32_t base = smem_u32(WIDE ? raw : ring);
      uint64_t* bfull = WIDE ? rfull : full;
      uint64_t* bempty = WIDE ? rempty : empty;
      const int per_half = NK / p.block_size;          // boxes of a column half
      const int nbox = per_half * (KV == kE2M1 ? 2 : (WIDE ? 1 : C::HALVES));
      const int hf = lane / per_half, bi = lane % per_half;  // E2M1: hf 1 loads scales
      const bool scales = KV == kE2M1 && hf == 1;
      const int box_scales = p.block_size * (D / 16) < 128 ? 128 : p.block_size * (D / 16);
      const uint32_t off = scales ? C::CODES + bi * box_scales : hf * C::HALFB + bi * p.block_size * ROWB;
      const CUtensorMap* tmap = v ? &tmap_v : &tmap_k;
      if constexpr (KV == kE2M1) {
        if (scales) tmap = v ? &tmap_s.v : &tmap_s.k;
      }
      int item = v;  // K of tile j is item 2 j of the ring, V item 2 j + 1
      int asked = 0, loads = 0, fixes = 0;  // units asked for; Qs loaded; units with a zeroed tail so far
      bool ok = true;
      uint32_t bx = blockIdx.x, by = blockIdx.y;
      TcUnit u;
      for (int n = 0; ok; ++n) {
        if (v == 0) {
          // the next unit there is, published to the other warps
          bool have = n == 0;
          u.b = -1;
          while (ok) {
            if (!have) {
              ok = wait(clc, asked - 1);
              if (!ok) break;
              have = clc_answer(smem_u32(s_clc), bx, by);
              if (!have) break;  // none is left, and none is asked for again
            }
            // one answer ahead, so that it has arrived when it is wanted
            __syncwarp();
            if (lane == 0) {
              fence_proxy_async_smem();  // the last answer has been read
              mbar_arrive_expect_tx(smem_u32(clc), 16);
              clc_ask(smem_u32(s_clc), smem_u32(clc));
            }
            __syncwarp();
            ++asked;
            if (tc_unit<NK, KV>(p, static_cast<int>(bx), static_cast<int>(by), u)) break;
            u.b = -1;
            have = false;
          }
          if (!ok) u.b = -1;
          const int slot = n % RU;
          if (n >= RU) ok = wait(uempty + slot, n / RU - 1) && ok;
          constexpr int W = sizeof(TcUnit) / 4;
          const uint32_t* from = reinterpret_cast<const uint32_t*>(&u);
          if (lane == 0) {
#pragma unroll
            for (int i = 0; i < W; ++i) s_unit[slot * C::UNIT + i] = from[i];
            mbar_arrive(smem_u32(ufull + slot));  // releases the slot's values to the readers
          }
          __syncwarp();
          if (u.b < 0) break;
        } else {
          if (!read_unit(n, u)) break;
          // Q of the unit, once every S of the last one has read its own
          if (n > 0) ok = wait(qempty, n - 1);
          if (!ok) break;
          if (lane == 0) {
            const uint32_t bytes = static_cast<uint32_t>(p.tile_q * G * 128);
            fence_proxy_async_smem();
            mbar_arrive_expect_tx(smem_u32(qfull), C::HALVES * bytes);
#pragma unroll
            for (int hh = 0; hh < C::HALVES; ++hh)  // rows (token, head), 128 bytes each
              tma_load_4d(smem_u32(q_sm) + hh * C::QHALF, &tmap_q, smem_u32(qfull), hh * 64, 0, u.h, u.row0);
          }
          __syncwarp();
          ++loads;
        }
        const int32_t* tbl = p.block_tables + static_cast<int64_t>(u.b) * p.max_blocks;
        // the block this lane's box of tile k holds; blocks that no row sees are
        // not looked up and read as zeros (outside the tensor map)
        auto block_of = [&](int k) {
          int phys = -1;
          if (lane < nbox && k < u.ntile) {
            const int t0 = u.tile(k) * NK + bi * p.block_size;
            if (u.sees(t0, t0 + p.block_size)) {
              phys = tbl[t0 / p.block_size];
              if (phys < 0 || phys >= p.num_blocks) {
                if (v == 0 && hf == 0) record_error(p.err, kDevErrBlockId);
                phys = -1;
              }
            }
          }
          return phys;
        };
        int phys = block_of(0);
        for (int k = 0; k < u.ntile; ++k, item += 2) {
          const int s = item % NRING;
          const int next = block_of(k + 1);
          if (item >= NRING) ok = wait(bempty + s, item / NRING - 1);
          if (!ok) break;
          const uint32_t bar = smem_u32(bfull + s);
          if (lane == 0) {
            fence_proxy_async_smem();
            mbar_arrive_expect_tx(bar, MOVED);
          }
          __syncwarp();
          if (lane < nbox) tma_load_4d(base + s * BYTES + off, tmap, bar, WIDE ? 0 : hf * 64, 0, u.h, phys);
          phys = next;
        }
        if (!WIDE && v == 1 && ok && u.v_tail(NK, p.block_size)) {
          // Rows of the last block past the sequence's end may hold anything
          // (NaN included): zero them once they have landed, P is 0 there.  Whole
          // blocks past it were loaded as zeros.
          const int last = item - 2, s = last % NRING;
          ok = wait(bfull + s, last / NRING);
          if (!ok) break;
          const int first = u.tail_first(NK);
          const int chunks = ((first + p.block_size - 1) / p.block_size * p.block_size - first) * 8;
          for (int c = lane; c < C::HALVES * chunks; c += 32) {
            const int hh = c / chunks, cc = c - hh * chunks;
            *reinterpret_cast<uint4*>(ring + s * C::TILE + hh * C::HALFB + first * 128 + cc * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(vfix + (fixes & 1)));
          ++fixes;
        }
      }
      if (lane == 0) {
        s_issued[v] = item;
        s_issued[2 + v] = v == 0 ? asked : loads;
      }
    } else if (WIDE && warp >= kConv) {
      // ------------------------------------------------------------ widening
      // of the unit's Q (bf16 -> f16, in place) and its K and V tiles (thread t:
      // key t of the tile, 16 codes -> 32 bytes at a time)
      if constexpr (WIDE) {
        static_assert(NK == 128, "a widening thread per key");
        const int t = (warp - kConv) * 32 + lane;
        int item = 0;
        bool ok = true;
        TcUnit u;
        for (int n = 0; ok && read_unit(n, u); ++n) {
          ok = wait(qfull, n);
          if (!ok) break;
          for (int i = t; i < C::HALVES * u.rows * 8; i += 128) {
            const int hh = i / (u.rows * 8);
            uint4* at = reinterpret_cast<uint4*>(q_sm + hh * C::QHALF + (i - hh * u.rows * 8) * 16);
            uint4 w = *at;
            w.x = pack_f16x2(bf16lo_to_f32(w.x), bf16hi_to_f32(w.x));
            w.y = pack_f16x2(bf16lo_to_f32(w.y), bf16hi_to_f32(w.y));
            w.z = pack_f16x2(bf16lo_to_f32(w.z), bf16hi_to_f32(w.z));
            w.w = pack_f16x2(bf16lo_to_f32(w.w), bf16hi_to_f32(w.w));
            *at = w;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(qready));
          for (int i = 0; i < 2 * u.ntile; ++i, ++item) {
            const int rs = item % NR, s = item % NS;
            ok = wait(rfull + rs, item / NR);
            if (ok && item >= NS) ok = wait(empty + s, item / NS - 1);
            if (!ok) break;
            // rows past the sequence's end may hold anything: zeros instead
            const bool live = u.tile(i >> 1) * NK + t < u.ctx;
            uint8_t* dst = ring + s * C::TILE + t * 128;
            if constexpr (KV == kE2M1)
              widen_e2m1<D>(raw + rs * C::RAW, dst, C::HALFB, t, p.block_size, live);
            else
              widen_e4m3<D>(raw + rs * C::RAW + t * D, dst, C::HALFB, t, live);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(smem_u32(full + s));
              mbar_arrive(smem_u32(rempty + rs));
            }
          }
        }
      }
    }
  } else {
    regs_inc<C::REGS_SOFTMAX>();
    // -------------------------------------------------------------- softmax
    const int grp = warp >> 2;
    const uint32_t lanes = tbase + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t t_s = lanes + COL_S + grp * NK, t_p = lanes + COL_P + grp * P_STEP, t_o = lanes + COL_O + grp * D;
    uint8_t* stage = s_stage + warp * C::STAGE;
    // r / G for a row r < 256 of the tile: exact, since r times the rounding of
    // the reciprocal (less than G / 65536) stays below 1 / G
    const uint32_t inv_g = (65536u + G - 1) / G;
    auto token_of = [&](int r) { return static_cast<int>(static_cast<uint32_t>(r) * inv_g >> 16); };
    int sk = 0, outs = 0;  // this group's tiles and its units with tiles so far
    bool ok = true;
    TcUnit u;
    for (int n = 0; ok && read_unit(n, u); ++n) {
      if (grp * M >= u.rows) continue;
      const int r_in = tid;                              // row of the tile
      const bool row_ok = r_in < u.rows;
      const bool warp_ok = warp * 32 < u.rows;           // some lane has a row
      const int tok = token_of(r_in), gh = r_in - tok * G;
      // what the row sees; a row past the tile's takes no mask (nothing of it
      // is ever written)
      constexpr int kFarPos = 0x3FFFFFFF;
      const int pos = row_ok ? u.pos0 + tok : kFarPos;
      const int lo = row_ok && p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
      const int pf = row_ok && pos >= 0 ? u.prefix : 0;
      constexpr float kLog2e = 1.4426950408889634f;
      const float qk = WIDE ? p.qk_log2 * __int_as_float(u.k_bits) : p.qk_log2;
      const float slope = (SCORE == kBiased || SCORE == kCappedBiased) && row_ok ? p.slopes[u.h * G + gh] * kLog2e : 0.f;
      const CapPoly<FAR> poly(qk, p);

      float m_used = -CUDART_INF_F, lsum = 0.f;
      for (int k = 0; k < u.ntile; ++k, ++sk) {
        ok = wait(sfull + grp, sk);
        if (!ok) break;
        tc_fence_after();
        if (warp_ok) {
          const int t0 = u.tile(k) * NK;
          auto is_masked = [&]() { return !__all_sync(kFull, (t0 + NK - 1 <= pos && t0 >= lo) || t0 + NK <= pf); };
          auto below = [&](int n, int w) {  // the first n keys of the tile, as bits of word w
            n -= 32 * w;
            return n <= 0 ? 0u : (n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u);
          };
          auto seen = [&](int w) {  // bit i: key t0 + 32 w + i is seen
            return (below(pos - t0 + 1, w) & ~below(lo - t0, w)) | below(pf - t0, w);
          };
          // rows past the tile's last hold what was in their shared memory: they do not
          // choose how the warp's scores are capped
          auto magnitude = [&](float abs_max) { return row_ok ? abs_max : 0.f; };
          float alpha = 1.f;
          bool resc = false;
          auto grow = [&](float mt) {  // the row's maximum of this tile
            if (m_used == -CUDART_INF_F) {
              m_used = mt;  // nothing accumulated yet for this row
            } else if (row_ok && mt > m_used + 8.f) {
              alpha = fast_exp2(m_used - mt);
              m_used = mt;
              resc = true;
            }
          };
          auto rescale = [&]() {
            if (!__any_sync(kFull, resc)) return;  // O holds tiles 0..k-1 (else PV(k-1) came before S(k))
#pragma unroll
            for (int c0 = 0; c0 < D; c0 += 32) {
              uint32_t u[2][16];
              tmem_ld16(t_o + c0, u[0]);
              tmem_ld16(t_o + c0 + 16, u[1]);
              tmem_wait_ld();
#pragma unroll
              for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                for (int i = 0; i < 16; ++i) u[hh][i] = __float_as_uint(__uint_as_float(u[hh][i]) * alpha);
              tmem_st16(t_o + c0, u[0]);
              tmem_st16(t_o + c0 + 16, u[1]);
            }
            lsum *= alpha;
          };
          float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          // weights of 32 keys, 2^(score - m), into S's columns; WAY: the scores are
          // raw products, raw products to be capped (small ones), done, or raw
          // products to be capped (up to kMidLimit caps)
          auto weights = [&](auto way, int c, const float* x) {
            constexpr int WAY = decltype(way)::value;
            const float mu = m_used == -CUDART_INF_F ? 0.f : m_used;
            const float2 neg_mu = make_float2(-mu, -mu), mult2 = make_float2(qk, qk);
            [[maybe_unused]] const float2 cap2 = make_float2(p.cap_log2, p.cap_log2);
            uint32_t hi[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 xx = make_float2(x[2 * i], x[2 * i + 1]);
              const float2 e = WAY == 0   ? __ffma2_rn(xx, mult2, neg_mu)
                               : WAY == 1 ? poly.minus(xx, neg_mu)
                               : WAY == 2 ? __fadd2_rn(xx, neg_mu)
                                          : __ffma2_rn(mid_tanh(xx, poly.y_mult), cap2, neg_mu);
              const float2 pp = make_float2(fast_exp2(e.x), fast_exp2(e.y));
              ls[i & 1] = __fadd2_rn(ls[i & 1], pp);
              hi[i] = WIDE ? pack_f16x2(pp.x, pp.y) : pack_bf16x2(pp.x, pp.y);
            }
            tmem_st16(t_p + 16 * c, hi);
          };
          if constexpr (PARTS) {
            // Scores that are not all small are read again, in parts of 32 that each
            // take their own way, by a loop whose code stays in the instruction cache
            // (the whole row's code for each way: 5 prompts of 301-1777, 28 + 4 heads
            // of 64, cap 30 75 us, this 62; all rows in parts 60, but 437 us for 345
            // where all are small, 4 chunks of 512 over 3584 of 128-wide heads).  P's
            // part takes columns that have been read.
            uint32_t ways = 0u;  // of each part: 0 small, 1 up to kMidLimit caps, 2 beyond
            float x[NK];
#pragma unroll
            for (int c = 0; c < NK / 32; ++c) tmem_ld32(t_s + 32 * c, x + 32 * c);
            tmem_wait_ld();
            const bool masked = is_masked();
#pragma unroll
            for (int c = 0; c < NK / 32; ++c) {
              const float am = magnitude(abs_max<32>(x + 32 * c));
              const bool small = __all_sync(kFull, poly.holds(am)), mid = __all_sync(kFull, am * poly.y_mult <= kMidLimit);
              ways |= (small ? 0u : mid ? 1u : 2u) << (2 * c);
            }
            if (masked) {
#pragma unroll
              for (int c = 0; c < NK / 32; ++c) {
                const uint32_t see = seen(c);
                mask_scores<32>(x + 32 * c, &see);
              }
            }
            float mt = row_max<NK>(x);
            mt = mt == -CUDART_INF_F ? mt : capped<FAR>(mt, qk, p.cap_log2, poly);
            grow(mt);
            rescale();
            if (ways == 0u) {
#pragma unroll
              for (int c = 0; c < NK / 32; ++c) weights(std::integral_constant<int, 1>{}, c, x + 32 * c);
            } else {
#pragma unroll 1
              for (int c = 0; c < NK / 32; ++c, ways >>= 2) {
                float x[32];
                tmem_ld32(t_s + 32 * c, x);
                tmem_wait_ld();
                const uint32_t way = ways & 3u, see = masked ? seen(c) : 0xFFFFFFFFu;
                if (way == 2u) cap_scores<32, FAR>(x, qk, p.cap_log2, poly, masked, &see);
                if (masked) mask_scores<32>(x, &see);
                if (way == 0u)
                  weights(std::integral_constant<int, 1>{}, c, x);
                else if (way == 1u)
                  weights(std::integral_constant<int, 3>{}, c, x);
                else
                  weights(std::integral_constant<int, 2>{}, c, x);
              }
            }
          } else {
            float x[NK];
#pragma unroll
            for (int c = 0; c < NK / 32; ++c) tmem_ld32(t_s + 32 * c, x + 32 * c);
            tmem_wait_ld();
            if constexpr (EARLY) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_u32(sfree + grp));  // S may be overwritten
            }
            const bool masked = is_masked();
            uint32_t see[NK / 32];
            if (masked) {
#pragma unroll
              for (int w = 0; w < NK / 32; ++w) see[w] = seen(w);
            }
            // Capped: the row maximum is taken of the raw products (a cap does not
            // change which is the largest), the cap enters with the exponent.
            bool small = false, mid = false;
            if constexpr (SCORE == kCapped) small = __all_sync(kFull, poly.holds(magnitude(abs_max<NK>(x))));
            if constexpr (SCORE == kCappedBiased) {
              if constexpr (MID) mid = __all_sync(kFull, magnitude(abs_max<NK>(x)) * poly.y_mult <= kMidLimit);
              if (mid) {
#pragma unroll
                for (int i = 0; i < NK; i += 2) {
                  const float2 z = __fmul2_rn(mid_tanh(make_float2(x[i], x[i + 1]), poly.y_mult),
                                              make_float2(p.cap_log2, p.cap_log2));
                  x[i] = z.x;
                  x[i + 1] = z.y;
                }
              } else {
                cap_scores<NK, FAR>(x, qk, p.cap_log2, poly, masked, see);
              }
            }
            if constexpr (SCORE == kBiased || SCORE == kCappedBiased) {
              const float mult = SCORE == kBiased ? qk : 1.f, base = slope * static_cast<float>(t0 - pos);
              const float2 mult2 = make_float2(mult, mult), slope2 = make_float2(slope, slope);
              const float2 base2 = make_float2(base, base);
#pragma unroll
              for (int i = 0; i < NK; i += 2) {
                const float2 at = make_float2(static_cast<float>(i), static_cast<float>(i + 1));
                const float2 z = __ffma2_rn(make_float2(x[i], x[i + 1]), mult2, __ffma2_rn(slope2, at, base2));
                x[i] = z.x;
                x[i + 1] = z.y;
              }
            }
            if (masked) mask_scores<NK>(x, see);
            float mt = row_max<NK>(x);
            if constexpr (SCORE == kPlain) mt *= qk;
            if constexpr (SCORE == kCapped) mt = mt == -CUDART_INF_F ? mt : capped<FAR>(mt, qk, p.cap_log2, poly);
            grow(mt);
            if (EARLY && sk > 0) {  // P(k-1)'s product has read it (and O holds tiles 0..k-1)
              ok = wait(pfree + grp, sk - 1);
              if (!ok) break;
              tc_fence_after();
            }
            rescale();
            auto each = [&](auto way) {
#pragma unroll
              for (int c = 0; c < NK / 32; ++c) weights(way, c, x + 32 * c);
            };
            if constexpr (SCORE == kPlain) {
              each(std::integral_constant<int, 0>{});
            } else if constexpr (SCORE == kCapped) {
              if (small) {
                each(std::integral_constant<int, 1>{});
              } else {
                cap_scores<NK, FAR>(x, qk, p.cap_log2, poly, masked, see);
                if (masked) mask_scores<NK>(x, see);
                each(std::integral_constant<int, 2>{});
              }
            } else {
              each(std::integral_constant<int, 2>{});
            }
          }
          lsum += (ls[0].x + ls[1].x) + (ls[0].y + ls[1].y);
          tmem_wait_st();
        } else if constexpr (EARLY) {
          if (lane == 0) mbar_arrive(smem_u32(sfree + grp));
          if (sk > 0) ok = wait(pfree + grp, sk - 1);
          if (!ok) break;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(pfull + grp));  // P is in TMEM
      }
      if (ok && u.ntile > 0) ok = wait(odone + grp, outs++);
      if (ok && warp_ok) {
        // ---- O leaves through the warp's staging, SB bytes of its rows per
        // pass, so that a store instruction writes whole pieces of that size
        // (four prompts of 1000 tokens: 88 us; 32 bytes of its row per lane and
        // store 90.5, 16 bytes 97; without any output 72)
        tc_fence_after();
        const float inv = lsum > 0.f ? (WIDE ? __int_as_float(u.v_bits) / lsum : 1.f / lsum) : 0.f;
        const bool direct = u.nsplit == 1;
        const float mult = direct ? inv : (WIDE ? __int_as_float(u.v_bits) : 1.f);
        float o[D];
        if (u.ntile > 0) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) tmem_ld32(t_o + 32 * c, o + 32 * c);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < D; ++i) o[i] = 0.f;
        }
        tc_fence_before();  // O has been read: the next unit's products may overwrite it after P's hand-over
        constexpr int CR = C::SB / 16;                   // 16-byte chunks of a row and pass
        // chunk c of row r, placed so that eight consecutive rows' chunks c lie
        // in distinct banks
        auto at = [&](int r, int c) { return stage + r * C::SB + ((c ^ (r * C::SB / 128 % CR)) << 4); };
        auto row_of = [&](int r) {                       // output row of the warp's row r
          const int rr = warp * 32 + r, tk = token_of(rr);
          return static_cast<int64_t>(u.row0 + tk) * H_q + u.h * G + (rr - tk * G);
        };
        // this lane stores chunk lane % CR of rows lane / CR + (32 / CR) i: byte
        // offsets in the output or the workspace, -1 past the tile's rows
        int64_t to[CR];
#pragma unroll
        for (int i = 0; i < CR; ++i) {
          const int r = lane / CR + (32 / CR) * i;
          const int64_t at_row = direct ? row_of(r) * (D * 2) : (row_of(r) * p.max_splits + u.split) * (D * 4);
          to[i] = warp * 32 + r < u.rows ? at_row + (lane % CR) * 16 : -1;
        }
        char* dst = direct ? static_cast<char*>(p.out) : reinterpret_cast<char*>(p.ws_o);
        auto leave = [&](int pass) {                     // SB bytes of every row
          __syncwarp();
          uint4 w[CR];
#pragma unroll
          for (int i = 0; i < CR; ++i) w[i] = *reinterpret_cast<const uint4*>(at(lane / CR + (32 / CR) * i, lane % CR));
#pragma unroll
          for (int i = 0; i < CR; ++i)
            if (to[i] >= 0) *reinterpret_cast<uint4*>(dst + to[i] + pass * C::SB) = w[i];
          __syncwarp();
        };
        if (direct) {
#pragma unroll
          for (int pass = 0; pass < D * 2 / C::SB; ++pass) {
#pragma unroll
            for (int i = 0; i < CR; ++i) {
              const float* v = o + pass * (C::SB / 2) + 8 * i;
              uint4 w;
              w.x = pack_bf16x2(v[0] * mult, v[1] * mult);
              w.y = pack_bf16x2(v[2] * mult, v[3] * mult);
              w.z = pack_bf16x2(v[4] * mult, v[5] * mult);
              w.w = pack_bf16x2(v[6] * mult, v[7] * mult);
              *reinterpret_cast<uint4*>(at(lane, i)) = w;
            }
            leave(pass);
          }
        } else {
#pragma unroll
          for (int pass = 0; pass < D * 4 / C::SB; ++pass) {
#pragma unroll
            for (int i = 0; i < CR; ++i) {
              const float* v = o + pass * (C::SB / 4) + 4 * i;
              *reinterpret_cast<float4*>(at(lane, i)) = make_float4(v[0] * mult, v[1] * mult, v[2] * mult, v[3] * mult);
            }
            leave(pass);
          }
        }
        if (!direct && row_ok) {
          float* ml = p.ws_ml + (row_of(lane) * p.max_splits + u.split) * 2;
          ml[0] = m_used;
          ml[1] = lsum;
        }
      }
    }
  }
  allow_next_grid();
  tc_fence_before();
  __syncthreads();
  if (warp == kLoadK && *s_abort) {  // what is still in flight lands before the CTA leaves
    constexpr int NRING = WIDE ? NR : NS;
    uint64_t* bfull = WIDE ? rfull : full;
    const int next_k = s_issued[0], next_v = s_issued[1], asked = s_issued[2], loads = s_issued[3];
    const int last = lane < NRING ? ring_last_item(lane, NRING, next_k, next_v) : -1;
    if (last >= 0) mbar_wait(smem_u32(bfull + lane), static_cast<uint32_t>((last / NRING) & 1), nullptr);
    if (lane == 0 && asked > 0) mbar_wait(smem_u32(clc), static_cast<uint32_t>((asked - 1) & 1), nullptr);
    if (lane == 0 && loads > 0) mbar_wait(smem_u32(qfull), static_cast<uint32_t>((loads - 1) & 1), nullptr);
  }
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

template <int D, int KV, int MODE>
cudaError_t launch_tc_t(const ChunkParams& p, const ChunkMaps& m, cudaStream_t stream) {
  auto kern = chunk_tc_kernel<D, KV, MODE>;
  using C = TcShape<D, KV, MODE>;
  // at least 120 KB: one CTA per SM (it holds all 512 TMEM columns)
  constexpr int smem = C::BYTES > 120 * 1024 ? C::BYTES : 120 * 1024;
  static int configured[64] = {};
  cudaError_t e = set_smem_once(kern, smem, configured);
  if (e != cudaSuccess) return e;
  const int tiles = p.n_tokens / p.tile_q + p.batch;
  ScaleMaps<KV> scales;
  if constexpr (KV == kE2M1) scales = {m.k_scales, m.v_scales};
  return launch_pdl(kern, dim3(tiles * p.num_kv_heads, p.max_splits), dim3(C::THREADS), smem, stream, m.q, m.k, m.v,
                    scales, p);
}

template <int D, int KV>
cudaError_t launch_tc_m(const ChunkParams& p, const ChunkMaps& m, cudaStream_t stream) {
  if (p.cap_far)
    return p.slopes != nullptr ? launch_tc_t<D, KV, kCappedBiased | kFar>(p, m, stream)
                               : launch_tc_t<D, KV, kCapped | kFar>(p, m, stream);
  if (p.slopes != nullptr)
    return p.cap_log2 > 0.f ? launch_tc_t<D, KV, kCappedBiased>(p, m, stream) : launch_tc_t<D, KV, kBiased>(p, m, stream);
  if (p.cap_log2 > 0.f) return launch_tc_t<D, KV, kCapped>(p, m, stream);
  return launch_tc_t<D, KV, kPlain>(p, m, stream);
}

template <int KV>
cudaError_t launch_tc(const ChunkParams& p, const ChunkMaps& m, cudaStream_t stream) {
  return p.head_dim == 128 ? launch_tc_m<128, KV>(p, m, stream) : launch_tc_m<64, KV>(p, m, stream);
}

}  // namespace
}  // namespace pkv
