// Attention of ragged chunks over E2M1 caches, row tiles of up to 16 rows (single
// tokens of up to 16 query heads per KV head, a few tokens of smaller groups);
// what it computes: chunk_common.cuh, what a cache holds: pkv.h.
//
// A CTA takes the rows of one tile of one (sequence, KV head) over one split of
// its visible keys, in 128-key steps: a warp copies its 32 keys of every step (a
// block's codes and scales lie behind one another) into a ring of its own and
// refills a slot as soon as it has read it, waiting for no other warp; the warps
// merge (m, l, O) through shared memory at the end.  The copies are the lanes' own
// 16-byte ones: a block of one head is 1152 bytes (576 with 64-wide heads), and
// bulk copies of that size came no faster than one per 58 cycles and SM whatever
// they hold (64 sequences of 512-8192 tokens, 64 + 8 heads of 128, 16-token blocks:
// 85.5 us where this takes 77; tensor-map boxes of codes and of scales 90.5).
//
// Both products have keys as the first operand's rows or columns and up to 8
// tile rows as the second's columns (NT of them: 1 or 2), mma.sync m16n8k16 of
// f16 with fp32 sums, so that the codes, widened once, serve every row:
//   S^T = K Q^T.  A lane reads a quarter of a key's row, 8 codes a word, two
//     products' worth, whose order of d is Q's to follow.  cvt makes f16 pairs of
//     its bytes, which are multiplied by the key's scale of that group, in pairs
//     too: exact, so S is that of the cache's values.
//   O^T += V^T P^T.  A lane needs pairs of keys at one d where the cache has
//     pairs of d of one key: it reads the same D / 8 d of its four keys and swaps
//     halves of their bytes before it widens them (a shift and a select for four
//     pairs).  All of them lie in one group, so that a pair of keys has one pair
//     of scales.
// Keys take the products' rows in an order (key_of) that spreads those reads over
// the banks.  P is rounded to f16: at most 2^-11 of each weight, next to the
// output's own 2^-8.  V past the sequence's end, and K and V of blocks that no
// row sees, have scale 0 (codes are finite whatever they are).
//
// Bound: the HBM stream of 9/8 D bytes per visible key and KV head, and close
// behind it the instructions: 647 of a warp per 32 keys of 128 (253 of them the
// ALU's, 148 of those conversions), of the 800 cycles that the stream leaves it.
// 8 sequences of 131,072 tokens: 195 us with the merge, 6.2 TB/s, 91 % of the
// measured copy; 64 of 512-8192 76 us, 4.6 TB/s, 68 %: a CTA's start (lengths,
// table, first keys, one after another) and end cost 1.2 us of its SM's time each
// time (200 sequences of 200: 23 us for 7.5 of bytes), and shorter ones, longer ones
// or none ahead of others come to the same; 64-wide heads 50 us, 51 %, with the same
// cost for half the bytes.  Measured and not kept: five CTAs per SM (83 and 221 us:
// 96 registers), two warps of 32 keys per CTA and eight CTAs (80-93 and 196; windowed
// single tokens 64 for 72, up to 16 rows 120 for 110), 64 keys per warp, equal
// ranges of all steps per CTA (88 us for 85 before the lanes' copies).

#include "chunk_common.cuh"

namespace pkv {
namespace {

template <int D, int NT, int BS>
struct E2M1Shape {
  static constexpr int STEP = kChunkE2M1Tile, KEYS = 32;    // keys of a step, and of a warp
  static constexpr int WARPS = STEP / KEYS, THREADS = 32 * WARPS, NG = KEYS / 16;
  static constexpr int ROWB = D / 2, SROWB = D / 16;        // bytes of a row's codes and scales
  static constexpr int TILE = BS * (ROWB + SROWB);          // of a block: its rows of codes, then of scales
  static constexpr int NBLK = KEYS / BS;                    // blocks of a warp's step
  static constexpr int STAGE = 2 * NBLK * TILE;             // a warp's step: K, then V
  static constexpr int CTAS = chunk_e2m1_ctas(NT == 1);
  static constexpr int NS = 2;
  static constexpr int DP = D + 4, R = 8 * NT;
  static constexpr int MERGE = WARPS * R * DP * 4 + WARPS * R * 2 * 4;
  static constexpr int RING = NS * WARPS * STAGE;
  static constexpr int BYTES = (RING > MERGE ? RING : MERGE) + kChunkMaxSplitBlocks * 4 + 128;
  // codes and scales of a group of 16 keys, from K's or V's start in a stage
  static constexpr int code_of(int g) { return 16 * g / BS * TILE + 16 * g % BS * ROWB; }
  static constexpr int scale_of(int g) { return 16 * g / BS * TILE + BS * ROWB + 16 * g % BS * SROWB; }
};

// Key of a 16-key group that is row i = 8 n + 4 j1 + 2 j0 + e of the products: the
// eight lanes that read 128 bytes of K together, and the lanes that read the same
// d of V, then have keys in different halves (64-byte rows) or quarters (32-byte
// rows) of 128 bytes.
template <int D>
__device__ __forceinline__ int key_of(int i) {
  return (i & 14) | ((i & 1) ^ (D == 128 ? (i >> 1) & 1 : (i >> 2) & 1));
}

// Copy 16 bytes global -> shared behind the thread's back, or zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Wait until the copies of all of this thread's groups but the last N have landed.
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// MODS: scores that are capped or biased.  FAR: a cap above kCapNear.
template <int D, int NT, int BS, bool MODS, bool FAR>
__global__ void __launch_bounds__(E2M1Shape<D, NT, BS>::THREADS, E2M1Shape<D, NT, BS>::CTAS)
    chunk_e2m1_kernel(const ChunkParams p) {
  using C = E2M1Shape<D, NT, BS>;
  constexpr int NS = C::NS, DP = C::DP, KS = D / 16, NG = C::NG, WARPS = C::WARPS;
  constexpr int KW = D / 32;  // words of codes that a lane takes of a key of K

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, j = lane & 3;
  const int G = p.group, H_q = p.num_q_heads;
  const int ntq = (p.max_q_len + p.tile_q - 1) / p.tile_q;
  const int h = blockIdx.y / ntq;
  const int i0 = (blockIdx.y - h * ntq) * p.tile_q;
  const int b = blockIdx.z, split = blockIdx.x;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
  int* s_blk = reinterpret_cast<int*>(smem + (C::RING > C::MERGE ? C::RING : C::MERGE));
  const uint32_t stage0 = smem_u32(smem) + warp * NS * C::STAGE;  // of this warp's ring

  wait_prior_grid();

  const ChunkSeq sq = chunk_seq(p, b, split == 0 && blockIdx.y == 0 && threadIdx.x == 0);
  if (i0 >= sq.n) return;
  const int i1 = min(sq.n, i0 + p.tile_q) - 1;
  const int rows = (i1 - i0 + 1) * G;
  const ChunkRange rg = chunk_range<C::STEP>(p, sq, i0, i1);
  const ChunkSplit sp(rg.n, p.split_tokens / C::STEP, split);
  const int nsplit = sp.nsplit, k0 = sp.k0, ntile = sp.ntile;
  if (split >= nsplit) return;
  const int64_t row_base = static_cast<int64_t>(sq.start + i0) * H_q + h * G;  // of row (0, g = 0)
  auto out_row = [&](int row) { return row_base + static_cast<int64_t>(row / G) * H_q + row % G; };

  // block ids of the split's keys; blocks that no row sees (behind the window,
  // past the last query) are not looked up and read as zeros
  constexpr int per_tile = C::STEP / BS;
  const int32_t* tbl = p.block_tables + static_cast<int64_t>(b) * p.max_blocks;
  for (int i = threadIdx.x; i < ntile * per_tile; i += blockDim.x) {
    const int t0 = rg.tile(k0 + i / per_tile) * C::STEP + (i % per_tile) * BS;
    int phys = -1;
    if (rg.sees(t0, t0 + BS)) {
      phys = tbl[t0 / BS];
      if (phys < 0 || phys >= p.num_blocks) {
        record_error(p.err, kDevErrBlockId);
        phys = -1;
      }
    }
    s_blk[i] = phys;
  }
  __syncthreads();

  // A warp's step is K's blocks and then V's, as they lie in the cache: PER lanes
  // copy one of them, 16 bytes each in turn, so that eight lanes read a line.
  constexpr int PIECES = 2 * C::NBLK, PER = 32 / PIECES, TURNS = (C::TILE / 16 + PER - 1) / PER;
  const int copied = lane / PER, sub = lane % PER;
  const bool is_v = copied >= C::NBLK;
  const uint8_t* cache = static_cast<const uint8_t*>(is_v ? p.v_cache : p.k_cache) +
                         static_cast<int64_t>(h) * C::TILE + sub * 16;
  const int64_t block_bytes = static_cast<int64_t>(p.num_kv_heads) * C::TILE;
  const uint32_t copy_to = stage0 + copied * C::TILE + sub * 16;
  const uint32_t blk0 = smem_u32(s_blk) + 4 * (warp * C::NBLK + (is_v ? copied - C::NBLK : copied));
  auto issue = [&](int k, int s) {  // step k into stage s, which this warp has read
    uint32_t phys[1];
    lds_words(blk0 + k * (4 * per_tile), phys);
    const bool there = static_cast<int>(phys[0]) >= 0;  // else no row sees the block: zeros
    const uint8_t* from = there ? cache + static_cast<int64_t>(phys[0]) * block_bytes : cache;
    const uint32_t to = copy_to + s * C::STAGE;
#pragma unroll
    for (int i = 0; i < TURNS; ++i)
      if ((i + 1) * PER * 16 <= C::TILE || i * PER + sub < C::TILE / 16)
        copy16(to + i * PER * 16, from + i * PER * 16, there);
  };
  int issued = 0;
#pragma unroll
  for (int i = 0; i < NS; ++i) {  // a group per step, empty past the last
    if (issued < ntile) issue(issued++, i);
    copies_end();
  }

  // Q as the second operand: row r of each n-tile; word c of the lane's quarter of
  // a row is two products, of d j D / 4 + 8 c + 0..3 and + 4..7
  uint32_t qb[NT][KS][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = 8 * nt + r;
    const uint16_t* q = static_cast<const uint16_t*>(p.q) + out_row(row) * D + j * (D / 4);
#pragma unroll
    for (int c = 0; c < KW; ++c) {
      const uint4 w = row < rows ? *reinterpret_cast<const uint4*>(q + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
      qb[nt][2 * c][0] = pack_f16x2(bf16lo_to_f32(w.x), bf16hi_to_f32(w.x));
      qb[nt][2 * c][1] = pack_f16x2(bf16lo_to_f32(w.y), bf16hi_to_f32(w.y));
      qb[nt][2 * c + 1][0] = pack_f16x2(bf16lo_to_f32(w.z), bf16hi_to_f32(w.z));
      qb[nt][2 * c + 1][1] = pack_f16x2(bf16lo_to_f32(w.w), bf16hi_to_f32(w.w));
    }
  }
  // this lane's rows of the tile: 8 nt + 2 j and + 1.  Per row: position, first
  // key of the window, end of the prefix, bias; a row past the tile's takes no
  // mask (nothing of it is ever written)
  constexpr float kLog2e = 1.4426950408889634f;
  int pos[NT][2], lo[NT][2], pf[NT][2];
  float slope[NT][2], m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = 8 * nt + 2 * j + e;
      constexpr int kFarPos = 0x7FFFFFFF;
      pos[nt][e] = row < rows ? sq.ctx - sq.n + i0 + row / G : kFarPos;
      lo[nt][e] = p.window > 0 && row < rows && pos[nt][e] >= p.window ? pos[nt][e] - p.window + 1 : 0;
      pf[nt][e] = pos[nt][e] >= 0 ? sq.prefix : 0;
      slope[nt][e] = p.slopes != nullptr && row < rows ? p.slopes[h * G + row % G] * kLog2e : 0.f;
      m[nt][e] = -CUDART_INF_F;
      l[nt][e] = 0.f;
    }
  // of all rows: keys [lo_all, hi_all] and those before pf_all are seen by every one
  int hi_all = 0x7FFFFFFF, lo_all = 0, pf_all = 0x7FFFFFFF;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      hi_all = min(hi_all, pos[nt][e]);
      lo_all = max(lo_all, lo[nt][e]);
      pf_all = min(pf_all, pf[nt][e]);
    }
  hi_all = __reduce_min_sync(kFull, hi_all);
  lo_all = __reduce_max_sync(kFull, lo_all);
  pf_all = __reduce_min_sync(kFull, pf_all);
  float qk_mult = p.qk_log2, v_mult = 1.f;
  if (p.k_scale != nullptr) {
    qk_mult *= p.k_scale[static_cast<int64_t>(b) * p.scale_stride + h];
    v_mult = p.v_scale[static_cast<int64_t>(b) * p.scale_stride + h];
  }
  const CapPoly<FAR> poly(qk_mult, p);
  const float ex_mult = p.cap_log2 > 0.f || p.slopes != nullptr ? 1.f : qk_mult;  // scores to log2 weights

  float o[NT][KS][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.f;

  // K: key of score rows r (and r + 8, eight further); V: keys of the products'
  // columns 2 j, 2 j + 1 (and 2 j + 8, 2 j + 9), the lane's D / 8 d of them
  const int kr = key_of<D>(r), kv0 = key_of<D>(2 * j), kv1 = key_of<D>(2 * j + 1);
  constexpr int VB = D / 16, GL = D / 64;  // code bytes of a lane per key of V; groups of its quarter of K
  constexpr int VAT = C::NBLK * C::TILE;   // V behind K
  const uint32_t at_k = stage0 + kr * C::ROWB + j * (4 * KW), at_ks = stage0 + kr * C::SROWB + j * GL;
  const uint32_t at_v0 = stage0 + VAT + kv0 * C::ROWB + r * VB, at_v1 = stage0 + VAT + kv1 * C::ROWB + r * VB;
  const uint32_t at_vs0 = stage0 + VAT + kv0 * C::SROWB + r * VB / 8, at_vs1 = stage0 + VAT + kv1 * C::SROWB + r * VB / 8;

  int s = 0;
  for (int k = 0; k < ntile; ++k) {
    copies_wait<NS - 1>();
    __syncwarp();  // every lane's copies of this step have landed
    const uint32_t stage = s * C::STAGE;
    const int t_warp = rg.tile(k0 + k) * C::STEP + warp * C::KEYS;  // this warp's first key
    {
      // ---- S^T of groups of 16 keys, two at a time: rows r, r + 8 (e >= 2) are keys
      // kr and kr + 8, columns 2 j, 2 j + 1 (odd e)
      float sc[NG][NT][4];
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) sc[g][nt][0] = sc[g][nt][1] = sc[g][nt][2] = sc[g][nt][3] = 0.f;
#pragma unroll
      for (int g0 = 0; g0 < NG; g0 += 2) {
        uint32_t kw[2][2][KW], ks[2][2];  // codes and scale codes of keys kr and kr + 8
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            lds_words(at_k + stage + C::code_of(g0 + g) + 8 * x * C::ROWB, kw[g][x]);
            const uint32_t at = at_ks + stage + C::scale_of(g0 + g) + 8 * x * C::SROWB;
            ks[g][x] = GL == 2 ? lds_half(at) : lds_byte(at);
          }
#pragma unroll
        for (int gl = 0; gl < GL; ++gl) {  // words 2 gl and 2 gl + 1 lie in one group
          uint32_t s2[2][2];
#pragma unroll
          for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              s2[g][x] = e4m3x2_to_f16x2(static_cast<uint16_t>(prmt(ks[g][x], 0u, gl == 0 ? 0x4400u : 0x4411u)));
#pragma unroll
          for (int c = 2 * gl; c < 2 * gl + 2; ++c)
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              uint32_t x[4], y[4];  // of keys kr and kr + 8
              e2m1x8_to_f16x2(kw[g][0][c], x);
              e2m1x8_to_f16x2(kw[g][1][c], y);
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                x[q] = mul_f16x2(x[q], s2[g][0]);
                y[q] = mul_f16x2(y[q], s2[g][1]);
              }
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t a[4] = {x[2 * e], y[2 * e], x[2 * e + 1], y[2 * e + 1]};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma_f16_pure(sc[g0 + g][nt], a, qb[nt][2 * c + e][0], qb[nt][2 * c + e][1]);
              }
            }
        }
      }
      // ---- V's codes and scales of the first two groups (with no more of them the
      // slot can be refilled under the softmax and P V)
      uint32_t vw[2][4][VB / 4], sv[2][4];  // of the lane's four keys
      auto load_v = [&](int g0) {
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            lds_words((i & 1 ? at_v1 : at_v0) + stage + C::code_of(g0 + g) + (i & 2 ? 8 * C::ROWB : 0), vw[g][i]);
            sv[g][i] = lds_byte((i & 1 ? at_vs1 : at_vs0) + stage + C::scale_of(g0 + g) + (i & 2 ? 8 * C::SROWB : 0));
          }
        if (g0 + 2 == NG) {
          __syncwarp();  // every lane has read the slot
          if (issued < ntile) issue(issued++, s);
          copies_end();
        }
      };
      load_v(0);
      // ---- scores, masks, online softmax with a lazy maximum (it moves when it
      // grows by more than 2^8, so that weights stay within 2^8)
      auto key_at = [&](int g, int e) { return t_warp + 16 * g + kr + (e < 2 ? 0 : 8); };
      if constexpr (MODS) {
        if (p.cap_log2 > 0.f) {
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) sc[g][nt][e] = capped<FAR>(sc[g][nt][e], qk_mult, p.cap_log2, poly);
        }
        if (p.slopes != nullptr) {
          const float mult = p.cap_log2 > 0.f ? 1.f : qk_mult;
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                sc[g][nt][e] = fmaf(sc[g][nt][e], mult, slope[nt][e & 1] * static_cast<float>(key_at(g, e) - pos[nt][e & 1]));
        }
      }
      const bool whole = (t_warp + C::KEYS - 1 <= hi_all && t_warp >= lo_all) || t_warp + C::KEYS <= pf_all;
      if (!whole) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int t = key_at(g, e), x = e & 1;
              if (!((t <= pos[nt][x] && t >= lo[nt][x]) || t < pf[nt][x])) sc[g][nt][e] = -CUDART_INF_F;
            }
        }
      }
      // (-inf: nothing seen yet, any seen key moves it)
      float mx[NT][2];
      bool up = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(sc[0][nt][e], sc[0][nt][e + 2]);
#pragma unroll
          for (int g = 1; g < NG; ++g) x = fmaxf(x, fmaxf(sc[g][nt][e], sc[g][nt][e + 2]));
          mx[nt][e] = ex_mult * x;
          up = up || mx[nt][e] > m[nt][e] + 8.f;
        }
      if (__any_sync(kFull, up)) {  // rare: only then the rows' maxima are put together
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = mx[nt][e];
#pragma unroll
            for (int sh = 4; sh < 32; sh <<= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, sh));
            const bool moves = x > m[nt][e] + 8.f;
            const float al = moves ? fast_exp2(m[nt][e] - x) : 1.f;
            if (moves) m[nt][e] = x;
            l[nt][e] *= al;
#pragma unroll
            for (int mt = 0; mt < KS; ++mt) {
              o[nt][mt][e] *= al;
              o[nt][mt][e + 2] *= al;
            }
          }
      }
      uint32_t pb[NG][NT][2];  // P^T as the second operand
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float mu[2] = {m[nt][0] == -CUDART_INF_F ? 0.f : m[nt][0], m[nt][1] == -CUDART_INF_F ? 0.f : m[nt][1]};
#pragma unroll
        for (int g = 0; g < NG; ++g) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[g][nt][e] = fast_exp2(fmaf(sc[g][nt][e], ex_mult, -mu[e & 1]));
          l[nt][0] += sc[g][nt][0] + sc[g][nt][2];
          l[nt][1] += sc[g][nt][1] + sc[g][nt][3];
          pb[g][nt][0] = movmatrix_trans(pack_f16x2(sc[g][nt][0], sc[g][nt][1]));
          pb[g][nt][1] = movmatrix_trans(pack_f16x2(sc[g][nt][2], sc[g][nt][3]));
        }
      }
      // ---- O^T += V^T P^T: product mt's rows r and r + 8 are d = r D / 8 + 2 mt and + 1
#pragma unroll
      for (int g0 = 0; g0 < NG; g0 += 2) {
        if (g0 > 0) load_v(g0);
        if (!whole) {  // keys past the sequence's end (a row that sees them all there is none): zeros
#pragma unroll
          for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (t_warp + 16 * (g0 + g) + (i & 1 ? kv1 : kv0) + (i & 2 ? 8 : 0) >= sq.ctx) sv[g][i] = 0u;
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const uint32_t s01 = e4m3x2_to_f16x2(static_cast<uint16_t>(prmt(sv[g][0], sv[g][1], 0x0040u))),
                         s23 = e4m3x2_to_f16x2(static_cast<uint16_t>(prmt(sv[g][2], sv[g][3], 0x0040u)));
#pragma unroll
          for (int q = 0; q < VB / 4; ++q) {
            // bytes of a pair of keys at one d: its even d, and its odd ones
            uint32_t x[2][2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t ka = vw[g][2 * i][q], kb = vw[g][2 * i + 1][q];
              e2m1x8_to_f16x2(bit_select(0x0F0F0F0Fu, ka, kb << 4), x[i][0]);
              e2m1x8_to_f16x2(bit_select(0x0F0F0F0Fu, ka >> 4, kb), x[i][1]);
            }
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
              const uint32_t a[4] = {mul_f16x2(x[0][0][mt], s01), mul_f16x2(x[0][1][mt], s01),
                                     mul_f16x2(x[1][0][mt], s23), mul_f16x2(x[1][1][mt], s23)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16_pure(o[nt][4 * q + mt], a, pb[g0 + g][nt][0], pb[g0 + g][nt][1]);
            }
          }
        }
      }
    }
    if (++s == NS) s = 0;
  }
  allow_next_grid();

  // ---- row sums over the lanes that share a row; the warps' results merge through shared memory
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int sh = 4; sh < 32; sh <<= 1) l[nt][e] += __shfl_xor_sync(kFull, l[nt][e], sh);
  __syncthreads();  // every warp is done with the stages
  float* s_o = reinterpret_cast<float*>(smem);  // [WARPS][R][DP]
  float* s_ml = s_o + WARPS * C::R * DP;        // [WARPS][R][2]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = 8 * nt + 2 * j + e;
      float* to = s_o + (warp * C::R + row) * DP + r * (D / 8);
#pragma unroll
      for (int mt = 0; mt < KS; mt += 2)
        *reinterpret_cast<float4*>(to + 2 * mt) =
            make_float4(o[nt][mt][e], o[nt][mt][e + 2], o[nt][mt + 1][e], o[nt][mt + 1][e + 2]);
      if (r == 0) {
        s_ml[(warp * C::R + row) * 2] = m[nt][e];
        s_ml[(warp * C::R + row) * 2 + 1] = l[nt][e];
      }
    }
  __syncthreads();

  for (int idx = threadIdx.x; idx < rows * (D / 2); idx += blockDim.x) {
    const int row = idx / (D / 2), d = 2 * (idx - row * (D / 2));
    float M = -CUDART_INF_F;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) M = fmaxf(M, s_ml[(w * C::R + row) * 2]);
    float a0 = 0.f, a1 = 0.f, lsum = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float2 ml = *reinterpret_cast<const float2*>(s_ml + (w * C::R + row) * 2);
      const float wt = ml.x == -CUDART_INF_F ? 0.f : fast_exp2(ml.x - M);
      const float2 v = *reinterpret_cast<const float2*>(s_o + (w * C::R + row) * DP + d);
      a0 += wt * v.x;
      a1 += wt * v.y;
      lsum += wt * ml.y;
    }
    const int64_t orow = out_row(row);
    if (nsplit == 1) {
      const float inv = lsum > 0.f ? v_mult / lsum : 0.f;
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + orow * D + d) = pack_bf16x2(a0 * inv, a1 * inv);
    } else {
      const int64_t slot = orow * p.max_splits + split;
      *reinterpret_cast<float2*>(p.ws_o + slot * D + d) = make_float2(a0 * v_mult, a1 * v_mult);
      if (d == 0) {
        p.ws_ml[slot * 2] = M;
        p.ws_ml[slot * 2 + 1] = lsum;
      }
    }
  }
}

template <int D, int NT, int BS, bool MODS, bool FAR>
cudaError_t launch_t(const ChunkParams& p, cudaStream_t stream) {
  using C = E2M1Shape<D, NT, BS>;
  auto kern = chunk_e2m1_kernel<D, NT, BS, MODS, FAR>;
  static int configured[64] = {};
  cudaError_t e = set_smem_once(kern, C::BYTES, configured);
  if (e != cudaSuccess) return e;
  const int ntq = (p.max_q_len + p.tile_q - 1) / p.tile_q;
  return launch_pdl(kern, dim3(p.max_splits, p.num_kv_heads * ntq, p.batch), dim3(C::THREADS), C::BYTES, stream, p);
}

template <int D, int NT, int BS>
cudaError_t launch_n(const ChunkParams& p, cudaStream_t stream) {
  if (p.cap_far) return launch_t<D, NT, BS, true, true>(p, stream);
  return p.cap_log2 > 0.f || p.slopes != nullptr ? launch_t<D, NT, BS, true, false>(p, stream)
                                                 : launch_t<D, NT, BS, false, false>(p, stream);
}

template <int D, int NT>
cudaError_t launch_b(const ChunkParams& p, cudaStream_t stream) {
  return p.block_size == 16 ? launch_n<D, NT, 16>(p, stream) : launch_n<D, NT, 32>(p, stream);
}

template <int D>
cudaError_t launch_d(const ChunkParams& p, cudaStream_t stream) {
  return p.max_q_len * p.group > 8 ? launch_b<D, 2>(p, stream) : launch_b<D, 1>(p, stream);
}

}  // namespace

cudaError_t launch_chunk_e2m1(const ChunkParams& p, cudaStream_t stream) {
  return p.head_dim == 128 ? launch_d<128>(p, stream) : launch_d<64>(p, stream);
}

}  // namespace pkv
