// Attention of ragged chunks over E2M1 caches, row tiles of up to 16 rows (single
// tokens of up to 16 query heads per KV head, a few tokens of smaller groups);
// what it computes: chunk_common.cuh, what a cache holds: pkv.h.
//
// A CTA takes the rows of one tile of one (sequence, KV head) over one split of
// its visible keys, in 128-key steps: warp w loads keys 32w..32w+31 of every
// step by TMA (a box of codes and a box of scales per block, of K and of V) into
// a ring of its own on barriers of its own, and refills a slot as soon as it has
// read it; the warps merge (m, l, O) through shared memory at the end.
//
// Both products have keys as the first operand's rows or columns and up to 8
// tile rows as the second's columns (NT of them: 1 or 2), mma.sync m16n8k16 of
// f16 with fp32 sums, so that the codes, widened once, serve every row:
//   S^T = K Q^T.  A lane's word of an ldmatrix row is 8 codes of one key: two
//     products' worth, whose order of d is Q's to follow.  cvt makes f16 pairs of
//     its bytes, which are multiplied by the key's scale of that group, in pairs
//     too: exact, so S is that of the cache's values.
//   O^T += V^T P^T.  A lane needs pairs of keys at one d where the cache has
//     pairs of d of one key: it reads the same D / 8 d of its four keys and swaps
//     halves of their bytes before it widens them (a shift and a select for four
//     pairs).  All of them lie in one group, so that a pair of keys has one pair
//     of scales.
// Keys take the products' rows in an order (key_of) that keeps those reads free
// of bank conflicts.  P is rounded to f16: at most 2^-11 of each weight, next to
// the output's own 2^-8.  V past the sequence's end has scale 0 (its codes are
// finite whatever they are).

#include "chunk_common.cuh"

namespace pkv {
namespace {

template <int D, int NT>
struct E2M1Shape {
  static constexpr int STEP = kChunkE2M1Tile, KEYS = STEP / 4;  // keys of a step, and of a warp
  static constexpr int ROWB = D / 2, SROWB = D / 16;      // bytes of a row's codes and scales
  static constexpr int CODEB = KEYS * ROWB;               // codes of K (or V) of a warp's step
  static constexpr int SCALEB = 256;                      // its scales: boxes of 64 bytes or more, 128 apart
  static constexpr int CTAS = chunk_e2m1_ctas(D, NT == 1);
  static constexpr int NS = D == 128 ? 2 : 4;
  static constexpr int STAGE = 4 * 2 * CODEB;
  static constexpr int DP = D + 4, R = 8 * NT;
  static constexpr int MERGE = 4 * R * DP * 4 + 4 * R * 2 * 4;
  static constexpr int RING = NS * (STAGE + 4 * 2 * SCALEB);
  static constexpr int BYTES = (RING > MERGE ? RING : MERGE) + 4 * NS * 8 + kChunkMaxSplitBlocks * 4 + 1024;
};

// Key of a 16-key group that is row i of the products.  128-wide heads: rows
// 2 j and 2 j + 1 are keys {0, 1, 4, 5}[j] and {2, 3, 6, 7}[j], 64-wide ones: j
// and j + 4.
template <int D>
__device__ __forceinline__ int key_of(int i) {
  return D == 128 ? (i & 12) | ((i & 1) << 1) | ((i >> 1) & 1) : (i & 8) | ((i & 1) << 2) | ((i >> 1) & 3);
}

// MODS: scores that are capped or biased.  FAR: a cap above kCapNear.
template <int D, int NT, bool MODS, bool FAR>
__global__ void __launch_bounds__(128, E2M1Shape<D, NT>::CTAS)
    chunk_e2m1_kernel(const __grid_constant__ ChunkMaps maps, const ChunkParams p) {
  using C = E2M1Shape<D, NT>;
  constexpr int NS = C::NS, DP = C::DP, KS = D / 16, CH = D / 32;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, j = lane & 3;
  const int G = p.group, H_q = p.num_q_heads;
  const int ntq = (p.max_q_len + p.tile_q - 1) / p.tile_q;
  const int h = blockIdx.y / ntq;
  const int i0 = (blockIdx.y - h * ntq) * p.tile_q;
  const int b = blockIdx.z, split = blockIdx.x;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + (C::RING > C::MERGE ? C::RING : C::MERGE));  // [NS][4]
  int* s_blk = reinterpret_cast<int*>(full + 4 * NS);
  // stage s of this warp: codes of K and of V, scales of K and of V
  const uint32_t codes0 = smem_u32(smem) + warp * 2 * C::CODEB;
  const uint32_t scales0 = smem_u32(smem) + NS * C::STAGE + warp * 2 * C::SCALEB;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 4 * NS; ++s) mbar_init(smem_u32(full + s), 1);
    fence_mbar_init();
    prefetch_tmap(&maps.k);
    prefetch_tmap(&maps.v);
    prefetch_tmap(&maps.k_scales);
    prefetch_tmap(&maps.v_scales);
  }
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
  const int bshift = p.block_size == 16 ? 4 : 5;
  const int per_tile = C::STEP >> bshift;
  const int32_t* tbl = p.block_tables + static_cast<int64_t>(b) * p.max_blocks;
  for (int i = threadIdx.x; i < ntile * per_tile; i += blockDim.x) {
    const int t0 = rg.tile(k0 + i / per_tile) * C::STEP + (i % per_tile) * p.block_size;
    int phys = -1;  // outside the tensor map: the TMA unit fills zeros
    if (rg.sees(t0, t0 + p.block_size)) {
      phys = tbl[t0 >> bshift];
      if (phys < 0 || phys >= p.num_blocks) {
        record_error(p.err, kDevErrBlockId);
        phys = -1;
      }
    }
    s_blk[i] = phys;
  }
  __syncthreads();

  // a warp's 32 keys are one or two blocks: lane 4 bx + w loads block bx of codes
  // of K, of V, scales of K, of V
  const int nbox = C::KEYS >> bshift;
  const int box_scales = p.block_size * C::SROWB < 128 ? 128 : p.block_size * C::SROWB;
  const int group_scales = bshift == 4 ? box_scales : 16 * C::SROWB;  // from a 16-key group's scales to the next's
  const int what = lane & 3, bx = lane >> 2;
  const CUtensorMap* tmap = what == 0 ? &maps.k : (what == 1 ? &maps.v : (what == 2 ? &maps.k_scales : &maps.v_scales));
  const uint32_t box_to = what < 2 ? codes0 + what * C::CODEB + bx * p.block_size * C::ROWB
                                   : scales0 + (what - 2) * C::SCALEB + bx * box_scales;
  const uint32_t stage_step = what < 2 ? C::STAGE : 4 * 2 * C::SCALEB;
  const uint32_t bar0 = smem_u32(full) + 8 * warp;  // of stage 0; 32 bytes on to the next stage's
  const uint32_t blk0 = smem_u32(s_blk) + 4 * (((warp * C::KEYS) >> bshift) + bx);
  auto issue = [&](int k, int s) {  // step k into stage s
    if (lane == 0) {
      fence_proxy_async_smem();  // this warp's reads of the slot come before the copy
      mbar_arrive_expect_tx(bar0 + 32 * s, 2 * C::KEYS * (C::ROWB + C::SROWB));
    }
    __syncwarp();
    if (bx < nbox) {
      uint32_t phys[1];
      lds_words(blk0 + k * (4 * per_tile), phys);
      tma_load_4d(box_to + s * stage_step, tmap, bar0 + 32 * s, 0, 0, h, static_cast<int>(phys[0]));
    }
  };
  int issued = 0;
  for (; issued < ntile && issued < NS; ++issued) issue(issued, issued);

  // Q as the second operand: row r of each n-tile; chunk c of 32 d is two
  // products, of the lane's d 32 c + 8 j + 0..3 and + 4..7
  uint32_t qb[NT][KS][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = 8 * nt + r;
    const uint16_t* q = static_cast<const uint16_t*>(p.q) + out_row(row) * D;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const uint4 w = row < rows ? *reinterpret_cast<const uint4*>(q + 32 * c + 8 * j) : make_uint4(0u, 0u, 0u, 0u);
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

  // K by ldmatrix: keys key_of(0-7), chunk 2 i; key_of(8-15), chunk 2 i; the same of chunk 2 i + 1
  const int key_k = key_of<D>((lane & 7) + ((lane >> 3) & 1) * 8), ch_k = lane >> 4;
  auto code_at = [](int key, int chunk) {  // 16-byte chunk of a row, as the TMA unit stores it
    return static_cast<uint32_t>(key * C::ROWB + ((chunk ^ (D == 128 ? (key >> 1) & 3 : (key >> 2) & 1)) << 4));
  };
  const uint32_t at_k = codes0 + code_at(key_k, ch_k);  // chunks 2 i + ch_k: the address with bit 5 flipped for i = 1
  // V: this lane's keys of the products' columns 2 j, 2 j + 1, 2 j + 8, 2 j + 9
  // (the last two: 8 rows on), and its D / 8 d of them
  const int kv0 = key_of<D>(2 * j), kv1 = key_of<D>(2 * j + 1);
  constexpr int VB = D / 16;                       // their code bytes
  const uint32_t v_in = D == 128 ? (r & 1) * 8 : (r & 3) * 4;
  const uint32_t at_v0 = codes0 + C::CODEB + code_at(kv0, D == 128 ? r >> 1 : r >> 2) + v_in,
                 at_v1 = codes0 + C::CODEB + code_at(kv1, D == 128 ? r >> 1 : r >> 2) + v_in;
  const int kr = key_of<D>(r);                     // key of score rows r (and r + 8, eight further)
  const uint32_t at_ks = scales0 + kr * C::SROWB, at_vs = scales0 + C::SCALEB + (D == 128 ? r : r >> 1);
  const uint32_t at_vs0 = at_vs + kv0 * C::SROWB, at_vs1 = at_vs + kv1 * C::SROWB;
  const uint32_t sel = j < 2 ? 0x2200u : 0x3311u;  // of four groups' scales those of the lane's d, each twice

  bool healthy = true;
  int s = 0;
  uint32_t parity = 0;
  for (int k = 0; k < ntile; ++k) {
    const bool arrived = mbar_wait(bar0 + 32 * s, parity, p.err);
    if (!__all_sync(kFull, arrived)) healthy = false;
    const uint32_t code_s = s * C::STAGE, scale_s = s * (4 * 2 * C::SCALEB);
    const int t_warp = rg.tile(k0 + k) * C::STEP + warp * C::KEYS;  // this warp's first key
    if (healthy) {
      // ---- S^T of two groups of 16 keys: rows r, r + 8 (e >= 2) are keys kr and
      // kr + 8, columns 2 j, 2 j + 1 (odd e)
      uint32_t kw[2][CH / 2][4], ksw[2][2][CH / 2];  // codes; scale codes of keys kr and kr + 8
#pragma unroll
      for (int g = 0; g < 2; ++g) {
#pragma unroll
        for (int e = 0; e < 2; ++e) lds_words(at_ks + scale_s + g * group_scales + 8 * e * C::SROWB, ksw[g][e]);
#pragma unroll
        for (int i = 0; i < CH / 2; ++i) ldsm_x4((at_k ^ (32 * i)) + code_s + g * 16 * C::ROWB, kw[g][i]);
      }
      float sc[2][NT][4];
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) sc[g][nt][0] = sc[g][nt][1] = sc[g][nt][2] = sc[g][nt][3] = 0.f;
#pragma unroll
      for (int i = 0; i < CH / 2; ++i)
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          const int c = 2 * i + cc;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            uint32_t x[4], y[4];  // of keys kr and kr + 8
            e2m1x8_to_f16x2(kw[g][i][2 * cc], x);
            e2m1x8_to_f16x2(kw[g][i][2 * cc + 1], y);
            // their scale pairs of the group that holds the lane's eight d
            const uint32_t sx = e4m3x2_to_f16x2(static_cast<uint16_t>(prmt(ksw[g][0][i], 0u, sel) >> (16 * cc))),
                           sy = e4m3x2_to_f16x2(static_cast<uint16_t>(prmt(ksw[g][1][i], 0u, sel) >> (16 * cc)));
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              x[q] = mul_f16x2(x[q], sx);
              y[q] = mul_f16x2(y[q], sy);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t a[4] = {x[2 * e], y[2 * e], x[2 * e + 1], y[2 * e + 1]};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_f16_pure(sc[g][nt], a, qb[nt][2 * c + e][0], qb[nt][2 * c + e][1]);
            }
          }
        }
      // ---- V's codes and scales: the slot can be refilled under the softmax and P V
      uint32_t vw[2][4][VB / 4], sv[2][4];  // of the lane's four keys
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lds_words((i & 1 ? at_v1 : at_v0) + code_s + g * 16 * C::ROWB + (i & 2 ? 8 * C::ROWB : 0), vw[g][i]);
          sv[g][i] = lds_byte((i & 1 ? at_vs1 : at_vs0) + scale_s + g * group_scales + (i & 2 ? 8 * C::SROWB : 0));
        }
      __syncwarp();
      if (issued < ntile) issue(issued++, s);
      // ---- scores, masks, online softmax with a lazy maximum (it moves when it
      // grows by more than 2^8, so that weights stay within 2^8)
      auto key_at = [&](int g, int e) { return t_warp + 16 * g + kr + (e < 2 ? 0 : 8); };
      if constexpr (MODS) {
        if (p.cap_log2 > 0.f) {
#pragma unroll
          for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) sc[g][nt][e] = capped<FAR>(sc[g][nt][e], qk_mult, p.cap_log2, poly);
        }
        if (p.slopes != nullptr) {
          const float mult = p.cap_log2 > 0.f ? 1.f : qk_mult;
#pragma unroll
          for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                sc[g][nt][e] = fmaf(sc[g][nt][e], mult, slope[nt][e & 1] * static_cast<float>(key_at(g, e) - pos[nt][e & 1]));
        }
      }
      if (!((t_warp + C::KEYS - 1 <= hi_all && t_warp >= lo_all) || t_warp + C::KEYS <= pf_all)) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int t = key_at(g, e), x = e & 1;
              if (!((t <= pos[nt][x] && t >= lo[nt][x]) || t < pf[nt][x])) sc[g][nt][e] = -CUDART_INF_F;
            }
          // (a key past the sequence's end is seen by no row, so that this is reached)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (t_warp + 16 * g + (i & 1 ? kv1 : kv0) + (i & 2 ? 8 : 0) >= sq.ctx) sv[g][i] = 0u;
        }
      }
      // (-inf: nothing seen yet, any seen key moves it)
      float mx[NT][2];
      bool up = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[nt][e] = ex_mult * fmaxf(fmaxf(sc[0][nt][e], sc[0][nt][e + 2]), fmaxf(sc[1][nt][e], sc[1][nt][e + 2]));
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
      uint32_t pb[2][NT][2];  // P^T as the second operand
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float mu[2] = {m[nt][0] == -CUDART_INF_F ? 0.f : m[nt][0], m[nt][1] == -CUDART_INF_F ? 0.f : m[nt][1]};
#pragma unroll
        for (int g = 0; g < 2; ++g) {
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
            for (int nt = 0; nt < NT; ++nt) mma_f16_pure(o[nt][4 * q + mt], a, pb[g][nt][0], pb[g][nt][1]);
          }
        }
      }
    }
    if (++s == NS) {
      s = 0;
      parity ^= 1u;
    }
  }
  if (!healthy && lane == 0) {
    // a copy of this warp's may still be landing: one more bounded wait each
    for (int kk = issued > NS ? issued - NS : 0; kk < issued; ++kk)
      mbar_wait(bar0 + 32 * (kk % NS), static_cast<uint32_t>((kk / NS) & 1), nullptr);
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
  float* s_o = reinterpret_cast<float*>(smem);  // [4 warps][R][DP]
  float* s_ml = s_o + 4 * C::R * DP;            // [4 warps][R][2]
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
    for (int w = 0; w < 4; ++w) M = fmaxf(M, s_ml[(w * C::R + row) * 2]);
    float a0 = 0.f, a1 = 0.f, lsum = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
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

template <int D, int NT, bool MODS, bool FAR>
cudaError_t launch_t(const ChunkParams& p, const ChunkMaps& m, cudaStream_t stream) {
  auto kern = chunk_e2m1_kernel<D, NT, MODS, FAR>;
  constexpr int smem = E2M1Shape<D, NT>::BYTES;
  static int configured[64] = {};
  cudaError_t e = set_smem_once(kern, smem, configured);
  if (e != cudaSuccess) return e;
  const int ntq = (p.max_q_len + p.tile_q - 1) / p.tile_q;
  return launch_pdl(kern, dim3(p.max_splits, p.num_kv_heads * ntq, p.batch), dim3(128), smem, stream, m, p);
}

template <int D, int NT>
cudaError_t launch_n(const ChunkParams& p, const ChunkMaps& m, cudaStream_t stream) {
  if (p.cap_far) return launch_t<D, NT, true, true>(p, m, stream);
  return p.cap_log2 > 0.f || p.slopes != nullptr ? launch_t<D, NT, true, false>(p, m, stream)
                                                 : launch_t<D, NT, false, false>(p, m, stream);
}

template <int D>
cudaError_t launch_d(const ChunkParams& p, const ChunkMaps& m, cudaStream_t stream) {
  return p.max_q_len * p.group > 8 ? launch_n<D, 2>(p, m, stream) : launch_n<D, 1>(p, m, stream);
}

}  // namespace

cudaError_t launch_chunk_e2m1(const ChunkParams& p, const ChunkMaps& m, cudaStream_t stream) {
  return p.head_dim == 128 ? launch_d<128>(p, m, stream) : launch_d<64>(p, m, stream);
}

}  // namespace pkv
