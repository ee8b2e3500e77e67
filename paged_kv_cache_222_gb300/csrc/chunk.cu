// Attention of ragged chunks of new tokens over the paged cache ([SC] "LLM
// inference: prefill, decode, KV cache", "9. Failure modes and limitations",
// item 3: chunked prefill beside decode steps; "4. Internal workings", step 4
// for chunks of one token), with scores that are capped, biased by distance,
// windowed or opened for a prefix (chunk_common.cuh).
//
// This file: the kernel for row tiles of up to 16 rows (a row is a new token
// and a query head of one KV head), and the merge of split pieces.
//
// A CTA takes the up to 16 rows of one tile of one (sequence, KV head) over
// one split of the tile's visible keys, in 64-key steps: warp w loads keys
// 16w..16w+15 of every step by TMA into its own part of a ring (K and V, one
// box of 16 tokens per lane and 128-byte column band), on barriers of its
// own, and refills its slot as soon as it has read it, so that no warp waits
// for another; the warps merge (m, l, O) through shared memory at the end.
// The products are mma.sync m16n8k16 products with fp32 sums: bf16
// for bf16 caches, f16 for E4M3 ones (every code is an f16).  P is rounded to
// that type: at most 2^-8 (bf16) or 2^-11 (f16) of each weight, next to the
// output's own 2^-8.  Bound: the HBM stream of 2 D bytes x type size per visible
// key and KV head.  64 sequences of 512-8192 tokens, 64 + 8 heads of 128, bf16,
// capped scores: 188-191 us with the merge, 6.5 TB/s, 96-97 % of the measured
// copy; 256 sequences of 1040 visible tokens in E4M3: 100 us, 5.5 TB/s, 82 %.
// There a call costs 18 us besides its stream, whatever the window: a CTA's
// first loads and the merge of its four warps, which CTAs that stream E4M3 are
// too busy to make up for (in bf16 it is 5 us).

#include <type_traits>

#include "chunk_common.cuh"

namespace pkv {
namespace {

constexpr int kSmallTile = kChunkSmallTile;  // keys per step

// CTAs per SM, and a ring that lets them fit: the smaller a row, the more of a
// CTA's life is its start and its merge, which others have to stream under.
// Up to 8 rows leave registers for four (E4M3 of 128 or bf16 of 64 wide: 256
// sequences of 1024 visible keys 102 -> 100 us and 90.8 -> 88, of 512 64 -> 59) or five
// (E4M3 of 64 wide: 78 -> 61, four 66), with two stages of bf16 rows of 128 three.
template <int D, bool FP8, bool TWO>
struct SmallShape {
  using L = Layout<D, FP8>;
  static constexpr int STAGE = 4 * L::STAGEB;             // 64 keys of K and V
  static constexpr int CTAS = chunk_small_ctas(D, FP8, !TWO);
  static constexpr int NS = (CTAS == 3 ? 65536 : (CTAS == 4 ? 49152 : 32768)) / STAGE;
  static constexpr int DP = D + 4;
  static constexpr int BYTES = NS * STAGE + 4 * NS * 8 + kChunkMaxSplitBlocks * 4 + 1024;
  static_assert(4 * 16 * DP * 4 + 4 * 16 * 2 * 4 <= NS * STAGE, "merge buffer fits the stages");
};

// TWO: tiles of more than 8 rows, S = Q K^T and O += P V with a lane's rows r
// and r + 8.  Up to 8 rows: the products transposed.  FAR: a cap above kCapNear.
template <int D, bool FP8, bool TWO, bool FAR>
__global__ void __launch_bounds__(128, SmallShape<D, FP8, TWO>::CTAS)
    chunk_small_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                       const ChunkParams p) {
  using L = Layout<D, FP8>;
  using C = SmallShape<D, FP8, TWO>;
  constexpr int KS = D / 16, NS = C::NS, STAGE = C::STAGE, DP = C::DP;
  // Up to 8 rows: S^T = K Q^T and O^T += V^T P^T, keys as the products' 16 rows
  // and tile rows as their 8 columns: half as many products as the other form,
  // which leaves half of its 16 rows empty, and half the registers of O (256
  // sequences of 1040 visible tokens: E4M3 112 -> 104 us; 1024 in bf16 165 -> 164, three CTAs per SM each).
  constexpr bool TR = !TWO;

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
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + NS * STAGE);  // [NS][4]: per stage and warp
  int* s_blk = reinterpret_cast<int*>(full + 4 * NS);
  const uint32_t stage0 = smem_u32(smem);

  if (threadIdx.x == 0) {
    for (int s = 0; s < 4 * NS; ++s) mbar_init(smem_u32(full + s), 1);
    fence_mbar_init();
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
  }
  wait_prior_grid();

  const ChunkSeq sq = chunk_seq(p, b, split == 0 && blockIdx.y == 0 && threadIdx.x == 0);
  if (i0 >= sq.n) return;
  const int i1 = min(sq.n, i0 + p.tile_q) - 1;
  const int rows = (i1 - i0 + 1) * G;
  const ChunkRange rg = chunk_range<kSmallTile>(p, sq, i0, i1);
  const ChunkSplit sp(rg.n, p.split_tokens / kSmallTile, split);
  const int nsplit = sp.nsplit, k0 = sp.k0, ntile = sp.ntile;
  if (split >= nsplit) return;
  const int64_t row_base = static_cast<int64_t>(sq.start + i0) * H_q + h * G;  // of row (0, g = 0)
  auto out_row = [&](int row) { return row_base + static_cast<int64_t>(row / G) * H_q + row % G; };

  // block ids of the split's keys; blocks that no row sees (behind the window,
  // past the last query) are not looked up and read as zeros
  const int bshift = p.block_size == 16 ? 4 : 5;
  const int per_tile = kSmallTile >> bshift;
  const int32_t* tbl = p.block_tables + static_cast<int64_t>(b) * p.max_blocks;
  for (int i = threadIdx.x; i < ntile * per_tile; i += blockDim.x) {
    const int t0 = rg.tile(k0 + i / per_tile) * kSmallTile + (i % per_tile) * p.block_size;
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

  auto issue = [&](int k) {
    const int s = k % NS;
    const uint32_t dst = stage0 + s * STAGE + warp * L::STAGEB;
    const uint32_t bar = smem_u32(full + 4 * s + warp);
    if (lane == 0) {
      fence_proxy_async_smem();  // this warp's reads of the slot come before the copy
      mbar_arrive_expect_tx(bar, L::STAGEB);
    }
    __syncwarp();
    if (lane < 2 * L::NBOX) {
      const int v = lane / L::NBOX, bx = lane % L::NBOX;
      const int o = warp * kTileTokens;  // token within the 64-key step
      tma_load_4d(dst + v * L::TILEB + bx * L::BOX_BYTES, v ? &tmap_v : &tmap_k, bar, bx * L::BOX_ELEMS,
                  o & (p.block_size - 1), h, s_blk[k * per_tile + (o >> bshift)]);
    }
  };
  int issued = 0;
  for (; issued < ntile && issued < NS; ++issued) issue(issued);

  // this lane's two rows of the tile: r, r + 8 (transposed: 2 j, 2 j + 1; its
  // fragments of Q still hold row r)
  const int ra = TR ? 2 * j : r, rb = TR ? 2 * j + 1 : r + 8;
  uint32_t qa[KS][4];
  {
    const uint16_t* q = static_cast<const uint16_t*>(p.q);
    const uint16_t* qra = r < rows ? q + out_row(r) * D : nullptr;
    const uint16_t* qrb = TWO && r + 8 < rows ? q + out_row(r + 8) * D : nullptr;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      if constexpr (!FP8) {
        const int d0 = 16 * ks + 2 * j;
        qa[ks][0] = qra ? *reinterpret_cast<const uint32_t*>(qra + d0) : 0u;
        qa[ks][1] = qrb ? *reinterpret_cast<const uint32_t*>(qrb + d0) : 0u;
        qa[ks][2] = qra ? *reinterpret_cast<const uint32_t*>(qra + d0 + 8) : 0u;
        qa[ks][3] = qrb ? *reinterpret_cast<const uint32_t*>(qrb + d0 + 8) : 0u;
      } else {  // f16, in the d-order of the widened E4M3 fragments
        const int d0 = 16 * ks + 4 * j;
        const uint2 wa = qra ? *reinterpret_cast<const uint2*>(qra + d0) : make_uint2(0u, 0u);
        const uint2 wb = qrb ? *reinterpret_cast<const uint2*>(qrb + d0) : make_uint2(0u, 0u);
        qa[ks][0] = pack_f16x2(bf16lo_to_f32(wa.x), bf16hi_to_f32(wa.x));
        qa[ks][1] = pack_f16x2(bf16lo_to_f32(wb.x), bf16hi_to_f32(wb.x));
        qa[ks][2] = pack_f16x2(bf16lo_to_f32(wa.y), bf16hi_to_f32(wa.y));
        qa[ks][3] = pack_f16x2(bf16lo_to_f32(wb.y), bf16hi_to_f32(wb.y));
      }
    }
  }
  // per row: position (-1 where it sees nothing), first key of the window
  auto pos_of = [&](int row) { return row < rows ? sq.ctx - sq.n + i0 + row / G : -1; };
  const int pos_a = pos_of(ra), pos_b = pos_of(rb);
  auto lo_of = [&](int pos) { return p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0; };
  const int lo_a = lo_of(pos_a), lo_b = lo_of(pos_b);
  const int pf_a = pos_a >= 0 ? sq.prefix : 0, pf_b = pos_b >= 0 ? sq.prefix : 0;
  constexpr float kLog2e = 1.4426950408889634f;
  float sl_a = 0.f, sl_b = 0.f;
  if (p.slopes != nullptr) {
    sl_a = ra < rows ? p.slopes[h * G + ra % G] * kLog2e : 0.f;
    sl_b = rb < rows ? p.slopes[h * G + rb % G] * kLog2e : 0.f;
  }
  float qk_mult = p.qk_log2, v_mult = 1.f;
  if constexpr (FP8) {
    qk_mult *= p.k_scale[static_cast<int64_t>(b) * p.scale_stride + h];
    v_mult = p.v_scale[static_cast<int64_t>(b) * p.scale_stride + h];
  }

  const CapPoly<FAR> poly(qk_mult, p);
  const float ex_mult = p.cap_log2 > 0.f || p.slopes != nullptr ? 1.f : qk_mult;  // scores to log2 weights

  float m_a = -CUDART_INF_F, m_b = -CUDART_INF_F, l_a = 0.f, l_b = 0.f;
  constexpr int NO = TR ? D / 16 : D / 8;  // products' accumulators of O
  float o[NO][4];
#pragma unroll
  for (int nt = 0; nt < NO; ++nt) o[nt][0] = o[nt][1] = o[nt][2] = o[nt][3] = 0.f;
  // ldmatrix lanes: K (tok 0-7,c)(tok 0-7,c+1)(tok 8-15,c)(tok 8-15,c+1);
  //                 V (tok 0-7,c)(tok 8-15,c)(tok 0-7,c+1)(tok 8-15,c+1)
  const int mq = lane >> 3;
  const int tok_k = (lane & 7) + (mq >> 1) * 8, ch_k = mq & 1;
  const int tok_v = (lane & 7) + (mq & 1) * 8, ch_v = mq >> 1;

  bool healthy = true;
  for (int k = 0; k < ntile; ++k) {
    const int s = k % NS;
    const bool arrived = mbar_wait(smem_u32(full + 4 * s + warp), static_cast<uint32_t>((k / NS) & 1), p.err);
    if (!__all_sync(kFull, arrived)) healthy = false;
    const uint32_t base = stage0 + s * STAGE + warp * L::STAGEB;
    const int t_warp = rg.tile(k0 + k) * kSmallTile + warp * kTileTokens;  // this warp's first key
    if constexpr (TR) {
      if (healthy) {
        // ---- S^T: keys r, r + 8 (e >= 2) of rows 2 j, 2 j + 1 (odd e), in two
        // accumulators to halve the chain
        float sc[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int pk = 0; pk < (FP8 ? KS / 2 : KS); ++pk) {
          uint32_t Rk[4];
          ldsm_x4(base + L::off(tok_k, 2 * pk + ch_k), Rk);
          if constexpr (!FP8) {
            const uint32_t a[4] = {Rk[0], Rk[2], Rk[1], Rk[3]};
            mma_bf16_16816(pk & 1 ? s2 : sc, a, qa[pk][0], qa[pk][2]);
            continue;
          }
#pragma unroll
          for (int e = 0; FP8 && e < 2; ++e) {  // a 16-byte chunk holds the 16 d of one k-step
            const uint32_t lo = Rk[e], hi = Rk[2 + e];
            const uint32_t a[4] = {e4m3x2_to_f16x2(static_cast<uint16_t>(lo & 0xFFFFu)),
                                   e4m3x2_to_f16x2(static_cast<uint16_t>(hi & 0xFFFFu)),
                                   e4m3x2_to_f16x2(static_cast<uint16_t>(lo >> 16)),
                                   e4m3x2_to_f16x2(static_cast<uint16_t>(hi >> 16))};
            mma_f16_16816(e ? s2 : sc, a, qa[(2 * pk + e) % KS][0], qa[(2 * pk + e) % KS][2]);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[e] += s2[e];
        const int ta = t_warp + r, tb = ta + 8;
        if (p.cap_log2 > 0.f) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[e] = capped<FAR>(sc[e], qk_mult, p.cap_log2, poly);
        }
        if (p.slopes != nullptr) {
          const float m = p.cap_log2 > 0.f ? 1.f : qk_mult;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sc[e] = fmaf(sc[e], m, (e & 1 ? sl_b : sl_a) * static_cast<float>((e < 2 ? ta : tb) - (e & 1 ? pos_b : pos_a)));
        }
        const auto whole = [&](int pos, int lo, int pf) {
          return (t_warp + kTileTokens - 1 <= pos && t_warp >= lo) || t_warp + kTileTokens <= pf;
        };
        if (!__all_sync(kFull, whole(pos_a, lo_a, pf_a) && whole(pos_b, lo_b, pf_b))) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int t = e < 2 ? ta : tb, pos = e & 1 ? pos_b : pos_a, lo = e & 1 ? lo_b : lo_a, pf = e & 1 ? pf_b : pf_a;
            if (!((t <= pos && t >= lo) || t < pf)) sc[e] = -CUDART_INF_F;
          }
        }
        float mx_a = fmaxf(sc[0], sc[2]), mx_b = fmaxf(sc[1], sc[3]);
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) {
          mx_a = fmaxf(mx_a, __shfl_xor_sync(kFull, mx_a, sh));
          mx_b = fmaxf(mx_b, __shfl_xor_sync(kFull, mx_b, sh));
        }
        mx_a *= ex_mult;
        mx_b *= ex_mult;
        const bool up_a = mx_a > m_a + 8.f, up_b = mx_b > m_b + 8.f;  // lazy maximum, as below
        if (__any_sync(kFull, up_a || up_b)) {
          const float al_a = up_a ? fast_exp2(m_a - mx_a) : 1.f, al_b = up_b ? fast_exp2(m_b - mx_b) : 1.f;
          if (up_a) m_a = mx_a;
          if (up_b) m_b = mx_b;
          l_a *= al_a;
          l_b *= al_b;
#pragma unroll
          for (int mt = 0; mt < NO; ++mt) {
            o[mt][0] *= al_a;
            o[mt][1] *= al_b;
            o[mt][2] *= al_a;
            o[mt][3] *= al_b;
          }
        }
        const float mu_a = m_a == -CUDART_INF_F ? 0.f : m_a, mu_b = m_b == -CUDART_INF_F ? 0.f : m_b;
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[e] = fast_exp2(fmaf(sc[e], ex_mult, e & 1 ? -mu_b : -mu_a));
        l_a += sc[0] + sc[2];
        l_b += sc[1] + sc[3];
        // ---- O^T += V^T P^T; rows of the first operand: 16 d, E4M3 the even ones
        // of a 16-d chunk and then the odd ones
        const uint32_t p0 = movmatrix_trans(FP8 ? pack_f16x2(sc[0], sc[1]) : pack_bf16x2(sc[0], sc[1])),
                       p1 = movmatrix_trans(FP8 ? pack_f16x2(sc[2], sc[3]) : pack_bf16x2(sc[2], sc[3]));
        const int vvalid = sq.ctx - t_warp;
        const uint32_t vt = base + L::TILEB;
        const auto add_pv = [&](auto tail) {
          constexpr bool TAIL = decltype(tail)::value;
          const uint32_t keep0 = ((2 * j < vvalid) ? 0x0000FFFFu : 0u) | ((2 * j + 1 < vvalid) ? 0xFFFF0000u : 0u);
          const uint32_t keep1 = ((2 * j + 8 < vvalid) ? 0x0000FFFFu : 0u) | ((2 * j + 9 < vvalid) ? 0xFFFF0000u : 0u);
#pragma unroll
          for (int q = 0; q < (FP8 ? KS / 2 : KS); ++q) {
            uint32_t Rv[4];
            ldsm_x4_trans(vt + L::off(tok_v, 2 * q + ch_v), Rv);
            if constexpr (TAIL) {
              Rv[0] &= keep0;
              Rv[1] &= keep1;
              Rv[2] &= keep0;
              Rv[3] &= keep1;
            }
            if constexpr (!FP8) {
              const uint32_t a[4] = {Rv[0], Rv[2], Rv[1], Rv[3]};
              mma_bf16_16816(o[q], a, p0, p1);
              continue;
            }
#pragma unroll
            for (int e = 0; FP8 && e < 2; ++e) {
              const uint32_t e0 = prmt(Rv[2 * e], 0u, 0x3120u);       // keys 0-7
              const uint32_t e1 = prmt(Rv[2 * e + 1], 0u, 0x3120u);   // keys 8-15
              const uint32_t a[4] = {e4m3x2_to_f16x2(static_cast<uint16_t>(e0 & 0xFFFFu)),
                                     e4m3x2_to_f16x2(static_cast<uint16_t>(e0 >> 16)),
                                     e4m3x2_to_f16x2(static_cast<uint16_t>(e1 & 0xFFFFu)),
                                     e4m3x2_to_f16x2(static_cast<uint16_t>(e1 >> 16))};
              mma_f16_16816(o[(2 * q + e) % NO], a, p0, p1);
            }
          }
        };
        if (vvalid < kTileTokens)
          add_pv(std::true_type{});
        else
          add_pv(std::false_type{});
      }
    } else if (healthy) {
      // ---- S = Q K^T: two 8-key n-tiles
      float sc[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
      if constexpr (!FP8) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          uint32_t Rk[4];
          ldsm_x4(base + L::off(tok_k, 2 * ks + ch_k), Rk);
          mma_bf16_16816(sc[0], qa[ks], Rk[0], Rk[1]);
          mma_bf16_16816(sc[1], qa[ks], Rk[2], Rk[3]);
        }
      } else {  // a 16-byte chunk holds the 16 d of one k-step
#pragma unroll
        for (int pk = 0; pk < KS / 2; ++pk) {
          uint32_t Rk[4];
          ldsm_x4(base + L::off(tok_k, 2 * pk + ch_k), Rk);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mma_f16_16816(sc[0], qa[2 * pk + e], e4m3x2_to_f16x2(static_cast<uint16_t>(Rk[e] & 0xFFFFu)),
                          e4m3x2_to_f16x2(static_cast<uint16_t>(Rk[e] >> 16)));
            mma_f16_16816(sc[1], qa[2 * pk + e], e4m3x2_to_f16x2(static_cast<uint16_t>(Rk[2 + e] & 0xFFFFu)),
                          e4m3x2_to_f16x2(static_cast<uint16_t>(Rk[2 + e] >> 16)));
          }
        }
      }
      // ---- scores, masks, online softmax (rows a: e = 0, 1; b: e = 2, 3).
      // Without cap and bias the multiplier waits for the exponent's FMA.  The
      // maximum is lazy: it moves when it grows by more than 2^8, so weights
      // stay within 2^8 and most steps rescale nothing.
      if (p.cap_log2 > 0.f) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[nt][e] = capped<FAR>(sc[nt][e], qk_mult, p.cap_log2, poly);
      }
      if (p.slopes != nullptr) {
        const float m = p.cap_log2 > 0.f ? 1.f : qk_mult;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int t = t_warp + 8 * nt + 2 * j + (e & 1);
            sc[nt][e] = fmaf(sc[nt][e], m, (e < 2 ? sl_a : sl_b) * static_cast<float>(t - (e < 2 ? pos_a : pos_b)));
          }
      }
      const auto whole = [&](int pos, int lo, int pf) {
        return (t_warp + kTileTokens - 1 <= pos && t_warp >= lo) || t_warp + kTileTokens <= pf;
      };
      if (!__all_sync(kFull, whole(pos_a, lo_a, pf_a) && whole(pos_b, lo_b, pf_b))) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int t = t_warp + 8 * nt + 2 * j + (e & 1);
            const int pos = e < 2 ? pos_a : pos_b, lo = e < 2 ? lo_a : lo_b, pf = e < 2 ? pf_a : pf_b;
            if (!((t <= pos && t >= lo) || t < pf)) sc[nt][e] = -CUDART_INF_F;
          }
      }
      float mx_a = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
      float mx_b = fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3]));
      mx_a = fmaxf(mx_a, __shfl_xor_sync(kFull, mx_a, 1));
      mx_a = fmaxf(mx_a, __shfl_xor_sync(kFull, mx_a, 2)) * ex_mult;
      mx_b = fmaxf(mx_b, __shfl_xor_sync(kFull, mx_b, 1));
      mx_b = fmaxf(mx_b, __shfl_xor_sync(kFull, mx_b, 2)) * ex_mult;
      // (-inf: nothing seen yet, any seen key moves it and there is nothing to rescale)
      const bool up_a = mx_a > m_a + 8.f, up_b = mx_b > m_b + 8.f;
      if (__any_sync(kFull, up_a || up_b)) {
        const float al_a = up_a ? fast_exp2(m_a - mx_a) : 1.f, al_b = up_b ? fast_exp2(m_b - mx_b) : 1.f;
        if (up_a) m_a = mx_a;
        if (up_b) m_b = mx_b;
        l_a *= al_a;
        l_b *= al_b;
#pragma unroll
        for (int nt = 0; nt < D / 8; ++nt) {
          o[nt][0] *= al_a;
          o[nt][1] *= al_a;
          o[nt][2] *= al_b;
          o[nt][3] *= al_b;
        }
      }
      const float mu_a = m_a == -CUDART_INF_F ? 0.f : m_a, mu_b = m_b == -CUDART_INF_F ? 0.f : m_b;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        sc[nt][0] = fast_exp2(fmaf(sc[nt][0], ex_mult, -mu_a));
        sc[nt][1] = fast_exp2(fmaf(sc[nt][1], ex_mult, -mu_a));
        l_a += sc[nt][0] + sc[nt][1];
        sc[nt][2] = fast_exp2(fmaf(sc[nt][2], ex_mult, -mu_b));
        sc[nt][3] = fast_exp2(fmaf(sc[nt][3], ex_mult, -mu_b));
        l_b += sc[nt][2] + sc[nt][3];
      }
      // ---- O += P V.  V rows at or past the end of the sequence may hold
      // anything (NaN included): zeroed in the fragments, P is 0 there.
      const int vvalid = sq.ctx - t_warp;
      const uint32_t vt = base + L::TILEB;
      uint32_t ph[4];
      if constexpr (FP8) {
        ph[0] = pack_f16x2(sc[0][0], sc[0][1]);
        ph[1] = pack_f16x2(sc[0][2], sc[0][3]);
        ph[2] = pack_f16x2(sc[1][0], sc[1][1]);
        ph[3] = pack_f16x2(sc[1][2], sc[1][3]);
      } else {
        ph[0] = pack_bf16x2(sc[0][0], sc[0][1]);
        ph[1] = pack_bf16x2(sc[0][2], sc[0][3]);
        ph[2] = pack_bf16x2(sc[1][0], sc[1][1]);
        ph[3] = pack_bf16x2(sc[1][2], sc[1][3]);
      }
      const auto add_pv = [&](auto tail) {
        constexpr bool TAIL = decltype(tail)::value;
        const uint32_t keep0 = ((2 * j < vvalid) ? 0x0000FFFFu : 0u) | ((2 * j + 1 < vvalid) ? 0xFFFF0000u : 0u);
        const uint32_t keep1 = ((2 * j + 8 < vvalid) ? 0x0000FFFFu : 0u) | ((2 * j + 9 < vvalid) ? 0xFFFF0000u : 0u);
#pragma unroll
        for (int q = 0; q < (FP8 ? KS / 2 : KS); ++q) {
          uint32_t Rv[4];
          ldsm_x4_trans(vt + L::off(tok_v, 2 * q + ch_v), Rv);
          if constexpr (TAIL) {
            Rv[0] &= keep0;
            Rv[1] &= keep1;
            Rv[2] &= keep0;
            Rv[3] &= keep1;
          }
          if constexpr (!FP8) {
            mma_bf16_16816(o[2 * q], ph, Rv[0], Rv[1]);
            mma_bf16_16816(o[2 * q + 1], ph, Rv[2], Rv[3]);
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // 16-d chunk 2 q + e: n-tile 2c its even d, 2c + 1 its odd d
              const uint32_t e0 = prmt(Rv[2 * e], 0u, 0x3120u);       // keys 0-7
              const uint32_t e1 = prmt(Rv[2 * e + 1], 0u, 0x3120u);   // keys 8-15
              const int c = 2 * q + e;
              mma_f16_16816(o[2 * c], ph, e4m3x2_to_f16x2(static_cast<uint16_t>(e0 & 0xFFFFu)),
                            e4m3x2_to_f16x2(static_cast<uint16_t>(e1 & 0xFFFFu)));
              mma_f16_16816(o[2 * c + 1], ph, e4m3x2_to_f16x2(static_cast<uint16_t>(e0 >> 16)),
                            e4m3x2_to_f16x2(static_cast<uint16_t>(e1 >> 16)));
            }
          }
        }
      };
      if (vvalid < kTileTokens)
        add_pv(std::true_type{});
      else
        add_pv(std::false_type{});
    }
    __syncwarp();  // this warp has read its part of the slot: refill it
    if (healthy && k + NS < ntile) issue(issued++);
  }
  if (!healthy && lane == 0) {
    // a copy of this warp's may still be landing: one more bounded wait each
    for (int kk = issued > NS ? issued - NS : 0; kk < issued; ++kk)
      mbar_wait(smem_u32(full + 4 * (kk % NS) + warp), static_cast<uint32_t>((kk / NS) & 1), nullptr);
  }
  allow_next_grid();

  // ---- row sums over the lanes that share a row; the warps' results merge through shared memory
#pragma unroll
  for (int sh = TR ? 4 : 1; sh < (TR ? 32 : 4); sh <<= 1) {
    l_a += __shfl_xor_sync(kFull, l_a, sh);
    l_b += __shfl_xor_sync(kFull, l_b, sh);
  }
  __syncthreads();  // every warp is done with the stages
  float* s_o = reinterpret_cast<float*>(smem);  // [4 warps][16][DP]
  float* s_ml = s_o + 4 * 16 * DP;              // [4 warps][16][2]
  {
    float* wo = s_o + warp * 16 * DP;
#pragma unroll
    for (int nt = 0; nt < NO; ++nt) {
      if constexpr (TR && !FP8) {  // d = 16 nt + r, + 8 of both rows
        wo[ra * DP + 16 * nt + r] = o[nt][0];
        wo[rb * DP + 16 * nt + r] = o[nt][1];
        wo[ra * DP + 16 * nt + 8 + r] = o[nt][2];
        wo[rb * DP + 16 * nt + 8 + r] = o[nt][3];
      } else if constexpr (TR) {   // d = 16 nt + 2 r, + 1
        *reinterpret_cast<float2*>(wo + ra * DP + 16 * nt + 2 * r) = make_float2(o[nt][0], o[nt][2]);
        *reinterpret_cast<float2*>(wo + rb * DP + 16 * nt + 2 * r) = make_float2(o[nt][1], o[nt][3]);
      } else if constexpr (!FP8) {
        *reinterpret_cast<float2*>(wo + r * DP + 8 * nt + 2 * j) = make_float2(o[nt][0], o[nt][1]);
        *reinterpret_cast<float2*>(wo + (r + 8) * DP + 8 * nt + 2 * j) = make_float2(o[nt][2], o[nt][3]);
      } else {  // columns 2j, 2j + 1 of n-tile 2c (2c + 1) are d = 16 c + 4 j, + 2 (+ 1, + 3)
        const int d = 16 * (nt >> 1) + 4 * j + (nt & 1);
        wo[r * DP + d] = o[nt][0];
        wo[r * DP + d + 2] = o[nt][1];
        wo[(r + 8) * DP + d] = o[nt][2];
        wo[(r + 8) * DP + d + 2] = o[nt][3];
      }
    }
    if ((TR ? r : j) == 0) {
      float* ml = s_ml + warp * 32;
      ml[2 * ra] = m_a;
      ml[2 * ra + 1] = l_a;
      ml[2 * rb] = m_b;
      ml[2 * rb + 1] = l_b;
    }
  }
  __syncthreads();

  for (int idx = threadIdx.x; idx < rows * (D / 2); idx += blockDim.x) {
    const int row = idx / (D / 2), d = 2 * (idx - row * (D / 2));
    float M = -CUDART_INF_F;
#pragma unroll
    for (int w = 0; w < 4; ++w) M = fmaxf(M, s_ml[w * 32 + 2 * row]);
    float a0 = 0.f, a1 = 0.f, lsum = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float mw = s_ml[w * 32 + 2 * row];
      const float wt = (mw == -CUDART_INF_F) ? 0.f : fast_exp2(mw - M);
      const float2 v = *reinterpret_cast<const float2*>(s_o + (w * 16 + row) * DP + d);
      a0 += wt * v.x;
      a1 += wt * v.y;
      lsum += wt * s_ml[w * 32 + 2 * row + 1];
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

// Merge of the split pieces: out = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s.
// A row (token, query head) is merged by W warps that share its pieces, eight
// pieces' rows in flight per warp; rows of one piece were written by the
// attention kernel itself.  Latency counts: one CTA per token with its heads in
// turn took 45 us for one token of 64 heads and 32 pieces.
template <int D, int W>
__global__ void __launch_bounds__(256) chunk_combine_kernel(const ChunkParams p, int nk) {
  constexpr int E = D / 32;  // elements per lane
  constexpr int BATCH = 8;
  __shared__ float s_acc[W > 1 ? 8 : 1][D];
  __shared__ float2 s_ml[8];
  wait_prior_grid();
  allow_next_grid();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = warp % W, tok = blockIdx.x, hq = blockIdx.y * (8 / W) + warp / W;
  int nsplit = 0;  // 0: this warp has no row to merge
  if (hq < p.num_q_heads) {
    const int b = warp_search(p.batch, tok, [&](int i) { return p.q_starts[i]; });
    const ChunkSeq sq = chunk_seq(p, b, false);
    const int i = tok - sq.start;
    if (i >= 0 && i < sq.n) {  // else a row of no sequence
      const int i0 = i / p.tile_q * p.tile_q, i1 = min(sq.n, i0 + p.tile_q) - 1;
      const int n = nk == 64 ? chunk_range<64>(p, sq, i0, i1).n : chunk_range<128>(p, sq, i0, i1).n;
      nsplit = ChunkSplit(n, p.split_tokens / nk, 0).nsplit;
      if (nsplit == 1) nsplit = 0;
    }
  }
  const int64_t row = static_cast<int64_t>(tok) * p.num_q_heads + hq;
  float acc[E], l = 0.f, M = -CUDART_INF_F;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  // this warp's pieces: part, part + W, ...
  const int mine = nsplit > part ? (nsplit - part + W - 1) / W : 0;
  if (mine > 0) {
    const float2* ml = reinterpret_cast<const float2*>(p.ws_ml) + row * p.max_splits;
    const float* po = p.ws_o + row * p.max_splits * D + lane * E;
    for (int s = lane; s < mine; s += 32) M = fmaxf(M, ml[part + s * W].x);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, x));
    for (int s0 = 0; s0 < mine; s0 += 32) {
      const float2 v = s0 + lane < mine ? ml[part + (s0 + lane) * W] : make_float2(-CUDART_INF_F, 0.f);
      const float wl = v.x == -CUDART_INF_F ? 0.f : fast_exp2(v.x - M);  // weight of piece s0 + lane
      l += wl * v.y;
      for (int s = s0; s < mine && s < s0 + 32; s += BATCH) {
        float u[BATCH][E];
#pragma unroll
        for (int q = 0; q < BATCH; ++q) {
          const float* src = po + static_cast<int64_t>(part + (s + q < mine ? s + q : s) * W) * D;
          if constexpr (E == 4) {
            const float4 w = *reinterpret_cast<const float4*>(src);
            u[q][0] = w.x;
            u[q][1] = w.y;
            u[q][2] = w.z;
            u[q][3] = w.w;
          } else {
            const float2 w = *reinterpret_cast<const float2*>(src);
            u[q][0] = w.x;
            u[q][1] = w.y;
          }
        }
#pragma unroll
        for (int q = 0; q < BATCH; ++q) {
          const float wt = __shfl_sync(kFull, wl, (s - s0 + q) & 31);
          if (s + q < mine) {
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += wt * u[q][e];
          }
        }
      }
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(kFull, l, x);
  }
  if constexpr (W > 1) {  // the warps' parts, by the row's first warp
    if (lane == 0) s_ml[warp] = make_float2(M, l);
#pragma unroll
    for (int e = 0; e < E; ++e) s_acc[warp][lane * E + e] = acc[e];
    __syncthreads();
    if (part != 0) return;
    const float own = M;
#pragma unroll
    for (int w = 1; w < W; ++w) M = fmaxf(M, s_ml[warp + w].x);
    const float w0 = own == -CUDART_INF_F ? 0.f : fast_exp2(own - M);
    l *= w0;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= w0;
#pragma unroll
    for (int w = 1; w < W; ++w) {
      const float2 v = s_ml[warp + w];
      const float wt = v.x == -CUDART_INF_F ? 0.f : fast_exp2(v.x - M);
      l += wt * v.y;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += wt * s_acc[warp + w][lane * E + e];
    }
  }
  if (nsplit == 0) return;
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + row * D + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2) dst[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
}

template <int D, bool FP8, bool TWO, bool FAR>
cudaError_t launch_small_t(const ChunkParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t stream) {
  auto kern = chunk_small_kernel<D, FP8, TWO, FAR>;
  constexpr int smem = SmallShape<D, FP8, TWO>::BYTES;
  static int configured[64] = {};
  cudaError_t e = set_smem_once(kern, smem, configured);
  if (e != cudaSuccess) return e;
  const int ntq = (p.max_q_len + p.tile_q - 1) / p.tile_q;
  return launch_pdl(kern, dim3(p.max_splits, p.num_kv_heads * ntq, p.batch), dim3(128), smem, stream, tk, tv, p);
}

template <int D, bool FP8>
cudaError_t launch_small_r(const ChunkParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t stream) {
  if (p.max_q_len * p.group > 8)
    return p.cap_far ? launch_small_t<D, FP8, true, true>(p, tk, tv, stream)
                     : launch_small_t<D, FP8, true, false>(p, tk, tv, stream);
  return p.cap_far ? launch_small_t<D, FP8, false, true>(p, tk, tv, stream)
                   : launch_small_t<D, FP8, false, false>(p, tk, tv, stream);
}

}  // namespace

cudaError_t launch_chunk_small(const ChunkParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                               cudaStream_t stream) {
  const bool fp8 = p.cache_dtype == kE4M3;
  if (p.head_dim == 128)
    return fp8 ? launch_small_r<128, true>(p, tk, tv, stream) : launch_small_r<128, false>(p, tk, tv, stream);
  return fp8 ? launch_small_r<64, true>(p, tk, tv, stream) : launch_small_r<64, false>(p, tk, tv, stream);
}

cudaError_t launch_chunk_combine(const ChunkParams& p, int nk, cudaStream_t stream) {
  // a whole CTA per row while the rows alone leave SMs idle and a warp would
  // have many pieces (9 pieces of 128 rows: 5 us slower than by warps)
  const bool few = static_cast<int64_t>(p.n_tokens) * p.num_q_heads <= 2048 && p.max_splits > 16;
  const dim3 grid(p.n_tokens, few ? p.num_q_heads : (p.num_q_heads + 7) / 8);
  if (p.head_dim == 128)
    return few ? launch_pdl(chunk_combine_kernel<128, 8>, grid, dim3(256), 0, stream, p, nk)
               : launch_pdl(chunk_combine_kernel<128, 1>, grid, dim3(256), 0, stream, p, nk);
  return few ? launch_pdl(chunk_combine_kernel<64, 8>, grid, dim3(256), 0, stream, p, nk)
             : launch_pdl(chunk_combine_kernel<64, 1>, grid, dim3(256), 0, stream, p, nk);
}

}  // namespace pkv
