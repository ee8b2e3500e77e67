// Attention of ragged chunks of new tokens over the paged cache on the
// 5th-generation tensor cores (what it computes: chunk_common.cuh).
//
// A CTA takes a row tile of one (sequence, KV head): up to 256 rows, a row
// being a new token and one of the KV head's query heads, as two groups of 128
// TMEM lanes, over one split of the tile's visible keys in 128-key tiles.
// Its warps have fixed roles:
//   0-7   softmax: thread t of group g is row 128 g + t
//   8     issues the products: S_g(k) = Q_g K(k)^T and O_g += P_g(k) V(k)
//   9, 10 load the K and the V tiles by TMA (one box per lane: a block's rows
//         of one 128-byte column half), alternately into one ring
//   12-15 (E4M3 caches) widen the loaded codes to f16 tiles of the ring
// TMEM: S of both groups (128 columns each) and O of both; P_g(k), 16-bit
// pairs, takes the first half of S_g's columns once the softmax has read them.
// The products are issued in the order
//   PV_0(k), S_0(k+1), PV_1(k), S_1(k+1), PV_0(k+1), ...
// so that one group's softmax runs under the other group's two products.  They
// execute in issue order: S_g(k+1) cannot overtake the PV_g(k) that reads P
// from its columns, and S_g(k) having completed (sfull) means that PV_g(k-1)
// has, so the softmax may then rescale O_g without a barrier of its own.
// The running maximum is lazy: O is rescaled only when the maximum grows by
// more than 2^8, so P stays within 2^8 (f16 holds that) and most tiles rescale
// nothing.  Sums, maxima and O are binary32; P is rounded to 16 bits (bf16
// 2^-8, f16 2^-11 of a weight), next to the output's own 2^-8.
//
// Every wait is bounded; a time-out records the error, raises the CTA's abort
// flag, which ends every role's loop, and the CTA drains its copies and
// products before it frees TMEM.

#include "chunk_common.cuh"
#include "pkv_tc.cuh"

namespace pkv {
namespace {

template <int D, bool FP8>
struct TcShape {
  static constexpr int M = 128, GROUPS = 2, ROWS = M * GROUPS, NK = 128;
  static constexpr int HALVES = D / 64;            // 128-byte column halves of a 16-bit row
  static constexpr int QHALF = ROWS * 128;
  static constexpr int QBYTES = HALVES * QHALF;
  static constexpr int HALFB = NK * 128;
  static constexpr int TILE = HALVES * HALFB;      // a 16-bit K or V tile
  static constexpr int RAW = NK * D;               // an E4M3 K or V tile
  static constexpr int NS = FP8 ? (D == 128 ? 3 : 6) : (D == 128 ? 4 : 8);
  static constexpr int NR = FP8 ? (D == 128 ? 4 : 8) : 0;
  static constexpr int NBARS = 2 * NS + 2 * NR + 4 * GROUPS + 2;
  static constexpr int BYTES = QBYTES + NS * TILE + NR * RAW + NBARS * 8 + 16 + 1024;
  static_assert(BYTES <= 232448, "shared memory per CTA");
  static constexpr int THREADS = FP8 ? 512 : 384;
  // registers: 384 x 168 or 512 x 128 at launch
  static constexpr int REGS_SOFTMAX = FP8 ? 176 : 200;
  static constexpr int REGS_OTHER = FP8 ? 80 : 104;
  static_assert(256 * REGS_SOFTMAX + (THREADS - 256) * REGS_OTHER <= THREADS * (FP8 ? 128 : 168), "register file");
};

// What a score is besides scale * q.k: nothing; capped; biased (capped or not).
constexpr int kPlain = 0, kCapped = 1, kBiased = 2;

__device__ __forceinline__ float min_nan(float a, float b) {  // NaN if one is
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// x := cap * tanh(x * y_mult) in log2 units, for the 128 scores of a row.
//
// Small arguments, |y| <= 1/2 in the whole warp (scores up to half the cap):
// tanh(y) = y (c0 + c1 y^2 + c2 y^4 + c3 y^6) with the coefficients of the
// least largest relative error on that range (5.4e-7: below 2^-15 of a
// weight's exponent for scores up to 25), powers of y_mult folded in: five
// packed FMA-pipe operations per two scores and nothing on the
// special-function unit, which the exponentials need.
// Others: 1 - 2 / (e^2y + 1), one reciprocal shared by four scores,
// 1 / a = b c d / (a b c d); 2y is held below 28 log2 units, where tanh is 1 to
// binary32 and the product of four cannot overflow.
template <int N>
__device__ __forceinline__ void cap_scores(float (&x)[N], float w_mult, float cap_log2, bool masked,
                                           const uint32_t (&see)[N / 32]) {
  constexpr float kY = 0.34657359027997264f;  // ln 2 / 2: y = kY * w
  const float y_mult = w_mult * kY;
  float am = 0.f;
#pragma unroll
  for (int i = 0; i < N; i += 2) am = max3f(am, fabsf(x[i]), fabsf(x[i + 1]));
  if (__all_sync(kFull, am * y_mult <= 0.5f) && y_mult > 1e-5f) {
    const float y2 = y_mult * y_mult, f0 = cap_log2 * y_mult;
    const float f1 = f0 * y2, f2 = f1 * y2, f3 = f2 * y2;
    const float2 c0 = make_float2(0.99999946f * f0, 0.99999946f * f0);
    const float2 c1 = make_float2(-0.33326318f * f1, -0.33326318f * f1);
    const float2 c2 = make_float2(0.13190297f * f2, 0.13190297f * f2);
    const float2 c3 = make_float2(-0.04440223f * f3, -0.04440223f * f3);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 v = make_float2(x[i], x[i + 1]);
      const float2 t = __fmul2_rn(v, v);
      float2 h = __ffma2_rn(c3, t, c2);
      h = __ffma2_rn(h, t, c1);
      h = __ffma2_rn(h, t, c0);
      h = __fmul2_rn(h, v);
      x[i] = h.x;
      x[i + 1] = h.y;
    }
    return;
  }
  if (masked) {  // what lies past the sequence's end may be NaN: it must not reach its neighbours
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (!((see[i / 32] >> (i % 32)) & 1u)) x[i] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    float q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = fast_exp2(min_nan(x[i + j] * w_mult, 28.f)) + 1.f;
    const float2 pr = __fmul2_rn(make_float2(q[0], q[2]), make_float2(q[1], q[3]));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(pr.x * pr.y));
    const float2 rp = __fmul2_rn(make_float2(r, r), make_float2(pr.y, pr.x));  // 1 / (q0 q1), 1 / (q2 q3)
    const float2 m2c = make_float2(-2.f * cap_log2, -2.f * cap_log2), c = make_float2(cap_log2, cap_log2);
    const float2 a = __ffma2_rn(__fmul2_rn(make_float2(rp.x, rp.x), make_float2(q[1], q[0])), m2c, c);
    const float2 b = __ffma2_rn(__fmul2_rn(make_float2(rp.y, rp.y), make_float2(q[3], q[2])), m2c, c);
    x[i] = a.x;
    x[i + 1] = a.y;
    x[i + 2] = b.x;
    x[i + 3] = b.y;
  }
}

template <int D, bool FP8, int MODE>
__global__ void __launch_bounds__(TcShape<D, FP8>::THREADS, 1)
    chunk_tc_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                    const ChunkParams p) {
  using C = TcShape<D, FP8>;
  constexpr int M = C::M, NK = C::NK, NS = C::NS, NR = C::NR, GROUPS = C::GROUPS;
  constexpr uint32_t COL_S = 0, COL_O = GROUPS * NK;  // + g * NK, + g * D
  constexpr uint32_t IDESC_S = FP8 ? idesc_f16(M, NK, false) : idesc_bf16(M, NK, false);
  constexpr uint32_t IDESC_PV = FP8 ? idesc_f16(M, D, true) : idesc_bf16(M, D, true);
  constexpr int kMma = 8, kProd = 9, kConv = 12;
  static_assert(COL_O + GROUPS * D <= 512, "TMEM columns");

  // the warp number as a broadcast: roles branch uniformly
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kFull, tid >> 5, 0);
  const int G = p.group, H_q = p.num_q_heads;
  wait_prior_grid();

  // ---- the CTA's row tile: number t of the sequences' tiles, longest first
  // within a sequence (its last tokens see the most keys)
  const int h = blockIdx.x % p.num_kv_heads;
  const int t = blockIdx.x / p.num_kv_heads;
  const int b = warp_search(p.batch, t, [&](int i) { return chunk_tile_base(p, i); });
  const ChunkSeq sq = chunk_seq(p, b, tid == 0 && blockIdx.y == 0 && h == 0);
  const int ntq = (sq.n + p.tile_q - 1) / p.tile_q;
  const int tile = ntq - 1 - (t - chunk_tile_base(p, b));
  if (tile < 0 || tile >= ntq) return;
  const int i0 = tile * p.tile_q, i1 = min(sq.n, i0 + p.tile_q) - 1;
  const int rows = (i1 - i0 + 1) * G;
  const ChunkRange rg = chunk_range<NK>(p, sq, i0, i1);
  const int per_split = p.split_tokens / NK;
  const int nsplit = max(1, (rg.n + per_split - 1) / per_split);
  const int split = blockIdx.y;
  if (split >= nsplit) return;
  const int k0 = split * per_split;
  const int ntile = min(rg.n - k0, per_split);
  const int ng = rows > M ? 2 : 1;
  // the sequence ends inside a block of the last tile (later tiles hold later keys)
  const int t_last = ntile > 0 ? rg.tile(k0 + ntile - 1) * NK : 0;
  const bool v_tail = ntile > 0 && sq.ctx - t_last < NK && (sq.ctx - t_last) % p.block_size != 0;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* q_sm = smem;                              // half hf, row r at hf * QHALF + r * 128
  uint8_t* ring = smem + C::QBYTES;                  // K(k) is item 2k, V(k) item 2k + 1
  uint8_t* raw = ring + NS * C::TILE;
  uint64_t* full = reinterpret_cast<uint64_t*>(raw + NR * C::RAW);
  uint64_t* empty = full + NS;
  uint64_t* rfull = empty + NS;
  uint64_t* rempty = rfull + NR;
  uint64_t* sfull = rempty + NR;    // [GROUPS]: S_g(k) is in TMEM
  uint64_t* pfull = sfull + GROUPS;  // [GROUPS]: P_g(k) is in TMEM
  uint64_t* odone = pfull + GROUPS;  // [GROUPS]: O_g is complete
  uint64_t* qfull = odone + GROUPS;
  uint64_t* vfix = qfull + 1;       // the last V tile's rows past the end are zeros
  uint64_t* done = vfix + 1;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(done + GROUPS);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(smem_u32(full + s), FP8 ? 4 : 1);
      mbar_init(smem_u32(empty + s), ng);
    }
    for (int s = 0; s < NR; ++s) {
      mbar_init(smem_u32(rfull + s), 1);
      mbar_init(smem_u32(rempty + s), 4);
    }
    for (int g = 0; g < GROUPS; ++g) {
      mbar_init(smem_u32(sfull + g), 1);
      mbar_init(smem_u32(pfull + g), 4);
      mbar_init(smem_u32(odone + g), 1);
      mbar_init(smem_u32(done + g), 1);
    }
    mbar_init(smem_u32(qfull), 4 * ng);
    mbar_init(smem_u32(vfix), 1);
    *s_abort = 0;
    fence_mbar_init();
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

  if (warp >= kMma) {
    regs_dec<C::REGS_OTHER>();
    if (warp == kMma || warp == kMma + 3) {
      // ------------------------------------------------------------ products
      // The whole warp walks this role, one lane's products are issued: see
      // tc_mma_ss_if.
      const int g = warp == kMma ? 0 : 1;
      const uint32_t leader = elect_one();
      const int nt = __shfl_sync(kFull, g < ng ? ntile : 0, 0);
      const uint32_t ring0 = __shfl_sync(kFull, smem_u32(ring), 0), q0 = __shfl_sync(kFull, smem_u32(q_sm), 0);
      const uint32_t c_s = tbase + COL_S + g * NK, c_o = tbase + COL_O + g * D;
      auto wait = [&](uint64_t* bar, int phase) {
        return __all_sync(kFull, wait_or_abort(smem_u32(bar), static_cast<uint32_t>(phase & 1), p.err, s_abort)) != 0;
      };
      const uint64_t a0 = smem_desc_sw128(q0 + g * M * 128, 0, 1024);
      auto issue_s = [&](int slot) {
        const uint64_t b0 = smem_desc_sw128(ring0 + slot * C::TILE, 0, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)  // descriptor addresses are in 16-byte units
          tc_mma_ss_if(leader, c_s, a0 + ((kk / 4) * C::QHALF + (kk % 4) * 32) / 16,
                       b0 + ((kk / 4) * C::HALFB + (kk % 4) * 32) / 16, IDESC_S, kk > 0 ? 1u : 0u);
        tc_commit_if(leader, smem_u32(sfull + g));
        tc_commit_if(leader, smem_u32(empty + slot));
      };
      bool ok = wait(qfull, 0);
      int slot = 0, use = 0;  // ring slot of the next item, and its use number
      auto next_slot = [&]() {
        if (++slot == NS) {
          slot = 0;
          ++use;
        }
      };
      if (nt > 0 && ok) {
        ok = wait(full, 0);
        if (ok) {
          tc_fence_after();
          issue_s(0);
        }
        next_slot();
      }
      for (int k = 0; k < nt && ok; ++k) {
        const int vslot = slot;
        ok = wait(full + vslot, use);
        if (!ok) break;
        if (!FP8 && k == nt - 1 && v_tail) {  // its loader has zeroed the rows past the sequence's end
          ok = wait(vfix, 0);
          if (!ok) break;
        }
        next_slot();
        const bool more = k + 1 < nt;
        if (more) ok = wait(full + slot, use);  // K(k+1), ahead of the wait for P
        const uint64_t v0 = smem_desc_sw128(ring0 + vslot * C::TILE, C::HALVES > 1 ? C::HALFB : 0, 1024);
        ok = ok && wait(pfull + g, k);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < NK / 16; ++kk)  // MN-major V: 8-key groups 1024 B apart, column halves HALFB apart
          tc_mma_ts_if(leader, c_o, c_s + kk * 8, v0 + kk * (2048 / 16), IDESC_PV, (k > 0 || kk > 0) ? 1u : 0u);
        tc_commit_if(leader, smem_u32(empty + vslot));
        if (more) {
          issue_s(slot);
          next_slot();
        } else {
          tc_commit_if(leader, smem_u32(odone + g));
        }
      }
      // nothing of this warp's may still be running when TMEM is freed
      tc_commit_if(leader, smem_u32(done + g));
      mbar_wait(smem_u32(done + g), 0u, nullptr);
    } else if (warp == kProd || warp == kProd + 1) {
      // ------------------------------------------------------------ loads
      const int v = warp - kProd;
      const CUtensorMap* tmap = v ? &tmap_v : &tmap_k;
      constexpr int ROWB = FP8 ? D : 128;              // bytes of a box row
      constexpr int BYTES = FP8 ? C::RAW : C::TILE;
      const int nring = FP8 ? NR : NS;
      const uint32_t base = smem_u32(FP8 ? raw : ring);
      uint64_t* bfull = FP8 ? rfull : full;
      uint64_t* bempty = FP8 ? rempty : empty;
      const int per_half = NK / p.block_size;          // boxes of a column half
      const int nbox = per_half * (FP8 ? 1 : C::HALVES);
      const int hf = lane / per_half, bi = lane % per_half;
      const uint32_t off = hf * C::HALFB + bi * p.block_size * ROWB;
      const int32_t* tbl = p.block_tables + static_cast<int64_t>(b) * p.max_blocks;
      // the block this lane's box of tile k holds; blocks that no row sees are
      // not looked up and read as zeros (outside the tensor map)
      auto block_of = [&](int k) {
        int phys = -1;
        if (lane < nbox && k < ntile) {
          const int t0 = rg.tile(k0 + k) * NK + bi * p.block_size;
          if (rg.sees(t0, t0 + p.block_size)) {
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
      int issued = 0;
      for (int k = 0; k < ntile; ++k) {
        const int item = 2 * k + v, s = item % nring;
        const int next = block_of(k + 1);
        bool go = true;
        if (lane == 0 && item >= nring)
          go = wait_or_abort(smem_u32(bempty + s), static_cast<uint32_t>((item / nring - 1) & 1), p.err, s_abort);
        if (!__shfl_sync(kFull, go ? 1 : 0, 0)) break;
        const uint32_t bar = smem_u32(bfull + s);
        if (lane == 0) {
          fence_proxy_async_smem();
          mbar_arrive_expect_tx(bar, BYTES);
        }
        __syncwarp();
        if (lane < nbox) tma_load_4d(base + s * BYTES + off, tmap, bar, hf * 64, 0, h, phys);
        phys = next;
        issued = k + 1;
      }
      if (!FP8 && v == 1 && v_tail && issued == ntile) {
        // Rows of the last block past the sequence's end may hold anything
        // (NaN included): zero them once they have landed, P is 0 there.  Whole
        // blocks past it were loaded as zeros.
        const int item = 2 * (ntile - 1) + 1, s = item % nring;
        bool ok = wait_or_abort(smem_u32(bfull + s), static_cast<uint32_t>((item / nring) & 1), p.err, s_abort);
        if (__all_sync(kFull, ok)) {
          const int first = sq.ctx - rg.tile(k0 + ntile - 1) * NK;
          const int chunks = ((first + p.block_size - 1) / p.block_size * p.block_size - first) * 8;
          for (int c = lane; c < C::HALVES * chunks; c += 32) {
            const int hh = c / chunks, cc = c - hh * chunks;
            *reinterpret_cast<uint4*>(ring + s * C::TILE + hh * C::HALFB + first * 128 + cc * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(vfix));
        }
      }
      if (lane == 0 && *s_abort) {  // the copies in flight land before the CTA leaves
        for (int k = 0; k < issued; ++k) {
          const int item = 2 * k + v;
          if (item + nring < 2 * issued) continue;
          mbar_wait(smem_u32(bfull + item % nring), static_cast<uint32_t>((item / nring) & 1), nullptr);
        }
      }
    } else if (FP8 && warp >= kConv) {
      // ------------------------------------------------------------ widening
      // thread t: key t of the tile, 16 codes -> 32 bytes at a time
      if constexpr (FP8) {
        const int key = (warp - kConv) * 32 + lane;
        constexpr int CH = D / 16;                     // 16-byte chunks of a raw row
        const uint32_t rsw = D == 128 ? (key & 7) : ((key >> 1) & 3);
        bool ok = true;
        for (int item = 0; item < 2 * ntile; ++item) {
          const int rs = item % NR, s = item % NS;
          ok = wait_or_abort(smem_u32(rfull + rs), static_cast<uint32_t>((item / NR) & 1), p.err, s_abort);
          if (ok && item >= NS)
            ok = wait_or_abort(smem_u32(empty + s), static_cast<uint32_t>((item / NS - 1) & 1), p.err, s_abort);
          if (!__all_sync(kFull, ok)) break;
          const uint8_t* src = raw + rs * C::RAW + key * D;
          uint8_t* dst = ring + s * C::TILE + key * 128;
          // rows past the sequence's end may hold anything: zeros instead
          const bool live = rg.tile(k0 + (item >> 1)) * NK + key < sq.ctx;
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            uint4 w = *reinterpret_cast<const uint4*>(src + ((c ^ rsw) << 4));
            if (!live) w = make_uint4(0u, 0u, 0u, 0u);
            uint4 a, e;
            a.x = e4m3x2_to_f16x2(static_cast<uint16_t>(w.x & 0xFFFFu));
            a.y = e4m3x2_to_f16x2(static_cast<uint16_t>(w.x >> 16));
            a.z = e4m3x2_to_f16x2(static_cast<uint16_t>(w.y & 0xFFFFu));
            a.w = e4m3x2_to_f16x2(static_cast<uint16_t>(w.y >> 16));
            e.x = e4m3x2_to_f16x2(static_cast<uint16_t>(w.z & 0xFFFFu));
            e.y = e4m3x2_to_f16x2(static_cast<uint16_t>(w.z >> 16));
            e.z = e4m3x2_to_f16x2(static_cast<uint16_t>(w.w & 0xFFFFu));
            e.w = e4m3x2_to_f16x2(static_cast<uint16_t>(w.w >> 16));
            uint8_t* to = dst + (c / 4) * C::HALFB;
            *reinterpret_cast<uint4*>(to + (((2 * (c % 4)) ^ (key & 7)) << 4)) = a;
            *reinterpret_cast<uint4*>(to + (((2 * (c % 4) + 1) ^ (key & 7)) << 4)) = e;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_u32(full + s));
            mbar_arrive(smem_u32(rempty + rs));
          }
        }
      }
    }
  } else {
    regs_inc<C::REGS_SOFTMAX>();
    const int grp = warp >> 2;
    if (grp < ng) {
      // ------------------------------------------------------------ softmax
      const int r_in = tid;                              // row of the tile
      const bool row_ok = r_in < rows;
      const bool warp_ok = warp * 32 < rows;             // some lane has a row
      const int64_t orow = (static_cast<int64_t>(sq.start) + i0 + r_in / G) * H_q + h * G + r_in % G;
      {  // this row of Q into shared memory, 128B-swizzled; f16 for E4M3 caches
        const uint16_t* qr = row_ok ? static_cast<const uint16_t*>(p.q) + orow * D : nullptr;
        uint4 w[D / 8];
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
          w[c] = qr ? *reinterpret_cast<const uint4*>(qr + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          if constexpr (FP8) {
            w[c].x = pack_f16x2(bf16lo_to_f32(w[c].x), bf16hi_to_f32(w[c].x));
            w[c].y = pack_f16x2(bf16lo_to_f32(w[c].y), bf16hi_to_f32(w[c].y));
            w[c].z = pack_f16x2(bf16lo_to_f32(w[c].z), bf16hi_to_f32(w[c].z));
            w[c].w = pack_f16x2(bf16lo_to_f32(w[c].w), bf16hi_to_f32(w[c].w));
          }
          *reinterpret_cast<uint4*>(q_sm + (c >> 3) * C::QHALF + r_in * 128 + (((c & 7) ^ (r_in & 7)) << 4)) = w[c];
        }
        fence_proxy_async_smem();  // the tensor core reads Q through the async proxy
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(qfull));
      }
      // what the row sees; a row past the tile's takes no mask (nothing of it
      // is ever written)
      constexpr int kFar = 0x3FFFFFFF;
      const int pos = row_ok ? sq.ctx - sq.n + i0 + r_in / G : kFar;
      const int lo = row_ok && p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
      const int pf = row_ok && pos >= 0 ? sq.prefix : 0;
      constexpr float kLog2e = 1.4426950408889634f;
      float qk = p.qk_log2, v_mult = 1.f;
      if constexpr (FP8) {
        qk *= p.k_scale[static_cast<int64_t>(b) * p.scale_stride + h];
        v_mult = p.v_scale[static_cast<int64_t>(b) * p.scale_stride + h];
      }
      const float slope = MODE == kBiased && row_ok ? p.slopes[h * G + r_in % G] * kLog2e : 0.f;
      // scores times ex_mult are log2 weights
      const float ex_mult = MODE != kPlain ? 1.f : qk;

      const uint32_t lanes = tbase + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      const uint32_t t_s = lanes + COL_S + grp * NK, t_o = lanes + COL_O + grp * D;
      const uint32_t b_sfull = smem_u32(sfull + grp), b_pfull = smem_u32(pfull + grp);
      float m_used = -CUDART_INF_F, lsum = 0.f;
      bool ok = true;
      for (int k = 0; k < ntile; ++k) {
        ok = __all_sync(kFull, wait_or_abort(b_sfull, static_cast<uint32_t>(k & 1), p.err, s_abort));
        if (!ok) break;
        tc_fence_after();
        if (warp_ok) {
          float x[NK];
#pragma unroll
          for (int c = 0; c < NK / 32; ++c) tmem_ld32(t_s + 32 * c, x + 32 * c);
          tmem_wait_ld();
          const int t0 = rg.tile(k0 + k) * NK;
          const bool whole = (t0 + NK - 1 <= pos && t0 >= lo) || t0 + NK <= pf;
          const bool masked = !__all_sync(kFull, whole);
          uint32_t see[NK / 32];  // bit i of word w: key t0 + 32 w + i is seen
          if (masked) {
            auto below = [&](int n, int w) {  // the first n keys of the tile
              n -= 32 * w;
              return n <= 0 ? 0u : (n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u);
            };
#pragma unroll
            for (int w = 0; w < NK / 32; ++w)
              see[w] = (below(pos - t0 + 1, w) & ~below(lo - t0, w)) | below(pf - t0, w);
          }
          if (MODE == kCapped || (MODE == kBiased && p.cap_log2 > 0.f)) cap_scores(x, qk, p.cap_log2, masked, see);
          if constexpr (MODE == kBiased) {
            const float mult = p.cap_log2 > 0.f ? 1.f : qk, base = slope * static_cast<float>(t0 - pos);
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
          if (masked) {
#pragma unroll
            for (int i = 0; i < NK; ++i)
              if (!((see[i / 32] >> (i % 32)) & 1u)) x[i] = -CUDART_INF_F;
          }
          float mt;
          {
            float mp[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              mp[j] = max3f(x[j], x[8 + j], x[16 + j]);
#pragma unroll
              for (int i = 24; i + 8 < NK; i += 16) mp[j] = max3f(mp[j], x[i + j], x[i + 8 + j]);
              mp[j] = fmaxf(mp[j], x[NK - 8 + j]);
            }
            mt = max3f(max3f(mp[0], mp[1], mp[2]), max3f(mp[3], mp[4], mp[5]), fmaxf(mp[6], mp[7])) * ex_mult;
          }
          float alpha = 1.f;
          bool resc = false;
          if (m_used == -CUDART_INF_F) {
            m_used = mt;  // nothing accumulated yet for this row
          } else if (row_ok && mt > m_used + 8.f) {
            alpha = fast_exp2(m_used - mt);
            m_used = mt;
            resc = true;
          }
          if (__any_sync(kFull, resc)) {  // O holds tiles 0..k-1 (PV(k-1) came before S(k))
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
          }
          const float mu = m_used == -CUDART_INF_F ? 0.f : m_used;
          const float2 neg_mu = make_float2(-mu, -mu), mult2 = make_float2(ex_mult, ex_mult);
          float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < NK / 32; ++c) {
            uint32_t hi[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 xx = make_float2(x[32 * c + 2 * i], x[32 * c + 2 * i + 1]);
              const float2 e = MODE != kPlain ? __fadd2_rn(xx, neg_mu) : __ffma2_rn(xx, mult2, neg_mu);
              const float2 pp = make_float2(fast_exp2(e.x), fast_exp2(e.y));
              ls[i & 1] = __fadd2_rn(ls[i & 1], pp);
              hi[i] = FP8 ? pack_f16x2(pp.x, pp.y) : pack_bf16x2(pp.x, pp.y);
            }
            tmem_st16(t_s + 16 * c, hi);
          }
          lsum += (ls[0].x + ls[1].x) + (ls[0].y + ls[1].y);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_pfull);  // P(k) is in TMEM
      }
      if (ok && ntile > 0) ok = __all_sync(kFull, wait_or_abort(smem_u32(odone + grp), 0u, p.err, s_abort));
      if (ok && warp_ok) {
        // ---- O leaves through this warp's part of the Q region (every S of
        // the group has completed), so that a store instruction writes whole
        // rows: direct outputs as bf16 rows, pieces as binary32 in 64-column
        // passes, both 128 bytes of a row per half
        tc_fence_after();
        const float inv = lsum > 0.f ? v_mult / lsum : 0.f;
        const float mult = nsplit == 1 ? inv : v_mult;
        auto stage = [&](int hf, int c) { return q_sm + hf * C::QHALF + r_in * 128 + ((c ^ (r_in & 7)) << 4); };
        auto row_of = [&](int r) {                       // output row of tile row r
          return (static_cast<int64_t>(sq.start) + i0 + r / G) * H_q + h * G + r % G;
        };
        if (nsplit == 1) {
#pragma unroll
          for (int c0 = 0; c0 < D; c0 += 32) {
            float o[32];
            if (ntile > 0) {
              tmem_ld32(t_o + c0, o);
              tmem_wait_ld();
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint4 w;
              w.x = pack_bf16x2(o[8 * i] * mult, o[8 * i + 1] * mult);
              w.y = pack_bf16x2(o[8 * i + 2] * mult, o[8 * i + 3] * mult);
              w.z = pack_bf16x2(o[8 * i + 4] * mult, o[8 * i + 5] * mult);
              w.w = pack_bf16x2(o[8 * i + 6] * mult, o[8 * i + 7] * mult);
              *reinterpret_cast<uint4*>(stage(c0 / 64, (c0 % 64) / 8 + i)) = w;
            }
          }
          __syncwarp();
          constexpr int CPR = D / 8;                     // 16-byte chunks of an output row
#pragma unroll
          for (int i = 0; i < CPR; ++i) {
            const int r = warp * 32 + (i * 32 + lane) / CPR, c = lane % CPR;
            if (r < rows)
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row_of(r) * D + c * 8) =
                  *reinterpret_cast<const uint4*>(q_sm + (c >> 3) * C::QHALF + r * 128 + (((c & 7) ^ (r & 7)) << 4));
          }
        } else {
          // 32 columns (128 bytes) of a row per pass, in the first half's rows
#pragma unroll
          for (int c0 = 0; c0 < D; c0 += 32) {
            float o[32];
            tmem_ld32(t_o + c0, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float4*>(stage(0, i)) = make_float4(o[4 * i] * mult, o[4 * i + 1] * mult,
                                                                    o[4 * i + 2] * mult, o[4 * i + 3] * mult);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r = warp * 32 + i * 4 + (lane >> 3), c = lane & 7;
              const float4 u = *reinterpret_cast<const float4*>(q_sm + r * 128 + ((c ^ (r & 7)) << 4));
              if (r < rows)
                *reinterpret_cast<float4*>(p.ws_o + (row_of(r) * p.max_splits + split) * D + c0 + c * 4) = u;
            }
            __syncwarp();
          }
          if (row_ok) {
            float* ml = p.ws_ml + (orow * p.max_splits + split) * 2;
            ml[0] = m_used;
            ml[1] = lsum;
          }
        }
      }
    }
  }
  allow_next_grid();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

template <int D, bool FP8, int MODE>
cudaError_t launch_tc_t(const ChunkParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t stream) {
  auto kern = chunk_tc_kernel<D, FP8, MODE>;
  // at least 120 KB: one CTA per SM (it holds all 512 TMEM columns)
  constexpr int smem = TcShape<D, FP8>::BYTES > 120 * 1024 ? TcShape<D, FP8>::BYTES : 120 * 1024;
  static int configured[64] = {};
  cudaError_t e = set_smem_once(kern, smem, configured);
  if (e != cudaSuccess) return e;
  const int tiles = p.n_tokens / p.tile_q + p.batch;
  return launch_pdl(kern, dim3(tiles * p.num_kv_heads, p.max_splits), dim3(TcShape<D, FP8>::THREADS), smem, stream,
                    tk, tv, p);
}

template <int D, bool FP8>
cudaError_t launch_tc_m(const ChunkParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t stream) {
  if (p.slopes != nullptr) return launch_tc_t<D, FP8, kBiased>(p, tk, tv, stream);
  if (p.cap_log2 > 0.f) return launch_tc_t<D, FP8, kCapped>(p, tk, tv, stream);
  return launch_tc_t<D, FP8, kPlain>(p, tk, tv, stream);
}

}  // namespace

cudaError_t launch_chunk_tc(const ChunkParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t stream) {
  const bool fp8 = p.cache_dtype == kE4M3;
  if (p.head_dim == 128)
    return fp8 ? launch_tc_m<128, true>(p, tk, tv, stream) : launch_tc_m<128, false>(p, tk, tv, stream);
  return fp8 ? launch_tc_m<64, true>(p, tk, tv, stream) : launch_tc_m<64, false>(p, tk, tv, stream);
}

}  // namespace pkv
