// Pieces shared by the ragged-chunk attention kernels (chunk.cu, chunk_e2m1.cu,
// chunk_tc.cuh):
// which sequence a token or a row tile belongs to, which keys a row tile sees,
// and the scores' definition.
//
// Query i of the n new tokens of a sequence with ctx tokens sits at position
// pos = ctx - n + i and sees key t when t < ctx and
//   t < prefix, or pos - window < t <= pos   (window 0: 0 <= t <= pos);
// a query before position 0 sees nothing.  Its score against key t is
//   z = scale q.k,   cap * tanh(z / cap) with a cap,   + slope (t - pos) with a bias.
#pragma once

#include "decode_common.cuh"

namespace pkv {

// One sequence of the call as the kernels see it.
struct ChunkSeq {
  int start, n, ctx, prefix;  // first query row, new tokens, tokens attended, tokens every query sees
  bool ok;                    // its row range lies inside the call's bounds
};

__device__ __forceinline__ int chunk_clamp_ctx(const ChunkParams& p, int ctx) {
  const int64_t cap = static_cast<int64_t>(p.max_blocks) * p.block_size;
  const int lim = static_cast<int>(cap < p.max_ctx ? cap : p.max_ctx);
  return ctx < 0 ? 0 : (ctx > lim ? lim : ctx);
}

// `note`: this thread records a range or length that had to be refused or clamped.
__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkParams& p, int b, bool note) {
  ChunkSeq s;
  const int q0 = p.q_starts[b], q1 = p.q_starts[b + 1];
  const int ctx_raw = p.context_lens[b];
  const int pfx = p.prefix_lens != nullptr ? p.prefix_lens[b] : 0;
  s.start = q0;
  s.ok = q0 >= 0 && q1 >= q0 && q1 <= p.n_tokens && q1 - q0 <= p.max_q_len;
  s.n = s.ok ? q1 - q0 : 0;
  s.ctx = chunk_clamp_ctx(p, ctx_raw);
  s.prefix = pfx < 0 ? 0 : (pfx < s.ctx ? pfx : s.ctx);
  if (note && (!s.ok || s.ctx != ctx_raw)) record_error(p.err, kDevErrContextLen);
  return s;
}

// Row tiles of the tcgen05 kernel: sequence b's tiles take numbers from
// floor(q_starts[b] / tile_q) + b on, which leaves each one room for its
// ceil(n / tile_q) tiles and needs no prefix sum; some numbers stay unused.
__device__ __forceinline__ int chunk_tile_base(const ChunkParams& p, int b) {
  const int q = p.q_starts[b];
  return (q < 0 ? 0 : (q > p.n_tokens ? p.n_tokens : q)) / p.tile_q + b;
}

// The keys that queries [i0, i1] of a sequence see, in tiles of NK tokens:
// tiles [0, na) for the prefix, then nb tiles from b0 on.
struct ChunkRange {
  int lo, hi, prefix;  // some query sees t iff lo <= t < hi or t < prefix
  int na, b0, n;       // n = na + the tiles of [lo, hi) past them
  __device__ __forceinline__ int tile(int k) const { return k < na ? k : b0 + (k - na); }
  __device__ __forceinline__ bool sees(int t0, int t1) const {  // any of tokens [t0, t1)
    return t0 < prefix || (t0 < hi && t1 > lo);
  }
};

template <int NK>
__device__ __forceinline__ ChunkRange chunk_range(const ChunkParams& p, const ChunkSeq& s, int i0, int i1) {
  ChunkRange r;
  const int pos0 = s.ctx - s.n + i0, pos1 = s.ctx - s.n + i1;
  r.hi = pos1 < 0 ? 0 : pos1 + 1;
  r.prefix = pos1 < 0 ? 0 : s.prefix;
  r.lo = p.window > 0 && pos0 >= p.window ? pos0 - p.window + 1 : 0;
  r.na = (r.prefix + NK - 1) / NK;
  const int first = r.lo / NK, end = (r.hi + NK - 1) / NK;
  r.b0 = first > r.na ? first : r.na;
  r.n = r.na + (end > r.b0 ? end - r.b0 : 0);
  return r;
}

// Split `split` of a row tile's n visible key tiles: as many splits as pieces of
// at most `most` tiles take, of even length.
struct ChunkSplit {
  int nsplit, k0, ntile;
  __device__ __forceinline__ ChunkSplit(int n, int most, int split) {
    nsplit = n > most ? (n + most - 1) / most : 1;
    const int each = (n + nsplit - 1) / nsplit;
    k0 = split * each;
    ntile = n - k0 < each ? n - k0 : each;
    if (ntile < 0) ntile = 0;
  }
};

// cap * tanh(score / cap), in two ways besides the exponential form; y = score / cap.
//
// Small scores: tanh(y) = y (c0 + c1 y^2 + c2 y^4) up to |y| = y_max, both from
// cap_coefficients: the capped score is off by less than 2^-13, next to the
// weight's own rounding.  Powers of the multipliers folded in, that is
// x * ((k2 x^2 + k1) x^2 + k0) for a raw product x: four packed FMA-pipe
// operations for two weights' exponents instead of one, and nothing on the
// special-function unit, which the exponentials need.  Where the powers pass
// binary32 (caps below about 1e-10 of the products) it holds for no score,
// since infinity times a product of 0 is NaN.
//
// Caps above 100 (kernels of their own), scores up to 0.35 of the cap: the error
// of so few coefficients would be more than the weight's rounding, so `far` has
// one more and binary32's own rounding.  Below it would only cost: biased prompts
// 6-18 %; chosen between at run time, all prompts 2-6 %.
template <bool FAR>
struct CapPoly {
  float2 k0, k1, k2;
  float y_mult;    // y = x * y_mult
  float y_max;     // |y| up to which the small scores' polynomial holds
  __device__ __forceinline__ CapPoly(float w_mult, const ChunkParams& p) {
    y_mult = w_mult * 0.34657359027997264f;  // ln 2 / 2: w = 2 y log2(e)
    const float y2 = y_mult * y_mult, f0 = p.cap_log2 * y_mult, f1 = f0 * y2, f2 = f1 * y2;
    // (up to kCapNear constants: they cost no registers)
    const float c0 = FAR ? p.cap_c[0] : kCapC[0], c1 = FAR ? p.cap_c[1] : kCapC[1];
    k0 = make_float2(c0 * f0, c0 * f0);
    k1 = make_float2(c1 * f1, c1 * f1);
    // positive also where the cap is so large that it underflows: a hidden
    // score, -inf, then stays -inf (0 times its square would be NaN)
    const float c2 = fmaxf((FAR ? p.cap_c[2] : kCapC[2]) * f2, 1.17549435e-38f);
    k2 = make_float2(c2, c2);
    y_max = f2 <= 3.4028235e38f ? (FAR ? p.cap_y_max : kCapLimit) : -1.f;
  }
  __device__ __forceinline__ bool holds(float abs_max) const { return abs_max * y_mult <= y_max; }
  __device__ __forceinline__ float2 minus(float2 x, float2 neg_mu) const {  // the capped scores - mu
    const float2 t = __fmul2_rn(x, x);
    return __ffma2_rn(__ffma2_rn(__ffma2_rn(k2, t, k1), t, k0), x, neg_mu);
  }
  __device__ __forceinline__ float of(float x) const {
    const float t = x * x;
    return fmaf(fmaf(k2.x, t, k1.x), t, k0.x) * x;
  }
  __device__ __forceinline__ bool far_holds(float x) const { return fabsf(x) * y_mult <= kCapLimit; }
  __device__ __forceinline__ float far(float x, float cap_log2) const {
    const float y = x * y_mult, t = y * y;
    return y * cap_log2 * fmaf(fmaf(fmaf(kCapC3, t, kCapC2), t, kCapC1), t, 1.f);
  }
};

// cap * tanh(score / cap) in log2 units of one raw product: a polynomial, or
// 1 - 2 / (e^2y + 1) from w = 2 y log2(e), above 0.35 of the cap off by less than
// 2^-22 of the cap, 2^-20 of the score.
template <bool FAR>
__device__ __forceinline__ float capped(float x, float w_mult, float cap_log2, const CapPoly<FAR>& poly) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fast_exp2(x * w_mult) + 1.f));
  // (which of the two is written first: 10 % of two-token decode in either case)
  if constexpr (FAR) {
    const float e = fmaf(-2.f * cap_log2, r, cap_log2);
    return poly.far_holds(x) ? poly.far(x, cap_log2) : e;
  } else {
    return poly.holds(fabsf(x)) ? poly.of(x) : fmaf(-2.f * cap_log2, r, cap_log2);
  }
}

}  // namespace pkv
