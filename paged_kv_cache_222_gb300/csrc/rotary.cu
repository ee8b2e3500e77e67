// Rotary positions and append in one pass: the new tokens' queries and keys
// are turned by their positions' angles, the queries returned, the keys and
// values written into their cache slots ([SC] "LLM inference: prefill, decode,
// KV cache", section "4. Internal workings", step 5, the append; FP8 E4M3 with
// per-head scales as in append.cu).
//
// Pair i of a head's first rotary_dim elements, (x1, x2) = (x[i], x[i + rd/2])
// in the half layout and (x[2i], x[2i+1]) in the interleaved one, becomes
//   (x1 c - x2 s, x2 c + x1 s),   c = mag cos(pos f_i), s = mag sin(pos f_i);
// the other elements pass through.  With several axes (time, height, width of
// images and video) pos is the token's position along the pair's own axis.  All
// in binary32, rounded once to bf16 or
// quantised once to E4M3 or E2M1 (whose groups of 16 elements may lie in two
// items: their largest magnitudes are exchanged between the row's lanes).
//
// Angles of far positions: f_i / 2 pi is taken as a 64-bit fixed-point
// fraction of a turn, so that pos * f_i modulo one turn is one wrapping 64-bit
// integer product, with no reduction and no 64-bit floating point per position.
// 1 / 2 pi and its product with f_i are each rounded to 53 bits and the fraction
// to 2^-64, which the product multiplies: at most |pos f_i| 2^-52 radians + |pos|
// 2^-65 turns, 2^-21 + 2^-31 radians at |pos f_i| = 2^31.  The top 32 bits of the
// product are the angle, rounded to binary32 (2^-25 of a turn).
//
// A CTA of 128 threads takes one token: its threads compute the token's (c, s)
// once for all heads into shared memory, under the first item's loads, then
// move 16-element items, the next one's loads in flight while one is turned
// and stored; an item is read whole before it is written, so the queries may
// be turned in place.  Bound: the bytes, each read and written once: 8192
// tokens of 64 + 8 heads of 128 (336 MB) take 55 us, 6.1 TB/s, 91 % of the
// measured copy (256 threads and four tokens per CTA 62 us, eight tokens 64 us;
// 32 registers fewer per thread for more resident CTAs spill: 100 us); 64
// tokens 3.8 us on the GPU, the latency of a position, its angles and a store.

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "decode_common.cuh"

namespace pkv {
namespace {

constexpr int kRotaryThreads = 128;

__device__ __forceinline__ uint64_t turn_step(double f) {
  double t = f * 0.15915494309189533577;  // 1 / 2 pi
  t -= floor(t);
  return __double2ull_rn(t * 18446744073709551616.0);  // 2^64
}

// Eight bf16 results at element `elem`.
__device__ __forceinline__ void store8_bf16(void* base, int64_t elem, const float (&x)[8]) {
  uint4 o;
  o.x = pack_bf16x2(x[0], x[1]);
  o.y = pack_bf16x2(x[2], x[3]);
  o.z = pack_bf16x2(x[4], x[5]);
  o.w = pack_bf16x2(x[6], x[7]);
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + elem) = o;
}

// Eight source elements as they lie in memory.
template <int SRC>
struct Raw8 {
  uint4 w[SRC == kEncBF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* base, int64_t elem) {
    if constexpr (SRC == kEncBF16) {
      w[0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + elem);
    } else {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + elem);
      w[0] = p[0];
      w[1] = p[1];
    }
  }
  __device__ __forceinline__ void widen(float (&x)[8]) const {
    if constexpr (SRC == kEncBF16) {
      const uint32_t v[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16lo_to_f32(v[i]);
        x[2 * i + 1] = bf16hi_to_f32(v[i]);
      }
    } else {
      const uint32_t v[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(v[i]);
    }
  }
};

// The lanes of a row (D / 16, all of them here) hold its elements in pieces of
// eight: this one x, piece px, and y, piece py.  Which lane holds a piece, and
// as which of the two: in the half layout pieces below half_pieces are x of
// their own number's lane and those up to turned_pieces y, half_pieces further
// on; any other lies at its place.  A group's scale needs both of its pieces'
// largest magnitude.
template <int D>
__device__ __forceinline__ void store_e2m1(uint8_t* tile, int block_size, int off, int px, int py, int half_pieces,
                                           int turned_pieces, float (&x)[8], float (&y)[8], float scale, bool scaled) {
  constexpr int LANES = D / 16;
  const int lane = threadIdx.x & 31, first = lane & ~(LANES - 1);
  const unsigned mask = ((1u << LANES) - 1u) << first;
  if (scaled) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = __fdiv_rn(x[i], scale);
      y[i] = __fdiv_rn(y[i], scale);
    }
  }
  const float mx = abs_max8(x), my = abs_max8(y);
  auto from = [&](int piece) {  // the largest magnitude of a piece
    const bool split = piece < turned_pieces && half_pieces > 0;
    const bool low = split && piece < half_pieces;
    const int at = first + (split ? (low ? piece : piece - half_pieces) : piece / 2);
    const float a = __shfl_sync(mask, mx, at), b = __shfl_sync(mask, my, at);
    return (split ? low : piece % 2 == 0) ? a : b;
  };
  const float gx = max_nan(mx, from(px ^ 1)), gy = max_nan(my, from(py ^ 1));  // of the pieces' groups
  const uint8_t sx = e2m1_group_scale(gx), sy = e2m1_group_scale(gy);
  uint8_t* codes = tile + off * (D / 2);
  uint8_t* scales = tile + block_size * (D / 2) + off * LANES;
  *reinterpret_cast<uint32_t*>(codes + px * 4) = e2m1_codes8<false>(x, gx, sx);
  *reinterpret_cast<uint32_t*>(codes + py * 4) = e2m1_codes8<false>(y, gy, sy);
  if (px % 2 == 0) scales[px / 2] = sx;
  if (py % 2 == 0) scales[py / 2] = sy;
}

template <int D, int SRC, int DST, bool INTER>
__global__ void __launch_bounds__(kRotaryThreads) rotary_append_kernel(const RotaryParams p) {
  __shared__ __align__(16) float2 s_cs[D / 2];  // read two at a time
  constexpr int PER_ROW = D / 16;                         // items of a row
  constexpr int PASS = kRotaryThreads / PER_ROW;          // rows per pass of the CTA
  const int half = p.rotary_dim / 2;
  const int hq = p.num_q_heads, hk = p.num_kv_heads;
  const int rows = hq + 2 * hk;                           // query, key, value rows of a token
  const int64_t tok = blockIdx.x;
  const int c = threadIdx.x % PER_ROW;                    // this thread's items: number c of its rows
  const bool inside = c < p.rotary_dim / 16;              // ... which turn (query and key rows)

  struct Item {
    Raw8<SRC> x, y;  // its two groups of eight elements
    int r;           // row of the token
  };
  int r = threadIdx.x / PER_ROW;                          // of the next item
  auto load = [&](Item& it) {
    it.r = r;
    if (r >= rows) return;
    const int kind = r < hq ? 0 : (r < hq + hk ? 1 : 2);
    const int h = kind == 0 ? r : (kind == 1 ? r - hq : r - hq - hk);
    const bool turned = inside && kind != 2;
    const int e0 = !INTER && turned ? 8 * c : 16 * c;
    const int e1 = !INTER && turned ? e0 + half : e0 + 8;
    const void* src = kind == 0 ? p.q : (kind == 1 ? p.k : p.v);
    const int64_t from = tok * (kind == 0 ? p.q_stride : (kind == 1 ? p.k_stride : p.v_stride)) + h * D;
    it.x.load(src, from + e0);
    it.y.load(src, from + e1);
    r += PASS;
  };
  wait_prior_grid();
  allow_next_grid();
  Item cur;
  load(cur);  // in flight while the angles are computed
  const int64_t slot = p.slots[tok];
  if (threadIdx.x < half) {
    const int axis = p.axes != nullptr ? p.axes[threadIdx.x] : 0;
    int64_t pos = 0;  // an axis that is none: not turned
    if (axis >= 0 && axis < p.num_axes)
      pos = p.positions[axis * p.position_stride + tok];
    else
      record_error(p.err, kDevErrAxis);
    const uint64_t turn = turn_step(p.inv_freq[threadIdx.x]) * static_cast<uint64_t>(pos);
    float sn, cs;
    sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077392578125e-10f, &sn, &cs);
    s_cs[threadIdx.x] = make_float2(cs * p.magnitude, sn * p.magnitude);
  }
  __syncthreads();

  while (cur.r < rows) {
    Item next;
    load(next);  // in flight while this one is turned and stored
    const int kind = cur.r < hq ? 0 : (cur.r < hq + hk ? 1 : 2);
    const int h = kind == 0 ? cur.r : (kind == 1 ? cur.r - hq : cur.r - hq - hk);
    const bool turned = inside && kind != 2;
    const int e0 = !INTER && turned ? 8 * c : 16 * c;
    const int e1 = !INTER && turned ? e0 + half : e0 + 8;
    float x[8], y[8];
    cur.x.widen(x);
    cur.y.widen(y);
    if (turned) {
      const float4* cs = reinterpret_cast<const float4*>(&s_cs[8 * c]);  // two (cos, sin) each
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 a = cs[i];
        if constexpr (INTER) {  // pairs 8c + 2i, 8c + 2i + 1 of the row
          float* v = i < 2 ? x + 4 * i : y + 4 * (i - 2);
          const float u0 = v[0], w0 = v[1], u1 = v[2], w1 = v[3];
          v[0] = u0 * a.x - w0 * a.y;
          v[1] = w0 * a.x + u0 * a.y;
          v[2] = u1 * a.z - w1 * a.w;
          v[3] = w1 * a.z + u1 * a.w;
        } else {
          const float u0 = x[2 * i], w0 = y[2 * i], u1 = x[2 * i + 1], w1 = y[2 * i + 1];
          x[2 * i] = u0 * a.x - w0 * a.y;
          y[2 * i] = w0 * a.x + u0 * a.y;
          x[2 * i + 1] = u1 * a.z - w1 * a.w;
          y[2 * i + 1] = w1 * a.z + u1 * a.w;
        }
      }
    }
    if (kind == 0) {
      const int64_t to = tok * p.out_stride + h * D;
      if (SRC == kEncBF16 && !turned) {  // passed through bit for bit
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.q_out) + to + e0) = cur.x.w[0];
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.q_out) + to + e1) = cur.y.w[0];
      } else {
        store8_bf16(p.q_out, to + e0, x);
        store8_bf16(p.q_out, to + e1, y);
      }
    } else {
      if (slot >= p.num_slots) {
        if (cur.r == hq && c == 0) record_error(p.err, kDevErrSlot);
      } else if (slot >= 0) {
        const int64_t blk = p.block_size == 16 ? slot >> 4 : slot >> 5;
        const int off = static_cast<int>(slot & (p.block_size - 1));
        const int64_t dst = ((blk * hk + h) * p.block_size + off) * D;
        void* cache = kind == 1 ? p.k_cache : p.v_cache;
        const float* scales = kind == 1 ? p.k_scale : p.v_scale;
        const float sc = DST != kEncBF16 && scales != nullptr ? scales[tok * p.scale_stride + h] : 1.f;
        if constexpr (DST == kEncE2M1) {
          store_e2m1<D>(static_cast<uint8_t*>(cache) + (blk * hk + h) * e2m1_tile_bytes(D, p.block_size), p.block_size,
                        off, e0 / 8, e1 / 8, turned && !INTER ? half / 8 : 0, p.rotary_dim / 8, x, y, sc, scales != nullptr);
        } else if (turned) {
          enc_store8<kEncF32, DST>(cache, dst + e0, x, uint4{}, sc);
          enc_store8<kEncF32, DST>(cache, dst + e1, y, uint4{}, sc);
        } else {
          enc_store8<SRC, DST>(cache, dst + e0, x, cur.x.w[0], sc);
          enc_store8<SRC, DST>(cache, dst + e1, y, cur.y.w[0], sc);
        }
      }
    }
    cur = next;
  }
}

template <int D, int SRC, int DST, bool INTER>
cudaError_t launch_rotary_t(const RotaryParams& p, cudaStream_t stream) {
  return launch_pdl(rotary_append_kernel<D, SRC, DST, INTER>, dim3(static_cast<unsigned>(p.n_tokens)),
                    dim3(kRotaryThreads), 0, stream, p);
}

template <int SRC, int DST>
cudaError_t launch_rotary_sd(const RotaryParams& p, cudaStream_t stream) {
  if (p.head_dim == 128)
    return p.interleaved ? launch_rotary_t<128, SRC, DST, true>(p, stream)
                         : launch_rotary_t<128, SRC, DST, false>(p, stream);
  return p.interleaved ? launch_rotary_t<64, SRC, DST, true>(p, stream)
                       : launch_rotary_t<64, SRC, DST, false>(p, stream);
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, cudaStream_t stream) {
  const bool bf = p.src_dtype == kEncBF16;
  if (p.cache_dtype == kEncBF16)
    return bf ? launch_rotary_sd<kEncBF16, kEncBF16>(p, stream) : launch_rotary_sd<kEncF32, kEncBF16>(p, stream);
  if (p.cache_dtype == kEncE2M1)
    return bf ? launch_rotary_sd<kEncBF16, kEncE2M1>(p, stream) : launch_rotary_sd<kEncF32, kEncE2M1>(p, stream);
  return bf ? launch_rotary_sd<kEncBF16, kEncE4M3>(p, stream) : launch_rotary_sd<kEncF32, kEncE4M3>(p, stream);
}

}  // namespace pkv
