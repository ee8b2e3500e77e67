// Rotary positions and append in one pass: the new tokens' queries and keys
// are turned by their positions' angles, the queries returned, the keys and
// values written into their cache slots ([SC] "LLM inference: prefill, decode,
// KV cache", section "4. Internal workings", step 5, the append; FP8 E4M3 with
// per-head scales as in append.cu).
//
// Pair i of a head's first rotary_dim elements, (x1, x2) = (x[i], x[i + rd/2])
// in the half layout and (x[2i], x[2i+1]) in the interleaved one, becomes
//   (x1 c - x2 s, x2 c + x1 s),   c = mag cos(pos f_i), s = mag sin(pos f_i);
// the other elements pass through.  All in binary32, rounded once to bf16 or
// quantised once to E4M3.
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
    const uint64_t turn = turn_step(p.inv_freq[threadIdx.x]) * static_cast<uint64_t>(p.positions[tok]);
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
        const int64_t dst = ((blk * hk + h) * p.block_size + (slot & (p.block_size - 1))) * D;
        void* cache = kind == 1 ? p.k_cache : p.v_cache;
        const float sc = DST == kEncE4M3 ? (kind == 1 ? p.k_scale : p.v_scale)[tok * p.scale_stride + h] : 1.f;
        if (turned) {
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
  return bf ? launch_rotary_sd<kEncBF16, kEncE4M3>(p, stream) : launch_rotary_sd<kEncF32, kEncE4M3>(p, stream);
}

}  // namespace pkv
