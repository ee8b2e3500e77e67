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
// integer product, exact up to f_i's own rounding (2^-53 of pos * f_i turns),
// with no reduction and no 64-bit floating point per position.  The top 32
// bits of it are the angle.
//
// A CTA takes TOK tokens: its threads first compute the tokens' (c, s) once
// for all heads into shared memory, then move 16-element items, each read
// whole before it is written (so the queries may be turned in place).  Bound:
// the bytes, each read and written once.

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "decode_common.cuh"

namespace pkv {
namespace {

constexpr int kRotaryThreads = 256;

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

template <int SRC, int DST, bool INTER, int TOK>
__global__ void __launch_bounds__(kRotaryThreads) rotary_append_kernel(const RotaryParams p) {
  __shared__ float2 s_cs[TOK][64];
  __shared__ int64_t s_slot[TOK];
  const int half = p.rotary_dim / 2;
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * TOK;
  const int ntok = static_cast<int>(p.n_tokens - tok0 < TOK ? p.n_tokens - tok0 : TOK);
  wait_prior_grid();
  allow_next_grid();
  for (int i = threadIdx.x; i < ntok * half; i += kRotaryThreads) {
    const int t = i / half, f = i - t * half;
    const uint64_t turn = turn_step(p.inv_freq[f]) * static_cast<uint64_t>(p.positions[tok0 + t]);
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077392578125e-10f, &s, &c);
    s_cs[t][f] = make_float2(c * p.magnitude, s * p.magnitude);
  }
  if (threadIdx.x < ntok) s_slot[threadIdx.x] = p.slots[tok0 + threadIdx.x];
  __syncthreads();

  const int D = p.head_dim, per_row = D / 16, rd16 = p.rotary_dim / 16;
  const int rows = p.num_q_heads + 2 * p.num_kv_heads;  // query, key, value rows of a token
  const int per_tok = rows * per_row;
  for (int idx = threadIdx.x; idx < ntok * per_tok; idx += kRotaryThreads) {
    const int t = TOK == 1 ? 0 : idx / per_tok;
    const int rem = idx - t * per_tok;
    const int row = rem / per_row, c = rem - row * per_row;
    const int64_t tok = tok0 + t;
    // the item's two groups of eight elements within the row
    const bool turned = c < rd16 && row < p.num_q_heads + p.num_kv_heads;
    const int e0 = !INTER && turned ? 8 * c : 16 * c;
    const int e1 = !INTER && turned ? e0 + half : e0 + 8;
    const int kind = row < p.num_q_heads ? 0 : (row < p.num_q_heads + p.num_kv_heads ? 1 : 2);
    const int h = kind == 0 ? row : (kind == 1 ? row - p.num_q_heads : row - p.num_q_heads - p.num_kv_heads);
    int64_t dst = 0;
    if (kind != 0) {
      const int64_t slot = s_slot[t];
      if (slot < 0) continue;
      if (slot >= p.num_slots) {
        if (rem == p.num_q_heads * per_row) record_error(p.err, kDevErrSlot);
        continue;
      }
      const int64_t blk = slot / p.block_size;
      dst = ((blk * p.num_kv_heads + h) * p.block_size + (slot - blk * p.block_size)) * D;
    }
    const void* src = kind == 0 ? p.q : (kind == 1 ? p.k : p.v);
    const int64_t from = tok * (kind == 0 ? p.q_stride : (kind == 1 ? p.k_stride : p.v_stride)) +
                         static_cast<int64_t>(h) * D;
    float x[8], y[8];
    uint4 rx, ry;
    enc_load8<SRC>(src, from + e0, x, rx);
    enc_load8<SRC>(src, from + e1, y, ry);
    if (turned) {
      const float2* cs = &s_cs[t][8 * c];
      if constexpr (INTER) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 a = cs[i], b = cs[4 + i];
          const float u = x[2 * i], w = x[2 * i + 1], u2 = y[2 * i], w2 = y[2 * i + 1];
          x[2 * i] = u * a.x - w * a.y;
          x[2 * i + 1] = w * a.x + u * a.y;
          y[2 * i] = u2 * b.x - w2 * b.y;
          y[2 * i + 1] = w2 * b.x + u2 * b.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 a = cs[i];
          const float u = x[i], w = y[i];
          x[i] = u * a.x - w * a.y;
          y[i] = w * a.x + u * a.y;
        }
      }
    }
    if (kind == 0) {
      const int64_t to = tok * p.out_stride + static_cast<int64_t>(h) * D;
      if (SRC == kEncBF16 && !turned) {  // passed through bit for bit
        enc_store8<SRC, kEncBF16>(p.q_out, to + e0, x, rx, 1.f);
        enc_store8<SRC, kEncBF16>(p.q_out, to + e1, y, ry, 1.f);
      } else {
        store8_bf16(p.q_out, to + e0, x);
        store8_bf16(p.q_out, to + e1, y);
      }
    } else {
      void* cache = kind == 1 ? p.k_cache : p.v_cache;
      const float sc = DST == kEncE4M3 ? (kind == 1 ? p.k_scale : p.v_scale)[tok * p.scale_stride + h] : 1.f;
      if (turned) {
        enc_store8<kEncF32, DST>(cache, dst + e0, x, rx, sc);
        enc_store8<kEncF32, DST>(cache, dst + e1, y, ry, sc);
      } else {
        enc_store8<SRC, DST>(cache, dst + e0, x, rx, sc);
        enc_store8<SRC, DST>(cache, dst + e1, y, ry, sc);
      }
    }
  }
}

template <int SRC, int DST, bool INTER>
cudaError_t launch_rotary_t(const RotaryParams& p, cudaStream_t stream) {
  // one token per CTA while that leaves SMs idle, else four, so that every
  // thread computes one angle of the CTA's tokens
  if (p.n_tokens <= 152 * 4)
    return launch_pdl(rotary_append_kernel<SRC, DST, INTER, 1>, dim3(static_cast<unsigned>(p.n_tokens)),
                      dim3(kRotaryThreads), 0, stream, p);
  return launch_pdl(rotary_append_kernel<SRC, DST, INTER, 4>, dim3(static_cast<unsigned>((p.n_tokens + 3) / 4)),
                    dim3(kRotaryThreads), 0, stream, p);
}

template <int SRC, int DST>
cudaError_t launch_rotary_sd(const RotaryParams& p, cudaStream_t stream) {
  return p.interleaved ? launch_rotary_t<SRC, DST, true>(p, stream) : launch_rotary_t<SRC, DST, false>(p, stream);
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, cudaStream_t stream) {
  const bool bf = p.src_dtype == kEncBF16;
  if (p.cache_dtype == kEncBF16)
    return bf ? launch_rotary_sd<kEncBF16, kEncBF16>(p, stream) : launch_rotary_sd<kEncF32, kEncBF16>(p, stream);
  return bf ? launch_rotary_sd<kEncBF16, kEncE4M3>(p, stream) : launch_rotary_sd<kEncF32, kEncE4M3>(p, stream);
}

}  // namespace pkv
