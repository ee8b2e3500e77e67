// KV append: scatter each new token's K/V rows into their cache slots, copying
// bf16 or quantising to FP8 E4M3 with a per-row, per-KV-head scale.
//
// What it computes: [SC] "LLM inference: prefill, decode, KV cache", section
// "4. Internal workings", step 5 (the new token's K/V are appended to the
// cache); FP8 E4M3 with per-head scales: [FN] "Sub-Millisecond Token
// Scheduling...", FAQ "How much HBM memory does FP8 KV-cache quantization
// save?".  Slot = physical_block * block_size + offset, negative = skip.
//
// Mapping: one thread per 8 consecutive elements of one (token, head) row, so a
// warp moves 2 (D=128) or 4 (D=64) whole rows with 16-byte (bf16) or 8-byte
// (E4M3) stores; loads are 16-byte (bf16 source) or 2x16-byte (f32 source).
// Grid-stride, so any number of rows fits a bounded grid.
//
// E2M1 caches: a thread per group of 16 elements, 8 code bytes and a scale byte
// (how codes are found without dividing by it: pkv_device.cuh).  Bound: a thread's
// loads and then its codes (14 instructions per element), so that neither HBM nor the
// ALU (58 %) is full: 16,384 tokens of 8 heads of 128 from bf16 20 us, 4.3 TB/s; 8
// elements of K and of V per thread, whose group's largest magnitude two lanes
// exchange, 26-34 us.  Head scales divide every element first: 65,536 such tokens 114
// us, without 65.
//
// read_kernel is the way back: a thread per 8 elements of a (token, head) row
// widens them (codes times scales; every code and code-times-scale product is
// exact in binary32), multiplies by the head's scale and rounds once.  16,384
// tokens of 8 heads of 128 from E2M1 to bf16 17.9 us, 4.8 TB/s; 16 elements per
// thread, whose 32-byte pieces of lines are written in two halves, 22.
//
// The slot-mapping kernel turns (sequence, logical position) pairs into those
// flat slots through the block tables ([SC] "PagedAttention & Memory
// Management (vLLM)": logical block j of a sequence lives in the physical
// block its table names).

#include "decode_common.cuh"

namespace pkv {
namespace {

constexpr int kBF16 = kEncBF16, kF32 = kEncF32;

template <int SRC, int DST>
__global__ void __launch_bounds__(256) append_kernel(AppendParams p) {
  // Let the next kernel in the stream start launching now (it waits for this
  // grid to finish before it reads anything), then wait for the previous one:
  // a slot written here may be one it still reads.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int D = p.head_dim;
  const int H = p.num_kv_heads;
  const int per_row = D / 8;
  const int64_t total = p.n_tokens * H * per_row;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t idx = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; idx < total;
       idx += stride) {
    const int64_t row = idx / per_row;  // token * H + head
    const int part = static_cast<int>(idx - row * per_row);
    const int64_t tok = row / H;
    const int h = static_cast<int>(row - tok * H);
    const int64_t slot = p.slots[tok];
    if (slot < 0) continue;
    if (slot >= p.num_slots) {
      if (part == 0 && h == 0) record_error(p.err, kDevErrSlot);
      continue;
    }
    const int64_t blk = slot / p.block_size;
    const int64_t off = slot - blk * p.block_size;
    const int64_t src_elem = row * D + part * 8;
    const int64_t dst_elem = ((blk * H + h) * p.block_size + off) * D + part * 8;
    float ks = 1.f, vs = 1.f;
    if constexpr (DST == kE4M3) {
      ks = p.k_scale[tok * p.scale_stride + h];
      vs = p.v_scale[tok * p.scale_stride + h];
    }
    float x[8];
    uint4 raw;
    enc_load8<SRC>(p.k_new, src_elem, x, raw);
    enc_store8<SRC, DST>(p.k_cache, dst_elem, x, raw, ks);
    enc_load8<SRC>(p.v_new, src_elem, x, raw);
    enc_store8<SRC, DST>(p.v_cache, dst_elem, x, raw, vs);
  }
}

// Pieces of (token, head) rows, `per_tok` of a token: a CTA takes whole tokens,
// threadIdx.y one of them and threadIdx.x its piece, so that nothing is divided.
template <class F>
__device__ __forceinline__ void for_pieces(int64_t n_tokens, int per_tok, F&& f) {
  for (int64_t tok = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y; tok < n_tokens;
       tok += static_cast<int64_t>(gridDim.x) * blockDim.y)
    for (int i = threadIdx.x; i < per_tok; i += blockDim.x) f(tok, i);
}

// Byte of a block's first tile: blocks and a block's bytes are 32-bit numbers.
__device__ __forceinline__ int64_t tile_at(int64_t block, int block_bytes) {
  return static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(block)) * static_cast<uint32_t>(block_bytes));
}

// A thread per group of 16 elements of K or of V.  SCALED: with heads' scales.
// From bf16, held to the 40 registers of 6 CTAs per SM (45 and 5: 24.2 us for 21.9; 7
// CTAs 25.7).
template <int SRC, bool SCALED>
__global__ void __launch_bounds__(256, SRC == kBF16 ? 6 : 1) append_e2m1_kernel(AppendParams p) {
  wait_prior_grid();
  allow_next_grid();
  const int D = p.head_dim, H = p.num_kv_heads, shift = p.block_size == 16 ? 4 : 5, to_row = D == 128 ? 3 : 2;
  const int tile = e2m1_tile_bytes(D, p.block_size), groups = H << to_row;
  for_pieces(p.n_tokens, 2 * groups, [&](int64_t tok, int i) {
    const int64_t slot = p.slots[tok];
    const bool kv = i >= groups;
    const int g = kv ? i - groups : i, h = g >> to_row, part = g & ((1 << to_row) - 1);
    const uint4* from = reinterpret_cast<const uint4*>(static_cast<const char*>(kv ? p.v_new : p.k_new) +
                                                       (tok * (H * D) + g * 16) * (SRC == kBF16 ? 2 : 4));
    uint4 w[SRC == kBF16 ? 2 : 4];
#pragma unroll
    for (int q = 0; q < (SRC == kBF16 ? 2 : 4); ++q) w[q] = from[q];
    if (slot < 0) return;
    if (slot >= p.num_slots) {
      if (i == 0) record_error(p.err, kDevErrSlot);
      return;
    }
    float x[2][8], amax;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if constexpr (SRC == kBF16) {
        const uint32_t v[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[q][2 * e] = bf16lo_to_f32(v[e]);
          x[q][2 * e + 1] = bf16hi_to_f32(v[e]);
        }
      } else {
        const uint4 a = w[SRC == kBF16 ? 0 : 2 * q], c = w[SRC == kBF16 ? 0 : 2 * q + 1];
        const uint32_t v[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) x[q][e] = __uint_as_float(v[e]);
      }
      if constexpr (SCALED) {
        const float s = (kv ? p.v_scale : p.k_scale)[tok * p.scale_stride + h];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[q][e] = __fdiv_rn(x[q][e], s);
      }
    }
    if constexpr (SRC == kBF16 && !SCALED) {  // on pairs
      uint32_t m = 0u;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t v[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) m = max_nan_bf16x2(m, v[e] & 0x7FFF7FFFu);
      }
      amax = max_nan(bf16lo_to_f32(m), bf16hi_to_f32(m));
    } else {
      amax = max_nan(abs_max8(x[0]), abs_max8(x[1]));
    }
    const int off = static_cast<int>(slot) & (p.block_size - 1);
    uint8_t* to = static_cast<uint8_t*>(kv ? p.v_cache : p.k_cache) + tile_at(slot >> shift, H * tile) + h * tile;
    const uint8_t sc = e2m1_group_scale(amax);
    constexpr bool SHORT = SRC == kBF16 && !SCALED;
    *reinterpret_cast<uint2*>(to + off * (D / 2) + part * 8) =
        make_uint2(e2m1_codes8<SHORT>(x[0], amax, sc), e2m1_codes8<SHORT>(x[1], amax, sc));
    to[p.block_size * (D / 2) + off * (D / 16) + part] = sc;
  });
}

// Eight elements of a row, piece `part` of it, as they lie in the tile of their
// block and head.
template <int SRC>
struct Raw8 {
  uint4 w;
  __device__ __forceinline__ void load(const uint8_t* tile, int D, int block_size, int off, int part) {
    if constexpr (SRC == kBF16) {
      w = *reinterpret_cast<const uint4*>(tile + (off * D + part * 8) * 2);
    } else if constexpr (SRC == kE4M3) {
      const uint2 c = *reinterpret_cast<const uint2*>(tile + off * D + part * 8);
      w.x = c.x;
      w.y = c.y;
    } else {
      w.x = *reinterpret_cast<const uint32_t*>(tile + off * (D / 2) + part * 4);
      w.y = tile[block_size * (D / 2) + off * (D / 16) + part / 2];
    }
  }
  __device__ __forceinline__ void widen(float (&x)[8]) const {
    if constexpr (SRC == kBF16) {
      const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16lo_to_f32(v[i]);
        x[2 * i + 1] = bf16hi_to_f32(v[i]);
      }
    } else {
      uint32_t h[4];
      if constexpr (SRC == kE4M3) {
        h[0] = e4m3x2_to_f16x2(static_cast<uint16_t>(w.x & 0xFFFFu));
        h[1] = e4m3x2_to_f16x2(static_cast<uint16_t>(w.x >> 16));
        h[2] = e4m3x2_to_f16x2(static_cast<uint16_t>(w.y & 0xFFFFu));
        h[3] = e4m3x2_to_f16x2(static_cast<uint16_t>(w.y >> 16));
      } else {
        const uint32_t s = e4m3x2_to_f16x2(static_cast<uint16_t>(w.y | (w.y << 8)));
        e2m1x8_to_f16x2(w.x, h);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = mul_f16x2(h[i], s);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = f16lo_to_f32(h[i]);
        x[2 * i + 1] = f16hi_to_f32(h[i]);
      }
    }
  }
};

// Eight results at element `elem`.
template <int DST>
__device__ __forceinline__ void store8(void* base, int64_t elem, const float (&x)[8]) {
  if constexpr (DST == kBF16) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + elem) =
        make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  } else {
    float4* to = reinterpret_cast<float4*>(static_cast<float*>(base) + elem);
    to[0] = make_float4(x[0], x[1], x[2], x[3]);
    to[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// A thread per 8 elements of K and of V: 16 bytes of bf16, so that a warp writes
// whole lines.
template <int SRC, int DST>
__global__ void __launch_bounds__(256) read_kernel(ReadParams p) {
  wait_prior_grid();
  allow_next_grid();
  const int D = p.head_dim, H = p.num_kv_heads, shift = p.block_size == 16 ? 4 : 5, to_row = D == 128 ? 4 : 3;
  const int tile = SRC == kE2M1 ? e2m1_tile_bytes(D, p.block_size) : p.block_size * D * (SRC == kBF16 ? 2 : 1);
  for_pieces(p.n_tokens, H << to_row, [&](int64_t tok, int i) {
    const int64_t slot = p.slots[tok], to = tok * (H * D) + i * 8;
    if (slot < 0 || slot >= p.num_slots) {
      if (slot >= 0 && i == 0) record_error(p.err, kDevErrSlot);
      const float zero[8] = {};
      store8<DST>(p.k_out, to, zero);
      store8<DST>(p.v_out, to, zero);
      return;
    }
    const int h = i >> to_row, part = i & ((1 << to_row) - 1);
    const int64_t base = tile_at(slot >> shift, H * tile) + h * tile;
    const int off = static_cast<int>(slot) & (p.block_size - 1);
    Raw8<SRC> raw[2];  // K's and V's, read together
    raw[0].load(static_cast<const uint8_t*>(p.k_cache) + base, D, p.block_size, off, part);
    raw[1].load(static_cast<const uint8_t*>(p.v_cache) + base, D, p.block_size, off, part);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      void* out = kv ? p.v_out : p.k_out;
      if constexpr (SRC == kBF16 && DST == kBF16) {  // bit for bit
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + to) = raw[kv].w;
      } else {
        float x[8];
        raw[kv].widen(x);
        const float* scale = kv ? p.v_scale : p.k_scale;
        if (scale != nullptr) {
          const float s = scale[tok * p.scale_stride + h];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= s;
        }
        store8<DST>(out, to, x);
      }
    }
  });
}

// Slot of each new token: the block table's entry for the token's logical
// block, times the block size, plus its offset in the block.  One thread per
// token; a negative position is padding (slot -1, nothing recorded).
__global__ void __launch_bounds__(256) slot_mapping_kernel(SlotParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  const int64_t cap = static_cast<int64_t>(p.max_blocks) * p.block_size;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < p.n; i += stride) {
    const int64_t pos = p.positions[i];
    int64_t slot = -1;
    if (pos >= 0) {
      const int64_t seq = p.seq_index != nullptr ? p.seq_index[i] : i;
      if (seq < 0 || seq >= p.num_seqs || pos >= cap) {
        record_error(p.err, kDevErrContextLen);
      } else {
        const int64_t j = pos / p.block_size;
        const int32_t blk = p.block_tables[seq * p.max_blocks + j];
        if (blk < 0 || blk >= p.num_blocks)
          record_error(p.err, kDevErrBlockId);
        else
          slot = static_cast<int64_t>(blk) * p.block_size + (pos - j * p.block_size);
      }
    }
    p.slots[i] = slot;
  }
}

// for_pieces over tokens of `per_tok` pieces.
template <class P>
cudaError_t launch_pieces(void (*kern)(P), const P& p, int64_t per_tok, cudaStream_t stream) {
  const dim3 block = per_tok < 256 ? dim3(static_cast<unsigned>(per_tok), static_cast<unsigned>(256 / per_tok)) : dim3(256);
  const int64_t want = (p.n_tokens + block.y - 1) / block.y;
  // two waves of the six CTAs that an SM holds (8192 tokens of 8 heads of 128 appended
  // and read back 19.4 us; one wave 20.8, four 19.5, a CTA per two tokens 20.1)
  return launch_pdl(kern, dim3(static_cast<unsigned>(want < 152 * 12 ? want : 152 * 12)), block, 0, stream, p);
}

}  // namespace

cudaError_t launch_slot_mapping(const SlotParams& p, cudaStream_t stream) {
  if (p.n == 0) return cudaSuccess;
  const int threads = 256;
  const int64_t want = (p.n + threads - 1) / threads;
  const int blocks = static_cast<int>(want < 152 * 8 ? want : 152 * 8);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, slot_mapping_kernel, p);
}

cudaError_t launch_read(const ReadParams& p, cudaStream_t stream) {
  void (*kern)(ReadParams);
  const bool bf = p.out_dtype == kBF16;
  if (p.cache_dtype == kBF16)
    kern = bf ? read_kernel<kBF16, kBF16> : read_kernel<kBF16, kF32>;
  else if (p.cache_dtype == kE4M3)
    kern = bf ? read_kernel<kE4M3, kBF16> : read_kernel<kE4M3, kF32>;
  else
    kern = bf ? read_kernel<kE2M1, kBF16> : read_kernel<kE2M1, kF32>;
  return launch_pieces(kern, p, static_cast<int64_t>(p.num_kv_heads) * (p.head_dim / 8), stream);
}

cudaError_t launch_append(const AppendParams& p, cudaStream_t stream) {
  if (p.cache_dtype == kE2M1) {
    const bool bf = p.src_dtype == kBF16, scaled = p.k_scale != nullptr;
    return launch_pieces(scaled ? (bf ? append_e2m1_kernel<kBF16, true> : append_e2m1_kernel<kF32, true>)
                                : (bf ? append_e2m1_kernel<kBF16, false> : append_e2m1_kernel<kF32, false>),
                         p, static_cast<int64_t>(p.num_kv_heads) * (p.head_dim / 8), stream);
  }
  const int64_t work = p.n_tokens * p.num_kv_heads * (p.head_dim / 8);
  if (work == 0) return cudaSuccess;
  const int threads = 256;
  const int64_t want = (work + threads - 1) / threads;
  const int blocks = static_cast<int>(want < 152 * 32 ? want : 152 * 32);
  void (*kern)(AppendParams);
  if (p.cache_dtype == kBF16)
    kern = p.src_dtype == kBF16 ? append_kernel<kBF16, kBF16> : append_kernel<kF32, kBF16>;
  else
    kern = p.src_dtype == kBF16 ? append_kernel<kBF16, kE4M3> : append_kernel<kF32, kE4M3>;
  // programmatic dependent launch: may be scheduled while the previous kernel
  // drains; the kernel itself waits for it before touching memory
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace pkv
