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
// E2M1 caches: a thread per group of 16 elements, which it reads whole, scales
// and packs into 8 code bytes and a scale byte (pkv_device.cuh).
//
// read_kernel is the way back: a thread per 16 elements of a (token, head) row
// widens them (codes times scales; every code and code-times-scale product is
// exact in binary32), multiplies by the head's scale and rounds once.
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

template <int SRC>
__global__ void __launch_bounds__(256) append_e2m1_kernel(AppendParams p) {
  wait_prior_grid();
  allow_next_grid();
  const int D = p.head_dim, H = p.num_kv_heads;
  const int per_row = D / kE2M1Group;
  const int64_t total = p.n_tokens * H * per_row;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  const int64_t tile = e2m1_tile_bytes(D, p.block_size);
  for (int64_t idx = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; idx < total; idx += stride) {
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
    const int off = static_cast<int>(slot - blk * p.block_size);
    const int64_t base = (blk * H + h) * tile;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      float x[2][8];
      uint4 raw;
      const void* src = kv ? p.v_new : p.k_new;
      enc_load8<SRC>(src, row * D + part * kE2M1Group, x[0], raw);
      enc_load8<SRC>(src, row * D + part * kE2M1Group + 8, x[1], raw);
      const float* scale = kv ? p.v_scale : p.k_scale;
      if (scale != nullptr) {
        const float s = scale[tok * p.scale_stride + h];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[0][i] = __fdiv_rn(x[0][i], s);
          x[1][i] = __fdiv_rn(x[1][i], s);
        }
      }
      const uint8_t sc = e2m1_group_scale(max_nan(abs_max8(x[0]), abs_max8(x[1])));
      uint8_t* to = static_cast<uint8_t*>(kv ? p.v_cache : p.k_cache) + base;
      *reinterpret_cast<uint2*>(to + off * (D / 2) + part * 8) =
          make_uint2(e2m1_codes8(x[0], sc), e2m1_codes8(x[1], sc));
      to[p.block_size * (D / 2) + off * per_row + part] = sc;
    }
  }
}

// Sixteen results at element `elem`.
template <int DST>
__device__ __forceinline__ void store16(void* base, int64_t elem, const float (&x)[16]) {
  if constexpr (DST == kBF16) {
    uint4* to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + elem);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      to[i] = make_uint4(pack_bf16x2(x[8 * i], x[8 * i + 1]), pack_bf16x2(x[8 * i + 2], x[8 * i + 3]),
                         pack_bf16x2(x[8 * i + 4], x[8 * i + 5]), pack_bf16x2(x[8 * i + 6], x[8 * i + 7]));
  } else {
    float4* to = reinterpret_cast<float4*>(static_cast<float*>(base) + elem);
#pragma unroll
    for (int i = 0; i < 4; ++i) to[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  }
}

// Eight f16x2 as floats.
__device__ __forceinline__ void widen16(const uint32_t (&h)[8], float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = f16lo_to_f32(h[i]);
    x[2 * i + 1] = f16hi_to_f32(h[i]);
  }
}

template <int SRC, int DST>
__global__ void __launch_bounds__(256) read_kernel(ReadParams p) {
  wait_prior_grid();
  allow_next_grid();
  const int D = p.head_dim, H = p.num_kv_heads;
  const int per_row = D / 16;
  const int64_t total = p.n_tokens * H * per_row;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  const int64_t tile = SRC == kE2M1 ? e2m1_tile_bytes(D, p.block_size)
                                    : static_cast<int64_t>(p.block_size) * D * (SRC == kBF16 ? 2 : 1);
  for (int64_t idx = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; idx < total; idx += stride) {
    const int64_t row = idx / per_row;  // token * H + head
    const int part = static_cast<int>(idx - row * per_row);
    const int64_t tok = row / H;
    const int h = static_cast<int>(row - tok * H);
    const int64_t slot = p.slots[tok];
    const bool live = slot >= 0 && slot < p.num_slots;
    if (slot >= p.num_slots && part == 0 && h == 0) record_error(p.err, kDevErrSlot);
    const int64_t blk = live ? slot / p.block_size : 0;
    const int off = live ? static_cast<int>(slot - blk * p.block_size) : 0;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      float x[16];
      if (live) {
        const uint8_t* from = static_cast<const uint8_t*>(kv ? p.v_cache : p.k_cache) + (blk * H + h) * tile;
        uint32_t hw[8];
        if constexpr (SRC == kBF16) {
          const uint4* q = reinterpret_cast<const uint4*>(from + (off * D + part * 16) * 2);
          const uint4 a = q[0], b = q[1];
          if constexpr (DST == kBF16) {  // bit for bit
            uint4* to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(kv ? p.v_out : p.k_out) + row * D + part * 16);
            to[0] = a;
            to[1] = b;
            continue;
          }
          const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[2 * i] = bf16lo_to_f32(w[i]);
            x[2 * i + 1] = bf16hi_to_f32(w[i]);
          }
        } else if constexpr (SRC == kE4M3) {
          const uint4 a = *reinterpret_cast<const uint4*>(from + off * D + part * 16);
          const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            hw[2 * i] = e4m3x2_to_f16x2(static_cast<uint16_t>(w[i] & 0xFFFFu));
            hw[2 * i + 1] = e4m3x2_to_f16x2(static_cast<uint16_t>(w[i] >> 16));
          }
          widen16(hw, x);
        } else {
          const uint2 a = *reinterpret_cast<const uint2*>(from + off * (D / 2) + part * 8);
          const uint32_t sc = from[p.block_size * (D / 2) + off * per_row + part];
          const uint32_t s2 = e4m3x2_to_f16x2(static_cast<uint16_t>(sc | (sc << 8)));
          uint32_t lo[4], hi[4];
          e2m1x8_to_f16x2(a.x, lo);
          e2m1x8_to_f16x2(a.y, hi);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            hw[i] = mul_f16x2(lo[i], s2);
            hw[4 + i] = mul_f16x2(hi[i], s2);
          }
          widen16(hw, x);
        }
        const float* scale = kv ? p.v_scale : p.k_scale;
        if (scale != nullptr) {
          const float s = scale[tok * p.scale_stride + h];
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] *= s;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = 0.f;
      }
      store16<DST>(kv ? p.v_out : p.k_out, row * D + part * 16, x);
    }
  }
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
  const int64_t want = (p.n_tokens * p.num_kv_heads * (p.head_dim / 16) + 255) / 256;
  const dim3 grid(static_cast<unsigned>(want < 152 * 32 ? want : 152 * 32));
  void (*kern)(ReadParams);
  const bool bf = p.out_dtype == kBF16;
  if (p.cache_dtype == kBF16)
    kern = bf ? read_kernel<kBF16, kBF16> : read_kernel<kBF16, kF32>;
  else if (p.cache_dtype == kE4M3)
    kern = bf ? read_kernel<kE4M3, kBF16> : read_kernel<kE4M3, kF32>;
  else
    kern = bf ? read_kernel<kE2M1, kBF16> : read_kernel<kE2M1, kF32>;
  return launch_pdl(kern, grid, dim3(256), 0, stream, p);
}

cudaError_t launch_append(const AppendParams& p, cudaStream_t stream) {
  if (p.cache_dtype == kE2M1) {
    const int64_t want = (p.n_tokens * p.num_kv_heads * (p.head_dim / kE2M1Group) + 255) / 256;
    const dim3 grid(static_cast<unsigned>(want < 152 * 32 ? want : 152 * 32));
    return launch_pdl(p.src_dtype == kBF16 ? append_e2m1_kernel<kBF16> : append_e2m1_kernel<kF32>, grid, dim3(256), 0,
                      stream, p);
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
