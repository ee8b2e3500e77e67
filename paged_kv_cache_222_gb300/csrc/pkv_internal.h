// Internal interface between the C ABI (api.cu) and the kernel translation
// units (append.cu, decode.cu).  Not installed; no stability promise.
#pragma once

#include <cmath>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace pkv {

// Mirrors PKV_DEVERR_* of pkv.h (kept separate so device code needs no C ABI).
constexpr int kDevErrWaitTimeout = 1;
constexpr int kDevErrBlockId = 2;
constexpr int kDevErrContextLen = 3;
constexpr int kDevErrSlot = 4;
constexpr int kDevErrAxis = 5;

// Tokens per pipeline tile: one mma M dimension of keys.
constexpr int kTileTokens = 16;
// Consumer warps per decode CTA.
constexpr int kDecodeWarps = 4;

enum KernelKind {
  kKindAppend = 0,
  kKindDecodeSplit = 1,
  kKindCombine = 2,
  kKindCascadePrefix = 3,
  kKindBlockCopy = 4,
  kKindMultiQuery = 5,
  kKindSlotMapping = 6,
  kKindChunk = 7,
  kKindRotary = 8,
  kKindCompact = 9,
  kKindRead = 10,
  kKindTables = 11,
  kNumKernelKinds = 12  // the trace aggregates by kind
};

// Decode work split: balanced stream-K ranges over the flattened
// (sequence, head, tile) space, or fixed `split_tokens` chunks per sequence.
constexpr int kModeStreamK = 0;
constexpr int kModeFixedSplit = 1;
// Largest batch the stream-K kernel takes (its tile prefix lives in shared
// memory); larger batches use fixed splits.
constexpr int kMaxStreamKBatch = 2048;

struct AppendParams {
  const void* k_new;
  const void* v_new;
  const int64_t* slots;
  void* k_cache;
  void* v_cache;
  const float* k_scale;
  const float* v_scale;
  int64_t scale_stride;
  int64_t n_tokens;
  int64_t num_slots;  // num_blocks * block_size
  int32_t block_size;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t src_dtype;    // PKV_BF16 / PKV_F32
  int32_t cache_dtype;  // PKV_BF16 / PKV_E4M3 / PKV_E2M1
  int* err;
};

// Token rows read back from the cache (append.cu).
struct ReadParams {
  const int64_t* slots;
  const void* k_cache;
  const void* v_cache;
  const float* k_scale;
  const float* v_scale;
  int64_t scale_stride;
  void* k_out;
  void* v_out;
  int64_t n_tokens;
  int64_t num_slots;  // num_blocks * block_size
  int32_t block_size;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t out_dtype;    // PKV_BF16 / PKV_F32
  int32_t cache_dtype;  // PKV_BF16 / PKV_E4M3 / PKV_E2M1
  int* err;
};

// Flat cache slots of new tokens from the block tables.
struct SlotParams {
  const int32_t* block_tables;  // [num_seqs, max_blocks]
  const int64_t* seq_index;     // [n] sequence of token i, or NULL: token i is sequence i
  const int64_t* positions;     // [n] logical position of token i (< 0: padding)
  int64_t* slots;               // [n] out: block * block_size + offset, -1 for padding
  int64_t n;
  int64_t num_blocks;
  int32_t num_seqs;
  int32_t max_blocks;
  int32_t block_size;
  int* err;
};

// Element types of K / V rows being encoded into the cache: the sources of
// an append (bf16, f32) and the cache's own (bf16, E4M3, E2M1).
constexpr int kEncBF16 = 0, kEncF32 = 1, kEncE4M3 = 2, kEncE2M1 = 3;

// E2M1 caches: the bytes of one (block, head) are block_size rows of D / 2 code
// bytes, then block_size rows of D / 16 scale bytes.  Codes and scales apart keep
// both of them in 16-byte pieces that the TMA unit moves.
constexpr int kE2M1Group = 16;  // elements that share a scale
constexpr int e2m1_code_row(int head_dim) { return head_dim / 2; }
constexpr int e2m1_scale_row(int head_dim) { return head_dim / kE2M1Group; }
constexpr int e2m1_tile_bytes(int head_dim, int block_size) {
  return block_size * (e2m1_code_row(head_dim) + e2m1_scale_row(head_dim));
}

struct DecodeParams {
  const void* q;              // bf16 [B, H_q, D]
  const int32_t* block_tables;  // [B, MB]
  const int32_t* context_lens;  // [B]
  float* out;                 // [B, H_q, D]
  float* ws_o;                // fixed split: [B, H_q, S, D]; stream-K: [2W, GP, D]
  float* ws_ml;               // fixed split: [B, H_q, S, 2]; stream-K: [2W, GP, 2]
  int* ws_q;                  // stream-K: tile prefix over sequences [B + 1];
                              // tcgen05 multi-token: the work-unit counter
  const float* k_scale;
  const float* v_scale;
  int64_t scale_stride;
  int64_t num_blocks;
  int32_t batch;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t group;              // G = H_q / H_kv
  int32_t head_dim;
  int32_t block_size;
  int32_t max_blocks;         // MB
  int32_t max_ctx;
  int32_t split_tokens;
  int32_t max_splits;
  float qk_log2_scale;        // softmax scale * log2(e)
  int32_t cache_dtype;
  int32_t mode;               // kModeStreamK / kModeFixedSplit
  int32_t workers;            // stream-K: warps of the persistent grid (W);
                              // tcgen05 multi-token: CTAs of the persistent grid
  // cascade (shared-prefix) decode; zero / -1 / NULL otherwise
  int32_t token_offset;       // fixed split: attend tokens [token_offset, ctx)
  int32_t force_partial;      // fixed split: always write partials, never `out`
  int32_t extra_slot;         // combine: first workspace slot of the prefix pieces (-1: none)
  int32_t extra_count;        // combine: number of prefix pieces per row
  int32_t slots_per_row;      // fixed split / cascade: workspace slots per (b, hq) row
  const int32_t* prefix_blocks;  // [prefix_len / block_size] physical blocks
  int32_t prefix_len;
  int32_t prefix_split_tokens;   // prefix tokens per prefix CTA (multiple of 64)
  // multi-token queries: q_len new tokens per sequence (1 for decode)
  int32_t q_len;
  // fixed split, fused append: each sequence's newest token (position
  // context_lens[b] - 1) is written from k_new / v_new [B, H_kv, D] into its
  // slot by the CTA that attends it, before that CTA's first load
  int32_t new_src;            // 0: no append; else kEncBF16 + 1 or kEncF32 + 1
  const void* k_new;
  const void* v_new;
  void* k_cache;
  void* v_cache;
  int* err;
};

// Whole-block copies between (or within) block pools: pair i copies block
// src[i] of the K and V caches to block dst[i].
struct CopyParams {
  const void* k_src;      // K cache the sources live in
  const void* v_src;
  void* k_dst;            // K cache the destinations live in
  void* v_dst;
  const int32_t* src;     // [n_pairs] source block ids
  const int32_t* dst;     // [n_pairs] destination block ids
  int64_t n_pairs;
  int64_t block_vec;      // 16-byte words per block of one cache
  int64_t src_blocks;     // valid source ids: [0, src_blocks)
  int64_t dst_blocks;     // valid destination ids: [0, dst_blocks)
  int32_t max_ctas;       // grid bound (0: as many as the copy can use)
  int* err;
};

// Attention of ragged chunks of new tokens over the paged cache (chunk.cu,
// chunk_e2m1.cu, chunk_tc.cuh).  Sequence b owns query rows [q_starts[b], q_starts[b + 1]);
// query i of its n sits at position context_lens[b] - n + i.
struct ChunkParams {
  const void* q;                 // bf16 [T, H_q, D]
  const void* k_cache;
  const void* v_cache;
  void* out;                     // bf16 [T, H_q, D]
  const int32_t* q_starts;       // [B + 1]
  const int32_t* block_tables;   // [B, MB]
  const int32_t* context_lens;   // [B]
  const float* slopes;           // [H_q] or NULL: score bias per token of distance
  const int32_t* prefix_lens;    // [B] or NULL: tokens every query of the sequence sees
  const float* k_scale;
  const float* v_scale;
  int64_t scale_stride;
  int64_t num_blocks;
  float* ws_o;                   // [T, H_q, S, D] partial rows (S > 1)
  float* ws_ml;                  // [T, H_q, S, 2]
  int32_t n_tokens;              // T
  int32_t batch;
  int32_t max_q_len;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t group;
  int32_t head_dim;
  int32_t block_size;
  int32_t max_blocks;
  int32_t max_ctx;
  int32_t window;                // tokens a query sees back, itself included (0: all)
  int32_t split_tokens;          // visible tokens per split (a multiple of 128)
  int32_t max_splits;
  int32_t tile_q;                // query tokens of one row tile
  float qk_log2;                 // scale * log2(e); with a cap: 2 * scale * log2(e) / cap
  float cap_log2;                // cap * log2(e), 0 without a cap
  float cap_c[3];                // small scores' tanh(y) / y: coefficients of 1, y^2, y^4 ...
  float cap_y_max;               // ... and the |y| = score / cap up to which they hold
  bool cap_far;                  // caps above kCapNear
  int32_t cache_dtype;
  int* err;
};

// Tensor maps of a chunk attention call: the queries (tcgen05 kernel), the
// caches' rows (E2M1: of codes) and an E2M1 cache's rows of scales.
struct ChunkMaps {
  CUtensorMap q, k, v, k_scales, v_scales;
};

// Rotary positions and append of new tokens (rotary.cu).
struct RotaryParams {
  const void* q;
  const void* k;
  const void* v;
  void* q_out;                   // bf16
  int64_t q_stride, k_stride, v_stride, out_stride;  // elements between tokens
  const int64_t* positions;      // [num_axes] rows of one per token, position_stride apart
  int64_t position_stride;
  const int32_t* axes;           // [rotary_dim / 2]: the axis of each pair, or NULL: axis 0
  int32_t num_axes;
  const double* inv_freq;        // [rotary_dim / 2], radians per position
  float magnitude;
  const int64_t* slots;
  void* k_cache;
  void* v_cache;
  const float* k_scale;
  const float* v_scale;
  int64_t scale_stride;
  int64_t n_tokens;
  int64_t num_slots;
  int32_t block_size;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t rotary_dim;
  int32_t interleaved;
  int32_t src_dtype;             // PKV_BF16 / PKV_F32
  int32_t cache_dtype;           // PKV_BF16 / PKV_E4M3 / PKV_E2M1
  int* err;
};

// In-place compaction of sequences' token rows (compact.cu).
struct CompactParams {
  void* k_cache;
  void* v_cache;
  const int32_t* block_tables;
  const int32_t* keep;           // [N] logical positions to keep
  const int32_t* keep_starts;    // [B + 1]
  const int32_t* dst_start;      // [B] or NULL: first destination (0)
  int64_t num_blocks;
  int32_t n_keep;                // N
  int32_t batch;
  int32_t max_keep;
  int32_t max_blocks;
  int32_t block_size;
  int32_t num_kv_heads;
  int32_t row_bytes;             // bytes of one token row of one head
  int32_t tile_bytes;            // from one (block, head) to the next
  int32_t tile_offset;           // of a (block, head)'s first row
  int* err;
};

// Tables, slots and positions of requests' new tokens (tables.cu).
struct ExtendParams {
  int32_t* block_tables;         // [B, MB]
  const int32_t* past_lens;      // [B]
  const int32_t* new_lens;       // [B]
  const int32_t* free_blocks;    // stack
  const int32_t* free_count;
  int32_t* context_lens;         // [B], may be past_lens
  int32_t* q_starts;             // [B + 1]
  int32_t* block_starts;         // [B + 1]
  int64_t* slots;                // [max_tokens]
  int64_t* positions;            // [max_tokens]
  int32_t* free_count_out;       // may be free_count
  int32_t* lacking;
  int64_t num_blocks;
  int64_t max_tokens;
  int32_t free_capacity;
  int32_t batch;
  int32_t max_blocks;
  int32_t block_size;
  int* err;
};

// Blocks that requests give back (tables.cu).
struct TruncateParams {
  const int32_t* block_tables;   // [B, MB]
  const int32_t* context_lens;   // [B]
  const int32_t* keep_lens;      // [B]
  int32_t* free_blocks;          // stack
  const int32_t* free_count;
  int32_t* block_starts;         // [B + 1]
  int32_t* free_count_out;       // may be free_count
  int64_t num_blocks;
  int32_t free_capacity;
  int32_t batch;
  int32_t max_blocks;
  int32_t block_size;
  int* err;
};

// Message returned by pkv_last_error() on this host thread.
void set_last_error(const char* msg);

// Configuration epoch (>= 1): pkv_shutdown starts a new one, after which every
// per-device set-up the launchers cached (shared-memory limits) is made again.
int config_epoch();

// Launchers (return the launch's cudaError_t; nothing is synchronised).
cudaError_t launch_copy_blocks(const CopyParams& p, cudaStream_t stream);
cudaError_t launch_append(const AppendParams& p, cudaStream_t stream);
cudaError_t launch_read(const ReadParams& p, cudaStream_t stream);
cudaError_t launch_extend(const ExtendParams& p, cudaStream_t stream);
cudaError_t launch_truncate(const TruncateParams& p, cudaStream_t stream);
cudaError_t launch_slot_mapping(const SlotParams& p, cudaStream_t stream);
cudaError_t launch_decode_split(const DecodeParams& p, const CUtensorMap& tmap_k,
                                const CUtensorMap& tmap_v, cudaStream_t stream);
cudaError_t launch_decode_combine(const DecodeParams& p, cudaStream_t stream);
cudaError_t launch_cascade_prefix(const DecodeParams& p, const CUtensorMap& tmap_k,
                                  const CUtensorMap& tmap_v, cudaStream_t stream);
cudaError_t launch_multi_query(const DecodeParams& p, const CUtensorMap& tmap_k,
                               const CUtensorMap& tmap_v, cudaStream_t stream);
// Multi-token queries of 64 or more rows per (sequence, KV head) on tcgen05
// (the cascade kernel's pipeline, one 128-row group per CTA).
cudaError_t launch_multi_query_tc(const DecodeParams& p, const CUtensorMap& tmap_k,
                                  const CUtensorMap& tmap_v, cudaStream_t stream);
// Ragged chunks: the mma.sync kernel (row tiles of up to 16 rows), the tcgen05
// kernel (row tiles of up to 256 rows) and the merge of their split pieces.
cudaError_t launch_chunk_small(const ChunkParams& p, const CUtensorMap& tmap_k, const CUtensorMap& tmap_v,
                               cudaStream_t stream);
cudaError_t launch_chunk_e2m1(const ChunkParams& p, cudaStream_t stream);
cudaError_t launch_chunk_tc(const ChunkParams& p, const ChunkMaps& maps, cudaStream_t stream);
cudaError_t launch_chunk_tc_e2m1(const ChunkParams& p, const ChunkMaps& maps, cudaStream_t stream);
// `nk`: keys per tile of the kernel that wrote the pieces.
cudaError_t launch_chunk_combine(const ChunkParams& p, int nk, cudaStream_t stream);
cudaError_t launch_rotary(const RotaryParams& p, cudaStream_t stream);
cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream);
// Self-test of the bounded waits (0: mbarrier wait; 1: tensor-core CTA abort
// path); records PKV_DEVERR_WAIT_TIMEOUT after about limit_ns.
cudaError_t launch_wait_selftest(int which, uint64_t limit_ns, int* err, cudaStream_t stream);
// Rows (q_len * G) from which multi-token queries take the tcgen05 kernel.
// Its speed hardly depends on the rows (0.68-0.70 of HBM from 8 to 128 rows
// on the 70B-class GQA batch); the mma.sync kernel measured 0.82 at 16 rows,
// 0.65 at 24, 0.63 at 32 and 0.41 at 40.
constexpr int kMultiQueryTcRows = 17;

// Multi-token query kernel: 64-token tiles, rows of (query token, head) pairs
// in 16-row warp groups; the block ids of one split staged in shared memory.
constexpr int kMultiQueryTile = 64;
constexpr int kMultiQueryMaxSplitBlocks = 1024;
// Token lanes (warps sharing the same 16 rows) for R rows per (sequence, head).
inline int multi_query_lanes(int rows) { return rows <= 16 ? 4 : (rows <= 32 ? 2 : 1); }

// Ragged chunks: rows of one row tile of the mma.sync and of the tcgen05
// kernel, and blocks of one split of the mma.sync kernel (their ids are staged
// in shared memory).
constexpr int kChunkSmallRows = 16;
constexpr int kChunkTcRows = 256;
constexpr int kChunkMaxSplitBlocks = 1024;
// Longest context: the end of its last key tile, and of the tile after it, are
// still 32-bit numbers.
constexpr int kChunkMaxContext = 0x7FFFFF00;
// Keys per tile: of the mma.sync kernels; of the tcgen05 kernel at most, and by
// its variant (chunk_tc.cuh: whether S(k+1) is issued ahead of P(k)'s product).
constexpr int kChunkSmallTile = 64, kChunkE2M1Tile = 128, kChunkTcTile = 128;
// CTAs per SM of the mma.sync kernels: over E2M1 caches (chunk_e2m1.cu), and by
// the bytes of a 64-key step over others (chunk.cu).
constexpr int chunk_e2m1_ctas(bool eight_rows) { return eight_rows ? 4 : 3; }
constexpr int chunk_small_ctas(int head_dim, bool fp8, bool eight_rows) {
  const int stage = 2 * kChunkSmallTile * head_dim * (fp8 ? 1 : 2);
  return !eight_rows || stage >= 32768 ? 3 : (stage == 16384 ? 4 : 5);
}
constexpr bool chunk_tc_early(bool fp8, bool mods) { return !fp8 && mods; }
constexpr int chunk_tc_tile(int head_dim, bool fp8, bool mods) {
  return head_dim == 128 && chunk_tc_early(fp8, mods) ? 64 : kChunkTcTile;
}

// Of a ring whose item i goes to slot i % slots, even items (K) issued by one
// loader up to next_k - 2 and odd ones (V) by another up to next_v - 2: the last
// item issued into `slot`, -1 if there was none.
constexpr int ring_last_item(int slot, int slots, int next_k, int next_v) {
  const int k = next_k - 2, v = next_v - 2;
  for (int i = k > v ? k : v; i >= 0; --i)
    if (i % slots == slot && i <= (i % 2 ? v : k)) return i;
  return -1;
}

// tanh(y) = y (c[0] + c[1] y^2 + c[2] y^4) for |y| <= y_max with cap times the
// error below 2^-13.  Caps up to 100: the coefficients of the least largest
// relative error on |y| <= 0.35, 2.9e-6.  Above, 1 exactly, so that the error
// falls with the score, and the other two such that what is left of the next
// term of the series, -17/315 y^6, is y^2 times a polynomial in y^2 with its two
// zeros placed for the least largest value up to y_max (a Chebyshev polynomial
// moved until its first zero is at 0: the others at 0.4641 and 0.9282 of y_max^2):
// 2.1e-3 y_max^7 of the cap.
constexpr double kCapNear = 100.0;
constexpr float kCapLimit = 0.35f, kCapC[3] = {0.99999713f, -0.33290954f, 0.12395031f};
inline void cap_coefficients(double cap, float (&c)[3], float& y_max) {
  if (cap <= kCapNear) {
    for (int i = 0; i < 3; ++i) c[i] = kCapC[i];
    y_max = kCapLimit;
    return;
  }
  const double a = std::pow(0.045 / cap, 1.0 / 7.0), next = -17.0 / 315.0;
  c[0] = 1.f;
  c[1] = static_cast<float>(-1.0 / 3.0 - next * 0.4641 * 0.9282 * a * a * a * a);
  c[2] = static_cast<float>(2.0 / 15.0 + next * (0.4641 + 0.9282) * a * a);
  y_max = static_cast<float>(a);
}

// tanh(y) = y (1 + kCapC1 y^2 + kCapC2 y^4 + kCapC3 y^6) for |y| <= kCapLimit, off
// by less than 4.1e-8 of itself: the least largest relative error with 1 exactly.
constexpr float kCapC1 = -0.33332663f, kCapC2 = 0.13299825f, kCapC3 = -0.0491485f;

// tanh(y) = y (kMidC0 + kMidC1 y^2 + ... + kMidC6 y^12) for |y| <= kMidLimit, off by less
// than 4.4e-7 with binary32's own rounding: 100 times that (kCapNear) is below
// 2^-13 of a weight.  The coefficients of the least largest error, the last one
// positive so that -inf, a hidden score, stays that.
constexpr float kMidLimit = 1.25f;
constexpr float kMidC0 = 0.999996483f, kMidC1 = -0.333242148f, kMidC2 = 0.132648036f, kMidC3 = -0.0516446903f,
                kMidC4 = 0.0176362358f, kMidC5 = -0.00432548998f, kMidC6 = 0.000525482697f;

// Rows of query heads one cascade prefix CTA covers: two groups of 128 TMEM
// lanes.
constexpr int kCascadeRowsTc = 256;
// Keys per cascade prefix tile (4 sub-tiles of kTileTokens).
constexpr int kCascadeTile = 64;
// Blocks of one cascade prefix range (their ids are staged in shared memory):
// a range holds at most this many times the block size of tokens.
constexpr int kCascadeMaxRangeBlocks = 256;

// Dynamic shared memory the split kernel needs for (head_dim, dtype, groups).
int decode_smem_bytes(int head_dim, int cache_dtype, int n_tiles8);

// Warps in the stream-K kernel's persistent grid on a GPU with `sms` SMs.
int streamk_grid_workers(int head_dim, int cache_dtype, int sms);

}  // namespace pkv
