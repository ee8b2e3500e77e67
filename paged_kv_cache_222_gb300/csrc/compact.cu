// In-place compaction of a paged cache: token rows that a sequence keeps move
// towards its front ([UI] "Architecting Multi-Tier Disaggregated KV-Cache
// Hierarchies...", "Predictive Prefetching and Attention-Salience Eviction
// Policy": tokens of low salience leave the cache; [SC] "LLM inference:
// prefill, decode, KV cache", "7. Practical applications", item 3: the
// accepted tokens of a verified draft stay).
//
//   row (dst_start + j) := row keep[j],   keep[j] >= dst_start + j
//
// for K and V of every head.  Because no source lies before its destination,
// rows read in order of j are never overwritten before they are read: a
// destination d written for entry j is the source of an entry j' > j only if
// keep[j'] = d < dst_start + j', which is refused.  Within a step of rows all
// reads come before a barrier and all writes after it, and the next step's
// rows are read before this step's are written.
//
// A CTA takes one (sequence, head, K or V, column band) and walks its rows in
// order; columns are independent, so few sequences are cut into bands of at
// least 64 bytes.  The rows' addresses (keep list, then block table) are
// looked up 256 at a time, a batch ahead.  Bound: the moved bytes, each read
// and written once: half of 32 x 4096 tokens of 8 heads of 128 (536 MB) takes
// 86.5 us, 6.2 TB/s, 93 % of the measured copy (without the next step's loads
// ahead 90 us; twice the rows per step 100, half of them 104; 128-byte bands
// for twice the CTAs 98: each then reads half a row's line).

#include "decode_common.cuh"

namespace pkv {
namespace {

constexpr int kCompactThreads = 256;
constexpr int kCompactUnroll = 4;

__device__ __forceinline__ int64_t compact_row(const CompactParams& p, const int32_t* tbl, int pos, int h, int& bad) {
  const int blk = tbl[pos / p.block_size];
  if (blk < 0 || blk >= p.num_blocks) {
    bad = kDevErrBlockId;
    return -1;
  }
  return (static_cast<int64_t>(blk) * p.num_kv_heads + h) * p.block_size + pos % p.block_size;
}

__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const CompactParams p, int band_bytes) {
  __shared__ int64_t s_src[2][kCompactThreads], s_dst[2][kCompactThreads];
  wait_prior_grid();
  allow_next_grid();
  const int bands = p.row_bytes / band_bytes;
  const int b = blockIdx.x;
  const int band = blockIdx.y % bands, hv = blockIdx.y / bands;
  const int h = hv >> 1;
  char* cache = static_cast<char*>((hv & 1) ? p.v_cache : p.k_cache) + band * band_bytes;
  const bool note = blockIdx.y == 0;  // one CTA of the sequence records what it refuses
  const int k0 = p.keep_starts[b], k1 = p.keep_starts[b + 1];
  const int first = p.dst_start != nullptr ? p.dst_start[b] : 0;
  if (k0 < 0 || k1 < k0 || k1 > p.n_keep || k1 - k0 > p.max_keep || first < 0) {
    if (note && threadIdx.x == 0) record_error(p.err, kDevErrContextLen);
    return;
  }
  const int n = k1 - k0;
  const int64_t cap = static_cast<int64_t>(p.max_blocks) * p.block_size;
  const int32_t* tbl = p.block_tables + static_cast<int64_t>(b) * p.max_blocks;

  // byte offsets of entry j's rows (-1: stays where it is, or refused)
  auto lookup = [&](int j, int64_t& src, int64_t& dst) {
    src = dst = -1;
    if (j >= n) return;
    const int64_t s = p.keep[k0 + j], d = static_cast<int64_t>(first) + j;
    if (s == d && s < cap) return;
    if (s < d || s >= cap) {
      if (note) record_error(p.err, kDevErrContextLen);
      return;
    }
    int bad = 0;
    src = compact_row(p, tbl, static_cast<int>(s), h, bad);
    dst = compact_row(p, tbl, static_cast<int>(d), h, bad);
    if (bad != 0) {
      if (note) record_error(p.err, bad);
      src = dst = -1;
      return;
    }
    src *= p.row_bytes;
    dst *= p.row_bytes;
  };

  // a step: 256 threads x 4 x 16 bytes; per_pass rows per 256 threads
  const int words = band_bytes / 16;
  const int per_pass = kCompactThreads / words;
  const int per_step = per_pass * kCompactUnroll;
  const int my_row = threadIdx.x / words, my_off = (threadIdx.x % words) * 16;
  int64_t ns, nd;
  lookup(threadIdx.x, ns, nd);
  for (int base = 0, buf = 0; base < n; base += kCompactThreads, buf ^= 1) {
    // buffer `buf` was last read two batches ago, before the barrier of the last one
    s_src[buf][threadIdx.x] = ns;
    s_dst[buf][threadIdx.x] = nd;
    __syncthreads();
    lookup(base + kCompactThreads + threadIdx.x, ns, nd);  // the next batch, in flight while this one moves
    const int here = min(n - base, kCompactThreads);
    uint4 v[kCompactUnroll], w[kCompactUnroll];
    auto load = [&](int r0, uint4 (&to)[kCompactUnroll]) {
#pragma unroll
      for (int u = 0; u < kCompactUnroll; ++u) {
        const int row = r0 + u * per_pass + my_row;
        const int64_t src = row < here ? s_src[buf][row] : -1;
        if (src >= 0) to[u] = __ldcg(reinterpret_cast<const uint4*>(cache + src + my_off));
      }
    };
    load(0, v);
    for (int r0 = 0; r0 < here; r0 += per_step) {
      __syncthreads();  // every row of the step has been read
      if (r0 + per_step < here) load(r0 + per_step, w);  // the next step's, in flight while this one's are written
#pragma unroll
      for (int u = 0; u < kCompactUnroll; ++u) {
        const int row = r0 + u * per_pass + my_row;
        const int64_t dst = row < here ? s_dst[buf][row] : -1;
        if (dst >= 0) *reinterpret_cast<uint4*>(cache + dst + my_off) = v[u];
      }
#pragma unroll
      for (int u = 0; u < kCompactUnroll; ++u) v[u] = w[u];
    }
  }
}

}  // namespace

cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream) {
  // column bands of at least 64 bytes while the CTAs are fewer than two per SM
  int band = p.row_bytes;
  while (band > 64 && static_cast<int64_t>(p.batch) * p.num_kv_heads * 2 * (p.row_bytes / band) < 2 * 152) band /= 2;
  const dim3 grid(p.batch, p.num_kv_heads * 2 * (p.row_bytes / band));
  return launch_pdl(compact_kernel, grid, dim3(kCompactThreads), 0, stream, p, band);
}

}  // namespace pkv
