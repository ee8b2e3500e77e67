// Block tables, slots and positions of a serving step, built on the GPU from the
// requests' lengths ([SC] "LLM inference: prefill, decode, KV cache",
// "PagedAttention & Memory Management (vLLM)": memory is taken on demand, a block
// at a time; [FN] "Paged KV-Cache with Radix Tree Prefix Cache": a table grows by
// taking a block from the free pool), with the free pool a stack in device memory.
//
// With have_b = ceil(past_b / bs), need_b = ceil((past_b + new_b) / bs) - have_b
// and their sums before request b, new block i of request b is entry
// count - 1 - (block_starts_b + i) of the stack, and token i of its new ones goes
// to position past_b + i.  Truncation puts blocks back the other way round, so
// that dropping what was just taken restores the stack.
//
// A plan kernel of one CTA sums the requests (a run of them per thread, one scan
// of the threads' sums) and decides whether the call goes through; a fill kernel
// gives every token its slot, or every freed block its place.  The fill finds a
// token's request in the sums that the plan wrote and needs nothing that a caller
// may have the plan overwrite in place: past_b = context_b - new_b, the old count
// = the new one + what was taken.  Up to kInline items the plan's own CTA fills
// (one launch).  Bound: latency, of a launch, the lengths, the scan, a free id or
// table entry, a store.  On the GPU 256 single tokens take 3.3 us, 120,570 tokens of
// 1024 requests 7.5 (two launches), 69,000 freed blocks 3.9; a call costs 6.5-10 us
// of the host's time, most of it for the seven outputs.

#include <algorithm>

#include "decode_common.cuh"

namespace pkv {
namespace {

constexpr int kPlanThreads = 1024, kFillThreads = 256;
constexpr int kInline = 2048;

struct Sums {
  int64_t a, b;
};

// Sums of the threads before this one, and of all of them.
__device__ __forceinline__ Sums block_scan(Sums v, Sums& total) {
  __shared__ Sums s_warp[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  Sums x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t a = __shfl_up_sync(kFull, x.a, d), b = __shfl_up_sync(kFull, x.b, d);
    if (lane >= d) {
      x.a += a;
      x.b += b;
    }
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  Sums before = {0, 0};
  total = {0, 0};
  for (int w = 0; w < warps; ++w) {
    if (w == warp) before = total;
    total.a += s_warp[w].a;
    total.b += s_warp[w].b;
  }
  return {before.a + x.a - v.a, before.b + x.b - v.b};
}

// Request of item t: largest b with starts[b] <= t, for a t below starts[batch];
// a whole warp, whose items lie between `first` and `last`.
__device__ __forceinline__ int request_of(const int32_t* starts, int batch, int first, int last, int t) {
  int lo = warp_search(batch, first, [&](int i) { return starts[i]; });
  int hi = lo + 1 + warp_search(batch - lo, last, [&](int i) { return starts[lo + i]; });  // starts[hi] > last
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// ------------------------------------------------------------ more tokens

// Tokens `from`, `from + step`, ... of the step; `from` is the same in no two
// threads, and a warp's are consecutive.
__device__ __forceinline__ void fill_tokens(const ExtendParams& p, int64_t from, int64_t step) {
  const int lane = threadIdx.x & 31, shift = p.block_size == 16 ? 4 : 5, mask = p.block_size - 1;
  const int total = p.q_starts[p.batch];
  const int count = *p.free_count_out + p.block_starts[p.batch];  // before the call
  for (int64_t t = from; t - lane < p.max_tokens; t += step) {
    int64_t slot = -1, pos = -1;
    if (t - lane < total) {  // the warp has tokens
      const int first = static_cast<int>(t - lane), last = min(first + 31, total - 1);
      const int b = request_of(p.q_starts, p.batch, first, last, min(static_cast<int>(t), last));
      if (t < total) {
        const int start = p.q_starts[b], past = p.context_lens[b] - (p.q_starts[b + 1] - start);
        const int at = past + static_cast<int>(t) - start;
        const int blk = at >> shift, have = (past >> shift) + ((past & mask) != 0);
        int32_t* entry = p.block_tables + static_cast<int64_t>(b) * p.max_blocks + blk;
        int id = blk >= have ? p.free_blocks[count - 1 - (p.block_starts[b] + blk - have)] : *entry;
        const bool ok = id >= 0 && id < p.num_blocks;
        if (!ok) {
          record_error(p.err, kDevErrBlockId);
          id = -1;
        }
        if (blk >= have && (at & mask) == 0) *entry = id;
        pos = at;
        slot = ok ? (static_cast<int64_t>(id) << shift) + (at & mask) : -1;
      }
    }
    if (t < p.max_tokens) {
      p.slots[t] = slot;
      p.positions[t] = pos;
    }
  }
}

__global__ void __launch_bounds__(kPlanThreads) extend_plan_kernel(const ExtendParams p, int inline_fill) {
  wait_prior_grid();
  allow_next_grid();
  const int shift = p.block_size == 16 ? 4 : 5, mask = p.block_size - 1;
  const int64_t cap = static_cast<int64_t>(p.max_blocks) << shift;
  const int each = (p.batch + blockDim.x - 1) / blockDim.x;
  const int b0 = min(static_cast<int>(threadIdx.x) * each, p.batch), b1 = min(b0 + each, p.batch);
  // tokens and blocks that request b gets; one that cannot have its tokens gets none
  auto wants = [&](int b, bool note, int& past) {
    past = p.past_lens[b];
    const int n = p.new_lens[b];
    if (past < 0 || n < 0 || static_cast<int64_t>(past) + n > cap) {
      if (note) record_error(p.err, kDevErrContextLen);
      return Sums{0, 0};
    }
    const int64_t end = static_cast<int64_t>(past) + n;
    return Sums{n, ((end + mask) >> shift) - ((static_cast<int64_t>(past) + mask) >> shift)};
  };
  Sums mine = {0, 0}, total;
  int past;
  for (int b = b0; b < b1; ++b) {
    const Sums w = wants(b, true, past);
    mine.a += w.a;
    mine.b += w.b;
  }
  const int count = *p.free_count;
  Sums at = block_scan(mine, total);
  const bool good = count >= 0 && count <= p.free_capacity;
  const bool goes = good && total.b <= count && total.a <= p.max_tokens;
  if (threadIdx.x == 0 && !good) record_error(p.err, kDevErrBlockId);
  if (threadIdx.x == 0 && total.a > p.max_tokens) record_error(p.err, kDevErrContextLen);
  // (what was read of a request is written only by the thread that read it; the
  // count was read by all before the scan's barrier)
  for (int b = b0; b < b1; ++b) {
    Sums w = wants(b, false, past);
    if (!goes) w = at = {0, 0};
    p.q_starts[b] = static_cast<int32_t>(at.a);
    p.block_starts[b] = static_cast<int32_t>(at.b);
    p.context_lens[b] = past + static_cast<int32_t>(w.a);
    at.a += w.a;
    at.b += w.b;
  }
  if (threadIdx.x == 0) {
    p.q_starts[p.batch] = goes ? static_cast<int32_t>(total.a) : 0;
    p.block_starts[p.batch] = goes ? static_cast<int32_t>(total.b) : 0;
    *p.free_count_out = goes ? count - static_cast<int32_t>(total.b) : count;
    const int64_t lack = good ? total.b - count : total.b;
    // a step that did not go through has a value other than 0, whatever it failed for
    *p.lacking = lack > 0 ? static_cast<int32_t>(min(lack, static_cast<int64_t>(0x7FFFFFFF))) : (goes ? 0 : -1);
  }
  if (inline_fill != 0) {
    __syncthreads();  // the sums are written
    fill_tokens(p, threadIdx.x, blockDim.x);
  }
}

__global__ void __launch_bounds__(kFillThreads) extend_fill_kernel(const ExtendParams p) {
  wait_prior_grid();
  allow_next_grid();
  fill_tokens(p, static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x,
              static_cast<int64_t>(gridDim.x) * blockDim.x);
}

// ------------------------------------------------------------ fewer tokens

__device__ __forceinline__ void fill_freed(const TruncateParams& p, int64_t from, int64_t step) {
  const int lane = threadIdx.x & 31, shift = p.block_size == 16 ? 4 : 5, mask = p.block_size - 1;
  const int total = p.block_starts[p.batch];
  const int count = *p.free_count_out - total;  // before the call
  for (int64_t t = from; t - lane < total; t += step) {
    const int first = static_cast<int>(t - lane), last = min(first + 31, total - 1);
    const int b = request_of(p.block_starts, p.batch, first, last, min(static_cast<int>(t), last));
    if (t < total) {
      const int keep = p.keep_lens[b];
      const int blk = (keep >> shift) + ((keep & mask) != 0) + static_cast<int>(t) - p.block_starts[b];
      int id = p.block_tables[static_cast<int64_t>(b) * p.max_blocks + blk];
      if (id < 0 || id >= p.num_blocks) {
        record_error(p.err, kDevErrBlockId);
        id = -1;
      }
      p.free_blocks[count + (total - 1 - static_cast<int>(t))] = id;
    }
  }
}

__global__ void __launch_bounds__(kPlanThreads) truncate_plan_kernel(const TruncateParams p, int inline_fill) {
  wait_prior_grid();
  allow_next_grid();
  const int shift = p.block_size == 16 ? 4 : 5, mask = p.block_size - 1;
  const int64_t cap = static_cast<int64_t>(p.max_blocks) << shift;
  const int each = (p.batch + blockDim.x - 1) / blockDim.x;
  const int b0 = min(static_cast<int>(threadIdx.x) * each, p.batch), b1 = min(b0 + each, p.batch);
  auto gives = [&](int b, bool note) -> int64_t {
    const int64_t ctx = p.context_lens[b], keep = p.keep_lens[b];
    if (keep < 0 || keep > ctx || ctx > cap) {
      if (note) record_error(p.err, kDevErrContextLen);
      return 0;
    }
    return ((ctx + mask) >> shift) - ((keep + mask) >> shift);
  };
  Sums mine = {0, 0}, total;
  for (int b = b0; b < b1; ++b) mine.a += gives(b, true);
  const int count = *p.free_count;
  Sums at = block_scan(mine, total);
  const bool goes = count >= 0 && total.a <= static_cast<int64_t>(p.free_capacity) - count;
  if (threadIdx.x == 0 && !goes) record_error(p.err, kDevErrBlockId);
  for (int b = b0; b < b1; ++b) {
    p.block_starts[b] = goes ? static_cast<int32_t>(at.a) : 0;
    at.a += gives(b, false);
  }
  if (threadIdx.x == 0) {
    p.block_starts[p.batch] = goes ? static_cast<int32_t>(total.a) : 0;
    *p.free_count_out = goes ? count + static_cast<int32_t>(total.a) : count;
  }
  if (inline_fill != 0) {
    __syncthreads();
    fill_freed(p, threadIdx.x, blockDim.x);
  }
}

__global__ void __launch_bounds__(kFillThreads) truncate_fill_kernel(const TruncateParams p) {
  wait_prior_grid();
  allow_next_grid();
  fill_freed(p, static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x,
             static_cast<int64_t>(gridDim.x) * blockDim.x);
}

dim3 plan_threads(int batch, int64_t items) {
  const int64_t want = std::max<int64_t>(batch, std::min<int64_t>(items, kInline));
  return dim3(static_cast<unsigned>(want >= kPlanThreads ? kPlanThreads : (want + 31) / 32 * 32 + (want == 0 ? 32 : 0)));
}

dim3 fill_grid(int64_t items) {
  const int64_t want = (items + kFillThreads - 1) / kFillThreads;
  return dim3(static_cast<unsigned>(want < 152 * 8 ? want : 152 * 8));
}

}  // namespace

cudaError_t launch_extend(const ExtendParams& p, cudaStream_t stream) {
  const bool here = p.max_tokens <= kInline;
  cudaError_t e = launch_pdl(extend_plan_kernel, dim3(1), plan_threads(p.batch, here ? p.max_tokens : 0), 0, stream, p,
                             here ? 1 : 0);
  if (e == cudaSuccess && !here)
    e = launch_pdl(extend_fill_kernel, fill_grid(p.max_tokens), dim3(kFillThreads), 0, stream, p);
  return e;
}

cudaError_t launch_truncate(const TruncateParams& p, cudaStream_t stream) {
  const int64_t most = std::min<int64_t>(static_cast<int64_t>(p.batch) * p.max_blocks, p.free_capacity);
  const bool here = most <= kInline;
  cudaError_t e = launch_pdl(truncate_plan_kernel, dim3(1), plan_threads(p.batch, here ? most : 0), 0, stream, p,
                             here ? 1 : 0);
  if (e == cudaSuccess && !here)
    e = launch_pdl(truncate_fill_kernel, fill_grid(most), dim3(kFillThreads), 0, stream, p);
  return e;
}

}  // namespace pkv
