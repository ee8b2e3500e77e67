// The tcgen05 kernel of chunk_tc.cuh for bf16 and E4M3 caches.

#include "chunk_tc.cuh"

namespace pkv {

cudaError_t launch_chunk_tc(const ChunkParams& p, const ChunkMaps& m, cudaStream_t stream) {
  if (p.cache_dtype == kE2M1) return launch_chunk_tc_e2m1(p, m, stream);
  return p.cache_dtype == kE4M3 ? launch_tc<kE4M3>(p, m, stream) : launch_tc<kBF16KV>(p, m, stream);
}

}  // namespace pkv
