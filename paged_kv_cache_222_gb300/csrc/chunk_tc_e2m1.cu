// The tcgen05 kernel of chunk_tc.cuh for E2M1 caches, compiled beside the
// others.

#include "chunk_tc.cuh"

namespace pkv {

cudaError_t launch_chunk_tc_e2m1(const ChunkParams& p, const ChunkMaps& m, cudaStream_t stream) {
  return launch_tc<kE2M1>(p, m, stream);
}

}  // namespace pkv
