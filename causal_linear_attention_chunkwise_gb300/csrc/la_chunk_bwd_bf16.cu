// la_chunk_bwd_bf16.cu -- the backward walks for short bf16 sequences, of one chunk.
#include "la_chunk_bwd.cuh"

namespace la {

cudaError_t launch_chunk_bwd_bf16(const ChunkBwd &p, int seqs, bool planes, cudaStream_t stream) {
  using T = __nv_bfloat16;
  if (planes) return run_chunk_bwd<BwdConfig<T, 64, 64, 1, 3>>(p, seqs, stream);
  return p.phi == LA_PHI_ELU1 ? run_chunk_bwd<BwdConfig<T, 64, 64, 2, 1>>(p, seqs, stream)
                              : run_chunk_bwd<BwdConfig<T, 64, 64, 1, 1>>(p, seqs, stream);
}

}  // namespace la
