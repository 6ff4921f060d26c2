// la_chunk_bwd_bf16.cu -- the backward walks for bf16 inputs as they are.
#include "la_chunk_bwd.cuh"

namespace la {

cudaError_t launch_chunk_bwd_bf16(const ChunkBwd &p, int seqs, bool wide, bool planes,
                                  cudaStream_t stream) {
  using T = __nv_bfloat16;
  if (wide)
    return planes ? run_chunk_bwd<BwdConfig<T, 128, 64, 1, 3>>(p, seqs, stream)
                  : run_chunk_bwd<BwdConfig<T, 128, 64, 1, 1>>(p, seqs, stream);
  return planes ? run_chunk_bwd<BwdConfig<T, 64, 64, 1, 3>>(p, seqs, stream)
                : run_chunk_bwd<BwdConfig<T, 64, 64, 1, 1>>(p, seqs, stream);
}

}  // namespace la
