// la_chunk_bwd_f32.cu -- the backward walks with inputs as three bf16 planes: fp32, and
// bf16 with phi = elu + 1 where an fp32 output is wanted.
#include "la_chunk_bwd.cuh"

namespace la {

cudaError_t launch_chunk_bwd_f32(const ChunkBwd &p, int seqs, bool wide, bool bf16,
                                 cudaStream_t stream) {
  if (bf16)
    return wide ? run_chunk_bwd<BwdConfig<__nv_bfloat16, 128, 32, 3, 3>>(p, seqs, stream)
                : run_chunk_bwd<BwdConfig<__nv_bfloat16, 64, 32, 3, 3>>(p, seqs, stream);
  return wide ? run_chunk_bwd<BwdConfig<float, 128, 32, 3, 3>>(p, seqs, stream)
              : run_chunk_bwd<BwdConfig<float, 64, 32, 3, 3>>(p, seqs, stream);
}

}  // namespace la
