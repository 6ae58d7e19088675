// chunk_window_tc.cu -- chunk attention on the tensor cores with a sliding window.
#include "chunk_tc_kernel.cuh"

namespace pda {

pda_status launch_chunk_window_tc(const ChunkParams& p, int D, pda_dtype kv_dtype, int dev,
                                  int sms, bool capped, void* workspace, cudaStream_t stream) {
  return launch_tc<true>(p, D, kv_dtype, dev, sms, capped, workspace, stream);
}

}  // namespace pda
