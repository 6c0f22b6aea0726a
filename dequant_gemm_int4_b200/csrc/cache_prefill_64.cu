// The tcgen05 attention kernels for heads of 64 elements.
#include "cache_prefill.cuh"

namespace int4lib {

cudaError_t launch_cache_prefill_64(const AttentionArgs& a, DType t, void* workspace, cudaStream_t stream) {
  return launch_prefill<64>(a, t, workspace, stream);
}

}  // namespace int4lib
