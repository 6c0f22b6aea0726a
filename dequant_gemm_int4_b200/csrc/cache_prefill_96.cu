// The tcgen05 attention kernels for heads of 96 elements.
#include "cache_prefill.cuh"

namespace int4lib {

cudaError_t launch_cache_prefill_96(const AttentionArgs& a, DType t, void* workspace, cudaStream_t stream) {
  return launch_prefill<96>(a, t, workspace, stream);
}

}  // namespace int4lib
