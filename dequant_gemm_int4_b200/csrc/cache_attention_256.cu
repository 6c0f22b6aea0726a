// The tensor-core attention kernels for heads of 256 elements.
#include "cache_attention.cuh"

namespace int4lib {

namespace {

template <class F>
bool pick(int group, bool asym, int rt, F&& f) {
  bool found = false;
  switch (group) {
    case 32:
      found = with_attention_cfg<256, 32>(asym, rt, f);
      break;
    case 64:
      found = with_attention_cfg<256, 64>(asym, rt, f);
      break;
    case 128:
      found = with_attention_cfg<256, 128>(asym, rt, f);
      break;
    case 256:
      found = with_attention_cfg<256, 256>(asym, rt, f);
      break;
    default:
      break;
  }
  return found;
}

}  // namespace

cudaError_t launch_cache_attention_256(const AttentionArgs& a, DType t, int rt, void* workspace,
                                      cudaStream_t stream) {
  cudaError_t e = cudaErrorInvalidValue;
  pick(a.cache.group, a.cache.zeros != nullptr, rt, [&](auto cfg) {
    using C = decltype(cfg);
    e = t == DType::BF16 ? launch_attention_cfg<__nv_bfloat16, C>(a, workspace, stream)
                         : launch_attention_cfg<__half, C>(a, workspace, stream);
  });
  return e;
}

int cache_attention_blocks_256(int group, bool asym, int rt) {
  int n = 0;
  pick(group, asym, rt, [&](auto cfg) { n = attention_blocks<decltype(cfg)>(); });
  return n;
}

}  // namespace int4lib
