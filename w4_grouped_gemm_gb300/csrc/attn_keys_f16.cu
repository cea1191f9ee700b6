// attn_keys_f16.cu -- the key kernels of attn_keys.cuh for fp16.
#include "attn_keys.cuh"

namespace lily {

cudaError_t launch_attn_keys_f16(const AttnArgs& a, const AttnSet& pa, const AttnSet& pb,
                                  const CUtensorMap& mk, const CUtensorMap& mv, bool first,
                                  cudaStream_t s) {
  return launch_keys_type<true>({a, pa, pb, mk, mv, first, s});
}

}  // namespace lily
