// Few-row attention kernels for heads of 64 (attention_few.hpp).
#include "attention_few.hpp"

namespace qlinear {

hipError_t launch_attention_few_64(const qlinear_kv_cache& c, const AttentionArgs& a, const attn::Plan& p,
                                   const attn::Partials& part, hipStream_t stream) {
  return attn::launch_few_width<64>(c, a, p, part, stream);
}

}  // namespace qlinear
