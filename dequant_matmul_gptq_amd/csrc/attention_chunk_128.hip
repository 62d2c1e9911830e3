// Chunk attention kernels for heads of 128 (attention_chunk.hpp).
#include "attention_chunk.hpp"

namespace qlinear {

hipError_t launch_attention_chunk_128(const qlinear_kv_cache& c, const AttentionArgs& a, const attn::Plan& p,
                                      const attn::Partials& part, hipStream_t stream) {
  return attn::launch_chunk_width<128>(c, a, p, part, stream);
}

}  // namespace qlinear
