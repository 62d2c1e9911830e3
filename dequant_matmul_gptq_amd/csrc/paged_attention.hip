// Attention over a paged cache, plain calls: the choice between the two kernels
// (attention_few.hpp, attention_chunk.hpp) by the plan of attention_plan.hpp.
#include "attention_plan.hpp"

namespace qlinear {

size_t paged_attention_workspace_need(const qlinear_kv_cache& cache, const AttentionArgs& a) {
  return attn::workspace_need(cache, a);
}

size_t paged_attention_workspace_bytes(const qlinear_kv_cache& cache, const AttentionArgs& a) {
  return attn::workspace_bytes(cache, a);
}

hipError_t launch_paged_attention(const qlinear_kv_cache& cache, const AttentionArgs& a, void* ws,
                                  hipStream_t stream) {
  auto few = [](int D) {
    return D == 64 ? launch_attention_few_64 : D == 128 ? launch_attention_few_128 : launch_attention_few_256;
  };
  auto chunk = [](int D) {
    return D == 64 ? launch_attention_chunk_64 : D == 128 ? launch_attention_chunk_128 : launch_attention_chunk_256;
  };
  return attn::launch_attention<attn::Partials>(cache, a, ws, few, chunk, stream);
}

}  // namespace qlinear
