// Attention of new tokens over a paged cache, one wave per (token, query
// head): 64 keys a step, one per lane, with the running maximum m and sum l of
// the softmax; o and l are scaled by exp(m_old - m_new) when m grows.
#include "qlinear_kernels.hpp"

namespace qlinear {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// Element d of cache row r of a pool.
__device__ __forceinline__ float cache_value(const void* pool, const uint16_t* scales, int64_t r, int d, int D,
                                             int bits, int group) {
  if (bits == 16) return (float)reinterpret_cast<const _Float16*>(pool)[r * D + d];
  const uint32_t* w = reinterpret_cast<const uint32_t*>(pool) + r * (D * bits / 32);
  const int pos = d * bits, k = pos >> 5, sh = pos & 31;
  uint32_t v = w[k] >> sh;
  if (sh + bits > 32) v |= w[k + 1] << (32 - sh);
  const float s = (float)__builtin_bit_cast(_Float16, scales[r * (D / group) + d / group]);
  return (float)(_Float16)(s * (float)((int)(v & ((1u << bits) - 1u)) - (1 << (bits - 1))));
}

__global__ __launch_bounds__(256) void attention_row_kernel(AttentionArgs a, qlinear_kv_cache c) {
  __shared__ float qs[4][256];
  const int D = c.head_dim, lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t row = (int64_t)blockIdx.x * 4 + wv;
  const bool live = row < (int64_t)a.tokens * a.q_heads;
  const int tok = live ? (int)(row / a.q_heads) : 0, h = live ? (int)(row % a.q_heads) : 0;
  const int hk = h / (a.q_heads / c.kv_heads);
  int b = -1, first = 0, last = 0;
  if (a.q_start) {
    for (int i = 0; i < a.batch; ++i)
      if (tok >= a.q_start[i] && tok < a.q_start[i + 1]) {
        b = i;
        first = a.q_start[i];
        last = a.q_start[i + 1];
      }
  } else {
    const int n = a.tokens / a.batch;
    b = tok / n;
    first = b * n;
    last = first + n;
  }
  for (int d = lane; d < D; d += 64)
    qs[wv][d] = live ? (float)__builtin_bit_cast(_Float16, a.q[tok * a.q_stride + (int64_t)h * D + d]) : 0.0f;
  __syncthreads();
  if (!live || b < 0) return;
  const int64_t cap = (int64_t)a.table_width * c.page_size;
  const int L = (int)min((int64_t)max(a.kv_len[b], 0), cap);
  const int p = L - (last - first) + (tok - first);
  const int lo = a.window > 0 ? max(0, p - a.window + 1) : 0;
  float m = -INFINITY, l = 0.0f, o[4] = {0, 0, 0, 0};
  auto slot = [&](int t) {
    int pg = a.block_table[(int64_t)b * a.table_width + t / c.page_size];
    pg = min(max(pg, 0), c.num_pages - 1);
    return ((int64_t)pg * c.kv_heads + hk) * c.page_size + t % c.page_size;
  };
  for (int t0 = lo; t0 <= p; t0 += 64) {
    const int t = t0 + lane;
    float s = -INFINITY;
    if (t <= p) {
      const int64_t r = slot(t);
      s = 0.0f;
      for (int d = 0; d < D; ++d) s += qs[wv][d] * cache_value(c.k, c.k_scales, r, d, D, c.bits, c.group);
      s *= a.scale * kLog2e;
    }
    float mx = s;
    for (int k = 1; k < 64; k <<= 1) mx = fmaxf(mx, __shfl_xor(mx, k));
    const float mn = fmaxf(m, mx);
    const float alpha = exp2f(m - mn), e = t <= p ? exp2f(s - mn) : 0.0f;
    float es = e;
    for (int k = 1; k < 64; k <<= 1) es += __shfl_xor(es, k);
    l = l * alpha + es;
    m = mn;
    for (int i = 0; i < 4; ++i) o[i] *= alpha;
    for (int j = 0; j < 64 && t0 + j <= p; ++j) {
      const float pj = __shfl(e, j);
      const int64_t r = slot(t0 + j);
      for (int i = 0; i < D / 64; ++i)
        o[i] += pj * cache_value(c.v, c.v_scales, r, lane + 64 * i, D, c.bits, c.group);
    }
  }
  for (int i = 0; i < D / 64; ++i)
    a.out[((int64_t)tok * a.q_heads + h) * D + lane + 64 * i] =
        __builtin_bit_cast(uint16_t, (_Float16)(l > 0.0f || l != l ? o[i] / l : 0.0f));
}

}  // namespace

size_t paged_attention_workspace_bytes(const qlinear_kv_cache&, const AttentionArgs&) { return 0; }

hipError_t launch_paged_attention(const qlinear_kv_cache& cache, const AttentionArgs& a, void*, hipStream_t stream) {
  const int64_t rows = (int64_t)a.tokens * a.q_heads;
  hipLaunchKernelGGL(attention_row_kernel, dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, stream, a, cache);
  return hipGetLastError();
}

}  // namespace qlinear
