// Attention of new tokens over a paged cache, one wave per (token, query
// head): 64 keys a step, one per lane, with the running maximum m and sum l of
// the softmax; o and l are scaled by exp(m_old - m_new) when m grows.
#include <stdlib.h>
#include "attention.hpp"

namespace qlinear {

namespace {

using namespace attn;

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

// Joins the partial results of a split call, one workgroup per row: the
// ranges' weights 2^(m - max m) first (kJoinBatch at a time in LDS), then the
// sum over ranges with D / 4 threads to a range and several loads in flight.
// Threads and ranges are added in a fixed order.
constexpr int kJoinBatch = 256;
template <int D>
__global__ __launch_bounds__(256) void attention_join_kernel(AttentionArgs a, Partials part, int splits) {
  constexpr int kSide = 256 / (D / 4);    // ranges at a time
  __shared__ float weight[kJoinBatch];
  __shared__ float tops[4], sums[4];
  __shared__ float4v o_part[kSide][D / 4];
  const int64_t row = blockIdx.x, rows = (int64_t)a.tokens * a.q_heads;
  const int tok = blockIdx.x / a.q_heads;
  if (a.q_start && (tok < a.q_start[0] || tok >= a.q_start[a.batch])) return;   // of no sequence
  const int t = threadIdx.x, side = t / (D / 4), d = t % (D / 4);
  float top = -INFINITY;
  for (int s = t; s < splits; s += 256) top = fmaxf(top, part.ml[s * rows + row].x);
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) top = fmaxf(top, __shfl_xor(top, k));
  if ((t & 63) == 0) tops[t >> 6] = top;
  __syncthreads();
  top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));

  float total = 0.0f;
  float4v o = {0, 0, 0, 0};
  for (int s0 = 0; s0 < splits; s0 += kJoinBatch) {
    const int n = min(kJoinBatch, splits - s0);
    if (s0) __syncthreads();
    if (t < n) {
      const float2 ml = part.ml[(s0 + t) * rows + row];
      // An empty range (m = -infinity) has weight 0 and its o is not written.
      const float f = ml.x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ml.x - top);
      weight[t] = ml.x == -INFINITY ? -1.0f : f;
      total += f * ml.y;
    }
    __syncthreads();
    const float4v* p = reinterpret_cast<const float4v*>(part.o) + ((int64_t)s0 * rows + row) * (D / 4) + d;
#pragma unroll 4
    for (int s = side; s < n; s += kSide) {
      const float f = weight[s];
      if (f >= 0.0f || f != f) o += f * p[s * rows * (D / 4)];
    }
  }
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) total += __shfl_xor(total, k);
  if ((t & 63) == 0) sums[t >> 6] = total;
  o_part[side][d] = o;
  __syncthreads();
  if (side != 0) return;
  total = sums[0] + sums[1] + sums[2] + sums[3];
#pragma unroll
  for (int i = 1; i < kSide; ++i) o += o_part[i][d];
  half4 y;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = (_Float16)(top == -INFINITY ? 0.0f : o[e] / total);
  *reinterpret_cast<half4*>(a.out + row * D + 4 * d) = y;
}

// Tokens a row tile can see at most, in steps.
int64_t plan_steps(const AttentionArgs& a) {
  int64_t n = a.max_kv_len;
  if (a.window > 0 && (int64_t)a.window + a.max_q_len < n) n = (int64_t)a.window + a.max_q_len;
  return n / kStep + 2;
}

constexpr int kFewRows = 64;       // most rows of a sequence per key/value head in the few-row kernel

Plan make_plan(const qlinear_kv_cache& c, const AttentionArgs& a) {
  const int64_t group = a.q_heads / c.kv_heads, rows = a.max_q_len * group;
  Plan p;
  p.rows = rows <= 16 || c.head_dim == 256 ? 16 : 32;   // two tiles of 256 wide heads do not fit the registers
  p.splits = 1;
  p.chunk = INT32_MAX;
  if (rows > kFewRows) return p;
  const int64_t tiles = (rows + p.rows - 1) / p.rows * c.kv_heads * a.batch;
  const int64_t steps = plan_steps(a);
  // A range is long enough that writing and reading its partial result is
  // about 1/25 of reading its keys and values, unless that leaves fewer than
  // two workgroups per CU; short enough for about 4096 workgroups.
  const int64_t row_bytes = c.bits == 16 ? 2 * c.head_dim : c.head_dim * c.bits / 8 + 2 * c.head_dim / c.group;
  const int64_t used = rows < p.rows ? rows : p.rows;
  const int64_t light = 25 * used * c.head_dim * 4 / (row_bytes * kStep);
  const int64_t even = (tiles * steps + 4095) / 4096;
  const int64_t fill = (tiles * steps + 511) / 512;
  int64_t chunk = even > light ? even : light;
  if (chunk > fill) chunk = fill;
  if (chunk < 4) chunk = 4;
  if (getenv("QL_CHUNK")) chunk = atoi(getenv("QL_CHUNK"));
  p.splits = (int)((steps + chunk - 1) / chunk);
  if (p.splits > 1) p.chunk = (int)chunk;
  return p;
}

}  // namespace

size_t paged_attention_workspace_bytes(const qlinear_kv_cache& cache, const AttentionArgs& a) {
  const Plan p = make_plan(cache, a);
  if (p.splits == 1) return 0;
  return (size_t)p.splits * a.tokens * a.q_heads * (cache.head_dim + 2) * sizeof(float);
}

hipError_t launch_paged_attention(const qlinear_kv_cache& cache, const AttentionArgs& a, void* ws,
                                  hipStream_t stream) {
  const Plan p = make_plan(cache, a);
  const int64_t rows = (int64_t)a.tokens * a.q_heads;
  if ((int64_t)a.max_q_len * (a.q_heads / cache.kv_heads) > kFewRows) {
    hipLaunchKernelGGL(attention_row_kernel, dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, stream, a, cache);
    return hipGetLastError();
  }
  Partials part = {};
  part.o = (float*)ws;
  if (p.splits > 1) part.ml = (float2*)(part.o + (int64_t)p.splits * rows * cache.head_dim);
  hipError_t e = cache.head_dim == 64    ? launch_attention_few_64(cache, a, p, part, stream)
                 : cache.head_dim == 128 ? launch_attention_few_128(cache, a, p, part, stream)
                                         : launch_attention_few_256(cache, a, p, part, stream);
  if (e != hipSuccess || p.splits == 1) return e;
  auto join = cache.head_dim == 64    ? attention_join_kernel<64>
              : cache.head_dim == 128 ? attention_join_kernel<128>
                                      : attention_join_kernel<256>;
  hipLaunchKernelGGL(join, dim3((unsigned)rows), dim3(256), 0, stream, a, part, p.splits);
  return hipGetLastError();
}

}  // namespace qlinear
