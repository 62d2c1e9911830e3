// Attention over a paged cache: the launch plan, the join of split calls, and
// the choice between the two kernels (attention_few.hpp, attention_chunk.hpp).
#include <stdlib.h>
#include "attention.hpp"

namespace qlinear {

namespace {

using namespace attn;

// Joins the partial results of a split launch, one workgroup per row: the
// ranges' weights 2^(m - max m) first (kJoinBatch at a time in LDS), then the
// sum over ranges with D / 4 threads to a range and several loads in flight.
// Threads and ranges are added in a fixed order.
// FEW: workgroup (row, key/value head, sequence); else (row tile and head,
// row).
constexpr int kJoinBatch = 256;
template <int D, bool FEW>
__global__ __launch_bounds__(256) void attention_join_kernel(AttentionArgs a, qlinear_kv_cache c, Plan plan,
                                                             Partials part) {
  constexpr int kSide = 256 / (D / 4);    // ranges at a time
  __shared__ float weight[kJoinBatch];
  __shared__ float tops[4], sums[4];
  __shared__ float4v o_part[kSide][D / 4];
  const int group = a.q_heads / c.kv_heads;
  Work w;
  int r, head;
  if constexpr (FEW) {
    r = blockIdx.x;
    head = blockIdx.y;
    sequence(a, c, blockIdx.z, w);
    const int64_t seq_rows = (int64_t)w.n * group;
    if (r >= seq_rows || seq_rows > plan.max_rows) return;
  } else {
    int tile = 0;
    head = blockIdx.x % c.kv_heads;
    if (!find_tile(a, c, plan, group, blockIdx.x / c.kv_heads, w, tile)) return;
    r = tile * kChunkRows + blockIdx.y;
    if (r >= w.n * group) return;
  }
  const int64_t out_row = (int64_t)(w.q0 + r / group) * a.q_heads + head * group + r % group;
  const int64_t row = FEW ? ((int64_t)w.b * c.kv_heads + head) * part.cap + r : out_row, rows = part.rows;
  const int splits = plan.splits;
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
      // An empty range (m = -infinity) has no o: weight -1 says so.
      const float f = ml.x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ml.x - top);
      weight[t] = ml.x == -INFINITY ? -1.0f : f;
      total += f * ml.y;
    }
    __syncthreads();
    const float4v* p = reinterpret_cast<const float4v*>(part.o) + (s0 * rows + row) * (D / 4) + d;
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
  *reinterpret_cast<half4*>(a.out + out_row * D + 4 * d) = y;
}

// Steps of `tokens` that a row tile can span at most.
int64_t plan_steps(const AttentionArgs& a, int tokens) {
  int64_t n = a.max_kv_len;
  if (a.window > 0 && (int64_t)a.window + a.max_q_len < n) n = (int64_t)a.window + a.max_q_len;
  return n / tokens + 2;
}

// The sequences of a call are served by their number of rows per key/value
// head: up to kFewRows by the few-row kernel, more by the chunk kernel. A call
// launches the kernels that it may need.
struct Route {
  bool few, chunk;
  Plan few_plan, chunk_plan;
  int few_cap;                      // rows per sequence and key/value head
  int64_t few_rows, chunk_rows;     // rows of the partial results, 0 if not split
};

Route make_route(const qlinear_kv_cache& c, const AttentionArgs& a) {
  const int64_t group = a.q_heads / c.kv_heads, most = a.max_q_len * group;
  Route r = {};
  r.chunk = most > kFewRows;
  r.few = !r.chunk || a.batch > 1;
  if (r.few) {
    Plan& p = r.few_plan;
    r.few_cap = (int)(most < kFewRows ? most : kFewRows);
    // Two tiles of 256 wide heads do not fit the registers.
    p.rows = r.few_cap <= 16 || c.head_dim == 256 ? 16 : 32;
    p.min_rows = 1;
    p.max_rows = kFewRows;
    p.splits = 1;
    p.chunk = INT32_MAX;
    const int64_t tiles = (int64_t)(r.few_cap + p.rows - 1) / p.rows * c.kv_heads * a.batch;
    const int64_t steps = plan_steps(a, kStep);
    // A range is long enough that writing and reading its partial result is
    // about 1/25 of reading its keys and values, unless that leaves fewer than
    // two workgroups per CU; short enough for about 4096 workgroups.
    const int64_t row_bytes = c.bits == 16 ? 2 * c.head_dim : c.head_dim * c.bits / 8 + 2 * c.head_dim / c.group;
    const int64_t used = r.few_cap < p.rows ? r.few_cap : p.rows;
    const int64_t light = 25 * used * c.head_dim * 4 / (row_bytes * kStep);
    const int64_t even = (tiles * steps + 4095) / 4096;
    const int64_t fill = (tiles * steps + 511) / 512;
    int64_t chunk = even > light ? even : light;
    if (chunk > fill) chunk = fill;
    if (chunk < 4) chunk = 4;
    if (getenv("QL_CHUNK")) chunk = atoi(getenv("QL_CHUNK"));
    p.splits = (int)((steps + chunk - 1) / chunk);
    if (p.splits > 1) {
      p.chunk = (int)chunk;
      r.few_rows = (int64_t)a.batch * c.kv_heads * r.few_cap;
    }
  }
  if (r.chunk) {
    Plan& p = r.chunk_plan;
    p.rows = kChunkRows;
    p.min_rows = r.few ? kFewRows + 1 : 1;
    p.max_rows = INT32_MAX;
    p.splits = 1;
    p.chunk = INT32_MAX;
    // Two workgroups per CU, each with at least eight steps.
    const int64_t groups = chunk_tiles(a, (int)group) * c.kv_heads;
    const int64_t steps = plan_steps(a, chunk_step(c.head_dim));
    int64_t splits = 512 / groups;
    if (splits > steps / 8) splits = steps / 8;
    if (getenv("QL_SPLITS")) splits = atoi(getenv("QL_SPLITS"));
    if (splits > 1) {
      p.chunk = (int)((steps + splits - 1) / splits);
      p.splits = (int)((steps + p.chunk - 1) / p.chunk);
      r.chunk_rows = (int64_t)a.tokens * a.q_heads;
    }
  }
  return r;
}

size_t partial_bytes(const Plan& p, int64_t rows, int D) { return (size_t)p.splits * rows * (D + 2) * sizeof(float); }

Partials partials(void* ws, const Plan& p, int64_t rows, int cap, int D) {
  Partials part = {};
  if (rows == 0) return part;
  part.o = (float*)ws;
  part.ml = (float2*)(part.o + (int64_t)p.splits * rows * D);
  part.rows = rows;
  part.cap = cap;
  return part;
}

}  // namespace

// The two kernels' launches follow one another on the stream and share the workspace.
size_t paged_attention_workspace_bytes(const qlinear_kv_cache& cache, const AttentionArgs& a) {
  const Route r = make_route(cache, a);
  const size_t few = partial_bytes(r.few_plan, r.few_rows, cache.head_dim);
  const size_t chunk = partial_bytes(r.chunk_plan, r.chunk_rows, cache.head_dim);
  return few > chunk ? few : chunk;
}

hipError_t launch_paged_attention(const qlinear_kv_cache& cache, const AttentionArgs& a, void* ws,
                                  hipStream_t stream) {
  const Route r = make_route(cache, a);
  const int D = cache.head_dim, group = a.q_heads / cache.kv_heads;
  if (r.chunk) {
    const Plan& p = r.chunk_plan;
    const Partials part = partials(ws, p, r.chunk_rows, 0, D);
    const hipError_t e = D == 64    ? launch_attention_chunk_64(cache, a, p, part, stream)
                         : D == 128 ? launch_attention_chunk_128(cache, a, p, part, stream)
                                    : launch_attention_chunk_256(cache, a, p, part, stream);
    if (e != hipSuccess) return e;
    if (r.chunk_rows > 0) {
      auto join = D == 64    ? attention_join_kernel<64, false>
                  : D == 128 ? attention_join_kernel<128, false>
                             : attention_join_kernel<256, false>;
      hipLaunchKernelGGL(join, dim3((unsigned)(chunk_tiles(a, group) * cache.kv_heads), kChunkRows), dim3(256), 0,
                         stream, a, cache, p, part);
      const hipError_t j = hipGetLastError();
      if (j != hipSuccess) return j;
    }
  }
  // Without q_start all sequences have the same length.
  if (r.few && (!r.chunk || a.q_start || (int64_t)(a.tokens / a.batch) * group <= kFewRows)) {
    const Plan& p = r.few_plan;
    const Partials part = partials(ws, p, r.few_rows, r.few_cap, D);
    const hipError_t e = D == 64    ? launch_attention_few_64(cache, a, p, part, stream)
                         : D == 128 ? launch_attention_few_128(cache, a, p, part, stream)
                                    : launch_attention_few_256(cache, a, p, part, stream);
    if (e != hipSuccess) return e;
    if (r.few_rows > 0) {
      auto join = D == 64    ? attention_join_kernel<64, true>
                  : D == 128 ? attention_join_kernel<128, true>
                             : attention_join_kernel<256, true>;
      hipLaunchKernelGGL(join, dim3((unsigned)r.few_cap, (unsigned)cache.kv_heads, (unsigned)a.batch), dim3(256), 0,
                         stream, a, cache, p, part);
      return hipGetLastError();
    }
  }
  return hipSuccess;
}

}  // namespace qlinear
