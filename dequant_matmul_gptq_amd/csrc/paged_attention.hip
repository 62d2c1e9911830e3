// Attention over a paged cache: the launch plan, the join of split calls, and
// the choice between the two kernels (attention_few.hpp, attention_chunk.hpp).
#include <stdlib.h>
#include "attention.hpp"

namespace qlinear {

namespace {

using namespace attn;

// The row of a join's workgroup: FEW, row r of (key/value head, sequence) in
// the grid's y and z; else row r of the tile and head in y. False: no such row.
struct JoinRow {
  int64_t out, part;     // row of the output, of the partial results
};
template <bool FEW>
__device__ __forceinline__ bool join_row(const AttentionArgs& a, const qlinear_kv_cache& c, const Plan& plan,
                                         const Partials& part, int r, JoinRow& j) {
  const int group = a.q_heads / c.kv_heads;
  Work w;
  int head;
  if constexpr (FEW) {
    head = blockIdx.y;
    sequence(a, c, blockIdx.z, w);
    const int64_t seq_rows = (int64_t)w.n * group;
    if (r >= seq_rows || seq_rows > plan.max_rows) return false;
  } else {
    int tile = 0;
    head = blockIdx.y % c.kv_heads;
    if (!find_tile(a, c, plan, group, blockIdx.y / c.kv_heads, w, tile)) return false;
    r += tile * kChunkRows;
    if (r >= w.n * group) return false;
  }
  j.out = (int64_t)(w.q0 + r / group) * a.q_heads + head * group + r % group;
  j.part = FEW ? ((int64_t)w.b * c.kv_heads + head) * part.cap + r : j.out;
  return true;
}

// Joins the partial results of a split launch: o = sum_s f_s o_s / sum_s f_s
// l_s with f_s = 2^(m_s - max m), an empty range (m = -infinity, o not
// written) left out. Bound by the latency of its reads, so few of them wait
// for one another. Up to kJoinFew ranges: one wave a row, all reads at once.
constexpr int kJoinFew = 16;
template <int D, bool FEW>
__global__ __launch_bounds__(256) void attention_join_few_kernel(AttentionArgs a, qlinear_kv_cache c, Plan plan,
                                                                 Partials part) {
  constexpr int kLanes = D / 4, kSide = 64 / kLanes;     // lanes to a range, ranges at a time
  const int lane = threadIdx.x & 63, side = lane / kLanes, d = lane % kLanes;
  JoinRow row;
  if (!join_row<FEW>(a, c, plan, part, blockIdx.x * 4 + (threadIdx.x >> 6), row)) return;
  const int splits = plan.splits;
  float2 ml = make_float2(-INFINITY, 0.0f);
  if (lane < splits) ml = part.ml[lane * part.rows + row.part];
  const float4v* p = reinterpret_cast<const float4v*>(part.o) + row.part * kLanes + d;
  float4v x[kJoinFew / kSide];
#pragma unroll
  for (int i = 0; i < kJoinFew / kSide; ++i) {
    const int s = i * kSide + side;
    x[i] = p[(s < splits ? s : 0) * part.rows * kLanes];
  }
  float top = ml.x;
#pragma unroll
  for (int k = 1; k < kJoinFew; k <<= 1) top = fmaxf(top, __shfl_xor(top, k, kJoinFew));
  top = __shfl(top, 0);
  const float f = ml.x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ml.x - top);
  float total = f * ml.y;
#pragma unroll
  for (int k = 1; k < kJoinFew; k <<= 1) total += __shfl_xor(total, k, kJoinFew);
  total = __shfl(total, 0);
  float4v o = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < kJoinFew / kSide; ++i) {
    const int s = i * kSide + side;
    const float fs = __shfl(f, s), ms = __shfl(ml.x, s);
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] += ms == -INFINITY ? 0.0f : fs * x[i][e];
  }
#pragma unroll
  for (int k = kLanes; k < 64; k <<= 1)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] += __shfl_xor(o[e], k);
  if (side != 0) return;
  half4 y;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = (_Float16)(top == -INFINITY ? 0.0f : o[e] / total);
  *reinterpret_cast<half4*>(a.out + row.out * D + 4 * d) = y;
}

// More ranges: a workgroup a row, the weights kJoinBatch at a time in LDS,
// then D / 4 threads to a range and several loads in flight. Threads and
// ranges are added in a fixed order.
constexpr int kJoinBatch = 256;
template <int D, bool FEW>
__global__ __launch_bounds__(256) void attention_join_kernel(AttentionArgs a, qlinear_kv_cache c, Plan plan,
                                                             Partials part) {
  constexpr int kSide = 256 / (D / 4);    // ranges at a time
  __shared__ float weight[kJoinBatch];
  __shared__ float tops[4], sums[4];
  __shared__ float4v o_part[kSide][D / 4];
  JoinRow at;
  if (!join_row<FEW>(a, c, plan, part, blockIdx.x, at)) return;
  const int64_t row = at.part, rows = part.rows;
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
      const float f = ml.x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ml.x - top);
      weight[t] = ml.x == -INFINITY ? -1.0f : f;       // -1: left out
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
  *reinterpret_cast<half4*>(a.out + at.out * D + 4 * d) = y;
}

template <int D, bool FEW>
hipError_t launch_join_width(const qlinear_kv_cache& c, const AttentionArgs& a, const Plan& p, const Partials& part,
                             int rows, dim3 grid, hipStream_t stream) {
  const bool few = p.splits <= kJoinFew;
  grid.x = (unsigned)(few ? (rows + 3) / 4 : rows);
  auto kernel = few ? attention_join_few_kernel<D, FEW> : attention_join_kernel<D, FEW>;
  hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, a, c, p, part);
  return hipGetLastError();
}

// `rows` rows for each place of the grid's y and z.
template <bool FEW>
hipError_t launch_join(const qlinear_kv_cache& c, const AttentionArgs& a, const Plan& p, const Partials& part,
                       int rows, dim3 grid, hipStream_t stream) {
  if (c.head_dim == 64) return launch_join_width<64, FEW>(c, a, p, part, rows, grid, stream);
  if (c.head_dim == 128) return launch_join_width<128, FEW>(c, a, p, part, rows, grid, stream);
  return launch_join_width<256, FEW>(c, a, p, part, rows, grid, stream);
}

// Steps of `tokens` tokens that a row tile spans at most.
int64_t plan_steps(const AttentionArgs& a, int tokens) {
  const int64_t reach = (int64_t)a.window + a.max_q_len;       // a window's start is inside a step
  if (a.window > 0 && reach < a.max_kv_len) return (reach + tokens - 1) / tokens + 1;
  return (a.max_kv_len + (int64_t)tokens - 1) / tokens;
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
    // Ranges for two workgroups per CU (what their registers allow), of 4 to
    // 64 steps: shorter ones cost more in partial results than they spread
    // (64 sequences of 2048 tokens, 64/8 heads: 96.8 us whole, 102.6, 107, 123
    // us in ranges of 64, 16, 4 steps), longer ones leave CUs idle at the end
    // (one of 32768: 31.0, 31.1, 40.1 us in ranges of 16, 64, 96).
    int64_t chunk = (tiles * steps + 511) / 512;
    if (chunk < 4) chunk = 4;
    if (chunk > 64) chunk = 64;
    if (getenv("QL_CHUNK")) chunk = atoi(getenv("QL_CHUNK"));
    p.splits = (int)((steps + chunk - 1) / chunk);
    if (p.splits < 1) p.splits = 1;
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
      // Splitting needs few workgroups, so the grid's y holds them.
      const hipError_t j = launch_join<false>(cache, a, p, part, kChunkRows,
                                              dim3(1, (unsigned)(chunk_tiles(a, group) * cache.kv_heads)), stream);
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
    if (r.few_rows > 0)
      return launch_join<true>(cache, a, p, part, r.few_cap,
                               dim3(1, (unsigned)cache.kv_heads, (unsigned)a.batch), stream);
  }
  return hipSuccess;
}

}  // namespace qlinear
