// Attention over a paged cache: the launch plan, the join of split calls, and
// the choice between the two kernels (attention_few.hpp, attention_chunk.hpp).
#include <type_traits>

#include "attention.hpp"

namespace qlinear {

namespace {

using namespace attn;

// A row of the output and its partial results.
template <bool FEW>
struct JoinRow {
  int64_t out;       // row of the output
  int parts;
  int64_t row;       // chunk kernel: row in each range's results
  int worker, head;  // few-row kernel: the first worker of the row's tile, ...
  bool tail;         // ... whose span ends in the tile (its second result, if it starts before)
  int in_tile;
  __device__ __forceinline__ int64_t part(int i, const qlinear_kv_cache& c, const Plan& plan,
                                          const Partials& p) const {
    if constexpr (!FEW) return i * p.rows + row;
    return (((int64_t)(worker + i) * c.kv_heads + head) * 2 + (i == 0 && tail ? 1 : 0)) * plan.rows + in_tile;
  }
};

// FEW: row r of the (key/value head, sequence) in the grid's y and z; else row
// r of the tile and head in y. False: no such row, or nothing to join.
template <bool FEW>
__device__ __forceinline__ bool join_row(const AttentionArgs& a, const qlinear_kv_cache& c, const Plan& plan, int r,
                                         JoinRow<FEW>& j) {
  const int group = a.q_heads / c.kv_heads;
  Work w;
  if constexpr (FEW) {
    j.head = blockIdx.y;
    sequence(a, c, blockIdx.z, w);
    const Item it = few_item(a, plan, group, w);
    const int tile = r >> __builtin_ctz(plan.rows);
    if (tile >= it.tiles || r >= w.n * group) return false;
    const Spans sp = few_spans(a, c, plan, group);
    if (sp.whole) return false;
    const unsigned start = few_before(a, c, plan, group, sp, w.b) + tile * it.steps, last = start + it.steps - 1;
    j.worker = (int)(start / (unsigned)sp.quota);
    j.parts = (int)(last / (unsigned)sp.quota) - j.worker + 1;
    if (j.parts == 1) return false;      // one worker had the whole tile
    j.tail = start > (unsigned)j.worker * sp.quota;
    j.in_tile = r & (plan.rows - 1);
  } else {
    int tile = 0;
    j.head = blockIdx.y % c.kv_heads;
    if (!find_tile(a, c, plan, group, blockIdx.y / c.kv_heads, w, tile)) return false;
    r += tile * kChunkRows;
    if (r >= w.n * group) return false;
    j.parts = plan.splits;
  }
  j.out = (int64_t)(w.q0 + r / group) * a.q_heads + j.head * group + r % group;
  if constexpr (!FEW) j.row = j.out;
  return true;
}

// Joins partial results: o = sum_i f_i o_i / sum_i f_i l_i with f_i =
// 2^(m_i - max m), an empty range (m = -infinity) left out. A wave takes
// kJoinAtOnce results at a time: bound by the latency of its reads, which do
// not wait for one another. WAVES waves to a row take turns, and their sums are
// joined the same way; all in a fixed order.
constexpr int kJoinAtOnce = 16;
template <int D, bool FEW, int WAVES>
__global__ __launch_bounds__(256) void attention_join_kernel(AttentionArgs a, qlinear_kv_cache c, Plan plan,
                                                             Partials part) {
  constexpr int kLanes = D / 4, kSide = 64 / kLanes;     // lanes to a result, results side by side
  __shared__ float4v o_all[4][kLanes];
  __shared__ float2 ml_all[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, side = lane / kLanes, d = lane % kLanes;
  JoinRow<FEW> row;
  if (!join_row<FEW>(a, c, plan, blockIdx.x * (4 / WAVES) + wave / WAVES, row)) return;
  float top = -INFINITY, total = 0.0f;
  float4v o = {0, 0, 0, 0};
  for (int i0 = wave % WAVES * kJoinAtOnce; i0 < row.parts; i0 += WAVES * kJoinAtOnce) {
    const int n = min(kJoinAtOnce, row.parts - i0);
    float2 ml = make_float2(-INFINITY, 0.0f);
    if (lane < n) ml = part.ml[row.part(i0 + lane, c, plan, part)];
    float4v x[kJoinAtOnce / kSide];
#pragma unroll
    for (int k = 0; k < kJoinAtOnce / kSide; ++k) {
      const int i = k * kSide + side;
      x[k] = reinterpret_cast<const float4v*>(part.o)[row.part(i0 + (i < n ? i : 0), c, plan, part) * kLanes + d];
    }
    float most = ml.x;
#pragma unroll
    for (int k = 1; k < kJoinAtOnce; k <<= 1) most = fmaxf(most, __shfl_xor(most, k, kJoinAtOnce));
    most = fmaxf(top, __shfl(most, 0));
    const float keep = top == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(top - most);
    const float f = ml.x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ml.x - most);
    top = most;
    float sum = f * ml.y;
#pragma unroll
    for (int k = 1; k < kJoinAtOnce; k <<= 1) sum += __shfl_xor(sum, k, kJoinAtOnce);
    total = total * keep + __shfl(sum, 0);
    o *= keep;
#pragma unroll
    for (int k = 0; k < kJoinAtOnce / kSide; ++k) {
      const int i = k * kSide + side;
      const float fi = __shfl(f, i), mi = __shfl(ml.x, i);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] += mi == -INFINITY ? 0.0f : fi * x[k][e];
    }
  }
#pragma unroll
  for (int k = kLanes; k < 64; k <<= 1)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] += __shfl_xor(o[e], k);
  if constexpr (WAVES > 1) {     // the whole workgroup is on one row
    if (side == 0) o_all[wave][d] = o;
    if (lane == 0) ml_all[wave] = make_float2(top, total);
    __syncthreads();
    if (wave != 0) return;
    top = fmaxf(fmaxf(ml_all[0].x, ml_all[1].x), fmaxf(ml_all[2].x, ml_all[3].x));
    total = 0.0f;
    o = float4v{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (ml_all[i].x == -INFINITY) continue;
      const float f = __builtin_amdgcn_exp2f(ml_all[i].x - top);
      total += f * ml_all[i].y;
      o += f * o_all[i][d];
    }
  }
  if (side != 0) return;
  half4 y;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = (_Float16)(top == -INFINITY ? 0.0f : o[e] / total);
  *reinterpret_cast<half4*>(a.out + row.out * D + 4 * d) = y;
}

// `rows` rows for each place of the grid's y and z, of about `parts` results.
template <bool FEW>
hipError_t launch_join(const qlinear_kv_cache& c, const AttentionArgs& a, const Plan& p, const Partials& part,
                       int rows, dim3 grid, int64_t parts, hipStream_t stream) {
  auto go = [&](auto kernel, int waves) {
    grid.x = (unsigned)((rows * waves + 3) / 4);
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, a, c, p, part);
    return hipGetLastError();
  };
  auto width = [&](auto waves) {
    constexpr int W = decltype(waves)::value;
    if (c.head_dim == 64) return go(attention_join_kernel<64, FEW, W>, W);
    if (c.head_dim == 128) return go(attention_join_kernel<128, FEW, W>, W);
    return go(attention_join_kernel<256, FEW, W>, W);
  };
  // Four waves to a row if one would make several turns (64 results: 10.2 us
  // with one wave, 5.1 us with four).
  return parts > kJoinAtOnce ? width(std::integral_constant<int, 4>{}) : width(std::integral_constant<int, 1>{});
}

// Up to this many steps a workgroup takes a tile whole, and nothing is joined
// (us, split and whole: one sequence of 400 tokens 10.3 and 10.6 (32/32 heads),
// 8.1 and 5.9 (32/8 heads of 64); of 1000 11.0 and 18.4; 64 of 400, 64/8 heads,
// 35.6 and 21.9). Past it the lengths decide on the device (see Spans).
constexpr int kWholeSteps = 16;

// Steps of `tokens` tokens that a row tile spans at most.
int64_t plan_steps(const AttentionArgs& a, int tokens) {
  const int64_t reach = (int64_t)a.window + a.max_q_len;       // a window's start is inside a step
  if (a.window > 0 && reach < a.max_kv_len) return (reach + tokens - 1) / tokens + 1;
  return (a.max_kv_len + (int64_t)tokens - 1) / tokens;
}

// Workgroups of a key/value head that the chip holds at once, and as many of
// them as get four steps each at least; rows of their partial results.
int few_slots(const qlinear_kv_cache& c, int rows) {
  const int slots = 256 * few_per_cu(c.head_dim, rows, c.bits) / c.kv_heads;
  return slots > 1 ? slots : 1;
}
int few_workers(const qlinear_kv_cache& c, int rows, int64_t tiles, int64_t steps) {
  const int64_t slots = few_slots(c, rows), quarter = (tiles * steps + 3) / 4;
  return (int)(slots < quarter ? slots : quarter > 1 ? quarter : 1);
}
int64_t few_partial_rows(const qlinear_kv_cache& c, int rows, int workers) {
  return (int64_t)workers * c.kv_heads * 2 * rows;
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
    const int64_t tiles = (int64_t)(r.few_cap + p.rows - 1) / p.rows * a.batch;
    const int64_t steps = plan_steps(a, kStep);
    if (steps > kWholeSteps) {
      p.slots = few_slots(c, p.rows);
      p.workers = few_workers(c, p.rows, tiles, steps);
      // One sequence this long is always cut. Past twice the slots spans hold
      // several tiles each, and whole ones would gain little.
      if (a.batch > 1 && tiles <= 2 * p.slots) p.whole = (int)(tiles / a.batch);
      r.few_rows = few_partial_rows(c, p.rows, p.workers);
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
    if (splits > 1) {
      p.chunk = (int)((steps + splits - 1) / splits);
      p.splits = (int)((steps + p.chunk - 1) / p.chunk);
      r.chunk_rows = (int64_t)a.tokens * a.q_heads;
    }
  }
  return r;
}

// `ranges` results of `rows` rows each.
size_t partial_bytes(int64_t ranges, int64_t rows, int D) { return (size_t)(ranges * rows * (D + 2)) * sizeof(float); }

Partials partials(void* ws, int64_t ranges, int64_t rows, int D) {
  Partials part = {};
  if (rows == 0) return part;
  part.o = (float*)ws;
  part.ml = (float2*)(part.o + ranges * rows * D);
  part.rows = rows;
  return part;
}

}  // namespace

// The two kernels' launches follow one another on the stream and share the workspace.
size_t paged_attention_workspace_need(const qlinear_kv_cache& cache, const AttentionArgs& a) {
  const Route r = make_route(cache, a);
  const size_t few = partial_bytes(1, r.few_rows, cache.head_dim);
  const size_t chunk = partial_bytes(r.chunk_plan.splits, r.chunk_rows, cache.head_dim);
  return few > chunk ? few : chunk;
}

// Smaller calls may need more (fewer rows are split further), so this goes over
// the kinds of plan that a call of at most these sizes may have, each at its most.
size_t paged_attention_workspace_bytes(const qlinear_kv_cache& c, const AttentionArgs& a) {
  const int64_t group = a.q_heads / c.kv_heads, most = a.max_q_len * group;
  const int64_t cap = most < kFewRows ? most : kFewRows;
  // A window's steps are one more where fewer new tokens reach less far than the length bound.
  auto steps_of = [&](int tokens) {
    const int64_t reach = (int64_t)a.window + a.max_q_len, all = a.max_kv_len;
    const int64_t seen = a.window > 0 && reach < all ? reach : all;
    return (seen + tokens - 1) / tokens + (a.window > 0 ? 1 : 0);
  };
  int64_t rows = 0;
  auto few = [&](int tile_rows, int64_t most_rows) {
    const int64_t tiles = (most_rows + tile_rows - 1) / tile_rows * a.batch;
    const int64_t r = few_partial_rows(c, tile_rows, few_workers(c, tile_rows, tiles, steps_of(kStep)));
    if (r > rows) rows = r;
  };
  if ((group <= kFewRows || a.batch > 1) && steps_of(kStep) > kWholeSteps) {
    if (c.head_dim == 256)
      few(16, cap);
    else if (group <= 16)
      few(16, cap < 16 ? cap : 16);
    if (c.head_dim != 256 && cap > 16) few(32, cap);
  }
  const int64_t ranges = steps_of(chunk_step(c.head_dim)) / 8;
  if (most > kFewRows && ranges > 1 && 512 / c.kv_heads > 1) {
    // Ranges times tiles times heads are 512 at most, of kChunkRows rows each.
    const int64_t all = ranges * a.tokens * a.q_heads;
    const int64_t r = all < 512 * kChunkRows ? all : 512 * kChunkRows;
    if (r > rows) rows = r;
  }
  return partial_bytes(1, rows, c.head_dim);
}

hipError_t launch_paged_attention(const qlinear_kv_cache& cache, const AttentionArgs& a, void* ws,
                                  hipStream_t stream) {
  const Route r = make_route(cache, a);
  const int D = cache.head_dim, group = a.q_heads / cache.kv_heads;
  if (r.chunk) {
    const Plan& p = r.chunk_plan;
    const Partials part = partials(ws, p.splits, r.chunk_rows, D);
    const hipError_t e = D == 64    ? launch_attention_chunk_64(cache, a, p, part, stream)
                         : D == 128 ? launch_attention_chunk_128(cache, a, p, part, stream)
                                    : launch_attention_chunk_256(cache, a, p, part, stream);
    if (e != hipSuccess) return e;
    if (r.chunk_rows > 0) {
      // Splitting needs few workgroups, so the grid's y holds them.
      const hipError_t j = launch_join<false>(cache, a, p, part, kChunkRows,
                                              dim3(1, (unsigned)(chunk_tiles(a, group) * cache.kv_heads)), p.splits, stream);
      if (j != hipSuccess) return j;
    }
  }
  // Without q_start all sequences have the same length.
  if (r.few && (!r.chunk || a.q_start || (int64_t)(a.tokens / a.batch) * group <= kFewRows)) {
    const Plan& p = r.few_plan;
    const Partials part = partials(ws, 1, r.few_rows, D);
    const hipError_t e = D == 64    ? launch_attention_few_64(cache, a, p, part, stream)
                         : D == 128 ? launch_attention_few_128(cache, a, p, part, stream)
                                    : launch_attention_few_256(cache, a, p, part, stream);
    if (e != hipSuccess) return e;
    if (r.few_rows > 0)
      return launch_join<true>(cache, a, p, part, r.few_cap,
                               dim3(1, (unsigned)cache.kv_heads, (unsigned)a.batch), p.workers / a.batch, stream);
  }
  return hipSuccess;
}

}  // namespace qlinear
