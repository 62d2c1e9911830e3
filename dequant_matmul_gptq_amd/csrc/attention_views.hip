// Attention over a paged cache, views: windows with sinks, and shared prefixes
// (see attention.hpp). Sinks go the way of plain calls. With shared prefixes each
// row of the output has results of its group's prefix and of its sequence's own
// tokens, whole or in parts, which a last launch joins:
//   o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i,  m = max m_i
#include "attention_plan.hpp"

namespace qlinear {

namespace {

using namespace attn;

auto few_launcher(int D) {
  return D == 64 ? launch_view_few_64 : D == 128 ? launch_view_few_128 : launch_view_few_256;
}
auto chunk_launcher(int D) {
  return D == 64 ? launch_view_chunk_64 : D == 128 ? launch_view_chunk_128 : launch_view_chunk_256;
}

// A row's results of one kind: result 0 at `first`, i at rest + i stride.
struct Results {
  int parts;
  int64_t first, rest, stride;
  __device__ __forceinline__ int64_t at(int i) const { return i == 0 ? first : rest + i * stride; }
};

struct SharedPlan {
  Plan few, chunk;
};

// Results of row `out` of the output as row r of the tile rows of sequence w
// and head.
__device__ __forceinline__ Results results_of(const ViewArgs& a, const qlinear_kv_cache& c, const SharedPlan& p,
                                              const ViewPartials& part, const Spans& sp, int group, const Work& w,
                                              int head, int r, int64_t out) {
  Results x = {1, (w.all ? 0 : part.rows) + out, 0, 0};       // whole
  if (w.n * group > kFewRows) {
    if (p.chunk.splits > 1) {
      x.parts = p.chunk.splits;
      x.first = x.rest = part.chunk0 + (w.all ? 0 : part.chunk_kinds - 1) * part.rows + out;
      x.stride = part.chunk_kinds * part.rows;
    }
    return x;
  }
  if (p.few.workers == 0 || sp.whole) return x;
  const Item it = few_item(a, p.few, group, w);
  const int tile = r >> __builtin_ctz(p.few.rows);
  const unsigned start = few_before(a, c, p.few, group, sp, w.b) + tile * it.steps, last = start + it.steps - 1;
  const int worker = (int)(start / (unsigned)sp.quota), parts = (int)(last / (unsigned)sp.quota) - worker + 1;
  if (parts == 1) return x;
  const bool tail = start > (unsigned)worker * sp.quota;
  x.parts = parts;
  x.rest = part.few0 + (((int64_t)worker * c.kv_heads + head) * 2) * p.few.rows + (r & (p.few.rows - 1));
  x.first = x.rest + (tail ? p.few.rows : 0);
  x.stride = (int64_t)c.kv_heads * 2 * p.few.rows;
  return x;
}

// Sequence of row `token` of q, 0 .. n - 1; all lanes together.
__device__ __forceinline__ int sequence_of(const ViewArgs& a, int n, int token) {
  if (!a.q_start) return min(token / (a.tokens / n), n - 1);
  const int lane = threadIdx.x & 63;
  for (int b0 = 0; b0 < n; b0 += 64) {
    const uint64_t past = __ballot(b0 + lane < n && a.q_start[b0 + lane + 1] > token);
    if (past) return b0 + __builtin_ctzll(past);
  }
  return n - 1;
}

template <int D, int WAVES>
__global__ __launch_bounds__(256) void shared_join_kernel(ViewArgs a, qlinear_kv_cache c, SharedPlan p,
                                                          ViewPartials part) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t out = (int64_t)blockIdx.x * (4 / WAVES) + wave / WAVES;
  if (out >= part.rows) return;
  const int token = (int)(out / a.q_heads), h = (int)(out - (int64_t)token * a.q_heads);
  const int group = a.q_heads / c.kv_heads, head = h / group;
  Work w;
  sequence(a, c, a.groups + sequence_of(a, a.batch - a.groups, token), w);
  // A row of no sequence, or of one that is longer than the call said.
  if (token < w.q0 || token >= w.q0 + w.n || w.n > a.max_q_len) return;
  const Spans sp = p.few.workers > 0 ? few_spans(a, c, p.few, group) : Spans{};
  const Results own = results_of(a, c, p, part, sp, group, w, head, (token - w.q0) * group + h % group, out);
  Results shared = {0, 0, 0, 0};
  const int g = group_of(a, w.row);
  if (g >= 0) {
    sequence(a, c, g, w);
    if (token >= w.q0 && token < w.q0 + w.n)
      shared = results_of(a, c, p, part, sp, group, w, head, (token - w.q0) * group + h % group, out);
  }
  join_results<D, WAVES>(
      part, shared.parts + own.parts, [&](int i) { return i < shared.parts ? shared.at(i) : own.at(i - shared.parts); },
      a.out + out * D);
}

// The plan of a call with shared prefixes: one for the prefixes and the
// sequences together. `rows`: partial results in all.
struct SharedRoute {
  bool chunk;
  SharedPlan plan;
  ViewPartials part;
  int64_t rows;
};

// Row tiles of the chunk kernel: of the prefixes, and of the sequences if any may be that long.
int64_t shared_tiles(const ViewArgs& a, int64_t group, bool own) {
  auto tiles = [&](int64_t sequences) { return (a.tokens * group + (kChunkRows - 1) * sequences) / kChunkRows; };
  return tiles(a.groups) + (own ? tiles(a.batch - a.groups) : 0);
}

SharedRoute make_shared_route(const qlinear_kv_cache& c, const ViewArgs& a) {
  const int64_t group = a.q_heads / c.kv_heads, prefix = a.tokens * group, own = a.max_q_len * group;
  const int64_t most = prefix > own ? prefix : own;
  SharedRoute r = {};
  r.part.rows = (int64_t)a.tokens * a.q_heads;
  r.rows = 2 * r.part.rows;
  r.chunk = most > kFewRows;
  const int64_t cap = most < kFewRows ? most : kFewRows;
  Plan& f = r.plan.few;
  // Tiles for the sequences that the few-row kernel is known to serve; one group
  // of more rows than that leaves the others.
  const int64_t likely = a.groups == 1 && prefix > kFewRows && own <= kFewRows ? own : cap;
  f.rows = likely <= 16 || c.head_dim == 256 ? 16 : 32;
  f.once = likely <= f.rows;
  f.min_rows = 1;
  f.max_rows = kFewRows;
  f.tiles = (int)((cap + f.rows - 1) / f.rows);
  const int64_t steps = (a.max_kv_len + (int64_t)kStep - 1) / kStep;
  if (steps > kWholeSteps) {
    const int64_t tiles = (int64_t)f.tiles * a.batch;
    f.slots = few_slots(c, f.rows);
    f.workers = few_workers(c, f.rows, tiles, steps);
    if (tiles <= 2 * f.slots) f.whole = f.tiles;
  }
  Plan& p = r.plan.chunk;
  p.rows = kChunkRows;
  p.min_rows = kFewRows + 1;
  p.max_rows = INT32_MAX;
  p.splits = 1;
  p.chunk = INT32_MAX;
  r.part.chunk0 = r.rows;
  r.part.chunk_kinds = own > kFewRows ? 2 : 1;
  if (r.chunk) {
    p.tiles = (int)shared_tiles(a, group, own > kFewRows);
    const int64_t groups = (int64_t)p.tiles * c.kv_heads;
    const int64_t length = own > kFewRows && a.max_kv_len > a.max_shared_len ? a.max_kv_len : a.max_shared_len;
    const int64_t chunk_steps = (length + chunk_step(c.head_dim) - 1) / chunk_step(c.head_dim);
    int64_t splits = 512 / groups;
    if (splits > chunk_steps / 8) splits = chunk_steps / 8;
    if (splits > 1) {
      p.chunk = (int)((chunk_steps + splits - 1) / splits);
      p.splits = (int)((chunk_steps + p.chunk - 1) / p.chunk);
      if (p.splits > 1) r.rows += (int64_t)p.splits * r.part.chunk_kinds * r.part.rows;
    }
  }
  r.part.few0 = r.rows;
  if (f.workers > 0) r.rows += few_partial_rows(c, f.rows, f.workers);
  return r;
}

}  // namespace

size_t sinks_attention_workspace_need(const qlinear_kv_cache& cache, const ViewArgs& a) {
  return workspace_need(cache, a);
}
size_t sinks_attention_workspace_bytes(const qlinear_kv_cache& cache, const ViewArgs& a) {
  return workspace_bytes(cache, a);
}
hipError_t launch_sinks_attention(const qlinear_kv_cache& cache, const ViewArgs& a, void* ws, hipStream_t stream) {
  return launch_attention<ViewPartials>(cache, a, ws, few_launcher, chunk_launcher, stream);
}

size_t shared_attention_workspace_need(const qlinear_kv_cache& cache, const ViewArgs& a) {
  return partial_bytes(1, make_shared_route(cache, a).rows, cache.head_dim);
}

// Enough for all smaller calls too: each part of the workspace at its most.
size_t shared_attention_workspace_bytes(const qlinear_kv_cache& c, const ViewArgs& a) {
  const int64_t group = a.q_heads / c.kv_heads, prefix = a.tokens * group, own = a.max_q_len * group;
  const int64_t most = prefix > own ? prefix : own, cap = most < kFewRows ? most : kFewRows;
  const int64_t rows = (int64_t)a.tokens * a.q_heads;
  int64_t few = 0, chunk = 0;
  const int64_t steps = (a.max_kv_len + (int64_t)kStep - 1) / kStep;
  if (steps > kWholeSteps)
    for (int tile : {16, 32}) {
      if (tile == 32 && (c.head_dim == 256 || cap <= 16)) continue;
      // A call of few rows may have tiles of 16 where this one has 32.
      const int64_t n = few_partial_rows(c, tile, few_workers(c, tile, (cap + tile - 1) / tile * a.batch, steps));
      if (n > few) few = n;
    }
  const int64_t length = a.max_kv_len > a.max_shared_len ? a.max_kv_len : a.max_shared_len;
  const int64_t ranges = (length + chunk_step(c.head_dim) - 1) / chunk_step(c.head_dim) / 8;
  if (most > kFewRows && ranges > 1 && 512 / c.kv_heads > 1) {
    // Ranges times tiles times heads are 512 at most, of kChunkRows rows each.
    const int64_t all = ranges * rows;
    chunk = (all < 512 * kChunkRows ? all : 512 * kChunkRows) * (own > kFewRows ? 2 : 1);
  }
  return partial_bytes(1, 2 * rows + chunk + few, c.head_dim);
}

hipError_t launch_shared_attention(const qlinear_kv_cache& cache, const ViewArgs& a, void* ws, hipStream_t stream) {
  const int D = cache.head_dim;
  SharedRoute r = make_shared_route(cache, a);
  r.part.o = (float*)ws;
  r.part.ml = (float2*)(r.part.o + r.rows * D);
  if (r.chunk) {
    const hipError_t e = chunk_launcher(D)(cache, a, r.plan.chunk, r.part, stream);
    if (e != hipSuccess) return e;
  }
  const hipError_t e = few_launcher(D)(cache, a, r.plan.few, r.part, stream);
  if (e != hipSuccess) return e;
  auto go = [&](auto kernel, int waves) {
    const unsigned grid = (unsigned)((r.part.rows * waves + 3) / 4);
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), 0, stream, a, cache, r.plan, r.part);
    return hipGetLastError();
  };
  auto width = [&](auto waves) {
    constexpr int W = decltype(waves)::value;
    if (D == 64) return go(shared_join_kernel<64, W>, W);
    if (D == 128) return go(shared_join_kernel<128, W>, W);
    return go(shared_join_kernel<256, W>, W);
  };
  // Four waves to a row if one would make several turns.
  const int64_t parts = r.plan.chunk.splits + r.plan.few.workers / a.batch;
  return parts > kJoinAtOnce && r.part.rows <= 1 << 20 ? width(std::integral_constant<int, 4>{})
                                                       : width(std::integral_constant<int, 1>{});
}

}  // namespace qlinear
