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

struct SharedPlan {
  Plan few, chunk;
};

// Sequence of row `token` of q, 0 .. n - 1; all lanes together.
__device__ __forceinline__ int sequence_of(const ViewArgs& a, int n, int token) {
  if (!a.q_start) return min(token / (a.tokens / n), n - 1);
  const int lane = threadIdx.x & 63;
  for (int b0 = 0; b0 < n; b0 += 64) {
    const uint64_t past = __ballot(b0 + lane < n && number(a.q_start, min(b0 + lane, n - 1) + 1) > token);
    if (past) return b0 + __builtin_ctzll(past);
  }
  return n - 1;
}

// Whether row `token` has results of (virtual) sequence b: not one of no
// sequence, of one that is longer than the call said, of no shared prefix.
__device__ __forceinline__ bool has_results(const ViewArgs& a, const qlinear_kv_cache& c, int b, int token) {
  Work w;
  sequence(a, c, b, w);
  return token >= w.q0 && token < w.q0 + w.n && (w.all || w.n <= a.max_q_len);
}

constexpr int kJoinRows = 16;      // of a wave, at most
// Joins the results of the rows of the output. WAVES == 1: a wave takes `rows`
// rows, and finds where their results are once for the heads of a token; most
// have two, which take no more than their loads. WAVES == 4: four waves to a row
// share its many results out.
template <int D, int WAVES>
__global__ __launch_bounds__(256) void shared_join_kernel(ViewArgs a, qlinear_kv_cache c, ViewPartials part, int rows,
                                                          int most, unsigned last) {
  constexpr int kOwn = D / 64;      // elements of a lane
  typedef float own_t __attribute__((ext_vector_type(kOwn)));
  typedef _Float16 half_t __attribute__((ext_vector_type(kOwn)));
  __shared__ own_t o_all[4][64];
  __shared__ float2 ml_all[4];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t first = ((int64_t)blockIdx.x * (4 / WAVES) + wave / WAVES) * rows;
  const own_t* os = reinterpret_cast<const own_t*>(part.o) + lane;
  int token = -1;
  bool own = false, shared = false;
  // Where the results are: row first + i's in lane i.
  int4 found[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) found[k] = part.found[k * part.rows + min(first + lane % kJoinRows, part.rows - 1)];
  auto of_row = [&](int4 x, int i) {
    return make_int4(__builtin_amdgcn_readlane(x.x, i), __builtin_amdgcn_readlane(x.y, i),
                     __builtin_amdgcn_readlane(x.z, i), __builtin_amdgcn_readlane(x.w, i));
  };
  for (int64_t out = first; out < first + rows && out < part.rows; ++out) {
    const int t = (int)(out / a.q_heads);
    if (t != token) {
      token = t;
      const int s = sequence_of(a, a.batch - a.groups, t), g = group_of(a, s);
      own = has_results(a, c, a.groups + s, t);
      shared = g >= 0 && has_results(a, c, g, t);
    }
    if (!own) continue;
    // Groups that overlap may have more tiles than the launch: then nobody wrote
    // these, and what they say stays in bounds.
    int4 y = of_row(found[0], (int)(out - first)), x = of_row(found[1], (int)(out - first));
    y.x = shared ? min(max(y.x, 0), most) : 0;
    x.x = min(max(x.x, 1), most);
    const int n = x.x + y.x;
    auto at = [&](int i) -> int64_t {
      const int j = i < y.x ? i : i - y.x;
      const unsigned row = i < y.x ? (j ? y.z + j * (unsigned)y.w : y.y) : (j ? x.z + j * (unsigned)x.w : x.y);
      return min(row, last);
    };
    // Results take turns of eight, whose loads do not wait for one another.
    constexpr int kTurn = 8;
    float top = -INFINITY, total = 0.0f;
    own_t o = 0.0f;
    const int each = (n + WAVES - 1) / WAVES, stop = min(n, (wave % WAVES + 1) * each);
    auto turn = [&](auto count, int i0) {
      constexpr int N = decltype(count)::value;
      float2 ml[N];
      own_t v[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int64_t r = at(min(i0 + i, stop - 1));
        ml[i] = part.ml[r];
        v[i] = os[r * 64];
      }
      float most = top;
#pragma unroll
      for (int i = 0; i < N; ++i) most = fmaxf(most, i0 + i < stop ? ml[i].x : -INFINITY);
      const float keep = top == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(top - most);
      total *= keep;
      o *= keep;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (i0 + i >= stop || ml[i].x == -INFINITY) continue;
        const float f = __builtin_amdgcn_exp2f(ml[i].x - most);
        total += f * ml[i].y;
        o += f * v[i];
      }
      top = most;
    };
    if (WAVES == 1 && n <= 2) {
      turn(std::integral_constant<int, 2>{}, 0);
    } else {
      for (int i0 = wave % WAVES * each; i0 < stop; i0 += kTurn) turn(std::integral_constant<int, kTurn>{}, i0);
    }
    if constexpr (WAVES > 1) {     // the whole workgroup is on one row
      o_all[wave][lane] = o;
      if (lane == 0) ml_all[wave] = make_float2(top, total);
      __syncthreads();
      if (wave == 0) {
        top = fmaxf(fmaxf(ml_all[0].x, ml_all[1].x), fmaxf(ml_all[2].x, ml_all[3].x));
        total = 0.0f;
        o = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (ml_all[i].x == -INFINITY) continue;
          const float f = __builtin_amdgcn_exp2f(ml_all[i].x - top);
          total += f * ml_all[i].y;
          o += f * o_all[i][lane];
        }
      }
      if (rows > 1) __syncthreads();
      if (wave != 0) continue;
    }
    half_t z;
#pragma unroll
    for (int e = 0; e < kOwn; ++e) z[e] = (_Float16)(top == -INFINITY ? 0.0f : o[e] / total);
    reinterpret_cast<half_t*>(a.out + out * D)[lane] = z;
  }
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

// Workgroups of a key/value head that the chip holds at once, two on a CU.
int chunk_slots(const qlinear_kv_cache& c) { return 512 / c.kv_heads > 1 ? 512 / c.kv_heads : 1; }

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
  if (r.chunk) {
    // Tiles are cut, on the device, where there are fewer than the chip holds.
    p.tiles = (int)shared_tiles(a, group, own > kFewRows);
    const int slots = chunk_slots(c);
    if (p.tiles < slots) {
      p.slots = p.tiles = slots;
      r.rows += (int64_t)p.tiles * c.kv_heads * kChunkRows;
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
  const SharedRoute r = make_shared_route(cache, a);
  return partial_bytes(1, r.rows, cache.head_dim) + 2 * r.part.rows * sizeof(int4);
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
  // (Fewer tiles may be cut where these are not.)
  if (most > kFewRows) chunk = (int64_t)chunk_slots(c) * c.kv_heads * kChunkRows;
  return partial_bytes(1, 2 * rows + chunk + few, c.head_dim) + 2 * rows * sizeof(int4);
}

hipError_t launch_shared_attention(const qlinear_kv_cache& cache, const ViewArgs& a, void* ws, hipStream_t stream) {
  const int D = cache.head_dim;
  SharedRoute r = make_shared_route(cache, a);
  r.part.o = (float*)ws;
  r.part.found = (int4*)(r.part.o + r.rows * D);
  r.part.ml = (float2*)(r.part.found + 2 * r.part.rows);
  if (r.chunk) {
    const hipError_t e = chunk_launcher(D)(cache, a, r.plan.chunk, r.part, stream);
    if (e != hipSuccess) return e;
  }
  const hipError_t e = few_launcher(D)(cache, a, r.plan.few, r.part, stream);
  if (e != hipSuccess) return e;
  // Four waves to a row if there may be many results; else as many rows to a wave
  // as leave the chip eight waves a CU and more.
  const int64_t parts = r.plan.chunk.slots + r.plan.few.workers / a.batch;
  const bool many = parts > 16 && r.part.rows <= 1 << 11;
  int rows = 1;
  static_assert(kJoinRows <= 64, "a lane for each");
  while (!many && rows < kJoinRows && r.part.rows / (2 * rows) >= 4096) rows *= 2;
  const int most = r.plan.chunk.slots > r.plan.few.workers ? r.plan.chunk.slots : r.plan.few.workers;
  const int64_t waves = (r.part.rows + rows - 1) / rows * (many ? 4 : 1);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, stream, a, cache, r.part, rows,
                       most > 1 ? most : 1, (unsigned)(r.rows - 1));
    return hipGetLastError();
  };
  if (D == 64) return many ? go(shared_join_kernel<64, 4>) : go(shared_join_kernel<64, 1>);
  if (D == 128) return many ? go(shared_join_kernel<128, 4>) : go(shared_join_kernel<128, 1>);
  return many ? go(shared_join_kernel<256, 4>) : go(shared_join_kernel<256, 1>);
}

}  // namespace qlinear
