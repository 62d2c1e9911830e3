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
// sequence, of one that is longer than the call said, of no shared prefix; with
// sinks, of the few-row kernel's.
__device__ __forceinline__ bool has_results(const ViewArgs& a, const qlinear_kv_cache& c, int b, int token) {
  Work w;
  sequence(a, c, b, w);
  return token >= w.q0 && token < w.q0 + w.n && (w.all || w.n <= a.max_q_len) &&
         (a.groups > 0 || (int64_t)w.n * (a.q_heads / c.kv_heads) <= kFewRows);
}

constexpr int kJoinRows = 16;      // of a wave, at most
// Joins the results of the rows of the output: a wave takes `rows` rows, and finds
// which sequence they are of once for the heads of a token. Most rows have two
// results, which take no more than their loads. (Four waves to a row lost: 2048
// rows of 33 results 12.9 us and 9.7 so, 7680 of 10 28 and 12.5; 128 rows of 64
// take 7.6.)
template <int D>
__global__ __launch_bounds__(256) void view_join_kernel(ViewArgs a, qlinear_kv_cache c, ViewPartials part, int rows,
                                                        int most, unsigned last) {
  constexpr int kOwn = D / 64;      // elements of a lane
  typedef float own_t __attribute__((ext_vector_type(kOwn)));
  typedef _Float16 half_t __attribute__((ext_vector_type(kOwn)));
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t first = ((int64_t)blockIdx.x * 4 + wave) * rows;
  const own_t* os = reinterpret_cast<const own_t*>(part.o) + lane;
  int token = -1;
  bool own = false, shared = false;
  // Where the results are: row first + i's in lane i.
  int4 found[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) found[k] = part.found[k * part.own0 + min(first + lane % kJoinRows, part.rows - 1)];
  auto of_row = [&](int4 x, int i) {
    return make_int4(__builtin_amdgcn_readlane(x.x, i), __builtin_amdgcn_readlane(x.y, i),
                     __builtin_amdgcn_readlane(x.z, i), __builtin_amdgcn_readlane(x.w, i));
  };
  for (int64_t out = first; out < first + rows && out < part.rows; ++out) {
    const int t = (int)(out / a.q_heads);
    if (t != token) {
      token = t;
      const int s = sequence_of(a, a.batch - a.groups, t), g = a.groups > 0 ? group_of(a, s) : -1;
      own = has_results(a, c, a.groups + s, t);
      shared = g >= 0 && has_results(a, c, g, t);
    }
    if (!own) continue;
    // Groups that overlap may have more tiles than the launch: then nobody wrote
    // these, and what they say stays in bounds.
    int4 y = of_row(found[0], (int)(out - first)), x = of_row(found[1], (int)(out - first));
    y.x = shared ? min(max(y.x, 0), most) : 0;
    x.x = min(max(x.x, 1), most);
    if (a.groups == 0 && x.x == 1) continue;      // it stands in the output
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
    auto turn = [&](auto count, int i0) {
      constexpr int N = decltype(count)::value;
      float2 ml[N];
      own_t v[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int64_t r = at(min(i0 + i, n - 1));
        ml[i] = part.ml[r];
        v[i] = os[r * 64];
      }
      float most = top;
#pragma unroll
      for (int i = 0; i < N; ++i) most = fmaxf(most, i0 + i < n ? ml[i].x : -INFINITY);
      const float keep = top == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(top - most);
      total *= keep;
      o *= keep;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (i0 + i >= n || ml[i].x == -INFINITY) continue;
        const float f = __builtin_amdgcn_exp2f(ml[i].x - most);
        total += f * ml[i].y;
        o += f * v[i];
      }
      top = most;
    };
    if (n <= 2) {
      turn(std::integral_constant<int, 2>{}, 0);
    } else {
      for (int i0 = 0; i0 < n; i0 += kTurn) turn(std::integral_constant<int, kTurn>{}, i0);
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
  bool long_rows;
  Plan few, chunk;
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
  r.part.rows = r.part.own0 = (int64_t)a.tokens * a.q_heads;
  r.rows = 2 * r.part.rows;
  r.long_rows = most > kFewRows;
  const int64_t cap = most < kFewRows ? most : kFewRows;
  Plan& f = r.few;
  // Tiles for the prefixes, which are the longer ones, if the few-row kernel likely
  // has them. Else two of 16 rows do better than one of 32 on own tokens, of which
  // there are few (20 sequences of 77 own tokens, 4 of them new, 64/8 heads, us:
  // float16 10 and 11.4, Q8 10.4 and 14.9; 30 of 4 to 900, Q8: 17.0 and 19.4).
  const int64_t group_rows = prefix / a.groups, own_rows = prefix / (a.batch - a.groups);
  const bool prefixes = group_rows <= kFewRows;
  const int64_t likely = likely_rows(cap, prefixes ? group_rows : own_rows);
  f.rows = !prefixes || likely <= 16 || c.head_dim == 256 ? 16 : 32;
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
  Plan& p = r.chunk;
  p.rows = kChunkRows;
  p.min_rows = kFewRows + 1;
  p.max_rows = INT32_MAX;
  p.splits = 1;
  p.chunk = INT32_MAX;
  r.part.chunk0 = r.rows;
  if (r.long_rows) {
    // Tiles are cut, on the device, where there are fewer than the chip holds: the
    // parts are no more than that.
    const int tiles = (int)shared_tiles(a, group, own > kFewRows);
    p.slots = chunk_slots(c);
    p.tiles = tiles > p.slots ? tiles : p.slots;
    r.rows += (int64_t)p.slots * c.kv_heads * kChunkRows;
  }
  r.part.few0 = r.rows;
  if (f.workers > 0) r.rows += few_partial_rows(c, f.rows, f.workers);
  return r;
}

}  // namespace

// As many rows to a wave as leave the chip eight waves a CU and more.
hipError_t attn::launch_view_join(const qlinear_kv_cache& c, const ViewArgs& a, const ViewPartials& part, int64_t total,
                                  int most, hipStream_t stream) {
  int rows = 1;
  static_assert(kJoinRows <= 64, "a lane for each");
  while (rows < kJoinRows && part.rows / (2 * rows) >= 4096) rows *= 2;
  const int64_t waves = (part.rows + rows - 1) / rows;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, stream, a, c, part, rows,
                       most > 1 ? most : 1, (unsigned)(total - 1));
    return hipGetLastError();
  };
  return c.head_dim == 64 ? go(view_join_kernel<64>) : c.head_dim == 128 ? go(view_join_kernel<128>)
                                                                         : go(view_join_kernel<256>);
}

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
  return partial_bytes(1, r.rows, cache.head_dim) + found_bytes(a);
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
  if (most > kFewRows) chunk = (int64_t)chunk_slots(c) * c.kv_heads * kChunkRows;
  return partial_bytes(1, 2 * rows + chunk + few, c.head_dim) + found_bytes(a);
}

hipError_t launch_shared_attention(const qlinear_kv_cache& cache, const ViewArgs& a, void* ws, hipStream_t stream) {
  const int D = cache.head_dim;
  SharedRoute r = make_shared_route(cache, a);
  r.part.o = (float*)ws;
  r.part.found = (int4*)(r.part.o + r.rows * D);
  r.part.ml = (float2*)(r.part.found + 2 * r.part.rows);
  if (r.long_rows) {
    const hipError_t e = chunk_launcher(D)(cache, a, r.chunk, r.part, stream);
    if (e != hipSuccess) return e;
  }
  const hipError_t e = few_launcher(D)(cache, a, r.few, r.part, stream);
  if (e != hipSuccess) return e;
  const int most = r.chunk.slots > r.few.workers ? r.chunk.slots : r.few.workers;
  return launch_view_join(cache, a, r.part, r.rows, most, stream);
}

}  // namespace qlinear
