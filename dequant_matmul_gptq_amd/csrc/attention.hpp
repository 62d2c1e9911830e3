// Attention of new tokens over a paged cache: what its kernels share. The
// mathematics, per query row r (a new token and a query head) over the tokens
// t it sees, in base 2 so that the exponential is one instruction:
//   x_t = scale log2(e) q.k_t;  m = max x_t;  l = sum 2^(x_t - m);
//   o = sum 2^(x_t - m) v_t / l
// built up over steps of tokens with the running m and l (o and l are
// multiplied by 2^(m_old - m_new) when m grows). Rows that see different
// parts of the cache, or parts of it handled by different workgroups, join
// the same way, in a fixed order.
//
// Both products run on the matrix cores in transposed form, S^T = K Q^T and
// O^T = V^T P^T. A lane of the accumulators then holds one query row: the
// softmax statistics are per-lane scalars, and the accumulator registers of
// S^T, rounded to float16, are the B operand of the second product as they
// stand, if its k index is counted in the order in which S^T's rows lie in
// the lanes. No weight crosses a lane.
//
// Views (ViewArgs): calls whose rows see other tokens than the last ones, by the
// same kernels in instances of their own.
//   Sinks: with a window, a sequence's first tokens are seen too. The steps
//   between them and the window are left out: a tile's steps are numbered
//   without them (Item::gap).
//   Shared prefixes: groups of sequences whose first tokens are the same cache
//   slots. A group's rows over its shared tokens, all of which they all see,
//   stand before the batch as a sequence of their own, and each sequence starts
//   after them; what both leave, float32, is joined as parts of a row are.
#pragma once

#include <type_traits>

#include "qlinear_kernels.hpp"

namespace qlinear {

// A call with sinks (groups == 0) or shared prefixes (groups > 0, no window, no
// sinks): batch is then groups + sequences.
struct ViewArgs : AttentionArgs {
  int sinks, groups;
  const int32_t *shared_start, *shared_len;      // shared_start NULL: one group of all
  int max_shared_len;                            // no plan asks for it: max_kv_len bounds the prefixes' steps too
};

// What a call takes of its workspace, and what is enough for it and for all
// smaller ones (attention_views.hip).
size_t sinks_attention_workspace_need(const qlinear_kv_cache& cache, const ViewArgs& a);
size_t sinks_attention_workspace_bytes(const qlinear_kv_cache& cache, const ViewArgs& a);
hipError_t launch_sinks_attention(const qlinear_kv_cache& cache, const ViewArgs& a, void* ws, hipStream_t stream);
size_t shared_attention_workspace_need(const qlinear_kv_cache& cache, const ViewArgs& a);
size_t shared_attention_workspace_bytes(const qlinear_kv_cache& cache, const ViewArgs& a);
hipError_t launch_shared_attention(const qlinear_kv_cache& cache, const ViewArgs& a, void* ws, hipStream_t stream);

namespace attn {

template <class Args>
constexpr bool kIsView = std::is_same_v<Args, ViewArgs>;

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef float float16v __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -3.4028234663852886e38f;

// A launch's plan. It serves the sequences whose rows per key/value head,
// (token, head of the group) pairs, number min_rows to max_rows, in tiles of
// `rows`.
//   Chunk kernel: each tile's visible tokens are cut into `splits` ranges of
//   `chunk` steps (the last range takes what is left).
//   Few-row kernel, workers == 0: a workgroup per tile. Else the tiles' steps
//   stand one after another, sequence by sequence, and each key/value head's
//   `workers` workgroups take equal spans of them (see Spans), or whole tiles
//   as well, if the launch has `whole` of them for each sequence (0: it has
//   not). `slots`: workgroups of a head that the chip holds at once.
struct Plan {
  int rows;
  int splits;
  int chunk;
  int workers, slots, whole;
  int min_rows, max_rows;
  // Views: tiles of a sequence (few-row kernel) or of all (chunk kernel) at most;
  // whether each row of the cache is read by one workgroup.
  int tiles;
  bool once;
};
constexpr int kStep = 32;          // tokens of a step, few-row kernel
constexpr int kChunkRows = 128;    // rows of a tile, chunk kernel
constexpr int kFewRows = 64;       // most rows of a sequence per key/value head in the few-row kernel
__host__ __device__ constexpr int chunk_step(int D) { return D == 256 ? 32 : 64; }   // tokens of its step

// Workgroups of the few-row kernel that a CU holds, by their registers: one of
// 256 wide heads or of 32 rows by 128, else two. With codes two of 32 by 128 are
// taken as well: they spill outside the loop of whole steps, and the unpacking
// wants the waves (8 sequences of 8192 tokens, 64/8 heads, 7 new tokens each, in
// us with one and two: float16 68 and 79, Q8 72 and 62, Q6 82 and 70, Q4 71 and
// 60; 4 new tokens: float16 53 and 70, Q8 44 and 49, Q6 50 and 51).
__host__ __device__ constexpr int few_per_cu(int head_dim, int rows, int bits) {
  return head_dim == 256 || (head_dim == 128 && rows == 32 && bits == 16) ? 1 : 2;
}

// Row tiles of the chunk kernel, at most, whatever the sequences' lengths.
inline int64_t chunk_tiles(const AttentionArgs& a, int group) {
  return ((int64_t)a.tokens * group + (kChunkRows - 1) * (int64_t)a.batch) / kChunkRows;
}

// Partial results, float32: o [.][rows][D] and (m, l) [.][rows]. Chunk kernel:
// [splits][rows of the output]. Few-row kernel: a worker's span starts and
// ends inside a tile, and what is between are whole tiles, so a worker has two
// partial results at most: [workers][kv_heads][2][plan.rows].
// Shared prefixes leave partial results where others write the output. All
// rows of those stand in one array: whole tiles [2][rows of the output] (0: of a
// prefix, 1: of a sequence's own tokens), the chunk kernel's ranges
// [items][kv_heads][kChunkRows] from row chunk0 on, the few-row kernel's from few0
// on. rows: of the output. found [2][rows] says where each row has its results of
// either kind: x of them, the first in row y, result i > 0 in row z + i w. The
// workgroup that has the first one writes it, so that the join need not look
// through the lengths again. Kind 1 starts at row own0; with sinks there is no
// other, and what is whole stands in the output.
struct Partials {
  float* o;
  float2* ml;
  int64_t rows;
};
struct ViewPartials : Partials {
  int64_t own0, chunk0, few0;
  int4* found;
};

// The kernels' loops come in kinds of step: whole ones that all rows see all
// of (kGrow: with the accumulators rescaled), edge ones with masks, and, where
// an edge step holds infinities or NaN (rare), the whole range again with
// careful steps. Kept apart so that the common loops hold no registers for the
// rare ones.
enum StepKind { kWhole, kGrow, kEdgeStep, kCareful };

// One workgroup's sequence, row tile and token range.
struct Work {
  int b;             // sequence
  int q0, n;         // first row of q, new tokens
  int len;           // cached tokens
  int row0, rows;    // first row of the tile among n * group, rows in it
  int p_min, p_max;  // positions of the tile's first and last token
  int lo_min, lo_max;  // first tokens they see
  // Views only:
  int row;           // of the block table
  int low;           // tokens below it are a shared prefix's
  bool all;          // all rows see all tokens: a shared prefix
};

// A sequence's length as its table bounds it, and so far below 2^31 that the
// tokens whose pages are looked up ahead have numbers too (kLookAhead past the
// last one at most: a step of 64, and the two after it).
constexpr int kLookAhead = 256;
constexpr int kMaxLength = INT32_MAX - 1023;
static_assert(kMaxLength <= INT32_MAX - kLookAhead);
__host__ __device__ __forceinline__ int bounded_length(int kv_len, int table_width, int page_size) {
  const int64_t len = max(kv_len, 0), cap = (int64_t)table_width * page_size;
  return min((int)(len < cap ? len : cap), kMaxLength);
}

// Rows q0 .. q1 - 1 of q, as far as there are such.
__host__ __device__ __forceinline__ void bounded_rows(int q0, int q1, int tokens, Work& w) {
  w.q0 = q0 > 0 ? q0 : 0;
  const int end = q1 < tokens ? q1 : tokens;
  w.n = end > w.q0 ? end - w.q0 : 0;
}

// Number i of an array that no launch writes: through the scalar cache where i
// is uniform.
__host__ __device__ __forceinline__ int number(const int32_t* p, int i) {
#ifdef __HIP_DEVICE_COMPILE__
  return ((const __attribute__((address_space(4))) int32_t*)(uintptr_t)p)[i];
#else
  return p[i];
#endif
}

// First row of sequence s of n (s == n: the row after the last).
__host__ __device__ __forceinline__ int first_row(const ViewArgs& a, int n, int s) {
  return a.q_start ? number(a.q_start, s) : s * (a.tokens / n);
}

// The group of sequence s, -1 if none.
__host__ __device__ __forceinline__ int group_of(const ViewArgs& a, int s) {
  if (!a.shared_start) return 0;
  int lo = 0, hi = a.groups;       // the last one that starts at s or before
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (number(a.shared_start, mid) <= s)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo > 0 && s < number(a.shared_start, lo) ? lo - 1 : -1;
}

// Sequence b's rows and length, bounded by what the buffers hold. With shared
// prefixes those come first (batch counts both), and the last step of it finds
// where own tokens start.
__host__ __device__ __forceinline__ void sequence_rows(const ViewArgs& a, const qlinear_kv_cache& c, int b, Work& w) {
  const int sequences = a.batch - a.groups;
  w.b = b;
  w.all = b < a.groups;
  w.low = 0;
  if (w.all) {
    const int s0 = a.shared_start ? min(max(number(a.shared_start, b), 0), sequences) : 0;
    const int s1 = a.shared_start ? min(number(a.shared_start, b + 1), sequences) : sequences;
    bounded_rows(first_row(a, sequences, s0), first_row(a, sequences, max(s0, s1)), a.tokens, w);
    w.len = bounded_length(number(a.shared_len, b), a.table_width, c.page_size);
    w.row = min(s0, sequences - 1);
    if (w.len == 0) w.n = 0;
    return;
  }
  w.row = b - a.groups;
  bounded_rows(first_row(a, sequences, w.row), first_row(a, sequences, w.row + 1), a.tokens, w);
  w.len = bounded_length(number(a.kv_len, w.row), a.table_width, c.page_size);
}
__host__ __device__ __forceinline__ void sequence_low(const ViewArgs& a, const qlinear_kv_cache& c, Work& w) {
  if (a.groups == 0 || w.all) return;
  const int g = group_of(a, w.row);
  if (g >= 0) w.low = bounded_length(number(a.shared_len, g), a.table_width, c.page_size);
}
__host__ __device__ __forceinline__ void sequence(const ViewArgs& a, const qlinear_kv_cache& c, int b, Work& w) {
  sequence_rows(a, c, b, w);
  sequence_low(a, c, w);
}
__device__ __forceinline__ void sequence(const AttentionArgs& a, const qlinear_kv_cache& c, int b, Work& w) {
  w.b = b;
  w.row = b;
  w.low = 0;
  w.all = false;
  if (a.q_start) {
    bounded_rows(a.q_start[b], a.q_start[b + 1], a.tokens, w);
  } else {
    w.n = a.tokens / a.batch;
    w.q0 = b * w.n;
  }
  w.len = bounded_length(a.kv_len[b], a.table_width, c.page_size);
}

__host__ __device__ __forceinline__ int first_seen(int p, int window) {
  // Below -1 all p see nothing; their differences to the largest windows would not fit.
  return window > 0 ? max(0, max(p, -1) - window + 1) : 0;
}

// The last token that new token `tok` of a sequence sees, and the first one
// (but for sinks) that a row with this last one does.
__host__ __device__ __forceinline__ int position(const AttentionArgs&, const Work& w, int tok) {
  return w.len - w.n + tok;
}
__host__ __device__ __forceinline__ int position(const ViewArgs&, const Work& w, int tok) {
  return w.all ? w.len - 1 : w.len - w.n + tok;
}
__host__ __device__ __forceinline__ int first_of(const AttentionArgs& a, const Work&, int p) {
  return first_seen(p, a.window);
}
__host__ __device__ __forceinline__ int first_of(const ViewArgs& a, const Work& w, int p) {
  return w.all ? 0 : max(w.low, first_seen(p, a.window));
}
// Whether a row that sees first .. p does not see token t.
__host__ __device__ __forceinline__ bool hidden(const AttentionArgs&, int t, int first, int p) {
  return t > p || t < first;
}
__host__ __device__ __forceinline__ bool hidden(const ViewArgs& a, int t, int first, int p) {
  return t > p || (t < first && t >= a.sinks);
}

// The tile of `tile_rows` rows from row0 on (group rows per token).
template <class Args>
__host__ __device__ __forceinline__ void row_tile(const Args& a, int group, int row0, int tile_rows, Work& w) {
  w.row0 = row0;
  w.rows = min(tile_rows, w.n * group - row0);
  w.p_min = position(a, w, row0 / group);
  w.p_max = position(a, w, (row0 + w.rows - 1) / group);
  w.lo_min = first_of(a, w, w.p_min);
  w.lo_max = first_of(a, w, w.p_max);
}

// Steps before a tile's window that hold sinks, if its window starts in step
// `first`, in steps of 2^shift tokens.
__host__ __device__ __forceinline__ int sink_steps(const AttentionArgs&, int, int) { return 0; }
__host__ __device__ __forceinline__ int sink_steps(const ViewArgs& a, int first, int shift) {
  return min((a.sinks >> shift) + ((a.sinks & ((1 << shift) - 1)) != 0), first);
}

// A sequence's page numbers, through the scalar cache where the place is
// uniform (the table is not written during a launch).
typedef const __attribute__((address_space(4))) int32_t* PageTable;
__device__ __forceinline__ PageTable page_table(const AttentionArgs& a, const Work& w) {
  return (PageTable)(uintptr_t)(a.block_table + (int64_t)w.b * a.table_width);
}
__device__ __forceinline__ PageTable page_table(const ViewArgs& a, const Work& w) {
  return (PageTable)(uintptr_t)(a.block_table + (int64_t)w.row * a.table_width);
}

// The page of token t: numbers are taken into the pool, table places to the
// sequence's last.
__device__ __forceinline__ int page_of(const qlinear_kv_cache& c, PageTable table, int page_shift, int last_page,
                                       int t) {
  return min(max(table[min(t >> page_shift, last_page)], 0), c.num_pages - 1);
}
// The pool row of token t in that page.
__device__ __forceinline__ int64_t pool_row(const qlinear_kv_cache& c, int page, int page_shift, int head, int t) {
  return (((int64_t)page * c.kv_heads + head) << page_shift) + (t & (c.page_size - 1));
}

// The sequence and row tile of tile number y, counting the tiles of the
// sequences of at least min_rows rows, found by all lanes together. False if
// there are fewer.
template <class Args>
__device__ __forceinline__ bool find_tile(const Args& a, const qlinear_kv_cache& c, const Plan& plan, int group, int y,
                                          Work& w, int& tile) {
  if (!kIsView<Args> && (!a.q_start || a.batch == 1)) {
    sequence(a, c, 0, w);
    const int per = (int)(((int64_t)w.n * group + kChunkRows - 1) / kChunkRows);
    if (per == 0 || (int64_t)w.n * group < plan.min_rows) return false;
    const int b = y / per;
    if (b >= a.batch) return false;
    sequence(a, c, b, w);
    tile = y - b * per;
    return true;
  }
  const int lane = threadIdx.x & 63;
  for (int b0 = 0; b0 < a.batch; b0 += 64) {
    int n = 0;
    if (b0 + lane < a.batch) {
      Work t;
      sequence(a, c, b0 + lane, t);
      const int64_t rows = (int64_t)t.n * group;
      n = rows < plan.min_rows ? 0 : (int)((rows + kChunkRows - 1) / kChunkRows);
    }
    int upto = n;
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) {
      const int o = __shfl_up(upto, k);
      if (lane >= k) upto += o;
    }
    const uint64_t past = __ballot(upto > y);
    if (past) {
      const int at = __builtin_ctzll(past);
      tile = y - __builtin_amdgcn_readlane(upto - n, at);
      sequence(a, c, b0 + at, w);
      return true;
    }
    y -= __builtin_amdgcn_readlane(upto, 63);
  }
  return false;
}

// ---- the chunk kernel's items with shared prefixes: a tile's steps in ranges of
// `chunk`, such that the chip is filled by what the lengths on the device are,
// and one round of workgroups takes them all (three groups of 8192, 4096 and 640
// tokens over Q8, 640, 288 and 32 rows a key/value head: 95 us with as many
// ranges for all tiles as the longest may have, 116 us with 66 items of 13 steps
// for 64 places, 81 us so; 50 us since that kernel spills nothing).
struct Ranges {
  int chunk;
  __device__ __forceinline__ int of(int steps) const { return steps <= chunk ? 1 : (steps + chunk - 1) / chunk; }
};
__device__ __forceinline__ int wave_total(int x) {
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) x += __shfl_xor(x, k);
  return __builtin_amdgcn_readfirstlane(x);
}
// Tiles, and each one's steps at most, of the lane's sequence of the 64 from b0
// on; none if it is not the chunk kernel's.
struct Tiles {
  int n, steps;
};
__device__ __forceinline__ Tiles chunk_tiles_of(const ViewArgs& a, const qlinear_kv_cache& c, const Plan& plan,
                                                int group, int shift, int b0) {
  const int b = b0 + (threadIdx.x & 63);
  Tiles t = {0, 1};
  if (b < a.batch) {
    Work w;
    sequence_rows(a, c, b, w);
    const int64_t rows = (int64_t)w.n * group;
    if (rows >= plan.min_rows) {
      sequence_low(a, c, w);
      t.n = (int)((rows + kChunkRows - 1) / kChunkRows);
      t.steps = max(((w.len - 1) >> shift) - (first_of(a, w, position(a, w, 0)) >> shift), 0) + 1;
      t.steps = min(t.steps, 1 << 22);     // 512 tiles' sum fits; a last range has the rest
    }
  }
  return t;
}
// t0: of the first 64 sequences, here and below.
__device__ __forceinline__ Ranges chunk_ranges(const ViewArgs& a, const qlinear_kv_cache& c, const Plan& plan,
                                               int group, int shift, const Tiles& t0) {
  int tiles = t0.n;
  unsigned total = t0.n * t0.steps;
  for (int b0 = 64; b0 < a.batch; b0 += 64) {
    const Tiles t = chunk_tiles_of(a, c, plan, group, shift, b0);
    tiles += t.n;
    total += t.n * t.steps;
  }
  tiles = wave_total(tiles);
  if (tiles >= plan.slots) return {INT32_MAX};
  total = wave_total(total);
  // Four steps at least (32 sequences behind 512 and 4096 tokens, 64/8 heads, us:
  // two 25.2 and 37.4, four 28.2 and 33.0, eight 33.0 and 37.0).
  Ranges ranges = {max(4, (int)((total + plan.slots - 1) / plan.slots))};
  int items = t0.n * ranges.of(t0.steps);
  for (int b0 = 64; b0 < a.batch; b0 += 64) {
    const Tiles t = chunk_tiles_of(a, c, plan, group, shift, b0);
    items += t.n * ranges.of(t.steps);
  }
  // Every tile's last range may be a short one.
  const int free = plan.slots - tiles;
  if (wave_total(items) > plan.slots) ranges.chunk = (int)((total + free - 1) / free);
  return ranges;
}
// Item y's sequence, tile, range and number of ranges, found by all lanes
// together. False if there are fewer.
__device__ __forceinline__ bool find_item(const ViewArgs& a, const qlinear_kv_cache& c, const Plan& plan, int group,
                                          int shift, const Tiles& t0, const Ranges& ranges, int y, Work& w, int& tile,
                                          int& split, int& splits) {
  Tiles t = t0;
  for (int b0 = 0;;) {
    const int each = ranges.of(t.steps), n = t.n * each;
    int upto = n;
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) {
      const int o = __shfl_up(upto, k);
      if ((int)(threadIdx.x & 63) >= k) upto += o;
    }
    const uint64_t past = __ballot(upto > y);
    if (past) {
      const int at = __builtin_ctzll(past);
      y -= __builtin_amdgcn_readlane(upto - n, at);
      splits = __builtin_amdgcn_readlane(each, at);
      tile = __builtin_amdgcn_readfirstlane(y / splits);
      split = y - tile * splits;
      sequence(a, c, b0 + at, w);
      return true;
    }
    y -= __builtin_amdgcn_readlane(upto, 63);
    b0 += 64;
    if (b0 >= a.batch) return false;
    t = chunk_tiles_of(a, c, plan, group, shift, b0);
  }
}

// ---- the few-row kernel's spans
// A sequence's row tiles, and the steps counted for each (from the first token
// that its first new token sees; 1 where none sees any, for the zeros).
// Views number the steps that their rows may see from 0 on: `sinks` steps of
// sinks, then from first_step on, which is `gap` further than its number. They
// count whole turns of a workgroup's waves, which cost what they cost however
// many of the waves have a step: else a span takes many short sequences, one
// after another (30 of 4 to 900 tokens behind three prefixes, 4 new ones each,
// 64/8 heads, Q8: 39 us with single steps, 18.5 us so).
struct Item {
  int tiles, steps, first_step;
  int sinks, gap;
  __host__ __device__ __forceinline__ int real(int step) const { return step < sinks ? step : step + gap; }
};
template <class Args>
__host__ __device__ __forceinline__ Item few_item(const Args& a, const Plan& plan, int group, const Work& w) {
  const int rows = w.n * group;
  Item it;
  it.tiles = rows > plan.max_rows ? 0 : (rows + plan.rows - 1) >> __builtin_ctz(plan.rows);
  it.first_step = first_of(a, w, position(a, w, 0)) / kStep;
  it.sinks = sink_steps(a, it.first_step, 5);
  it.gap = it.first_step - it.sinks;
  it.steps = it.sinks + max((w.len - 1) / kStep - it.first_step, 0) + 1;
  if constexpr (kIsView<Args>) it.steps = (it.steps + 3) & ~3;      // whole turns, see Item
  return it;
}
static_assert(kStep == 1 << 5);
// Steps of the 64 sequences from b0 on, one per lane, with their running sum.
// (The entry point bounds the slots of all tables, so that the sums fit.)
struct Costs {
  int own, upto;
  int q0, n, len, tiles, steps;     // the lane's sequence, each of its tiles' steps
  int row, low, all;
  // Sequence b, from the lane that holds it.
  __device__ __forceinline__ void get(int b, Work& w) const {
    w.b = b;
    w.q0 = __builtin_amdgcn_readlane(q0, b & 63);
    w.n = __builtin_amdgcn_readlane(n, b & 63);
    w.len = __builtin_amdgcn_readlane(len, b & 63);
    w.row = __builtin_amdgcn_readlane(row, b & 63);
    w.low = __builtin_amdgcn_readlane(low, b & 63);
    w.all = __builtin_amdgcn_readlane(all, b & 63);
  }
  __device__ __forceinline__ void set(const Work& w, const Item& it) {
    q0 = w.q0;
    n = w.n;
    len = w.len;
    row = w.row;
    low = w.low;
    all = w.all;
    tiles = it.tiles;
    steps = it.tiles > 0 ? it.steps : 0;
    own = upto = it.tiles * it.steps;
  }
};
template <class Args>
__device__ __forceinline__ Costs few_costs(const Args& a, const qlinear_kv_cache& c, const Plan& plan,
                                           int group, int b0) {
  const int lane = threadIdx.x & 63;
  Costs k = {};
  if (b0 + lane < a.batch) {
    Work w;
    sequence(a, c, b0 + lane, w);
    k.set(w, few_item(a, plan, group, w));
  }
#pragma unroll
  for (int n = 1; n < 64; n <<= 1) {
    const int o = __shfl_up(k.upto, n);
    if (lane >= n) k.upto += o;
  }
  return k;
}
// The steps of all sequences, and each worker's: whole turns of its four
// waves, one at least. costs: of the first 64.
//
// whole: every workgroup takes one tile, and nothing is joined. A span that
// cuts tiles pays for its second start and the join, about as much as 13 steps
// of a lone workgroup; a whole tile's workgroup pays by being the last one. A
// full chip's step takes about 1.25 times a lone workgroup's for each one that
// a CU holds, a partly full one's less in proportion. So tiles are taken whole
// if the longest, at the load of all of them, is done within 13 lone steps of
// what the spans take. Both sides measured, us, spans and whole, 64/8 heads of
// 128: float16: 16 sequences of 700 tokens 22.1 and 19.6, of 2100 36.1 and 40.9;
// 64 of 1100 59.9 and 52.9; 48 of 1 to 4000 73.3 and 114; Q4: 64 of 1100 38.3 and
// 28.8, of 2100 54.8 and 45.6, 128 of 1100 66.9 and 56.8, of 700 42.0 and 44.6.
//
// Every workgroup, and every one of the join, goes over all sequences for this,
// 64 at a time: work that grows with the square of the batch. Single tokens over
// 600 cached ones, 64/8 heads of 128, float16, us (and the cache's bytes at a
// large copy's rate): 512 sequences 266 (245), 1024 594 (489), 2048 1417 (979);
// 8/1 heads: 1024 101 (61), 16384 4933 (979). Batches past a thousand sequences
// are better cut by the caller.
struct Spans {
  Costs costs;
  int total, quota, tiles;
  bool whole;
};
__device__ __forceinline__ int few_tiles(const Costs& k) {
  static_assert(kFewRows <= 4 * 16, "four tiles of a sequence at most");
  int tiles = 0;
#pragma unroll
  for (int n = 0; n < 4; ++n) tiles += __builtin_popcountll(__ballot(k.tiles > n));
  return tiles;
}
template <class Args>
__device__ __forceinline__ Spans few_spans(const Args& a, const qlinear_kv_cache& c, const Plan& plan,
                                           int group) {
  Spans s;
  if (a.batch == 1) {      // no lane work on the way to the first load
    Work w;
    sequence(a, c, 0, w);
    s.costs.set(w, few_item(a, plan, group, w));
    s.total = __builtin_amdgcn_readfirstlane(s.costs.upto);
    s.tiles = __builtin_amdgcn_readfirstlane(s.costs.tiles);
  } else {
    s.costs = few_costs(a, c, plan, group, 0);
    s.total = __builtin_amdgcn_readlane(s.costs.upto, 63);
    s.tiles = few_tiles(s.costs);
  }
  for (int b0 = 64; b0 < a.batch; b0 += 64) {
    const Costs k = few_costs(a, c, plan, group, b0);
    s.total += __builtin_amdgcn_readlane(k.upto, 63);
    s.tiles += few_tiles(k);
  }
  s.quota = (int)((((unsigned)s.total + plan.workers - 1) / (unsigned)plan.workers + 3) & ~3u);
  if (plan.whole > 0) {
    // In a lone workgroup's steps; full: what one is worth on a full chip.
    const float full = 1.25f * (float)few_per_cu(c.head_dim, plan.rows, c.bits) / (float)plan.slots;
    const float spans = fmaxf((float)s.quota, full * (float)s.total) + 13.0f;
    const int most = (int)(spans / fmaxf(1.0f, full * (float)s.tiles));
    s.whole = !__any(s.costs.steps > most);
    for (int b0 = 64; b0 < a.batch && s.whole; b0 += 64) s.whole = !__any(few_costs(a, c, plan, group, b0).steps > most);
  } else {
    s.whole = false;
  }
  return s;
}
// The sequence w that holds step `at` (below the total), and the steps before it.
template <class Args>
__device__ __forceinline__ void few_find(const Args& a, const qlinear_kv_cache& c, const Plan& plan, int group,
                                        const Spans& s, int at, int& before, Work& w) {
  Costs k = s.costs;
  before = 0;
  for (int b0 = 0;; b0 += 64, k = few_costs(a, c, plan, group, b0)) {
    const uint64_t past = __ballot(before + k.upto > at);
    if (past || b0 + 64 >= a.batch) {
      const int i = past ? __builtin_ctzll(past) : 0;
      before += __builtin_amdgcn_readlane(k.upto - k.own, i);
      k.get(b0 + i, w);
      return;
    }
    before += __builtin_amdgcn_readlane(k.upto, 63);
  }
}
// The steps before sequence b.
template <class Args>
__device__ __forceinline__ int few_before(const Args& a, const qlinear_kv_cache& c, const Plan& plan,
                                          int group, const Spans& s, int b) {
  Costs k = s.costs;
  int before = 0;
  for (int b0 = 0; b >= 64; b -= 64) {
    before += __builtin_amdgcn_readlane(k.upto, 63);
    b0 += 64;
    k = few_costs(a, c, plan, group, b0);
  }
  return before + __builtin_amdgcn_readlane(k.upto - k.own, b);
}

// Lane swaps: both halves' (rows of 16 lanes', pairwise) values of x in every lane.
struct Two {
  float a, b;
};
__device__ __forceinline__ Two swap32(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return {__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1])};
}
__device__ __forceinline__ Two swap16(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return {__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1])};
}
__device__ __forceinline__ float max32(float x) {
  const Two t = swap32(x);
  return fmaxf(t.a, t.b);
}
__device__ __forceinline__ float max16(float x) {
  const Two t = swap16(x);
  return fmaxf(t.a, t.b);
}
__device__ __forceinline__ float sum32(float x) {
  const Two t = swap32(x);
  return t.a + t.b;
}
__device__ __forceinline__ float sum16(float x) {
  const Two t = swap16(x);
  return t.a + t.b;
}

__device__ __forceinline__ half2v as_half2(uint32_t x) { return __builtin_bit_cast(half2v, x); }
__device__ __forceinline__ uint32_t as_u32(half2v x) { return __builtin_bit_cast(uint32_t, x); }
__device__ __forceinline__ uint32_t lo_halves(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x05040100u);
}
__device__ __forceinline__ uint32_t hi_halves(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x07060302u);
}

// Non-finite float16 halves of a pair, as bit 15 of each half: adding to the
// magnitude carries into that bit from 0x7C00 (infinity) or 0x7C01 (NaN) on.
constexpr uint32_t kTops = 0x80008000u, kOnes = 0x3C003C00u;   // kOnes: a pair of 1.0
__device__ __forceinline__ uint32_t nonfinite_halves(uint32_t x) { return ((x & ~kTops) + 0x04000400u) & kTops; }
__device__ __forceinline__ uint32_t nan_halves(uint32_t x) { return ((x & ~kTops) + 0x03FF03FFu) & kTops; }
// Whole halves, or 1.0, where bit 15 says so.
__device__ __forceinline__ uint32_t spread_top(uint32_t f) { return f | (f - (f >> 15)); }
__device__ __forceinline__ uint32_t ones_at(uint32_t f) { return (f >> 1) - (f >> 5); }
// Masks of a pair's halves.
__device__ __forceinline__ uint32_t both(bool lo, bool hi) { return (lo ? 0x0000FFFFu : 0u) | (hi ? 0xFFFF0000u : 0u); }

// ---- codes to values. A code in the low bits of a half, OR-ed into float16
// 1024.0, is 1024 + code exactly; minus 1024 + half of the range it is the
// signed code exactly, and one product with the block's scale rounds as the
// codec does.
constexpr uint32_t kMagic = 0x64006400u;

template <int B>
__device__ __forceinline__ half2v code_pair(uint32_t codes, half2v scale) {
  const half2v bias = {(_Float16)(-1024.0f - (float)(1 << (B - 1))), (_Float16)(-1024.0f - (float)(1 << (B - 1)))};
  return (as_half2(codes | kMagic) + bias) * scale;
}

}  // namespace attn

// Launchers of the views' kernels, one file per head width (see attention_views.hip).
#define QLINEAR_VIEW_LAUNCHER(name)                                                                               \
  hipError_t name(const qlinear_kv_cache& c, const ViewArgs& a, const attn::Plan& p, const attn::ViewPartials& part, \
                  hipStream_t stream)
QLINEAR_VIEW_LAUNCHER(launch_view_few_64);
QLINEAR_VIEW_LAUNCHER(launch_view_few_128);
QLINEAR_VIEW_LAUNCHER(launch_view_few_256);
QLINEAR_VIEW_LAUNCHER(launch_view_chunk_64);
QLINEAR_VIEW_LAUNCHER(launch_view_chunk_128);
QLINEAR_VIEW_LAUNCHER(launch_view_chunk_256);

// Launchers, one file per head width (see paged_attention.hip).
hipError_t launch_attention_few_64(const qlinear_kv_cache& c, const AttentionArgs& a, const attn::Plan& p,
                                   const attn::Partials& part, hipStream_t stream);
hipError_t launch_attention_few_128(const qlinear_kv_cache& c, const AttentionArgs& a, const attn::Plan& p,
                                    const attn::Partials& part, hipStream_t stream);
hipError_t launch_attention_few_256(const qlinear_kv_cache& c, const AttentionArgs& a, const attn::Plan& p,
                                    const attn::Partials& part, hipStream_t stream);
hipError_t launch_attention_chunk_64(const qlinear_kv_cache& c, const AttentionArgs& a, const attn::Plan& p,
                                     const attn::Partials& part, hipStream_t stream);
hipError_t launch_attention_chunk_128(const qlinear_kv_cache& c, const AttentionArgs& a, const attn::Plan& p,
                                      const attn::Partials& part, hipStream_t stream);
hipError_t launch_attention_chunk_256(const qlinear_kv_cache& c, const AttentionArgs& a, const attn::Plan& p,
                                      const attn::Partials& part, hipStream_t stream);

}  // namespace qlinear
