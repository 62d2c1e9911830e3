// Log probabilities of given tokens, entropy and top alternatives of rows of
// logits x with maximum m, in base 2:
//   t_i = (x_i - m) log2(e);  l = sum 2^t_i;  s = sum 2^t_i t_i
//   log p_i = (t_i - log2 l) ln 2;  H = (log2 l - s / l) ln 2
// Of float16, t_i is one fused multiply-add, x_i log2(e) - c with c = RNE(m
// log2 e), whose rounding is the same in t and l and cancels; float32's lowest
// values, as masks have them, would overflow there. The top ones are the
// largest keys (order of the value, lower index), so ties are settled.
//
// Bound by reading the logits once: a workgroup holds its part of a row in
// registers between the maximum, the sums and the search. Rows are cut into
// parts where there are few of them, or where a row is longer than the
// registers; a second launch joins the parts. The search: the k-th largest of
// 64 maxima, over a 64th of the part each, is below the k-th largest element or
// equal to it. What is not below it (about k to 2 k elements of rows without
// order) goes to LDS and is ranked there by counting larger keys. Where too many
// are equal to it (rows with masks), the first ones by index are taken in order.
//
// Measured: 2047 rows of 32000 float16 logits 27.5 us without alternatives (4.8
// TB/s, what a large copy reaches), 33.6 with 5, 36 with 20, 46 with 64; float32
// with 5 56.7; 1000 of 65536 with 20 39.8; one row of 131072 float32 with 20, in
// 128 parts, 5.4 and the join 6.6, 17.9 with the host's call. With all elements converted once and kept
// (256 registers) the first took 65 with 5; with the largest of 64 columns for 64
// alternatives, which leaves too many above it now and then, 711 with 64.
#include <type_traits>

#include "qlinear_kernels.hpp"

namespace qlinear {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kCandidates = 512;
constexpr int kMaxParts = kThreads;      // of a row that is cut for the sake of more workgroups
constexpr int kMaxGroups = 16;           // of elements that a thread holds: 1, 2, 4, 8 or 16
// Turns of the join's threads over a row's parts. A float32 row of the longest that
// starts inside a group has one part more than there are threads.
constexpr int kJoinTurns = 2;
static_assert((QLINEAR_MAX_VOCAB + 3 - 1) / (kThreads * kMaxGroups * 4) + 1 <= kJoinTurns * kThreads);
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

typedef _Float16 half2v __attribute__((ext_vector_type(2)));

// Values as integers in their order, NaN on top, both zeros the same; never 0.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);
  return x != x ? ~0u : b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __builtin_bit_cast(float, u == ~0u ? 0x7FC00000u : u & 0x80000000u ? u ^ 0x80000000u : ~u);
}
__device__ __forceinline__ uint64_t make_key(float x, int i) {
  return (uint64_t)ordered(x) << 32 | (uint32_t)(INT32_MAX - i);
}

// t of an element x of type T (see above). A row or part of -infinity alone has t = x.
template <typename T>
__device__ __forceinline__ float exponent(float x, float m) {
  const float base = m == -INFINITY ? 0.0f : m;
  return sizeof(T) == 4 ? (x - base) * kLog2e : fmaf(x, kLog2e, -(base * kLog2e));
}
template <typename T>
__device__ __forceinline__ float log_p(float x, float m, float log2_l) {
  if constexpr (sizeof(T) == 2) return (exponent<T>(x, m) - log2_l) * kLn2;
  return x - (m == -INFINITY ? 0.0f : m) - log2_l * kLn2;      // the lowest value has one too
}
// t of a part's maximum in a row of maximum m: what its own c is above the row's.
template <typename T>
__device__ __forceinline__ float exponent_of_part(float part, float m) {
#pragma clang fp contract(off)
  if constexpr (sizeof(T) == 4) return exponent<T>(part, m);
  const float base = m == -INFINITY ? 0.0f : m;
  const float c = part * kLog2e, all = base * kLog2e;
  return c - all;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) v = fmaxf(v, __shfl_xor(v, k));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) v += __shfl_xor(v, k);
  return v;
}

struct Shared {
  float lane_max[kWaves][64];
  float l[kWaves], s[kWaves];
  float least[kWaves];
  int ties[kWaves];
  uint64_t best[kWaves];
  uint64_t candidates[kCandidates];
  int count;
};

// A value that the k-th largest element is not below: the k-th largest of 64
// maxima (column: that of a lane of all waves) or, for more than 32, where those
// would leave too many above it, of 256 (sh.lane_max). top: the largest.
__device__ __forceinline__ float threshold(Shared& sh, float column, float top, int k) {
  if (k == 1) return top;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  int larger = 0;
  float mine = column;
  if (k <= 32) {
#pragma unroll
    for (int j = 0; j < 64; ++j)
      larger += __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, column), j)) > mine ? 1 : 0;
  } else {
    mine = sh.lane_max[wave][lane];
    for (int j = 0; j < kThreads; j += 4) {
      const float4 v = *reinterpret_cast<const float4*>(&sh.lane_max[0][0] + j);
      larger += (v.x > mine) + (v.y > mine) + (v.z > mine) + (v.w > mine);
    }
  }
  float v = larger < k ? mine : INFINITY;
#pragma unroll
  for (int j = 1; j < 64; j <<= 1) v = fminf(v, __shfl_xor(v, j));
  if (k <= 32) return v;
  if (lane == 0) sh.least[wave] = v;
  __syncthreads();
  return fminf(fminf(sh.least[0], sh.least[1]), fminf(sh.least[2], sh.least[3]));
}

// Which of its keys a thread passes on, by their values.
enum Pass { kNotBelow, kAbove, kAll };

// Calls put(rank, key) for the k largest keys of all threads, of which one is
// `least` or larger. each(pass, f) calls f(key) for the thread's own keys that are
// to be passed on, and tied(turn, f) for those of turn 0 .. turns - 1 that have the
// value `least`; turns are in the order of indexes, and in a turn threads are.
// Fewer than k: the others are not put. Returns how many there were to choose from.
template <typename Each, typename Tied, typename Put>
__device__ __forceinline__ int top_keys(int k, Shared& sh, Each each, int turns, Tied tied, Put put) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  auto push = [&](uint64_t key) {
    const int at = atomicAdd(&sh.count, 1);
    if (at < kCandidates) sh.candidates[at] = key;
  };
  each(std::integral_constant<int, kNotBelow>{}, push);
  __syncthreads();
  int n = sh.count;
  if (n > kCandidates) {
    // Many of one value: those above it, and of it the first ones by index.
    __syncthreads();
    if (threadIdx.x == 0) sh.count = 0;
    __syncthreads();
    each(std::integral_constant<int, kAbove>{}, push);
    __syncthreads();
    n = sh.count;
    for (int turn = 0; turn < turns && n < k; ++turn) {
      int own = 0;
      tied(turn, [&](uint64_t) { ++own; });
      int upto = own;
#pragma unroll
      for (int j = 1; j < 64; j <<= 1) {
        const int o = __shfl_up(upto, j);
        if (lane >= j) upto += o;
      }
      if (lane == 63) sh.ties[wave] = upto;
      __syncthreads();
      int at = n + upto - own, all = 0;
#pragma unroll
      for (int j = 0; j < kWaves; ++j) {
        if (j < wave) at += sh.ties[j];
        all += sh.ties[j];
      }
      tied(turn, [&](uint64_t key) {
        if (at < k) sh.candidates[at] = key;
        ++at;
      });
      n = min(n + all, k);
      __syncthreads();
    }
  }
  if (n <= kCandidates) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const uint64_t key = sh.candidates[i];
      int rank = 0;
#pragma unroll 4
      for (int j = 0; j < n; ++j) rank += sh.candidates[j] > key ? 1 : 0;
      if (rank < k) put(rank, key);
    }
    return n;
  }
  // More different values than that are above it: one maximum after another.
  uint64_t last = ~0ull;
  for (int r = 0; r < k; ++r) {
    uint64_t best = 0;
    each(std::integral_constant<int, kAll>{}, [&](uint64_t key) {
      if (key < last && key > best) best = key;
    });
#pragma unroll
    for (int j = 1; j < 64; j <<= 1) {
      const uint64_t o = __shfl_xor(best, j);
      best = o > best ? o : best;
    }
    __syncthreads();
    if (lane == 0) sh.best[wave] = best;
    __syncthreads();
    for (int j = 0; j < kWaves; ++j) best = sh.best[j] > best ? sh.best[j] : best;
    if (threadIdx.x == 0) put(r, best);
    last = best;
  }
  return n;
}

// A part's results (m the maximum, l and s as above), or a row's.
struct Sums {
  float m, l, s;
};

// Partial results: float4 (m, l, s, 0) and `top` keys, 0 where there are
// fewer, of each row's parts.
struct Parts {
  float4* sums;
  uint64_t* keys;
  int per_row;
};

__device__ __forceinline__ float load1(const uint16_t* p) { return (float)__builtin_bit_cast(_Float16, *p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }

// What one thread writes for a row.
template <typename T>
__device__ __forceinline__ void write_row(const LogprobArgs& a, int row, const Sums& r) {
  const float log_l = log2f(r.l);
  if (a.logprob) {
    const int token = a.tokens[row];
    float y = __builtin_nanf("");
    if ((unsigned)token < (unsigned)a.vocab) {
      const float x = load1(static_cast<const T*>(a.logits) + row * a.stride + token);
      y = log_p<T>(x, r.m, log_l);
    }
    a.logprob[row] = y;
  }
  if (a.entropy) {
    const float h = (log_l - r.s / r.l) * kLn2;
    a.entropy[row] = h < 0.0f ? 0.0f : h;
  }
}
template <typename T>
__device__ __forceinline__ void write_top(const LogprobArgs& a, int row, const Sums& r, int rank, uint64_t key) {
  const int64_t at = (int64_t)row * a.top + rank;
  a.top_logprob[at] = log_p<T>(unordered((uint32_t)(key >> 32)), r.m, log2f(r.l));
  a.top_id[at] = INT32_MAX - (int)(uint32_t)key;
}

// Four or eight elements as loaded.
template <typename T>
struct Group {
  static constexpr int kSize = 16 / sizeof(T);
  uint4 v;
  __device__ __forceinline__ float get(int e) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (sizeof(T) == 4)
      return __builtin_bit_cast(float, w[e]);
    else
      return (float)__builtin_bit_cast(half2v, w[e / 2])[e % 2];
  }
  __device__ __forceinline__ void none() {
    const uint32_t w = sizeof(T) == 4 ? 0xFF800000u : 0xFC00FC00u;
    v = make_uint4(w, w, w, w);
  }
  // Elements at .. of a row of n; what is outside it is -infinity.
  __device__ __forceinline__ void load(const T* row, int at, int n) {
    if (at >= 0 && at <= n - kSize) {
      v = *reinterpret_cast<const uint4*>(row + at);
      return;
    }
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < kSize; ++e) {
      uint32_t x = sizeof(T) == 4 ? 0xFF800000u : 0xFC00u;
      if (at + e >= 0 && at + e < n) {
        if constexpr (sizeof(T) == 4)
          x = __builtin_bit_cast(uint32_t, row[at + e]);
        else
          x = row[at + e];
      }
      w[e * sizeof(T) / 4] |= sizeof(T) == 4 ? x : x << 16 * (e % 2);
    }
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
  // NaN is left out.
  __device__ __forceinline__ float max() const {
    if constexpr (sizeof(T) == 4) {
      return fmaxf(fmaxf(get(0), get(1)), fmaxf(get(2), get(3)));
    } else {
      const half2v a = __builtin_elementwise_max(__builtin_bit_cast(half2v, v.x), __builtin_bit_cast(half2v, v.y));
      const half2v b = __builtin_elementwise_max(__builtin_bit_cast(half2v, v.z), __builtin_bit_cast(half2v, v.w));
      const half2v c = __builtin_elementwise_max(a, b);
      return fmaxf((float)c[0], (float)c[1]);
    }
  }
};

// NG groups a thread; a workgroup has part blockIdx % per_row of a row.
template <typename T, int NG>
__global__ __launch_bounds__(kThreads) void logprob_kernel(LogprobArgs a, Parts parts) {
  constexpr int G = Group<T>::kSize;
  __shared__ Shared sh;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int row = blockIdx.x / parts.per_row, part = blockIdx.x % parts.per_row;
  const T* p = static_cast<const T*>(a.logits) + row * a.stride;
  // Groups are aligned in memory: a row's first and last may be others' in part.
  const int shift = (int)((uintptr_t)p / sizeof(T) % G);
  const int first = (part * NG * kThreads + t) * G - shift;     // the thread's groups start kThreads * G elements apart
  if (t == 0) sh.count = 0;

  auto place = [&](int i) { return first + i * kThreads * G; };
  Group<T> x[NG];
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    // Groups that are not whole read the row's second, which is, instead of branching.
    const bool whole = place(i) >= 0 && place(i) <= a.vocab - G;
    if (a.vocab >= 2 * G) x[i].v = *reinterpret_cast<const uint4*>(p + (whole ? place(i) : G - shift));
    if (!whole) x[i].none();
  }
  if (a.vocab < 2 * G || shift != 0 || a.vocab % G != 0) {
    // A row's first group is a thread's first, its last one any.
    const int last = (a.vocab - 1 + shift) / G * G - shift, i_last = (last - first) / (kThreads * G);
    const bool has_last = last >= first && last == place(i_last) && i_last < NG;
    if (place(0) > -G && place(0) < a.vocab) x[0].load(p, place(0), a.vocab);
    Group<T> end;
    end.none();
    if (has_last) end.load(p, last, a.vocab);
#pragma unroll
    for (int i = 0; i < NG; ++i)
      if (has_last && i == i_last) x[i] = end;
  }

  // The elements stay as loaded: converted ones are not kept from one use to the next.
  auto keep = [&]() {
#pragma unroll
    for (int i = 0; i < NG; ++i) asm("" : "+v"(x[i].v.x), "+v"(x[i].v.y), "+v"(x[i].v.z), "+v"(x[i].v.w));
  };
  keep();
  float mine = -INFINITY;
#pragma unroll
  for (int i = 0; i < NG; ++i) mine = fmaxf(mine, x[i].max());
  keep();
  sh.lane_max[wave][lane] = mine;
  __syncthreads();
  float column = sh.lane_max[0][lane];
#pragma unroll
  for (int j = 1; j < kWaves; ++j) column = fmaxf(column, sh.lane_max[j][lane]);
  Sums r;
  r.m = wave_max(column);
  float l = 0.0f, s = 0.0f;
#pragma unroll
  for (int i = 0; i < NG; ++i)
#pragma unroll
    for (int e = 0; e < G; ++e) {
      const float d = exponent<T>(x[i].get(e), r.m), y = __builtin_amdgcn_exp2f(d);
      l += y;
      s = fmaf(y, fmaxf(d, -3e38f), s);      // 0 times -infinity adds nothing
    }
  l = wave_sum(l);
  s = wave_sum(s);
  if (lane == 0) {
    sh.l[wave] = l;
    sh.s[wave] = s;
  }
  __syncthreads();
  r.l = r.s = 0.0f;
#pragma unroll
  for (int j = 0; j < kWaves; ++j) {
    r.l += sh.l[j];
    r.s += sh.s[j];
  }
  const bool direct = parts.per_row == 1;
  if (t == 0) {
    if (direct)
      write_row<T>(a, row, r);
    else
      parts.sums[blockIdx.x] = make_float4(r.m, r.l, r.s, 0.0f);
  }
  if (a.top == 0) return;

  keep();
  const float least = threshold(sh, column, r.m, a.top);
  const bool nan = r.l != r.l;        // there may be NaN, which no maximum shows
  // The thread's groups that hold one of the largest: few, so they are loaded again.
  unsigned groups = 0;
#pragma unroll
  for (int i = 0; i < NG; ++i) groups |= x[i].max() >= least || nan ? 1u << i : 0u;
  auto keys_of = [&](int i, auto wanted, auto f) {
    Group<T> y;
    y.load(p, place(i), a.vocab);
#pragma unroll
    for (int e = 0; e < G; ++e) {
      const int at = place(i) + e;
      if (wanted(y.get(e)) && at >= 0 && at < a.vocab) f(make_key(y.get(e), at));
    }
  };
  const int found = top_keys(
      a.top, sh,
      [&](auto pass, auto f) {
        constexpr int kPass = decltype(pass)::value;
#pragma unroll 1
        for (unsigned m = kPass == kAll ? (1u << NG) - 1 : groups; m != 0; m &= m - 1)
          keys_of(__builtin_ctz(m),
                  [&](float y) { return kPass == kAll || !(kPass == kAbove ? y <= least : y < least); }, f);
      },
      NG, [&](int i, auto f) { keys_of(i, [&](float y) { return y == least; }, f); },
      [&](int rank, uint64_t key) {
        if (direct)
          write_top<T>(a, row, r, rank, key);
        else
          parts.keys[(int64_t)blockIdx.x * a.top + rank] = key;
      });
  // A part of fewer elements than that (never a whole row).
  if (!direct && t < a.top && t >= found) parts.keys[(int64_t)blockIdx.x * a.top + t] = 0;
}

// A workgroup joins a row's parts.
template <typename T>
__global__ __launch_bounds__(kThreads) void logprob_join_kernel(LogprobArgs a, Parts parts) {
  __shared__ Shared sh;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, row = blockIdx.x;
  const int64_t p0 = (int64_t)row * parts.per_row;
  const uint64_t* keys = parts.keys + p0 * a.top;
  const int n = parts.per_row * a.top;
  if (t == 0) sh.count = 0;
  float4 v[kJoinTurns];
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < kJoinTurns; ++j) {
    const int i = t + j * kThreads;
    v[j] = make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
    if (i < parts.per_row) v[j] = parts.sums[p0 + i];
    m = fmaxf(m, v[j].x);
  }
  // The thread's keys, in the order of their places: loads of a turn do not wait for
  // one another (one row of 131072 with 20 alternatives: 7.7 us with one after another, 6.4 so).
  constexpr int kTurn = 8;
  auto own = [&](auto f) {
#pragma unroll 1
    for (int i0 = t; i0 < n; i0 += kTurn * kThreads) {
      uint64_t key[kTurn];
#pragma unroll
      for (int j = 0; j < kTurn; ++j) key[j] = keys[min(i0 + j * kThreads, n - 1)];
#pragma unroll
      for (int j = 0; j < kTurn; ++j)
        if (i0 + j * kThreads < n) f(key[j]);
    }
  };
  uint64_t most = 0;
  own([&](uint64_t key) { most = key > most ? key : most; });
  // NaN, which is no column's maximum here either, is looked for where there is one.
  const bool none = most == 0, odd = (uint32_t)(most >> 32) == ~0u;
  const float mine = none || odd ? -INFINITY : unordered((uint32_t)(most >> 32));

  m = wave_max(m);
  if (lane == 0) sh.s[wave] = m;
  sh.lane_max[wave][lane] = mine;
  __syncthreads();
  Sums r;
  r.m = fmaxf(fmaxf(sh.s[0], sh.s[1]), fmaxf(sh.s[2], sh.s[3]));
  float column = sh.lane_max[0][lane];
#pragma unroll
  for (int j = 1; j < kWaves; ++j) column = fmaxf(column, sh.lane_max[j][lane]);
  __syncthreads();
  float l = 0.0f, s = 0.0f;
#pragma unroll
  for (int j = 0; j < kJoinTurns; ++j) {
    if (v[j].x == -INFINITY && v[j].y == 0.0f) continue;
    const float d = exponent_of_part<T>(v[j].x, r.m), f = __builtin_amdgcn_exp2f(d);
    l += f * v[j].y;
    s += f > 0.0f ? f * fmaf(v[j].y, d, v[j].z) : 0.0f;      // d may be -infinity
  }
  l = wave_sum(l);
  s = wave_sum(s);
  if (lane == 0) {
    sh.l[wave] = l;
    sh.s[wave] = s;
  }
  __syncthreads();
  r.l = r.s = 0.0f;
#pragma unroll
  for (int j = 0; j < kWaves; ++j) {
    r.l += sh.l[j];
    r.s += sh.s[j];
  }
  if (t == 0) write_row<T>(a, row, r);
  if (a.top == 0) return;
  const float least = threshold(sh, column, wave_max(column), a.top);
  const uint32_t from = ordered(least);
  // Keys stand in the order of indexes where their values are the same.
  top_keys(
      a.top, sh,
      [&](auto pass, auto f) {
        constexpr int kPass = decltype(pass)::value;
        if (none || (kPass != kAll && (uint32_t)(most >> 32) < from)) return;
        own([&](uint64_t key) {
          const uint32_t v = (uint32_t)(key >> 32);
          if (key != 0 && (kPass == kAll || (kPass == kAbove ? v > from : v >= from))) f(key);
        });
      },
      (n + kThreads - 1) / kThreads,
      [&](int turn, auto f) {
        const int i = turn * kThreads + t;
        if (i < n && (uint32_t)(keys[i] >> 32) == from) f(keys[i]);
      },
      [&](int rank, uint64_t key) { write_top<T>(a, row, r, rank, key); });
}

struct Plan {
  int groups;      // of a thread
  int parts;
};

// As few parts as give every CU two workgroups.
constexpr int kWanted = 512;
Plan make_plan(int rows, int vocab, bool f32, bool whole) {
  const int size = f32 ? 4 : 8;
  // Rows that start inside a group (not `whole`) may have one more.
  auto parts = [&](int groups) {
    const int64_t all = (int64_t)vocab + (whole ? 0 : size - 1), part = kThreads * groups * size;
    return (int)((all + part - 1) / part);
  };
  int g = kMaxGroups;
  while (g > 1 && (int64_t)rows * parts(g) < kWanted && parts(g / 2) <= kMaxParts) g /= 2;
  const int n = parts(g);
  while (g > 1 && parts(g / 2) == n) g /= 2;
  return {g, n};
}

}  // namespace

// Whether all rows start at whole groups.
static bool whole_rows(const LogprobArgs& a) {
  return ((uintptr_t)a.logits & 15) == 0 && (a.rows == 1 || a.stride * (a.f32 ? 4 : 2) % 16 == 0);
}

size_t logprob_workspace_need(const LogprobArgs& a) {
  const Plan p = make_plan(a.rows, a.vocab, a.f32, whole_rows(a));
  return p.parts == 1 ? 0 : (size_t)a.rows * p.parts * (sizeof(float4) + sizeof(uint64_t) * a.top);
}

size_t logprob_workspace_bytes(const LogprobArgs& a) {
  // Fewer rows are cut into more parts, but only while they are below kWanted in all
  // (halving a part doubles their number at most); shorter rows have fewer.
  const int64_t most = (int64_t)a.rows * make_plan(1 << 22, a.vocab, a.f32, false).parts;
  const size_t parts = make_plan(1, a.vocab, a.f32, false).parts == 1 ? 0 : most > 2 * kWanted ? most : 2 * kWanted;
  return parts * (sizeof(float4) + sizeof(uint64_t) * a.top);
}

hipError_t launch_logprob(const LogprobArgs& a, void* ws, hipStream_t stream) {
  const Plan p = make_plan(a.rows, a.vocab, a.f32, whole_rows(a));
  Parts parts = {(float4*)ws, nullptr, p.parts};
  if (p.parts > 1) parts.keys = (uint64_t*)(parts.sums + (int64_t)a.rows * p.parts);
  auto go = [&](auto type) {
    using T = decltype(type);
    auto kernel = p.groups == 1   ? logprob_kernel<T, 1>
                  : p.groups == 2 ? logprob_kernel<T, 2>
                  : p.groups == 4 ? logprob_kernel<T, 4>
                  : p.groups == 8 ? logprob_kernel<T, 8>
                                  : logprob_kernel<T, 16>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(a.rows * p.parts)), dim3(kThreads), 0, stream, a, parts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.parts == 1) return e;
    hipLaunchKernelGGL(logprob_join_kernel<T>, dim3((unsigned)a.rows), dim3(kThreads), 0, stream, a, parts);
    return hipGetLastError();
  };
  return a.f32 ? go(float{}) : go(uint16_t{});
}

}  // namespace qlinear
