// Attention for few query rows per key/value head (single tokens, drafts):
// bound by reading the cache. The rows of one sequence and key/value head,
// up to 16 NT (token, head of the group) pairs, are the columns of 16-wide
// matrix-core tiles, so that the cache is read once for all of them.
//
// A workgroup takes a span of steps of 32 tokens, equal for all, of one
// sequence or several, so that lengths of any mix fill the chip evenly (32
// sequences of 1 to 8191 tokens, 64/8 heads: 98 us with each sequence cut by
// itself, 77 us so). Its four waves take steps in turn, each with its own
// running maximum and sums, and join at the end of each sequence. Keys and
// values go from memory straight into matrix fragments, with no LDS between:
//   - S^T tile i (16 tokens): lane (c, g) = (l % 16, l / 16) holds key c's
//     elements of k-group g. float16: 8 elements at 32 f + 8 g for fragment
//     f, so that four lanes cover 64 contiguous bytes of a row. Quantized:
//     the lane's fragments are one contiguous run of D / 4 elements, which
//     has one scale per 32 elements at most; q is laid out in the order in
//     which the codes unpack.
//   - O^T: lane (c, g) holds tokens 4 g .. + 3 and 16 + 4 g .. + 3 (the rows
//     of S^T in its accumulators) and elements W c .. W c + W - 1 of them
//     (W = 8, 4 at D = 64); fragment j pairs up element j of its 8 tokens by
//     byte permutes (float16) or while unpacking (codes of two tokens share
//     a register's halves).
// A step's key loads are issued before the previous step's softmax, its
// value loads after the previous step's second product.
//
// Measured, each call's cache cold: 16 sequences of 4096 tokens, 32/32 heads
// of 128, float16: 168 us, 6.4 TB/s; 64 of 2048, 64/8 heads: float16 90 us, 6.0
// TB/s, Q8 55, Q6 58, Q4 45 us (unpacking bounds those); one of 32768: 31 us.
#pragma once

#include <type_traits>

#include "attention.hpp"

namespace qlinear {
namespace attn {

constexpr int kFewWaves = 4;
constexpr int kAllButVmem = 0x78F;     // what may move across a scheduling barrier

// Raw registers of one step. Scales have a register each: two 16-bit values
// that live across the loop would be packed into one where they are loaded,
// which waits for them there.
template <int D, int B>
struct KeyRaw {
  static constexpr int kScales = D == 256 ? 2 : 1;
  // words of a lane's row part (D / 4 codes, or D / 32 fragments of float16)
  static constexpr int kWords = B == 16 ? D / 8 : D / 4 * B / 32;
  uint32_t w[2][kWords];
  uint32_t s[2][kScales];
};

template <int D, int B>
struct ValueRaw {
  static constexpr int W = D == 64 ? 4 : 8;     // elements of a token per lane and part
  static constexpr int U = D / (16 * W);        // parts (128 elements apart)
  static constexpr int kWords = B == 16 ? W / 2 : B == 6 ? 2 : (W * B + 31) / 32;
  uint32_t w[8][U][kWords];
  uint32_t s[8][U];
};

// Loads of 4, 2 and 1 words, 4-byte aligned. What this workgroup alone reads,
// once (ONCE), goes past the caches, whose lines serve nobody then.
typedef u32x4 __attribute__((aligned(4))) u32x4_a4;
typedef u32x2 __attribute__((aligned(4))) u32x2_a4;
template <bool ONCE>
__device__ __forceinline__ u32x4 load4(const void* p) {
  const u32x4_a4* w = static_cast<const u32x4_a4*>(p);
  if constexpr (ONCE)
    return __builtin_nontemporal_load(w);
  else
    return *w;
}
template <bool ONCE>
__device__ __forceinline__ u32x2 load2(const void* p) {
  const u32x2_a4* w = static_cast<const u32x2_a4*>(p);
  if constexpr (ONCE)
    return __builtin_nontemporal_load(w);
  else
    return *w;
}
template <bool ONCE>
__device__ __forceinline__ uint32_t load1(const void* p) {
  const uint32_t* w = static_cast<const uint32_t*>(p);
  if constexpr (ONCE)
    return __builtin_nontemporal_load(w);
  else
    return *w;
}

template <int N, bool ONCE>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const uint32_t* p) {
#pragma unroll
  for (int i = 0; i + 4 <= N; i += 4) {
    const u32x4 v = load4<ONCE>(p + i);
    w[i] = v[0];
    w[i + 1] = v[1];
    w[i + 2] = v[2];
    w[i + 3] = v[3];
  }
  if constexpr (N % 4 >= 2) {
    const u32x2 v = load2<ONCE>(p + N / 4 * 4);
    w[N / 4 * 4] = v[0];
    w[N / 4 * 4 + 1] = v[1];
  }
  if constexpr (N % 2 == 1) w[N - 1] = load1<ONCE>(p + N - 1);
}

// Keys of tile i: pool row r0 is its first token's.
template <int D, int B, bool ONCE>
__device__ __forceinline__ void load_keys(KeyRaw<D, B>& k, int i, const qlinear_kv_cache& c, int group_shift,
                                          int64_t r0, int col, int g) {
  if constexpr (B == 16) {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(c.k) + r0 * D + col * D + 8 * g;
#pragma unroll
    for (int f = 0; f < D / 32; ++f) {
      const u32x4 v = load4<ONCE>(p + 32 * f);
#pragma unroll
      for (int e = 0; e < 4; ++e) k.w[i][4 * f + e] = v[e];
    }
  } else {
    constexpr int kN = KeyRaw<D, B>::kWords;
    load_words<kN, ONCE>(k.w[i], reinterpret_cast<const uint32_t*>(c.k) + r0 * (4 * kN) + col * (4 * kN) + g * kN);
    const int per = D >> group_shift;
#pragma unroll
    for (int s = 0; s < KeyRaw<D, B>::kScales; ++s)
      k.s[i][s] = c.k_scales[r0 * per + col * per + ((g * (D / 4) + 32 * s) >> group_shift)];
  }
}

// Values of tile i: tokens 4 g .. 4 g + 3 of it.
template <int D, int B, bool ONCE>
__device__ __forceinline__ void load_values(ValueRaw<D, B>& v, int i, const qlinear_kv_cache& c, int group_shift,
                                            int64_t r0, int col, int g) {
  constexpr int W = ValueRaw<D, B>::W;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int row = 4 * g + t;
#pragma unroll
    for (int u = 0; u < ValueRaw<D, B>::U; ++u) {
      auto& w = v.w[4 * i + t][u];
      if constexpr (B == 16) {
        load_words<W / 2, ONCE>(w, reinterpret_cast<const uint32_t*>(c.v) + r0 * (D / 2) + row * (D / 2) + u * 64 +
                                 col * (W / 2));
      } else {
        const char* p = reinterpret_cast<const char*>(c.v) + r0 * (D * B / 8) + row * (D * B / 8) + u * (16 * B);
        if constexpr (W * B == 64) {
          load_words<2, ONCE>(w, reinterpret_cast<const uint32_t*>(p + col * 8));
        } else if constexpr (W * B == 32) {
          w[0] = load1<ONCE>(p + col * 4);
        } else if constexpr (W * B == 16) {
          w[0] = *reinterpret_cast<const uint16_t*>(p + col * 2);
        } else {
          // Six bits: 8 codes are 6 bytes, 2-byte aligned; at W = 4 two lanes share them.
          const uint16_t* q = reinterpret_cast<const uint16_t*>(p + (W == 8 ? col : col / 2) * 6);
          w[0] = (uint32_t)q[0] | ((uint32_t)q[1] << 16);
          w[1] = q[2];
        }
        const int per = D >> group_shift;
        v.s[4 * i + t][u] = c.v_scales[r0 * per + row * per + ((u * 128 + col * W) >> group_shift)];
      }
    }
  }
}

// Fragment f of tile i's keys.
template <int D, int B>
__device__ __forceinline__ half8 key_fragment(const KeyRaw<D, B>& k, int i, int f) {
  u32x4 r;
  if constexpr (B == 16) {
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = k.w[i][4 * f + e];
  } else {
    const _Float16 s = __builtin_bit_cast(_Float16, (uint16_t)k.s[i][KeyRaw<D, B>::kScales == 1 ? 0 : f / 4]);
    const half2v s2 = {s, s};
    if constexpr (B == 8) {          // 2 words, byte order
#pragma unroll
      for (int e = 0; e < 4; ++e)
        r[e] = as_u32(code_pair<8>(__builtin_amdgcn_perm(0u, k.w[i][2 * f + e / 2], e % 2 ? 0x0C030C02u : 0x0C010C00u),
                                   s2));
    } else if constexpr (B == 4) {   // 1 word: pairs (e, e + 4)
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] = as_u32(code_pair<4>((k.w[i][f] >> (4 * e)) & 0x000F000Fu, s2));
    } else {                         // units 2 (f / 2) and + 1 of 48 bits: pairs across them
      const uint32_t* w = &k.w[i][f / 2 * 3];
      // unit a: bits 0 .. 47 of w[0..2], unit b: bits 48 .. 95
      uint32_t x, y;
      if (f % 2 == 0) {              // codes 0 .. 3: windows at bits 0 and 12
        const uint32_t b0 = __builtin_amdgcn_alignbit(w[2], w[1], 16);
        x = lo_halves(w[0], b0);
        y = lo_halves(w[0] >> 12, b0 >> 12);
      } else {                       // codes 4 .. 7: windows at bits 24 and 36
        x = lo_halves(__builtin_amdgcn_alignbit(w[1], w[0], 24), w[2] >> 8);
        y = lo_halves(w[1] >> 4, w[2] >> 20);
      }
      r[0] = as_u32(code_pair<6>(x & 0x003F003Fu, s2));
      r[1] = as_u32(code_pair<6>((x >> 6) & 0x003F003Fu, s2));
      r[2] = as_u32(code_pair<6>(y & 0x003F003Fu, s2));
      r[3] = as_u32(code_pair<6>((y >> 6) & 0x003F003Fu, s2));
    }
  }
  return __builtin_bit_cast(half8, r);
}

// Element (0 .. D / 4 - 1, of the lane's run for codes; of its fragments for
// float16) that position e of fragment f multiplies.
template <int D, int B>
__device__ __forceinline__ constexpr int q_element(int f, int e) {
  if (B == 4) return 8 * f + e / 2 + 4 * (e % 2);
  if (B == 6) return 8 * (f / 2 * 2 + e % 2) + 4 * (f % 2) + e / 2;
  return 8 * f + e;
}

// Fragments of part u's W elements over the lane's 8 tokens.
template <int D, int B>
__device__ __forceinline__ void value_fragments(const ValueRaw<D, B>& v, int u, int col,
                                                u32x4 (&r)[ValueRaw<D, B>::W]) {
  constexpr int W = ValueRaw<D, B>::W;
#pragma unroll
  for (int t = 0; t < 4; ++t) {       // tokens 2 t, 2 t + 1
    const uint32_t* a = v.w[2 * t][u];
    const uint32_t* b = v.w[2 * t + 1][u];
    if constexpr (B == 16) {
#pragma unroll
      for (int j = 0; j < W / 2; ++j) {
        r[2 * j][t] = lo_halves(a[j], b[j]);
        r[2 * j + 1][t] = hi_halves(a[j], b[j]);
      }
    } else {
      const half2v s = as_half2(lo_halves(v.s[2 * t][u], v.s[2 * t + 1][u]));
      if constexpr (B == 8) {
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const uint32_t k = j % 4;
          r[j][t] = as_u32(code_pair<8>(__builtin_amdgcn_perm(b[j / 4], a[j / 4], 0x0C000C00u | k | ((4u + k) << 16)), s));
        }
      } else if constexpr (B == 4) {
#pragma unroll
        for (int h = 0; h < W / 4; ++h) {
          const uint32_t x = h ? hi_halves(a[0], b[0]) : lo_halves(a[0], b[0]);
#pragma unroll
          for (int j = 0; j < 4; ++j) r[4 * h + j][t] = as_u32(code_pair<4>((x >> (4 * j)) & 0x000F000Fu, s));
        }
      } else {
        uint32_t x[4];
        if constexpr (W == 8) {
          x[0] = lo_halves(a[0], b[0]);
          x[1] = lo_halves(a[0] >> 12, b[0] >> 12);
          x[2] = lo_halves(__builtin_amdgcn_alignbit(a[1], a[0], 24), __builtin_amdgcn_alignbit(b[1], b[0], 24));
          x[3] = lo_halves(a[1] >> 4, b[1] >> 4);
        } else {                       // the lane's half of the 48 bits
          const uint32_t sh = 24 * (col & 1);
          const uint32_t p = (uint32_t)((((uint64_t)a[1] << 32) | a[0]) >> sh);
          const uint32_t q = (uint32_t)((((uint64_t)b[1] << 32) | b[0]) >> sh);
          x[0] = lo_halves(p, q);
          x[1] = lo_halves(p >> 12, q >> 12);
        }
#pragma unroll
        for (int j = 0; j < W; ++j) r[j][t] = as_u32(code_pair<6>((x[j / 2] >> (6 * (j % 2))) & 0x003F003Fu, s));
      }
    }
  }
}

// What the infinities and NaN of a value fragment add to the rows that see
// their tokens (column of `sees`: 1.0 where the row does): counts of tokens
// with +infinity or NaN, and of ones with -infinity or NaN, from the same
// matrix product as the finite values. sum: element r of the fragment's
// result at sum[r * stride].
__device__ __forceinline__ void add_nonfinite(const u32x4& v, const u32x4& sees, float* sum, int stride) {
  u32x4 up, down;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const uint32_t any = nonfinite_halves(v[t]), nan = nan_halves(v[t]);
    up[t] = ones_at((any & ~v[t]) | nan);
    down[t] = ones_at((any & v[t]) | nan);
  }
  const half8 b = __builtin_bit_cast(half8, sees);
  const float4v zero = {0, 0, 0, 0};
  const float4v nu = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, up), b, zero, 0, 0, 0);
  const float4v nd = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, down), b, zero, 0, 0, 0);
#pragma unroll
  for (int r = 0; r < 4; ++r)
    sum[r * stride] += (nu[r] > 0.0f ? INFINITY : 0.0f) - (nd[r] > 0.0f ? INFINITY : 0.0f);
}

template <int D, int B, int NT, bool ONCE>
__global__ __launch_bounds__(64 * kFewWaves, few_per_cu(D, 16 * NT, B)) void attention_few_kernel(
    AttentionArgs a, qlinear_kv_cache c, Plan plan, Partials part) {
  typedef ValueRaw<D, B> VR;
  constexpr int W = VR::W, U = VR::U, kTiles = D / 16, kFrags = D / 32;
  constexpr int kRow = D + 4;     // LDS row of the join, in floats
  __shared__ float join[NT][kFewWaves][16][kRow];
  __shared__ float2 join_ml[NT][kFewWaves][16];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int group = a.q_heads / c.kv_heads;
  const int head = blockIdx.x % c.kv_heads, worker = blockIdx.x / c.kv_heads;
  const int page_shift = __builtin_ctz(c.page_size);
  const int group_shift = B == 16 ? 0 : __builtin_ctz(c.group);

  // This workgroup's steps: `at` to `stop` of all, from step i0 of tile `tile`.
  Work w;
  Item it;
  int tile, i0 = 0, at, stop;
  if (plan.workers == 0) {
    sequence(a, c, blockIdx.y, w);
    it = few_item(a, plan, group, w);
    tile = worker;
    if (tile >= it.tiles) return;
    at = 0;
    stop = it.steps;
  } else {
    const Spans sp = few_spans(a, c, plan, group);
    if (sp.whole) {
      const int b = worker / plan.whole;
      if (b >= a.batch) return;
      if (b < 64)
        sp.costs.get(b, w);
      else
        sequence(a, c, b, w);
      it = few_item(a, plan, group, w);
      tile = worker - b * plan.whole;
      if (tile >= it.tiles) return;
      at = 0;
      stop = it.steps;
    } else {
      if (worker >= plan.workers || (int64_t)worker * sp.quota >= sp.total) return;
      at = worker * sp.quota;
      stop = min(at + sp.quota, sp.total);
      int before;
      few_find(a, c, plan, group, sp, at, before, w);
      it = few_item(a, plan, group, w);
      tile = (unsigned)(at - before) / (unsigned)it.steps;
      i0 = at - before - tile * it.steps;
    }
  }
  int slot = 0;                // of a partial result

  for (;;) {
  const int taken = min(it.steps - i0, stop - at);
  const bool alone = taken == it.steps;
  row_tile(a, group, tile * 16 * NT, 16 * NT, w);
  const int begin = max(it.first_step + i0, w.lo_min / kStep);
  const int end = min(it.first_step + i0 + taken, w.p_max < 0 ? 0 : w.p_max / kStep + 1);
  const int64_t part_row0 = (((int64_t)worker * c.kv_heads + head) * 2 + slot) * (16 * NT);

  // Rows: column col of tile nt is row row0 + 16 nt + col of the sequence.
  int pos[NT], first[NT];
  half8 q[NT][kFrags];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = 16 * nt + col;
    const bool live = r < w.rows;
    const int rr = w.row0 + (live ? r : 0);
    const int tok = rr / group, h = head * group + rr % group;
    pos[nt] = w.len - w.n + tok;
    first[nt] = first_seen(pos[nt], a.window);
    const uint16_t* p = a.q + (w.q0 + tok) * a.q_stride + (int64_t)h * D;
    uint32_t run[D / 8];
#pragma unroll
    for (int f = 0; f < kFrags; ++f) {
      u32x4 v = {0, 0, 0, 0};
      if (live)
        v = *reinterpret_cast<const u32x4*>(p + (B == 16 ? 32 * f + 8 * g : g * (D / 4) + 8 * f));
#pragma unroll
      for (int e = 0; e < 4; ++e) run[4 * f + e] = v[e];
    }
#pragma unroll
    for (int f = 0; f < kFrags; ++f) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int x = q_element<D, B>(f, e);
        q[nt][f][e] = as_half2(run[x / 2])[x % 2];
      }
    }
  }

  const PageTable table = page_table(a, w.b);
  const int last_page = max(w.len - 1, 0) >> page_shift;
  float4v o[NT][kTiles];
  float m[NT], l[NT];
  const float sc = a.scale * kLog2e;

  bool nonfinite = false;      // this wave's rows of join hold what infinities and NaN add
  KeyRaw<D, B> kr;
  VR vr;
  // Pool rows of a step's two tiles; their pages are looked up a step ahead.
  int pages[2];
  int64_t rows[2];
  auto look_up = [&](int step) {
#pragma unroll
    for (int i = 0; i < 2; ++i) pages[i] = page_of(c, table, page_shift, last_page, step * kStep + 16 * i);
  };
  auto keys = [&](int step) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      rows[i] = pool_row(c, pages[i], page_shift, head, step * kStep + 16 * i);
      load_keys<D, B, ONCE>(kr, i, c, group_shift, rows[i], col, g);
    }
  };
  auto values = [&](int step) {
#pragma unroll
    for (int i = 0; i < 2; ++i) load_values<D, B, ONCE>(vr, i, c, group_shift, rows[i], col, g);
    look_up(step + kFewWaves);
  };

  // One step; kind: see StepKind. False: an edge step has infinities or NaN
  // that only some rows see.
  auto one_step = [&](auto kind, int step) __attribute__((always_inline)) -> bool {
    constexpr bool kEdge = decltype(kind)::value != kWhole, kSplit = decltype(kind)::value == kCareful;
    const int t0 = step * kStep;
    // Whole steps are never the wave's last (see below): their loads stand
    // in no branch, which would make the waits for them whole.
    const bool more = !kEdge || step + kFewWaves < end;
    // S^T: tile i, row 4 g + r of it in register r.
    float4v s[NT][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[nt][i] = float4v{0, 0, 0, 0};
#pragma unroll
      for (int f = 0; f < kFrags; ++f) {
        const half8 kf = key_fragment<D, B>(kr, i, f);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          s[nt][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, q[nt][f], s[nt][i], 0, 0, 0);
      }
    }
    if (more) keys(step + kFewWaves);
    // Memory loads stay in this order: keys are waited for first.
    __builtin_amdgcn_sched_barrier(kAllButVmem);

    half8 p[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = s[nt][i / 4][i % 4] * sc;
      if constexpr (kEdge) {      // hide what the row does not see
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int t = t0 + 16 * (i / 4) + 4 * g + i % 4;
          if (t > pos[nt] || t < first[nt]) x[i] = -INFINITY;
        }
      }
      float mx = x[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) mx = fmaxf(mx, x[i]);
      mx = max32(max16(mx));
      const float mn = fmaxf(m[nt], mx);
      const float base = mn == -INFINITY ? 0.0f : mn;
      const float alpha = __builtin_amdgcn_exp2f(m[nt] - base);
      m[nt] = mn;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float e = __builtin_amdgcn_exp2f(x[i] - base);
        sum += e;
        p[nt][i] = (_Float16)e;
      }
      l[nt] = l[nt] * alpha + sum;
#pragma unroll
      for (int j = 0; j < kTiles; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[nt][j][r] *= alpha;
    }

#pragma unroll
    for (int u = 0; u < U; ++u) {
      u32x4 vf[W];
      value_fragments<D, B>(vr, u, col, vf);
      if constexpr (kEdge) {
        // Tokens that no row sees may hold anything: zero.
        uint32_t bad = 0;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int ta = t0 + 16 * (t / 2) + 4 * g + 2 * (t % 2);
          const uint32_t keep = both(ta <= w.p_max && ta >= w.lo_min, ta < w.p_max && ta + 1 >= w.lo_min);
#pragma unroll
          for (int j = 0; j < W; ++j) {
            vf[j][t] &= keep;
            bad |= nonfinite_halves(vf[j][t]);
          }
        }
        // A weight of 0 does not hide an infinity or NaN from the rows that
        // do not see it (0 times infinity). Such values are taken out here, and
        // what they add is kept apart, in this wave's rows of `join`.
        const bool apart = w.p_min != w.p_max && __any(bad != 0);
        if (!kSplit && apart) return false;
        if (kSplit && apart) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (!nonfinite)
              for (int d = lane; d < 16 * kRow; d += 64) (&join[nt][wave][0][0])[d] = 0.0f;
            u32x4 sees;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const int ta = t0 + 16 * (t / 2) + 4 * g + 2 * (t % 2);
              sees[t] = kOnes & both(ta <= pos[nt] && ta >= first[nt], ta < pos[nt] && ta + 1 >= first[nt]);
            }
#pragma unroll
            for (int j = 0; j < W; ++j) {
              add_nonfinite(vf[j], sees, &join[nt][wave][col][128 * u + 4 * W * g + j], W);
              __builtin_amdgcn_sched_barrier(0);     // rare: few registers matter more than overlap
            }
          }
#pragma unroll
          for (int j = 0; j < W; ++j)
#pragma unroll
            for (int t = 0; t < 4; ++t) vf[j][t] &= ~spread_top(nonfinite_halves(vf[j][t]));
          nonfinite = true;
        }
      }
#pragma unroll
      for (int j = 0; j < W; ++j)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          o[nt][u * W + j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, vf[j]), p[nt],
                                                                    o[nt][u * W + j], 0, 0, 0);
    }
    if (more) values(step + kFewWaves);
    return true;
  };

  int step;
  auto start = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt] = -INFINITY;
      l[nt] = 0.0f;
#pragma unroll
      for (int j = 0; j < kTiles; ++j) o[nt][j] = float4v{0, 0, 0, 0};
    }
    step = begin + wave;
    if (step < end) {
      look_up(step);
      keys(step);
      values(step);
    }
  };
  auto steps_to = [&](auto kind, int to) __attribute__((always_inline)) -> bool {
    // With nothing pending at its entry (vmcnt 0, the other counters open), a
    // loop's waits are counted from its own loads alone, and leave those of
    // the next step in flight.
    if (step < to) __builtin_amdgcn_s_waitcnt(0x0F70);
    for (; step < to; step += kFewWaves)
      if (!one_step(kind, step)) return false;
    return true;
  };
  start();
  // Steps at the window's start, whole steps, steps at the diagonal: two rounds
  // of whole and then edge steps, so that each kind's code is there once.
  const int whole_lo = (w.lo_max + kStep - 1) / kStep, whole_hi = max((w.p_min + 1) / kStep, whole_lo);
  bool done = true;
  for (int round = 0; round < 2 && done; ++round) {
    steps_to(std::integral_constant<int, kWhole>{}, min(round ? whole_hi : begin, end - kFewWaves));
    done = steps_to(std::integral_constant<int, kEdgeStep>{}, round ? end : min(whole_lo, end));
  }
  if (!done) {
    start();
    steps_to(std::integral_constant<int, kCareful>{}, end);
  }

  // The four waves join. Register r of O^T tile u W + j is element
  // 128 u + 4 W g + W r + j of row col.
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const float sum = sum32(sum16(l[nt]));
    if (g == 0) join_ml[nt][wave][col] = make_float2(m[nt], sum);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int j = 0; j < W; j += 4) {
          float4v* at = reinterpret_cast<float4v*>(&join[nt][wave][col][128 * u + 4 * W * g + W * r + j]);
          float4v v = {o[nt][u * W + j][r], o[nt][u * W + j + 1][r], o[nt][u * W + j + 2][r], o[nt][u * W + j + 3][r]};
          if (nonfinite) v += *at;
          *at = v;
        }
  }
  __syncthreads();
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    // Thread: row t / 16 of the tile, D / 16 elements of it.
    const int row = threadIdx.x >> 4, d0 = (threadIdx.x & 15) * 4;
    const int rr = 16 * nt + row;
    if (rr < w.rows) {
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < kFewWaves; ++i) top = fmaxf(top, join_ml[nt][i][row].x);
      const float base = top == -INFINITY ? 0.0f : top;
      float f[kFewWaves], total = 0.0f;
#pragma unroll
      for (int i = 0; i < kFewWaves; ++i) {
        f[i] = __builtin_amdgcn_exp2f(join_ml[nt][i][row].x - base);
        total += f[i] * join_ml[nt][i][row].y;
      }
      const int tok = (w.row0 + rr) / group, h = head * group + (w.row0 + rr) % group;
      const int pr = w.len - w.n + tok, fr = first_seen(pr, a.window);
      const int64_t out_row = (int64_t)(w.q0 + tok) * a.q_heads + h;
      const float inv = pr < fr ? 0.0f : 1.0f / total;
#pragma unroll
      for (int d = 0; d < D / 64; ++d) {
        float4v v = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < kFewWaves; ++i) {
          const float4v x = *reinterpret_cast<const float4v*>(&join[nt][i][row][d * 64 + d0]);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] += f[i] * x[e];
        }
        if (alone) {
          half4 y;
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = (_Float16)(pr < fr ? 0.0f : v[e] * inv);
          *reinterpret_cast<half4*>(a.out + out_row * D + d * 64 + d0) = y;
        } else {
          *reinterpret_cast<float4v*>(part.o + (part_row0 + rr) * D + d * 64 + d0) = v;
        }
      }
      if (!alone && d0 == 0) {
        // A range that the row sees part of, all of it at -infinity, is not an empty one.
        const bool sees = max(fr, begin * kStep) <= min(pr, end * kStep - 1);
        part.ml[part_row0 + rr] = make_float2(top == -INFINITY && sees ? kLowest : top, total);
      }
    }
  }

  at += taken;
  if (at >= stop) break;
  slot = 1;                    // a second partial result is the span's end
  i0 = 0;
  if (++tile == it.tiles) {
    do {
      sequence(a, c, w.b + 1, w);
      it = few_item(a, plan, group, w);
    } while (it.tiles == 0);
    tile = 0;
  }
  __syncthreads();             // the join's rows have been read
  }
}

template <int D, int B>
hipError_t launch_few(const qlinear_kv_cache& c, const AttentionArgs& a, const Plan& p, const Partials& part,
                      hipStream_t stream) {
  const int group = a.q_heads / c.kv_heads;
  const int64_t most = (int64_t)a.max_q_len * group;
  const int tiles = (int)(((most < p.max_rows ? most : p.max_rows) + p.rows - 1) / p.rows);
  const int workgroups = p.whole * a.batch > p.workers ? p.whole * a.batch : p.workers;
  const dim3 grid = p.workers ? dim3((unsigned)(c.kv_heads * workgroups))
                              : dim3((unsigned)(c.kv_heads * tiles), (unsigned)a.batch);
  // One tile per sequence and key/value head reads each cache row once, more of
  // them share it through L2 (both sides measured, cold: 64 sequences of 2048
  // tokens, 64/8 heads, one tile 98.2 us with plain loads, 87.4 us past the
  // caches; 8 of 8192 with 7 new tokens each, two tiles, 69.3 and 76.7 us).
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(64 * kFewWaves), 0, stream, a, c, p, part);
    return hipGetLastError();
  };
  if (p.rows == 16)
    return tiles == 1 ? go(attention_few_kernel<D, B, 1, true>) : go(attention_few_kernel<D, B, 1, false>);
  if constexpr (D < 256)
    return tiles == 1 ? go(attention_few_kernel<D, B, 2, true>) : go(attention_few_kernel<D, B, 2, false>);
  return hipErrorInvalidValue;      // no plan has more rows for 256 wide heads
}

template <int D>
hipError_t launch_few_width(const qlinear_kv_cache& c, const AttentionArgs& a, const Plan& p, const Partials& part,
                            hipStream_t stream) {
  if (c.bits == 16) return launch_few<D, 16>(c, a, p, part, stream);
  if (c.bits == 8) return launch_few<D, 8>(c, a, p, part, stream);
  if (c.bits == 6) return launch_few<D, 6>(c, a, p, part, stream);
  return launch_few<D, 4>(c, a, p, part, stream);
}

}  // namespace attn
}  // namespace qlinear
