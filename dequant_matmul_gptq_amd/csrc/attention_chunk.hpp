// Attention for many query rows per key/value head (prompts and chunks of
// them): bound by the matrix cores and the exponentials. A workgroup takes
// 128 (token, head of the group) rows of one sequence and key/value head, 32
// to a wave, and goes over the tokens they see in steps of 64 (32 at D = 256,
// where two steps of 64 would not leave room for a second workgroup in LDS).
//
// A step's keys and values are staged in LDS as float16 [token][D], two steps
// deep, with one barrier per step: the next step's are asked for before this
// one is multiplied (float16: straight from memory to LDS; quantized: through
// registers, dequantized by all waves together after this step's products).
// The barrier does not wait for loads to LDS, so each wave waits for its own
// before it. At D = 64 and 128 the compiler waits for them already before this
// step's first LDS read, so that there a second workgroup on the CU covers
// their latency, not this one's products. The 32 x 32 x 16 products:
//   - S^T = K Q^T: keys are rows (A: 16-byte LDS reads), q stays in registers.
//     Accumulator register r of lane (n, h) = (l % 32, l / 32) is token
//     8 (r / 4) + 4 h + r % 4 and query row n.
//   - O^T = V^T P^T: P^T is S^T's registers in order, so fragment element
//     8 h + i of a 16-token chunk is token 8 (i / 4) + 4 h + i % 4: V^T's
//     fragments are two transposing LDS reads of four tokens each.
// 16-byte pieces of a row sit at places exclusive-or-ed with the row number,
// so that the lanes of one LDS cycle hit different banks.
//
// Measured: a prompt of 8192 tokens, 64/8 heads of 128, float16: 1160 us, 948
// TFLOP/s of the visible pairs, 72% of what a library product of 8192 cubed
// reaches when warm (1325). Its cycles are half matrix products, half softmax
// and waits, those for the next step's rows (see above) among them, at a clock
// that the power limit holds near 1.8 GHz: the same call on zeros takes 870 us.
// Tiles of 32 tokens with the next one's products in between this one's
// exponentials, ordered by hand, took as many cycles (1160 to 1190 us). 511
// tokens at 16384 over Q8, 40/40 heads: 235 us, 15 of them the join; its
// unpacking is hidden (a third fewer instructions there changed nothing). 4096
// tokens of 16/4 heads of 256, one workgroup per CU by its registers (32 to 57 of
// them spilled, outside the loops of whole steps but for one): 258 us, 533
// TFLOP/s; over Q8 / Q6 / Q4 242, 268, 255 us.
#pragma once

#include <type_traits>

#include "attention.hpp"

namespace qlinear {
namespace attn {

constexpr int kChunkThreads = 256;
constexpr int kAheadK = 6, kAheadV = 4;     // fragments read ahead of the products

// The place of 16-byte piece x of row `row`. Keys are read eight rows of one
// piece in a cycle. Values are read four rows of 64 neighbouring bytes, and
// unpacked codes stored as four rows of pieces four apart: both groups of four
// pieces and the pieces in them are exchanged (groups alone: 4 stores on one
// bank, 511 tokens at 16384 over Q8 254 us instead of 247).
template <int D>
__device__ __forceinline__ int key_piece(int row, int x) {
  return D == 64 ? x ^ ((row >> 1) & 7) : x ^ (row & 15);
}
template <int D>
__device__ __forceinline__ int value_piece(int row, int x) {
  return D == 64 ? x ^ ((row >> 1) & 1) * 5 : x ^ (row & 3) * 5;
}

// Element order inside 8 neighbouring ones as codes unpack: place e holds
// element order(e). 4 and 6 bits unpack pairs four elements apart.
template <int B>
__device__ __forceinline__ constexpr int unpacked(int e) {
  return B == 4 || B == 6 ? e / 2 + 4 * (e % 2) : e;
}

// Eight codes (B words / 4) to eight values in unpacking order.
template <int B>
__device__ __forceinline__ u32x4 decode8(uint32_t a, uint32_t b, half2v s) {
  u32x4 r;
  if constexpr (B == 8) {
    r[0] = as_u32(code_pair<8>(__builtin_amdgcn_perm(0u, a, 0x0C010C00u), s));
    r[1] = as_u32(code_pair<8>(__builtin_amdgcn_perm(0u, a, 0x0C030C02u), s));
    r[2] = as_u32(code_pair<8>(__builtin_amdgcn_perm(0u, b, 0x0C010C00u), s));
    r[3] = as_u32(code_pair<8>(__builtin_amdgcn_perm(0u, b, 0x0C030C02u), s));
  } else if constexpr (B == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = as_u32(code_pair<4>((a >> (4 * i)) & 0x000F000Fu, s));
  } else {   // 48 bits in a and the low half of b: windows at bits 0 / 24 and 12 / 36
    const uint32_t x = lo_halves(a, __builtin_amdgcn_alignbit(b, a, 24));
    const uint32_t y = lo_halves(a >> 12, b >> 4);
    r[0] = as_u32(code_pair<6>(x & 0x003F003Fu, s));
    r[1] = as_u32(code_pair<6>((x >> 6) & 0x003F003Fu, s));
    r[2] = as_u32(code_pair<6>(y & 0x003F003Fu, s));
    r[3] = as_u32(code_pair<6>((y >> 6) & 0x003F003Fu, s));
  }
  return r;
}

// Scheduling of a run of N matrix products fed by R LDS reads each: `Ahead`
// products' reads first, then one product for every further R reads.
template <int N, int R, int Ahead>
__device__ __forceinline__ void feed_ahead() {
  constexpr int kMfma = 0x8, kDsRead = 0x100;
  __builtin_amdgcn_sched_group_barrier(kDsRead, R * Ahead, 0);
#pragma unroll
  for (int i = 0; i < N - Ahead; ++i) {
    __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
    __builtin_amdgcn_sched_group_barrier(kDsRead, R, 0);
  }
  __builtin_amdgcn_sched_group_barrier(kMfma, Ahead, 0);
}

template <int D, int B>
struct ChunkShape {
  static constexpr int T = chunk_step(D);              // tokens of a step
  static constexpr int kPieces = D / 8;                // 16-byte pieces of a row
  static constexpr int kRun = T * D / kChunkThreads;   // elements of a row a thread dequantizes
  static constexpr int kRunWords = B == 16 ? 1 : kRun * B / 32;
};

template <int D, int B>
__global__ __launch_bounds__(kChunkThreads, D == 256 ? 1 : 2) void attention_chunk_kernel(AttentionArgs a,
                                                                                          qlinear_kv_cache c,
                                                                                          Plan plan, Partials part) {
  typedef ChunkShape<D, B> Sh;
  constexpr int T = Sh::T, kKeyTiles = T / 32, kFrags = D / 16, kOutTiles = D / 32;
  __shared__ __attribute__((aligned(16))) uint16_t ks[2][T * D];
  __shared__ __attribute__((aligned(16))) uint16_t vs[2][T * D];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n32 = lane & 31, h = lane >> 5;
  const int group = a.q_heads / c.kv_heads;
  const int head = blockIdx.x % c.kv_heads, split = blockIdx.y;
  const int page_shift = __builtin_ctz(c.page_size);
  const int group_shift = B == 16 ? 0 : __builtin_ctz(c.group);

  // Later rows see more tokens: they start first.
  Work w;
  int tile = 0;
  if (!find_tile(a, c, plan, group, (gridDim.x - 1 - blockIdx.x) / c.kv_heads, w, tile)) return;
  row_tile(a, group, tile * kChunkRows, kChunkRows, w);
  const int step_lo = w.lo_min / T;
  const int step_end = w.p_max < 0 ? 0 : w.p_max / T + 1;
  const int begin = step_lo + split * plan.chunk;
  const int end = split == plan.splits - 1 ? step_end : min(begin + plan.chunk, step_end);
  if (begin >= end && plan.splits > 1) {   // nothing in this range
    for (int r = threadIdx.x; r < w.rows; r += kChunkThreads) {
      const int rr = w.row0 + r;
      part.ml[split * part.rows + (int64_t)(w.q0 + rr / group) * a.q_heads + head * group + rr % group] =
          make_float2(-INFINITY, 0.0f);
    }
    return;
  }

  // This lane's query row, and what the wave's rows see.
  const int row = 32 * wave + n32;
  const bool live = row < w.rows;
  const int rr = w.row0 + (live ? row : 0);
  const int tok = rr / group, qh = head * group + rr - tok * group;
  const int pos = w.len - w.n + tok, first = first_seen(pos, a.window);
  const int64_t out_row = (int64_t)(w.q0 + tok) * a.q_heads + qh;
  const int wr0 = w.row0 + 32 * wave, wr1 = w.row0 + min(32 * wave + 31, w.rows - 1);
  const int wp_max = w.len - w.n + wr1 / group, wlo_min = first_seen(w.len - w.n + wr0 / group, a.window);

  half8 q[kFrags];
  {
    const uint16_t* p = a.q + (w.q0 + tok) * a.q_stride + (int64_t)qh * D + 8 * h;
    // The kernel's scale is positive: a negative one turns q, 0 makes it 0 (NaN
    // where it is not finite).
    const uint32_t flip = a.scale < 0.0f ? kTops : 0u, keep = a.scale == 0.0f ? 0u : ~0u;
#pragma unroll
    for (int f = 0; f < kFrags; ++f) {
      u32x4 v = *reinterpret_cast<const u32x4*>(p + 16 * f);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = ((v[e] ^ flip) & keep) | (spread_top(nonfinite_halves(v[e])) & ~keep);
      const half8 x = __builtin_bit_cast(half8, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) q[f][e] = x[unpacked<B>(e)];
    }
  }
  const float slack = 8.0f / (a.scale == 0.0f ? 1.0f : fabsf(a.scale) * kLog2e);
  const float sc = a.scale == 0.0f ? 1.0f : fabsf(a.scale) * kLog2e;

  const PageTable table = page_table(a, w.b);
  const int last_page = max(w.len - 1, 0) >> page_shift;

  // ---- staging
  typedef __attribute__((address_space(3))) uint16_t* Lds;
  typedef __attribute__((address_space(3))) u32x4* Lds4;
  // float16: a wave brings in every fourth 1024-byte group of rows, each lane
  // the 16 bytes whose place in LDS is its own. The groups' pages are looked
  // up a step ahead.
  constexpr int kGroupRows = 1024 / (2 * D), kGroups = T / kGroupRows / 4;
  int pages[kGroups];
  auto look_up = [&](int step) {
    if constexpr (B == 16)
#pragma unroll
      for (int i = 0; i < kGroups; ++i)
        pages[i] = page_of(c, table, page_shift, last_page, step * T + (4 * i + wave) * kGroupRows);
  };
  auto stage_direct = [&](int step, Lds kn, Lds vn) {
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const int r0 = (4 * i + wave) * kGroupRows;
      const int64_t pool = pool_row(c, pages[i], page_shift, head, step * T + r0) * D;
      // lane's row and piece in LDS order
      const int r = r0 + lane / Sh::kPieces, x = lane % Sh::kPieces;
      typedef const __attribute__((address_space(1))) void* gptr;
      typedef __attribute__((address_space(3))) void* lptr;
      const int in = (lane / Sh::kPieces) * D;
      __builtin_amdgcn_global_load_lds((gptr)((const uint16_t*)c.k + pool + in + key_piece<D>(r, x) * 8),
                                       (lptr)(kn + r0 * D), 16, 0, 0);
      __builtin_amdgcn_global_load_lds((gptr)((const uint16_t*)c.v + pool + in + value_piece<D>(r, x) * 8),
                                       (lptr)(vn + r0 * D), 16, 0, 0);
    }
  };
  // Quantized: a thread takes kRun neighbouring elements of one token.
  uint32_t kw[Sh::kRunWords], vw[Sh::kRunWords];
  uint16_t kscale = 0, vscale = 0;
  constexpr int kPerRow = D / Sh::kRun;
  const int my_row = threadIdx.x / kPerRow, my_run = threadIdx.x % kPerRow;
  auto fetch = [&](int step) {
    if constexpr (B != 16) {
      const int t = step * T + my_row;
      const int64_t pool = pool_row(c, page_of(c, table, page_shift, last_page, t), page_shift, head, t);
      const uint32_t* kp = (const uint32_t*)c.k + pool * (D * B / 32) + my_run * Sh::kRunWords;
      const uint32_t* vp = (const uint32_t*)c.v + pool * (D * B / 32) + my_run * Sh::kRunWords;
#pragma unroll
      for (int i = 0; i < Sh::kRunWords; ++i) {
        kw[i] = kp[i];
        vw[i] = vp[i];
      }
      const int64_t at = pool * (D >> group_shift) + ((my_run * Sh::kRun) >> group_shift);
      kscale = c.k_scales[at];
      vscale = c.v_scales[at];
    }
  };
  auto unpack = [&](Lds kn, Lds vn) {
    if constexpr (B != 16) {
      const _Float16 sk = __builtin_bit_cast(_Float16, kscale), sv = __builtin_bit_cast(_Float16, vscale);
#pragma unroll
      for (int i = 0; i < Sh::kRun / 8; ++i) {
        uint32_t ka, kb = 0, va, vb = 0;
        if constexpr (B == 4) {
          ka = kw[i];
          va = vw[i];
        } else if constexpr (B == 8) {
          ka = kw[2 * i];
          kb = kw[2 * i + 1];
          va = vw[2 * i];
          vb = vw[2 * i + 1];
        } else {
          const int o = i / 2 * 3;     // 48 bits at bit 0 or 48 of three words
          ka = i % 2 ? __builtin_amdgcn_alignbit(kw[o + 2], kw[o + 1], 16) : kw[o];
          kb = i % 2 ? kw[o + 2] >> 16 : kw[o + 1];
          va = i % 2 ? __builtin_amdgcn_alignbit(vw[o + 2], vw[o + 1], 16) : vw[o];
          vb = i % 2 ? vw[o + 2] >> 16 : vw[o + 1];
        }
        const int x = my_run * (Sh::kRun / 8) + i;
        *(Lds4)(kn + my_row * D + key_piece<D>(my_row, x) * 8) = decode8<B>(ka, kb, half2v{sk, sk});
        *(Lds4)(vn + my_row * D + value_piece<D>(my_row, x) * 8) = decode8<B>(va, vb, half2v{sv, sv});
      }
    }
  };

  // V^T fragment of 16-token chunk cc, 32-element tile dt: lane (d = l % 32)
  // gets tokens 16 cc + 4 h + 0 .. 3 and + 8 of element 32 dt + d.
  auto value_fragment = [&](Lds vc, int cc, int dt) {
    typedef short short4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) short4* Lds2;
    const int j = lane & 15, sub = (lane >> 4) & 1;
    const int x = 4 * dt + 2 * sub + (j & 3) / 2;     // 16-byte piece
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 16 * cc + 8 * i + 4 * h + j / 4;
      const short4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (Lds2)(vc + t * D + value_piece<D>(t, x) * 8 + (j & 1) * 4));
      const u32x2 u = __builtin_bit_cast(u32x2, v);
      r[2 * i] = u[0];
      r[2 * i + 1] = u[1];
    }
    return r;
  };

  float16v o[kOutTiles];
  float m, l;

  // One step: rows in kc, vc; the next step's go to kn, vn, which are apart (restrict).
  // kind: see StepKind. False: an edge step has infinities or NaN that only
  // some rows see.
  auto one_step = [&](auto kind, int step, Lds __restrict__ kc, Lds __restrict__ vc, Lds __restrict__ kn,
                      Lds __restrict__ vn) __attribute__((always_inline)) -> bool {
    constexpr bool kSplit = decltype(kind)::value == kCareful;
    const int t0 = step * T;
    constexpr bool kEdge = decltype(kind)::value == kEdgeStep || kSplit;
    if (decltype(kind)::value != kGrow && step + 1 < end) {
      if constexpr (B == 16) {
        stage_direct(step + 1, kn, vn);
        look_up(step + 2);
      } else {
        fetch(step + 1);
      }
    }

    bool nonfinite = false;
    if constexpr (kEdge) {
      // Values of tokens that no row sees may be anything: zero. A weight of
      // 0 does not hide an infinity or NaN of a token that only some rows see.
      uint32_t bad = 0;
      for (int i = threadIdx.x; i < T * D / 8; i += kChunkThreads) {
        const int t = t0 + i / Sh::kPieces;
        const Lds4 at = (Lds4)(vc + i * 8);
        if (t > w.p_max || t < w.lo_min) {
          *at = u32x4{0, 0, 0, 0};
        } else {
          const u32x4 v = *at;
#pragma unroll
          for (int e = 0; e < 4; ++e) bad |= nonfinite_halves(v[e]);
        }
      }
      nonfinite = __syncthreads_or(bad != 0) && w.p_min != w.p_max;
      if (!kSplit && nonfinite) return false;
    }

    const bool active = !kEdge || (t0 <= wp_max && t0 + T - 1 >= wlo_min);
    half8 p[T / 16];
    if (active) {
      float16v s[kKeyTiles];
#pragma unroll
      for (int k = 0; k < kKeyTiles; ++k)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[k][r] = 0.0f;
#pragma unroll
      for (int f = 0; f < kFrags; ++f)
#pragma unroll
        for (int k = 0; k < kKeyTiles; ++k) {
          const int key = 32 * k + n32;
          const half8 kf = __builtin_bit_cast(half8, *(Lds4)(kc + key * D + key_piece<D>(key, 2 * f + h) * 8));
          s[k] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, q[f], s[k], 0, 0, 0);
        }
      feed_ahead<kFrags * kKeyTiles, 1, kAheadK>();
      __builtin_amdgcn_sched_barrier(0);

      if constexpr (kEdge) {
#pragma unroll
        for (int k = 0; k < kKeyTiles; ++k)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int t = t0 + 32 * k + 8 * (r / 4) + 4 * h + r % 4;
            if (t > pos || t < first) s[k][r] = -INFINITY;
          }
      }
      float mx = s[0][0];
#pragma unroll
      for (int k = 0; k < kKeyTiles; ++k)
#pragma unroll
        for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[k][r]);
      mx = max32(mx);
      if constexpr (decltype(kind)::value == kWhole) {
        if (__any(mx > m + slack)) return false;
      } else {
        const float mn = fmaxf(m, mx);
        const float alpha = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m * sc - mn * sc);
        m = mn;
        l *= alpha;
#pragma unroll
        for (int d = 0; d < kOutTiles; ++d)
#pragma unroll
          for (int r = 0; r < 16; ++r) o[d][r] *= alpha;
      }
      const float base = m == -INFINITY ? 0.0f : m * sc;
      float sum = 0.0f;
#pragma unroll
      for (int k = 0; k < kKeyTiles; ++k)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float e = __builtin_amdgcn_exp2f(s[k][r] * sc - base);
          sum += e;
          p[2 * k + r / 8][r % 8] = (_Float16)e;
        }
      l += sum;
    }

    if (kSplit && nonfinite) {
      // What infinities and NaN add to the rows that see them: counts of
      // tokens with +infinity or NaN, and with -infinity or NaN, from the
      // same product with weights of 1. Then they are taken out of LDS.
      if (active) {
#pragma unroll 1
        for (int cc = 0; cc < T / 16; ++cc) {
          u32x4 sees;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = t0 + 16 * cc + 8 * (i / 2) + 4 * h + 2 * (i % 2);
            sees[i] = kOnes & both(t <= pos && t >= first, t < pos && t + 1 >= first);
          }
#pragma unroll
          for (int d = 0; d < kOutTiles; ++d) {
            const u32x4 v = value_fragment(vc, cc, d);
            u32x4 up, down;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t any = nonfinite_halves(v[i]), nan = nan_halves(v[i]);
              up[i] = ones_at((any & ~v[i]) | nan);
              down[i] = ones_at((any & v[i]) | nan);
            }
            float16v zero;
#pragma unroll
            for (int r = 0; r < 16; ++r) zero[r] = 0.0f;
            const half8 b8 = __builtin_bit_cast(half8, sees);
            const float16v nu = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, up), b8, zero, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 16; ++r) o[d][r] += nu[r] > 0.0f ? INFINITY : 0.0f;
            const float16v nd =
                __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, down), b8, zero, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 16; ++r) o[d][r] -= nd[r] > 0.0f ? INFINITY : 0.0f;
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < T * D / 8; i += kChunkThreads) {
        const Lds4 at = (Lds4)(vc + i * 8);
        u32x4 v = *at;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] &= ~spread_top(nonfinite_halves(v[e]));
        *at = v;
      }
      __syncthreads();
    }

    if (active) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int cc = 0; cc < T / 16; ++cc)
#pragma unroll
        for (int d = 0; d < kOutTiles; ++d)
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, value_fragment(vc, cc, d)), p[cc],
                                                        o[d], 0, 0, 0);
      feed_ahead<T / 16 * kOutTiles, 2, kAheadV>();
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (B != 16) {
      if (step + 1 < end) unpack(kn, vn);
    }
    return true;
  };

  auto start = [&]() {
#pragma unroll
    for (int d = 0; d < kOutTiles; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[d][r] = 0.0f;
    m = -INFINITY;
    l = 0.0f;
    if (begin >= end) return;
    look_up(begin);
    if constexpr (B == 16) {
      stage_direct(begin, (Lds)ks[0], (Lds)vs[0]);
      look_up(begin + 1);
    } else {
      fetch(begin);
      unpack((Lds)ks[0], (Lds)vs[0]);
    }
  };
  int step = begin, buf = 0;
  // Everyone's rows are in LDS and nobody reads the others any more. A barrier
  // does not wait for loads from memory to LDS, so each wave waits for its own
  // first (vmcnt 0, the other counters open); the compiler's waits are for its
  // own reads alone, and not at every width.
  auto meet = [&]() __attribute__((always_inline)) {
    if constexpr (B == 16) {
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0x0F70);
    }
    __syncthreads();
  };
  // Steps of one kind up to `to`; each turns the buffers.
  auto steps_to = [&](auto kind, int to) __attribute__((always_inline)) -> bool {
    while (step < to) {
      for (; step < to; ++step, buf ^= 1) {
        meet();
        if (!one_step(kind, step, (Lds)ks[buf], (Lds)vs[buf], (Lds)ks[buf ^ 1], (Lds)vs[buf ^ 1])) break;
      }
      if constexpr (decltype(kind)::value == kWhole) {
        if (step < to) {
          one_step(std::integral_constant<int, kGrow>{}, step, (Lds)ks[buf], (Lds)vs[buf], (Lds)ks[buf ^ 1],
                   (Lds)vs[buf ^ 1]);
          ++step;
          buf ^= 1;
        }
      } else {
        return step == to;
      }
    }
    return true;
  };
  start();
  bool done = true;
  // Steps at the window's start, whole steps, steps at the diagonal: two rounds
  // of whole and then edge steps, so that each kind's code is there once.
  const int whole_lo = (w.lo_max + T - 1) / T, whole_hi = max((w.p_min + 1) / T, whole_lo);
  for (int round = 0; round < 2 && done; ++round) {
    steps_to(std::integral_constant<int, kWhole>{}, min(round ? whole_hi : begin, end));
    done = steps_to(std::integral_constant<int, kEdgeStep>{}, round ? end : min(whole_lo, end));
  }
  if (!done) {
    meet();                // the staging under way ends before the first step's starts again
    step = begin;
    buf = 0;
    start();
    steps_to(std::integral_constant<int, kCareful>{}, end);
  }

  // Register r of tile d is element 32 d + 8 (r / 4) + 4 h + r % 4 as stored.
  l = sum32(l);
  if (!live) return;
  const bool none = pos < first;     // sees no token
  if (plan.splits == 1) {
    const float inv = 1.0f / l;
    uint16_t* out = a.out + out_row * D;
#pragma unroll
    for (int d = 0; d < kOutTiles; ++d)
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        half4 y;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = (_Float16)(none ? 0.0f : o[d][r + e] * inv);
        const int at = 32 * d + 2 * r + 4 * h;
        if constexpr (unpacked<B>(1) == 1) {
          *reinterpret_cast<half4*>(out + at) = y;
        } else {
          // places 4 h .. + 3 of the 8 hold elements 2 h, 2 h + 4, 2 h + 1, 2 h + 5
          const int base8 = 32 * d + 2 * r;
          *reinterpret_cast<half2v*>(out + base8 + 2 * h) = half2v{y[0], y[2]};
          *reinterpret_cast<half2v*>(out + base8 + 2 * h + 4) = half2v{y[1], y[3]};
        }
      }
  } else {
    float* out = part.o + (split * part.rows + out_row) * D;
#pragma unroll
    for (int d = 0; d < kOutTiles; ++d)
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        const int base8 = 32 * d + 2 * r;
        if constexpr (unpacked<B>(1) == 1) {
          *reinterpret_cast<float4v*>(out + base8 + 4 * h) = float4v{o[d][r], o[d][r + 1], o[d][r + 2], o[d][r + 3]};
        } else {
          *reinterpret_cast<float2*>(out + base8 + 2 * h) = make_float2(o[d][r], o[d][r + 2]);
          *reinterpret_cast<float2*>(out + base8 + 2 * h + 4) = make_float2(o[d][r + 1], o[d][r + 3]);
        }
      }
    if (h == 0) {
      // A range that the row sees part of, all of it at -infinity, is not an empty one.
      const bool sees = max(first, begin * T) <= min(pos, end * T - 1);
      part.ml[split * part.rows + out_row] = make_float2(m == -INFINITY ? (sees ? kLowest : m) : m * sc, l);
    }
  }
}

template <int D, int B>
hipError_t launch_chunk(const qlinear_kv_cache& c, const AttentionArgs& a, const Plan& p, const Partials& part,
                        hipStream_t stream) {
  const int group = a.q_heads / c.kv_heads;
  // Key/value heads are neighbours in the grid: with 8 of them (or a multiple)
  // one XCD's L2 sees the keys and values of its own heads only.
  const dim3 grid((unsigned)(chunk_tiles(a, group) * c.kv_heads), (unsigned)p.splits);
  hipLaunchKernelGGL((attention_chunk_kernel<D, B>), grid, dim3(kChunkThreads), 0, stream, a, c, p, part);
  return hipGetLastError();
}

template <int D>
hipError_t launch_chunk_width(const qlinear_kv_cache& c, const AttentionArgs& a, const Plan& p, const Partials& part,
                              hipStream_t stream) {
  if (c.bits == 16) return launch_chunk<D, 16>(c, a, p, part, stream);
  if (c.bits == 8) return launch_chunk<D, 8>(c, a, p, part, stream);
  if (c.bits == 6) return launch_chunk<D, 6>(c, a, p, part, stream);
  return launch_chunk<D, 4>(c, a, p, part, stream);
}

}  // namespace attn
}  // namespace qlinear
