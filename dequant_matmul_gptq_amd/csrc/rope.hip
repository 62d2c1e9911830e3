// Rotary positions, alone or with the append to a paged cache. Pair (a, b) of
// a head turns by the token's angle: (a c - b s, b c + a s), (c, s) from a
// float32 table. Each product and the sum is rounded once (no fused
// multiply-add), so that the result, and with it the codes of a quantized
// cache, is the same wherever the formula is computed in float32.
//
// HBM-bound at many tokens, launch latency at few. A lane holds 8 elements of
// a head (16-byte accesses), a row's D / 8 lanes are neighbours in one wave,
// and in the half layout each also loads its partner's 8 elements (the same
// cache lines). A thread goes over several heads of one token, so that the
// table's row is read once for them. A wave reads all of its rows' elements
// before it writes any, so a row may be rotated in place. Quantized blocks
// are groups of neighbouring lanes, whose maximum takes lane swaps.
#include <type_traits>

#include "qlinear_kernels.hpp"

namespace qlinear {

namespace {

constexpr int kThreads = 256;

union Half8 {
  uint4 v;
  uint16_t b[8];
};

// Stores past the caches' allocation: what is written here is more than they
// keep, and the lines they hold for it would be the next kernels' inputs (8192
// tokens of 64/8 heads: 93 us with plain stores, 52 us; followed by their
// attention 1237.5, 1208.5 us; 512 tokens 31.5, 28.8 us; 64 tokens the same).
__device__ __forceinline__ void store_past(uint4* p, const uint4& v) {
  typedef uint32_t u4 __attribute__((ext_vector_type(4)));
  __builtin_nontemporal_store(__builtin_bit_cast(u4, v), reinterpret_cast<u4*>(p));
}

__device__ __forceinline__ float half_value(uint16_t b) { return (float)__builtin_bit_cast(_Float16, b); }

// The codec's codes and scale of one lane's 8 elements of a block of G (see
// kv_codec.hip), written to words + the lane's place u.
template <int B, int G>
__device__ __forceinline__ void encode8(const Half8& x, int u, uint32_t* words, uint16_t* scales) {
  // Magnitudes as integers: their order is the float16 order, with NaN on top.
  int m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, (int)(x.b[i] & 0x7FFFu));
#pragma unroll
  for (int k = 1; k < G / 8; k <<= 1) m = max(m, __shfl_xor(m, k));
  constexpr int kHalf = 1 << (B - 1);
  const _Float16 s16 = (_Float16)(half_value((uint16_t)m) / (float)(kHalf - 1));
  const float s = (float)s16;
  uint64_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float r = s > 0.0f ? __builtin_rintf(half_value(x.b[i]) / s) : 0.0f;
    r = fminf(fmaxf(r, (float)-kHalf), (float)(kHalf - 1));
    w |= (uint64_t)(uint32_t)((int)r + kHalf) << (i * B);
  }
  if constexpr (B == 4) {
    words[u] = (uint32_t)w;
  } else if constexpr (B == 8) {
    reinterpret_cast<uint2*>(words)[u] = make_uint2((uint32_t)w, (uint32_t)(w >> 32));
  } else {   // 8 six-bit codes are 6 bytes: 2-byte aligned
    uint16_t* p = reinterpret_cast<uint16_t*>(words) + 3 * u;
    p[0] = (uint16_t)w;
    p[1] = (uint16_t)(w >> 16);
    p[2] = (uint16_t)(w >> 32);
  }
  if (u % (G / 8) == 0) scales[u / (G / 8)] = __builtin_bit_cast(uint16_t, s16);
}

// B: 0 rotates q rows only, 16 appends to a float16 cache, 8 / 6 / 4 to a
// quantized one with blocks of G. Rows of a token: q heads, k heads, v heads.
// H: rows a thread goes over, all of them read before the first is written;
// reads past the last row, or of a partner that is not needed, take an address
// in reach instead of a branch.
template <int B, int G, int H, bool HALF>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a, qlinear_kv_cache c) {
  const int D = a.head_dim, U = D / 8;
  const int lane = threadIdx.x & 63;
  // A cache's head widths are powers of two.
  const int rows_per_wave = B == 0 ? 64 / U : 64 >> __builtin_ctz(U);
  const int in_wave = B == 0 ? lane / U : lane >> __builtin_ctz(U), u = lane - in_wave * U;
  if (in_wave >= rows_per_wave) return;
  const int t = blockIdx.x;
  const int total = B == 0 ? a.q_heads : a.q_heads + 2 * c.kv_heads;
  const int wave = blockIdx.y * (kThreads / 64) + (threadIdx.x >> 6);
  const int row0 = wave * rows_per_wave * H + in_wave;

  const bool rotated = u * 8 < a.rot_dim;
  const int half_units = a.rot_dim / 16;
  const bool low = u < half_units;
  const int partner = !rotated ? u : low ? u + half_units : u - half_units;

  const uint16_t* q = a.q + t * a.q_stride;
  const uint16_t* k = a.k + t * a.k_stride;
  const uint16_t* v = a.v + t * a.v_stride;
  Half8 x[H], o[H];      // the row's 8 elements, and in the half layout their partners
#pragma unroll
  for (int n = 0; n < H; ++n) {
    const int row = min(row0 + n * rows_per_wave, total - 1);
    const uint16_t* src = q + (int64_t)row * D;
    if constexpr (B != 0) {
      const int kv = row - a.q_heads;
      if (kv >= 0) src = kv < c.kv_heads ? k + (int64_t)kv * D : v + (int64_t)(kv - c.kv_heads) * D;
    }
    x[n].v = *reinterpret_cast<const uint4*>(src + u * 8);
    if constexpr (HALF) o[n].v = *reinterpret_cast<const uint4*>(src + partner * 8);
  }

  // (cos, sin) of the lane's pairs: 8 in the half layout, 4 else.
  constexpr int kPairs = HALF ? 8 : 4;
  float cs[2 * kPairs];
  if (rotated) {
    const int p = a.positions[t];
    const bool known = (unsigned)p < (unsigned)a.table_rows;
    const float4* src = reinterpret_cast<const float4*>(a.table + (int64_t)(known ? p : 0) * a.rot_dim) +
                        (HALF ? (low ? u : u - half_units) * 4 : u * 2);
#pragma unroll
    for (int i = 0; i < kPairs / 2; ++i) {
      const float4 w = src[i];
      cs[4 * i] = w.x;
      cs[4 * i + 1] = w.y;
      cs[4 * i + 2] = w.z;
      cs[4 * i + 3] = w.w;
    }
#pragma unroll
    for (int i = 0; i < 2 * kPairs; ++i) cs[i] = known ? cs[i] : __builtin_nanf("");
  } else {
#pragma unroll
    for (int i = 0; i < 2 * kPairs; ++i) cs[i] = 0.0f;
  }
  int slot = -1, slots = 0;
  if constexpr (B != 0) {
    slot = a.slots[t];
    slots = c.num_pages * c.page_size;
  }

#pragma unroll
  for (int n = 0; n < H; ++n) {
    const int row = row0 + n * rows_per_wave;
    if (row >= total) break;
    const bool is_q = B == 0 || row < a.q_heads;
    const bool is_v = B != 0 && row >= a.q_heads + c.kv_heads;
    if (rotated && !is_v) {
#pragma clang fp contract(off)
      Half8 r;
      if constexpr (HALF) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p = half_value(x[n].b[i]) * cs[2 * i], s = half_value(o[n].b[i]) * cs[2 * i + 1];
          r.b[i] = __builtin_bit_cast(uint16_t, (_Float16)(p + (low ? -s : s)));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = half_value(x[n].b[2 * i]), s = half_value(x[n].b[2 * i + 1]);
          r.b[2 * i] = __builtin_bit_cast(uint16_t, (_Float16)(p * cs[2 * i] - s * cs[2 * i + 1]));
          r.b[2 * i + 1] = __builtin_bit_cast(uint16_t, (_Float16)(s * cs[2 * i] + p * cs[2 * i + 1]));
        }
      }
      x[n] = r;
    }
    if (is_q) {
      store_past(reinterpret_cast<uint4*>(a.q_out + t * a.out_stride + (int64_t)row * D + u * 8), x[n].v);
    } else if constexpr (B != 0) {
      if ((unsigned)slot >= (unsigned)slots) continue;
      // Row of (page, head, slot in page) in the pools.
      const int head = row - a.q_heads - (is_v ? c.kv_heads : 0);
      const int page = slot >> __builtin_ctz(c.page_size), place = slot & (c.page_size - 1);
      const int64_t r = ((int64_t)page * c.kv_heads + head) * c.page_size + place;
      void* pool = is_v ? c.v : c.k;
      if constexpr (B == 16)
        reinterpret_cast<uint4*>(pool)[r * U + u] = x[n].v;
      else
        encode8<B, G>(x[n], u, reinterpret_cast<uint32_t*>(pool) + r * (D * B / 32),
                      (is_v ? c.v_scales : c.k_scales) + r * (D / G));
    }
  }
}

// ---- with norms of the heads
// A q or k row is first scaled, x^ = x w / sqrt(mean x^2 + eps), its lanes adding
// up the squares by lane moves; then it is rotated as above, in float32, and
// rounded once. In the half layout the partner's x^ comes from its lane instead
// of memory.
//
// Bound by its instructions as much as by memory at many tokens, so: sums and
// products with float16 operands as they are (fused multiply-adds with mixed
// types, whose addend -0 keeps zeros' signs), the hardware's reciprocal root (one
// unit in the last place), 32-bit offsets, partners by DPP moves inside the
// multiplications. 8191 tokens of 64/8 heads of 128: float16 63.5 us, Q8 76.6 (61.0
// and 62.5 without norms); with the partners and their weights loaded, and a
// precise root, 130 and 163.

// Lane moves inside rows of 16 lanes (DPP controls).
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140, kRight8 = 0x128, kLeft4 = 0x104,
              kRight4 = 0x114;
template <int CTRL, int BANKS = 15>
__device__ __forceinline__ float moved(float v, float old = 0.0f) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, old), __builtin_bit_cast(int, v),
                                                               CTRL, 15, BANKS, BANKS == 15));
}
// v of lane l ^ 16.
__device__ __forceinline__ float across16(float v, int lane) {
  const uint32_t x = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  return __builtin_bit_cast(float, (uint32_t)(lane & 16 ? r[0] : r[1]));
}

// Sum over a row's U neighbouring lanes, u the lane's place among them.
template <bool POW2>
__device__ __forceinline__ float row_sum(float v, int lane, int u, int U) {
  if constexpr (POW2) {      // 8, 16 or 32
    v += moved<kXor1>(v);
    v += moved<kXor2>(v);
    v += moved<kMirror8>(v);      // four lanes have the same sum by now, and so on
    if (U > 8) v += moved<kMirror16>(v);
    if (U > 16) v += across16(v, lane);
    return v;
  } else {         // lane u holds the sum of u .. u + 2 k - 1 after a turn
    for (int k = 1; k < U; k <<= 1) {
      const float o = __shfl_down(v, k);
      v += u + k < U ? o : 0.0f;
    }
    return __shfl(v, lane - u);
  }
}

// Rows of a token, threads and H as in rope_kernel.
template <int B, int G, int H, bool HALF>
__global__ __launch_bounds__(kThreads) void norm_rope_kernel(RopeArgs a, qlinear_kv_cache c) {
  const int D = a.head_dim, U = D / 8;
  const int lane = threadIdx.x & 63;
  const int rows_per_wave = B == 0 ? 64 / U : 64 >> __builtin_ctz(U);
  const int in_wave = B == 0 ? lane / U : lane >> __builtin_ctz(U), u = lane - in_wave * U;
  if (in_wave >= rows_per_wave) return;
  const int t = blockIdx.x;
  const int total = B == 0 ? a.q_heads : a.q_heads + 2 * c.kv_heads;
  const int wave = blockIdx.y * (kThreads / 64) + (threadIdx.x >> 6);
  const int row0 = wave * rows_per_wave * H + in_wave;
  const bool rotated = u * 8 < a.rot_dim;
  const int half_units = a.rot_dim / 16;
  const bool low = u < half_units;

  const uint16_t* q = a.q + t * a.q_stride;
  const uint16_t* k = B == 0 ? q : a.k + t * a.k_stride;
  const uint16_t* v = B == 0 ? q : a.v + t * a.v_stride;
  // Rows without a norm, as v's, read themselves for weights; no branches.
  const uint16_t *wq = a.q_norm ? a.q_norm : q, *wk = B != 0 && a.k_norm ? a.k_norm : k;
  const int wq_stride = a.q_norm ? (int)a.q_norm_stride : D, wk_stride = B != 0 && a.k_norm ? (int)a.k_norm_stride : D;
  Half8 x[H], w[H];
#pragma unroll
  for (int n = 0; n < H; ++n) {
    const int row = min(row0 + n * rows_per_wave, total - 1);
    const bool is_q = B == 0 || row < a.q_heads, is_k = !is_q && row < a.q_heads + c.kv_heads;
    const int head = is_q ? row : row - a.q_heads - (is_k ? 0 : c.kv_heads);
    const uint16_t *src = is_q ? q : is_k ? k : v, *p = is_q ? wq : is_k ? wk : v;
    x[n].v = *reinterpret_cast<const uint4*>(src + (unsigned)(head * D + u * 8));
    w[n].v = *reinterpret_cast<const uint4*>(p + (unsigned)(head * (is_q ? wq_stride : is_k ? wk_stride : D) + u * 8));
  }

  // (cos, sin) of the lane's pairs: 8 in the half layout, 4 else; the sine
  // with the sign that the lane's own element has for it.
  constexpr int kPairs = HALF ? 8 : 4;
  float cs[kPairs], sn[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    cs[i] = 1.0f;
    sn[i] = 0.0f;
  }
  if (rotated) {
    const int p = __builtin_amdgcn_readfirstlane(a.positions[t]);
    if ((unsigned)p < (unsigned)a.table_rows) {
      const float4* src = reinterpret_cast<const float4*>(a.table + (int64_t)p * a.rot_dim) +
                          (HALF ? (low ? u : u - half_units) * 4 : u * 2);
#pragma unroll
      for (int i = 0; i < kPairs / 2; ++i) {
        const float4 z = src[i];
        cs[2 * i] = z.x;
        sn[2 * i] = HALF && low ? -z.y : z.y;
        cs[2 * i + 1] = z.z;
        sn[2 * i + 1] = HALF && low ? -z.w : z.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) cs[i] = sn[i] = __builtin_nanf("");
    }
  }
  int slot = -1;
  if constexpr (B != 0) {
    slot = __builtin_amdgcn_readfirstlane(a.slots[t]);
    if ((unsigned)slot >= (unsigned)(c.num_pages * c.page_size)) slot = -1;
  }

  // The weights as loaded: without this the compiler loads their halves one by
  // one where they are used.
#pragma unroll
  for (int n = 0; n < H; ++n) asm("" : "+v"(w[n].v.x), "+v"(w[n].v.y), "+v"(w[n].v.z), "+v"(w[n].v.w));

  float f[H][8];
#pragma unroll
  for (int n = 0; n < H; ++n) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(half_value(x[n].b[i]), half_value(x[n].b[i]), sum);
    const float inv = __builtin_amdgcn_rsqf(__builtin_fmaf(row_sum<B != 0>(sum, lane, u, U), a.per_element, a.eps));
#pragma unroll
    for (int i = 0; i < 8; ++i)
      f[n][i] = __builtin_fmaf(half_value(w[n].b[i]), __builtin_fmaf(half_value(x[n].b[i]), inv, -0.0f), -0.0f);
  }
  if (B != 0 && (!a.q_norm || !a.k_norm)) {
#pragma unroll
    for (int n = 0; n < H; ++n) {
      const bool normed = (row0 + n * rows_per_wave < a.q_heads ? a.q_norm : a.k_norm) != nullptr;
#pragma unroll
      for (int i = 0; i < 8; ++i) f[n][i] = normed ? f[n][i] : half_value(x[n].b[i]);
    }
  }

  float y[H][8];
  if constexpr (HALF) {
    auto turn = [&](auto partner) __attribute__((always_inline)) {
#pragma clang fp contract(off)
#pragma unroll
      for (int n = 0; n < H; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i) y[n][i] = f[n][i] * cs[i] + partner(f[n][i]) * sn[i];
    };
    // Lanes half_units apart exchange their elements.
    const int half = B == 0 ? 0 : half_units;
    if (half == 8)
      turn([](float z) { return moved<kRight8>(z); });
    else if (half == 4)
      turn([](float z) { return moved<kRight4, 10>(z, moved<kLeft4, 5>(z, z)); });
    else if (half == 2)
      turn([](float z) { return moved<kXor2>(z); });
    else if (half == 1)
      turn([](float z) { return moved<kXor1>(z); });
    else if (half == 16)
      turn([&](float z) { return across16(z, lane); });
    else
      turn([&](float z) { return __shfl(z, !rotated ? lane : low ? lane + half_units : lane - half_units); });
  } else {
#pragma clang fp contract(off)
#pragma unroll
    for (int n = 0; n < H; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[n][2 * i] = f[n][2 * i] * cs[i] - f[n][2 * i + 1] * sn[i];
        y[n][2 * i + 1] = f[n][2 * i + 1] * cs[i] + f[n][2 * i] * sn[i];
      }
  }
  if (a.rot_dim < D) {       // 0 times a partner that is not finite is not 0
#pragma unroll
    for (int n = 0; n < H; ++n)
#pragma unroll
      for (int i = 0; i < 8; ++i) y[n][i] = rotated ? y[n][i] : f[n][i];
  }

  int64_t pool_row = 0;      // of (page, head 0, place in the page) in the pools
  if constexpr (B != 0)
    pool_row = (int64_t)(slot >> __builtin_ctz(c.page_size)) * c.kv_heads * c.page_size + (slot & (c.page_size - 1));
#pragma unroll
  for (int n = 0; n < H; ++n) {
    const int row = row0 + n * rows_per_wave;
    if (row >= total) break;
    const bool is_q = B == 0 || row < a.q_heads, is_v = B != 0 && row >= a.q_heads + c.kv_heads;
    Half8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.b[i] = __builtin_bit_cast(uint16_t, (_Float16)y[n][i]);
    if (is_v) r = x[n];
    if (is_q) {
      store_past(reinterpret_cast<uint4*>(a.q_out + t * a.out_stride + (unsigned)(row * D + u * 8)), r.v);
    } else if constexpr (B != 0) {
      if (slot < 0) continue;
      const int head = row - a.q_heads - (is_v ? c.kv_heads : 0);
      const int64_t p = pool_row + (int64_t)head * c.page_size;
      void* pool = is_v ? c.v : c.k;
      if constexpr (B == 16)
        reinterpret_cast<uint4*>(pool)[p * U + u] = r.v;
      else
        encode8<B, G>(r, u, reinterpret_cast<uint32_t*>(pool) + p * (D * B / 32),
                      (is_v ? c.v_scales : c.k_scales) + p * (D / G));
    }
  }
}

template <int B, int G>
hipError_t launch(const RopeArgs& a, const qlinear_kv_cache& c, hipStream_t stream) {
  const int rows_per_group = 64 / (a.head_dim / 8) * (kThreads / 64);
  const int total = B == 0 ? a.q_heads : a.q_heads + 2 * c.kv_heads;
  // One row a thread for few tokens; up to four once there are tokens enough
  // to fill the chip, as many as share a token's rows out evenly.
  int groups = (total + rows_per_group - 1) / rows_per_group, rows = 1;
  if (a.tokens >= 256) {
    groups = (groups + 3) / 4;
    rows = (total + rows_per_group * groups - 1) / (rows_per_group * groups);
  }
  const dim3 grid((unsigned)a.tokens, (unsigned)groups);
  const bool half = a.layout == QLINEAR_ROPE_HALF, norm = a.q_norm || a.k_norm;
  auto go = [&](auto h) {
    constexpr int H = decltype(h)::value;
    auto kernel = norm ? (half ? norm_rope_kernel<B, G, H, true> : norm_rope_kernel<B, G, H, false>)
                       : (half ? rope_kernel<B, G, H, true> : rope_kernel<B, G, H, false>);
    hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, a, c);
    return hipGetLastError();
  };
  if (rows == 1) return go(std::integral_constant<int, 1>{});
  if (rows == 2) return go(std::integral_constant<int, 2>{});
  if (rows == 3) return go(std::integral_constant<int, 3>{});
  return go(std::integral_constant<int, 4>{});
}

template <int B>
hipError_t launch_group(const RopeArgs& a, const qlinear_kv_cache& c, hipStream_t stream) {
  if (c.group == 32) return launch<B, 32>(a, c, stream);
  if (c.group == 64) return launch<B, 64>(a, c, stream);
  return launch<B, 128>(a, c, stream);
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t stream) { return launch<0, 32>(a, qlinear_kv_cache{}, stream); }

hipError_t launch_rope_append(const RopeArgs& a, const qlinear_kv_cache& cache, hipStream_t stream) {
  if (cache.bits == 16) return launch<16, 32>(a, cache, stream);
  if (cache.bits == 8) return launch_group<8>(a, cache, stream);
  if (cache.bits == 6) return launch_group<6>(a, cache, stream);
  return launch_group<4>(a, cache, stream);
}

}  // namespace qlinear
