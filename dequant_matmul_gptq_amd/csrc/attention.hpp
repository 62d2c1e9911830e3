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
#pragma once

#include "qlinear_kernels.hpp"

namespace qlinear {
namespace attn {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef float float16v __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -3.4028234663852886e38f;

// The launch's plan: row tiles of `rows` (token, head of the group) pairs,
// each tile's visible tokens cut into `splits` ranges of `chunk` steps of
// kStep tokens (the last range takes what is left).
struct Plan {
  int rows;
  int splits;
  int chunk;
};
constexpr int kStep = 32;

// Partial results of a split call: o [splits][tokens * q_heads][D] and
// (m, l) [splits][tokens * q_heads], float32.
struct Partials {
  float* o;
  float2* ml;
};

// One workgroup's sequence, row tile and token range.
struct Work {
  int b;             // sequence
  int q0, n;         // first row of q, new tokens
  int len;           // cached tokens
  int row0, rows;    // first row of the tile among n * group, rows in it
  int p_min, p_max;  // positions of the tile's first and last token
  int lo_min, lo_max;  // first tokens they see
};

// Sequence b's rows and length, bounded by what the buffers hold.
__device__ __forceinline__ void sequence(const AttentionArgs& a, const qlinear_kv_cache& c, int b, Work& w) {
  w.b = b;
  if (a.q_start) {
    const int q0 = max(a.q_start[b], 0), q1 = min(a.q_start[b + 1], a.tokens);
    w.q0 = q0;
    w.n = max(q1 - q0, 0);
  } else {
    w.n = a.tokens / a.batch;
    w.q0 = b * w.n;
  }
  const int64_t cap = (int64_t)a.table_width * c.page_size;
  w.len = (int)min((int64_t)max(a.kv_len[b], 0), cap);
}

__device__ __forceinline__ int first_seen(int p, int window) { return window > 0 ? max(0, p - window + 1) : 0; }

// The tile of `tile_rows` rows from row0 on (group rows per token).
__device__ __forceinline__ void row_tile(const AttentionArgs& a, int group, int row0, int tile_rows, Work& w) {
  w.row0 = row0;
  w.rows = min(tile_rows, w.n * group - row0);
  w.p_min = w.len - w.n + row0 / group;
  w.p_max = w.len - w.n + (row0 + w.rows - 1) / group;
  w.lo_min = first_seen(w.p_min, a.window);
  w.lo_max = first_seen(w.p_max, a.window);
}

// First pool row of token slot t's 16-token tile (t a multiple of 16): page
// numbers are taken into the pool and table places to the sequence's last.
__device__ __forceinline__ int64_t tile_row(const AttentionArgs& a, const qlinear_kv_cache& c, const int32_t* table,
                                            int page_shift, int last_page, int head, int t) {
  const int pg = min(max(table[min(t >> page_shift, last_page)], 0), c.num_pages - 1);
  return (((int64_t)pg * c.kv_heads + head) << page_shift) + (t & (c.page_size - 1));
}

// Maximum and sum over the four lanes l % 16 == c (l / 16 = 0 .. 3).
__device__ __forceinline__ float swap16(float v) { return __shfl_xor(v, 16); }
__device__ __forceinline__ float swap32(float v) { return __shfl_xor(v, 32); }

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

// Launchers, one file per head width (see paged_attention.hip).
hipError_t launch_attention_few_64(const qlinear_kv_cache& c, const AttentionArgs& a, const attn::Plan& p,
                                   const attn::Partials& part, hipStream_t stream);
hipError_t launch_attention_few_128(const qlinear_kv_cache& c, const AttentionArgs& a, const attn::Plan& p,
                                    const attn::Partials& part, hipStream_t stream);
hipError_t launch_attention_few_256(const qlinear_kv_cache& c, const AttentionArgs& a, const attn::Plan& p,
                                    const attn::Partials& part, hipStream_t stream);

}  // namespace qlinear
