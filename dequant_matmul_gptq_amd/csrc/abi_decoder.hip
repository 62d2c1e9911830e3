// extern "C" entry points of the operators between a decoder's linear layers
// (paged cache, rotary positions, attention, norm): host-side validation,
// then launches on the caller's stream. Nothing here allocates memory or
// synchronizes.
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "attention.hpp"

namespace {

using namespace qlinear;

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

int hip_status(hipError_t e) { return e == hipSuccess ? QLINEAR_OK : QLINEAR_ERR_HIP; }

constexpr int64_t kMaxSlots = (int64_t)1 << 30;
// Tokens and norm rows are a grid dimension, whose threads must stay below 2^32.
constexpr int kMaxRows = (1 << 22) - 1;
// Query rows of one attention call (a workgroup of 256 threads takes 128 rows
// of a sequence and key/value head, or fewer where a sequence ends).
constexpr int64_t kMaxQueryRows = (int64_t)1 << 29;
// With shared prefixes each row of the output has two results and more in the
// workspace (69 GB of 256 wide heads at this bound), which are numbered in 31 bits.
constexpr int64_t kMaxSharedRows = (int64_t)1 << 25;
// Token slots that a call's block tables name: its steps (32 tokens, four row
// tiles at most) are counted in 32 bits.
constexpr int64_t kMaxTableSlots = (int64_t)1 << 33;

// Logits of one call: with at most kMaxRows rows its parts (16384 elements at
// least where there are several) are a grid below 2^24 workgroups.
constexpr int64_t kMaxLogits = (int64_t)1 << 37;

int check_cache(const qlinear_kv_cache* c) {
  if (!c || !c->k || !c->v || c->num_pages < 1 || c->kv_heads < 1) return QLINEAR_ERR_INVALID_ARGUMENT;
  const int P = c->page_size, D = c->head_dim;
  if (P != 16 && P != 32 && P != 64 && P != 128 && P != 256) return QLINEAR_ERR_UNSUPPORTED;
  if (D != 64 && D != 128 && D != 256) return QLINEAR_ERR_UNSUPPORTED;
  if (c->bits != 16 && c->bits != 8 && c->bits != 6 && c->bits != 4) return QLINEAR_ERR_UNSUPPORTED;
  if ((int64_t)c->num_pages * P > kMaxSlots || c->kv_heads > 4096) return QLINEAR_ERR_UNSUPPORTED;
  if (c->bits != 16) {
    if ((c->group != 32 && c->group != 64 && c->group != 128) || D % c->group != 0) return QLINEAR_ERR_UNSUPPORTED;
    if (!c->k_scales || !c->v_scales) return QLINEAR_ERR_INVALID_ARGUMENT;
    if (!aligned(c->k_scales, 16) || !aligned(c->v_scales, 16)) return QLINEAR_ERR_MISALIGNED;
  }
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return QLINEAR_ERR_MISALIGNED;
  return QLINEAR_OK;
}

// Shape of the rotation (rot_dim == 0 only where the caller allows it).
int check_rotation(int32_t head_dim, int32_t rot_dim, int32_t layout, const int32_t* positions, const float* table,
                   int32_t table_rows) {
  if (layout != QLINEAR_ROPE_HALF && layout != QLINEAR_ROPE_INTERLEAVED) return QLINEAR_ERR_UNSUPPORTED;
  if (head_dim % 16 != 0 || head_dim > 512 || rot_dim % 16 != 0 || rot_dim > head_dim) return QLINEAR_ERR_UNSUPPORTED;
  if (rot_dim == 0) return QLINEAR_OK;
  if (!positions || !table || table_rows < 1) return QLINEAR_ERR_INVALID_ARGUMENT;
  if (!aligned(positions, 4) || !aligned(table, 16)) return QLINEAR_ERR_MISALIGNED;
  return QLINEAR_OK;
}

// A [tokens][heads][head_dim] operand with a token stride.
int check_rows(const void* p, int64_t stride, int32_t heads, int32_t head_dim) {
  if (!p || stride < (int64_t)heads * head_dim) return QLINEAR_ERR_INVALID_ARGUMENT;
  if (stride % 8 != 0) return QLINEAR_ERR_UNSUPPORTED;
  if (!aligned(p, 16)) return QLINEAR_ERR_MISALIGNED;
  return QLINEAR_OK;
}

// Sizes shared by the attention call and its workspace query.
int check_attention(const qlinear_kv_cache* cache, int32_t tokens, int32_t q_heads, int32_t batch, int32_t max_q_len,
                    int32_t max_kv_len, int32_t window) {
  const int st = check_cache(cache);
  if (st != QLINEAR_OK) return st;
  if (tokens < 0 || batch < 0 || q_heads < 1 || max_q_len < 0 || max_kv_len < 0 || window < 0)
    return QLINEAR_ERR_INVALID_ARGUMENT;
  if (q_heads % cache->kv_heads != 0 || q_heads > 65535 || batch > 65535) return QLINEAR_ERR_UNSUPPORTED;
  if ((int64_t)tokens * q_heads > kMaxQueryRows || (int64_t)batch * cache->kv_heads > kMaxQueryRows / 128)
    return QLINEAR_ERR_UNSUPPORTED;
  return QLINEAR_OK;
}

int check_logprob(int32_t rows, int32_t vocab, int32_t logit_bits, int32_t top, LogprobArgs& a) {
  if (rows < 0 || vocab < 1 || top < 0 || top > vocab) return QLINEAR_ERR_INVALID_ARGUMENT;
  if ((logit_bits != 16 && logit_bits != 32) || vocab > QLINEAR_MAX_VOCAB || top > QLINEAR_MAX_TOP ||
      rows > kMaxRows || (int64_t)rows * vocab > kMaxLogits)
    return QLINEAR_ERR_UNSUPPORTED;
  a.rows = rows;
  a.vocab = vocab;
  a.f32 = logit_bits == 32;
  a.top = top;
  return QLINEAR_OK;
}

// The rest of what a call is checked for; `rows` of block tables.
int check_attention_call(const qlinear_kv_cache* cache, const uint16_t* q, int64_t q_stride, int32_t tokens,
                         int32_t q_heads, int32_t batch, const int32_t* q_start, const int32_t* kv_len,
                         const int32_t* block_table, int32_t table_width, float scale, const uint16_t* out,
                         int64_t rows) {
  if (table_width < 1 || !isfinite(scale)) return QLINEAR_ERR_INVALID_ARGUMENT;
  if (!q_start && tokens % batch != 0) return QLINEAR_ERR_INVALID_ARGUMENT;
  if (rows * table_width > kMaxTableSlots / cache->page_size) return QLINEAR_ERR_UNSUPPORTED;
  const int st = check_rows(q, q_stride, q_heads, cache->head_dim);
  if (st != QLINEAR_OK) return st;
  if (!kv_len || !block_table || !out) return QLINEAR_ERR_INVALID_ARGUMENT;
  if (!aligned(out, 16) || !aligned(q_start, 4) || !aligned(kv_len, 4) || !aligned(block_table, 4))
    return QLINEAR_ERR_MISALIGNED;
  return QLINEAR_OK;
}

// Sizes of a call with shared prefixes and of its workspace query.
int check_shared(const qlinear_kv_cache* cache, int32_t tokens, int32_t q_heads, int32_t batch, int32_t max_q_len,
                 int32_t max_kv_len, int32_t groups, int32_t max_shared_len) {
  const int st = check_attention(cache, tokens, q_heads, batch, max_q_len, max_kv_len, 0);
  if (st != QLINEAR_OK) return st;
  if (groups < 1 || max_shared_len < 0) return QLINEAR_ERR_INVALID_ARGUMENT;
  if ((int64_t)batch + groups > 65535 || ((int64_t)batch + groups) * cache->kv_heads > kMaxQueryRows / 128 ||
      (int64_t)tokens * q_heads > kMaxSharedRows)
    return QLINEAR_ERR_UNSUPPORTED;
  return QLINEAR_OK;
}

ViewArgs view_sizes(const AttentionArgs& sizes, int32_t sinks, int32_t groups, int32_t max_shared_len) {
  ViewArgs a = {};
  static_cast<AttentionArgs&>(a) = sizes;
  a.batch += groups;
  a.sinks = sinks;
  a.groups = groups;
  a.max_shared_len = max_shared_len;
  return a;
}

AttentionArgs attention_sizes(int32_t tokens, int32_t q_heads, int32_t batch, int32_t max_q_len, int32_t max_kv_len,
                              int32_t window) {
  AttentionArgs a = {};
  a.tokens = tokens;
  a.q_heads = q_heads;
  a.batch = batch;
  a.max_q_len = max_q_len < tokens ? (max_q_len > 1 ? max_q_len : 1) : tokens;
  a.max_kv_len = max_kv_len;
  a.window = window;
  return a;
}

// Norm weights of q and k heads: one for all heads, or one a head; NULL: no norm.
struct Norms {
  const uint16_t* q = nullptr;
  int32_t q_heads = 1;
  const uint16_t* k = nullptr;
  int32_t k_heads = 1;
  float eps = 0.0f;
};
int set_norms(const Norms& n, int32_t q_heads, int32_t kv_heads, int32_t head_dim, RopeArgs& a) {
  if (!(n.eps >= 0.0f) || !isfinite(n.eps)) return QLINEAR_ERR_INVALID_ARGUMENT;
  if ((n.q && n.q_heads != 1 && n.q_heads != q_heads) || (n.k && n.k_heads != 1 && n.k_heads != kv_heads))
    return QLINEAR_ERR_INVALID_ARGUMENT;
  if (!aligned(n.q, 16) || !aligned(n.k, 16)) return QLINEAR_ERR_MISALIGNED;
  a.q_norm = n.q;
  a.k_norm = n.k;
  a.q_norm_stride = n.q_heads == 1 ? 0 : head_dim;
  a.k_norm_stride = n.k_heads == 1 ? 0 : head_dim;
  // The kernel's reciprocal root takes a subnormal number for zero, and a head of
  // zeros would be 0 times infinity. A head of anything else has a mean square of
  // 2^-57 at least, beside which either eps is nothing.
  a.eps = n.eps > 0.0f && n.eps < FLT_MIN ? FLT_MIN : n.eps;
  a.per_element = 1.0f / (float)head_dim;
  return QLINEAR_OK;
}

// rot_dim == 0 needs no positions or table.
int rotate(const uint16_t* x, int64_t x_stride, int32_t tokens, int32_t heads, int32_t head_dim, const Norms& norms,
           const int32_t* positions, const float* table, int32_t table_rows, int32_t rot_dim, int32_t layout,
           uint16_t* out, int64_t out_stride, void* stream) {
  if (tokens < 0 || heads < 0 || head_dim < 1 || rot_dim < 0) return QLINEAR_ERR_INVALID_ARGUMENT;
  if (heads > 65535 || tokens > kMaxRows) return QLINEAR_ERR_UNSUPPORTED;
  if (tokens == 0 || heads == 0) return QLINEAR_OK;
  RopeArgs a = {};
  int st = check_rotation(head_dim, rot_dim, layout, positions, table, table_rows);
  if (st == QLINEAR_OK) st = check_rows(x, x_stride, heads, head_dim);
  if (st == QLINEAR_OK) st = check_rows(out, out_stride, heads, head_dim);
  if (st == QLINEAR_OK) st = set_norms(norms, heads, 0, head_dim, a);
  if (st != QLINEAR_OK) return st;
  a.q = x;
  a.q_stride = x_stride;
  a.q_out = out;
  a.out_stride = out_stride;
  a.q_heads = heads;
  a.head_dim = head_dim;
  a.tokens = tokens;
  a.positions = positions;
  a.table = table;
  a.table_rows = table_rows;
  a.rot_dim = rot_dim;
  a.layout = layout;
  return hip_status(launch_rope(a, (hipStream_t)stream));
}

int append(const qlinear_kv_cache* cache, const uint16_t* q, int64_t q_stride, int32_t q_heads, const uint16_t* k,
           int64_t k_stride, const uint16_t* v, int64_t v_stride, uint16_t* q_out, int64_t q_out_stride, int32_t tokens,
           const Norms& norms, const int32_t* positions, const int32_t* slots, const float* table, int32_t table_rows,
           int32_t rot_dim, int32_t layout, void* stream) {
  int st = check_cache(cache);
  if (st != QLINEAR_OK) return st;
  if (tokens < 0 || q_heads < 0 || rot_dim < 0) return QLINEAR_ERR_INVALID_ARGUMENT;
  if (q_heads > 65535 || tokens > kMaxRows) return QLINEAR_ERR_UNSUPPORTED;
  if (tokens == 0) return QLINEAR_OK;
  const int D = cache->head_dim;
  st = check_rotation(D, rot_dim, layout, positions, table, table_rows);
  if (st == QLINEAR_OK) st = check_rows(k, k_stride, cache->kv_heads, D);
  if (st == QLINEAR_OK) st = check_rows(v, v_stride, cache->kv_heads, D);
  if (st == QLINEAR_OK && q_heads > 0) st = check_rows(q, q_stride, q_heads, D);
  if (st == QLINEAR_OK && q_heads > 0) st = check_rows(q_out, q_out_stride, q_heads, D);
  RopeArgs a = {};
  if (st == QLINEAR_OK) st = set_norms(norms, q_heads, cache->kv_heads, D, a);
  if (st != QLINEAR_OK) return st;
  if (!slots) return QLINEAR_ERR_INVALID_ARGUMENT;
  if (!aligned(slots, 4)) return QLINEAR_ERR_MISALIGNED;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out = q_out;
  a.out_stride = q_out_stride;
  a.q_heads = q_heads;
  a.head_dim = D;
  a.tokens = tokens;
  a.positions = positions;
  a.slots = slots;
  a.table = table;
  a.table_rows = table_rows;
  a.rot_dim = rot_dim;
  a.layout = layout;
  return hip_status(launch_rope_append(a, *cache, (hipStream_t)stream));
}

}  // namespace

extern "C" {

int qlinear_rope(const uint16_t* x, int64_t x_stride, int32_t tokens, int32_t heads, int32_t head_dim,
                 const int32_t* positions, const float* table, int32_t table_rows, int32_t rot_dim, int32_t layout,
                 uint16_t* out, int64_t out_stride, void* stream) {
  if (rot_dim < 1) return QLINEAR_ERR_INVALID_ARGUMENT;
  return rotate(x, x_stride, tokens, heads, head_dim, {}, positions, table, table_rows, rot_dim, layout, out,
                out_stride, stream);
}

int qlinear_norm_rope(const uint16_t* x, int64_t x_stride, int32_t tokens, int32_t heads, int32_t head_dim,
                      const uint16_t* weight, int32_t weight_heads, float eps, const int32_t* positions,
                      const float* table, int32_t table_rows, int32_t rot_dim, int32_t layout, uint16_t* out,
                      int64_t out_stride, void* stream) {
  if (tokens > 0 && heads > 0 && !weight) return QLINEAR_ERR_INVALID_ARGUMENT;
  return rotate(x, x_stride, tokens, heads, head_dim, {weight, weight_heads, nullptr, 1, eps}, positions, table,
                table_rows, rot_dim, layout, out, out_stride, stream);
}

int qlinear_rope_append(const qlinear_kv_cache* cache, const uint16_t* q, int64_t q_stride, int32_t q_heads,
                        const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride, uint16_t* q_out,
                        int64_t q_out_stride, int32_t tokens, const int32_t* positions, const int32_t* slots,
                        const float* table, int32_t table_rows, int32_t rot_dim, int32_t layout, void* stream) {
  return append(cache, q, q_stride, q_heads, k, k_stride, v, v_stride, q_out, q_out_stride, tokens, {}, positions,
                slots, table, table_rows, rot_dim, layout, stream);
}

int qlinear_norm_rope_append(const qlinear_kv_cache* cache, const uint16_t* q, int64_t q_stride, int32_t q_heads,
                             const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride, uint16_t* q_out,
                             int64_t q_out_stride, int32_t tokens, const uint16_t* q_norm, int32_t q_norm_heads,
                             const uint16_t* k_norm, int32_t k_norm_heads, float eps, const int32_t* positions,
                             const int32_t* slots, const float* table, int32_t table_rows, int32_t rot_dim,
                             int32_t layout, void* stream) {
  return append(cache, q, q_stride, q_heads, k, k_stride, v, v_stride, q_out, q_out_stride, tokens,
                {q_norm, q_norm_heads, k_norm, k_norm_heads, eps}, positions, slots, table, table_rows, rot_dim, layout,
                stream);
}

int qlinear_paged_attention_workspace_bytes(const qlinear_kv_cache* cache, int32_t tokens, int32_t q_heads,
                                            int32_t batch, int32_t max_q_len, int32_t max_kv_len, int32_t window,
                                            size_t* bytes) {
  if (!bytes) return QLINEAR_ERR_INVALID_ARGUMENT;
  const int st = check_attention(cache, tokens, q_heads, batch, max_q_len, max_kv_len, window);
  if (st != QLINEAR_OK) return st;
  *bytes = tokens == 0 || batch == 0
               ? 0
               : paged_attention_workspace_bytes(
                     *cache, attention_sizes(tokens, q_heads, batch, max_q_len, max_kv_len, window));
  return QLINEAR_OK;
}

int qlinear_paged_attention(const qlinear_kv_cache* cache, const uint16_t* q, int64_t q_stride, int32_t tokens,
                            int32_t q_heads, int32_t batch, const int32_t* q_start, const int32_t* kv_len,
                            const int32_t* block_table, int32_t table_width, int32_t max_q_len, int32_t max_kv_len,
                            float scale, int32_t window, uint16_t* out, void* workspace, size_t workspace_bytes,
                            void* stream) {
  int st = check_attention(cache, tokens, q_heads, batch, max_q_len, max_kv_len, window);
  if (st != QLINEAR_OK) return st;
  if (tokens == 0 || batch == 0) return QLINEAR_OK;
  st = check_attention_call(cache, q, q_stride, tokens, q_heads, batch, q_start, kv_len, block_table, table_width, scale,
                            out, batch);
  if (st != QLINEAR_OK) return st;
  AttentionArgs a = attention_sizes(tokens, q_heads, batch, max_q_len, max_kv_len, window);
  a.q = q;
  a.q_stride = q_stride;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.block_table = block_table;
  a.table_width = table_width;
  a.scale = scale;
  a.out = out;
  const size_t need = paged_attention_workspace_need(*cache, a);
  if (need > 0 && (!workspace || workspace_bytes < need)) return QLINEAR_ERR_WORKSPACE;
  if (need > 0 && !aligned(workspace, 16)) return QLINEAR_ERR_MISALIGNED;
  return hip_status(launch_paged_attention(*cache, a, workspace, (hipStream_t)stream));
}

int qlinear_paged_attention_sinks_workspace_bytes(const qlinear_kv_cache* cache, int32_t tokens, int32_t q_heads,
                                                  int32_t batch, int32_t max_q_len, int32_t max_kv_len, int32_t window,
                                                  int32_t sinks, size_t* bytes) {
  if (!bytes) return QLINEAR_ERR_INVALID_ARGUMENT;
  const int st = check_attention(cache, tokens, q_heads, batch, max_q_len, max_kv_len, window);
  if (st != QLINEAR_OK) return st;
  if (sinks < 0) return QLINEAR_ERR_INVALID_ARGUMENT;
  *bytes = tokens == 0 || batch == 0
               ? 0
               : sinks_attention_workspace_bytes(
                     *cache, view_sizes(attention_sizes(tokens, q_heads, batch, max_q_len, max_kv_len, window), sinks, 0, 0));
  return QLINEAR_OK;
}

int qlinear_paged_attention_sinks(const qlinear_kv_cache* cache, const uint16_t* q, int64_t q_stride, int32_t tokens,
                                  int32_t q_heads, int32_t batch, const int32_t* q_start, const int32_t* kv_len,
                                  const int32_t* block_table, int32_t table_width, int32_t max_q_len,
                                  int32_t max_kv_len, float scale, int32_t window, int32_t sinks, uint16_t* out,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_attention(cache, tokens, q_heads, batch, max_q_len, max_kv_len, window);
  if (st != QLINEAR_OK) return st;
  if (sinks < 0) return QLINEAR_ERR_INVALID_ARGUMENT;
  if (tokens == 0 || batch == 0) return QLINEAR_OK;
  st = check_attention_call(cache, q, q_stride, tokens, q_heads, batch, q_start, kv_len, block_table, table_width, scale,
                            out, batch);
  if (st != QLINEAR_OK) return st;
  ViewArgs a = view_sizes(attention_sizes(tokens, q_heads, batch, max_q_len, max_kv_len, window), sinks, 0, 0);
  a.q = q;
  a.q_stride = q_stride;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.block_table = block_table;
  a.table_width = table_width;
  a.scale = scale;
  a.out = out;
  const size_t need = sinks_attention_workspace_need(*cache, a);
  if (need > 0 && (!workspace || workspace_bytes < need)) return QLINEAR_ERR_WORKSPACE;
  if (need > 0 && !aligned(workspace, 16)) return QLINEAR_ERR_MISALIGNED;
  return hip_status(launch_sinks_attention(*cache, a, workspace, (hipStream_t)stream));
}

int qlinear_paged_attention_shared_workspace_bytes(const qlinear_kv_cache* cache, int32_t tokens, int32_t q_heads,
                                                   int32_t batch, int32_t max_q_len, int32_t max_kv_len,
                                                   int32_t groups, int32_t max_shared_len, size_t* bytes) {
  if (!bytes) return QLINEAR_ERR_INVALID_ARGUMENT;
  const int st = check_shared(cache, tokens, q_heads, batch, max_q_len, max_kv_len, groups, max_shared_len);
  if (st != QLINEAR_OK) return st;
  *bytes = tokens == 0 || batch == 0
               ? 0
               : shared_attention_workspace_bytes(
                     *cache, view_sizes(attention_sizes(tokens, q_heads, batch, max_q_len, max_kv_len, 0), 0, groups,
                                        max_shared_len));
  return QLINEAR_OK;
}

int qlinear_paged_attention_shared(const qlinear_kv_cache* cache, const uint16_t* q, int64_t q_stride, int32_t tokens,
                                   int32_t q_heads, int32_t batch, const int32_t* q_start, const int32_t* kv_len,
                                   const int32_t* block_table, int32_t table_width, int32_t groups,
                                   const int32_t* shared_start, const int32_t* shared_len, int32_t max_q_len,
                                   int32_t max_kv_len, int32_t max_shared_len, float scale, uint16_t* out,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_shared(cache, tokens, q_heads, batch, max_q_len, max_kv_len, groups, max_shared_len);
  if (st != QLINEAR_OK) return st;
  if (tokens == 0 || batch == 0) return QLINEAR_OK;
  st = check_attention_call(cache, q, q_stride, tokens, q_heads, batch, q_start, kv_len, block_table, table_width, scale,
                            out, (int64_t)batch + groups);
  if (st != QLINEAR_OK) return st;
  if (!shared_len || (!shared_start && groups != 1)) return QLINEAR_ERR_INVALID_ARGUMENT;
  if (!aligned(shared_start, 4) || !aligned(shared_len, 4)) return QLINEAR_ERR_MISALIGNED;
  ViewArgs a =
      view_sizes(attention_sizes(tokens, q_heads, batch, max_q_len, max_kv_len, 0), 0, groups, max_shared_len);
  a.q = q;
  a.q_stride = q_stride;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.block_table = block_table;
  a.table_width = table_width;
  a.scale = scale;
  a.out = out;
  a.shared_start = shared_start;
  a.shared_len = shared_len;
  const size_t need = shared_attention_workspace_need(*cache, a);
  if (need > 0 && (!workspace || workspace_bytes < need)) return QLINEAR_ERR_WORKSPACE;
  if (need > 0 && !aligned(workspace, 16)) return QLINEAR_ERR_MISALIGNED;
  return hip_status(launch_shared_attention(*cache, a, workspace, (hipStream_t)stream));
}

int qlinear_copy_pages(const qlinear_kv_cache* caches_host, int32_t count, const int32_t* pairs, int32_t moves,
                       void* stream) {
  if (count < 0 || moves < 0) return QLINEAR_ERR_INVALID_ARGUMENT;
  if (count == 0) return QLINEAR_OK;
  if (!caches_host) return QLINEAR_ERR_INVALID_ARGUMENT;
  for (int i = 0; i < count; ++i) {
    const qlinear_kv_cache &a = caches_host[0], &b = caches_host[i];
    const int st = check_cache(&b);
    if (st != QLINEAR_OK) return st;
    if (a.num_pages != b.num_pages || a.page_size != b.page_size || a.kv_heads != b.kv_heads ||
        a.head_dim != b.head_dim || a.bits != b.bits || (a.bits != 16 && a.group != b.group))
      return QLINEAR_ERR_UNSUPPORTED;
  }
  if (moves == 0) return QLINEAR_OK;
  if (!pairs) return QLINEAR_ERR_INVALID_ARGUMENT;
  if (!aligned(pairs, 8)) return QLINEAR_ERR_MISALIGNED;
  return hip_status(launch_copy_pages(caches_host, count, pairs, moves, (hipStream_t)stream));
}

int qlinear_rms_norm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, int32_t M, int32_t K,
                     float eps, uint16_t* y, uint16_t* residual_out, void* stream) {
  if (M < 0 || K < 1 || !(eps >= 0.0f) || !isfinite(eps)) return QLINEAR_ERR_INVALID_ARGUMENT;
  if (K > (1 << 24) || M > kMaxRows) return QLINEAR_ERR_UNSUPPORTED;
  if (M == 0) return QLINEAR_OK;
  if (!x || !weight || !y || y == residual_out) return QLINEAR_ERR_INVALID_ARGUMENT;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(y, 16) ||
      !aligned(residual_out, 16))
    return QLINEAR_ERR_MISALIGNED;
  return hip_status(launch_rms_norm(x, residual, weight, M, K, eps, y, residual_out, (hipStream_t)stream));
}

int qlinear_token_logprobs_workspace_bytes(int32_t rows, int32_t vocab, int32_t logit_bits, int32_t top,
                                           size_t* bytes) {
  if (!bytes) return QLINEAR_ERR_INVALID_ARGUMENT;
  LogprobArgs a = {};
  const int st = check_logprob(rows, vocab, logit_bits, top, a);
  if (st != QLINEAR_OK) return st;
  *bytes = rows == 0 ? 0 : logprob_workspace_bytes(a);
  return QLINEAR_OK;
}

int qlinear_token_logprobs(const void* logits, int64_t stride, int32_t rows, int32_t vocab, int32_t logit_bits,
                           const int32_t* tokens, int32_t top, float* logprob, float* entropy, float* top_logprob,
                           int32_t* top_id, void* workspace, size_t workspace_bytes, void* stream) {
  LogprobArgs a = {};
  const int st = check_logprob(rows, vocab, logit_bits, top, a);
  if (st != QLINEAR_OK) return st;
  if (rows == 0) return QLINEAR_OK;
  if (!logits || stride < vocab || (logprob && !tokens) || (top > 0 && (!top_logprob || !top_id)))
    return QLINEAR_ERR_INVALID_ARGUMENT;
  if (!aligned(logits, logit_bits / 8) || !aligned(tokens, 4) || !aligned(logprob, 4) || !aligned(entropy, 4) ||
      !aligned(top_logprob, 4) || !aligned(top_id, 4))
    return QLINEAR_ERR_MISALIGNED;
  if (!logprob && !entropy && top == 0) return QLINEAR_OK;
  a.logits = logits;
  a.stride = stride;
  a.tokens = tokens;
  a.logprob = logprob;
  a.entropy = entropy;
  a.top_logprob = top_logprob;
  a.top_id = top_id;
  const size_t need = logprob_workspace_need(a);
  if (need > 0 && (!workspace || workspace_bytes < need)) return QLINEAR_ERR_WORKSPACE;
  if (need > 0 && !aligned(workspace, 16)) return QLINEAR_ERR_MISALIGNED;
  return hip_status(launch_logprob(a, workspace, (hipStream_t)stream));
}

}  // extern "C"
