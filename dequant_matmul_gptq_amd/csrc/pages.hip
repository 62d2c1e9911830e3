// Page copies inside the caches of a model's layers: for every pair, the
// target page's bytes become the source page's, in each layer's k and v pools
// and their scales. One launch covers up to kMaxLayers layers (their pool
// pointers travel in the kernel's arguments) and all pairs.
//
// HBM-bound: every page byte is read and written once. A page's pools are cut
// into pieces of kPiece bytes, one workgroup each, four 16-byte loads in
// flight per thread; stores leave no lines in the caches, whose room the
// sources can use (one page of 1 MiB in each of 32 layers: 22.0 us with plain
// stores, 11.5 us = 5.9 TB/s; 151 pages in each of 16: 280, 271 us = 5.3 TB/s).
#include "qlinear_kernels.hpp"

namespace qlinear {

namespace {

constexpr int kThreads = 256;
constexpr int kLoads = 4;
constexpr int kPiece = kThreads * kLoads * 16;
constexpr int kMaxLayers = 64;

typedef uint32_t u4 __attribute__((ext_vector_type(4)));

struct LayerPools {
  uint4* pool[kMaxLayers][2];     // k, v
  uint4* scales[kMaxLayers][2];
};

__global__ __launch_bounds__(kThreads) void copy_pages_kernel(LayerPools layers, const int2* __restrict__ pairs,
                                                              int num_pages, int pieces, int scale_pieces,
                                                              int64_t page_units, int64_t scale_units) {
  const int per_pair = 2 * (pieces + scale_pieces);
  const int2 pair = pairs[blockIdx.x / per_pair];
  if ((unsigned)pair.x >= (unsigned)num_pages || (unsigned)pair.y >= (unsigned)num_pages) return;
  int j = blockIdx.x % per_pair;
  const bool is_scale = j >= 2 * pieces;
  if (is_scale) j -= 2 * pieces;
  const int n = is_scale ? scale_pieces : pieces;
  const int side = j >= n ? 1 : 0;
  const int64_t units = is_scale ? scale_units : page_units;
  uint4* base = is_scale ? layers.scales[blockIdx.y][side] : layers.pool[blockIdx.y][side];
  const uint4* src = base + pair.x * units;
  uint4* dst = base + pair.y * units;
  const int64_t first = (int64_t)(j - side * n) * (kThreads * kLoads) + threadIdx.x;
  uint4 v[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i)
    if (first + i * kThreads < units) v[i] = src[first + i * kThreads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i)
    if (first + i * kThreads < units)
      __builtin_nontemporal_store(__builtin_bit_cast(u4, v[i]), reinterpret_cast<u4*>(dst + first + i * kThreads));
}

}  // namespace

hipError_t launch_copy_pages(const qlinear_kv_cache* caches, int count, const int32_t* pairs, int moves,
                             hipStream_t stream) {
  const qlinear_kv_cache& c = caches[0];
  const int64_t slots = (int64_t)c.kv_heads * c.page_size;
  const int64_t page_bytes = slots * c.head_dim * c.bits / 8;
  const int64_t scale_bytes = c.bits == 16 ? 0 : slots * (c.head_dim / c.group) * 2;
  const int pieces = (int)((page_bytes + kPiece - 1) / kPiece);
  const int scale_pieces = (int)((scale_bytes + kPiece - 1) / kPiece);
  const int per_pair = 2 * (pieces + scale_pieces);
  // gridDim.x stays below 2^31 work items' worth of workgroups.
  const int max_moves = (int)((((int64_t)1 << 31) / kThreads - 1) / per_pair);
  for (int l0 = 0; l0 < count; l0 += kMaxLayers) {
    const int n = count - l0 < kMaxLayers ? count - l0 : kMaxLayers;
    LayerPools layers = {};
    for (int i = 0; i < n; ++i) {
      const qlinear_kv_cache& s = caches[l0 + i];
      layers.pool[i][0] = (uint4*)s.k;
      layers.pool[i][1] = (uint4*)s.v;
      layers.scales[i][0] = (uint4*)s.k_scales;
      layers.scales[i][1] = (uint4*)s.v_scales;
    }
    for (int m0 = 0; m0 < moves; m0 += max_moves) {
      const int m = moves - m0 < max_moves ? moves - m0 : max_moves;
      hipLaunchKernelGGL(copy_pages_kernel, dim3((unsigned)(m * per_pair), (unsigned)n), dim3(kThreads), 0, stream,
                         layers, reinterpret_cast<const int2*>(pairs) + m0, c.num_pages, pieces, scale_pieces,
                         page_bytes / 16, scale_bytes / 16);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

}  // namespace qlinear
