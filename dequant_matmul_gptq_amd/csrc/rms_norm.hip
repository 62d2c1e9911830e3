// Root-mean-square norm with the residual's addition:
//   h = RNE_fp16(x + residual),  y = RNE_fp16(h / sqrt(mean h^2 + eps) * w)
// per row of K elements. The sum of squares is float32 over the rounded h, so
// that the norm is of what the residual stream keeps; both roundings are the
// outputs' own.
//
// HBM-bound: reads x and the residual and writes h and y once, 8 bytes per
// element. A row stays in registers between the sum and the scaling (up to
// 32768 elements, kRegRow); longer rows, and rows whose length is not a
// multiple of 8 (their 16-byte loads would not be aligned), are read again.
#include <type_traits>

#include "qlinear_kernels.hpp"

namespace qlinear {

namespace {

constexpr int kRegRow = 32768;

union Half8 {
  uint4 v;
  _Float16 h[8];
};

// PAST: stores that leave no lines in the caches, which hold less than what a
// large call writes, and then keep its inputs instead (8192 x 8192 with a
// residual, on the same buffers again: 102.8 us with plain stores, 79.9 us;
// 100000 x 512: 71.7, 57.8 us; on other buffers each time 98 us = 5.5 TB/s).
// What a small call writes is read from the caches next.
template <bool PAST>
__device__ __forceinline__ void store8(uint16_t* p, const uint4& v) {
  typedef uint32_t u4 __attribute__((ext_vector_type(4)));
  if constexpr (PAST)
    __builtin_nontemporal_store(__builtin_bit_cast(u4, v), reinterpret_cast<u4*>(p));
  else
    *reinterpret_cast<uint4*>(p) = v;
}

// Sum over the T threads that share a row (neighbours in a wave, or waves).
template <int T>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
  for (int k = 1; k < (T < 64 ? T : 64); k <<= 1) v += __shfl_xor(v, k);
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < T / 64; ++i) v += part[i];
  }
  return v;
}

// T threads a row, NC 16-byte chunks a thread; T <= 64 puts 256 / T rows in a workgroup.
template <int T, int NC, bool PAST>
__global__ __launch_bounds__(T <= 64 ? 256 : T) void rms_norm_kernel(
    const uint16_t* x, const uint16_t* residual, const uint16_t* __restrict__ weight, int M, int K, float eps,
    uint16_t* y, uint16_t* residual_out) {
  __shared__ float part[T < 64 ? 1 : T / 64];
  const int t = threadIdx.x % T;
  const int m = T <= 64 ? blockIdx.x * (256 / T) + threadIdx.x / T : blockIdx.x;
  if (m >= M) return;   // whole rows (T <= 64), which meet no barrier
  const int64_t row = (int64_t)m * K;
  Half8 h[NC];
  float sum = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int k = (c * T + t) * 8;
    if (k >= K) continue;
    h[c].v = *reinterpret_cast<const uint4*>(x + row + k);
    if (residual) {
      Half8 r;
      r.v = *reinterpret_cast<const uint4*>(residual + row + k);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c].h[i] = (_Float16)((float)h[c].h[i] + (float)r.h[i]);
    }
    if (residual_out) store8<PAST>(residual_out + row + k, h[c].v);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += (float)h[c].h[i] * (float)h[c].h[i];
  }
  const float inv = 1.0f / sqrtf(row_sum<T>(sum, part) / (float)K + eps);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int k = (c * T + t) * 8;
    if (k >= K) continue;
    Half8 w;
    w.v = *reinterpret_cast<const uint4*>(weight + k);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[c].h[i] = (_Float16)((float)h[c].h[i] * inv * (float)w.h[i]);
    store8<PAST>(y + row + k, h[c].v);
  }
}

// Any K, element by element; each thread reads again what it read itself, so
// outputs may be the inputs' buffers (h comes back from residual_out where x
// or the residual may have been overwritten by it).
__global__ __launch_bounds__(256) void rms_norm_any_kernel(const uint16_t* x, const uint16_t* residual,
                                                           const uint16_t* __restrict__ weight, int K, float eps,
                                                           uint16_t* y, uint16_t* residual_out) {
  __shared__ float part[4];
  const int64_t row = (int64_t)blockIdx.x * K;
  auto h_of = [&](int k) {
    const _Float16 a = __builtin_bit_cast(_Float16, x[row + k]);
    if (!residual) return a;
    return (_Float16)((float)a + (float)__builtin_bit_cast(_Float16, residual[row + k]));
  };
  float sum = 0.0f;
  for (int k = threadIdx.x; k < K; k += 256) {
    const _Float16 h = h_of(k);
    if (residual_out) residual_out[row + k] = __builtin_bit_cast(uint16_t, h);
    sum += (float)h * (float)h;
  }
  const float inv = 1.0f / sqrtf(row_sum<256>(sum, part) / (float)K + eps);
  for (int k = threadIdx.x; k < K; k += 256) {
    const _Float16 h = residual_out ? __builtin_bit_cast(_Float16, residual_out[row + k]) : h_of(k);
    const float w = (float)__builtin_bit_cast(_Float16, weight[k]);
    y[row + k] = __builtin_bit_cast(uint16_t, (_Float16)((float)h * inv * w));
  }
}

}  // namespace

hipError_t launch_rms_norm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, int M, int K,
                           float eps, uint16_t* y, uint16_t* residual_out, hipStream_t stream) {
  if (K % 8 != 0 || K > kRegRow) {
    hipLaunchKernelGGL(rms_norm_any_kernel, dim3((unsigned)M), dim3(256), 0, stream, x, residual, weight, K, eps, y,
                       residual_out);
    return hipGetLastError();
  }
  const bool past = (int64_t)M * K >= 1 << 19;      // outputs of a MiB
  auto go = [&](auto threads, auto chunks) {
    constexpr int T = decltype(threads)::value, NC = decltype(chunks)::value;
    constexpr int kRows = T <= 64 ? 256 / T : 1;
    auto kernel = past ? rms_norm_kernel<T, NC, true> : rms_norm_kernel<T, NC, false>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)((M + kRows - 1) / kRows)), dim3(T <= 64 ? 256 : T), 0, stream, x,
                       residual, weight, M, K, eps, y, residual_out);
    return hipGetLastError();
  };
  std::integral_constant<int, 1> one;
  std::integral_constant<int, 4> four;
  std::integral_constant<int, 256> group;
  if (K <= 64) return go(std::integral_constant<int, 8>{}, one);
  if (K <= 128) return go(std::integral_constant<int, 16>{}, one);
  if (K <= 512) return go(std::integral_constant<int, 64>{}, one);
  if (K <= 2048) return go(group, one);
  if (K <= 4096) return go(group, std::integral_constant<int, 2>{});
  if (K <= 8192) return go(group, four);
  return go(std::integral_constant<int, 1024>{}, four);
}

}  // namespace qlinear
