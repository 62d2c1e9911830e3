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
#include "qlinear_kernels.hpp"

namespace qlinear {

namespace {

constexpr int kRegRow = 32768;

union Half8 {
  uint4 v;
  _Float16 h[8];
};

// Sum over the T threads that share a row (T == 64: one wave).
template <int T>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) v += __shfl_xor(v, k);
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < T / 64; ++i) v += part[i];
  }
  return v;
}

// T threads a row, NC 16-byte chunks a thread; T == 64 puts four rows in a workgroup.
template <int T, int NC>
__global__ __launch_bounds__(T == 64 ? 256 : T) void rms_norm_kernel(
    const uint16_t* x, const uint16_t* residual, const uint16_t* __restrict__ weight, int M, int K, float eps,
    uint16_t* y, uint16_t* residual_out) {
  __shared__ float part[T / 64];
  const int t = threadIdx.x % T;
  const int m = T == 64 ? blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  if (m >= M) return;   // whole waves only (T == 64), which meet no barrier
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
    if (residual_out) *reinterpret_cast<uint4*>(residual_out + row + k) = h[c].v;
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
    *reinterpret_cast<uint4*>(y + row + k) = h[c].v;
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
  auto go = [&](auto kernel, int threads, int rows) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)((M + rows - 1) / rows)), dim3(threads), 0, stream, x, residual, weight,
                       M, K, eps, y, residual_out);
    return hipGetLastError();
  };
  if (K % 8 != 0 || K > kRegRow) {
    hipLaunchKernelGGL(rms_norm_any_kernel, dim3((unsigned)M), dim3(256), 0, stream, x, residual, weight, K, eps, y,
                       residual_out);
    return hipGetLastError();
  }
  if (K <= 512) return go(rms_norm_kernel<64, 1>, 256, 4);
  if (K <= 2048) return go(rms_norm_kernel<256, 1>, 256, 1);
  if (K <= 4096) return go(rms_norm_kernel<256, 2>, 256, 1);
  if (K <= 8192) return go(rms_norm_kernel<256, 4>, 256, 1);
  return go(rms_norm_kernel<1024, 4>, 1024, 1);
}

}  // namespace qlinear
