// RMS norm with the residual's addition and 8-bit rows, and its gradient
// (sm_103a):
//
//   h = x + residual;  rstd = 1 / sqrt(mean h^2 + eps);  y = h * rstd * gamma
//   scale = max(max |y|, 1e-30) / 448;  q = rne_e4m3(y / scale)
//
//   n = h * rstd;  g = dy * gamma;  c = mean(g n)
//   dx = rstd * (g - n c) + dh;  dgamma = sum over rows of dy n
//
// One CTA per row with the row in fp32 in shared memory: every input element
// is read once and every output written once.

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "../../include/mpopt.h"
#include "internal.h"

namespace mpopt {
namespace {

constexpr int kThreads = 256;
constexpr float kE4m3Max = 448.f;
constexpr float kAmaxFloor = 1e-30f;

__device__ __forceinline__ float load_elem(const void* p, int64_t i, int dtype) {
  return dtype == kBf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
}

__device__ __forceinline__ void store_elem(void* p, int64_t i, int dtype, float v) {
  if (dtype == kBf16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<float*>(p)[i] = v;
}

// Sum and maximum over the CTA, the same value in every thread.
template <bool kMax>
__device__ __forceinline__ float block_reduce(float v, float* warp_vals) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const float o = __shfl_xor_sync(0xffffffffu, v, off);
    v = kMax ? fmaxf(v, o) : v + o;
  }
  __syncthreads();                     // the previous reduction has been read
  if ((threadIdx.x & 31) == 0) warp_vals[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = warp_vals[0];
  for (int w = 1; w < kThreads / 32; ++w) t = kMax ? fmaxf(t, warp_vals[w]) : t + warp_vals[w];
  return t;
}

__device__ __forceinline__ uint8_t e4m3_bits(float v) {
  return __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}

__global__ void __launch_bounds__(kThreads) rmsnorm_kernel(const __grid_constant__ RmsnormArgs a) {
  extern __shared__ float row[];
  __shared__ float warp_vals[kThreads / 32];
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    float ss = 0.f;
    for (int64_t c = threadIdx.x; c < a.cols; c += kThreads) {
      float v = load_elem(a.x, r * a.x_ld + c, a.dtype);
      if (a.residual) v += load_elem(a.residual, r * a.residual_ld + c, a.dtype);
      if (a.h) store_elem(a.h, r * a.h_ld + c, a.dtype, v);
      row[c] = v;
      ss += v * v;
    }
    float rstd = 1.f;
    if (a.norm) {
      rstd = 1.f / sqrtf(block_reduce<false>(ss, warp_vals) / static_cast<float>(a.cols) + a.eps);
      if (a.rstd && threadIdx.x == 0) a.rstd[r] = rstd;
    }
    float amax = 0.f;
    for (int64_t c = threadIdx.x; c < a.cols; c += kThreads) {
      float y = row[c];
      if (a.norm) y = y * rstd * load_elem(a.gamma, c, a.gamma_dtype);
      row[c] = y;
      amax = fmaxf(amax, fabsf(y));
      if (a.y) store_elem(a.y, r * a.y_ld + c, kBf16, y);
    }
    if (a.q) {
      const float scale = fmaxf(block_reduce<true>(amax, warp_vals), kAmaxFloor) / kE4m3Max;
      if (threadIdx.x == 0) a.q_scale[r] = scale;
      const float inv = 1.f / scale;
      for (int64_t c = threadIdx.x; c < a.cols; c += kThreads) a.q[r * a.q_ld + c] = e4m3_bits(row[c] * inv);
    }
    __syncthreads();                   // the row is free again
  }
}

// CTA b takes rows b, b + gridDim.x, ... and keeps its part of dgamma in
// partial[b].
__global__ void __launch_bounds__(kThreads) rmsnorm_grad_kernel(const __grid_constant__ RmsnormGradArgs a) {
  extern __shared__ float rows[];
  __shared__ float warp_vals[kThreads / 32];
  float* n_row = rows;
  float* g_row = rows + a.cols;
  float* part = a.dgamma ? a.partial + static_cast<int64_t>(blockIdx.x) * a.cols : nullptr;
  bool first = true;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const float rstd = a.rstd[r];
    float dot = 0.f;
    for (int64_t c = threadIdx.x; c < a.cols; c += kThreads) {
      const float n = load_elem(a.h, r * a.h_ld + c, a.dtype) * rstd;
      const float dy = load_elem(a.dy, r * a.dy_ld + c, kBf16);
      const float g = dy * load_elem(a.gamma, c, a.gamma_dtype);
      if (part) part[c] = first ? dy * n : part[c] + dy * n;   // this thread's own column
      n_row[c] = n;
      g_row[c] = g;
      dot += g * n;
    }
    first = false;
    if (a.dx) {
      const float mean = block_reduce<false>(dot, warp_vals) / static_cast<float>(a.cols);
      for (int64_t c = threadIdx.x; c < a.cols; c += kThreads) {
        float v = rstd * (g_row[c] - n_row[c] * mean);
        if (a.dh) v += load_elem(a.dh, r * a.dh_ld + c, a.dtype);
        store_elem(a.dx, r * a.dx_ld + c, a.dtype, v);
      }
      __syncthreads();
    }
  }
}

__global__ void __launch_bounds__(kThreads)
dgamma_kernel(const float* partial, int n_partial, int64_t cols, float* dgamma, int accumulate) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (c >= cols) return;
  float s = 0.f;
  for (int p = 0; p < n_partial; ++p) s += partial[static_cast<int64_t>(p) * cols + c];
  dgamma[c] = accumulate ? dgamma[c] + s : s;
}

}  // namespace

cudaError_t launch_rmsnorm(const RmsnormArgs& a, cudaStream_t stream) {
  if (a.rows <= 0) return cudaSuccess;
  const int smem = static_cast<int>(a.cols * sizeof(float));
  cudaError_t e = cudaFuncSetAttribute(rmsnorm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t grid = a.rows < (int64_t(1) << 30) ? a.rows : (int64_t(1) << 30);
  rmsnorm_kernel<<<static_cast<unsigned>(grid), kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_rmsnorm_grad(const RmsnormGradArgs& a, cudaStream_t stream) {
  const int64_t grid = a.rows < kNormPartialRows ? a.rows : kNormPartialRows;
  if (grid > 0) {
    const int smem = static_cast<int>(2 * a.cols * sizeof(float));
    cudaError_t e = cudaFuncSetAttribute(rmsnorm_grad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    prof_begin(OPT_KERNEL_RMSNORM_GRAD, 1, a.rows, a.cols, stream);
    rmsnorm_grad_kernel<<<static_cast<unsigned>(grid), kThreads, smem, stream>>>(a);
    prof_end(stream);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (!a.dgamma) return cudaSuccess;
  prof_begin(OPT_KERNEL_RMSNORM_DGAMMA, 1, a.rows, a.cols, stream);
  dgamma_kernel<<<static_cast<unsigned>((a.cols + kThreads - 1) / kThreads), kThreads, 0, stream>>>(
      a.partial, static_cast<int>(grid), a.cols, a.dgamma, a.accumulate);
  prof_end(stream);
  return cudaGetLastError();
}

}  // namespace mpopt
