// Cross-entropy of rows of logits and its gradient (sm_103a):
//
//   lse = m + log(sum_j exp(x_j - m)), m = max_j x_j;  loss = lse - x_label
//   dx_j = (exp(x_j - m) / sum - [j = label]) * scale * weight
//
// Bound by HBM: a row is read for its maximum and sum, kept together in one pass
// (a thread's sum is scaled when its maximum grows), and the gradient written.
// The second reading of the row comes out of L2.  A row of up to 1024 columns
// belongs to a warp, a longer one to a CTA.  Groups of 16 bytes begin at the
// row's first multiple of 16 bytes, the elements around them go to one thread
// each.

#include "elements.cuh"
#include "internal.h"
#include "overlap.cuh"

namespace mpopt {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// e^d for d <= 0 (0 below 2^-126): d log2 e is rounded once, which is 2^-24 |d|
// of the value, beside 2 units of the instruction.
__device__ __forceinline__ float exp_of(float d) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(d * kLog2e));
  return e;
}

// The largest value and the sum of exp(x - max) of some logits; max -inf: none yet.
struct Stat {
  float top, sum;
};

__device__ __forceinline__ float anchor(float top) { return top == -INFINITY ? 0.f : top; }

__device__ __forceinline__ Stat join(Stat a, Stat b) {
  const float top = fmaxf(a.top, b.top), at = anchor(top);
  return Stat{top, a.sum * exp_of(a.top - at) + b.sum * exp_of(b.top - at)};
}

template <typename T>
struct Group {
  static constexpr int kN = 16 / sizeof(T);
};

__device__ __forceinline__ void load_group(const __nv_bfloat16* p, float (&v)[8]) { load8(p, v); }
__device__ __forceinline__ void load_group(const float* p, float (&v)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
}
__device__ __forceinline__ void store_group(__nv_bfloat16* p, const float (&v)[8]) { store8(p, v); }
__device__ __forceinline__ void store_group(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

template <int kN>
__device__ __forceinline__ void add_to(Stat& s, const float (&v)[kN]) {
  float top = s.top;
#pragma unroll
  for (int j = 0; j < kN; ++j) top = fmaxf(top, v[j]);
  const float at = anchor(top);
  float sum = s.sum * exp_of(s.top - at);
#pragma unroll
  for (int j = 0; j < kN; ++j) sum += exp_of(v[j] - at);
  s.top = top;
  s.sum = sum;
}

template <typename T, int kTPR>
__global__ void __launch_bounds__(kTPR == 32 ? 256 : kTPR)
cross_entropy_kernel(const __grid_constant__ opt_cross_entropy_args a) {
  constexpr int kRows = kTPR == 32 ? 8 : 1, kN = Group<T>::kN, kWarps = kTPR / 32;
  __shared__ Stat parts[kWarps];
  let_next_start();
  wait_for_predecessors();
  const int t = threadIdx.x % kTPR;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kTPR;
  if (r >= a.rows) return;                       // whole warps of a CTA with a row to each
  const T* x = static_cast<const T*>(a.logits) + r * a.logits_ld;
  T* g = a.dlogits ? static_cast<T*>(a.dlogits) + r * a.dlogits_ld : nullptr;
  const int64_t label = a.index_dtype == OPT_INDEX_INT32 ? static_cast<const int32_t*>(a.labels)[r]
                                                         : static_cast<const int64_t*>(a.labels)[r];
  const bool counts = label >= 0 && label < a.cols;
  const int64_t ahead = (-(reinterpret_cast<uintptr_t>(x) / sizeof(T)) & (kN - 1));
  const int64_t head = ahead < a.cols ? ahead : a.cols, groups = (a.cols - head) / kN, end = head + groups * kN;
  // the column outside of the groups that this thread has, or -1
  const int64_t edge = t < head ? t : t < head + a.cols - end ? end + t - head : -1;
  const float at_label = counts ? load_elem(x + label) : 0.f;
  Stat s{-INFINITY, 0.f};
  if (counts || a.lse) {
    if (edge >= 0) {
      const float v[1] = {load_elem(x + edge)};
      add_to(s, v);
    }
#pragma unroll 4
    for (int64_t i = t; i < groups; i += kTPR) {
      float v[kN];
      load_group(x + head + i * kN, v);
      add_to(s, v);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const Stat o{__shfl_xor_sync(0xffffffffu, s.top, off), __shfl_xor_sync(0xffffffffu, s.sum, off)};
      s = join(s, o);
    }
    if constexpr (kTPR > 32) {
      if ((t & 31) == 0) parts[t >> 5] = s;
      __syncthreads();
      s = parts[0];
      for (int w = 1; w < kWarps; ++w) s = join(s, parts[w]);
    }
    if (t == 0) {
      const bool none = s.sum == 0.f;            // an empty row
      const float log_sum = logf(s.sum);
      if (a.lse) a.lse[r] = none ? -INFINITY : s.top + log_sum;
      if (a.loss) a.loss[r] = !counts ? 0.f : none ? INFINITY : log_sum - (at_label - anchor(s.top));
    }
  } else if (t == 0 && a.loss) {
    a.loss[r] = 0.f;
  }
  if (!g) return;
  if constexpr (kTPR == 32) __syncwarp();         // dlogits may be logits: the label's is read before it is written
  const bool zero = !counts || s.sum == 0.f;
  const float w = a.weight ? a.weight[r] * a.scale : a.scale;
  const float inv = 1.f / s.sum, at = anchor(s.top);
  auto gradient = [&](float v, int64_t c) { return zero ? 0.f : (exp_of(v - at) * inv - (c == label ? 1.f : 0.f)) * w; };
  if (edge >= 0) store_elem(g + edge, gradient(load_elem(x + edge), edge));
  const bool together = ((reinterpret_cast<uintptr_t>(g + head)) & 15u) == 0;
#pragma unroll 4
  for (int64_t i = t; i < groups; i += kTPR) {
    const int64_t c = head + i * kN;
    float v[kN];
    load_group(x + c, v);
#pragma unroll
    for (int j = 0; j < kN; ++j) v[j] = gradient(v[j], c + j);
    if (together) {
      store_group(g + c, v);
    } else {
#pragma unroll
      for (int j = 0; j < kN; ++j) store_elem(g + c + j, v[j]);
    }
  }
}

template <typename T>
cudaError_t launch_rows(const opt_cross_entropy_args& a, cudaStream_t stream) {
  if (a.cols <= 1024)
    return launch_overlapped(cross_entropy_kernel<T, 32>, dim3(static_cast<unsigned>((a.rows + 7) / 8)), 256, 0, stream, 0, a);
  return launch_overlapped(cross_entropy_kernel<T, 512>, dim3(static_cast<unsigned>(a.rows)), 512, 0, stream, 0, a);
}

}  // namespace

cudaError_t launch_cross_entropy(const opt_cross_entropy_args& a, cudaStream_t stream) {
  return a.dtype == kBf16 ? launch_rows<__nv_bfloat16>(a, stream) : launch_rows<float>(a, stream);
}

}  // namespace mpopt
