// RMS norm with the residual's addition and 8-bit rows, and its gradient
// (sm_103a):
//
//   h = x + residual;  rstd = 1 / sqrt(mean h^2 + eps);  y = h * rstd * gamma
//   scale = max(max |y|, 1e-30) / 448;  q = rne_e4m3(y / scale)
//
//   n = h * rstd;  g = dy * gamma;  c = mean(g n)
//   dx = rstd * (g - n c) + dh;  dgamma = sum over rows of dy n
//
// All of it is bound by HBM: every input element is read once and every
// output written once, a row staying in registers between its statistics and
// its outputs.  A row of up to 1024 columns belongs to one warp (no barrier,
// eight rows to a CTA), a longer one to a CTA of 128 to 512 threads, up to
// 16384 columns in registers; longer rows are kept in fp32 in shared memory.
// Where every row starts on 16 bytes a thread moves 8 elements at a time,
// otherwise single elements, neighbours in neighbouring lanes.

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "../../include/mpopt.h"
#include "internal.h"
#include "overlap.cuh"

namespace mpopt {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kAmaxFloor = 1e-30f;
constexpr int kLongThreads = 512;             // rows longer than the register kernels take
constexpr int64_t kRegisterCols = 16384;

// ------------------------------------------------------------- elements --

__device__ __forceinline__ float load_elem(const float* p) { return *p; }
__device__ __forceinline__ float load_elem(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_elem(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_elem(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// Plain loads: an output may be one of the inputs (h over x, dx over dh).
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  unpack8(*reinterpret_cast<const uint4*>(p), v);
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint8_t e4m3(float v) { return __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3); }

// A thread's share of a row: kNV groups of 8 columns.  With kVec group i
// starts at column (i * kTPR + t) * 8, otherwise its element j is column
// (i * 8 + j) * kTPR + t.
template <int kTPR, bool kVec>
__device__ __forceinline__ int column(int i, int j, int t) {
  return kVec ? (i * kTPR + t) * 8 + j : (i * 8 + j) * kTPR + t;
}

template <int kTPR, bool kVec, typename T>
__device__ __forceinline__ void load_group(const T* row, int i, int t, int cols, float (&v)[8]) {
  if constexpr (kVec) {
    const int c = column<kTPR, true>(i, 0, t);
    if (c < cols) {
      load8(row + c, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = column<kTPR, false>(i, j, t);
      v[j] = c < cols ? load_elem(row + c) : 0.f;
    }
  }
}

template <int kTPR, bool kVec, typename T>
__device__ __forceinline__ void store_group(T* row, int i, int t, int cols, const float (&v)[8]) {
  if constexpr (kVec) {
    const int c = column<kTPR, true>(i, 0, t);
    if (c < cols) store8(row + c, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = column<kTPR, false>(i, j, t);
      if (c < cols) store_elem(row + c, v[j]);
    }
  }
}

// A group times inv in e4m3, 8 bytes.
template <int kTPR>
__device__ __forceinline__ void store_e4m3(uint8_t* row, int i, int t, int cols, const float (&v)[8], float inv) {
  const int c = column<kTPR, true>(i, 0, t);
  if (c < cols)
    *reinterpret_cast<uint2*>(row + c) =
        make_uint2(e4m3x2(v[0] * inv, v[1] * inv) | (e4m3x2(v[2] * inv, v[3] * inv) << 16),
                   e4m3x2(v[4] * inv, v[5] * inv) | (e4m3x2(v[6] * inv, v[7] * inv) << 16));
}

template <int kTPR, bool kVec>
__device__ __forceinline__ void load_gamma(const void* gamma, int dtype, int i, int t, int cols, float (&v)[8]) {
  if (dtype == kBf16) load_group<kTPR, kVec>(static_cast<const __nv_bfloat16*>(gamma), i, t, cols, v);
  else load_group<kTPR, kVec>(static_cast<const float*>(gamma), i, t, cols, v);
}

// Sum or maximum over the kTPR threads of a row, the same value in each, in a
// fixed order.  `vals` is used by one reduction between two barriers.
template <int kTPR, bool kMax>
__device__ __forceinline__ float row_reduce(float v, float* vals) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const float o = __shfl_xor_sync(0xffffffffu, v, off);
    v = kMax ? fmaxf(v, o) : v + o;
  }
  if constexpr (kTPR > 32) {
    if ((threadIdx.x & 31) == 0) vals[threadIdx.x >> 5] = v;
    __syncthreads();
    v = vals[0];
#pragma unroll
    for (int w = 1; w < kTPR / 32; ++w) v = kMax ? fmaxf(v, vals[w]) : v + vals[w];
  }
  return v;
}

// The sums of kU rows at once, one barrier for all of them.
template <int kTPR, int kU>
__device__ __forceinline__ void rows_reduce(float (&v)[kU], float (*vals)[kTPR / 32]) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
#pragma unroll
    for (int u = 0; u < kU; ++u) v[u] += __shfl_xor_sync(0xffffffffu, v[u], off);
  if constexpr (kTPR > 32) {
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int u = 0; u < kU; ++u) vals[u][threadIdx.x >> 5] = v[u];
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      v[u] = vals[u][0];
#pragma unroll
      for (int w = 1; w < kTPR / 32; ++w) v[u] += vals[u][w];
    }
  }
}

// -------------------------------------------------------------- forward --

// One row per group of kTPR threads.
template <typename T, int kTPR, int kNV, bool kVec>
__global__ void __launch_bounds__(kTPR == 32 ? 256 : kTPR)
rmsnorm_kernel(const __grid_constant__ RmsnormArgs a) {
  constexpr int kThreads = kTPR == 32 ? 256 : kTPR;
  constexpr int kRows = kThreads / kTPR;
  __shared__ float vals[2][kTPR / 32];
  let_next_start();
  wait_for_predecessors();
  const int t = threadIdx.x % kTPR;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kTPR;
  if (r >= a.rows) return;                       // kTPR == 32: whole warps; otherwise the grid is exact
  const int cols = static_cast<int>(a.cols);       // kNormMaxCols at most
  float v[kNV][8];
  {
    const T* x = static_cast<const T*>(a.x) + r * a.x_ld;
#pragma unroll
    for (int i = 0; i < kNV; ++i) load_group<kTPR, kVec>(x, i, t, cols, v[i]);
  }
  if (a.residual) {
    const T* p = static_cast<const T*>(a.residual) + r * a.residual_ld;
    float w[kNV][8];
#pragma unroll
    for (int i = 0; i < kNV; ++i) load_group<kTPR, kVec>(p, i, t, cols, w[i]);
#pragma unroll
    for (int i = 0; i < kNV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] += w[i][j];
  }
  if (a.h) {
    T* h = static_cast<T*>(a.h) + r * a.h_ld;
#pragma unroll
    for (int i = 0; i < kNV; ++i) store_group<kTPR, kVec>(h, i, t, cols, v[i]);
  }
  if (a.norm) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kNV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += v[i][j] * v[i][j];
    ss = row_reduce<kTPR, false>(ss, vals[0]);
    const float rstd = 1.f / sqrtf(ss / static_cast<float>(cols) + a.eps);
    if (a.rstd && t == 0) a.rstd[r] = rstd;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      float g[8];
      load_gamma<kTPR, kVec>(a.gamma, a.gamma_dtype, i, t, cols, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * g[j];
    }
  }
  if (a.y) {
    __nv_bfloat16* y = reinterpret_cast<__nv_bfloat16*>(a.y) + r * a.y_ld;
#pragma unroll
    for (int i = 0; i < kNV; ++i) store_group<kTPR, kVec>(y, i, t, cols, v[i]);
  }
  if (a.q) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < kNV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // columns past the end hold zeros times rstd, which may be NaN: fmaxf drops it
        amax = fmaxf(amax, fabsf(v[i][j]));
      }
    const float scale = fmaxf(row_reduce<kTPR, true>(amax, vals[1]), kAmaxFloor) / kE4m3Max;
    if (t == 0) a.q_scale[r] = scale;
    const float inv = 1.f / scale;
    uint8_t* q = a.q + r * a.q_ld;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      if constexpr (kVec) {
        store_e4m3<kTPR>(q, i, t, cols, v[i], inv);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int c = column<kTPR, false>(i, j, t);
          if (c < cols) q[c] = e4m3(v[i][j] * inv);
        }
      }
    }
  }
}

// bf16 rows without a residual stay packed in registers and are unpacked at
// each use: half the registers a column, so twice the bytes in flight (the
// loads are all there is to wait for; unpacked, 14336 x 4096 in e4m3 took 33
// us, 5.4 TB/s).
template <int kTPR, int kNV>
__global__ void __launch_bounds__(kTPR) rmsnorm_packed_kernel(const __grid_constant__ RmsnormArgs a) {
  __shared__ float vals[2][kTPR / 32];
  let_next_start();
  wait_for_predecessors();
  const int t = threadIdx.x;
  const int64_t r = blockIdx.x;
  const int cols = static_cast<int>(a.cols);       // kNormMaxCols at most
  uint4 raw[kNV];
  {
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x) + r * a.x_ld;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = column<kTPR, true>(i, 0, t);
      raw[i] = c < cols ? *reinterpret_cast<const uint4*>(x + c) : make_uint4(0, 0, 0, 0);
    }
  }
  float rstd = 1.f;
  if (a.norm) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      float v[8];
      unpack8(raw[i], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += v[j] * v[j];
    }
    ss = row_reduce<kTPR, false>(ss, vals[0]);
    rstd = 1.f / sqrtf(ss / static_cast<float>(cols) + a.eps);
    if (a.rstd && t == 0) a.rstd[r] = rstd;
  }
  auto values = [&](int i, float (&v)[8]) {
    unpack8(raw[i], v);
    if (a.norm) {
      float g[8];
      load_gamma<kTPR, true>(a.gamma, a.gamma_dtype, i, t, cols, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = v[j] * rstd * g[j];
    }
  };
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kNV; ++i) {
    const int c = column<kTPR, true>(i, 0, t);
    if (a.h && c < cols) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.h) + r * a.h_ld + c) = raw[i];
    float v[8];
    values(i, v);
    if (a.y) store_group<kTPR, true>(reinterpret_cast<__nv_bfloat16*>(a.y) + r * a.y_ld, i, t, cols, v);
    // columns past the end hold zeros times rstd, which may be NaN: fmaxf drops it
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
  }
  if (a.q) {
    const float scale = fmaxf(row_reduce<kTPR, true>(amax, vals[1]), kAmaxFloor) / kE4m3Max;
    if (t == 0) a.q_scale[r] = scale;
    const float inv = 1.f / scale;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      float v[8];
      values(i, v);
      store_e4m3<kTPR>(a.q + r * a.q_ld, i, t, cols, v, inv);
    }
  }
}

// A long row in fp32 in shared memory.
template <typename T>
__global__ void __launch_bounds__(kLongThreads) rmsnorm_long_kernel(const __grid_constant__ RmsnormArgs a) {
  extern __shared__ float row[];
  __shared__ float vals[2][kLongThreads / 32];
  let_next_start();
  wait_for_predecessors();
  const int64_t r = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + r * a.x_ld;
  const T* res = a.residual ? static_cast<const T*>(a.residual) + r * a.residual_ld : nullptr;
  T* h = a.h ? static_cast<T*>(a.h) + r * a.h_ld : nullptr;
  float ss = 0.f;
  for (int64_t c = threadIdx.x; c < a.cols; c += kLongThreads) {
    float v = load_elem(x + c);
    if (res) v += load_elem(res + c);
    if (h) store_elem(h + c, v);
    row[c] = v;
    ss += v * v;
  }
  float rstd = 1.f;
  if (a.norm) {
    rstd = 1.f / sqrtf(row_reduce<kLongThreads, false>(ss, vals[0]) / static_cast<float>(a.cols) + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[r] = rstd;
  }
  float amax = 0.f;
  for (int64_t c = threadIdx.x; c < a.cols; c += kLongThreads) {   // this thread's own columns
    float y = row[c];
    if (a.norm)
      y = y * rstd *
          (a.gamma_dtype == kBf16 ? load_elem(static_cast<const __nv_bfloat16*>(a.gamma) + c)
                                  : static_cast<const float*>(a.gamma)[c]);
    row[c] = y;
    amax = fmaxf(amax, fabsf(y));
    if (a.y) store_elem(reinterpret_cast<__nv_bfloat16*>(a.y) + r * a.y_ld + c, y);
  }
  if (a.q) {
    const float scale = fmaxf(row_reduce<kLongThreads, true>(amax, vals[1]), kAmaxFloor) / kE4m3Max;
    if (threadIdx.x == 0) a.q_scale[r] = scale;
    const float inv = 1.f / scale;
    for (int64_t c = threadIdx.x; c < a.cols; c += kLongThreads) a.q[r * a.q_ld + c] = e4m3(row[c] * inv);
  }
}

// ------------------------------------------------------------- gradient --

// A group of 8 elements as loaded (bf16 stays packed until it is used).
template <typename T, bool kVec>
struct Raw {
  float v[8];
  __device__ __forceinline__ void get(float (&out)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) out[j] = v[j];
  }
};
template <>
struct Raw<__nv_bfloat16, true> {
  uint4 w;
  __device__ __forceinline__ void get(float (&out)[8]) const { unpack8(w, out); }
};

template <int kTPR, bool kVec, typename T>
__device__ __forceinline__ void load_raw(const T* row, int i, int t, int cols, Raw<T, kVec>& r) {
  if constexpr (kVec && sizeof(T) == 2) {
    const int c = column<kTPR, true>(i, 0, t);
    r.w = c < cols ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0, 0, 0, 0);
  } else {
    load_group<kTPR, kVec>(row, i, t, cols, r.v);
  }
}

// The gradient walks over many rows per CTA with a barrier in each, so it lives
// from rows that are independent of one another.  bf16 at 16 columns a thread:
// kU = 2 rows at a time share a barrier, and the loads run ahead of them in a
// ring (every thread copies the 16-byte pieces of the coming rows that it will
// itself use into its own places in shared memory, with cp.async: no registers,
// no barrier).  The other forms load a row into registers, with as many CTAs to
// an SM as that leaves; fp32, twice the bytes for the same work, reaches 6.1
// TB/s so, and a ring of the two rows that fit took it down to 4.5.
template <typename T, int kTPR, int kNV, bool kVec>
struct GradConfig {
  static constexpr int kThreads = kTPR == 32 ? 256 : kTPR;
  static constexpr bool kRing = kVec && sizeof(T) == 2 && kNV == 2;
  static constexpr int kU = kRing ? 2 : 1;
  static constexpr int kPieces = 3 * kNV;                                  // of a row: h, dh, dy
  static constexpr int kStageBytes = kU * kPieces * kThreads * 16;
  // CTAs to an SM: without the ring registers for 64 (bf16) or 80 (fp32) a
  // thread at 16 columns each, half as many CTAs at 32
  static constexpr int plain_ctas() {
    if (!kVec || kNV > 2) return kTPR == 32 && kNV > 2 ? 2 : 1;
    const int n = (sizeof(T) == 2 ? 1024 : 768) / kThreads;
    return n < 1 ? 1 : n;
  }
  static constexpr int kCtas = kRing ? 512 / kThreads : plain_ctas();
  static constexpr int kStages = kRing ? (216 * 1024) / kCtas / kStageBytes : 0;
  static_assert(!kRing || kStages >= 2, "the ring holds the rows in use and the ones on their way");
  static constexpr int kBytes = kStages * kStageBytes;
};

__device__ __forceinline__ void copy16(uint4* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// CTA b takes rows b, b + gridDim.x, ... (a row to a warp where kTPR is 32); a
// thread's columns stay the same, so its part of dgamma stays in registers, and
// the CTA writes its partial sums once.
template <typename T, int kTPR, int kNV, bool kVec>
__global__ void __launch_bounds__(kTPR == 32 ? 256 : kTPR, (GradConfig<T, kTPR, kNV, kVec>::kCtas))
rmsnorm_grad_kernel(const __grid_constant__ RmsnormGradArgs a) {
  using C = GradConfig<T, kTPR, kNV, kVec>;
  constexpr int kThreads = C::kThreads, kU = C::kU;
  constexpr int kRows = kThreads / kTPR;
  extern __shared__ uint4 ring[];              // [kStages][kU][kPieces][kThreads]
  __shared__ float vals[2][kU][kTPR / 32];
  __shared__ float join[kRows > 1 ? kRows * kTPR * 8 : 1];
  let_next_start();
  wait_for_predecessors();
  const int t = threadIdx.x % kTPR, sub = threadIdx.x / kTPR;
  const int cols = static_cast<int>(a.cols);       // kNormMaxCols at most
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  const float inv_cols = 1.f / static_cast<float>(cols);
  float part[kNV][8];
#pragma unroll
  for (int i = 0; i < kNV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) part[i][j] = 0.f;

  // this thread's pieces of rows r, r + step into stage s; a commit in any
  // case, so that the count of groups is that of stages
  auto fetch = [&](int64_t r, int s) {
    uint4* p = ring + static_cast<size_t>(s) * (kU * C::kPieces * kThreads) + threadIdx.x;
#pragma unroll
    for (int u = 0; u < kU; ++u, r += step)
      if (r < a.rows) {
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
          const int c = column<kTPR, true>(i, 0, t);
          if (c < cols) {
            uint4* q = p + (u * C::kPieces + i) * kThreads;
            copy16(q, static_cast<const T*>(a.h) + r * a.h_ld + c);
            if (a.dh) copy16(q + kNV * kThreads, static_cast<const T*>(a.dh) + r * a.dh_ld + c);
            copy16(q + 2 * kNV * kThreads, a.dy + r * a.dy_ld + c);
          }
        }
      }
    copy_commit();
  };
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRows + sub;
  if constexpr (C::kRing) {
    for (int s = 0; s < C::kStages - 1; ++s) fetch(r0 + s * kU * step, s);
  }
  int parity = 0, stage = 0;
  for (int64_t r = r0; r < a.rows; r += kU * step, parity ^= 1) {
    Raw<T, kVec> h[kU][kNV], dh[kU][kNV];
    Raw<__nv_bfloat16, kVec> dy[kU][kNV];
    float rstd[kU], dot[kU];
    if constexpr (C::kRing) {
      copy_wait<C::kStages - 2>();
      const uint4* p = ring + static_cast<size_t>(stage) * (kU * C::kPieces * kThreads) + threadIdx.x;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const bool row = r + u * step < a.rows;
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
          const bool in = row && column<kTPR, true>(i, 0, t) < cols;       // nothing was copied for the others
          const uint4* q = p + (u * C::kPieces + i) * kThreads;
          const uint4 zero = make_uint4(0, 0, 0, 0);
          h[u][i].w = in ? q[0] : zero;
          dh[u][i].w = in && a.dh ? q[kNV * kThreads] : zero;
          dy[u][i].w = in ? q[2 * kNV * kThreads] : zero;
        }
      }
    } else {
      const T* hp = static_cast<const T*>(a.h) + r * a.h_ld;
      const __nv_bfloat16* yp = reinterpret_cast<const __nv_bfloat16*>(a.dy) + r * a.dy_ld;
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        load_raw<kTPR, kVec>(hp, i, t, cols, h[0][i]);
        load_raw<kTPR, kVec>(yp, i, t, cols, dy[0][i]);
      }
      if (a.dh) {
        const T* sp = static_cast<const T*>(a.dh) + r * a.dh_ld;
#pragma unroll
        for (int i = 0; i < kNV; ++i) load_raw<kTPR, kVec>(sp, i, t, cols, dh[0][i]);
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      rstd[u] = r + u * step < a.rows ? a.rstd[r + u * step] : 0.f;
      dot[u] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      float gamma[8];
      load_gamma<kTPR, kVec>(a.gamma, a.gamma_dtype, i, t, cols, gamma);
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        float n[8], g[8];
        h[u][i].get(n);
        dy[u][i].get(g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float p = g[j] * n[j];            // dy h; rstd comes in once a sum
          part[i][j] += p * rstd[u];
          dot[u] += p * gamma[j];
        }
      }
    }
    if constexpr (C::kRing) {
      // the stage read one turn ago (its values are in use by now) takes the rows kStages - 1 turns ahead
      const int next = stage == 0 ? C::kStages - 1 : stage - 1;
      fetch(r + (C::kStages - 1) * kU * step, next);
      if (++stage == C::kStages) stage = 0;
    }
    if (a.dx) {
      rows_reduce<kTPR, kU>(dot, vals[parity]);
      // rstd (g - n mean(g n)) = rstd g - (rstd^3 mean(g h)) h
      float back[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) back[u] = -rstd[u] * rstd[u] * rstd[u] * (dot[u] * inv_cols);
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        float gamma[8];
        load_gamma<kTPR, kVec>(a.gamma, a.gamma_dtype, i, t, cols, gamma);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          if (r + u * step >= a.rows) break;
          float n[8], g[8], d[8];
          h[u][i].get(n);
          dy[u][i].get(g);
          if (a.dh) {
            dh[u][i].get(d);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) d[j] = 0.f;
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] += rstd[u] * (g[j] * gamma[j]) + back[u] * n[j];
          store_group<kTPR, kVec>(static_cast<T*>(a.dx) + (r + u * step) * a.dx_ld, i, t, cols, d);
        }
      }
    }
  }
  if (!a.dgamma) return;
  float* out = a.partial + static_cast<int64_t>(blockIdx.x) * a.cols;
  if constexpr (kRows == 1) {
#pragma unroll
    for (int i = 0; i < kNV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = column<kTPR, kVec>(i, j, t);
        if (c < cols) out[c] = part[i][j];
      }
  } else {
    // the warps' sums of 8 * kTPR columns at a time, added in order
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) join[(sub * 8 + j) * kTPR + t] = part[i][j];
      __syncthreads();
      for (int e = threadIdx.x; e < 8 * kTPR; e += kThreads) {
        float s = join[e];
        for (int w = 1; w < kRows; ++w) s += join[w * 8 * kTPR + e];
        const int c = column<kTPR, kVec>(i, e / kTPR, e % kTPR);
        if (c < cols) out[c] = s;
      }
    }
  }
}

// Rows longer than the registers hold: n and g in shared memory, the partial
// sums of dgamma in the workspace (each thread its own columns).
template <typename T>
__global__ void __launch_bounds__(kLongThreads) rmsnorm_grad_long_kernel(const __grid_constant__ RmsnormGradArgs a) {
  extern __shared__ float rows[];
  __shared__ float vals[2][kLongThreads / 32];
  let_next_start();
  wait_for_predecessors();
  float* n_row = rows;
  float* g_row = rows + a.cols;
  float* part = a.dgamma ? a.partial + static_cast<int64_t>(blockIdx.x) * a.cols : nullptr;
  int parity = 0;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x, parity ^= 1) {
    const float rstd = a.rstd[r];
    const T* h = static_cast<const T*>(a.h) + r * a.h_ld;
    const __nv_bfloat16* dy = reinterpret_cast<const __nv_bfloat16*>(a.dy) + r * a.dy_ld;
    float dot = 0.f;
    for (int64_t c = threadIdx.x; c < a.cols; c += kLongThreads) {
      const float n = load_elem(h + c) * rstd, d = load_elem(dy + c);
      const float g = d * (a.gamma_dtype == kBf16 ? load_elem(static_cast<const __nv_bfloat16*>(a.gamma) + c)
                                                  : static_cast<const float*>(a.gamma)[c]);
      if (part) part[c] = r == blockIdx.x ? d * n : part[c] + d * n;
      n_row[c] = n;
      g_row[c] = g;
      dot += g * n;
    }
    if (a.dx) {
      const float mean = row_reduce<kLongThreads, false>(dot, vals[parity]) / static_cast<float>(a.cols);
      T* dx = static_cast<T*>(a.dx) + r * a.dx_ld;
      for (int64_t c = threadIdx.x; c < a.cols; c += kLongThreads) {
        float v = rstd * (g_row[c] - n_row[c] * mean);
        if (a.dh) v += load_elem(static_cast<const T*>(a.dh) + r * a.dh_ld + c);
        store_elem(dx + c, v);
      }
    }
  }
}

// dgamma (+)= the partial sums, in a fixed order: a CTA takes 32 columns, its
// 32 warps every 32nd partial row, ten loads in flight together, and the warps'
// sums are added in order.
__global__ void __launch_bounds__(1024)
dgamma_kernel(const float* partial, int n_partial, int64_t cols, float* dgamma, int accumulate) {
  __shared__ float sums[32][32];
  let_next_start();
  wait_for_predecessors();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float s = 0.f;
  if (c < cols) {
    constexpr int kBatch = 10;
    for (int p0 = warp; p0 < n_partial; p0 += 32 * kBatch) {
      float v[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int p = p0 + 32 * j;
        v[j] = p < n_partial ? partial[static_cast<int64_t>(p) * cols + c] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) s += v[j];
    }
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < cols) {
#pragma unroll
    for (int w = 1; w < 32; ++w) s += sums[w][lane];
    dgamma[c] = accumulate ? dgamma[c] + s : s;
  }
}

// -------------------------------------------------------------- launches --

bool aligned(const void* p, int64_t ld, int64_t rows, int es, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) % bytes) == 0 && (rows <= 1 || (ld * es) % bytes == 0);
}

// Raises a kernel's shared-memory limit once per thread and device.
template <auto kKernel>
cudaError_t allow_smem(int bytes) {
  static thread_local int configured_dev = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev == configured_dev) return e;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) configured_dev = dev;
  return e;
}

template <typename T, int kTPR, int kNV>
cudaError_t forward_config(const RmsnormArgs& a, bool vec, cudaStream_t stream) {
  constexpr int kThreads = kTPR == 32 ? 256 : kTPR;
  constexpr int kRows = kThreads / kTPR;
  const unsigned grid = static_cast<unsigned>((a.rows + kRows - 1) / kRows);
  return launch_overlapped(vec ? rmsnorm_kernel<T, kTPR, kNV, true> : rmsnorm_kernel<T, kTPR, kNV, false>, grid, kThreads,
                           0, stream, 0, a);
}

template <typename T>
cudaError_t forward_typed(const RmsnormArgs& a, cudaStream_t stream) {
  const int es = static_cast<int>(sizeof(T));
  const bool vec = a.cols % 8 == 0 && aligned(a.x, a.x_ld, a.rows, es, 16) &&
                   aligned(a.residual, a.residual_ld, a.residual ? a.rows : 1, es, 16) &&
                   aligned(a.h, a.h_ld, a.h ? a.rows : 1, es, 16) && aligned(a.y, a.y_ld, a.y ? a.rows : 1, 2, 16) &&
                   aligned(a.q, a.q_ld, a.q ? a.rows : 1, 1, 8) && aligned(a.gamma, 0, 1, 1, 16);
  if constexpr (sizeof(T) == 2) {
    // from 2049 columns on; a row of fewer is too short for CTAs of this kind
    if (vec && !a.residual && a.cols > 2048 && a.cols <= kRegisterCols) {
      const unsigned grid = static_cast<unsigned>(a.rows);
      if (a.cols <= 4096) return launch_overlapped(rmsnorm_packed_kernel<128, 4>, grid, 128, 0, stream, 0, a);
      if (a.cols <= 8192) return launch_overlapped(rmsnorm_packed_kernel<256, 4>, grid, 256, 0, stream, 0, a);
      return launch_overlapped(rmsnorm_packed_kernel<512, 4>, grid, 512, 0, stream, 0, a);
    }
  }
  if (a.cols <= 256) return forward_config<T, 32, 1>(a, vec, stream);
  if (a.cols <= 512) return forward_config<T, 32, 2>(a, vec, stream);
  if (a.cols <= 1024) return forward_config<T, 32, 4>(a, vec, stream);
  if (a.cols <= 2048) return forward_config<T, 128, 2>(a, vec, stream);
  if (a.cols <= 4096) return forward_config<T, 256, 2>(a, vec, stream);
  if (a.cols <= 8192) return forward_config<T, 512, 2>(a, vec, stream);
  if (a.cols <= kRegisterCols) return forward_config<T, 512, 4>(a, vec, stream);
  const cudaError_t e = allow_smem<rmsnorm_long_kernel<T>>(static_cast<int>(kNormMaxCols * sizeof(float)));
  if (e != cudaSuccess) return e;
  return launch_overlapped(rmsnorm_long_kernel<T>, static_cast<unsigned>(a.rows), kLongThreads, a.cols * sizeof(float),
                           stream, 0, a);
}

// CTAs of a kernel that the GPU holds at a time (kept per thread and device).
template <auto kKernel>
int resident_ctas(int threads, int smem) {
  static thread_local int cached_dev = -1, cached = 1;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (dev != cached_dev) {
    int per_sm = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kKernel, threads, smem) != cudaSuccess || per_sm < 1)
      per_sm = 1;
    cached = per_sm * num_sms();
    cached_dev = dev;
  }
  return cached;
}

template <typename T, int kTPR, int kNV, bool kVec>
cudaError_t grad_launch(const RmsnormGradArgs& a, int* grid, cudaStream_t stream) {
  constexpr int kThreads = kTPR == 32 ? 256 : kTPR;
  constexpr int kRows = kThreads / kTPR;
  constexpr int kSmem = GradConfig<T, kTPR, kNV, kVec>::kBytes;
  int64_t n = (a.rows + kRows - 1) / kRows;
  const cudaError_t e = allow_smem<rmsnorm_grad_kernel<T, kTPR, kNV, kVec>>(kSmem);
  if (e != cudaSuccess) return e;
  const int64_t most = resident_ctas<rmsnorm_grad_kernel<T, kTPR, kNV, kVec>>(kThreads, kSmem);
  if (n > most) n = most;
  if (n > kNormPartialRows) n = kNormPartialRows;
  *grid = static_cast<int>(n);
  return launch_overlapped(rmsnorm_grad_kernel<T, kTPR, kNV, kVec>, static_cast<unsigned>(*grid), kThreads, kSmem, stream,
                           0, a);
}

template <typename T, int kTPR, int kNV>
cudaError_t grad_config(const RmsnormGradArgs& a, bool vec, int* grid, cudaStream_t stream) {
  return vec ? grad_launch<T, kTPR, kNV, true>(a, grid, stream) : grad_launch<T, kTPR, kNV, false>(a, grid, stream);
}

template <typename T>
cudaError_t grad_typed(const RmsnormGradArgs& a, int* grid, cudaStream_t stream) {
  const int es = static_cast<int>(sizeof(T));
  const bool vec = a.cols % 8 == 0 && aligned(a.h, a.h_ld, a.rows, es, 16) && aligned(a.dy, a.dy_ld, a.rows, 2, 16) &&
                   aligned(a.dh, a.dh_ld, a.dh ? a.rows : 1, es, 16) &&
                   aligned(a.dx, a.dx_ld, a.dx ? a.rows : 1, es, 16) && aligned(a.gamma, 0, 1, 1, 16);
  if (a.cols <= 256) return grad_config<T, 32, 1>(a, vec, grid, stream);
  if (a.cols <= 512) return grad_config<T, 32, 2>(a, vec, grid, stream);
  if (a.cols <= 1024) return grad_config<T, 32, 4>(a, vec, grid, stream);
  if (a.cols <= 2048) return grad_config<T, 128, 2>(a, vec, grid, stream);
  if (a.cols <= 4096) return grad_config<T, 256, 2>(a, vec, grid, stream);
  if (a.cols <= 8192) return grad_config<T, 512, 2>(a, vec, grid, stream);
  if (a.cols <= kRegisterCols) return grad_config<T, 512, 4>(a, vec, grid, stream);
  const cudaError_t e = allow_smem<rmsnorm_grad_long_kernel<T>>(static_cast<int>(2 * kNormGradMaxCols * sizeof(float)));
  if (e != cudaSuccess) return e;
  const int64_t n = a.rows < num_sms() ? a.rows : num_sms();
  *grid = static_cast<int>(n < kNormPartialRows ? n : kNormPartialRows);
  return launch_overlapped(rmsnorm_grad_long_kernel<T>, static_cast<unsigned>(*grid), kLongThreads,
                           2 * a.cols * sizeof(float), stream, 0, a);
}

}  // namespace

cudaError_t launch_rmsnorm(const RmsnormArgs& a, cudaStream_t stream) {
  if (a.rows <= 0) return cudaSuccess;
  return a.dtype == kBf16 ? forward_typed<__nv_bfloat16>(a, stream) : forward_typed<float>(a, stream);
}

cudaError_t launch_rmsnorm_grad(const RmsnormGradArgs& a, cudaStream_t stream) {
  int grid = 0;
  if (a.rows > 0) {
    prof_begin(OPT_KERNEL_RMSNORM_GRAD, 1, a.rows, a.cols, stream);
    const cudaError_t e =
        a.dtype == kBf16 ? grad_typed<__nv_bfloat16>(a, &grid, stream) : grad_typed<float>(a, &grid, stream);
    prof_end(stream);
    if (e != cudaSuccess) return e;
  }
  if (!a.dgamma) return cudaSuccess;
  prof_begin(OPT_KERNEL_RMSNORM_DGAMMA, 1, a.rows, a.cols, stream);
  const cudaError_t e = launch_overlapped(dgamma_kernel, static_cast<unsigned>((a.cols + 31) / 32), 1024, 0, stream, 0,
                                          static_cast<const float*>(a.partial), grid, a.cols, a.dgamma, a.accumulate);
  prof_end(stream);
  return e;
}

}  // namespace mpopt
