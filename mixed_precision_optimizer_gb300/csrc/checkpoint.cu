// Activation checkpoints in 8 bits (sm_103a): e4m3 codes with a power of two for
// every 32 columns of a row, and their way back.
//
//   2^e, the smallest with max |x| <= 448 * 2^e;  q = rne_e4m3(x * 2^-e)
//   z = q * 2^e;  y = act(z);  dz = dy * act'(z)
//
// Both are bound by HBM: every element is read once and written once.  Powers of
// two cost no rounding, so z needs no more than e4m3's four significant bits and
// a bf16 output is z itself.  Where rows start on 16 bytes a thread has 8
// elements, four neighbouring lanes a block of 32; otherwise a warp has a
// block, an element to each lane.

#include "activation.cuh"
#include "elements.cuh"
#include "internal.h"
#include "overlap.cuh"

namespace mpopt {
namespace {

constexpr int kThreads = 256;
constexpr int kBlock = OPT_CHECKPOINT_BLOCK;
constexpr int kMinExp = -116;            // the smallest code is 2^-9: restored values stay normal numbers
constexpr int kMaxExp = 120;             // of the largest finite value, 2^128 less a step
constexpr float kMaxTop = 240.f;         // the largest code there: 256 * 2^120 would be an infinity

// Magnitude as an integer, 0 for an infinity or a NaN.
__device__ __forceinline__ uint32_t magnitude(float v) {
  const uint32_t u = __float_as_uint(v) & 0x7fffffffu;
  return u < 0x7f800000u ? u : 0u;
}

// The exponent e of a block whose largest magnitude has these bits:
// 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exponent(uint32_t amax) {
  const int e = static_cast<int>(amax >> 23) - 127 - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < kMinExp ? kMinExp : e;
}

__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// An infinity becomes a NaN: the conversion would saturate it.
__device__ __forceinline__ float code_input(float v, float inv) {
  return fabsf(v) == __uint_as_float(0x7f800000u) ? __uint_as_float(0x7fc00000u) : v * inv;
}

__device__ __forceinline__ float below_infinity(float v) { return v != v ? v : fminf(fmaxf(v, -kMaxTop), kMaxTop); }

struct SaveArgs {
  const void* x;
  uint8_t *q, *scale;
  int64_t rows, cols, x_ld, q_ld, scale_ld;
  int64_t groups;        // of 8 columns to a row (vector access)
};

template <typename T>
__global__ void __launch_bounds__(kThreads) checkpoint_save_kernel(const __grid_constant__ SaveArgs a) {
  let_next_start();
  wait_for_predecessors();
  // four lanes to a block of 32 columns; lanes past the row's last group take part with zeros
  const int64_t per_row = (a.groups + 3) & ~int64_t(3);
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t r = at / per_row;
  const int64_t g = at - r * per_row;
  const bool in = r < a.rows && g < a.groups;
  float v[8];
  if (in) {
    load8(static_cast<const T*>(a.x) + r * a.x_ld + g * 8, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
  }
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = max(amax, magnitude(v[j]));
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  if (!in) return;
  const int e = scale_exponent(amax);
  const float inv = power_of_two(-e);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = code_input(v[j], inv);
  if (e == kMaxExp) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = below_infinity(v[j]);
  }
  *reinterpret_cast<uint2*>(a.q + r * a.q_ld + g * 8) =
      make_uint2(e4m3x2(v[0], v[1]) | (e4m3x2(v[2], v[3]) << 16), e4m3x2(v[4], v[5]) | (e4m3x2(v[6], v[7]) << 16));
  if ((g & 3) == 0) a.scale[r * a.scale_ld + g / 4] = static_cast<uint8_t>(e + 127);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) checkpoint_save_single_kernel(const __grid_constant__ SaveArgs a) {
  let_next_start();
  wait_for_predecessors();
  const int64_t blocks = (a.cols + kBlock - 1) / kBlock;
  const int64_t at = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / 32;
  const int64_t r = at / blocks, b = at - r * blocks;
  if (r >= a.rows) return;                           // whole warps
  const int64_t c = b * kBlock + (threadIdx.x & 31);
  const bool in = c < a.cols;
  const float v = in ? load_elem(static_cast<const T*>(a.x) + r * a.x_ld + c) : 0.f;
  const int e = scale_exponent(__reduce_max_sync(0xffffffffu, magnitude(v)));
  const float t = code_input(v, power_of_two(-e));
  if (in) a.q[r * a.q_ld + c] = e4m3(e == kMaxExp ? below_infinity(t) : t);
  if ((threadIdx.x & 31) == 0) a.scale[r * a.scale_ld + b] = static_cast<uint8_t>(e + 127);
}

// --------------------------------------------------------------- restore --

struct RestoreArgs {
  opt_checkpoint_args a;
  int64_t groups;
};

// Two codes as fp32; e4m3 values are exact in fp16.
__device__ __forceinline__ float2 decode2(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes & 0xffffu), __NV_E4M3);
  return __half22float2(__half2(h));
}

// Bytes that no checkpoint has are taken as the nearest that it may have.
__device__ __forceinline__ float scale_of(uint8_t byte) {
  const int b = byte, least = 127 + kMinExp;
  return power_of_two((b < least ? least : b > 127 + kMaxExp ? 127 + kMaxExp : b) - 127);
}

template <int kAct>
__global__ void __launch_bounds__(kThreads) checkpoint_restore_kernel(const __grid_constant__ RestoreArgs p) {
  let_next_start();
  wait_for_predecessors();
  const opt_checkpoint_args& a = p.a;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t r = at / p.groups, g = at - r * p.groups;
  if (r >= a.rows) return;
  const uint2 w = *reinterpret_cast<const uint2*>(a.q + r * a.q_ld + g * 8);
  const float s = scale_of(a.scale[r * a.scale_ld + g / 4]);
  float dy[8];
  if (a.dz) load8(reinterpret_cast<const __nv_bfloat16*>(a.dy) + r * a.dy_ld + g * 8, dy);
  float z[8], v[8];
  const uint32_t u[2] = {w.x, w.y};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 d = decode2(u[j / 2] >> (j % 2 * 16));
    z[2 * j] = d.x * s;
    z[2 * j + 1] = d.y * s;
  }
  if (a.z) store8(reinterpret_cast<__nv_bfloat16*>(a.z) + r * a.z_ld + g * 8, z);
  if (a.y) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = activate<kAct>(z[j]);
    store8(reinterpret_cast<__nv_bfloat16*>(a.y) + r * a.y_ld + g * 8, v);
  }
  if (a.dz) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = dy[j] * activate_grad<kAct>(z[j]);
    store8(reinterpret_cast<__nv_bfloat16*>(a.dz) + r * a.dz_ld + g * 8, v);
  }
}

template <int kAct>
__global__ void __launch_bounds__(kThreads) checkpoint_restore_single_kernel(const __grid_constant__ RestoreArgs p) {
  let_next_start();
  wait_for_predecessors();
  const opt_checkpoint_args& a = p.a;
  const int64_t blocks = (a.cols + kBlock - 1) / kBlock;
  const int64_t at = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / 32;
  const int64_t r = at / blocks, b = at - r * blocks;
  const int64_t c = b * kBlock + (threadIdx.x & 31);
  if (r >= a.rows || c >= a.cols) return;
  const float z = decode2(a.q[r * a.q_ld + c]).x * scale_of(a.scale[r * a.scale_ld + b]);
  if (a.z) store_elem(reinterpret_cast<__nv_bfloat16*>(a.z) + r * a.z_ld + c, z);
  if (a.y) store_elem(reinterpret_cast<__nv_bfloat16*>(a.y) + r * a.y_ld + c, activate<kAct>(z));
  if (a.dz)
    store_elem(reinterpret_cast<__nv_bfloat16*>(a.dz) + r * a.dz_ld + c,
               load_elem(reinterpret_cast<const __nv_bfloat16*>(a.dy) + r * a.dy_ld + c) * activate_grad<kAct>(z));
}

// Whether every row starts on `bytes` bytes.
bool rows_on(const void* p, int64_t ld, int es, int64_t rows, uintptr_t bytes) {
  return !p || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && (rows <= 1 || static_cast<uintptr_t>(ld) * es % bytes == 0));
}

dim3 grid_of(int64_t threads) { return dim3(static_cast<unsigned>((threads + kThreads - 1) / kThreads)); }

template <int kAct>
cudaError_t restore_with(const RestoreArgs& p, bool vec, dim3 grid, cudaStream_t stream) {
  return vec ? launch_overlapped(checkpoint_restore_kernel<kAct>, grid, kThreads, 0, stream, 0, p)
             : launch_overlapped(checkpoint_restore_single_kernel<kAct>, grid, kThreads, 0, stream, 0, p);
}

}  // namespace

cudaError_t launch_checkpoint_save(const void* x, int64_t x_ld, int dtype, int64_t rows, int64_t cols, uint8_t* q,
                                   int64_t q_ld, uint8_t* scale, int64_t scale_ld, cudaStream_t stream) {
  const int es = dtype == kBf16 ? 2 : 4;
  const bool vec = cols % 8 == 0 && rows_on(x, x_ld, es, rows, 16) && rows_on(q, q_ld, 1, rows, 8);
  const SaveArgs a{x, q, scale, rows, cols, x_ld, q_ld, scale_ld, cols / 8};
  if (vec) {
    const dim3 grid = grid_of(rows * ((cols / 8 + 3) & ~int64_t(3)));
    return dtype == kBf16 ? launch_overlapped(checkpoint_save_kernel<__nv_bfloat16>, grid, kThreads, 0, stream, 0, a)
                          : launch_overlapped(checkpoint_save_kernel<float>, grid, kThreads, 0, stream, 0, a);
  }
  const dim3 grid = grid_of(rows * ((cols + kBlock - 1) / kBlock) * 32);
  return dtype == kBf16 ? launch_overlapped(checkpoint_save_single_kernel<__nv_bfloat16>, grid, kThreads, 0, stream, 0, a)
                        : launch_overlapped(checkpoint_save_single_kernel<float>, grid, kThreads, 0, stream, 0, a);
}

cudaError_t launch_checkpoint_restore(const opt_checkpoint_args& a, cudaStream_t stream) {
  const bool vec = a.cols % 8 == 0 && rows_on(a.q, a.q_ld, 1, a.rows, 8) && rows_on(a.dy, a.dy_ld, 2, a.rows, 16) &&
                   rows_on(a.z, a.z_ld, 2, a.rows, 16) && rows_on(a.y, a.y_ld, 2, a.rows, 16) &&
                   rows_on(a.dz, a.dz_ld, 2, a.rows, 16);
  const RestoreArgs p{a, a.cols / 8};
  const dim3 grid = grid_of(vec ? a.rows * (a.cols / 8) : a.rows * ((a.cols + kBlock - 1) / kBlock) * 32);
  switch (a.act) {
    case OPT_ACT_RELU: return restore_with<OPT_ACT_RELU>(p, vec, grid, stream);
    case OPT_ACT_GELU: return restore_with<OPT_ACT_GELU>(p, vec, grid, stream);
    case OPT_ACT_SILU: return restore_with<OPT_ACT_SILU>(p, vec, grid, stream);
    default: return restore_with<OPT_ACT_NONE>(p, vec, grid, stream);
  }
}

}  // namespace mpopt
