// Activation checkpoints in 8 bits (sm_103a): e4m3 codes with a power of two for
// every 32 columns of a row, and their way back.
//
//   2^e, the smallest with max |x| <= 448 * 2^e;  q = rne_e4m3(x * 2^-e)
//   z = q * 2^e;  y = act(z);  dz = dy * act'(z)
//
// Both are bound by HBM: every element is read once and written once.  Powers of
// two cost no rounding, so z needs no more than e4m3's four significant bits and
// a bf16 output is z itself.  Where rows start on 16 bytes a thread has 8 columns
// of four (two) rows, four neighbouring lanes a block of 32: 8192 x 14336 in bf16
// 54 us (0.99 of the measured copy rate), back through GELU with its gradient 126
// (0.98); a row a thread and a flat grid, whose 64-bit divisions are a third of
// the instructions, took 89 and 158.  Otherwise a warp has a block, an element to
// each lane.

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
};

// A CTA's share where rows start on 16 bytes: 2^log_tpr threads to a row, a group
// of 8 columns to each, and kRows rows to a thread, whose loads are on their way
// together.
struct Tiles {
  int log_tpr;
  uint32_t slices;       // CTAs to a row
};

struct Place {
  int64_t row, group;    // of the first row
  int step;              // rows from one of a thread's to the next
};

template <int kRows>
__device__ __forceinline__ Place place_of(const Tiles& t) {
  const uint32_t block = blockIdx.x / t.slices, slice = blockIdx.x - block * t.slices;
  const int step = kThreads >> t.log_tpr;
  return Place{static_cast<int64_t>(block) * step * kRows + (threadIdx.x >> t.log_tpr),
               (static_cast<int64_t>(slice) << t.log_tpr) + (threadIdx.x & ((1 << t.log_tpr) - 1)), step};
}

// A group as loaded, and the largest of its magnitudes as the bits of an fp32 value
// (an infinity's or a NaN's where it has one).
template <typename T>
struct Group;
template <>
struct Group<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void clear() { w = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&v)[8]) const { unpack8(w, v); }
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t k = 0x7fff7fffu;
    const uint32_t m = __vmaxu2(__vmaxu2(w.x & k, w.y & k), __vmaxu2(w.z & k, w.w & k));
    return max(m << 16, m & 0xffff0000u);
  }
};
template <>
struct Group<float> {
  float v[8];
  __device__ __forceinline__ void load(const float* p) { load8(p, v); }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
  }
  __device__ __forceinline__ void get(float (&out)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) out[j] = v[j];
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
    return m;
  }
};

// The maximum over the four lanes of a block.
__device__ __forceinline__ uint32_t block_max(uint32_t v) {
  v = max(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return max(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

constexpr int kSaveRows = 4;

template <typename T>
__global__ void __launch_bounds__(kThreads) checkpoint_save_kernel(const __grid_constant__ SaveArgs a,
                                                                   const __grid_constant__ Tiles tiles) {
  let_next_start();
  wait_for_predecessors();
  const Place at = place_of<kSaveRows>(tiles);
  Group<T> x[kSaveRows];
  bool in[kSaveRows];
#pragma unroll
  for (int u = 0; u < kSaveRows; ++u) {
    const int64_t r = at.row + u * at.step;
    in[u] = r < a.rows && at.group * 8 < a.cols;       // lanes past the row take part with zeros
    if (in[u]) x[u].load(static_cast<const T*>(a.x) + r * a.x_ld + at.group * 8);
    else x[u].clear();
  }
#pragma unroll
  for (int u = 0; u < kSaveRows; ++u) {
    uint32_t amax = block_max(x[u].top());
    float v[8];
    x[u].get(v);
    const bool odd = __any_sync(0xffffffffu, amax >= 0x7f800000u);
    if (odd) {                                   // an infinity or a NaN in one of the warp's blocks
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, magnitude(v[j]));
      amax = block_max(m);
    }
    if (!in[u]) continue;
    const int64_t r = at.row + u * at.step;
    const int e = scale_exponent(amax);
    const float inv = power_of_two(-e);
    if (odd || e == kMaxExp) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = code_input(v[j], inv);
      if (e == kMaxExp) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = below_infinity(v[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= inv;
    }
    *reinterpret_cast<uint2*>(a.q + r * a.q_ld + at.group * 8) =
        make_uint2(e4m3x2(v[0], v[1]) | (e4m3x2(v[2], v[3]) << 16), e4m3x2(v[4], v[5]) | (e4m3x2(v[6], v[7]) << 16));
    if ((at.group & 3) == 0) a.scale[r * a.scale_ld + at.group / 4] = static_cast<uint8_t>(e + 127);
  }
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

constexpr int kRestoreRows = 2;

template <int kAct>
__global__ void __launch_bounds__(kThreads) checkpoint_restore_kernel(const __grid_constant__ opt_checkpoint_args a,
                                                                      const __grid_constant__ Tiles tiles) {
  let_next_start();
  wait_for_predecessors();
  const Place at = place_of<kRestoreRows>(tiles);
  const int64_t c = at.group * 8;
  if (c >= a.cols) return;
  uint2 w[kRestoreRows];
  uint8_t byte[kRestoreRows];
  uint4 dy[kRestoreRows];
#pragma unroll
  for (int u = 0; u < kRestoreRows; ++u) {
    const int64_t r = at.row + u * at.step;
    if (r >= a.rows) break;
    w[u] = *reinterpret_cast<const uint2*>(a.q + r * a.q_ld + c);
    byte[u] = a.scale[r * a.scale_ld + at.group / 4];
    if (a.dz) dy[u] = *reinterpret_cast<const uint4*>(a.dy + r * a.dy_ld + c);
  }
#pragma unroll
  for (int u = 0; u < kRestoreRows; ++u) {
    const int64_t r = at.row + u * at.step;
    if (r >= a.rows) break;
    const float s = scale_of(byte[u]);
    float z[8], v[8];
    const uint32_t q[2] = {w[u].x, w[u].y};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 d = decode2(q[j / 2] >> (j % 2 * 16));
      z[2 * j] = d.x * s;
      z[2 * j + 1] = d.y * s;
    }
    if (a.z) store8(reinterpret_cast<__nv_bfloat16*>(a.z) + r * a.z_ld + c, z);
    if (a.dz) {                                  // y and the derivative share their sigmoid
      float g[8];
      unpack8(dy[u], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = activate<kAct>(z[j]);
        g[j] *= activate_grad<kAct>(z[j]);
      }
      store8(reinterpret_cast<__nv_bfloat16*>(a.dz) + r * a.dz_ld + c, g);
    } else if (a.y) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = activate<kAct>(z[j]);
    }
    if (a.y) store8(reinterpret_cast<__nv_bfloat16*>(a.y) + r * a.y_ld + c, v);
  }
}

template <int kAct>
__global__ void __launch_bounds__(kThreads) checkpoint_restore_single_kernel(const __grid_constant__ opt_checkpoint_args a) {
  let_next_start();
  wait_for_predecessors();
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

// At least the four threads of a block to a row.
Tiles tiles_of(int64_t cols) {
  const int64_t groups = cols / 8;
  int log_tpr = 2;
  while (log_tpr < 8 && (int64_t(1) << log_tpr) < groups) ++log_tpr;
  return Tiles{log_tpr, static_cast<uint32_t>((groups + (int64_t(1) << log_tpr) - 1) >> log_tpr)};
}

dim3 grid_of(const Tiles& t, int64_t rows, int rows_per_thread) {
  const int64_t per_cta = static_cast<int64_t>(kThreads >> t.log_tpr) * rows_per_thread;
  return dim3(static_cast<unsigned>((rows + per_cta - 1) / per_cta * t.slices));
}

template <typename T>
cudaError_t save(const SaveArgs& a, bool vec, cudaStream_t stream) {
  if (vec) {
    const Tiles t = tiles_of(a.cols);
    return launch_overlapped(checkpoint_save_kernel<T>, grid_of(t, a.rows, kSaveRows), kThreads, 0, stream, 0, a, t);
  }
  return launch_overlapped(checkpoint_save_single_kernel<T>, grid_of(a.rows * ((a.cols + kBlock - 1) / kBlock) * 32), kThreads, 0,
                           stream, 0, a);
}

template <int kAct>
cudaError_t restore(const opt_checkpoint_args& a, bool vec, cudaStream_t stream) {
  if (vec) {
    const Tiles t = tiles_of(a.cols);
    return launch_overlapped(checkpoint_restore_kernel<kAct>, grid_of(t, a.rows, kRestoreRows), kThreads, 0, stream, 0, a, t);
  }
  return launch_overlapped(checkpoint_restore_single_kernel<kAct>, grid_of(a.rows * ((a.cols + kBlock - 1) / kBlock) * 32),
                           kThreads, 0, stream, 0, a);
}

}  // namespace

cudaError_t launch_checkpoint_save(const void* x, int64_t x_ld, int dtype, int64_t rows, int64_t cols, uint8_t* q,
                                   int64_t q_ld, uint8_t* scale, int64_t scale_ld, cudaStream_t stream) {
  const bool vec = cols % 8 == 0 && rows_on(x, x_ld, dtype == kBf16 ? 2 : 4, rows, 16) && rows_on(q, q_ld, 1, rows, 8);
  const SaveArgs a{x, q, scale, rows, cols, x_ld, q_ld, scale_ld};
  return dtype == kBf16 ? save<__nv_bfloat16>(a, vec, stream) : save<float>(a, vec, stream);
}

cudaError_t launch_checkpoint_restore(const opt_checkpoint_args& a, cudaStream_t stream) {
  const bool vec = a.cols % 8 == 0 && rows_on(a.q, a.q_ld, 1, a.rows, 8) && rows_on(a.dy, a.dy_ld, 2, a.rows, 16) &&
                   rows_on(a.z, a.z_ld, 2, a.rows, 16) && rows_on(a.y, a.y_ld, 2, a.rows, 16) &&
                   rows_on(a.dz, a.dz_ld, 2, a.rows, 16);
  switch (a.act) {
    case OPT_ACT_RELU: return restore<OPT_ACT_RELU>(a, vec, stream);
    case OPT_ACT_GELU: return restore<OPT_ACT_GELU>(a, vec, stream);
    case OPT_ACT_SILU: return restore<OPT_ACT_SILU>(a, vec, stream);
    default: return restore<OPT_ACT_NONE>(a, vec, stream);
  }
}

}  // namespace mpopt
