// RMS norm with the residual's addition and 8-bit rows, and its gradient
// (sm_103a):
//
//   h = x + residual;  rstd = 1 / sqrt(mean h^2 + eps);  y = h * rstd * gamma
//   scale = max(max |y|, 1e-30) / 448;  q = rne_e4m3(y * (1 / scale))
//
//   n = h * rstd;  g = dy * gamma;  c = mean(g n)
//   dx = rstd * (g - n c) + dh;  dgamma = sum over rows of dy n
//
// All of it is bound by HBM: every input element is read once and every
// output written once, a row staying in registers between its statistics and
// its outputs.  A row of up to 1024 columns belongs to one warp (no barrier,
// eight rows to a CTA), a longer one to a CTA of 128 to 512 threads, up to
// 16384 columns in registers; longer rows are kept in fp32 in shared memory.
// Where every row starts on 16 bytes a thread moves 8 elements at a time
// (kVector).  Rows of an odd width start anywhere, but where all tensors' rows
// start equally far past a multiple of 8 elements (dense ones do), the groups
// of 8 begin at the row's first multiple of 8, and the up to 14 elements before
// the first and after the last group go to one thread each (kShifted).
// Otherwise single elements, neighbours in neighbouring lanes (kSingle).

#include "../../include/mpopt.h"
#include "elements.cuh"
#include "internal.h"
#include "overlap.cuh"

namespace mpopt {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kAmaxFloor = 1e-30f;
constexpr int kLongThreads = 512;             // rows longer than the register kernels take
constexpr int64_t kRegisterCols = 16384;

enum Access : int { kSingle = 0, kVector = 1, kShifted = 2 };

// -------------------------------------------------------- a thread's share --

// A thread's share of a row: kNV groups of 8 columns.  With kSingle element j
// of group i is column (i * 8 + j) * kTPR + t.  Otherwise the group starts at
// column first + (i * kTPR + t) * 8 and there are groups up to column `end`: 0 and
// the width with kVector; with kShifted `first` is where the row has its first
// multiple of 8 elements, `end` where no whole group is left, and `edge` the
// column outside of them that this thread takes (-1: none).
struct Share {
  int first, end, edge;
};

template <int kAccess>
__device__ __forceinline__ Share share_of(int64_t start, int cols, int t) {
  Share s{0, cols, -1};
  if constexpr (kAccess == kShifted) {
    const int head = static_cast<int>(-start & 7);
    s.first = head < cols ? head : cols;
    s.end = s.first + ((cols - s.first) & ~7);
    const int e = t < 8 ? t : s.end + t - 8;
    if (t < 8 ? e < s.first : t < 16 && e < cols) s.edge = e;
  }
  return s;
}

template <int kTPR, int kAccess>
__device__ __forceinline__ int column(const Share& s, int i, int j, int t) {
  return kAccess == kSingle ? (i * 8 + j) * kTPR + t : s.first + (i * kTPR + t) * 8 + j;
}

template <int kTPR, int kAccess, typename T>
__device__ __forceinline__ void load_group(const T* row, const Share& s, int i, int t, float (&v)[8]) {
  if constexpr (kAccess != kSingle) {
    const int c = column<kTPR, kAccess>(s, i, 0, t);
    if (c < s.end) {
      load8(row + c, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = column<kTPR, kAccess>(s, i, j, t);
      v[j] = c < s.end ? load_elem(row + c) : 0.f;
    }
  }
}

template <int kTPR, int kAccess, typename T>
__device__ __forceinline__ void store_group(T* row, const Share& s, int i, int t, const float (&v)[8]) {
  if constexpr (kAccess == kSingle) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = column<kTPR, kAccess>(s, i, j, t);
      if (c < s.end) store_elem(row + c, v[j]);
    }
  } else {
    const int c = column<kTPR, kAccess>(s, i, 0, t);
    if (c < s.end) store8(row + c, v);
  }
}

// The same with kShifted for an output whose groups do not start on 16 bytes:
// a warp's groups go through shared memory (256 floats a warp), so that
// neighbouring lanes store neighbouring columns.  The whole warp calls.
template <int kTPR, typename T>
__device__ __forceinline__ void spread_group(T* row, const Share& s, int i, int t, const float (&v)[8], float* staging) {
  const int lane = t & 31, base = column<kTPR, kShifted>(s, i, 0, t - lane);
  float* mine = staging + (threadIdx.x >> 5) * 256;
  reinterpret_cast<float4*>(mine)[lane] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(mine)[32 + lane] = make_float4(v[4], v[5], v[6], v[7]);
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int e = k * 32 + lane;                   // element e % 8 of lane e / 8
    if (base + e < s.end) store_elem(row + base + e, mine[(e & 4) * 32 + (e / 8) * 4 + (e & 3)]);
  }
  __syncwarp();
}

// A group times inv in e4m3, 8 bytes.
template <int kTPR, int kAccess>
__device__ __forceinline__ void store_e4m3(uint8_t* row, const Share& s, int i, int t, const float (&v)[8], float inv) {
  if constexpr (kAccess == kSingle) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = column<kTPR, kAccess>(s, i, j, t);
      if (c < s.end) row[c] = e4m3(v[j] * inv);
    }
  } else {
    const int c = column<kTPR, kAccess>(s, i, 0, t);
    if (c < s.end)
      *reinterpret_cast<uint2*>(row + c) =
          make_uint2(e4m3x2(v[0] * inv, v[1] * inv) | (e4m3x2(v[2] * inv, v[3] * inv) << 16),
                     e4m3x2(v[4] * inv, v[5] * inv) | (e4m3x2(v[6] * inv, v[7] * inv) << 16));
  }
}

__device__ __forceinline__ float gamma_elem(const void* gamma, int dtype, int c) {
  return dtype == kBf16 ? load_elem(static_cast<const __nv_bfloat16*>(gamma) + c) : static_cast<const float*>(gamma)[c];
}

// With kShifted gamma's groups do not start on 16 bytes: single elements.
template <int kTPR, int kAccess, typename T>
__device__ __forceinline__ void load_gamma_typed(const T* gamma, const Share& s, int i, int t, float (&v)[8]) {
  if constexpr (kAccess == kShifted) {
    const int c = column<kTPR, kAccess>(s, i, 0, t);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c < s.end ? load_elem(gamma + c + j) : 0.f;
  } else {
    load_group<kTPR, kAccess>(gamma, s, i, t, v);
  }
}
template <int kTPR, int kAccess>
__device__ __forceinline__ void load_gamma(const void* gamma, int dtype, const Share& s, int i, int t, float (&v)[8]) {
  if (dtype == kBf16) load_gamma_typed<kTPR, kAccess>(static_cast<const __nv_bfloat16*>(gamma), s, i, t, v);
  else load_gamma_typed<kTPR, kAccess>(static_cast<const float*>(gamma), s, i, t, v);
}

// A group of 8 elements as loaded (bf16 stays packed until it is used).
template <typename T, int kAccess>
struct Raw {
  float v[8];
  __device__ __forceinline__ void get(float (&out)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) out[j] = v[j];
  }
};
struct PackedRaw {
  uint4 w;
  __device__ __forceinline__ void get(float (&out)[8]) const { unpack8(w, out); }
};
template <>
struct Raw<__nv_bfloat16, kVector> : PackedRaw {};
template <>
struct Raw<__nv_bfloat16, kShifted> : PackedRaw {};

template <int kTPR, int kAccess, typename T>
__device__ __forceinline__ void load_raw(const T* row, const Share& s, int i, int t, Raw<T, kAccess>& r) {
  if constexpr (kAccess != kSingle && sizeof(T) == 2) {
    const int c = column<kTPR, kAccess>(s, i, 0, t);
    r.w = c < s.end ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0, 0, 0, 0);
  } else {
    load_group<kTPR, kAccess>(row, s, i, t, r.v);
  }
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
template <typename T, int kTPR, int kNV, int kAccess>
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
  const int cols = static_cast<int>(a.cols);       // kRegisterCols at most
  const Share s = share_of<kAccess>(a.shift + r * a.x_ld, cols, t);
  const bool edge = kAccess == kShifted && s.edge >= 0;
  float v[kNV][8], ve = 0.f;
  {
    const T* x = static_cast<const T*>(a.x) + r * a.x_ld;
#pragma unroll
    for (int i = 0; i < kNV; ++i) load_group<kTPR, kAccess>(x, s, i, t, v[i]);
    if (edge) ve = load_elem(x + s.edge);
  }
  if (a.residual) {
    const T* p = static_cast<const T*>(a.residual) + r * a.residual_ld;
    float w[kNV][8], we = 0.f;
#pragma unroll
    for (int i = 0; i < kNV; ++i) load_group<kTPR, kAccess>(p, s, i, t, w[i]);
    if (edge) we = load_elem(p + s.edge);
#pragma unroll
    for (int i = 0; i < kNV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] += w[i][j];
    ve += we;
  }
  if (a.h) {
    T* h = static_cast<T*>(a.h) + r * a.h_ld;
#pragma unroll
    for (int i = 0; i < kNV; ++i) store_group<kTPR, kAccess>(h, s, i, t, v[i]);
    if (edge) store_elem(h + s.edge, ve);
  }
  if (a.norm) {
    float ss = ve * ve;
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
      load_gamma<kTPR, kAccess>(a.gamma, a.gamma_dtype, s, i, t, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * g[j];
    }
    if (edge) ve = ve * rstd * gamma_elem(a.gamma, a.gamma_dtype, s.edge);
  }
  if (a.y) {
    __nv_bfloat16* y = reinterpret_cast<__nv_bfloat16*>(a.y) + r * a.y_ld;
#pragma unroll
    for (int i = 0; i < kNV; ++i) store_group<kTPR, kAccess>(y, s, i, t, v[i]);
    if (edge) store_elem(y + s.edge, ve);
  }
  if (a.q) {
    float amax = fabsf(ve);
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
    for (int i = 0; i < kNV; ++i) store_e4m3<kTPR, kAccess>(q, s, i, t, v[i], inv);
    if (edge) q[s.edge] = e4m3(ve * inv);
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
  const int cols = static_cast<int>(a.cols);       // kRegisterCols at most
  const Share s = share_of<kVector>(0, cols, t);
  uint4 raw[kNV];
  {
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x) + r * a.x_ld;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = column<kTPR, kVector>(s, i, 0, t);
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
      load_gamma<kTPR, kVector>(a.gamma, a.gamma_dtype, s, i, t, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = v[j] * rstd * g[j];
    }
  };
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kNV; ++i) {
    const int c = column<kTPR, kVector>(s, i, 0, t);
    if (a.h && c < cols) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.h) + r * a.h_ld + c) = raw[i];
    float v[8];
    values(i, v);
    if (a.y) store_group<kTPR, kVector>(reinterpret_cast<__nv_bfloat16*>(a.y) + r * a.y_ld, s, i, t, v);
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
      store_e4m3<kTPR, kVector>(a.q + r * a.q_ld, s, i, t, v, inv);
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

// The gradient walks over many rows per CTA with a barrier in each, so it lives
// from rows that are independent of one another.  bf16 at 16 columns a thread:
// kU = 2 rows at a time share a barrier, and the loads run ahead of them in a
// ring (every thread copies the 16-byte pieces of the coming rows that it will
// itself use into its own places in shared memory, with cp.async: no registers,
// no barrier).  The other forms load a row into registers, with as many CTAs to
// an SM as that leaves; fp32, twice the bytes for the same work, reaches 6.1
// TB/s so, and a ring of the two rows that fit took it down to 4.5.  With
// kShifted a thread's gamma lies in fp32 in its own places in shared memory,
// since its groups do not start on 16 bytes of gamma, and the rows' edges take
// registers: 80 a thread (8192 x 2545 in bf16: 49 us, with 64 or 128 55 and 58;
// in bf16 two CTAs of 512 need 64: 4096 x 4097 53 us, one CTA 69),
// for a warp's row of two groups 128 (8192 x 505: 12.3 us, with 80 18.2), and
// rows of 513 to 1024 columns take 128 threads instead of a warp (5000 x 1023:
// 21 us against 23, in fp32 26 against 32).  Single elements took 149 us for
// 8192 x 2545.
template <typename T, int kTPR, int kNV, int kAccess>
struct GradConfig {
  static constexpr int kThreads = kTPR == 32 ? 256 : kTPR;
  static constexpr bool kRing = kAccess == kVector && sizeof(T) == 2 && kNV == 2;
  static constexpr int kU = kRing ? 2 : 1;
  static constexpr int kPieces = 3 * kNV;                                  // of a row: h, dh, dy
  static constexpr int kStageBytes = kU * kPieces * kThreads * 16;
  // CTAs to an SM: without the ring registers for 64 (bf16) or 80 (fp32) a
  // thread at 16 columns each, half as many CTAs at 32
  static constexpr int plain_ctas() {
    if (kAccess == kSingle || kNV > 2) return kTPR == 32 && kNV > 2 ? 2 : 1;
    if (kAccess == kShifted && kTPR == 32 && kNV == 2) return 2;
    const int n = (sizeof(T) == 2 && (kAccess != kShifted || kThreads == 512) ? 1024 : 768) / kThreads;
    return n < 1 ? 1 : n;
  }
  static constexpr int kCtas = kRing ? 512 / kThreads : plain_ctas();
  static constexpr int kStages = kRing ? (216 * 1024) / kCtas / kStageBytes : 0;
  static_assert(!kRing || kStages >= 2, "the ring holds the rows in use and the ones on their way");
  static constexpr int kBytes = kAccess == kShifted ? kThreads * (kNV + 1) * 32 : kStages * kStageBytes;
};

// CTA b takes rows b, b + gridDim.x, ... (a row to a warp where kTPR is 32, with
// kSingle and kVector rows next to one another); a thread's columns stay the
// same, so its part of dgamma stays in registers, and the CTA writes its partial
// sums once.  With kShifted gridDim.x is a multiple of 8 (or the number of rows),
// which gives all rows of a CTA one shift.
template <typename T, int kTPR, int kNV, int kAccess>
__global__ void __launch_bounds__(kTPR == 32 ? 256 : kTPR, (GradConfig<T, kTPR, kNV, kAccess>::kCtas))
rmsnorm_grad_kernel(const __grid_constant__ RmsnormGradArgs a) {
  using C = GradConfig<T, kTPR, kNV, kAccess>;
  constexpr int kThreads = C::kThreads, kU = C::kU;
  constexpr int kRows = kThreads / kTPR;
  extern __shared__ uint4 ring[];              // [kStages][kU][kPieces][kThreads]; 
                                               // kShifted: gamma, [kNV][2][kThreads], and the warps' staging
  __shared__ float vals[2][kU][kTPR / 32];
  __shared__ float join[kRows > 1 ? kRows * kTPR * 8 : 1];
  let_next_start();
  wait_for_predecessors();
  const int t = threadIdx.x % kTPR, sub = threadIdx.x / kTPR;
  const int cols = static_cast<int>(a.cols);       // kRegisterCols at most
  const Share s = share_of<kAccess>(a.shift + blockIdx.x * a.h_ld, cols, t);
  const bool edge = kAccess == kShifted && s.edge >= 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  const float inv_cols = 1.f / static_cast<float>(cols);
  float part[kNV][8], part_e = 0.f;
#pragma unroll
  for (int i = 0; i < kNV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) part[i][j] = 0.f;

  // this thread's pieces of rows r, r + step into stage s; a commit in any
  // case, so that the count of groups is that of stages
  auto fetch = [&](int64_t r, int at) {
    uint4* p = ring + static_cast<size_t>(at) * (kU * C::kPieces * kThreads) + threadIdx.x;
#pragma unroll
    for (int u = 0; u < kU; ++u, r += step)
      if (r < a.rows) {
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
          const int c = column<kTPR, kVector>(s, i, 0, t);
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
  const int64_t r0 = kAccess == kShifted ? blockIdx.x + static_cast<int64_t>(sub) * gridDim.x
                                         : static_cast<int64_t>(blockIdx.x) * kRows + sub;
  float4* own_gamma = reinterpret_cast<float4*>(ring) + threadIdx.x;
  if constexpr (kAccess == kShifted) {
    if (r0 < a.rows) {
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        float g[8];
        load_gamma<kTPR, kAccess>(a.gamma, a.gamma_dtype, s, i, t, g);
        own_gamma[(2 * i) * kThreads] = make_float4(g[0], g[1], g[2], g[3]);
        own_gamma[(2 * i + 1) * kThreads] = make_float4(g[4], g[5], g[6], g[7]);
      }
    }
  }
  const float gamma_e = edge ? gamma_elem(a.gamma, a.gamma_dtype, s.edge) : 0.f;
  auto gamma_group = [&](int i, float (&g)[8]) {
    if constexpr (kAccess == kShifted) {
      const float4 p = own_gamma[(2 * i) * kThreads], q = own_gamma[(2 * i + 1) * kThreads];
      g[0] = p.x, g[1] = p.y, g[2] = p.z, g[3] = p.w, g[4] = q.x, g[5] = q.y, g[6] = q.z, g[7] = q.w;
    } else {
      load_gamma<kTPR, kAccess>(a.gamma, a.gamma_dtype, s, i, t, g);
    }
  };
  if constexpr (C::kRing) {
    for (int at = 0; at < C::kStages - 1; ++at) fetch(r0 + at * kU * step, at);
  }
  int parity = 0, stage = 0;
  for (int64_t r = r0; r < a.rows; r += kU * step, parity ^= 1) {
    Raw<T, kAccess> h[kU][kNV], dh[kU][kNV];
    Raw<__nv_bfloat16, kAccess> dy[kU][kNV];
    float rstd[kU], dot[kU], he = 0.f, dhe = 0.f, dye = 0.f;      // kShifted has kU = 1
    if constexpr (C::kRing) {
      copy_wait<C::kStages - 2>();
      const uint4* p = ring + static_cast<size_t>(stage) * (kU * C::kPieces * kThreads) + threadIdx.x;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const bool row = r + u * step < a.rows;
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
          const bool in = row && column<kTPR, kVector>(s, i, 0, t) < cols;       // nothing was copied for the others
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
        load_raw<kTPR, kAccess>(hp, s, i, t, h[0][i]);
        load_raw<kTPR, kAccess>(yp, s, i, t, dy[0][i]);
      }
      if (edge) {
        he = load_elem(hp + s.edge);
        dye = load_elem(yp + s.edge);
        if (a.dh) dhe = load_elem(static_cast<const T*>(a.dh) + r * a.dh_ld + s.edge);
      }
      if (a.dh) {
        const T* sp = static_cast<const T*>(a.dh) + r * a.dh_ld;
#pragma unroll
        for (int i = 0; i < kNV; ++i) load_raw<kTPR, kAccess>(sp, s, i, t, dh[0][i]);
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
      gamma_group(i, gamma);
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        float n[8], g[8];
        h[u][i].get(n);
        dy[u][i].get(g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float p = g[j] * (n[j] * rstd[u]);     // n first: of order one whatever h's size
          part[i][j] += p;
          dot[u] += p * gamma[j];
        }
      }
    }
    if constexpr (kAccess == kShifted) {
      const float p = dye * (he * rstd[0]);
      part_e += p;
      dot[0] += p * gamma_e;
    }
    if constexpr (C::kRing) {
      // the stage read one turn ago (its values are in use by now) takes the rows kStages - 1 turns ahead
      const int next = stage == 0 ? C::kStages - 1 : stage - 1;
      fetch(r + (C::kStages - 1) * kU * step, next);
      if (++stage == C::kStages) stage = 0;
    }
    if (a.dx) {
      rows_reduce<kTPR, kU>(dot, vals[parity]);
      // rstd (g - n mean(g n)) = rstd g - (rstd mean(g n) rstd) h, in this order: mean(g n) is of g's
      // size, and rstd^2 stays in fp32's range wherever the forward pass's squares do (rstd^3 does not:
      // a row of 1e14 lost its projection).  n formed once more here: in fp32 85.4 us against 81.5 for
      // 8192 x 4096.
      float back[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) back[u] = -(rstd[u] * (dot[u] * inv_cols)) * rstd[u];
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        float gamma[8];
        gamma_group(i, gamma);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          if (r + u * step >= a.rows) break;     // the same for a warp
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
          T* dx = static_cast<T*>(a.dx) + (r + u * step) * a.dx_ld;
          if (kAccess == kShifted && !a.dx_grouped)
            spread_group<kTPR>(dx, s, i, t, d, reinterpret_cast<float*>(ring + 2 * kNV * kThreads));
          else
            store_group<kTPR, kAccess>(dx, s, i, t, d);
        }
      }
      if (edge)
        store_elem(static_cast<T*>(a.dx) + r * a.dx_ld + s.edge, dhe + (rstd[0] * (dye * gamma_e) + back[0] * he));
    }
  }
  if (!a.dgamma) return;
  float* out = a.partial + static_cast<int64_t>(blockIdx.x) * a.cols;
  if constexpr (kRows == 1) {
#pragma unroll
    for (int i = 0; i < kNV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = column<kTPR, kAccess>(s, i, j, t);
        if (c < s.end) out[c] = part[i][j];
      }
    if (edge) out[s.edge] = part_e;
  } else {
    // the warps' sums of 8 * kTPR columns at a time, added in order
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) join[(sub * 8 + j) * kTPR + t] = part[i][j];
      __syncthreads();
      for (int e = threadIdx.x; e < 8 * kTPR; e += kThreads) {
        float sum = join[e];
        for (int w = 1; w < kRows; ++w) sum += join[w * 8 * kTPR + e];
        const int c = column<kTPR, kAccess>(s, i, e / kTPR, e % kTPR);
        if (c < s.end) out[c] = sum;
      }
    }
    if constexpr (kAccess == kShifted) {
      __syncthreads();
      join[sub * kTPR + t] = part_e;
      __syncthreads();
      if (sub == 0 && edge) {
        float sum = part_e;
        for (int w = 1; w < kRows; ++w) sum += join[w * kTPR + t];
        out[s.edge] = sum;
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

// How far past a multiple of 8 elements the first rows of all given tensors
// start, if it is the same for all and stays so from row to row; otherwise -1.
// The first one is always given.
struct RowTensor {
  const void* p;
  int64_t ld;
  int es;
};
template <int kN>
int common_shift(const RowTensor (&tensors)[kN], int64_t rows) {
  int shift = -1;
  int64_t ld = 0;
  for (const RowTensor& x : tensors) {
    if (!x.p) continue;
    const int own = static_cast<int>((reinterpret_cast<uintptr_t>(x.p) / x.es) & 7);
    if (shift >= 0 && (own != shift || (rows > 1 && ((x.ld - ld) & 7) != 0))) return -1;
    shift = own, ld = x.ld;
  }
  return shift;
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
cudaError_t forward_config(const RmsnormArgs& a, Access access, cudaStream_t stream) {
  constexpr int kThreads = kTPR == 32 ? 256 : kTPR;
  constexpr int kRows = kThreads / kTPR;
  const unsigned grid = static_cast<unsigned>((a.rows + kRows - 1) / kRows);
  return launch_overlapped(access == kVector    ? rmsnorm_kernel<T, kTPR, kNV, kVector>
                           : access == kShifted ? rmsnorm_kernel<T, kTPR, kNV, kShifted>
                                                : rmsnorm_kernel<T, kTPR, kNV, kSingle>,
                           grid, kThreads, 0, stream, 0, a);
}

template <typename T>
cudaError_t forward_typed(RmsnormArgs a, cudaStream_t stream) {
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
  Access access = vec ? kVector : kSingle;
  if (!vec && a.cols <= kRegisterCols) {
    a.shift = common_shift({{a.x, a.x_ld, es}, {a.residual, a.residual_ld, es}, {a.h, a.h_ld, es},
                            {a.y, a.y_ld, 2}, {a.q, a.q_ld, 1}}, a.rows);
    if (a.shift >= 0) access = kShifted;
  }
  if (a.cols <= 256) return forward_config<T, 32, 1>(a, access, stream);
  if (a.cols <= 512) return forward_config<T, 32, 2>(a, access, stream);
  if (a.cols <= 1024) return forward_config<T, 32, 4>(a, access, stream);
  if (a.cols <= 2048) return forward_config<T, 128, 2>(a, access, stream);
  if (a.cols <= 4096) return forward_config<T, 256, 2>(a, access, stream);
  if (a.cols <= 8192) return forward_config<T, 512, 2>(a, access, stream);
  if (a.cols <= kRegisterCols) return forward_config<T, 512, 4>(a, access, stream);
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

template <typename T, int kTPR, int kNV, int kAccess>
cudaError_t grad_launch(const RmsnormGradArgs& a, int* grid, cudaStream_t stream) {
  constexpr int kThreads = kTPR == 32 ? 256 : kTPR;
  constexpr int kRows = kThreads / kTPR;
  constexpr int kSmem = GradConfig<T, kTPR, kNV, kAccess>::kBytes;
  int64_t n = (a.rows + kRows - 1) / kRows;
  const cudaError_t e = allow_smem<rmsnorm_grad_kernel<T, kTPR, kNV, kAccess>>(kSmem);
  if (e != cudaSuccess) return e;
  const int64_t most = resident_ctas<rmsnorm_grad_kernel<T, kTPR, kNV, kAccess>>(kThreads, kSmem);
  if (n > most) n = most;
  if (n > kNormPartialRows) n = kNormPartialRows;
  if (kAccess == kShifted) {
    // a multiple of 8, or as many CTAs as rows (then no CTA has a second row);
    // never more than the rows, for which the workspace has been sized
    n = n < most && n < kNormPartialRows ? (n + 7) / 8 * 8 : n < 8 ? 8 : n / 8 * 8;
    if (n > a.rows) n = a.rows;
  }
  *grid = static_cast<int>(n);
  return launch_overlapped(rmsnorm_grad_kernel<T, kTPR, kNV, kAccess>, static_cast<unsigned>(*grid), kThreads, kSmem, stream,
                           0, a);
}

template <typename T, int kTPR, int kNV>
cudaError_t grad_config(const RmsnormGradArgs& a, Access access, int* grid, cudaStream_t stream) {
  if (access == kVector) return grad_launch<T, kTPR, kNV, kVector>(a, grid, stream);
  if (access == kShifted) return grad_launch<T, kTPR, kNV, kShifted>(a, grid, stream);
  return grad_launch<T, kTPR, kNV, kSingle>(a, grid, stream);
}

template <typename T>
cudaError_t grad_typed(RmsnormGradArgs a, int* grid, cudaStream_t stream) {
  const int es = static_cast<int>(sizeof(T));
  const bool vec = a.cols % 8 == 0 && aligned(a.h, a.h_ld, a.rows, es, 16) && aligned(a.dy, a.dy_ld, a.rows, 2, 16) &&
                   aligned(a.dh, a.dh_ld, a.dh ? a.rows : 1, es, 16) &&
                   aligned(a.dx, a.dx_ld, a.dx ? a.rows : 1, es, 16) && aligned(a.gamma, 0, 1, 1, 16);
  Access access = vec ? kVector : kSingle;
  if (!vec && a.cols <= kRegisterCols) {
    // dx has no part in the choice: its bits do not depend on where it lies
    const RowTensor h{a.h, a.h_ld, es};
    a.shift = common_shift({h, {a.dy, a.dy_ld, 2}, {a.dh, a.dh_ld, es}}, a.rows);
    if (a.shift >= 0) {
      access = kShifted;
      a.dx_grouped = common_shift({h, {a.dx, a.dx_ld, es}}, a.rows) >= 0;
    }
  }
  if (a.cols <= 256) return grad_config<T, 32, 1>(a, access, grid, stream);
  if (a.cols <= 512) return grad_config<T, 32, 2>(a, access, grid, stream);
  if (a.cols <= 1024) {
    if (access == kShifted) return grad_launch<T, 128, 1, kShifted>(a, grid, stream);
    return vec ? grad_launch<T, 32, 4, kVector>(a, grid, stream) : grad_launch<T, 32, 4, kSingle>(a, grid, stream);
  }
  if (a.cols <= 2048) return grad_config<T, 128, 2>(a, access, grid, stream);
  if (a.cols <= 4096) return grad_config<T, 256, 2>(a, access, grid, stream);
  if (a.cols <= 8192) return grad_config<T, 512, 2>(a, access, grid, stream);
  if (a.cols <= kRegisterCols) return grad_config<T, 512, 4>(a, access, grid, stream);
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
