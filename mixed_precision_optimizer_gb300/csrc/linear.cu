// The linear layer's products on the 5th-generation tensor cores (sm_103a):
//
//   forward   y = act(x w^T + bias) + residual        bf16 or e4m3 operands
//   dx        (dz w) * act'(z)                        bf16
//   dw        dz^T x (+ main_grad)                    bf16 operands, fp32 result
//
// All three are out[b][a] = sum_k A[a][k] B[b][k], where `a` is the index that
// is contiguous in the output: a TMEM lane is an `a` and a TMEM column a `b`,
// so a warp's loads and stores of one column are contiguous whatever the
// output's row distance and alignment, and the bias and the weight scale of a
// lane are one register.  An operand stored [index][k] is K-major, one stored
// [k][index] (w in dx, both operands of dw) MN-major: no transposed copy is
// made.
//
// One CTA per 128 x 128 tile: warp 0 loads k-blocks of 128 bytes by TMA into a
// ring, warp 1 issues the MMAs, warps 2-5 run the epilogue.  Out-of-range rows
// and columns are filled with zeros by the TMA and never stored.

#include <cuda_bf16.h>

#include "../../include/mpopt.h"
#include "internal.h"
#include "tc_common.cuh"

namespace mpopt {
namespace {

constexpr int BM = 128;                        // A indices of a tile (TMEM lanes)
constexpr int BN = 128;                        // B indices of a tile (TMEM columns)
constexpr int kStages = 6;
constexpr int kStageA = BM * kRowBytes;
constexpr int kStageB = BN * kRowBytes;
constexpr int kStageBytes = kStageA + kStageB;
constexpr int kEpiWarps = 4;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kTmemCols = BN;
constexpr uint32_t kSmemBytes = kStages * kStageBytes + 1024 /*align*/ + 256 /*barriers*/;
static_assert(kSmemBytes <= 232448, "dynamic shared memory above the 227 KB a CTA may use");

struct LinearParams {
  LinearArgs g;
  int k_blocks;
  int64_t tiles_a;
};

// ------------------------------------------------------------ activations --

// sqrt(2/pi) and the cubic's coefficient of the tanh form of GELU; with
// (1 + tanh u) / 2 = sigmoid(2 u) both activations are u * sigmoid(t(u)).
__device__ __forceinline__ float sigmoid(float t) { return 1.f / (1.f + __expf(-t)); }

constexpr float kGelu2 = 1.5957691216057308f;   // 2 sqrt(2/pi)
constexpr float kGeluCubic = 0.044715f;

__device__ __forceinline__ float activate(float z, int act) {
  if (act == OPT_ACT_RELU) return z > 0.f || z != z ? z : 0.f;
  if (act == OPT_ACT_GELU) return z * sigmoid(kGelu2 * (z + kGeluCubic * z * z * z));
  if (act == OPT_ACT_SILU) return z * sigmoid(z);
  return z;
}

__device__ __forceinline__ float activate_grad(float z, int act) {
  if (act == OPT_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  if (act == OPT_ACT_GELU) {
    const float p = sigmoid(kGelu2 * (z + kGeluCubic * z * z * z));
    return p + z * p * (1.f - p) * (kGelu2 * (1.f + 3.f * kGeluCubic * z * z));
  }
  if (act == OPT_ACT_SILU) {
    const float p = sigmoid(z);
    return p + z * p * (1.f - p);
  }
  return 1.f;
}

__device__ __forceinline__ float bf16_at(const uint16_t* p, int64_t i) {
  return __uint_as_float(static_cast<uint32_t>(p[i]) << 16);
}

__device__ __forceinline__ uint16_t to_bf16(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// ------------------------------------------------------------ tensor cores --

// Instruction descriptor: fp32 accumulator (bits 4-5 = 1), operand formats in
// bits 7-9 and 10-12 (kind::f16: 1 = bf16; kind::f8f6f4: 0 = e4m3), MN-major
// operands flagged in bits 15 (A) and 16 (B), N >> 3 in bits 17-22, M >> 4 in
// bits 24-28.
__host__ __device__ constexpr uint32_t linear_idesc(bool fp8, bool a_mn, bool b_mn, int m, int n) {
  return (1u << 4) | ((fp8 ? 0u : 1u) << 7) | ((fp8 ? 0u : 1u) << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

template <bool kFp8>
__device__ __forceinline__ void mma_1cta(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  if constexpr (kFp8)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void commit_1cta(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// `count` rows (K-major: one box of `count` rows) or columns (MN-major: boxes
// of 64 columns x 64 k rows) of an operand, from `index`, k-block `kb`.
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap* map, uint32_t bar, bool mn, int index,
                                             int count, int kb, int elems) {
  if (mn) {
    for (int j = 0; j < count / 64; ++j) tma_load_2d(dst + j * kMnBlockBytes, map, bar, index + 64 * j, kb * elems);
  } else {
    tma_load_2d(dst, map, bar, kb * elems, index);
  }
}

// -------------------------------------------------------------- epilogue --

// Column j of the tile is output row b0 + j; this lane is output column `a`.
template <bool kFp8>
__device__ __forceinline__ void epilogue_columns(const LinearArgs& g, int64_t a, int64_t b0, const float (&v)[32]) {
  if (a >= g.na) return;
  const int n = static_cast<int>(g.nb - b0 < 32 ? g.nb - b0 : 32);
  if (g.mode == kLinearDw) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < n) {
        float* p = g.dw + (b0 + j) * g.dw_ld + a;
        *p = g.accumulate ? *p + v[j] : v[j];
      }
    return;
  }
  if (g.mode == kLinearDx) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < n) {
        float d = v[j];
        if (g.z_in) d *= activate_grad(bf16_at(g.z_in, (b0 + j) * g.z_ld + a), g.act);
        g.y[(b0 + j) * g.y_ld + a] = to_bf16(d);
      }
    return;
  }
  const float wscale = kFp8 ? g.a_scale[a] : 1.f;
  float bias = 0.f;
  if (g.bias)
    bias = g.bias_dtype == kBf16 ? bf16_at(static_cast<const uint16_t*>(g.bias), a)
                                 : static_cast<const float*>(g.bias)[a];
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (j < n) {
      float z = v[j];
      if (kFp8) z *= wscale * g.b_scale[b0 + j];
      z += bias;
      if (g.z_out) g.z_out[(b0 + j) * g.z_ld + a] = to_bf16(z);
      float y = activate(z, g.act);
      if (g.residual) y += bf16_at(g.residual, (b0 + j) * g.residual_ld + a);
      g.y[(b0 + j) * g.y_ld + a] = to_bf16(y);
    }
}

// ---------------------------------------------------------------- kernel --

template <bool kFp8>
__global__ void __launch_bounds__(kThreads, 1)
linear_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
              const __grid_constant__ LinearParams P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* status = P.g.header;
  constexpr int kElems = kFp8 ? 128 : 64;
  const bool a_mn = P.g.A.mn_major != 0, b_mn = P.g.B.mn_major != 0;
  const int64_t a0 = static_cast<int64_t>(blockIdx.x % P.tiles_a) * BM;
  const int64_t b0 = static_cast<int64_t>(blockIdx.x / P.tiles_a) * BN;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(acc_full), 1);
    *abort_flag = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty), acc_bar = smem_u32(acc_full);

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t sa0 = smem_u32(smem), sb0 = sa0 + kStages * kStageA;
      uint32_t s = 0, ph = 0;
      int kb = 0;
      for (; kb < P.k_blocks; ++kb) {
        if (!mbar_wait(empty0 + 8 * s, ph ^ 1u, abort_flag, status, kStatusTimeoutEmpty)) break;
        mbar_expect_tx(full0 + 8 * s, kStageBytes);
        load_operand(sa0 + s * kStageA, &map_a, full0 + 8 * s, a_mn, static_cast<int>(a0), BM, kb, kElems);
        load_operand(sb0 + s * kStageB, &map_b, full0 + 8 * s, b_mn, static_cast<int>(b0), BN, kb, kElems);
        if (++s == kStages) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (kb < P.k_blocks) {
        // aborting: give copies in flight time to land before the CTA exits
        const unsigned long long t0 = global_ns();
        while (global_ns() - t0 < 10000000ull) {
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = linear_idesc(kFp8, a_mn, b_mn, BM, BN);
      const uint32_t sa0 = smem_u32(smem), sb0 = sa0 + kStages * kStageA;
      const uint64_t ad0 = a_mn ? smem_desc_mn(sa0) : smem_desc(sa0);
      const uint64_t bd0 = b_mn ? smem_desc_mn(sb0) : smem_desc(sb0);
      // one MMA's K step: 32 bytes of a K-major row, or 16 rows of an MN-major block
      const uint32_t ka = (a_mn ? 16 * kRowBytes : 32) >> 4, kb_step = (b_mn ? 16 * kRowBytes : 32) >> 4;
      uint32_t s = 0, ph = 0;
      for (int kb = 0; kb < P.k_blocks; ++kb) {
        if (!mbar_wait(full0 + 8 * s, ph, abort_flag, status, kStatusTimeoutFull)) break;
        tc_fence_after();
        const uint64_t ad = ad0 + s * (kStageA >> 4), bd = bd0 + s * (kStageB >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_1cta<kFp8>(tmem_base, ad + ka * kk, bd + kb_step * kk, idesc, (kb > 0 || kk > 0) ? 1u : 0u);
        commit_1cta(empty0 + 8 * s);
        if (++s == kStages) {
          s = 0;
          ph ^= 1u;
        }
      }
      // also after an aborted loop: the MMAs issued complete before TMEM goes
      commit_1cta(acc_bar);
      const unsigned long long t0 = global_ns();
      while (!mbar_try(acc_bar, 0)) {
        if (global_ns() - t0 > kWaitLimitNs) {
          *abort_flag = 1u;
          atomicCAS(status, 0u, static_cast<uint32_t>(kStatusTimeoutDrain));
          break;
        }
      }
    }
  } else {
    const int quarter = warp & 3;
    const bool ready = mbar_wait(acc_bar, 0, abort_flag, status, kStatusTimeoutAcc) && !*abort_flag;
    if (__all_sync(0xffffffffu, ready)) {
      tc_fence_after();
      for (int c = 0; c < BN && b0 + c < P.g.nb; c += 32) {
        float v[32];
        tmem_ld32(tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + c, v);
        epilogue_columns<kFp8>(P.g, a0 + quarter * 32 + lane, b0 + c, v);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols) : "memory");
  }
}

// ------------------------------------------------------- smaller kernels --

// Column sums of dz, in a fixed order: a CTA takes 32 columns, its 8 warps
// every eighth row, and the warps' sums are added in order.
__global__ void __launch_bounds__(256)
column_sums_kernel(const uint16_t* dz, int64_t ld, int64_t m, int64_t n, float* out, int accumulate) {
  __shared__ float sums[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float s = 0.f;
  if (c < n)
    for (int64_t r = warp; r < m; r += 8) s += bf16_at(dz, r * ld + c);
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < n) {
    float t = 0.f;
    for (int w = 0; w < 8; ++w) t += sums[w][lane];
    out[c] = accumulate ? out[c] + t : t;
  }
}

template <typename T>
__global__ void __launch_bounds__(256)
repack_kernel(const T* src, int64_t src_ld, T* dst, int64_t dst_ld, int64_t rows, int64_t cols) {
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
    for (int64_t c = threadIdx.x; c < cols; c += 256) dst[r * dst_ld + c] = src[r * src_ld + c];
}

// -------------------------------------------------------------- host side --

// 2-D map of an operand: K-major [index][k], box of 128 bytes of k x
// `box_rows` indices; MN-major [k][index], box of 64 indices x 64 k.
cudaError_t make_operand_map(CUtensorMap* map, const LinearOperand& o, int64_t n_index, int64_t nk, bool fp8,
                             int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const int es = fp8 ? 1 : 2;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(o.mn_major ? n_index : nk),
                              static_cast<cuuint64_t>(o.mn_major ? nk : n_index)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(o.ld * es)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(kRowBytes / es), static_cast<cuuint32_t>(o.mn_major ? 64 : box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                        const_cast<void*>(o.p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <bool kFp8>
cudaError_t launch_typed(const CUtensorMap& ma, const CUtensorMap& mb, const LinearParams& P, int64_t grid,
                         cudaStream_t stream) {
  const cudaError_t e =
      cudaFuncSetAttribute(linear_kernel<kFp8>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  linear_kernel<kFp8><<<static_cast<unsigned>(grid), kThreads, kSmemBytes, stream>>>(ma, mb, P);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t stream) {
  if (a.na <= 0 || a.nb <= 0) return cudaSuccess;
  LinearParams P{};
  P.g = a;
  const int elems = a.fp8 ? 128 : 64;
  P.k_blocks = static_cast<int>((a.nk + elems - 1) / elems);
  P.tiles_a = (a.na + BM - 1) / BM;
  const int64_t grid = P.tiles_a * ((a.nb + BN - 1) / BN);
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  CUtensorMap ma, mb;
  cudaError_t e;
  if ((e = make_operand_map(&ma, a.A, a.na, a.nk, a.fp8 != 0, BM)) != cudaSuccess) return e;
  if ((e = make_operand_map(&mb, a.B, a.nb, a.nk, a.fp8 != 0, BN)) != cudaSuccess) return e;
  return a.fp8 ? launch_typed<true>(ma, mb, P, grid, stream) : launch_typed<false>(ma, mb, P, grid, stream);
}

cudaError_t launch_column_sums(const uint16_t* dz, int64_t ld, int64_t m, int64_t n, float* out, int accumulate,
                               cudaStream_t stream) {
  column_sums_kernel<<<static_cast<unsigned>((n + 31) / 32), 256, 0, stream>>>(dz, ld, m, n, out, accumulate);
  return cudaGetLastError();
}

cudaError_t launch_repack(const void* src, int64_t src_ld, void* dst, int64_t dst_ld, int64_t rows, int64_t cols,
                          int esize, cudaStream_t stream) {
  const int64_t grid = rows < 65536 ? rows : 65536;
  if (esize == 1)
    repack_kernel<uint8_t><<<static_cast<unsigned>(grid), 256, 0, stream>>>(
        static_cast<const uint8_t*>(src), src_ld, static_cast<uint8_t*>(dst), dst_ld, rows, cols);
  else
    repack_kernel<uint16_t><<<static_cast<unsigned>(grid), 256, 0, stream>>>(
        static_cast<const uint16_t*>(src), src_ld, static_cast<uint16_t*>(dst), dst_ld, rows, cols);
  return cudaGetLastError();
}

}  // namespace mpopt
