// The linear layer's products on the 5th-generation tensor cores (sm_103a):
//
//   forward   y = act(x w^T + bias) + residual        bf16 or e4m3 operands
//   dx        (dz w) * act'(z)                        bf16
//   dw        dz^T x (+ main_grad)                    bf16 operands, fp32 result
//
// All three are out[b][a] = sum_k A[a][k] B[b][k], where `a` is the index that
// is contiguous in the output.  An operand stored [index][k] is K-major, one
// stored [k][index] (w in dx, both operands of dw) MN-major: no transposed
// copy is made.
//
// linear_pair_kernel takes large products, linear_split_kernel the others.
// Both load k-blocks of 128 bytes by TMA; out-of-range rows and columns are
// filled with zeros there and never stored.

#include <cuda_bf16.h>

#include "../../include/mpopt.h"
#include "activation.cuh"
#include "internal.h"
#include "overlap.cuh"
#include "tc_common.cuh"

namespace mpopt {
namespace {

constexpr int BM = 128;                        // TMEM lanes of a CTA: output indices of the MMA's A operand
constexpr int kStageA = BM * kRowBytes;

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

// main_grad += without reading it: each element gets one addition per launch,
// rounded to nearest in fp32, in L2 (subnormal values and results become zero),
// so the result does not depend on an order.
__device__ __forceinline__ void red_add(float* p, float v) {
  asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(p), "f"(v) : "memory");
}
__device__ __forceinline__ void red_add(float4* p, float4 v) {
  asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

// -------------------------------------------------------------- epilogue --

// What the epilogue needs of this lane's output column `a` throughout a tile.
struct LaneColumn {
  int64_t a;
  float scale, bias;
};

template <int kMode, bool kFp8>
__device__ __forceinline__ LaneColumn lane_column(const LinearArgs& g, int64_t a) {
  LaneColumn c{a, 1.f, 0.f};
  if (kMode == kLinearForward && a < g.na) {
    if (kFp8) c.scale = g.a_scale[a];
    if (g.bias)
      c.bias = g.bias_dtype == kBf16 ? bf16_at(static_cast<const uint16_t*>(g.bias), a)
                                     : static_cast<const float*>(g.bias)[a];
  }
  return c;
}

// kN accumulator columns: column j is output row b0 + j, this lane output
// column c.a; a warp's accesses of one column are contiguous.
template <int kMode, bool kFp8, int kN>
__device__ __forceinline__ void epilogue_columns(const LinearArgs& g, const LaneColumn& c, int64_t b0,
                                                 const float* v) {
  if (c.a >= g.na) return;
  const int n = static_cast<int>(g.nb - b0 < kN ? g.nb - b0 : kN);
  static_assert(kMode != kLinearDw, "dw has its rows on the lanes");
  if constexpr (kMode == kLinearDx) {
    uint16_t zr[kN];
    if (g.z_in) {
#pragma unroll
      for (int j = 0; j < kN; ++j)
        if (j < n) zr[j] = __ldcs(g.z_in + (b0 + j) * g.z_ld + c.a);
    }
    with_activation(g.z_in ? g.act : OPT_ACT_NONE, [&](auto act) {
#pragma unroll
      for (int j = 0; j < kN; ++j)
        if (j < n) {
          float d = v[j];
          if (act.value != OPT_ACT_NONE)
            d *= activate_grad<act.value>(__uint_as_float(static_cast<uint32_t>(zr[j]) << 16));
          g.y[(b0 + j) * g.y_ld + c.a] = to_bf16(d);
        }
    });
  } else {
    uint16_t rr[kN];
    if (g.residual) {
#pragma unroll
      for (int j = 0; j < kN; ++j)
        if (j < n) rr[j] = g.residual[(b0 + j) * g.residual_ld + c.a];
    }
    with_activation(g.act, [&](auto act) {
#pragma unroll
      for (int j = 0; j < kN; ++j)
        if (j < n) {
          float z = v[j];
          if (kFp8) z *= c.scale * g.b_scale[b0 + j];
          z += c.bias;
          if (g.z_out) __stcs(g.z_out + (b0 + j) * g.z_ld + c.a, to_bf16(z));
          float y = activate<act.value>(z);
          if (g.residual) y += __uint_as_float(static_cast<uint32_t>(rr[j]) << 16);
          g.y[(b0 + j) * g.y_ld + c.a] = to_bf16(y);
        }
    });
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// kN values that every lane shares: p[col0 .. col0 + kN - 1], 0 past the end.
template <int kN>
__device__ __forceinline__ void load_shared_cols(const void* p, int dtype, int64_t col0, int64_t cols, float (&out)[kN]) {
  if (dtype == kBf16) {
    const uint16_t* q = static_cast<const uint16_t*>(p) + col0;
    if (col0 + kN <= cols && (reinterpret_cast<uintptr_t>(q) & 15u) == 0) {
#pragma unroll
      for (int i = 0; i < kN / 8; ++i) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(q) + i);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          out[8 * i + 2 * k] = __uint_as_float(u[k] << 16);
          out[8 * i + 2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < kN; ++j) out[j] = col0 + j < cols ? bf16_at(q, j) : 0.f;
    }
  } else {
    const float* q = static_cast<const float*>(p) + col0;
    if (col0 + kN <= cols && (reinterpret_cast<uintptr_t>(q) & 15u) == 0) {
#pragma unroll
      for (int i = 0; i < kN / 4; ++i) {
        const float4 w = __ldg(reinterpret_cast<const float4*>(q) + i);
        out[4 * i] = w.x;
        out[4 * i + 1] = w.y;
        out[4 * i + 2] = w.z;
        out[4 * i + 3] = w.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kN; ++j) out[j] = col0 + j < cols ? q[j] : 0.f;
    }
  }
}

// Two elements to a word, by index.
template <int kWords>
__device__ __forceinline__ float block_elem(const uint32_t (&raw)[kWords], int j) {
  return __uint_as_float(j & 1 ? raw[j >> 1] & 0xffff0000u : raw[j >> 1] << 16);
}

// The same with the lanes on output rows: this lane holds columns col .. col +
// kN - 1 of row `row`.  Rows that start on 16 bytes move in 16-byte pieces;
// others are turned in the warp's `table`, so that a warp's accesses cover runs
// of kN columns.
struct RowAccess {
  bool in_vec, out_vec;        // residual / z_in, and y, z (or dw)
};

template <int kN>
constexpr int kTableWords = 32 * (kN + 1);

template <int kN>
__device__ __forceinline__ void load_row_in(const uint16_t* p, int64_t ld, int64_t row, int64_t rows, int64_t col,
                                            int64_t cols, bool vec, uint32_t* table, int lane,
                                            uint32_t (&raw)[kN / 2]) {
  if (vec && col + kN <= cols) {
    const uint4* q = reinterpret_cast<const uint4*>(p + row * ld + col);
#pragma unroll
    for (int i = 0; i < kN / 8; ++i) {
      const uint4 w = row < rows ? q[i] : make_uint4(0, 0, 0, 0);    // a plain load: y may be the residual
      raw[4 * i] = w.x, raw[4 * i + 1] = w.y, raw[4 * i + 2] = w.z, raw[4 * i + 3] = w.w;
    }
    return;
  }
  const int sub = lane / kN, c = lane % kN;
  const int64_t row0 = row - lane;
  uint16_t got[kN];                   // 32 rows, 32 / kN at a time, all loads in flight together
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int64_t rr = row0 + i * (32 / kN) + sub;
    got[i] = rr < rows && col + c < cols ? p[rr * ld + col + c] : 0;
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kN; ++i) table[(i * (32 / kN) + sub) * (kN + 1) + c] = got[i];
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kN / 2; ++i)
    raw[i] = table[lane * (kN + 1) + 2 * i] | (table[lane * (kN + 1) + 2 * i + 1] << 16);
}

template <int kN>
__device__ __forceinline__ void store_row_out(uint16_t* p, int64_t ld, int64_t row, int64_t rows, int64_t col,
                                              int64_t cols, bool vec, uint32_t* table, int lane, const float (&v)[kN]) {
  if (vec && col + kN <= cols) {
    if (row < rows) {
      uint4* q = reinterpret_cast<uint4*>(p + row * ld + col);
#pragma unroll
      for (int i = 0; i < kN / 8; ++i)
        q[i] = make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                          pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
    }
    return;
  }
  const int sub = lane / kN, c = lane % kN;
  const int64_t row0 = row - lane;
  __syncwarp();
#pragma unroll
  for (int j = 0; j < kN; ++j) table[lane * (kN + 1) + j] = to_bf16(v[j]);
  __syncwarp();
#pragma unroll
  for (int r = 0; r < 32; r += 32 / kN) {
    const int64_t rr = row0 + r + sub;
    if (rr < rows && col + c < cols) p[rr * ld + col + c] = static_cast<uint16_t>(table[(r + sub) * (kN + 1) + c]);
  }
}

template <int kN>
__device__ __forceinline__ void store_row_dw(float* p, int64_t ld, int64_t row, int64_t rows, int64_t col,
                                             int64_t cols, bool vec, bool add, float* table, int lane,
                                             const float (&v)[kN]) {
  if (vec && col + kN <= cols) {
    if (row < rows) {
      float4* q = reinterpret_cast<float4*>(p + row * ld + col);
#pragma unroll
      for (int i = 0; i < kN / 4; ++i) {
        const float4 x = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        if (add) red_add(q + i, x);
        else q[i] = x;
      }
    }
    return;
  }
  const int sub = lane / kN, c = lane % kN;          // 32 rows, 32 / kN at a time
  const int64_t row0 = row - lane;
  __syncwarp();
#pragma unroll
  for (int j = 0; j < kN; ++j) table[lane * (kN + 1) + j] = v[j];
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int r = i * (32 / kN) + sub;
    const float x = table[r * (kN + 1) + c];
    if (row0 + r < rows && col + c < cols) {
      if (add) red_add(p + (row0 + r) * ld + col + c, x);
      else p[(row0 + r) * ld + col + c] = x;
    }
  }
}

template <int kMode, bool kFp8, int kN>
__device__ __forceinline__ void epilogue_row(const LinearArgs& g, const RowAccess& access, float row_scale, int64_t row,
                                             int64_t col, uint32_t* table, int lane, float (&v)[kN]) {
  if constexpr (kMode == kLinearDw) {
    store_row_dw<kN>(g.dw, g.dw_ld, row, g.nb, col, g.na, access.out_vec, g.accumulate != 0,
                     reinterpret_cast<float*>(table), lane, v);
  } else {
    const uint16_t* in = kMode == kLinearDx ? g.z_in : g.residual;
    uint32_t raw[kN / 2];
    if (in)
      load_row_in<kN>(in, kMode == kLinearDx ? g.z_ld : g.residual_ld, row, g.nb, col, g.na, access.in_vec, table, lane,
                      raw);
    if constexpr (kMode == kLinearDx) {
      if (in)
        with_activation(g.act, [&](auto act) {
#pragma unroll
          for (int j = 0; j < kN; ++j) v[j] *= activate_grad<act.value>(block_elem(raw, j));
        });
    } else {
      float t[kN];
      if constexpr (kFp8) {
        load_shared_cols(g.a_scale, kFp32, col, g.na, t);
#pragma unroll
        for (int j = 0; j < kN; ++j) v[j] *= row_scale * t[j];
      }
      if (g.bias) {
        load_shared_cols(g.bias, g.bias_dtype, col, g.na, t);
#pragma unroll
        for (int j = 0; j < kN; ++j) v[j] += t[j];
      }
      if (g.z_out) store_row_out<kN>(g.z_out, g.z_ld, row, g.nb, col, g.na, access.out_vec, table, lane, v);
      with_activation(g.act, [&](auto act) {
#pragma unroll
        for (int j = 0; j < kN; ++j) v[j] = activate<act.value>(v[j]);
      });
      if (in) {
#pragma unroll
        for (int j = 0; j < kN; ++j) v[j] += block_elem(raw, j);
      }
    }
    store_row_out<kN>(g.y, g.y_ld, row, g.nb, col, g.na, access.out_vec, table, lane, v);
  }
}

// The operands' orders by product: forward K-major both, dx A MN-major, dw both.
template <int kMode>
struct Order {
  static constexpr bool a_mn = kMode != kLinearForward;
  static constexpr bool b_mn = kMode == kLinearDw;
};

// ----------------------------------------------------------- split kernel --
//
// Products with too few 256 x 256 tiles for the pair kernel: from one token,
// where the time is that of reading the weights once, to a few hundred.
//   kRows false  (up to 64 output rows) a CTA computes 128 output columns, on
//                the TMEM lanes, x kBN = 16, 32 or 64 rows, so that a few tokens
//                do not pay for a wide tile
//   kRows true   128 output rows, on the lanes, x kBN = 64 columns: a lane's
//                columns move in 16-byte pieces
// Where the tiles are too few for the GPU, a cluster of 2, 4 or 8 CTAs splits
// the k-blocks of one tile and joins the partial sums through distributed
// shared memory: rank r adds the ranks' sums of its share of the TMEM columns
// in rank order and runs their epilogue, so the result does not depend on
// timing and needs no workspace or second launch.  About 100 KB of shared
// memory a CTA, so that two fit on an SM and one's start and end overlap the
// other's main loop.
//   warp 0     TMA producer      warp 1     TMEM allocation, MMA issuer
//   warps 2-5  epilogue, one TMEM lane quarter each
// dw runs in segments as in the pair kernel (below).

constexpr int kSplitEpiWarps = 4;
constexpr int kSplitThreads = 64 + 32 * kSplitEpiWarps;
constexpr int kMaxSplit = 8;
constexpr int kDwSegment = 12;               // k-blocks of dw accumulated in TMEM at a time

template <int kBN>
struct SplitConfig {
  static constexpr int kStageB = kBN * kRowBytes;
  static constexpr int kStageBytes = kStageA + kStageB;
  static_assert(kBN == 16 || kBN == 32 || kBN == 64, "stages, and what join() loads at a time, are chosen for these");
  static constexpr int kStages = kBN == 16 ? 6 : kBN == 32 ? 5 : 4;
  static constexpr uint32_t kSmemBytes = kStages * kStageBytes + 1024 /*align*/ + 256 /*barriers*/;
  static constexpr int kTmemCols = 2 * kBN < 32 ? 32 : 2 * kBN;     // two accumulators
  static_assert(kSmemBytes <= 116224, "two CTAs shall fit on an SM");
  // in the ring's place, once its MMAs are done: the partial sums, then a
  // turning table for each epilogue warp
  static constexpr int kPartBytes = BM * kBN * 4;
  static_assert(kBN < 64 || kPartBytes + kSplitEpiWarps * kTableWords<32> * 4 <= kStages * kStageBytes,
                "partial sums and tables larger than the ring they replace");
};

struct SplitParams {
  LinearArgs g;
  int k_blocks;        // of the whole product
  int per_rank;        // k-blocks of one CTA of the cluster
  int segment;         // k-blocks accumulated in TMEM at a time
  int split;           // CTAs that share a tile; divides the cluster's size
  int64_t tiles_m;     // tiles along the lanes' index
  int64_t tiles;
  RowAccess access;
};

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

template <int kSplit>
struct SplitTag {
  static constexpr int value = kSplit;
};

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr));
  return v;
}

// The work of CTA `block` of a product's CTAs (maps and params are kernel
// parameters).
template <int kMode, bool kFp8, int kBN, bool kRows>
__device__ __forceinline__ void split_tile(const CUtensorMap& map_a, const CUtensorMap& map_b, const SplitParams& P,
                                           int64_t block) {
  using C = SplitConfig<kBN>;
  constexpr int kElems = kFp8 ? 128 : 64;
  // the MMA's A operand is the lanes' index: output rows (the product's B) or columns (its A)
  constexpr bool a_mn = kRows ? Order<kMode>::b_mn : Order<kMode>::a_mn;
  constexpr bool b_mn = kRows ? Order<kMode>::a_mn : Order<kMode>::b_mn;
  static_assert(!b_mn || kBN % 64 == 0, "an MN-major operand is staged 64 indices at a time");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStageBytes);
  uint64_t* empty = full + C::kStages;
  uint64_t* acc_full = empty + C::kStages;     // [2]
  uint64_t* acc_empty = acc_full + 2;          // [2]
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* status = P.g.header;
  // the CTAs first_rank .. first_rank + split - 1 of the cluster share a tile
  const int in_cluster = P.split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int rank = in_cluster & (P.split - 1), first_rank = in_cluster - rank;
  const int64_t tile = block / P.split;
  const bool exists = tile < P.tiles;          // the last cluster may have CTAs to spare
  const int64_t m0 = tile % P.tiles_m * BM, n0 = tile / P.tiles_m * kBN;   // first lane's and first column's index
  const int64_t n_end = kRows ? P.g.na : P.g.nb;
  // this CTA's k-blocks; the last ranks may have none, and their sums are zero
  const int kb0 = min(rank * P.per_rank, P.k_blocks), kb1 = exists ? min(kb0 + P.per_rank, P.k_blocks) : kb0;

  const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty);
  const uint32_t sa0 = smem_u32(smem), sb0 = sa0 + C::kStages * kStageA;
  // k-block kb into stage s, by the producer
  auto load_stage = [&](int kb, uint32_t s) {
    mbar_expect_tx(full0 + 8 * s, C::kStageBytes);
    load_operand(sa0 + s * kStageA, &map_a, full0 + 8 * s, a_mn, static_cast<int>(m0), BM, kb, kElems);
    load_operand(sb0 + s * C::kStageB, &map_b, full0 + 8 * s, b_mn, static_cast<int>(n0), kBN, kb, kElems);
  };
  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_a)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_b)) : "memory");
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&acc_full[a]), 1);
      mbar_init(smem_u32(&acc_empty[a]), 32 * kSplitEpiWarps);
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    wait_for_predecessors();
    // the first loads fly while the CTA sets up: the ring is empty
    for (int s = 0; s < C::kStages && kb0 + s < kb1; ++s) load_stage(kb0 + s, s);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(C::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  wait_for_predecessors();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int quarter = warp & 3;
  const int64_t index = m0 + quarter * 32 + lane;     // this lane's
  LaneColumn lane_col{index, 1.f, 0.f};
  float row_scale = 1.f;
  if constexpr (kRows) {
    if (kFp8 && index < P.g.nb) row_scale = P.g.b_scale[index];
  } else {
    lane_col = lane_column<kMode, kFp8>(P.g, index);
  }
  constexpr int kSum = kMode == kLinearDw ? kBN : 1;
  float sum[kSum];
  bool ready = false;          // epilogue warps: the accumulator holds this CTA's sums

  if (warp == 0) {
    if (lane == 0) {
      uint32_t s = 0, ph = 0;                       // second time round the ring and on
      int kb = kb0 + C::kStages;
      for (; kb < kb1; ++kb) {
        if (!mbar_wait(empty0 + 8 * s, ph, abort_flag, status, kStatusTimeoutEmpty)) break;
        load_stage(kb, s);
        if (++s == C::kStages) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (kb < kb1) {
        // aborting: give copies in flight time to land before the CTA exits
        const unsigned long long t0 = global_ns();
        while (global_ns() - t0 < 10000000ull) {
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && kb1 > kb0) {
      constexpr uint32_t idesc = linear_idesc(kFp8, a_mn, b_mn, BM, kBN);
      const uint64_t ad0 = a_mn ? smem_desc_mn(sa0) : smem_desc(sa0);
      const uint64_t bd0 = b_mn ? smem_desc_mn(sb0) : smem_desc(sb0);
      // one MMA's K step: 32 bytes of a K-major row, or 16 rows of an MN-major block
      constexpr uint32_t ka = (a_mn ? 16 * kRowBytes : 32) >> 4, kbs = (b_mn ? 16 * kRowBytes : 32) >> 4;
      uint32_t s = 0, ph = 0, use = 0;
      bool ok = true;
      for (int k0 = kb0; ok && k0 < kb1; k0 += P.segment, ++use) {
        const uint32_t acc = use & 1;
        if (!mbar_wait(smem_u32(&acc_empty[acc]), ((use >> 1) & 1u) ^ 1u, abort_flag, status, kStatusTimeoutAccFree))
          break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * kBN;
        const int k1 = min(k0 + P.segment, kb1);
        for (int kb = k0; kb < k1; ++kb) {
          if (!mbar_wait(full0 + 8 * s, ph, abort_flag, status, kStatusTimeoutFull)) {
            ok = false;
            break;
          }
          const uint64_t ad = ad0 + s * (kStageA >> 4), bd = bd0 + s * (C::kStageB >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_1cta<kFp8>(d_tmem, ad + ka * kk, bd + kbs * kk, idesc, (kb > k0 || kk > 0) ? 1u : 0u);
          commit_1cta(empty0 + 8 * s);
          if (++s == C::kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (ok) commit_1cta(smem_u32(&acc_full[acc]));
      }
      // every MMA issued by this thread has completed before TMEM goes
      commit_1cta(smem_u32(drain));
      const unsigned long long t0 = global_ns();
      while (!mbar_try(smem_u32(drain), 0)) {
        if (global_ns() - t0 > kWaitLimitNs) {
          *abort_flag = 1u;
          atomicCAS(status, 0u, static_cast<uint32_t>(kStatusTimeoutDrain));
          break;
        }
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < kSum; ++c) sum[c] = 0.f;
    uint32_t use = 0;
    ready = exists;
    if constexpr (kRows && kMode != kLinearDw) {
      // the residual or pre-activation of this rank's share comes from DRAM while the MMAs run
      const uint16_t* in = kMode == kLinearDx ? P.g.z_in : P.g.residual;
      const int64_t c = n0 + rank * (kBN / P.split);
      if (exists && in && index < P.g.nb && c < P.g.na)
        prefetch_l2(in + index * (kMode == kLinearDx ? P.g.z_ld : P.g.residual_ld) + c);
    }
    for (int k0 = kb0; ready && k0 < kb1; k0 += P.segment, ++use) {
      const uint32_t acc = use & 1;
      ready = __all_sync(0xffffffffu, mbar_wait(smem_u32(&acc_full[acc]), (use >> 1) & 1u, abort_flag, status,
                                                kStatusTimeoutAcc));
      if (!ready) break;
      tc_fence_after();
      if constexpr (kMode == kLinearDw) {
#pragma unroll
        for (int c = 0; c < kBN; c += 16) {
          float v[16];
          tmem_ld16(tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * kBN + c, v);
#pragma unroll
          for (int j = 0; j < 16; ++j) sum[c + j] += v[j];
        }
        tc_fence_before();
        mbar_arrive_local(smem_u32(&acc_empty[acc]));
      }
    }
  }

  __syncwarp();
  // The sums of the tile's columns c, c + 1, ...
  auto finish = [&](int c, auto& v) {
    constexpr int kN = sizeof(v) / sizeof(float);
    if constexpr (kRows) {
      uint32_t* table = reinterpret_cast<uint32_t*>(smem + C::kPartBytes) + (warp - 2) * kTableWords<32>;
      epilogue_row<kMode, kFp8, kN>(P.g, P.access, row_scale, index, n0 + c, table, lane, v);
    } else {
      epilogue_columns<kMode, kFp8, kN>(P.g, lane_col, n0 + c, v);
    }
  };
  // columns c .. c + 15 of this CTA's own sums
  auto own_sums = [&](int c, float* v) {
    if constexpr (kMode == kLinearDw) {
#pragma unroll
      for (int k = 0; k < kBN; k += 16)
        if (k == c)
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = sum[k + j];
    } else if (kb1 > kb0) {
      float w[16];
      tmem_ld16(tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + c, w);
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = w[j];
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = 0.f;
    }
  };
  // This rank's share of the columns of a cluster of kSplit, up to 32 at a
  // time with every peer's words and the epilogue's inputs in flight together
  // (at most 64 words a lane).
  auto join = [&](auto split_tag) {
    constexpr int kSplit = decltype(split_tag)::value, kPer = kBN / kSplit;
    constexpr int kMost = kMode == kLinearDw ? 16 : 32;          // dw keeps its sums in registers
    constexpr int kN = kPer > kMost ? kMost : kPer < 4 ? 4 : kPer;     // kPer 2 (16 columns, 8 ranks): half of a word
    const uint32_t base = smem_u32(smem) + (quarter * 32 + lane) * 16;
#pragma unroll
    for (int c0 = 0; c0 < kPer; c0 += kN) {
      const int c = rank * kPer + c0, c4 = c & ~3;
      if (n0 + c >= n_end) break;
      float v[kN];
      float4 w[kSplit][kN / 4];
#pragma unroll
      for (int p = 0; p < kSplit; ++p) {
        const uint32_t peer = peer_addr(base, static_cast<uint32_t>(first_rank + p));
#pragma unroll
        for (int i = 0; i < kN / 4; ++i) w[p][i] = ld_cluster_f32x4(peer + (c4 / 4 + i) * (BM * 16));
      }
#pragma unroll
      for (int i = 0; i < kN / 4; ++i) {
        float4 t = w[0][i];
#pragma unroll
        for (int p = 1; p < kSplit; ++p) {
          t.x += w[p][i].x;
          t.y += w[p][i].y;
          t.z += w[p][i].z;
          t.w += w[p][i].w;
        }
        v[4 * i] = t.x;
        v[4 * i + 1] = t.y;
        v[4 * i + 2] = t.z;
        v[4 * i + 3] = t.w;
      }
      if constexpr (kPer < 4) {
        float part_word[kPer];
        part_word[0] = c & 2 ? v[2] : v[0];
        part_word[1] = c & 2 ? v[3] : v[1];
        finish(c, part_word);
      } else {
        finish(c, v);
      }
    }
  };
  if (P.split == 1) {
    if (ready) {
      constexpr int kN = kBN < 32 || kMode == kLinearDw ? 16 : 32;
#pragma unroll
      for (int c = 0; c < kBN; c += kN) {
        if (n0 + c >= n_end) break;
        float v[kN];
        own_sums(c, v);
        if constexpr (kN == 32) own_sums(c + 16, v + 16);
        finish(c, v);
      }
    }
  } else {
    // the sums take the place of the ring: its MMAs have completed (acc_full).
    // Four columns of a lane are one 16-byte word: part[column / 4][lane]
    float4* part = reinterpret_cast<float4*>(smem);
    if (ready) {
#pragma unroll
      for (int c = 0; c < kBN; c += 16) {
        float v[16];
        own_sums(c, v);
#pragma unroll
        for (int j = 0; j < 16; j += 4)
          part[(c + j) / 4 * BM + quarter * 32 + lane] = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
      }
    }
    __syncwarp();
    cluster_sync();
    if (ready) {
      if (P.split == 2) join(SplitTag<2>{});
      else if (P.split == 4) join(SplitTag<4>{});
      else join(SplitTag<8>{});
    }
    __syncwarp();
    cluster_sync();          // no CTA leaves while another reads its sums
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(C::kTmemCols)
                 : "memory");
  }
}

template <int kMode, bool kFp8, int kBN, bool kRows>
__global__ void __launch_bounds__(kSplitThreads, 2)
linear_split_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                    const __grid_constant__ SplitParams P) {
  let_next_start();
  split_tile<kMode, kFp8, kBN, kRows>(map_a, map_b, P, blockIdx.x);
}

// The column sums of dz, in a fixed order.  CTA (x, y) takes 64 columns of the
// rows of its y-th slice, each of its six warps every sixth of them, two
// columns to a lane, and adds its warps' sums in order; with one slice that is
// the result, otherwise the slices' sums go to `partial` and join_sums_kernel
// adds them in order.
struct ColumnSums {
  const uint16_t* dz;
  int64_t ld, m, n;
  float *out, *partial;
  int accumulate;
  int vec;             // both columns of a lane in one 4-byte load
};
constexpr int kSumCols = 64;

__device__ __forceinline__ void column_sums(const ColumnSums& p, int64_t x, int64_t y, int64_t slices) {
  __shared__ float2 sums[kSplitThreads / 32][32];
  constexpr int kWarps = kSplitThreads / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t c = x * kSumCols + 2 * lane;
  const int64_t per = (p.m + slices - 1) / slices;
  const int64_t r0 = per * y, r1 = r0 + per < p.m ? r0 + per : p.m;
  float2 s = make_float2(0.f, 0.f);
  if (c < p.n) {
    // sixteen rows' loads in flight together
    constexpr int kBatch = 16;
    const int64_t two = c + 1 < p.n ? 1 : 0;         // past the last column: that one again, not stored
    for (int64_t q = r0 + warp; q < r1; q += kWarps * kBatch) {
      uint32_t v[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int64_t r = q + j * kWarps;
        const uint16_t* x = p.dz + r * p.ld + c;
        v[j] = r >= r1 ? 0u : p.vec ? *reinterpret_cast<const uint32_t*>(x) : x[0] | static_cast<uint32_t>(x[two]) << 16;
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        s.x += __uint_as_float(v[j] << 16);
        s.y += __uint_as_float(v[j] & 0xffff0000u);
      }
    }
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      s.x += sums[w][lane].x;
      s.y += sums[w][lane].y;
    }
    float* o = slices > 1 ? p.partial + y * p.n : p.out;
    const bool add = slices == 1 && p.accumulate;
    if (c < p.n) o[c] = add ? o[c] + s.x : s.x;
    if (c + 1 < p.n) o[c + 1] = add ? o[c + 1] + s.y : s.y;
  }
}

__global__ void __launch_bounds__(kSplitThreads) column_sums_kernel(const __grid_constant__ ColumnSums p) {
  let_next_start();
  wait_for_predecessors();
  column_sums(p, blockIdx.x, blockIdx.y, gridDim.y);
}

__global__ void __launch_bounds__(128)
join_sums_kernel(const float* partial, int slices, int64_t n, float* out, int accumulate) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
  let_next_start();
  wait_for_predecessors();
  if (c >= n) return;
  float s = 0.f;
#pragma unroll 8
  for (int p = 0; p < slices; ++p) s += partial[p * n + c];
  out[c] = accumulate ? out[c] + s : s;
}

// dx, dw and dbias of a short batch in one launch: CTAs 0 .. dx_blocks - 1
// compute dx, the next dw_blocks dw, the others 64 columns of dbias each.  The
// three are independent and each alone leaves most of the GPU idle; every
// result has the bits that it has from a launch of its own.
struct GradParams {
  SplitParams dx, dw;
  ColumnSums sums;
  int64_t dx_blocks, dw_blocks;      // multiples of the cluster's size
};

template <int kBN, bool kRows>
__global__ void __launch_bounds__(kSplitThreads, 2)
linear_grad_kernel(const __grid_constant__ CUtensorMap dx_a, const __grid_constant__ CUtensorMap dx_b,
                   const __grid_constant__ CUtensorMap dw_a, const __grid_constant__ CUtensorMap dw_b,
                   const __grid_constant__ GradParams P) {
  const int64_t block = blockIdx.x;
  let_next_start();
  if (block < P.dx_blocks) {
    split_tile<kLinearDx, false, kBN, kRows>(dx_a, dx_b, P.dx, block);
  } else if (block < P.dx_blocks + P.dw_blocks) {
    split_tile<kLinearDw, false, 64, true>(dw_a, dw_b, P.dw, block - P.dx_blocks);
  } else {
    const int64_t x = block - P.dx_blocks - P.dw_blocks;
    wait_for_predecessors();
    if (x * kSumCols < P.sums.n) column_sums(P.sums, x, 0, 1);
  }
}

// ----------------------------------------------------------- pair kernel --
//
// Large products: CTA pairs, persistent over tiles of 256 rows x 256 (or 128)
// columns with cta_group::2 MMAs, the structure of the Newton-Schulz GEMMs.
// Each CTA stages 128 output rows' and 128 (64) output columns' operand (32 KB
// per 128-byte k-block, where two separate 128 x 256 tiles would stage 96 KB
// between them) and receives the accumulators of its own 128 rows.  Two
// accumulators let the epilogue of one tile overlap the main loop of the next.
// 8192 x 14336 x 4096: 498 us alone, 1.93 PFLOP/s; in e4m3 281 us, 3.4 PFLOP/s;
// back to back the power limit sets the clock (1.55 PFLOP/s in bf16).
//   warp 0      TMA producer (both CTAs; bytes counted on the even CTA's barrier)
//   warp 1      TMEM allocation; in the even CTA the MMA issuer
//   warps 2-9   epilogue: two warps per TMEM lane quarter, half of the columns
//               each (four and a quarter each, at 96 registers: no faster)
//   warp 10     even CTA: claims tiles from a launch-wide counter and publishes
//               them to both CTAs, so the tiles in flight stay neighbours that
//               share operand panels in L2
//
// Here a TMEM lane is an output row `b` and a TMEM column an output column
// `a`: a lane's 32 columns pack into 16-byte pieces of its row, are staged in
// shared memory and leave by TMA stores (main_grad += by TMA reductions, one
// addition per element).  With the lanes on `a`, as in the split kernel's short form, each
// column was a 64-byte store of its own and the epilogue, not the MMAs, set
// the pace: 22 us per tile whatever k was, against 17 us of MMAs at k = 4096.
// Outputs that TMA cannot address (base or row distance not a multiple of 16
// bytes) are turned in shared memory and stored 64 bytes at a time.
//
// dw sums over the tokens, and the tensor cores truncate each addition to the
// accumulator: a sum of 16384 tokens comes out low by 1.6e-5 of its value when
// the terms' signs are random and by 6.5e-5 when they are one (half of it where
// two CTAs share the k-blocks).  So dw runs in segments of kDwSegment k-blocks
// (768 tokens: 6e-7 at any number of tokens): the epilogue adds each segment's accumulator to registers
// with rounding additions while the MMAs of the next segment run into the
// other accumulator.  Two segments are also the time that a tile's stores have
// before the MMAs stall: 8 k-blocks cost 6 % against one segment for all
// (8192 tokens, 14336 x 4096), 16 and more 2 % or less.

constexpr int kPairEpiWarps = 8;
constexpr int kPairThreads = 96 + 32 * kPairEpiWarps;
constexpr int kTileSlots = 3;
constexpr int kDoneWord = kSchedWord + 1;    // header words beside the tile counter: CTAs that have finished,
constexpr int kTakenWord = kSchedWord + 2;   // and tiles claimed in all
constexpr int kBlockBytes = 32 * 128;   // a staged block: 32 rows of 128 bytes
constexpr uint32_t kTileConsumers = 2 + 1 + 2 * kPairEpiWarps;

template <int kMode, int kBN>
struct PairConfig {
  static constexpr int kBarrierReserve = 384;
  static constexpr int kHalf = kBN / 2;                      // columns staged by one CTA, and of an epilogue warp
  static constexpr int kStageB = kHalf * kRowBytes;
  static constexpr int kStageBytes = kStageA + kStageB;
  // per epilogue warp two blocks: y and z; y and the input (residual or
  // pre-activation), which TMA loads while the MMAs run; or y's or dw's in turn.
  // The second one is the turning table of inputs and outputs that cannot move
  // 16 bytes at a time.
  static constexpr int kWarpScratch = 2 * kBlockBytes;
  static constexpr int kTableAt = kBlockBytes;
  static constexpr int kStages = (227 * 1024 - 1024 - kBarrierReserve - kPairEpiWarps * kWarpScratch) / kStageBytes;
  static constexpr int kTmemCols = 2 * kBN;                  // two accumulators
  static constexpr int kBarrierBytes = (2 * kStages + 5 + 2 * kTileSlots + kPairEpiWarps) * 8 + 8 + 4 * kTileSlots;
  static_assert(kBarrierBytes <= kBarrierReserve, "barrier block larger than its reservation");
  static constexpr uint32_t kSmemBytes =
      kStages * kStageBytes + kPairEpiWarps * kWarpScratch + 1024 /*align*/ + kBarrierReserve;
  static_assert(kSmemBytes <= 232448, "dynamic shared memory above the 227 KB a CTA may use");
};

struct PairParams {
  LinearArgs g;
  int k_blocks;
  int segment;         // k-blocks accumulated in TMEM at a time
  int tiles_a, tiles_b, total_tiles;
  int out_tma;         // y (or dw) moves through map_out, z through map_z
  int in_vec;          // residual / z_in rows start on 16 bytes
  int in_tma;          // and there is no z: the input comes through map_z
};

struct PairSplitParams {
  PairParams p;
  RowAccess access;
  int per_pair;        // k-blocks of one pair of the cluster
  int tile0;           // the launch's first tile
};

// Tiles in groups of kGroupB tiles along b, a-major inside a group: about 76
// tiles are in flight, a block of 12 x 6.3 tiles that shares its panels (4 and 6
// wide: up to 5 % slower on 8192 x 14336 x 4096 and its gradients; 8 and 16 within 2 %).
constexpr int kGroupB = 12;

__device__ __forceinline__ void pair_tile(const PairParams& P, int tile, int& ta, int& tb) {
  const int per_group = kGroupB * P.tiles_a;
  const int grp = tile / per_group, r = tile - grp * per_group;
  const int width = min(kGroupB, P.tiles_b - grp * kGroupB);
  ta = r / width;
  tb = grp * kGroupB + (r - ta * width);
}

template <bool kFp8>
__device__ __forceinline__ void mma_pair(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  if constexpr (kFp8)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    mma(tmem_d, adesc, bdesc, idesc, accumulate);
}

// A box of a 2-D map into this CTA's shared memory, completing on `bar`, a
// shared::cluster address that may be the even CTA's barrier.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_store_block(const CUtensorMap* map, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(src)
               : "memory");
}

// The block is added to global memory, fp32, each element once.
__device__ __forceinline__ void tma_add_block(const CUtensorMap* map, uint32_t src, int x, int y) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(src)
               : "memory");
}

// Lane t stages 32 columns of row t of a block of 32 rows x 64 bf16 columns
// (128 bytes, 128-byte swizzle) for a TMA store; `half` 32: the upper ones.
__device__ __forceinline__ void stage_row(uint8_t* buf, int lane, int half, const float (&v)[32]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t phys = static_cast<uint32_t>(q + half / 8) ^ (static_cast<uint32_t>(lane) & 7u);
    *reinterpret_cast<uint4*>(buf + lane * 128 + phys * 16) =
        make_uint4(pack_bf16(v[8 * q], v[8 * q + 1]), pack_bf16(v[8 * q + 2], v[8 * q + 3]),
                   pack_bf16(v[8 * q + 4], v[8 * q + 5]), pack_bf16(v[8 * q + 6], v[8 * q + 7]));
  }
}

// The same columns of a block that TMA loaded, two elements to a word.
__device__ __forceinline__ void unstage_row(const uint8_t* buf, int lane, int half, uint32_t (&raw)[16]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t phys = static_cast<uint32_t>(q + half / 8) ^ (static_cast<uint32_t>(lane) & 7u);
    const uint4 w = *reinterpret_cast<const uint4*>(buf + lane * 128 + phys * 16);
    raw[4 * q] = w.x;
    raw[4 * q + 1] = w.y;
    raw[4 * q + 2] = w.z;
    raw[4 * q + 3] = w.w;
  }
}

// The warp's 32 x 32 words of scratch as a turning table: (row, col) at
// row * 32 + (col ^ row), free of bank conflicts by rows and by columns.
__device__ __forceinline__ int turn(int row, int col) { return row * 32 + (col ^ row); }

// A 32 x 32 block of a bf16 input, lane t's row t (row0 + t) in `raw`, two
// elements to a word; zeros outside the matrix.
__device__ __forceinline__ void load_block(const uint16_t* p, int64_t ld, int64_t row0, int64_t col0, int64_t rows,
                                           int64_t cols, bool vec, uint32_t* table, int lane, uint32_t (&raw)[16]) {
  if (vec && col0 + 32 <= cols) {
    const bool ok = row0 + lane < rows;
    const uint4* q = reinterpret_cast<const uint4*>(p + (row0 + lane) * ld + col0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 w = ok ? q[i] : make_uint4(0, 0, 0, 0);   // a plain load: y may be the residual
      raw[4 * i] = w.x;
      raw[4 * i + 1] = w.y;
      raw[4 * i + 2] = w.z;
      raw[4 * i + 3] = w.w;
    }
    return;
  }
  if (vec) {                               // the matrix ends inside the block
    const uint16_t* q = p + (row0 + lane) * ld + col0;
    const int n = row0 + lane < rows ? static_cast<int>(cols - col0) : 0;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      raw[i] = (2 * i < n ? q[2 * i] : 0u) | (2 * i + 1 < n ? static_cast<uint32_t>(q[2 * i + 1]) << 16 : 0u);
    return;
  }
  const bool ok = col0 + lane < cols;
  uint16_t got[32];                        // all loads in flight together
#pragma unroll
  for (int r = 0; r < 32; ++r) got[r] = ok && row0 + r < rows ? p[(row0 + r) * ld + col0 + lane] : 0;
#pragma unroll
  for (int r = 0; r < 32; ++r) table[turn(r, lane)] = got[r];
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 16; ++i) raw[i] = table[turn(lane, 2 * i)] | (table[turn(lane, 2 * i + 1)] << 16);
  __syncwarp();
}

// A block that TMA cannot store: turned through the table, then 32 columns of
// one row at a time.
template <typename T, typename F>
__device__ __forceinline__ void store_turned(T* p, int64_t ld, int64_t row0, int64_t col0, int64_t rows, int64_t cols,
                                             float* table, int lane, const float (&v)[32], F&& put) {
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 32; ++j) table[turn(lane, j)] = v[j];
  __syncwarp();
  if (col0 + lane < cols) {
    const int n = static_cast<int>(rows - row0 < 32 ? rows - row0 : 32);
    T* q = p + row0 * ld + col0 + lane;
#pragma unroll 8
    for (int r = 0; r < n; ++r) put(q + r * ld, table[turn(r, lane)]);
  }
  __syncwarp();
}

template <int kMode, bool kFp8, int kBN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
linear_pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                   const __grid_constant__ CUtensorMap map_out, const __grid_constant__ CUtensorMap map_z,
                   const __grid_constant__ PairParams P) {
  using C = PairConfig<kMode, kBN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* scratch = smem + C::kStages * C::kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(scratch + kPairEpiWarps * C::kWarpScratch);   // even CTA: both CTAs' copies landed
  uint64_t* empty = full + C::kStages;            // both CTAs: stage free again
  uint64_t* acc_full = empty + C::kStages;        // [2] both CTAs: accumulator ready
  uint64_t* acc_empty = acc_full + 2;              // [2] even CTA: both epilogues have read it
  uint64_t* drain = acc_empty + 2;                 // even CTA: all MMAs complete
  uint64_t* tile_full = drain + 1;                 // [kTileSlots] both CTAs: next tile published
  uint64_t* tile_empty = tile_full + kTileSlots;   // [kTileSlots] even CTA: every role has read it
  uint64_t* in_full = tile_empty + kTileSlots;     // [kPairEpiWarps] the warp's input block has landed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(in_full + kPairEpiWarps);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  volatile int* tile_ring = reinterpret_cast<volatile int*>(tmem_slot + 2);   // [kTileSlots]

  constexpr int kElems = kFp8 ? 128 : 64;
  // the MMA's A operand holds output rows (the product's B), its B operand output columns
  constexpr bool a_mn = Order<kMode>::b_mn, b_mn = Order<kMode>::a_mn;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  uint32_t* status = P.g.header;
  let_next_start();

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&acc_full[a]), 1);
      mbar_init(smem_u32(&acc_empty[a]), 2 * 32 * kPairEpiWarps);
    }
    mbar_init(smem_u32(drain), 1);
    for (int k = 0; k < kTileSlots; ++k) {
      mbar_init(smem_u32(&tile_full[k]), 1);
      mbar_init(smem_u32(&tile_empty[k]), kTileConsumers);
    }
    for (int w = 0; w < kPairEpiWarps; ++w) mbar_init(smem_u32(&in_full[w]), 1);
    *abort_flag = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0 && lane < 4) {
    const CUtensorMap* map = lane == 0 ? &map_a : lane == 1 ? &map_b : lane == 2 ? &map_out : &map_z;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(C::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  wait_for_predecessors();
  tc_fence_before();
  cluster_sync();            // barriers of both CTAs initialised, TMEM allocated in both
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true, issued = false;
      const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty);
      const uint32_t full0_even = peer_addr(full0, 0);
      const uint32_t sa0 = smem_u32(smem), sb0 = sa0 + C::kStages * kStageA;
      const uint32_t tempty_even = peer_addr(smem_u32(&tile_empty[0]), 0);
      uint32_t s = 0, ph = 0;
      int tile = pair;             // the first tile; the others come through the ring
      for (uint32_t seq = 0; ok; ++seq) {
        int ta, tb;
        pair_tile(P, tile, ta, tb);
        const int ai = tb * 256 + static_cast<int>(rank) * BM, bi = ta * kBN + static_cast<int>(rank) * C::kHalf;
        for (int kb = 0; kb < P.k_blocks; ++kb) {
          if (!mbar_wait(empty0 + 8 * s, ph ^ 1u, abort_flag, status, kStatusTimeoutEmpty)) {
            ok = false;
            break;
          }
          const uint32_t fb = full0_even + 8 * s;
          if (rank == 0) mbar_expect_tx(full0 + 8 * s, 2 * C::kStageBytes);
          const uint32_t sa = sa0 + s * kStageA, sb = sb0 + s * C::kStageB;
          if constexpr (a_mn) {
            tma_load_2d_pair(sa, &map_a, fb, ai, kb * kElems);
            tma_load_2d_pair(sa + kMnBlockBytes, &map_a, fb, ai + 64, kb * kElems);
          } else {
            tma_load_2d_pair(sa, &map_a, fb, kb * kElems, ai);
          }
          if constexpr (b_mn) {
            tma_load_2d_pair(sb, &map_b, fb, bi, kb * kElems);
            if constexpr (kBN == 256) tma_load_2d_pair(sb + kMnBlockBytes, &map_b, fb, bi + 64, kb * kElems);
          } else {
            tma_load_2d_pair(sb, &map_b, fb, kb * kElems, bi);
          }
          issued = true;
          if (++s == C::kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
        const uint32_t slot = seq % kTileSlots, sph = (seq / kTileSlots) & 1u;
        if (!ok) break;
        if (!(rank == 0 ? mbar_wait(smem_u32(&tile_full[slot]), sph, abort_flag, status, kStatusTimeoutTile)
                        : mbar_wait_acq_cluster(smem_u32(&tile_full[slot]), sph, abort_flag, status,
                                                kStatusTimeoutTile))) {
          ok = false;
          break;
        }
        tile = tile_ring[slot];
        if (rank == 0) mbar_arrive_local(smem_u32(&tile_empty[slot]));
        else mbar_arrive_remote(tempty_even + 8 * slot);
        if (tile >= P.total_tiles) break;
      }
      if (!ok && issued) {
        // aborting: give copies in flight time to land before the CTA exits
        const unsigned long long t0 = global_ns();
        while (global_ns() - t0 < 10000000ull) {
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = linear_idesc(kFp8, a_mn, b_mn, 256, kBN);
      const uint32_t sa0 = smem_u32(smem), sb0 = sa0 + C::kStages * kStageA;
      const uint64_t ad0 = a_mn ? smem_desc_mn(sa0) : smem_desc(sa0);
      const uint64_t bd0 = b_mn ? smem_desc_mn(sb0) : smem_desc(sb0);
      constexpr uint32_t ka = (a_mn ? 16 * kRowBytes : 32) >> 4, kbs = (b_mn ? 16 * kRowBytes : 32) >> 4;
      const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty);
      uint32_t s = 0, ph = 0, use = 0;          // use: accumulator uses so far
      bool ok = true;
      for (uint32_t lt = 0; ok; ++lt) {
        for (int k0 = 0; ok && k0 < P.k_blocks; k0 += P.segment, ++use) {
          const uint32_t acc = use & 1;
          if (!mbar_wait(smem_u32(&acc_empty[acc]), ((use >> 1) & 1u) ^ 1u, abort_flag, status,
                         kStatusTimeoutAccFree)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + acc * kBN;
          const int k1 = min(k0 + P.segment, P.k_blocks);
          for (int kb = k0; kb < k1; ++kb) {
            if (!mbar_wait(full0 + 8 * s, ph, abort_flag, status, kStatusTimeoutFull)) {
              ok = false;
              break;
            }
            const uint64_t ad = ad0 + s * (kStageA >> 4), bd = bd0 + s * (C::kStageB >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_pair<kFp8>(d_tmem, ad + ka * kk, bd + kbs * kk, idesc, (kb > k0 || kk > 0) ? 1u : 0u);
            mma_commit_pair(empty0 + 8 * s);
            if (++s == C::kStages) {
              s = 0;
              ph ^= 1u;
            }
          }
          if (ok) mma_commit_pair(smem_u32(&acc_full[acc]));
        }
        const uint32_t slot = lt % kTileSlots, sph = (lt / kTileSlots) & 1u;
        if (!ok || !mbar_wait(smem_u32(&tile_full[slot]), sph, abort_flag, status, kStatusTimeoutTile)) break;
        const int tile = tile_ring[slot];
        mbar_arrive_local(smem_u32(&tile_empty[slot]));
        if (tile >= P.total_tiles) break;
      }
      // every MMA issued by this thread has completed before TMEM goes
      mma_commit_local(smem_u32(drain));
      const unsigned long long t0 = global_ns();
      while (!mbar_try(smem_u32(drain), 0)) {
        if (global_ns() - t0 > kWaitLimitNs) {
          *abort_flag = 1u;
          atomicCAS(status, 0u, static_cast<uint32_t>(kStatusTimeoutDrain));
          break;
        }
      }
    }
  } else if (warp < 2 + kPairEpiWarps) {
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t empty_even = peer_addr(smem_u32(&acc_empty[0]), 0);
    const uint32_t tempty_even = peer_addr(smem_u32(&tile_empty[0]), 0);
    uint8_t* stage = scratch + (warp - 2) * C::kWarpScratch;
    uint32_t* table = reinterpret_cast<uint32_t*>(stage + C::kTableAt);
    const uint32_t in_bar = smem_u32(&in_full[warp - 2]);
    uint32_t blocks = 0;                 // dw: blocks staged so far
    uint32_t in_phase = 0;
    uint32_t use = 0;
    bool ok = true;
    int tile = pair;
    for (uint32_t lt = 0; ok; ++lt) {
      if (lt > 0) {
        const uint32_t slot = (lt - 1) % kTileSlots, sph = ((lt - 1) / kTileSlots) & 1u;
        int got = 1;
        if (lane == 0) {
          got = (rank == 0 ? mbar_wait(smem_u32(&tile_full[slot]), sph, abort_flag, status, kStatusTimeoutTile)
                           : mbar_wait_acq_cluster(smem_u32(&tile_full[slot]), sph, abort_flag, status,
                                                   kStatusTimeoutTile))
                    ? 1
                    : 0;
          if (got) {
            tile = tile_ring[slot];
            if (rank == 0) mbar_arrive_local(smem_u32(&tile_empty[slot]));
            else mbar_arrive_remote(tempty_even + 8 * slot);
          }
        }
        got = __shfl_sync(0xffffffffu, got, 0);
        tile = __shfl_sync(0xffffffffu, tile, 0);
        if (!got || tile >= P.total_tiles) break;
      }
      int ta, tb;
      pair_tile(P, tile, ta, tb);
      const int64_t row0 = static_cast<int64_t>(tb) * 256 + rank * BM + quarter * 32;
      const int64_t col0 = static_cast<int64_t>(ta) * kBN + half * C::kHalf;
      const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + half * C::kHalf;
      if constexpr (kMode == kLinearDw) {
        float sum[C::kHalf];
#pragma unroll
        for (int c = 0; c < C::kHalf; ++c) sum[c] = 0.f;
        for (int k0 = 0; k0 < P.k_blocks; k0 += P.segment, ++use) {
          const uint32_t acc = use & 1;
          ok = __all_sync(0xffffffffu,
                          mbar_wait(smem_u32(&acc_full[acc]), (use >> 1) & 1u, abort_flag, status, kStatusTimeoutAcc));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < C::kHalf; c += 16) {
            float v[16];
            tmem_ld16(lane_addr + acc * kBN + c, v);
#pragma unroll
            for (int j = 0; j < 16; ++j) sum[c + j] += v[j];
          }
          tc_fence_before();
          mbar_arrive_remote(empty_even + acc * 8);
        }
        if (!ok) break;
        if (row0 < P.g.nb) {
#pragma unroll
          for (int c = 0; c < C::kHalf; c += 32) {
            if (col0 + c >= P.g.na) break;
            if (P.out_tma) {
              uint8_t* const buf = stage + (blocks++ & 1) * kBlockBytes;
              if (lane == 0) bulk_wait_read_1();     // the store that last used this block has read it
              __syncwarp();
#pragma unroll
              for (int q = 0; q < 8; ++q)            // 128-byte swizzle
                *reinterpret_cast<float4*>(buf + lane * 128 + ((q ^ (lane & 7)) * 16)) =
                    make_float4(sum[c + 4 * q], sum[c + 4 * q + 1], sum[c + 4 * q + 2], sum[c + 4 * q + 3]);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                const int x = static_cast<int>(col0 + c), y = static_cast<int>(row0);
                if (P.g.accumulate) tma_add_block(&map_out, smem_u32(buf), x, y);
                else tma_store_block(&map_out, smem_u32(buf), x, y);
                bulk_commit();
              }
            } else {
              float v[32];
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = sum[c + j];
              const bool add = P.g.accumulate != 0;
              store_turned(P.g.dw, P.g.dw_ld, row0, col0 + c, P.g.nb, P.g.na, reinterpret_cast<float*>(table), lane, v,
                           [add](float* p, float x) {
                             if (add) red_add(p, x);
                             else *p = x;
                           });
            }
          }
        }
      } else {
        const uint16_t* in = kMode == kLinearDx ? P.g.z_in : P.g.residual;
        const int64_t in_ld = kMode == kLinearDx ? P.g.z_ld : P.g.residual_ld;
        const bool live = row0 < P.g.nb;
        // the first input block comes while the MMAs run
        auto load_in = [&](int c) {
          if (lane == 0) {
            mbar_expect_tx(in_bar, kBlockBytes);
            tma_load_2d(smem_u32(stage + kBlockBytes), &map_z, in_bar, static_cast<int>(col0) + c, static_cast<int>(row0));
          }
        };
        const bool in_tma = P.in_tma != 0;
        if (in_tma && live && col0 < P.g.na) load_in(0);
        if (in && !in_tma && row0 + lane < P.g.nb) {
          // rows that TMA cannot read come into L2 meanwhile
          const uint16_t* p = in + (row0 + lane) * in_ld + col0;
          for (int64_t c = 0; c < C::kHalf && col0 + c < P.g.na; c += 64) prefetch_l2(p + c);
        }
        const bool alternate = P.out_tma && !in && !(kMode == kLinearForward && P.g.z_out);
        float row_scale = 1.f;
        if (kFp8 && row0 + lane < P.g.nb) row_scale = P.g.b_scale[row0 + lane];
        const uint32_t acc = use & 1;
        ok = __all_sync(0xffffffffu,
                        mbar_wait(smem_u32(&acc_full[acc]), (use >> 1) & 1u, abort_flag, status, kStatusTimeoutAcc));
        if (!ok) break;
        ++use;
        tc_fence_after();
        for (int c = 0; c < C::kHalf && live && col0 + c < P.g.na; c += 32) {
          const int64_t col = col0 + c;
          uint8_t* const buf = alternate ? stage + (c & 64 ? kBlockBytes : 0) : stage;
          uint32_t raw[16];
          if (!(c & 32)) {                             // a new block: its staging area's last store has read it
            if (lane == 0) {
              if (alternate && c > 0) bulk_wait_read_1();
              else bulk_wait_read_0();
            }
            __syncwarp();
            if (in_tma) {
              ok = __all_sync(0xffffffffu, mbar_wait(in_bar, in_phase, abort_flag, status, kStatusTimeoutWload));
              if (!ok) break;
              in_phase ^= 1u;
            }
          }
          if (in_tma) {
            unstage_row(stage + kBlockBytes, lane, c & 32, raw);
            if ((c & 32) && c + 32 < C::kHalf && col + 32 < P.g.na) {
              __syncwarp();                            // every lane has read the block: the next one may land in it
              load_in(c + 32);
            }
          } else if (in) {
            load_block(in, in_ld, row0, col, P.g.nb, P.g.na, P.in_vec != 0, table, lane, raw);
          }
          float v[32];
          tmem_ld32(lane_addr + acc * kBN + c, v);
          if constexpr (kMode == kLinearDx) {
            if (in)
              with_activation(P.g.act, [&](auto act) {
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] *= activate_grad<act.value>(block_elem(raw, j));
              });
          } else {
            float t[32];
            if constexpr (kFp8) {
              load_shared_cols(P.g.a_scale, kFp32, col, P.g.na, t);
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] *= row_scale * t[j];
            }
            if (P.g.bias) {
              load_shared_cols(P.g.bias, P.g.bias_dtype, col, P.g.na, t);
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] += t[j];
            }
            if (P.g.z_out) {
              if (P.out_tma) stage_row(stage + kBlockBytes, lane, c & 32, v);
              else
                store_turned(P.g.z_out, P.g.z_ld, row0, col, P.g.nb, P.g.na, reinterpret_cast<float*>(table), lane, v,
                             [](uint16_t* p, float x) { *p = to_bf16(x); });
            }
            with_activation(P.g.act, [&](auto act) {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = activate<act.value>(v[j]);
            });
            if (in) {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] += block_elem(raw, j);
            }
          }
          if (P.out_tma) {
            stage_row(buf, lane, c & 32, v);
            if ((c & 32) || col + 32 >= P.g.na) {          // both halves of the block, or the last one
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                const int x = static_cast<int>(col) - (c & 32), y = static_cast<int>(row0);
                tma_store_block(&map_out, smem_u32(buf), x, y);
                if (kMode == kLinearForward && P.g.z_out) tma_store_block(&map_z, smem_u32(stage + kBlockBytes), x, y);
                bulk_commit();
              }
            }
          } else {
            store_turned(P.g.y, P.g.y_ld, row0, col, P.g.nb, P.g.na, reinterpret_cast<float*>(table), lane, v,
                         [](uint16_t* p, float x) { *p = to_bf16(x); });
          }
        }
        if (!ok) break;
        tc_fence_before();
        mbar_arrive_remote(empty_even + acc * 8);
      }
    }
    if (!ok && lane == 0) {
      // aborting: give an input block in flight time to land before the CTA exits
      const unsigned long long t0 = global_ns();
      while (global_ns() - t0 < 10000000ull) {
      }
    }
    if (lane == 0) bulk_wait_all();        // stores complete before the CTA exits
  } else if (lane == 0 && rank == 0) {
    const uint32_t ring_odd = peer_addr(smem_u32(const_cast<int*>(tile_ring)), 1);
    const uint32_t tfull_odd = peer_addr(smem_u32(&tile_full[0]), 1);
    // A counter that did not start at zero gives no tile out of range: it ends
    // the claims early, and the last CTA finds tiles missing.
    const uint32_t left = static_cast<uint32_t>(P.total_tiles - npairs);
    uint32_t taken = 0;
    for (uint32_t seq = 0;; ++seq) {
      const uint32_t slot = seq % kTileSlots, sph = (seq / kTileSlots) & 1u;
      if (!mbar_wait(smem_u32(&tile_empty[slot]), sph ^ 1u, abort_flag, status, kStatusTimeoutTile)) break;
      const uint32_t claim = atomicAdd(status + kSchedWord, 1u);
      const int tile = claim < left ? npairs + static_cast<int>(claim) : P.total_tiles;
      taken += claim < left ? 1u : 0u;
      tile_ring[slot] = tile;
      st_cluster_u32(ring_odd + 4 * slot, static_cast<uint32_t>(tile));
      mbar_arrive_local(smem_u32(&tile_full[slot]));
      mbar_arrive_remote(tfull_odd + 8 * slot);
      if (tile >= P.total_tiles) break;
    }
    if (taken) atomicAdd(status + kTakenWord, taken);
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();            // no CTA leaves while its partner may still signal it
  if (threadIdx.x == 0) {
    // the last CTA to finish (every claim is made by then) leaves the header zero
    __threadfence();
    const uint32_t before = atomicAdd(status + kDoneWord, 1u);
    bool whole = before < gridDim.x;
    if (before == gridDim.x - 1) {
      whole = atomicExch(status + kTakenWord, 0u) == static_cast<uint32_t>(P.total_tiles - npairs);
      atomicExch(status + kSchedWord, 0u);
      atomicExch(status + kDoneWord, 0u);
    }
    if (!whole) atomicCAS(status, 0u, static_cast<uint32_t>(kStatusHeader));
  }
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(C::kTmemCols)
                 : "memory");
  }
}

// ------------------------------------------------- pair kernel, k split --
//
// A last wave that less than half fills the GPU, or a product with that few
// tiles: a cluster of two CTA pairs splits the k-blocks of one 256 x 256 tile
// (four pairs: slower, the GPU holds too few clusters of eight such CTAs).
// Every CTA leaves its sums in its shared memory, and the CTAs of the same 128
// rows add their shares of the columns in order, as in the split kernel, and
// run its epilogue.
//   warp 0     TMA producer
//   warp 1     TMEM allocation; in the even CTA of a pair the MMA issuer
//   warps 2-9  epilogue: two warps per TMEM lane quarter, half of the columns each

constexpr int kPairSplitThreads = 64 + 32 * kPairEpiWarps;
constexpr int kPairSplit = 2;                  // pairs of a cluster

struct PairSplitConfig {
  static constexpr int kBN = 256;
  static constexpr int kStageBytes = 2 * kStageA;
  static constexpr int kStages = 6;
  static constexpr int kPartBytes = BM * kBN * 4;
  static constexpr uint32_t kSmemBytes = kStages * kStageBytes + 1024 /*align*/ + 256 /*barriers*/;
  static_assert(kSmemBytes <= 232448, "dynamic shared memory above the 227 KB a CTA may use");
  static_assert(kPartBytes + kPairEpiWarps * kTableWords<32> * 4 <= kStages * kStageBytes,
                "partial sums and tables larger than the ring they replace");
};

// Arrive on `bar` in the CTAs of `mask` once all MMAs of this thread have completed.
__device__ __forceinline__ void mma_commit_mask(uint32_t bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(mask)
      : "memory");
}

template <int kMode, bool kFp8>
__global__ void __launch_bounds__(kPairSplitThreads, 1)
linear_pair_split_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                         const __grid_constant__ PairSplitParams P) {
  using C = PairSplitConfig;
  constexpr int kSplit = kPairSplit;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStageBytes);   // even CTA: both CTAs' copies landed
  uint64_t* empty = full + C::kStages;             // both CTAs: stage free again
  uint64_t* acc_full = empty + C::kStages;         // [2] both CTAs: accumulator ready
  uint64_t* acc_empty = acc_full + 2;              // [2] even CTA: both epilogues have read it
  uint64_t* drain = acc_empty + 2;                 // even CTA: all MMAs complete
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile uint32_t* abort_flag = tmem_slot + 1;

  constexpr int kElems = kFp8 ? 128 : 64;
  // the MMA's A operand holds output rows (the product's B), its B operand output columns
  constexpr bool a_mn = Order<kMode>::b_mn, b_mn = Order<kMode>::a_mn;
  constexpr int kTmemCols = kMode == kLinearDw ? 512 : 256;       // dw: two accumulators
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t cta = cluster_rank(), rank = cta & 1u, even = cta & ~1u;
  const int part = static_cast<int>(cta >> 1);                    // which share of the k-blocks
  const uint16_t both = static_cast<uint16_t>(3u << even);
  uint32_t* status = P.p.g.header;
  const int kb0 = min(part * P.per_pair, P.p.k_blocks), kb1 = min(kb0 + P.per_pair, P.p.k_blocks);
  int ta, tb;
  pair_tile(P.p, P.tile0 + static_cast<int>(blockIdx.x) / (2 * kSplit), ta, tb);
  let_next_start();

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&acc_full[a]), 1);
      mbar_init(smem_u32(&acc_empty[a]), 2 * 32 * kPairEpiWarps);
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0 && lane < 2) {
    const CUtensorMap* map = lane == 0 ? &map_a : &map_b;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  wait_for_predecessors();
  tc_fence_before();
  cluster_sync();            // barriers of all CTAs initialised, TMEM allocated
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t sa0 = smem_u32(smem), sb0 = sa0 + C::kStages * kStageA;
  const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty);
  const int quarter = warp & 3, half = (warp - 2) >> 2;
  constexpr int kSum = kMode == kLinearDw ? 128 : 1;
  float sum[kSum];
  bool ready = false;

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t full_even = peer_addr(full0, even);
      const int ai = tb * 256 + static_cast<int>(rank) * BM, bi = ta * C::kBN + static_cast<int>(rank) * 128;
      uint32_t s = 0, ph = 0;
      int kb = kb0;
      for (; kb < kb1; ++kb) {
        if (!mbar_wait(empty0 + 8 * s, ph ^ 1u, abort_flag, status, kStatusTimeoutEmpty)) break;
        const uint32_t fb = full_even + 8 * s;
        if (rank == 0) mbar_expect_tx(full0 + 8 * s, 2 * C::kStageBytes);
        const uint32_t sa = sa0 + s * kStageA, sb = sb0 + s * kStageA;
        if constexpr (a_mn) {
          tma_load_2d_pair(sa, &map_a, fb, ai, kb * kElems);
          tma_load_2d_pair(sa + kMnBlockBytes, &map_a, fb, ai + 64, kb * kElems);
        } else {
          tma_load_2d_pair(sa, &map_a, fb, kb * kElems, ai);
        }
        if constexpr (b_mn) {
          tma_load_2d_pair(sb, &map_b, fb, bi, kb * kElems);
          tma_load_2d_pair(sb + kMnBlockBytes, &map_b, fb, bi + 64, kb * kElems);
        } else {
          tma_load_2d_pair(sb, &map_b, fb, kb * kElems, bi);
        }
        if (++s == C::kStages) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (kb < kb1) {
        // aborting: give copies in flight time to land before the CTA exits
        const unsigned long long t0 = global_ns();
        while (global_ns() - t0 < 10000000ull) {
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0 && kb1 > kb0) {
      constexpr uint32_t idesc = linear_idesc(kFp8, a_mn, b_mn, 256, C::kBN);
      const uint64_t ad0 = a_mn ? smem_desc_mn(sa0) : smem_desc(sa0);
      const uint64_t bd0 = b_mn ? smem_desc_mn(sb0) : smem_desc(sb0);
      constexpr uint32_t ka = (a_mn ? 16 * kRowBytes : 32) >> 4, kbs = (b_mn ? 16 * kRowBytes : 32) >> 4;
      uint32_t s = 0, ph = 0, use = 0;
      bool ok = true;
      for (int k0 = kb0; ok && k0 < kb1; k0 += P.p.segment, ++use) {
        const uint32_t acc = use & 1;
        if (!mbar_wait(smem_u32(&acc_empty[acc]), ((use >> 1) & 1u) ^ 1u, abort_flag, status, kStatusTimeoutAccFree))
          break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * C::kBN;
        const int k1 = min(k0 + P.p.segment, kb1);
        for (int kb = k0; kb < k1; ++kb) {
          if (!mbar_wait(full0 + 8 * s, ph, abort_flag, status, kStatusTimeoutFull)) {
            ok = false;
            break;
          }
          const uint64_t ad = ad0 + s * (kStageA >> 4), bd = bd0 + s * (kStageA >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_pair<kFp8>(d_tmem, ad + ka * kk, bd + kbs * kk, idesc, (kb > k0 || kk > 0) ? 1u : 0u);
          mma_commit_mask(empty0 + 8 * s, both);
          if (++s == C::kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (ok) mma_commit_mask(smem_u32(&acc_full[acc]), both);
      }
      // every MMA issued by this thread has completed before TMEM goes
      mma_commit_local(smem_u32(drain));
      const unsigned long long t0 = global_ns();
      while (!mbar_try(smem_u32(drain), 0)) {
        if (global_ns() - t0 > kWaitLimitNs) {
          *abort_flag = 1u;
          atomicCAS(status, 0u, static_cast<uint32_t>(kStatusTimeoutDrain));
          break;
        }
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < kSum; ++c) sum[c] = 0.f;
    const uint32_t empty_even = peer_addr(smem_u32(&acc_empty[0]), even);
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + half * 128;
    ready = true;
    uint32_t use = 0;
    for (int k0 = kb0; ready && k0 < kb1; k0 += P.p.segment, ++use) {
      const uint32_t acc = use & 1;
      ready = __all_sync(0xffffffffu, mbar_wait(smem_u32(&acc_full[acc]), (use >> 1) & 1u, abort_flag, status,
                                                kStatusTimeoutAcc));
      if (!ready) break;
      tc_fence_after();
      if constexpr (kMode == kLinearDw) {
#pragma unroll
        for (int c = 0; c < 128; c += 16) {
          float v[16];
          tmem_ld16(lane_addr + acc * C::kBN + c, v);
#pragma unroll
          for (int j = 0; j < 16; ++j) sum[c + j] += v[j];
        }
        tc_fence_before();
        mbar_arrive_remote(empty_even + acc * 8);
      }
    }
    // the sums take the place of the ring: the pair's MMAs have completed
    // (acc_full).  Four columns of a lane are one 16-byte word: [column / 4][lane]
    if (ready) {
      float4* sums = reinterpret_cast<float4*>(smem);
#pragma unroll
      for (int c = 0; c < 128; c += 16) {
        float v[16];
        if constexpr (kMode == kLinearDw) {
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = sum[c + j];
        } else if (kb1 > kb0) {
          tmem_ld16(lane_addr + c, v);
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 16; j += 4)
          sums[(half * 128 + c + j) / 4 * BM + quarter * 32 + lane] = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
      }
    }
  }
  __syncwarp();
  cluster_sync();
  if (ready) {
    const LinearArgs& g = P.p.g;
    const int64_t row = static_cast<int64_t>(tb) * 256 + rank * BM + quarter * 32 + lane;
    float row_scale = 1.f;
    if (kFp8 && row < g.nb) row_scale = g.b_scale[row];
    uint32_t* table = reinterpret_cast<uint32_t*>(smem + C::kPartBytes) + (warp - 2) * kTableWords<32>;
    const uint32_t base = smem_u32(smem) + (quarter * 32 + lane) * 16;
    constexpr int kShare = C::kBN / kSplit / 2;                   // columns of this warp
#pragma unroll
    for (int c0 = 0; c0 < kShare; c0 += 32) {
      const int c = (part * 2 + half) * kShare + c0;
      const int64_t col = static_cast<int64_t>(ta) * C::kBN + c;
      if (col >= g.na) break;
      float v[32];
      float4 w[kSplit][8];
#pragma unroll
      for (int q = 0; q < kSplit; ++q) {
        const uint32_t peer = peer_addr(base, 2u * q + rank);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[q][i] = ld_cluster_f32x4(peer + (c / 4 + i) * (BM * 16));
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float4 t = w[0][i];
#pragma unroll
        for (int q = 1; q < kSplit; ++q) {
          t.x += w[q][i].x;
          t.y += w[q][i].y;
          t.z += w[q][i].z;
          t.w += w[q][i].w;
        }
        v[4 * i] = t.x;
        v[4 * i + 1] = t.y;
        v[4 * i + 2] = t.z;
        v[4 * i + 3] = t.w;
      }
      epilogue_row<kMode, kFp8, 32>(g, P.access, row_scale, row, col, table, lane, v);
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();            // no CTA leaves while another reads its sums or may still signal it
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols) : "memory");
  }
}

// ------------------------------------------------------- smaller kernels --

// Operand copies with rows on 16 bytes, up to three in one launch.  A thread
// writes one 16-byte piece of a row from as many single-element loads; a warp's
// loads of one turn lie within 512 bytes of a row.
template <typename T>
__global__ void __launch_bounds__(256) repack_kernel(const __grid_constant__ RepackBatch batch) {
  constexpr int kN = 16 / sizeof(T);
  let_next_start();
  wait_for_predecessors();
  int64_t piece = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  int i = 0;
  while (i < batch.n && piece >= batch.m[i].pieces) piece -= batch.m[i++].pieces;
  if (i == batch.n) return;
  const RepackMatrix& m = batch.m[i];
  const int64_t per_row = m.dst_ld / kN;
  const int64_t r = piece / per_row, c = (piece - r * per_row) * kN;
  const T* src = static_cast<const T*>(m.src) + r * m.src_ld + c;
  alignas(16) T v[kN];
#pragma unroll
  for (int j = 0; j < kN; ++j) v[j] = c + j < m.cols ? src[j] : T(0);
  *reinterpret_cast<uint4*>(static_cast<T*>(m.dst) + r * m.dst_ld + c) = *reinterpret_cast<const uint4*>(v);
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

bool rows_on_16(const void* p, int64_t ld, int64_t rows, int es) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (rows <= 1 || (ld * es) % 16 == 0);
}

// 2-D map of an output [rows][cols] in blocks of 32 rows x 128 bytes (128-byte
// swizzle); false when TMA cannot address it.
bool make_block_map(CUtensorMap* map, const void* p, int64_t ld, int64_t rows, int64_t cols, bool fp32) {
  const int es = fp32 ? 4 : 2;
  EncodeTiledFn fn = encode_fn();
  if (!fn || !rows_on_16(p, ld, rows, es)) return false;
  if (rows <= 1) ld = (cols + 7) / 8 * 8;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld * es)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(kRowBytes / es), 32};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p),
            dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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

int k_blocks_of(const LinearArgs& a) {
  const int64_t elems = a.fp8 ? 128 : 64;
  return static_cast<int>((a.nk + elems - 1) / elems);
}

template <int kMode>
PairParams pair_params(const LinearArgs& a, int bn, int total_tiles) {
  PairParams P{};
  P.g = a;
  P.k_blocks = k_blocks_of(a);
  P.segment = kMode == kLinearDw ? kDwSegment : P.k_blocks;
  P.tiles_a = static_cast<int>((a.na + bn - 1) / bn);
  P.tiles_b = static_cast<int>((a.nb + 255) / 256);
  P.total_tiles = total_tiles;
  return P;
}

template <int kMode>
RowAccess row_access(const LinearArgs& a) {
  RowAccess r{};
  if (kMode == kLinearDw) {
    r.out_vec = rows_on_16(a.dw, a.dw_ld, a.nb, 4);
  } else {
    r.out_vec = rows_on_16(a.y, a.y_ld, a.nb, 2) && (!a.z_out || rows_on_16(a.z_out, a.z_ld, a.nb, 2));
    r.in_vec = kMode == kLinearDx ? rows_on_16(a.z_in, a.z_ld, a.nb, 2)
                                  : rows_on_16(a.residual, a.residual_ld, a.nb, 2);
  }
  return r;
}

// The first `tiles` tiles.
template <int kMode, bool kFp8, int kBN>
cudaError_t launch_pair(const LinearArgs& a, int64_t tiles, cudaStream_t stream) {
  using C = PairConfig<kMode, kBN>;
  PairParams P = pair_params<kMode>(a, kBN, static_cast<int>(tiles));
  CUtensorMap ma, mb, mo{}, mz{};
  cudaError_t e;
  if ((e = make_operand_map(&ma, a.A, a.na, a.nk, kFp8, C::kHalf)) != cudaSuccess) return e;
  if ((e = make_operand_map(&mb, a.B, a.nb, a.nk, kFp8, BM)) != cudaSuccess) return e;
  if constexpr (kMode == kLinearDw) {
    P.out_tma = make_block_map(&mo, a.dw, a.dw_ld, a.nb, a.na, true);
  } else {
    P.out_tma = make_block_map(&mo, a.y, a.y_ld, a.nb, a.na, false) &&
                (!a.z_out || make_block_map(&mz, a.z_out, a.z_ld, a.nb, a.na, false));
    const uint16_t* in = kMode == kLinearDx ? a.z_in : a.residual;
    const int64_t in_ld = kMode == kLinearDx ? a.z_ld : a.residual_ld;
    P.in_vec = rows_on_16(in, in_ld, a.nb, 2);
    if (in && !P.in_vec && a.z_out) P.out_tma = 0;       // the table would take z's staging area
    P.in_tma = in && P.out_tma && P.in_vec && !a.z_out && make_block_map(&mz, in, in_ld, a.nb, a.na, false);
  }
  if ((e = allow_smem<linear_pair_kernel<kMode, kFp8, kBN>>(C::kSmemBytes)) != cudaSuccess) return e;
  const int max_pairs = num_sms() / 2;
  const int grid = 2 * (P.total_tiles < max_pairs ? P.total_tiles : max_pairs);
  return launch_overlapped(linear_pair_kernel<kMode, kFp8, kBN>, static_cast<unsigned>(grid), kPairThreads, C::kSmemBytes,
                           stream, 0, mb, ma, mo, mz, P);
}

// Tiles tile0 .. tile0 + tiles - 1 of 256 x 256, each by a cluster of pairs.
template <int kMode, bool kFp8>
cudaError_t launch_pair_split(const LinearArgs& a, int64_t tile0, int64_t tiles, cudaStream_t stream) {
  PairSplitParams P{};
  P.p = pair_params<kMode>(a, 256, static_cast<int>(tile0 + tiles));
  P.access = row_access<kMode>(a);
  P.per_pair = (P.p.k_blocks + kPairSplit - 1) / kPairSplit;
  P.tile0 = static_cast<int>(tile0);
  CUtensorMap ma, mb;
  cudaError_t e;
  if ((e = make_operand_map(&ma, a.A, a.na, a.nk, kFp8, 128)) != cudaSuccess) return e;
  if ((e = make_operand_map(&mb, a.B, a.nb, a.nk, kFp8, BM)) != cudaSuccess) return e;
  if ((e = allow_smem<linear_pair_split_kernel<kMode, kFp8>>(PairSplitConfig::kSmemBytes)) != cudaSuccess) return e;
  return launch_overlapped(linear_pair_split_kernel<kMode, kFp8>, static_cast<unsigned>(tiles * 2 * kPairSplit),
                           kPairSplitThreads, PairSplitConfig::kSmemBytes, stream, 2 * kPairSplit, mb, ma, P);
}

// Parameters and operand maps of a split product: m on the lanes, n on the columns.
template <int kMode, bool kFp8, int kBN, bool kRows>
cudaError_t plan_split(const LinearArgs& a, SplitParams* P, CUtensorMap* m, CUtensorMap* n) {
  P->g = a;
  P->k_blocks = k_blocks_of(a);
  P->tiles_m = ((kRows ? a.nb : a.na) + BM - 1) / BM;
  P->tiles = P->tiles_m * (((kRows ? a.na : a.nb) + kBN - 1) / kBN);
  // split while the CTAs still run at once, two to an SM, and each keeps 4
  // k-blocks (8 or 12: 10 to 50 % slower on 100 x 776 x 1000 and 1 x 2048 x 2048;
  // one CTA to an SM: 15 % slower on 331 x 2048 x 1024 and 64 x 4096 x 4096)
  P->split = 1;
  while (P->split < kMaxSplit && P->tiles * P->split * 2 <= 2 * num_sms() && P->k_blocks >= P->split * 2 * 4)
    P->split *= 2;
  P->per_rank = (P->k_blocks + P->split - 1) / P->split;
  P->segment = kMode == kLinearDw ? kDwSegment : P->k_blocks;
  P->access = row_access<kMode>(a);
  if (P->tiles > (int64_t(1) << 27)) return cudaErrorInvalidValue;
  const cudaError_t e = make_operand_map(kRows ? n : m, a.A, a.na, a.nk, kFp8, kRows ? kBN : BM);
  return e != cudaSuccess ? e : make_operand_map(kRows ? m : n, a.B, a.nb, a.nk, kFp8, kRows ? BM : kBN);
}

template <int kMode, bool kFp8, int kBN, bool kRows>
cudaError_t launch_split(const LinearArgs& a, cudaStream_t stream) {
  SplitParams P{};
  CUtensorMap m, n;
  cudaError_t e = plan_split<kMode, kFp8, kBN, kRows>(a, &P, &m, &n);
  if (e != cudaSuccess) return e;
  constexpr uint32_t kSmem = SplitConfig<kBN>::kSmemBytes;
  if ((e = allow_smem<linear_split_kernel<kMode, kFp8, kBN, kRows>>(kSmem)) != cudaSuccess) return e;
  return launch_overlapped(linear_split_kernel<kMode, kFp8, kBN, kRows>, static_cast<unsigned>(P.tiles * P.split),
                           kSplitThreads, kSmem, stream, P.split, m, n, P);
}

template <int kBN, bool kRows>
cudaError_t launch_grad(const LinearArgs& dx, const LinearArgs& dw, const ColumnSums* sums, cudaStream_t stream) {
  GradParams P{};
  CUtensorMap xm, xn, wm, wn;
  cudaError_t e;
  if ((e = plan_split<kLinearDx, false, kBN, kRows>(dx, &P.dx, &xm, &xn)) != cudaSuccess) return e;
  if ((e = plan_split<kLinearDw, false, 64, true>(dw, &P.dw, &wm, &wn)) != cudaSuccess) return e;
  const int cluster = P.dx.split > P.dw.split ? P.dx.split : P.dw.split;
  const auto whole = [cluster](int64_t blocks) { return (blocks + cluster - 1) / cluster * cluster; };
  P.dx_blocks = whole(P.dx.tiles * P.dx.split);
  P.dw_blocks = whole(P.dw.tiles * P.dw.split);
  int64_t blocks = P.dx_blocks + P.dw_blocks;
  if (sums) {
    P.sums = *sums;
    blocks += whole((sums->n + kSumCols - 1) / kSumCols);
  }
  constexpr uint32_t kSmem = SplitConfig<kBN>::kSmemBytes > SplitConfig<64>::kSmemBytes ? SplitConfig<kBN>::kSmemBytes
                                                                                     : SplitConfig<64>::kSmemBytes;
  if ((e = allow_smem<linear_grad_kernel<kBN, kRows>>(kSmem)) != cudaSuccess) return e;
  return launch_overlapped(linear_grad_kernel<kBN, kRows>, static_cast<unsigned>(blocks), kSplitThreads, kSmem, stream,
                           cluster, xm, xn, wm, wn, P);
}

// How a product runs.
struct Plan {
  int pair_width;        // of the pair kernel's tiles, or 0: the split kernel
  int64_t pair_tiles;    // by the pair kernel, the first ones
  int64_t tail_tiles;    // 256 x 256 tiles after them, by clusters of pairs
};

// The pair kernels take products of more than 128 rows (128 x 4096 x 4096: 25 us
// against 13 of the split kernel) once 256 x 128 tiles fill the pairs (64 of
// them: the split kernel takes 9.4 us for 2048 x 1024 x 1024 against 11.7), or
// from 24 tiles of 256 x 256 with 32 k-blocks if clusters of pairs split them
// (512 x 4096 x 4096, 32 tiles: 18 us against 25; 512 x 2048 x 2048, 16: 12.2
// against 10.1).  dw of a few tokens is little more than its stores: there twice
// the tiles (1 x 2048 x 2048, 128 tiles of 128: 10.9 us split against 12.0, and
// dx shares the launch).
//
// Measured cycles of a tile: 560 a k-block and 7000 besides when it is 256 wide,
// 500 and 4500 when 128 (both wait for their operands from L2: 58 and 49 bytes a
// cycle per SM), so the narrow one pays where it fills the last wave better or
// the sum is short.  A last wave of clusters takes 26000 besides its share of the
// k-blocks, the start of its own launch included (8192 x 4096 x 4096's dw: 187
// -> 179 us, 837 x 6784 x 8856: 112 -> 95 us).
Plan plan_product(const LinearArgs& a) {
  const int64_t pairs = num_sms() / 2, kb = k_blocks_of(a);
  const int64_t tiles_b = (a.nb + 255) / 256;
  const int64_t t256 = tiles_b * ((a.na + 255) / 256), t128 = tiles_b * ((a.na + 127) / 128);
  if (a.nb <= 128 || t128 >= (int64_t(1) << 30)) return Plan{};
  const auto waves = [pairs](int64_t t) { return (t + pairs - 1) / pairs; };
  const int64_t full = t256 / pairs * pairs, rest = t256 - full;
  if (t256 >= 24 && t256 <= pairs / kPairSplit && kb >= 32) return Plan{256, 0, t256};
  if (t128 < pairs * (a.mode == kLinearDw && kb <= 2 ? 2 : 1)) return Plan{};
  const int64_t tile256 = 560 * kb + 7000, tile128 = 500 * kb + 4500;
  const int64_t c256 = waves(t256) * tile256, c128 = waves(t128) * tile128;
  if (full > 0 && rest > 0 && rest <= pairs / kPairSplit) {
    const int64_t tail = full / pairs * tile256 + 560 * ((kb + kPairSplit - 1) / kPairSplit) + 26000;
    if (tail < c256 && tail < c128) return Plan{256, full, rest};
  }
  return c256 <= c128 ? Plan{256, t256, 0} : Plan{128, t128, 0};
}

// Rows to a tile of a split product with the lanes on the columns, or 0: the
// lanes on the rows.  The former read the weights' tile once for up to 64 rows
// (64 x 14336 x 4096: 24 us against 26, 50 x 8576 x 984: 9 against 13), but
// store 2 bytes a lane: with few k-blocks that shows (64 x 1024 x 1024 in e4m3:
// 7.1 us against 5.4).
int column_lanes(const LinearArgs& a) {
  if (a.nb <= 16) return 16;
  if (a.nb <= 32) return 32;
  return a.nb <= 64 && k_blocks_of(a) >= 16 ? 64 : 0;
}

template <int kMode, bool kFp8>
cudaError_t launch_product(const LinearArgs& a, cudaStream_t stream) {
  const Plan plan = plan_product(a);
  if (plan.pair_width) {
    cudaError_t e = cudaSuccess;
    if (plan.pair_tiles > 0)
      e = plan.pair_width == 256 ? launch_pair<kMode, kFp8, 256>(a, plan.pair_tiles, stream)
                                 : launch_pair<kMode, kFp8, 128>(a, plan.pair_tiles, stream);
    if (e != cudaSuccess || plan.tail_tiles == 0) return e;
    return launch_pair_split<kMode, kFp8>(a, plan.pair_tiles, plan.tail_tiles, stream);
  }
  if constexpr (kMode != kLinearDw) {
    switch (column_lanes(a)) {
      case 16: return launch_split<kMode, kFp8, 16, false>(a, stream);
      case 32: return launch_split<kMode, kFp8, 32, false>(a, stream);
      case 64: return launch_split<kMode, kFp8, 64, false>(a, stream);
      default: break;
    }
  }
  return launch_split<kMode, kFp8, 64, true>(a, stream);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t stream) {
  if (a.na <= 0 || a.nb <= 0) return cudaSuccess;
  if (a.mode == kLinearDx) return launch_product<kLinearDx, false>(a, stream);
  if (a.mode == kLinearDw) return launch_product<kLinearDw, false>(a, stream);
  return a.fp8 ? launch_product<kLinearForward, true>(a, stream) : launch_product<kLinearForward, false>(a, stream);
}

namespace {

ColumnSums plan_sums(const ColumnSumArgs& a) {
  const bool vec = a.n % 2 == 0 && (reinterpret_cast<uintptr_t>(a.dz) & 3u) == 0 && (a.m <= 1 || a.ld % 2 == 0);
  return ColumnSums{a.dz, a.ld, a.m, a.n, a.out, a.partial, a.accumulate, vec};
}

}  // namespace

bool linear_grad_fits(const LinearArgs& dx, const LinearArgs& dw) {
  return plan_product(dx).pair_width == 0 && plan_product(dw).pair_width == 0;
}

cudaError_t launch_linear_grad(const LinearArgs& dx, const LinearArgs& dw, const ColumnSumArgs* sums,
                               cudaStream_t stream) {
  ColumnSums s{};
  if (sums) s = plan_sums(*sums);
  const ColumnSums* p = sums ? &s : nullptr;
  switch (column_lanes(dx)) {
    case 16: return launch_grad<16, false>(dx, dw, p, stream);
    case 32: return launch_grad<32, false>(dx, dw, p, stream);
    case 64: return launch_grad<64, false>(dx, dw, p, stream);
    default: return launch_grad<64, true>(dx, dw, p, stream);
  }
}

cudaError_t launch_column_sums(const ColumnSumArgs& a, cudaStream_t stream) {
  const unsigned gx = static_cast<unsigned>((a.n + kSumCols - 1) / kSumCols);
  const int64_t slices = column_sum_slices(a.m, a.n);
  const cudaError_t e = launch_overlapped(column_sums_kernel, dim3(gx, static_cast<unsigned>(slices)), kSplitThreads, 0,
                                          stream, 0, plan_sums(a));
  if (e != cudaSuccess || slices == 1) return e;
  return launch_overlapped(join_sums_kernel, static_cast<unsigned>((a.n + 127) / 128), 128, 0, stream, 0,
                           static_cast<const float*>(a.partial), static_cast<int>(slices), a.n, a.out, a.accumulate);
}

cudaError_t launch_repack(const RepackBatch& batch, int esize, cudaStream_t stream) {
  int64_t pieces = 0;
  for (int i = 0; i < batch.n; ++i) pieces += batch.m[i].pieces;
  const int64_t grid = (pieces + 255) / 256;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  if (grid == 0) return cudaSuccess;
  return launch_overlapped(esize == 1 ? repack_kernel<uint8_t> : repack_kernel<uint16_t>, static_cast<unsigned>(grid),
                           256, 0, stream, 0, batch);
}

}  // namespace mpopt
