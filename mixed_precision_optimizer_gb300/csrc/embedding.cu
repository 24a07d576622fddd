// Embedding lookup and its gradient (sm_103a):
//
//   y[r] = table[token[r]] * scale
//   dtable[v] += scale * sum over the rows r with token[r] = v of dy[r]
//
// The lookup copies rows.  The gradient first sorts the rows by token, so that
// the rows of one token are neighbours and one thread adds a column of all of
// them in registers: dtable is touched once for each distinct token and no
// addition is atomic.
//   embedding_rank_kernel  few rows: each row's place by comparing its token with
//                          all others
//   embedding_sort_kernel  more rows: a stable radix sort of (token, row) by one
//                          cluster
//   embedding_sums_kernel  sums the runs of equal tokens within pieces of the
//                          sorted rows; a run that crosses a piece's border
//                          leaves a partial sum for each piece
//   embedding_join_kernel  adds the partial sums of such runs in order

#include "cluster.cuh"
#include "elements.cuh"
#include "internal.h"
#include "overlap.cuh"

namespace mpopt {
namespace {

constexpr int kThreads = 256;

bool rows_on_16(const void* p, int64_t ld, int es, int64_t rows) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || static_cast<uintptr_t>(ld) * es % 16 == 0);
}

__device__ __forceinline__ int64_t token_at(const void* tokens, int index_dtype, int64_t r) {
  return index_dtype == OPT_INDEX_INT32 ? static_cast<int64_t>(static_cast<const int32_t*>(tokens)[r])
                                        : static_cast<const int64_t*>(tokens)[r];
}

// --------------------------------------------------------------- columns --

// Four columns as loaded (bf16 stays packed until it is used), or one.
template <typename T, int kN>
struct Raw {
  float v[kN];
  __device__ __forceinline__ void load(const T* p);
  __device__ __forceinline__ float get(int j) const { return v[j]; }
};
template <>
struct Raw<__nv_bfloat16, 4> {
  uint2 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ float get(int j) const {
    const uint32_t u = j < 2 ? w.x : w.y;
    return __uint_as_float(j & 1 ? u & 0xffff0000u : u << 16);
  }
};

// One, 4 or 8 neighbouring columns.
__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
  const float4 f = *reinterpret_cast<const float4*>(p);
  v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&v)[4]) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(u.x << 16), v[1] = __uint_as_float(u.x & 0xffff0000u);
  v[2] = __uint_as_float(u.y << 16), v[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
}
template <typename T, int kN>
__device__ __forceinline__ void load_columns(const T* p, float (&v)[kN]) {
  if constexpr (kN == 8) load8(p, v);
  else if constexpr (kN == 4) load4(p, v);
  else v[0] = load_elem(p);
}
template <typename T, int kN>
__device__ __forceinline__ void store_columns(T* p, const float (&v)[kN]) {
  if constexpr (kN == 8) store8(p, v);
  else if constexpr (kN == 4) store4(p, v);
  else store_elem(p, v[0]);
}

template <typename T, int kN>
__device__ __forceinline__ void Raw<T, kN>::load(const T* p) {
  load_columns(p, v);
}

// ---------------------------------------------------------------- lookup --

// A thread has some columns of kRows rows, whose loads are on their way together:
// first the tokens, then the table's rows; 2^log_tpr threads to a row.  The columns
// are 16 bytes of the wider type (4, or 8 where both are bf16: neighbouring lanes
// store neighbouring 16 bytes; 8 columns of an fp32 output took 16384 x 4096
// from 59 to 66 us, four take 54), or one where rows do not start on 16 bytes.
constexpr int kRows = 4;
template <typename T, typename O, bool kVec>
constexpr int kLookupCols = !kVec ? 1 : sizeof(T) == 2 && sizeof(O) == 2 ? 8 : 4;
template <typename T, typename O, bool kVec>
__global__ void __launch_bounds__(kThreads) embedding_kernel(const __grid_constant__ opt_embedding_args a, int log_tpr,
                                                             uint32_t slices) {
  constexpr int kN = kLookupCols<T, O, kVec>;
  let_next_start();
  wait_for_predecessors();
  const uint32_t block = blockIdx.x / slices, slice = blockIdx.x - block * slices;
  const int64_t c = ((static_cast<int64_t>(slice) << log_tpr) + (threadIdx.x & ((1 << log_tpr) - 1))) * kN;
  if (c >= a.cols) return;
  const int per_step = kThreads >> log_tpr;
  const int64_t r0 = static_cast<int64_t>(block) * per_step * kRows + (threadIdx.x >> log_tpr);
  int64_t token[kRows];
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int64_t r = r0 + u * per_step;
    token[u] = r < a.rows ? token_at(a.tokens, a.index_dtype, r) : -1;
  }
  float v[kRows][kN];
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    if (token[u] >= 0 && token[u] < a.vocab) {
      const T* src = static_cast<const T*>(a.table) + token[u] * a.table_ld + c;
      load_columns(src, v[u]);
#pragma unroll
      for (int j = 0; j < kN; ++j) v[u][j] *= a.scale;
    } else {
#pragma unroll
      for (int j = 0; j < kN; ++j) v[u][j] = 0.f;
    }
  }
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int64_t r = r0 + u * per_step;
    if (r >= a.rows) return;
    O* dst = static_cast<O*>(a.y) + r * a.y_ld + c;
    store_columns(dst, v[u]);
  }
}

template <typename T, typename O>
cudaError_t lookup(const opt_embedding_args& a, cudaStream_t stream) {
  const bool vec = a.cols % 8 == 0 && rows_on_16(a.table, a.table_ld, sizeof(T), a.vocab) &&
                   rows_on_16(a.y, a.y_ld, sizeof(O), a.rows);
  const int64_t groups = a.cols / (vec ? kLookupCols<T, O, true> : 1);
  int log_tpr = 0;
  while (log_tpr < 8 && (int64_t(1) << log_tpr) < groups) ++log_tpr;
  const int64_t slices = (groups + (int64_t(1) << log_tpr) - 1) >> log_tpr, per_cta = (kThreads >> log_tpr) * kRows;
  const dim3 grid(static_cast<unsigned>((a.rows + per_cta - 1) / per_cta * slices));
  return vec ? launch_overlapped(embedding_kernel<T, O, true>, grid, kThreads, 0, stream, 0, a, log_tpr, static_cast<uint32_t>(slices))
             : launch_overlapped(embedding_kernel<T, O, false>, grid, kThreads, 0, stream, 0, a, log_tpr, static_cast<uint32_t>(slices));
}

// ------------------------------------------------------------------ sort --

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxBits = 10;                     // of a digit: [32][1024] counters fit shared memory
constexpr int kSortCluster = 8;

struct SortArgs {
  const void* tokens;
  int index_dtype;
  int64_t rows, vocab;
  EmbeddingScratch ws;
  int passes, bits;
  int64_t per_warp;      // rows of one warp, a multiple of 32
};

// Least significant digit first.  Every warp owns consecutive rows; a digit's
// place is the rows of smaller digits, plus those with this digit of lower
// CTAs, of lower warps, and earlier ones of the warp: a stable order.  Bound by
// latency (20 us for 16384 rows in two passes, 52 between events for 65536): the
// first kHeld keys of a lane are loaded at once and kept for the second look at
// them, and every CTA stores its totals into the others' memory.
constexpr int kHeld = 4;

__global__ void __launch_bounds__(kSortThreads) embedding_sort_kernel(const __grid_constant__ SortArgs a) {
  extern __shared__ uint32_t counts[];            // [kSortWarps][bins], then [CTAs][bins] totals
  __shared__ uint32_t scan[kSortWarps];
  let_next_start();
  wait_for_predecessors();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = cluster_rank(), ctas = cluster_size();
  const int bins = 1 << a.bits;
  uint32_t* total = counts + kSortWarps * bins;
  uint32_t* mine = counts + warp * bins;
  const int64_t first = (static_cast<int64_t>(rank) * kSortWarps + warp) * a.per_warp;
  const int64_t last = first + a.per_warp < a.rows ? first + a.per_warp : a.rows;
  cluster_sync();                                 // every CTA has begun
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.bits;
    const uint32_t *key_in = a.ws.key[pass & 1], *row_in = a.ws.row[pass & 1];
    uint32_t *key_out = a.ws.key[(pass & 1) ^ 1], *row_out = a.ws.row[(pass & 1) ^ 1];
    auto key_at = [&](int64_t i) {
      if (i >= last) return 0u;
      if (pass) return key_in[i];
      const int64_t t = token_at(a.tokens, a.index_dtype, i);
      return static_cast<uint32_t>(t >= 0 && t < a.vocab ? t : a.vocab);
    };
    auto row_at = [&](int64_t i) { return pass && i < last ? row_in[i] : static_cast<uint32_t>(i); };
    uint32_t held[kHeld], held_row[kHeld];
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
      held[k] = key_at(first + k * 32 + lane);
      held_row[k] = row_at(first + k * 32 + lane);
    }
    for (int i = threadIdx.x; i < kSortWarps * bins; i += kSortThreads) counts[i] = 0;
    __syncthreads();
    // the lanes with this lane's digit (none beyond the last row: they share a digit that does not exist)
    auto same_digit = [&](int64_t i, uint32_t key, uint32_t& digit) {
      digit = i < last ? (key >> shift) & (bins - 1) : static_cast<uint32_t>(bins);
      return __match_any_sync(0xffffffffu, digit);
    };
    auto count = [&](int64_t i, uint32_t key) {
      uint32_t digit;
      const uint32_t same = same_digit(i, key, digit);
      if (i < last && lane == __ffs(same) - 1) mine[digit] += __popc(same);
      __syncwarp();
    };
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (first + k * 32 < last) count(first + k * 32 + lane, held[k]);
    for (int64_t i = first + kHeld * 32 + lane; i - lane < last; i += 32) count(i, key_at(i));
    __syncthreads();
    // one thread to a digit (bins <= threads)
    const int d = threadIdx.x;
    if (d < bins) {
      uint32_t sum = 0;
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t n = counts[w * bins + d];
        counts[w * bins + d] = sum;
        sum += n;
      }
      for (uint32_t r = 0; r < ctas; ++r) store_peer(at_peer(total + rank * bins + d, r), sum);
    }
    cluster_sync();
    uint32_t before = 0, all = 0;
    if (d < bins) {
      for (uint32_t r = 0; r < ctas; ++r) {
        const uint32_t n = total[r * bins + d];
        if (r < rank) before += n;
        all += n;
      }
    }
    // exclusive sum of `all` over the digits
    uint32_t up = all;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, up, off);
      if (lane >= off) up += o;
    }
    if (lane == 31) scan[warp] = up;
    __syncthreads();
    uint32_t base = lane < warp ? scan[lane] : 0u;               // the warps before this one
    base = __reduce_add_sync(0xffffffffu, base) + up - all + before;
    if (d < bins) {
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) counts[w * bins + d] += base;
    }
    __syncthreads();
    auto place = [&](int64_t i, uint32_t key, uint32_t row) {
      uint32_t digit;
      const uint32_t same = same_digit(i, key, digit);
      if (i < last) {
        const uint32_t at = mine[digit] + __popc(same & ((1u << lane) - 1));
        key_out[at] = key;
        row_out[at] = row;
      }
      __syncwarp();
      if (i < last && lane == __ffs(same) - 1) mine[digit] += __popc(same);
      __syncwarp();
    };
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (first + k * 32 < last) place(first + k * 32 + lane, held[k], held_row[k]);
    for (int64_t i = first + kHeld * 32 + lane; i - lane < last; i += 32) place(i, key_at(i), row_at(i));
    cluster_sync();              // the next pass reads what other CTAs wrote, and writes to their totals
  }
}

// ------------------------------------------------------------------ rank --

// A row's place is the number of smaller tokens and of equal ones before it.  Every
// CTA has 32 rows and the tokens of all, 1024 at a time in shared memory, of
// which each of a row's eight threads compares an eighth: rows^2 comparisons over
// all SMs in one step without a barrier between CTAs.  Bound by latency for few rows,
// by the comparisons for many (between events 777 rows take 10 us, 4096 14, 8192 25,
// 16384 58; the radix sort 18 and, from 4096 rows on, 25).
constexpr int kRankRows = 32, kRankTile = 1024;
constexpr int64_t kRankMost = 8192;

__global__ void __launch_bounds__(kThreads) embedding_rank_kernel(const __grid_constant__ SortArgs a) {
  __shared__ __align__(16) uint32_t tile[kRankTile];
  let_next_start();
  wait_for_predecessors();
  const int rows = static_cast<int>(a.rows), part = threadIdx.x & 7;
  const int row = blockIdx.x * kRankRows + static_cast<int>(threadIdx.x >> 3);
  auto key_at = [&](int i) {
    if (i >= rows) return 0xffffffffu;                  // above all: no row is behind it
    const int64_t t = token_at(a.tokens, a.index_dtype, i);
    return static_cast<uint32_t>(t >= 0 && t < a.vocab ? t : a.vocab);
  };
  const uint32_t mine = key_at(row);
  uint32_t before = 0;
  for (int first = 0; first < rows; first += kRankTile) {
    __syncthreads();
    for (int i = threadIdx.x; i < kRankTile; i += kThreads) tile[i] = key_at(first + i);
    __syncthreads();
    if (first + kRankTile <= row || first > row) {      // all of them before the row, or all behind it
      const bool behind = first > row;
#pragma unroll 8
      for (int i = part * 4; i < kRankTile; i += 32) {
        const uint4 k = *reinterpret_cast<const uint4*>(tile + i);
        if (behind) before += (k.x < mine) + (k.y < mine) + (k.z < mine) + (k.w < mine);
        else before += (k.x <= mine) + (k.y <= mine) + (k.z <= mine) + (k.w <= mine);
      }
    } else {
      for (int i = part; i < kRankTile; i += 8) before += first + i < row ? tile[i] <= mine : tile[i] < mine;
    }
  }
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) before += __shfl_xor_sync(0xffffffffu, before, off);
  if (part == 0 && row < rows) {
    a.ws.key[0][before] = mine;
    a.ws.row[0][before] = static_cast<uint32_t>(row);
  }
}

// ------------------------------------------------------------------ sums --

struct SumArgs {
  opt_embedding_grad_args a;
  const uint32_t *key, *row;
  float* partial;          // [pieces][2][cols]
  uint32_t slices;         // CTAs to a piece
  int piece;               // rows
};

// 4 columns to a thread, 16 bytes of the table, or one.
template <bool kVec>
constexpr int kSumCols = kVec ? 4 : 1;
constexpr int kAhead = 8;                        // rows on their way to a thread together
constexpr int kJoinAhead = 8;

// A run's sum goes to the table if the run lies within the piece, else to the
// piece's first partial row (a run that came from the piece before) or its
// second (a run that starts here and goes on).  What the table holds at a run's
// end is loaded with the run's last row.  Bound by HBM: 16384 rows of 4096 bf16
// columns into a table of 128256 rows take 59 us, 0.9 of the measured copy rate;
// with four rows on their way instead of eight 95, with each row's place filled
// again as it is used 165 (a wait for one load waits for others).
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) embedding_sums_kernel(const __grid_constant__ SumArgs p) {
  constexpr int kN = kSumCols<kVec>;
  __shared__ uint32_t key[kEmbeddingPiece + 2], row[kEmbeddingPiece];
  let_next_start();
  wait_for_predecessors();
  const opt_embedding_grad_args& a = p.a;
  const uint32_t piece = blockIdx.x / p.slices;
  const int64_t first = static_cast<int64_t>(piece) * p.piece;
  const int n = static_cast<int>(a.rows - first < p.piece ? a.rows - first : p.piece);
  const uint32_t none = static_cast<uint32_t>(a.vocab);
  // key[0] and key[n + 1]: the neighbouring pieces' (a token outside the table where there is none)
  for (int i = threadIdx.x; i < n + 2; i += kThreads) {
    const int64_t at = first + i - 1;
    key[i] = at >= 0 && at < a.rows ? p.key[at] : none;
  }
  for (int i = threadIdx.x; i < n; i += kThreads) row[i] = p.row[first + i];
  __syncthreads();
  const int64_t c = (static_cast<int64_t>(blockIdx.x - piece * p.slices) * kThreads + threadIdx.x) * kN;
  if (c >= a.cols) return;
  const T* dy = static_cast<const T*>(a.dy) + c;
  float* table = a.dtable + c;
  float sum[kN];
#pragma unroll
  for (int j = 0; j < kN; ++j) sum[j] = 0.f;
  bool from_before = key[0] == key[1];
  for (int i0 = 0; i0 < n; i0 += kAhead) {
    Raw<T, kN> next[kAhead];
    float old[kAhead][kN];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u;
      if (i >= n || key[i + 1] == none) break;
      next[u].load(dy + row[i] * a.dy_ld);
      if (key[i + 2] != key[i + 1]) load_columns(static_cast<const float*>(table) + key[i + 1] * a.cols, old[u]);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u;
      if (i >= n) return;
      const uint32_t v = key[i + 1];
      if (v == none) return;                     // and so are all rows behind it
#pragma unroll
      for (int j = 0; j < kN; ++j) sum[j] += next[u].get(j);
      const bool ends_here = key[i + 2] != v;
      if (ends_here || i + 1 == n) {
        if (from_before || !ends_here) {
          store_columns(p.partial + (2 * static_cast<int64_t>(piece) + (from_before ? 0 : 1)) * a.cols + c, sum);
        } else {
#pragma unroll
          for (int j = 0; j < kN; ++j) old[u][j] += sum[j] * a.scale;
          store_columns(table + v * a.cols, old[u]);
        }
        from_before = false;
#pragma unroll
        for (int j = 0; j < kN; ++j) sum[j] = 0.f;
      }
    }
  }
}

// The CTA of the piece in which a run starts that goes on behind it.
template <bool kVec>
__global__ void __launch_bounds__(kThreads) embedding_join_kernel(const __grid_constant__ SumArgs p) {
  constexpr int kN = kSumCols<kVec>;
  let_next_start();
  wait_for_predecessors();
  const opt_embedding_grad_args& a = p.a;
  const uint32_t piece = blockIdx.x / p.slices;
  const int64_t start = static_cast<int64_t>(piece) * p.piece, last = start + p.piece - 1;
  if (last + 1 >= a.rows) return;
  const uint32_t v = p.key[last];
  if (v >= static_cast<uint32_t>(a.vocab) || p.key[last + 1] != v) return;
  if (piece > 0 && p.key[start - 1] == v && p.key[start] == v) return;        // it started earlier
  // the run's last piece: the first one behind this that it does not fill, or, where
  // that does not begin with it, the one before; each warp looks at 32 pieces a time
  int64_t last_piece = piece + 1;
  for (uint32_t full = 0xffffffffu; full == 0xffffffffu;) {
    const int64_t end = (last_piece + static_cast<int>(threadIdx.x & 31) + 1) * p.piece - 1;
    full = __ballot_sync(0xffffffffu, end < a.rows && p.key[end] == v);
    last_piece += full == 0xffffffffu ? 32 : __ffs(~full) - 1;
  }
  if (last_piece * p.piece >= a.rows || p.key[last_piece * p.piece] != v) --last_piece;
  const int64_t c = (static_cast<int64_t>(blockIdx.x - piece * p.slices) * kThreads + threadIdx.x) * kN;
  if (c >= a.cols) return;
  float sum[kN], old[kN];
  float* table = a.dtable + v * a.cols + c;
  load_columns(static_cast<const float*>(table), old);
  load_columns(static_cast<const float*>(p.partial) + (2 * static_cast<int64_t>(piece) + 1) * a.cols + c, sum);
  for (int64_t q0 = piece + 1; q0 <= last_piece; q0 += kJoinAhead) {
    float part[kJoinAhead][kN];
#pragma unroll
    for (int u = 0; u < kJoinAhead; ++u)
      if (q0 + u <= last_piece) load_columns(static_cast<const float*>(p.partial) + 2 * (q0 + u) * a.cols + c, part[u]);
#pragma unroll
    for (int u = 0; u < kJoinAhead; ++u)
      if (q0 + u <= last_piece) {
#pragma unroll
        for (int j = 0; j < kN; ++j) sum[j] += part[u][j];
      }
  }
#pragma unroll
  for (int j = 0; j < kN; ++j) old[j] += sum[j] * a.scale;
  store_columns(table, old);
}

// 4 columns to a thread where rows of dy, the table and the partial sums start on 16 bytes.
bool grad_vec(const opt_embedding_grad_args& a) {
  return a.cols % 8 == 0 && rows_on_16(a.dy, a.dy_ld, a.dtype == kBf16 ? 2 : 4, a.rows) &&
         reinterpret_cast<uintptr_t>(a.dtable) % 16 == 0;
}

SumArgs sum_args(const opt_embedding_grad_args& a, const EmbeddingScratch& ws, int sorted, bool vec) {
  const int64_t per_cta = kThreads * (vec ? kSumCols<true> : 1);
  return SumArgs{a, ws.key[sorted], ws.row[sorted], ws.partial, static_cast<uint32_t>((a.cols + per_cta - 1) / per_cta),
                 embedding_piece(a.rows)};
}

}  // namespace

cudaError_t launch_embedding(const opt_embedding_args& a, cudaStream_t stream) {
  if (a.dtype == kBf16)
    return a.y_dtype == kBf16 ? lookup<__nv_bfloat16, __nv_bfloat16>(a, stream) : lookup<__nv_bfloat16, float>(a, stream);
  return a.y_dtype == kBf16 ? lookup<float, __nv_bfloat16>(a, stream) : lookup<float, float>(a, stream);
}

cudaError_t launch_embedding_sort(const opt_embedding_grad_args& a, const EmbeddingScratch& ws, int* sorted,
                                  cudaStream_t stream) {
  if (a.rows <= kRankMost) {
    const SortArgs s{a.tokens, a.index_dtype, a.rows, a.vocab, ws, 0, 0, 0};
    *sorted = 0;
    return launch_overlapped(embedding_rank_kernel, dim3(static_cast<unsigned>((a.rows + kRankRows - 1) / kRankRows)), kThreads, 0,
                             stream, 0, s);
  }
  int key_bits = 1;                              // of tokens 0 .. vocab
  while (a.vocab >> key_bits) ++key_bits;
  SortArgs s{a.tokens, a.index_dtype, a.rows, a.vocab, ws, (key_bits + kMaxBits - 1) / kMaxBits, 0, 0};
  s.bits = (key_bits + s.passes - 1) / s.passes;
  const int cluster = kSortCluster;
  const int64_t warps = static_cast<int64_t>(cluster) * kSortWarps;
  s.per_warp = ((a.rows + warps - 1) / warps + 31) & ~int64_t(31);
  *sorted = s.passes & 1;
  const size_t smem = static_cast<size_t>(kSortWarps + cluster) * (size_t(1) << s.bits) * 4;
  const cudaError_t e = cudaFuncSetAttribute(embedding_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (kSortWarps + kSortCluster) * (1 << kMaxBits) * 4);
  if (e != cudaSuccess) return e;
  return launch_overlapped(embedding_sort_kernel, dim3(static_cast<unsigned>(cluster)), kSortThreads, smem, stream, cluster, s);
}

cudaError_t launch_embedding_sums(const opt_embedding_grad_args& a, const EmbeddingScratch& ws, int sorted,
                                  cudaStream_t stream) {
  const bool vec = grad_vec(a);
  const SumArgs p = sum_args(a, ws, sorted, vec);
  const dim3 grid(static_cast<unsigned>(embedding_pieces(a.rows) * p.slices));
  if (a.dtype == kBf16)
    return vec ? launch_overlapped(embedding_sums_kernel<__nv_bfloat16, true>, grid, kThreads, 0, stream, 0, p)
               : launch_overlapped(embedding_sums_kernel<__nv_bfloat16, false>, grid, kThreads, 0, stream, 0, p);
  return vec ? launch_overlapped(embedding_sums_kernel<float, true>, grid, kThreads, 0, stream, 0, p)
             : launch_overlapped(embedding_sums_kernel<float, false>, grid, kThreads, 0, stream, 0, p);
}

cudaError_t launch_embedding_join(const opt_embedding_grad_args& a, const EmbeddingScratch& ws, int sorted,
                                  cudaStream_t stream) {
  const bool vec = grad_vec(a);
  const SumArgs p = sum_args(a, ws, sorted, vec);
  const dim3 grid(static_cast<unsigned>(embedding_pieces(a.rows) * p.slices));
  return vec ? launch_overlapped(embedding_join_kernel<true>, grid, kThreads, 0, stream, 0, p)
             : launch_overlapped(embedding_join_kernel<false>, grid, kThreads, 0, stream, 0, p);
}

}  // namespace mpopt
