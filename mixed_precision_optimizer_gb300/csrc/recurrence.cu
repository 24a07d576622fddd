// Gated recurrence along the rows of packed sequences, and its gradient (sm_103a):
//
//   h_t = h_{t-1} + c_t (x_t - h_{t-1}),  c = 1 / (1 + exp(-gate))
//   l_t = dy_t + (1 - c_{t+1}) l_{t+1};  dx_t = c_t l_t
//   dgate_t = c_t (1 - c_t) l_t (x_t - h_{t-1})
//
// Rows t1 .. t2 take a state h to  B + (1 - C) h,  where B is their result from
// h = 0 and 1 - C the product of their 1 - c; the gradient passes them the same
// way backwards.  C is kept, not 1 - C: slow channels have c far below 2^-24.
// Two such pieces, the first (C1, B1) and behind it (C2, B2), make
//   C = C1 + C2 - C1 C2,  B = B2 + (1 - C2) B1
// A piece in which a sequence starts or ends does not depend on the state before
// it: C = kReset, and B is selected, not multiplied, so that an infinity or a NaN
// stays in its own sequence.
//
// A warp has 64 columns, two to a lane, and 16 rows (bf16; fp32 8) at a time in
// shared memory, fetched with cp.async while it works on the rows before.  Its
// eight warps' pieces, and those of the CTAs of a cluster, which take the next
// rows each, are joined through (distributed) shared memory; then every thread
// runs through its rows again from the right state.  Bound by HBM: x and gate
// are read once (and dy), the outputs written once; a state for every 16 rows
// in fp32 is all that the gradient needs of the forward pass.

#include "elements.cuh"
#include "internal.h"
#include "overlap.cuh"

namespace mpopt {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kCols = 64;                        // of a CTA
constexpr int kMaxCluster = 8;                   // a warp of a CTA for each
constexpr float kReset = 2.f;

// ---------------------------------------------------------------- pieces --

struct Piece {
  float c, b;
};
__device__ __forceinline__ Piece then(Piece first, Piece second) {
  if (second.c >= kReset) return second;
  return Piece{first.c >= kReset ? kReset : fmaf(second.c, 1.f - first.c, first.c),
               fmaf(-second.c, first.b, first.b) + second.b};
}
__device__ __forceinline__ float through(Piece p, float h) { return p.c >= kReset ? p.b : fmaf(-p.c, h, h) + p.b; }

// 1 / (1 + e^-g) from two approximate instructions of 2 units each; the rounding
// of g log2 e adds 2^-24 |g| of the value.  0 below g = -87.
__device__ __forceinline__ float exp_neg(float g) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * g));
  return e;
}
__device__ __forceinline__ float update_gate(float g) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + exp_neg(g)));
  return r;
}
// 1 - c, as exact as c where c is near one too.
__device__ __forceinline__ float one_minus(float c, float g) { return g > 0.f ? c * exp_neg(g) : 1.f - c; }

// --------------------------------------------------------------- cluster --

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t at_peer(const void* p, uint32_t rank) {
  uint32_t m;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(m)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
  return m;
}
__device__ __forceinline__ void store_peer(uint32_t at, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}
__device__ __forceinline__ void store_peer(uint32_t at, int64_t v) {
  asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}

// ----------------------------------------------------------------- layout --

template <typename T>
struct Rows {
  static constexpr int kS = 32 / sizeof(T);              // of a thread at a time
  static constexpr int kChunk = kWarps * kS;             // of a CTA at a time
  static constexpr int kTile = kS * kCols * sizeof(T);   // bytes of a warp's rows of one tensor
};

struct Plan {
  int cluster, ranges, groups;      // CTAs to a cluster; shares of the sequences; shares of the columns
  int64_t length;                   // rows of a sequence without starts
};

// The sequences and rows of a cluster.
struct Span {
  int64_t seq, seq_end, row, row_end;
};

struct Shared {
  float4* pieces;        // [2][kWarps][32]: two columns' (c, b) of a warp
  float4* inbox;         // [2][cluster][32]: of a CTA
  int* first;            // [kChunk] with starts: the sequence that a row starts, or -1
  int* last;             // [kChunk]              the sequence that a row ends, or -1
  Span* span;
};

template <typename T, int kTensors>
struct Layout {
  static constexpr int kStage = kTensors * Rows<T>::kTile * kWarps;
  static size_t bytes(int cluster) {
    return 2 * kStage + 2 * kWarps * 512 + (cluster > 1 ? 2 * cluster * 512 : 0) + 2 * Rows<T>::kChunk * 4 + 64;
  }
  static __device__ __forceinline__ Shared carve(uint8_t* base, int cluster) {
    Shared s;
    base += 2 * kStage;
    s.pieces = reinterpret_cast<float4*>(base);
    s.inbox = s.pieces + 2 * kWarps * 32;
    s.first = reinterpret_cast<int*>(s.inbox + (cluster > 1 ? 2 * cluster * 32 : 0));
    s.last = s.first + Rows<T>::kChunk;
    s.span = reinterpret_cast<Span*>(s.last + Rows<T>::kChunk);
    return s;
  }
};

// -------------------------------------------------------------- sequences --

__device__ __forceinline__ int64_t start_at(const int32_t* starts, int64_t i, int64_t rows) {
  const int64_t v = starts[i];
  return v < 0 ? 0 : v > rows ? rows : v;
}

// First index in [0, n] whose start is not below v (n: none), by one warp: 32 probes a step.
__device__ __forceinline__ int64_t lower_bound(const int32_t* starts, int64_t n, int64_t v, int lane) {
  int64_t lo = 0, hi = n;                        // starts before lo are below v, those from hi on are not
  while (hi > lo) {
    const int64_t step = (hi - lo + 31) / 32, at = lo + lane * step;
    const int k = __popc(__ballot_sync(0xffffffffu, at < hi && starts[at] < v));
    if (k == 0) return lo;
    const int64_t next_hi = lo + k * step;
    lo += (k - 1) * step + 1;
    hi = next_hi < hi ? next_hi : hi;
  }
  return lo;
}

// The share of the sequences that this cluster has.  With starts, rank 0 reads
// them and tells the others: the CTAs of a cluster loop over the same rows
// whatever becomes of the array meanwhile.
template <bool kRagged>
__device__ __forceinline__ Span span_of(const Plan& plan, const int32_t* starts, int64_t rows, int64_t sequences,
                                        int range, uint32_t rank, const Shared& sh) {
  if constexpr (!kRagged) {
    const int64_t s0 = sequences * range / plan.ranges, s1 = sequences * (range + 1) / plan.ranges;
    return Span{s0, s1, s0 * plan.length, s1 * plan.length};
  } else {
    const int lane = threadIdx.x & 31;
    if (rank == 0 && threadIdx.x < 32) {
      const int64_t s0 = range == 0 ? 0 : lower_bound(starts, sequences, rows * range / plan.ranges, lane);
      const int64_t s1 = range + 1 == plan.ranges ? sequences
                                                  : lower_bound(starts, sequences, rows * (range + 1) / plan.ranges, lane);
      const int64_t r0 = start_at(starts, s0, rows), r1 = start_at(starts, s1, rows);
      for (int i = lane; i < plan.cluster * 4; i += 32) {
        const int64_t v = i % 4 == 0 ? s0 : i % 4 == 1 ? s1 : i % 4 == 2 ? r0 : r1;
        if (plan.cluster > 1) store_peer(at_peer(reinterpret_cast<int64_t*>(sh.span) + i % 4, i / 4), v);
        else reinterpret_cast<int64_t*>(sh.span)[i] = v;
      }
    }
    if (plan.cluster > 1) cluster_sync();
    else __syncthreads();
    return *sh.span;
  }
}

// Which of a warp's rows start or end a sequence: a bit for each, and in lane j
// the sequence that row j starts (ends).
struct Marks {
  uint32_t start, end;
  int start_seq, end_seq;
};

template <typename T>
__device__ __forceinline__ Marks marks_equal(const Plan& plan, const Span& span, int64_t row, int lane) {
  const int64_t r = row + lane;
  const bool in = lane < Rows<T>::kS && r >= span.row && r < span.row_end;
  Marks m;
  m.start_seq = m.end_seq = in ? static_cast<int>(static_cast<uint32_t>(r) / static_cast<uint32_t>(plan.length)) : 0;
  m.start = __ballot_sync(0xffffffffu, in && r == m.start_seq * plan.length);
  m.end = __ballot_sync(0xffffffffu, in && r + 1 == (m.start_seq + 1) * plan.length);
  return m;
}

// With starts, for the rows [row, row + kChunk) of the CTA.  `next` moves along the
// sequences with the rows: starts before it (kBack: behind it) are of no use to
// these rows and those that are taken after them.  All threads call.
template <typename T, bool kBack>
__device__ __forceinline__ void mark_rows(const int32_t* starts, int64_t rows, const Span& span, int64_t row, int64_t& next,
                                          const Shared& sh) {
  constexpr int kChunk = Rows<T>::kChunk;
  const int64_t r0 = row > span.row ? row : span.row;
  const int64_t r1 = row + kChunk < span.row_end ? row + kChunk : span.row_end;
  for (int i = threadIdx.x; i < 2 * kChunk; i += kThreads) sh.first[i] = -1;       // first and last
  for (int done = kThreads; done == kThreads; next += kBack ? -done : done) {
    const int64_t i = kBack ? next - threadIdx.x : next + threadIdx.x;
    const bool there = i >= span.seq && i <= span.seq_end;
    const int64_t v = there ? start_at(starts, i, rows) : 0;
    done = __syncthreads_count(there && (kBack ? v > r1 : v < r0));
  }
  int64_t at = next;
  for (int within = kThreads; within == kThreads; at += kBack ? -kThreads : kThreads) {
    const int64_t i = kBack ? at - threadIdx.x : at + threadIdx.x;
    const bool there = i >= span.seq && i <= span.seq_end;
    const int64_t v = there ? start_at(starts, i, rows) : 0;
    if (there && r0 < r1) {
      if (i < span.seq_end && v >= r0 && v < r1 && start_at(starts, i + 1, rows) > v) sh.first[v - row] = static_cast<int>(i);
      if (i > span.seq && v > r0 && v <= r1 && start_at(starts, i - 1, rows) < v) sh.last[v - 1 - row] = static_cast<int>(i - 1);
    }
    within = __syncthreads_count(there && (kBack ? v >= r0 : v <= r1));
  }
}

template <typename T>
__device__ __forceinline__ Marks marks_of(const Shared& sh, int warp, int lane) {
  Marks m;
  const bool in = lane < Rows<T>::kS;
  m.start_seq = in ? sh.first[warp * Rows<T>::kS + lane] : -1;
  m.end_seq = in ? sh.last[warp * Rows<T>::kS + lane] : -1;
  m.start = __ballot_sync(0xffffffffu, m.start_seq >= 0);
  m.end = __ballot_sync(0xffffffffu, m.end_seq >= 0);
  return m;
}

// out[s] <- in[s] (zeros without in) for the span's sequences that have no row.
__device__ __forceinline__ void pass_empty(const int32_t* starts, const Span& span, float* out, const float* in,
                                           int64_t col, int64_t cols) {
  if (!out) return;
  for (int64_t s = span.seq + threadIdx.x; s < span.seq_end; s += kThreads)
    if (starts[s + 1] <= starts[s])
      for (int64_t c = col; c < col + kCols && c < cols; ++c) out[s * cols + c] = in ? in[s * cols + c] : 0.f;
}

// --------------------------------------------------------------- elements --

// Copies a warp's rows of one tensor to its place in shared memory, [kS][64], zeros
// where there is no row or column.
template <typename T, bool kVec>
__device__ __forceinline__ void fetch_rows(uint8_t* dst, const void* src, int64_t ld, int64_t row, const Span& span,
                                           int64_t col, int64_t cols, int lane) {
  constexpr int kS = Rows<T>::kS;
  const T* p = static_cast<const T*>(src);
  if constexpr (kVec) {
    constexpr int kPer = 16 / sizeof(T), kPieces = kCols / kPer;      // 16-byte pieces of a row
#pragma unroll
    for (int i = 0; i < kS * kPieces / 32; ++i) {
      const int k = i * 32 + lane;
      const int64_t r = row + k / kPieces, c = col + k % kPieces * kPer;
      const bool in = r >= span.row && r < span.row_end && c < cols;
      const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst)) + k * 16;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(p + (in ? r * ld + c : 0)),
                   "r"(in ? 16 : 0)
                   : "memory");
    }
  } else {
    T* to = reinterpret_cast<T*>(dst);
#pragma unroll 8
    for (int k = lane; k < kS * kCols; k += 32) {
      const int64_t r = row + k / kCols, c = col + k % kCols;
      const bool in = r >= span.row && r < span.row_end && c < cols;
      store_elem(to + k, in ? load_elem(p + r * ld + c) : 0.f);
    }
  }
}

// A lane's two columns of a row in shared memory: neighbours (kVec), or 32 apart.
template <typename T, bool kVec>
__device__ __forceinline__ void pair_at(const uint8_t* tile, int j, int lane, float (&v)[2]) {
  const T* row = reinterpret_cast<const T*>(tile) + j * kCols;
  if constexpr (!kVec) {
    v[0] = load_elem(row + lane);
    v[1] = load_elem(row + 32 + lane);
  } else if constexpr (sizeof(T) == 2) {
    const uint32_t u = reinterpret_cast<const uint32_t*>(row)[lane];
    v[0] = __uint_as_float(u << 16);
    v[1] = __uint_as_float(u & 0xffff0000u);
  } else {
    const float2 f = reinterpret_cast<const float2*>(row)[lane];
    v[0] = f.x;
    v[1] = f.y;
  }
}

template <bool kVec>
__device__ __forceinline__ int64_t column(int64_t col, int lane, int k) {
  return kVec ? col + 2 * lane + k : col + 32 * k + lane;
}

// Stores a lane's two columns; with kVec the number of columns is a multiple of 8.
template <typename T, bool kVec>
__device__ __forceinline__ void store_pair(T* row, int64_t col, int64_t cols, int lane, float a, float b) {
  if constexpr (kVec) {
    const int64_t c = column<true>(col, lane, 0);
    if (c < cols) {
      if constexpr (sizeof(T) == 2) *reinterpret_cast<uint32_t*>(row + c) = pack2(a, b);
      else *reinterpret_cast<float2*>(row + c) = make_float2(a, b);
    }
  } else {
    if (column<false>(col, lane, 0) < cols) store_elem(row + column<false>(col, lane, 0), a);
    if (column<false>(col, lane, 1) < cols) store_elem(row + column<false>(col, lane, 1), b);
  }
}

template <bool kVec>
__device__ __forceinline__ void load_state(const float* states, int64_t seq, int64_t col, int64_t cols, int lane,
                                           float (&v)[2]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t c = column<kVec>(col, lane, k);
    v[k] = states && c < cols ? states[seq * cols + c] : 0.f;
  }
}

// The state that a warp's rows begin with, and in `carry` the one behind the rows of
// the whole cluster: the pieces of the CTAs and warps in between, in order.
// kBack: rows, warps and CTAs are taken from the last to the first.  Pieces and
// inbox alternate between two places with the turns (`parity`): a thread writes
// to one again only after a barrier that all threads reach when they have
// read it.
template <bool kBack>
__device__ __forceinline__ void exchange(const Shared& sh, int parity, int cluster, uint32_t rank, int warp, int lane,
                                         const Piece (&mine)[2], float (&carry)[2], float (&state)[2]) {
  float4* pieces = sh.pieces + parity * kWarps * 32;
  pieces[warp * 32 + lane] = make_float4(mine[0].c, mine[0].b, mine[1].c, mine[1].b);
  __syncthreads();
  auto both = [](const float4& p, float (&h)[2]) {
    h[0] = through(Piece{p.x, p.y}, h[0]);
    h[1] = through(Piece{p.z, p.w}, h[1]);
  };
  state[0] = carry[0];
  state[1] = carry[1];
  if (cluster > 1) {
    float4* inbox = sh.inbox + parity * cluster * 32;
    if (warp < cluster) {                        // warp w tells CTA w of the cluster this CTA's piece
      Piece p[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        const float4 q = pieces[(kBack ? kWarps - 1 - i : i) * 32 + lane];
        p[0] = then(p[0], Piece{q.x, q.y});
        p[1] = then(p[1], Piece{q.z, q.w});
      }
      store_peer(at_peer(inbox + rank * 32 + lane, warp), make_float4(p[0].c, p[0].b, p[1].c, p[1].b));
    }
    cluster_sync();
    for (int i = 0; i < cluster; ++i) {
      const int q = kBack ? cluster - 1 - i : i;
      if (q == static_cast<int>(rank)) {
        state[0] = carry[0];
        state[1] = carry[1];
      }
      both(inbox[q * 32 + lane], carry);
    }
  }
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    const int w = kBack ? kWarps - 1 - i : i;
    if (kBack ? w > warp : w < warp) both(pieces[w * 32 + lane], state);
  }
  if (cluster == 1) {
#pragma unroll
    for (int i = 0; i < kWarps; ++i) both(pieces[(kBack ? kWarps - 1 - i : i) * 32 + lane], carry);
  }
}

// --------------------------------------------------------------- forward --

template <typename T, bool kVec, bool kRagged>
__global__ void __launch_bounds__(kThreads, 2)
recurrence_kernel(const __grid_constant__ opt_recurrence_args a, const __grid_constant__ Plan plan) {
  constexpr int kS = Rows<T>::kS, kChunk = Rows<T>::kChunk, kTile = Rows<T>::kTile;
  using L = Layout<T, 2>;
  extern __shared__ __align__(128) uint8_t smem[];
  let_next_start();
  wait_for_predecessors();
  const Shared sh = L::carve(smem, plan.cluster);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = plan.cluster > 1 ? cluster_rank() : 0;
  const int64_t id = blockIdx.x / plan.cluster, col = id % plan.groups * kCols;
  if (plan.cluster > 1) cluster_sync();          // every CTA of the cluster has begun
  const Span span = span_of<kRagged>(plan, a.starts, a.rows, a.sequences, static_cast<int>(id / plan.groups), rank, sh);
  if (kRagged && rank == 0) pass_empty(a.starts, span, a.hT, a.h0, col, a.cols);
  const int64_t base = span.row / kS * kS, step = static_cast<int64_t>(plan.cluster) * kChunk;
  const int64_t turns = span.row_end > span.row ? (span.row_end - base + step - 1) / step : 0;
  int64_t next = span.seq;
  auto row_of = [&](int64_t turn) { return base + turn * step + static_cast<int64_t>(rank) * kChunk; };
  auto stage = [&](int64_t turn) { return smem + (turn & 1) * L::kStage + warp * 2 * kTile; };
  auto fetch = [&](int64_t turn) {
    if (turn < turns) {
      const int64_t r = row_of(turn) + warp * kS;
      fetch_rows<T, kVec>(stage(turn), a.x, a.x_ld, r, span, col, a.cols, lane);
      fetch_rows<T, kVec>(stage(turn) + kTile, a.gate, a.gate_ld, r, span, col, a.cols, lane);
    }
    copy_commit();
  };
  fetch(0);
  float carry[2] = {0.f, 0.f};
  for (int64_t turn = 0; turn < turns; ++turn) {
    copy_wait<0>();
    __syncwarp();
    fetch(turn + 1);                             // over the rows of the turn before, which this warp is done with
    const int64_t row = row_of(turn) + warp * kS;
    Marks m;
    if constexpr (kRagged) {
      mark_rows<T, false>(a.starts, a.rows, span, row_of(turn), next, sh);
      m = marks_of<T>(sh, warp, lane);
    } else {
      m = marks_equal<T>(plan, span, row, lane);
    }
    const uint8_t *xs = stage(turn), *gs = xs + kTile;
    float c[kS][2];
    Piece mine[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
    for (int j = 0; j < kS; ++j) {
      float g[2], x[2];
      pair_at<T, kVec>(gs, j, lane, g);
      pair_at<T, kVec>(xs, j, lane, x);
      const bool in = row + j >= span.row && row + j < span.row_end;
      if (m.start >> j & 1) {
        float h0[2];
        load_state<kVec>(a.h0, __shfl_sync(0xffffffffu, m.start_seq, j), col, a.cols, lane, h0);
        mine[0].b = h0[0];
        mine[1].b = h0[1];
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        c[j][k] = in ? update_gate(g[k]) : 0.f;
        mine[k].b = fmaf(c[j][k], x[k] - mine[k].b, mine[k].b);
        mine[k].c = fmaf(c[j][k], 1.f - mine[k].c, mine[k].c);
      }
    }
    if (m.start) mine[0].c = mine[1].c = kReset;
    float h[2];
    exchange<false>(sh, static_cast<int>(turn & 1), plan.cluster, rank, warp, lane, mine, carry, h);
    if (a.states && row >= span.row && row < span.row_end)
      store_pair<float, kVec>(a.states + row / kS * a.cols, col, a.cols, lane, h[0], h[1]);
    T* y = static_cast<T*>(a.y) + row * a.y_ld;
#pragma unroll
    for (int j = 0; j < kS; ++j, y += a.y_ld) {
      float x[2];
      pair_at<T, kVec>(xs, j, lane, x);
      if (m.start >> j & 1) load_state<kVec>(a.h0, __shfl_sync(0xffffffffu, m.start_seq, j), col, a.cols, lane, h);
#pragma unroll
      for (int k = 0; k < 2; ++k) h[k] = fmaf(c[j][k], x[k] - h[k], h[k]);
      if (row + j >= span.row && row + j < span.row_end) store_pair<T, kVec>(y, col, a.cols, lane, h[0], h[1]);
      if ((m.end >> j & 1) && a.hT)
        store_pair<float, kVec>(a.hT + __shfl_sync(0xffffffffu, m.end_seq, j) * a.cols, col, a.cols, lane, h[0], h[1]);
    }
    __syncwarp();                                // the tile may be written over
  }
}

// One row to each sequence: nothing depends on another row.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) recurrence_step_kernel(const __grid_constant__ opt_recurrence_args a,
                                                                   int64_t slices) {
  constexpr int kN = kVec ? 8 : 1;
  let_next_start();
  wait_for_predecessors();
  const int64_t r = blockIdx.x / slices;
  const int64_t c = ((blockIdx.x - r * slices) * kThreads + threadIdx.x) * kN;
  if (c >= a.cols) return;
  float x[kN], g[kN], h[kN];
#pragma unroll
  for (int j = 0; j < kN; ++j) h[j] = 0.f;
  if constexpr (kVec) {
    load8(static_cast<const T*>(a.x) + r * a.x_ld + c, x);
    load8(static_cast<const T*>(a.gate) + r * a.gate_ld + c, g);
    if (a.h0) load8(a.h0 + r * a.cols + c, h);
  } else {
    x[0] = load_elem(static_cast<const T*>(a.x) + r * a.x_ld + c);
    g[0] = load_elem(static_cast<const T*>(a.gate) + r * a.gate_ld + c);
    if (a.h0) h[0] = a.h0[r * a.cols + c];
  }
#pragma unroll
  for (int j = 0; j < kN; ++j) h[j] = fmaf(update_gate(g[j]), x[j] - h[j], h[j]);
  if constexpr (kVec) {
    store8(static_cast<T*>(a.y) + r * a.y_ld + c, h);
    if (a.hT) store8(a.hT + r * a.cols + c, h);
  } else {
    store_elem(static_cast<T*>(a.y) + r * a.y_ld + c, h[0]);
    if (a.hT) a.hT[r * a.cols + c] = h[0];
  }
}

// -------------------------------------------------------------- gradient --

// From the last row to the first.  Each warp runs through its rows forward from
// the saved state for x_t - h_{t-1}, then backward.
template <typename T, bool kVec, bool kRagged>
__global__ void __launch_bounds__(kThreads, 2)
recurrence_grad_kernel(const __grid_constant__ opt_recurrence_grad_args a, const __grid_constant__ Plan plan) {
  constexpr int kS = Rows<T>::kS, kChunk = Rows<T>::kChunk, kTile = Rows<T>::kTile;
  using L = Layout<T, 3>;
  extern __shared__ __align__(128) uint8_t smem[];
  let_next_start();
  wait_for_predecessors();
  const Shared sh = L::carve(smem, plan.cluster);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = plan.cluster > 1 ? cluster_rank() : 0;
  const int64_t id = blockIdx.x / plan.cluster, col = id % plan.groups * kCols;
  if (plan.cluster > 1) cluster_sync();          // every CTA of the cluster has begun
  const Span span = span_of<kRagged>(plan, a.starts, a.rows, a.sequences, static_cast<int>(id / plan.groups), rank, sh);
  if (kRagged && rank == 0) pass_empty(a.starts, span, a.dh0, a.dhT, col, a.cols);
  const int64_t base = span.row / kS * kS, step = static_cast<int64_t>(plan.cluster) * kChunk;
  const int64_t turns = span.row_end > span.row ? (span.row_end - base + step - 1) / step : 0;
  int64_t next = span.seq_end;
  auto row_of = [&](int64_t turn) { return base + (turns - 1 - turn) * step + static_cast<int64_t>(rank) * kChunk; };
  auto stage = [&](int64_t turn) { return smem + (turn & 1) * L::kStage + warp * 3 * kTile; };
  auto fetch = [&](int64_t turn) {
    if (turn < turns) {
      const int64_t r = row_of(turn) + warp * kS;
      fetch_rows<T, kVec>(stage(turn), a.x, a.x_ld, r, span, col, a.cols, lane);
      fetch_rows<T, kVec>(stage(turn) + kTile, a.gate, a.gate_ld, r, span, col, a.cols, lane);
      fetch_rows<T, kVec>(stage(turn) + 2 * kTile, a.dy, a.dy_ld, r, span, col, a.cols, lane);
    }
    copy_commit();
  };
  fetch(0);
  float carry[2] = {0.f, 0.f};
  for (int64_t turn = 0; turn < turns; ++turn) {
    const int64_t row = row_of(turn) + warp * kS;
    float h[2];
    load_state<kVec>(row >= span.row && row < span.row_end ? a.states : nullptr, row / kS, col, a.cols, lane, h);
    copy_wait<0>();
    __syncwarp();
    fetch(turn + 1);                             // over the rows of the turn before, which this warp is done with
    Marks m;
    if constexpr (kRagged) {
      mark_rows<T, true>(a.starts, a.rows, span, row_of(turn), next, sh);
      m = marks_of<T>(sh, warp, lane);
    } else {
      m = marks_equal<T>(plan, span, row, lane);
    }
    const uint8_t *xs = stage(turn), *gs = xs + kTile, *ys = gs + kTile;
    float c[kS][2], d[kS][2];
#pragma unroll
    for (int j = 0; j < kS; ++j) {
      float g[2], x[2];
      pair_at<T, kVec>(gs, j, lane, g);
      pair_at<T, kVec>(xs, j, lane, x);
      const bool in = row + j >= span.row && row + j < span.row_end;
      if (m.start >> j & 1) load_state<kVec>(a.h0, __shfl_sync(0xffffffffu, m.start_seq, j), col, a.cols, lane, h);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        c[j][k] = in ? update_gate(g[k]) : 0.f;
        d[j][k] = x[k] - h[k];
        h[k] = fmaf(c[j][k], d[j][k], h[k]);
      }
    }
    Piece mine[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
    for (int j = kS - 1; j >= 0; --j) {
      float dy[2];
      pair_at<T, kVec>(ys, j, lane, dy);
      if (m.end >> j & 1) {
        float dhT[2];
        load_state<kVec>(a.dhT, __shfl_sync(0xffffffffu, m.end_seq, j), col, a.cols, lane, dhT);
        mine[0].b = dhT[0];
        mine[1].b = dhT[1];
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float l = dy[k] + mine[k].b;
        mine[k].b = (m.start >> j & 1) ? 0.f : fmaf(-c[j][k], l, l);
        mine[k].c = fmaf(c[j][k], 1.f - mine[k].c, mine[k].c);
      }
    }
    if (m.start | m.end) mine[0].c = mine[1].c = kReset;
    float b[2];                                  // (1 - c) l of the row behind
    exchange<true>(sh, static_cast<int>(turn & 1), plan.cluster, rank, warp, lane, mine, carry, b);
    T* dx = static_cast<T*>(a.dx) + (row + kS - 1) * a.dx_ld;
    T* dg = static_cast<T*>(a.dgate) + (row + kS - 1) * a.dgate_ld;
#pragma unroll
    for (int j = kS - 1; j >= 0; --j, dx -= a.dx_ld, dg -= a.dgate_ld) {
      float dy[2], g[2], ox[2], og[2];
      pair_at<T, kVec>(ys, j, lane, dy);
      pair_at<T, kVec>(gs, j, lane, g);
      if (m.end >> j & 1) load_state<kVec>(a.dhT, __shfl_sync(0xffffffffu, m.end_seq, j), col, a.cols, lane, b);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float l = dy[k] + b[k];
        ox[k] = c[j][k] * l;
        og[k] = ox[k] * one_minus(c[j][k], g[k]) * d[j][k];
        b[k] = fmaf(-c[j][k], l, l);
      }
      if (row + j >= span.row && row + j < span.row_end) {
        store_pair<T, kVec>(dx, col, a.cols, lane, ox[0], ox[1]);
        store_pair<T, kVec>(dg, col, a.cols, lane, og[0], og[1]);
      }
      if (m.start >> j & 1) {
        if (a.dh0)
          store_pair<float, kVec>(a.dh0 + __shfl_sync(0xffffffffu, m.start_seq, j) * a.cols, col, a.cols, lane, b[0], b[1]);
        b[0] = b[1] = 0.f;
      }
    }
    __syncwarp();                                // the tile may be written over
  }
}

// ---------------------------------------------------------------- launch --

bool rows_on(const void* p, int64_t ld, int es, int64_t rows, uintptr_t bytes) {
  return !p || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && (rows <= 1 || static_cast<uintptr_t>(ld) * es % bytes == 0));
}

// How many CTAs share the rows of a sequence (a cluster) and how many shares the
// sequences make, so that two CTAs of 64 columns to an SM have as few turns as
// possible.  A share of ragged sequences is taken to be longer than the others by
// an average sequence.
Plan make_plan(int64_t rows, int64_t cols, int64_t sequences, bool ragged, int chunk) {
  Plan best{1, 1, static_cast<int>((cols + kCols - 1) / kCols), ragged ? 0 : rows / sequences};
  const int64_t target = 2 * num_sms(), average = (rows + sequences - 1) / sequences;
  double least = 0;
  for (int cluster = 1; cluster <= kMaxCluster; cluster *= 2) {
    int64_t ranges = target / (static_cast<int64_t>(best.groups) * cluster);
    if (ranges < 1) {
      if (cluster > 1) break;
      ranges = 1;
    }
    if (ranges > sequences) ranges = sequences;
    const int64_t most = ranges == 1 ? rows
                         : ragged    ? rows / ranges + average
                                     : (sequences + ranges - 1) / ranges * average;
    const int64_t turns = (most + cluster * chunk - 1) / (static_cast<int64_t>(cluster) * chunk);
    const int64_t waves = (ranges * best.groups * cluster + target - 1) / target;
    const double cost = static_cast<double>(turns * waves) * (cluster > 1 ? 1.25 : 1.0);
    if (cluster == 1 || cost < least) {
      least = cost;
      best.cluster = cluster;
      best.ranges = static_cast<int>(ranges);
    }
  }
  return best;
}

template <typename Kernel, typename Args>
cudaError_t launch_plan(Kernel kernel, const Args& a, const Plan& plan, size_t smem, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int64_t ctas = static_cast<int64_t>(plan.cluster) * plan.groups * plan.ranges;
  return launch_overlapped(kernel, dim3(static_cast<unsigned>(ctas)), kThreads, smem, stream, plan.cluster, a, plan);
}

template <typename T, bool kVec>
cudaError_t forward(const opt_recurrence_args& a, cudaStream_t stream) {
  if (!a.starts && a.rows == a.sequences) {
    const int64_t per_cta = kThreads * (kVec ? 8 : 1), slices = (a.cols + per_cta - 1) / per_cta;
    return launch_overlapped(recurrence_step_kernel<T, kVec>, dim3(static_cast<unsigned>(a.rows * slices)), kThreads, 0, stream,
                             0, a, slices);
  }
  const Plan plan = make_plan(a.rows, a.cols, a.sequences, a.starts != nullptr, Rows<T>::kChunk);
  const size_t smem = Layout<T, 2>::bytes(plan.cluster);
  return a.starts ? launch_plan(recurrence_kernel<T, kVec, true>, a, plan, smem, stream)
                  : launch_plan(recurrence_kernel<T, kVec, false>, a, plan, smem, stream);
}

template <typename T, bool kVec>
cudaError_t backward(const opt_recurrence_grad_args& a, cudaStream_t stream) {
  const Plan plan = make_plan(a.rows, a.cols, a.sequences, a.starts != nullptr, Rows<T>::kChunk);
  const size_t smem = Layout<T, 3>::bytes(plan.cluster);
  return a.starts ? launch_plan(recurrence_grad_kernel<T, kVec, true>, a, plan, smem, stream)
                  : launch_plan(recurrence_grad_kernel<T, kVec, false>, a, plan, smem, stream);
}

}  // namespace

cudaError_t launch_recurrence(const opt_recurrence_args& a, cudaStream_t stream) {
  const int es = a.dtype == kBf16 ? 2 : 4;
  const bool vec = a.cols % 8 == 0 && rows_on(a.x, a.x_ld, es, a.rows, 16) && rows_on(a.gate, a.gate_ld, es, a.rows, 16) &&
                   rows_on(a.y, a.y_ld, es, a.rows, 16) && rows_on(a.h0, a.cols, 4, 1, 16) &&
                   rows_on(a.hT, a.cols, 4, 1, 16) && rows_on(a.states, a.cols, 4, 1, 8);
  if (a.dtype == kBf16) return vec ? forward<__nv_bfloat16, true>(a, stream) : forward<__nv_bfloat16, false>(a, stream);
  return vec ? forward<float, true>(a, stream) : forward<float, false>(a, stream);
}

cudaError_t launch_recurrence_grad(const opt_recurrence_grad_args& a, cudaStream_t stream) {
  const int es = a.dtype == kBf16 ? 2 : 4;
  const bool vec = a.cols % 8 == 0 && rows_on(a.dy, a.dy_ld, es, a.rows, 16) && rows_on(a.x, a.x_ld, es, a.rows, 16) &&
                   rows_on(a.gate, a.gate_ld, es, a.rows, 16) && rows_on(a.dx, a.dx_ld, es, a.rows, 16) &&
                   rows_on(a.dgate, a.dgate_ld, es, a.rows, 16) && rows_on(a.dh0, a.cols, 4, 1, 8);
  if (a.dtype == kBf16) return vec ? backward<__nv_bfloat16, true>(a, stream) : backward<__nv_bfloat16, false>(a, stream);
  return vec ? backward<float, true>(a, stream) : backward<float, false>(a, stream);
}

}  // namespace mpopt
