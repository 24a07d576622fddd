// Gated recurrence along the rows of packed sequences, and its gradient (sm_103a):
//
//   h_t = h_{t-1} + c_t (x_t - h_{t-1}),  c = 1 / (1 + exp(-gate))
//   l_t = dy_t + (1 - c_{t+1}) l_{t+1};  dx_t = c_t l_t
//   dgate_t = c_t (1 - c_t) l_t (x_t - h_{t-1})
//
// Rows t1 .. t2 take a state h to  P h + B, where B is their result from h = 0 and P
// the product of their 1 - c; the gradient passes them the same way backwards.
// Two such pieces, the first (P1, B1) and behind it (P2, B2), make
//   P = P1 P2,  B = B2 + P2 B1
// Both c and 1 - c are taken from the smaller of them, which keeps its digits however
// far the gate is open or closed: (1 - c) v is v - c v where c < 1/2, one rounding
// of v, and the product with 1 - c beyond.  A piece in which a
// sequence starts or ends does not depend on the state before it: P = kReset,
// and B is selected, not multiplied, so that an infinity or a NaN stays in its
// own sequence.
//
// A warp has 64 columns, two to a lane (or 128, four), and 8 rows at a time in shared
// memory, fetched with cp.async while it works on the rows before.  The pieces of
// its CTA's eight or 16 warps, and those of the CTAs of a cluster, which take the
// next rows each, are joined through (distributed) shared memory; then every
// thread applies the pieces up to each of its rows to the right state (the gradient,
// whose registers do not hold them, runs through its rows again; that way the
// forward pass takes 12 % longer).  x and gate are read once (and dy), the outputs
// written once: HBM's floor is 60 us for 16384 x 4096 in bf16, 50 for the gradient of
// 8192 x 4096.  They take 99 and 103: a turn of 512 (384) rows is a chain of the
// pieces, their join, the mail and the outputs, 3.1 (4.7) us, with 27 (59)
// instructions an element.  A state for every 8 rows in fp32 is all that the gradient
// needs of the forward pass.

#include <climits>

#include "cluster.cuh"
#include "elements.cuh"
#include "internal.h"
#include "overlap.cuh"

namespace mpopt {
namespace {

constexpr int kStepThreads = 256;
constexpr int kMaxCluster = kMostClusterCtas;
constexpr int kS = kRecurrenceStateRows;         // rows of a thread at a time
constexpr float kReset = -1.f;                   // a product of 1 - c is not below 0
__device__ __forceinline__ bool is_reset(float p) { return p < -0.5f; }

// ---------------------------------------------------------------- pieces --

struct Piece {
  float p, b;
};
__device__ __forceinline__ Piece then(Piece first, Piece second) {
  if (is_reset(second.p)) return second;
  return Piece{is_reset(first.p) ? kReset : first.p * second.p, fmaf(second.p, first.b, second.b)};
}
__device__ __forceinline__ float through(Piece q, float h) { return is_reset(q.p) ? q.b : fmaf(q.p, h, q.b); }

// A row's gate: w = c where gate < 0, and -(1 - c), with its sign bit even where that is
// 0, where the gate is open.  |w| = e / (1 + e), e = exp(-|gate|), from two approximate
// instructions of 2 units each; the rounding of gate log2 e adds 2^-24 |gate| of the
// value.  0 beyond |gate| = 87.  From c alone 1 - c would be off by 2^-24 of 1, that is 1 %
// of itself at a gate of 12 and all of it from 17 on; the selects that this takes cost
// the forward pass 7 % (16384 x 4096: 99 us for 92) and the gradient 11 % (8192 x 4096
// packed: 103 for 91 to 94).
__device__ __forceinline__ float gate_of(float g) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * fabsf(g)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return __uint_as_float(__float_as_uint(e * r) | (~__float_as_uint(g) & 0x80000000u));
}
__device__ __forceinline__ bool is_open(float w) { return __float_as_int(w) < 0; }
// h + c (x - h)
__device__ __forceinline__ float advance(float w, float x, float h) { return fmaf(w, x - h, is_open(w) ? x : h); }
// (1 - c) v
__device__ __forceinline__ float keep(float w, float v) { return fmaf(-w, v, is_open(w) ? 0.f : v); }
// c v and (1 - c) v: the smaller is a product, the other what it leaves of v.
struct Parts {
  float taken, kept;
};
__device__ __forceinline__ Parts parts_of(float w, float v) {
  const float small = fabsf(w) * v, large = v - small;
  return is_open(w) ? Parts{large, small} : Parts{small, large};
}

// Two columns' pieces with one row more, advance() and keep() by packed instructions
// (one column at a time 16384 x 4096 takes 4 % longer; with the gates packed too, 20 %:
// more registers than there are).
__device__ __forceinline__ void add_row(float wa, float wb, float xa, float xb, Piece& a, Piece& b) {
  const float2 n = make_float2(-wa, -wb), d = make_float2(a.b - xa, b.b - xb), p = make_float2(a.p, b.p);
  const float2 h = __ffma2_rn(n, d, make_float2(is_open(wa) ? xa : a.b, is_open(wb) ? xb : b.b));
  const float2 q = __ffma2_rn(n, p, make_float2(is_open(wa) ? 0.f : p.x, is_open(wb) ? 0.f : p.y));
  a = Piece{q.x, h.x};
  b = Piece{q.y, h.y};
}

// ----------------------------------------------------------------- layout --

// kC columns to a lane, 32 kC to a CTA.
template <typename T, int kC>
constexpr int kTile = kS * 32 * kC * static_cast<int>(sizeof(T));   // bytes of a warp's rows of one tensor

// CTAs to an SM, by registers and shared memory.
template <typename T, int kC, int kW>
constexpr int kForwardCtas = kW == 16 ? (sizeof(T) == 2 ? 2 : 1) : kC == 4 ? 2 : sizeof(T) == 2 ? 4 : 3;
template <int kW>
constexpr int kBackwardCtas = kW == 16 ? 1 : 3;

struct Plan {
  int cluster, ranges, groups;      // CTAs to a cluster; shares of the sequences; shares of the columns
  int length;                       // rows of a sequence without starts
};

// The sequences and rows of a cluster; both are at most 2^30.
struct Span {
  int seq, seq_end, row, row_end;
};

struct Shared {
  float2* pieces;        // [2][kWarps][kCols]: (p, b) of a warp's rows; then of all warps' before it
  float2* inbox;         // [2][cluster][kCols]: of a CTA's rows
  float* state;          // [2][kCols]: before the CTA's rows
  int* first;            // [kChunk] with starts: the sequence that a row starts (set where one does)
  int* last;             // [kChunk]              the sequence that a row ends
  Span* span;
  Mailbox mail;
};

template <typename T, int kC, int kW, int kTensors>
struct Layout {
  static constexpr int kCols = 32 * kC, kWarps = kW, kThreads = 32 * kW, kChunk = kW * kS;
  static constexpr int kStage = kTensors * kTile<T, kC> * kWarps;
  static size_t bytes(int cluster) {
    return 2 * kStage + (2 * kWarps * 8 + (cluster > 1 ? 2 * cluster * 8 : 0) + 2 * 4) * kCols + 2 * kChunk * 4 + sizeof(Span) + 16;
  }
  static __device__ __forceinline__ Shared carve(uint8_t* base, int cluster) {
    Shared s;
    base += 2 * kStage;
    s.pieces = reinterpret_cast<float2*>(base);
    s.inbox = s.pieces + 2 * kWarps * kCols;
    s.state = reinterpret_cast<float*>(s.inbox + (cluster > 1 ? 2 * cluster * kCols : 0));
    s.first = reinterpret_cast<int*>(s.state + 2 * kCols);
    s.last = s.first + kChunk;
    s.span = reinterpret_cast<Span*>(s.last + kChunk);
    s.mail.bar = reinterpret_cast<uint64_t*>(s.span + 1);
    return s;
  }
};

// -------------------------------------------------------------- sequences --

__device__ __forceinline__ int start_at(const int32_t* starts, int i, int rows) {
  const int v = starts[i];
  return v < 0 ? 0 : v > rows ? rows : v;
}

// First index in [0, n] whose start is not below v (n: none), by one warp: 32 probes a step.
__device__ __forceinline__ int lower_bound(const int32_t* starts, int n, int v, int lane) {
  int lo = 0, hi = n;                            // starts before lo are below v, those from hi on are not
  while (hi > lo) {
    const int step = (hi - lo + 31) / 32;
    const int64_t at = lo + static_cast<int64_t>(lane) * step;
    const int k = __popc(__ballot_sync(0xffffffffu, at < hi && starts[at] < v));
    if (k == 0) return lo;
    const int64_t next_hi = lo + static_cast<int64_t>(k) * step;
    lo += (k - 1) * step + 1;
    hi = next_hi < hi ? static_cast<int>(next_hi) : hi;
  }
  return lo;
}

__device__ __forceinline__ int share(int64_t n, int part, int parts) { return static_cast<int>(n * part / parts); }

// The share of the sequences that this cluster has.  With starts, rank 0 reads
// them and tells the others: the CTAs of a cluster loop over the same rows
// whatever becomes of the array meanwhile.
template <bool kRagged>
__device__ __forceinline__ Span span_of(const Plan& plan, const int32_t* starts, int rows, int sequences, int range,
                                        uint32_t rank, const Shared& sh) {
  if constexpr (!kRagged) {
    const int s0 = share(sequences, range, plan.ranges), s1 = share(sequences, range + 1, plan.ranges);
    return Span{s0, s1, s0 * plan.length, s1 * plan.length};
  } else {
    const int lane = threadIdx.x & 31;
    if (rank == 0 && threadIdx.x < 32) {
      const int s0 = range == 0 ? 0 : lower_bound(starts, sequences, share(rows, range, plan.ranges), lane);
      const int s1 = range + 1 == plan.ranges ? sequences : lower_bound(starts, sequences, share(rows, range + 1, plan.ranges), lane);
      const int r0 = start_at(starts, s0, rows), r1 = start_at(starts, s1, rows);
      for (int i = lane; i < plan.cluster * 4; i += 32) {
        const int v = i % 4 == 0 ? s0 : i % 4 == 1 ? s1 : i % 4 == 2 ? r0 : r1;
        if (plan.cluster > 1) store_peer(at_peer(reinterpret_cast<int*>(sh.span) + i % 4, i / 4), static_cast<uint32_t>(v));
        else reinterpret_cast<int*>(sh.span)[i] = v;
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

// How far a warp's rows have come along the starts: `near` is the first start from
// its rows on (kBack: the last one before the rows it has looked at), so that
// most groups of rows are known to have no mark by one comparison; `next`, with
// starts, the first sequence that does not start before the rows.
struct Cursor {
  int near, next;
};
template <bool kBack>
__device__ __forceinline__ Cursor first_cursor(const Span& span) {
  return kBack ? Cursor{span.row_end, span.seq_end + 1} : Cursor{span.row, span.seq};
}

// Sequences of one length.
template <bool kBack>
__device__ __forceinline__ Marks marks_equal(const Plan& plan, const Span& span, int row, Cursor& at, int lane) {
  Marks m{0, 0, 0, 0};
  if (row >= span.row_end) return m;
  if (kBack ? at.near > row + kS : at.near < row) {
    const uint32_t len = static_cast<uint32_t>(plan.length);
    at.near = static_cast<int>(static_cast<uint32_t>(kBack ? row + kS : row + plan.length - 1) / len * len);
  }
  if (kBack ? at.near < row : at.near > row + kS) return m;
  const int r = row + lane;
  const bool in = lane < kS && r >= span.row && r < span.row_end;
  const int seq = in ? r / plan.length : 0, rest = r - seq * plan.length;
  m.start_seq = m.end_seq = seq;
  m.start = __ballot_sync(0xffffffffu, in && rest == 0);
  m.end = __ballot_sync(0xffffffffu, in && rest == plan.length - 1);
  return m;
}

// With starts; the span's end counts as one.
template <bool kBack>
__device__ __forceinline__ Marks marks_ragged(const int32_t* starts, int rows, const Span& span, int row, Cursor& at,
                                              const Shared& sh, int warp, int lane) {
  const int r0 = row > span.row ? row : span.row, r1 = row + kS < span.row_end ? row + kS : span.row_end;
  Marks m{0, 0, -1, -1};
  if (r0 >= r1 || (kBack ? at.near < row : at.near > row + kS)) return m;
  for (int n = 32; n == 32;) {
    const int i = kBack ? at.next - 1 - lane : at.next + lane;
    const bool there = i >= span.seq && i <= span.seq_end;
    const int v = there ? start_at(starts, i, rows) : 0;
    n = __popc(__ballot_sync(0xffffffffu, there && (kBack ? v >= r0 : v < r0)));
    at.next += kBack ? -n : n;
  }
  if (kBack) at.near = at.next > span.seq ? start_at(starts, at.next - 1, rows) : -1;
  else at.near = at.next <= span.seq_end ? start_at(starts, at.next, rows) : INT_MAX;
  int *first = sh.first + warp * kS, *last = sh.last + warp * kS;
  uint32_t start = 0, end = 0;
  for (int64_t base = at.next;; base += 32) {
    const int64_t i = base + lane;
    const int v = i <= span.seq_end ? start_at(starts, static_cast<int>(i), rows) : INT_MAX;
    const uint32_t here = __ballot_sync(0xffffffffu, v <= r1);
    if (here >> lane & 1) {
      if (i < span.seq_end && v >= r0 && v < r1 && start_at(starts, static_cast<int>(i + 1), rows) > v) {
        first[v - row] = static_cast<int>(i);
        start |= 1u << (v - row);
      }
      if (i > span.seq && v > r0 && start_at(starts, static_cast<int>(i - 1), rows) < v) {
        last[v - 1 - row] = static_cast<int>(i - 1);
        end |= 1u << (v - 1 - row);
      }
    }
    if (here != 0xffffffffu) break;
  }
  m.start = __reduce_or_sync(0xffffffffu, start);
  m.end = __reduce_or_sync(0xffffffffu, end);
  if (m.start | m.end) {
    __syncwarp();
    if (m.start >> lane & 1) m.start_seq = first[lane];
    if (m.end >> lane & 1) m.end_seq = last[lane];
    __syncwarp();
  }
  return m;
}

// out[s] <- in[s] (zeros without in) for the span's sequences that have no row.
template <int kCols>
__device__ __forceinline__ void pass_empty(const int32_t* starts, const Span& span, float* out, const float* in,
                                           int col, int cols) {
  if (!out) return;
  for (int s = span.seq + static_cast<int>(threadIdx.x); s < span.seq_end; s += static_cast<int>(blockDim.x))
    if (starts[s + 1] <= starts[s])
      for (int64_t c = static_cast<int64_t>(s) * cols + col, n = min(kCols, cols - col); n > 0; ++c, --n) out[c] = in ? in[c] : 0.f;
}

// --------------------------------------------------------------- elements --

// Copies a warp's rows of one tensor to its place in shared memory, [kS][kCols], zeros
// where there is no row or column.  `whole`: they are all there.
template <typename T, int kC, bool kVec>
__device__ __forceinline__ void fetch_rows(uint8_t* dst, const void* src, int64_t ld, int row, const Span& span,
                                           int col, int cols, int lane, bool whole) {
  constexpr int kCols = 32 * kC;
  const T* p = static_cast<const T*>(src);
  if constexpr (kVec) {
    constexpr int kPer = 16 / sizeof(T), kPieces = kCols / kPer, kStep = 32 / kPieces;   // 16-byte pieces of a row, rows a step
    static_assert(kPieces <= 32, "a step takes whole rows");
    const int r0 = row + lane / kPieces, c = col + lane % kPieces * kPer;
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst)) + lane * 16;
    if (whole) {
      const T* q = p + r0 * ld + c;
#pragma unroll
      for (int i = 0; i < kS / kStep; ++i, q += kStep * ld)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * 512), "l"(q) : "memory");
    } else {
#pragma unroll
      for (int i = 0; i < kS / kStep; ++i) {
        const int r = r0 + i * kStep;
        const bool in = r >= span.row && r < span.row_end && c < cols;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + i * 512), "l"(p + (in ? r * ld + c : 0)),
                     "r"(in ? 16 : 0)
                     : "memory");
      }
    }
  } else {
    T* to = reinterpret_cast<T*>(dst);
#pragma unroll
    for (int k = 0; k < kC; ++k) {
      const int c = col + k * 32 + lane;
#pragma unroll
      for (int j = 0; j < kS; ++j) {
        const bool in = whole || (row + j >= span.row && row + j < span.row_end && c < cols);
        const T* q = p + (in ? static_cast<int64_t>(row + j) * ld + c : 0);
        T* at = to + j * kCols + k * 32 + lane;
        if constexpr (sizeof(T) == 4)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(at))),
                       "l"(q), "r"(in ? 4 : 0)
                       : "memory");
        else
          store_elem(at, in ? load_elem(q) : 0.f);
      }
    }
  }
}

// A lane's columns of a row in shared memory: neighbours (kVec), or 32 apart.
template <typename T, int kC, bool kVec>
__device__ __forceinline__ void columns_at(const uint8_t* tile, int j, int lane, float (&v)[kC]) {
  const T* row = reinterpret_cast<const T*>(tile) + j * 32 * kC;
  if constexpr (!kVec) {
#pragma unroll
    for (int k = 0; k < kC; ++k) v[k] = load_elem(row + 32 * k + lane);
  } else if constexpr (sizeof(T) == 2) {
    uint32_t u[kC / 2];
    if constexpr (kC == 2) {
      u[0] = reinterpret_cast<const uint32_t*>(row)[lane];
    } else {
      const uint2 w = reinterpret_cast<const uint2*>(row)[lane];
      u[0] = w.x, u[1] = w.y;
    }
#pragma unroll
    for (int k = 0; k < kC; ++k) v[k] = __uint_as_float(k & 1 ? u[k / 2] & 0xffff0000u : u[k / 2] << 16);
  } else if constexpr (kC == 2) {
    const float2 f = reinterpret_cast<const float2*>(row)[lane];
    v[0] = f.x, v[1] = f.y;
  } else {
    const float4 f = reinterpret_cast<const float4*>(row)[lane];
    v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
  }
}

template <int kC, bool kVec>
__device__ __forceinline__ int column(int lane, int k) {
  return kVec ? kC * lane + k : 32 * k + lane;
}

// Stores a lane's columns; with kVec the number of columns is a multiple of 8.
template <typename T, int kC, bool kVec>
__device__ __forceinline__ void store_columns(T* row, int col, int cols, int lane, const float (&v)[kC]) {
  if constexpr (kVec) {
    const int c = col + kC * lane;
    if (c >= cols) return;
    if constexpr (sizeof(T) == 2) {
      if constexpr (kC == 2) *reinterpret_cast<uint32_t*>(row + c) = pack2(v[0], v[1]);
      else *reinterpret_cast<uint2*>(row + c) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
    } else {
      if constexpr (kC == 2) *reinterpret_cast<float2*>(row + c) = make_float2(v[0], v[1]);
      else *reinterpret_cast<float4*>(row + c) = make_float4(v[0], v[1], v[2], v[3]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < kC; ++k)
      if (col + column<kC, false>(lane, k) < cols) store_elem(row + col + column<kC, false>(lane, k), v[k]);
  }
}

template <int kC, bool kVec>
__device__ __forceinline__ void load_state(const float* states, int seq, int col, int cols, int lane,
                                           float (&v)[kC]) {
  const float* from = states + static_cast<int64_t>(seq) * cols;
#pragma unroll
  for (int k = 0; k < kC; ++k) {
    const int c = col + column<kC, kVec>(lane, k);
    v[k] = states && c < cols ? from[c] : 0.f;
  }
}

// The state that a warp's rows begin with.  The first kCols threads of a CTA have a
// column each: they join the warps' pieces to what stands before every warp, tell
// the CTAs of the cluster the whole of it, and keep in `carry` the state behind
// all their rows.  kBack: rows, warps and CTAs are taken from the last to the
// first.  The places alternate with the turns: a thread writes to one again only
// after a barrier, or a message from every CTA, that comes when it has been read.
// From a message that does not come on, `carry` is NaN.
template <int kC, int kW, bool kVec, bool kBack>
__device__ __forceinline__ void exchange(const Shared& sh, int turn, int cluster, uint32_t rank, int warp, int lane,
                                         const Piece (&mine)[kC], float& carry, int& lost_at, float (&state)[kC]) {
  constexpr int kCols = 32 * kC, kWarps = kW;
  const int parity = turn & 1;
  float2* pieces = sh.pieces + parity * kWarps * kCols;
  float* before = sh.state + parity * kCols;
#pragma unroll
  for (int k = 0; k < kC; ++k) pieces[warp * kCols + column<kC, kVec>(lane, k)] = make_float2(mine[k].p, mine[k].b);
  __syncthreads();
  const int c = threadIdx.x;
  Piece all{1.f, 0.f};
  if (c < kCols) {
    float2 q[kWarps];
#pragma unroll
    for (int i = 0; i < kWarps; ++i) q[i] = pieces[i * kCols + c];
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const int w = kBack ? kWarps - 1 - i : i;
      pieces[w * kCols + c] = make_float2(all.p, all.b);
      all = then(all, Piece{q[w].x, q[w].y});
    }
    if (cluster == 1) {
      before[c] = carry;
      carry = through(all, carry);
    } else {
      float2* inbox = sh.inbox + parity * cluster * kCols;
      const bool there = exchange_message(sh.mail, turn, c == 0, static_cast<uint32_t>(cluster) * kCols * 8, lost_at, [&] {
        for (int i = 0; i < cluster; ++i) sh.mail.send(turn, inbox + rank * kCols + c, i, make_float2(all.p, all.b));
      });
      if (!there) carry = __uint_as_float(0x7fc00000u);
      for (int i = 0; i < cluster; ++i) {
        const int w = kBack ? cluster - 1 - i : i;
        if (w == static_cast<int>(rank)) before[c] = carry;
        const float2 q = inbox[w * kCols + c];
        carry = there ? through(Piece{q.x, q.y}, carry) : carry;
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kC; ++k) {
    const int at = column<kC, kVec>(lane, k);
    const float2 q = pieces[warp * kCols + at];
    state[k] = through(Piece{q.x, q.y}, before[at]);
  }
}

// --------------------------------------------------------------- forward --

template <bool kValue>
struct Flag {
  static constexpr bool value = kValue;
};

template <typename T, int kC, int kW, bool kVec, bool kRagged>
__global__ void __launch_bounds__(32 * kW, (kForwardCtas<T, kC, kW>))
recurrence_kernel(const __grid_constant__ opt_recurrence_args a, const __grid_constant__ Plan plan) {
  constexpr int kCols = 32 * kC;
  using L = Layout<T, kC, kW, 2>;
  extern __shared__ __align__(128) uint8_t smem[];
  let_next_start();
  wait_for_predecessors();
  const Shared sh = L::carve(smem, plan.cluster);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = plan.cluster > 1 ? cluster_rank() : 0;
  const int id = blockIdx.x / plan.cluster;
  const int rows = static_cast<int>(a.rows), cols = static_cast<int>(a.cols), col = id % plan.groups * kCols;
  if (plan.cluster > 1) {                        // every CTA of the cluster has begun
    if (threadIdx.x == 0) sh.mail.init();
    cluster_sync();
  }
  const Span span = span_of<kRagged>(plan, a.starts, rows, static_cast<int>(a.sequences), id / plan.groups, rank, sh);
  if (kRagged && rank == 0) pass_empty<kCols>(a.starts, span, a.hT, a.h0, col, cols);
  const int base = span.row / kS * kS, step = plan.cluster * L::kChunk;
  const int turns = span.row_end > span.row ? (span.row_end - base + step - 1) / step : 0;
  int row = base + (static_cast<int>(rank) * kW + warp) * kS;
  Cursor at = first_cursor<false>(span);
  auto stage = [&](int turn) { return smem + (turn & 1) * L::kStage + warp * 2 * kTile<T, kC>; };
  auto fetch = [&](int r, int turn) {
    if (r < span.row_end) {
      const bool whole = r >= span.row && r + kS <= span.row_end && col + kCols <= cols;
      fetch_rows<T, kC, kVec>(stage(turn), a.x, a.x_ld, r, span, col, cols, lane, whole);
      fetch_rows<T, kC, kVec>(stage(turn) + kTile<T, kC>, a.gate, a.gate_ld, r, span, col, cols, lane, whole);
    }
    copy_commit();
  };
  fetch(row, 0);
  float carry = 0.f;                             // the first kCols threads: behind all rows so far
  int lost_at = kNoneLost;                       // a message of the cluster's
  for (int turn = 0; turn < turns; ++turn, row += step) {
    copy_wait<0>();
    __syncwarp();
    fetch(row + step, turn + 1);                 // over the rows of the turn before, which this warp is done with
    Marks m;
    if constexpr (kRagged) m = marks_ragged<false>(a.starts, rows, span, row, at, sh, warp, lane);
    else m = marks_equal<false>(plan, span, row, at, lane);
    const uint8_t *xs = stage(turn), *gs = xs + kTile<T, kC>;
    Piece upto[kS][kC], mine[kC];                // of the rows up to each, of all
#pragma unroll
    for (int k = 0; k < kC; ++k) mine[k] = Piece{1.f, 0.f};
    auto pieces = [&](auto plain) {              // plain: all rows are there, no sequence starts or ends
#pragma unroll
      for (int j = 0; j < kS; ++j) {
        float g[kC], x[kC];
        columns_at<T, kC, kVec>(gs, j, lane, g);
        columns_at<T, kC, kVec>(xs, j, lane, x);
        const bool in = plain.value || (row + j >= span.row && row + j < span.row_end);
        if (!plain.value && (m.start >> j & 1)) {
          float h0[kC];
          load_state<kC, kVec>(a.h0, __shfl_sync(0xffffffffu, m.start_seq, j), col, cols, lane, h0);
#pragma unroll
          for (int k = 0; k < kC; ++k) mine[k].b = h0[k];
        }
#pragma unroll
        for (int k = 0; k < kC; k += 2) {
          // a row that is not there leaves both alone, whatever lies in its place
          if (in) add_row(gate_of(g[k]), gate_of(g[k + 1]), x[k], x[k + 1], mine[k], mine[k + 1]);
          upto[j][k] = mine[k];
          upto[j][k + 1] = mine[k + 1];
        }
      }
      if (!plain.value && m.start) {
#pragma unroll
        for (int k = 0; k < kC; ++k) mine[k].p = kReset;
      }
    };
    const bool plain = row >= span.row && row + kS <= span.row_end && (m.start | m.end) == 0;
    if (plain) pieces(Flag<true>{});
    else pieces(Flag<false>{});
    float h[kC];
    exchange<kC, kW, kVec, false>(sh, turn, plan.cluster, rank, warp, lane, mine, carry, lost_at, h);
    if (a.states && row >= span.row && row < span.row_end)
      store_columns<float, kC, kVec>(a.states + static_cast<int64_t>(row / kS) * cols, col, cols, lane, h);
    T* y = static_cast<T*>(a.y) + static_cast<int64_t>(row) * a.y_ld;
    auto outputs = [&](auto plain) {
#pragma unroll
      for (int j = 0; j < kS; ++j, y += a.y_ld) {
        const bool in = plain.value || (row + j >= span.row && row + j < span.row_end);
        const bool begun = !plain.value && (m.start & ((2u << j) - 1)) != 0;      // a sequence, among these rows
        float v[kC];
#pragma unroll
        for (int k = 0; k < kC; k += 2) {
          const Piece p = upto[j][k], q = upto[j][k + 1];
          const float2 f = __ffma2_rn(make_float2(p.p, q.p), make_float2(h[k], h[k + 1]), make_float2(p.b, q.b));
          v[k] = begun ? p.b : f.x;
          v[k + 1] = begun ? q.b : f.y;
        }
        if (in) store_columns<T, kC, kVec>(y, col, cols, lane, v);
        if (!plain.value && (m.end >> j & 1) && a.hT)
          store_columns<float, kC, kVec>(a.hT + static_cast<int64_t>(__shfl_sync(0xffffffffu, m.end_seq, j)) * cols, col, cols,
                                         lane, v);
      }
    };
    if (plain) outputs(Flag<true>{});
    else outputs(Flag<false>{});
    __syncwarp();                                // the tile may be written over
  }
  if (plan.cluster > 1) {                        // nobody leaves while mail to it is on its way
    cluster_sync();
    leave_mail(sh.mail, lost_at);
  }
}

// One row to each sequence: nothing depends on another row.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kStepThreads) recurrence_step_kernel(const __grid_constant__ opt_recurrence_args a,
                                                                   uint32_t slices) {
  constexpr int kN = kVec ? 8 : 1;
  let_next_start();
  wait_for_predecessors();
  const uint32_t block = blockIdx.x / slices;
  const int64_t r = block, c = static_cast<int64_t>((blockIdx.x - block * slices) * kStepThreads + threadIdx.x) * kN;
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
  for (int j = 0; j < kN; ++j) h[j] = advance(gate_of(g[j]), x[j], h[j]);
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
// the saved state for (1 - c) (x_t - h_{t-1}), then backward twice.
template <typename T, int kC, int kW, bool kVec, bool kRagged>
__global__ void __launch_bounds__(32 * kW, kBackwardCtas<kW>)
recurrence_grad_kernel(const __grid_constant__ opt_recurrence_grad_args a, const __grid_constant__ Plan plan) {
  constexpr int kCols = 32 * kC;
  using L = Layout<T, kC, kW, 3>;
  extern __shared__ __align__(128) uint8_t smem[];
  let_next_start();
  wait_for_predecessors();
  const Shared sh = L::carve(smem, plan.cluster);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = plan.cluster > 1 ? cluster_rank() : 0;
  const int id = blockIdx.x / plan.cluster;
  const int rows = static_cast<int>(a.rows), cols = static_cast<int>(a.cols), col = id % plan.groups * kCols;
  if (plan.cluster > 1) {                        // every CTA of the cluster has begun
    if (threadIdx.x == 0) sh.mail.init();
    cluster_sync();
  }
  const Span span = span_of<kRagged>(plan, a.starts, rows, static_cast<int>(a.sequences), id / plan.groups, rank, sh);
  if (kRagged && rank == 0) pass_empty<kCols>(a.starts, span, a.dh0, a.dhT, col, cols);
  const int base = span.row / kS * kS, step = plan.cluster * L::kChunk;
  const int turns = span.row_end > span.row ? (span.row_end - base + step - 1) / step : 0;
  int row = base + (turns - 1) * step + (static_cast<int>(rank) * kW + warp) * kS;
  Cursor at = first_cursor<true>(span);
  auto stage = [&](int turn) { return smem + (turn & 1) * L::kStage + warp * 3 * kTile<T, kC>; };
  auto fetch = [&](int r, int turn) {
    if (r >= base && r < span.row_end) {
      const bool whole = r >= span.row && r + kS <= span.row_end && col + kCols <= cols;
      fetch_rows<T, kC, kVec>(stage(turn), a.x, a.x_ld, r, span, col, cols, lane, whole);
      fetch_rows<T, kC, kVec>(stage(turn) + kTile<T, kC>, a.gate, a.gate_ld, r, span, col, cols, lane, whole);
      fetch_rows<T, kC, kVec>(stage(turn) + 2 * kTile<T, kC>, a.dy, a.dy_ld, r, span, col, cols, lane, whole);
    }
    copy_commit();
  };
  auto saved = [&](int r, float (&h)[kC]) {      // h before row r, where that is a row of the span
    load_state<kC, kVec>(r >= span.row && r < span.row_end ? a.states : nullptr, r / kS, col, cols, lane, h);
  };
  float coming[kC];
  fetch(row, 0);
  saved(row, coming);
  float carry = 0.f;                             // the first kCols threads: behind all rows so far
  int lost_at = kNoneLost;                       // a message of the cluster's
  for (int turn = 0; turn < turns; ++turn, row -= step) {
    copy_wait<0>();
    __syncwarp();
    float h[kC];
#pragma unroll
    for (int k = 0; k < kC; ++k) h[k] = coming[k];
    fetch(row - step, turn + 1);                 // over the rows of the turn before, which this warp is done with
    saved(row - step, coming);
    Marks m;
    if constexpr (kRagged) m = marks_ragged<true>(a.starts, rows, span, row, at, sh, warp, lane);
    else m = marks_equal<true>(plan, span, row, at, lane);
    const uint8_t *xs = stage(turn), *gs = xs + kTile<T, kC>, *ys = gs + kTile<T, kC>;
    float w[kS][kC], q[kS][kC];                  // q = (1 - c) (x_t - h_{t-1})
    Piece mine[kC];
#pragma unroll
    for (int k = 0; k < kC; ++k) mine[k] = Piece{1.f, 0.f};
    auto pieces = [&](auto plain) {              // plain: all rows are there, no sequence starts or ends
#pragma unroll
      for (int j = 0; j < kS; ++j) {
        float g[kC], x[kC];
        columns_at<T, kC, kVec>(gs, j, lane, g);
        columns_at<T, kC, kVec>(xs, j, lane, x);
        const bool in = plain.value || (row + j >= span.row && row + j < span.row_end);
        if (!plain.value && (m.start >> j & 1))
          load_state<kC, kVec>(a.h0, __shfl_sync(0xffffffffu, m.start_seq, j), col, cols, lane, h);
#pragma unroll
        for (int k = 0; k < kC; ++k) {
          w[j][k] = in ? gate_of(g[k]) : 0.f;
          q[j][k] = parts_of(w[j][k], x[k] - h[k]).kept;
          h[k] = in ? advance(w[j][k], x[k], h[k]) : h[k];
        }
      }
#pragma unroll
      for (int j = kS - 1; j >= 0; --j) {
        float dy[kC];
        columns_at<T, kC, kVec>(ys, j, lane, dy);
        const bool in = plain.value || (row + j >= span.row && row + j < span.row_end);
        if (!plain.value && (m.end >> j & 1)) {
          float dhT[kC];
          load_state<kC, kVec>(a.dhT, __shfl_sync(0xffffffffu, m.end_seq, j), col, cols, lane, dhT);
#pragma unroll
          for (int k = 0; k < kC; ++k) mine[k].b = dhT[k];
        }
#pragma unroll
        for (int k = 0; k < kC; ++k) {
          const float l = dy[k] + mine[k].b;
          mine[k].b = !in ? mine[k].b : !plain.value && (m.start >> j & 1) ? 0.f : keep(w[j][k], l);
          mine[k].p = keep(w[j][k], mine[k].p);
        }
      }
      if (!plain.value && (m.start | m.end)) {
#pragma unroll
        for (int k = 0; k < kC; ++k) mine[k].p = kReset;
      }
    };
    const bool plain = row >= span.row && row + kS <= span.row_end && (m.start | m.end) == 0;
    if (plain) pieces(Flag<true>{});
    else pieces(Flag<false>{});
    float b[kC];                                 // (1 - c) l of the row behind
    exchange<kC, kW, kVec, true>(sh, turn, plan.cluster, rank, warp, lane, mine, carry, lost_at, b);
    T* dx = static_cast<T*>(a.dx) + static_cast<int64_t>(row + kS - 1) * a.dx_ld;
    T* dg = static_cast<T*>(a.dgate) + static_cast<int64_t>(row + kS - 1) * a.dgate_ld;
    auto outputs = [&](auto plain) {
#pragma unroll
      for (int j = kS - 1; j >= 0; --j, dx -= a.dx_ld, dg -= a.dgate_ld) {
        float dy[kC], ox[kC], og[kC];
        columns_at<T, kC, kVec>(ys, j, lane, dy);
        const bool in = plain.value || (row + j >= span.row && row + j < span.row_end);
        if (!plain.value && (m.end >> j & 1))
          load_state<kC, kVec>(a.dhT, __shfl_sync(0xffffffffu, m.end_seq, j), col, cols, lane, b);
        if (in) {
#pragma unroll
          for (int k = 0; k < kC; ++k) {
            const Parts l = parts_of(w[j][k], dy[k] + b[k]);
            ox[k] = l.taken;
            og[k] = ox[k] * q[j][k];
            b[k] = l.kept;
          }
          store_columns<T, kC, kVec>(dx, col, cols, lane, ox);
          store_columns<T, kC, kVec>(dg, col, cols, lane, og);
        }
        if (!plain.value && (m.start >> j & 1)) {
          if (a.dh0)
            store_columns<float, kC, kVec>(a.dh0 + static_cast<int64_t>(__shfl_sync(0xffffffffu, m.start_seq, j)) * cols, col,
                                           cols, lane, b);
#pragma unroll
          for (int k = 0; k < kC; ++k) b[k] = 0.f;
        }
      }
    };
    if (plain) outputs(Flag<true>{});
    else outputs(Flag<false>{});
    __syncwarp();                                // the tile may be written over
  }
  if (plan.cluster > 1) {                        // nobody leaves while mail to it is on its way
    cluster_sync();
    leave_mail(sh.mail, lost_at);
  }
}

// ---------------------------------------------------------------- launch --

bool rows_on(const void* p, int64_t ld, int es, int64_t rows, uintptr_t bytes) {
  return !p || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && (rows <= 1 || static_cast<uintptr_t>(ld) * es % bytes == 0));
}

// How many CTAs share the rows of a sequence (a cluster) and how many shares the
// sequences make, so that the CTAs that the SMs hold at once have as few turns as
// possible.  A share of ragged sequences is taken to be longer than the others by
// three average sequences.
template <auto kKernel, typename L, typename Args>
cudaError_t launch_rows(const Args& a, cudaStream_t stream) {
  const int64_t average = (a.rows + a.sequences - 1) / a.sequences;
  const bool ragged = a.starts != nullptr;
  Plan plan{1, 1, static_cast<int>((a.cols + L::kCols - 1) / L::kCols), ragged ? 0 : static_cast<int>(average)};
  const int groups = plan.groups;
  double least = 0;
  for (int cluster = 1; cluster <= kMaxCluster; ++cluster) {
    int held = 0;
    const cudaError_t e = clusters_at_once<kKernel>(cluster, L::kThreads, L::bytes(kMaxCluster), &held);
    if (e != cudaSuccess) return e;
    held *= cluster;
    int64_t ranges = held / (static_cast<int64_t>(groups) * cluster);
    if (ranges < 1) {
      if (cluster > 1) break;
      ranges = 1;
    }
    if (ranges > a.sequences) ranges = a.sequences;
    const int64_t most = ranges == 1 ? a.rows
                         : ragged    ? a.rows / ranges + 3 * average
                                     : (a.sequences + ranges - 1) / ranges * average;
    const int64_t turns = (most + cluster * L::kChunk - 1) / (cluster * L::kChunk);
    const int64_t waves = (ranges * groups * cluster + held - 1) / held;
    const double cost = static_cast<double>(turns * waves) * (cluster > 1 ? 1.25 : 1.0);
    if (cluster == 1 || cost < least) {
      least = cost;
      plan.cluster = cluster;
      plan.ranges = static_cast<int>(ranges);
    }
  }
  const int64_t ctas = static_cast<int64_t>(plan.cluster) * groups * plan.ranges;
  return launch_overlapped(kKernel, dim3(static_cast<unsigned>(ctas)), L::kThreads, L::bytes(plan.cluster), stream, plan.cluster, a,
                           plan);
}

template <typename T, int kC, int kW, bool kVec>
cudaError_t run_forward(const opt_recurrence_args& a, cudaStream_t stream) {
  using L = Layout<T, kC, kW, 2>;
  return a.starts ? launch_rows<recurrence_kernel<T, kC, kW, kVec, true>, L>(a, stream)
                  : launch_rows<recurrence_kernel<T, kC, kW, kVec, false>, L>(a, stream);
}

template <typename T, int kW, bool kVec>
cudaError_t run_backward(const opt_recurrence_grad_args& a, cudaStream_t stream) {
  using L = Layout<T, 2, kW, 3>;
  return a.starts ? launch_rows<recurrence_grad_kernel<T, 2, kW, kVec, true>, L>(a, stream)
                  : launch_rows<recurrence_grad_kernel<T, 2, kW, kVec, false>, L>(a, stream);
}

// The time is that of the turns, one after another, until the columns fill the
// GPU: narrow recurrences take 16 warps, that is twice the rows, a turn (16384
// rows in bf16, back to back: 512 columns 54 us forward and 50 backward, with 8
// warps 59 and 96; 2048 columns 60 and 87, with 8 warps 102 and 131).  The gradient
// in bf16 beyond kFewGradCols columns has 8, three CTAs to an SM: 8192 packed rows of
// 4096 columns 99 us and 100 with 16, of 6144 133 and 151, of 4095, one element at a
// time, 459 and 657 (8192 columns the other way round: 175 and 151).  In fp32, whose
// registers leave room for two such CTAs only, it has 16 throughout: 8192 rows of
// 2560 columns 72 us and 118 with 8, of 4096 108 and 167, of 4095 244 and 431.  From
// kWideCols on the forward pass has four columns to a lane: half the instructions
// around a row's arithmetic (4096 columns 98 us, with two columns 108 by 16 warps and
// 109 by 8; 2048 columns 94, with two 60: too few CTAs).
constexpr int64_t kWideCols = 4096, kFewGradCols = 2048;

template <typename T, bool kVec>
cudaError_t forward(const opt_recurrence_args& a, cudaStream_t stream) {
  if (!a.starts && a.rows == a.sequences) {
    const int64_t per_cta = kStepThreads * (kVec ? 8 : 1), slices = (a.cols + per_cta - 1) / per_cta;
    return launch_overlapped(recurrence_step_kernel<T, kVec>, dim3(static_cast<unsigned>(a.rows * slices)), kStepThreads, 0, stream,
                             0, a, static_cast<uint32_t>(slices));
  }
  if (a.cols < kWideCols) return run_forward<T, 2, 16, kVec>(a, stream);
  return run_forward<T, kVec && sizeof(T) == 2 ? 4 : 2, 8, kVec>(a, stream);
}

template <typename T, bool kVec>
cudaError_t backward(const opt_recurrence_grad_args& a, cudaStream_t stream) {
  if constexpr (sizeof(T) == 2) {
    if (a.cols > kFewGradCols) return run_backward<T, 8, kVec>(a, stream);
  }
  return run_backward<T, 16, kVec>(a, stream);
}

}  // namespace

cudaError_t launch_recurrence(const opt_recurrence_args& a, cudaStream_t stream) {
  const int es = a.dtype == kBf16 ? 2 : 4;
  const bool vec = a.cols % 8 == 0 && rows_on(a.x, a.x_ld, es, a.rows, 16) && rows_on(a.gate, a.gate_ld, es, a.rows, 16) &&
                   rows_on(a.y, a.y_ld, es, a.rows, 16) && rows_on(a.h0, a.cols, 4, 1, 16) &&
                   rows_on(a.hT, a.cols, 4, 1, 16) && rows_on(a.states, a.cols, 4, 1, 16);
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
