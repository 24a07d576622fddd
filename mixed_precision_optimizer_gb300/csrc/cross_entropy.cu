// Cross-entropy of rows of logits and its gradient (sm_103a):
//
//   lse = m + log(sum_j exp(x_j - m)), m = max_j x_j;  loss = lse - x_label
//   dx_j = (exp(x_j - m) / sum - [j = label]) * scale * weight
//
// Bound by HBM.  cross_entropy_cluster_kernel keeps a row on the chip: up to eight
// CTAs of a cluster share it, each thread reads its 64 elements once, takes their
// exponentials from its own maximum, and scales them when the row's maximum and
// sum are known: one exponential an element (with two, one for the sum and one
// for the gradient, 8192 x 128256 in bf16 took 1190 us; with 32 elements a thread
// and 16 CTAs 990; now 802 to 823, 5.2 TB/s).  The CTAs stay for many rows, and the next
// rows' elements are on their way (cp.async) meanwhile: what remains is a row's
// chain of maximum, sum, mail and scaling, which two CTAs to an SM overlap.
// cross_entropy_kernel reads the row twice, the second time out of L1 or L2: rows
// of up to 1024 columns by a warp each, and those beyond eight CTAs' reach by a
// CTA.
// Groups of 16 bytes begin at the row's first multiple of 16 bytes, the elements
// around them go to one thread each.

#include "cluster.cuh"
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

// ---------------------------------------------------------------- cluster --

constexpr int kElems = 64;                       // of a thread
constexpr int kMaxCluster = kMostClusterCtas;

template <typename T, int kThreads>
struct Config {
  static constexpr int kGroups = kElems / Group<T>::kN;            // of a thread
  static constexpr int kStageBytes = kGroups * kThreads * 16;
  static constexpr int kCtas = 512 / kThreads;                     // to an SM: 128 registers a thread
  static constexpr int kStages = 192 * 1024 / kCtas / kStageBytes; // rows on their way
  static constexpr int kBytes = kStages * kStageBytes;
  static_assert(kStages >= 1, "the ring holds a row's share");
};

// A row in elements: the first group's column, the groups, the column behind the last.
struct Place {
  int head, groups, end;
};

template <typename T>
__device__ __forceinline__ Place place_of(const T* x, int cols) {
  constexpr int kN = Group<T>::kN;
  const int ahead = static_cast<int>(-(reinterpret_cast<uintptr_t>(x) / sizeof(T)) & (kN - 1));
  Place p;
  p.head = ahead < cols ? ahead : cols;
  p.groups = static_cast<uint32_t>(cols - p.head) / kN;
  p.end = p.head + p.groups * kN;
  return p;
}

// The maximum of a group; a NaN counts only where there is nothing else.
__device__ __forceinline__ float group_max(const uint4& w, const __nv_bfloat16*) {
  auto two = [](uint32_t u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); };
  const __nv_bfloat162 m = __hmax2(__hmax2(two(w.x), two(w.y)), __hmax2(two(w.z), two(w.w)));
  return fmaxf(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float group_max(const uint4& w, const float*) {
  return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
}
__device__ __forceinline__ void group_values(const uint4& w, float (&v)[8]) { unpack8(w, v); }
__device__ __forceinline__ void group_values(const uint4& w, float (&v)[4]) {
  v[0] = __uint_as_float(w.x), v[1] = __uint_as_float(w.y), v[2] = __uint_as_float(w.z), v[3] = __uint_as_float(w.w);
}

// The Stat of all that the lanes hold, in every lane.
__device__ __forceinline__ Stat warp_join(Stat s) {
  float top = s.top;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  float sum = s.sum * exp_of(s.top - anchor(top));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  return Stat{top, sum};
}

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, (Config<T, kThreads>::kCtas))
cross_entropy_cluster_kernel(const __grid_constant__ opt_cross_entropy_args a, int cluster) {
  using C = Config<T, kThreads>;
  constexpr int kN = Group<T>::kN, kWarps = kThreads / 32, kGroups = C::kGroups;
  extern __shared__ uint4 ring[];                // [kStages][kGroups][kThreads]
  __shared__ float2 parts[2][kMaxCluster * kWarps];        // every warp's of the cluster
  __shared__ uint64_t bars[2];
  let_next_start();
  wait_for_predecessors();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, cols = static_cast<int>(a.cols);
  const int rank = cluster > 1 ? static_cast<int>(cluster_rank()) : 0;
  const Mailbox mail{bars};
  if (cluster > 1) {                             // every CTA of the cluster has begun
    if (t == 0) mail.init();
    cluster_sync();
  }
  const int64_t step = gridDim.x / cluster;
  const int mine = rank * kGroups * kThreads + t;          // this thread's first group
  auto row_at = [&](int64_t r) { return static_cast<const T*>(a.logits) + r * a.logits_ld; };
  auto label_at = [&](int64_t r) {
    const int64_t v = a.index_dtype == OPT_INDEX_INT32 ? static_cast<int64_t>(static_cast<const int32_t*>(a.labels)[r])
                                                       : static_cast<const int64_t*>(a.labels)[r];
    return v >= 0 && v < cols ? static_cast<int>(v) : -1;
  };
  // row r into a stage, this thread's own places; a commit in any case
  auto fetch = [&](int64_t r, int stage) {
    if (r < a.rows) {
      const T* x = row_at(r);
      const Place p = place_of(x, cols);
      const T* from = x + p.head + mine * kN;
      uint4* to = ring + stage * kGroups * kThreads + t;
#pragma unroll
      for (int i = 0; i < kGroups; ++i)
        if (mine + i * kThreads < p.groups) copy16(to + i * kThreads, from + i * kThreads * kN);
    }
    copy_commit();
  };
  int64_t r = blockIdx.x / cluster;
  for (int s = 0; s < C::kStages; ++s) fetch(r + s * step, s);
  int label = label_at(r), next_label = -1;      // the grid has no more clusters than rows
  int lost_at = kNoneLost;                       // a message of the cluster's
  for (int k = 0, stage = 0; r < a.rows; ++k, r += step, label = next_label, stage = stage + 1 == C::kStages ? 0 : stage + 1) {
    const T* x = row_at(r);
    const Place p = place_of(x, cols);
    if (r + step < a.rows) next_label = label_at(r + step);
    const float w = a.weight ? a.weight[r] * a.scale : a.scale;
    // the column outside of the groups that this thread has, or -1
    const int edge = rank ? -1 : t < p.head ? t : t < p.head + cols - p.end ? p.end + t - p.head : -1;
    const float at_edge = edge >= 0 ? load_elem(x + edge) : -INFINITY;
    copy_wait<C::kStages - 1>();
    const uint4* from = ring + stage * kGroups * kThreads + t;
    float e[kGroups][kN], top = at_edge;
    {
      uint4 raw[kGroups];
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        const uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;       // -inf
        raw[i] = mine + i * kThreads < p.groups ? from[i * kThreads] : make_uint4(none, none, none, none);
        top = fmaxf(top, group_max(raw[i], static_cast<const T*>(nullptr)));
      }
#pragma unroll
      for (int i = 0; i < kGroups; ++i) group_values(raw[i], e[i]);
    }
    // the label's group and its place there, where it is this thread's
    const int hot = label - p.head, away = hot / kN - mine;
    const bool hot_here = label >= 0 && hot >= 0 && hot < p.groups * kN && away >= 0 && away < kGroups * kThreads &&
                          away % kThreads == 0;
    float at_label = at_edge;
    if (hot_here) at_label = load_elem(reinterpret_cast<const T*>(from + away) + (hot & (kN - 1)));
    const float own = anchor(top), edge_e = exp_of(at_edge - own);
    float sum = edge_e;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      float part = 0.f;
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        e[i][j] = exp_of(e[i][j] - own);
        part += e[i][j];
      }
      sum += part;
    }
    fetch(r + C::kStages * step, stage);         // over what this thread has read
    Stat s = warp_join(Stat{top, sum});
    if (cluster > 1) {                           // lane i tells CTA i
      const bool there = exchange_message(mail, k, t == 0, static_cast<uint32_t>(cluster) * kWarps * 8, lost_at, [&] {
        if (lane < cluster) mail.send(k, &parts[k & 1][rank * kWarps + warp], lane, make_float2(s.top, s.sum));
      });
      if (!__all_sync(0xffffffffu, there) && lost_at == kNoneLost) lost_at = k;      // a warp reads and sends as one
    } else {
      if (lane == 0) parts[k & 1][warp] = make_float2(s.top, s.sum);
      __syncthreads();
    }
    s = Stat{-INFINITY, 0.f};
    for (int i = lane; i < cluster * kWarps; i += 32) {
      const float2 q = parts[k & 1][i];
      s = join(s, Stat{q.x, q.y});
    }
    s = warp_join(s);
    if (lost_at != kNoneLost) s.sum = __uint_as_float(0x7fc00000u);
    const bool none = s.sum == 0.f;              // an empty row
    if (rank == 0 && t == 0) {
      if (a.lse) a.lse[r] = none ? -INFINITY : s.top + logf(s.sum);
      if (a.loss && label < 0) a.loss[r] = 0.f;
    }
    if (a.loss && label >= 0 && (hot_here || edge == label))
      a.loss[r] = none ? INFINITY : logf(s.sum) - (at_label - anchor(s.top));
    if (!a.dlogits) continue;
    T* g = static_cast<T*>(a.dlogits) + r * a.dlogits_ld;
    const bool zero = label < 0 || none;
    const float inv = exp_of(top - anchor(s.top)) / s.sum, inv_w = inv * w;
    if (edge >= 0) store_elem(g + edge, zero ? 0.f : (edge_e * inv - (edge == label ? 1.f : 0.f)) * w);
    const bool together = (reinterpret_cast<uintptr_t>(g + p.head) & 15u) == 0;
    T* to = g + p.head + mine * kN;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      if (mine + i * kThreads >= p.groups) break;
      if (zero) {
#pragma unroll
        for (int j = 0; j < kN; ++j) e[i][j] = 0.f;
      } else if (hot_here && away == i * kThreads) {
#pragma unroll
        for (int j = 0; j < kN; ++j) e[i][j] = (e[i][j] * inv - (j == (hot & (kN - 1)) ? 1.f : 0.f)) * w;
      } else {
#pragma unroll
        for (int j = 0; j < kN; ++j) e[i][j] *= inv_w;
      }
      if (together) {
        store_group(to + i * kThreads * kN, e[i]);
      } else {
#pragma unroll
        for (int j = 0; j < kN; ++j) store_elem(to + i * kThreads * kN + j, e[i][j]);
      }
    }
  }
  if (cluster > 1) {                             // nobody leaves while mail to it is on its way
    cluster_sync();
    leave_mail(mail, lost_at);
  }
}

template <typename T, int kThreads>
cudaError_t launch_cluster(const opt_cross_entropy_args& a, int cluster, cudaStream_t stream) {
  using C = Config<T, kThreads>;
  const size_t smem = C::kBytes;
  int most = 0;
  const cudaError_t e = clusters_at_once<cross_entropy_cluster_kernel<T, kThreads>>(cluster, kThreads, smem, &most);
  if (e != cudaSuccess) return e;
  const int64_t clusters = a.rows < most ? a.rows : most;
  return launch_overlapped(cross_entropy_cluster_kernel<T, kThreads>, dim3(static_cast<unsigned>(clusters * cluster)), kThreads,
                           smem, stream, cluster, a, cluster);
}

template <typename T>
cudaError_t launch_rows(const opt_cross_entropy_args& a, cudaStream_t stream) {
  if (a.cols <= 1024)
    return launch_overlapped(cross_entropy_kernel<T, 32>, dim3(static_cast<unsigned>((a.rows + 7) / 8)), 256, 0, stream, 0, a);
  if (a.cols <= 64 * kElems) return launch_cluster<T, 64>(a, 1, stream);
  if (a.cols <= 128 * kElems) return launch_cluster<T, 128>(a, 1, stream);
  int cluster = 1;
  while (cluster < kMaxCluster && a.cols > static_cast<int64_t>(cluster) * 256 * kElems) cluster *= 2;
  if (a.cols <= static_cast<int64_t>(cluster) * 256 * kElems) return launch_cluster<T, 256>(a, cluster, stream);
  return launch_overlapped(cross_entropy_kernel<T, 1024>, dim3(static_cast<unsigned>(a.rows)), 1024, 0, stream, 0, a);
}

}  // namespace

cudaError_t launch_cross_entropy(const opt_cross_entropy_args& a, cudaStream_t stream) {
  return a.dtype == kBf16 ? launch_rows<__nv_bfloat16>(a, stream) : launch_rows<float>(a, stream);
}

}  // namespace mpopt
