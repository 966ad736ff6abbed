// kld_beam.cu -- beam search over logit rows: the selection over beams and
// vocabulary, and the reordering of the beams' states.
//
// Selection. For every group g of W beams with running scores s_w,
//   c(w, j) = s_w + x_wj - lse_w,   lse_w = ln sum_j e^x_wj,
// and the k largest c over (w, j) leave, best first, ties to the lowest
// w * V + j. One read of the logits: a row's columns are split over CTAs,
// each keeping its part of lse (sums of e^(x - m) in fp32 with a thread-level
// frame m that moves only when a value exceeds it by kRaise, fp64 merges, so
// rows of any magnitude, the type's lowest value included, are summed right)
// and the entries that can still
// be among the row's k largest; the last CTA of a group to finish (a ticket)
// merges lse in fp64, scores the kept entries in fp64 and sorts the best k.
//
// What can still be among the k largest: any k entries give a bound, since
// at least k are >= the least of them. The CTA takes its first tile's lane
// maxima, of each warp the ceil(k / warps)-th largest, and the least of
// those: a few shuffles, and only some 1-2 % of a tile lies above. Entries
// at or above the bound go to a list in shared memory, thinned once more in
// the same way at the end. Should the list overflow (large ties, rising
// rows) the part is done again 256 columns at a time with exact pruning.
//
// Bound by HBM for large batches (one read of s bytes an element, one
// exponential), by latency for a few rows.
#include <climits>

#include "kld_internal.h"
#include "kld_packed.cuh"

namespace kld {
namespace {

using packed::neg_inf;
using packed::Type;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = 16;                     // columns of a thread per tile
constexpr int kList = 1024;                  // entries of the shared list
constexpr float kL = 1.4426950408889634f;
constexpr double kLD = static_cast<double>(kL);
constexpr float kRaise = 5.f;                // nats a value may exceed its thread's frame by
constexpr float kLowest = -3.402823466e38f;  // frame before any value

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// e^(lambda d) for the frames' merges, lambda = L ln 2 = 1 + 1.4e-8 as in the sums.
__device__ __forceinline__ double scale_of(float from, float to) {
  return exp2((static_cast<double>(from) - static_cast<double>(to)) * kLD);
}
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ double warp_max(double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmax(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ uint64_t order_key(double x) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(x));
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}
__device__ __forceinline__ double key_value(uint64_t k) {
  const uint64_t b = (k >> 63) ? (k & 0x7fffffffffffffffull) : ~k;
  return __longlong_as_double(static_cast<long long>(b));
}

// The n-th largest (n >= 1) of the warp's values, ties counted apart; -inf
// when fewer than n are above -inf.
template <typename T>
__device__ __forceinline__ T warp_nth(T x, int n) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const T none = -INFINITY;
  T m = warp_max(x);
  for (int i = 1; i < n; ++i) {
    const unsigned who = __ballot_sync(0xffffffffu, x == m);
    if (lane == __ffs(static_cast<int>(who)) - 1) x = none;
    m = warp_max(x);
  }
  return m;
}

// A lower bound of the k-th largest value of the CTA from one value per
// thread: the least of the warps' ceil(k / warps)-th largest.
template <typename T>
__device__ __forceinline__ T block_bound(T x, int k, T* sh) {
  const T m = warp_nth(x, (k + kWarps - 1) / kWarps);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = m;
  __syncthreads();
  T t = sh[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) t = sh[w] < t ? sh[w] : t;
  __syncthreads();
  return t;
}

// The shared list: order keys of the values and their indices (a key's ties
// go to the lowest index).
struct List {
  uint64_t key[kList];
  uint32_t idx[kList];
  int count;
};
__device__ __forceinline__ void push(List& l, uint64_t key, uint32_t idx) {
  const int at = atomicAdd(&l.count, 1);
  if (at < kList) {
    l.key[at] = key;
    l.idx[at] = idx;
  }
}
// Keeps the k best of the list (all when fewer), sorted best first: every
// entry counts those that beat it. Called by the whole CTA, count <= kList.
__device__ void prune(List& l, int k) {
  __syncthreads();
  const int n = l.count;
  constexpr int kEach = kList / kThreads;
  uint64_t key[kEach];
  uint32_t idx[kEach];
  int rank[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = static_cast<int>(threadIdx.x) + e * kThreads;
    rank[e] = i < n ? 0 : INT_MAX;
    key[e] = i < n ? l.key[i] : 0;
    idx[e] = i < n ? l.idx[i] : 0;
  }
  for (int e = 0; e < kEach; ++e) {
    if (e * kThreads >= n) break;
    if (static_cast<int>(threadIdx.x) + e * kThreads >= n) continue;
    int c = 0;
    for (int i = 0; i < n; ++i) {
      const uint64_t o = l.key[i];
      c += (o > key[e] || (o == key[e] && l.idx[i] < idx[e])) ? 1 : 0;
    }
    rank[e] = c;
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    if (rank[e] < k) {
      l.key[rank[e]] = key[e];
      l.idx[rank[e]] = idx[e];
    }
  }
  if (threadIdx.x == 0) l.count = n < k ? n : k;
  __syncthreads();
}

struct Select {
  const void* logits;
  int64_t ld;               // elements between rows
  const float* scores;      // [groups, beams]
  const uint8_t* finished;  // nullable
  int32_t eos;
  int beams, k;
  int64_t V;
  int parts;                // CTAs per row
  int64_t slice;            // columns per CTA (a multiple of the tile's)
  int cap;                  // entries a CTA may leave
  // workspace
  float2* sums;             // [rows * parts]: frame m, sum of e^(x - m)
  int* counts;              // [rows * parts]
  float2* entries;          // [rows * parts][cap]: value, column (bits)
  unsigned* tickets;        // [groups], zero between launches
  uint32_t* flags;
  // outputs [groups, k]
  float* out_scores;
  int32_t* out_tokens;
  int32_t* out_parents;
};

struct SelectShared {
  List list;
  float bound[kWarps];
  double dbound[kWarps];
  float F[kWarps], S[kWarps];
  int kept;
  int last;
  float m[KLD_BEAM_MAX_BEAMS];      // lse = m + lns
  double lns[KLD_BEAM_MAX_BEAMS];   // NaN: the beam offers nothing
  float score[KLD_BEAM_MAX_BEAMS];
};

// Column j of a row, -inf outside.
template <int DT>
__device__ __forceinline__ float value_at(const char* row, int64_t j, int64_t V) {
  return j >= 0 && j < V ? Type<DT>::load(row + j * Type<DT>::kBytes) : neg_inf();
}

// A tile: each thread NV vectors of 16 bytes, vector v of thread t being the
// tile's (v * kThreads + t)-th.
template <int DT>
struct Tile {
  static constexpr int E = 16 / Type<DT>::kBytes;
  static constexpr int NV = kPer / E;
  uint32_t w[4 * NV];
  __device__ void load(const char* row, int64_t j0, int64_t j1, int64_t V, int off) {
    // columns [j0, j1) of the vector grid, which starts `off` columns before the row
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t g = j0 + (v * kThreads + static_cast<int>(threadIdx.x)) * E;
      const int64_t j = g - off;
      uint4 x;
      if (g < j1 && j >= 0 && j + E <= V) {
        x = __ldcs(reinterpret_cast<const uint4*>(row + j * Type<DT>::kBytes));
      } else {
        float y[E];
#pragma unroll
        for (int k = 0; k < E; ++k) y[k] = g < j1 ? value_at<DT>(row, j + k, V) : neg_inf();
        x = Type<DT>::vec(y);
      }
      *reinterpret_cast<uint4*>(&w[4 * v]) = x;
    }
  }
  __device__ static int64_t column(int64_t j0, int k, int off) {
    return j0 + ((k / E) * kThreads + static_cast<int>(threadIdx.x)) * E + k % E - off;
  }
};

// Best k entries of columns [g0, g1) of the vector grid, exactly, 256 columns
// at a time (the path of a part whose list overflowed).
template <int DT>
__device__ __noinline__ void slow_part(List& l, const char* row, int64_t g0, int64_t g1, int off,
                                       int64_t V, int k) {
  __syncthreads();
  if (threadIdx.x == 0) l.count = 0;
  __syncthreads();
  uint64_t least = 0;  // key of the k-th best once k are known
  bool full = false;
  for (int64_t g = g0; g < g1; g += kThreads) {
    const int64_t j = g + threadIdx.x - off;
    const float x = g + threadIdx.x < g1 ? value_at<DT>(row, j, V) : neg_inf();
    const uint64_t key = order_key(static_cast<double>(x));
    // columns rise, so an equal value later never replaces an earlier one
    if (x > neg_inf() && (!full || key > least)) push(l, key, static_cast<uint32_t>(j));
    __syncthreads();
    if (l.count > kList - kThreads) {
      prune(l, k);
      full = l.count == k;
      if (full) least = l.key[k - 1];
    }
    __syncthreads();
  }
  prune(l, k);
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 4) kld_beam_select_kernel(const Select a) {
  __shared__ SelectShared sh;
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int64_t part = blockIdx.x;
  const int64_t r = part / a.parts;
  const int64_t group = r / a.beams;
  const int64_t V = a.V;
  const float score = __ldg(a.scores + r);
  const bool done = a.finished && __ldg(a.finished + r);
  const bool live = !done && score > neg_inf() && score < INFINITY;
  if (tid == 0) {
    sh.list.count = 0;
    sh.kept = 0;
    if (!(score < INFINITY) && part % a.parts == 0) atomicOr(a.flags, KLD_BEAM_BAD_SCORE);
  }
  __syncthreads();

  if (live) {
    const char* row = static_cast<const char*>(a.logits) + r * a.ld * Type<DT>::kBytes;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / Type<DT>::kBytes);
    const int64_t g0 = (part % a.parts) * a.slice;
    int64_t g1 = g0 + a.slice;
    if (g1 > V + off) g1 = V + off;
    constexpr int64_t kTile = static_cast<int64_t>(kThreads) * kPer;
    float F = kLowest, S = 0.f, T = neg_inf();
    Tile<DT> t;
    if (g0 < g1) t.load(row, g0, g1, V, off);
    for (int64_t g = g0; g < g1; g += kTile) {
      float x[kPer];
      Type<DT>::unpack16(t.w, x);
      if (g + kTile < g1) t.load(row, g + kTile, g1, V, off);
      float m = x[0];
#pragma unroll
      for (int k = 1; k < kPer; ++k) m = fmaxf(m, x[k]);
      if (m > F + kRaise) {
        S *= ex2((F - m) * kL);
        F = m;
      }
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < kPer; ++k) s += ex2((x[k] - F) * kL);
      S += s;
      if (g == g0) T = block_bound(m, a.k, sh.bound);
      if (m >= T && m > neg_inf()) {
#pragma unroll
        for (int k = 0; k < kPer; ++k)
          if (x[k] >= T && x[k] > neg_inf())
            push(sh.list, order_key(static_cast<double>(x[k])),
                 static_cast<uint32_t>(Tile<DT>::column(g, k, off)));
      }
    }
    // this CTA's frame and sum
    {
      const float f = warp_max(F);
      float s = S * ex2((F - f) * kL);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == 0) {
        sh.F[warp] = f;
        sh.S[warp] = s;
      }
    }
    __syncthreads();
    int n = sh.list.count;
    if (n > kList) {
      slow_part<DT>(sh.list, row, g0, g1, off, V, a.k);
      n = sh.list.count;
    }
    double T2 = -INFINITY;
    if (n > a.cap) {
      double best = -INFINITY;
      for (int i = tid; i < n; i += kThreads) best = fmax(best, key_value(sh.list.key[i]));
      T2 = block_bound(best, a.k, sh.dbound);
    }
    float2* to = a.entries + part * a.cap;
    for (int i = tid; i < n; i += kThreads) {
      const double x = key_value(sh.list.key[i]);
      if (x >= T2) {
        const int at = atomicAdd(&sh.kept, 1);
        if (at < a.cap) to[at] = make_float2(static_cast<float>(x), __uint_as_float(sh.list.idx[i]));
      }
    }
    __syncthreads();
    if (sh.kept > a.cap) {  // ties at the bound: the exact k best
      prune(sh.list, a.k);
      if (tid < sh.list.count)
        to[tid] = make_float2(static_cast<float>(key_value(sh.list.key[tid])),
                              __uint_as_float(sh.list.idx[tid]));
      if (tid == 0) sh.kept = sh.list.count;
      __syncthreads();
    }
    if (tid == 0) {
      float f = sh.F[0];
      for (int w = 1; w < kWarps; ++w) f = fmaxf(f, sh.F[w]);
      double s = 0.0;
      for (int w = 0; w < kWarps; ++w) s += scale_of(sh.F[w], f) * sh.S[w];
      a.sums[part] = make_float2(f, static_cast<float>(s));
    }
  }
  if (tid == 0) a.counts[part] = live ? sh.kept : 0;

  // ---- the group's last CTA merges
  __threadfence();
  __syncthreads();
  if (tid == 0) {
    const unsigned parts = static_cast<unsigned>(a.beams * a.parts);
    const unsigned seen = atomicAdd(a.tickets + group, 1u);
    sh.last = seen == parts - 1u;
    if (sh.last) a.tickets[group] = 0u;
  }
  __syncthreads();
  if (!sh.last) return;
  __threadfence();

  const int64_t row0 = group * a.beams, part0 = row0 * a.parts;
  for (int w = warp; w < a.beams; w += kWarps) {
    const float sc = __ldcg(a.scores + row0 + w);
    const bool fin = a.finished && __ldcg(a.finished + row0 + w);
    double lns = __longlong_as_double(0x7ff8000000000000ll);
    float f = kLowest;
    if (!fin && sc > neg_inf() && sc < INFINITY) {
      for (int p = lane; p < a.parts; p += 32)
        f = fmaxf(f, __ldcg(a.sums + part0 + static_cast<int64_t>(w) * a.parts + p).x);
      f = warp_max(f);
      double s = 0.0;
      for (int p = lane; p < a.parts; p += 32) {
        const float2 v = __ldcg(a.sums + part0 + static_cast<int64_t>(w) * a.parts + p);
        s += scale_of(v.x, f) * v.y;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      // NaN, +inf or nothing but -inf: no candidates
      if (s > 0.0 && s < 1e300)
        lns = log(s);
      else if (lane == 0)
        atomicOr(a.flags, KLD_BEAM_NONFINITE);
    }
    if (lane == 0) {
      sh.m[w] = f;
      sh.lns[w] = lns;
      sh.score[w] = sc;
    }
  }
  if (tid == 0) sh.list.count = 0;
  __syncthreads();

  const int lists = a.beams * a.parts;
  // Score of entry i of list l; false when there is none.
  auto scored = [&](int l, int i, double& s, uint32_t& flat) {
    const int w = l / a.parts;
    const double lns = sh.lns[w];
    if (!(lns == lns)) return false;
    const float2 e = __ldcg(a.entries + (part0 + l) * a.cap + i);
    s = static_cast<double>(sh.score[w]) +
        ((static_cast<double>(e.x) - static_cast<double>(sh.m[w])) - lns);
    flat = static_cast<uint32_t>(w) * static_cast<uint32_t>(V) + __float_as_uint(e.y);
    return true;
  };
  double best = -INFINITY;
  for (int l = warp; l < lists; l += kWarps) {
    const int n = __ldcg(a.counts + part0 + l);
    for (int i = lane; i < n; i += 32) {
      double s;
      uint32_t flat;
      if (scored(l, i, s, flat)) best = fmax(best, s);
    }
  }
  const double bound = block_bound(best, a.k, sh.dbound);
  for (int l = warp; l < lists; l += kWarps) {
    const int n = __ldcg(a.counts + part0 + l);
    for (int i = lane; i < n; i += 32) {
      double s;
      uint32_t flat;
      if (scored(l, i, s, flat) && s >= bound) push(sh.list, order_key(s), flat);
    }
  }
  auto offer_finished = [&]() {
    // a finished beam stays as it is: one candidate, its eos
    if (a.finished && tid < a.beams && __ldcg(a.finished + row0 + tid)) {
      const float sc = sh.score[tid];
      if (sc > neg_inf() && sc < INFINITY)
        push(sh.list, order_key(static_cast<double>(sc)),
             static_cast<uint32_t>(tid) * static_cast<uint32_t>(V) + static_cast<uint32_t>(a.eos));
    }
  };
  offer_finished();
  __syncthreads();
  if (sh.list.count > kList) {
    // ties at the bound: again, one list at a time with exact pruning
    __syncthreads();
    if (tid == 0) sh.list.count = 0;
    __syncthreads();
    offer_finished();
    for (int l = 0; l < lists; ++l) {
      const int n = __ldcg(a.counts + part0 + l);
      for (int i = tid; i < n; i += kThreads) {
        double s;
        uint32_t flat;
        if (scored(l, i, s, flat) && s >= bound) push(sh.list, order_key(s), flat);
      }
      __syncthreads();
      if (sh.list.count > kList - kThreads) prune(sh.list, a.k);
      __syncthreads();
    }
  }
  prune(sh.list, a.k);
  if (tid < a.k) {
    const int64_t o = group * a.k + tid;
    const bool some = tid < sh.list.count;
    const uint32_t flat = some ? sh.list.idx[tid] : 0u;
    a.out_scores[o] = some ? static_cast<float>(key_value(sh.list.key[tid])) : neg_inf();
    a.out_tokens[o] = some ? static_cast<int32_t>(flat % static_cast<uint32_t>(V)) : -1;
    a.out_parents[o] = some ? static_cast<int32_t>(flat / static_cast<uint32_t>(V)) : -1;
  }
}

// -------------------------------------------------------------- reordering
//
// state[g, w] <- state[g, parent[g, w]] in place, for the first len positions
// of each run. A thread owns one 16-byte (or smaller) column of a group's W
// rows: it reads the rows that other beams take, then writes the beams that
// change, so no copy of the state and no exchange between threads is needed,
// and beams that keep their slot cost nothing. Bound by HBM: the distinct
// sources are read once (a source of two beams again from L2), each changed
// beam is written once.

constexpr int kStatesPerLaunch = 48;
constexpr int kSpan = 4;  // columns of a thread (kThreads apart)

struct StateDesc {
  char* p;
  int64_t row_stride, outer_stride;  // bytes
  int64_t run;                       // bytes of a full run (all positions)
  int64_t unit;                      // bytes of one position; 0: no time axis
  int32_t outer;
  uint32_t spans;                    // CTAs per run
  uint32_t first;                    // first CTA of this state
};
struct Reorder {
  StateDesc s[kStatesPerLaunch];
  int n, beams;
  const int32_t* parents;
  const int32_t* lengths;  // nullable
  uint32_t* flags;
};
static_assert(sizeof(Reorder) <= 4000, "kernel parameters");

template <typename Vec, int kMaxBeams>
__global__ void __launch_bounds__(kThreads) kld_beam_reorder_kernel(const __grid_constant__ Reorder a) {
  __shared__ int src[kMaxBeams];        // -1: the beam keeps its slot
  __shared__ int64_t bytes[kMaxBeams];  // of the run that the beam takes over
  __shared__ int64_t longest;
  const int tid = static_cast<int>(threadIdx.x);
  int i = 0;
  while (i + 1 < a.n && a.s[i + 1].first <= blockIdx.x) ++i;
  const StateDesc& s = a.s[i];
  const uint32_t item = blockIdx.x - s.first;
  const uint32_t span = item % s.spans;
  const uint32_t rest = item / s.spans;
  const int outer = static_cast<int>(rest % static_cast<uint32_t>(s.outer));
  const int64_t group = rest / static_cast<uint32_t>(s.outer);
  const int64_t x0 = static_cast<int64_t>(span) * (kThreads * kSpan * static_cast<int>(sizeof(Vec)));
  if (tid == 0) longest = 0;
  __syncthreads();
  if (tid < a.beams) {
    int p = __ldg(a.parents + group * a.beams + tid);
    if (p < -1 || p >= a.beams) {
      if (span == 0) atomicOr(a.flags, KLD_BEAM_BAD_PARENT);
      p = -1;
    }
    int64_t n = 0;
    if (p >= 0 && p != tid) {
      n = s.run;
      if (a.lengths && s.unit) {
        const int64_t len = __ldg(a.lengths + group * a.beams + p);
        n = len <= 0 ? 0 : (len * s.unit < n ? len * s.unit : n);
      }
      if (n > x0) atomicMax(reinterpret_cast<unsigned long long*>(&longest),
                            static_cast<unsigned long long>(n));
    }
    src[tid] = n > x0 ? p : -1;
    bytes[tid] = n;
  }
  __syncthreads();
  if (longest == 0) return;
  char* base = s.p + group * a.beams * s.row_stride + static_cast<int64_t>(outer) * s.outer_stride;
#pragma unroll 1
  for (int k = 0; k < kSpan; ++k) {
    const int64_t x = x0 + static_cast<int64_t>(k * kThreads + tid) * static_cast<int>(sizeof(Vec));
    if (x >= longest) break;
    Vec v[kMaxBeams];
#pragma unroll
    for (int w = 0; w < kMaxBeams; ++w) {
      if (w < a.beams && src[w] >= 0) {
        const char* from = base + src[w] * s.row_stride + x;
        if (x + static_cast<int64_t>(sizeof(Vec)) <= bytes[w]) {
          v[w] = __ldcg(reinterpret_cast<const Vec*>(from));
        } else {
          // the run's last bytes, one by one
          unsigned char* b = reinterpret_cast<unsigned char*>(&v[w]);
#pragma unroll
          for (int q = 0; q < static_cast<int>(sizeof(Vec)); ++q)
            b[q] = x + q < bytes[w] ? __ldcg(reinterpret_cast<const unsigned char*>(from) + q) : 0;
        }
      }
    }
#pragma unroll
    for (int w = 0; w < kMaxBeams; ++w) {
      if (w < a.beams && src[w] >= 0) {
        char* to = base + w * s.row_stride + x;
        if (x + static_cast<int64_t>(sizeof(Vec)) <= bytes[w]) {
          *reinterpret_cast<Vec*>(to) = v[w];
        } else {
          const unsigned char* b = reinterpret_cast<const unsigned char*>(&v[w]);
#pragma unroll
          for (int q = 0; q < static_cast<int>(sizeof(Vec)); ++q)
            if (x + q < bytes[w]) to[q] = static_cast<char>(b[q]);
        }
      }
    }
  }
}

// Widest vector a group of `beams` rows may hold in registers: 16 bytes up to
// 16 beams, 8 up to 32, 4 up to 64 (64 registers each).
int widest(int beams) { return beams <= 16 ? 16 : (beams <= 32 ? 8 : 4); }

template <typename Vec>
cudaError_t launch_reorder_vec(const Reorder& a, unsigned grid, cudaStream_t s) {
  if (a.beams <= 4)
    kld_beam_reorder_kernel<Vec, 4><<<grid, kThreads, 0, s>>>(a);
  else if (a.beams <= 8)
    kld_beam_reorder_kernel<Vec, 8><<<grid, kThreads, 0, s>>>(a);
  else if (a.beams <= 16)
    kld_beam_reorder_kernel<Vec, 16><<<grid, kThreads, 0, s>>>(a);
  else if constexpr (sizeof(Vec) <= 8) {
    if (a.beams <= 32)
      kld_beam_reorder_kernel<Vec, 32><<<grid, kThreads, 0, s>>>(a);
    else if constexpr (sizeof(Vec) <= 4)
      kld_beam_reorder_kernel<Vec, 64><<<grid, kThreads, 0, s>>>(a);
    else
      return cudaErrorInvalidValue;
  } else {
    return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace

BeamPlan plan_beam(int64_t rows, int64_t V, int off, int sm_count) {
  // About 16 slices an SM over all rows (four waves of four CTAs) keep the
  // SMs evenly busy; a slice is at least one tile. parts * rows stays below
  // 16 * SMs + 2 * rows, the workspace's size.
  constexpr int64_t tile = static_cast<int64_t>(kThreads) * kPer;
  BeamPlan p;
  const int64_t target = static_cast<int64_t>(sm_count) * 16;
  p.slice = (rows * V + target - 1) / target;
  p.slice = (p.slice + tile - 1) / tile * tile;
  // the grid of vectors starts up to `off` columns before a row
  p.parts = static_cast<int>((V + off + p.slice - 1) / p.slice);
  return p;
}

cudaError_t launch_beam_select(const BeamSelect& b, int sm_count, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(b.groups) * b.beams;
  const int eb = elem_bytes(b.dtype);
  const bool aligned = (reinterpret_cast<uintptr_t>(b.logits) & 15u) == 0 && b.ld * eb % 16 == 0;
  const BeamPlan p = plan_beam(rows, b.V, aligned ? 0 : 16 / eb - 1, sm_count);
  Select a;
  a.logits = b.logits;
  a.ld = b.ld;
  a.scores = b.scores;
  a.finished = b.finished;
  a.eos = b.eos;
  a.beams = b.beams;
  a.k = b.k;
  a.V = b.V;
  a.parts = p.parts;
  a.slice = p.slice;
  a.cap = b.cap;
  a.sums = b.sums;
  a.counts = b.counts;
  a.entries = b.entries;
  a.tickets = b.tickets;
  a.flags = b.flags;
  a.out_scores = b.out_scores;
  a.out_tokens = b.out_tokens;
  a.out_parents = b.out_parents;
  const unsigned grid = static_cast<unsigned>(rows * p.parts);
  switch (b.dtype) {
    case KLD_F32: kld_beam_select_kernel<KLD_F32><<<grid, kThreads, 0, stream>>>(a); break;
    case KLD_BF16: kld_beam_select_kernel<KLD_BF16><<<grid, kThreads, 0, stream>>>(a); break;
    case KLD_F16: kld_beam_select_kernel<KLD_F16><<<grid, kThreads, 0, stream>>>(a); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

cudaError_t launch_beam_reorder(const kld_state_t* states, int n, const int32_t* parents,
                                const int32_t* lengths, int groups, int beams, uint32_t* flags,
                                cudaStream_t stream) {
  // One launch per vector width (and per kStatesPerLaunch states).
  for (int width = 16; width >= 1; width >>= 1) {
    Reorder a;
    a.n = 0;
    a.beams = beams;
    a.parents = parents;
    a.lengths = lengths;
    a.flags = flags;
    uint64_t grid = 0;
    auto flush = [&]() -> cudaError_t {
      if (a.n == 0) return cudaSuccess;
      cudaError_t e;
      const unsigned g = static_cast<unsigned>(grid);
      switch (width) {
        case 16: e = launch_reorder_vec<uint4>(a, g, stream); break;
        case 8: e = launch_reorder_vec<uint2>(a, g, stream); break;
        case 4: e = launch_reorder_vec<unsigned int>(a, g, stream); break;
        case 2: e = launch_reorder_vec<unsigned short>(a, g, stream); break;
        default: e = launch_reorder_vec<unsigned char>(a, g, stream); break;
      }
      a.n = 0;
      grid = 0;
      return e;
    };
    for (int i = 0; i < n; ++i) {
      const kld_state_t& t = states[i];
      const int64_t run = t.positions * t.position_bytes;
      if (run == 0 || t.outer == 0) continue;
      const uint64_t bits = reinterpret_cast<uintptr_t>(t.data) | static_cast<uint64_t>(t.row_stride) |
                            (t.outer > 1 ? static_cast<uint64_t>(t.outer_stride) : 0u);
      int w = widest(beams);
      while (w > 1 && (bits & static_cast<uint64_t>(w - 1))) w >>= 1;
      if (w != width) continue;
      StateDesc d;
      d.p = static_cast<char*>(t.data);
      d.row_stride = t.row_stride;
      d.outer_stride = t.outer_stride;
      d.run = run;
      d.unit = t.timed ? t.position_bytes : 0;
      d.outer = static_cast<int32_t>(t.outer);
      const int64_t span = static_cast<int64_t>(kThreads) * kSpan * width;
      d.spans = static_cast<uint32_t>((run + span - 1) / span);
      const uint64_t ctas = static_cast<uint64_t>(d.spans) * static_cast<uint64_t>(t.outer) *
                            static_cast<uint64_t>(groups);
      if (ctas > 0x7fffffffu) return cudaErrorInvalidConfiguration;
      if (a.n == kStatesPerLaunch || grid + ctas > 0x7fffffffu) {
        const cudaError_t e = flush();
        if (e != cudaSuccess) return e;
      }
      d.first = static_cast<uint32_t>(grid);
      a.s[a.n++] = d;
      grid += ctas;
    }
    const cudaError_t e = flush();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace kld
