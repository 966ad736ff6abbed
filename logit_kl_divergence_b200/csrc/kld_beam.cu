// kld_beam.cu -- beam search over logit rows: the selection over beams and
// vocabulary, and the reordering of the beams' states.
//
// Selection. For every group g of W beams with running scores s_w,
//   c(w, j) = s_w + x_wj - lse_w,   lse_w = ln sum_j e^x_wj,
// and the k largest c over (w, j) leave, best first, ties to the lowest
// w * V + j. One read of the logits: a row's columns are split over CTAs,
// each keeping its part of lse (sums of e^(x - m) with a thread-level
// frame m that moves only when a value exceeds it by kRaise, fp64 merges, so
// rows of any magnitude, the type's lowest value included, are summed right;
// fp32 exponentials, and their sums over a thread's 16 columns and a warp in
// fp32, err by 2e-6 in lse at most, as the scores' own fp32 does, and alike in
// equal rows) and the entries that can still be among the row's k largest; the
// last CTA of a group to finish (a ticket) merges lse in fp64, scores the kept
// entries in fp64 and sorts the best k.
//
// What can still be among the k largest: any k entries give a bound, since
// at least k are >= the least of them. The CTA takes its lanes'
// maxima, of each warp the few largest, and the k-th largest of those: close
// to the k-th largest of the tiles so far. The bound is renewed after 1, 2,
// 4, ... tiles, so that about k entries pass it from one time to the next.
// They go to a list in shared memory. Should the list overflow
// (large ties, rising rows) the part is done again 256 columns at a time with
// exact pruning. The merge does the same with the lists' maxima: only lists
// whose maximum reaches the k-th largest of them are read.
//
// Bound by latency for a few rows (4 rows of 32000 bf16: 12 us), by instruction
// issue and the bounds' barriers for many: 16 instructions an element, one
// exponential among them, at 55 % of the issue slots. 256 rows of 151936 bf16
// take 48 us (fp32 50); HBM alone would take 12. Rows of 151937, most of which
// have to be shifted, take 53 us at 19 instructions (fp32 65): 48 and 51 when a
// thread's columns followed the memory's grid, which equal beams cannot have.
#include <climits>
#include <type_traits>

#include "kld_internal.h"
#include "kld_packed.cuh"

namespace kld {
namespace {

using packed::neg_inf;
using packed::Type;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCtasPerSm = 4;                // of the selection
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
// Integers in the order of the values (zeros of either sign are one).
__device__ __forceinline__ uint64_t order_key(double x) {
  const uint64_t b = x == 0.0 ? 0ull : static_cast<uint64_t>(__double_as_longlong(x));
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}
// The same of an fp32 value, in 32 bits.
__device__ __forceinline__ uint32_t order_key32(float x) {
  const uint32_t b = x == 0.f ? 0u : __float_as_uint(x);
  return (b >> 31) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value32(uint32_t k) {
  return __uint_as_float((k >> 31) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ double key_value(uint64_t k) {
  const uint64_t b = (k >> 63) ? (k & 0x7fffffffffffffffull) : ~k;
  return __longlong_as_double(static_cast<long long>(b));
}

// A lower bound of the k-th largest value of the CTA from one value per
// thread: the k-th largest of every warp's `each` (<= 32) largest, -inf when
// those are fewer than k.
struct BoundShared {
  float cand[kWarps * 32];
  float bound;
};
__device__ __forceinline__ float block_bound(float x, int k, int each, BoundShared& sh) {
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const float none = neg_inf();
  for (int i = 0; i < each; ++i) {
    const float m = warp_max(x);
    const unsigned who = __ballot_sync(0xffffffffu, x == m);
    if (lane == __ffs(static_cast<int>(who)) - 1) {
      sh.cand[warp * each + i] = x;
      x = none;
    }
  }
  __syncthreads();
  const int n = kWarps * each;  // callers give each >= k / kWarps
  if (tid < n) {
    const float v = sh.cand[tid];
    int above = 0;
#pragma unroll 8
    for (int i = 0; i < n; ++i) above += sh.cand[i] > v || (sh.cand[i] == v && i < tid) ? 1 : 0;
    if (above == k - 1) sh.bound = v;
  }
  __syncthreads();
  return sh.bound;
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
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const uint64_t o = l.key[i];
      const uint32_t j = l.idx[i];
      c += static_cast<int>(o > key[e]) + static_cast<int>(o == key[e] && j < idx[e]);
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
  float4* sums;             // [rows * parts]: frame m, sum of e^(x - m), largest entry, entries (bits)
  float2* entries;          // [rows * parts][cap]: value, column (bits)
  unsigned* tickets;        // [groups], zero between launches
  uint32_t* flags;
  // outputs [groups, k]
  float* out_scores;
  int32_t* out_tokens;
  int32_t* out_parents;
};

constexpr int kMaxLists = kBeamMaxLists;

struct SelectShared {
  List list;
  BoundShared bound;
  float F[kWarps], S[kWarps];
  int last;
  // the merge
  float m[KLD_BEAM_MAX_BEAMS];      // lse = m + lns
  double lns[KLD_BEAM_MAX_BEAMS];   // NaN: the beam offers nothing
  float score[KLD_BEAM_MAX_BEAMS];
  int chosen;
  float top[kMaxLists];             // the lists' largest entries
  uint16_t count[kMaxLists];
  uint32_t choice[kMaxLists];       // beam << 16 | list
};

// Column j of a row, -inf from j1 on.
template <int DT>
__device__ __forceinline__ float value_at(const char* row, int64_t j, int64_t j1) {
  return j < j1 ? Type<DT>::load(row + j * Type<DT>::kBytes) : neg_inf();
}

// A row and what its reading needs: the bytes it starts past a 16-byte
// boundary, and the matrix's first and last byte (whole 16-byte vectors that
// lie between them may be read).
struct Row {
  const char* p;
  uint32_t mis;
  const char *begin, *end;
};

// A tile: each thread NV vectors of E columns, a warp's NV * 32 vectors one
// after another from the row's start on. The columns that a thread sums do not
// depend on where the row lies, so equal rows have equal sums (on the memory's
// own grid their log-sum-exps differed by 1e-8, which broke ties between
// beams).
template <int DT>
struct Tile {
  static constexpr int E = 16 / Type<DT>::kBytes;
  static constexpr int NV = kPer / E;
  uint32_t w[4 * NV];
  // A thread's first vector of the tile; the others follow 32 apart.
  __device__ __forceinline__ static int first() {
    return static_cast<int>(threadIdx.x >> 5) * (32 * NV) + static_cast<int>(threadIdx.x & 31);
  }
  __device__ static int64_t column(int64_t j0, int k) { return j0 + (first() + k / E * 32) * E + k % E; }
  // The lane's maximum, and the sum of e^(lambda (x - F)) (16-bit values are
  // never widened for either).
  __device__ __forceinline__ float max() const {
    if constexpr (DT == KLD_F32) {
      float m = __uint_as_float(w[0]);
#pragma unroll
      for (int k = 1; k < 16; ++k) m = fmaxf(m, __uint_as_float(w[k]));
      return m;
    } else {
      uint32_t m = w[0];
#pragma unroll
      for (int k = 1; k < 8; ++k) {
        if constexpr (DT == KLD_BF16)
          asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(w[k]));
        else
          asm("max.f16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(w[k]));
      }
      return fmaxf(lo(m), hi(m));
    }
  }
  __device__ __forceinline__ static float lo(uint32_t x) {
    if constexpr (DT == KLD_BF16) return __uint_as_float(x << 16);
    else return __half2float(__ushort_as_half(static_cast<unsigned short>(x & 0xffffu)));
  }
  __device__ __forceinline__ static float hi(uint32_t x) {
    if constexpr (DT == KLD_BF16) return __uint_as_float(x & 0xffff0000u);
    else return __half2float(__ushort_as_half(static_cast<unsigned short>(x >> 16)));
  }
  __device__ __forceinline__ float sum(float F) const {
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float d0, d1;
      if constexpr (DT == KLD_F32) {
        d0 = __uint_as_float(w[2 * k]) - F;
        d1 = __uint_as_float(w[2 * k + 1]) - F;
      } else if constexpr (DT == KLD_BF16) {
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tsub.f32.bf16 %0, lo, %3;\n\t"
            "sub.f32.bf16 %1, hi, %3;\n\t}"
            : "=f"(d0), "=f"(d1) : "r"(w[k]), "f"(F));
      } else {
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tsub.f32.f16 %0, lo, %3;\n\t"
            "sub.f32.f16 %1, hi, %3;\n\t}"
            : "=f"(d0), "=f"(d1) : "r"(w[k]), "f"(F));
      }
      s0 += ex2(d0 * kL);
      s1 += ex2(d1 * kL);
    }
    return s0 + s1;
  }
  __device__ __forceinline__ float value(int k) const {
    if constexpr (DT == KLD_F32) return __uint_as_float(w[k]);
    else return (k & 1) ? hi(w[k >> 1]) : lo(w[k >> 1]);
  }
  // Bits of the elements that are >= T and above -inf.
  __device__ __forceinline__ unsigned at_least(float T) const {
    unsigned hits = 0u;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const float x = value(k);
      hits |= x >= T && x > neg_inf() ? 1u << k : 0u;
    }
    return hits;
  }
};

// A tile on its way. Rows that start inside a 16-byte vector (kShift) are
// loaded as the aligned vectors that hold their first bytes, and shifted when
// the tile is taken: a lane gets the words it lacks from the next lane, the
// last one from the warp's next vector. (Loading two vectors for each one and
// shifting at once, with the wait that this brings: 32x8x151937 bf16 58 us,
// fp32 66.)
template <int DT, bool kShift>
struct Ahead {
  using T = Tile<DT>;
  static constexpr int NV = T::NV, E = T::E;
  uint32_t w[4 * NV + (kShift ? 4 : 0)];
  bool raw;  // not shifted yet

  // Columns [j0, j0 + tile) of the row, -inf from j1 on.
  __device__ __forceinline__ void load(const Row& row, int64_t j0, int64_t j1) {
    constexpr int64_t kCols = static_cast<int64_t>(kThreads) * kPer;
    const char* tile = row.p + j0 * Type<DT>::kBytes;
    const char* at = tile + T::first() * 16;
    raw = false;
    if (j0 + kCols <= j1) {  // the whole tile, for all threads
      if constexpr (!kShift) {
#pragma unroll
        for (int v = 0; v < NV; ++v) vector(at + v * 512, v);
        return;
      } else if (tile - row.mis >= row.begin && tile + kThreads * NV * 16 + 16 - row.mis <= row.end) {
        at -= row.mis;
#pragma unroll
        for (int v = 0; v < NV; ++v) vector(at + v * 512, v);
        if ((threadIdx.x & 31) == 0) vector(at + NV * 512, NV);
        raw = true;
        return;
      }
    }
    // A row's last tile, and the matrix's first when it starts inside a vector.
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t j = T::column(j0, v * E);
      const char* p = at + v * 512;
      if (j + E <= j1 && !kShift) {
        vector(p, v);
      } else if (kShift && j + E <= j1 && p - row.mis >= row.begin && p + 32 - row.mis <= row.end) {
        uint32_t x[8];
        *reinterpret_cast<uint4*>(x) = __ldg(reinterpret_cast<const uint4*>(p - row.mis));
        *reinterpret_cast<uint4*>(x + 4) = __ldg(reinterpret_cast<const uint4*>(p - row.mis) + 1);
        packed::shift_bytes<4, DT == KLD_F32>(x, row.mis);
#pragma unroll
        for (int k = 0; k < 4; ++k) w[4 * v + k] = x[k];
      } else {
        float y[E];
#pragma unroll
        for (int k = 0; k < E; ++k) y[k] = value_at<DT>(row.p, j + k, j1);
        *reinterpret_cast<uint4*>(&w[4 * v]) = Type<DT>::vec(y);
      }
    }
  }
  __device__ __forceinline__ void vector(const char* p, int v) {
    *reinterpret_cast<uint4*>(&w[4 * v]) = __ldcs(reinterpret_cast<const uint4*>(p));
  }
  // The tile in place (the whole warp together; mis and raw are the CTA's).
  __device__ __forceinline__ void take(T& t, uint32_t mis) const {
    if (kShift && raw) {
      switch (mis >> 2) {
        case 0: return rotate<0>(t, mis);
        case 1: return rotate<1>(t, mis);
        case 2: return rotate<2>(t, mis);
        default: return rotate<3>(t, mis);
      }
    }
#pragma unroll
    for (int k = 0; k < 4 * NV; ++k) t.w[k] = w[k];
  }
  // Words kWords on, and half a word more where mis has one.
  template <int kWords>
  __device__ __forceinline__ void rotate(T& t, uint32_t mis) const {
    constexpr bool kHalf = DT != KLD_F32;
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const uint32_t bits = (mis & 3u) * 8u;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      uint32_t x[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = w[4 * v + k];
#pragma unroll
      for (int k = 0; k < kWords + (kHalf ? 1 : 0); ++k) {
        const uint32_t give = lane == 0 ? w[kShift ? 4 * (v + 1) + k : 0] : x[k];
        x[4 + k] = __shfl_sync(0xffffffffu, give, (lane + 1) & 31);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        t.w[4 * v + k] = kHalf ? __funnelshift_r(x[kWords + k], x[kWords + k + 1], bits) : x[kWords + k];
    }
  }
};

// Best k entries of columns [g0, g1), exactly, 256 columns at a time (the path
// of a part whose list overflowed).
template <int DT>
__device__ __noinline__ void slow_part(List& l, const char* row, int64_t g0, int64_t g1, int k) {
  __syncthreads();
  if (threadIdx.x == 0) l.count = 0;
  __syncthreads();
  uint64_t least = 0;  // key of the k-th best once k are known
  bool full = false;
  for (int64_t g = g0; g < g1; g += kThreads) {
    const int64_t j = g + threadIdx.x;
    const float x = value_at<DT>(row, j, g1);
    const uint64_t key = order_key32(x);
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
__global__ void __launch_bounds__(kThreads, kCtasPerSm) kld_beam_select_kernel(const Select a) {
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
    if (!(score < INFINITY) && part % a.parts == 0) atomicOr(a.flags, KLD_BEAM_BAD_SCORE);
  }
  __syncthreads();

  if (live) {
    Row row;
    row.begin = static_cast<const char*>(a.logits);
    row.end = row.begin + ((gridDim.x / a.parts - 1) * a.ld + V) * Type<DT>::kBytes;
    row.p = row.begin + r * a.ld * Type<DT>::kBytes;
    row.mis = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row.p) & 15u);
    const int64_t g0 = (part % a.parts) * a.slice;
    const int64_t g1 = g0 + a.slice < V ? g0 + a.slice : V;
    constexpr int64_t kTile = static_cast<int64_t>(kThreads) * kPer;
    float F = kLowest, T = neg_inf(), top = neg_inf();  // top: of the lane, so far
    // In fp64 from one tile to the next: equal terms round alike, so a long
    // fp32 sum drifts (6e-6 over 64 rows of 2^24 columns of two values).
    double S = 0.0;
    int renew = 0, tile = 0;  // the tile that renews the bound next
    auto pass = [&](auto shift) {
      Ahead<DT, decltype(shift)::value> next;
      if (g0 < g1) next.load(row, g0, g1);
      for (int64_t g = g0; g < g1; g += kTile) {
        Tile<DT> t;
        next.take(t, row.mis);
        if (g + kTile < g1) next.load(row, g + kTile, g1);
        const float m = fmaxf(t.max(), neg_inf());  // -inf where all are NaN
        if (m > F + kRaise) {
          S *= ex2((F - m) * kL);
          F = m;
        }
        S += t.sum(F);
        top = fmaxf(top, m);
        if (tile++ == renew) {
          // after 1, 2, 4, 8, ... tiles: each time about k more entries pass
          T = block_bound(top, a.k, min(32, a.k / kWarps + 5), sh.bound);
          renew = 2 * renew + 1;
        }
        if (m >= T && m > neg_inf()) {
          // Only the columns are noted: taking a value out of 16 registers by
          // its number costs more than reading the few again at the end.
          for (unsigned hits = t.at_least(T); hits; hits &= hits - 1u) {
            const int at = atomicAdd(&sh.list.count, 1);
            if (at < kList)
              sh.list.idx[at] =
                  static_cast<uint32_t>(Tile<DT>::column(g, __ffs(static_cast<int>(hits)) - 1));
          }
        }
      }
    };
    if (row.mis == 0)
      pass(std::false_type{});
    else
      pass(std::true_type{});
    // this CTA's frame and sum
    {
      const float f = warp_max(F);
      float s = static_cast<float>(S) * ex2((F - f) * kL);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == 0) {
        sh.F[warp] = f;
        sh.S[warp] = s;
      }
    }
    __syncthreads();
    if (sh.list.count > kList) {
      slow_part<DT>(sh.list, row.p, g0, g1, a.k);
    } else {
      for (int i = tid; i < sh.list.count; i += kThreads)
        sh.list.key[i] = order_key32(value_at<DT>(row.p, sh.list.idx[i], V));
      __syncthreads();
      if (sh.list.count > a.cap) prune(sh.list, a.k);
    }
    const int n = sh.list.count;
    float2* to = a.entries + part * a.cap;
    top = neg_inf();
    for (int i = tid; i < n; i += kThreads) {
      const float x = key_value32(static_cast<uint32_t>(sh.list.key[i]));
      top = fmaxf(top, x);
      to[i] = make_float2(x, __uint_as_float(sh.list.idx[i]));
    }
    top = warp_max(top);
    __syncthreads();
    if (lane == 0) sh.bound.cand[warp] = top;
    __syncthreads();
    if (tid == 0) {
      float f = sh.F[0];
      for (int w = 1; w < kWarps; ++w) {
        f = fmaxf(f, sh.F[w]);
        top = fmaxf(top, sh.bound.cand[w]);
      }
      double s = 0.0;
      for (int w = 0; w < kWarps; ++w) s += scale_of(sh.F[w], f) * sh.S[w];
      a.sums[part] = make_float4(f, static_cast<float>(s), top, __int_as_float(n));
    }
  } else if (tid == 0) {
    a.sums[part] = make_float4(kLowest, 0.f, neg_inf(), __int_as_float(0));
  }

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
        const float4 v = __ldcg(a.sums + part0 + static_cast<int64_t>(w) * a.parts + p);
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
  if (tid == 0) sh.list.count = sh.chosen = 0;
  const int lists = a.beams * a.parts;
  for (int l = tid; l < lists; l += kThreads) {
    const float4 v = __ldcg(a.sums + part0 + l);
    sh.top[l] = v.z;
    sh.count[l] = static_cast<uint16_t>(__float_as_int(v.w));
  }
  __syncthreads();

  // The score of a value of beam w (NaN: the beam offers nothing).
  auto scored = [&](int w, float x) {
    return static_cast<double>(sh.score[w]) +
           ((static_cast<double>(x) - static_cast<double>(sh.m[w])) - sh.lns[w]);
  };
  // Bounds are taken in fp32, scores rounded down: one instruction a maximum.
  float best = neg_inf();
  // list l goes to warp l % kWarps, so that few lists leave no warp without
  for (int l = warp + kWarps * lane; l < lists; l += kThreads)
    if (sh.count[l]) best = fmaxf(best, __double2float_rd(scored(l / a.parts, sh.top[l])));
  float bound = block_bound(best, a.k, min(32, a.k / kWarps + 5), sh.bound);
  for (int l = tid; l < lists; l += kThreads) {
    const int w = l / a.parts;
    if (sh.count[l] && scored(w, sh.top[l]) >= static_cast<double>(bound))
      sh.choice[atomicAdd(&sh.chosen, 1)] = static_cast<uint32_t>(w) << 16 | static_cast<uint32_t>(l);
  }
  __syncthreads();
  // Entries of the chosen lists, `cap` (a power of two) places each.
  const int shift = 31 - __clz(a.cap);
  const int places = sh.chosen << shift;
  constexpr int kHold = 8;  // places a thread reads at a time
  float2 v[kHold];
  auto read = [&](int e0) {  // places e0 + i * kThreads, all on their way together
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      const int e = e0 + i * kThreads;
      const int l = e < places ? sh.choice[e >> shift] & 0xffffu : 0, at = e & (a.cap - 1);
      const bool have = e < places && at < sh.count[l];
      v[i] = have ? __ldcg(a.entries + (part0 + l) * a.cap + at) : make_float2(neg_inf(), 0.f);
    }
  };
  auto best_of = [&](int e0) {
#pragma unroll
    for (int i = 0; i < kHold; ++i)
      if (v[i].x > neg_inf())
        best = fmaxf(best, __double2float_rd(scored(sh.choice[(e0 + i * kThreads) >> shift] >> 16, v[i].x)));
  };
  auto offer = [&](int e0) {
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      if (v[i].x > neg_inf()) {
        const uint32_t w = sh.choice[(e0 + i * kThreads) >> shift] >> 16;
        const double s = scored(w, v[i].x);
        if (s >= static_cast<double>(bound))
          push(sh.list, order_key(s), w * static_cast<uint32_t>(V) + __float_as_uint(v[i].y));
      }
    }
  };
  constexpr int kStep = kThreads * kHold;
  auto offer_all = [&]() {
    if (places <= kStep) {
      offer(tid);
    } else {
      for (int e = tid; e < places; e += kStep) {
        read(e);
        offer(e);
      }
    }
    __syncthreads();
  };
  if (places <= kStep) read(tid);
  offer_all();
  // Read by all before a finished beam's push may raise it: the branch holds
  // barriers, so every thread has to take the same side of it.
  const int offered = sh.list.count;
  __syncthreads();
  if (offered > kThreads) {
    // Few lists for k, or long ones: a closer bound from their entries (a
    // list holds at least k, or all its part has).
    best = neg_inf();
    if (places <= kStep) {
      best_of(tid);
    } else {
      for (int e = tid; e < places; e += kStep) {
        read(e);
        best_of(e);
      }
    }
    bound = fmaxf(bound, block_bound(best, a.k, min(32, max(a.k, 5)), sh.bound));
    if (tid == 0) sh.list.count = 0;
    __syncthreads();
    offer_all();
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
    // ties at the bound: again, 256 places at a time with exact pruning
    __syncthreads();
    if (tid == 0) sh.list.count = 0;
    __syncthreads();
    offer_finished();
    for (int e = tid; e - tid < places; e += kThreads) {
      const uint32_t c = e < places ? sh.choice[e >> shift] : 0u;
      const int l = c & 0xffffu, at = e & (a.cap - 1);
      if (e < places && at < sh.count[l]) {
        const float2 x = __ldcg(a.entries + (part0 + l) * a.cap + at);
        const double s = scored(c >> 16, x.x);
        if (s >= static_cast<double>(bound))
          push(sh.list, order_key(s), (c >> 16) * static_cast<uint32_t>(V) + __float_as_uint(x.y));
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
  int64_t positions;
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
        n = len <= 0 ? 0 : (len < s.positions ? len * s.unit : n);
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

BeamPlan plan_beam(int64_t rows, int64_t V, int sm_count) {
  // CTAs per row: the number that takes the fewest rounds of CTAs times a
  // CTA's time, in tiles, whose fixed part (the bound, the list, the ticket)
  // is worth about kFixed of them. Measured at 256 rows of 151936 bf16: 8 parts
  // 58 us, 2 parts (one round of 512) 48 us; 8 rows take one tile a CTA.
  // parts * rows stays below kBeamSlices + 2 * rows, the workspace's size.
  constexpr int64_t tile = static_cast<int64_t>(kThreads) * kPer;
  constexpr int64_t kFixed = 4;
  const int64_t slots = static_cast<int64_t>(sm_count) * kCtasPerSm;
  const int64_t tiles = (V + tile - 1) / tile;
  int64_t most = kBeamSlices / rows;
  most = most < 1 ? 1 : (most < tiles ? most : tiles);
  int64_t best = 1, cost = INT64_MAX;
  for (int64_t n = 1; n <= most; ++n) {
    const int64_t per = (tiles + n - 1) / n;
    const int64_t c = (rows * n + slots - 1) / slots * (per + kFixed);
    if (c < cost) {
      cost = c;
      best = per;
    }
  }
  BeamPlan p;
  p.slice = best * tile;
  p.parts = static_cast<int>((tiles + best - 1) / best);
  return p;
}

cudaError_t launch_beam_select(const BeamSelect& b, int sm_count, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(b.groups) * b.beams;
  const BeamPlan p = plan_beam(rows, b.V, sm_count);
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
  // A state's widest vectors, and its CTAs of them.
  auto width_of = [&](const kld_state_t& t) {
    const uint64_t bits = reinterpret_cast<uintptr_t>(t.data) | static_cast<uint64_t>(t.row_stride) |
                          (t.outer > 1 ? static_cast<uint64_t>(t.outer_stride) : 0u);
    int w = widest(beams);
    while (w > 1 && (bits & static_cast<uint64_t>(w - 1))) w >>= 1;
    return w;
  };
  auto spans_of = [&](const kld_state_t& t, int width) {
    const int64_t span = static_cast<int64_t>(kThreads) * kSpan * width;
    return (t.positions * t.position_bytes - 1) / span + 1;
  };
  constexpr int64_t kMostCtas = 0x7fffffff;
  for (int i = 0; i < n; ++i) {  // refused before any is moved
    const kld_state_t& t = states[i];
    if (t.positions * t.position_bytes == 0 || t.outer == 0) continue;
    if (spans_of(t, width_of(t)) > kMostCtas / t.outer / groups) return cudaErrorInvalidConfiguration;
  }
  // One launch per vector width (and per kStatesPerLaunch states).
  for (int width = 16; width >= 1; width >>= 1) {
    Reorder a;
    a.n = 0;
    a.beams = beams;
    a.parents = parents;
    a.lengths = lengths;
    a.flags = flags;
    int64_t grid = 0;
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
      if (width_of(t) != width) continue;
      StateDesc d;
      d.p = static_cast<char*>(t.data);
      d.row_stride = t.row_stride;
      d.outer_stride = t.outer_stride;
      d.run = run;
      d.unit = t.timed ? t.position_bytes : 0;
      d.positions = t.positions;
      d.outer = static_cast<int32_t>(t.outer);
      d.spans = static_cast<uint32_t>(spans_of(t, width));
      const int64_t ctas = static_cast<int64_t>(d.spans) * t.outer * groups;
      if (a.n == kStatesPerLaunch || grid + ctas > kMostCtas) {
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
