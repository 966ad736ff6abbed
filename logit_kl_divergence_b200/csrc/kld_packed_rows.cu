// kld_packed_rows.cu -- the statistic and the gradient of KL(P_base || P_quant)
// with the base rows read from an 8-bit logit checkpoint (kld_packed.cuh) and
// the quant rows dense (fp32, bf16, f16) or from a checkpoint of their own.
//
// The sums are those of the row pass (kld_rows_kernel.cuh, whose log-ratio,
// polynomial and packed-pair helpers are used here): with L = log2(e), an
// integer frame F near the base row's maximum, a centre K and
// x_j = q_j - b_j + K,
//   e_j = 2^(b_j L - F),  S = sum e_j,  A = sum e_j x_j,
//   C = sum e_j (e^x_j - 1 - x_j),  B = A + C = sum e_j (e^x_j - 1),
//   KL = -A/S + log1p(B/S),  sum_j e^q_j = (S + B) 2^F e^-K,
//   grad_j = scale * (softmax(q)_j - softmax(b)_j).
// One exponential an element; e^x - 1 - x is x^2 times a polynomial for
// |x| <= 2.5 (two degrees by the warp's largest |x|). Steps of a warp that hold
// a larger or non-finite x take a second exponential, h_j = e_j e^x_j, and sum
// it apart (Q, with their e in D), so B = A + C over the others plus Q - D.
// Nothing of the size of KL is got by subtracting rounded exponentials, so
// rows that are nearly equal or nearly one-hot keep their accuracy, and so do
// rows whose two distributions hardly meet. F and K belong to a
// warp and move only when a value exceeds the maximum they were set at by
// more than four nats. Sums run in fp32 over a lane's part of the row (a few
// hundred terms) and its warp, in fp64 from there on.
//
// One read of the logits for both passes. A row belongs to a thread-block
// cluster of 1, 2, 4 or 8 CTAs, each taking a run of its 512-column chunks;
// a warp streams its chunks through shared-memory slots of its own with
// cp.async (every global read whole 16-byte vectors in order). After the
// sums are merged (every warp leaves its sums in the shared memory of all of
// the cluster's CTAs, one cluster barrier) the gradient pass walks the chunks
// backwards: those still in their slots are not read again, the others come
// back from L2. No wait in this kernel depends on another launch.
//
// Alignment: chunks follow the 16-byte grid of the dense operand (the quant
// rows, else the gradient), so a row that starts `off` elements into a
// vector has its codes shifted by as many bytes (kOff), and the vectors that
// cross the row's ends go element by element.
//
// Rows whose sums are not finite and positive (NaN or +inf, an empty row, a
// base entry above -inf where quant is -inf, magnitudes near the type's
// limit) are done again by slow_row in fp64 from the definitions.
#include <climits>

#include "kld_internal.h"
#include "kld_packed.cuh"
#include "kld_rows_kernel.cuh"

namespace kld {
namespace {
namespace from_packed {

using namespace packed;

constexpr int kFromPack = 3;  // quant operand from a checkpoint
constexpr int kThreads = 128;
constexpr int kCtasPerSm = 5;  // 20 warps of at most 96 registers
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 512;   // columns a warp takes at a time
constexpr int kDepth = 4;     // chunks in flight per warp
constexpr int kMaxCluster = 8;
constexpr float kNoFrame = -1.0e30f;
constexpr uint32_t kExcludedFlags = KLD_ROW_NONFINITE | KLD_ROW_EMPTY;

// ------------------------------------------------------------- small pieces

// 2^d for a whole d <= 0 (0 below the normal range), exactly.
__device__ __forceinline__ double pow2d(float d) {
  return d < -1022.f ? 0.0
                     : __longlong_as_double(static_cast<long long>(static_cast<int>(d) + 1023) << 52);
}
// The type whose quant values stay packed in the sums (see Packed), or 0.
template <int QT>
constexpr int kPacked16 = QT == KLD_BF16 || QT == KLD_F16 ? QT : 0;

// Two values that are of the 16-bit type, packed.
template <int QT>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (QT == KLD_BF16) {
    return (__float_as_uint(lo) >> 16) | (__float_as_uint(hi) & 0xffff0000u);
  } else {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
__device__ __forceinline__ float sum_lanes(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_peer(uint32_t local, uint32_t rank, uint32_t word) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(local), "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(word) : "memory");
}

__device__ __forceinline__ void min_peer(uint32_t local, uint32_t rank, uint32_t value) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(local), "r"(rank));
  asm volatile("red.shared::cluster.min.s32 [%0], %1;" ::"r"(a), "r"(value) : "memory");
}

// The operand a kernel argument describes: dense rows, or codes and headers.
struct Operands {
  const uint8_t* bcodes;
  const uint32_t* bheads;
  const void* quant;        // dense [N, V], or codes [N, nb * 128]
  const uint32_t* qheads;   // headers of packed quant rows
  const int32_t* tok;       // nullable
  int64_t N, V, nb;
};
struct Outputs {
  kld_row_t* rows;
  double* kld;      // per-row copies, each nullable
  double* nll;
  int32_t* amax_b;
  int32_t* amax_q;
  void* grad;       // nullable: statistic only
  float scale;
};

// Quant operand traits: bytes of one element, elements of a lane's
// contiguous group and groups of a lane's 16 columns of a chunk.
template <int QT>
struct Quant {
  static constexpr int kBytes = QT == KLD_F32 ? 4 : (QT == kFromPack ? 1 : 2);
  static constexpr int kGroup = QT == KLD_F32 ? 4 : 8;
  static constexpr int kGroups = 16 / kGroup;
};
// A chunk's slot in shared memory: the codes and their blocks' headers (from
// 16 codes and one block before the chunk on when shifted), and the quant
// operand likewise.
constexpr int kCodeBytes = kChunk + 16;
constexpr int kHeadBytes = 32;
template <int QT>
struct Slot {
  static constexpr int kHeads = kCodeBytes;
  static constexpr int kQuant = kCodeBytes + kHeadBytes;
  static constexpr int kBytes =
      kQuant + (QT == kFromPack ? kCodeBytes + kHeadBytes : kChunk * Quant<QT>::kBytes);
};

struct RowPtr {
  const uint8_t* bcodes;
  const uint32_t* bheads;
  const char* quant;        // dense row, or codes
  const uint32_t* qheads;
  int off;                  // columns before the row in its first 16-byte vector
};

// What a lane copies of chunk 0; chunk c lies c * (bytes of a chunk) further.
struct LanePtr {
  const uint8_t* bcodes;
  const uint32_t* bheads;
  const char* quant;       // dense values, or codes
  const uint32_t* qheads;
};
template <int QT, bool kOff>
__device__ __forceinline__ LanePtr lane_ptr(const RowPtr& rp, int lane) {
  LanePtr p;
  const int64_t at = static_cast<int64_t>(lane - (kOff ? 1 : 0)) * 16;
  p.bcodes = rp.bcodes + at;
  p.bheads = rp.bheads + lane - (kOff ? 1 : 0);
  p.qheads = nullptr;
  if (QT == kFromPack) {
    p.quant = rp.quant + at;
    p.qheads = rp.qheads + lane - (kOff ? 1 : 0);
  } else {
    p.quant = rp.quant + (lane * 16 - (kOff ? rp.off * Quant<QT>::kBytes : 0));
  }
  return p;
}

// Starts the copies of chunk c into a slot (all lanes; one commit group is
// the caller's). inner: everything the chunk's copies read lies inside the
// row's buffers; otherwise each copy is checked.
template <int QT, bool kOff>
__device__ __forceinline__ void fetch(const LanePtr& p, const RowPtr& rp, int64_t V, int64_t nb,
                                      int c, bool inner, uint32_t slot, int lane) {
  constexpr int kHeadsRead = kOff ? 5 : 4;
  constexpr int kVecs = kChunk * Quant<QT>::kBytes / 512;  // 16-byte vectors a lane copies of dense rows
  const uint8_t* bc = p.bcodes + static_cast<int64_t>(c) * kChunk;
  const uint32_t* bh = p.bheads + static_cast<int64_t>(c) * (kChunk / kBlock);
  const char* qc = p.quant + static_cast<int64_t>(c) * (kChunk * Quant<QT>::kBytes);
  const uint32_t* qh = QT == kFromPack ? p.qheads + static_cast<int64_t>(c) * (kChunk / kBlock) : nullptr;
  const uint32_t q = slot + Slot<QT>::kQuant;
  if (inner) {
    copy16(slot + lane * 16, bc);
    if (kOff && lane == 0) copy16(slot + 512, bc + 512);
    if (lane < kHeadsRead) {
      copy4(slot + Slot<QT>::kHeads + lane * 4, bh);
      if (QT == kFromPack) copy4(q + kCodeBytes + lane * 4, qh);
    }
    if (QT == kFromPack) {
      copy16(q + lane * 16, qc);
      if (kOff && lane == 0) copy16(q + 512, qc + 512);
    } else {
#pragma unroll
      for (int k = 0; k < kVecs; ++k) copy16(q + k * 512 + lane * 16, qc + k * 512);
    }
    return;
  }
  const int64_t coded = nb * kBlock;
  const int64_t at = static_cast<int64_t>(c) * kChunk + (lane - (kOff ? 1 : 0)) * 16;
  const bool here = at >= 0 && at < coded, tail = kOff && lane == 0 && at + 512 < coded;
  if (here) copy16(slot + lane * 16, bc);
  if (tail) copy16(slot + 512, bc + 512);
  const int64_t h = static_cast<int64_t>(c) * (kChunk / kBlock) + lane - (kOff ? 1 : 0);
  if (lane < kHeadsRead && h >= 0 && h < nb) {
    copy4(slot + Slot<QT>::kHeads + lane * 4, bh);
    if (QT == kFromPack) copy4(q + kCodeBytes + lane * 4, qh);
  }
  if (QT == kFromPack) {
    if (here) copy16(q + lane * 16, qc);
    if (tail) copy16(q + 512, qc + 512);
  } else {
    constexpr int E = 16 / Quant<QT>::kBytes;
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int64_t j = static_cast<int64_t>(c) * kChunk + (k * 32 + lane) * E - (kOff ? rp.off : 0);
      if (j >= 0 && j + E <= V) copy16(q + k * 512 + lane * 16, qc + k * 512);
    }
  }
}

// G (4 or 8) values of a checkpoint row from its slot: `at` is the first
// column's offset in the chunk's code grid (at least -off for kOff). Blocks
// with masks or bad values (bit 8 of the headers, gathered in `special`) give
// wrong values unless kMasks.
template <int G, bool kOff, bool kMasks>
__device__ __forceinline__ void slot_values(const unsigned char* codes, const uint32_t* heads,
                                            int at, uint32_t& special, float* o) {
  uint32_t w[G / 4 + 1];
  if (!kOff) {
    if (G == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(codes + at);
      w[0] = v.x;
      w[G / 4 - 1] = v.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(codes + at);
    }
  } else {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(codes + 16 + (at & ~3));
#pragma unroll
    for (int k = 0; k <= G / 4; ++k) w[k] = p[k];
    const uint32_t bits = (at & 3) * 8;
#pragma unroll
    for (int k = 0; k < G / 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], bits);
  }
  const uint32_t* h = heads + (at >> 7) + (kOff ? 1 : 0);
  const uint32_t h0 = h[0];
  const int cut = kOff ? kBlock - (at & (kBlock - 1)) : G;  // columns of the first block
  const uint32_t h1 = kOff && cut < G ? h[1] : h0;          // a group may cross into the next one
  special |= h0 | h1;
  if (kMasks) {
    const Scale s = scale_of(h0), t = scale_of(h1);
#pragma unroll
    for (int k = 0; k < G / 4; ++k) decode4(w[k], s, o + 4 * k);
    if (kOff && cut < G) {
      float y[G];
#pragma unroll
      for (int k = 0; k < G / 4; ++k) decode4(w[k], t, y + 4 * k);
#pragma unroll
      for (int k = 0; k < G; ++k)
        if (k >= cut) o[k] = y[k];
    }
  } else {
    float s0, f0, s1, f1;
    plain_scale(h0, s0, f0);
    if (kOff) plain_scale(h1, s1, f1);
#pragma unroll
    for (int k = 0; k < G; k += 2) {
      const uint32_t x = w[k / 4];
      const float m0 = (k & 2) ? magic_byte<2>(x) : magic_byte<0>(x);
      const float m1 = (k & 2) ? magic_byte<3>(x) : magic_byte<1>(x);
      if (kOff) {
        o[k] = fmaf(m0, k < cut ? s0 : s1, k < cut ? f0 : f1);
        o[k + 1] = fmaf(m1, k + 1 < cut ? s0 : s1, k + 1 < cut ? f0 : f1);
      } else {
        upk(fma2(pk(m0, m1), splat(s0), splat(f0)), o[k], o[k + 1]);
      }
    }
  }
}

// One value of each operand by plain loads.
template <int QT>
__device__ __forceinline__ float base_at(const RowPtr& rp, int64_t j) {
  return decode1(rp.bcodes[j], __ldg(rp.bheads + j / kBlock));
}
template <int QT>
__device__ __forceinline__ float quant_at(const RowPtr& rp, int64_t j) {
  if constexpr (QT == kFromPack)
    return decode1(static_cast<uint8_t>(rp.quant[j]), __ldg(rp.qheads + j / kBlock));
  else
    return Type<QT>::load(rp.quant + j * Quant<QT>::kBytes);
}

// A lane's column of its group g in a chunk, from the chunk's start.
template <int QT>
__device__ __forceinline__ int group_col(int g, int lane) {
  return (g * 32 + lane) * Quant<QT>::kGroup;
}

// A lane's 16 columns of a chunk that lies inside the row: base values, and
// quant values (packed ones for the 16-bit types), wrong where a block is
// special (bit 8 of the result).
template <int QT, bool kOff>
__device__ __forceinline__ uint32_t step_plain(int off, const unsigned char* slot, int lane,
                                               float* b, float* q, uint32_t* qw) {
  constexpr int G = Quant<QT>::kGroup;
  uint32_t special = 0u;
#pragma unroll
  for (int g = 0; g < Quant<QT>::kGroups; ++g) {
    const int at = group_col<QT>(g, lane) - (kOff ? off : 0);
    slot_values<G, kOff, false>(slot, reinterpret_cast<const uint32_t*>(slot + Slot<QT>::kHeads),
                                at, special, b + g * G);
    const unsigned char* qs = slot + Slot<QT>::kQuant;
    if constexpr (QT == kFromPack) {
      slot_values<G, kOff, false>(qs, reinterpret_cast<const uint32_t*>(qs + kCodeBytes), at,
                                  special, q + g * G);
    } else {
      const uint4 w = *reinterpret_cast<const uint4*>(qs + group_col<QT>(g, lane) * Quant<QT>::kBytes);
      if constexpr (QT == KLD_F32) {
        q[4 * g] = __uint_as_float(w.x);
        q[4 * g + 1] = __uint_as_float(w.y);
        q[4 * g + 2] = __uint_as_float(w.z);
        q[4 * g + 3] = __uint_as_float(w.w);
      } else {
        qw[4 * g] = w.x;
        qw[4 * g + 1] = w.y;
        qw[4 * g + 2] = w.z;
        qw[4 * g + 3] = w.w;
      }
    }
  }
  return special;
}

// The same for any chunk, quant values unpacked: masks and bad blocks read as
// such, groups that cross the row's ends element by element, -inf outside.
template <int QT, bool kOff>
__device__ __forceinline__ void step_general(const RowPtr& rp, int64_t V, int c,
                                             const unsigned char* slot, int lane, float* b,
                                             float* q) {
  constexpr int G = Quant<QT>::kGroup;
  const int off = kOff ? rp.off : 0;
  uint32_t special = 0u;
#pragma unroll
  for (int g = 0; g < Quant<QT>::kGroups; ++g) {
    const int at = group_col<QT>(g, lane) - off;
    const int64_t j = static_cast<int64_t>(c) * kChunk + at;
    float* bg = b + g * G;
    float* qg = q + g * G;
    if (j >= 0 && j + G <= V) {
      slot_values<G, kOff, true>(slot, reinterpret_cast<const uint32_t*>(slot + Slot<QT>::kHeads),
                                 at, special, bg);
      const unsigned char* qs = slot + Slot<QT>::kQuant;
      if constexpr (QT == kFromPack) {
        slot_values<G, kOff, true>(qs, reinterpret_cast<const uint32_t*>(qs + kCodeBytes), at,
                                   special, qg);
      } else {
        const uint4 w = *reinterpret_cast<const uint4*>(qs + (at + off) * Quant<QT>::kBytes);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < G; ++k)
          qg[k] = QT == KLD_F32 ? __uint_as_float(ww[k & 3]) : q_el<kPacked16<QT>>(nullptr, ww, k);
      }
    } else {
#pragma unroll
      for (int k = 0; k < G; ++k) {
        const bool in = j + k >= 0 && j + k < V;
        bg[k] = in ? base_at<QT>(rp, j + k) : neg_inf();
        qg[k] = in ? quant_at<QT>(rp, j + k) : neg_inf();
      }
    }
  }
}

// --------------------------------------------------------------- row state

// A warp's sums, as they are merged.
struct Part {
  float F, K;      // frame (a whole number; kNoFrame before any value), centre
  float S, A, C;   // over the polynomial steps
  float D, E, Q;   // over the others: sums of e, e x, h
  float mb, mq;    // maxima of its columns
};
constexpr int kPartWords = 10;
static_assert(sizeof(Part) == 4 * kPartWords, "Part is stored word by word");
constexpr int kMaxParts = kMaxCluster * kWarps;

// The row's merged sums and what the gradient pass needs of them.
struct Total {
  double S, A, B, q;  // sum of e, e x, e (e^x - 1), e e^x over all steps
  float F, K;
  float mb, mq;
  float Fq;        // frame of the quant row's exponentials
  float cb, cq;    // scale / (their sums in the frames)
  int good;
};

struct Shared {
  Part part[kMaxParts];  // every warp of the cluster, written by its owner
  Total total;
  int ib, iq;            // lowest columns of the maxima (rank 0's are the row's)
  // slow_row: block reductions
  double dsum[kWarps];
  float fmax_[2][kWarps];
  uint32_t flags;
};

// What a lane keeps of its part of the row: its warp's frame and centre
// (uniform), its sums (Part), its maxima and the first chunks they are in.
struct State {
  float F, K, T;  // T: a value above it moves the frame and the centre
  int form;       // order of the log-ratio's roundings (ratio_form)
  float S, A, C, D, E, Q;
  float mb, mq;
  int ib, iq;
};

// Moves a warp's frame to its step's maximum M (um: the lane's own), rebasing
// the lanes' sums exactly in F and by
//   A' = A + d S,  C' = e^d C + (e^d - 1) A + (e^d - 1 - d) S,
//   E' = E + d D,  Q' = e^d Q
// in K (d its change).
template <int QT>
__device__ __forceinline__ void raise(State& s, const float* b, const float* q, const uint32_t* qw,
                                      float um, float M) {
  float qm = 0.f;
#pragma unroll
  for (int k = 15; k >= 0; --k)
    if (b[k] == M) qm = q_el<kPacked16<QT>>(q, qw, k);
  const unsigned who = __ballot_sync(0xffffffffu, um == M);
  qm = __shfl_sync(0xffffffffu, qm, __ffs(static_cast<int>(who)) - 1);
  const float K = fabsf(qm) < INFINITY ? M - qm : s.K;  // a masked or NaN quant entry sets none
  const float F = floorf(M * kLog2e);
  if (s.F != kNoFrame) {
    const float sc = static_cast<float>(pow2d(s.F - F));
    const float d = K - s.K;
    const float lam = static_cast<float>(kLambda);
    const float ld = lam * d;
    float e1, phi;  // e^ld - 1, e^ld - 1 - ld
    if (fabsf(d) <= kTau) {
      phi = d * d * phi_q(d);
      e1 = ld + phi;
    } else {
      e1 = ex2(d * kLog2e) - 1.f;
      phi = e1 - ld;
    }
    s.C = sc * (s.C + e1 * s.C + e1 * lam * s.A + phi * s.S);
    s.A = sc * (s.A + d * s.S);
    s.S *= sc;
    s.E = sc * (s.E + d * s.D);
    s.D *= sc;
    s.Q = sc * (s.Q + e1 * s.Q);
  }
  s.F = F;
  s.K = K;
  s.T = M + kRaiseMargin;
  s.form = ratio_form(M, K);
}

// S += e, A += e x, C += e (e^x - 1 - x) with tier T's polynomial.
template <int T>
__device__ __forceinline__ void add_poly(State& s, const float* b, const f2* x) {
  const f2 L2 = splat(kLog2e), nf = splat(-s.F);
  // Two accumulator sets halve the dependent-add chains.
  f2 S[2] = {splat(0.f), splat(0.f)}, A[2] = {splat(0.f), splat(0.f)}, C[2] = {splat(0.f), splat(0.f)};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float u0, u1;
    upk(fma2(pk(b[2 * k], b[2 * k + 1]), L2, nf), u0, u1);
    const f2 e = pk(ex2(u0), ex2(u1));
    const f2 t = mul2(e, x[k]);
    S[k & 1] = add2(S[k & 1], e);
    A[k & 1] = add2(A[k & 1], t);
    C[k & 1] = fma2(mul2(t, x[k]), phi_q2<T>(x[k]), C[k & 1]);
  }
  float v0, v1;
  upk(add2(S[0], S[1]), v0, v1);
  s.S += v0 + v1;
  upk(add2(A[0], A[1]), v0, v1);
  s.A += v0 + v1;
  upk(add2(C[0], C[1]), v0, v1);
  s.C += v0 + v1;
}

// Adds a chunk's 16 columns of a lane (the whole warp together) to its
// state. Entries whose bit in `valid` is 0 are -inf in both operands (masks,
// columns outside the row): they have weight 0 and take x = 0. i: the
// warp's number of the chunk.
template <int QT>
__device__ __forceinline__ void add_step(State& s, const float* b, const float* q,
                                         const uint32_t* qw, unsigned valid, int i) {
  constexpr int kPk = kPacked16<QT>;
  const float mb = tree_max<16, false>(b);
  float mq;
  if constexpr (kPk != 0) {
    uint32_t m2 = qw[0];
#pragma unroll
    for (int w = 1; w < 8; ++w) m2 = Packed<kPk>::max2(m2, qw[w]);
    mq = fmaxf(Packed<kPk>::lo(m2), Packed<kPk>::hi(m2));
  } else {
    mq = tree_max<16, false>(q);
  }
  if (__any_sync(0xffffffffu, mb > s.T)) raise<QT>(s, b, q, qw, mb, warp_max(mb));
  f2 x[8];
  float ax;
  if (s.form == 0) {
    ax = log_ratios<16, 0, kPk>(b, q, valid, s.K, x, qw);
  } else {
    float y[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) y[k] = q_el<kPk>(q, qw, k);
    ax = s.form == 1 ? log_ratios<16, 1>(b, y, valid, s.K, x) : log_ratios<16, 2>(b, y, valid, s.K, x);
  }
  if (__all_sync(0xffffffffu, ax <= kTauA)) {
    add_poly<0>(s, b, x);
  } else if (__all_sync(0xffffffffu, ax <= kTauB)) {
    add_poly<1>(s, b, x);
  } else if (__all_sync(0xffffffffu, ax <= kTau)) {
    add_poly<2>(s, b, x);
  } else {
    // Large or non-finite log-ratios. A masked base entry has e = 0 and gives
    // its h to Q; x = -inf with a base entry above -inf makes E non-finite,
    // which sends the row to slow_row.
    float D = 0.f, E = 0.f, Q = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float xs[2];
      upk(x[k], xs[0], xs[1]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float bk = b[2 * k + h];
        const float e = ex2(fmaf(bk, kLog2e, -s.F));
        D += e;
        E += bk == neg_inf() ? 0.f : e * xs[h];
        Q += ex2(fmaf(q_el<kPk>(q, qw, 2 * k + h) + s.K, kLog2e, -s.F));
      }
    }
    s.D += D;
    s.E += E;
    s.Q += Q;
  }
  if (mb > s.mb) {
    s.mb = mb;
    s.ib = i;
  }
  if (mq > s.mq) {
    s.mq = mq;
    s.iq = i;
  }
}

// add_step for a chunk that crosses the row's ends or holds masked or bad
// blocks. By value, so that the caller's state stays in registers.
template <int QT, bool kOff>
__device__ __noinline__ State add_general(State s, const RowPtr rp, int64_t V, int c,
                                          const unsigned char* slot, int lane, int i) {
  float b[16], q[16];
  uint32_t qw[8];
  step_general<QT, kOff>(rp, V, c, slot, lane, b, q);
  unsigned valid = 0u;
#pragma unroll
  for (int k = 0; k < 16; ++k)
    if (b[k] != neg_inf() || q[k] != neg_inf()) valid |= 1u << k;
  if constexpr (kPacked16<QT> != 0) {
#pragma unroll
    for (int k = 0; k < 8; ++k) qw[k] = pack16<QT>(q[2 * k], q[2 * k + 1]);
  }
  add_step<QT>(s, b, q, qw, valid, i);
  return s;
}

// The parts of a row merged by one warp, in fp64, to the largest frame and
// the centre of the part that holds the row's maximum.
__device__ __noinline__ void merge(Shared& sh, int parts, float scale) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  float F = kNoFrame, mb = neg_inf(), mq = neg_inf();
  for (int i = lane; i < parts; i += 32) {
    F = fmaxf(F, sh.part[i].F);
    mb = fmaxf(mb, sh.part[i].mb);
    mq = fmaxf(mq, sh.part[i].mq);
  }
  F = warp_max(F);
  mb = warp_max(mb);
  mq = warp_max(mq);
  int best = INT_MAX;
  for (int i = lane; i < parts; i += 32)
    if (sh.part[i].mb == mb) best = min(best, i);
  best = __reduce_min_sync(0xffffffffu, best);
  const float K = best < parts ? sh.part[best].K : 0.f;
  double S = 0.0, A = 0.0, C = 0.0, D = 0.0, E = 0.0, Q = 0.0;
  for (int i = lane; i < parts; i += 32) {
    const Part p = sh.part[i];
    if (p.S == 0.f && p.D == 0.f && p.E == 0.f && p.Q == 0.f) continue;
    const double sc = pow2d(p.F - F);
    const double d = static_cast<double>(K) - static_cast<double>(p.K);
    double e1 = 0.0, phi = 0.0;
    if (d != 0.0) {
      e1 = expm1(kLambda * d);
      phi = e1 - kLambda * d;
    }
    const double s = p.S, a = p.A, c = p.C;
    S += sc * s;
    A += sc * (a + d * s);
    C += sc * (c + e1 * c + e1 * kLambda * a + phi * s);
    D += sc * p.D;
    E += sc * (p.E + d * p.D);
    Q += sc * (p.Q + e1 * p.Q);
  }
  S = warp_sum(S);
  A = warp_sum(A);
  C = warp_sum(C);
  D = warp_sum(D);
  E = warp_sum(E);
  Q = warp_sum(Q);
  if (lane == 0) {
    Total t;
    t.S = S + D;
    t.A = A + E;
    t.B = kLambda * A + C + (Q - D);
    t.q = S + (kLambda * A + C) + Q;
    t.F = F;
    t.K = K;
    t.mb = mb;
    t.mq = mq;
    t.good = t.S > 0.0 && t.S < 1e300 && fabs(t.A) < 1e300 && t.q > 0.0 && t.q < 1e300 &&
             fabsf(F) < 1e6f && fabsf(K) < 1e6f;
    // sum_j 2^(q_j L) = t.q 2^(F - K L): its whole part is the quant row's frame
    const double at = static_cast<double>(F) - static_cast<double>(K) * kLog2eD;
    t.Fq = static_cast<float>(floor(at));
    t.cb = static_cast<float>(scale / t.S);
    t.cq = static_cast<float>(scale / (t.q * exp2(at - floor(at))));
    sh.total = t;
  }
}

// The row from its definitions in fp64, by one whole CTA (every CTA of the
// row's cluster does it for itself): for rows the fp32 sums cannot hold.
struct Slow {
  float mb, mq;
  double Sb, Sq, kl;
  uint32_t flags;
};
__device__ double block_sum(Shared& sh, double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.dsum[threadIdx.x >> 5] = x;
  __syncthreads();
  double s = 0.0;
  for (int w = 0; w < kWarps; ++w) s += sh.dsum[w];
  return s;
}
template <int QT>
__device__ __noinline__ void slow_row(Shared& sh, const RowPtr& rp, int64_t V, Slow& out) {
  const int tid = static_cast<int>(threadIdx.x);
  if (tid == 0) sh.flags = 0u;
  __syncthreads();
  float mb = neg_inf(), mq = neg_inf();
  uint32_t f = 0u;
  for (int64_t j = tid; j < V; j += kThreads) {
    const float b = base_at<QT>(rp, j), q = quant_at<QT>(rp, j);
    if (!(b < INFINITY) || !(q < INFINITY)) f |= KLD_ROW_NONFINITE;  // NaN or +inf
    if (b > neg_inf() && q == neg_inf()) f |= KLD_ROW_INF_KL;
    mb = fmaxf(mb, b);
    mq = fmaxf(mq, q);
  }
  mb = warp_max(mb);
  mq = warp_max(mq);
  if (f) atomicOr(&sh.flags, f);
  if ((tid & 31) == 0) {
    sh.fmax_[0][tid >> 5] = mb;
    sh.fmax_[1][tid >> 5] = mq;
  }
  __syncthreads();
  for (int w = 0; w < kWarps; ++w) {
    mb = fmaxf(mb, sh.fmax_[0][w]);
    mq = fmaxf(mq, sh.fmax_[1][w]);
  }
  f = sh.flags;
  if (f & KLD_ROW_NONFINITE)
    f = KLD_ROW_NONFINITE;
  else if (mb == neg_inf() || mq == neg_inf())
    f = KLD_ROW_EMPTY;
  double sb = 0.0, sq = 0.0, a = 0.0;
  if (!(f & kExcludedFlags)) {
    for (int64_t j = tid; j < V; j += kThreads) {
      const double b = static_cast<double>(base_at<QT>(rp, j)) - mb;
      const double q = static_cast<double>(quant_at<QT>(rp, j)) - mq;
      const double e = exp(b);
      sb += e;
      sq += exp(q);
      if (b > -INFINITY && q > -INFINITY) a += e * (b - q);
    }
  }
  sb = block_sum(sh, sb);
  sq = block_sum(sh, sq);
  a = block_sum(sh, a);
  out.mb = mb;
  out.mq = mq;
  out.Sb = sb;
  out.Sq = sq;
  out.kl = (f & KLD_ROW_INF_KL) ? INFINITY : a / sb - log(sb) + log(sq);
  out.flags = f;
}

// Gradient of columns [j0, j1) of a row slow_row has done (zero on excluded
// rows), one element a thread.
template <int QT, int OT>
__device__ __noinline__ void slow_grad(const RowPtr& rp, int64_t j0, int64_t j1, const Slow& s,
                                       char* grow, float scale) {
  const float cb = static_cast<float>(1.0 / s.Sb), cq = static_cast<float>(1.0 / s.Sq);
  for (int64_t j = j0 + threadIdx.x; j < j1; j += kThreads) {
    float g = 0.f;
    if (!(s.flags & kExcludedFlags)) {
      const float p = __fmul_rn(ex2((base_at<QT>(rp, j) - s.mb) * kLog2e), cb);
      const float r = __fmul_rn(ex2((quant_at<QT>(rp, j) - s.mq) * kLog2e), cq);
      g = __fmul_rn(scale, __fsub_rn(r, p));
    }
    Type<OT>::store(grow + j * Type<OT>::kBytes, g);
  }
}

// The row's record (and its per-field copies), by one thread. ln_b, ln_q:
// ln sum e^(lam (x - m)) of the two rows, m their maxima.
template <int QT>
__device__ void write_row(const Operands& in, const Outputs& out, const RowPtr& rp, int64_t r,
                          double kl, double lam, float mb, float mq, double ln_b, double ln_q,
                          int ib, int iq, uint32_t flags) {
  const double nan = __longlong_as_double(0x7ff8000000000000ll);
  kld_row_t rec;
  rec.kld = rec.nll = rec.nll_base = nan;
  rec.argmax_base = rec.argmax_quant = -1;
  float dp = __int_as_float(0x7fc00000);
  const bool ok = !(flags & kExcludedFlags);
  if (ok) {
    rec.kld = kl;
    rec.argmax_base = ib;
    rec.argmax_quant = iq;
  }
  if (in.tok) {
    const int32_t t = __ldg(in.tok + r);
    if (t < 0 || t >= in.V) {
      flags |= KLD_ROW_BAD_TOKEN;
    } else if (ok) {
      const float b = base_at<QT>(rp, t), q = quant_at<QT>(rp, t);
      rec.nll = ln_q + lam * (static_cast<double>(mq) - static_cast<double>(q));
      rec.nll_base = ln_b + lam * (static_cast<double>(mb) - static_cast<double>(b));
      if (q == neg_inf()) flags |= KLD_ROW_INF_NLL;
      if (b == neg_inf()) flags |= KLD_ROW_INF_NLL_BASE;
      dp = static_cast<float>(exp(-rec.nll) - exp(-rec.nll_base));
    }
  }
  rec.flags = flags;
  rec.dp = dp;
  out.rows[r] = rec;
  if (out.kld) out.kld[r] = rec.kld;
  if (out.nll) out.nll[r] = rec.nll;
  if (out.amax_b) out.amax_b[r] = rec.argmax_base;
  if (out.amax_q) out.amax_q[r] = rec.argmax_quant;
}

// A lane's 16 gradient values of the chunk that starts at column j0 of the
// row's grid. check: the chunk may cross the row's ends.
template <int QT, int OT>
__device__ __forceinline__ void store_grad(char* grow, int64_t j0, int64_t V, int lane, bool check,
                                           const float* x) {
  constexpr int G = Quant<QT>::kGroup;
  constexpr int OE = 16 / Type<OT>::kBytes;  // elements of an output vector
  // All of a row's groups lie alike on the 16-byte grid of the output.
  char* at = grow + (j0 + lane * G) * Type<OT>::kBytes;
  const uint32_t mis = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(at)) & 15u;
#pragma unroll
  for (int g = 0; g < Quant<QT>::kGroups; ++g) {
    char* dst = at + g * 32 * G * Type<OT>::kBytes;
    const float* y = x + g * G;
    const int64_t j = j0 + group_col<QT>(g, lane);
    if ((!check || (j >= 0 && j + G <= V)) && (OE <= G ? mis == 0u : (mis & 7u) == 0u)) {
      if (OE <= G) {
#pragma unroll
        for (int k = 0; k < G; k += OE)
          __stcs(reinterpret_cast<uint4*>(dst + k * Type<OT>::kBytes), Type<OT>::vec(y + k));
      } else {
        const float z[8] = {y[0], y[1], y[2], y[3], 0.f, 0.f, 0.f, 0.f};
        const uint4 w = Type<OT>::vec(z);
        __stcs(reinterpret_cast<uint2*>(dst), make_uint2(w.x, w.y));
      }
    } else {
#pragma unroll
      for (int k = 0; k < G; ++k)
        if (j + k >= 0 && j + k < V) Type<OT>::store(dst + k * Type<OT>::kBytes, y[k]);
    }
  }
}

// ------------------------------------------------------------------ kernel

// grid = N * C CTAs, clusters of C = gridDim / N; slots: shared-memory slots
// per warp (>= kDepth).
template <int QT, int OT, bool kOff>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    kld_packed_rows_kernel(const Operands in, const Outputs out, int C, int slots) {
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ Shared sh;
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int64_t r = blockIdx.x / C;
  const int rank = C > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int64_t V = in.V, nb = in.nb;
  if (C > 1) cluster_arrive();  // peers may be written to once all have started
  if (tid == 0) sh.ib = sh.iq = INT_MAX;

  RowPtr rp;
  rp.bcodes = in.bcodes + r * nb * kBlock;
  rp.bheads = in.bheads + r * nb;
  rp.qheads = nullptr;
  char* grow = out.grad ? static_cast<char*>(out.grad) + r * V * Type<OT>::kBytes : nullptr;
  if (QT == kFromPack) {
    rp.quant = static_cast<const char*>(in.quant) + r * nb * kBlock;
    rp.qheads = in.qheads + r * nb;
    rp.off = kOff ? static_cast<int>((reinterpret_cast<uintptr_t>(grow) & 15u) / Type<OT>::kBytes) : 0;
  } else {
    rp.quant = static_cast<const char*>(in.quant) + r * V * Quant<QT>::kBytes;
    rp.off = kOff ? static_cast<int>((reinterpret_cast<uintptr_t>(rp.quant) & 15u) / Quant<QT>::kBytes) : 0;
  }
  const int off = kOff ? rp.off : 0;

  // This CTA's chunks [c0, c1); warp w takes c0 + w + i * kWarps, i < n.
  const int chunks = static_cast<int>((V + off + kChunk - 1) / kChunk);
  const int c0 = static_cast<int>(static_cast<int64_t>(chunks) * rank / C);
  const int c1 = static_cast<int>(static_cast<int64_t>(chunks) * (rank + 1) / C);
  const int n = c0 + warp < c1 ? (c1 - c0 - warp + kWarps - 1) / kWarps : 0;
  // Chunks [in0, in1) lie inside the row (their vectors whole, their headers
  // and shifted codes in the row's buffers).
  const int in0 = kOff ? 1 : 0;
  const int in1 = static_cast<int>((V + off) / kChunk);
  const LanePtr lp = lane_ptr<QT, kOff>(rp, lane);
  unsigned char* my = ring + static_cast<size_t>(warp) * slots * Slot<QT>::kBytes;
  const uint32_t my32 = smem_u32(my);
  const int first = c0 + warp;
  auto inner = [&](int c) { return c >= in0 && c < in1; };
  auto load = [&](int i, int slot) {
    const int c = first + i * kWarps;
    fetch<QT, kOff>(lp, rp, V, nb, c, inner(c), my32 + slot * Slot<QT>::kBytes, lane);
  };

  State st;
  st.F = kNoFrame;
  st.K = 0.f;
  st.T = neg_inf();
  st.form = 0;
  st.S = st.A = st.C = st.D = st.E = st.Q = 0.f;
  st.mb = st.mq = neg_inf();
  st.ib = st.iq = 0;

  // ---- sums
#pragma unroll
  for (int i = 0; i < kDepth; ++i) {
    if (i < n) load(i, i);
    copy_commit();
  }
  int cur = 0, nxt = kDepth == slots ? 0 : kDepth;  // slots of chunks i and i + kDepth
  for (int i = 0; i < n; ++i) {
    copy_wait<kDepth - 1>();
    __syncwarp();
    const int c = first + i * kWarps;
    const unsigned char* slot = my + cur * Slot<QT>::kBytes;
    bool general = !inner(c);
    float b[16], q[16];
    uint32_t qw[8];
    if (!general) {
      const uint32_t special = step_plain<QT, kOff>(off, slot, lane, b, q, qw);
      general = __any_sync(0xffffffffu, (special & 256u) != 0u);
    }
    if (!general)
      add_step<QT>(st, b, q, qw, 0xffffu, i);
    else
      st = add_general<QT, kOff>(st, rp, V, c, slot, lane, i);
    __syncwarp();
    if (i + kDepth < n) load(i + kDepth, nxt);
    copy_commit();
    if (++cur == slots) cur = 0;
    if (++nxt == slots) nxt = 0;
  }

  // ---- merge: lanes, then every warp of the cluster
  {
    Part w;
    w.F = st.F;
    w.K = st.K;
    w.S = sum_lanes(st.S);
    w.A = sum_lanes(st.A);
    w.C = sum_lanes(st.C);
    w.D = sum_lanes(st.D);
    w.E = sum_lanes(st.E);
    w.Q = sum_lanes(st.Q);
    w.mb = warp_max(st.mb);
    w.mq = warp_max(st.mq);
    if (C > 1) cluster_wait();  // every CTA of the cluster has started
    if (lane < C) {             // lane k leaves the part with CTA k
      const uint32_t* words = reinterpret_cast<const uint32_t*>(&w);
      const uint32_t at = smem_u32(&sh.part[rank * kWarps + warp]);
#pragma unroll
      for (int k = 0; k < kPartWords; ++k) {
        if (C > 1)
          store_peer(at + 4 * k, static_cast<uint32_t>(lane), words[k]);
        else
          reinterpret_cast<uint32_t*>(&sh.part[warp])[k] = words[k];
      }
    }
    __syncwarp();
  }
  if (C > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  if (warp == 0) merge(sh, C * kWarps, out.scale);
  __syncthreads();
  // Lowest columns of the row's maxima: the lanes that hold one look through
  // the first chunk in which it appeared; rank 0 collects.
  if (n > 0 && (st.mb == sh.total.mb || st.mq == sh.total.mq)) {
    for (int which = 0; which < 2; ++which) {
      const float m = which ? sh.total.mq : sh.total.mb;
      if ((which ? st.mq : st.mb) != m) continue;
      const int64_t c = first + (which ? st.iq : st.ib) * kWarps;
      for (int k = 0; k < 16; ++k) {
        const int at = group_col<QT>(k / Quant<QT>::kGroup, lane) + k % Quant<QT>::kGroup - off;
        const int64_t j = c * kChunk + at;
        if (j < 0 || j >= V) continue;
        if ((which ? quant_at<QT>(rp, j) : base_at<QT>(rp, j)) == m) {
          if (C > 1)
            min_peer(smem_u32(which ? &sh.iq : &sh.ib), 0u, static_cast<uint32_t>(j));
          else
            atomicMin(which ? &sh.iq : &sh.ib, static_cast<int>(j));
          break;
        }
      }
    }
  }
  if (!sh.total.good) {  // the same in every thread of the cluster
    copy_wait<0>();
    Slow s;
    slow_row<QT>(sh, rp, V, s);
    if (grow) {
      const int64_t j0 = static_cast<int64_t>(c0) * kChunk - off;
      const int64_t j1 = static_cast<int64_t>(c1) * kChunk - off;
      slow_grad<QT, OT>(rp, j0 < 0 ? 0 : j0, j1 < V ? j1 : V, s, grow, out.scale);
    }
    if (C > 1) {
      __syncwarp();
      cluster_arrive();
      cluster_wait();
    }
    __syncthreads();
    if (rank == 0 && tid == 0)
      write_row<QT>(in, out, rp, r, s.kl, 1.0, s.mb, s.mq, log(s.Sb), log(s.Sq), sh.ib, sh.iq,
                    s.flags);
    return;
  }

  // ---- gradient, chunks backwards: the last `slots` of them are still here
  if (grow) {
    const f2 L2 = splat(kLog2e), fb = splat(-sh.total.F), fq = splat(-sh.total.Fq);
    const f2 cb2 = splat(sh.total.cb), cq2 = splat(sh.total.cq), zero2 = splat(0.f);
    cur = n > 0 ? (n - 1) % slots : 0;
    for (int i = n - 1; i >= 0; --i) {
      copy_wait<kDepth - 1>();
      __syncwarp();
      const int c = first + i * kWarps;
      const unsigned char* slot = my + cur * Slot<QT>::kBytes;
      bool general = !inner(c);
      float b[16], q[16];
      uint32_t qw[8];
      if (!general) {
        const uint32_t special = step_plain<QT, kOff>(off, slot, lane, b, q, qw);
        general = __any_sync(0xffffffffu, (special & 256u) != 0u);
        if constexpr (kPacked16<QT> != 0) {
#pragma unroll
          for (int k = 0; k < 16; ++k) q[k] = q_el<kPacked16<QT>>(nullptr, qw, k);
        }
      }
      if (general) step_general<QT, kOff>(rp, V, c, slot, lane, b, q);
#pragma unroll
      for (int k = 0; k < 16; k += 2) {
        float u0, u1, v0, v1;
        upk(fma2(pk(b[k], b[k + 1]), L2, fb), u0, u1);
        upk(fma2(pk(q[k], q[k + 1]), L2, fq), v0, v1);
        // Products rounded apart, so equal rows give exactly zero: as FMAs
        // with zero, since a packed product may be joined with the
        // difference into one FMA (measured: 2.5e-8 p instead of 0).
        const f2 pr = fma2(pk(ex2(u0), ex2(u1)), cb2, zero2);
        const f2 rr = fma2(pk(ex2(v0), ex2(v1)), cq2, zero2);
        upk(sub2(rr, pr), b[k], b[k + 1]);
      }
      store_grad<QT, OT>(grow, static_cast<int64_t>(c) * kChunk - off, V, lane, general, b);
      __syncwarp();
      if (i - slots >= 0) load(i - slots, cur);
      copy_commit();
      if (--cur < 0) cur = slots - 1;
    }
  }
  copy_wait<0>();
  if (C > 1) {
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  }
  __syncthreads();
  if (rank == 0 && tid == 0) {
    const Total& t = sh.total;
    // ln(q / S), by the difference where the rows are close
    const double x = t.B / t.S;
    const double up = x > -0.5 ? log1p(x) : log(t.q / t.S);
    const double lse_b = kLn2 * (static_cast<double>(t.F) + log2(t.S));
    write_row<QT>(in, out, rp, r, up - kLambda * (t.A / t.S), kLambda, t.mb, t.mq,
                  lse_b - kLambda * static_cast<double>(t.mb),
                  lse_b + up - kLambda * (static_cast<double>(t.K) + static_cast<double>(t.mq)),
                  sh.ib, sh.iq, 0u);
  }
}

// -------------------------------------------------------------------- host

// Launch shape: CTAs per row and shared-memory slots per warp.
struct Shape {
  int cluster, slots;
};
template <int QT>
Shape shape_for(int64_t N, int64_t V, int sm_count) {
  // Shared memory of kCtasPerSm CTAs an SM.
  const int most = 44 * 1024 / (kWarps * Slot<QT>::kBytes);
  const int64_t chunks = (V + kChunk - 1) / kChunk + 1;
  // Few rows are split until the CTAs fill the SMs (or a warp has one chunk).
  int c = 1;
  while (c < kMaxCluster && N * c < static_cast<int64_t>(sm_count) * kCtasPerSm &&
         chunks > static_cast<int64_t>(c) * kWarps)
    c *= 2;
  int64_t s = (chunks + c * kWarps - 1) / (c * kWarps) + 1;
  if (s > most) s = most;
  if (s < kDepth) s = kDepth;
  return {c, static_cast<int>(s)};
}

template <int QT, int OT, bool kOff>
cudaError_t launch_shape(const Operands& in, const Outputs& out, int sm_count, cudaStream_t s) {
  const Shape sh = shape_for<QT>(in.N, in.V, sm_count);
  const int smem = kWarps * sh.slots * Slot<QT>::kBytes;
  auto kern = kld_packed_rows_kernel<QT, OT, kOff>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(in.N * sh.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = static_cast<unsigned>(sh.cluster);
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, in, out, sh.cluster, sh.slots);
}

template <int QT, int OT>
cudaError_t launch_off(const Operands& in, const Outputs& out, int sm_count, cudaStream_t s) {
  // Rows on the 16-byte grid of the dense operand need no byte shift.
  const void* grid = QT == kFromPack ? out.grad : in.quant;
  const int64_t bytes = in.V * (QT == kFromPack ? Type<OT>::kBytes : Quant<QT>::kBytes);
  const bool on = grid == nullptr ||
                  ((reinterpret_cast<uintptr_t>(grid) & 15u) == 0 && (in.N == 1 || bytes % 16 == 0));
  return on ? launch_shape<QT, OT, false>(in, out, sm_count, s)
            : launch_shape<QT, OT, true>(in, out, sm_count, s);
}

template <int QT>
cudaError_t launch_out(const Operands& in, const Outputs& out, kld_dtype_t ot, int sm_count,
                       cudaStream_t s) {
  switch (ot) {
    case KLD_F32: return launch_off<QT, KLD_F32>(in, out, sm_count, s);
    case KLD_BF16: return launch_off<QT, KLD_BF16>(in, out, sm_count, s);
    case KLD_F16: return launch_off<QT, KLD_F16>(in, out, sm_count, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace from_packed
}  // namespace

cudaError_t launch_packed_rows(const PackedRows& a, int sm_count, cudaStream_t stream) {
  using namespace from_packed;
  Operands in;
  in.bcodes = a.base_codes;
  in.bheads = a.base_heads;
  in.quant = a.quant_codes ? static_cast<const void*>(a.quant_codes) : a.quant;
  in.qheads = a.quant_heads;
  in.tok = a.token_ids;
  in.N = a.N;
  in.V = a.V;
  in.nb = (a.V + packed::kBlock - 1) / packed::kBlock;
  Outputs out;
  out.rows = a.rows;
  out.kld = a.kld;
  out.nll = a.nll;
  out.amax_b = a.amax_b;
  out.amax_q = a.amax_q;
  out.grad = a.grad;
  out.scale = a.scale;
  const kld_dtype_t ot = a.grad ? a.grad_dtype : KLD_F32;
  if (a.quant_codes) return launch_out<kFromPack>(in, out, ot, sm_count, stream);
  switch (a.quant_dtype) {
    case KLD_F32: return launch_out<KLD_F32>(in, out, ot, sm_count, stream);
    case KLD_BF16: return launch_out<KLD_BF16>(in, out, ot, sm_count, stream);
    case KLD_F16: return launch_out<KLD_F16>(in, out, ot, sm_count, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace kld
