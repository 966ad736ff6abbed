// kld_packed_rows.cuh -- the statistic and the gradient of KL(P_base || P_quant)
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
// |x| <= 2.5 (three degrees by the warp's largest |x|). Steps of a warp that hold
// a larger or non-finite x take a second exponential, h_j = e_j e^x_j, and sum
// it apart (Q, with their e in D), so B = A + C over the others plus Q - D. Q
// is summed as 2^(q_j L - G) in a frame G near those steps' quant maximum: in
// the base row's frame an argument of 100 would be rounded by 4e-6.
// The polynomial steps get nothing of the size of KL by subtracting rounded
// exponentials, so rows that are nearly equal or nearly one-hot keep their
// accuracy, and so do rows whose two distributions hardly meet. Q - D is such
// a difference: one large log-ratio in a step that holds the row's mass
// leaves an absolute error of about 1e-7 in KL. F and K belong to a
// warp and move only when a value exceeds the maximum they were set at by
// more than four nats. Sums run in fp32 over a lane's 16 columns of a chunk,
// from there over at most kFold chunks and the warp, in fp64 beyond. (Equal
// terms round alike, so their errors add up: in sums of one fp32 addition a
// term, gradients of rows of one value were off by 3e-5 over 2^20 columns.)
//
// Rows whose sums are not finite and positive (NaN or +inf, an empty row, a
// base entry above -inf where quant is -inf, magnitudes near the type's
// limit) are done again by slow_row in fp64 from the definitions.
//
// Device code of kld_packed_rows.cu.
#pragma once

#include <climits>

#include "kld_internal.h"
#include "kld_packed.cuh"
#include "kld_rows_kernel.cuh"

namespace kld {
namespace {
namespace from_packed {

using namespace packed;

constexpr int kFromPack = 3;  // quant operand from a checkpoint
constexpr int kChunk = 512;   // columns a warp takes at a time
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
// Shared-memory loads by 32-bit address (ordered with the volatile waits).
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t x;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(a));
  return x;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 x;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(a));
  return x;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 x;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "r"(a));
  return x;
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

// Starts the copies of chunk c, which lies inside the row, into a slot (all
// lanes; the commit is the caller's).
template <int QT, bool kOff>
__device__ __forceinline__ void fetch(const LanePtr& p, int c, uint32_t slot, int lane) {
  const uint8_t* bc = p.bcodes + static_cast<int64_t>(c) * kChunk;
  const uint32_t* bh = p.bheads + static_cast<int64_t>(c) * (kChunk / kBlock);
  const char* qc = p.quant + static_cast<int64_t>(c) * (kChunk * Quant<QT>::kBytes);
  const uint32_t q = slot + Slot<QT>::kQuant;
  copy16(slot + lane * 16, bc);
  if (kOff && lane == 0) copy16(slot + 512, bc + 512);
  if (lane < (kOff ? 5 : 4)) {
    copy4(slot + Slot<QT>::kHeads + lane * 4, bh);
    if (QT == kFromPack)
      copy4(q + kCodeBytes + lane * 4, p.qheads + static_cast<int64_t>(c) * (kChunk / kBlock));
  }
  if (QT == kFromPack) {
    copy16(q + lane * 16, qc);
    if (kOff && lane == 0) copy16(q + 512, qc + 512);
  } else {
#pragma unroll
    for (int k = 0; k < kChunk * Quant<QT>::kBytes / 512; ++k)
      copy16(q + k * 512 + lane * 16, qc + k * 512);
  }
}

// G (4 or 8) values of a checkpoint row from its slot: `at` is the first
// column's offset in the chunk's code grid (at least -off for kOff), h0 its
// block's header, h1 that of the last column (kOff: a group may cross into
// the next block). Blocks with masks or bad values (bit 8 of the headers,
// gathered in `special`) give wrong values.
template <int G, bool kOff>
__device__ __forceinline__ void slot_values(uint32_t codes, uint32_t h0, uint32_t h1,
                                            int at, uint32_t& special, float* o) {
  uint32_t w[G / 4 + 1];
  if (!kOff) {
    if (G == 8) {
      const uint2 v = lds64(codes + at);
      w[0] = v.x;
      w[G / 4 - 1] = v.y;
    } else {
      w[0] = lds32(codes + at);
    }
  } else {
    const uint32_t p = codes + 16 + (at & ~3);
#pragma unroll
    for (int k = 0; k <= G / 4; ++k) w[k] = lds32(p + 4 * k);
    const uint32_t bits = (at & 3) * 8;
#pragma unroll
    for (int k = 0; k < G / 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], bits);
  }
  const int cut = kOff ? kBlock - (at & (kBlock - 1)) : G;  // columns of the first block
  special |= h0;
  if (kOff) special |= h1;
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

// Headers of a lane's groups of a chunk.
template <int QT, bool kOff>
struct Heads {
  static constexpr int kN = Quant<QT>::kGroups;
  uint32_t b[kN], bx[kOff ? kN : 1];
  uint32_t q[QT == kFromPack ? kN : 1], qx[QT == kFromPack && kOff ? kN : 1];
  // From shared memory: the headers of the chunk's first block (of the one
  // before it when shifted) and on.
  __device__ __forceinline__ void load(uint32_t base, uint32_t quant, int off, int lane) {
#pragma unroll
    for (int g = 0; g < kN; ++g) {
      const int at = group_col<QT>(g, lane) - (kOff ? off : 0);
      const uint32_t k0 = ((at >> 7) + (kOff ? 1 : 0)) * 4;
      const uint32_t k1 = (((at + Quant<QT>::kGroup - 1) >> 7) + 1) * 4;
      b[g] = lds32(base + k0);
      if (kOff) bx[g] = lds32(base + k1);
      if (QT == kFromPack) q[g] = lds32(quant + k0);
      if (QT == kFromPack && kOff) qx[g] = lds32(quant + k1);
    }
  }
};

// A lane's 16 columns of a chunk that lies inside the row: base values, and
// quant values (packed ones for the 16-bit types), wrong where a block is
// special (bit 8 of the result).
template <int QT, bool kOff>
__device__ __forceinline__ uint32_t step_plain(int off, uint32_t codes, uint32_t quant, const Heads<QT, kOff>& h,
                                               int lane, float* b, float* q, uint32_t* qw) {
  constexpr int G = Quant<QT>::kGroup;
  uint32_t special = 0u;
#pragma unroll
  for (int g = 0; g < Quant<QT>::kGroups; ++g) {
    const int at = group_col<QT>(g, lane) - (kOff ? off : 0);
    slot_values<G, kOff>(codes, h.b[g], h.bx[kOff ? g : 0], at, special, b + g * G);
    if constexpr (QT == kFromPack) {
      slot_values<G, kOff>(quant, h.q[g], h.qx[kOff ? g : 0], at, special, q + g * G);
    } else {
      const uint4 w = lds128(quant + group_col<QT>(g, lane) * Quant<QT>::kBytes);
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

// A lane's 16 columns of any chunk, straight from global memory: masks and
// bad blocks read as such, -inf outside the row.
template <int QT>
__device__ __forceinline__ void step_global(const RowPtr& rp, int64_t V, int c, int lane, float* b,
                                            float* q) {
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const int64_t j = static_cast<int64_t>(c) * kChunk + group_col<QT>(k / Quant<QT>::kGroup, lane) +
                      k % Quant<QT>::kGroup - rp.off;
    const bool in = j >= 0 && j < V;
    b[k] = in ? base_at<QT>(rp, j) : neg_inf();
    q[k] = in ? quant_at<QT>(rp, j) : neg_inf();
  }
}

// --------------------------------------------------------------- row state

// A warp's sums, as they are merged.
struct Part {
  float F, K;      // frame (a whole number; kNoFrame before any value), centre
  float S, A, C;   // over the polynomial steps
  float D, E;      // over the others: sums of e, e x
  float G, Q;      // and of 2^(q L - G), G their quant exponentials' frame
  float mb, mq;    // maxima of its columns
};
constexpr int kPartWords = 11;
static_assert(sizeof(Part) == 4 * kPartWords, "Part is stored word by word");

// The row's merged sums and what the gradient pass needs of them.
struct Total {
  double S, A, B, q;  // sum of e, e x, e (e^x - 1), e e^x over all steps
  float F, K;
  float mb, mq;
  // The gradient's frames, floor(log2) of the rows' whole sums, so that its
  // exponentials are the softmax values within a factor of two wherever the
  // rows peak; scale / (the sums in them), in (scale / 2, scale]. The two are
  // formed alike: equal rows give equal values.
  float Fb, Fq, cb, cq;
  int good;
};

// Block reductions of slow_row.
struct SlowShared {
  double dsum[32];
  float fmax_[2][32];
  int first[2];  // lowest columns of the maxima
  uint32_t flags;
};


// What a lane keeps of its part of the row: its warp's frame and centre
// (uniform), its sums (Part), its maxima and the first chunks they are in.
struct State {
  float F, K, T;  // T: a value above it moves the frame and the centre
  int form;       // order of the log-ratio's roundings (ratio_form)
  f2 S, A, C;     // pairs of fp32
  float D, E, G, Q;
  float mb, mq;
  int ib, iq;
};

// Moves a warp's frame to its step's maximum M (um: the lane's own), rebasing
// the lanes' sums exactly in F and by
//   A' = A + d S,  C' = e^d C + (e^d - 1) A + (e^d - 1 - d) S,  E' = E + d D
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
    float S[2], A[2], C[2];
    upk(s.S, S[0], S[1]);
    upk(s.A, A[0], A[1]);
    upk(s.C, C[0], C[1]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      C[k] = sc * (C[k] + e1 * C[k] + e1 * lam * A[k] + phi * S[k]);
      A[k] = sc * (A[k] + d * S[k]);
      S[k] *= sc;
    }
    s.S = pk(S[0], S[1]);
    s.A = pk(A[0], A[1]);
    s.C = pk(C[0], C[1]);
    s.E = sc * (s.E + d * s.D);
    s.D *= sc;
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
  f2 S, A, C;  // of the step: one addition to the long sums a step
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float u0, u1;
    upk(fma2(pk(b[2 * k], b[2 * k + 1]), L2, nf), u0, u1);
    const f2 e = pk(ex2(u0), ex2(u1));
    const f2 t = mul2(e, x[k]);
    S = k == 0 ? e : add2(S, e);
    A = k == 0 ? t : add2(A, t);
    C = k == 0 ? mul2(mul2(t, x[k]), phi_q2<T>(x[k])) : fma2(mul2(t, x[k]), phi_q2<T>(x[k]), C);
  }
  s.S = add2(s.S, S);
  s.A = add2(s.A, A);
  s.C = add2(s.C, C);
}

// Adds a chunk's 16 columns of a lane (the whole warp together) to its
// state. Entries whose bit in `valid` is 0 are -inf in both operands (masks,
// columns outside the row): they have weight 0 and take x = 0. i: the
// chunk's number. special: some block of the lane's is masked or bad (bit 8);
// then nothing is added and the result is false. kPlain: the values come from
// slot_values, where an entry is -inf only if its block's step is past 2^95
// (plain_scale); such rows are left to slow_row.
template <int QT, bool kPlain>
__device__ __forceinline__ bool add_step(State& s, const float* b, const float* q,
                                         const uint32_t* qw, uint32_t special, unsigned valid, int i) {
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
  // One vote for the two rare cases.
  if (__any_sync(0xffffffffu, (special & 256u) != 0u || mb > s.T)) {
    if (__any_sync(0xffffffffu, (special & 256u) != 0u)) return false;
    raise<QT>(s, b, q, qw, mb, warp_max(mb));
  }
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
  // The warp's largest |x| by its bits (NaN is above infinity there).
  ax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(ax)));
  if (ax <= kTauA) {
    add_poly<0>(s, b, x);
  } else if (ax <= kTauB) {
    add_poly<1>(s, b, x);
  } else if (ax <= kTau) {
    add_poly<2>(s, b, x);
  } else {
    // Large or non-finite log-ratios. A masked base entry has e = 0 and gives
    // its h to Q; x = -inf with a base entry above -inf makes E non-finite,
    // which sends the row to slow_row, as a block too wide for plain_scale does.
    const float none = kPlain ? __int_as_float(0x7fc00000) : 0.f;
    const float G = floorf(warp_max(mq) * kLog2e);
    if (G > s.G) {
      s.Q *= static_cast<float>(pow2d(s.G - G));
      s.G = G;
    }
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
        E += bk == neg_inf() ? none : e * xs[h];
        Q += ex2(fmaf(q_el<kPk>(q, qw, 2 * k + h), kLog2e, -s.G));
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
  return true;
}

// A warp's part from its lanes' states (the whole warp together).
__device__ __forceinline__ Part part_of(const State& s) {
  Part w;
  w.F = s.F;
  w.K = s.K;
  float v0, v1;
  upk(s.S, v0, v1);
  w.S = sum_lanes(v0 + v1);
  upk(s.A, v0, v1);
  w.A = sum_lanes(v0 + v1);
  upk(s.C, v0, v1);
  w.C = sum_lanes(v0 + v1);
  w.D = sum_lanes(s.D);
  w.E = sum_lanes(s.E);
  w.G = s.G;
  w.Q = sum_lanes(s.Q);
  w.mb = warp_max(s.mb);
  w.mq = warp_max(s.mq);
  return w;
}

// A lane's sums over blocks of kFold chunks, for rows that have more.
constexpr int kFold = 256;
struct Long {
  float F, K, G;
  double S, A, C, D, E, Q;
};
// Moves a lane's sums there (`first`: nothing is there yet), rebasing what is
// as raise does.
__device__ __noinline__ State fold(State s, Long* l, bool first) {
  if (first) {
    l->F = l->G = kNoFrame;
    l->K = 0.f;
    l->S = l->A = l->C = l->D = l->E = l->Q = 0.0;
  }
  if (s.F != l->F || s.K != l->K) {
    const double sc = pow2d(l->F - s.F);
    const double d = static_cast<double>(s.K) - static_cast<double>(l->K);
    const double e1 = expm1(kLambda * d), phi = e1 - kLambda * d;
    if (l->F != kNoFrame) {
      l->C = sc * (l->C + e1 * l->C + e1 * kLambda * l->A + phi * l->S);
      l->A = sc * (l->A + d * l->S);
      l->E = sc * (l->E + d * l->D);
      l->S *= sc;
      l->D *= sc;
    }
    l->F = s.F;
    l->K = s.K;
  }
  if (s.G > l->G) {
    l->Q *= pow2d(l->G - s.G);
    l->G = s.G;
  }
  float v0, v1;
  upk(s.S, v0, v1);
  l->S += static_cast<double>(v0) + v1;
  upk(s.A, v0, v1);
  l->A += static_cast<double>(v0) + v1;
  upk(s.C, v0, v1);
  l->C += static_cast<double>(v0) + v1;
  l->D += s.D;
  l->E += s.E;
  l->Q += s.Q;
  s.S = s.A = s.C = splat(0.f);
  s.D = s.E = s.Q = 0.f;
  return s;
}
// A warp's part from what was moved (the whole warp together).
__device__ __noinline__ Part part_of_long(const State s, const Long* l) {
  Part w;
  w.F = l->F;
  w.K = l->K;
  w.S = static_cast<float>(warp_sum(l->S));
  w.A = static_cast<float>(warp_sum(l->A));
  w.C = static_cast<float>(warp_sum(l->C));
  w.D = static_cast<float>(warp_sum(l->D));
  w.E = static_cast<float>(warp_sum(l->E));
  w.G = l->G;
  w.Q = static_cast<float>(warp_sum(l->Q));
  w.mb = warp_max(s.mb);
  w.mq = warp_max(s.mq);
  return w;
}
__device__ __forceinline__ State fresh_state() {
  State s;
  s.F = kNoFrame;
  s.K = 0.f;
  s.T = neg_inf();
  s.form = 0;
  s.S = s.A = s.C = splat(0.f);
  s.D = s.E = s.Q = 0.f;
  s.G = kNoFrame;
  s.mb = s.mq = neg_inf();
  s.ib = s.iq = 0;
  return s;
}

// Chunks a warp puts off: those that hold masked or bad blocks are done after
// the others, out of the way of the hot loops. Past kLater chunks the rest
// are found again by put_off.
constexpr int kLater = 16;
struct Later {
  int chunk[kLater];
};
// Whether chunk c is one of them (the whole warp together; exactly as the
// hot loops decide).
template <int QT, bool kOff>
__device__ __forceinline__ bool put_off(const RowPtr& rp, int64_t nb, int c, int lane) {
  const int64_t k = static_cast<int64_t>(c) * (kChunk / kBlock) + lane - 1;
  uint32_t h = 0u;
  if (lane < 5 && (lane > 0 || (kOff && rp.off > 0)) && k >= 0 && k < nb) {
    h = __ldg(rp.bheads + k);
    if (QT == kFromPack) h |= __ldg(rp.qheads + k);
  }
  return __any_sync(0xffffffffu, (h & 256u) != 0u);
}

// add_step for a chunk put off.
template <int QT>
__device__ __noinline__ State add_later(State s, const RowPtr rp, int64_t V, int c, int lane) {
  float b[16], q[16];
  uint32_t qw[8];
  step_global<QT>(rp, V, c, lane, b, q);
  unsigned valid = 0u;
#pragma unroll
  for (int k = 0; k < 16; ++k)
    if (b[k] != neg_inf() || q[k] != neg_inf()) valid |= 1u << k;
  if constexpr (kPacked16<QT> != 0) {
#pragma unroll
    for (int k = 0; k < 8; ++k) qw[k] = pack16<QT>(q[2 * k], q[2 * k + 1]);
  }
  // Out of order: a maximum that equals one of a later chunk comes first.
  const float mb = s.mb, mq = s.mq;
  const int ib = s.ib, iq = s.iq;
  s.mb = s.mq = neg_inf();
  add_step<QT, false>(s, b, q, qw, 0u, valid, c);
  if (mb > s.mb || (mb == s.mb && ib < c)) {
    s.mb = mb;
    s.ib = ib;
  }
  if (mq > s.mq || (mq == s.mq && iq < c)) {
    s.mq = mq;
    s.iq = iq;
  }
  return s;
}

// The parts of a row merged by one warp, in fp64, to the largest frame and
// the centre of the part that holds the row's maximum. grad: the gradient's
// frames too, the base row's on lane 0 and the quant row's on lane 1.
__device__ __noinline__ void merge(const Part* part, int parts, float scale, bool grad, Total* total) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  float F = kNoFrame, mb = neg_inf(), mq = neg_inf();
  for (int i = lane; i < parts; i += 32) {
    F = fmaxf(F, part[i].F);
    mb = fmaxf(mb, part[i].mb);
    mq = fmaxf(mq, part[i].mq);
  }
  F = warp_max(F);
  mb = warp_max(mb);
  mq = warp_max(mq);
  int best = INT_MAX;
  for (int i = lane; i < parts; i += 32)
    if (part[i].mb == mb) best = min(best, i);
  best = __reduce_min_sync(0xffffffffu, best);
  const float K = best < parts ? part[best].K : 0.f;
  double S = 0.0, A = 0.0, C = 0.0, D = 0.0, E = 0.0, Q = 0.0;
  for (int i = lane; i < parts; i += 32) {
    const Part p = part[i];
    if (p.Q != 0.f)  // from its frame to the row's: 2^(F - K L) is the unit there
      Q += p.Q * exp2(static_cast<double>(p.G) - static_cast<double>(F) + static_cast<double>(K) * kLog2eD);
    if (p.S == 0.f && p.D == 0.f && p.E == 0.f) continue;
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
  }
  S = warp_sum(S);
  A = warp_sum(A);
  C = warp_sum(C);
  D = warp_sum(D);
  E = warp_sum(E);
  Q = warp_sum(Q);
  const double q = S + (kLambda * A + C) + Q;
  if (lane == 0) {
    Total& t = *total;
    t.S = S + D;
    t.A = A + E;
    t.B = kLambda * A + C + (Q - D);
    t.q = q;
    t.F = F;
    t.K = K;
    t.mb = mb;
    t.mq = mq;
    t.good = t.S > 0.0 && t.S < 1e300 && fabs(t.A) < 1e300 && q > 0.0 && q < 1e300 &&
             fabsf(F) < 1e6f && fabsf(K) < 1e6f;
  }
  if (grad && lane < 2) {
    // sum_j 2^(b_j L) = (S + D) 2^F, sum_j 2^(q_j L) = q 2^(F - K L)
    const double at = log2(lane == 0 ? S + D : q) + static_cast<double>(F) -
                      (lane == 0 ? 0.0 : static_cast<double>(K) * kLog2eD);
    const float frame = static_cast<float>(floor(at)), c = static_cast<float>(scale * exp2(floor(at) - at));
    *(lane == 0 ? &total->Fb : &total->Fq) = frame;
    *(lane == 0 ? &total->cb : &total->cq) = c;
  }
}

// The row from its definitions in fp64, by one whole CTA (every CTA of the
// row's cluster does it for itself): for rows the fp32 sums cannot hold.
struct Slow {
  float mb, mq;
  int ib, iq;
  double Sb, Sq, kl;
  uint32_t flags;
};
__device__ double block_sum(SlowShared& sh, double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.dsum[threadIdx.x >> 5] = x;
  __syncthreads();
  double s = 0.0;
  for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w) s += sh.dsum[w];
  return s;
}
template <int QT>
__device__ __noinline__ void slow_row(SlowShared& sh, const RowPtr& rp, int64_t V, Slow& out) {
  const int tid = static_cast<int>(threadIdx.x);
  if (tid == 0) {
    sh.flags = 0u;
    sh.first[0] = sh.first[1] = INT_MAX;
  }
  __syncthreads();
  float mb = neg_inf(), mq = neg_inf();
  uint32_t f = 0u;
  for (int64_t j = tid; j < V; j += blockDim.x) {
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
  for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w) {
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
    int ib = INT_MAX, iq = INT_MAX;
    for (int64_t j = tid; j < V; j += blockDim.x) {
      const double b = static_cast<double>(base_at<QT>(rp, j)) - mb;
      const double q = static_cast<double>(quant_at<QT>(rp, j)) - mq;
      const double e = exp(b);
      sb += e;
      sq += exp(q);
      if (b > -INFINITY && q > -INFINITY) a += e * (b - q);
      if (b == 0.0) ib = min(ib, static_cast<int>(j));
      if (q == 0.0) iq = min(iq, static_cast<int>(j));
    }
    if (ib < INT_MAX) atomicMin(&sh.first[0], ib);
    if (iq < INT_MAX) atomicMin(&sh.first[1], iq);
  }
  sb = block_sum(sh, sb);
  sq = block_sum(sh, sq);
  a = block_sum(sh, a);
  out.mb = mb;
  out.mq = mq;
  out.ib = sh.first[0];
  out.iq = sh.first[1];
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
  for (int64_t j = j0 + threadIdx.x; j < j1; j += blockDim.x) {
    float g = 0.f;
    if (!(s.flags & kExcludedFlags)) {
      const float p = __fmul_rn(ex2((base_at<QT>(rp, j) - s.mb) * kLog2e), cb);
      const float r = __fmul_rn(ex2((quant_at<QT>(rp, j) - s.mq) * kLog2e), cq);
      g = __fmul_rn(scale, __fsub_rn(r, p));
    }
    Type<OT>::store(grow + j * Type<OT>::kBytes, g);
  }
}

// A row's token and both operands at it.
struct Token {
  int id;    // -1: no token ids; -2: outside [0, V)
  float b, q;
};
template <int QT>
__device__ __forceinline__ Token token_of(const Operands& in, const RowPtr& rp, int64_t r) {
  Token t = {-1, 0.f, 0.f};
  if (in.tok) {
    t.id = __ldg(in.tok + r);
    if (t.id < 0 || t.id >= in.V) {
      t.id = -2;
    } else {
      t.b = base_at<QT>(rp, t.id);
      t.q = quant_at<QT>(rp, t.id);
    }
  }
  return t;
}

// The row's record (and its per-field copies), by one thread. ln_b, ln_q:
// ln sum e^(lam (x - m)) of the two rows, m their maxima.
__device__ void write_row(const Outputs& out, const Token& tok, int64_t r, double kl, double lam, float mb, float mq, double ln_b, double ln_q,
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
  if (tok.id != -1) {
    if (tok.id < 0) {
      flags |= KLD_ROW_BAD_TOKEN;
    } else if (ok) {
      const float b = tok.b, q = tok.q;
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

// What the gradient of a row needs of its sums.
struct GradScale {
  float Fb, Fq, cb, cq;
  __device__ __forceinline__ explicit GradScale(const Total& t) : Fb(t.Fb), Fq(t.Fq), cb(t.cb), cq(t.cq) {}
};
// The gradient of 16 columns (into b).
__device__ __forceinline__ void grad_values(const GradScale& t, float* b, const float* q) {
  const f2 L2 = splat(kLog2e), fb = splat(-t.Fb), fq = splat(-t.Fq);
  const f2 cb2 = splat(t.cb), cq2 = splat(t.cq), zero2 = splat(0.f);
#pragma unroll
  for (int k = 0; k < 16; k += 2) {
    float u0, u1, v0, v1;
    upk(fma2(pk(b[k], b[k + 1]), L2, fb), u0, u1);
    upk(fma2(pk(q[k], q[k + 1]), L2, fq), v0, v1);
    // Products rounded apart, so equal rows give exactly zero: as FMAs with
    // zero, since a packed product may be joined with the difference into
    // one FMA (measured: 2.5e-8 p instead of 0).
    const f2 pr = fma2(pk(ex2(u0), ex2(u1)), cb2, zero2);
    const f2 rr = fma2(pk(ex2(v0), ex2(v1)), cq2, zero2);
    upk(sub2(rr, pr), b[k], b[k + 1]);
  }
}

// The record of a row from its sums, by one thread.
__device__ void write_total(const Outputs& out, const Token& tok, int64_t r, const Total& t, int ib,
                            int iq) {
  // ln(q / S), by the difference where the rows are close
  const double x = t.B / t.S;
  const double up = x > -0.5 ? log1p(x) : log(t.q / t.S);
  const double lse_b = kLn2 * (static_cast<double>(t.F) + log2(t.S));
  write_row(out, tok, r, up - kLambda * (t.A / t.S), kLambda, t.mb, t.mq,
                lse_b - kLambda * static_cast<double>(t.mb),
                lse_b + up - kLambda * (static_cast<double>(t.K) + static_cast<double>(t.mq)),
                ib, iq, 0u);
}

// A lane's 16 gradient values of a chunk: at: the address of its first group
// (all groups of a row lie alike on the output's 16-byte grid; whole: on
// it, as far as a group's vectors need).
template <int QT, int OT>
__device__ __forceinline__ bool whole_vectors(const char* at) {
  constexpr uint32_t bytes = Quant<QT>::kGroup * Type<OT>::kBytes < 16 ? 8u : 16u;
  return (reinterpret_cast<uintptr_t>(at) & (bytes - 1u)) == 0;
}
template <int QT, int OT>
__device__ __forceinline__ void store_whole(char* at, const float* x) {
  constexpr int G = Quant<QT>::kGroup;
  constexpr int OE = 16 / Type<OT>::kBytes;  // elements of an output vector
#pragma unroll
  for (int g = 0; g < Quant<QT>::kGroups; ++g) {
    char* dst = at + g * 32 * G * Type<OT>::kBytes;
    const float* y = x + g * G;
    if (OE <= G) {
#pragma unroll
      for (int k = 0; k < G; k += OE)
        __stcs(reinterpret_cast<uint4*>(dst + k * Type<OT>::kBytes), Type<OT>::vec(y + k));
    } else {
      const float z[8] = {y[0], y[1], y[2], y[3], 0.f, 0.f, 0.f, 0.f};
      const uint4 w = Type<OT>::vec(z);
      __stcs(reinterpret_cast<uint2*>(dst), make_uint2(w.x, w.y));
    }
  }
}
// The same one by one, for groups that are not on the output's grid.
template <int QT, int OT>
__device__ __forceinline__ void store_singly(char* at, const float* x) {
  constexpr int G = Quant<QT>::kGroup;
#pragma unroll
  for (int k = 0; k < 16; ++k)
    Type<OT>::store(at + (k / G * 32 * G + k % G) * Type<OT>::kBytes, x[k]);
}
// One by one, those of a chunk's columns from j0 on that lie in the row.
template <int QT, int OT>
__device__ __forceinline__ void store_checked(char* grow, int64_t j0, int64_t V, int lane,
                                              const float* x) {
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const int64_t j = j0 + group_col<QT>(k / Quant<QT>::kGroup, lane) + k % Quant<QT>::kGroup;
    if (j >= 0 && j < V) Type<OT>::store(grow + j * Type<OT>::kBytes, x[k]);
  }
}

// The gradient of a chunk put off.
template <int QT, int OT>
__device__ __noinline__ void grad_later(const GradScale gs, const RowPtr rp, char* grow, int64_t V,
                                        int c, int lane) {
  float b[16], q[16];
  step_global<QT>(rp, V, c, lane, b, q);
  grad_values(gs, b, q);
  store_checked<QT, OT>(grow, static_cast<int64_t>(c) * kChunk - rp.off, V, lane, b);
}

// -------------------------------------------------------------------- host

inline Operands operands_of(const PackedRows& a) {
  Operands in;
  in.bcodes = a.base_codes;
  in.bheads = a.base_heads;
  in.quant = a.quant_codes ? static_cast<const void*>(a.quant_codes) : a.quant;
  in.qheads = a.quant_heads;
  in.tok = a.token_ids;
  in.N = a.N;
  in.V = a.V;
  in.nb = (a.V + packed::kBlock - 1) / packed::kBlock;
  return in;
}
inline Outputs outputs_of(const PackedRows& a) {
  Outputs out;
  out.rows = a.rows;
  out.kld = a.kld;
  out.nll = a.nll;
  out.amax_b = a.amax_b;
  out.amax_q = a.amax_q;
  out.grad = a.grad;
  out.scale = a.scale;
  return out;
}
// Whether all rows lie on the 16-byte grid of the dense operand (then no
// byte shift is needed).
template <int QT, int OT>
bool on_grid(const Operands& in, const Outputs& out) {
  const void* grid = QT == kFromPack ? out.grad : in.quant;
  const int64_t bytes = in.V * (QT == kFromPack ? Type<OT>::kBytes : Quant<QT>::kBytes);
  return grid == nullptr ||
         ((reinterpret_cast<uintptr_t>(grid) & 15u) == 0 && (in.N == 1 || bytes % 16 == 0));
}

}  // namespace from_packed
}  // namespace
}  // namespace kld
