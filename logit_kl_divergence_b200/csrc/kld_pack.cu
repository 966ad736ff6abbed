// kld_pack.cu -- writing and restoring the 8-bit logit checkpoint (format
// and its arithmetic: kld_packed.cuh).
#include "kld_internal.h"
#include "kld_packed.cuh"

namespace kld {
namespace {

using namespace packed;

constexpr int kThreads = 256;
constexpr int kUnit = 16;                       // elements of one thread's step
constexpr int kLanes = kBlock / kUnit;          // lanes that share a block
constexpr float kMagic = 12582912.f;            // 1.5 * 2^23: x + kMagic rounds x to a whole number

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float min3_nan(float a, float b, float c) {
  float y;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// Exponent of a finite x >= 0: floor(log2 x), -127 for zero and subnormals.
__device__ __forceinline__ int exponent(float x) {
  return static_cast<int>(__float_as_uint(x) >> 23) - 127;
}

// A warp's steps over groups of units, `per` groups a row, in the order of a
// grid-stride loop: row and group advance by a stride split the same way (a
// 64-bit division a step cost more than the step's work).
struct Steps {
  int64_t row;
  uint32_t group;
  __device__ __forceinline__ Steps(int64_t start, uint32_t per)
      : row(start / per), group(static_cast<uint32_t>(start % per)) {}
  __device__ __forceinline__ void add(const Steps& d, uint32_t per) {
    row += d.row;
    group += d.group;
    if (group >= per) {
      group -= per;
      ++row;
    }
  }
};
// Units of a lane in a group, 32 apart, loaded together. Measured at 2048
// rows: fp32 rows of 151936 253 us with two, 266 with one; shifted bf16 rows
// of 131073 184 us with one, 192 with two; four spill or halve the CTAs.
template <bool kAligned>
constexpr int kPackUnits = kAligned ? 2 : 1;
constexpr int kUnpackUnits = 4;  // bf16 checkpoint to fp32 316 us, one by one 370 us

// 16 elements of a row from column j on. Full units whose 16-byte vectors
// lie inside the tensor [begin, end) take vector loads, shifted into place
// where the row does not start on a 16-byte boundary; the others go element
// by element, -inf past V.
template <int DT, bool kAligned>
__device__ __forceinline__ void load_unit(const char* row, int64_t j, int64_t V,
                                          const char* begin, const char* end, float* x) {
  constexpr int eb = Type<DT>::kBytes;
  constexpr int nv = kUnit * eb / 16;
  const char* p = row + j * eb;
  if (kAligned) {
    if (j + kUnit <= V) {
      uint32_t w[4 * nv];
#pragma unroll
      for (int k = 0; k < nv; ++k)
        *reinterpret_cast<uint4*>(&w[4 * k]) = __ldcs(reinterpret_cast<const uint4*>(p) + k);
      Type<DT>::unpack16(w, x);
      return;
    }
  } else {
    const uint32_t mis = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15u);
    const char* a = p - mis;
    if (j + kUnit <= V && a >= begin && a + 16 * (nv + 1) <= end) {
      uint32_t w[4 * nv + 4];
#pragma unroll
      for (int k = 0; k <= nv; ++k)
        *reinterpret_cast<uint4*>(&w[4 * k]) = __ldg(reinterpret_cast<const uint4*>(a) + k);
      shift_bytes<4 * nv>(w, mis);
      Type<DT>::unpack16(w, x);
      return;
    }
  }
#pragma unroll
  for (int k = 0; k < kUnit; ++k)
    x[k] = j + k < V ? Type<DT>::load(p + k * eb) : neg_inf();
}

// Header and codes of a lane's unit; the 8 lanes of a block agree on its
// extremes by three shuffles (the whole warp together; live: the lane has a
// unit). Units with -inf, NaN or a magnitude of 2^126 take the slow branch
// (the extremes test fails there and only there).
__device__ __forceinline__ void pack_unit(const float* x, bool live, int lane, uint32_t& head,
                                          uint4& out) {
  float lo = 0.f, hi = 0.f;
  bool masked = false, some = true, bad = false;
  if (live) {
    lo = hi = x[0];
#pragma unroll
    for (int k = 1; k < kUnit - 1; k += 2) {
      lo = min3_nan(lo, x[k], x[k + 1]);
      hi = max3_nan(hi, x[k], x[k + 1]);
    }
    lo = min3_nan(lo, x[kUnit - 1], x[kUnit - 1]);
    hi = max3_nan(hi, x[kUnit - 1], x[kUnit - 1]);
    if (!(lo > -kLimit && hi < kLimit)) {
      lo = kLimit;
      hi = -kLimit;
      some = false;
#pragma unroll
      for (int k = 0; k < kUnit; ++k) {
        if (x[k] == neg_inf()) {
          masked = true;
        } else if (!(fabsf(x[k]) < kLimit)) {
          bad = true;
        } else {
          some = true;
          lo = fminf(lo, x[k]);
          hi = fmaxf(hi, x[k]);
        }
      }
    }
  }
  // Lanes without an unmasked entry leave the extremes to the others.
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const unsigned group = 0xffu << (lane & 24);
  const unsigned has_some = __ballot_sync(0xffffffffu, some);
  const unsigned has_mask = __ballot_sync(0xffffffffu, masked);
  const unsigned has_bad = __ballot_sync(0xffffffffu, bad);
  uint32_t c[4] = {0u, 0u, 0u, 0u};
  if (has_bad & group) {
    head = kBadHead;
  } else if (!(has_some & group)) {
    head = kMaskedHead;
  } else if (live) {
    int e = exponent(hi - lo) - 7;
    e = max(e, exponent(fmaxf(fabsf(lo), fabsf(hi))) - 20);
    e = max(e, -126);
    float up = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e
    if (rintf(hi * up) - rintf(lo * up) > 254.f) {
      ++e;
      up *= 0.5f;
    }
    const int base = static_cast<int>(rintf(lo * up)) - 1;
    head = static_cast<uint32_t>(base) << 9 | (has_mask & group ? 256u : 0u) |
           static_cast<uint32_t>(e + 128);
    // bits(x * up + kMagic) - bits(kMagic) is the whole number n.
    const uint32_t zero = __float_as_uint(kMagic) + static_cast<uint32_t>(base);
    uint32_t n[kUnit];
#pragma unroll
    for (int k = 0; k < kUnit; ++k) n[k] = __float_as_uint(fmaf(x[k], up, kMagic)) - zero;
    if (masked) {
#pragma unroll
      for (int k = 0; k < kUnit; ++k)
        if (x[k] == neg_inf()) n[k] = 0u;
    }
    // the low bytes, four to a word
#pragma unroll
    for (int k = 0; k < 4; ++k)
      c[k] = __byte_perm(__byte_perm(n[4 * k], n[4 * k + 1], 0x0040),
                         __byte_perm(n[4 * k + 2], n[4 * k + 3], 0x0040), 0x5410);
  }
  out = make_uint4(c[0], c[1], c[2], c[3]);
}

// One pass over the logits: a lane holds kPackUnits units of 16 elements in
// registers and writes each one's codes as one vector. Bound by HBM: it reads
// s and writes 1 + 1/32 bytes per element; 2048 x 151936 bf16 in 197 us, 4.8
// TB/s (fp32 253 us, 6.2 TB/s).
template <int DT, bool kAligned>
__global__ void __launch_bounds__(kThreads)
    kld_pack_kernel(const void* __restrict__ logits, int64_t N, int64_t V, int64_t nb,
                    uint8_t* __restrict__ codes, uint32_t* __restrict__ heads) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const uint32_t upr = static_cast<uint32_t>(nb * kLanes);  // units per row
  const uint32_t per = (upr + 32 * kPackUnits<kAligned> - 1) / (32 * kPackUnits<kAligned>);
  const char* begin = static_cast<const char*>(logits);
  const char* end = begin + N * V * Type<DT>::kBytes;
  constexpr int kWarps = kThreads / 32;
  const Steps stride(static_cast<int64_t>(gridDim.x) * kWarps, per);
  for (Steps at(static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5), per); at.row < N;
       at.add(stride, per)) {
    const char* row = begin + at.row * V * Type<DT>::kBytes;
    const uint32_t u0 = at.group * (32 * kPackUnits<kAligned>) + lane;
    float x[kPackUnits<kAligned>][kUnit];
#pragma unroll
    for (int i = 0; i < kPackUnits<kAligned>; ++i)
      if (u0 + 32 * i < upr)
        load_unit<DT, kAligned>(row, static_cast<int64_t>(u0 + 32 * i) * kUnit, V, begin, end, x[i]);
#pragma unroll
    for (int i = 0; i < kPackUnits<kAligned>; ++i) {
      const uint32_t u = u0 + 32 * i;
      uint32_t head;
      uint4 c;
      pack_unit(x[i], u < upr, lane, head, c);
      if (u < upr) {
        *reinterpret_cast<uint4*>(codes + (at.row * upr + u) * kUnit) = c;
        if ((lane & (kLanes - 1)) == 0) heads[at.row * nb + u / kLanes] = head;
      }
    }
  }
}

// Restores the values: a lane writes whole 16-byte vectors of a row (E
// elements each), so that stores are whole and in order whatever the row's
// alignment: a row that starts `off` elements into a vector has its codes
// shifted by as many bytes instead. Bound by HBM: reads 1 + 1/32 and writes the
// output's bytes per element; 2048 x 151936 to fp32 in 316 us, 5.0 TB/s.
template <int OT>
__global__ void __launch_bounds__(kThreads)
    kld_unpack_kernel(const uint8_t* __restrict__ codes, const uint32_t* __restrict__ heads,
                      int64_t N, int64_t V, int64_t nb, void* __restrict__ out) {
  constexpr int eb = Type<OT>::kBytes;
  constexpr int E = 16 / eb;
  constexpr int NW = E / 4;  // code words of a vector
  const uint32_t upr = static_cast<uint32_t>((V + E - 1) / E + 1);  // vectors that touch a row, at most
  const uint32_t per = (upr + 32 * kUnpackUnits - 1) / (32 * kUnpackUnits);
  constexpr int kWarps = kThreads / 32;
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const Steps stride(static_cast<int64_t>(gridDim.x) * kWarps, per);
  for (Steps at(static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5), per); at.row < N;
       at.add(stride, per)) {
    char* row = static_cast<char*>(out) + at.row * V * eb;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / eb);
    const uint8_t* crow = codes + at.row * nb * kBlock;
    const uint32_t* hrow = heads + at.row * nb;
    const int64_t j0 = static_cast<int64_t>(at.group * (32 * kUnpackUnits) + lane) * E - off;
    // all of the group's codes and headers are on their way before the first is used
    uint32_t w[kUnpackUnits][NW + 1], h0[kUnpackUnits], h1[kUnpackUnits];
    const uint32_t bits = static_cast<uint32_t>(j0 & 3) * 8u;
#pragma unroll
    for (int i = 0; i < kUnpackUnits; ++i) {
      const int64_t j = j0 + i * (32 * E);  // first column of the vector
      if (j < 0 || j + E > V) continue;
      // The E code bytes from column j on: whole words, then a byte shift.
      const uint32_t* wp = reinterpret_cast<const uint32_t*>(crow + (j & ~static_cast<int64_t>(3)));
      if (NW == 2 && off == 0) {
        const uint2 v = __ldcs(reinterpret_cast<const uint2*>(wp));
        w[i][0] = v.x;
        w[i][NW - 1] = v.y;
      } else {
#pragma unroll
        for (int k = 0; k < NW; ++k) w[i][k] = __ldg(wp + k);
      }
      w[i][NW] = bits ? __ldg(wp + NW) : 0u;
      h0[i] = __ldg(hrow + j / kBlock);
      h1[i] = off ? __ldg(hrow + (j + E - 1) / kBlock) : h0[i];
    }
#pragma unroll
    for (int i = 0; i < kUnpackUnits; ++i) {
      const int64_t j = j0 + i * (32 * E);
      if (j >= 0 && j + E <= V) {
        float x[E];
        if (off) {
#pragma unroll
          for (int k = 0; k < NW; ++k) w[i][k] = __funnelshift_r(w[i][k], w[i][k + 1], bits);
        }
        if ((h0[i] | h1[i]) & 256u) {
          // masked or bad blocks
          const int cut = kBlock - static_cast<int>(j & (kBlock - 1));
          float y[E];
          const Scale s0 = scale_of(h0[i]), s1 = scale_of(h1[i]);
#pragma unroll
          for (int k = 0; k < NW; ++k) {
            decode4(w[i][k], s0, x + 4 * k);
            decode4(w[i][k], s1, y + 4 * k);
          }
#pragma unroll
          for (int k = 0; k < E; ++k)
            if (k >= cut) x[k] = y[k];
        } else {
          const int cut = kBlock - static_cast<int>(j & (kBlock - 1));
          float a0, b0, a1, b1;
          plain_scale(h0[i], a0, b0);
          plain_scale(h1[i], a1, b1);
#pragma unroll
          for (int k = 0; k < E; ++k) {
            const uint32_t y = w[i][k / 4];
            const float m = k % 4 == 0 ? magic_byte<0>(y) : (k % 4 == 1 ? magic_byte<1>(y)
                          : (k % 4 == 2 ? magic_byte<2>(y) : magic_byte<3>(y)));
            x[k] = fmaf(m, k < cut ? a0 : a1, k < cut ? b0 : b1);
          }
        }
        __stcs(reinterpret_cast<uint4*>(row + j * eb), Type<OT>::vec(x));
      } else {
        for (int k = 0; k < E; ++k) {
          const int64_t c = j + k;
          if (c >= 0 && c < V) Type<OT>::store(row + c * eb, decode1(crow[c], hrow[c / kBlock]));
        }
      }
    }
  }
}

int blocks_for(int64_t groups, int sm_count) {
  const int64_t need = (groups + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t most = static_cast<int64_t>(sm_count) * 8;
  return static_cast<int>(need < most ? need : most);
}

template <int DT>
cudaError_t pack_typed(const void* logits, int64_t N, int64_t V, uint8_t* codes, uint32_t* heads,
                       int sm_count, cudaStream_t s) {
  const int64_t nb = (V + kBlock - 1) / kBlock;
  const bool aligned = (reinterpret_cast<uintptr_t>(logits) & 15u) == 0 &&
                       (N == 1 || V * Type<DT>::kBytes % 16 == 0);
  const int64_t group = 32 * (aligned ? kPackUnits<true> : kPackUnits<false>);
  const int grid = blocks_for(N * ((nb * kLanes + group - 1) / group), sm_count);
  if (aligned)
    kld_pack_kernel<DT, true><<<grid, kThreads, 0, s>>>(logits, N, V, nb, codes, heads);
  else
    kld_pack_kernel<DT, false><<<grid, kThreads, 0, s>>>(logits, N, V, nb, codes, heads);
  return cudaGetLastError();
}

template <int OT>
cudaError_t unpack_typed(const uint8_t* codes, const uint32_t* heads, int64_t N, int64_t V,
                         void* out, int sm_count, cudaStream_t s) {
  constexpr int E = 16 / Type<OT>::kBytes;
  const int64_t nb = (V + kBlock - 1) / kBlock;
  const int64_t per = ((V + E - 1) / E + 1 + 32 * kUnpackUnits - 1) / (32 * kUnpackUnits);
  kld_unpack_kernel<OT><<<blocks_for(N * per, sm_count), kThreads, 0, s>>>(codes, heads, N, V, nb,
                                                                         out);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_pack(const void* logits, int64_t N, int64_t V, kld_dtype_t dtype,
                        uint8_t* codes, uint32_t* heads, int sm_count, cudaStream_t stream) {
  switch (dtype) {
    case KLD_F32: return pack_typed<KLD_F32>(logits, N, V, codes, heads, sm_count, stream);
    case KLD_BF16: return pack_typed<KLD_BF16>(logits, N, V, codes, heads, sm_count, stream);
    case KLD_F16: return pack_typed<KLD_F16>(logits, N, V, codes, heads, sm_count, stream);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_unpack(const uint8_t* codes, const uint32_t* heads, int64_t N, int64_t V,
                          void* out, kld_dtype_t out_dtype, int sm_count, cudaStream_t stream) {
  switch (out_dtype) {
    case KLD_F32: return unpack_typed<KLD_F32>(codes, heads, N, V, out, sm_count, stream);
    case KLD_BF16: return unpack_typed<KLD_BF16>(codes, heads, N, V, out, sm_count, stream);
    case KLD_F16: return unpack_typed<KLD_F16>(codes, heads, N, V, out, sm_count, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace kld
