// kld_pack.cu -- writing and restoring the 8-bit logit checkpoint (format
// and its arithmetic: kld_packed.cuh).
#include <cmath>
#include <type_traits>

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
// Units of a lane in a group, 32 apart, loaded together as they lie in memory
// (as many as 64 registers hold). Measured at 2048 rows: bf16 rows of 151936
// 157 us with three, 166 with two, 207 with four; fp32 244 us with two, 247
// with one; shifted bf16 rows of 131073 169 us with one, 178 with two.
template <int DT, bool kAligned>
constexpr int kPackUnits = kAligned ? (Type<DT>::kBytes == 2 ? 3 : 2) : 1;
constexpr int kUnpackUnits = 4;  // 2048 x 151936 to fp32 251 us, with two 298, with eight 249 (bf16 of 131073: 147, 171, 158)

// 16 elements of a row from column j on, as they lie in memory. Full units
// whose 16-byte vectors lie inside the tensor [begin, end) take vector loads,
// shifted into place where the row does not start on a 16-byte boundary; the
// others go element by element, -inf past V.
template <int DT, bool kAligned>
__device__ __forceinline__ void load_unit(const char* row, int64_t j, int64_t V,
                                          const char* begin, const char* end, uint32_t* raw) {
  constexpr int eb = Type<DT>::kBytes;
  constexpr int nv = kUnit * eb / 16;
  const char* p = row + j * eb;
  if (kAligned) {
    if (j + kUnit <= V) {
#pragma unroll
      for (int k = 0; k < nv; ++k) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p) + k);
        raw[4 * k] = v.x;
        raw[4 * k + 1] = v.y;
        raw[4 * k + 2] = v.z;
        raw[4 * k + 3] = v.w;
      }
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
#pragma unroll
      for (int k = 0; k < 4 * nv; ++k) raw[k] = w[k];
      return;
    }
  }
  if constexpr (eb == 4) {
#pragma unroll
    for (int k = 0; k < kUnit; ++k)
      raw[k] = j + k < V ? reinterpret_cast<const uint32_t*>(p)[k] : 0xff800000u;
  } else {
    constexpr uint32_t none = DT == KLD_BF16 ? 0xff80u : 0xfc00u;
#pragma unroll
    for (int k = 0; k < kUnit; k += 2) {
      const uint16_t* e = reinterpret_cast<const uint16_t*>(p) + k;
      raw[k / 2] = (j + k < V ? e[0] : none) | (j + k + 1 < V ? e[1] : none) << 16;
    }
  }
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
  uint32_t has_mask = 0u;
  bool none = false, any_bad = false;  // of the lane's block
  if (__any_sync(0xffffffffu, masked || bad || !some)) {
    const unsigned group = 0xffu << (lane & 24);
    has_mask = __ballot_sync(0xffffffffu, masked) & group ? 256u : 0u;
    none = !(__ballot_sync(0xffffffffu, some) & group);
    any_bad = __ballot_sync(0xffffffffu, bad) & group;
  }
  uint32_t c[4] = {0u, 0u, 0u, 0u};
  if (any_bad) {
    head = kBadHead;
  } else if (none) {
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
    const int even = base + (base & 1);
    head = static_cast<uint32_t>(base) << 9 | has_mask | static_cast<uint32_t>(e + 128);
    // The low byte of x * up + kMagic - even is n - even: the sum has steps of
    // one, and an even shift keeps ties where they are. Bytes rise by the
    // odd one that is left without a carry (codes are at most 255).
    const float zero = kMagic - static_cast<float>(even);
    const uint32_t odd = (base & 1) ? 0x01010101u : 0u;
    uint32_t n[kUnit];
#pragma unroll
    for (int k = 0; k < kUnit; ++k) n[k] = __float_as_uint(fmaf(x[k], up, zero));
#pragma unroll
    for (int k = 0; k < 4; ++k)  // the low bytes, four to a word
      c[k] = __byte_perm(__byte_perm(n[4 * k], n[4 * k + 1], 0x0040),
                         __byte_perm(n[4 * k + 2], n[4 * k + 3], 0x0040), 0x5410) + odd;
    if (masked) {
#pragma unroll
      for (int k = 0; k < kUnit; ++k)
        if (x[k] == neg_inf()) c[k / 4] &= ~(0xffu << 8 * (k % 4));
    }
  }
  out = make_uint4(c[0], c[1], c[2], c[3]);
}

// One pass over the logits: a lane holds kPackUnits units of 16 elements in
// registers and writes each one's codes as one vector. Bound by HBM: it reads
// s and writes 1 + 1/32 bytes per element; 2048 x 151936 bf16 in 157 us, 6.0
// TB/s (fp32 244 us, 6.4 TB/s). kMask: entries at or below mask_at become -inf.
template <int DT, bool kAligned, bool kMask>
__global__ void __launch_bounds__(kThreads)
    kld_pack_kernel(const void* __restrict__ logits, int64_t N, int64_t V, int64_t nb, float mask_at,
                    uint8_t* __restrict__ codes, uint32_t* __restrict__ heads) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const uint32_t upr = static_cast<uint32_t>(nb * kLanes);  // units per row
  constexpr int kUnits = kPackUnits<DT, kAligned>;
  const uint32_t per = (upr + 32 * kUnits - 1) / (32 * kUnits);
  const char* begin = static_cast<const char*>(logits);
  const char* end = begin + N * V * Type<DT>::kBytes;
  constexpr int kWarps = kThreads / 32;
  const Steps stride(static_cast<int64_t>(gridDim.x) * kWarps, per);
  for (Steps at(static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5), per); at.row < N;
       at.add(stride, per)) {
    const char* row = begin + at.row * V * Type<DT>::kBytes;
    const uint32_t u0 = at.group * (32 * kUnits) + lane;
    uint32_t raw[kUnits][kUnit * Type<DT>::kBytes / 4];
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
      if (u0 + 32 * i < upr)
        load_unit<DT, kAligned>(row, static_cast<int64_t>(u0 + 32 * i) * kUnit, V, begin, end, raw[i]);
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const uint32_t u = u0 + 32 * i;
      float x[kUnit];
      Type<DT>::unpack16(raw[i], x);
      if constexpr (kMask) {
#pragma unroll
        for (int k = 0; k < kUnit; ++k) x[k] = x[k] <= mask_at ? neg_inf() : x[k];
      }
      uint32_t head;
      uint4 c;
      pack_unit(x, u < upr, lane, head, c);
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
// shifted by as many bytes instead (kOff). A group of vectors whose blocks are
// all plain has neither checks nor masks between its loads and its stores.
// Bound by HBM: reads 1 + 1/32 and writes the output's bytes per element; 2048 x
// 151936 to fp32 in 251 us, 6.2 TB/s (bf16 150 us, 6.3 TB/s).
template <int OT, bool kOff>
__global__ void __launch_bounds__(kThreads)
    kld_unpack_kernel(const uint8_t* __restrict__ codes, const uint32_t* __restrict__ heads,
                      int64_t N, int64_t V, int64_t nb, void* __restrict__ out) {
  constexpr int eb = Type<OT>::kBytes;
  constexpr int E = 16 / eb;
  constexpr int NW = E / 4;       // code words of a vector
  constexpr int kStep = 32 * E;   // columns of a warp's vectors, a whole number of blocks
  const uint32_t upr = static_cast<uint32_t>((V + E - 1) / E + (kOff ? 1 : 0));  // vectors that touch a row, at most
  const uint32_t per = (upr + 32 * kUnpackUnits - 1) / (32 * kUnpackUnits);
  constexpr int kWarps = kThreads / 32;
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const Steps stride(static_cast<int64_t>(gridDim.x) * kWarps, per);
  for (Steps at(static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5), per); at.row < N;
       at.add(stride, per)) {
    char* row = static_cast<char*>(out) + at.row * V * eb;
    const int off = kOff ? static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / eb) : 0;
    const uint8_t* crow = codes + at.row * nb * kBlock;
    const uint32_t* hrow = heads + at.row * nb;
    const int64_t first = static_cast<int64_t>(at.group) * (kStep * kUnpackUnits) - off;
    const int64_t j0 = first + lane * E;
    char* dst = row + j0 * eb;
    bool whole = first >= 0 && first + kStep * kUnpackUnits <= V;
    if (whole) {
      // All of the group lies in the row; codes and headers are on their way
      // before the first is used.
      uint32_t w[kUnpackUnits][NW + 1], h0[kUnpackUnits], h1[kUnpackUnits], special = 0u;
      const uint32_t* wp = reinterpret_cast<const uint32_t*>(crow + (j0 & ~static_cast<int64_t>(3)));
      const uint32_t* hp = hrow + j0 / kBlock;
      const int more = static_cast<int>((j0 + E - 1) / kBlock - j0 / kBlock);  // the last column's block
      const uint32_t bits = static_cast<uint32_t>(j0 & 3) * 8u;
#pragma unroll
      for (int i = 0; i < kUnpackUnits; ++i) {
        if (NW == 2 && !kOff) {
          const uint2 v = __ldcs(reinterpret_cast<const uint2*>(wp + i * (kStep / 4)));
          w[i][0] = v.x;
          w[i][NW - 1] = v.y;
        } else {
#pragma unroll
          for (int k = 0; k < NW; ++k) w[i][k] = __ldg(wp + i * (kStep / 4) + k);
          if (kOff) w[i][NW] = bits ? __ldg(wp + i * (kStep / 4) + NW) : 0u;
        }
        h0[i] = __ldg(hp + i * (kStep / kBlock));
        h1[i] = kOff ? __ldg(hp + i * (kStep / kBlock) + more) : h0[i];
      }
#pragma unroll
      for (int i = 0; i < kUnpackUnits; ++i) special |= special_bits(h0[i]) | special_bits(h1[i]);
      whole = !(special & 256u);
      if (whole) {
        const int cut = kBlock - static_cast<int>(j0 & (kBlock - 1));  // the first block's columns
#pragma unroll
        for (int i = 0; i < kUnpackUnits; ++i) {
          float x[E], a0, b0, a1, b1;
          plain_scale(h0[i], a0, b0);
          if (kOff) plain_scale(h1[i], a1, b1);
#pragma unroll
          for (int k = 0; k < E; ++k) {
            if (kOff && k % 4 == 0) w[i][k / 4] = __funnelshift_r(w[i][k / 4], w[i][k / 4 + 1], bits);
            const uint32_t y = w[i][k / 4];
            const float m = k % 4 == 0 ? magic_byte<0>(y) : (k % 4 == 1 ? magic_byte<1>(y)
                          : (k % 4 == 2 ? magic_byte<2>(y) : magic_byte<3>(y)));
            x[k] = kOff ? fmaf(m, k < cut ? a0 : a1, k < cut ? b0 : b1) : fmaf(m, a0, b0);
          }
          __stcs(reinterpret_cast<uint4*>(dst + i * (32 * 16)), Type<OT>::vec(x));
        }
      }
    }
    if (!whole) {
      // a row's ends, special blocks
#pragma unroll 1
      for (int i = 0; i < kUnpackUnits; ++i) {
        const int64_t j = j0 + i * kStep;
        float x[E];
#pragma unroll
        for (int k = 0; k < E; ++k)
          x[k] = j + k >= 0 && j + k < V ? decode1(crow[j + k], __ldg(hrow + (j + k) / kBlock)) : 0.f;
        if (j >= 0 && j + E <= V) {
          __stcs(reinterpret_cast<uint4*>(dst + i * (32 * 16)), Type<OT>::vec(x));
        } else {
#pragma unroll
          for (int k = 0; k < E; ++k)
            if (j + k >= 0 && j + k < V) Type<OT>::store(row + (j + k) * eb, x[k]);
        }
      }
    }
  }
}

// CTAs for so many groups of a warp: enough for every SM several times over,
// so that the last ones to finish weigh little (2048 x 151936 fp32: 32 a SM
// 244 us, 8 a SM 254 us).
int blocks_for(int64_t groups, int sm_count) {
  const int64_t need = (groups + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t most = static_cast<int64_t>(sm_count) * 32;
  return static_cast<int>(need < most ? need : most);
}

template <int DT, bool kMask>
cudaError_t pack_typed(const void* logits, int64_t N, int64_t V, float mask_at, uint8_t* codes,
                       uint32_t* heads, int sm_count, cudaStream_t s) {
  const int64_t nb = (V + kBlock - 1) / kBlock;
  const bool aligned = (reinterpret_cast<uintptr_t>(logits) & 15u) == 0 &&
                       (N == 1 || V * Type<DT>::kBytes % 16 == 0);
  const int64_t group = 32 * (aligned ? kPackUnits<DT, true> : kPackUnits<DT, false>);
  const int grid = blocks_for(N * ((nb * kLanes + group - 1) / group), sm_count);
  if (aligned)
    kld_pack_kernel<DT, true, kMask><<<grid, kThreads, 0, s>>>(logits, N, V, nb, mask_at, codes, heads);
  else
    kld_pack_kernel<DT, false, kMask><<<grid, kThreads, 0, s>>>(logits, N, V, nb, mask_at, codes, heads);
  return cudaGetLastError();
}

template <int OT>
cudaError_t unpack_typed(const uint8_t* codes, const uint32_t* heads, int64_t N, int64_t V,
                         void* out, int sm_count, cudaStream_t s) {
  constexpr int E = 16 / Type<OT>::kBytes;
  const int64_t nb = (V + kBlock - 1) / kBlock;
  const bool aligned = (reinterpret_cast<uintptr_t>(out) & 15u) == 0 && (N == 1 || V * Type<OT>::kBytes % 16 == 0);
  const int64_t vectors = (V + E - 1) / E + (aligned ? 0 : 1);
  const int grid = blocks_for(N * ((vectors + 32 * kUnpackUnits - 1) / (32 * kUnpackUnits)), sm_count);
  if (aligned)
    kld_unpack_kernel<OT, false><<<grid, kThreads, 0, s>>>(codes, heads, N, V, nb, out);
  else
    kld_unpack_kernel<OT, true><<<grid, kThreads, 0, s>>>(codes, heads, N, V, nb, out);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_pack(const void* logits, int64_t N, int64_t V, kld_dtype_t dtype, float mask_at,
                        uint8_t* codes, uint32_t* heads, int sm_count, cudaStream_t stream) {
  auto typed = [&](auto kind) {
    constexpr int DT = decltype(kind)::value;
    // as the logits hold it: -1e9 in bf16 is a little above -1e9
    if (DT == KLD_BF16) mask_at = __bfloat162float(__float2bfloat16_rn(mask_at));
    if (DT == KLD_F16) mask_at = __half2float(__float2half_rn(mask_at));
    return mask_at > -INFINITY
               ? pack_typed<DT, true>(logits, N, V, mask_at, codes, heads, sm_count, stream)
               : pack_typed<DT, false>(logits, N, V, mask_at, codes, heads, sm_count, stream);
  };
  switch (dtype) {
    case KLD_F32: return typed(std::integral_constant<int, KLD_F32>{});
    case KLD_BF16: return typed(std::integral_constant<int, KLD_BF16>{});
    case KLD_F16: return typed(std::integral_constant<int, KLD_F16>{});
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
