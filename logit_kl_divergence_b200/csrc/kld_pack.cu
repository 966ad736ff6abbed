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

// One pass over the logits: a thread holds 16 elements in registers, the 8
// lanes of a block agree on its extremes by three shuffles and each writes
// its 16 codes as one vector. Bound by HBM: it reads s and writes 1 + 1/32
// bytes per element. Blocks with -inf, NaN or a magnitude of 2^126 take the
// slow branch (the extremes test fails there and only there).
template <int DT, bool kAligned>
__global__ void __launch_bounds__(kThreads)
    kld_pack_kernel(const void* __restrict__ logits, int64_t N, int64_t V, int64_t nb,
                    uint8_t* __restrict__ codes, uint32_t* __restrict__ heads) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const int64_t upr = nb * kLanes;  // units per row
  const int64_t total = N * upr;
  const char* begin = static_cast<const char*>(logits);
  const char* end = begin + N * V * Type<DT>::kBytes;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
  // Warps run whole: the loop condition is the warp's first unit.
  for (int64_t u0 = static_cast<int64_t>(blockIdx.x) * kThreads + (threadIdx.x & ~31u); u0 < total;
       u0 += stride) {
    const int64_t u = u0 + lane;
    const bool live = u < total;
    const int64_t r = live ? u / upr : 0;
    const int64_t j = live ? (u - r * upr) * kUnit : 0;
    float x[kUnit];
    float lo = 0.f, hi = 0.f;
    bool masked = false, some = true, bad = false;
    if (live) {
      load_unit<DT, kAligned>(begin + r * V * Type<DT>::kBytes, j, V, begin, end, x);
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
    if (!live) continue;
    uint32_t head, c[4] = {0u, 0u, 0u, 0u};
    if (has_bad & group) {
      head = kBadHead;
    } else if (!(has_some & group)) {
      head = kMaskedHead;
    } else {
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
#pragma unroll
      for (int k = 0; k < kUnit; ++k) {
        uint32_t n = __float_as_uint(fmaf(x[k], up, kMagic)) - zero;
        if (masked && x[k] == neg_inf()) n = 0u;
        c[k >> 2] |= (n & 255u) << (8 * (k & 3));
      }
    }
    *reinterpret_cast<uint4*>(codes + u * kUnit) = make_uint4(c[0], c[1], c[2], c[3]);
    if ((lane & (kLanes - 1)) == 0) heads[u / kLanes] = head;
  }
}

// Restores the values: a thread writes one 16-byte vector of a row (E
// elements), so that stores are whole and in order whatever the row's
// alignment: a row that starts `off` elements into a vector has its codes
// shifted by as many bytes instead. Bound by HBM: reads 1 + 1/32 and writes
// the output's bytes per element.
template <int OT>
__global__ void __launch_bounds__(kThreads)
    kld_unpack_kernel(const uint8_t* __restrict__ codes, const uint32_t* __restrict__ heads,
                      int64_t N, int64_t V, int64_t nb, void* __restrict__ out) {
  constexpr int eb = Type<OT>::kBytes;
  constexpr int E = 16 / eb;
  constexpr int NW = E / 4;  // code words of a vector
  const int64_t upr = (V + E - 1) / E + 1;  // vectors that touch a row, at most
  const int64_t total = N * upr;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
  char* O = static_cast<char*>(out);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; t < total; t += stride) {
    const int64_t r = t / upr;
    char* row = O + r * V * eb;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / eb);
    const int64_t j = (t - r * upr) * E - off;  // first column of the vector
    if (j >= V) continue;
    const uint8_t* crow = codes + r * nb * kBlock;
    const uint32_t* hrow = heads + r * nb;
    if (j >= 0 && j + E <= V) {
      // The E code bytes from column j on: whole words, then a byte shift.
      const uint32_t* wp = reinterpret_cast<const uint32_t*>(crow + (j & ~static_cast<int64_t>(3)));
      const uint32_t bits = static_cast<uint32_t>(j & 3) * 8u;
      uint32_t w[NW + 1];
      if (NW == 2 && (j & 7) == 0) {
        const uint2 v = __ldcs(reinterpret_cast<const uint2*>(wp));
        w[0] = v.x;
        w[NW - 1] = v.y;
      } else {
#pragma unroll
        for (int k = 0; k < NW; ++k) w[k] = __ldg(wp + k);
      }
      w[NW] = bits ? __ldg(wp + NW) : 0u;
#pragma unroll
      for (int k = 0; k < NW; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], bits);
      const int64_t k0 = j / kBlock, k1 = (j + E - 1) / kBlock;
      float x[E];
      const Scale s0 = scale_of(__ldg(hrow + k0));
#pragma unroll
      for (int k = 0; k < NW; ++k) decode4(w[k], s0, x + 4 * k);
      if (k1 != k0) {  // the vector crosses into the next block
        const Scale s1 = scale_of(__ldg(hrow + k1));
        const int cut = static_cast<int>(k1 * kBlock - j);
        float y[E];
#pragma unroll
        for (int k = 0; k < NW; ++k) decode4(w[k], s1, y + 4 * k);
#pragma unroll
        for (int k = 0; k < E; ++k)
          if (k >= cut) x[k] = y[k];
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

int blocks_for(int64_t units, int sm_count) {
  const int64_t need = (units + kThreads - 1) / kThreads;
  const int64_t most = static_cast<int64_t>(sm_count) * 8;  // 8 CTAs of 256 threads fill an SM
  return static_cast<int>(need < most ? need : most);
}

template <int DT>
cudaError_t pack_typed(const void* logits, int64_t N, int64_t V, uint8_t* codes, uint32_t* heads,
                       int sm_count, cudaStream_t s) {
  const int64_t nb = (V + kBlock - 1) / kBlock;
  const int grid = blocks_for(N * nb * kLanes, sm_count);
  const bool aligned = (reinterpret_cast<uintptr_t>(logits) & 15u) == 0 &&
                       (N == 1 || V * Type<DT>::kBytes % 16 == 0);
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
  kld_unpack_kernel<OT><<<blocks_for(N * ((V + E - 1) / E + 1), sm_count), kThreads, 0, s>>>(
      codes, heads, N, V, nb, out);
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
