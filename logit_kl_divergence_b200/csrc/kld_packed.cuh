// kld_packed.cuh -- the 8-bit logit checkpoint's format and the element
// access shared by the kernels that write and read it (kld_pack.cu,
// kld_packed_rows.cu). Device code only.
//
// Format. A row of V logits is cut into blocks of kBlock = 128 columns (the
// last one padded), each with one 32-bit header and 128 one-byte codes. A
// block's values are whole multiples of a power of two, its step 2^e:
//
//   n_j  = rint(x_j / 2^e),   base = min_j n_j - 1,   code_j = n_j - base,
//   value_j = (base + code_j) * 2^e,    |value_j - x_j| <= 2^(e-1),
//
// code 0 stands for -inf, e is the smallest integer >= floor(log2 max|x|) - 20
// (and >= -126) for which every code fits in 1..255. Scaling by a power of
// two and rounding to whole numbers below 2^22 are exact in fp32, so a code
// is decided by no rounded quantity (any fp32 or fp64 evaluation gives the
// same bits) and every value is an fp32 number. The price against a freely
// chosen step is a step up to twice as long (1.44 times on average). Only
// values on the step's grid are stored exactly; the others are off by at most
// R / 254 where the block spans R, or 2^-21 max|x| where that is more.
//   header = base << 9 | (some code is 0) << 8 | (e + 128)
// The low byte is 2..248 for a block with an unmasked entry, 0 for a fully
// masked one (header 256) and 255 for a block that held NaN, +inf or a
// magnitude of 2^126 or more (kBadHead; its values read as NaN).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "kld_stats.h"

namespace kld {
namespace packed {

constexpr int kBlock = 128;
constexpr uint32_t kMaskedHead = 256u;
constexpr uint32_t kBadHead = 0x1ffu;  // base 0, some code is 0, low byte 255
constexpr float kLimit = 8.507059173023462e37f;  // 2^126

// One block's decoding constants: value = (2^23 + code + shift) * step, where
// shift = base - 2^23 (|shift| < 2^24) and the sum are exact.
struct Scale {
  float step, shift;
  bool masked;  // some code is 0: those entries are -inf
  __device__ __forceinline__ float value(float magic) const { return (magic + shift) * step; }
};
__device__ __forceinline__ Scale scale_of(uint32_t head) {
  Scale s;
  const uint32_t eb = head & 255u;
  // The step's exponent field: e + 127 = eb - 1; a bad block's (255) is NaN,
  // a masked block's (0) is not used.
  const uint32_t field = eb == 255u ? 0x7fc00000u : (eb - 1u) << 23;
  s.step = eb == 0u ? 1.f : __uint_as_float(field);
  s.shift = static_cast<float>((static_cast<int32_t>(head) >> 9) - (1 << 23));
  s.masked = (head & 256u) != 0u && eb != 255u;
  return s;
}
// A block that is not special has no masks or bad values (bit 8 of its header
// is 0) and a step below 2^96 (a low byte below 224: adding 32 does not reach
// bit 8). Bit 8 of this, or of an OR of several, tells.
__device__ __forceinline__ uint32_t special_bits(uint32_t head) { return head | (head + 32u); }
// Decoding constants of such a block, value = (2^23 + code) * step + off with
// off = (base - 2^23) * step exact, in a few integer and FMA-pipe operations:
// the step's bits are the low byte less one in the exponent field; 1.5 * 2^23 +
// base is made by its bits. A step past 2^104 can make off, and with it every
// value, -inf, and does nothing else wrong.
__device__ __forceinline__ void plain_scale(uint32_t head, float& step, float& off) {
  step = __uint_as_float(head * 0x00800000u - 0x00800000u);
  const float b = __uint_as_float(0x4b400000u + static_cast<uint32_t>(static_cast<int32_t>(head) >> 9));
  off = (b - 20971520.f) * step;  // base - 2^23, exactly
}
// Byte k of w as the float 2^23 + byte, in one byte permute (written out:
// the compiler's own choice took 1.5 to 2 instructions).
template <int K>
__device__ __forceinline__ float magic_byte(uint32_t w) {
  uint32_t y;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(y) : "r"(w), "r"(0x4b000000u), "n"(0x7650 + K));
  return __uint_as_float(y);
}
__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xff800000u); }

// The value of a code of any block.
__device__ __forceinline__ float decode1(uint32_t code, uint32_t head) {
  const Scale s = scale_of(head);
  const float v = s.value(__uint_as_float(0x4b000000u | code));
  return s.masked && code == 0u ? neg_inf() : v;
}

// ------------------------------------------------------------ element types

template <int DT>
struct Type;
template <>
struct Type<KLD_F32> {
  static constexpr int kBytes = 4;
  __device__ static float load(const void* p) { return __ldg(static_cast<const float*>(p)); }
  __device__ static void store(void* p, float x) { *static_cast<float*>(p) = x; }
  // 16 elements from 16 words.
  __device__ static void unpack16(const uint32_t* w, float* o) {
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] = __uint_as_float(w[k]);
  }
  // A 16-byte vector of elements.
  __device__ static uint4 vec(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};
template <>
struct Type<KLD_BF16> {
  static constexpr int kBytes = 2;
  __device__ static float load(const void* p) {
    return __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const unsigned short*>(p))) << 16);
  }
  __device__ static void store(void* p, float x) {
    *static_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(x);
  }
  __device__ static void unpack16(const uint32_t* w, float* o) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      o[2 * k] = __uint_as_float(w[k] << 16);
      o[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
  __device__ static uint4 vec(const float* x) {
    uint4 v;
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
      w[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return v;
  }
};
template <>
struct Type<KLD_F16> {
  static constexpr int kBytes = 2;
  __device__ static float load(const void* p) {
    return __half2float(__ushort_as_half(__ldg(static_cast<const unsigned short*>(p))));
  }
  __device__ static void store(void* p, float x) { *static_cast<__half*>(p) = __float2half_rn(x); }
  __device__ static void unpack16(const uint32_t* w, float* o) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
      o[2 * k] = f.x;
      o[2 * k + 1] = f.y;
    }
  }
  __device__ static uint4 vec(const float* x) {
    uint4 v;
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __half2 h = __floats2half2_rn(x[2 * k], x[2 * k + 1]);
      w[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return v;
  }
};

// NW words that start `mis` bytes (0 <= mis < 16) into the NW + 4 words w:
// a two-stage shift by whole words, then a funnel shift by bytes, which a mis
// that is a multiple of 4 (kWords) does not need.
template <int NW, bool kWords = false>
__device__ __forceinline__ void shift_bytes(uint32_t* w, uint32_t mis) {
  const bool two = (mis & 8u) != 0u, one = (mis & 4u) != 0u;
#pragma unroll
  for (int i = 0; i < NW + 2; ++i) w[i] = two ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < NW + 1; ++i) w[i] = one ? w[i + 1] : w[i];
  if constexpr (!kWords) {
    const uint32_t bits = (mis & 3u) * 8u;
#pragma unroll
    for (int i = 0; i < NW; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], bits);
  }
}

}  // namespace packed
}  // namespace kld
