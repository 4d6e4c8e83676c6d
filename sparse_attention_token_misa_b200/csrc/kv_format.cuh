// The forms a latent row is held in (include/misa_latent.h) and the arithmetic
// between them and bf16.
//
// An e4m3 (e2m1) number, its bits moved to the top of bf16's exponent and
// mantissa fields, is that number times 2^-120 (2^-126): the fields line up, the
// exponents differ by the two biases, and subnormal numbers stay right because
// both fields are read the same way.  One bf16 product with a power of two then
// gives element * 2^e, exactly: at most 4 significant bits, and an exponent that
// the writer's range of e keeps among the normal bf16 numbers.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "../../include/misa_latent.h"

namespace misa {

constexpr int kKvGroup = 32;                          // entries of one scale
constexpr int kKvGroups = MISA_MLA_DV / kKvGroup;     // 16 scale bytes a row
constexpr int kKvRope = MISA_MLA_DQK - MISA_MLA_DV;   // 64 rotary entries, always bf16

__host__ __device__ constexpr int kv_code_bytes(int fmt) {
  return fmt == MISA_KV_BF16 ? MISA_MLA_DV * 2 : fmt == MISA_KV_MX8 ? MISA_MLA_DV : MISA_MLA_DV / 2;
}
// byte offset of the rotary entries, and the row's bytes (a multiple of 16)
__host__ __device__ constexpr int kv_rope_offset(int fmt) {
  return kv_code_bytes(fmt) + (fmt == MISA_KV_BF16 ? 0 : kKvGroups);
}
__host__ __device__ constexpr int kv_row_bytes(int fmt) { return kv_rope_offset(fmt) + kKvRope * 2; }

#ifdef __CUDACC__

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf16x2_of(uint32_t bits) { return bits | (bits << 16); }

// What scale byte b multiplies the moved bits by: 2^(b - 127 + shift), shift =
// 120 or 126, as one factor while that is a bf16 number and as two behind it
// (`second`, else 0).  Byte 255 is NaN.
template <int kFmt>
__device__ __forceinline__ uint32_t kv_scale(uint32_t b, uint32_t* second) {
  constexpr uint32_t kShift = kFmt == MISA_KV_MX8 ? 120u : 126u;
  *second = 0u;
  if (b + kShift <= 254u) return bf16x2_of((b + kShift) << 7);
  if (b == 255u) return bf16x2_of(0x7FC0u);
  *second = bf16x2_of((b + kShift - 127u) << 7);
  return bf16x2_of(254u << 7);
}

// Two entries of the pair of bytes (MX8) or of byte (MX4) `kPair` of w, moved to bf16 fields.
template <int kPair>
__device__ __forceinline__ uint32_t moved_mx8(uint32_t w) {   // bytes 2 kPair, 2 kPair + 1
  const uint32_t x = __byte_perm(w, 0u, kPair ? 0x3424 : 0x1404);
  return (x & 0x80008000u) | ((x >> 4) & 0x07F007F0u);
}
template <int kPair>
__device__ __forceinline__ uint32_t moved_mx4(uint32_t low, uint32_t w) {   // low = w << 4
  const uint32_t x = __byte_perm(low, w, 0x4000 | (kPair << 12) | (kPair << 4));   // bytes 1 and 3: the even and odd entry
  return (x & 0x80008000u) | ((x >> 6) & 0x01C001C0u);
}

// Eight consecutive entries as bf16: codes in w0 (and w1 for MX8).
template <int kFmt>
__device__ __forceinline__ uint4 kv_decode8(uint32_t w0, uint32_t w1, uint32_t scale, uint32_t second) {
  uint4 y;
  if (kFmt == MISA_KV_MX8) {
    y = make_uint4(moved_mx8<0>(w0), moved_mx8<1>(w0), moved_mx8<0>(w1), moved_mx8<1>(w1));
  } else {
    const uint32_t low = w0 << 4;
    y = make_uint4(moved_mx4<0>(low, w0), moved_mx4<1>(low, w0), moved_mx4<2>(low, w0), moved_mx4<3>(low, w0));
  }
  y = make_uint4(mul_bf16x2(y.x, scale), mul_bf16x2(y.y, scale), mul_bf16x2(y.z, scale), mul_bf16x2(y.w, scale));
  if (second)
    y = make_uint4(mul_bf16x2(y.x, second), mul_bf16x2(y.y, second), mul_bf16x2(y.z, second), mul_bf16x2(y.w, second));
  return y;
}

// Scale byte of a group whose largest |entry| has these bf16 bits (sign clear):
// e = the smallest with amax <= 448 * 2^e (6 * 2^e), clamped.  448 = 1.75 * 2^8
// and 6 = 1.5 * 2^2, so e is amax's exponent - 8 (2), one more if its mantissa is
// above 1.75 (1.5).
template <int kFmt>
__device__ __forceinline__ uint32_t kv_scale_byte(uint32_t amax) {
  if (amax >= 0x7F80u) return 255u;
  constexpr int kTop = kFmt == MISA_KV_MX8 ? 8 : 2;
  constexpr uint32_t kMant = kFmt == MISA_KV_MX8 ? 0x60u : 0x40u;
  constexpr int kMax = (kFmt == MISA_KV_MX8 ? 119 : 125) + 127;
  const int b = static_cast<int>(amax >> 7) - kTop + ((amax & 0x7Fu) > kMant ? 1 : 0);
  return static_cast<uint32_t>(b < 10 ? 10 : b > kMax ? kMax : b);   // 10 = -117 + 127
}

#endif  // __CUDACC__

}  // namespace misa
