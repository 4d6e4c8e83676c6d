// The forms a latent row is held in (include/misa_latent.h) and the arithmetic
// between them and bf16.
//
// An e4m3 (e2m1) number, its bits moved to the top of bf16's exponent and
// mantissa fields, is that number times 2^-120 (2^-126): the fields line up, the
// exponents differ by the two biases, and subnormal numbers stay right because
// both fields are read the same way.  A bf16 product with 2^120 (2^126) gives the
// element and one with its scale element * 2^e, both exactly: at most 4
// significant bits, and an exponent that the writer's range of e keeps among the
// normal bf16 numbers.  A scale byte is itself the exponent field of its power of
// two: byte 255 is infinity, and its group's zeros become NaN; byte 0, which is
// never written, is 0.
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
template <uint32_t kSelect>   // bytes of a (0-3) and b (4-7) by nibble; 8 + i: the sign of byte i, eight times
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "n"(kSelect));
  return d;
}

// 2^(b - 127) twice.
__device__ __forceinline__ uint32_t kv_scale(uint32_t b) { return b * 0x00800080u; }

// Two entries as elements in bf16.  The element bytes go to the upper bytes of
// the two halves, the first one's sign between them; one arithmetic shift moves
// both, with the signs copied into the bits that the mask then clears.
template <int kPair>
__device__ __forceinline__ uint32_t element2_mx8(uint32_t w) {   // bytes 2 kPair, 2 kPair + 1
  const uint32_t x = kPair ? prmt<0x3A20>(w, 0u) : prmt<0x1800>(w, 0u);
  return mul_bf16x2((static_cast<int32_t>(x) >> 4) & 0x87F087F0u, 0x7B807B80u);
}
template <int kPair>
__device__ __forceinline__ uint32_t element2_mx4(uint32_t low, uint32_t w) {   // byte kPair; low = w << 4
  const uint32_t x = prmt<0x4800 | (kPair << 12) | (kPair << 8) | (kPair << 4)>(low, w);
  return mul_bf16x2((static_cast<int32_t>(x) >> 6) & 0x81C081C0u, 0x7E807E80u);
}

// Eight consecutive entries as bf16: codes in w0 (and w1 for MX8), scale = kv_scale.
template <int kFmt>
__device__ __forceinline__ uint4 kv_decode8(uint32_t w0, uint32_t w1, uint32_t scale) {
  if (kFmt == MISA_KV_MX8)
    return make_uint4(mul_bf16x2(element2_mx8<0>(w0), scale), mul_bf16x2(element2_mx8<1>(w0), scale),
                      mul_bf16x2(element2_mx8<0>(w1), scale), mul_bf16x2(element2_mx8<1>(w1), scale));
  const uint32_t low = w0 << 4;
  return make_uint4(mul_bf16x2(element2_mx4<0>(low, w0), scale), mul_bf16x2(element2_mx4<1>(low, w0), scale),
                    mul_bf16x2(element2_mx4<2>(low, w0), scale), mul_bf16x2(element2_mx4<3>(low, w0), scale));
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
