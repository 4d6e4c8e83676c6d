// The latent cache written and read back (include/misa_latent.h).
//
// Both kernels are one pass over the rows and bound by HBM.  A thread takes 16
// bytes of bf16, eight entries: 64 such pieces of latent entries and 8 of rotary
// ones make a row of 72, so the four pieces that share a scale are four
// neighbouring lanes of one warp (72 and 32 are multiples of 4).
#include "kv_format.cuh"
#include "launch.h"
#include "misa_device.cuh"

namespace misa {

namespace {

constexpr int kPieces = MISA_MLA_DQK / 8;      // 72
constexpr int kCodePieces = MISA_MLA_DV / 8;   // 64
constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint32_t d;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tcvt.u32.u8 %0, b;\n\t}" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

template <int kFmt>
__global__ void __launch_bounds__(kThreads)
append_kv_kernel(const uint16_t* __restrict__ rows, int64_t npieces, int n_new, const int32_t* __restrict__ counts,
                 const int32_t* __restrict__ len, uint8_t* __restrict__ cache, int64_t seq_stride, int64_t L_cap,
                 uint32_t* err) {
  constexpr int kRow = kv_row_bytes(kFmt);
  pdl_wait_inputs();
  pdl_allow_next();
  const int64_t g = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (g >= npieces) return;   // npieces is a multiple of 4: the lanes of a group leave together
  const int64_t row = g / kPieces;
  const int piece = static_cast<int>(g - row * kPieces);
  const int b = static_cast<int>(row / n_new);
  const int i = static_cast<int>(row - static_cast<int64_t>(b) * n_new);
  const int64_t l0 = len[b];
  const int cnt = counts ? counts[b] : n_new;
  if (cnt < 0 || cnt > n_new || l0 < 0 || l0 + cnt > L_cap) {
    if (i == 0 && piece == 0) record_error(err, MISA_DEVERR_BAD_LEN);
    return;
  }
  if (i >= cnt) return;
  const uint4 x = __ldcs(reinterpret_cast<const uint4*>(rows) + g);
  uint8_t* dst = cache + static_cast<int64_t>(b) * seq_stride + (l0 + i) * kRow;
  if (kFmt == MISA_KV_BF16) {
    *reinterpret_cast<uint4*>(dst + piece * 16) = x;
    return;
  }
  if (piece >= kCodePieces) {
    *reinterpret_cast<uint4*>(dst + kv_rope_offset(kFmt) + (piece - kCodePieces) * 16) = x;
    return;
  }
  // the largest of |entry| as bf16 bits: they order as the numbers do, infinity and NaN on top
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) amax = max(amax, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
  const unsigned quad = 0xFu << (threadIdx.x & 28);
  amax = max(amax, __shfl_xor_sync(quad, amax, 1));
  amax = max(amax, __shfl_xor_sync(quad, amax, 2));
  const uint32_t sb = kv_scale_byte<kFmt>(amax);
  // 2^-e, a normal fp32 number; a group with an infinity or NaN holds zeros under its scale byte
  const float inv = sb == 255u ? 0.f : __uint_as_float((254u - sb) << 23);
  uint32_t code[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float lo = sb == 255u ? 0.f : __uint_as_float(w[j] << 16) * inv;
    const float hi = sb == 255u ? 0.f : __uint_as_float(w[j] & 0xFFFF0000u) * inv;
    code[j] = kFmt == MISA_KV_MX8 ? e4m3x2(lo, hi) : e2m1x2(lo, hi);
  }
  if (kFmt == MISA_KV_MX8)
    *reinterpret_cast<uint2*>(dst + piece * 8) = make_uint2(code[0] | (code[1] << 16), code[2] | (code[3] << 16));
  else
    *reinterpret_cast<uint32_t*>(dst + piece * 4) = code[0] | (code[1] << 8) | (code[2] << 16) | (code[3] << 24);
  if ((piece & 3) == 0) dst[kv_code_bytes(kFmt) + (piece >> 2)] = static_cast<uint8_t>(sb);
}

struct ReadParams {
  const uint8_t* cache;
  int64_t nseq, seq_stride, L;
  const int32_t* seq_of;
  const int32_t* idx;
  int64_t idx_stride;
  const int32_t* first;
  const int32_t* prefix_len;
  int64_t n, npieces;
  uint16_t* out;
  uint32_t* err;
};

template <int kFmt>
__global__ void __launch_bounds__(kThreads) read_kv_kernel(const ReadParams p) {
  constexpr int kRow = kv_row_bytes(kFmt);
  pdl_wait_inputs();
  pdl_allow_next();
  const int64_t g = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (g >= p.npieces) return;
  const int64_t row = g / kPieces;
  const int piece = static_cast<int>(g - row * kPieces);
  const int64_t t = row / p.n;
  const int64_t i = row - t * p.n;
  const int64_t seq = p.seq_of[t];
  int64_t s = -1;
  if (seq < 0 || seq >= p.nseq) {
    if (piece == 0 && i == 0) record_error(p.err, MISA_DEVERR_BAD_SEQ);
  } else if (p.idx) {
    s = p.idx[t * p.idx_stride + i];
    if (s < -1 || s >= p.L) {
      if (piece == 0) record_error(p.err, MISA_DEVERR_BAD_INDEX);
      s = -1;
    }
  } else {
    const int64_t f = p.first ? p.first[t] : 0;
    if (f < 0) {
      if (piece == 0 && i == 0) record_error(p.err, MISA_DEVERR_BAD_INDEX);
    } else {
      const int64_t end = p.prefix_len && p.prefix_len[t] < p.L ? p.prefix_len[t] : p.L;
      if (f + i < end) s = f + i;
    }
  }
  uint4 y = make_uint4(0u, 0u, 0u, 0u);
  if (s >= 0) {
    const uint8_t* src = p.cache + seq * p.seq_stride + s * kRow;
    if (kFmt == MISA_KV_BF16) {
      y = *reinterpret_cast<const uint4*>(src + piece * 16);
    } else if (piece >= kCodePieces) {
      y = *reinterpret_cast<const uint4*>(src + kv_rope_offset(kFmt) + (piece - kCodePieces) * 16);
    } else {
      uint2 c;
      if (kFmt == MISA_KV_MX8) c = *reinterpret_cast<const uint2*>(src + piece * 8);
      else c = make_uint2(*reinterpret_cast<const uint32_t*>(src + piece * 4), 0u);
      y = kv_decode8<kFmt>(c.x, c.y, kv_scale(src[kv_code_bytes(kFmt) + (piece >> 2)]));
    }
  }
  __stcs(reinterpret_cast<uint4*>(p.out) + g, y);
}

}  // namespace

cudaError_t launch_append_kv(const uint16_t* rows, int64_t nseq, int n_new, const int32_t* counts, const int32_t* len,
                             int fmt, void* cache, int64_t seq_stride, int64_t L_cap, uint32_t* err,
                             cudaStream_t stream) {
  const int64_t npieces = nseq * n_new * kPieces;
  const int64_t ctas = (npieces + kThreads - 1) / kThreads;
  auto kern = fmt == MISA_KV_BF16  ? append_kv_kernel<MISA_KV_BF16>
              : fmt == MISA_KV_MX8 ? append_kv_kernel<MISA_KV_MX8>
                                   : append_kv_kernel<MISA_KV_MX4>;
  return launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, stream, 0, rows, npieces, n_new, counts,
                    len, static_cast<uint8_t*>(cache), seq_stride, L_cap, err);
}

cudaError_t launch_read_kv(const void* cache, int fmt, int64_t nseq, int64_t seq_stride, int64_t L,
                           const int32_t* seq_of, int T, const int32_t* idx, int64_t idx_stride, const int32_t* first,
                           const int32_t* prefix_len, int64_t n, uint16_t* out, uint32_t* err, cudaStream_t stream) {
  ReadParams p = {static_cast<const uint8_t*>(cache), nseq, seq_stride, L, seq_of, idx, idx_stride, first, prefix_len,
                  n, static_cast<int64_t>(T) * n * kPieces, out, err};
  const int64_t ctas = (p.npieces + kThreads - 1) / kThreads;
  auto kern = fmt == MISA_KV_BF16  ? read_kv_kernel<MISA_KV_BF16>
              : fmt == MISA_KV_MX8 ? read_kv_kernel<MISA_KV_MX8>
                                   : read_kv_kernel<MISA_KV_MX4>;
  return launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, stream, 0, p);
}

}  // namespace misa
