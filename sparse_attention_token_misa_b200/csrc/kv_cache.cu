// The latent cache written and read back (include/misa_latent.h).
//
// Both kernels are one pass over the rows and bound by HBM, if few enough
// instructions go into a row (writing mx4 takes 0.70 of the issue slots, reading 0.39).  A warp takes several rows, four at a time: its lanes
// first find a row each (its sequence, its place in the cache), then all lanes take
// each of the four rows' 64 pieces of eight latent entries, two pieces a lane, and
// the 4 x 8 rotary pieces once.  The four pieces that share a scale are four
// neighbouring lanes.  (A thread that found its own piece's row spent more on that
// than on the piece: 65,536 rows of mx4 took 35 us to read.)  Measured, 65,536 rows
// with the cache not in L2: mx8 118 MB read in 20.5 us (5.8 TB/s), listed rows 22.6,
// written 22.6; mx4 102 MB 18.4, 20.5 and 22.5; bf16 151 MB 24.6 (a plain copy:
// 22.5 to 24.5).
#include "kv_format.cuh"
#include "launch.h"
#include "misa_device.cuh"

namespace misa {

namespace {

constexpr int kPieces = MISA_MLA_DQK / 8;      // 72
constexpr int kCodePieces = MISA_MLA_DV / 8;   // 64
constexpr int kThreads = 128;
constexpr int kMaxEach = 32;                   // rows of a warp

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

// Eight latent entries of a row to its codes; the four lanes of a group together.
template <int kFmt>
__device__ __forceinline__ void write_piece(uint8_t* dst, int piece, uint4 x) {
  if (kFmt == MISA_KV_BF16) {
    *reinterpret_cast<uint4*>(dst + piece * 16) = x;
    return;
  }
  // the largest of |entry| as bf16 bits: they order as the numbers do, infinity and NaN on top
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) amax = max(amax, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
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

// nrows = nseq * n_new < 2^31; each: rows of a warp, a multiple of 4.
template <int kFmt>
__global__ void __launch_bounds__(kThreads)
append_kv_kernel(const uint16_t* __restrict__ rows, uint32_t nrows, uint32_t each, int n_new, const int32_t* __restrict__ counts,
                 const int32_t* __restrict__ len, uint8_t* __restrict__ cache, int64_t seq_stride, int64_t L_cap,
                 uint32_t* err) {
  constexpr int kRow = kv_row_bytes(kFmt);
  pdl_wait_inputs();
  pdl_allow_next();
  const uint32_t lane = threadIdx.x & 31, row0 = (blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * each;
  if (row0 >= nrows) return;
  const uint32_t count = min(each, nrows - row0);
  uint8_t* mine = nullptr;   // where row row0 + lane goes
  if (lane < count) {
    const uint32_t row = row0 + lane, b = row / static_cast<uint32_t>(n_new);
    const int i = static_cast<int>(row - b * static_cast<uint32_t>(n_new));
    const int64_t l0 = __ldg(len + b);
    const int cnt = counts ? __ldg(counts + b) : n_new;
    if (cnt < 0 || cnt > n_new || l0 < 0 || l0 + cnt > L_cap) {
      if (i == 0) record_error(err, MISA_DEVERR_BAD_LEN);
    } else if (i < cnt) {
      mine = cache + b * seq_stride + (l0 + i) * kRow;
    }
  }
#pragma unroll 1
  for (uint32_t g = 0; g < count; g += 4) {
    const uint4* src = reinterpret_cast<const uint4*>(rows) + static_cast<int64_t>(row0 + g) * kPieces;
    uint8_t* dst[4];
    uint4 x[4][2], rope = make_uint4(0u, 0u, 0u, 0u);
    uint8_t* rope_dst = reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), g + (lane >> 3)));
    if (rope_dst) rope = __ldcs(src + (lane >> 3) * kPieces + kCodePieces + (lane & 7));
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      dst[r] = reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), g + r));
#pragma unroll
      for (int u = 0; u < 2; ++u) x[r][u] = dst[r] ? __ldcs(src + r * kPieces + 32 * u + lane) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (!dst[r]) continue;
      write_piece<kFmt>(dst[r], static_cast<int>(lane), x[r][0]);
      write_piece<kFmt>(dst[r], static_cast<int>(lane) + 32, x[r][1]);
    }
    if (rope_dst) *reinterpret_cast<uint4*>(rope_dst + kv_rope_offset(kFmt) + (lane & 7) * 16) = rope;
  }
}

struct ReadParams {
  const uint8_t* cache;
  int64_t nseq, seq_stride, L;
  const int32_t* seq_of;
  const int32_t* idx;
  int64_t idx_stride;
  const int32_t* first;
  const int32_t* prefix_len;
  uint32_t n, nrows, each;   // nrows = T * n < 2^31; each: rows of a warp, a multiple of 4
  uint16_t* out;
  uint32_t* err;
};

// Where output row `row` comes from in the cache, -1: zeros.
template <int kFmt>
__device__ __forceinline__ int64_t source_of(const ReadParams& p, uint32_t row) {
  const uint32_t t = row / p.n;
  const int64_t i = row - t * p.n;
  const int64_t seq = __ldg(p.seq_of + t);
  int64_t s = -1;
  if (seq < 0 || seq >= p.nseq) {
    if (i == 0) record_error(p.err, MISA_DEVERR_BAD_SEQ);
  } else if (p.idx) {
    s = __ldg(p.idx + t * p.idx_stride + i);
    if (s < -1 || s >= p.L) {
      record_error(p.err, MISA_DEVERR_BAD_INDEX);
      s = -1;
    }
  } else {
    const int64_t f = p.first ? __ldg(p.first + t) : 0;
    if (f < 0) {
      if (i == 0) record_error(p.err, MISA_DEVERR_BAD_INDEX);
    } else {
      const int64_t last = p.prefix_len ? __ldg(p.prefix_len + t) : p.L;
      if (f + i < (last < p.L ? last : p.L)) s = f + i;
    }
  }
  return s < 0 ? -1 : seq * p.seq_stride + s * kv_row_bytes(kFmt);
}

template <int kFmt>
__global__ void __launch_bounds__(kThreads) read_kv_kernel(const ReadParams p) {
  pdl_wait_inputs();
  pdl_allow_next();
  const uint32_t lane = threadIdx.x & 31, row0 = (blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * p.each;
  if (row0 >= p.nrows) return;
  const uint32_t count = min(p.each, p.nrows - row0);
  const long long mine = lane < count ? source_of<kFmt>(p, row0 + lane) : -1;
#pragma unroll 1
  for (uint32_t g = 0; g < count; g += 4) {
    uint4* out = reinterpret_cast<uint4*>(p.out) + static_cast<int64_t>(row0 + g) * kPieces;
    uint4 y[4][2], rope = make_uint4(0u, 0u, 0u, 0u);
    uint32_t scale[4][2];
    const long long rope_at = __shfl_sync(0xffffffffu, mine, g + (lane >> 3));
    if (rope_at >= 0) rope = __ldg(reinterpret_cast<const uint4*>(p.cache + rope_at + kv_rope_offset(kFmt) + (lane & 7) * 16));
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const long long at = __shfl_sync(0xffffffffu, mine, g + r);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t piece = lane + 32 * u;
        y[r][u] = make_uint4(0u, 0u, 0u, 0u);
        scale[r][u] = 0u;
        if (at < 0) continue;
        if (kFmt == MISA_KV_BF16) {
          y[r][u] = __ldg(reinterpret_cast<const uint4*>(p.cache + at + piece * 16));
        } else if (kFmt == MISA_KV_MX8) {
          const uint2 c = __ldg(reinterpret_cast<const uint2*>(p.cache + at + piece * 8));
          y[r][u].x = c.x;
          y[r][u].y = c.y;
        } else {
          y[r][u].x = __ldg(reinterpret_cast<const uint32_t*>(p.cache + at + piece * 4));
        }
        if (kFmt != MISA_KV_BF16) scale[r][u] = __ldg(p.cache + at + kv_code_bytes(kFmt) + (piece >> 2));
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (g + r >= count) break;
#pragma unroll
      for (int u = 0; u < 2; ++u)   // (an absent row's scale is zero)
        __stcs(out + r * kPieces + lane + 32 * u,
               kFmt == MISA_KV_BF16 ? y[r][u] : kv_decode8<kFmt>(y[r][u].x, y[r][u].y, kv_scale(scale[r][u])));
    }
    if (g + (lane >> 3) < count) __stcs(out + (lane >> 3) * kPieces + kCodePieces + (lane & 7), rope);
  }
}

// Rows of a warp: 4 until there are more than 128 warps an SM, so that a decode step's
// few rows spread out; finding the rows costs least a row when a warp has 32.
uint32_t rows_each(uint32_t nrows) {
  uint32_t each = 4;
  while (each < kMaxEach && nrows / each > 128u * static_cast<uint32_t>(device_sm_count())) each *= 2;
  return each;
}
uint32_t ctas_for(uint32_t nrows, uint32_t each) {
  const uint32_t rows = each * (kThreads / 32);
  return nrows / rows + (nrows % rows != 0);
}

}  // namespace

cudaError_t launch_append_kv(const uint16_t* rows, int64_t nseq, int n_new, const int32_t* counts, const int32_t* len,
                             int fmt, void* cache, int64_t seq_stride, int64_t L_cap, uint32_t* err,
                             cudaStream_t stream) {
  const uint32_t nrows = static_cast<uint32_t>(nseq * n_new);
  const uint32_t each = rows_each(nrows);
  auto kern = fmt == MISA_KV_BF16  ? append_kv_kernel<MISA_KV_BF16>
              : fmt == MISA_KV_MX8 ? append_kv_kernel<MISA_KV_MX8>
                                   : append_kv_kernel<MISA_KV_MX4>;
  return launch_pdl(kern, dim3(ctas_for(nrows, each)), dim3(kThreads), 0, stream, 0, rows, nrows, each, n_new, counts,
                    len, static_cast<uint8_t*>(cache), seq_stride, L_cap, err);
}

cudaError_t launch_read_kv(const void* cache, int fmt, int64_t nseq, int64_t seq_stride, int64_t L,
                           const int32_t* seq_of, int T, const int32_t* idx, int64_t idx_stride, const int32_t* first,
                           const int32_t* prefix_len, int64_t n, uint16_t* out, uint32_t* err, cudaStream_t stream) {
  ReadParams p = {static_cast<const uint8_t*>(cache), nseq, seq_stride, L, seq_of, idx, idx_stride, first, prefix_len,
                  static_cast<uint32_t>(n), static_cast<uint32_t>(T * n), 0u, out, err};
  p.each = rows_each(p.nrows);
  auto kern = fmt == MISA_KV_BF16  ? read_kv_kernel<MISA_KV_BF16>
              : fmt == MISA_KV_MX8 ? read_kv_kernel<MISA_KV_MX8>
                                   : read_kv_kernel<MISA_KV_MX4>;
  return launch_pdl(kern, dim3(ctas_for(p.nrows, p.each)), dim3(kThreads), 0, stream, 0, p);
}

}  // namespace misa
