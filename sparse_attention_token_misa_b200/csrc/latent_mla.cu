// Attention over a latent cache held in 16, 8 or 4 bits: the listed rows of each
// query, or all rows of its prefix (include/misa_latent.h).
//
//   out[t, h] = sum_i p_i v_i / sum_i p_i,  p_i = exp(scale * q[t, h] . k_i)
//
// One pass over the rows with a running maximum m and sum l: a row whose score
// is above m first scales the sums by 2^(m - m').  One CTA per query and eight
// heads, one warp per head: the tile of rows is brought to bf16 in shared memory
// once for the eight, each lane keeps 18 of the query's entries and 16 of the
// output's.
#include "kv_format.cuh"
#include "launch.h"
#include "misa_device.cuh"

namespace misa {

namespace {

constexpr int kHeads = 8;      // heads (warps) of a CTA
constexpr int kTile = 16;      // rows staged at a time
constexpr int kPieces = MISA_MLA_DQK / 8;

template <int kFmt>
__device__ __forceinline__ uint4 row_piece(const uint8_t* src, int piece) {
  if (kFmt == MISA_KV_BF16) return *reinterpret_cast<const uint4*>(src + piece * 16);
  if (piece >= MISA_MLA_DV / 8)
    return *reinterpret_cast<const uint4*>(src + kv_rope_offset(kFmt) + (piece - MISA_MLA_DV / 8) * 16);
  uint2 c;
  if (kFmt == MISA_KV_MX8) c = *reinterpret_cast<const uint2*>(src + piece * 8);
  else c = make_uint2(*reinterpret_cast<const uint32_t*>(src + piece * 4), 0u);
  uint32_t second;
  const uint32_t scale = kv_scale<kFmt>(src[kv_code_bytes(kFmt) + (piece >> 2)], &second);
  return kv_decode8<kFmt>(c.x, c.y, scale, second);
}

template <int kFmt>
__global__ void __launch_bounds__(kHeads * 32) latent_mla_kernel(const LatentArgs p) {
  __shared__ uint4 sRow[kTile][kPieces];
  __shared__ int32_t sId[kTile];
  pdl_wait_inputs();
  pdl_allow_next();
  const int groups = (p.Hq + kHeads - 1) / kHeads;
  const int t = static_cast<int>(blockIdx.x) / groups;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = (static_cast<int>(blockIdx.x) - t * groups) * kHeads + warp;
  const bool live = h < p.Hq;
  int64_t seq = p.seq_of[t];
  int64_t n = p.idx ? p.k : min(static_cast<int64_t>(p.prefix_len[t]), p.L);
  if (seq < 0 || seq >= p.nseq) {
    if (threadIdx.x == 0) record_error(p.err, MISA_DEVERR_BAD_SEQ);
    seq = 0;
    n = 0;
  }
  const uint8_t* base = static_cast<const uint8_t*>(p.cache) + seq * p.seq_stride;
  float q[18], o[16];
  const __nv_bfloat16* qrow =
      reinterpret_cast<const __nv_bfloat16*>(p.q) + (static_cast<int64_t>(t) * p.Hq + (live ? h : 0)) * MISA_MLA_DQK;
#pragma unroll
  for (int j = 0; j < 18; ++j) q[j] = __bfloat162float(qrow[lane + 32 * j]) * p.scale_log2;
#pragma unroll
  for (int j = 0; j < 16; ++j) o[j] = 0.f;
  const float kNegInf = -__int_as_float(0x7f800000);
  float m = kNegInf, l = 0.f;
  for (int64_t s0 = 0; s0 < n; s0 += kTile) {
    __syncthreads();
    if (threadIdx.x < kTile) {
      int32_t id = -1;
      if (s0 + threadIdx.x < n) {
        id = p.idx ? p.idx[static_cast<int64_t>(t) * p.idx_stride + s0 + threadIdx.x] : static_cast<int32_t>(s0 + threadIdx.x);
        if (id < -1 || id >= p.L) {
          record_error(p.err, MISA_DEVERR_BAD_INDEX);
          id = -1;
        }
      }
      sId[threadIdx.x] = id;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < kTile * kPieces; c += kHeads * 32) {
      const int r = c / kPieces, piece = c - r * kPieces;
      if (sId[r] >= 0) sRow[r][piece] = row_piece<kFmt>(base + sId[r] * static_cast<int64_t>(kv_row_bytes(kFmt)), piece);
    }
    __syncthreads();
    for (int r = 0; r < kTile; ++r) {
      if (sId[r] < 0) continue;
      const __nv_bfloat16* row = reinterpret_cast<const __nv_bfloat16*>(&sRow[r][0]);
      float v[18], s = 0.f;
#pragma unroll
      for (int j = 0; j < 18; ++j) {
        v[j] = __bfloat162float(row[lane + 32 * j]);
        s += q[j] * v[j];
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      if (s > m) {
        const float f = exp2f(m - s);
        l *= f;
#pragma unroll
        for (int j = 0; j < 16; ++j) o[j] *= f;
        m = s;
      }
      const float w = m == kNegInf ? 0.f : exp2f(s - m);
      l += w;
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j] += w * v[j];
    }
  }
  if (!live) return;
  const int64_t row = static_cast<int64_t>(t) * p.Hq + h;
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j)
    reinterpret_cast<__nv_bfloat16*>(p.out)[row * MISA_MLA_DV + lane + 32 * j] = __float2bfloat16_rn(o[j] * inv);
  if (p.lse && lane == 0) p.lse[row] = l > 0.f || l != l ? (m + log2f(l)) * 0.69314718055994531f : kNegInf;
}

}  // namespace

size_t latent_mla_scratch_bytes(int, int, int64_t) { return 0; }

cudaError_t launch_latent_mla(const LatentArgs& a, cudaStream_t stream) {
  const int64_t grid = static_cast<int64_t>(a.T) * ((a.Hq + kHeads - 1) / kHeads);
  auto kern = a.fmt == MISA_KV_BF16  ? latent_mla_kernel<MISA_KV_BF16>
              : a.fmt == MISA_KV_MX8 ? latent_mla_kernel<MISA_KV_MX8>
                                     : latent_mla_kernel<MISA_KV_MX4>;
  return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(kHeads * 32), 0, stream, 0, a);
}

}  // namespace misa
