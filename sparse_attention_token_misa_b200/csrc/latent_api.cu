// C ABI of the latent cache (include/misa_latent.h): host-side argument checks
// and launches.
#include <cmath>

#include "kv_format.cuh"
#include "launch.h"

namespace {

constexpr size_t kErrBytes = 256;
constexpr int64_t kMax31 = static_cast<int64_t>(1) << 31;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool known(int fmt) { return fmt == MISA_KV_BF16 || fmt == MISA_KV_MX8 || fmt == MISA_KV_MX4; }
misa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MISA_OK : MISA_ERR_CUDA; }

misa_status check_cache(const void* cache, int fmt, int64_t nseq, int64_t seq_stride, int64_t L) {
  if (!cache || !known(fmt) || nseq < 1 || L < 1) return MISA_ERR_INVALID_ARG;
  if (L >= kMax31 || nseq >= kMax31) return MISA_ERR_UNSUPPORTED;
  if (!aligned16(cache) || seq_stride < 0 || seq_stride % 16 != 0) return MISA_ERR_INVALID_ARG;
  if (nseq > 1 && seq_stride < L * misa::kv_row_bytes(fmt)) return MISA_ERR_INVALID_ARG;
  return MISA_OK;
}

misa_status check_ws(const void* ws, size_t have, size_t need) {
  if (!ws || have < need) return MISA_ERR_WORKSPACE;
  return aligned16(ws) ? MISA_OK : MISA_ERR_INVALID_ARG;
}

// The checks both attention calls share, then the launch.  n: the rows a query
// has at most (k, or L).
misa_status attend(misa::LatentArgs& a, int64_t n, float scale, void* ws, size_t ws_bytes, misa_stream_t stream) {
  if (!a.q || !a.seq_of || !a.out || a.T < 1 || a.Hq < 1) return MISA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || scale < 0.f) return MISA_ERR_INVALID_ARG;
  misa_status st = check_cache(a.cache, a.fmt, a.nseq, a.seq_stride, a.L);
  if (st != MISA_OK) return st;
  if (!aligned16(a.q) || !aligned16(a.out)) return MISA_ERR_INVALID_ARG;
  a.scale_log2 = scale * 1.4426950408889634f;
  if (!std::isfinite(a.scale_log2)) return MISA_ERR_UNSUPPORTED;   // infinity times a score of 0 would be NaN
  if (a.Hq > MISA_MAX_HEADS || static_cast<int64_t>(a.T) * a.Hq >= kMax31 || a.T >= (1 << 29))
    return MISA_ERR_UNSUPPORTED;
  // a TMA map reads bf16 rows: its strides are 40 bits
  if (a.fmt == MISA_KV_BF16 && (a.seq_stride >> 40 || (a.L * misa::kv_row_bytes(MISA_KV_BF16)) >> 40))
    return MISA_ERR_UNSUPPORTED;
  st = check_ws(ws, ws_bytes, kErrBytes + misa::latent_mla_scratch_bytes(a.T, a.Hq, n));
  if (st != MISA_OK) return st;
  a.err = static_cast<uint32_t*>(ws);
  a.scratch = static_cast<uint8_t*>(ws) + kErrBytes;
  return cuda_status(misa::launch_latent_mla(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int64_t misa_kv_row_bytes(int fmt) { return known(fmt) ? misa::kv_row_bytes(fmt) : 0; }

misa_status misa_append_kv(const uint16_t* rows, int64_t nseq, int n_new, const int32_t* counts, const int32_t* len,
                           int fmt, void* cache, int64_t cache_seq_stride, int64_t L_cap, void* workspace,
                           size_t workspace_bytes, misa_stream_t stream) {
  if (!rows || !len || n_new < 1) return MISA_ERR_INVALID_ARG;
  misa_status st = check_cache(cache, fmt, nseq, cache_seq_stride, L_cap);
  if (st != MISA_OK) return st;
  if (!aligned16(rows)) return MISA_ERR_INVALID_ARG;
  if (nseq * n_new >= kMax31) return MISA_ERR_UNSUPPORTED;
  st = check_ws(workspace, workspace_bytes, kErrBytes);
  if (st != MISA_OK) return st;
  return cuda_status(misa::launch_append_kv(rows, nseq, n_new, counts, len, fmt, cache, cache_seq_stride, L_cap,
                                            static_cast<uint32_t*>(workspace), reinterpret_cast<cudaStream_t>(stream)));
}

misa_status misa_read_kv(const void* cache, int fmt, int64_t nseq, int64_t cache_seq_stride, int64_t L,
                         const int32_t* seq_of, int T, const int32_t* idx, int64_t idx_stride, const int32_t* first,
                         const int32_t* prefix_len, int64_t n, uint16_t* out, void* workspace, size_t workspace_bytes,
                         misa_stream_t stream) {
  if (!seq_of || !out || T < 1 || n < 1) return MISA_ERR_INVALID_ARG;
  if (idx && (first || prefix_len || idx_stride < n)) return MISA_ERR_INVALID_ARG;
  misa_status st = check_cache(cache, fmt, nseq, cache_seq_stride, L);
  if (st != MISA_OK) return st;
  if (!aligned16(out)) return MISA_ERR_INVALID_ARG;
  if (n >= kMax31 || T * n >= kMax31) return MISA_ERR_UNSUPPORTED;
  st = check_ws(workspace, workspace_bytes, kErrBytes);
  if (st != MISA_OK) return st;
  return cuda_status(misa::launch_read_kv(cache, fmt, nseq, cache_seq_stride, L, seq_of, T, idx, idx_stride, first,
                                          prefix_len, n, out, static_cast<uint32_t*>(workspace),
                                          reinterpret_cast<cudaStream_t>(stream)));
}

misa_status misa_sparse_mla_q(const uint16_t* q, const void* cache, int fmt, int64_t nseq, int64_t cache_seq_stride,
                              int64_t L, const int32_t* seq_of, int T, int Hq, const int32_t* idx, int k,
                              int64_t idx_stride, float scale, uint16_t* out, float* lse, void* workspace,
                              size_t workspace_bytes, misa_stream_t stream) {
  if (!idx || k < 1 || idx_stride < k) return MISA_ERR_INVALID_ARG;
  if (k > MISA_MAX_TOPK || fmt == MISA_KV_BF16) return MISA_ERR_UNSUPPORTED;
  misa::LatentArgs a = {q, cache, fmt, nseq, cache_seq_stride, L, seq_of, nullptr, idx, k, idx_stride, T, Hq, 0.f, out,
                        lse, nullptr, nullptr};
  return attend(a, k, scale, workspace, workspace_bytes, stream);
}

misa_status misa_prefix_mla(const uint16_t* q, const void* cache, int fmt, int64_t nseq, int64_t cache_seq_stride,
                            int64_t L, const int32_t* seq_of, const int32_t* prefix_len, int T, int Hq, float scale,
                            uint16_t* out, float* lse, void* workspace, size_t workspace_bytes, misa_stream_t stream) {
  if (!prefix_len) return MISA_ERR_INVALID_ARG;
  misa::LatentArgs a = {q, cache, fmt, nseq, cache_seq_stride, L, seq_of, prefix_len, nullptr, 0, 0, T, Hq, 0.f, out,
                        lse, nullptr, nullptr};
  return attend(a, L, scale, workspace, workspace_bytes, stream);
}

}  // extern "C"
