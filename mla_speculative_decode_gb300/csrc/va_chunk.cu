// va_chunk.cu -- attention of ragged chunks of new tokens over the latent
// cache: entry points and the CUDA-core path.
//
// Request b brings n_b new tokens (one for a decode step, hundreds for a piece
// of a prompt) and P_b cached prefix keys; the new tokens' own rows are its
// last keys.  Token i sits at position P_b + i and sees key j when
//   j <= P_b + i  and  (no window, or j > P_b + i - window, or j < sinks).
// The output is the latent attention of the verify calls (softmax over 576
// columns, value = the first 512) in one pass over the visible keys with a
// running maximum and sum.
#include <string.h>

#include "va_chunk.cuh"

#ifndef VA_API
#define VA_API extern "C" __attribute__((visibility("default")))
#endif

namespace va {
namespace {

constexpr int kRowThreads = 256;   // 8 warps, a row each

bool aligned(const void* ptr, size_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }

// CUDA-core path: one warp per (token, head) row.
__global__ void __launch_bounds__(kRowThreads) chunk_fma_kernel(const ChunkParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t warp = int64_t(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
  const int64_t warps = int64_t(gridDim.x) * (kRowThreads / 32);
  uint32_t bits = 0u;
  for (int b = 0; b < p.B; ++b) {
    const ChunkReq r = chunk_req(p, b);
    if (r.bad) bits |= VA_STATUS_BAD_INDPTR;
    const int64_t rows = int64_t(r.n) * p.H;
    // the warp whose turn it is among all rows of the batch
    const int64_t g0 = int64_t(r.q0) * p.H;
    for (int64_t k = (warp - g0 % warps + warps) % warps; k < rows; k += warps) {
      bool bad_slot = false;
      chunk_row(p, r, int(k / p.H), int(k % p.H), lane, &bad_slot);
      if (bad_slot) bits |= VA_STATUS_BAD_SLOT;
    }
  }
  if (lane == 0 && bits) atomicOr(p.status, bits);
}

}  // namespace

int chunk_check(const ChunkParams& p, bool paged, float sm_scale, int flags, const void* ws) {
  if (!p.kv || !p.prefix_len || !p.q_indptr || !ws) return VA_ERR_NULL;
  if (p.total_q > 0 && (!p.q || !p.lse)) return VA_ERR_NULL;
  if (paged ? (!p.slot_idx || !p.kv_indptr) : !p.kv_start) return VA_ERR_NULL;
  if (p.B < 1 || p.B > 65535 || p.H < 1 || p.total_q < 0) return VA_ERR_SHAPE;
  if (int64_t(p.total_q) * p.H > VA_CHUNK_ROWS_MAX) return VA_ERR_SHAPE;
  if (p.num_slots < 1 || p.kv_stride < VA_D_QK || p.window < 0 || p.sinks < 0) return VA_ERR_SHAPE;
  if (flags < VA_PATH_AUTO || flags > VA_PATH_TC_1SM || !isfinite(sm_scale)) return VA_ERR_SHAPE;
  if (p.kv_stride % 8 != 0 || !aligned(p.q, 16) || !aligned(p.kv, 16) || !aligned(ws, 256) ||
      !aligned(p.lse, 4) || !aligned(p.prefix_len, 4) || !aligned(p.q_indptr, 4) ||
      !aligned(p.slot_idx, 4) || !aligned(p.kv_indptr, 4) || !aligned(p.kv_start, 8))
    return VA_ERR_ALIGN;
  return VA_OK;
}

namespace {

int chunk_common(ChunkParams& p, bool paged, float sm_scale, int flags, void* ws, size_t ws_bytes,
                 cudaStream_t st) {
  const int rc = chunk_check(p, paged, sm_scale, flags, ws);
  if (rc != VA_OK) return rc;
  if (p.total_q > 0 && !p.out) return VA_ERR_NULL;
  if (!aligned(p.out, 16)) return VA_ERR_ALIGN;
  if (ws_bytes < va_chunk_workspace_bytes(p.B, p.total_q, p.H, flags)) return VA_ERR_WORKSPACE;
  DeviceInfo di;
  const int rd = device_info(&di);
  if (rd != VA_OK) return rd;
  p.num_entries = 0x7fffffff;
  p.scale_log2 = sm_scale * kLog2e;
  p.status = static_cast<uint32_t*>(ws);
  if (cudaMemsetAsync(ws, 0, sizeof(uint32_t), st) != cudaSuccess) return VA_ERR_LAUNCH;
  if (p.total_q == 0) return VA_OK;
  const int64_t rows = int64_t(p.total_q) * p.H;
  const int64_t want = (rows + kRowThreads / 32 - 1) / (kRowThreads / 32);
  const int64_t wave = int64_t(di.num_sms) * 8;
  chunk_fma_kernel<<<unsigned(want < wave ? want : wave), kRowThreads, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? VA_OK : VA_ERR_LAUNCH;
}

}  // namespace
}  // namespace va

VA_API size_t va_chunk_workspace_bytes(int B, int total_q, int H, int flags) {
  if (B < 1 || B > 65535 || total_q < 0 || H < 1 || flags < VA_PATH_AUTO ||
      flags > VA_PATH_TC_1SM || int64_t(total_q) * H > VA_CHUNK_ROWS_MAX)
    return 0;
  return va::kHeaderBytes;
}

VA_API int va_chunk_attn_paged(const void* q, const void* kv_pool, int64_t num_slots,
                               int64_t kv_row_stride, const int32_t* slot_idx,
                               const int32_t* kv_indptr, const int32_t* prefix_len,
                               const int32_t* q_indptr, int B, int total_q, int H, float sm_scale,
                               int window, int sinks, int flags, void* workspace,
                               size_t workspace_bytes, void* out, float* lse,
                               va_stream_t stream) {
  va::ChunkParams p;
  memset(&p, 0, sizeof p);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.kv = static_cast<const __nv_bfloat16*>(kv_pool);
  p.num_slots = num_slots;
  p.kv_stride = kv_row_stride;
  p.slot_idx = slot_idx;
  p.kv_indptr = kv_indptr;
  p.prefix_len = prefix_len;
  p.q_indptr = q_indptr;
  p.B = B;
  p.total_q = total_q;
  p.H = H;
  p.window = window;
  p.sinks = sinks;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  return va::chunk_common(p, true, sm_scale, flags, workspace, workspace_bytes,
                          reinterpret_cast<cudaStream_t>(stream));
}

VA_API int va_chunk_attn_contiguous(const void* q, const void* kv_pool, int64_t num_slots,
                                    int64_t kv_row_stride, const int64_t* kv_start,
                                    const int32_t* prefix_len, const int32_t* q_indptr, int B,
                                    int total_q, int H, float sm_scale, int window, int sinks,
                                    int flags, void* workspace, size_t workspace_bytes, void* out,
                                    float* lse, va_stream_t stream) {
  va::ChunkParams p;
  memset(&p, 0, sizeof p);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.kv = static_cast<const __nv_bfloat16*>(kv_pool);
  p.num_slots = num_slots;
  p.kv_stride = kv_row_stride;
  p.kv_start = kv_start;
  p.prefix_len = prefix_len;
  p.q_indptr = q_indptr;
  p.B = B;
  p.total_q = total_q;
  p.H = H;
  p.window = window;
  p.sinks = sinks;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  return va::chunk_common(p, false, sm_scale, flags, workspace, workspace_bytes,
                          reinterpret_cast<cudaStream_t>(stream));
}
