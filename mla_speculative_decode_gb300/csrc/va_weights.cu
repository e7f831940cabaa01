// va_weights.cu -- attention weight that each cached key receives from a
// chunk's rows, added to a running total per list entry:
//   weights_out[e] = weights_in[e] + sum over the rows r that see the key of
//                    exp(s_r - lse_r)
// with s_r the scaled score and lse_r the row's log-sum-exp from the attention
// call.  Which rows see a key is exactly what the attention call applied
// (causal, window, sinks).  The entry point and the CUDA-core path
// (VA_PATH_FMA); the tensor-core path is in va_weights_tc.cu.
#include <string.h>

#include "va_weights.cuh"

#ifndef VA_API
#define VA_API extern "C" __attribute__((visibility("default")))
#endif

namespace va {
namespace {

constexpr int kWeightThreads = 256;   // 8 warps, a key each

struct WeightParams {
  ChunkParams c;
  const float* win;
  float* wout;
};

// CUDA-core path: one warp per (request, key); a token's heads are summed
// first and then added to the key's total, so no partial sum is long.
__global__ void __launch_bounds__(kWeightThreads) weights_fma_kernel(const WeightParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t warp = int64_t(blockIdx.x) * (kWeightThreads / 32) + (threadIdx.x >> 5);
  const int64_t warps = int64_t(gridDim.x) * (kWeightThreads / 32);
  const ChunkParams& c = p.c;
  uint32_t bits = 0u;
  int64_t turn = 0;
  const int requests = chunk_requests(c, lane);
  for (int b = 0; b < c.B; ++b) {
    const ChunkReq r = chunk_req(c, b, b >= requests);
    if (r.bad) bits |= VA_STATUS_BAD_INDPTR;
    const int N = r.nlist < r.P + r.n ? r.nlist : r.P + r.n;
    for (int64_t k = (warp - turn % warps + warps) % warps; k < N; k += warps) {
      const int j = int(k);
      const int64_t kr = chunk_key_row(c, r, j);
      float total = 0.f;
      const int i0 = j > r.P ? j - r.P : 0;   // the first token that sees it, if any does
      if (i0 >= r.n || (j >= c.sinks && j < window_first(c.window, r.P + i0))) {
      } else if (kr < 0) {
        bits |= VA_STATUS_BAD_SLOT;
      } else {
        const uint32_t* k32 = reinterpret_cast<const uint32_t*>(c.kv + kr * c.kv_stride);
        uint32_t kv[9];
#pragma unroll
        for (int x = 0; x < 9; ++x) kv[x] = k32[32 * x + lane];
        for (int i = i0; i < r.n; ++i) {
          if (j >= c.sinks && j < window_first(c.window, r.P + i)) break;   // nor any later token
          float token = 0.f;
          for (int h = 0; h < c.H; ++h) {
            const size_t row = (size_t(r.q0) + i) * c.H + h;
            const float lse = c.lse[row];
            const uint32_t* q32 = reinterpret_cast<const uint32_t*>(c.q + row * kDqk);
            float s = 0.f;
#pragma unroll
            for (int x = 0; x < 9; ++x) {
              const uint32_t q = q32[32 * x + lane];
              s = fmaf(bf16lo(q), bf16lo(kv[x]), s);
              s = fmaf(bf16hi(q), bf16hi(kv[x]), s);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            // a row at -inf saw no key and gives no weight
            if (lse != -INFINITY) token += exp2f(fmaf(s, c.scale_log2, -lse * kLog2e));
          }
          total += token;
        }
      }
      if (lane == 0) {
        const int64_t e = r.base + j;
        p.wout[e] = (p.win ? p.win[e] : 0.f) + total;
      }
    }
    turn += N;
  }
  if (lane == 0 && bits) atomicOr(c.status, bits);
}

struct WeightsLayout {
  size_t flags, entry, cont, sums, total;
};

WeightsLayout weights_layout(int64_t num_entries) {
  WeightsLayout L;
  L.flags = kHeaderBytes;
  L.entry = L.flags + align256(kWeightClusters * sizeof(uint32_t));
  L.cont = L.entry + align256(kWeightClusters * sizeof(int32_t));
  L.sums = L.cont + align256(size_t(kWeightClusters) * 256 * sizeof(float));
  L.total = L.sums + align256(size_t(num_entries) * sizeof(float));
  return L;
}

bool aligned4(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 3u) == 0; }

}  // namespace
}  // namespace va

VA_API size_t va_kv_weights_workspace_bytes(int B, int total_q, int H, int64_t num_entries,
                                            int flags) {
  if (B < 1 || B > 65535 || total_q < 0 || H < 1 || flags < VA_PATH_AUTO ||
      flags > VA_PATH_TC_1SM || int64_t(total_q) * H > VA_CHUNK_ROWS_MAX || num_entries < 0 ||
      num_entries > va::kKeysMax)
    return 0;
  if (flags == VA_PATH_FMA) return va::kHeaderBytes;
  return va::weights_layout(num_entries).total;
}

VA_API int va_kv_weights_paged(const void* q, const void* kv_pool, int64_t num_slots,
                               int64_t kv_row_stride, const int32_t* slot_idx,
                               const int32_t* kv_indptr, const int32_t* prefix_len,
                               const int32_t* q_indptr, const float* lse, const float* weights_in,
                               int64_t num_entries, int B, int total_q, int H, float sm_scale,
                               int window, int sinks, int flags, void* workspace,
                               size_t workspace_bytes, float* weights_out, va_stream_t stream) {
  using namespace va;
  WeightParams p;
  memset(&p, 0, sizeof p);
  ChunkParams& c = p.c;
  c.q = static_cast<const __nv_bfloat16*>(q);
  c.kv = static_cast<const __nv_bfloat16*>(kv_pool);
  c.num_slots = num_slots;
  c.kv_stride = kv_row_stride;
  c.slot_idx = slot_idx;
  c.kv_indptr = kv_indptr;
  c.prefix_len = prefix_len;
  c.q_indptr = q_indptr;
  c.num_entries = num_entries;
  c.B = B;
  c.total_q = total_q;
  c.H = H;
  c.window = window;
  c.sinks = sinks;
  c.lse = const_cast<float*>(lse);
  const int rc = chunk_check(c, true, sm_scale, flags, workspace);
  if (rc != VA_OK) return rc;
  if (!weights_out && num_entries != 0) return VA_ERR_NULL;
  if (num_entries < 0 || num_entries > kKeysMax) return VA_ERR_SHAPE;
  if (!aligned4(weights_in) || !aligned4(weights_out)) return VA_ERR_ALIGN;
  if (workspace_bytes < va_kv_weights_workspace_bytes(B, total_q, H, num_entries, flags))
    return VA_ERR_WORKSPACE;
  DeviceInfo di;
  const int rd = device_info(&di);
  if (rd != VA_OK) return rd;
  c.scale_log2 = sm_scale * kLog2e;
  c.status = static_cast<uint32_t*>(workspace);
  p.win = weights_in;
  p.wout = weights_out;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // (no rows at all: there is no map of them to launch the tensor-core kernel with)
  if (flags != VA_PATH_FMA && total_q > 0) {
    // Two-SM products when the average request has more than one row tile of the
    // one-SM kernel (32 requests of 8k keys: 64 rows 72 us with one SM and 73 with
    // two, 128 rows 116 and 77, 256 rows 205 and 74; 4 of 16k keys: 29 and 28, 41
    // and 31, 64 and 30).
    const int busy = B < total_q ? B : total_q;
    const bool pair = flags != VA_PATH_TC_1SM && int64_t(total_q) * H > 64 * int64_t(busy);
    const WeightsLayout L = weights_layout(num_entries);
    uint8_t* w = static_cast<uint8_t*>(workspace);
    WeightTcParams t;
    memset(&t, 0, sizeof t);
    t.c = c;
    t.c.scale_log2 = tc_scale_log2(sm_scale);
    t.win = weights_in;
    t.wout = weights_out;
    const int clusters = pair ? di.pairs : di.num_sms;
    const int most = pair ? kWeightClusters / 2 : kWeightClusters;
    t.clusters = clusters < most ? clusters : most;
    t.tile_keys = pair ? 256 : 128;
    t.cta_flags = reinterpret_cast<uint32_t*>(w + L.flags);
    t.cont_entry = reinterpret_cast<int32_t*>(w + L.entry);
    t.cont = reinterpret_cast<float*>(w + L.cont);
    t.sums = reinterpret_cast<float*>(w + L.sums);
    return launch_weights_tc(t, pair, st) == cudaSuccess ? VA_OK : VA_ERR_LAUNCH;
  }
  if (cudaMemsetAsync(workspace, 0, sizeof(uint32_t), st) != cudaSuccess) return VA_ERR_LAUNCH;
  const int64_t want = (num_entries + kWeightThreads / 32 - 1) / (kWeightThreads / 32);
  const int64_t wave = int64_t(di.num_sms) * 8;
  weights_fma_kernel<<<unsigned(want < 1 ? 1 : want < wave ? want : wave), kWeightThreads, 0,
                       st>>>(p);
  return cudaGetLastError() == cudaSuccess ? VA_OK : VA_ERR_LAUNCH;
}
