// va_evict.cu -- eviction from the cache by accumulated attention weight.
//
// Request b keeps `budget` of its L = prefix_len[b] list entries when L is
// larger: the first `sinks`, the last `recent`, and of the entries between
// them the m = budget - sinks - recent with the largest weights (ties: the
// lower index; NaN counts as -inf).  The kept entries stay in list order and
// move to the front of the request's list, with their weights; the evicted
// slots go back to the free list.
//
// The m-th largest weight is found by a radix selection on the weights mapped
// to unsigned integers of the same order: a histogram of the leading digit of
// the candidates, the digit where the count from the top reaches m, and so on
// through the digits.  Every entry above that threshold stays, and of the
// entries equal to it as many as are still wanted, in index order.
#include <math.h>
#include <string.h>

#include "va_common.cuh"

#ifndef VA_API
#define VA_API extern "C" __attribute__((visibility("default")))
#endif

namespace va {
namespace {

constexpr int kEvictThreads = 1024;
constexpr int kDigits = 256;

struct EvictParams {
  const int32_t* slot_idx;
  const int32_t* kv_indptr;
  const int32_t* prefix_len;
  const float* weights;
  int64_t num_entries;
  int B, budget, sinks, recent;
  int32_t* free_slots;
  int64_t free_capacity;
  const int32_t* free_head;
  int32_t* slot_out;
  int32_t* prefix_out;
  float* weights_out;
  int32_t* head_out;
  uint32_t* status;
};

// A weight as an unsigned integer of the same order.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (isnan(w)) w = -INFINITY;
  w += 0.f;   // -0 and +0 are equal
  const uint32_t u = __float_as_uint(w);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A request's list: [base, base + L) inside the arrays whatever they hold.
__device__ __forceinline__ int evict_list(const EvictParams& p, int b, int64_t* base, bool* bad) {
  int64_t i0 = p.kv_indptr[b], i1 = p.kv_indptr[b + 1];
  int L = p.prefix_len[b];
  if (i0 < 0 || i1 < i0 || i1 > p.num_entries) {
    *bad = true;
    i0 = i0 < 0 ? 0 : (i0 > p.num_entries ? p.num_entries : i0);
    i1 = i1 < i0 ? i0 : (i1 > p.num_entries ? p.num_entries : i1);
  }
  if (L < 0) { L = 0; *bad = true; }
  if (L > i1 - i0) { L = int(i1 - i0); *bad = true; }
  *base = i0;
  return L;
}

__device__ __forceinline__ int64_t evicted_of(const EvictParams& p, int b) {
  int64_t base;
  bool bad = false;
  const int L = evict_list(p, b, &base, &bad);
  return L > p.budget ? L - p.budget : 0;
}

// Sum of v over the block (every thread gets it).
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (lane == 0) red[warp] = v;
  __syncthreads();
  int64_t t = 0;
#pragma unroll
  for (int w = 0; w < kEvictThreads / 32; ++w) t += red[w];
  return t;
}

// One CTA per request.
__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const EvictParams p) {
  __shared__ int64_t red[kEvictThreads / 32];
  __shared__ uint32_t hist[kDigits];
  __shared__ uint32_t s_digit, s_above;
  __shared__ uint2 wsum[kEvictThreads / 32];
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool bad = false;
  int64_t base;
  const int L = evict_list(p, b, &base, &bad);
  if (bad && tid == 0 && p.status) atomicOr(p.status, VA_STATUS_BAD_INDPTR);
  const int nfreed = L > p.budget ? L - p.budget : 0;

  // place of the request's first evicted slot in the free list
  int64_t before = 0, total = 0;
  if (p.free_slots) {
    int64_t mine_before = 0, mine = 0;
    for (int x = tid; x < p.B; x += kEvictThreads) {
      const int64_t n = evicted_of(p, x);
      mine += n;
      if (x < b) mine_before += n;
    }
    before = block_sum(mine_before, red);
    total = block_sum(mine, red);
  }
  const int64_t free0 = p.free_slots ? int64_t(*p.free_head) - total + before : 0;

  const int lo = nfreed ? p.sinks : 0, hi = nfreed ? L - p.recent : 0;   // candidates
  const int m = p.budget - p.sinks - p.recent;                          // of which stay
  uint32_t prefix = 0, want = uint32_t(m > 0 ? m : 0);
  if (nfreed && m > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int d = tid; d < kDigits; d += kEvictThreads) hist[d] = 0;
      __syncthreads();
      for (int i = lo + tid; i < hi; i += kEvictThreads) {
        const uint32_t k = weight_key(p.weights[base + i]);
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
          atomicAdd(&hist[(k >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        uint32_t above = 0;
        int d = kDigits - 1;
        while (d > 0 && above + hist[d] < want) above += hist[d--];
        s_digit = uint32_t(d);
        s_above = above;
      }
      __syncthreads();
      prefix |= s_digit << shift;
      want -= s_above;
      __syncthreads();
    }
  }
  // `prefix` is the threshold's key; `want` entries equal to it stay

  // compaction, a block of entries at a time: the output never passes the input
  uint32_t kept = 0, equal = 0;   // before this block of entries
  for (int i0 = 0; i0 < L; i0 += kEvictThreads) {
    const int i = i0 + tid;
    const bool in = i < L;
    const int slot = in ? p.slot_idx[base + i] : 0;
    const float w = in ? p.weights[base + i] : 0.f;
    const bool cand = in && i >= lo && i < hi;
    const uint32_t k = cand ? weight_key(w) : 0u;
    const bool eq = cand && m > 0 && k == prefix;
    const bool above = in && (!cand || (m > 0 && k > prefix));
    const uint32_t beq = __ballot_sync(0xffffffffu, eq);
    const uint32_t babove = __ballot_sync(0xffffffffu, above);
    if (lane == 0) wsum[warp] = make_uint2(uint32_t(__popc(beq)), uint32_t(__popc(babove)));
    __syncthreads();
    uint32_t e0 = equal, a0 = 0, et = 0, at = 0;
    for (int x = 0; x < kEvictThreads / 32; ++x) {
      const uint2 s = wsum[x];
      if (x < warp) { e0 += s.x; a0 += s.y; }
      et += s.x;
      at += s.y;
    }
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t my_eq = e0 + uint32_t(__popc(beq & below));
    const bool keep = above || (eq && my_eq < want);
    // kept entries before this one in the block: those above, and the equal
    // ones that still fit
    const uint32_t eq_kept = (my_eq < want ? my_eq : want) - (equal < want ? equal : want);
    const uint32_t at_out = kept + a0 + uint32_t(__popc(babove & below)) + eq_kept;
    if (in) {
      if (keep) {
        p.slot_out[base + at_out] = slot;
        p.weights_out[base + at_out] = w;
      } else if (p.free_slots) {
        const int64_t f = free0 + (i - int64_t(at_out));
        if (f >= 0 && f < p.free_capacity)
          p.free_slots[f] = slot;
        else if (p.status)
          atomicOr(p.status, VA_STATUS_BAD_DST);
      }
    }
    const uint32_t after = equal + et;
    kept += at + (after < want ? after : want) - (equal < want ? equal : want);
    equal = after;
    __syncthreads();
  }
}

// The new lengths and the free list's head, once every request's CTA has read
// the old ones (the outputs may be the inputs' own buffers).
__global__ void __launch_bounds__(kEvictThreads) evict_finish_kernel(const EvictParams p) {
  __shared__ int64_t red[kEvictThreads / 32];
  int64_t mine = 0;
  for (int b = threadIdx.x; b < p.B; b += kEvictThreads) {
    int64_t base;
    bool bad = false;
    const int L = evict_list(p, b, &base, &bad);
    p.prefix_out[b] = L < p.budget ? L : p.budget;
    mine += L > p.budget ? L - p.budget : 0;
  }
  if (!p.free_slots) return;
  const int64_t total = block_sum(mine, red);
  if (threadIdx.x == 0) {
    const int64_t head = int64_t(*p.free_head) - total;
    *p.head_out = int32_t(head < 0 ? 0 : head);
  }
}

bool aligned4(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 3u) == 0; }

}  // namespace
}  // namespace va

VA_API int va_kv_evict(const int32_t* slot_idx, const int32_t* kv_indptr,
                       const int32_t* prefix_len, const float* weights, int64_t num_entries, int B,
                       int budget, int sinks, int recent, int32_t* free_slots,
                       int64_t free_capacity, const int32_t* free_head, int32_t* slot_idx_out,
                       int32_t* prefix_len_out, float* weights_out, int32_t* free_head_out,
                       uint32_t* status, va_stream_t stream) {
  using namespace va;
  if (!slot_idx || !kv_indptr || !prefix_len || !weights || !slot_idx_out || !prefix_len_out ||
      !weights_out)
    return VA_ERR_NULL;
  if (free_slots && (!free_head || !free_head_out)) return VA_ERR_NULL;
  if (B < 1 || B > 65535 || num_entries < 0 || num_entries > 0x7fffffff || budget < 0 ||
      sinks < 0 || recent < 0 || int64_t(sinks) + recent > budget ||
      (free_slots && free_capacity < 0))
    return VA_ERR_SHAPE;
  if (!aligned4(slot_idx) || !aligned4(kv_indptr) || !aligned4(prefix_len) || !aligned4(weights) ||
      !aligned4(free_slots) || !aligned4(free_head) || !aligned4(slot_idx_out) ||
      !aligned4(prefix_len_out) || !aligned4(weights_out) || !aligned4(free_head_out) ||
      !aligned4(status))
    return VA_ERR_ALIGN;
  DeviceInfo di;
  const int rc = device_info(&di);
  if (rc != VA_OK) return rc;
  EvictParams p;
  memset(&p, 0, sizeof p);
  p.slot_idx = slot_idx;
  p.kv_indptr = kv_indptr;
  p.prefix_len = prefix_len;
  p.weights = weights;
  p.num_entries = num_entries;
  p.B = B;
  p.budget = budget;
  p.sinks = sinks;
  p.recent = recent;
  p.free_slots = free_slots;
  p.free_capacity = free_capacity;
  p.free_head = free_head;
  p.slot_out = slot_idx_out;
  p.prefix_out = prefix_len_out;
  p.weights_out = weights_out;
  p.head_out = free_head_out;
  p.status = status;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  evict_kernel<<<unsigned(B), kEvictThreads, 0, st>>>(p);
  if (cudaGetLastError() != cudaSuccess) return VA_ERR_LAUNCH;
  evict_finish_kernel<<<1, kEvictThreads, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? VA_OK : VA_ERR_LAUNCH;
}
