// va_chunk.cuh -- what the chunk-attention kernels, the weight kernels and
// their host code share: launch parameters, a request's bounds, which keys a
// token sees, and one row's attention on CUDA cores.
#pragma once

#include <math.h>

#include "va_common.cuh"

namespace va {

// Arguments of a chunk call (va_chunk_attn_*, va_kv_weights_paged), by value.
// Request b's new tokens are query tokens q_indptr[b] .. q_indptr[b+1] - 1; its
// keys are P = prefix_len[b] prefix rows followed by the new tokens' own rows.
struct ChunkParams {
  const __nv_bfloat16* q;      // [total_q, H, 576]
  const __nv_bfloat16* kv;     // [num_slots, kv_stride]
  int64_t num_slots;
  int64_t kv_stride;           // elements
  const int32_t* slot_idx;     // paged
  const int32_t* kv_indptr;    // paged: [B+1]
  const int64_t* kv_start;     // contiguous: [B] (NULL when paged)
  const int32_t* prefix_len;   // [B]
  const int32_t* q_indptr;     // [B+1]
  int64_t num_entries;         // entries of slot_idx (weights call), else 2^31 - 1
  int B, total_q, H;
  int window, sinks;           // window 0: every earlier key is visible
  float scale_log2;            // sm_scale * log2(e)
  uint32_t* status;
  __nv_bfloat16* out;          // [total_q, H, 512]
  float* lse;                  // [total_q, H]
};

// A request's bounds.  Whatever the device arrays hold, 0 <= q0 <= q0 + n <=
// total_q, P >= 0 and [base, base + nlist) lies inside the slot list, so no
// later access leaves a buffer.
struct ChunkReq {
  int P;         // prefix length (clamped to what the list holds)
  int n;         // new tokens
  int q0;        // first query token
  int nlist;     // keys that have a list entry (contiguous: P + n)
  int64_t base;  // paged: offset into slot_idx; contiguous: first pool row
  bool bad;      // bounds were clamped (VA_STATUS_BAD_INDPTR)
};

__device__ inline ChunkReq chunk_req(const ChunkParams& p, int b) {
  ChunkReq r;
  const int a0 = p.q_indptr[b], a1 = p.q_indptr[b + 1];
  int q0 = a0 < 0 ? 0 : (a0 > p.total_q ? p.total_q : a0);
  int q1 = a1 < q0 ? q0 : (a1 > p.total_q ? p.total_q : a1);
  r.bad = q0 != a0 || q1 != a1;
  r.q0 = q0;
  r.n = q1 - q0;
  int P = p.prefix_len[b];
  if (P < 0) { P = 0; r.bad = true; }
  if (p.kv_start) {
    // a prefix longer than the pool cannot be there
    if (P > p.num_slots) { P = int(p.num_slots); r.bad = true; }
    if (P > 0x7fffffff - r.n) { P = 0x7fffffff - r.n; r.bad = true; }
    r.base = p.kv_start[b];
    r.nlist = P + r.n;
  } else {
    int64_t i0 = p.kv_indptr[b], i1 = p.kv_indptr[b + 1];
    if (i0 < 0 || i1 < i0 || i1 > p.num_entries) {
      r.bad = true;
      i0 = i0 < 0 ? 0 : (i0 > p.num_entries ? p.num_entries : i0);
      i1 = i1 < i0 ? i0 : (i1 > p.num_entries ? p.num_entries : i1);
    }
    const int nl = int(i1 - i0);
    if (nl - r.n < P) {   // a list shorter than prefix + tokens: the prefix gives way
      r.bad = true;
      P = nl > r.n ? nl - r.n : 0;
    }
    r.base = i0;
    r.nlist = nl;
  }
  r.P = P;
  return r;
}

// Pool row of key j (0 <= j < P + n), or -1 when it has none.
__device__ inline int64_t chunk_key_row(const ChunkParams& p, const ChunkReq& r, int j) {
  if (j >= r.nlist) return -1;
  const int64_t s = p.kv_start ? r.base + j : int64_t(p.slot_idx[r.base + j]);
  return (s >= 0 && s < p.num_slots) ? s : -1;
}

// First key past the sinks that the token at position `pos` (= P + its index)
// sees: pos - window + 1, or 0 without a window.
__device__ inline int window_first(int window, int pos) {
  return window > 0 && pos >= window ? pos - window + 1 : 0;
}

// One (token, head) row's attention over every key it sees, by one warp in
// 32-bit arithmetic: lane l holds columns 64k + 2l and 64k + 2l + 1 (k < 9) of
// the query and of each key row; the first eight pairs are also its columns of
// the value and of the output.  Hidden keys are not read at all, so nothing
// they hold (NaN, infinities) reaches the row.
__device__ inline void chunk_row(const ChunkParams& p, const ChunkReq& r, int i, int h, int lane,
                                 bool* bad_slot) {
  const size_t row = (size_t(r.q0) + i) * p.H + h;
  const uint32_t* q32 = reinterpret_cast<const uint32_t*>(p.q + row * kDqk);
  uint32_t q[9];
#pragma unroll
  for (int k = 0; k < 9; ++k) q[k] = q32[32 * k + lane];
  float acc[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) acc[k] = 0.f;
  // the row sum in two levels, 64 keys and their totals, so that its rounding
  // does not grow with a long context
  float m = -INFINITY, l = 0.f, l64 = 0.f;
  const int pos = r.P + i;
  const int first = window_first(p.window, pos);
  const int nsink = p.sinks < first ? p.sinks : first;
  const int count = nsink + (pos + 1 - first);
  for (int c = 0; c < count; ++c) {
    const int j = c < nsink ? c : c - nsink + first;
    const int64_t kr = chunk_key_row(p, r, j);
    if (kr < 0) {
      *bad_slot = true;
      continue;
    }
    const uint32_t* k32 = reinterpret_cast<const uint32_t*>(p.kv + kr * p.kv_stride);
    uint32_t kv[9];
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 9; ++k) kv[k] = k32[32 * k + lane];
#pragma unroll
    for (int k = 0; k < 9; ++k) {
      s = fmaf(bf16lo(q[k]), bf16lo(kv[k]), s);
      s = fmaf(bf16hi(q[k]), bf16hi(kv[k]), s);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= p.scale_log2;
    if (s > m) {
      const float a = exp2f(m - s);   // 0 when nothing was seen before
      l *= a;
      l64 *= a;
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[k] *= a;
      m = s;
    }
    const float e = m == -INFINITY && !isnan(s) ? 0.f : exp2f(s - m);
    l64 += e;
    if ((c & 63) == 63) {
      l += l64;
      l64 = 0.f;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      acc[2 * k] = fmaf(e, bf16lo(kv[k]), acc[2 * k]);
      acc[2 * k + 1] = fmaf(e, bf16hi(kv[k]), acc[2 * k + 1]);
    }
  }
  l += l64;
  const float inv = l == 0.f ? 0.f : 1.f / l;   // a row that saw no key: out 0, lse -inf
  uint32_t* o32 = reinterpret_cast<uint32_t*>(p.out + row * kDv);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const __nv_bfloat162 o = __floats2bfloat162_rn(acc[2 * k] * inv, acc[2 * k + 1] * inv);
    o32[32 * k + lane] = *reinterpret_cast<const uint32_t*>(&o);
  }
  if (lane == 0) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Checks shared by the chunk calls (va_chunk.cu).
int chunk_check(const ChunkParams& p, bool paged, float sm_scale, int flags, const void* ws);

}  // namespace va
