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
//
// Two paths: the tensor cores -- a kernel for few rows per request
// (va_decode_tc.cu), one for many (va_prefill_tc.cu), and between them that of the
// verify calls in its chunk mode (va_tc.cu) -- followed by chunk_finish_kernel,
// which merges the splits; and one warp per row on CUDA cores (VA_PATH_FMA), an
// independent implementation that the finish kernel also uses for the rare rows
// that the products may have spoilt (see kFlagHiddenNonfinite).
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
    if (chunk_ends(p, b)) break;
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

// Merge of the splits (and the call's status word).  Split s of a row left its
// normalised partial o_s and lse_s; with L = ln sum_s exp(lse_s) the row is
// sum_s exp(lse_s - L) o_s, in a fixed order.  A row is taken by one warp, or,
// when there are too few rows to fill the SMs that way, by the kW = 8 warps of a
// CTA, each with every eighth split; a lane holds 16 of the 512 columns.  Rows of
// units in one split are final already and only passed over.  Bound by the
// partials' bytes (2 KB per row and split, mostly from L2) and, with few rows, by
// the latency of the unit's entry, the lse values and the partials.  (Rows dealt
// out before looking whether their unit needs anything took 87 us for the 278k
// rows of three prompts, all of them final.)
constexpr int kFinishThreads = 256;
constexpr int kFinishWarps = kFinishThreads / 32;
constexpr int kMaxNs = 544;   // splits of a unit: at most all items of a launch (see below)

template <int kW>
__global__ void __launch_bounds__(kFinishThreads) chunk_finish_kernel(const ChunkTcParams p) {
  static_assert(kW == 1 || kW == kFinishWarps, "a warp or a CTA per row");
  __shared__ float weight[kFinishWarps][kMaxNs];
  __shared__ ChunkUnit list[kFinishThreads];   // units to merge (b < 0: ~b, to compute again)
  __shared__ int warp_count[kFinishWarps];
  __shared__ float4 sums[kW == 1 ? 1 : kFinishWarps][kDv / 4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_wait();                // the split kernel's results are complete
  griddep_launch_dependents();   // the next kernel may start its set-up
  const int U = p.sched.unit_rows;
  const int total_units = p.totals[0];
  constexpr int kRowsPerCta = kFinishWarps / kW;
  float* w = weight[warp];
  // every CTA's status bits; which units a hidden key may have spoilt is looked
  // up only when there is one
  uint32_t bits = 0u;
  {
    const int n = p.totals[1] * p.ctas;
#pragma unroll 4
    for (int i = tid; i < n; i += kFinishThreads) bits |= p.cta_flags[i];
    if (blockIdx.x == 0)
      for (int i = tid; i < p.pack_blocks; i += kFinishThreads) bits |= p.pack_flags[i] & ~kPackMissing;
  }
  const bool hidden = __syncthreads_or((bits & kFlagHiddenNonfinite) != 0u);
  // (a CTA that gave up a wait has not written the entries of the units that it
  // did not reach: then nothing is merged, and the status word says so)
  const bool gave_up = __syncthreads_or((bits & VA_STATUS_TIMEOUT) != 0u);
  for (int u0 = 0; !gave_up && u0 < total_units; u0 += kFinishThreads) {
    // which of 256 units need work: listed in the same order by every CTA
    ChunkUnit unit;
    unit.ns = 1;
    uint32_t f = 0u;
    if (u0 + tid < total_units) {
      unit = p.units[u0 + tid];
      if (hidden)
        for (int s = 0; s < unit.ns; ++s)
          for (int c = 0; c < p.ctas; ++c)
            f |= p.cta_flags[size_t(unit.item + s * unit.istride) * p.ctas + c];
      if (f & kFlagHiddenNonfinite) unit.b = ~unit.b;
    }
    const bool need = unit.ns > 1 || (f & kFlagHiddenNonfinite);
    const uint32_t ballot = __ballot_sync(0xffffffffu, need);
    if (lane == 0) warp_count[warp] = __popc(ballot);
    __syncthreads();
    int at = __popc(ballot & ((1u << lane) - 1u)), count = 0;
#pragma unroll
    for (int k = 0; k < kFinishWarps; ++k) {
      at += k < warp ? warp_count[k] : 0;
      count += warp_count[k];
    }
    if (need) list[at] = unit;
    __syncthreads();
    for (int id = int(blockIdx.x) * kRowsPerCta + (kW == 1 ? warp : 0); id < count * U;
         id += int(gridDim.x) * kRowsPerCta) {
      const ChunkUnit& x = list[id / U];
      const int r = id % U;
      if (r >= x.rows) continue;
      if (x.b < 0) {   // a hidden key may have spoilt the unit's rows
        if (kW == 1 || warp == 0) {
          bool bad = false;
          chunk_row(p, chunk_req(p, ~x.b), (x.i0 + r) / p.H, (x.i0 + r) % p.H, lane, &bad);
        }
        continue;
      }
      const int ns = x.ns < kMaxNs ? x.ns : kMaxNs;
      auto slot = [&](int s) -> size_t {
        return size_t(s == 0 ? x.pslot : x.pslot1 + (s - 1) * x.pstride) * U + r;
      };
      float m = -INFINITY;
      for (int s = lane; s < ns; s += 32) {
        const float ls = p.part_lse[slot(s)];
        w[s] = ls;
        m = fmaxf(m, ls);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      float z = 0.f;
      for (int s = lane; s < ns; s += 32)
        if (w[s] != -INFINITY) z += expf(w[s] - m);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
      const float L = z == 0.f ? -INFINITY : m + logf(z);
      for (int s = lane; s < ns; s += 32) w[s] = w[s] == -INFINITY ? 0.f : expf(w[s] - L);
      __syncwarp();
      if (lane == 0 && (kW == 1 || warp == 0)) p.lse[x.row0 + r] = L;
      // columns 4 * lane + 128 q .. + 3
      float4 acc[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int s = kW == 1 ? 0 : warp; s < ns; s += kW) {
        const float4* src = reinterpret_cast<const float4*>(p.part_o + slot(s) * kDv) + lane;
        const float ws = w[s];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 v = src[32 * q];
          acc[q].x = fmaf(ws, v.x, acc[q].x);
          acc[q].y = fmaf(ws, v.y, acc[q].y);
          acc[q].z = fmaf(ws, v.z, acc[q].z);
          acc[q].w = fmaf(ws, v.w, acc[q].w);
        }
      }
      __syncwarp();   // w is read
      uint2* out = reinterpret_cast<uint2*>(p.out + size_t(x.row0 + r) * kDv);
      auto pack = [](float4 v) -> uint2 {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
        return make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      };
      if constexpr (kW == 1) {
#pragma unroll
        for (int q = 0; q < 4; ++q) out[32 * q + lane] = pack(acc[q]);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) sums[warp][32 * q + lane] = acc[q];
        __syncthreads();
        if (tid < kDv / 4) {
          float4 t = sums[0][tid];
#pragma unroll
          for (int k = 1; k < kW; ++k) {
            const float4 v = sums[k][tid];
            t.x += v.x;
            t.y += v.y;
            t.z += v.z;
            t.w += v.w;
          }
          out[tid] = pack(t);
        }
        __syncthreads();
      }
    }
    __syncthreads();   // the list is read
  }
  // the status word: every CTA's bits, and requests whose bounds were clamped
  if (blockIdx.x == 0) {
    __shared__ uint32_t s_bits;
    if (tid == 0) s_bits = 0u;
    __syncthreads();
    bits &= ~kFlagHiddenNonfinite;
    for (int b = tid; b < p.B; b += kFinishThreads)
      if (chunk_req(p, b).bad) bits |= VA_STATUS_BAD_INDPTR;
    if (bits) atomicOr(&s_bits, bits);
    __syncthreads();
    if (tid == 0) *p.status = s_bits;
  }
}

// ------------------------------------------------------------- host side

// Clusters of the tensor-core kernel that a GB300's 152 SMs hold at most; the
// workspace is sized for them, so that sizing it takes no device call.
constexpr int kMaxSms = 152, kMaxPairs = 76, kMaxQuads = 38;
static_assert(kMaxNs >= kMaxSms && kMaxNs >= kSplitWaves * kMaxPairs, "splits of a unit");
// Paged rows are packed side by side for the prefill kernel (va_prefill_tc.cu),
// which pays from this many query rows per request on, on the average: then about
// three units read the packed rows instead of gathering them.  64 heads, split
// kernel against prefill kernel: 32 requests of 8k keys, 512 rows 342 and 331 us,
// 768 rows 514 and 428, 2048 rows 1292 and 883; 4 requests of 16k keys, 117 and 124,
// 150 and 144, 323 and 261.  Enormous lists, whose copy would not, are left to the
// split kernel.
constexpr int kPrefillRows = 640;
constexpr int64_t kPackEntriesMax = int64_t(1) << 21;

// Requests up to which the split kernel is taken.  Each of its clusters looks through
// all requests for its piece, so a launch's time grows with their square; the decode and
// prefill kernels look once per SM.  64 heads' worth of rows, split kernel against the
// other: 128 rows of 8k keys, 64 requests 280 and 299 us, 128 702 and 568, 256 1371 and
// 1106; 256 rows of 4k keys against the prefill kernel, 245 and 250, 667 and 444, 939 and
// 830; 1024 requests of 1k keys 2164 and 668, 4159 and 959.  (65535 requests of 200
// rows took 14 s.)  Lists too long to be packed go to the decode kernel, which reads the
// keys once per 64 rows, from more requests on only (256 rows: 512 requests of 4.5k keys
// 2542 and 3029 us, 1024 of 2.2k 5155 and 3639, 4096 of 600 69.8 and 7.8 ms).
constexpr int kSplitRequests = 96, kSplitRequestsLong = 768;

struct ChunkPlan {
  bool decode;       // va_decode_tc.cu
  bool prefill;      // va_prefill_tc.cu
  bool pair;
  int unit_rows, ctas, max_clusters;
  int units_bound;   // units the batch can have
  int max_waves;     // waves of clusters in the grid
  int pack_blocks;
  size_t off_units, off_flags, off_lse, off_o, off_pack_flags, off_valid, off_tails, off_pack, total;
};

// By the average request's rows.  Up to 64, one unit of the decode kernel (64 rows
// each in 32 requests of 8k paged keys: 89 us, the split kernel 143; with 128 rows,
// two units, 161 and 146).  Up to 128, the split kernel with a pair of SMs per
// unit.  Above that products of two SMs (128 rows: one-SM products 146 us, two-SM
// 191; 192 rows: 234 and 183): the prefill kernel where keys lie side by side
// (192 rows: split 162 us, prefill 131; 4 requests of 16k keys, 82 and 55) or can be
// packed (see kPrefillRows), else the split kernel.  Batches of many requests: see
// kSplitRequests.
ChunkPlan chunk_plan(int B, int total_q, int H, int64_t num_entries, int flags) {
  ChunkPlan c;
  memset(&c, 0, sizeof c);
  const int64_t rows = int64_t(total_q) * H;
  const int busy = B < total_q ? B : total_q;   // requests with tokens, at most
  const bool paged = num_entries > 0, many = B > kSplitRequests;
  c.decode = flags != VA_PATH_TC_1SM && rows <= (many ? 128 : 64) * int64_t(busy);
  c.pair = flags != VA_PATH_TC_1SM && rows > 128 * int64_t(busy);
  c.prefill = c.pair && (!paged || ((many || rows >= kPrefillRows * int64_t(busy)) &&
                                    num_entries <= kPackEntriesMax));
  if (c.pair && !c.prefill && B > kSplitRequestsLong) {
    c.decode = true;
    c.pair = false;
  }
  c.unit_rows = c.decode ? 64 : c.pair ? 256 : 128;
  c.ctas = c.decode ? 1 : c.pair ? 4 : 2;
  c.max_clusters = c.decode ? kMaxSms : c.pair ? kMaxQuads : kMaxPairs;
  c.units_bound = int((rows + c.unit_rows - 1) / c.unit_rows) + busy;
  // (fewer clusters than the most may be resident: the waves are counted for
  // three quarters of them at least, see launch)
  const int waves = (c.units_bound + c.max_clusters * 3 / 4 - 1) / (c.max_clusters * 3 / 4);
  c.max_waves = waves > kSplitWaves ? waves : kSplitWaves;
  // the decode and prefill kernels: an item and two slots per CTA or cluster
  const bool even = c.decode || c.prefill;
  const size_t items = even ? size_t(c.max_clusters) : size_t(c.max_waves) * c.max_clusters;
  const size_t slots = size_t(even ? 2 : kSplitWaves) * c.max_clusters;
  c.off_units = kHeaderBytes;
  c.off_flags = c.off_units + align256(size_t(c.units_bound) * sizeof(ChunkUnit));
  c.off_lse = c.off_flags + align256(items * c.ctas * sizeof(uint32_t));
  c.off_o = c.off_lse + align256(slots * c.unit_rows * sizeof(float));
  c.off_pack_flags = c.off_o + align256(slots * c.unit_rows * kDv * sizeof(float));
  c.total = c.off_pack_flags;
  if (c.prefill) {
    constexpr size_t kRowBytes = kDqk * sizeof(__nv_bfloat16);
    c.pack_blocks = int((num_entries + 255) / 256);
    // (entries rounded up to whole blocks; two words more for the last tile's bits)
    c.off_valid = c.off_pack_flags + align256(size_t(c.pack_blocks) * sizeof(uint32_t));
    c.off_tails = c.off_valid + align256((size_t(c.pack_blocks) * 8 + 4) * sizeof(uint32_t));
    c.off_pack = c.off_tails + align256(size_t(B) * 64 * kRowBytes);
    c.total = c.off_pack + size_t(num_entries) * kRowBytes;
  }
  return c;
}

// What va_prefill_tc.cu reads, laid out for its boxes.  The first `pack_blocks`
// blocks (paged calls): every listed row that lies in a tile some token sees, at
// its list position in `packed` (zeros for a key without a row), and a bit per
// entry that has one.  Then a block per request: its last tile, when that is not
// whole, with zeros behind the request's last key.  A warp takes 32 entries (or 8
// rows of a tail): a lane finds the pool row of one, then the warp copies four rows
// at a time, all loads before the stores.  Bound by HBM: 1152 B read and written
// per key.
constexpr int kPackThreads = 256;

// Rows k .. k + 3 of the warp's: lane x holds row x's pool row (-1: zeros, -2: no
// copy); row x goes to dst + x rows.
__device__ __forceinline__ void copy_rows(const ChunkParams& p, int64_t row, int count, uint4* dst,
                                          int lane) {
  constexpr int kChunks = kDqk / 8;   // 72 chunks of 16 bytes
  for (int k = 0; k < count; k += 4) {
    uint4 v[4][3];
    int64_t src[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      src[x] = __shfl_sync(0xffffffffu, row, k + x);
      const uint4* s = reinterpret_cast<const uint4*>(p.kv + (src[x] > 0 ? src[x] : 0) * p.kv_stride);
#pragma unroll
      for (int c = 0; c < 3; ++c) {
        v[x][c] = make_uint4(0u, 0u, 0u, 0u);
        if (src[x] >= 0 && lane + 32 * c < kChunks) v[x][c] = s[lane + 32 * c];
      }
    }
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int c = 0; c < 3; ++c)
        if (src[x] >= -1 && lane + 32 * c < kChunks)
          dst[size_t(k + x) * kChunks + lane + 32 * c] = v[x][c];
  }
}

__global__ void __launch_bounds__(kPackThreads) chunk_pack_kernel(const ChunkTcParams p) {
  griddep_wait();                // the stream's previous kernel has completed
  griddep_launch_dependents();   // the attention kernel may start its set-up
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (int(blockIdx.x) >= p.pack_blocks) {
    const int b = int(blockIdx.x) - p.pack_blocks;
    const ChunkReq r = chunk_req(p, b);
    const int N = r.nlist < r.P + r.n ? r.nlist : r.P + r.n;
    if (N % 64 == 0 || r.n == 0) return;
    const int i0 = 8 * warp, j = N / 64 * 64 + i0 + lane;
    const int64_t row = lane < 8 && j < N ? chunk_key_row(p, r, j) : -1;
    copy_rows(p, row, 8,
              reinterpret_cast<uint4*>(const_cast<__nv_bfloat16*>(p.tails) +
                                       (size_t(b) * 64 + i0) * kDqk), lane);
    return;
  }
  const int64_t e = int64_t(blockIdx.x) * kPackThreads + tid, e0 = e - lane;
  int64_t row = -2;
  bool bad = false;
  const int requests = chunk_requests(p, lane);
  const bool sorted = chunk_lists_sorted(p, lane);
  // what request b makes of the entry
  auto look = [&](int b) {
    const ChunkReq r = chunk_req(p, b);
    const int64_t j = e - r.base;
    const int first = window_first(p.window, r.P);
    if (r.n > 0 && j >= 0 && j < r.P + r.n && j < r.nlist &&
        (j >= (first & ~63) || j < (int64_t(p.sinks) + 63) / 64 * 64)) {
      row = chunk_key_row(p, r, int(j));
      bad |= row < 0 && (j >= first || j < p.sinks);
    }
  };
  if (e < p.num_entries && sorted) {
    int lo = 0, hi = p.B;   // the last list that begins at or before e
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.kv_indptr[mid] <= e) lo = mid;
      else hi = mid;
    }
    if (lo < requests) look(lo);
  } else if (e < p.num_entries) {   // bounds in error: any request's list may hold it
    for (int b = 0; b < requests; ++b) look(b);
  }
  const uint32_t have = __ballot_sync(0xffffffffu, row >= 0);
  if (lane == 0) const_cast<uint32_t*>(p.valid)[e0 >> 5] = have;
  const bool any_bad = __syncthreads_or(bad), missing = __syncthreads_or(row == -1);
  if (tid == 0)
    p.pack_flags[blockIdx.x] = (any_bad ? VA_STATUS_BAD_SLOT : 0u) | (missing ? kPackMissing : 0u);
  copy_rows(p, row, 32, reinterpret_cast<uint4*>(const_cast<__nv_bfloat16*>(p.packed) + e0 * kDqk),
            lane);
}

cudaError_t launch_pack(const ChunkTcParams& p, cudaStream_t st) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(unsigned(p.pack_blocks + p.B), 1, 1);
  cfg.blockDim = dim3(kPackThreads, 1, 1);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_pack_kernel, p);
}

cudaError_t launch_finish(const ChunkTcParams& p, int units_bound, int num_sms, cudaStream_t st) {
  const int64_t wave = int64_t(num_sms) * 8;   // CTAs
  const int64_t rows = int64_t(p.total_q) * p.H;
  // a CTA per row while one wave of CTAs covers the rows, else a warp per row
  const bool cta_rows = rows <= wave;
  const int64_t ids = int64_t(units_bound) * p.sched.unit_rows;   // rows, padded to units
  const int64_t want = cta_rows ? ids : (ids + kFinishWarps - 1) / kFinishWarps;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(unsigned(want < wave ? want : wave), 1, 1);
  cfg.blockDim = dim3(kFinishThreads, 1, 1);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cta_rows ? cudaLaunchKernelEx(&cfg, chunk_finish_kernel<kFinishWarps>, p)
                  : cudaLaunchKernelEx(&cfg, chunk_finish_kernel<1>, p);
}

}  // namespace

int chunk_check(const ChunkParams& p, bool paged, float sm_scale, int flags, const void* ws) {
  if (!p.kv || !p.prefix_len || !p.q_indptr || !ws) return VA_ERR_NULL;
  if (p.total_q > 0 && (!p.q || !p.lse)) return VA_ERR_NULL;
  // (an empty list has no address)
  if (paged ? ((!p.slot_idx && p.num_entries != 0) || !p.kv_indptr) : !p.kv_start) return VA_ERR_NULL;
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
  if (p.num_entries < 0 || p.num_entries > kKeysMax) return VA_ERR_SHAPE;
  if (p.num_slots > 0x7fffff00) return VA_ERR_SHAPE;   // rows are named by 32-bit coordinates
  if (ws_bytes < va_chunk_workspace_bytes(p.B, p.total_q, p.H, p.num_entries, flags))
    return VA_ERR_WORKSPACE;
  DeviceInfo di;
  const int rd = device_info(&di);
  if (rd != VA_OK) return rd;
  p.scale_log2 = sm_scale * kLog2e;
  p.status = static_cast<uint32_t*>(ws);
  const int64_t rows = int64_t(p.total_q) * p.H;
  // (no entries at all: no keys, and nothing to lay out for the tensor cores)
  if (flags == VA_PATH_FMA || rows == 0 || (!p.kv_start && p.num_entries == 0)) {
    if (cudaMemsetAsync(ws, 0, sizeof(uint32_t), st) != cudaSuccess) return VA_ERR_LAUNCH;
    if (rows == 0) return VA_OK;
    const int64_t want = (rows + kRowThreads / 32 - 1) / (kRowThreads / 32);
    const int64_t wave = int64_t(di.num_sms) * 8;
    chunk_fma_kernel<<<unsigned(want < wave ? want : wave), kRowThreads, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? VA_OK : VA_ERR_LAUNCH;
  }
  const ChunkPlan c = chunk_plan(p.B, p.total_q, p.H, p.num_entries, flags);
  uint8_t* w = static_cast<uint8_t*>(ws);
  ChunkTcParams t;
  memset(&t, 0, sizeof t);
  static_cast<ChunkParams&>(t) = p;
  t.scale_log2 = tc_scale_log2(sm_scale);
  const int resident = c.decode ? di.num_sms : c.pair ? di.quads : di.pairs;
  t.sched.unit_rows = c.unit_rows;
  t.sched.clusters = resident < c.max_clusters ? resident : c.max_clusters;
  if (!c.decode && t.sched.clusters < c.max_clusters * 3 / 4) return VA_ERR_UNSUPPORTED;
  t.ctas = c.ctas;
  t.totals = reinterpret_cast<int32_t*>(w) + 4;
  t.units = reinterpret_cast<ChunkUnit*>(w + c.off_units);
  t.cta_flags = reinterpret_cast<uint32_t*>(w + c.off_flags);
  t.part_lse = reinterpret_cast<float*>(w + c.off_lse);
  t.part_o = reinterpret_cast<float*>(w + c.off_o);
  cudaError_t e;
  if (c.prefill) {
    t.tails = reinterpret_cast<const __nv_bfloat16*>(w + c.off_tails);
    if (!p.kv_start) {
      t.packed = reinterpret_cast<const __nv_bfloat16*>(w + c.off_pack);
      t.valid = reinterpret_cast<const uint32_t*>(w + c.off_valid);
      t.pack_flags = reinterpret_cast<uint32_t*>(w + c.off_pack_flags);
      t.pack_blocks = c.pack_blocks;
    }
    if (launch_pack(t, st) != cudaSuccess) return VA_ERR_LAUNCH;
    e = launch_prefill_tc(t, t.sched.clusters, st);
  } else if (c.decode) {
    e = launch_decode_tc(t, t.sched.clusters, st);
  } else {
    // (at most max_waves * max_clusters items, which the workspace is sized for)
    const int waves = (c.units_bound + t.sched.clusters - 1) / t.sched.clusters;
    t.sched.max_waves = waves > kSplitWaves ? waves : kSplitWaves;
    e = launch_chunk_tc(t, t.sched.max_waves * t.sched.clusters, c.pair, st);
  }
  if (e != cudaSuccess) return VA_ERR_LAUNCH;
  t.scale_log2 = p.scale_log2;   // (rows that it computes again are CUDA-core rows)
  return launch_finish(t, c.units_bound, di.num_sms, st) == cudaSuccess ? VA_OK : VA_ERR_LAUNCH;
}

}  // namespace
}  // namespace va

VA_API size_t va_chunk_workspace_bytes(int B, int total_q, int H, int64_t num_entries,
                                       int flags) {
  if (num_entries < 0 || num_entries > va::kKeysMax || B < 1 || B > 65535 || total_q < 0 || H < 1 ||
      flags < VA_PATH_AUTO || flags > VA_PATH_TC_1SM || int64_t(total_q) * H > VA_CHUNK_ROWS_MAX)
    return 0;
  if (total_q == 0 || flags == VA_PATH_FMA) return va::kHeaderBytes;
  return va::chunk_plan(B, total_q, H, num_entries, flags).total;
}

VA_API int va_chunk_attn_paged(const void* q, const void* kv_pool, int64_t num_slots,
                               int64_t kv_row_stride, const int32_t* slot_idx,
                               const int32_t* kv_indptr, const int32_t* prefix_len,
                               const int32_t* q_indptr, int64_t num_entries, int B, int total_q,
                               int H, float sm_scale, int window, int sinks, int flags,
                               void* workspace, size_t workspace_bytes, void* out, float* lse,
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
  p.num_entries = num_entries;
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
