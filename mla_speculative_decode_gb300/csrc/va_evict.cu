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
// through the digits (12, 10 and 10 bits).  Every entry above that threshold
// stays, and of the entries equal to it as many as are still wanted, in index
// order.
//
// One cluster of CTAs per request, as many (1 to 8) as the SMs hold for the
// batch at once.  The list is read four times, from L2 after the first: the
// histogram of the first digit; that of the second digit, which also collects
// the candidates that match the first in shared memory, so that the third
// digit needs no reading; a count of what stays; and the compaction.
// Histograms are added across the cluster through distributed shared memory by
// every CTA.  For the last two a warp owns a contiguous piece of the list: it
// counts what stays of it, the warps exchange their counts once, and each then
// compacts its piece on its own, with no barrier in the loop (runs of a CTA's
// entries with a prefix sum over the CTA for each took 3.5 us a run of 4096, three
// times as long).  In place, an output may lie where another warp still reads:
// the kept entries then wait in shared memory until the cluster has read all of
// a window of the list -- the whole list when what stays of it fits.
// Bound by latency: barriers and dependent reads for a short list (4096 entries:
// 11.7 us, of which three digits take a third).  Of long ones (64 lists of 20k to 200k
// entries, 76 us, a sixth of the memory's rate counted once) the compaction takes a
// third, the passes of the first two digits and the count a sixth each; every list has
// the same number of CTAs, so those of the longest, 49.7k entries each, have twice an
// equal share of all entries, and the launch lasts as long as they do.
#include <math.h>
#include <string.h>

#include "va_common.cuh"
#include "va_sm100.cuh"

#ifndef VA_API
#define VA_API extern "C" __attribute__((visibility("default")))
#endif

namespace va {
namespace {

constexpr int kEvictThreads = 512;
constexpr int kWarps = kEvictThreads / 32;
constexpr int kBits1 = 12, kBits2 = 10, kBits3 = 10;   // digits, from the top
constexpr int kCtaBudget = 2;   // CTAs that an SM's registers and shared memory hold
constexpr int kPer = 8;                                // entries of a thread and step
constexpr int kBatch = 16;                             // of a thread at once in the histograms
constexpr int kList = 4096;                            // collected candidates per CTA
// Entries at most: positions are 32-bit, and threads step past a list's end by up to
// two batches, warps by a piece of it (1/128 of a list, of 2^31 entries 2^24).
constexpr int64_t kEntriesMax = 0x7fffffff - (1 << 25);
constexpr int kHeld = 10240;                           // kept entries that a CTA can hold back

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
  int ctas;     // CTAs per request
  bool finish;  // a second kernel writes the lengths and the head
  bool hold;    // in place: kept entries wait in shared memory (kHeld per CTA)
};

// A weight as an unsigned integer of the same order.
__device__ __forceinline__ uint32_t weight_key(float w) {
  w = fmaxf(w, -INFINITY) + 0.f;   // NaN counts as -inf; -0 and +0 are equal
  const uint32_t u = __float_as_uint(w);
  return u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
}
// ... and back.
__device__ __forceinline__ float key_weight(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
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
  for (int w = 0; w < kWarps; ++w) t += red[w];
  return t;
}

__device__ __forceinline__ uint4 ld_cluster_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

struct EvictSmem {
  uint32_t hist1[1 << kBits1];
  uint32_t hist2[1 << kBits2];
  uint32_t hist3[1 << kBits3];
  uint32_t wsum[kWarps];
  uint2 count[kWarps];         // a warp's entries that stay whatever the others are; equal ones
  uint2 total[2];              // this CTA's, by the window's parity
  uint32_t nlist, digit, above;
  int64_t red[kWarps];
  // low 20 bits of the candidates that match the first digit; later, when
  // the launch asks for it, kHeld kept entries (slot, weight)
  alignas(16) uint32_t list[kList];
};
constexpr size_t kHeldBytes = size_t(kHeld) * 8 - sizeof(uint32_t) * kList;   // beyond `list`

// The digit at which the counts from the top of the histogram, added over the
// cluster's CTAs, reach `want` (>= 1), and the count above it.  A thread holds
// kN consecutive bins (the first kBins / kN threads).  Ends with the block in
// step; the cluster has to have met since the histogram was filled.
template <int kBins>
__device__ void find_digit(EvictSmem& sm, const uint32_t* hist, int ctas, uint32_t want) {
  constexpr int kN = kBins / kEvictThreads;
  static_assert(kBins == kN * kEvictThreads, "a run of bins per thread");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t = kEvictThreads - 1 - tid;   // threads in order hold bins from the top down
  uint32_t bin[kN];
#pragma unroll
  for (int k = 0; k < kN; ++k) bin[k] = 0;
  const uint32_t at = smem_u32(hist + t * kN);
#pragma unroll 4
  for (int c = 0; c < ctas; ++c) {
    const uint32_t a = sm100::mapa(at, uint32_t(c));
    if constexpr (kN % 4 == 0) {
#pragma unroll
      for (int k = 0; k < kN; k += 4) {
        const uint4 v = ld_cluster_v4(a + 4u * uint32_t(k));
        bin[k] += v.x; bin[k + 1] += v.y; bin[k + 2] += v.z; bin[k + 3] += v.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < kN; ++k) bin[k] += ld_cluster(a + 4u * uint32_t(k));
    }
  }
  uint32_t mine = 0;
#pragma unroll
  for (int k = 0; k < kN; ++k) mine += bin[k];
  uint32_t sum = mine;   // inclusive over the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 31) sm.wsum[warp] = sum;
  __syncthreads();
  uint32_t before = 0;   // the warps before this one: a warp's worth of sums
  {
    uint32_t x = lane < warp ? sm.wsum[lane] : 0u;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    before = x;
  }
  uint32_t above = before + sum - mine;
  if (above < want && want <= above + mine) {
    int k = kN - 1;
    for (; k > 0 && above + bin[k] < want; --k) above += bin[k];
    sm.digit = uint32_t(t * kN + k);
    sm.above = above;
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kEvictThreads, 2) evict_kernel(const EvictParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  EvictSmem& sm = *reinterpret_cast<EvictSmem*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = p.ctas, rank = int(sm100::cluster_ctarank());
  const int b = int(blockIdx.x) / ctas;
  for (int d = tid; d < (1 << kBits1); d += kEvictThreads) sm.hist1[d] = 0;
  for (int d = tid; d < (1 << kBits2); d += kEvictThreads) sm.hist2[d] = 0;
  for (int d = tid; d < (1 << kBits3); d += kEvictThreads) sm.hist3[d] = 0;
  if (tid == 0) sm.nlist = 0;
  griddep_wait();                // the stream's previous kernel has completed
  griddep_launch_dependents();   // the next kernel may start its set-up
  bool bad = false;
  int64_t base;
  const int L = evict_list(p, b, &base, &bad);
  if (bad && tid == 0 && rank == 0 && p.status) atomicOr(p.status, VA_STATUS_BAD_INDPTR);
  const int nfreed = L > p.budget ? L - p.budget : 0;

  // place of the request's first evicted slot in the free list
  int64_t free0 = 0;
  if (p.free_slots) {
    int64_t before = 0, all = 0;
    for (int x = tid; x < p.B; x += kEvictThreads) {
      const int64_t n = evicted_of(p, x);
      all += n;
      if (x < b) before += n;
    }
    before = block_sum(before, sm.red);
    all = block_sum(all, sm.red);
    const int64_t head = *p.free_head;
    free0 = head - all + before;
    if (!p.finish && blockIdx.x == 0 && tid == 0)
      *p.head_out = int32_t(head - all < 0 ? 0 : head - all);
  }
  if (nfreed == 0 && p.slot_out == p.slot_idx && p.weights_out == p.weights) {
    // in place, and all of it stays: every CTA of the cluster leaves (the
    // length written is the one they all clamp theirs to)
    if (!p.finish && rank == 0 && tid == 0) p.prefix_out[b] = L;
    return;
  }
  __syncthreads();

  // this CTA's part of the list, and the candidates within it
  const int part = (L + ctas - 1) / ctas;
  const int p0 = rank * part < L ? rank * part : L, p1 = p0 + part < L ? p0 + part : L;
  const int lo = nfreed ? p.sinks : 0, hi = nfreed ? L - p.recent : 0;   // all candidates
  const int c0 = p0 > lo ? p0 : lo, c1 = p1 < hi ? p1 : hi;
  const int m = p.budget - p.sinks - p.recent;                          // of which stay
  uint32_t thr = 0xffffffffu, want = 0u;   // threshold's key; entries equal to it that stay
  if (nfreed && m > 0) {
    const float* w = p.weights + base;
    want = uint32_t(m);
    // all of this CTA's candidates, kBatch loads of a thread on their way at once,
    // the last ones included
    auto each = [&](auto&& use) {
      for (int i0 = c0 + tid; i0 < c1; i0 += kBatch * kEvictThreads) {
        float x[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int i = i0 + k * kEvictThreads;
          x[k] = i < c1 ? w[i] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (i0 + k * kEvictThreads < c1) use(weight_key(x[k]));
      }
    };
    each([&](uint32_t k) { atomicAdd(&sm.hist1[k >> (kBits2 + kBits3)], 1u); });
    sm100::cluster_sync();
    find_digit<1 << kBits1>(sm, sm.hist1, ctas, want);
    const uint32_t d1 = sm.digit;
    want -= sm.above;
    __syncthreads();
    each([&](uint32_t k) {
      if ((k >> (kBits2 + kBits3)) == d1) {
        atomicAdd(&sm.hist2[(k >> kBits3) & ((1u << kBits2) - 1u)], 1u);
        const uint32_t at = atomicAdd(&sm.nlist, 1u);
        if (at < kList) sm.list[at] = k & ((1u << (kBits2 + kBits3)) - 1u);
      }
    });
    sm100::cluster_sync();
    find_digit<1 << kBits2>(sm, sm.hist2, ctas, want);
    const uint32_t d2 = sm.digit;
    want -= sm.above;
    const uint32_t nlist = sm.nlist;
    __syncthreads();
    constexpr uint32_t kLow = (1u << kBits3) - 1u;
    if (nlist <= kList) {
      for (uint32_t i = tid; i < nlist; i += kEvictThreads)
        if ((sm.list[i] >> kBits3) == d2) atomicAdd(&sm.hist3[sm.list[i] & kLow], 1u);
    } else {   // more matched the first digit than the list holds
      const uint32_t d12 = d1 << kBits2 | d2;
      each([&](uint32_t k) {
        if ((k >> kBits3) == d12) atomicAdd(&sm.hist3[k & kLow], 1u);
      });
    }
    sm100::cluster_sync();
    find_digit<1 << kBits3>(sm, sm.hist3, ctas, want);
    thr = (d1 << kBits2 | d2) << kBits3 | sm.digit;
    want -= sm.above;
  }
  const float T = key_weight(thr);   // (NaN, which equals and exceeds nothing, when none stays)
  const int32_t* slot_in = p.slot_idx + base;
  const float* w_in = p.weights + base;
  int32_t* slot_o = p.slot_out + base;
  float* w_o = p.weights_out + base;
  uint2* held = reinterpret_cast<uint2*>(sm.list);
  // the request's evicted slots: their places in the free list, and whether all
  // of them lie inside it
  int32_t* fr = p.free_slots ? p.free_slots + free0 : nullptr;
  const bool fits = free0 >= 0 && free0 + nfreed <= p.free_capacity;
  const uint32_t below = (1u << lane) - 1u;
  constexpr int kStep = 32 * kPer;   // entries of a warp's step

  // Windows of the list: all of it, unless what is kept has to be held back and a
  // CTA's share does not fit, when a window is what fits even if all of it stays.
  int window = L;
  uint32_t kept = 0, equal = 0;   // kept, and equal to the threshold, before the window
  for (int w0 = 0, parity = 0; w0 < L; parity ^= 1) {
    const int w1 = L - w0 < window ? L : w0 + window;
    // this warp's piece
    const int piece = (w1 - w0 + ctas * kWarps - 1) / (ctas * kWarps);
    const int at0 = w0 + (rank * kWarps + warp) * piece;
    const int q0 = at0 < w1 ? at0 : w1, q1 = q0 + piece < w1 ? q0 + piece : w1;
    uint32_t n_stay = 0, n_eq = 0;
    for (int i0 = q0; i0 < q1; i0 += kStep) {
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int i = i0 + 32 * k + lane;
        if (i < q1) {
          const float x = w_in[i];
          const bool cand = i >= lo && i < hi;
          n_stay += !cand || x > T ? 1u : 0u;
          n_eq += cand && fmaxf(x, -INFINITY) == T ? 1u : 0u;
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      n_stay += __shfl_xor_sync(0xffffffffu, n_stay, o);
      n_eq += __shfl_xor_sync(0xffffffffu, n_eq, o);
    }
    if (lane == 0) sm.count[warp] = make_uint2(n_stay, n_eq);
    __syncthreads();
    // what the warps before this one count, in the CTA and (below) the cluster
    uint32_t my_stay = 0, my_eq = 0, cta_stay = 0, cta_eq = 0;
#pragma unroll
    for (int x = 0; x < kWarps; ++x) {
      const uint2 c = sm.count[x];
      if (x < warp) { my_stay += c.x; my_eq += c.y; }
      cta_stay += c.x;
      cta_eq += c.y;
    }
    if (tid == 0) sm.total[parity] = make_uint2(cta_stay, cta_eq);
    sm100::cluster_sync();
    // Equal entries stay while fewer than `want` came before: e of them, up to a
    // place, have kept min(e, want).
    auto eq_kept = [&](uint32_t e) { return e < want ? e : want; };
    uint32_t all_stay = 0, all_eq = 0, cta_at = 0, cta_eq_at = 0, most = 0;
    for (int c = 0; c < ctas; ++c) {
      const uint32_t a = sm100::mapa(smem_u32(&sm.total[parity]), uint32_t(c));
      if (c == rank) { cta_at = all_stay; cta_eq_at = all_eq; }
      const uint32_t n = ld_cluster(a), e = ld_cluster(a + 4);
      const uint32_t both = n + eq_kept(equal + all_eq + e) - eq_kept(equal + all_eq);
      most = both > most ? both : most;
      all_stay += n;
      all_eq += e;
    }
    if (p.hold && most > uint32_t(kHeld)) {   // (the whole cluster; a smaller window fits)
      window = ctas * kHeld;
      continue;
    }
    const uint32_t k0 = kept - eq_kept(equal);   // kept before the window, without equal ones
    const uint32_t out0 = k0 + cta_at + eq_kept(equal + cta_eq_at);   // this CTA's first output
    uint32_t stay = k0 + cta_at + my_stay, eq = equal + cta_eq_at + my_eq;
    for (int i0 = q0; i0 < q1; i0 += kStep) {
      int s[kPer];
      float v[kPer];
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int i = i0 + 32 * k + lane;
        s[k] = i < q1 ? slot_in[i] : 0;
        v[k] = i < q1 ? w_in[i] : 0.f;
      }
      // The usual step: candidates all of them, none equal to the threshold.
      bool other = i0 < lo || i0 + kStep > (hi < q1 ? hi : q1) || (fr && !fits);
#pragma unroll
      for (int k = 0; k < kPer; ++k) other |= fmaxf(v[k], -INFINITY) == T;
      if (!__any_sync(0xffffffffu, other)) {
        const uint32_t e0 = eq_kept(eq);
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const bool a = v[k] > T;
          const uint32_t ba = __ballot_sync(0xffffffffu, a);
          const uint32_t at = stay + e0 + uint32_t(__popc(ba & below));
          stay += uint32_t(__popc(ba));
          if (a && p.hold) {
            held[at - out0] = make_uint2(uint32_t(s[k]), __float_as_uint(v[k]));
          } else if (a) {
            slot_o[at] = s[k];
            w_o[at] = v[k];
          } else if (fr) {
            fr[i0 + 32 * k + lane - int(at)] = s[k];
          }
        }
        continue;
      }
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int i = i0 + 32 * k + lane;
        const bool in = i < q1, cand = i >= lo && i < hi;
        const bool a = in && (!cand || v[k] > T);
        const bool e = in && cand && fmaxf(v[k], -INFINITY) == T;
        const uint32_t ba = __ballot_sync(0xffffffffu, a), be = __ballot_sync(0xffffffffu, e);
        uint32_t e_at = eq;
        if (be) {   // (few, as a rule)
          e_at += uint32_t(__popc(be & below));
          eq += uint32_t(__popc(be));
        }
        const uint32_t at = stay + uint32_t(__popc(ba & below)) + eq_kept(e_at);
        stay += uint32_t(__popc(ba));
        const bool keep = a || (e && e_at < want);
        if (keep) {
          if (p.hold) {
            held[at - out0] = make_uint2(uint32_t(s[k]), __float_as_uint(v[k]));
          } else {
            slot_o[at] = s[k];
            w_o[at] = v[k];
          }
        }
        if (fr && in && !keep) {
          const int f = i - int(at);
          if (fits || (free0 + f >= 0 && free0 + f < p.free_capacity))
            fr[f] = s[k];
          else if (p.status)
            atomicOr(p.status, VA_STATUS_BAD_DST);
        }
      }
    }
    if (p.hold) {
      sm100::cluster_sync();   // the window has been read
      const uint32_t n = cta_stay + eq_kept(equal + cta_eq_at + cta_eq) - eq_kept(equal + cta_eq_at);
      for (uint32_t k = tid; k < n; k += kEvictThreads) {
        slot_o[out0 + k] = int32_t(held[k].x);
        w_o[out0 + k] = __uint_as_float(held[k].y);
      }
    }
    equal += all_eq;
    kept = k0 + all_stay + eq_kept(equal);
    w0 = w1;
    __syncthreads();   // count and held are read
  }
  sm100::cluster_sync();   // no CTA leaves while another reads its shared memory
  // (in place: the old length has been read by the whole cluster)
  if (!p.finish && rank == 0 && tid == 0) p.prefix_out[b] = L - nfreed;
}

// The new lengths and the free list's head, where they replace the old ones
// that every request's CTAs read first.
__global__ void __launch_bounds__(kEvictThreads) evict_finish_kernel(const EvictParams p) {
  __shared__ int64_t red[kWarps];
  griddep_wait();
  griddep_launch_dependents();
  int64_t mine = 0;
  for (int b = threadIdx.x; b < p.B; b += kEvictThreads) {
    int64_t base;
    bool bad = false;
    const int L = evict_list(p, b, &base, &bad);
    p.prefix_out[b] = L < p.budget ? L : p.budget;
    mine += L > p.budget ? L - p.budget : 0;
  }
  const int64_t total = block_sum(mine, red);
  if (threadIdx.x == 0) {
    const int64_t head = int64_t(*p.free_head) - total;
    *p.head_out = int32_t(head < 0 ? 0 : head);
  }
}

bool aligned4(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 3u) == 0; }

}  // namespace

cudaError_t init_evict() {
  return cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              int(sizeof(EvictSmem) + kHeldBytes));
}

}  // namespace va

VA_API int va_kv_evict(const int32_t* slot_idx, const int32_t* kv_indptr,
                       const int32_t* prefix_len, const float* weights, int64_t num_entries, int B,
                       int budget, int sinks, int recent, int32_t* free_slots,
                       int64_t free_capacity, const int32_t* free_head, int32_t* slot_idx_out,
                       int32_t* prefix_len_out, float* weights_out, int32_t* free_head_out,
                       uint32_t* status, va_stream_t stream) {
  using namespace va;
  if (!kv_indptr || !prefix_len || !prefix_len_out) return VA_ERR_NULL;
  // (empty lists have no address)
  if (num_entries != 0 && (!slot_idx || !weights || !slot_idx_out || !weights_out))
    return VA_ERR_NULL;
  if (free_slots && (!free_head || !free_head_out)) return VA_ERR_NULL;
  if (B < 1 || B > 65535 || num_entries < 0 || num_entries > kEntriesMax || budget < 0 ||
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
  // A length or head that is rewritten while other requests' CTAs still read
  // it for their place in the free list is left to a second kernel.
  p.finish = free_slots && (prefix_len_out == prefix_len || free_head_out == free_head);
  // As many CTAs per request as the batch leaves room for at once, and no more
  // than its average list has steps for (64 lists of 20k to 200k entries: four
  // CTAs each 76 us; two 94; eight, in two waves, 140).
  int ctas = 1;
  while (ctas < 8 && int64_t(2 * ctas) * B <= kCtaBudget * di.num_sms &&
         num_entries / B > int64_t(ctas) * kPer * kEvictThreads)
    ctas *= 2;
  p.ctas = ctas;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(ctas);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(unsigned(B) * unsigned(ctas), 1, 1);
  cfg.blockDim = dim3(kEvictThreads, 1, 1);
  p.hold = slot_idx_out == slot_idx || weights_out == weights;
  cfg.dynamicSmemBytes = sizeof(EvictSmem) + (p.hold ? kHeldBytes : 0);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, evict_kernel, p) != cudaSuccess) return VA_ERR_LAUNCH;
  if (!p.finish) return VA_OK;
  cfg.gridDim = dim3(1, 1, 1);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_finish_kernel, p) == cudaSuccess ? VA_OK : VA_ERR_LAUNCH;
}
