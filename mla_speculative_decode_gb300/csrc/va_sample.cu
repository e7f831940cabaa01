// va_sample.cu -- tokens drawn from rows of logits, and acceptance of a draft tree by
// sampling.
//
// A row l_i, i < V, with m = max l and w_i = exp((l_i - m) / T), is cut to the k largest
// logits, of those to the shortest run, largest first, that holds top_p of their mass, and
// to w_i >= min_p.  Equal logits rank by index.  What is kept is therefore every logit above
// a value, and the first few of those equal to it: (above, ties).  The token is the first in
// index order at which the kept mass so far exceeds uniform * (kept mass).
//
// Masses are whole numbers, w_i in units of 2^-43 (a row has 2^20 logits at most), so that
// sums do not depend on their order.  w_i itself has 32-bit accuracy: the exponent's factor
// log2(e) / T comes in two parts, so that its rounding does not tilt the distribution.
//
// One cluster of CTAs per row.  Each CTA reads its part of the row once, into shared
// memory, and takes the maximum; then, by row:
//   - with top-k or top-p, a histogram of counts and masses over -log2 w in steps of 1/64
//     octave, added over the cluster; the step in which the border lies; the values in that
//     step, gathered by every CTA, cut again by 512, and the few left taken largest first.
//     (Where too many values share a step, the border is found digit by digit of the
//     ordered values instead.)
//   - the kept mass of each warp's piece of the row, and, in the CTA where the drawn mass
//     falls, the token.
#include <cuda_fp16.h>
#include <math.h>
#include <string.h>

#include "va_accept.cuh"
#include "va_common.cuh"
#include "va_sm100.cuh"

#ifndef VA_API
#define VA_API extern "C" __attribute__((visibility("default")))
#endif

namespace va {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCtasMax = 8;               // of a cluster
constexpr int kBins = 2048;               // of the histogram: 32 octaves
constexpr int kPer = kBins / kThreads;    // bins of a thread
constexpr int kSub = 512;                 // parts of a bin
constexpr int kList = 2048;               // values of one bin, of a whole row
constexpr int kRounds = 8;                // values taken out of a part of a bin
constexpr float kBinsPerOctave = 64.f;
constexpr int kUnit = 43;                 // masses count 2^-43
constexpr float kNothing = -46.f;         // a height whose mass is 0
static_assert(kSub == kThreads, "a part of a bin per thread");

struct SampleParams {
  const void* root;      // rows of the prefix (trees), or NULL
  const void* logits;
  int64_t stride;        // elements between rows of logits
  int64_t V;
  int group;             // rows that share their settings (tree: T + 1)
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* uniform;
  int32_t* tokens;
  float* logprob;        // or NULL
  uint32_t* status;      // or NULL
  bool clear_status;
  int ctas;              // of a row
  bool staged;           // the row's parts fit shared memory
};

struct alignas(16) SampleSmem {
  uint32_t cnt[kBins];   // values of a bin
  uint32_t lo[kBins];    // their masses, in 2^-(23 + octave): low 12 bits summed,
  uint32_t hi[kBins];    // and the rest
  float list[kList];     // this CTA's values of the border's bin
  float merged[kList];   // the row's
  uint32_t nlist;
  float min_above;       // min-p keeps what is above
  // what the cluster's CTAs tell each other
  float x_max[kCtasMax];
  uint32_t x_total[kCtasMax][2];
  uint32_t x_mass[kCtasMax][2];
  uint32_t x_eq[kCtasMax];
  uint32_t x_first[kCtasMax];
  // within the CTA
  float w_max[kWarps];
  uint64_t w_mass[kWarps];
  uint32_t w_eq[kWarps];
  uint64_t s_mass[kWarps];
  uint32_t s_cnt[kWarps];
  // results of a search
  uint32_t f_bin, f_cnt, f_in;
  uint64_t f_mass;
};

// ------------------------------------------------------------- small pieces

__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld_cluster_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

template <typename T>
__device__ __forceinline__ void unpack(const uint4& r, float (&x)[16 / sizeof(T)]);
template <>
__device__ __forceinline__ void unpack<float>(const uint4& r, float (&x)[4]) {
  x[0] = __uint_as_float(r.x); x[1] = __uint_as_float(r.y);
  x[2] = __uint_as_float(r.z); x[3] = __uint_as_float(r.w);
}
template <>
__device__ __forceinline__ void unpack<__nv_bfloat16>(const uint4& r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void unpack<__half>(const uint4& r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __half2float(__ushort_as_half(uint16_t(w[i] & 0xffffu)));
    x[2 * i + 1] = __half2float(__ushort_as_half(uint16_t(w[i] >> 16)));
  }
}
template <typename T>
__device__ __forceinline__ T minus_inf();
template <>
__device__ __forceinline__ float minus_inf<float>() { return -INFINITY; }
template <>
__device__ __forceinline__ __nv_bfloat16 minus_inf<__nv_bfloat16>() {
  return __ushort_as_bfloat16(0xff80u);
}
template <>
__device__ __forceinline__ __half minus_inf<__half>() { return __ushort_as_half(0xfc00u); }

// A value as an unsigned integer of the opposite order (the largest first), and back.
__device__ __forceinline__ uint32_t down_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);   // -0 and +0 are equal
  return ~(u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u));
}
__device__ __forceinline__ float down_value(uint32_t key) {
  const uint32_t k = ~key;
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// What a row's weights are made of.
struct Scale {
  float m, c_hi, c_lo;
  // -h is the distance from the maximum in octaves: it falls with the value, and never rises
  __device__ __forceinline__ float height(float l) const { return (l == m ? 0.f : l - m) * c_hi; }
  __device__ __forceinline__ float weight(float l) const {
    const float x = l == m ? 0.f : l - m, h = x * c_hi;
    return h > kNothing ? sm100::ex2_approx(fmaf(x, c_lo, h)) : 0.f;
  }
  __device__ __forceinline__ int bin(float h) const {
    return int(fminf(h * -kBinsPerOctave, float(kBins - 1)));
  }
};

// A weight, or a sum of a few, in units of 2^-43.
__device__ __forceinline__ uint64_t mass_of(float e) {
  const uint32_t b = __float_as_uint(e);
  const int up = int(b >> 23) - 150 + kUnit;   // of the 24-bit mantissa
  const uint64_t f = uint64_t((b & 0x7fffffu) | 0x800000u);
  if (up >= 0) return f << up;
  return up < -32 ? 0 : (f + (uint64_t(1) << (-up - 1))) >> -up;
}
// The same in units of 2^-(23 + octave), for a weight of that octave (or less).
__device__ __forceinline__ uint32_t octave_mass(float e, int octave) {
  const uint32_t b = __float_as_uint(e);
  const float v = b < 0x00800000u ? 0.f : __uint_as_float(b + (uint32_t(octave) << 23));
  return __float_as_uint(fminf(v, 1.f) + 1.f) - 0x3f800000u;
}
__device__ __forceinline__ uint64_t from_octave(uint64_t mass, int octave) {
  const int down = octave - (kUnit - 23);
  return down <= 0 ? mass << -down : mass >> down;
}
// ... and back, rounded up (a part of a sum stays a part of it).
__device__ __forceinline__ uint64_t to_octave(uint64_t mass, int octave) {
  const int up = octave - (kUnit - 23);
  return up >= 0 ? mass << up : (mass + (uint64_t(1) << -up) - 1) >> -up;
}

// The least whole number not below p * mass, 0 < p < 1.
__device__ __forceinline__ uint64_t part_of(float p, uint64_t mass) {
  const uint64_t q = __float2ull_rz(p * 0x1p63f);
  const uint64_t hi = __umul64hi(q, mass), lo = q * mass;
  return ((hi << 1) | (lo >> 63)) + ((lo << 1) != 0 ? 1 : 0);
}

// What is kept of a row: values above `above`, and the first `ties` equal to it.
struct Cut {
  float above;
  uint32_t ties;
};

// This CTA's part of a row, vectors of 16 bytes [v0, v1) counted from the 16-byte boundary
// at or before the row's first element.
template <typename T>
struct Part {
  static constexpr int kE = 16 / int(sizeof(T));
  const T* row;       // element 0
  const uint4* mem;   // vector v0, in shared memory (NULL: not staged)
  int64_t V;
  int skew;           // elements between the boundary and the row
  int v0, v1;
  __device__ __forceinline__ uint4 from_global(int v) const {
    const int64_t i0 = int64_t(v) * kE - skew;
    if (i0 >= 0 && i0 + kE <= V) return *reinterpret_cast<const uint4*>(row + i0);
    union { T e[kE]; uint4 q; } u;
#pragma unroll
    for (int j = 0; j < kE; ++j) u.e[j] = i0 + j >= 0 && i0 + j < V ? row[i0 + j] : minus_inf<T>();
    return u.q;
  }
  // NaN counts as -inf
  __device__ __forceinline__ void load(int v, float (&x)[kE]) const {
    unpack<T>(mem ? mem[v - v0] : from_global(v), x);
#pragma unroll
    for (int j = 0; j < kE; ++j) x[j] = fmaxf(x[j], -INFINITY);
  }
  // a warp's piece, in index order
  __device__ __forceinline__ void piece(int warp, int* p0, int* p1) const {
    const int n = (v1 - v0 + kWarps - 1) / kWarps;
    *p0 = v0 + warp * n < v1 ? v0 + warp * n : v1;
    *p1 = *p0 + n < v1 ? *p0 + n : v1;
  }
  template <typename F>
  __device__ __forceinline__ void each(F&& use) const {
    for (int v = v0 + int(threadIdx.x); v < v1; v += kThreads) {
      float x[kE];
      load(v, x);
#pragma unroll
      for (int j = 0; j < kE; ++j) use(x[j]);
    }
  }
};

// Exclusive sums over the block of a count and a mass, in thread order.
__device__ __forceinline__ void block_scan(SampleSmem& sm, uint32_t& cnt, uint64_t& mass) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t c0 = cnt;
  const uint64_t m0 = mass;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t c = __shfl_up_sync(0xffffffffu, cnt, o);
    const uint64_t m = __shfl_up_sync(0xffffffffu, mass, o);
    if (lane >= o) { cnt += c; mass += m; }
  }
  if (lane == 31) {
    sm.s_cnt[warp] = cnt;
    sm.s_mass[warp] = mass;
  }
  __syncthreads();
  cnt -= c0;
  mass -= m0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w)
    if (w < warp) { cnt += sm.s_cnt[w]; mass += sm.s_mass[w]; }
  __syncthreads();
}

__device__ __forceinline__ float block_max(SampleSmem& sm, float v) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (lane == 0) sm.w_max[warp] = v;
  __syncthreads();
  v = sm.w_max[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) v = fmaxf(v, sm.w_max[w]);
  __syncthreads();
  return v;
}

// ------------------------------------------------------------ border search

// The histogram's bins of this thread, added over the cluster; masses in 2^-43.
struct Bins {
  uint32_t cnt[kPer];
  uint64_t mass[kPer];
};

__device__ __forceinline__ void gather_bins(SampleSmem& sm, int ctas, Bins& b) {
  const int t = int(threadIdx.x) * kPer;
  uint64_t low[kPer], high[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) { b.cnt[k] = 0; low[k] = high[k] = 0; }
  static_assert(kPer == 4, "a 16-byte read per array");
  for (int c = 0; c < ctas; ++c) {
    const uint4 n = ld_cluster_v4(sm100::mapa(smem_u32(sm.cnt + t), uint32_t(c)));
    const uint4 l = ld_cluster_v4(sm100::mapa(smem_u32(sm.lo + t), uint32_t(c)));
    const uint4 h = ld_cluster_v4(sm100::mapa(smem_u32(sm.hi + t), uint32_t(c)));
    b.cnt[0] += n.x; b.cnt[1] += n.y; b.cnt[2] += n.z; b.cnt[3] += n.w;
    low[0] += l.x; low[1] += l.y; low[2] += l.z; low[3] += l.w;
    high[0] += h.x; high[1] += h.y; high[2] += h.z; high[3] += h.w;
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k)
    b.mass[k] = from_octave(low[k] + (high[k] << 12), (t + k) >> 6);
}

struct Found {
  int bin;         // kBins: none
  uint32_t cnt;    // above it
  uint64_t mass;
  uint32_t in;     // values in it
};

// The first bin at which the count, or the mass, from the top reaches `want` (>= 1).
__device__ __forceinline__ Found find_bin(SampleSmem& sm, const Bins& b, bool by_mass, uint64_t want) {
  if (threadIdx.x == 0) sm.f_bin = kBins;
  uint32_t cnt = 0;
  uint64_t mass = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) { cnt += b.cnt[k]; mass += b.mass[k]; }
  const uint32_t c1 = cnt;
  const uint64_t m1 = mass;
  block_scan(sm, cnt, mass);
  const uint64_t before = by_mass ? mass : cnt, mine = by_mass ? m1 : c1;
  if (before < want && want <= before + mine) {
    bool found = false;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (!found && (by_mass ? mass + b.mass[k] : uint64_t(cnt + b.cnt[k])) >= want) {
        found = true;
        sm.f_bin = uint32_t(int(threadIdx.x) * kPer + k);
        sm.f_cnt = cnt;
        sm.f_mass = mass;
        sm.f_in = b.cnt[k];
      }
      if (!found) { cnt += b.cnt[k]; mass += b.mass[k]; }
    }
  }
  __syncthreads();
  const Found f = {int(sm.f_bin), sm.f_cnt, sm.f_mass, sm.f_in};
  __syncthreads();
  return f;
}

// The row's values of one bin (weights from `least` on) in every CTA's `merged`, and their counts and masses over
// kSub parts of the bin in cnt, lo and hi.  The cluster has met since the histogram was read.
template <typename T>
__device__ __forceinline__ int gather_list(SampleSmem& sm, const Part<T>& part, const Scale& s, int ctas,
                                           int bin, float least) {
  const int tid = int(threadIdx.x);
  part.each([&](float l) {
    const float h = s.height(l);
    if (s.bin(h) == bin && s.weight(l) >= least) {
      const uint32_t at = atomicAdd(&sm.nlist, 1u);
      if (at < kList) sm.list[at] = l;
    }
  });
  sm100::cluster_sync();
  sm.cnt[tid] = sm.lo[tid] = sm.hi[tid] = 0;
  __syncthreads();
  int n = 0;
  const int octave = bin >> 6;
  for (int c = 0; c < ctas; ++c) {
    const int nc = min(int(ld_cluster(sm100::mapa(smem_u32(&sm.nlist), uint32_t(c)))), kList);
    const uint32_t from = sm100::mapa(smem_u32(sm.list), uint32_t(c));
    for (int i = tid; i < nc && n + i < kList; i += kThreads) {
      const float l = __uint_as_float(ld_cluster(from + 4u * uint32_t(i)));
      sm.merged[n + i] = l;
      const float h = s.height(l);
      const int sub = int(h * (-kBinsPerOctave * kSub)) & (kSub - 1);
      const uint32_t w = octave_mass(s.weight(l), octave);
      atomicAdd(&sm.cnt[sub], 1u);
      atomicAdd(&sm.lo[sub], w & 0xfffu);
      atomicAdd(&sm.hi[sub], w >> 12);
    }
    n += nc;
  }
  __syncthreads();
  return min(n, kList);
}

// The border among the values of one bin (gather_list has run): `want` of their count, or of
// their mass (in the octave's unit), from the top.  False if the values in the border's part
// are too many different ones.  *mass: what of the bin is kept, in the octave's unit.
__device__ __forceinline__ bool border_in_list(SampleSmem& sm, const Scale& s, int n, int bin, bool by_mass,
                                               uint64_t want, Cut* cut, uint64_t* mass_out) {
  const int tid = int(threadIdx.x), octave = bin >> 6;
  if (tid == 0) sm.f_bin = kSub;
  uint32_t cnt = sm.cnt[tid];
  uint64_t mass = uint64_t(sm.lo[tid]) + (uint64_t(sm.hi[tid]) << 12);
  const uint32_t c1 = cnt;
  const uint64_t m1 = mass;
  block_scan(sm, cnt, mass);
  const uint64_t before = by_mass ? mass : cnt, mine = by_mass ? m1 : c1;
  if (before < want && want <= before + mine) {
    sm.f_bin = uint32_t(tid);
    sm.f_cnt = cnt;
    sm.f_mass = mass;
  }
  __syncthreads();
  const int sub = int(sm.f_bin);
  if (sub == kSub) return false;
  uint64_t left = want - (by_mass ? sm.f_mass : uint64_t(sm.f_cnt));
  mass = sm.f_mass;
  constexpr int kMine = kList / kThreads;
  float v[kMine];
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    const int i = tid + k * kThreads;
    v[k] = i < n ? sm.merged[i] : -INFINITY;
    if (i < n && (int(s.height(v[k]) * (-kBinsPerOctave * kSub)) & (kSub - 1)) != sub)
      v[k] = -INFINITY;
  }
  for (int round = 0; round < kRounds; ++round) {
    float top = v[0];
#pragma unroll
    for (int k = 1; k < kMine; ++k) top = fmaxf(top, v[k]);
    top = block_max(sm, top);
    if (top == -INFINITY) return false;   // (-inf itself is the last bin's)
    uint32_t eq = 0;
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const uint32_t n_eq = __popc(__ballot_sync(0xffffffffu, v[k] == top));
      eq += n_eq;
      if (v[k] == top) v[k] = -INFINITY;
    }
    if ((tid & 31) == 0) sm.w_eq[tid >> 5] = eq;
    __syncthreads();
    eq = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) eq += sm.w_eq[w];
    __syncthreads();
    const uint32_t w = octave_mass(s.weight(top), octave);
    const uint64_t all = by_mass ? uint64_t(eq) * w : uint64_t(eq);
    if (left <= all) {
      const uint64_t ties = by_mass ? (left + w - 1) / w : left;
      cut->above = top;
      cut->ties = uint32_t(ties);
      *mass_out = mass + ties * w;
      return true;
    }
    left -= all;
    mass += uint64_t(eq) * w;
  }
  return false;
}

// The border over the whole row, digit by digit (11, 11, 10 bits) of the ordered values:
// for rows with thousands of values in one bin.  *mass: what is kept, in 2^-43.
template <typename T>
__device__ void border_by_digits(SampleSmem& sm, const Part<T>& part, const Scale& s, int ctas,
                                 bool by_mass, uint64_t want, Cut* cut, uint64_t* mass_out) {
  const int tid = int(threadIdx.x);
  unsigned long long* sums = reinterpret_cast<unsigned long long*>(sm.lo);   // lo and hi
  uint32_t prefix = 0;
  uint64_t left = want, mass = 0;
  Bins b;
  for (int level = 0; level < 3; ++level) {
    const int shift = level == 0 ? 21 : (level == 1 ? 10 : 0);
    const uint32_t mask = level < 2 ? 2047u : 1023u;
    const int above = level == 0 ? 32 : (level == 1 ? 21 : 10);
    sm100::cluster_sync();   // the histogram has been read
    for (int i = tid; i < kBins; i += kThreads) { sm.cnt[i] = 0; sums[i] = 0; }
    __syncthreads();
    part.each([&](float l) {
      const uint32_t key = down_key(l);
      if (s.height(l) > kNothing && (above == 32 || (key >> above) == prefix)) {
        const uint32_t d = (key >> shift) & mask;
        atomicAdd(&sm.cnt[d], 1u);
        const uint64_t w = mass_of(s.weight(l));
        if (w) atomicAdd(&sums[d], (unsigned long long)w);
      }
    });
    sm100::cluster_sync();
    const int t = tid * kPer;
#pragma unroll
    for (int k = 0; k < kPer; ++k) { b.cnt[k] = 0; b.mass[k] = 0; }
    for (int c = 0; c < ctas; ++c) {
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        b.cnt[k] += ld_cluster(sm100::mapa(smem_u32(sm.cnt + t + k), uint32_t(c)));
        const uint32_t a = sm100::mapa(smem_u32(sums + t + k), uint32_t(c));
        b.mass[k] += uint64_t(ld_cluster(a)) | (uint64_t(ld_cluster(a + 4)) << 32);
      }
    }
    const Found f = find_bin(sm, b, by_mass, left);
    if (f.bin == kBins) {   // (a rounding of the total: all of it is kept)
      cut->above = -INFINITY;
      cut->ties = 0;
      return;
    }
    prefix = (prefix << (level == 0 ? 0 : (level == 1 ? 11 : 10))) | uint32_t(f.bin);
    left -= by_mass ? f.mass : uint64_t(f.cnt);
    mass += f.mass;
  }
  cut->above = down_value(prefix);
  const uint64_t w = mass_of(s.weight(cut->above));
  cut->ties = by_mass ? uint32_t((left + (w ? w : 1) - 1) / (w ? w : 1)) : uint32_t(left);
  *mass_out = mass + cut->ties * w;
}

// ------------------------------------------------------------------ kernel

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SampleSmem& sm = *reinterpret_cast<SampleSmem*>(smem_raw);
  constexpr int kE = Part<T>::kE;
  const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int ctas = p.ctas, rank = int(sm100::cluster_ctarank());
  const int r = int(blockIdx.x) / ctas, g = r / p.group, at = r - g * p.group;
  sm100::cluster_arrive_relaxed();   // (every CTA of the cluster runs before any writes to it)
  for (int i = tid; i < kBins; i += kThreads) sm.cnt[i] = sm.lo[i] = sm.hi[i] = 0;
  if (tid == 0) sm.nlist = 0;
  griddep_wait();                // the stream's previous kernel has completed
  griddep_launch_dependents();   // the next kernel may start its set-up
  if (p.clear_status && blockIdx.x == 0 && tid == 0) *p.status = 0u;

  const float temp = p.temperature ? p.temperature[g] : 1.f;
  const int top_k = p.top_k ? p.top_k[g] : 0;
  const float top_p = p.top_p ? p.top_p[g] : 1.f;
  const float min_p = p.min_p ? p.min_p[g] : 0.f;
  const bool greedy = !(temp > 0.f);
  const bool use_k = !greedy && top_k > 0 && top_k < p.V;
  const bool use_p = !greedy && top_p < 1.f;
  Part<T> part;
  part.row = p.group == 1 ? static_cast<const T*>(p.logits) + int64_t(r) * p.stride
             : at == 0    ? static_cast<const T*>(p.root) + int64_t(g) * p.V
                          : static_cast<const T*>(p.logits) +
                                (int64_t(g) * (p.group - 1) + (at - 1)) * p.V;
  part.V = p.V;
  part.skew = int((reinterpret_cast<uintptr_t>(part.row) / sizeof(T)) % kE);
  const int nv = int((p.V + part.skew + kE - 1) / kE), per = (nv + ctas - 1) / ctas;
  part.v0 = rank * per < nv ? rank * per : nv;
  part.v1 = part.v0 + per < nv ? part.v0 + per : nv;
  part.mem = nullptr;

  // ---- the row's part into shared memory, and its maximum
  float top = -INFINITY;
  {
    uint4* stage = reinterpret_cast<uint4*>(smem_raw + sizeof(SampleSmem));
    constexpr int kBatch = 4;
    for (int v = part.v0 + tid; v < part.v1; v += kBatch * kThreads) {
      uint4 q[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (v + k * kThreads < part.v1) q[k] = part.from_global(v + k * kThreads);
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (v + k * kThreads < part.v1) {
          float x[kE];
          unpack<T>(q[k], x);
#pragma unroll
          for (int j = 0; j < kE; ++j) top = fmaxf(top, x[j]);
          if (p.staged) stage[v + k * kThreads - part.v0] = q[k];
        }
    }
    if (p.staged) part.mem = stage;
  }
  top = block_max(sm, top);
  sm100::cluster_wait();
  if (tid < ctas) sm100::st_cluster_f32(sm100::mapa(smem_u32(&sm.x_max[rank]), uint32_t(tid)), top);
  sm100::cluster_sync();
  top = sm.x_max[0];
  for (int c = 1; c < ctas; ++c) top = fmaxf(top, sm.x_max[c]);

  Scale s;
  s.m = top;
  {   // log2(e) / T in two parts
    constexpr float kHi = 1.4426950216293335f, kLo = 1.925962989e-8f;
    const float t = fminf(fmaxf(temp, 0x1p-100f), 3.4e38f);
    s.c_hi = kHi / t;
    s.c_lo = (fmaf(-s.c_hi, t, kHi) + kLo) / t;
  }
  Cut cut = {-INFINITY, 0u};

  if (top == -INFINITY) {   // nothing to draw from (the whole cluster leaves)
    if (rank == 0 && tid == 0) {
      p.tokens[r] = 0;
      if (p.logprob) p.logprob[r] = -INFINITY;
      if (p.status && !p.clear_status) atomicOr(p.status, VA_STATUS_EMPTY_ROW);
    }
    return;
  }
  if (greedy) {   // the lowest index of the largest
    uint32_t first = 0xffffffffu;
    for (int v = part.v0 + tid; v < part.v1 && first == 0xffffffffu; v += kThreads) {
      float x[kE];
      part.load(v, x);
#pragma unroll
      for (int j = kE - 1; j >= 0; --j)
        if (x[j] == top) first = uint32_t(int64_t(v) * kE - part.skew + j);
    }
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) sm.w_eq[warp] = first;
    __syncthreads();
    if (tid == 0) {
      for (int w = 0; w < kWarps; ++w) first = min(first, sm.w_eq[w]);
      sm100::st_cluster_u32(sm100::mapa(smem_u32(&sm.x_first[rank]), 0u), first);
    }
    sm100::cluster_sync();
    if (rank == 0 && tid == 0) {
      for (int c = 0; c < ctas; ++c) first = min(first, sm.x_first[c]);
      p.tokens[r] = int32_t(first);
      if (p.logprob) p.logprob[r] = 0.f;
    }
    return;
  }

  if (use_k || use_p) {
    // ---- histogram of the heights.  Weights below (1 - top_p) / V cannot reach the
    // border (all of them together weigh less than what top_p drops of a total >= 1).
    const float dropped = use_p && !use_k ? (1.f - fmaxf(top_p, 0.f)) / float(p.V) * 0.999f : 0.f;
    uint64_t total = 0;
    for (int v = part.v0 + tid; v < part.v1; v += kThreads) {
      float x[kE], sum = 0.f;
      part.load(v, x);
#pragma unroll
      for (int j = 0; j < kE; ++j) {
        const float h = s.height(x[j]);
        if (!(h > kNothing)) continue;   // (top-k may count as many of these as it likes)
        const int bin = s.bin(h);
        if (use_p) {
          const float e = s.weight(x[j]);
          sum += e;
          if (e >= dropped) {
            const uint32_t w = octave_mass(e, bin >> 6);
            atomicAdd(&sm.lo[bin], w & 0xfffu);
            atomicAdd(&sm.hi[bin], w >> 12);
            atomicAdd(&sm.cnt[bin], 1u);
          }
        } else {
          atomicAdd(&sm.cnt[bin], 1u);
        }
      }
      total += mass_of(sum);
    }
    if (use_p && !use_k) {   // the row's mass
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
      if (lane == 0) sm.w_mass[warp] = total;
      __syncthreads();
      if (tid < ctas) {
        total = 0;
        for (int w = 0; w < kWarps; ++w) total += sm.w_mass[w];
        const uint32_t a = sm100::mapa(smem_u32(&sm.x_total[rank][0]), uint32_t(tid));
        sm100::st_cluster_u32(a, uint32_t(total));
        sm100::st_cluster_u32(a + 4, uint32_t(total >> 32));
      }
    }
    sm100::cluster_sync();
    Bins bins;
    gather_bins(sm, ctas, bins);
    int listed = -1, n = 0;   // bin whose values are in `merged`
    uint64_t kept = 0;
    bool done_p = !use_p;
    if (use_k) {
      const Found f = find_bin(sm, bins, false, uint64_t(top_k));
      const int bin = f.bin;
      uint64_t in_bin = 0;
      bool ok = bin < kBins - 1 && f.in <= kList;
      if (bin == kBins) {   // fewer than k have a mass: all of them stay
        ok = true;
        uint32_t n_all = 0;
        kept = 0;
#pragma unroll
        for (int k = 0; k < kPer; ++k) kept += bins.mass[k];
        const uint64_t mine = kept;
        block_scan(sm, n_all, kept);
        kept += mine;   // (the last thread's is the total)
        if (tid == kThreads - 1) sm.f_mass = kept;
        __syncthreads();
        kept = sm.f_mass;
        __syncthreads();
      } else if (ok) {
        n = gather_list(sm, part, s, ctas, bin, dropped);
        listed = bin;
        ok = border_in_list(sm, s, n, bin, false, uint64_t(top_k) - f.cnt, &cut, &in_bin);
        kept = f.mass + from_octave(in_bin, bin >> 6);
      }
      if (!ok) {
        listed = -1;
        border_by_digits(sm, part, s, ctas, false, uint64_t(top_k), &cut, &kept);
        if (use_p) {
          Cut c2 = {-INFINITY, 0u};
          uint64_t m2;
          const uint64_t want_p = top_p > 0.f ? part_of(top_p, kept) : 1u;
          border_by_digits(sm, part, s, ctas, true, want_p > 0 ? want_p : 1u, &c2, &m2);
          if (c2.above > cut.above || (c2.above == cut.above && c2.ties < cut.ties)) cut = c2;
          done_p = true;
        }
      }
    } else {
      kept = 0;
      for (int c = 0; c < ctas; ++c)
        kept += uint64_t(sm.x_total[c][0]) | (uint64_t(sm.x_total[c][1]) << 32);
    }
    if (!done_p) {
      uint64_t want = top_p > 0.f ? part_of(top_p, kept) : 1u;
      want = want > 0 ? want : 1u;
      const Found f = find_bin(sm, bins, true, want);
      const int bin = f.bin;
      if (bin < kBins) {   // (else, by a rounding of the total, all of it stays)
        const uint64_t inside = to_octave(want - f.mass, bin >> 6);
        Cut c2 = {-INFINITY, 0u};
        uint64_t m2;
        bool ok = bin < kBins - 1 && f.in <= kList;
        if (ok) {
          if (bin != listed) {
            if (listed >= 0) {   // the first list has been read by the whole cluster
              sm100::cluster_sync();
              if (tid == 0) sm.nlist = 0;
              __syncthreads();
            }
            n = gather_list(sm, part, s, ctas, bin, dropped);
          }
          ok = border_in_list(sm, s, n, bin, true, inside > 0 ? inside : 1u, &c2, &m2);
        }
        if (!ok) border_by_digits(sm, part, s, ctas, true, want, &c2, &m2);
        if (c2.above > cut.above || (c2.above == cut.above && c2.ties < cut.ties)) cut = c2;
      }
    }
  }
  if (min_p > 0.f) {   // the largest value below m + T ln(min_p)
    if (tid == 0) {    // (64 bits are slow: one thread)
      const double gap = double(temp) * log(double(min_p));
      const double t = double(top) + fmin(gap, 0.0);
      const float f = __double2float_rd(t);
      sm.min_above = double(f) == t ? nextafterf(f, -INFINITY) : f;
    }
    __syncthreads();
    const float f = sm.min_above;
    if (f >= cut.above) cut = {f, 0u};
  }

  // ---- kept masses, piece by piece in index order
  const uint64_t tie_mass = cut.ties ? mass_of(s.weight(cut.above)) : 0;
  int p0, p1;
  part.piece(warp, &p0, &p1);
  uint64_t mass = 0;
  uint32_t eq = 0;
  for (int v = p0 + lane; v < p1; v += 32) {
    float x[kE], sum = 0.f;
    part.load(v, x);
    bool any = false;
#pragma unroll
    for (int j = 0; j < kE; ++j) {
      any |= x[j] > cut.above;
      eq += x[j] == cut.above ? 1u : 0u;
    }
    if (any) {
#pragma unroll
      for (int j = 0; j < kE; ++j) sum += x[j] > cut.above ? s.weight(x[j]) : 0.f;
      mass += mass_of(sum);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mass += __shfl_xor_sync(0xffffffffu, mass, o);
    eq += __shfl_xor_sync(0xffffffffu, eq, o);
  }
  if (lane == 0) {
    sm.w_mass[warp] = mass;
    sm.w_eq[warp] = eq;
  }
  __syncthreads();
  if (tid < ctas) {
    uint64_t m = 0;
    uint32_t e = 0;
    for (int w = 0; w < kWarps; ++w) { m += sm.w_mass[w]; e += sm.w_eq[w]; }
    const uint32_t a = sm100::mapa(smem_u32(&sm.x_mass[rank][0]), uint32_t(tid));
    sm100::st_cluster_u32(a, uint32_t(m));
    sm100::st_cluster_u32(a + 4, uint32_t(m >> 32));
    sm100::st_cluster_u32(sm100::mapa(smem_u32(&sm.x_eq[rank]), uint32_t(tid)), e);
  }
  sm100::cluster_sync();   // (the last time that a CTA touches another's memory is before it)

  // ---- where the drawn mass falls
  auto tied = [&](uint32_t e) { return uint64_t(e < cut.ties ? e : cut.ties) * tie_mass; };
  uint64_t all = 0, before = 0;
  uint32_t all_eq = 0, eq_before = 0;
  for (int c = 0; c < ctas; ++c) {
    if (c == rank) { before = all; eq_before = all_eq; }
    all += uint64_t(sm.x_mass[c][0]) | (uint64_t(sm.x_mass[c][1]) << 32);
    all_eq += sm.x_eq[c];
  }
  const uint64_t total = all + tied(all_eq);
  const float u = p.uniform[r];
  const uint64_t u64 = u >= 1.f ? ~uint64_t(0) : (u > 0.f ? __float2ull_rz(u * 0x1p64f) : 0);
  const uint64_t drawn = __umul64hi(u64, total);   // < total: the token is the first past it
  for (int w = 0; w < warp; ++w) { before += sm.w_mass[w]; eq_before += sm.w_eq[w]; }
  if (drawn < before + tied(eq_before) ||
      drawn >= before + sm.w_mass[warp] + tied(eq_before + sm.w_eq[warp]))
    return;
  for (int vb = p0; vb < p1; vb += 32) {   // this warp's piece holds it
    const int v = vb + lane;
    float x[kE];
    uint32_t my_eq = 0;
    float sum = 0.f;
    if (v < p1) {
      part.load(v, x);
#pragma unroll
      for (int j = 0; j < kE; ++j) {
        sum += x[j] > cut.above ? s.weight(x[j]) : 0.f;
        my_eq += x[j] == cut.above ? 1u : 0u;
      }
    }
    const uint64_t mine = sum > 0.f ? mass_of(sum) : 0;
    uint64_t m = mine;
    uint32_t e = my_eq;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t m1 = __shfl_up_sync(0xffffffffu, m, o);
      const uint32_t e1 = __shfl_up_sync(0xffffffffu, e, o);
      if (lane >= o) { m += m1; e += e1; }
    }
    const uint64_t m_at = before + m - mine;
    uint32_t e_at = eq_before + e - my_eq;
    const bool here = drawn >= m_at + tied(e_at) && drawn < m_at + mine + tied(e_at + my_eq);
    if (__any_sync(0xffffffffu, here)) {
      if (here) {
        int pick = 0;
        bool found = false;
        float run = 0.f;
#pragma unroll
        for (int j = 0; j < kE; ++j) {
          const bool a = x[j] > cut.above, b = x[j] == cut.above && e_at < cut.ties;
          if (a) run += s.weight(x[j]);
          if (x[j] == cut.above) ++e_at;
          if ((a || b) && !found) {
            pick = j;   // (the last kept one, should a rounding leave none)
            found = drawn < m_at + (run > 0.f ? mass_of(run) : 0) + tied(e_at);
          }
        }
        float l = x[0];
#pragma unroll
        for (int j = 1; j < kE; ++j) l = pick == j ? x[j] : l;
        p.tokens[r] = int32_t(int64_t(v) * kE - part.skew + pick);
        if (p.logprob) {
          // ln(w / total): near a total of 1 from what it exceeds 1 by
          const uint64_t one = uint64_t(1) << kUnit;
          const float ln = total < 2 * one && total >= one
                               ? log1pf(float(total - one) * 0x1p-43f)
                               : logf(float(total) * 0x1p-43f);
          const float t = fminf(fmaxf(temp, 0x1p-100f), 3.4e38f);
          p.logprob[r] = (l == top ? 0.f : (l - top) / t) - ln;
        }
      }
      return;
    }
    before += __shfl_sync(0xffffffffu, m, 31);
    eq_before += __shfl_sync(0xffffffffu, e, 31);
  }
}

// -------------------------------------------------------------------- host

constexpr size_t kStageMax = 190 * 1024 - sizeof(SampleSmem);   // staged bytes of a CTA at most
constexpr size_t kStageTwo = 112 * 1024 - sizeof(SampleSmem);   // with two CTAs on an SM
constexpr int64_t kRowsMax = int64_t(1) << 23;

bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int launch_sample(SampleParams& p, int dtype, int64_t rows, int num_sms, va_stream_t stream) {
  const size_t elem = dtype == VA_F32 ? 4 : 2;
  const int64_t vecs = (p.V * int64_t(elem) + 15) / 16 + 1;
  auto bytes = [&](int ctas) { return size_t((vecs + ctas - 1) / ctas) * 16; };
  // As many CTAs per row as leave two on an SM, and more while SMs are idle.
  int ctas = 1;
  while (ctas < kCtasMax &&
         (bytes(ctas) > kStageTwo || (rows * ctas * 2 <= 2 * num_sms && bytes(ctas) > 4096)))
    ctas *= 2;
  p.ctas = ctas;
  p.staged = bytes(ctas) <= kStageMax;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(ctas);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(unsigned(rows * ctas), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = sizeof(SampleSmem) + (p.staged ? bytes(ctas) : 0);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e;
  if (dtype == VA_F32)
    e = cudaLaunchKernelEx(&cfg, sample_kernel<float>, p);
  else if (dtype == VA_BF16)
    e = cudaLaunchKernelEx(&cfg, sample_kernel<__nv_bfloat16>, p);
  else
    e = cudaLaunchKernelEx(&cfg, sample_kernel<__half>, p);
  return e == cudaSuccess ? VA_OK : VA_ERR_LAUNCH;
}

struct TreeLayout {
  size_t tokens, logprob, total;
};
TreeLayout tree_layout(int B, int T) {
  const size_t rows = size_t(B) * (size_t(T) + 1);
  TreeLayout L;
  L.tokens = kHeaderBytes;
  L.logprob = L.tokens + align256(rows * sizeof(int32_t));
  L.total = L.logprob + align256(rows * sizeof(float));
  return L;
}

}  // namespace

cudaError_t init_sample() {
  const int smem = int(sizeof(SampleSmem) + kStageMax);
  cudaError_t e = cudaFuncSetAttribute(sample_kernel<float>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(sample_kernel<__nv_bfloat16>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(sample_kernel<__half>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem);
  return e;
}

}  // namespace va

VA_API int va_sample(const void* logits, int64_t row_stride, int dtype, int64_t rows, int64_t V,
                     const float* temperature, const int32_t* top_k, const float* top_p,
                     const float* min_p, const float* uniform, int32_t* tokens, float* logprob,
                     uint32_t* status, va_stream_t stream) {
  using namespace va;
  if (rows != 0 && (!logits || !uniform || !tokens)) return VA_ERR_NULL;
  if (rows < 0 || rows > kRowsMax || V < 1 || V > VA_SAMPLE_V_MAX || dtype < VA_F32 ||
      dtype > VA_F16 || row_stride < 0 || row_stride > (int64_t(1) << 40))
    return VA_ERR_SHAPE;
  const size_t elem = dtype == VA_F32 ? 4 : 2;
  if (!aligned_to(logits, elem) || !aligned_to(temperature, 4) || !aligned_to(top_k, 4) ||
      !aligned_to(top_p, 4) || !aligned_to(min_p, 4) || !aligned_to(uniform, 4) ||
      !aligned_to(tokens, 4) || !aligned_to(logprob, 4) || !aligned_to(status, 4))
    return VA_ERR_ALIGN;
  DeviceInfo di;
  const int rc = device_info(&di);
  if (rc != VA_OK || rows == 0) return rc;
  SampleParams p;
  memset(&p, 0, sizeof p);
  p.logits = logits;
  p.stride = row_stride;
  p.V = V;
  p.group = 1;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.uniform = uniform;
  p.tokens = tokens;
  p.logprob = logprob;
  p.status = status;
  return launch_sample(p, dtype, rows, di.num_sms, stream);
}

VA_API size_t va_tree_accept_sampled_workspace_bytes(int B, int T) {
  if (B < 1 || B > 65535 || T < 1 || T > VA_T_MAX) return 0;
  return va::tree_layout(B, T).total;
}

VA_API int va_tree_accept_sampled(const void* root_logits, const void* logits, int dtype, int64_t V,
                                  const int32_t* draft_tokens, const int32_t* tree_parent,
                                  const int32_t* draft_slots, int B, int T,
                                  const float* temperature, const int32_t* top_k,
                                  const float* top_p, const float* min_p, const float* uniform,
                                  void* workspace, size_t workspace_bytes, int32_t* accept_len,
                                  int32_t* accept_nodes, int32_t* accept_slots,
                                  int32_t* bonus_token, float* logprob, va_stream_t stream) {
  using namespace va;
  if (!root_logits || !logits || !draft_tokens || !tree_parent || !uniform || !workspace ||
      !accept_len || !accept_nodes || !bonus_token)
    return VA_ERR_NULL;
  if (B < 1 || B > 65535 || T < 1 || T > VA_T_MAX || V < 1 || V > VA_SAMPLE_V_MAX ||
      dtype < VA_F32 || dtype > VA_F16)
    return VA_ERR_SHAPE;
  const size_t elem = dtype == VA_F32 ? 4 : 2;
  if (!aligned_to(root_logits, elem) || !aligned_to(logits, elem) || !aligned_to(draft_tokens, 4) ||
      !aligned_to(tree_parent, 4) || !aligned_to(draft_slots, 4) || !aligned_to(temperature, 4) ||
      !aligned_to(top_k, 4) || !aligned_to(top_p, 4) || !aligned_to(min_p, 4) ||
      !aligned_to(uniform, 4) || !aligned_to(workspace, 256) || !aligned_to(accept_len, 4) ||
      !aligned_to(accept_nodes, 4) || !aligned_to(accept_slots, 4) ||
      !aligned_to(bonus_token, 4) || !aligned_to(logprob, 4))
    return VA_ERR_ALIGN;
  const TreeLayout L = tree_layout(B, T);
  if (workspace_bytes < L.total) return VA_ERR_WORKSPACE;
  DeviceInfo di;
  int rc = device_info(&di);
  if (rc != VA_OK) return rc;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  SampleParams p;
  memset(&p, 0, sizeof p);
  p.root = root_logits;
  p.logits = logits;
  p.stride = V;
  p.V = V;
  p.group = T + 1;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.uniform = uniform;
  p.tokens = reinterpret_cast<int32_t*>(w + L.tokens);
  p.logprob = logprob ? logprob : reinterpret_cast<float*>(w + L.logprob);
  p.status = reinterpret_cast<uint32_t*>(w);
  p.clear_status = true;
  rc = launch_sample(p, dtype, int64_t(B) * (T + 1), di.num_sms, stream);
  if (rc != VA_OK) return rc;
  // the walk reads each row's token as the one chunk of an argmax, and its logprob as the value
  AcceptParams a;
  memset(&a, 0, sizeof a);
  a.V = V;
  a.tokens = draft_tokens;
  a.parent = tree_parent;
  a.slots = draft_slots;
  a.B = B;
  a.T = T;
  a.chunks = 1;
  a.part_val = p.logprob;
  a.part_idx = p.tokens;
  a.flag_empty = true;
  a.status = p.status;
  a.accept_len = accept_len;
  a.accept_nodes = accept_nodes;
  a.accept_slots = accept_slots;
  a.bonus = bonus_token;
  return launch_accept_walk(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? VA_OK
                                                                                       : VA_ERR_LAUNCH;
}
