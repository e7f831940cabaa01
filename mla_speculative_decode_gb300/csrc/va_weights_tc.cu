// va_weights_tc.cu -- attention weight per key on the tcgen05 tensor cores.
//
// The sum over rows wants a key's scores in one thread: the product is turned
// round, S^T = K Q^T, with 128 keys per CTA as the rows of the accumulator (a
// tensor-memory lane, so a thread, per key) and query rows as its columns.  A
// thread then adds exp2(s * scale - lse) over the columns in registers; no
// reduction across threads is needed, and lse comes from shared memory by
// broadcast.
//
// Two shapes:
//   one-SM products (M = 128 keys, N = up to 64 query rows): decode batches.
//     Bound by HBM: every key row is read once.  The request's query rows stay
//     in shared memory (nine slots of 8 KB, one per 64-column block) while its
//     keys stream past, and N follows the rows there are.
//   two-SM products (clusters of 2, M = 256 keys, N = 256 query rows): chunks.
//     Bound by the tensor cores: a key tile stays in shared memory (nine slots
//     of 16 KB) while the request's query rows stream past it in blocks of 64
//     columns through four slots; each CTA brings half of a block, so that an SM
//     reads 32 bytes per cycle for its products.
// Keys arrive by 16-byte cp.async gathers, in three groups of three column
// blocks with barriers of their own, so that the next key tile's first group
// loads as soon as the products of this one's first group are done.  Queries
// arrive by TMA boxes.
//
// Work: with a key tile and a tile of query rows that sees some of it as one
// step, the batch is one long row of steps (request, key tile, row tile).  Each
// cluster takes an equal run of it, whatever the lengths.  A run that begins
// inside a key tile's row tiles leaves that tile's share in a slot of its own,
// every other share goes to sums[entry]; weights_finish_kernel adds them in a
// fixed order.
//
// Measured: 8 requests of one token, 64 heads, 1k to 65k paged keys (282 MB):
// 68 us, the kernel 58 of them at 4.9 TB/s (a bare gather of such rows: 5.6).  256
// tokens, 64 heads, 16k keys in front: 229 us, 70% of the cuBLAS rate; the tensor
// pipe is active 57% of a launch.  What the rest is has not been taken apart: the
// waits between steps, the exponentials of a tile's last columns, and the query rows,
// which at the pipe's full rate would take 9.7 TB/s from L2.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <string.h>

#include "va_sm100.cuh"
#include "va_weights.cuh"

#ifdef VA_TEST_HOOKS
// Test build only: the gate of va_tc.cu, for the producer warps of this kernel.
__device__ const int32_t* g_va_weights_gate = nullptr;
#endif

namespace va {

extern PFN_cuTensorMapEncodeTiled_v12000 g_encode;   // va_tc.cu, resolved by va_init

#ifdef VA_TEST_HOOKS
cudaError_t set_weights_gate(const int32_t* flag) {
  return cudaMemcpyToSymbol(g_va_weights_gate, &flag, sizeof(flag));
}
#endif

namespace {

using namespace sm100;

constexpr int kEpilogue = 256;         // warps 0-7: scores to sums
constexpr int kProducers = 256;        // warps 8-15: keys
constexpr int kMmaWarp = 16;           // products
constexpr int kQueryWarp = 17;         // boxes of query rows
constexpr int kThreads = 576;
constexpr uint32_t kProducerBar = 1, kEpilogueBar = 2;   // named barriers
constexpr int kKeys = 128;             // keys per CTA and tile
constexpr int kBlocks = kDqk / 64;     // 9 column blocks
constexpr uint16_t kBoth = 0x3;        // cluster ranks of a pair
constexpr int kGroups = 3;             // of three column blocks
constexpr uint32_t kKSlot = kKeys * 128u;
constexpr long long kWaitCycles = 4000000000ll;   // wait bound in SM cycles (~2 s)
// After a wait gave up: time for the boxes in flight to land before the CTA leaves.
constexpr long long kDrainCycles = 2000000ll;

template <bool kPair>
struct WCfg {
  static constexpr int kCtas = kPair ? 2 : 1;
  static constexpr int kTileKeys = kCtas * kKeys;
  static constexpr int kTileRows = kPair ? 256 : 64;          // query rows of a step
  static constexpr int kCtaRows = kTileRows / kCtas;          // of which a CTA holds
  static constexpr int kQSlots = kPair ? 4 : kBlocks;
  static constexpr uint32_t kQSlot = uint32_t(kCtaRows) * 128u;
  static constexpr uint32_t kTmemCols = 2 * kTileRows;        // two S buffers

  static constexpr int B_KFULL = 0;                    // [3] a group of key blocks landed
  static constexpr int B_KFULLP = B_KFULL + kGroups;   // [3] the odd rank's (pair)
  static constexpr int B_KEMPTY = B_KFULLP + kGroups;  // [3] its products are done
  static constexpr int B_QFULL = B_KEMPTY + kGroups;   // [kQSlots]
  static constexpr int B_QEMPTY = B_QFULL + kQSlots;   // [kQSlots]
  static constexpr int B_SFULL = B_QEMPTY + kQSlots;   // [2]
  static constexpr int B_SEMPTY = B_SFULL + 2;         // [2]
  static constexpr int B_FIN = B_SEMPTY + 2;
  static constexpr int kNumBars = B_FIN + 1;

  static constexpr uint32_t kOffTmemSlot = 512;
  static constexpr uint32_t kOffAbort = 516;
  static constexpr uint32_t kOffFlags = 520;
  static constexpr uint32_t kOffSrow = 1024;    // int32 [2][128] pool rows of a key tile
  static constexpr uint32_t kOffLse = 2048;     // float [2][256] lse * log2(e) of a step's rows
  static constexpr uint32_t kOffPart = 4096;    // float [128] the second half's sums
  static constexpr uint32_t kOffK = 5120;
  static constexpr uint32_t kOffQ = kOffK + kBlocks * kKSlot;
  static constexpr uint32_t kSmemBytes = kOffQ + kQSlots * kQSlot + 1024;
  static_assert(8 * kNumBars <= int(kOffTmemSlot), "barrier area");
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

// A place in the row of steps.  Every role of a cluster walks its run with one
// of these, so they agree without talking.
struct Walk {
  const ChunkParams& p;
  int tile_keys, tile_rows;
  ChunkReq r;
  int b, N;
  int kt, rt, lo, hi;   // key tile; row tile within [lo, hi)
  int64_t left;         // steps left, this one included

  __device__ Walk(const ChunkParams& p_, int tk, int tr) : p(p_), tile_keys(tk), tile_rows(tr) {}

  __device__ int first_key() const { return window_first(p.window, r.P); }
  __device__ int sink_tiles() const {
    const int s = p.sinks < N ? p.sinks : N;
    return p.window > 0 ? (s + tile_keys - 1) / tile_keys : 0;
  }
  __device__ void load(int b_) {
    b = b_;
    r = chunk_req(p, b);
    N = r.nlist < r.P + r.n ? r.nlist : r.P + r.n;
  }
  // Row tiles whose tokens see some key of tile kt: tokens from the tile's
  // first key on, up to the last whose window still reaches its last key.
  __device__ void rows_of(int t, int* l, int* h) const {
    const int64_t k0 = int64_t(t) * tile_keys;
    const int64_t i0 = k0 > r.P ? k0 - r.P : 0;
    int64_t i1 = r.n;
    if (p.window > 0 && k0 >= p.sinks) {
      const int64_t e = k0 + tile_keys - 1 + p.window - r.P;
      if (e < i1) i1 = e;
    }
    *l = int(i0 * p.H / tile_rows);
    *h = i1 > i0 ? int((i1 * p.H + tile_rows - 1) / tile_rows) : *l;
  }
  // Key tiles before `full` see every row (no window); the steps of a request.
  __device__ int full_tiles() const {
    const int tiles = (N + tile_keys - 1) / tile_keys;
    if (p.window > 0) return 0;
    const int f = r.P / tile_keys + 1;
    return f < tiles ? f : tiles;
  }
  __device__ int next_tile(int t) const {   // the tile after t - 1 that some token sees
    const int w = p.window > 0 ? first_key() / tile_keys : 0;
    return t >= sink_tiles() && t < w ? w : t;
  }
  __device__ int64_t steps() const {
    if (r.n == 0 || N == 0) return 0;
    const int tiles = (N + tile_keys - 1) / tile_keys;
    const int full = full_tiles();
    int64_t n = int64_t(full) * ((int64_t(r.n) * p.H + tile_rows - 1) / tile_rows);
    for (int t = next_tile(full); t < tiles; t = next_tile(t + 1)) {
      int l, h;
      rows_of(t, &l, &h);
      n += h - l;
    }
    return n;
  }
  // Step `at` (>= 0, within it) of request b.
  __device__ void seek(int64_t at) {
    const int full = full_tiles();
    const int64_t nrt = (int64_t(r.n) * p.H + tile_rows - 1) / tile_rows;
    if (at < full * nrt) {
      kt = int(at / nrt);
      rows_of(kt, &lo, &hi);
      rt = lo + int(at % nrt);
      return;
    }
    at -= full * nrt;
    const int tiles = (N + tile_keys - 1) / tile_keys;
    for (kt = next_tile(full); kt < tiles; kt = next_tile(kt + 1)) {
      rows_of(kt, &lo, &hi);
      if (at < hi - lo) break;
      at -= hi - lo;
    }
    rt = lo + int(at);
  }
  // The next step (only while left > 1).
  __device__ void next() {
    --left;
    if (left <= 0) return;
    if (++rt < hi) return;
    kt = next_tile(kt + 1);
    while (r.n == 0 || int64_t(kt) * tile_keys >= N) {
      if (b + 1 >= p.B) { left = 0; return; }
      load(b + 1);
      kt = next_tile(0);
    }
    rows_of(kt, &lo, &hi);
    rt = lo;
  }
};

// The run of cluster c of C: its first step and length.  Whole warps call it.
__device__ void find_run(Walk& w, int c, int C, int lane) {
  constexpr uint32_t kAll = 0xffffffffu;
  int64_t total = 0, s0 = 0;   // s0: steps of request `lane`, kept for B <= 32
  for (int b0 = 0; b0 < w.p.B; b0 += 32) {
    int64_t s = 0;
    if (b0 + lane < w.p.B) {
      w.load(b0 + lane);
      s = w.steps();
    }
    // (no run goes past the steps counted here, so none reaches the batch's end)
    const uint32_t ends = __ballot_sync(kAll, chunk_ends(w.p, b0 + lane));
    if (ends && lane >= __ffs(int(ends)) - 1) s = 0;
    if (b0 == 0) s0 = s;
    total += s;
    if (ends) break;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
  const int64_t begin = total * c / C, end = total * (c + 1) / C;
  w.left = end - begin;
  if (w.left == 0) return;
  int64_t before = 0;
  for (int b0 = 0; b0 < w.p.B; b0 += 32) {
    int64_t s = s0;
    if (b0 > 0) {
      s = 0;
      if (b0 + lane < w.p.B) {
        w.load(b0 + lane);
        s = w.steps();
      }
    }
    int64_t sum = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(kAll, sum, o);
      if (lane >= o) sum += x;
    }
    const uint32_t mine = __ballot_sync(kAll, begin >= before + sum - s && begin < before + sum);
    if (mine) {
      const int src = __ffs(int(mine)) - 1;
      const int64_t first = before + __shfl_sync(kAll, sum - s, src);
      w.load(b0 + src);
      w.seek(begin - first);
      return;
    }
    before += __shfl_sync(kAll, sum, 31);
  }
}

template <bool kPair>
__global__ void __launch_bounds__(kThreads, 1)
    weights_tc_kernel(const __grid_constant__ WeightTcParams p,
                      const __grid_constant__ CUtensorMap tmap_q) {
  using C = WCfg<kPair>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sb = (raw + 1023u) & ~1023u;
  uint8_t* gb = smem_raw + (sb - raw);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gb + C::kOffAbort);
  uint32_t* cta_flags = reinterpret_cast<uint32_t*>(gb + C::kOffFlags);
  auto bar = [&](int i) -> uint32_t { return sb + 8u * uint32_t(i); };
  auto fail = [&]() {
    *abort_flag = 1;
    atomicOr(cta_flags, VA_STATUS_TIMEOUT);
  };
  const int hh = kPair ? int(cluster_ctarank()) : 0;   // which 128 keys (and query rows)
  const int cluster = int(blockIdx.x) / C::kCtas;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) tma_prefetch(&tmap_q);

  griddep_wait();                // the stream's previous kernel has completed
  griddep_launch_dependents();   // weights_finish_kernel may start its set-up
  if (blockIdx.x == 0 && tid == 0) *p.c.status = 0u;
  Walk w(p.c, C::kTileKeys, C::kTileRows);
  find_run(w, cluster, int(gridDim.x) / C::kCtas, lane);
  // a run that begins inside a key tile's rows leaves a share in its slot
  const bool cont = w.left > 0 && w.rt > w.lo;
  if (tid == 0 && hh == 0)
    p.cont_entry[cluster] = cont ? int(w.r.base) + w.kt * C::kTileKeys : -1;
  if (w.left == 0) {   // every CTA of the cluster leaves together
    if (tid == 0) p.cta_flags[blockIdx.x] = 0u;
    return;
  }

  if (tid == 0) {
    for (int i = 0; i < C::kNumBars; ++i) {
      uint32_t cnt = 1;
      if (i >= C::B_KFULL && i < C::B_KFULL + kGroups) cnt = kProducers;
      // in a pair the odd rank's eight epilogue warps add one arrival each
      if (i >= C::B_SEMPTY && i < C::B_SEMPTY + 2) cnt = kEpilogue + (kPair ? kEpilogue / 32 : 0);
      mbar_init(bar(i), cnt);
    }
    *abort_flag = 0;
    *cta_flags = 0u;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    if constexpr (kPair) tmem_alloc_pair(sb + C::kOffTmemSlot, C::kTmemCols);
    else tmem_alloc(sb + C::kOffTmemSlot, C::kTmemCols);
  }
  tc_fence_before();
  if constexpr (kPair) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gb + C::kOffTmemSlot);

  if (warp >= kEpilogue / 32 && warp < kMmaWarp) {
    // ---- keys: a tile's 128 rows, in three groups of column blocks; a warp
    // instruction copies 128 bytes of each of four rows
    const int ptid = tid - kEpilogue;
    int* srow = reinterpret_cast<int*>(gb + C::kOffSrow);
    const int pw = ptid >> 5;
    bool ok = true;
#ifdef VA_TEST_HOOKS
    {
      bool open = true;
      if (ptid == 0 && g_va_weights_gate) {
        const long long t0 = clock64();
        while (open && *reinterpret_cast<const volatile int32_t*>(g_va_weights_gate) == 0) {
          open = clock64() - t0 <= kWaitCycles;
          __nanosleep(2000);
        }
      }
      ok = named_sync_and(kProducerBar, kProducers, open);
    }
#endif
    int visit = 0, kt = -1, b = -1;
    for (; ok && w.left > 0; w.next()) {
      if (w.kt == kt && w.b == b) continue;   // another row tile of the same keys
      kt = w.kt;
      b = w.b;
      int* rows = srow + (visit & 1) * kKeys;
      if (ptid < kKeys) {
        const int j = kt * C::kTileKeys + hh * kKeys + ptid;
        rows[ptid] = j < w.N ? int(chunk_key_row(w.p, w.r, j)) : -1;
      }
#pragma unroll 1
      for (int g = 0; g < kGroups; ++g) {
        bool got = true;
        if (ptid == 0 && visit > 0)
          got = mbar_wait(bar(C::B_KEMPTY + g), uint32_t(visit - 1) & 1u, abort_flag, kWaitCycles);
        if (!named_sync_and(kProducerBar, kProducers, got)) {
          ok = false;
          break;
        }
        const uint32_t slot0 = sb + C::kOffK + uint32_t(3 * g) * kKSlot;
#pragma unroll 2
        for (int key = pw * 4 + (lane >> 3); key < kKeys; key += (kProducers / 32) * 4) {
          const int row = rows[key];
          const __nv_bfloat16* src = w.p.kv + (row >= 0 ? int64_t(row) * w.p.kv_stride : 0) +
                                     192 * g + (lane & 7) * 8;
          const uint32_t nb = row >= 0 ? 16u : 0u;
          const uint32_t dst =
              slot0 + uint32_t(key) * 128u + uint32_t(((lane & 7) ^ (key & 7)) * 16);
#pragma unroll
          for (int c = 0; c < 3; ++c) cp_async16(dst + uint32_t(c) * kKSlot, src + 64 * c, nb);
        }
        cp_async_arrive_noinc(bar(C::B_KFULL + g));
      }
      if (!ok) break;
      ++visit;
    }
    if (!ok && ptid == 0) fail();
    cp_async_wait_all();
  } else if (warp == kMmaWarp) {
    // ---- products: the even rank's, for both CTAs of a pair
    bool ok = true;
    if (hh == 0) {
      int step = 0, visit = -1, qload = -1, kt = -1, b = -1, qb = -1, qrt = -1;
      for (; w.left > 0; ++step) {
        const bool new_k = w.kt != kt || w.b != b;
        const bool new_q = kPair || w.rt != qrt || w.b != qb;
        if (new_k) ++visit;
        if (new_q) ++qload;
        kt = w.kt;
        b = w.b;
        qb = w.b;
        qrt = w.rt;
        // query rows of the step: N of the product (a multiple of 16)
        int n16 = C::kTileRows;
        if constexpr (!kPair) {
          const int rows = w.r.n * w.p.H - w.rt * C::kTileRows;
          n16 = rows < C::kTileRows ? (rows + 15) & ~15 : C::kTileRows;
        }
        const uint32_t idesc = idesc_bf16(uint32_t(C::kTileKeys), uint32_t(n16), 0, 0);
        w.next();
        const bool last_k = w.left <= 0 || w.kt != kt || w.b != b;
        const bool last_q = kPair || w.left <= 0 || w.rt != qrt || w.b != qb;
        const int bs = step & 1;
        ok = step < 2 || __all_sync(0xffffffffu,
                                    mbar_wait<kPair>(bar(C::B_SEMPTY + bs),
                                                     uint32_t((step >> 1) - 1) & 1u, abort_flag,
                                                     kWaitCycles));
        tc_fence_after();
        const uint32_t d = tmem + uint32_t(C::kTileRows * bs);
#pragma unroll 1
        for (int c = 0; ok && c < kBlocks; ++c) {
          const int g = c / 3;
          bool got = true;
          if (new_k && c == 3 * g) {
            got = mbar_wait(bar(C::B_KFULL + g), uint32_t(visit) & 1u, abort_flag, kWaitCycles) &&
                  (!kPair || mbar_wait<true>(bar(C::B_KFULLP + g), uint32_t(visit) & 1u, abort_flag,
                                             kWaitCycles));
          }
          const int at = kPair ? kBlocks * step + c : c;
          const int qs = at % C::kQSlots;
          const uint32_t qpar = uint32_t(kPair ? at / C::kQSlots : qload) & 1u;
          if (new_q)
            got = got && mbar_wait<kPair>(bar(C::B_QFULL + qs), qpar, abort_flag, kWaitCycles);
          if (!__all_sync(0xffffffffu, got)) {
            ok = false;
            break;
          }
          if (new_k && c == 3 * g) fence_proxy_async_cta();   // the copies, seen by the tensor core
          tc_fence_after();
          const uint64_t ad = smem_desc(sb + C::kOffK + uint32_t(c) * kKSlot, 16, 1024, kSwizzle128B);
          const uint64_t bd =
              smem_desc(sb + C::kOffQ + uint32_t(qs) * C::kQSlot, 16, 1024, kSwizzle128B);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint32_t acc = (c | kk) != 0 ? 1u : 0u;
              if constexpr (kPair) mma2_ss(d, ad + uint64_t(2 * kk), bd + uint64_t(2 * kk), idesc, acc);
              else mma_ss(d, ad + uint64_t(2 * kk), bd + uint64_t(2 * kk), idesc, acc);
            }
            if (last_q) {
              if constexpr (kPair) mma2_commit_mc(bar(C::B_QEMPTY + qs), kBoth);
              else mma_commit(bar(C::B_QEMPTY + qs));
            }
            if (last_k && c == 3 * g + 2) {
              if constexpr (kPair) mma2_commit_mc(bar(C::B_KEMPTY + g), kBoth);
              else mma_commit(bar(C::B_KEMPTY + g));
            }
          }
          __syncwarp();
        }
        if (!ok) {
          if (lane == 0) fail();
          break;
        }
        if constexpr (kPair) mma2_commit_mc_warp(bar(C::B_SFULL + bs), kBoth);
        else mma_commit_warp(bar(C::B_SFULL + bs));
      }
      if constexpr (kPair) mma2_commit_mc_warp(bar(C::B_FIN), kBoth);
      else mma_commit_warp(bar(C::B_FIN));
    } else {
      // the odd rank's key groups, forwarded to the even rank whose products
      // read them
      const uint32_t fullp = mapa(bar(C::B_KFULLP), 0);
      int visit = -1, kt = -1, b = -1;
      for (; ok && w.left > 0; w.next()) {
        if (w.kt == kt && w.b == b) continue;
        kt = w.kt;
        b = w.b;
        ++visit;
        for (int g = 0; g < kGroups; ++g) {
          if (!__all_sync(0xffffffffu, mbar_wait(bar(C::B_KFULL + g), uint32_t(visit) & 1u,
                                                 abort_flag, kWaitCycles))) {
            if (lane == 0) fail();
            ok = false;
            break;
          }
          fence_proxy_async_cta();
          if (lane == 0) mbar_arrive_remote(fullp + 8u * uint32_t(g));
          __syncwarp();
        }
      }
    }
    // products read both CTAs' memories until their last commit
    (void)mbar_wait(bar(C::B_FIN), 0, nullptr, kWaitCycles);
    __syncwarp();
  } else if (warp == kQueryWarp) {
    // ---- query rows: a box of the CTA's share of the step's rows per column
    // block.  In a pair both CTAs' boxes land on the even rank's barrier.
    if (lane == 0) {
      bool ok = true;
      int step = 0, qload = -1, qb = -1, qrt = -1;
      for (; ok && w.left > 0; w.next(), ++step) {
        if (!kPair && w.rt == qrt && w.b == qb) continue;   // resident
        ++qload;
        qb = w.b;
        qrt = w.rt;
        const int row = w.r.q0 * w.p.H + w.rt * C::kTileRows + hh * C::kCtaRows;
        for (int c = 0; c < kBlocks; ++c) {
          const int at = kPair ? kBlocks * step + c : c;
          const int qs = at % C::kQSlots;
          const int use = kPair ? at / C::kQSlots : qload;
          if (use > 0 && !mbar_wait(bar(C::B_QEMPTY + qs), uint32_t(use - 1) & 1u, abort_flag,
                                    kWaitCycles)) {
            fail();
            ok = false;
            break;
          }
          const uint32_t dst = sb + C::kOffQ + uint32_t(qs) * C::kQSlot;
          if (hh == 0) mbar_arrive_expect_tx(bar(C::B_QFULL + qs), uint32_t(C::kCtas) * C::kQSlot);
          if constexpr (kPair)
            tma_load_3d_pair(dst, &tmap_q, 0, row, c, mapa(bar(C::B_QFULL + qs), 0));
          else
            tma_load_3d(dst, &tmap_q, 0, row, c, bar(C::B_QFULL + qs));
        }
      }
      (void)mbar_wait(bar(C::B_FIN), 0, nullptr, kWaitCycles);
      // after an abort boxes may still be in flight: a bounded time to land
      if (*abort_flag)
        for (const long long t0 = clock64(); clock64() - t0 < kDrainCycles;) {}
    }
    __syncwarp();
  } else {
    // ---- epilogue: thread = key; the two halves take half of the columns each
    const int etid = tid, half = warp >> 2, q4 = warp & 3;
    const int r = q4 * 32 + lane;
    constexpr int kHalf = C::kTileRows / 2;
    float* lse = reinterpret_cast<float*>(gb + C::kOffLse);
    float* part = reinterpret_cast<float*>(gb + C::kOffPart);
    const uint32_t tl = tmem + (uint32_t(q4 * 32) << 16) + uint32_t(kHalf * half);
    const uint32_t sempty = kPair ? mapa(bar(C::B_SEMPTY), 0) : 0u;
    const float sc = p.c.scale_log2;
    const int window = p.c.window, sinks = p.c.sinks;
    float total = 0.f;
    bool to_slot = cont;
    bool ok = true;
    for (int step = 0; w.left > 0; ++step) {
      const int bs = step & 1;
      const int R = w.r.n * w.p.H, row0 = w.rt * C::kTileRows;
      // the step's lse; +inf for a row that saw nothing (lse -inf): no weight
      bool clean = true;
      if (etid < C::kTileRows) {
        const int row = row0 + etid;
        float l = INFINITY;
        if (row < R) {
          const float x = w.p.lse[size_t(w.r.q0) * w.p.H + row];
          if (x != -INFINITY) l = x * kLog2e;
        }
        lse[bs * 256 + etid] = l;
        clean = l != INFINITY;
      }
      // The columns (rows of the step) that see this thread's key are one run
      // [c_lo, c_hi): from its own token on, up to the last token whose window
      // reaches it.  Most steps lie inside it for every key.
      const int k0 = w.kt * C::kTileKeys + hh * kKeys;
      const int j = k0 + r;
      int c_lo, c_hi;
      {
        const int64_t lo = int64_t(j - w.r.P) * w.p.H - row0;
        int64_t hi = R - row0;
        if (window > 0 && j >= sinks) {
          const int64_t x = (int64_t(j) + window - w.r.P) * w.p.H - row0;
          hi = x < hi ? x : hi;
        }
        c_lo = lo < 0 ? 0 : lo > C::kTileRows ? C::kTileRows : int(lo);
        c_hi = hi < 0 ? 0 : hi > C::kTileRows ? C::kTileRows : int(hi);
      }
      if (c_lo > 0 || c_hi < C::kTileRows) clean = false;
      // what the step's end needs of this place
      const int N = w.N, tile0 = w.kt * C::kTileKeys, kt = w.kt, b = w.b;
      const int64_t base = w.r.base;
      const int cols = R - row0 < C::kTileRows ? R - row0 : C::kTileRows;
      w.next();
      const bool last_k = w.left <= 0 || w.kt != kt || w.b != b;
      clean = named_sync_and(kEpilogueBar, kEpilogue, clean);
      const bool got = mbar_wait(bar(C::B_SFULL + bs), uint32_t(step >> 1) & 1u, abort_flag,
                                 kWaitCycles);
      if (!__all_sync(0xffffffffu, got)) ok = false;
      if (ok) {
        tc_fence_after();
        float sum = 0.f;
#pragma unroll 1
        for (int c0 = 0; c0 < kHalf; c0 += 32) {
          if (kHalf * half + c0 >= cols) break;   // (a warp's lanes agree)
          uint32_t sv[32];
          tmem_ld32(tl + uint32_t(C::kTileRows * bs + c0), sv);
          tmem_wait_ld();
          const float4* l4 =
              reinterpret_cast<const float4*>(lse + bs * 256 + kHalf * half + c0);
          if (clean) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const float4 l = l4[c];
              sum += (ex2_approx(fmaf(__uint_as_float(sv[4 * c]), sc, -l.x)) +
                      ex2_approx(fmaf(__uint_as_float(sv[4 * c + 1]), sc, -l.y))) +
                     (ex2_approx(fmaf(__uint_as_float(sv[4 * c + 2]), sc, -l.z)) +
                      ex2_approx(fmaf(__uint_as_float(sv[4 * c + 3]), sc, -l.w)));
            }
          } else {
            // a score that is hidden, or of a row without weight, is not used
            // at all, whatever it is
            const int lo = c_lo - (kHalf * half + c0), hi = c_hi - (kHalf * half + c0);
            auto term = [&](int c, float l) -> float {
              return c >= lo && c < hi && l < INFINITY
                         ? ex2_approx(fmaf(__uint_as_float(sv[c]), sc, -l))
                         : (l != l && c >= lo && c < hi ? l : 0.f);
            };
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const float4 l = l4[c];
              sum += (term(4 * c, l.x) + term(4 * c + 1, l.y)) +
                     (term(4 * c + 2, l.z) + term(4 * c + 3, l.w));
            }
          }
        }
        tc_fence_before();
        total += sum;
        if (hh == 0) {
          mbar_arrive(bar(C::B_SEMPTY + bs));
        } else {
          __syncwarp();
          if (lane == 0) mbar_arrive_remote_relaxed(sempty + 8u * uint32_t(bs));
        }
      }
      if (!named_sync_and(kEpilogueBar, kEpilogue, ok)) {
        if (etid == 0) fail();
        break;
      }
      if (last_k) {
        if (half) part[r] = total;
        named_sync(kEpilogueBar, kEpilogue);
        if (!half && j < N) {
          const float v = total + part[r];
          if (to_slot) p.cont[size_t(cluster) * 256 + (j - tile0)] = v;
          else p.sums[base + j] = v;
        }
        total = 0.f;
        to_slot = false;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0) p.cta_flags[blockIdx.x] = *cta_flags;
  if constexpr (kPair) {
    cluster_sync();
    if (warp == kMmaWarp) {
      tc_fence_after();
      tmem_dealloc_pair(tmem, C::kTmemCols);
    }
  } else if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// weights_out = weights_in + the key's sums: its tile's share in `sums`, then the
// shares of the clusters whose runs began inside the tile, in cluster order.  A
// thread per entry; keys that no token sees keep their totals.
__global__ void __launch_bounds__(256) weights_finish_kernel(const WeightTcParams p) {
  __shared__ int heads[kWeightClusters];
  __shared__ uint32_t s_bits;
  const ChunkParams& c = p.c;
  const int tid = threadIdx.x;
  uint32_t bits = 0u;
  if (tid == 0) s_bits = 0u;
  // the entry's request: the last list that begins at or before it, or, where the
  // bounds are in error, any whose keys it is among (the bounds are inputs of the
  // call, so they are read before the wait)
  const int requests = chunk_requests(c, tid & 31);
  const bool sorted = chunk_lists_sorted(c, tid & 31);
  const int64_t e = int64_t(blockIdx.x) * 256 + tid;
  ChunkReq r;
  r.n = r.P = r.nlist = 0;
  r.base = 0;
  if (e < c.num_entries && sorted) {
    int lo = 0, hi = c.B;   // indptr[lo] <= e (or lo = 0), indptr[hi] > e (or hi = B)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (c.kv_indptr[mid] <= e) lo = mid;
      else hi = mid;
    }
    r = chunk_req(c, lo, lo >= requests);
  } else if (e < c.num_entries) {
    for (int b = 0; b < c.B; ++b) {
      const ChunkReq x = chunk_req(c, b, b >= requests);
      const int64_t j = e - x.base;
      if (j >= 0 && j < x.nlist && j < x.P + x.n) {
        r = x;
        break;
      }
    }
  }
  griddep_wait();                // the sums are complete
  griddep_launch_dependents();   // the next kernel may start its set-up
  for (int i = tid; i < p.clusters; i += 256) heads[i] = p.cont_entry[i];
  for (int i = tid; i < p.clusters * (p.tile_keys / kKeys); i += 256) bits |= p.cta_flags[i];
  // (a CTA that gave up a wait has not written the shares of its last tiles: then
  // every key keeps its total, and the status word says so)
  const bool gave_up = __syncthreads_or((bits & VA_STATUS_TIMEOUT) != 0u);
  const int64_t j64 = e - r.base;
  const int N = r.nlist < r.P + r.n ? r.nlist : r.P + r.n;
  if (e < c.num_entries && j64 >= 0 && j64 < N) {
    const int j = int(j64);
    // the tokens that see key j: from its own (or the first) to the last whose
    // window reaches it
    const int first = j > r.P ? j - r.P : 0;
    int64_t last = r.n - 1;
    if (c.window > 0 && j >= c.sinks && int64_t(j) + c.window - 1 - r.P < last)
      last = int64_t(j) + c.window - 1 - r.P;
    float v = 0.f;
    if (first <= last && !gave_up) {
      if (chunk_key_row(c, r, j) < 0) {
        bits |= VA_STATUS_BAD_SLOT;
      } else {
        const int in_tile = j % p.tile_keys;
        const int tile = int(e) - in_tile;
        v = p.sums[e];
        for (int i = 0; i < p.clusters; ++i)
          if (heads[i] == tile) v += p.cont[size_t(i) * 256 + in_tile];
      }
    }
    p.wout[e] = (p.win ? p.win[e] : 0.f) + v;
  }
  if (blockIdx.x == 0)
    for (int b = tid; b < c.B; b += 256)
      if (chunk_req(c, b).bad) bits |= VA_STATUS_BAD_INDPTR;
  if (bits) atomicOr(&s_bits, bits);
  __syncthreads();
  if (tid == 0 && s_bits) atomicOr(c.status, s_bits);
}

}  // namespace

cudaError_t init_weights_tc() {
  constexpr cudaFuncAttribute kSmem = cudaFuncAttributeMaxDynamicSharedMemorySize;
  const cudaError_t e =
      cudaFuncSetAttribute(weights_tc_kernel<false>, kSmem, int(WCfg<false>::kSmemBytes));
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(weights_tc_kernel<true>, kSmem, int(WCfg<true>::kSmemBytes));
}

// p.clusters, p.tile_keys and the workspace pointers are set by the caller.
cudaError_t launch_weights_tc(const WeightTcParams& p, bool pair, cudaStream_t st) {
  const int ctas = pair ? 2 : 1;
  CUtensorMap tq;
  memset(&tq, 0, sizeof tq);
  if (p.c.total_q > 0) {
    if (!g_encode) return cudaErrorNotSupported;
    cuuint64_t dims[3] = {64u, cuuint64_t(p.c.total_q) * cuuint64_t(p.c.H), cuuint64_t(kBlocks)};
    cuuint64_t strides[2] = {cuuint64_t(kDqk) * 2u, 128u};
    cuuint32_t box[3] = {64u, uint32_t(pair ? WCfg<true>::kCtaRows : WCfg<false>::kCtaRows), 1u};
    cuuint32_t estr[3] = {1u, 1u, 1u};
    if (g_encode(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16*>(p.c.q), dims,
                 strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                 CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorNotSupported;
  }
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(unsigned(ctas * p.clusters), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = pair ? WCfg<true>::kSmemBytes : WCfg<false>::kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(ctas);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = pair ? cudaLaunchKernelEx(&cfg, weights_tc_kernel<true>, p, tq)
                             : cudaLaunchKernelEx(&cfg, weights_tc_kernel<false>, p, tq);
  if (e != cudaSuccess) return e;
  const int64_t blocks = (p.c.num_entries + 255) / 256;
  cfg.gridDim = dim3(unsigned(blocks < 1 ? 1 : blocks), 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, weights_finish_kernel, p);
}

}  // namespace va
