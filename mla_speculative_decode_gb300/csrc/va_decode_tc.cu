// va_decode_tc.cu -- chunk attention of few rows per request (a decode batch:
// one token, up to 64 heads) on the tcgen05 tensor cores, one SM per piece.
//
// With at most 64 rows the pass is bound by reading the keys, so a key row has
// to enter an SM once and serve both products.  The split kernel (va_tc.cu)
// cannot do that: its 128 x 512 accumulator fills an SM's tensor memory, so the
// scores live on another SM and the keys are gathered twice.  Here the second
// product is turned round,
//     S = Q K^T        (M = 64 rows, N = 64 keys, 36 products of depth 16)
//     O^T += V^T P^T   (M = 128 value columns, four times; N = the rows there
//                       are, up to 64; depth 64 keys)
// and both accumulators fit one SM: O^T takes 4 x 64 columns of tensor memory, S
// two buffers of 64.  The same shared-memory tile of 64 gathered rows is the
// K-major B operand of the first product and the MN-major A operand of the
// second.  Shared memory: two key tiles (2 x 72 KB), the unit's queries (72 KB)
// and P (8 KB).
//
// Warps: 0-7 softmax (row = lane of a half-filled quadrant, two warps share a
// quadrant, each 32 of a tile's 64 keys) and write-out (value column = lane),
// 8-14 gather keys (16-byte cp.async, or one TMA box per tile of a contiguous
// pool), 15 issues the products and the boxes of queries.
//
// Work: the tiles of all units (64 rows of a request; a decode request is one
// unit) form one row of steps, and every SM takes an equal run of it, whatever
// the lengths.  A unit inside one run goes straight to out and lse; of a unit cut
// by run ends each piece leaves an fp32 partial for the merge (va_chunk.cu).
//
// Measured: 32 requests of one token, 64 heads, 1k to 32k paged keys (701 MB): 177 us,
// 4.0 TB/s, where a kernel that only gathers such rows reaches 5.6.  A tile takes
// about 5200 cycles: its copies 3700 if nothing disturbs them, and with two tiles of
// shared memory a tile's products, softmax and release (2800) overlap the next one's
// copies only in part.  (Slower: copies without the producers' barrier 182 to 208,
// the next rows brought into L2 first 210, more copying warps 191 to 211.)  One
// thread issues a group's products; elected one by one they took it to 192.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <string.h>

#include "va_chunk.cuh"
#include "va_sm100.cuh"

namespace va {

extern PFN_cuTensorMapEncodeTiled_v12000 g_encode;   // va_tc.cu, resolved by va_init

namespace {

using namespace sm100;

constexpr int kSoftmax = 256;          // warps 0-7
constexpr int kProducers = 224;        // warps 8-14
constexpr int kMmaWarp = 15;
constexpr int kThreads = 512;
constexpr uint32_t kSoftmaxBar = 1, kProducerBar = 2;   // named barriers
constexpr int kRows = 64, kTile = 64, kBlocks = kDqk / 64;
constexpr int kGroups = 3;             // of three 64-column blocks: what is loaded and released as one
constexpr uint32_t kSlot = kTile * 128u;               // one 64-column block of a tile
constexpr uint32_t kTileBytes = kBlocks * kSlot;
constexpr int kValidRing = 4;
constexpr uint32_t kTmemCols = 512, kTmemO = 0, kTmemS = 256;
constexpr long long kWaitCycles = 4000000000ll;   // wait bound in SM cycles (~2 s)
constexpr long long kDrainCycles = 2000000ll;     // after an abort: boxes in flight land
constexpr float kRescaleLog2 = 8.f;

// What a unit costs besides its tiles, in tiles: queries in, rows out.  (64 requests
// with a window of 4096: 0 98.7 us, 1 98.1, 2 96.3, 4 98.7.)
using Run = ChunkRun<kRows, 2>;

// Barriers.
constexpr int B_KFULL = 0;                     // [2][kGroups] column blocks of a key tile landed
constexpr int B_KEMPTY = B_KFULL + 2 * kGroups;   // [2][kGroups] both products of them are done
constexpr int B_SFULL = B_KEMPTY + 2 * kGroups;   // [2]
constexpr int B_SEMPTY = B_SFULL + 2;          // [2]
constexpr int B_VREADY = B_SEMPTY + 2;         // [kValidRing] a tile's key-validity mask
constexpr int B_PFULL = B_VREADY + kValidRing;
constexpr int B_PFREE = B_PFULL + 1;           // the second product has read P (and O is final)
constexpr int B_QFULL = B_PFREE + 1;
constexpr int B_QEMPTY = B_QFULL + 1;
constexpr int B_OFULL = B_QEMPTY + 1;          // a piece's last product is done
constexpr int B_OFREE = B_OFULL + 1;           // its O has been read
constexpr int B_FIN = B_OFREE + 1;
constexpr int kNumBars = B_FIN + 1;

// Shared layout (offsets from a 1024-byte aligned base).
constexpr uint32_t kOffTmemSlot = 256, kOffAbort = 260, kOffFlags = 264;
constexpr uint32_t kOffValid = 272;    // uint64 [kValidRing]
constexpr uint32_t kOffSrow = 512;     // int32 [2][64] pool rows of a tile
constexpr uint32_t kOffMx = 1024;      // float [2][64] half maxima, then half sums
constexpr uint32_t kOffAlpha = 1536;   // float [64] rescale factors; at the end 1 / row sum
constexpr uint32_t kOffK = 2048;
constexpr uint32_t kOffQ = kOffK + 2 * kTileBytes;
constexpr uint32_t kOffP = kOffQ + kTileBytes;
constexpr uint32_t kEnd = kOffP + kRows * 128u;
constexpr uint32_t kSmemBytes = kEnd + 1024;
static_assert(8 * kNumBars <= int(kOffTmemSlot) && kOffValid + 8 * kValidRing <= kOffSrow, "header");
static_assert(kOffK % 1024 == 0 && kSmemBytes <= 232448, "shared memory budget");

__global__ void __launch_bounds__(kThreads, 1)
    decode_tc_kernel(const __grid_constant__ ChunkTcParams p, const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_q) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sb = (raw + 1023u) & ~1023u;
  uint8_t* gb = smem_raw + (sb - raw);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gb + kOffAbort);
  uint32_t* cta_flags = reinterpret_cast<uint32_t*>(gb + kOffFlags);
  auto bar = [&](int i) -> uint32_t { return sb + 8u * uint32_t(i); };
  auto wait = [&](int i, uint32_t parity) -> bool {
    return mbar_wait(bar(i), parity & 1u, abort_flag, kWaitCycles);
  };
  auto fail = [&]() {
    *abort_flag = 1;
    atomicOr(cta_flags, VA_STATUS_TIMEOUT);
  };
  const int cta = int(blockIdx.x);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    tma_prefetch(&tmap_q);
    if (p.kv_start) tma_prefetch(&tmap_k);
  }
  griddep_wait();                // the stream's previous kernel has completed
  griddep_launch_dependents();   // the merge may start its set-up
  Run w(p);
  const int all_units = find_run(w, cta, int(gridDim.x), lane);
  if (cta == 0 && tid == 0) {
    p.totals[0] = all_units;
    p.totals[1] = int(gridDim.x);
  }
  if (!w.more()) {
    if (tid == 0) p.cta_flags[cta] = 0u;
    return;
  }
  // the first tile's slots load during the set-up
  const bool producer = warp >= 8 && warp < kMmaWarp;
  const int ptid = tid - kSoftmax;
  auto fetch = [&](const Run& x) -> int {   // raw pool row of this thread's key of the step's tile
    const int j = x.key() + ptid;
    if (!x.t.sees(j) || j >= x.r.nlist) return -1;
    if (p.kv_start) {
      const int64_t row = x.r.base + j;
      return row >= 0 && row < p.num_slots && row <= 0x7fffffff ? int(row) : -1;
    }
    return __ldg(p.slot_idx + x.r.base + j);
  };
  const int raw0 = producer && ptid < kTile ? fetch(w) : -1;

  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      uint32_t cnt = 1;
      if (i >= B_KFULL && i < B_KFULL + 2 * kGroups) cnt = kProducers + 1;   // copies + producer 0
      if (i == B_SEMPTY || i == B_SEMPTY + 1 || i == B_PFULL || i == B_OFREE) cnt = kSoftmax;
      mbar_init(bar(i), cnt);
    }
    *abort_flag = 0;
    *cta_flags = 0u;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(sb + kOffTmemSlot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gb + kOffTmemSlot);

  if (producer) {
    // ---- keys: 64 rows of a tile; a warp instruction copies 128 bytes of each of
    // four rows (one column block).  The tile's rows are staged first; then, as
    // each group of column blocks is released, the warps share its 3 x 16
    // instructions.  After a wait gave up a warp stays in step, copying nothing.
    int* srow = reinterpret_cast<int*>(gb + kOffSrow);
    uint32_t* valid32 = reinterpret_cast<uint32_t*>(gb + kOffValid);
    const int pw = ptid >> 5;
    int rawrow = raw0;
    bool ok = true, bad_slot = false;
    int box_step[2] = {-1, -1};   // the last step loaded by boxes into each half
    for (int s = 0; w.more(); ++s) {
      const int half = s & 1;
      const int tk0 = w.key();
      if (ptid < kTile) {
        const int row = rawrow >= 0 && int64_t(rawrow) < p.num_slots ? rawrow : -1;
        srow[half * kTile + ptid] = row;
        bad_slot |= w.t.sees(tk0 + ptid) && row < 0;
        const uint32_t v = __ballot_sync(0xffffffffu, row >= 0);
        if (lane == 0) valid32[(s % kValidRing) * 2 + (ptid >> 5)] = v;
      }
      named_sync(kProducerBar, kProducers);
      const int64_t row0 = p.kv_start ? w.r.base + tk0 : -1;
      const bool box = p.kv_start && w.t.whole(tk0) && tk0 + kTile <= w.r.nlist && row0 >= 0 &&
                       row0 + kTile <= p.num_slots && row0 + kTile <= 0x7fffffff;
      w.next();
      if (ptid < kTile && w.more()) rawrow = fetch(w);
      if (ptid == 0) {
        mbar_arrive(bar(B_VREADY + s % kValidRing));
        box_step[half] = box ? s : -1;
      }
      const uint32_t dst0 = sb + kOffK + uint32_t(half) * kTileBytes;
#pragma unroll 1
      for (int g = 0; g < kGroups; ++g) {
        const int full = B_KFULL + half * kGroups + g;
        if (s >= 2 && ok) {
          bool got = true;
          if (lane == 0) got = wait(B_KEMPTY + half * kGroups + g, uint32_t((s >> 1) - 1));
          ok = __all_sync(0xffffffffu, got);
          if (!ok && lane == 0) fail();
        }
        if (ptid == 0) {
          if (box && ok) {
            mbar_arrive_expect_tx(bar(full), 3 * kSlot);
            tma_load_3d(dst0 + uint32_t(3 * g) * kSlot, &tmap_k, 0, int(row0), 3 * g, bar(full));
          } else {
            mbar_arrive(bar(full));
          }
        }
        if (!box && ok) {
#pragma unroll
          for (int x = 0; x < 7; ++x) {
            const int u = pw + x * (kProducers / 32);   // block of the group x four keys
            if (u < 3 * kTile / 4) {
              const int c = 3 * g + (u >> 4);
              const int key = 4 * (u & 15) + (lane >> 3);
              const int row = srow[half * kTile + key];
              const __nv_bfloat16* src =
                  p.kv + (row >= 0 ? int64_t(row) * p.kv_stride : 0) + 64 * c + (lane & 7) * 8;
              cp_async16(dst0 + uint32_t(c) * kSlot + uint32_t(key) * 128u +
                             uint32_t(((lane & 7) ^ (key & 7)) * 16),
                         src, row >= 0 ? 16u : 0u);
            }
          }
        }
        cp_async_arrive_noinc(bar(full));
      }
    }
    if (bad_slot) atomicOr(cta_flags, VA_STATUS_BAD_SLOT);
    cp_async_wait_all();
    if (ptid == 0) {
      (void)mbar_wait(bar(B_FIN), 0, nullptr, kWaitCycles);
      // after an abort, boxes still in flight land before the CTA can leave
      if (*abort_flag)
        for (int i = 0; i < 2 * kGroups; ++i)
          if (box_step[i / kGroups] >= 0)
            (void)mbar_wait(bar(B_KFULL + i), uint32_t(box_step[i / kGroups] >> 1) & 1u, nullptr,
                            kDrainCycles);
    }
  } else if (warp == kMmaWarp) {
    // ---- products.  The second product of a tile goes as soon as its P is there
    // -- it is what frees the tile's shared memory -- and the first product of the
    // next tile group by group as it lands, whichever comes first; at a unit's end
    // the second goes first, as the next unit's queries are still to come.
    //
    // Queries: one box of 64 rows per unit, as soon as the last product that
    // reads the unit before is done (rows past the request's end are another's,
    // or zeros past the tensor; they are not used).  The lane that issues it also
    // writes the unit's entry for the merge, when its first tile is in this run.
    int loads = 0;
    auto queries = [&]() {
      ++loads;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(B_QFULL), kTileBytes);
        tma_load_3d(sb + kOffQ, &tmap_q, 0, w.r.q0 * p.H + w.unit * kRows, 0, bar(B_QFULL));
        if (w.k == 0) {
          ChunkUnit u;
          u.row0 = w.r.q0 * p.H + w.unit * kRows;
          u.rows = w.rows();
          u.ns = w.owner(w.g + w.t.ntiles - 1) - cta + 1;
          // slots 2c: the piece a run begins with; 2c + 1: a piece begun later
          u.pslot = 2 * cta + (w.g > w.begin(cta) ? 1 : 0);
          u.pslot1 = 2 * (cta + 1);
          u.pstride = 2;
          u.item = cta;
          u.istride = 1;
          u.b = w.b;
          u.i0 = w.unit * kRows;
          p.units[w.unit0 + w.unit] = u;
        }
      }
      __syncwarp();
    };
    constexpr uint32_t idesc_s = idesc_bf16(kRows, kTile, 0, 0);
    bool ok = true;
    int piece = 0;
    auto second = [&](int s, int n16, bool first, bool last) -> bool {
      if (first && piece > 0 && !__all_sync(0xffffffffu, wait(B_OFREE, uint32_t(piece - 1))))
        return false;
      if (!__all_sync(0xffffffffu, wait(B_PFULL, uint32_t(s)))) return false;
      tc_fence_after();
      const uint32_t idesc_o = idesc_bf16(128, uint32_t(n16), 1, 0);
      const uint32_t v0 = sb + kOffK + uint32_t(s & 1) * kTileBytes;
      const uint64_t bd = smem_desc(sb + kOffP, 16, 1024, kSwizzle128B);
      if (elect_one()) {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint64_t ad = smem_desc(v0 + uint32_t(2 * m) * kSlot, kSlot, 1024, kSwizzle128B);
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            mma_ss(tmem + kTmemO + uint32_t(64 * m), ad + uint64_t((uint32_t(k) * 2048u) >> 4),
                   bd + uint64_t((uint32_t(k) * 32u) >> 4), idesc_o, (!first || k > 0) ? 1u : 0u);
          // blocks 0-2, 3-5 and 6-8 are done with after value blocks 0-3, 4-5, 6-7
          if (m > 0) mma_commit(bar(B_KEMPTY + (s & 1) * kGroups + m - 1));
        }
        mma_commit(bar(B_PFREE));
        if (last) mma_commit(bar(B_OFULL));
      }
      __syncwarp();
      if (last) ++piece;
      return true;
    };
    // the tile whose second product is still to be issued
    int s = 0, qload = 0;
    queries();
    bool pending = false, pend_first = false, pend_last = false;
    int pend_n = 0;
    bool first = true;
    while (ok && w.more()) {
      const bool last = w.last_tile();
      const int n16 = (w.rows() + 15) & ~15;
      const int full = B_KFULL + (s & 1) * kGroups;
      if (pending && (first || !__all_sync(0xffffffffu,
                                           mbar_test(bar(full), uint32_t(s >> 1) & 1u)))) {
        ok = second(s - 1, pend_n, pend_first, pend_last);
        pending = false;
        if (!ok) break;
      }
      bool got = s < 2 || wait(B_SEMPTY + (s & 1), uint32_t((s >> 1) - 1));
      if (first) {
        got = got && wait(B_QFULL, uint32_t(qload));
        ++qload;
      }
      if (!__all_sync(0xffffffffu, got)) {
        ok = false;
        break;
      }
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        ok = ok && __all_sync(0xffffffffu, wait(full + g, uint32_t(s >> 1)));
        if (!ok) break;
        fence_proxy_async_cta();   // the producers' copies, seen by the tensor core
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int c = 3 * g; c < 3 * g + 3; ++c) {
            const uint64_t ad = smem_desc(sb + kOffQ + uint32_t(c) * kSlot, 16, 1024, kSwizzle128B);
            const uint64_t bd = smem_desc(
                sb + kOffK + uint32_t(s & 1) * kTileBytes + uint32_t(c) * kSlot, 16, 1024, kSwizzle128B);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ss(tmem + kTmemS + uint32_t(64 * (s & 1)), ad + uint64_t(2 * kk),
                     bd + uint64_t(2 * kk), idesc_s, (c | kk) != 0 ? 1u : 0u);
          }
          if (g + 1 == kGroups) {
            mma_commit(bar(B_SFULL + (s & 1)));
            if (last) mma_commit(bar(B_QEMPTY));
          }
        }
        __syncwarp();
      }
      if (!ok) break;
      if (pending && !second(s - 1, pend_n, pend_first, pend_last)) {
        ok = false;
        break;
      }
      pending = true;
      pend_first = first;
      pend_last = last;
      pend_n = n16;
      first = last;
      ++s;
      w.next();
      if (last && w.more()) {
        if (!__all_sync(0xffffffffu, wait(B_QEMPTY, uint32_t(qload - 1)))) {
          ok = false;
          break;
        }
        queries();
      }
    }
    if (ok && pending) ok = second(s - 1, pend_n, pend_first, pend_last);
    if (!ok && lane == 0) fail();
    mma_commit_warp(bar(B_FIN));
    (void)mbar_wait(bar(B_FIN), 0, nullptr, kWaitCycles);
    // after an abort, a box of queries may still be in flight
    if (*abort_flag) (void)mbar_wait(bar(B_QFULL), uint32_t(loads - 1) & 1u, nullptr, kDrainCycles);
    __syncwarp();
  } else {
    // ---- softmax and write-out
    const int half = warp >> 2, q4 = warp & 3;
    const int r = q4 * 16 + (lane & 15);        // S: row r of 64 sits in lane r % 16 of its quadrant
    const bool row_lane = lane < 16;
    const uint32_t lanes = tmem + (uint32_t(q4 * 32) << 16);
    float* mx = reinterpret_cast<float*>(gb + kOffMx);
    float* alpha_s = reinterpret_cast<float*>(gb + kOffAlpha);
    volatile uint64_t* valid_ring = reinterpret_cast<volatile uint64_t*>(gb + kOffValid);
    const bool raw_scores = p.scale_log2 > 0.f;
    const float sc = raw_scores ? p.scale_log2 : 1.f;
    bool ok = true, hidden_nonfinite = false;
    int s = 0, piece = 0;
    while (w.more() && ok) {
      // one piece: the tiles of this unit that lie in the run
      const int rows = w.rows();
      const bool row_ok = row_lane && r < rows;
      const int row0 = w.unit * kRows;
      const size_t grow = size_t(w.r.q0) * p.H + row0;   // row of out and lse
      const int pos = w.r.P + (row0 + (row_ok ? r : 0)) / p.H;
      const int first = window_first(p.window, pos);
      const int pos_a = w.r.P + row0 / p.H;              // first and last row's position
      const int first_z = window_first(p.window, w.t.k1 - 1);
      const bool starts = w.k == 0;
      const bool begins = w.g > w.begin(cta);            // (not the piece the run begins with)
      float m_ref = -INFINITY, l = 0.f;
      bool fresh = true, ends = false;
      for (bool more = true; more; ++s) {
        const int tk0 = w.key();
        more = !w.last_tile();
        ends = w.k + 1 == w.t.ntiles;
        w.next();
        // which of this row's 32 keys it sees, while the scores are on their way
        uint64_t vis = ~0ull;
        if (tk0 + kTile > pos_a + 1 || (tk0 < first_z && tk0 + kTile > p.sinks))
          vis = low_bits(pos + 1 - tk0) & (~low_bits(first - tk0) | low_bits(p.sinks - tk0));
        bool got = wait(B_VREADY + s % kValidRing, uint32_t(s / kValidRing));
        const uint32_t held = got ? uint32_t(valid_ring[s % kValidRing] >> (32 * half)) : 0u;
        const uint32_t v32 = row_ok ? uint32_t(vis >> (32 * half)) & held : 0u;
        const bool all_seen = __all_sync(0xffffffffu, v32 == 0xffffffffu || !row_lane);
        got = got && wait(B_SFULL + (s & 1), uint32_t(s >> 1));
        const bool wok = __all_sync(0xffffffffu, got);
        float x[32];
        float mth = -INFINITY;
        if (wok) {
          tc_fence_after();
          uint32_t sv[32];
          tmem_ld32(lanes + kTmemS + uint32_t(64 * (s & 1) + 32 * half), sv);
          tmem_wait_ld();
          tc_fence_before();
          mbar_arrive(bar(B_SEMPTY + (s & 1)));
          if (row_ok && held != v32) {
            // a hidden key whose score is not finite (see kFlagHiddenNonfinite)
#pragma unroll
            for (int c = 0; c < 32; ++c)
              hidden_nonfinite |= (((held & ~v32) >> c) & 1u) && (sv[c] & 0x7f800000u) == 0x7f800000u;
          }
          // With a positive scale (the usual case) the scores stay raw, their
          // maximum is scaled, and each exponent is one multiply-add; otherwise
          // they are scaled here.
          if (all_seen && raw_scores) {
#pragma unroll
            for (int c = 0; c < 32; ++c) x[c] = __uint_as_float(sv[c]);
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              x[c] = ((v32 >> c) & 1u) ? __uint_as_float(sv[c]) * (raw_scores ? 1.f : p.scale_log2)
                                       : -INFINITY;
          }
          float t4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int c = 4; c < 32; ++c) t4[c & 3] = fmaxf(t4[c & 3], x[c]);
          if (row_ok) mth = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * sc;
        }
        if (row_lane) mx[half * kRows + r] = mth;
        // One barrier per tile: the halves' maxima are in place, and whether any
        // row's reference moves (either half's maximum alone decides that).
        const bool calm = wok && !(mth > m_ref + kRescaleLog2);
        float alpha = 1.f;
        if (!named_sync_and(kSoftmaxBar, kSoftmax, calm)) {
          if (!named_sync_and(kSoftmaxBar, kSoftmax, wok)) {
            if (tid == 0) fail();
            ok = false;
            break;
          }
          const float mt = fmaxf(mx[r], mx[kRows + r]);
          if (row_lane && mt > m_ref + kRescaleLog2) {
            alpha = ex2_approx(m_ref - mt);   // 0 when nothing was seen before
            l *= alpha;
            m_ref = mt;
          }
          if (half == 0 && row_lane) alpha_s[r] = alpha;
          const bool pfree = s == 0 || wait(B_PFREE, uint32_t(s - 1));   // O is final
          if (!named_sync_and(kSoftmaxBar, kSoftmax, __all_sync(0xffffffffu, pfree))) {
            if (tid == 0) fail();
            ok = false;
            break;
          }
          if (!fresh) {
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {   // 32 rows (columns of O) of one of two blocks of values
              const uint32_t at = lanes + kTmemO + uint32_t(64 * (2 * half + (c >> 1)) + 32 * (c & 1));
              uint32_t v[32];
              tmem_ld32(at, v);
              tmem_wait_ld();
              const float* a = alpha_s + 32 * (c & 1);
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * a[e]);
              tmem_st32(at, v);
            }
            tmem_wait_st();
            tc_fence_before();
          }
        }
        // The probabilities round to bf16, the type of the values that they are
        // multiplied with; the row sum takes them unrounded, in 32 bits.  Each is off by
        // at most 2^-8 of itself, as the output's own rounding is; together they put the
        // output 1.75e-3 to 1.85e-3 of its norm from the 64-bit one, where rounding that
        // alone makes 1.66e-3.
        const float mr = m_ref == -INFINITY ? 0.f : m_ref;
        uint32_t pk[16];
        float lt = 0.f;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float a = ex2_approx(fmaf(x[2 * c], sc, -mr)), b = ex2_approx(fmaf(x[2 * c + 1], sc, -mr));
          lt += a + b;
          const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
          pk[c] = *reinterpret_cast<const uint32_t*>(&h);
        }
        l += lt;
        // P's buffer is free once the tile before has been multiplied (should
        // this wait give up, the next tile's end the piece for everyone)
        if (s > 0 && !wait(B_PFREE, uint32_t(s - 1))) fail();
        fresh = false;
        // this row's 32 keys (K-major, 128-byte swizzle)
        if (row_lane) {
          uint8_t* prow = gb + kOffP + r * 128;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4*>(prow + (((4 * half + j) ^ (r & 7)) * 16)) =
                make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
        }
        fence_proxy_async_cta();   // P, read by the tensor core
        mbar_arrive(bar(B_PFULL));
      }
      if (!ok) break;
      // the piece's row sums, lse and normalised rows
      if (row_lane) mx[half * kRows + r] = l;
      named_sync(kSoftmaxBar, kSoftmax);
      const bool direct = starts && ends;
      const size_t slot = size_t(2 * cta + (begins ? 1 : 0));
      if (half == 0 && row_lane) {
        const float lt = mx[r] + mx[kRows + r];
        const float lse = lt == 0.f ? -INFINITY : (m_ref + log2f(lt)) * kLn2;
        alpha_s[r] = lt == 0.f ? 0.f : 1.f / lt;
        if (row_ok) {
          if (direct) p.lse[grow + r] = lse;
          else p.part_lse[slot * kRows + r] = lse;
        }
      }
      const bool fin = wait(B_OFULL, uint32_t(piece));
      if (!named_sync_and(kSoftmaxBar, kSoftmax, __all_sync(0xffffffffu, fin))) {
        if (tid == 0) fail();
        ok = false;
        break;
      }
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        const int block = 2 * half + (c >> 1), rr0 = 32 * (c & 1);
        if (rr0 >= rows) continue;
        uint32_t v[32];
        tmem_ld32(lanes + kTmemO + uint32_t(64 * block + rr0), v);
        tmem_wait_ld();
        const int col = 128 * block + 32 * q4 + lane;
        const float* inv = alpha_s + rr0;
        if (direct) {
          // two rows at a time: lanes pair up, the even one stores the first
          // row's two columns, the odd one the second's
          __nv_bfloat16* dst = p.out + (grow + rr0 + (lane & 1)) * kDv + (col & ~1);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float a = __uint_as_float(v[e]) * inv[e], b = __uint_as_float(v[e + 1]) * inv[e + 1];
            const float give = lane & 1 ? a : b;
            const float take = __shfl_xor_sync(0xffffffffu, give, 1);
            const __nv_bfloat162 h = lane & 1 ? __floats2bfloat162_rn(take, b)
                                              : __floats2bfloat162_rn(a, take);
            if (rr0 + e + (lane & 1) < rows)
              *reinterpret_cast<__nv_bfloat162*>(dst + size_t(e) * kDv) = h;
          }
        } else {
          float* dst = p.part_o + (slot * kRows + rr0) * kDv + col;
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (rr0 + e < rows) dst[size_t(e) * kDv] = __uint_as_float(v[e]) * inv[e];
        }
      }
      tc_fence_before();
      mbar_arrive(bar(B_OFREE));
      ++piece;
      named_sync(kSoftmaxBar, kSoftmax);   // alpha_s has been read
    }
    if (hidden_nonfinite) atomicOr(cta_flags, kFlagHiddenNonfinite);
  }

  tc_fence_before();
  __syncthreads();
  if (tid == 0) p.cta_flags[cta] = *cta_flags;
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Rows of 576 features as column blocks of 64: a box of 64 rows x `blocks`.
bool encode(CUtensorMap* m, const __nv_bfloat16* base, int64_t rows, int64_t stride, int blocks) {
  cuuint64_t dims[3] = {64u, cuuint64_t(rows), cuuint64_t(kBlocks)};
  cuuint64_t strides[2] = {cuuint64_t(stride) * 2u, 128u};
  cuuint32_t box[3] = {64u, 64u, uint32_t(blocks)};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16*>(base), dims,
                  strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t init_decode_tc() {
  return cudaFuncSetAttribute(decode_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              int(kSmemBytes));
}

cudaError_t launch_decode_tc(const ChunkTcParams& p, int ctas, cudaStream_t st) {
  CUtensorMap tk, tq;
  memset(&tk, 0, sizeof tk);
  memset(&tq, 0, sizeof tq);
  if (!g_encode || !encode(&tq, p.q, int64_t(p.total_q) * p.H, kDqk, kBlocks)) return cudaErrorNotSupported;
  if (p.kv_start && !encode(&tk, p.kv, p.num_slots, p.kv_stride, kBlocks / kGroups)) return cudaErrorNotSupported;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(unsigned(ctas), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_tc_kernel, p, tk, tq);
}

}  // namespace va
