// va_prefill_tc.cu -- chunk attention of many rows per request (pieces of
// prompts) on the tcgen05 tensor cores, persistent.
//
// The mathematics and the division of labour are the split kernel's
// (va_tc.cu): a unit is 256 query rows on a cluster of four, S = Q K^T on two
// SMs (rank 0, 1: M = 256 over both, queries in tensor memory, keys from shared
// memory), O += P V on the other two (rank 2, 3: O fills their tensor memory), P
// crosses over distributed shared memory.  Bound by the tensor cores, with two
// products of unequal width sharing the work.  What many units change:
//
//  - A cluster does not end with its unit.  The tiles of all units form one row of
//    steps, every cluster takes an equal run of it, and the roles walk the run
//    without meeting at unit ends: while the PV SMs multiply a unit's last tiles
//    and write its rows out, the QK SMs load the next unit's queries and go on.
//    (One unit per cluster launch costs about 11 us besides its tiles, as much as
//    a dozen of them: a prompt of 1500 tokens spent half its time there, and a
//    last, partly filled wave of clusters on top.)  A unit cut by run ends leaves
//    an fp32 partial per piece for the merge (va_chunk.cu), a whole one goes
//    straight to out and lse.
//  - Keys lie side by side (contiguous pools, or paged lists packed first), so
//    everything arrives by TMA boxes from one thread per SM.  The boxes of a pair
//    complete on the barrier of the SM that issues the products, for both.  A
//    request's last, partial tile comes from a copy with zeros behind it, so that
//    nothing that follows a request in memory enters a product.
//  - The QK SMs' ring holds five slots of 36 KB: a slot takes an SM's 32 keys of a
//    tile, or a quarter of its 128 query rows, which pass through the ring like
//    tiles on their way to tensor memory.
//  - The two softmax warpgroups take alternate tiles, a thread a row of 64 keys, so
//    a tile's scores, exponentials and probabilities have two tiles' time.  Only the
//    row's reference maximum goes from tile to tile.  (Sharing every tile, 32 keys a
//    thread, a tile's chain of load, maximum, barrier, exponentials and hand-over
//    took 1600 cycles, longer than its products.)  And one thread issues a tile's
//    products in one go: with an election per product they went out every 37 to 41
//    cycles, where the tensor cores need 32.  Either change alone gained 0 to 4%,
//    both 15%.
//
// A request of 512 tokens, 64 heads, with 16k keys in front: 780 us, 78% of the
// cuBLAS rate; per tile about 1590 cycles, of which the QK SMs' tensor cores work
// 1152.
//
// Every wait is bounded; a role that gives up sets VA_STATUS_TIMEOUT and its CTA
// drains its copies and products before it leaves.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <string.h>

#include "va_chunk.cuh"
#include "va_sm100.cuh"

namespace va {

extern PFN_cuTensorMapEncodeTiled_v12000 g_encode;   // va_tc.cu, resolved by va_init

namespace {

using namespace sm100;

constexpr int kThreads = 384;          // warps: 0 boxes, 1 products, 2 P copies, 4-11 rows
constexpr int kCtas = 4;
constexpr int kRows = 128;             // of a CTA; a unit has two CTAs' worth
constexpr int kUnitRows = 2 * kRows;
constexpr int kTile = 64, kBlocks = kDqk / 64;
constexpr int kSlotRows = 32;          // keys (or query rows) of a ring slot
constexpr uint32_t kBlockBytes = kSlotRows * 128u;
constexpr uint32_t kSlotBytes = kBlocks * kBlockBytes;      // 36 KB
constexpr int kRing = 5;
constexpr int kQSlots = kRows / kSlotRows;
constexpr uint32_t kVBlock = kTile * 128u;                  // 64 keys x 64 value columns
constexpr uint32_t kVTileBytes = 4 * kVBlock;               // a CTA's four blocks of a tile
constexpr int kVRing = 4;
// P buffer: 128 rows x 64 keys bf16 (K-major, 128-byte swizzle), the rows'
// rescale factors, four warps' flags; one bulk copy to the PV CTA.
constexpr uint32_t kPBytes = kRows * 128;
constexpr uint32_t kPAlpha = kPBytes, kPFlags = kPAlpha + 4 * kRows, kPPayload = kPFlags + 16;
constexpr uint32_t kPBufBytes = 17 * 1024;
constexpr int kPBufs = 3;
// Row sums of units on their way to the PV CTA.  When a tile has been staged, the
// product of the tile kPBufs + 2 before it is done (two staging buffers, kPBufs at
// the PV CTA), and the sums of the unit before that one's have been read: with
// units of one tile those of kPBufs + 2 more may wait, besides the new ones.
constexpr int kFinRing = kPBufs + 3;
constexpr int kSoftmax = 256;          // warps 4-11
constexpr uint32_t kRowBar = 1;        // their named barrier
constexpr uint32_t kCmdDone = 0xFFFFFFFFu, kCmdUnit = 0x80000000u;
constexpr uint32_t kTmemCols = 512, kTmemQ = 0, kTmemS = 320;
constexpr uint16_t kQkMask = 0x3, kPvMask = 0xC;
constexpr long long kWaitCycles = 4000000000ll;   // wait bound in SM cycles (~2 s)
constexpr long long kDrainCycles = 2000000ll;     // after an abort: boxes in flight land
constexpr float kRescaleLog2 = 8.f;

// What a unit costs besides its tiles, in tiles: queries into tensor memory, the
// pipeline's fill, rows out of it: about 8000 cycles, and a tile takes 1590.  (Three
// prompts of 517 to 2047 tokens: 4 494 us, 5 461, 6 451, 7 458, 9 472.)
constexpr int kUnitCost = 6;
using Run = ChunkRun<kUnitRows, kUnitCost>;

// Barriers: one layout in all four CTAs, QK and PV sides side by side.
// (Keys and queries land on barriers of their own although they share the slots:
// an odd rank that is ahead may have its keys on the way into a slot whose
// queries the even rank is still waiting for.)
constexpr int B_KFULL = 0;                     // [kRing] QK, even rank: both CTAs' keys in a slot
constexpr int B_QFULL = B_KFULL + kRing;       // [kQSlots] QK: a quarter of the CTA's queries
constexpr int B_EMPTY = B_QFULL + kQSlots;     // [kRing] QK: slot read
constexpr int B_SFULL = B_EMPTY + kRing;       // [2]
constexpr int B_SEMPTY = B_SFULL + 2;          // [2]
constexpr int B_QREADY = B_SEMPTY + 2;         // a unit's queries in tensor memory
constexpr int B_QREADYP = B_QREADY + 1;        // ... the odd rank's
constexpr int B_PFREE = B_QREADYP + 1;         // [kPBufs] QK; committed by PV
constexpr int B_VFULL = B_PFREE + kPBufs;      // [kVRing] PV, even rank
constexpr int B_VEMPTY = B_VFULL + kVRing;     // [kVRing] PV
constexpr int B_PFULL = B_VEMPTY + kVRing;     // [kPBufs] PV; bulk copies from QK
constexpr int B_PFULLP = B_PFULL + kPBufs;     // [kPBufs] PV, even rank: the odd rank's
constexpr int B_OGO = B_PFULLP + kPBufs;       // PV: a command for the row warps
constexpr int B_OCORR = B_OGO + 1;             // PV: rows rescaled
constexpr int B_ODONE = B_OCORR + 1;           // PV: products before a rescale done
constexpr int B_OFULL = B_ODONE + 1;           // PV: a unit's products done
constexpr int B_OFREE = B_OFULL + 1;           // PV: its O has been read
constexpr int B_FIN = B_OFREE + 1;             // [kFinRing] PV: row sums from QK
constexpr int B_STGFULL = B_FIN + kFinRing;    // [2] QK: a P staging buffer written
constexpr int B_STGFREE = B_STGFULL + 2;       // [2] QK: read by its copy
constexpr int B_REF = B_STGFREE + 2;           // [2][4] QK: a tile's references, by quadrant
constexpr int B_MMAFIN = B_REF + 8;
constexpr int kNumBars = B_MMAFIN + 1;

// Shared layout (offsets from a 1024-byte aligned base).
constexpr uint32_t kOffTmemSlot = 512, kOffAbort = 516, kOffCmd = 520, kOffFlags = 524;
constexpr uint32_t kOffRun = 544;              // RunPlace
constexpr uint32_t kOffPeerAny = 640;          // PV, even rank: uint32 [kPBufs]
constexpr uint32_t kOffRef = 1024;             // QK: float [2][128] reference maxima, by tile parity
constexpr uint32_t kOffSum = 2048;             // QK: float [2][2][128] partial sums, their references
constexpr uint32_t kOffFin = 1024;             // PV: float [kFinRing][128] 1 / row sum
constexpr uint32_t kOffK = 4096;               // QK: ring
constexpr uint32_t kOffStage = kOffK + kRing * kSlotBytes;   // QK: P staging [2]
constexpr uint32_t kOffP = 4096;               // PV: P buffers
constexpr uint32_t kOffV = kOffP + kPBufs * kPBufBytes;
constexpr uint32_t kOffOut = kOffV + kVRing * kVTileBytes;   // PV: write-out staging
constexpr uint32_t kOutRow = 128 + 16;         // a row's 128 bytes, padded over the banks
constexpr uint32_t kEndQK = kOffStage + 2 * kPBufBytes;
constexpr uint32_t kEndPV = kOffOut + 8 * 32 * kOutRow;
constexpr uint32_t kSmemBytes = (kEndQK > kEndPV ? kEndQK : kEndPV) + 1024;
static_assert(8 * kNumBars <= int(kOffTmemSlot), "barrier area");
static_assert(kOffFin + kFinRing * kRows * 4 <= kOffP, "row sums");
static_assert(kOffStage % 1024 == 0 && kOffV % 1024 == 0 && kSmemBytes <= 232448, "layout");

struct RunPlace {
  int64_t g, end, total;
  int b, unit, unit0, k, runs;
};
static_assert(kOffRun + sizeof(RunPlace) <= kOffPeerAny, "header");

// Two probabilities as the second product takes them, in bf16 like the values; the row
// sum takes them unrounded, in 32 bits.  Each is off by at most 2^-8 of itself, as the
// output's own rounding is; together they put the output 1.8e-3 to 2.2e-3 of its norm from
// the 64-bit one, where rounding that alone makes 1.66e-3.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b, float& sum) {
  sum += a + b;
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

struct Maps {
  CUtensorMap k, v, kt, vt, q;   // keys and values; of the tails; queries
};

// Where the tile of the step lies: rows of the keys' map, or of the tails' (the
// request's last, partial tile), or past the end (zeros) where the list has none.
struct TileAt {
  int row;
  bool tail;
};
__device__ __forceinline__ TileAt tile_at(const ChunkTcParams& p, const Run& w) {
  const int tk0 = w.key();
  const int N = w.r.nlist < w.r.P + w.r.n ? w.r.nlist : w.r.P + w.r.n;
  const int64_t rows = p.packed ? p.num_entries : p.num_slots;
  const int64_t row = w.r.base + tk0;
  TileAt t;
  t.tail = tk0 < N && tk0 + kTile > N;
  t.row = t.tail ? w.b * kTile : int(tk0 >= N || row < -kTile || row > rows ? rows : row);
  return t;
}

// Tiles of the rest of a run.
__device__ int64_t tiles_of(Run w) {
  int64_t n = 0;
  for (; w.more(); w.next_piece()) n += w.piece();
  return n;
}

__global__ void __launch_bounds__(kThreads, 1)
    prefill_tc_kernel(const __grid_constant__ ChunkTcParams p, const __grid_constant__ Maps maps) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sb = (raw + 1023u) & ~1023u;
  uint8_t* gb = smem_raw + (sb - raw);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gb + kOffAbort);
  uint32_t* cta_flags = reinterpret_cast<uint32_t*>(gb + kOffFlags);
  auto bar = [&](int i) -> uint32_t { return sb + 8u * uint32_t(i); };
  // waits for a phase by its number (from 0); the second kind for barriers that
  // another CTA completes
  auto wait = [&](int i, int phase) -> bool {
    return mbar_wait(bar(i), uint32_t(phase) & 1u, abort_flag, kWaitCycles);
  };
  auto wait_far = [&](int i, int phase) -> bool {
    return mbar_wait<true>(bar(i), uint32_t(phase) & 1u, abort_flag, kWaitCycles);
  };
  auto fail = [&]() {
    *abort_flag = 1;
    atomicOr(cta_flags, VA_STATUS_TIMEOUT);
  };
  const uint32_t rank = cluster_ctarank();
  const bool qk = rank < 2u, even = (rank & 1u) == 0u;
  const int hh = int(rank & 1u);               // which 128 rows of the unit
  const uint32_t lead = rank & 2u, mate = rank ^ 1u, other = rank ^ 2u;
  const int cluster = int(blockIdx.x) / kCtas;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    tma_prefetch(qk ? &maps.k : &maps.v);
    tma_prefetch(qk ? &maps.kt : &maps.vt);
    if (qk) tma_prefetch(&maps.q);
  }
  if (tid == 32) {
    for (int i = 0; i < kNumBars; ++i) {
      uint32_t cnt = 1;
      // the odd rank's eight row warps add one arrival each
      if (i == B_OCORR || i == B_OFREE) cnt = kSoftmax + kSoftmax / 32;
      // a tile's four softmax warps, of both CTAs of the pair or of one
      if (i == B_SEMPTY || i == B_SEMPTY + 1) cnt = 8;
      if (i == B_STGFULL || i == B_STGFULL + 1) cnt = 4;
      if (i == B_QREADY) cnt = kSoftmax;
      if (i == B_QREADYP) cnt = kSoftmax / 32;
      if (i >= B_FIN && i < B_FIN + kFinRing) cnt = 4;   // the first four row warps
      mbar_init(bar(i), cnt);
    }
    *abort_flag = 0;
    *cta_flags = 0u;
    fence_mbar_init();
  }
  griddep_wait();                // the stream's previous kernel has completed
  griddep_launch_dependents();   // the merge may start its set-up
  RunPlace* place = reinterpret_cast<RunPlace*>(gb + kOffRun);
  Run w(p);
  if (warp == 0) {
    const int units = find_run(w, cluster, int(gridDim.x) / kCtas, lane);
    if (lane == 0) {
      *place = RunPlace{w.g, w.end, w.total, w.b, w.unit, w.unit0, w.k, w.runs};
      if (blockIdx.x == 0) {
        p.totals[0] = units;
        p.totals[1] = int(gridDim.x) / kCtas;
      }
    }
  }
  __syncthreads();
  if (place->g >= place->end) {   // every CTA of the cluster leaves together
    if (tid == 0) p.cta_flags[blockIdx.x] = 0u;
    return;
  }
  if (warp != 0) {
    w.load(place->b);
    w.unit = place->unit;
    w.tiles();
    w.unit0 = place->unit0;
    w.k = place->k;
    w.g = place->g;
    w.end = place->end;
    w.total = place->total;
    w.runs = place->runs;
  }
  if (warp == 2) tmem_alloc_pair(sb + kOffTmemSlot, kTmemCols);
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gb + kOffTmemSlot);
  const int half = (warp - 4) >> 2, q4 = warp & 3;   // row warps: column half, lane quadrant

  if (qk) {
    // ================================================================ QK CTA
    if (warp == 0) {
      // ---- boxes: a unit's queries in four quarters, then its keys' tiles
      if (lane == 0) {
        bool ok = true;
        int f = 0;   // ring entry
        bool first = true;
        const uint32_t lead_full = mapa(bar(B_KFULL), lead);
        for (; ok && w.more(); w.next()) {
          if (first) {
            const int row = w.r.q0 * p.H + w.unit * kUnitRows + hh * kRows;
            for (int i = 0; ok && i < kQSlots; ++i, ++f) {
              const int s = f % kRing;
              ok = f < kRing || wait(B_EMPTY + s, f / kRing - 1);
              if (!ok) break;
              mbar_arrive_expect_tx(bar(B_QFULL + i), kSlotBytes);
              tma_load_3d(sb + kOffK + uint32_t(s) * kSlotBytes, &maps.q, 0, row + kSlotRows * i, 0,
                          bar(B_QFULL + i));
            }
            if (even && w.k == 0) {   // the unit's entry, for the merge
              ChunkUnit u;
              u.row0 = w.r.q0 * p.H + w.unit * kUnitRows;
              u.rows = w.rows();
              u.ns = w.owner(w.g + w.t.ntiles - 1) - cluster + 1;
              // slots 2c: the piece a run begins with; 2c + 1: a piece begun later
              u.pslot = 2 * cluster + (w.g > w.begin(cluster) ? 1 : 0);
              u.pslot1 = 2 * (cluster + 1);
              u.pstride = 2;
              u.item = cluster;
              u.istride = 1;
              u.b = w.b;
              u.i0 = w.unit * kUnitRows;
              p.units[w.unit0 + w.unit] = u;
            }
          }
          first = w.last_tile();
          if (!ok) break;
          const int s = f % kRing;
          ok = f < kRing || wait(B_EMPTY + s, f / kRing - 1);
          if (!ok) break;
          // both CTAs' keys land on the even rank's barrier
          if (even) mbar_arrive_expect_tx(bar(B_KFULL + s), 2 * kSlotBytes);
          const TileAt t = tile_at(p, w);
          tma_load_3d_pair(sb + kOffK + uint32_t(s) * kSlotBytes, t.tail ? &maps.kt : &maps.k, 0,
                           t.row + kSlotRows * hh, 0, lead_full + 8u * uint32_t(s));
          ++f;
        }
        if (!ok) fail();
        (void)mbar_wait(bar(B_MMAFIN), 0, nullptr, kWaitCycles);
        if (*abort_flag)
          for (const long long t0 = clock64(); clock64() - t0 < kDrainCycles;) {}
      }
      __syncwarp();
    } else if (warp == 1) {
      // ---- products S[T % 2] = Q K^T, issued by the even rank for both
      if (even) {
        constexpr uint32_t idesc = idesc_bf16(kUnitRows, kTile, 0, 0);
        bool ok = true;
        int f = 0, u = 0, n = 0;   // ring entry, unit, tiles left of the unit's piece
        uint32_t kphase = 0;       // bit s: parity of slot s's next keys
        for (int T = 0; n > 0 || w.more(); ++T, ++f, --n) {
          bool got = true;
          if (n == 0) {
            n = w.piece();
            w.next_piece();
            got = wait(B_QREADY, u) && wait_far(B_QREADYP, u);
            ++u;
            f += kQSlots;
          }
          const int s = f % kRing, bs = T & 1;
          got = got && wait_far(B_KFULL + s, int(kphase >> s & 1u)) &&
                (T < 2 || wait_far(B_SEMPTY + bs, (T >> 1) - 1));
          if (!__all_sync(0xffffffffu, got)) {
            ok = false;
            break;
          }
          kphase ^= 1u << s;
          fence_proxy_async_cta();
          tc_fence_after();
          const uint32_t d = tmem + kTmemS + 64u * uint32_t(bs);
          const uint64_t b0 = smem_desc(sb + kOffK + uint32_t(s) * kSlotBytes, 16, 1024, kSwizzle128B);
          if (elect_one()) {
#pragma unroll
            for (int c = 0; c < kBlocks; ++c)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma2_ts(d, tmem + kTmemQ + 8u * uint32_t(4 * c + kk),
                        b0 + uint64_t((uint32_t(c) * kBlockBytes + uint32_t(kk) * 32u) >> 4), idesc,
                        (c | kk) != 0 ? 1u : 0u);
            mma2_commit_mc(bar(B_SFULL + bs), kQkMask);
            mma2_commit_mc(bar(B_EMPTY + s), kQkMask);
          }
          __syncwarp();
        }
        if (!ok && lane == 0) fail();
        mma2_commit_mc_warp(bar(B_MMAFIN), kQkMask);
      }
      // products read both CTAs' memories until their last commit
      (void)mbar_wait<true>(bar(B_MMAFIN), 0, nullptr, kWaitCycles);
      __syncwarp();
    } else if (warp == 2) {
      // ---- P to the PV CTA of the same rows, a copy per tile
      if (lane == 0) {
        const uint32_t pv_p = mapa(sb + kOffP, other), pv_pfull = mapa(bar(B_PFULL), other);
        const int64_t steps = tiles_of(w);
        bool ok = true;
        int T = 0;
        for (; T < steps; ++T) {
          const int bs = T & 1, pb = T % kPBufs;
          ok = wait(B_STGFULL + bs, T >> 1) && (T < kPBufs || wait_far(B_PFREE + pb, T / kPBufs - 1));
          if (!ok) break;
          bulk_copy_to_cluster(pv_p + uint32_t(pb) * kPBufBytes,
                               sb + kOffStage + uint32_t(bs) * kPBufBytes, kPPayload,
                               pv_pfull + 8u * uint32_t(pb));
          bulk_commit();
          bulk_wait_read<0>();
          mbar_arrive(bar(B_STGFREE + bs));
        }
        // the PV CTAs' last releases land before this shared memory goes away
        for (int t = T > kPBufs ? T - kPBufs : 0; ok && t < T; ++t)
          ok = wait_far(B_PFREE + t % kPBufs, t / kPBufs);
        if (!ok) fail();
      }
      __syncwarp();
    } else if (warp >= 4) {
      // ---- softmax: the warpgroups take alternate tiles, a thread a row's 64
      // keys.  A row's reference maximum goes from tile to tile, so from warp to warp
      // of a quadrant, through shared memory; everything else of a tile -- its
      // scores, exponentials and probabilities -- has two tiles' time.  Each
      // warpgroup keeps its own part of a row's sum, to the reference of its last
      // tile.
      const int wg = half;
      const int r = q4 * 32 + lane;
      const uint32_t tl = tmem + (uint32_t(q4 * 32) << 16);
      float* ref_s = reinterpret_cast<float*>(gb + kOffRef);
      float* sum_s = reinterpret_cast<float*>(gb + kOffSum);
      const uint32_t pv_fin = mapa(sb + kOffFin, other);
      const uint32_t pv_finbar = mapa(bar(B_FIN), other);
      const uint32_t sempty_lead = mapa(bar(B_SEMPTY), lead);
      const uint32_t qready_lead = mapa(bar(B_QREADYP), lead);
      const bool raw_scores = p.scale_log2 > 0.f;
      const float sc = raw_scores ? p.scale_log2 : 1.f;
      bool ok = true, hidden_nonfinite = false, bad_slot = false;
      int T = 0, f = 0;
      int last_b = -1;          // request of the piece before,
      bool all_valid = false;   // and whether every key of it has a row
      for (int u = 0; w.more(); ++u) {
        // one piece: the tiles of this unit that lie in the run
        const int rows = w.rows() - hh * kRows;            // of this CTA
        const bool row_ok = r < rows;
        const int ur = w.unit * kUnitRows + hh * kRows;    // first row within the request
        const size_t grow = size_t(w.r.q0) * p.H + ur;
        const int pos = w.r.P + (ur + (row_ok ? r : 0)) / p.H;
        const int first = window_first(p.window, pos);
        const int pos_a = w.r.P + w.unit * kUnitRows / p.H;   // the unit's first position
        const int first_z = window_first(p.window, w.t.k1 - 1);
        const int64_t base = w.r.base;
        const int k1 = w.t.k1, first_a = w.t.first;
        const int N = w.r.nlist < w.r.P + w.r.n ? w.r.nlist : w.r.P + w.r.n;
        const bool direct = w.k == 0 && w.piece() == w.t.ntiles;
        const size_t slot = size_t(2 * cluster + (w.g > w.begin(cluster) ? 1 : 0));
        bad_slot |= k1 > N;   // the list ends before the unit's last token's own key
        if (w.b != last_b) {
          last_b = w.b;
          bool all = true;
          if (p.valid) {   // any key of the blocks that the list touches without one
            for (int64_t k = base / 256 + (tid - 128); k * 256 < base + N; k += kSoftmax)
              all = all && !(p.pack_flags[k] & kPackMissing);
          } else {
            all = base >= 0 && base + N <= p.num_slots;
          }
          all_valid = named_sync_and(kRowBar, kSoftmax, all);
        }
        // The unit's queries: this warp's quarter of the rows, column blocks 0-4
        // or 5-8, into tensor memory, once the products of the unit before are done
        // (its last scores are complete).
        {
          const int s = (f + q4) % kRing;
          const bool got = __all_sync(
              0xffffffffu, wait(B_QFULL + q4, u) &&
                               (T == 0 || wait(B_SFULL + ((T - 1) & 1), (T - 1) >> 1)));
          if (got) {
            tc_fence_after();
            const uint32_t row_addr = sb + kOffK + uint32_t(s) * kSlotBytes + uint32_t(lane) * 128u;
#pragma unroll 1
            for (int c = half ? 5 : 0; c < (half ? 9 : 5); ++c) {
              uint32_t v[32];
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const uint4 x = ld_shared_v4(row_addr + uint32_t(c) * kBlockBytes +
                                             uint32_t((j ^ (lane & 7)) * 16));
                v[4 * j] = x.x; v[4 * j + 1] = x.y; v[4 * j + 2] = x.z; v[4 * j + 3] = x.w;
              }
              tmem_st32(tl + kTmemQ + 32u * uint32_t(c), v);
            }
          }
          tmem_wait_st();
          tc_fence_before();
          if (!named_sync_and(kRowBar, kSoftmax, got)) {
            if (tid == 128) fail();
            break;
          }
          if (tid == 128)
            for (int i = 0; i < kQSlots; ++i) mbar_arrive(bar(B_EMPTY + (f + i) % kRing));
          if (even) {
            mbar_arrive(bar(B_QREADY));
          } else {
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(qready_lead);
          }
          f += kQSlots;
        }
        float m_ref = -INFINITY, l = 0.f;   // of this warpgroup's last tile
        ChunkTiles tiles = w.t;   // (the tile's index is all that moves)
        const int n = w.piece();
        tiles.t0 = w.k;
        w.next_piece();
        // Tiles that lie inside for every row of the unit, with a row behind every
        // key: [0, in_a) among the sinks and [in_b, in_c) of the window (counted from
        // the piece's first).
        int in_a = 0, in_b = 0, in_c = 0;
        if (all_valid) {
          // tiles of the list that all rows reach (a list may end before their own keys)
          const int seen = (pos_a + 1 < N ? pos_a + 1 : N) / kTile;
          const int whole = p.sinks / kTile < seen ? p.sinks / kTile : seen;
          in_a = (tiles.nst < whole ? tiles.nst : whole) - tiles.t0;
          // list tile x >= wt is the unit's tile x - wt + nst
          const int from = (first_z + kTile - 1) / kTile;
          in_b = (from > tiles.wt ? from : tiles.wt) - tiles.wt + tiles.nst - tiles.t0;
          in_c = seen - tiles.wt + tiles.nst - tiles.t0;
        }
        // (after a wait gave up a warp goes on to the unit's end, where all agree)
        for (int i = (T & 1) == wg ? 0 : 1; ok && i < n; i += 2) {
          const int t = T + i, bs = wg;
          const bool inside = i < in_a || (i >= in_b && i < in_c);
          uint64_t v64 = ~0ull;   // which of the tile's 64 keys this row sees
          if (!inside) {
            const int tk0 = tiles.tile_key(i);
            uint64_t valid = 0ull;
            if (p.valid) {
              const int c = N - tk0;   // of them in the list
              const int64_t e = base + tk0;
              if (c > 0) {
                const uint32_t* v = p.valid + (e >> 5);
                const uint32_t x0 = __ldg(v), x1 = __ldg(v + 1), x2 = __ldg(v + 2);
                valid = (uint64_t(__funnelshift_r(x1, x2, uint32_t(e) & 31u)) << 32 |
                         __funnelshift_r(x0, x1, uint32_t(e) & 31u)) & low_bits(c);
              }
            } else {
              const int64_t a = base + tk0;   // pool row of the first
              const int64_t lo = -a, hi = p.num_slots - a;
              valid = low_bits(hi > 64 ? 64 : int(hi < 0 ? 0 : hi)) &
                      ~low_bits(lo > 64 ? 64 : int(lo < 0 ? 0 : lo));
              const uint64_t seen =
                  low_bits(k1 - tk0) & (~low_bits(first_a - tk0) | low_bits(p.sinks - tk0));
              bad_slot |= (seen & ~valid) != 0ull;
            }
            const uint64_t vis =
                low_bits(pos + 1 - tk0) & (~low_bits(first - tk0) | low_bits(p.sinks - tk0));
            v64 = vis & valid;
          }
          ok = __all_sync(0xffffffffu, wait(B_SFULL + bs, t >> 1));
          if (!ok) break;
          float x[64];
          tc_fence_after();
          {
            uint32_t a[32], b[32];
            tmem_ld32(tl + kTmemS + 64u * uint32_t(bs), a);
            tmem_ld32(tl + kTmemS + 64u * uint32_t(bs) + 32u, b);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              x[c] = __uint_as_float(a[c]);
              x[32 + c] = __uint_as_float(b[c]);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (even) mbar_arrive(bar(B_SEMPTY + bs));
            else mbar_arrive_remote_relaxed(sempty_lead + 8u * uint32_t(bs));
          }
          // With a positive scale (the usual case) the scores stay raw, their
          // maximum is scaled, and each exponent is one multiply-add.
          if (v64 != ~0ull || !raw_scores) {
            if (row_ok) {
              // a hidden key whose score is not finite (see kFlagHiddenNonfinite)
#pragma unroll
              for (int c = 0; c < 64; ++c)
                hidden_nonfinite |= !((v64 >> c) & 1ull) &&
                                    (__float_as_uint(x[c]) & 0x7f800000u) == 0x7f800000u;
            }
#pragma unroll
            for (int c = 0; c < 64; ++c)
              x[c] = ((v64 >> c) & 1ull) ? x[c] * (raw_scores ? 1.f : p.scale_log2) : -INFINITY;
          }
          float t4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int c = 4; c < 64; ++c) t4[c & 3] = fmaxf(t4[c & 3], x[c]);
          // (a row past the unit's is not written, and must not move anything)
          const float mt =
              row_ok ? fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * sc : -INFINITY;
          // the reference of the tile before, and on to the tile after
          float before = -INFINITY;
          if (i > 0) {
            if (!wait(B_REF + 4 * (bs ^ 1) + q4, (t - 1) >> 1)) fail();
            before = ref_s[(bs ^ 1) * kRows + r];
          }
          float now = before, alpha = 1.f;
          if (mt > before + kRescaleLog2) {
            now = mt;
            alpha = ex2_approx(before - mt);   // 0 when nothing was seen before
          }
          ref_s[bs * kRows + r] = now;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_REF + 4 * bs + q4));
          if (now != m_ref) {
            l *= ex2_approx(m_ref - now);   // (NaN stays)
            m_ref = now;
          }
          const float mr = now == -INFINITY ? 0.f : now;
          // the copy two tiles back has read the staging buffer
          if (t >= 2 && !wait(B_STGFREE + bs, (t >> 1) - 1)) fail();
          uint8_t* stg = gb + kOffStage + uint32_t(bs) * kPBufBytes;
          float lt = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint32_t pk[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
              pk[c] = pack_bf16(ex2_approx(fmaf(x[8 * j + 2 * c], sc, -mr)),
                                ex2_approx(fmaf(x[8 * j + 2 * c + 1], sc, -mr)), lt);
            *reinterpret_cast<uint4*>(stg + r * 128 + ((j ^ (r & 7)) * 16)) =
                make_uint4(pk[0], pk[1], pk[2], pk[3]);
          }
          l += lt;
          reinterpret_cast<float*>(stg + kPAlpha)[r] = alpha;
          const uint32_t moved = __ballot_sync(0xffffffffu, alpha != 1.f);
          if (lane == 0) reinterpret_cast<uint32_t*>(stg + kPFlags)[q4] = moved ? 1u : 0u;
          fence_proxy_async_cta();   // staging writes, read by the bulk copy
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_STGFULL + bs));
        }
        T += n;
        f += n;
        // row sums: the two warpgroups' parts, to the unit's last reference
        sum_s[wg * kRows + r] = l;
        sum_s[(2 + wg) * kRows + r] = m_ref;
        if (!named_sync_and(kRowBar, kSoftmax, ok)) {
          if (tid == 128) fail();
          break;
        }
        if (wg == 0) {
          const float l1 = sum_s[kRows + r], m1 = sum_s[3 * kRows + r];
          const float m = fmaxf(m_ref, m1);
          float lt = 0.f;
          if (m_ref != -INFINITY || l != 0.f) lt += l * ex2_approx(m_ref - m);
          if (m1 != -INFINITY || l1 != 0.f) lt += l1 * ex2_approx(m1 - m);
          const float lse = lt == 0.f ? -INFINITY : (m + log2f(lt)) * kLn2;
          if (row_ok) {
            if (direct) p.lse[grow + r] = lse;
            else p.part_lse[slot * kUnitRows + hh * kRows + r] = lse;
          }
          st_cluster_f32(pv_fin + uint32_t((u % kFinRing) * kRows + r) * 4u, lt == 0.f ? 0.f : 1.f / lt);
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(pv_finbar + 8u * uint32_t(u % kFinRing));
        }
      }
      if (bad_slot) atomicOr(cta_flags, VA_STATUS_BAD_SLOT);
      if (hidden_nonfinite) atomicOr(cta_flags, kFlagHiddenNonfinite);
    }
  } else {
    // ================================================================ PV CTA
    volatile uint32_t* cmd = reinterpret_cast<volatile uint32_t*>(gb + kOffCmd);
    if (warp == 0) {
      // ---- boxes: the CTA's value blocks of each tile ({0,1,4,5} + 2h)
      if (lane == 0) {
        bool ok = true;
        const uint32_t lead_full = mapa(bar(B_VFULL), lead);
        for (int T = 0; w.more(); ++T, w.next()) {
          const int s = T % kVRing;
          if (T >= kVRing && !wait(B_VEMPTY + s, T / kVRing - 1)) {
            ok = false;
            break;
          }
          if (even) mbar_arrive_expect_tx(bar(B_VFULL + s), 2 * kVTileBytes);
          const TileAt t = tile_at(p, w);
          const CUtensorMap* m = t.tail ? &maps.vt : &maps.v;
          const uint32_t dst = sb + kOffV + uint32_t(s) * kVTileBytes;
          tma_load_3d_pair(dst, m, 0, t.row, 2 * hh, lead_full + 8u * uint32_t(s));
          tma_load_3d_pair(dst + 2 * kVBlock, m, 0, t.row, 4 + 2 * hh, lead_full + 8u * uint32_t(s));
        }
        if (!ok) fail();
        (void)mbar_wait(bar(B_MMAFIN), 0, nullptr, kWaitCycles);
        if (*abort_flag)
          for (const long long t0 = clock64(); clock64() - t0 < kDrainCycles;) {}
      }
      __syncwarp();
    } else if (warp == 1 && even) {
      // ---- products O += P V, for both CTAs; commands to the row warps
      constexpr uint32_t idesc = idesc_bf16(kUnitRows, 256, 0, 1);
      const uint32_t m_cmd = mapa(sb + kOffCmd, mate), m_ogo = mapa(bar(B_OGO), mate);
      auto command = [&](uint32_t c) {
        if (lane == 0) {
          *cmd = c;
          mbar_arrive(bar(B_OGO));
          st_cluster_u32(m_cmd, c);
          mbar_arrive_remote(m_ogo);
        }
        __syncwarp();
      };
      // a P buffer's barrier expects one arrival, ours, that carries the bytes of
      // the QK CTA's copy into it
      const int64_t steps = tiles_of(w);
      if (lane == 0)
        for (int t = 0; t < kPBufs && t < steps; ++t) mbar_arrive_expect_tx(bar(B_PFULL + t), kPPayload);
      __syncwarp();
      bool ok = true, first = false;
      int u = 0, nresc = 0, n = 0;   // units begun, rescales, tiles left of the unit's piece
      for (int T = 0; n > 0 || w.more(); ++T) {
        first = n == 0;
        if (first) {
          n = w.piece();
          w.next_piece();
        }
        const int pb = T % kPBufs, s = T % kVRing;
        const bool got = (!first || u == 0 || wait_far(B_OFREE, u - 1)) &&
                         wait_far(B_VFULL + s, T / kVRing) && wait_far(B_PFULL + pb, T / kPBufs) &&
                         wait_far(B_PFULLP + pb, T / kPBufs);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        const uint32_t pbase = sb + kOffP + uint32_t(pb) * kPBufBytes;
        const volatile uint32_t* flags =
            reinterpret_cast<const volatile uint32_t*>(gb + kOffP + pb * kPBufBytes + kPFlags);
        const uint32_t any = flags[0] | flags[1] | flags[2] | flags[3] |
                             reinterpret_cast<const volatile uint32_t*>(gb + kOffPeerAny)[pb];
        if (__any_sync(0xffffffffu, any != 0) && !first) {
          // rows change reference: O must be final before the row warps rescale
          // it, and rescaled before this tile's product
          mma2_commit_mc_warp(bar(B_ODONE), uint16_t(1u << rank));
          bool g = __all_sync(0xffffffffu, wait(B_ODONE, nresc));
          if (g) {
            command(uint32_t(pb));
            g = __all_sync(0xffffffffu, wait_far(B_OCORR, nresc));
          }
          ++nresc;
          if (!g) {
            ok = false;
            break;
          }
        }
        fence_proxy_async_cta();
        tc_fence_after();
        const uint64_t ad = smem_desc(pbase, 16, 1024, kSwizzle128B);
        if (elect_one()) {
#pragma unroll
          for (int q = 0; q < kDv / 256; ++q) {
            const uint64_t bd = smem_desc(sb + kOffV + uint32_t(s) * kVTileBytes + uint32_t(2 * q) * kVBlock,
                                          kVBlock, 1024, kSwizzle128B);
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)
              mma2_ss(tmem + uint32_t(256 * q), ad + uint64_t((uint32_t(k) * 32u) >> 4),
                      bd + uint64_t((uint32_t(k) * 2048u) >> 4), idesc, (!first || k > 0) ? 1u : 0u);
          }
          mma2_commit_mc(bar(B_VEMPTY + s), kPvMask);
          // re-armed before its release can reach the QK CTA
          if (T + kPBufs < steps) mbar_arrive_expect_tx(bar(B_PFULL + pb), kPPayload);
          mma2_commit_mc(bar(B_PFREE + pb), kQkMask);
        }
        __syncwarp();
        if (--n == 0) {   // the unit's last product here: its rows may be written out
          mma2_commit_mc_warp(bar(B_OFULL), kPvMask);
          command(kCmdUnit);
          ++u;
        }
      }
      // (the last unit's rows have been read before its command is overwritten)
      if (ok && u > 0) ok = __all_sync(0xffffffffu, wait_far(B_OFREE, u - 1));
      if (!ok && lane == 0) fail();
      command(kCmdDone);
      mma2_commit_mc_warp(bar(B_MMAFIN), kPvMask);
      (void)mbar_wait(bar(B_MMAFIN), 0, nullptr, kWaitCycles);
      __syncwarp();
    } else if (warp == 1) {
      // ---- odd rank: forwards its P buffers' arrivals, and whether their rows
      // rescale, to the even rank, and re-arms them
      const uint32_t pfullp = mapa(bar(B_PFULLP), mate), peer_any = mapa(sb + kOffPeerAny, mate);
      const int64_t steps = tiles_of(w);
      if (lane == 0)
        for (int t = 0; t < kPBufs && t < steps; ++t) mbar_arrive_expect_tx(bar(B_PFULL + t), kPPayload);
      __syncwarp();
      for (int64_t T = 0; T < steps; ++T) {
        const int pb = int(T % kPBufs);
        if (!__all_sync(0xffffffffu, wait_far(B_PFULL + pb, int(T / kPBufs)))) {
          if (lane == 0) fail();
          break;
        }
        fence_proxy_async_cta();
        if (lane == 0) {
          const volatile uint32_t* fl = reinterpret_cast<const volatile uint32_t*>(
              gb + kOffP + uint32_t(pb) * kPBufBytes + kPFlags);
          st_cluster_u32(peer_any + 4u * uint32_t(pb), fl[0] | fl[1] | fl[2] | fl[3]);
          if (T + kPBufs < steps) mbar_arrive_expect_tx(bar(B_PFULL + pb), kPPayload);
          mbar_arrive_remote(pfullp + 8u * uint32_t(pb));
        }
        __syncwarp();
      }
      // products read this CTA's memory until their last commit
      (void)mbar_wait<true>(bar(B_MMAFIN), 0, nullptr, kWaitCycles);
      __syncwarp();
    } else if (warp >= 4) {
      // ---- row warps: rescale O on command, and write a unit's rows out;
      // warpgroup `half` owns 256 of the 512 columns
      const int r = q4 * 32 + lane;
      const uint32_t tl = tmem + (uint32_t(q4 * 32) << 16) + 256u * uint32_t(half);
      const uint32_t ocorr_lead = mapa(bar(B_OCORR), lead), ofree_lead = mapa(bar(B_OFREE), lead);
      uint8_t* stg = gb + kOffOut + uint32_t(warp - 4) * (32 * kOutRow);
      for (int k = 0, u = 0;; ++k) {
        if (!__all_sync(0xffffffffu, wait_far(B_OGO, k))) {
          if (lane == 0) fail();
          break;
        }
        const uint32_t c = *cmd;
        if (c == kCmdDone) break;
        if (c != kCmdUnit) {
          const float a = reinterpret_cast<const float*>(gb + kOffP + c * kPBufBytes + kPAlpha)[r];
          tc_fence_after();
          if (__any_sync(0xffffffffu, a != 1.f)) {
#pragma unroll 1
            for (int cc = 0; cc < 8; ++cc) {
              uint32_t v[32];
              tmem_ld32(tl + 32u * uint32_t(cc), v);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * a);
              tmem_st32(tl + 32u * uint32_t(cc), v);
            }
            tmem_wait_st();
          }
          tc_fence_before();
          if (even) {
            mbar_arrive(bar(B_OCORR));
          } else {
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(ocorr_lead);
          }
          continue;
        }
        const int rows = w.rows() - hh * kRows - q4 * 32;   // of this warp's 32
        const int ur = w.unit * kUnitRows + hh * kRows + q4 * 32;
        const size_t grow = size_t(w.r.q0) * p.H + ur;
        const bool direct = w.k == 0 && w.piece() == w.t.ntiles;
        const size_t prow = (size_t(2 * cluster + (w.g > w.begin(cluster) ? 1 : 0))) * kUnitRows +
                            hh * kRows + q4 * 32;
        w.next_piece();
        const bool got = wait_far(B_OFULL, u) && wait_far(B_FIN + u % kFinRing, u / kFinRing);
        if (!__all_sync(0xffffffffu, got)) {
          if (lane == 0) fail();
          break;
        }
        tc_fence_after();
        const float inv = reinterpret_cast<const volatile float*>(gb + kOffFin)[(u % kFinRing) * kRows + r];
        ++u;
        // 128 bytes of each of the warp's rows at a time -- 64 columns as bf16, or
        // 32 of an fp32 partial -- through shared memory, so that the stores are
        // whole lines of a row
        const int passes = direct ? 4 : 8;
#pragma unroll 1
        for (int pass = 0; pass < passes; ++pass) {
          uint32_t o[32];
          if (direct) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t v[32];
              tmem_ld32(tl + 64u * uint32_t(pass) + 32u * uint32_t(h), v);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(v[2 * e]) * inv,
                                                                __uint_as_float(v[2 * e + 1]) * inv);
                o[16 * h + e] = *reinterpret_cast<const uint32_t*>(&b2);
              }
            }
          } else {
            tmem_ld32(tl + 32u * uint32_t(pass), o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv);
          }
          if (pass + 1 == passes) {   // O has been read: the next unit's products may go
            tc_fence_before();
            if (even) {
              mbar_arrive(bar(B_OFREE));
            } else {
              __syncwarp();
              if (lane == 0) mbar_arrive_remote(ofree_lead);
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(stg + uint32_t(lane) * kOutRow + 16 * j) =
                make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
          __syncwarp();
          uint8_t* dst = direct ? reinterpret_cast<uint8_t*>(p.out + grow * kDv + 256 * half + 64 * pass)
                                : reinterpret_cast<uint8_t*>(p.part_o + prow * kDv + 256 * half + 32 * pass);
          const size_t pitch = direct ? size_t(kDv) * 2 : size_t(kDv) * 4;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int row = 4 * i + (lane >> 3);
            if (row < rows)
              *reinterpret_cast<uint4*>(dst + row * pitch + (lane & 7) * 16) =
                  *reinterpret_cast<const uint4*>(stg + uint32_t(row) * kOutRow + (lane & 7) * 16);
          }
          __syncwarp();
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (tid == 0) p.cta_flags[blockIdx.x] = *cta_flags;
  // every CTA has finished every role before any frees its tensor memory or
  // leaves: products and arrivals cross between them
  cluster_sync();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// Rows of 576 features as column blocks of 64: a box of `rows` x `blocks`.
bool encode(CUtensorMap* m, const __nv_bfloat16* base, int64_t n, int64_t stride, int rows, int blocks) {
  cuuint64_t dims[3] = {64u, cuuint64_t(n), cuuint64_t(kBlocks)};
  cuuint64_t strides[2] = {cuuint64_t(stride) * 2u, 128u};
  cuuint32_t box[3] = {64u, uint32_t(rows), uint32_t(blocks)};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16*>(base), dims,
                  strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t init_prefill_tc() {
  return cudaFuncSetAttribute(prefill_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              int(kSmemBytes));
}

cudaError_t launch_prefill_tc(const ChunkTcParams& p, int clusters, cudaStream_t st) {
  if (!g_encode) return cudaErrorNotSupported;
  const __nv_bfloat16* kv = p.packed ? p.packed : p.kv;
  const int64_t rows = p.packed ? p.num_entries : p.num_slots;
  const int64_t stride = p.packed ? kDqk : p.kv_stride;
  const int64_t tail_rows = int64_t(p.B) * kTile;
  Maps m;
  memset(&m, 0, sizeof m);
  if (!encode(&m.k, kv, rows, stride, kSlotRows, kBlocks) || !encode(&m.v, kv, rows, stride, kTile, 2) ||
      !encode(&m.kt, p.tails, tail_rows, kDqk, kSlotRows, kBlocks) ||
      !encode(&m.vt, p.tails, tail_rows, kDqk, kTile, 2) ||
      !encode(&m.q, p.q, int64_t(p.total_q) * p.H, kDqk, kSlotRows, kBlocks))
    return cudaErrorNotSupported;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCtas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(unsigned(kCtas * clusters), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, prefill_tc_kernel, p, m);
}

}  // namespace va
