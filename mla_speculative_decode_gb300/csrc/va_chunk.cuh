// va_chunk.cuh -- what the chunk-attention kernels, the weight kernels and
// their host code share: launch parameters, a request's bounds, which keys a
// token sees, and one row's attention on CUDA cores.
#pragma once

#include <math.h>

#include "va_common.cuh"

namespace va {

// What a cluster of the split kernel costs besides its tiles (set-up, fill,
// drain and write-out, about 11 us), in tiles; and the most waves of clusters that
// units are split for.  (A batch that needs more waves than that for its units
// alone is split only as far as its last wave has room.  So at most kSplitWaves
// waves' items are parts of split units, or 2 waves' when the units alone need
// more: that bounds the partials.)
constexpr int kFixedTiles = 10;
constexpr int kSplitWaves = 7;

// List positions are 32-bit: a request's keys, and the entries of all lists, stay below
// 2^31 with some key tiles to spare.
constexpr int kKeysMax = 0x7fffffff - 1024;

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
  int64_t num_entries;         // entries of slot_idx (contiguous: 0)
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

// (`ended`: the request lies behind the batch's end, see chunk_ends, and brings no
// tokens)
__device__ inline ChunkReq chunk_req(const ChunkParams& p, int b, bool ended = false) {
  ChunkReq r;
  const int a0 = p.q_indptr[b], a1 = p.q_indptr[b + 1];
  int q0 = a0 < 0 ? 0 : (a0 > p.total_q ? p.total_q : a0);
  int q1 = a1 < q0 ? q0 : (a1 > p.total_q ? p.total_q : a1);
  r.bad = q0 != a0 || q1 != a1;
  if (ended) q1 = q0;
  r.q0 = q0;
  r.n = q1 - q0;
  int P = p.prefix_len[b];
  if (P < 0) { P = 0; r.bad = true; }
  if (p.kv_start) {
    // a prefix longer than the pool cannot be there
    if (P > p.num_slots) { P = int(p.num_slots); r.bad = true; }
    if (P > kKeysMax - r.n) { P = kKeysMax - r.n; r.bad = true; }
    // (a start behind the pool, or so far before it that no key reaches it, names no
    // row: clamped, so that no sum with a list position overflows)
    const int64_t at = p.kv_start[b], before = -(int64_t(1) << 31);
    r.base = at > p.num_slots ? p.num_slots : at < before ? before : at;
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

// Whether request b's query bounds decrease, which ends the batch before it: only
// bounds that never do are sure to name no row twice, and no more rows than q has.
// (b past the batch: false.)
__device__ inline bool chunk_ends(const ChunkParams& p, int b) {
  return b < p.B && p.q_indptr[b + 1] < p.q_indptr[b];
}

// Requests before the batch's end.  A whole warp takes part.
__device__ inline int chunk_requests(const ChunkParams& p, int lane) {
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const uint32_t ends = __ballot_sync(0xffffffffu, chunk_ends(p, b0 + lane));
    if (ends) return b0 + __ffs(int(ends)) - 1;
  }
  return p.B;
}

// Whether the bounds of the requests' lists never decrease: then the list that an
// entry lies in is the last one that begins at or before it.  A whole warp takes part.
__device__ inline bool chunk_lists_sorted(const ChunkParams& p, int lane) {
  bool falls = false;
  for (int b = lane; b < p.B; b += 32) falls |= p.kv_indptr[b + 1] < p.kv_indptr[b];
  return !__any_sync(0xffffffffu, falls);
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

// ---------------------------------------------------------------- schedule
//
// Work is cut where the tokens are: a unit is `unit_rows` consecutive rows
// (token, head) of one request, and a unit's keys are tiles of 64 list
// positions: the tiles that hold sinks, then those from the first key that the
// unit's first token sees to the last token's own key.  Lengths live on the
// device, so a launch has a fixed grid of clusters ("items") and each cluster
// finds its own piece: (request, unit, split of the unit's tiles).

// The tiles of one unit, or of one split of them.
struct ChunkTiles {
  int t0;       // first tile, counted through the unit's tiles
  int ntiles;
  int nst;      // tiles that hold sinks, before the window's
  int wt;       // the window's first tile, as a list position / 64
  int k1;       // keys past the unit's last token start here
  int first;    // first key past the sinks that the unit's first token sees
  int sinks;
  __device__ int tile_key(int t) const {
    const int g = t0 + t;
    return (g < nst ? g : g - nst + wt) * 64;
  }
  // whether some row of the unit sees key j
  __device__ bool sees(int j) const { return j < k1 && (j >= first || j < sinks); }
  // whether some row sees every key of the tile that starts at key tk0
  __device__ bool whole(int tk0) const {
    return tk0 + 64 <= k1 && (tk0 >= first || tk0 + 64 <= sinks);
  }
};

// The n lowest bits of a 64-bit mask (any n).
__device__ __forceinline__ uint64_t low_bits(int n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
}

// All tiles of rows [row0, row0 + rows) of a request (rows >= 1).
__device__ inline ChunkTiles chunk_tiles(const ChunkParams& p, const ChunkReq& r, int row0,
                                         int rows) {
  ChunkTiles t;
  const int i0 = row0 / p.H, i1 = (row0 + rows - 1) / p.H;
  t.k1 = r.P + i1 + 1;
  t.first = window_first(p.window, r.P + i0);
  t.sinks = p.sinks;
  const int s = p.sinks < t.first ? p.sinks : t.first;   // sinks before the window
  t.nst = (s + 63) / 64;
  t.wt = t.first / 64 > t.nst ? t.first / 64 : t.nst;
  t.t0 = 0;
  t.ntiles = t.nst + (t.k1 + 63) / 64 - t.wt;
  return t;
}

struct ChunkSched {
  int unit_rows;   // 64 (decode kernel), 128, or 256 with two-SM products
  int clusters;    // clusters resident at once
  int max_waves;   // waves of clusters that the grid holds
};

struct ChunkItem {
  int b, unit, split;
  int units;        // of the request
  int ns;           // splits of each of the request's units
  int unit0;        // units of the requests before it
  int item0;        // its first item
  int pslot0;       // its first partial slot (requests with ns > 1 have units * ns)
  int total_units, total_items;   // of the batch (valid for item 0)
  bool live;
};

// A request's units and the tiles of its longest (last) unit.
__device__ inline void chunk_work(const ChunkParams& p, const ChunkSched& s, int b, int* units,
                                  int* tiles) {
  const ChunkReq r = chunk_req(p, b);
  const int rows = r.n * p.H;
  *units = (rows + s.unit_rows - 1) / s.unit_rows;
  *tiles = 0;
  if (rows > 0) {
    const int row0 = (*units - 1) * s.unit_rows;
    *tiles = chunk_tiles(p, r, row0, rows - row0).ntiles;
  }
}

// Item `item` of the batch; a whole warp takes part, lane l looking at requests
// l, l + 32, ...  A split takes at most `chunk` tiles, so a request with t tiles
// gets ns = ceil(t / chunk) splits and units * ns items.  For each number k of
// waves of clusters that could hold the batch, the smallest chunk whose items fit
// is found (grown by eighths from the average), and the k with the least
// k * (chunk + kFixedTiles) is taken: k rounds of a split's tiles and of what a
// cluster costs besides.  Items run split by split, and within a split from the
// last unit (the most keys) to the first, so that units that read the same keys
// run together.
__device__ inline ChunkItem chunk_item(const ChunkParams& p, const ChunkSched& s, int item,
                                       int lane) {
  constexpr uint32_t kAll = 0xffffffffu;
  const int B = chunk_requests(p, lane);
  int u0 = 0, t0 = 0;   // requests 0 .. 31 stay in registers
  int64_t work = 0;
  for (int b = lane; b < B; b += 32) {
    int u, t;
    chunk_work(p, s, b, &u, &t);
    if (b < 32) { u0 = u; t0 = t; }
    work += int64_t(u) * t;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) work += __shfl_xor_sync(kAll, work, o);
  int all_units = 0;
  for (int b = lane; b < B; b += 32) {
    int u = u0, t = t0;
    if (b >= 32) chunk_work(p, s, b, &u, &t);
    all_units += u;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all_units += __shfl_xor_sync(kAll, all_units, o);
  // (one split per unit fits the grid whatever the lengths: its waves hold all
  // units that the batch can have)
  int chunk = 0x3fffffff;
  int64_t best = INT64_MAX;
  const int k0 = (all_units + s.clusters - 1) / s.clusters;
  for (int k = k0 < 1 ? 1 : k0;
       k <= s.max_waves && (k <= kSplitWaves || best == INT64_MAX); ++k) {
    int64_t c = (work + int64_t(k) * s.clusters - 1) / (int64_t(k) * s.clusters);
    if (c < 1) c = 1;
    if (k * (c + kFixedTiles) >= best) continue;   // could not be better even if it fitted
    for (int n = INT32_MAX; c < 0x3fffffff; c += c / 8 + 1) {
      n = 0;
      for (int b = lane; b < B; b += 32) {
        int u = u0, t = t0;
        if (b >= 32) chunk_work(p, s, b, &u, &t);
        n += u * int((t + c - 1) / c);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(kAll, n, o);
      if (n <= k * s.clusters) break;
    }
    if (k * (c + kFixedTiles) < best) {
      best = k * (c + kFixedTiles);
      chunk = int(c);
    }
    if (c <= kFixedTiles) break;   // shorter splits only add to what clusters cost
  }
  ChunkItem it;
  it.live = false;
  it.b = it.unit = it.split = it.units = it.ns = it.unit0 = it.item0 = it.pslot0 = 0;
  int items = 0, slots = 0, units = 0;   // of the requests before this round
  for (int b0 = 0; b0 < B; b0 += 32) {
    const int b = b0 + lane;
    int u = u0, t = t0;
    if (b0 > 0) {
      u = t = 0;
      if (b < B) chunk_work(p, s, b, &u, &t);
    }
    const int ns = (t + chunk - 1) / chunk;
    const int n_items = u * ns, n_slots = ns > 1 ? n_items : 0;
    int ci = n_items, cs = n_slots, cu = u;   // inclusive sums
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(kAll, ci, o), c = __shfl_up_sync(kAll, cs, o),
                d = __shfl_up_sync(kAll, cu, o);
      if (lane >= o) { ci += a; cs += c; cu += d; }
    }
    const uint32_t mine =
        __ballot_sync(kAll, item >= items + ci - n_items && item < items + ci);
    if (mine) {
      const int src = __ffs(int(mine)) - 1;
      it.live = true;
      it.b = b0 + src;
      it.units = __shfl_sync(kAll, u, src);
      it.ns = __shfl_sync(kAll, ns, src);
      it.unit0 = units + __shfl_sync(kAll, cu, src) - it.units;
      it.item0 = items + __shfl_sync(kAll, ci, src) - it.units * it.ns;
      it.pslot0 = slots + __shfl_sync(kAll, cs, src) - (it.ns > 1 ? it.units * it.ns : 0);
      const int k = item - it.item0;
      it.split = k / it.units;
      it.unit = it.units - 1 - k % it.units;
      if (item != 0) break;
    }
    items += __shfl_sync(kAll, ci, 31);
    slots += __shfl_sync(kAll, cs, 31);
    units += __shfl_sync(kAll, cu, 31);
  }
  it.total_units = units;
  it.total_items = items;
  return it;
}

// A place in the row of steps: the tiles of all units (kRows query rows each) of
// the batch, request by request, unit by unit, each unit's preceded by kCost places
// for what a unit costs besides its tiles.  A launch cuts the row into equal runs,
// one for each of its CTAs or clusters; every role of those walks its run with one
// of these, so that they agree without talking.
template <int kRows, int kCost>
struct ChunkRun {
  const ChunkParams& p;
  ChunkReq r;
  ChunkTiles t;        // all tiles of the unit
  int b, unit, units, unit0;   // request, unit within it, its units, units before it
  int k;               // tile within the unit
  int64_t g, end;      // place of this step in the row; of the run's end
  int64_t total;       // places of the batch
  int runs;            // runs it is cut into

  __device__ explicit ChunkRun(const ChunkParams& p_) : p(p_) {}
  __device__ int rows() const {
    const int n = r.n * p.H - unit * kRows;
    return n < kRows ? n : kRows;
  }
  __device__ void load(int b_) {
    b = b_;
    r = chunk_req(p, b);
    units = (r.n * p.H + kRows - 1) / kRows;
    unit = 0;
  }
  __device__ void tiles() { t = chunk_tiles(p, r, unit * kRows, rows()); }
  __device__ int key() const { return t.tile_key(k); }
  __device__ bool more() const { return g < end; }
  __device__ bool last_tile() const { return k + 1 == t.ntiles || g + 1 >= end; }
  // The next step of the run, if there is one (see more).
  __device__ void next() {
    if (++g >= end) return;
    if (++k < t.ntiles) return;
    g += kCost;
    if (g >= end) return;
    k = 0;
    if (++unit >= units) {
      unit0 += units;
      do load(b + 1);
      while (units == 0 && b + 1 < p.B);
    }
    tiles();
  }
  // The steps of this unit that lie in the run from here on, and the step after
  // them.
  __device__ int piece() const { return int(t.ntiles - k < end - g ? t.ntiles - k : end - g); }
  __device__ void next_piece() {
    const int n = piece() - 1;
    k += n;
    g += n;
    next();
  }
  // First place of run c, and the run that place x is in.
  __device__ int64_t begin(int c) const { return total * c / runs; }
  __device__ int owner(int64_t x) const {
    int c = int(x * runs / total);
    while (c + 1 < runs && begin(c + 1) <= x) ++c;
    while (c > 0 && begin(c) > x) --c;
    return c;
  }
};

// Places and units of requests b0 + lane: a lane counts a request of at most two
// units by itself, the warp together one of more.
template <int kRows, int kCost>
__device__ int64_t count_steps(ChunkRun<kRows, kCost>& w, int b0, int lane, int* units) {
  constexpr uint32_t kAll = 0xffffffffu;
  int64_t mine = 0;
  *units = 0;
  if (b0 + lane < w.p.B) {
    w.load(b0 + lane);
    *units = w.units;
    if (w.units <= 2)
      for (; w.unit < w.units; ++w.unit) {
        w.tiles();
        mine += w.t.ntiles;
      }
  }
  for (uint32_t many = __ballot_sync(kAll, *units > 2); many; many &= many - 1) {
    const int src = __ffs(int(many)) - 1;
    w.load(b0 + src);
    int64_t n = 0;
    for (w.unit = lane; w.unit < w.units; w.unit += 32) {
      w.tiles();
      n += w.t.ntiles;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(kAll, n, o);
    if (lane == src) mine = n;
  }
  return mine + int64_t(*units) * kCost;
}

// Run c's first step and end (see more), of at most `grid` runs; returns the
// batch's units in total.  A whole warp takes part.
template <int kRows, int kCost>
__device__ int find_run(ChunkRun<kRows, kCost>& w, int c, int grid, int lane) {
  constexpr uint32_t kAll = 0xffffffffu;
  int64_t total = 0, s0 = 0;
  int all_units = 0, n0 = 0;
  for (int b0 = 0; b0 < w.p.B; b0 += 32) {
    int n;
    int64_t s = count_steps(w, b0, lane, &n);
    const uint32_t ends = __ballot_sync(kAll, chunk_ends(w.p, b0 + lane));
    if (ends && lane >= __ffs(int(ends)) - 1) s = n = 0;
    if (b0 == 0) { s0 = s; n0 = n; }
    total += s;
    all_units += n;
    if (ends) break;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total += __shfl_xor_sync(kAll, total, o);
    all_units += __shfl_xor_sync(kAll, all_units, o);
  }
  w.total = total;
  w.runs = total < grid ? int(total) : grid;
  w.g = w.end = 0;
  if (c >= w.runs) return all_units;
  w.g = w.begin(c);
  w.end = w.begin(c + 1);
  int64_t before = 0;
  int units = 0;
  for (int b0 = 0; b0 < w.p.B; b0 += 32) {
    int64_t s = s0;
    int n = n0;
    if (b0 > 0) s = count_steps(w, b0, lane, &n);
    int64_t sum = s;
    int nsum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(kAll, sum, o);
      const int y = __shfl_up_sync(kAll, nsum, o);
      if (lane >= o) { sum += x; nsum += y; }
    }
    const uint32_t mine = __ballot_sync(kAll, w.g >= before + sum - s && w.g < before + sum);
    if (mine) {
      const int src = __ffs(int(mine)) - 1;
      int64_t at = w.g - before - __shfl_sync(kAll, sum - s, src);   // steps into the request
      w.unit0 = units + __shfl_sync(kAll, nsum - n, src);
      w.load(b0 + src);
      for (int u0 = 0;; u0 += 32) {   // 32 units at a time
        int64_t t = 0;
        w.unit = u0 + lane;
        if (w.unit < w.units) {
          w.tiles();
          t = w.t.ntiles + kCost;
        }
        int64_t cum = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t x = __shfl_up_sync(kAll, cum, o);
          if (lane >= o) cum += x;
        }
        const uint32_t in = __ballot_sync(kAll, at >= cum - t && at < cum);
        if (in) {
          const int u = __ffs(int(in)) - 1;
          // (a run that begins in a unit's cost begins with its first tile)
          const int k = int(at - __shfl_sync(kAll, cum - t, u)) - kCost;
          w.k = k < 0 ? 0 : k;
          w.g += k < 0 ? -k : 0;
          w.unit = u0 + u;
          w.tiles();
          return all_units;
        }
        at -= __shfl_sync(kAll, cum, 31);
        if (u0 + 32 >= w.units) break;   // (cannot be: the step lies in this request)
      }
      break;
    }
    before += __shfl_sync(kAll, sum, 31);
    units += __shfl_sync(kAll, nsum, 31);
  }
  w.g = w.end;
  return all_units;
}

// One unit's entry in the workspace, written by its first split's cluster for
// the kernel that merges the splits.
struct alignas(16) ChunkUnit {
  int row0, rows;        // rows of out / lse
  int ns;                // splits that hold keys (1: already in out and lse)
  int pslot;             // partial slot of split 0 ...
  int pslot1, pstride;   // ... of split 1, and from there on
  int item, istride;     // item of split 0, and from split to split
  int b, i0;             // request, row within it
};

// Arguments of the tensor-core launch and of the merge.
struct ChunkTcParams : ChunkParams {
  ChunkSched sched;
  int ctas;              // CTAs per item
  int32_t* totals;       // [2]: units, items (written by item 0)
  ChunkUnit* units;
  uint32_t* cta_flags;   // [items][ctas] status bits of each CTA
  // many rows per request (va_prefill_tc.cu):
  const __nv_bfloat16* packed;  // paged: [num_entries, 576] the listed rows side by side
  const uint32_t* valid;        // paged: bit e set when entry e has a pool row
  const __nv_bfloat16* tails;   // [B * 64, 576]: each request's last, partial tile, zeros behind it
  uint32_t* pack_flags;         // [pack_blocks] status bits of the packing
  int pack_blocks;
  float* part_lse;       // [slots][unit_rows]
  float* part_o;         // [slots][unit_rows][512], normalised by the split's row sum
};

// Bit of a CTA's status word: a hidden key's score was not finite, so products
// with its value may have spoilt rows that do not see it; the merge kernel
// computes the unit's rows again on CUDA cores.
constexpr uint32_t kFlagHiddenNonfinite = 0x80000000u;

// Bit of a packing block's status word: one of its entries that were copied has no
// pool row.
constexpr uint32_t kPackMissing = 0x80000000u;

// Tensor-core kernels: va_decode_tc.cu for few rows per request (units of 64
// rows, an item per CTA, two partial slots each), else va_tc.cu.
cudaError_t launch_decode_tc(const ChunkTcParams& p, int ctas, cudaStream_t st);
// va_prefill_tc.cu: many rows per request (units of 256 rows, an item per
// cluster, two partial slots each), keys side by side.
cudaError_t launch_prefill_tc(const ChunkTcParams& p, int clusters, cudaStream_t st);
cudaError_t launch_chunk_tc(const ChunkTcParams& p, int grid_items, bool pair, cudaStream_t st);

// The scale, for base-2 exponents, of scores from the tensor cores.  They accumulate a
// score in 36 steps that round towards zero.  What that takes off depends on how the
// partial sums run: 4.5e-7 s on the average for keys and queries without structure,
// 1.4e-7 s where the last columns make up the score, 1.1e-6 s where the first ones do
// or all do evenly, up to 1.5e-6 s where half of them cancel the others.  The scale
// makes up the average, in the attention and in the weight kernels alike: a weight
// exp(s - lse) from an attention call's own lse then keeps no trace of what was lost
// (totals of rows with scores up to 33: 2e-7 high; with the scale made up in the
// weights alone 1.25e-5), and lse agrees better with an exact one (there 2e-6 off instead
// of 1.4e-5).  The CUDA-core path rounds to nearest and takes the scale as it is.
inline float tc_scale_log2(float sm_scale) {
  return float(double(sm_scale) * 1.4426950408889634 * (1.0 + 4.5e-7));
}

// Checks shared by the chunk calls (va_chunk.cu).
int chunk_check(const ChunkParams& p, bool paged, float sm_scale, int flags, const void* ws);

}  // namespace va
