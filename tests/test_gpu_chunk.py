"""Chunk attention (va_chunk_attn_paged, va_chunk_attn_contiguous) against the
fp64 oracle (needs an sm_103 GPU): ragged lengths from zero, windows and sinks,
strides, bad bounds and slots, NaN where nothing may look, capture, streams."""
import numpy as np
import pytest
import torch

import synth
from tests import _chunk

pytestmark = pytest.mark.gpu

PATHS = {"fma": 1, "tc": 2, "tc1sm": 3}


@pytest.fixture(scope="module")
def va():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mla_speculative_decode_gb300 as m
    m.build()
    m.init()
    return m


CASES = [
    # P, n, H
    ([0], [1], 1),
    ([1], [1], 8),
    ([63], [1], 8),
    ([64], [1], 64),
    ([0], [2], 3),
    ([0], [65], 5),
    ([500], [17], 8),
    ([129, 0, 64, 3], [1, 1, 1, 1], 16),
    ([0, 200, 31, 7], [3, 0, 40, 1], 5),
    ([0, 0, 10], [0, 0, 5], 2),
    ([300, 2, 0, 77, 129], [1, 1, 33, 64, 5], 24),
    ([1000], [3], 128),
    ([90, 700], [50, 1], 64),
]


@pytest.mark.parametrize("path", list(PATHS.values()), ids=list(PATHS))
@pytest.mark.parametrize("layout", ["paged", "contiguous"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_ragged_chunks(va, case, layout, path):
    P, n, H = CASES[case]
    c = _chunk.make(P, n, H, seed=100 + case, layout=layout, list_gap=case % 3)
    out, lse = _chunk.call(va, c, flags=path)
    _chunk.check(c, out, lse)


WINDOWS = [(1, 0), (1, 1), (2, 5), (17, 0), (64, 4), (65, 64), (128, 63), (200, 100),
           (100000, 3), (7, 100000)]


@pytest.mark.parametrize("path", list(PATHS.values()), ids=list(PATHS))
@pytest.mark.parametrize("layout", ["paged", "contiguous"])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_window_and_sinks(va, window, sinks, layout, path):
    c = _chunk.make([430, 0, 91, 5], [37, 66, 1, 0], 6, seed=window + 7 * sinks, layout=layout)
    out, lse = _chunk.call(va, c, flags=path, window=window, sinks=sinks)
    _chunk.check(c, out, lse, window=window, sinks=sinks)


@pytest.mark.parametrize("path", list(PATHS.values()), ids=list(PATHS))
@pytest.mark.parametrize("layout", ["paged", "contiguous"])
def test_rows_without_a_request_are_left_and_wide_pool_rows_are_skipped(va, layout, path):
    c = _chunk.make([120, 33], [9, 4], 8, seed=3, layout=layout, stride=640, q_before=2, q_behind=5)
    total = c.q.shape[0]
    out = torch.full((total, 8, 512), 7.5, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((total, 8), -3.25, device="cuda")
    c.q[:2] = float("nan")
    c.q[-5:] = float("nan")
    _chunk.call(va, c, flags=path, out=out, lse=lse)
    _chunk.check(c, out, lse)
    for rows in (slice(0, 2), slice(total - 5, total)):
        assert bool((out[rows] == 7.5).all()) and bool((lse[rows] == -3.25).all())
    # a narrow view of a wide pool
    if layout == "paged":
        pool = c.dev("pool")
        o2, l2 = va.chunk_attn_paged(c.dev("q"), pool[:, :576], c.dev("slot_idx"),
                                     c.dev("kv_indptr"), c.dev("prefix_len"), c.dev("q_indptr"),
                                     sm_scale=synth.SM_SCALE, flags=path)
        assert torch.equal(o2[2:-5], out[2:-5]) and torch.equal(l2[2:-5], lse[2:-5])


@pytest.mark.parametrize("path", list(PATHS.values()), ids=list(PATHS))
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
@pytest.mark.parametrize("layout", ["paged", "contiguous"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_a_token_does_not_see_does_not_reach_it(va, bad, layout, window, sinks, path):
    """Later tokens' keys and keys outside the window hold NaN or infinities:
    the tokens that do not see them are as without them, the others NaN."""
    P, n, H = [150, 20], [40, 12], 8
    c = _chunk.make(P, n, H, seed=11, layout=layout)
    for b, j in ((0, 160), (0, 189), (0, 60), (1, 25), (1, 31)):
        c.pool[int(c.key_rows[b][j])] = bad
    out, lse = _chunk.call(va, c, flags=path, window=window, sinks=sinks)
    ref = _chunk.reference(c, window=window, sinks=sinks)
    assert np.isfinite(ref[1]).any() and np.isnan(ref[1]).any()
    # the bound on the scores comes from the finite rows alone
    spread = _chunk.reference(_chunk.make(P, n, H, seed=11, layout=layout), window=window,
                              sinks=sinks)[3]
    fin = np.isfinite(ref[1])
    o = out.float().cpu().numpy().astype(np.float64)
    l = lse.cpu().numpy().astype(np.float64)
    np.testing.assert_array_equal(np.isfinite(l), fin)
    np.testing.assert_array_equal(np.isfinite(o).all(-1), fin)
    assert np.all(np.abs(o - ref[0])[fin] <= _chunk.out_bound(ref[0], ref[2], spread, 200)[fin])
    assert np.all(np.abs(l - ref[1])[fin] <= _chunk.lse_bound(ref[1], spread, 200)[fin])


@pytest.mark.parametrize("path", list(PATHS.values()), ids=list(PATHS))
def test_slots_outside_the_pool_are_skipped_and_flagged(va, path):
    c = _chunk.make([70, 64], [3, 2], 8, seed=5)
    for b, j, v in ((0, 3, -1), (0, 71, 10 ** 6), (1, 0, c.pool.shape[0])):
        c.slot_idx[int(c.kv_indptr[b]) + j] = v
        c.key_rows[b][j] = -1
    call = _chunk.call(va, c, flags=path, prepare=True)
    out, lse = call()
    _chunk.check(c, out, lse)
    assert va.read_status(call.workspace) == va.STATUS_BAD_SLOT
    # every key gone: the rows are empty
    c.slot_idx[:] = -1
    c.key_rows = [np.full(len(r), -1) for r in c.key_rows]
    out, lse = _chunk.call(va, c, flags=path)
    _chunk.check(c, out, lse)


@pytest.mark.parametrize("path", list(PATHS.values()), ids=list(PATHS))
def test_bad_bounds_are_clamped_and_flagged(va, path):
    # a list shorter than prefix + tokens: the prefix gives way
    c = _chunk.make([70, 5], [3, 2], 8, seed=6)
    c.prefix_len[0] = 90
    call = _chunk.call(va, c, flags=path, prepare=True)
    out, lse = call()
    _chunk.check(c, out, lse)
    assert va.read_status(call.workspace) == va.STATUS_BAD_INDPTR
    # a negative prefix counts as none: the tokens are the list's first keys
    c = _chunk.make([0, 5], [3, 2], 8, seed=7)
    c.prefix_len[0] = -4
    call = _chunk.call(va, c, flags=path, prepare=True)
    out, lse = call()
    _chunk.check(c, out, lse)
    assert va.read_status(call.workspace) == va.STATUS_BAD_INDPTR
    # query offsets outside q are cut off
    c = _chunk.make([4, 5], [3, 2], 8, seed=8)
    call = _chunk.call(va, c, flags=path, prepare=True)
    call()
    assert va.read_status(call.workspace) == 0
    c.q_indptr[2] = 1000
    call = _chunk.call(va, c, flags=path, prepare=True)
    call()
    assert va.read_status(call.workspace) == va.STATUS_BAD_INDPTR


@pytest.mark.parametrize("B,P,T,H", [(700, 0, 2, 128), (500, 61, 3, 128), (400, 10, 17, 16)])
@pytest.mark.parametrize("layout", ["paged", "contiguous"])
def test_many_units_of_one_or_two_tiles(va, B, P, T, H, layout):
    """Short requests by the hundred: row sums of many units are on their way at once."""
    c = _chunk.make([P] * B, [T] * B, H, seed=17, layout=layout)
    call = _chunk.call(va, c, prepare=True)
    first = [x.clone() for x in call()]
    fma_out, fma_lse = _chunk.call(va, c, flags=1)     # the CUDA-core path, on every row
    assert float((first[1] - fma_lse).abs().max()) < 1e-4
    d = (first[0].float() - fma_out.float()).abs()
    assert float((d - 2 * 2.0 ** -8 * fma_out.float().abs()).max()) < 2e-2
    for _ in range(5):
        out, lse = call()
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert va.read_status(call.workspace) == 0


@pytest.mark.parametrize("T,H,flags", [(1, 8, 0), (2, 64, 0), (40, 8, 0), (40, 8, 3), (40, 8, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
def test_contiguous_rows_that_leave_the_pool(va, T, H, flags, window, sinks):
    """Starts before the pool, near its end and far outside: keys without a row are
    skipped and reported."""
    c = _chunk.make([70, 200, 130, 30], [T] * 4, H, seed=16, layout="contiguous", unused_nan=False)
    rows = c.pool.shape[0]
    starts = [-33, rows - 150, 1 << 40, -(1 << 62)]
    c.kv_start = torch.tensor(starts, dtype=torch.int64)
    for b, at in enumerate(starts):
        r = np.arange(c.P[b] + T, dtype=np.int64) + at
        c.key_rows[b] = np.where((r >= 0) & (r < rows), r, -1)
    call = _chunk.call(va, c, flags=flags, window=window, sinks=sinks, prepare=True)
    out, lse = call()
    _chunk.check(c, out, lse, window=window, sinks=sinks)
    assert va.read_status(call.workspace) == va.STATUS_BAD_SLOT


@pytest.mark.parametrize("layout", ["paged", "contiguous"])
@pytest.mark.parametrize("B,T,H,flags", [(40, 6, 8, 0), (40, 1, 1, 0), (5, 10, 64, 0), (5, 50, 64, 0),
                                         (70, 50, 64, 0), (9, 33, 16, 1), (9, 33, 16, 3)])
def test_query_bounds_that_decrease_end_the_batch(va, B, T, H, flags, layout):
    """q_indptr 0, T, 0, T, ...: many requests claim the same rows, more in all than q
    has.  The first has them; the others bring none."""
    c = _chunk.make([30] * B, [T] + [0] * (B - 1), H, seed=15, layout=layout)
    call = _chunk.call(va, c, flags=flags, prepare=True)
    first = [x.clone() for x in call()]
    assert va.read_status(call.workspace) == 0
    c.q_indptr[2::2] = 0
    call = _chunk.call(va, c, flags=flags, prepare=True)
    out, lse = call()
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert va.read_status(call.workspace) == va.STATUS_BAD_INDPTR


@pytest.mark.parametrize("path", list(PATHS.values()), ids=list(PATHS))
@pytest.mark.parametrize("sm_scale", [0.0, -0.05, 1.0])
def test_scales(va, sm_scale, path):
    c = _chunk.make([100, 0], [5, 9], 8, seed=9, scale=0.25)
    out, lse = _chunk.call(va, c, flags=path, sm_scale=sm_scale)
    _chunk.check(c, out, lse, sm_scale=sm_scale)


def test_no_tokens_at_all(va):
    c = _chunk.make([10, 3], [0, 0], 4, seed=10)
    out, lse = _chunk.call(va, c)
    assert out.shape == (0, 4, 512) and lse.shape == (0, 4)
    # room for rows, none owned: nothing is written
    c = _chunk.make([10, 3], [0, 0], 4, seed=10, q_behind=6)
    out = torch.full((6, 4, 512), 2.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((6, 4), 2.0, device="cuda")
    _chunk.call(va, c, out=out, lse=lse)
    assert bool((out == 2).all()) and bool((lse == 2).all())


def test_captured_call_serves_other_lengths(va):
    """One captured graph, replayed with other lengths and lists; two graphs
    with a workspace each may overlap."""
    c = _chunk.make([150, 40, 9], [4, 1, 30], 8, seed=12)
    d = _chunk.make([10, 190, 77], [20, 14, 1], 8, seed=13, pool_rows=c.pool.shape[0])
    bufs = {k: c.dev(k) for k in ("q", "pool", "kv_indptr", "prefix_len", "q_indptr")}
    n = max(c.slot_idx.numel(), d.slot_idx.numel())
    bufs["slot_idx"] = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    bufs["slot_idx"][:c.slot_idx.numel()] = c.slot_idx.cuda()
    call = va.prepare_chunk_paged(bufs["q"], bufs["pool"], bufs["slot_idx"], bufs["kv_indptr"],
                                  bufs["prefix_len"], bufs["q_indptr"], sm_scale=synth.SM_SCALE)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = call()
    g.replay()
    _chunk.check(c, out, lse)
    for k in ("q", "pool", "kv_indptr", "prefix_len", "q_indptr"):
        bufs[k].copy_(getattr(d, k))
    bufs["slot_idx"][:d.slot_idx.numel()] = d.slot_idx.cuda()
    g.replay()
    _chunk.check(d, out, lse)


def test_other_streams_and_repeat(va):
    c = _chunk.make([700, 40], [3, 20], 16, seed=14)
    call = _chunk.call(va, c, prepare=True)
    out, lse = call()
    first = out.clone(), lse.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    # two calls at once, each with its own workspace and outputs
    other = _chunk.call(va, c, prepare=True)
    with torch.cuda.stream(side):
        for _ in range(20):
            other()
    for _ in range(20):
        call()
    torch.cuda.synchronize()
    assert torch.equal(out, first[0]) and torch.equal(other.result[0], first[0])


def test_refusals(va):
    c = _chunk.make([10], [3], 4, seed=15)
    a = [c.dev(k) for k in ("q", "pool", "slot_idx", "kv_indptr", "prefix_len", "q_indptr")]
    ok = dict(sm_scale=0.1)
    for i, t, e in ((0, a[0].float(), TypeError), (0, a[0][:, :, :512], ValueError),
                    (0, c.q, ValueError), (1, a[1][:, :512], ValueError), (1, a[1].t(), ValueError),
                    (2, a[2].long(), TypeError), (3, a[3][:1], ValueError),
                    (5, a[5][:1], ValueError), (5, a[5].long(), TypeError)):
        bad = list(a)
        bad[i] = t
        with pytest.raises(e):
            va.chunk_attn_paged(*bad, **ok)
    for kw in (dict(window=-1), dict(sinks=-1), dict(flags=9), dict(sm_scale=float("nan"))):
        with pytest.raises(va.VaError):
            va.chunk_attn_paged(*a, **(ok | kw))
    with pytest.raises(ValueError):
        va.chunk_attn_paged(*a, **ok, out=torch.empty(3, 4, 511, dtype=torch.bfloat16,
                                                      device="cuda"))
    with pytest.raises(va.VaError) as e:
        va.chunk_attn_paged(*a, **ok, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == -4


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 5), (33, 70)])
def test_many_rows_per_request_read_packed_lists(va, window, sinks):
    """640 query rows and more per request: the call packs the listed rows
    first (invisible ones not at all, ones without a row as zeros that count for
    nothing)."""
    c = _chunk.make([400, 0, 130], [40, 33, 1], 64, seed=40 + window, stride=584, list_gap=3,
                    q_before=1, q_behind=2)
    for b, j in ((0, 7), (0, 410), (1, 2), (2, 0)):
        c.slot_idx[int(c.kv_indptr[b]) + j] = -1 if j % 2 else c.pool.shape[0] + j
        c.key_rows[b][j] = -1
    call = _chunk.call(va, c, window=window, sinks=sinks, prepare=True)
    assert call.workspace.numel() > va.load().va_chunk_workspace_bytes(3, c.q.shape[0], 64, 0, 0)
    out, lse = call()
    _chunk.check(c, out, lse, window=window, sinks=sinks)
    own = slice(1, -2)                   # rows no request owns hold whatever they held
    first = out[own].clone()
    assert va.read_status(call.workspace) == va.STATUS_BAD_SLOT
    call()
    assert torch.equal(out[own], first)


def test_packed_lists_with_nan_where_nothing_may_look(va):
    P, n, H = [300], [60], 32
    c = _chunk.make(P, n, H, seed=50)
    for j in (305, 340, 359, 100, 3):
        c.pool[int(c.key_rows[0][j])] = float("nan")
    for window, sinks in ((0, 0), (90, 2), (150, 8)):
        out, lse = _chunk.call(va, c, window=window, sinks=sinks)
        ref = _chunk.reference(c, window=window, sinks=sinks)
        fin = np.isfinite(ref[1])
        np.testing.assert_array_equal(np.isfinite(lse.cpu().numpy()), fin)
        np.testing.assert_array_equal(np.isfinite(out.float().cpu().numpy()).all(-1), fin)
        spread = _chunk.reference(_chunk.make(P, n, H, seed=50), window=window, sinks=sinks)[3]
        err = np.abs(out.float().cpu().numpy() - ref[0])[fin]
        assert np.all(err <= _chunk.out_bound(ref[0], ref[2], spread, 400)[fin])


@pytest.mark.parametrize("P,n,H", [([2000], [64], 16), ([5000, 0], [40, 3], 64),
                                   ([0], [700], 8), ([9000], [1], 128), ([64] * 40, [2] * 40, 8),
                                   ([700] * 70, [3] * 70, 64)])
@pytest.mark.parametrize("layout", ["paged", "contiguous"])
def test_longer_batches(va, P, n, H, layout):
    """More units, splits and waves than the small cases have; rows sampled."""
    c = _chunk.make(P, n, H, seed=60, layout=layout)
    out, lse = _chunk.call(va, c)
    fma_out, fma_lse = _chunk.call(va, c, flags=1)     # the CUDA-core path, on every row
    assert float((lse - fma_lse).abs().max()) < 1e-4
    d = (out.float() - fma_out.float()).abs()
    assert float((d - 2 * 2.0 ** -8 * fma_out.float().abs()).max()) < 2e-2
    for b in sorted({0, len(P) - 1}):                  # and against the oracle, whole requests
        t = slice(int(c.q_indptr[b]), min(int(c.q_indptr[b + 1]), int(c.q_indptr[b]) + 4))
        sub = _chunk.Chunk(P=[P[b]], n=[t.stop - t.start], H=H, q=c.q[t], pool=c.pool,
                           key_rows=[c.key_rows[b]], slot_idx=c.slot_idx, kv_indptr=c.kv_indptr,
                           prefix_len=c.prefix_len,
                           q_indptr=torch.tensor([0, t.stop - t.start], dtype=torch.int32))
        _chunk.check(sub, out[t], lse[t])


@pytest.mark.parametrize("P,n,H,window", [([0, 0, 0], [700, 333, 1000], 64, 0),
                                          ([3000, 100], [90, 257], 64, 200), ([4000], [64], 128, 0),
                                          ([900] * 24, [1] * 24, 64, 0)])
def test_calls_back_to_back_give_the_same_bits(va, P, n, H, window):
    """Many calls in a row, nothing waited for between them: each one's rows are
    the first one's, bit for bit."""
    c = _chunk.make(P, n, H, seed=70, layout="contiguous" if n[0] == 700 else "paged")
    call = _chunk.call(va, c, window=window, prepare=True)
    out, lse = call()
    first = out.clone(), lse.clone()
    assert bool(torch.isfinite(first[1]).all())
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(60):
        out.fill_(9.0)
        for _ in range(4):
            call()
        differ += (out != first[0]).sum() + (lse != first[1]).sum()
    assert int(differ) == 0
    assert va.read_status(call.workspace) == 0
