"""Attention-weight totals per key (va_kv_weights_paged) against the fp64
oracle (needs an sm_103 GPU)."""
import numpy as np
import pytest
import torch

import oracle
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


def run(va, c, lse, w, **kw):
    return va.kv_weights(c.dev("q"), c.dev("pool"), c.dev("slot_idx"), c.dev("kv_indptr"),
                         c.dev("prefix_len"), c.dev("q_indptr"), lse, w,
                         **(dict(sm_scale=synth.SM_SCALE) | kw))


def check(c, got, lse, w, spread, *, window=0, sinks=0, sm_scale=synth.SM_SCALE, fresh=None):
    """Entries of the requests' keys within the error bound of the sum (each term
    off by the score's error, the rounding of lse and exp2, a running sum of as
    many terms as there are rows), all others untouched."""
    ref = oracle.chunk_weights(synth.as_u16(c.q), synth.as_u16(c.pool), c.key_rows, c.P,
                               c.q_indptr.numpy(), lse, sm_scale, window, sinks)
    got = got.cpu().numpy().astype(np.float64)
    before = np.zeros_like(got) if w is None else w.astype(np.float64)
    left = np.ones(got.shape, dtype=bool)
    for b, x in enumerate(ref):
        e = slice(int(c.kv_indptr[b]), int(c.kv_indptr[b]) + len(x))
        left[e] = False
        rel = _chunk.score_error(spread) + 2.0 ** -22 * np.max(np.abs(lse[np.isfinite(lse)]),
                                                              initial=0.0)
        rel += (c.n[b] * c.H + 2) * 2.0 ** -24
        bound = rel * x + 2.0 ** -23 * np.abs(before[e] + x) + 1e-30
        err = np.abs(got[e] - (before[e] + x))
        assert np.all(err <= bound), (b, float(np.max(err / (bound + 1e-300))))
    np.testing.assert_array_equal(got[left], (before if fresh is None else fresh)[left])


CASES = [
    ([0], [1], 1), ([1], [1], 8), ([127], [1], 64), ([128], [1], 128), ([0], [70], 5),
    ([600], [17], 8), ([129, 0, 64, 3], [1, 1, 1, 1], 16), ([0, 200, 31, 7], [3, 0, 40, 1], 5),
    ([300, 2, 0, 77, 129], [1, 1, 33, 64, 5], 24), ([90, 700], [50, 1], 64), ([256], [2], 33),
]


@pytest.mark.parametrize("path", list(PATHS.values()), ids=list(PATHS))
@pytest.mark.parametrize("window,sinks", [(0, 0), (30, 3), (1, 0), (130, 70)])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_weights(va, case, window, sinks, path):
    P, n, H = CASES[case]
    c = _chunk.make(P, n, H, seed=200 + case, list_gap=case % 3, q_before=case % 2, q_behind=3)
    _, lse, _, spread = _chunk.reference(c, window=window, sinks=sinks)
    lse = np.where(np.isnan(lse), 7.0, lse).astype(np.float32)
    rng = np.random.default_rng(case)
    w = rng.exponential(size=c.slot_idx.numel()).astype(np.float32)
    got = run(va, c, torch.from_numpy(lse).cuda(), torch.from_numpy(w).cuda(), window=window,
              sinks=sinks, flags=path)
    check(c, got, lse, w, spread, window=window, sinks=sinks)
    # totals that start at zero, and in place
    got = run(va, c, torch.from_numpy(lse).cuda(), None, window=window, sinks=sinks, flags=path)
    check(c, got, lse, None, spread, window=window, sinks=sinks)
    t = torch.from_numpy(w).cuda()
    run(va, c, torch.from_numpy(lse).cuda(), t, window=window, sinks=sinks, flags=path,
        weights_out=t)
    check(c, t, lse, w, spread, window=window, sinks=sinks)


@pytest.mark.parametrize("path", list(PATHS.values()), ids=list(PATHS))
def test_keys_without_a_row_and_rows_without_a_key(va, path):
    c = _chunk.make([70, 64], [3, 2], 8, seed=5)
    for b, j, v in ((0, 3, -1), (0, 71, 10 ** 6), (1, 0, c.pool.shape[0])):
        c.slot_idx[int(c.kv_indptr[b]) + j] = v
        c.key_rows[b][j] = -1
    _, lse, _, spread = _chunk.reference(c)
    lse = lse.astype(np.float32)
    lse[1, 3] = lse[4, 0] = -np.inf          # rows that saw nothing give nothing
    call = va.prepare_kv_weights(c.dev("q"), c.dev("pool"), c.dev("slot_idx"), c.dev("kv_indptr"),
                                 c.dev("prefix_len"), c.dev("q_indptr"),
                                 torch.from_numpy(lse).cuda(), None, sm_scale=synth.SM_SCALE,
                                 flags=path)
    check(c, call(), lse, None, spread)
    assert va.read_status(call.workspace) == va.STATUS_BAD_SLOT


@pytest.mark.parametrize("path", list(PATHS.values()), ids=list(PATHS))
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_a_token_does_not_see_gets_nothing_from_it(va, bad, path):
    P, n, H = [100], [20], 8
    c = _chunk.make(P, n, H, seed=21)
    ref = _chunk.reference(c, window=50, sinks=2)
    lse = ref[1].astype(np.float32)
    c.q[5:7] = bad                       # two tokens whose own weights are lost
    j = np.arange(120)
    seen = ((j <= 105) & ((j > 55) | (j < 2))) | ((j <= 106) & ((j > 56) | (j < 2)))
    got = run(va, c, torch.from_numpy(lse).cuda(), None, window=50, sinks=2, flags=path)
    got = got.cpu().numpy()
    assert not np.isfinite(got[seen]).any()
    assert np.isfinite(got[~seen]).all()


@pytest.mark.parametrize("path", list(PATHS.values()), ids=list(PATHS))
def test_weights_are_the_same_every_time(va, path):
    c = _chunk.make([900, 40], [40, 2], 16, seed=22)
    _, lse = _chunk.call(va, c)
    first = run(va, c, lse, None, flags=path)
    for _ in range(5):
        assert torch.equal(run(va, c, lse, None, flags=path), first)
    # every row's weights sum to one
    want = [m * 16 for m in c.n]
    for b in range(2):
        e = slice(int(c.kv_indptr[b]), int(c.kv_indptr[b + 1]))
        assert abs(float(first[e].double().sum()) - want[b]) <= 1e-4 * want[b]


def test_no_tokens_copies_the_totals(va):
    c = _chunk.make([10, 3], [0, 0], 4, seed=10)
    w = torch.rand(13, device="cuda")
    got = run(va, c, torch.empty(0, 4, device="cuda"), w, weights_out=torch.zeros(13, device="cuda"))
    assert torch.equal(got, w)


def test_refusals(va):
    c = _chunk.make([10], [3], 4, seed=15)
    lse = torch.zeros(3, 4, device="cuda")
    with pytest.raises(ValueError):
        run(va, c, lse[:2], None)
    with pytest.raises(TypeError):
        run(va, c, lse.double(), None)
    with pytest.raises(ValueError):
        run(va, c, lse, torch.zeros(5, device="cuda"))
    with pytest.raises(ValueError):
        run(va, c, lse, torch.zeros(13))
    with pytest.raises(va.VaError):
        run(va, c, lse, None, window=-2)
    with pytest.raises(va.VaError) as e:
        run(va, c, lse, None, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert e.value.code == -4
