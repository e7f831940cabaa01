"""Weight totals of batches that end early, of entries that no request's keys cover, and
on other streams (needs an sm_103 GPU)."""
import numpy as np
import pytest
import torch

import oracle
import synth
from tests import _chunk

pytestmark = pytest.mark.gpu

PATHS = {"auto": 0, "fma": 1, "tc1sm": 3}


@pytest.fixture(scope="module")
def va():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mla_speculative_decode_gb300 as m
    m.build()
    m.init()
    return m


def args(c):
    return [c.dev(k) for k in ("q", "pool", "slot_idx", "kv_indptr", "prefix_len", "q_indptr")]


@pytest.mark.parametrize("path", list(PATHS.values()), ids=list(PATHS))
@pytest.mark.parametrize("B,T,H", [(3, 5, 4), (40, 3, 8), (3, 40, 8), (70, 2, 64)])
@pytest.mark.parametrize("end", [1, 2])
def test_query_bounds_that_decrease_end_the_batch(va, B, T, H, end, path):
    """q_indptr falls by one after `end` requests: those before have their rows'
    weights, that one and those behind it add nothing to their totals."""
    c = _chunk.make([70] * B, [T] * B, H, seed=400 + B, list_gap=2)
    lse = _chunk.call(va, c)[1]
    w = torch.rand(c.slot_idx.numel(), generator=torch.Generator().manual_seed(1)).cuda()
    whole = va.kv_weights(*args(c), lse, w, sm_scale=synth.SM_SCALE, flags=path)
    c.q_indptr[end + 1:] -= T + 1
    call = va.prepare_kv_weights(*args(c), lse, w, sm_scale=synth.SM_SCALE, flags=path)
    got = call()
    e = int(c.kv_indptr[end])
    assert torch.equal(got[e:], w[e:])
    # (the sums of a key may be cut into runs at other places: their order)
    assert bool((whole[:e] != w[:e]).any())
    assert torch.allclose(got[:e], whole[:e], rtol=T * H * 2.0 ** -23, atol=1e-30)
    assert va.read_status(call.workspace) == va.STATUS_BAD_INDPTR


@pytest.mark.parametrize("path", list(PATHS.values()), ids=list(PATHS))
@pytest.mark.parametrize("ind", [[50, 100, 20, 40], [700, 1300, 0, 600], [300, 301, 100, 290]])
@pytest.mark.parametrize("window,sinks", [(0, 0), (9, 2)])
def test_list_bounds_that_decrease(va, ind, window, sinks, path):
    """The request whose bounds decrease has an empty list; the one behind it has its
    own, although it lies before the first one's."""
    n, H = 7, 8
    L = [ind[1] - ind[0], 0, ind[3] - ind[2]]
    P = [max(0, L[0] - n), 0, L[2] - n]
    c = _chunk.make(P, [min(n, L[0]), 2, n], H, seed=430)
    slots = c.slot_idx.numpy()
    two = slots[c.kv_indptr[2]:c.kv_indptr[2] + L[2]]
    lists = np.full(1400, -5, dtype=np.int32)
    lists[ind[0]:ind[1]] = slots[:L[0]]
    lists[ind[2]:ind[3]] = two
    c.slot_idx = torch.from_numpy(lists)
    c.key_rows[1] = np.full(2, -1)
    c.kv_indptr = torch.tensor(ind, dtype=torch.int32)
    _, lse, _, spread = _chunk.reference(c, window=window, sinks=sinks)
    lse = lse.astype(np.float32)
    w = np.random.default_rng(431).random(1400).astype(np.float32)
    call = va.prepare_kv_weights(*args(c), torch.from_numpy(lse).cuda(),
                                 torch.from_numpy(w).cuda(), sm_scale=synth.SM_SCALE,
                                 window=window, sinks=sinks, flags=path)
    got = call().cpu().numpy()
    ref = oracle.chunk_weights(synth.as_u16(c.q), synth.as_u16(c.pool), c.key_rows, c.P,
                               c.q_indptr.numpy(), lse, synth.SM_SCALE, window, sinks)
    want = w.astype(np.float64)
    for b in (0, 2):
        want[ind[b]:ind[b] + L[b]] += ref[b]
    rel = _chunk.score_error(spread) + 2.0 ** -22 * np.abs(lse[np.isfinite(lse)]).max() \
        + (n * H + 2) * 2.0 ** -24
    assert np.all(np.abs(got - want) <= rel * (want - w) + 2.0 ** -23 * want)
    assert va.read_status(call.workspace) == va.STATUS_BAD_INDPTR


@pytest.mark.parametrize("path", list(PATHS.values()), ids=list(PATHS))
def test_a_prepared_call_gives_uncovered_entries_the_totals_of_its_time(va, path):
    """Entries behind a request's keys: weights_in as it is when the call runs (zero
    without one), not as it was when the call was prepared."""
    c = _chunk.make([30, 5], [3, 2], 8, seed=410, list_gap=4)
    lse = _chunk.call(va, c)[1]
    w = torch.rand(c.slot_idx.numel(), generator=torch.Generator().manual_seed(2)).cuda()
    call = va.prepare_kv_weights(*args(c), lse, w, sm_scale=synth.SM_SCALE, flags=path)
    call()
    w += 1
    got = call()
    behind = np.concatenate([np.arange(int(c.kv_indptr[b]) + c.P[b] + c.n[b],
                                       int(c.kv_indptr[b + 1])) for b in range(2)])
    assert behind.size == 8
    assert torch.equal(got[behind], w[behind])
    fresh = va.prepare_kv_weights(*args(c), lse, None, sm_scale=synth.SM_SCALE, flags=path)
    fresh().fill_(7.0)
    assert bool((fresh()[behind] == 0).all())


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("start", [False, True])
def test_totals_without_weights_out_on_another_stream(va, start, handle):
    """All of the call's work is on the stream it was given: what is still queued on the
    current stream does not come between."""
    c = _chunk.make([30, 5], [3, 2], 8, seed=411, list_gap=4)
    lse = _chunk.call(va, c)[1]
    w = torch.rand(c.slot_idx.numel(), generator=torch.Generator().manual_seed(3)).cuda()
    w = w if start else None
    want = va.kv_weights(*args(c), lse, w, sm_scale=synth.SM_SCALE)
    a = args(c)
    side = torch.cuda.Stream()
    first = torch.empty(c.slot_idx.numel(), dtype=torch.float32, pin_memory=True)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)          # the current stream is busy for 0.1 s
    got = va.kv_weights(*a, lse, w, sm_scale=synth.SM_SCALE,
                        stream=side.cuda_stream if handle else side)
    side.synchronize()
    assert not torch.cuda.current_stream().query()
    with torch.cuda.stream(side):
        first.copy_(got, non_blocking=True)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(first, want.cpu()) and torch.equal(got, want)


@pytest.mark.parametrize("path", list(PATHS.values()), ids=list(PATHS))
def test_no_tokens_at_all_in_many_requests(va, path):
    """A call without query rows copies the totals of every request's keys, reports bad
    bounds, and touches nothing else."""
    c = _chunk.make([10, 0, 700, 3] * 20, [0] * 80, 4, seed=412, list_gap=2)
    w = torch.rand(c.slot_idx.numel(), generator=torch.Generator().manual_seed(5)).cuda()
    c.prefix_len[7] = -1
    call = va.prepare_kv_weights(*args(c), torch.empty(0, 4, device="cuda"), w,
                                 weights_out=torch.full_like(w, -2.0), sm_scale=synth.SM_SCALE,
                                 flags=path)
    got = call().cpu()
    want = torch.full_like(got, -2.0)
    for b in range(80):
        e = int(c.kv_indptr[b])
        n = max(int(c.prefix_len[b]), 0)
        want[e:e + n] = w[e:e + n].cpu()
    assert torch.equal(got, want)
    assert va.read_status(call.workspace) == va.STATUS_BAD_INDPTR
