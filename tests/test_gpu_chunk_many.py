"""Chunk attention of batches of hundreds and thousands of requests (needs an sm_103 GPU)."""
import numpy as np
import pytest
import torch

import synth
from tests import _chunk
from tests.test_gpu_chunk_long import marked, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def va():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mla_speculative_decode_gb300 as m
    m.build()
    m.init()
    return m


@pytest.mark.parametrize("layout", ["paged", "contiguous"])
@pytest.mark.parametrize("B", [96, 97, 300])
@pytest.mark.parametrize("n,H", [(1, 100), (2, 64), (3, 64), (1, 200), (5, 100)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
def test_every_key_counts_once(va, n, H, B, window, sinks, layout):
    """Requests of n tokens and of none, with 0 to 400 keys in front."""
    rng = np.random.default_rng(B + H)
    P = rng.integers(0, 400, size=B).tolist()
    ns = [n if rng.random() < 0.9 else 0 for _ in range(B)]
    c = marked(P, ns, H, seed=560, layout=layout)
    call = _chunk.call(va, c, window=window, sinks=sinks, prepare=True)
    out, lse = call()
    ref, ref_lse, spread = reference(c, window, sinks)
    N = 400 + n
    rel = 2.0 ** -7 * (1 + 2.0 ** -7) + 2 * _chunk.score_error(spread) + 2 * N * 2.0 ** -24
    assert bool(((out.double() - ref).abs() <= rel * ref + 1e-30).all())
    bound = _chunk.score_error(spread) + N * 2.0 ** -24 + 2.0 ** -22 * ref_lse.abs()
    assert bool(((lse.double() - ref_lse).abs() <= bound).all())
    assert va.read_status(call.workspace) == 0


@pytest.mark.parametrize("L,entries", [(6, 0), (6, 1 << 22), (30, 0)])
def test_the_largest_batch(va, L, entries):
    """65535 requests of one token of 200 heads.  With 4 Mi entries the lists are too long
    to be packed.  The time does not grow with the square of the requests."""
    B, H = 65535, 200
    g = torch.Generator(device="cuda").manual_seed(561)
    q = torch.randn(B, H, 576, generator=g, device="cuda", dtype=torch.bfloat16)
    pool = torch.randn(5000, 576, generator=g, device="cuda", dtype=torch.bfloat16)
    slots = torch.randint(0, 5000, (max(entries, B * L),), generator=g, device="cuda",
                          dtype=torch.int32)
    ind = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    P = torch.full((B,), L - 1, dtype=torch.int32, device="cuda")
    call = va.prepare_chunk_paged(q, pool, slots, ind * L, P, ind, sm_scale=synth.SM_SCALE)
    call()
    a, b = torch.cuda.Event(True), torch.cuda.Event(True)
    a.record()
    out, lse = call()
    b.record()
    b.synchronize()
    assert a.elapsed_time(b) < 500, a.elapsed_time(b)      # ms
    assert va.read_status(call.workspace) == 0
    # the last requests, in 64 bits
    for r in (0, 31, 32, 40000, B - 1):
        k = pool[slots[r * L:(r + 1) * L].long()].double()
        s = (q[r].double() @ k.t()) * synth.SM_SCALE
        want = torch.logsumexp(s, -1)
        assert float((lse[r].double() - want).abs().max()) < 1e-4
        o = torch.softmax(s, -1) @ k[:, :512]
        mass = torch.softmax(s, -1) @ k[:, :512].abs()
        assert bool(((out[r].double() - o).abs() <= 2.0 ** -8 * 1.02 * (o.abs() + mass)).all())
