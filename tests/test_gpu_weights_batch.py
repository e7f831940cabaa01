"""Weight totals of batches that end early (needs an sm_103 GPU)."""
import numpy as np
import pytest
import torch

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
