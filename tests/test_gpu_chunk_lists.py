"""Chunk attention over lists that are not what the header asks for: shorter than
the new tokens.  Flagged, and the same rows on every path (needs an sm_103 GPU)."""
import numpy as np
import pytest
import torch

from tests import _chunk

pytestmark = pytest.mark.gpu

# prefill (packed lists) from 640 query rows per request on, the CUDA-core path, the
# split kernel
PATHS = {"auto": 0, "fma": 1, "tc1sm": 3}


@pytest.fixture(scope="module")
def va():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mla_speculative_decode_gb300 as m
    m.build()
    m.init()
    return m


def cut_list(c, b, m):
    """Request b's list ends after m entries, fewer than its new tokens: the prefix
    gives way altogether, and the tokens past the list have no row."""
    ind = c.kv_indptr.numpy().copy()
    gone = int(ind[b + 1] - ind[b]) - m
    s = c.slot_idx.numpy()
    c.slot_idx = torch.from_numpy(np.concatenate([s[:ind[b] + m], s[ind[b + 1]:]]))
    ind[b + 1:] -= gone
    c.kv_indptr = torch.from_numpy(ind)
    assert m < c.n[b]
    c.key_rows[b] = np.concatenate([c.key_rows[b][:m], np.full(c.n[b] - m, -1)])
    c.P[b] = 0


@pytest.mark.parametrize("path", list(PATHS.values()), ids=list(PATHS))
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3), (70, 65)])
@pytest.mark.parametrize("P,n,H,m", [(0, 100, 64, 10), (30, 100, 8, 64), (5, 300, 8, 130),
                                     (0, 70, 16, 1), (0, 200, 8, 0)])
def test_a_list_shorter_than_the_new_tokens(va, P, n, H, m, window, sinks, path):
    c = _chunk.make([P, 40], [n, 90], H, seed=300 + m)
    cut_list(c, 0, m)
    call = _chunk.call(va, c, flags=path, window=window, sinks=sinks, prepare=True)
    out, lse = call()
    _chunk.check(c, out, lse, window=window, sinks=sinks)
    assert va.read_status(call.workspace) == va.STATUS_BAD_INDPTR | va.STATUS_BAD_SLOT
