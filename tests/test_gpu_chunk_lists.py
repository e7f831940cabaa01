"""Chunk attention over lists that are not what the header asks for: shorter than the new
tokens, with bounds that decrease, or outside the pool.  Flagged, and the same rows on
every path (needs an sm_103 GPU)."""
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


@pytest.mark.parametrize("path", list(PATHS.values()), ids=list(PATHS))
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 2), (100, 0), (64, 130)])
@pytest.mark.parametrize("ind", [[0, 600, 200, 800], [300, 900, 0, 600], [600, 1200, 0, 600]])
def test_list_bounds_that_decrease(va, ind, window, sinks, path):
    """The request whose bounds decrease has an empty list; those behind it have
    theirs, also where two requests' lists share entries.  What the workspace held
    before shows nowhere."""
    n, H, L = 20, 64, 600
    c = _chunk.make([L - n, 0, L - n], [n, n, n], H, seed=420, unused_nan=False)
    rng = np.random.default_rng(421)
    slots = rng.permutation(c.pool.shape[0])[:1200].astype(np.int32)
    c.slot_idx = torch.from_numpy(slots)
    c.kv_indptr = torch.tensor(ind, dtype=torch.int32)
    c.key_rows = [slots[ind[0]:ind[1]].astype(np.int64), np.full(n, -1),
                  slots[ind[2]:ind[3]].astype(np.int64)]
    ws = torch.full((va.load().va_chunk_workspace_bytes(3, 3 * n, H, 1200, path),), 0x41,
                    dtype=torch.uint8, device="cuda")
    out, lse = _chunk.call(va, c, flags=path, window=window, sinks=sinks, workspace=ws)
    _chunk.check(c, out, lse, window=window, sinks=sinks)
    assert va.read_status(ws) == va.STATUS_BAD_INDPTR | va.STATUS_BAD_SLOT


@pytest.mark.parametrize("H,flags", [(8, 0), (16, 0), (64, 0), (64, 1), (64, 3), (200, 0)])
def test_contiguous_starts_at_the_ends_of_64_bits(va, H, flags):
    """Rows that cannot be, however far outside the pool they start: no key has one."""
    c = _chunk.make([70, 200, 130, 90], [7] * 4, H, seed=440, layout="contiguous",
                    unused_nan=False)
    c.kv_start = torch.tensor([2 ** 63 - 1, -2 ** 63, 2 ** 63 - 100, int(c.kv_start[3])],
                              dtype=torch.int64)
    for b in range(3):
        c.key_rows[b] = np.full(c.P[b] + 7, -1)
    call = _chunk.call(va, c, flags=flags, prepare=True)
    out, lse = call()
    _chunk.check(c, out, lse)
    assert va.read_status(call.workspace) == va.STATUS_BAD_SLOT
