"""The largest lists that the chunk, weight and eviction calls take: the kernels count list
positions in 32 bits and step past a list's end by up to a tile (or a block's step), so
longer ones are refused before any device work."""
import pytest

import mla_speculative_decode_gb300 as va
from tests.test_abi_chunk_cpu import CHUNK, EVICT, WEIGHTS

LISTS = 2 ** 31 - 1025             # chunk and weight calls
EVICTED = 2 ** 31 - 2 ** 25 - 1    # eviction


@pytest.fixture(scope="module")
def lib():
    va.build()
    return va.load()


@pytest.mark.parametrize("n,good", [(LISTS, True), (LISTS + 1, False), (2 ** 31 - 1, False)])
def test_lists_of_attention_and_weights(lib, n, good):
    want = (-5, -7) if good else (-2,)
    for flags in range(4):
        assert lib.va_chunk_attn_paged(*(CHUNK | dict(n=n, flags=flags)).values()) in want
        assert lib.va_kv_weights_paged(*(WEIGHTS | dict(n=n, flags=flags)).values()) in want
        assert (lib.va_chunk_workspace_bytes(2, 5, 8, n, flags) > 0) == good
        assert (lib.va_kv_weights_workspace_bytes(2, 5, 8, n, flags) > 0) == good


@pytest.mark.parametrize("n,good", [(EVICTED, True), (EVICTED + 1, False), (2 ** 31 - 1, False)])
def test_lists_of_eviction(lib, n, good):
    assert lib.va_kv_evict(*(EVICT | dict(n=n)).values()) in ((-5, -7) if good else (-2,))


def test_an_empty_list_may_be_null(lib):
    """num_entries 0: there is nothing to point to (an empty tensor's address is NULL)."""
    none = dict(n=0, slot=None)
    assert lib.va_chunk_attn_paged(*(CHUNK | none).values()) in (-5, -7)
    assert lib.va_chunk_attn_paged(*(CHUNK | none | dict(indptr=None)).values()) == -1
    assert lib.va_kv_weights_paged(*(WEIGHTS | none | dict(wout=None)).values()) in (-5, -7)
    assert lib.va_kv_weights_paged(*(WEIGHTS | none | dict(ws=None)).values()) == -1
    none |= dict(w=None, so=None, wo=None)
    assert lib.va_kv_evict(*(EVICT | none).values()) in (-5, -7)
    assert lib.va_kv_evict(*(EVICT | none | dict(po=None)).values()) == -1


def test_batches_of_many_requests_pack_their_lists(lib):
    """More than 128 rows per request, more than 96 requests: room for the listed rows."""
    f = lib.va_chunk_workspace_bytes
    n = 20000
    for B, packs in ((96, False), (97, True), (4096, True)):
        assert (f(B, 3 * B, 64, n, 0) - f(B, 3 * B, 64, 1, 0) >= (n - 1) * 1152) == packs
        assert f(B, 2 * B, 64, n, 0) == f(B, 2 * B, 64, 1, 0)         # 128 rows: no packing
        assert f(B, 3 * B, 64, n, 3) == f(B, 3 * B, 64, 1, 3)
    assert f(4096, 3 * 4096, 64, 1 << 22, 0) == f(4096, 3 * 4096, 64, 1 << 23, 0)
