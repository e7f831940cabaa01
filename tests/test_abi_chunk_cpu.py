"""Argument checks of the chunk, weight and eviction entry points: every refusal
comes before any device work, so all of them show on a machine without a GPU."""
import pytest

import mla_speculative_decode_gb300 as va

A16 = 0x10000      # fake, never dereferenced
A256 = 0x20000


@pytest.fixture(scope="module")
def lib():
    va.build()
    return va.load()


CHUNK = dict(q=A16, kv=A16, num_slots=4096, stride=576, slot=A16, indptr=A16, prefix=A16,
             qind=A16, n=1000, B=2, total_q=5, H=8, scale=0.07, window=0, sinks=0, flags=0,
             ws=A256, ws_bytes=1 << 40, out=A16, lse=A16, stream=None)


def _paged(lib, **over):
    return lib.va_chunk_attn_paged(*(CHUNK | over).values())


def _contiguous(lib, **over):
    a = CHUNK | dict(slot=A16) | over
    a.pop("indptr")
    a.pop("n")
    return lib.va_chunk_attn_contiguous(*a.values())


COMMON = [
    (dict(q=None), -1), (dict(kv=None), -1), (dict(slot=None), -1), (dict(prefix=None), -1),
    (dict(qind=None), -1), (dict(ws=None), -1), (dict(out=None), -1), (dict(lse=None), -1),
    (dict(B=0), -2), (dict(B=65536), -2), (dict(H=0), -2), (dict(total_q=-1), -2),
    (dict(total_q=1 << 22, H=8), -2), (dict(num_slots=0), -2), (dict(stride=512), -2),
    (dict(window=-1), -2), (dict(sinks=-1), -2), (dict(flags=4), -2), (dict(flags=-1), -2),
    (dict(scale=float("inf")), -2),
    (dict(stride=580), -3), (dict(q=A16 + 8), -3), (dict(kv=A16 + 2), -3), (dict(out=A16 + 4), -3),
    (dict(ws=A256 + 16), -3), (dict(lse=A16 + 2), -3), (dict(prefix=A16 + 2), -3),
    (dict(qind=A16 + 1), -3), (dict(slot=A16 + 2), -3),
    (dict(ws_bytes=100), -4),
]


@pytest.mark.parametrize("over,code", COMMON + [(dict(indptr=None), -1),
                                                (dict(indptr=A16 + 2), -3), (dict(n=-1), -2),
                                                (dict(n=1 << 31), -2)])
def test_paged_chunk_errors(lib, over, code):
    assert _paged(lib, **over) == code


@pytest.mark.parametrize("over,code", COMMON + [(dict(slot=A16 + 4), -3)])
def test_contiguous_chunk_errors(lib, over, code):
    assert _contiguous(lib, **over) == code


def test_good_chunk_calls_end_at_the_device_check(lib):
    for flags in range(4):
        assert _paged(lib, flags=flags) in (-5, -7)
        assert _contiguous(lib, flags=flags) in (-5, -7)
    # no rows: q, out and lse may be NULL
    assert _paged(lib, total_q=0, q=None, out=None, lse=None) in (-5, -7)


def test_chunk_workspace_bytes(lib):
    f = lib.va_chunk_workspace_bytes
    for bad in ((0, 1, 1, 0, 0), (65536, 1, 1, 0, 0), (1, -1, 1, 0, 0), (1, 1, 0, 0, 0),
                (1, 1 << 24, 2, 0, 0), (1, 1, 1, 0, 4), (1, 1, 1, 0, -1), (1, 1, 1, -1, 0),
                (1, 1, 1, 1 << 31, 0)):
        assert f(*bad) == 0
    for B, total_q, H in ((1, 0, 1), (1, 1, 1), (8, 4096, 64), (65535, 1, 1), (1, 1 << 17, 128)):
        for flags in range(4):
            assert 256 <= f(B, total_q, H, 0, flags) < 1 << 32
    # many rows per request: the listed rows are packed first
    assert 0 <= f(1, 512, 64, 20000, 0) - f(1, 512, 64, 0, 0) - 20000 * 1152 < 1 << 16
    assert f(1, 10, 64, 20000, 0) - f(1, 10, 64, 0, 0) >= 20000 * 1152
    for few in (1, 2, 3, 9):
        assert f(1, few, 64, 20000, 0) == f(1, few, 64, 1, 0)


WEIGHTS = dict(q=A16, kv=A16, num_slots=4096, stride=576, slot=A16, indptr=A16, prefix=A16,
               qind=A16, lse=A16, win=None, n=1000, B=2, total_q=5, H=8, scale=0.07, window=0,
               sinks=0, flags=0, ws=A256, ws_bytes=1 << 40, wout=A16, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(q=None), -1), (dict(kv=None), -1), (dict(slot=None), -1), (dict(indptr=None), -1),
    (dict(prefix=None), -1), (dict(qind=None), -1), (dict(lse=None), -1), (dict(ws=None), -1),
    (dict(wout=None), -1),
    (dict(n=-1), -2), (dict(n=1 << 31), -2), (dict(B=0), -2), (dict(H=0), -2),
    (dict(window=-1), -2), (dict(sinks=-1), -2), (dict(flags=4), -2),
    (dict(wout=A16 + 2), -3), (dict(win=A16 + 1), -3), (dict(q=A16 + 8), -3),
    (dict(ws=A256 + 16), -3), (dict(ws_bytes=100), -4),
])
def test_weights_errors(lib, over, code):
    assert lib.va_kv_weights_paged(*(WEIGHTS | over).values()) == code


def test_good_weights_calls_end_at_the_device_check(lib):
    for over in (dict(), dict(win=A16), dict(total_q=0, q=None, lse=None), dict(flags=1)):
        assert lib.va_kv_weights_paged(*(WEIGHTS | over).values()) in (-5, -7)


def test_weights_workspace_bytes(lib):
    f = lib.va_kv_weights_workspace_bytes
    for bad in ((0, 1, 1, 1, 0), (1, -1, 1, 1, 0), (1, 1, 0, 1, 0), (1, 1, 1, -1, 0),
                (1, 1, 1, 1 << 31, 0), (1, 1, 1, 1, 9)):
        assert f(*bad) == 0
    assert 256 <= f(8, 4096, 64, 1 << 20, 0) < 1 << 32
    assert 256 <= f(1, 0, 1, 0, 0)


EVICT = dict(slot=A16, indptr=A16, prefix=A16, w=A16, n=1000, B=2, budget=100, sinks=4, recent=10,
             free=A16, cap=50, head=A16, so=A16, po=A16, wo=A16, ho=A16, status=None, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(slot=None), -1), (dict(indptr=None), -1), (dict(prefix=None), -1), (dict(w=None), -1),
    (dict(so=None), -1), (dict(po=None), -1), (dict(wo=None), -1), (dict(head=None), -1),
    (dict(ho=None), -1),
    (dict(B=0), -2), (dict(B=65536), -2), (dict(n=-1), -2), (dict(n=1 << 31), -2),
    (dict(budget=-1), -2), (dict(sinks=-1), -2), (dict(recent=-1), -2),
    (dict(budget=13), -2), (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), -2), (dict(cap=-1), -2),
    (dict(slot=A16 + 2), -3), (dict(w=A16 + 1), -3), (dict(ho=A16 + 2), -3),
    (dict(status=A16 + 2), -3),
])
def test_evict_errors(lib, over, code):
    assert lib.va_kv_evict(*(EVICT | over).values()) == code


def test_good_evict_calls_end_at_the_device_check(lib):
    assert lib.va_kv_evict(*EVICT.values()) in (-5, -7)
    assert lib.va_kv_evict(*(EVICT | dict(free=None, head=None, ho=None)).values()) in (-5, -7)
