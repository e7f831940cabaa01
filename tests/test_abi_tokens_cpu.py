"""Argument checks of the entry points around attention (rotary positions, cache rows, sampling):
every refusal comes before any device work, so all of them show on a machine without a
GPU; and the frequencies, which are host arithmetic."""
import ctypes
import math

import pytest

import mla_speculative_decode_gb300 as va

A16 = 0x10000      # fake, never dereferenced
FREQ = (ctypes.c_double * 128)(*([0.5] * 128))
F = ctypes.addressof(FREQ)
BAD = (ctypes.c_double * 128)(*([0.5] * 31 + [float("nan")] + [0.5] * 96))
HUGE = (ctypes.c_double * 128)(*([0.5, 2.0 ** 40] + [0.5] * 126))


@pytest.fixture(scope="module")
def lib():
    va.build()
    return va.load()


ROPE = dict(x=A16, xt=512, xh=64, out=A16 + 4096, ot=512, oh=64, dtype=1, pos=A16, tokens=5,
            heads=8, width=64, off=0, rot=64, freq=F, amp=1.0, flags=0, stream=None)


def rope(lib, **over):
    return lib.va_rope(*(ROPE | over).values())


@pytest.mark.parametrize("over,code", [
    (dict(x=None), -1), (dict(out=None), -1), (dict(pos=None), -1), (dict(freq=None), -1),
    (dict(tokens=-1), -2), (dict(tokens=1 << 31), -2), (dict(heads=0), -2),
    (dict(heads=65536), -2), (dict(width=0), -2), (dict(width=63), -2), (dict(rot=63), -2),
    (dict(rot=0), -2), (dict(rot=-2), -2), (dict(rot=66), -2), (dict(off=1), -2), (dict(off=-1), -2),
    (dict(rot=258, width=512, xh=512, oh=512, ot=4096), -2), (dict(off=2 ** 31 - 1), -2),
    (dict(dtype=3), -2), (dict(dtype=-1), -2), (dict(flags=4), -2), (dict(flags=-1), -2),
    (dict(amp=float("nan")), -2), (dict(freq=ctypes.addressof(BAD)), -2),
    (dict(freq=ctypes.addressof(HUGE)), -2),
    (dict(xt=-1), -2), (dict(oh=-1), -2), (dict(xt=(1 << 40) + 1), -2),
    # one token is at most a launch; a tensor spans at most 2^50 elements
    (dict(heads=65535, width=16385, xh=16385, oh=16385, xt=1 << 31, ot=1 << 31), -2),
    (dict(tokens=2 ** 31 - 1, xt=1 << 20), -2), (dict(tokens=2 ** 31 - 1, ot=1 << 20), -2),
    (dict(heads=65535, xh=1 << 35, ot=1 << 30), -2),
    (dict(oh=63), -2), (dict(ot=511), -2), (dict(oh=0), -2), (dict(ot=0), -2),
    (dict(ot=64, oh=64), -2), (dict(ot=64, oh=319), -2),
    (dict(x=A16 + 1), -3), (dict(out=A16 + 1), -3), (dict(pos=A16 + 2), -3),
    (dict(dtype=0, x=A16 + 2), -3),
])
def test_rope_errors(lib, over, code):
    assert rope(lib, **over) == code


@pytest.mark.parametrize("over", [
    dict(), dict(dtype=0), dict(dtype=2, flags=3), dict(x=A16 + 2), dict(xt=0, xh=0),
    dict(tokens=0, x=None, out=None, pos=None), dict(ot=64, oh=320), dict(tokens=1, ot=0),
    dict(heads=1, oh=0, ot=64), dict(width=65, off=1, xh=65, oh=65, ot=520), dict(rot=2),
    dict(width=256, rot=256, xh=256, oh=256, xt=2048, ot=2048), dict(tokens=2 ** 31 - 1),
    dict(heads=65535, width=16384, xh=16384, oh=16384, xt=1 << 31, ot=1 << 31)])
def test_good_rope_calls_end_at_the_device_check(lib, over):
    assert rope(lib, **over) in (-5, -7)


APPEND = dict(pool=A16, num_slots=100, stride=576, kv=A16, row=576, dtype=1, w=A16, eps=1e-6,
              slots=A16, pos=A16, tokens=5, freq=F, amp=1.0, flags=0, q=A16, qt=512, qh=64,
              qo=A16, qot=512, qoh=64, heads=8, status=None, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(pool=None), -1), (dict(kv=None), -1), (dict(slots=None), -1), (dict(pos=None), -1),
    (dict(freq=None), -1), (dict(q=None), -1), (dict(qo=None), -1),
    (dict(num_slots=0), -2), (dict(num_slots=1 << 31), -2), (dict(stride=568), -2),
    (dict(row=-8), -2), (dict(dtype=3), -2), (dict(tokens=-1), -2), (dict(tokens=1 << 31), -2),
    (dict(heads=-1), -2), (dict(heads=65536), -2), (dict(flags=2), -2), (dict(eps=-1.0), -2),
    (dict(eps=float("nan")), -2), (dict(amp=float("inf")), -2),
    (dict(freq=ctypes.addressof(BAD)), -2), (dict(qoh=32), -2), (dict(qt=-1), -2),
    (dict(num_slots=2 ** 31 - 1, stride=1 << 20), -2), (dict(tokens=2 ** 31 - 1, row=1 << 20), -2),
    (dict(stride=580), -3), (dict(row=580), -3), (dict(pool=A16 + 8), -3), (dict(kv=A16 + 8), -3),
    (dict(w=A16 + 8), -3), (dict(slots=A16 + 2), -3), (dict(pos=A16 + 1), -3),
    (dict(status=A16 + 2), -3), (dict(q=A16 + 1), -3), (dict(qo=A16 + 1), -3),
])
def test_append_errors(lib, over, code):
    assert lib.va_kv_append_paged(*(APPEND | over).values()) == code


@pytest.mark.parametrize("over", [
    dict(), dict(heads=0, q=None, qo=None), dict(w=None), dict(dtype=0), dict(q=A16 + 2),
    dict(tokens=0, kv=None, slots=None, pos=None, q=None, qo=None), dict(tokens=1, row=1)])
def test_good_append_calls_end_at_the_device_check(lib, over):
    assert lib.va_kv_append_paged(*(APPEND | over).values()) in (-5, -7)


INV = dict(rot=64, base=10000.0, scaling=3, factor=40.0, orig=4096, fast=32.0, slow=1.0, out=F)


@pytest.mark.parametrize("over,code", [
    (dict(out=None), -1), (dict(rot=0), -2), (dict(rot=63), -2), (dict(rot=258), -2),
    (dict(base=1.0), -2), (dict(base=float("inf")), -2), (dict(base=float("nan")), -2),
    (dict(scaling=4), -2), (dict(scaling=-1), -2), (dict(factor=0.5), -2),
    (dict(factor=float("nan")), -2), (dict(scaling=1, factor=0.0), -2), (dict(orig=0), -2),
    (dict(slow=0.0), -2), (dict(fast=0.5), -2), (dict(fast=float("inf")), -2),
    (dict(rot=2, scaling=2), -2)])
def test_frequency_errors(lib, over, code):
    assert lib.va_rope_inv_freq(*(INV | over).values()) == code


def test_frequencies():
    plain = va.rope_inv_freq(64, 10000.0)
    assert plain == pytest.approx([10000.0 ** (-i / 32) for i in range(32)], rel=1e-14)
    assert va.rope_inv_freq(64, scaling="linear", factor=4.0) == \
        pytest.approx([f / 4 for f in plain], rel=1e-14)
    # the slowest pair's wavelength grows by the factor, the fastest keeps its own
    ntk = va.rope_inv_freq(64, scaling="ntk", factor=8.0)
    assert ntk[0] == 1.0 and ntk[-1] == pytest.approx(plain[-1] / 8, rel=1e-12)
    yarn = va.rope_inv_freq(64, scaling="yarn", factor=40.0, original_len=4096)
    for i, (f, y) in enumerate(zip(plain, yarn)):
        turns = 4096 * f / (2 * math.pi)
        assert f / 40 * (1 - 1e-14) <= y <= f * (1 + 1e-14)
        if turns > 32 * plain[0] / plain[1]:      # a pair or more beyond the border
            assert y == pytest.approx(f, rel=1e-14)
        if turns < plain[1] / plain[0]:
            assert y == pytest.approx(f / 40, rel=1e-14)
    assert va.rope_inv_freq(2) == [1.0] and len(va.rope_inv_freq(256)) == 128
    with pytest.raises(ValueError):
        va.rope_inv_freq(64, scaling="other")
    with pytest.raises(va.VaError):
        va.rope_inv_freq(63)


A256 = 0x20000
SAMPLE = dict(logits=A16, stride=1000, dtype=0, rows=3, V=1000, t=A16, k=A16, p=A16, m=A16, u=A16,
              tok=A16, lp=A16, status=None, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(logits=None), -1), (dict(u=None), -1), (dict(tok=None), -1),
    (dict(rows=-1), -2), (dict(rows=(1 << 23) + 1), -2), (dict(V=0), -2),
    (dict(V=(1 << 20) + 1), -2), (dict(dtype=3), -2), (dict(dtype=-1), -2), (dict(stride=-1), -2),
    (dict(stride=(1 << 40) + 1), -2), (dict(rows=1 << 23, stride=1 << 30), -2),
    (dict(logits=A16 + 2), -3), (dict(dtype=1, logits=A16 + 1), -3), (dict(t=A16 + 2), -3),
    (dict(k=A16 + 2), -3), (dict(p=A16 + 2), -3), (dict(m=A16 + 2), -3), (dict(u=A16 + 2), -3),
    (dict(tok=A16 + 2), -3), (dict(lp=A16 + 2), -3), (dict(status=A16 + 2), -3),
])
def test_sample_errors(lib, over, code):
    assert lib.va_sample(*(SAMPLE | over).values()) == code


@pytest.mark.parametrize("over", [
    dict(), dict(t=None, k=None, p=None, m=None, lp=None), dict(dtype=1, logits=A16 + 2),
    dict(stride=0), dict(V=1 << 20, rows=1 << 23), dict(rows=0, logits=None, u=None, tok=None)])
def test_good_sample_calls_end_at_the_device_check(lib, over):
    assert lib.va_sample(*(SAMPLE | over).values()) in (-5, -7)


TREE = dict(root=A16, logits=A16, dtype=0, V=1000, tok=A16, par=A16, slots=A16, B=2, T=8, t=A16,
            k=A16, p=A16, m=A16, u=A16, ws=A256, n=1 << 20, alen=A16, nodes=A16, aslots=A16,
            bonus=A16, lp=A16, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(root=None), -1), (dict(logits=None), -1), (dict(tok=None), -1), (dict(par=None), -1),
    (dict(u=None), -1), (dict(ws=None), -1), (dict(alen=None), -1), (dict(nodes=None), -1),
    (dict(bonus=None), -1), (dict(B=0), -2), (dict(B=65536), -2), (dict(T=0), -2), (dict(T=65), -2),
    (dict(V=0), -2), (dict(V=(1 << 20) + 1), -2), (dict(dtype=3), -2),
    (dict(root=A16 + 2), -3), (dict(ws=A256 + 16), -3), (dict(aslots=A16 + 2), -3),
    (dict(slots=A16 + 1), -3), (dict(lp=A16 + 2), -3), (dict(u=A16 + 2), -3), (dict(k=A16 + 1), -3),
    (dict(n=300), -4),
])
def test_sampled_acceptance_errors(lib, over, code):
    assert lib.va_tree_accept_sampled(*(TREE | over).values()) == code


def test_good_sampled_acceptance_calls_end_at_the_device_check(lib):
    for over in (dict(), dict(t=None, k=None, p=None, m=None), dict(slots=None, aslots=None, lp=None),
                 dict(dtype=2, root=A16 + 2), dict(V=1 << 20)):
        assert lib.va_tree_accept_sampled(*(TREE | over).values()) in (-5, -7)
    f = lib.va_tree_accept_sampled_workspace_bytes
    assert f(0, 1) == f(1, 0) == f(65536, 1) == f(1, 65) == 0
    assert f(1, 1) == 256 * 3 and f(65535, 64) >= 256 + 8 * 65535 * 65
    assert lib.va_tree_accept_sampled(*(TREE | dict(n=f(2, 8))).values()) in (-5, -7)
    assert lib.va_tree_accept_sampled(*(TREE | dict(n=f(2, 8) - 1)).values()) == -4
