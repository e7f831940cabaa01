"""Rotary positions and the new tokens' cache rows (va_rope, va_kv_append_paged) against the
oracle in 64 bits (needs an sm_103 GPU)."""
import numpy as np
import pytest
import torch

import oracle
from tests import _tokens

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def va():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mla_speculative_decode_gb300 as m
    m.build()
    m.init()
    return m


def heads(tokens, H, width, dtype, seed, buf_width=None, col=0, device="cuda"):
    """[tokens, H, width] inside a buffer whose other columns hold NaN."""
    g = torch.Generator().manual_seed(seed)
    buf = torch.full((tokens, H, buf_width or width), float("nan"), dtype=dtype, device=device)
    x = buf[..., col:col + width]
    x.copy_(torch.randn(tokens, H, width, generator=g).to(dtype))
    return buf, x


def positions(n, seed, hi=1 << 20, lo=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(lo, hi, (n,), generator=g, dtype=torch.int32).cuda()


def check(got, x, pos, freq, **kw):
    xs = _tokens.f64(x)
    want = oracle.rope(xs, pos.cpu().numpy(), freq, **kw)
    kw.pop("inverse", None)
    bound = _tokens.rope_bound(want, xs, x.dtype, len(freq), **kw)
    err = np.abs(_tokens.f64(got) - np.where(bound == 0, xs, want))
    assert np.all(err <= bound), float(np.max(err - bound))


CASES = [
    # tokens, heads, width, rot, offset
    (1, 1, 64, 64, 0), (1, 8, 64, 64, 0), (3, 5, 64, 64, 0), (257, 16, 64, 64, 0),
    (33, 7, 192, 64, 128), (130, 3, 80, 48, 0), (20, 4, 96, 32, 64), (7, 2, 256, 256, 0),
    (5, 3, 7, 2, 3), (9, 2, 65, 64, 1), (40, 1, 50, 6, 44), (6, 4, 130, 2, 0), (2, 130, 24, 16, 8),
]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,H,width,rot,off", CASES)
def test_rope_matches_the_oracle(va, tokens, H, width, rot, off, interleaved, dtype):
    _, x = heads(tokens, H, width, dtype, 1)
    pos = positions(tokens, 2)
    freq = va.rope_inv_freq(rot)
    kw = dict(rot_offset=off, interleaved=interleaved)
    got = va.rope(x, pos, freq, **kw)
    check(got, x, pos, freq, **kw)
    same = x.clone()
    assert va.rope(same, pos, freq, out=same, **kw) is same
    assert torch.equal(same, got)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("scaling", ["linear", "ntk", "yarn"])
def test_scaled_inverse_and_amplitude(va, scaling, interleaved):
    freq = va.rope_inv_freq(64, 50000.0, scaling=scaling, factor=16.0, original_len=4096)
    _, x = heads(50, 6, 128, F32, 3)
    pos = positions(50, 4)
    kw = dict(rot_offset=64, interleaved=interleaved, amplitude=1.277, inverse=True)
    check(va.rope(x, pos, freq, **kw), x, pos, freq, **kw)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("x_at,out_at", [((192, 128), (576, 512)), ((192, 128), (67, 1)),
                                         ((71, 3), (576, 512)), ((68, 4), (72, 8))])
def test_views_of_wider_tensors(va, dtype, interleaved, x_at, out_at):
    """From one tensor's columns into another's, aligned to 16 bytes or not; what lies
    beside the columns stays."""
    _, x = heads(37, 9, 64, dtype, 5, *x_at)
    buf, out = heads(37, 9, 64, dtype, 6, *out_at)
    pos = positions(37, 7)
    freq = va.rope_inv_freq(64)
    before = buf.clone()
    got = va.rope(x, pos, freq, interleaved=interleaved, out=out)
    check(got, x, pos, freq, interleaved=interleaved)
    beside = torch.ones(buf.shape[-1], dtype=torch.bool)
    beside[out_at[1]:out_at[1] + 64] = False
    assert torch.equal(buf[..., beside].isnan(), before[..., beside].isnan())


def test_other_orders_of_tokens_and_heads(va):
    freq = va.rope_inv_freq(32)
    pos = positions(21, 8)
    base = heads(6, 21, 64, BF16, 9)[1]              # heads outside tokens
    x = base.transpose(0, 1)
    check(va.rope(x, pos, freq), x, pos, freq)
    out = torch.empty(6, 21, 64, dtype=BF16, device="cuda").transpose(0, 1)
    check(va.rope(x, pos, freq, out=out), x, pos, freq)
    one = heads(21, 1, 64, BF16, 10)[1].expand(21, 6, 64)   # one head seen as six
    check(va.rope(one, pos, freq), one, pos, freq)


def test_far_and_negative_positions(va):
    """Angles of positions to the ends of 32 bits.  The reference's own product p f is off
    by 2^-53 of up to 2^31 radians there: 2.4e-7 of |a| + |b|, added to the bound."""
    freq = va.rope_inv_freq(64)
    _, x = heads(8, 2, 64, F32, 11)
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1000003, -77777777, 2 ** 30],
                       dtype=torch.int32, device="cuda")
    got = _tokens.f64(va.rope(x, pos, freq))
    xs = _tokens.f64(x)
    want = oracle.rope(xs, pos.cpu().numpy(), freq)
    bound = _tokens.rope_bound(want, xs, F32, 32) + 2.0 ** -22 * _tokens.pair_sums(xs, 0, 32, False)
    assert np.all(np.abs(got - want) <= bound)
    assert torch.equal(va.rope(x, pos, freq)[0], x[0])          # position 0


def test_negative_frequencies_turn_the_other_way(va):
    """Small ones too, at far positions: they keep all their bits.  (Angles of a few radians,
    of which the reference's product loses 2^-53.)"""
    freq = [-1e-9, -3.3e-10, -1e-20, -7.7e-10, -2.9e-9, 1.1e-12, -5.5e-10, 0.0]
    _, x = heads(6, 2, 16, F32, 13)
    pos = torch.tensor([0, 1, 2 ** 31 - 1, -2 ** 31, 1000003, 2 ** 30 + 12345], dtype=torch.int32,
                       device="cuda")
    check(va.rope(x, pos, freq), x, pos, freq)
    other = _tokens.f64(va.rope(x, pos, [-f for f in freq], inverse=True))
    # the same angle but for its last place, 2^-34 of a turn, and 2^-24 of it
    bound = (2 * np.pi * 2.0 ** -34 + 8 * 2.0 ** -24) * _tokens.pair_sums(_tokens.f64(x), 0, 8, False)
    assert np.all(np.abs(_tokens.f64(va.rope(x, pos, freq)) - other) <= bound)


def test_frequencies_of_whole_turns(va):
    """Frequencies of 2 pi times a whole number and one over a power of two turn by exact
    fractions: eighths and quarters of a turn at every position."""
    freq = [2 * np.pi * t for t in (0.25, 0.125, -0.25, 1.0, 3.0, 0.0, 0.5, -0.125)]
    pos = torch.arange(-20, 20, dtype=torch.int32, device="cuda")
    _, x = heads(40, 3, 16, F32, 12)
    check(va.rope(x, pos, freq), x, pos, freq)


def test_gradient_is_the_inverse_rotation(va):
    """<g, rope(x + h) - rope(x)> = <inverse(g), h>: against the oracle's own differences."""
    freq = va.rope_inv_freq(32)
    _, x = heads(9, 4, 48, F32, 13)
    _, g = heads(9, 4, 48, F32, 14)
    pos = positions(9, 15)
    kw = dict(rot_offset=8, interleaved=True, amplitude=0.8)
    dx = _tokens.f64(va.rope(g, pos, freq, inverse=True, **kw))
    xs, gs, p = _tokens.f64(x), _tokens.f64(g), pos.cpu().numpy()
    rng = np.random.default_rng(16)
    for _ in range(20):
        h = rng.normal(size=xs.shape)
        diff = ((oracle.rope(xs + h, p, freq, **kw) - oracle.rope(xs - h, p, freq, **kw)) * gs).sum() / 2
        # every entry of dx is off by less than 10 * 2^-24 of its pair's |g| sum (copied: 0)
        slack = (10 * 2.0 ** -24 * _tokens.pair_sums(gs, 8, 16, True) * np.abs(h)).sum() + 1e-9
        assert abs(diff - (dx * h).sum()) <= slack


def test_many_items_take_the_wide_variant(va):
    """2^20 items and more, and fewer: a row's result is the same."""
    freq = va.rope_inv_freq(64)
    _, x = heads(2100, 64, 64, BF16, 17)
    pos = positions(2100, 18)
    for inter in (False, True):
        big = va.rope(x, pos, freq, interleaved=inter)
        small = va.rope(x[2000:], pos[2000:].contiguous(), freq, interleaved=inter)
        assert torch.equal(big[2000:], small)
        check(small, x[2000:], pos[2000:], freq, interleaved=inter)


def test_no_tokens(va):
    x = torch.empty(0, 4, 64, dtype=BF16, device="cuda")
    assert va.rope(x, torch.empty(0, dtype=torch.int32, device="cuda"), va.rope_inv_freq(64)).shape \
        == x.shape


def rows(tokens, dtype, seed, stride=576):
    g = torch.Generator().manual_seed(seed)
    buf = torch.full((tokens, stride), float("nan"), dtype=dtype)
    buf[:, :576] = (torch.randn(tokens, 576, generator=g) * 3).to(dtype)
    return buf.cuda()[:, :576]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,H,norm,stride", [(1, 0, True, 576), (1, 8, True, 576),
                                                  (9, 64, True, 640), (130, 5, False, 584),
                                                  (7, 1, False, 576)])
def test_append_matches_the_oracle(va, tokens, H, norm, stride, interleaved, dtype):
    pool = torch.full((300, stride), float("nan"), dtype=BF16, device="cuda")
    kv = rows(tokens, dtype, 20, 576 + 8 * (tokens % 3))
    g = torch.Generator().manual_seed(21)
    slots = torch.randperm(300, generator=g)[:tokens].to(torch.int32).cuda()
    pos = positions(tokens, 22)
    w = (1 + 0.3 * torch.randn(512, generator=g)).to(dtype).cuda() if norm else None
    freq = va.rope_inv_freq(64, scaling="yarn", factor=40.0, original_len=4096)
    amp = 1.3688
    q_pe = heads(tokens, H, 64, BF16, 23, 192, 128)[1] if H else None
    buf, q_out = heads(tokens, H, 64, BF16, 24, 576, 512) if H else (None, None)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got_pool, got_q = va.kv_append(pool, kv, slots, pos, freq, norm_weight=w, interleaved=interleaved,
                                   amplitude=amp, q_pe=q_pe, q_out=q_out, status=status)
    assert got_pool is pool and got_q is q_out and int(status) == 0
    kv64 = _tokens.f64(kv)
    want = oracle.latent_rows(kv64, pos.cpu().numpy(), freq, None if w is None else _tokens.f64(w),
                              1e-6, interleaved, amp)
    got = _tokens.f64(pool)[slots.cpu().numpy(), :576]
    bound = _tokens.row_bound(want, kv64, 32, norm=norm, interleaved=interleaved, amplitude=amp)
    assert np.all(np.abs(got - want) <= bound), float(np.max(np.abs(got - want) - bound))
    # other rows, and columns from 576 on, are left
    rest = torch.ones(300, dtype=torch.bool)
    rest[slots.long().cpu()] = False
    assert bool(pool[rest.cuda()].isnan().all()) and bool(pool[:, 576:].isnan().all())
    if H:
        check(q_out, q_pe, pos, freq, interleaved=interleaved, amplitude=amp)
        assert bool(buf[..., :512].isnan().all())


def test_append_skips_slots_outside_the_pool(va):
    pool = torch.zeros(16, 576, dtype=BF16, device="cuda")
    kv = rows(6, BF16, 30)
    slots = torch.tensor([3, -1, 16, 2 ** 31 - 1, -2 ** 31, 5], dtype=torch.int32, device="cuda")
    pos = positions(6, 31)
    q_pe = heads(6, 4, 64, BF16, 32)[1]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, q = va.kv_append(pool, kv, slots, pos, va.rope_inv_freq(64), q_pe=q_pe, status=status)
    assert int(status) == va.STATUS_BAD_SLOT
    live = pool.abs().sum(1) > 0
    assert live.nonzero().flatten().tolist() == [3, 5]
    check(q, q_pe, pos, va.rope_inv_freq(64))


def test_append_rotates_queries_in_place_and_askew(va):
    """q_out may be q_pe; queries that are not 16-byte aligned take a launch of their own."""
    pool = torch.zeros(16, 576, dtype=BF16, device="cuda")
    kv, pos = rows(5, BF16, 33), positions(5, 34)
    slots = torch.arange(5, dtype=torch.int32, device="cuda")
    freq = va.rope_inv_freq(64)
    for at in ((576, 512), (67, 3)):
        _, q = heads(5, 7, 64, BF16, 35, *at)
        x = q.clone()
        va.kv_append(pool, kv, slots, pos, freq, q_pe=q, q_out=q)
        check(q, x, pos, freq)


def test_append_large_batch(va):
    """More query items than the narrow variant takes, and hundreds of rows."""
    n, H = 2100, 64
    pool = torch.zeros(n + 50, 576, dtype=BF16, device="cuda")
    kv, pos = rows(n, BF16, 36), positions(n, 37)
    slots = torch.randperm(n + 50, generator=torch.Generator().manual_seed(38))[:n].to(torch.int32).cuda()
    freq = va.rope_inv_freq(64)
    w = torch.ones(512, dtype=BF16, device="cuda")
    q_pe = heads(n, H, 64, BF16, 39)[1]
    _, q = va.kv_append(pool, kv, slots, pos, freq, norm_weight=w, q_pe=q_pe)
    assert torch.equal(q, va.rope(q_pe, pos, freq))
    small = torch.zeros_like(pool)
    for a in range(0, n, 700):
        va.kv_append(small, kv[a:a + 700], slots[a:a + 700].contiguous(),
                     pos[a:a + 700].contiguous(), freq, norm_weight=w)
    assert torch.equal(pool, small)
    want = oracle.latent_rows(_tokens.f64(kv[:64]), pos[:64].cpu().numpy(), freq, np.ones(512))
    got = _tokens.f64(pool)[slots[:64].cpu().numpy()]
    assert np.all(np.abs(got - want) <= _tokens.row_bound(want, _tokens.f64(kv[:64]), 32, norm=True))


def test_zero_rows_and_rows_of_nan(va):
    """A row of zeros is normalised by eps alone; NaN stays in its own row."""
    pool = torch.zeros(4, 576, dtype=BF16, device="cuda")
    kv = rows(3, F32, 40)
    kv[0] = 0
    kv[1, 5] = float("nan")
    w = torch.ones(512, device="cuda")
    va.kv_append(pool, kv, torch.arange(3, dtype=torch.int32, device="cuda"), positions(3, 41),
                 va.rope_inv_freq(64), norm_weight=w)
    assert bool((pool[0] == 0).all()) and bool(pool[1, :512].isnan().all())
    assert bool(pool[2].isfinite().all()) and bool((pool[3] == 0).all())


def test_captured_calls_follow_their_buffers(va):
    """Positions, slots and rows are read when a graph is replayed; frequencies are not."""
    pool = torch.zeros(32, 576, dtype=BF16, device="cuda")
    kv, pos = rows(4, BF16, 42), positions(4, 43)
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    freq = va.rope_inv_freq(64)
    q_pe = heads(4, 8, 64, BF16, 44)[1]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    append = va.prepare_kv_append(pool, kv, slots, pos, freq, q_pe=q_pe, stream=st)
    turn = va.prepare_rope(q_pe, pos, freq, inverse=True, stream=st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        append()
        turn()
    for seed in (45, 46):
        kv.copy_(rows(4, BF16, seed))
        pos.copy_(positions(4, seed))
        slots.copy_(torch.randperm(32, generator=torch.Generator().manual_seed(seed))[:4])
        pool.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = torch.zeros_like(pool)
        _, q = va.kv_append(want, kv, slots, pos, freq, q_pe=q_pe)
        assert torch.equal(pool, want) and torch.equal(append.result[1], q)
        assert torch.equal(turn.result, va.rope(q_pe, pos, freq, inverse=True))


def test_refusals(va):
    x = torch.zeros(3, 4, 64, dtype=BF16, device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    f = va.rope_inv_freq(64)
    for bad in (lambda: va.rope(x.cpu(), pos, f), lambda: va.rope(x[0], pos, f),
                lambda: va.rope(x, pos[:2], f), lambda: va.rope(x, pos.cpu(), f),
                lambda: va.rope(x[..., ::2], pos, f[:16]),
                lambda: va.rope(x, pos, f, out=torch.zeros(3, 4, 65, dtype=BF16, device="cuda")),
                lambda: va.rope(x, pos, torch.zeros(32, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: va.rope(x.double(), pos, f), lambda: va.rope(x, pos.long(), f),
                lambda: va.rope(x, pos, f, out=x.float())):
        with pytest.raises(TypeError):
            bad()
    for kw in (dict(inv_freq=f + [1.0]), dict(inv_freq=f, rot_offset=1),
               dict(inv_freq=f, rot_offset=-1), dict(inv_freq=[float("nan")]), dict(inv_freq=[]),
               dict(inv_freq=f, amplitude=float("inf"))):
        with pytest.raises(va.VaError):
            va.rope(x, pos, **kw)
    # rows of the output that overlap
    with pytest.raises(va.VaError):
        va.rope(x, pos, f, out=torch.zeros(3, 1, 64, dtype=BF16, device="cuda").expand(3, 4, 64))
    pool = torch.zeros(8, 576, dtype=BF16, device="cuda")
    kv = torch.zeros(3, 576, dtype=BF16, device="cuda")
    slots = torch.zeros(3, dtype=torch.int32, device="cuda")
    w = torch.ones(512, dtype=BF16, device="cuda")
    for bad in (lambda: va.kv_append(pool, kv[:, :575], slots, pos, f),
                lambda: va.kv_append(pool, kv, slots[:1], pos, f),
                lambda: va.kv_append(pool, kv, slots, pos, f[:5]),
                lambda: va.kv_append(pool, kv, slots, pos, f, norm_weight=w[:100].contiguous()),
                lambda: va.kv_append(pool, kv, slots, pos, f, q_out=x),
                lambda: va.kv_append(pool, kv, slots, pos, f, q_pe=x[:2])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: va.kv_append(pool, kv, slots, pos, f, norm_weight=w.float()),
                lambda: va.kv_append(pool, kv, slots, pos, f, q_pe=x.float()),
                lambda: va.kv_append(pool.float(), kv, slots, pos, f)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(va.VaError):
        va.kv_append(pool, kv, slots, pos, f, eps=-1.0)
    odd = torch.zeros(3 * 580, dtype=BF16, device="cuda").view(3, 580)[:, :576]
    with pytest.raises(va.VaError):
        va.kv_append(pool, odd, slots, pos, f)
