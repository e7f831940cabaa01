"""Tokens drawn from rows of logits, and tree acceptance by sampling (va_sample,
va_tree_accept_sampled), against the oracle in 64 bits (needs an sm_103 GPU).

How far a mass may be off, in units of 2^-24 of itself: the exponent (l - m) / T loses three
roundings of itself, at most 20 for a token whose mass matters here (e^-20 of the largest's, a
hundred thousand times, is 2e-4 of a row), so 60, also where it is taken in two parts, to the
maximum of a part of the row and from there; the powers of two 4 each; the sum of a step's
weights 5, of a lane's steps (32 at most) 32, the whole numbers 2.  In all 107, less than 2^-17.2 of
every weight, hence of every sum of them: BOUND.  Where the oracle finds every comparison decided by
more than BOUND of the kept mass, the token has to be the oracle's; elsewhere it has to be
a token whose stretch lies as near.  ln of a share is then off by 2 BOUND, and rounds
to 2^-24 of itself and of the two logarithms it is made of (at most 40 together)."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
BOUND = 2.0 ** -17.2
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def va():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mla_speculative_decode_gb300 as m
    m.build()
    m.init()
    return m


def model_logits(n, V, seed, dtype=F32, sharp=1.0):
    """A broad tail and some likely tokens."""
    g = torch.Generator().manual_seed(seed)
    x = 2.0 * torch.randn(n, V, generator=g)
    k = min(V, 40)
    x.scatter_add_(1, torch.randint(0, V, (n, k), generator=g),
                   9.0 + 3.0 * torch.randn(n, k, generator=g))
    return (x * sharp).to(dtype)


def dev(x, dtype=F32):
    return None if x is None else torch.tensor(x, dtype=dtype, device="cuda")


def near(row, token, u, temperature, top_k, top_p, min_p):
    """Whether some uniform within 4 BOUND of u, and some top_p as near, gives the token."""
    for dp in (0.0, -2 * BOUND, 2 * BOUND):
        for du in np.linspace(-4 * BOUND, 4 * BOUND, 65):
            p = top_p + dp if top_p < 1 else top_p
            if oracle.draw(row, min(max(u + du, 0.0), 1 - 1e-12), temperature, top_k, p, min_p)[0] \
                    == token:
                return True
    return False


def check(va, logits, u, *, temperature=None, top_k=None, top_p=None, min_p=None, sure=0.75, **kw):
    """logits: a CPU tensor, or a CUDA view of one.  `sure`: share of rows that the oracle
    finds decided by more than BOUND, at least (it depends on the inputs alone)."""
    n = logits.shape[0]
    d = logits if logits.is_cuda else logits.cuda()
    tok, lp = va.sample(d, dev(u), temperature=dev(temperature), top_k=dev(top_k, torch.int32),
                        top_p=dev(top_p), min_p=dev(min_p), **kw)
    again, lp2 = va.sample(d, dev(u), temperature=dev(temperature), top_k=dev(top_k, torch.int32),
                           top_p=dev(top_p), min_p=dev(min_p))
    assert torch.equal(tok, again) and torch.equal(lp, lp2)
    tok, lp = tok.cpu().numpy(), lp.cpu().numpy().astype(np.float64)
    host = d.float().cpu().numpy()
    f32 = lambda x, i, other: other if x is None else float(np.float32(x[i]))  # noqa: E731
    decided = 0
    for i in range(n):
        s = (f32(temperature, i, 1.0), 0 if top_k is None else int(top_k[i]), f32(top_p, i, 1.0),
             f32(min_p, i, 0.0))
        s = s[:2] + (1.0 if s[2] != s[2] else s[2], 0.0 if s[3] != s[3] else s[3])
        ui = f32(u, i, None)
        want, want_lp, margin = oracle.draw(host[i], ui, *s)
        if margin > BOUND:
            decided += 1
            assert tok[i] == want, (i, int(tok[i]), want, margin, s, ui)
            if want_lp == -np.inf:
                assert lp[i] == -np.inf
            else:
                assert abs(lp[i] - want_lp) <= 2 * BOUND + 2.0 ** -24 * (abs(want_lp) + 40)
        else:
            assert near(host[i], tok[i], ui, *s), (i, int(tok[i]), want, margin)
    assert decided >= sure * n, (decided, n)
    return tok, lp


def settings(n, seed):
    r = np.random.default_rng(seed)
    return dict(temperature=r.choice([0.0, 0.5, 0.8, 1.0, 1.5], n).tolist(),
                top_k=r.choice([0, 1, 2, 20, 50, 700], n).tolist(),
                top_p=r.choice([1.0, 0.3, 0.8, 0.9, 0.99], n).tolist(),
                min_p=r.choice([0.0, 0.0, 0.01, 0.2], n).tolist())


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 31, 127, 1000, 4099, 32000, 129280])
def test_mixed_settings_match_the_oracle(va, V, dtype):
    n = 24 if V < 10000 else 10
    u = np.random.default_rng(V).random(n).tolist()
    check(va, model_logits(n, V, V, dtype), u, **settings(n, V + 1))


@pytest.mark.parametrize("which", ["none", "top_k", "top_p", "min_p", "temperature"])
@pytest.mark.parametrize("V", [257, 50021])
def test_one_setting_at_a_time(va, V, which):
    n = 12
    u = np.random.default_rng(5).random(n).tolist()
    s = settings(n, 6)
    check(va, model_logits(n, V, 7, F32), u, **({which: s[which]} if which != "none" else {}))


@pytest.mark.parametrize("rows,V", [(1, 129280), (3, 129281), (70, 9001), (160, 2000), (330, 700),
                                    (700, 90)])
def test_batches_of_all_sizes(va, rows, V):
    """Eight CTAs a row down to one."""
    u = np.random.default_rng(8).random(rows).tolist()
    check(va, model_logits(rows, V, 9), u, **settings(rows, 10))


@pytest.mark.parametrize("V,dtype", [(262144, F32), (400003, F32), (1 << 20, F32), (1 << 20, BF16)])
def test_long_rows(va, V, dtype):
    """Up to the largest: parts of a row that do not fit shared memory are read again."""
    u = [0.3, 0.7, 0.11]
    check(va, model_logits(3, V, 11, dtype), u, temperature=[1.0, 0.8, 1.2], top_k=[0, 50, 1000],
          top_p=[1.0, 0.95, 0.9], min_p=[0.0, 0.0, 0.01], sure=0.6)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_at_any_stride_and_alignment(va, dtype):
    n, V = 9, 1003
    u = np.random.default_rng(12).random(n).tolist()
    s = settings(n, 13)
    base = model_logits(n, V, 14, dtype)
    for width, col in ((1003, 0), (1005, 1), (1011, 3), (1024, 5), (1031, 8)):
        buf = torch.full((n, width + 8), INF, dtype=dtype, device="cuda")   # must not be read
        view = buf[:, col:col + V]
        view.copy_(base)
        check(va, view, u, **s)
    check(va, base[:1].cuda().expand(n, V), u, **s)        # one row for all


def stretches(va, row, n, **kw):
    """Tokens of one row for n uniforms spread evenly: each token comes as often as its
    share of the kept mass says, to one."""
    V = row.shape[0]
    u = (np.arange(n) + 0.5) / n
    tok, _ = va.sample(row.cuda()[None].expand(n, V), dev(u),
                       **{k: dev([v] * n, torch.int32 if k == "top_k" else F32) for k, v in kw.items()})
    tok = tok.cpu().numpy()
    assert (np.diff(tok) >= 0).all()          # index order
    return np.bincount(tok, minlength=V)


def shares(row, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    l = row.double().numpy()
    w = np.exp((l - l.max()) / temperature)
    order = np.argsort(-l, kind="stable")[:top_k or None]
    if top_p < 1:
        c = np.cumsum(w[order])
        order = order[:int(np.searchsorted(c, float(np.float32(top_p)) * c[-1])) + 1]
    keep = np.zeros(len(l), bool)
    keep[order] = True
    keep &= w >= min_p
    return np.where(keep, w, 0) / w[keep].sum()


@pytest.mark.parametrize("kw", [dict(), dict(temperature=0.7), dict(top_k=40), dict(top_p=0.9),
                                dict(top_k=300, top_p=0.8), dict(min_p=0.05),
                                dict(temperature=2.5, top_p=0.95)])
def test_tokens_come_as_often_as_they_should(va, kw):
    row = model_logits(1, 5003, 15)[0]
    n = 20000
    got, p = stretches(va, row, n, **kw), shares(row, **kw)
    assert np.all(np.abs(got - n * p) <= 1 + n * 2 * BOUND)


@pytest.mark.parametrize("V", [300, 5000, 100003])
def test_equal_logits(va, V):
    """Weights of exactly 1: borders and draws come out to the token.  The long rows have
    more equal values than a list holds."""
    row = torch.full((1, V), 3.25)
    u = [0.0, 0.25, 0.5, 1 - 2.0 ** -24]
    def tokens(**kw):
        return va.sample(row.cuda().expand(4, V), dev(u), **kw)[0].tolist()
    at = lambda n: [min(int(np.floor(x * n)), n - 1) for x in u]  # noqa: E731
    assert tokens() == at(V)
    assert tokens(top_k=dev([7] * 4, torch.int32)) == at(7)
    assert tokens(top_p=dev([0.5] * 4)) == at((V + 1) // 2)
    assert tokens(top_p=dev([0.0] * 4)) == [0] * 4
    assert tokens(min_p=dev([1.0] * 4)) == at(V)
    n = int(np.ceil(float(np.float32(0.3)) * 129))
    assert tokens(top_k=dev([129] * 4, torch.int32), top_p=dev([0.3] * 4)) == at(n)


@pytest.mark.parametrize("V", [5000, 60000])
@pytest.mark.parametrize("spread", [1e-3, 1e-6])
def test_thousands_of_values_close_together(va, V, spread):
    """All values within one step of the histogram (the border is found digit by digit)."""
    g = torch.Generator().manual_seed(16)
    row = 1.0 + spread * torch.rand(1, V, generator=g)
    order = torch.sort(row[0], descending=True, stable=True)[1]
    k, n = 1234, 4000
    got = stretches(va, row[0], n, top_k=k)
    p = shares(row[0], top_k=k)
    assert np.all(np.abs(got - n * p) <= 1 + n * 2 * BOUND)
    assert set(np.flatnonzero(got)) <= set(order[:k].tolist())
    p = shares(row[0], top_p=0.4)
    got = stretches(va, row[0], n, top_p=0.4)
    # (the border itself may lie a few values off: BOUND of V of them)
    assert np.abs(np.cumsum(got) / n - np.cumsum(p)).max() <= 1 / n + 4 * BOUND
    few = int(np.flatnonzero(p).size)
    assert set(np.flatnonzero(got)) <= set(order[:few + 2 + int(4 * BOUND * V)].tolist())
    got = stretches(va, row[0], n, top_k=k, top_p=0.5)
    assert set(np.flatnonzero(got)) <= set(order[:k // 2 + 2].tolist())


def test_many_equal_among_different(va):
    """Ties at the border of top-k and top-p: the lower indices stay."""
    g = torch.Generator().manual_seed(17)
    row = torch.randint(0, 12, (1, 20000), generator=g).float() * 0.25
    for kw in (dict(top_k=1700), dict(top_k=100), dict(top_p=0.13), dict(top_p=0.7),
               dict(top_k=5000, top_p=0.5)):
        n = 6000
        p = shares(row[0], **kw)
        got = stretches(va, row[0], n, **kw)
        assert np.abs(np.cumsum(got) / n - np.cumsum(p)).max() <= 1 / n + 4 * BOUND
        assert not got[p == 0].any() or "top_p" in kw


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V,sigma", [(50000, 0.3), (129280, 1.0), (129281, 2.0), (262144, 1.5)])
def test_borders_among_thousands_of_tokens(va, V, sigma, dtype):
    """Rows whose mass lies in thousands of tokens: tokens for evenly spread uniforms follow the
    shares, to BOUND of the mass (a border may lie off by that much, too: 2 BOUND and one
    token at either end), and only kept tokens come."""
    g = torch.Generator().manual_seed(V)
    row = (sigma * torch.randn(V, generator=g)).to(dtype)
    n = 400
    for kw in (dict(top_p=0.5), dict(top_p=0.9), dict(top_p=0.99), dict(top_p=0.9, min_p=0.01),
               dict(temperature=1.7, top_p=0.95), dict(top_k=3000), dict(top_k=3000, top_p=0.8),
               dict(top_k=V // 3), dict(top_k=V // 3, top_p=0.6, min_p=0.002)):
        p = shares(row, **kw)
        got = stretches(va, row, n, **kw)
        token = p[p > 0].max()
        assert np.abs(np.cumsum(got) / n - np.cumsum(p)).max() <= 1 / n + 4 * BOUND + token, kw
        stray = np.flatnonzero((p == 0) & (got > 0))
        if "top_p" not in kw:
            assert stray.size == 0, kw
        elif stray.size:     # beyond the border by no more than BOUND of the mass
            l = row.double().numpy() / kw.get("temperature", 1.0)
            w = np.exp(l - l.max())
            between = (l >= l[stray].min()) & (p == 0)
            assert w[between].sum() <= 4 * BOUND * w.sum() + w[between].max(), kw


def check_stretches(va, row, s, seed):
    """Each row's token is kept and its stretch holds the uniform, both to BOUND; s: settings of
    every row."""
    n, V = row.shape
    u = np.random.default_rng(seed).random(n).astype(np.float32)
    tok, _ = va.sample(row.cuda(), dev(u.tolist()), temperature=dev(s["temperature"]),
                       top_k=dev(s["top_k"], torch.int32), top_p=dev(s["top_p"]),
                       min_p=dev(s["min_p"]))
    for i, t in enumerate(tok.tolist()):
        T, k, p, m = (float(np.float32(s[x][i])) for x in ("temperature", "top_k", "top_p", "min_p"))
        l = row[i].double().numpy() / T
        w = np.exp(l - l.max())
        order = np.argsort(-l, kind="stable")[:int(k) or V]
        before = np.concatenate([[0.0], np.cumsum(w[order])])
        mass, before = before[-1], before[:-1]
        keep = np.zeros(V, bool)
        keep[order[before < p * mass] if p < 1 else order] = True
        keep &= w >= m * (1 - BOUND)
        rank = int(np.flatnonzero(order == t)[0])       # (among the k largest, exactly)
        assert before[rank] < (p + 2 * BOUND) * mass and w[t] >= m * (1 - BOUND)
        # the token's stretch holds u, but for BOUND of both sides' masses, and of the border's
        # (kept or dropped on either side of the drawn one, and in the whole)
        c = np.cumsum(np.where(keep, w, 0.0))
        tol = 8 * BOUND * mass / c[-1] + w[t] / c[-1]
        assert c[t] / c[-1] - w[t] / c[-1] - tol <= u[i] <= c[t] / c[-1] + tol, (i, t)


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("V,sigma", [(9001, 0.1), (70001, 0.5), (70001, 0.02), (300000, 0.1)])
def test_flat_rows_with_any_filters(va, V, sigma, dtype):
    """No token is likely: borders of top-k and top-p lie among values that are close together."""
    g = torch.Generator().manual_seed(V + int(100 * sigma))
    n = 10
    row = (sigma * torch.randn(n, V, generator=g)).to(dtype)
    s = dict(temperature=[0.6, 1.0, 1.3, 1.0, 0.8, 1.0, 30.0, 1.0, 0.7, 1.0],
             top_k=[0, 20, 0, 200, 1000, 3000, 50, 0, 4000, 0],
             top_p=[0.5, 1.0, 0.9, 0.95, 0.8, 1.0, 0.9, 0.999, 0.9, 0.9999],
             min_p=[0.0, 0.0, 0.02, 0.1, 0.0, 0.0, 0.0, 0.0, 0.5, 0.0])
    check_stretches(va, row, s, V)


@pytest.mark.parametrize("V,step", [(50000, 0.125), (262144, 0.125), (262144, 2.0), (1 << 20, 0.5)])
def test_thousands_of_ties_at_the_border(va, V, step):
    """Large logits of a 16-bit type: few different values, each thousands of times, and a
    top-k of thousands."""
    g = torch.Generator().manual_seed(V)
    n = 9
    row = ((torch.randn(n, V, generator=g) * 2 + 20) / step).round().mul(step).to(BF16)
    row[8] = 20.0
    s = dict(temperature=[1.0, 1.0, 2.0, 1.0, 1.0, 0.7, 1.0, 1.0, 1.0],
             top_k=[0, 0, 0, 10000, 5000, 0, 20000, V // 2, 0],
             top_p=[0.9, 0.99, 0.5, 1.0, 0.8, 0.95, 0.9999, 0.999, 0.9],
             min_p=[0.0, 0.0, 0.0, 0.0, 0.0, 0.05, 0.3, 0.0, 0.0])
    check_stretches(va, row, s, V)


@pytest.mark.parametrize("V", [3000, 6000, 20000])
@pytest.mark.parametrize("levels", [2, 5])
def test_few_different_logits(va, V, levels):
    """Hundreds to thousands of ties at every border."""
    n = 40
    g = torch.Generator().manual_seed(V + levels)
    row = torch.randint(0, levels, (n, V), generator=g).float() * 0.5
    s = settings(n, 50)
    s["temperature"] = [t or 1.0 for t in s["temperature"]]
    check(va, row, np.random.default_rng(51).random(n).tolist(), sure=0.5, **s)


def test_likely_tokens_at_one_end_of_the_row(va):
    """Token ids sorted by frequency: all that is listed lies in the first part of the row."""
    V, n = 60000, 24
    row = model_logits(n, V, 52).sort(-1, descending=True)[0]
    s = settings(n, 53)
    check(va, row, np.random.default_rng(54).random(n).tolist(), **s)
    check(va, row.flip(-1).contiguous(), np.random.default_rng(55).random(n).tolist(), **s)


def test_masked_rows(va):
    V = 3000
    row = torch.full((8, V), -INF)
    row[0, 17] = -3.0                                     # one token
    row[1, [5, 900, 2999]] = torch.tensor([1.0, 2.0, 0.5])
    row[3] = torch.finfo(F32).min                         # the type's lowest value throughout
    row[4] = torch.finfo(F32).min
    row[4, 40] = 0.0
    row[5, [7, 8]] = INF                                  # they share the mass
    row[5, 9] = 100.0
    row[6] = NAN
    row[7] = NAN
    row[7, [1, 2]] = torch.tensor([-1.0, -1.0])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    u = [0.6] * 8
    for kw in (dict(), dict(top_k=dev([50] * 8, torch.int32)), dict(top_p=dev([0.9] * 8)),
               dict(min_p=dev([0.1] * 8)),
               dict(top_k=dev([50] * 8, torch.int32), top_p=dev([0.999] * 8))):
        status.zero_()
        tok, lp = va.sample(row.cuda(), dev(u), status=status, **kw)
        t, lp = tok.tolist(), lp.tolist()
        assert int(status) == va.STATUS_EMPTY_ROW
        w = np.exp(np.array([1.0, 2.0, 0.5]) - 2.0)
        share = np.cumsum(w) / w.sum()
        assert t[0] == 17 and lp[0] == 0
        assert t[1] == (5, 900, 2999)[int(np.searchsorted(share, 0.6))]
        assert (t[2], t[6]) == (0, 0) and lp[2] == lp[6] == -INF
        n = 50 if "top_k" in kw else V
        n = int(np.ceil(0.9 * n - 1e-6)) if "top_p" in kw and "top_k" not in kw else n
        assert t[3] == int(0.6 * n) and abs(lp[3] + np.log(n)) < 1e-5
        assert t[4] == 40 and lp[4] == 0
        assert t[5] == 8 and abs(lp[5] + np.log(2)) < 1e-6
        assert t[7] == 2
    status.zero_()
    tok, lp = va.sample(row.cuda(), dev(u), temperature=dev([0.0] * 8), status=status)
    assert tok.tolist() == [17, 900, 0, 0, 40, 7, 0, 1] and int(status) == va.STATUS_EMPTY_ROW
    assert lp.tolist() == [0, 0, -INF, 0, 0, 0, -INF, 0]
    va.sample(row[:2].cuda(), dev(u[:2]))                 # without a status word


def test_ends_of_the_settings(va):
    V = 2000
    x = model_logits(1, V, 18)
    x[0, 77] = x[0, 1500] = float(x.max()) + 1.0         # two largest
    row = x.cuda()
    one = lambda u=0.7, **kw: va.sample(  # noqa: E731
        row, dev([u]), **{k: dev([v], torch.int32 if k == "top_k" else F32)
                          for k, v in kw.items()})[0].item()
    for t in (0.0, -1.0, -0.0, NAN):
        assert one(temperature=t) == 77
    for t in (1e-30, 1e-45, 1e-10):                       # only the largest have a mass
        assert one(0.2, temperature=t) == 77 and one(0.7, temperature=t) == 1500
    for t in (1e30, INF):                                 # every token the same
        assert one(0.7, temperature=t) == int(np.float32(0.7) * np.float64(V))
    assert one(top_k=1) == 77 and one(top_k=2) == 1500
    for kw in (dict(top_k=0), dict(top_k=-5), dict(top_k=V), dict(top_k=2 ** 31 - 1),
               dict(top_p=1.0), dict(top_p=7.0), dict(top_p=NAN), dict(top_p=INF),
               dict(min_p=0.0), dict(min_p=-1.0), dict(min_p=NAN)):
        assert one(0.31, **kw) == one(0.31), kw
    for p in (0.0, -1.0, 1e-30, 1e-45, -INF):
        assert one(top_p=p) == 77
    for p in (1.0, 2.0, INF):
        assert one(0.2, min_p=p) == 77 and one(0.7, min_p=p) == 1500
    first = int((x[0] > -30).nonzero()[0])
    for u in (0.0, -1.0, NAN, -INF):
        assert one(u) == first
    for u in (1.0, 5.0, INF, 1 - 2.0 ** -24):
        assert one(u, top_k=2) == 1500


def test_top_p_close_to_one(va):
    row = model_logits(1, 30000, 19)[0]
    for p in (1 - 2.0 ** -24, 1 - 2.0 ** -20, 0.999999):
        n = 3000
        got = stretches(va, row, n, top_p=p)
        assert np.abs(np.cumsum(got) / n - np.cumsum(shares(row))).max() <= 1 / n + 2e-6 + 4 * BOUND


def test_rows_are_left_alone_and_outputs_given(va):
    """Given outputs are written, each row by itself; no rows: nothing."""
    x = model_logits(4, 500, 20).cuda()
    u = dev([0.1, 0.5, 0.9, 0.3])
    tok = torch.full((4,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((4,), 7.0, device="cuda")
    got = va.sample(x, u, tokens=tok, logprob=lp)
    assert got[0] is tok and got[1] is lp
    want = [va.sample(x[i:i + 1], u[i:i + 1]) for i in range(4)]
    assert tok.tolist() == [w[0].item() for w in want] and lp.tolist() == [w[1].item() for w in want]
    e = torch.empty(0, 500, device="cuda")
    assert va.sample(e, torch.empty(0, device="cuda"))[0].numel() == 0


def tree(B, T, V, seed, dtype=F32):
    r = np.random.default_rng(seed)
    lg = model_logits(B * (T + 1), V, seed, dtype).view(B, T + 1, V)
    par = np.array([[r.integers(-1, i) if i else -1 for i in range(T)] for _ in range(B)], np.int32)
    best = torch.topk(lg.float(), min(3, V), -1)[1].numpy()
    tok = np.array([[best[b, par[b, i] + 1, r.integers(0, min(3, V))] for i in range(T)]
                    for b in range(B)], np.int32)
    slots = r.permutation(4 * B * T)[:B * T].reshape(B, T).astype(np.int32)
    return lg, par, tok, slots, r.random((B, T + 1)).astype(np.float32)


@pytest.mark.parametrize("B,T,V,dtype", [(1, 1, 37, F32), (3, 16, 5003, F32), (8, 16, 32000, BF16),
                                         (2, 64, 9000, F16), (1, 16, 129280, F32), (20, 5, 300, F32),
                                         (24, 16, 900, F32)])
def test_tree_acceptance(va, B, T, V, dtype):
    lg, par, tok, slots, u = tree(B, T, V, 21 + B, dtype)
    s = settings(B, 22)
    d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    call = va.prepare_tree_accept_sampled(
        lg[:, 0].contiguous().cuda(), lg[:, 1:].contiguous().cuda(), d(tok), d(par), d(u),
        temperature=dev(s["temperature"]), top_k=dev(s["top_k"], torch.int32),
        top_p=dev(s["top_p"]), min_p=dev(s["min_p"]), draft_slots=d(slots))
    got = [x.cpu().numpy() for x in call()]
    assert va.read_status(call.workspace) == 0
    # every position's draw is the one that sample makes of its row
    drawn, lp = va.sample(lg.view(-1, V).cuda(), d(u.reshape(-1)),
                          **{k: dev(np.repeat(v, T + 1).tolist(), torch.int32 if k == "top_k" else F32)
                             for k, v in s.items()})
    drawn = drawn.view(B, T + 1).cpu().numpy()
    np.testing.assert_array_equal(got[4].reshape(-1), lp.cpu().numpy())
    # ... and the walk is the greedy one along them
    onehot = lambda t: np.eye(V, dtype=np.float32)[t]  # noqa: E731
    for b in range(B):
        w = oracle.tree_accept(onehot(drawn[b:b + 1, 0]), onehot(drawn[b:b + 1, 1:]), tok[b:b + 1],
                               par[b:b + 1], slots[b:b + 1])
        for k in range(4):
            np.testing.assert_array_equal(got[k][b], w[k][0])
    # draws against the oracle, along the path
    for b in range(min(B, 3)):
        for at in [0] + [int(x) + 1 for x in got[1][b] if x >= 0][:3]:
            one = [float(np.float32(s[k][b])) for k in ("temperature", "top_k", "top_p", "min_p")]
            want, _, margin = oracle.draw(lg[b, at].float().numpy(), float(u[b, at]), one[0],
                                          int(one[1]), one[2], one[3])
            assert margin <= BOUND or drawn[b, at] == want


def test_greedy_settings_give_the_greedy_walk(va):
    lg, par, tok, slots, u = tree(6, 16, 2000, 30)
    d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    a = (lg[:, 0].contiguous().cuda(), lg[:, 1:].contiguous().cuda(), d(tok), d(par))
    got = va.tree_accept_sampled(*a, d(u), temperature=torch.zeros(6, device="cuda"),
                                 draft_slots=d(slots))
    want = va.tree_accept(*a, d(slots))
    for x, y in zip(got[:4], want[:4]):
        assert torch.equal(x, y)
    assert bool((got[4] == 0).all())


def test_tree_status_and_optional_outputs(va):
    lg, par, tok, slots, u = tree(2, 4, 100, 31)
    d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    par[1, 2] = 3                                   # not an earlier node
    lg[0, 3] = -INF                                 # a position without a token
    a = (lg[:, 0].contiguous().cuda(), lg[:, 1:].contiguous().cuda(), d(tok), d(par), d(u))
    outs = (torch.empty(2, dtype=torch.int32, device="cuda"),
            torch.empty(2, 4, dtype=torch.int32, device="cuda"), None,
            torch.empty(2, dtype=torch.int32, device="cuda"), None)
    call = va.prepare_tree_accept_sampled(*a, outputs=outs)
    call()
    assert va.read_status(call.workspace) == va.STATUS_BAD_PARENT | va.STATUS_EMPTY_ROW
    full = va.tree_accept_sampled(*a)
    assert torch.equal(full[0], outs[0]) and torch.equal(full[1], outs[1]) \
        and torch.equal(full[3], outs[3]) and bool((full[2] == -1).all())
    good = va.prepare_tree_accept_sampled(*a[:3], d(np.full((2, 4), -1, np.int32)), a[4],
                                          workspace=call.workspace)
    lg[0, 3] = 0.0
    a[1].copy_(lg[:, 1:])
    good()
    assert va.read_status(call.workspace) == 0      # rewritten by every call


def test_tree_emits_the_target_distribution(va):
    """The first emitted token of a tree, over evenly spread uniforms at the prefix, comes as
    often as sampling the target alone would give it, whatever was drafted."""
    B, T, V = 4000, 2, 30
    row = model_logits(1, V, 32)[0]
    lg = model_logits(1, V, 33)[0].expand(B, T, V).contiguous()
    tok = torch.tensor([[int(row.argmax()), 3]] * B, dtype=torch.int32)
    par = torch.tensor([[-1, -1]] * B, dtype=torch.int32)
    u = torch.rand(B, T + 1, generator=torch.Generator().manual_seed(34))
    u[:, 0] = (torch.arange(B) + 0.5) / B
    n, nodes, _, bonus, _ = va.tree_accept_sampled(row.expand(B, V).contiguous().cuda(), lg.cuda(),
                                                   tok.cuda(), par.cuda(), u.cuda())
    first = torch.where(n.cpu() > 0, tok.gather(1, nodes[:, :1].cpu().clamp(min=0).long())[:, 0],
                        bonus.cpu())
    got = np.bincount(first.numpy(), minlength=V)
    assert np.all(np.abs(got - B * shares(row)) <= 1 + 2 * B * BOUND)


def test_captured_calls_follow_their_buffers(va):
    """Logits, settings and uniforms are read when a graph is replayed."""
    n, V, B, T = 5, 3001, 2, 6
    x, u = model_logits(n, V, 35).cuda(), dev([0.5] * n)
    s = settings(n, 36)
    s = {k: dev(v, torch.int32 if k == "top_k" else F32) for k, v in s.items()}
    lg, par, tok, slots, tu = tree(B, T, V, 37)
    d = lambda y: torch.from_numpy(np.ascontiguousarray(y)).cuda()  # noqa: E731
    ta = [lg[:, 0].contiguous().cuda(), lg[:, 1:].contiguous().cuda(), d(tok), d(par), d(tu)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    one = va.prepare_sample(x, u, stream=st, **s)
    two = va.prepare_tree_accept_sampled(*ta, stream=st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        one()
        two()
    for seed in (38, 39, 40):
        x.copy_(model_logits(n, V, seed))
        u.copy_(torch.rand(n, generator=torch.Generator().manual_seed(seed)))
        for k, v in settings(n, seed).items():
            s[k].copy_(torch.tensor(v))
        lg, par, tok, slots, tu = tree(B, T, V, seed)
        for t, v in zip(ta, (lg[:, 0], lg[:, 1:], torch.from_numpy(tok), torch.from_numpy(par),
                             torch.from_numpy(tu))):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(one.result, va.sample(x, u, **s)):
            assert torch.equal(got, want)
        for got, want in zip(two.result, va.tree_accept_sampled(*ta)):
            assert torch.equal(got, want)


def test_memory_of_a_given_stream(va):
    """Memory taken for a call on a busy stream is not given to the current one."""
    x, u = model_logits(64, 5000, 41).cuda(), torch.rand(64, device="cuda")
    lg, par, tok, slots, tu = tree(2, 6, 3001, 42)
    d = lambda y: torch.from_numpy(np.ascontiguousarray(y)).cuda()  # noqa: E731
    ta = [lg[:, 0].contiguous().cuda(), lg[:, 1:].contiguous().cuda(), d(tok), d(par), d(tu)]
    side = torch.cuda.Stream()
    for make in (lambda: va.prepare_sample(x, u, stream=side),
                 lambda: va.prepare_tree_accept_sampled(*ta, stream=side)):
        make()()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(400_000_000)       # 0.2 s
        call = make()
        call()
        places = [(t.data_ptr(), t.numel() * t.element_size())
                  for t in (call.workspace, *call.result) if t is not None]
        del call
        new = [torch.empty(n, dtype=torch.uint8, device="cuda") for _, n in places]
        assert not any(a.data_ptr() < p + m and p < a.data_ptr() + a.numel()
                       for p, m in places for a in new)
        assert not side.query()
        side.synchronize()


def test_calls_on_two_streams_at_once(va):
    """Long and short rows, one CTA each and clusters, prepared and captured: what each gives by
    itself."""
    V = 60000
    calls, alone = [], []
    for i, n in enumerate((3, 40, 200, 7)):
        x = model_logits(n, V, 60 + i, (F32, BF16)[i % 2]).cuda()
        s = settings(n, 61 + i)
        u = dev(np.random.default_rng(62 + i).random(n).tolist())
        calls.append(dict(logits=x, uniform=u, temperature=dev(s["temperature"]),
                          top_k=dev(s["top_k"], torch.int32), top_p=dev(s["top_p"]),
                          min_p=dev(s["min_p"])))
        alone.append([t.clone() for t in va.sample(**calls[-1])])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    graphs = []
    for c, s in zip(calls, streams):
        call = va.prepare_sample(**c)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
        graphs.append((g, call))
    for _ in range(5):
        for i, (c, s) in enumerate(zip(calls, streams)):
            with torch.cuda.stream(s):
                got[i].append(va.sample(**c))
                graphs[i][0].replay()
    torch.cuda.synchronize()
    for i, want in enumerate(alone):
        for tok, lp in got[i] + [graphs[i][1].result]:
            assert torch.equal(tok, want[0]) and torch.equal(lp, want[1])


def test_refusals(va):
    x, u = torch.zeros(3, 10, device="cuda"), torch.zeros(3, device="cuda")
    k = torch.zeros(3, dtype=torch.int32, device="cuda")
    for bad in (lambda: va.sample(x.cpu(), u), lambda: va.sample(x[0], u),
                lambda: va.sample(x, u[:2]), lambda: va.sample(x, u.cpu()),
                lambda: va.sample(x[:, ::2], u), lambda: va.sample(x, u, top_k=k[:1]),
                lambda: va.sample(x, u, tokens=k[:2]), lambda: va.sample(x, u, top_p=u.cpu())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: va.sample(x.double(), u), lambda: va.sample(x, u.double()),
                lambda: va.sample(x, u, top_k=u), lambda: va.sample(x, u, temperature=k),
                lambda: va.sample(x, u, logprob=k)):
        with pytest.raises(TypeError):
            bad()
    for bad in (torch.zeros(3, 0, device="cuda"),
                torch.zeros(3, (1 << 20) + 1, dtype=BF16, device="cuda")):
        with pytest.raises(va.VaError):
            va.sample(bad, u)
    lg, par, tok, slots, tu = tree(2, 4, 100, 43)
    d = lambda y: torch.from_numpy(np.ascontiguousarray(y)).cuda()  # noqa: E731
    a = dict(root_logits=lg[:, 0].contiguous().cuda(), logits=lg[:, 1:].contiguous().cuda(),
             draft_tokens=d(tok), tree_parent=d(par), uniform=d(tu))
    for over in (dict(root_logits=a["root_logits"][:1]), dict(logits=a["logits"][0]),
                 dict(logits=lg.cuda()[:, 1:]), dict(draft_tokens=a["draft_tokens"][:1]),
                 dict(uniform=a["uniform"][:, :4].contiguous()), dict(top_p=u),
                 dict(draft_slots=a["draft_tokens"][:1])):
        with pytest.raises(ValueError):
            va.tree_accept_sampled(**(a | over))
    for over in (dict(root_logits=a["root_logits"].to(BF16)), dict(uniform=a["tree_parent"]),
                 dict(draft_tokens=a["draft_tokens"].long())):
        with pytest.raises(TypeError):
            va.tree_accept_sampled(**(a | over))
    with pytest.raises(va.VaError):
        va.tree_accept_sampled(**a, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
