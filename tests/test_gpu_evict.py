"""Eviction by accumulated weight (va_kv_evict) against the oracle, exactly, and
the whole loop a server runs: chunk attention, weights, eviction, and verify over
the lists that are left (needs an sm_103 GPU)."""
import numpy as np
import pytest
import torch

import oracle
import synth
from tests import _chunk, _gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def va():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mla_speculative_decode_gb300 as m
    m.build()
    m.init()
    return m


def _weights(kind, n, rng):
    if kind == "floats":
        return rng.exponential(size=n).astype(np.float32)
    if kind == "ties":
        return rng.integers(0, 3, size=n).astype(np.float32)
    if kind == "equal":
        return np.full(n, 0.25, dtype=np.float32)
    if kind == "close":       # neighbours that differ in the last bit only
        return (np.float32(1.0).view(np.int32) + rng.integers(0, 5, size=n)).astype(
            np.int32).view(np.float32)
    w = rng.normal(size=n).astype(np.float32)
    special = np.array([np.nan, np.inf, -np.inf, -0.0, 0.0, 1e-42, -1e-42], dtype=np.float32)
    at = rng.random(n) < 0.6
    w[at] = rng.choice(special, size=int(at.sum()))
    return w


def _run(va, L, gap, w_kind, budget, sinks, recent, *, seed, free=True, inplace=False):
    rng = np.random.default_rng(seed)
    B = len(L)
    indptr = np.concatenate([[0], np.cumsum([x + gap for x in L])]).astype(np.int32)
    n = int(indptr[-1])
    slots = rng.permutation(4 * n + 5)[:n].astype(np.int32)
    w = _weights(w_kind, n, rng)
    freed_total = sum(max(0, x - budget) for x in L)
    cap = freed_total + 9
    head = freed_total + 4
    fl = -np.arange(1, cap + 1, dtype=np.int32)
    t = [torch.from_numpy(x).cuda() for x in
         (slots, indptr, np.array(L, dtype=np.int32), w, fl, np.array([head], dtype=np.int32))]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = (t[0], t[2], t[3], t[5]) if inplace else \
        (torch.full_like(t[0], -9), torch.full_like(t[2], -9), torch.full_like(t[3], -9.0),
         torch.full_like(t[5], -9))
    kw = dict(free_slots=t[4], free_head=t[5]) if free else {}
    got = va.kv_evict(t[0], t[1], t[2], t[3], budget=budget, sinks=sinks, recent=recent,
                      outputs=outs, status=status, **kw)
    torch.cuda.synchronize()
    want_s = slots.copy() if inplace else np.full(n, -9, np.int32)
    want_w = w.copy() if inplace else np.full(n, -9.0, np.float32)
    freed = []
    for b in range(B):
        e = int(indptr[b])
        kept, gone = oracle.evict(slots[e:e + L[b]], w[e:e + L[b]], budget, sinks, recent)
        want_s[e:e + len(kept)] = slots[e + kept]
        want_w[e:e + len(kept)] = w[e + kept]
        freed += slots[e + gone].tolist()
    np.testing.assert_array_equal(got[0].cpu().numpy(), want_s)
    np.testing.assert_array_equal(got[2].cpu().numpy().view(np.int32), want_w.view(np.int32))
    np.testing.assert_array_equal(got[1].cpu().numpy(), [min(x, budget) for x in L])
    assert int(status.item()) == 0
    if free:
        h = head - len(freed)
        assert int(got[3].item()) == h
        want_f = fl.copy()
        want_f[h:head] = freed
        np.testing.assert_array_equal(t[4].cpu().numpy(), want_f)
    else:
        assert got[3] is None


KINDS = ["floats", "ties", "equal", "close", "special"]
CUTS = [
    # L, budget, sinks, recent
    ([100], 50, 0, 0),
    ([1, 0, 5, 2000], 4, 1, 2),
    ([3000, 1025, 1024, 1023, 7], 1000, 4, 128),
    ([2500], 2499, 3, 7),
    ([500, 501], 0, 0, 0),
    ([777, 50], 60, 60, 0),
    ([777, 50], 60, 0, 60),
    ([5000], 100, 10, 90),
    ([40], 40, 1, 1),
    ([9000, 20000], 6000, 4, 512),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("cut", range(len(CUTS)))
def test_evict_matches_the_oracle(va, cut, kind):
    L, budget, sinks, recent = CUTS[cut]
    for inplace in (False, True):
        _run(va, L, cut % 3, kind, budget, sinks, recent, seed=cut * 10 + KINDS.index(kind),
             inplace=inplace)
    _run(va, L, 1, kind, budget, sinks, recent, seed=cut, free=False)


@pytest.mark.parametrize("L", [70000, 200000, 600000])
def test_long_lists(va, L):
    _run(va, [L, L // 3], 5, "floats", 16384, 4, 1024, seed=L, inplace=True)
    _run(va, [L], 0, "ties", L // 2, 4, 1024, seed=L, inplace=True)


def test_many_requests(va):
    rng = np.random.default_rng(3)
    L = rng.integers(0, 400, size=300).tolist()
    _run(va, L, 2, "floats", 100, 4, 16, seed=4)


def test_free_list_without_room_and_bad_bounds_are_flagged(va):
    slots = torch.arange(20, dtype=torch.int32, device="cuda")
    w = torch.arange(20, dtype=torch.float32, device="cuda")
    ind = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    fl = torch.full((30,), -1, dtype=torch.int32, device="cuda")
    head = torch.tensor([3], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = (torch.zeros_like(slots), torch.zeros(1, dtype=torch.int32, device="cuda"),
           torch.zeros_like(w), torch.zeros_like(head))
    n = torch.tensor([20], dtype=torch.int32, device="cuda")
    va.kv_evict(slots, ind, n, w, budget=15, free_slots=fl, free_head=head, outputs=out,
                status=status)
    assert int(status.item()) == va.STATUS_BAD_DST
    assert int(out[3].item()) == 0 and fl[:3].tolist() == [2, 3, 4] and int(fl[3]) == -1
    # a length past the list, and a list past the arrays
    for ind_v, n_v, left in (([0, 20], 50, 15), ([0, 100], 20, 15), ([-3, 20], 20, 15),
                             ([0, 20], -1, 0), ([30, 40], 5, 0)):
        status.zero_()
        out[1].fill_(-1)
        va.kv_evict(slots, torch.tensor(ind_v, dtype=torch.int32, device="cuda"),
                    torch.tensor([n_v], dtype=torch.int32, device="cuda"), w, budget=15,
                    outputs=out, status=status)
        assert int(status.item()) == va.STATUS_BAD_INDPTR and int(out[1].item()) == left


def test_refusals(va):
    slots = torch.arange(20, dtype=torch.int32, device="cuda")
    w = torch.arange(20, dtype=torch.float32, device="cuda")
    ind = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    n = torch.tensor([20], dtype=torch.int32, device="cuda")
    for kw in (dict(budget=-1), dict(budget=4, sinks=3, recent=2), dict(budget=4, sinks=-1),
               dict(budget=4, recent=-1)):
        with pytest.raises(va.VaError):
            va.kv_evict(slots, ind, n, w, **kw)
    for bad, e in (((slots.long(), ind, n, w), TypeError), ((slots, ind[:1], n, w), ValueError),
                   ((slots, ind, n, w[:4]), ValueError), ((slots.cpu(), ind, n, w), ValueError)):
        with pytest.raises(e):
            va.kv_evict(*bad, budget=4)
    with pytest.raises(ValueError):
        va.kv_evict(slots, ind, n, w, budget=4, free_slots=slots.clone())


def test_chunk_weights_evict_verify_in_one_graph(va):
    """Prompt chunk, weights of its last tokens, eviction onto the free list, a
    draft tree whose slots come from that list, and tree verify over the lists
    that are left: captured once, replayed, checked against the oracle."""
    B, H, T, budget, sinks, recent = 2, 16, 4, 96, 4, 16
    P, n = [130, 40], [60, 75]
    c = _chunk.make(P, n, H, seed=31, list_gap=T, unused_nan=False)
    d = {k: c.dev(k) for k in ("q", "pool", "slot_idx", "kv_indptr", "prefix_len", "q_indptr")}
    L = torch.tensor([p + m for p, m in zip(P, n)], dtype=torch.int32, device="cuda")
    gone = sum(p + m - budget for p, m in zip(P, n))
    free = torch.full((gone + 8,), -1, dtype=torch.int32, device="cuda")
    head = torch.tensor([gone + 8], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(32)
    q2 = synth._bf16_normal((B * T, H, 576), g)
    draft = synth._bf16_normal((B * T, 576), g)
    tok = torch.randint(0, 1000, (B, 3, 4), generator=g, dtype=torch.int32)
    lp = torch.log_softmax(torch.randn(B, 3, 4, generator=g), dim=-1)
    dq2, ddraft, dtok, dlp = q2.cuda(), draft.cuda(), tok.cuda(), lp.cuda()
    w = torch.zeros(c.slot_idx.numel(), device="cuda")
    s_out, w_out = d["slot_idx"].clone(), torch.zeros_like(w)
    len_out, h_out = torch.zeros_like(L), torch.zeros_like(head)
    attn = va.prepare_chunk_paged(d["q"], d["pool"], d["slot_idx"], d["kv_indptr"],
                                  d["prefix_len"], d["q_indptr"], sm_scale=synth.SM_SCALE)
    weigh = va.prepare_kv_weights(d["q"], d["pool"], d["slot_idx"], d["kv_indptr"],
                                  d["prefix_len"], d["q_indptr"], attn.result[1], None,
                                  sm_scale=synth.SM_SCALE, weights_out=w)
    evict = va.prepare_kv_evict(d["slot_idx"], d["kv_indptr"], L, w, budget=budget, sinks=sinks,
                                recent=recent, free_slots=free, free_head=head,
                                outputs=(s_out, len_out, w_out, h_out))
    ws, ns = va.alloc_workspace(B, T, H)
    rows = torch.arange(T, device="cuda")
    # where each request's draft slots go in its list: behind the kept entries
    at = (d["kv_indptr"][:B, None].long() + budget + rows[None]).reshape(-1)

    def step():
        attn()
        weigh()
        evict()
        par, _, _, loc = va.tree_build(dtok, dlp, T, free, h_out, outputs=tree)
        s_out[at] = loc
        d["pool"].index_copy_(0, loc.long(), ddraft)
        return par, loc, va.verify_attn_paged(dq2, d["pool"], s_out, d["kv_indptr"], len_out, par,
                                              sm_scale=synth.SM_SCALE, workspace=ws, nsplit=ns)

    tree = tuple(torch.empty(B, T, dtype=torch.int32, device="cuda") for _ in range(3)) + (
        torch.empty(B * T, dtype=torch.int32, device="cuda"),)
    pool0 = d["pool"].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        par, loc, (vo, vl) = step()
    for _ in range(2):
        d["pool"].copy_(pool0)
        graph.replay()
    torch.cuda.synchronize()
    # chunk attention and the eviction of the weights it measured
    _chunk.check(c, *attn.result)
    freed, slots_left = [], []
    ww = w.cpu().numpy()
    for b in range(B):
        e, N = int(c.kv_indptr[b]), P[b] + n[b]
        kept, gone_b = oracle.evict(c.slot_idx.numpy()[e:e + N], ww[e:e + N], budget, sinks, recent)
        slots_left.append(c.slot_idx.numpy()[e + kept])
        freed += c.slot_idx.numpy()[e + gone_b].tolist()
    h0 = gone + 8 - len(freed)
    assert free.cpu().numpy()[h0:h0 + len(freed)].tolist() == freed
    assert loc.cpu().tolist() == freed[:B * T] and int(h_out.item()) == h0 + B * T
    # the verify step over what is left
    pool = pool0.cpu()
    pool[loc.cpu().long()] = draft
    lists = np.concatenate([np.concatenate([slots_left[b], loc.cpu().numpy()[b * T:(b + 1) * T]])
                            for b in range(B)]).astype(np.int32)
    indptr = np.arange(B + 1, dtype=np.int32) * (budget + T)
    bits, _ = oracle.tree_bits(par.cpu().numpy())
    ro, rl, _ = oracle.verify_attn(synth.as_u16(q2), synth.as_u16(pool), lists, indptr,
                                   np.full(B, budget, dtype=np.int32), bits, synth.SM_SCALE)
    _gpu.compare(vo, vl, ro, rl)


@pytest.mark.parametrize("L,budget", [([30000], 25000), ([200000, 40000, 9000], 100000),
                                      ([90000], 11000)])
def test_in_place_with_more_kept_than_a_block_holds(va, L, budget):
    for kind in ("floats", "ties"):
        _run(va, L, 3, kind, budget, 4, 1024, seed=budget, inplace=True)
    _run(va, L, 0, "equal", budget, 0, budget // 2, seed=budget, inplace=True)
