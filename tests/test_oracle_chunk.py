"""Pins of the oracle's chunk attention, weight totals and eviction (CPU)."""
import itertools

import numpy as np
import pytest
import torch

import oracle
import synth
from tests import _chunk


def test_sees_by_hand():
    assert oracle.chunk_sees(3, 0, 9).tolist() == [True] * 4
    assert oracle.chunk_sees(5, 2, 1).tolist() == [True, False, False, False, True, True]
    assert oracle.chunk_sees(5, 1, 0).tolist() == [False] * 5 + [True]
    assert oracle.chunk_sees(2, 100, 0).tolist() == [True] * 3


@pytest.mark.parametrize("window,sinks", [(0, 0), (5, 2), (1, 0)])
def test_chunk_attention_equals_the_library_routine(window, sinks):
    c = _chunk.make([11, 0, 3], [4, 7, 0], 2, seed=1, q_before=1)
    out, lse, mass, spread = _chunk.reference(c, window=window, sinks=sinks)
    assert np.isnan(out[0]).all()
    for b in range(3):
        if c.n[b] == 0:
            continue
        t = slice(int(c.q_indptr[b]), int(c.q_indptr[b + 1]))
        q = c.q[t].double().transpose(0, 1)
        k = c.pool[torch.from_numpy(c.key_rows[b])][:, :576].double()
        pos = c.P[b] + torch.arange(c.n[b])[:, None]
        j = torch.arange(c.P[b] + c.n[b])[None]
        mask = j <= pos
        if window:
            mask &= (pos - j < window) | (j < sinks)
        o = torch.nn.functional.scaled_dot_product_attention(
            q, k[None].expand(2, -1, -1), k[None, :, :512].expand(2, -1, -1), attn_mask=mask,
            scale=synth.SM_SCALE)
        np.testing.assert_allclose(out[t], o.transpose(0, 1).numpy(), rtol=1e-10, atol=1e-12)
        s = (q @ k.T) * synth.SM_SCALE
        want = torch.logsumexp(s.masked_fill(~mask, -np.inf), -1).transpose(0, 1).numpy()
        np.testing.assert_allclose(lse[t], want, rtol=1e-12)


def test_keys_without_a_row_are_no_keys():
    c = _chunk.make([6], [2], 1, seed=2)
    c.key_rows[0][[0, 3]] = -1
    out, lse, _, _ = _chunk.reference(c)
    keep = [1, 2, 4, 5, 6, 7]
    k = oracle._widen(synth.as_u16(c.pool))[c.key_rows[0][keep]][:, :576]
    q = oracle._widen(synth.as_u16(c.q))
    s = synth.SM_SCALE * (q[1, 0] @ k.T)
    assert abs(lse[1, 0] - np.log(np.exp(s).sum())) < 1e-10
    c.key_rows[0][:] = -1
    out, lse, _, _ = _chunk.reference(c)
    assert np.all(out == 0) and np.all(np.isneginf(lse))


@pytest.mark.parametrize("window,sinks", [(0, 0), (4, 1)])
def test_weights_are_the_softmax_weights_summed(window, sinks):
    c = _chunk.make([9, 0], [5, 3], 3, seed=3)
    _, lse, _, _ = _chunk.reference(c, window=window, sinks=sinks)
    w = oracle.chunk_weights(synth.as_u16(c.q), synth.as_u16(c.pool), c.key_rows, c.P,
                             c.q_indptr.numpy(), lse, synth.SM_SCALE, window, sinks)
    for b in range(2):
        assert abs(w[b].sum() - c.n[b] * 3) < 1e-9      # every row's weights sum to one
        q = oracle._widen(synth.as_u16(c.q))
        k = oracle._widen(synth.as_u16(c.pool))[c.key_rows[b]][:, :576]
        want = np.zeros(len(w[b]))
        for i, h in itertools.product(range(c.n[b]), range(3)):
            see = np.zeros(len(want), dtype=bool)
            see[:c.P[b] + i + 1] = oracle.chunk_sees(c.P[b] + i, window, sinks)
            e = np.where(see, np.exp(synth.SM_SCALE * (k @ q[int(c.q_indptr[b]) + i, h])), 0)
            want += e / e.sum()
        np.testing.assert_allclose(w[b], want, rtol=1e-10)


def test_evict_by_hand():
    kept, gone = oracle.evict(list("abcdefgh"), [9, 1, 5, 5, 0, 5, 2, 0], 5, 1, 1)
    # first and last stay; of b..g the three largest, equal ones from the left
    assert kept.tolist() == [0, 2, 3, 5, 7] and gone.tolist() == [1, 4, 6]
    kept, gone = oracle.evict(range(4), [np.nan, -np.inf, 0, np.nan], 2, 0, 0)
    assert kept.tolist() == [0, 2] and gone.tolist() == [1, 3]
    kept, gone = oracle.evict(range(3), [1, 2, 3], 3, 0, 0)
    assert kept.tolist() == [0, 1, 2] and gone.size == 0


@pytest.mark.parametrize("seed", range(20))
def test_evict_keeps_the_heaviest_subset(seed):
    """Of all subsets of the allowed size the kept one weighs most, and among
    those it is the first in index order."""
    rng = np.random.default_rng(seed)
    L, sinks, recent = 8, int(rng.integers(0, 3)), int(rng.integers(0, 3))
    budget = sinks + recent + int(rng.integers(0, L - sinks - recent))
    w = rng.integers(0, 4, size=L).astype(float)
    kept, gone = oracle.evict(range(L), w, budget, sinks, recent)
    assert sorted(kept.tolist() + gone.tolist()) == list(range(L))
    free = [j for j in range(sinks, L - recent)]
    best = max(itertools.combinations(free, budget - sinks - recent),
               key=lambda s: (sorted((w[j] for j in s), reverse=True), [-j for j in s]))
    fixed = set(range(sinks)) | set(range(L - recent, L))
    got = [j for j in kept.tolist() if j not in fixed]
    assert sum(w[j] for j in got) == sum(w[j] for j in best)
    assert sorted(got) == sorted(best)
