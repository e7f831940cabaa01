"""Chunk attention over long lists, every element of every row (needs an sm_103 GPU).

The queries look at the rotary columns only, so the latent columns are free to say
which key they belong to: column t holds 1 for the keys of tiles t, t + 256, ..., column
256 + k for keys k, k + 256, ... of a list.  An output is then the softmax weight of a
few known keys, at least one of each tile of 64 among them: a tile, a key or a piece that
is lost, doubled or swapped changes it by as much as itself, where random values would
average it away.  The weights themselves are summed in 64 bits."""
import math

import pytest
import torch

import synth
from tests import _chunk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def va():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mla_speculative_decode_gb300 as m
    m.build()
    m.init()
    return m


def marked(P, n, H, *, seed, layout):
    c = _chunk.make(P, n, H, seed=seed, layout=layout, unused_nan=False)
    c.q[..., :512] = 0
    for rows in c.key_rows:
        r, j = torch.from_numpy(rows), torch.arange(len(rows))
        c.pool[r, :512] = 0
        c.pool[r, j // 64 % 256] = 1
        c.pool[r, 256 + j % 256] = 1
    return c


def reference(c, window, sinks):
    """out and lse of every row, [total_q, H, 512] and [total_q, H], in 64 bits, and the
    spread of the scores."""
    out = torch.empty(*c.q.shape[:2], 512, dtype=torch.float64, device="cuda")
    lse = torch.empty(*c.q.shape[:2], dtype=torch.float64, device="cuda")
    spread = 0.0
    for b, rows in enumerate(c.key_rows):
        k = c.pool[torch.from_numpy(rows), 512:576].cuda().double()
        N, pad = len(rows), -len(rows) % (64 * 256)
        j = torch.arange(N, device="cuda")
        step = max(1, (1 << 26) // (N * c.H))
        for i0 in range(0, c.n[b], step):
            i1 = min(c.n[b], i0 + step)
            t = slice(int(c.q_indptr[b]) + i0, int(c.q_indptr[b]) + i1)
            q = c.q[t, :, 512:].cuda().double()
            s = torch.einsum("ihd,jd->ihj", q, k) * synth.SM_SCALE
            spread = max(spread, float((q.abs().amax(0) @ k.abs().amax(0)).max()) * synth.SM_SCALE)
            pos = c.P[b] + torch.arange(i0, i1, device="cuda")[:, None]
            see = j <= pos
            if window:
                see &= (j > pos - window) | (j < sinks)
            s.masked_fill_(~see[:, None], -math.inf)
            lse[t] = torch.logsumexp(s, -1)
            p = torch.nn.functional.pad(torch.exp(s - lse[t][..., None]), (0, pad))
            out[t, :, :256] = p.view(i1 - i0, c.H, -1, 256, 64).sum((2, 4))
            out[t, :, 256:] = p.view(i1 - i0, c.H, -1, 256).sum(2)
    return out, lse, spread


CASES = {
    # P, n, H, layout, window, sinks
    "decode": ([9000, 1, 64, 4095, 12345, 63], [1] * 6, 64, "paged", 0, 0),
    "decode_h8": ([40000, 17], [1, 1], 8, "paged", 0, 0),
    "decode_contiguous": ([20001, 777, 128], [1] * 3, 64, "contiguous", 0, 0),
    "decode_window": ([30000, 900, 5000], [1] * 3, 64, "paged", 4096, 4),
    "two_units": ([7000, 129], [1, 1], 128, "paged", 0, 0),
    "short_chunks": ([8000, 1000, 0], [9, 3, 8], 32, "paged", 0, 0),
    "tokens_and_a_chunk": ([500] * 15 + [3000], [1] * 15 + [130], 64, "paged", 0, 0),
    "long_chunk": ([40000], [301], 8, "paged", 0, 0),
    "chunks": ([5000, 0, 300], [130, 77, 65], 64, "paged", 0, 0),
    "prompts": ([0, 0], [700, 333], 64, "contiguous", 0, 0),
    "far_chunk": ([60000], [257], 8, "contiguous", 0, 0),
    "window_chunk": ([9000, 40], [150, 90], 64, "paged", 1024, 64),
    "window_contiguous": ([3000], [200], 64, "contiguous", 300, 70),
}


@pytest.mark.parametrize("flags", [0, 3])
@pytest.mark.parametrize("case", list(CASES))
def test_every_key_counts_once_in_every_row(va, case, flags):
    P, n, H, layout, window, sinks = CASES[case]
    c = marked(P, n, H, seed=540, layout=layout)
    call = _chunk.call(va, c, flags=flags, window=window, sinks=sinks, prepare=True)
    out, lse = call()
    ref, ref_lse, spread = reference(c, window, sinks)
    N = max(p + m for p, m in zip(P, n))
    # weights are not negative, so an output's own size bounds what it is made of
    err = (out.double() - ref).abs()
    rel = 2.0 ** -7 * (1 + 2.0 ** -7) + 2 * _chunk.score_error(spread) + 2 * N * 2.0 ** -24
    assert bool((err <= rel * ref + 1e-30).all()), float((err / (ref + 1e-30)).max())
    lerr = (lse.double() - ref_lse).abs()
    bound = _chunk.score_error(spread) + N * 2.0 ** -24 + 2.0 ** -22 * ref_lse.abs()
    assert bool((lerr <= bound).all()), float(lerr.max())
    assert va.read_status(call.workspace) == 0
