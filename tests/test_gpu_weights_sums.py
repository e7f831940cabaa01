"""Weight totals from the lse that the attention calls return: each row gives its keys one
in all, however large the scores, and however they come about (needs an sm_103 GPU)."""
import numpy as np
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


def queries(kind, c, g):
    """Rows whose largest scores are about 200."""
    if kind == "large":
        return (40 * torch.randn(c.q.shape, generator=g)).bfloat16()
    # a key's own row, the second half turned round: the sum over the columns climbs
    # to three times what is left of it
    j = torch.randint(0, c.P[0], c.q.shape[:2], generator=g)
    q = 32 * c.pool[torch.from_numpy(c.key_rows[0])[j]][..., :576].float()
    q[..., 288:] *= -0.7
    return q.bfloat16()


# The tensor cores take a score's 36 steps in the same order in both calls, and both give
# the same scale to it, so the two scores are the same number whatever the steps lost.
# What is left, relative to a row's sum of one:
#  - lse: the sum of maximum and logarithm rounds (2^-24 of it), so does its turn into
#    the natural logarithm and back (the two factors are off by 0.27 * 2^-24 in all),
#    and, of a unit in pieces, once more in the merge: 4.3 * 2^-24 |lse|
#  - exponentials and logarithms of both calls: 2^-20
#  - sums: 16 pairs of a tile one after the other, at most 13 tiles, 8 groups of a
#    block's columns four times, at most 5 blocks: 96 * 2^-24 at most
@pytest.mark.parametrize("kind", ["large", "cancel"])
@pytest.mark.parametrize("flags", [0, 3])
@pytest.mark.parametrize("layout,n,H", [("paged", 1, 64), ("paged", 1, 8), ("paged", 2, 64),
                                        ("paged", 20, 64), ("contiguous", 20, 64),
                                        ("paged", 40, 8)])
def test_every_row_gives_one(va, layout, n, H, flags, kind):
    c = _chunk.make([700], [n], H, seed=520, layout=layout)
    c.q = queries(kind, c, torch.Generator().manual_seed(521))
    lse = _chunk.call(va, c, flags=flags)[1]
    assert float(lse.mean()) > 150
    slots = torch.from_numpy(c.key_rows[0].astype(np.int32)).cuda()
    w = va.kv_weights(c.dev("q"), c.dev("pool"), slots, c.dev("kv_indptr"), c.dev("prefix_len"),
                      c.dev("q_indptr"), lse, sm_scale=synth.SM_SCALE, flags=flags)
    rel = abs(float(w.double().sum()) / (n * H) - 1)
    assert rel <= 4.3 * 2.0 ** -24 * float(lse.abs().mean()) + 2.0 ** -20 + 96 * 2.0 ** -24, rel
