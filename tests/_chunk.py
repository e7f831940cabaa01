"""Inputs, references and error bounds of the chunk-attention, weight and
eviction tests."""
from __future__ import annotations

from dataclasses import dataclass, field
from typing import List, Optional

import numpy as np
import torch

import oracle
import synth


@dataclass
class Chunk:
    """A batch of ragged chunks with its host-side description."""
    P: List[int]
    n: List[int]
    H: int
    q: torch.Tensor
    pool: torch.Tensor
    key_rows: List[np.ndarray]          # pool row of every key, -1: none
    slot_idx: torch.Tensor
    kv_indptr: torch.Tensor
    prefix_len: torch.Tensor
    q_indptr: torch.Tensor
    kv_start: Optional[torch.Tensor] = None
    extra: dict = field(default_factory=dict)

    def dev(self, name):
        return getattr(self, name).cuda()


def make(P, n, H, *, seed, layout="paged", stride=576, list_gap=0, q_before=0, q_behind=0,
         unused_nan=True, pool_rows=None, scale=1.0):
    """list_gap: list entries behind each request's keys; q_before, q_behind:
    query rows that no request owns.  Pool rows that no list names, and pool
    columns past 576, hold NaN."""
    g = torch.Generator().manual_seed(seed)
    B = len(P)
    lens = [p + m for p, m in zip(P, n)]
    total = sum(lens)
    rows = pool_rows or total + total // 3 + 17 + 5 * B
    pool = synth._bf16_normal((rows, stride), g) * scale
    if stride > 576:
        pool[:, 576:] = float("nan")
    tokens = q_before + sum(n) + q_behind
    q = synth._bf16_normal((tokens, H, 576), g) if tokens else \
        torch.empty(0, H, 576, dtype=torch.bfloat16)
    q_indptr = np.concatenate([[0], np.cumsum(n)]).astype(np.int32) + q_before
    indptr = np.concatenate([[0], np.cumsum([v + list_gap for v in lens])]).astype(np.int32)
    key_rows, start = [], None
    if layout == "paged":
        perm = torch.randperm(rows, generator=g)[:total].numpy()
        at = 0
        for v in lens:
            key_rows.append(perm[at:at + v].astype(np.int64))
            at += v
    else:
        start, at = [], 3
        for v in lens:
            start.append(at)
            key_rows.append(np.arange(at, at + v))
            at += v + 2
    # entries behind a request's keys name a row that must not be read
    slots = np.full(int(indptr[-1]), -5, dtype=np.int32)
    for b, r in enumerate(key_rows):
        slots[indptr[b]:indptr[b] + len(r)] = r
    if unused_nan:
        used = torch.zeros(rows, dtype=torch.bool)
        for r in key_rows:
            used[torch.from_numpy(r)] = True
        pool[~used] = float("nan")
    return Chunk(P=list(P), n=list(n), H=H, q=q, pool=pool.to(torch.bfloat16), key_rows=key_rows,
                 slot_idx=torch.from_numpy(slots), kv_indptr=torch.from_numpy(indptr),
                 prefix_len=torch.tensor(P, dtype=torch.int32),
                 q_indptr=torch.from_numpy(q_indptr),
                 kv_start=None if start is None else torch.tensor(start, dtype=torch.int64))


def call(va, c, *, out=None, lse=None, prepare=False, **kw):
    kw = dict(sm_scale=synth.SM_SCALE, out=out, lse=lse) | kw
    if c.kv_start is not None:
        f = va.prepare_chunk_contiguous if prepare else va.chunk_attn_contiguous
        return f(c.dev("q"), c.dev("pool"), c.dev("kv_start"), c.dev("prefix_len"),
                 c.dev("q_indptr"), **kw)
    f = va.prepare_chunk_paged if prepare else va.chunk_attn_paged
    return f(c.dev("q"), c.dev("pool"), c.dev("slot_idx"), c.dev("kv_indptr"),
             c.dev("prefix_len"), c.dev("q_indptr"), **kw)


def reference(c, *, window=0, sinks=0, sm_scale=synth.SM_SCALE):
    return oracle.chunk_attn(synth.as_u16(c.q), synth.as_u16(c.pool), c.key_rows, c.P,
                             c.q_indptr.numpy(), sm_scale, window, sinks)


# Error bounds, from the kernels' arithmetic alone.
#  - A score is a sum of 576 exact products accumulated in 32 bits, 16 at a time
#    on the tensor cores (36 roundings, each at most 2^-23 of the sum of the
#    products' magnitudes, truncation included); the warp's sum on CUDA cores
#    has fewer than 36 roundings on any path too (18 products and 5 levels of a
#    tree).  So |ds| <= 36 * 2^-23 * spread, spread = max scale * sum |q k|.
#  - exp2 and log2 add a few units of 2^-22 of the value; the row's maximum,
#    scaled, rounds to 2^-24 of itself: in all at most 2^-20 for the scores here.
#  - p rounds to bf16 on the tensor cores (half a step: 2^-8 of p), the output
#    rounds to bf16 (2^-8 of it), both sums of at most N terms are kept in 32 bits
#    (N * 2^-24 of the terms' magnitudes).
def score_error(spread):
    return 36 * 2.0 ** -23 * spread + 2.0 ** -20


def out_bound(out, mass, spread, N):
    rel = 2 * score_error(spread) + 2 * N * 2.0 ** -24
    return 2.0 ** -8 * (1 + 2.0 ** -7) * (np.abs(out) + mass) + rel * mass + 1e-30


def lse_bound(lse, spread, N):
    return score_error(spread) + N * 2.0 ** -24 + 2.0 ** -22 * np.abs(lse)


def check(c, got_out, got_lse, *, window=0, sinks=0, sm_scale=synth.SM_SCALE, ref=None):
    ref_out, ref_lse, mass, spread = ref or reference(c, window=window, sinks=sinks,
                                                      sm_scale=sm_scale)
    o = got_out.float().cpu().numpy().astype(np.float64)
    l = got_lse.cpu().numpy().astype(np.float64)
    N = max(p + m for p, m in zip(c.P, c.n))
    own = np.zeros(o.shape[0], dtype=bool)
    for b in range(len(c.P)):
        own[int(c.q_indptr[b]):int(c.q_indptr[b + 1])] = True
    o, l, ref_out, ref_lse, mass = (x[own] for x in (o, l, ref_out, ref_lse, mass))
    fin = np.isfinite(ref_lse)
    np.testing.assert_array_equal(np.isneginf(l), np.isneginf(ref_lse))
    np.testing.assert_array_equal(np.isnan(l), np.isnan(ref_lse))
    assert np.all(o[np.isneginf(ref_lse)] == 0)
    assert np.all(np.isnan(o[np.isnan(ref_lse)]))
    err = np.abs(o - ref_out)[fin]
    bound = out_bound(ref_out, mass, spread, N)[fin]
    assert np.all(err <= bound), (float(np.max(err - bound)), float(err.max()))
    lerr = np.abs(l[fin] - ref_lse[fin])
    lb = lse_bound(ref_lse, spread, N)[fin]
    assert np.all(lerr <= lb), (float(np.max(lerr - lb)), float(lerr.max()))
