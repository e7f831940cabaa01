"""Operators of the paged latent cache, as a serving program calls them.

  attn     attention of each request's new tokens over its cache (prompt chunks
           and single tokens in one batch, causal)
  window   the same with a sliding window and a few first tokens that stay
           visible
  weights  attention weight that each cached key received from the new tokens,
           added to a running total
  evict    the keys with the least accumulated weight leave the cache: the slot
           lists are compacted and the freed slots go back to the free list

One latent row per key (576 wide: 512 latent columns, which are also the value,
and 64 rotary columns), shared by all heads; pool rows are named by a slot list
per request, or follow one another.
"""
import math
import random

import numpy as np
import torch

own = False

D_QK, D_V = 576, 512
SM_SCALE = 1.0 / math.sqrt(192.0)
DEV = "cuda"


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one request decodes one token at 8 heads per rank: the smallest call
        dict(name="attn_token_h8_4k", op="attn", layout="paged", B=1, H=8, q_lo=1, q_hi=1,
             p_lo=4096, p_hi=4096, window=0, sinks=0, lens=1),
        # a decode batch: every request one token, contexts from 1k to 32k
        dict(name="attn_token_batch_h64", op="attn", layout="paged", B=32, H=64, q_lo=1, q_hi=1,
             p_lo=1024, p_hi=32768, window=0, sinks=0, lens=2),
        # continuous batching: short and long pieces of prompts over caches of all lengths
        dict(name="attn_mixed_h64", op="attn", layout="paged", B=8, H=64, q_lo=1, q_hi=509,
             p_lo=1, p_hi=16384, window=0, sinks=0, lens=1123),
        # one chunk of a long prompt
        dict(name="attn_chunk_h64_16k", op="attn", layout="paged", B=1, H=64, q_lo=512, q_hi=512,
             p_lo=16384, p_hi=16384, window=0, sinks=0, lens=4),
        # whole fresh prompts of odd lengths, in contiguous rows
        dict(name="attn_prompt_h64", op="attn", layout="contiguous", B=3, H=64, q_lo=517,
             q_hi=2047, p_lo=0, p_hi=0, window=0, sinks=0, lens=5),
        # a chunk at the far end of a 200k context at 8 heads per rank, contiguous rows
        dict(name="attn_chunk_h8_200k", op="attn", layout="contiguous", B=1, H=8, q_lo=256,
             q_hi=256, p_lo=200000, p_hi=200000, window=0, sinks=0, lens=6),
        # a decode batch over long contexts of which a window stays visible
        dict(name="window_token_batch_h64", op="window", layout="paged", B=64, H=64, q_lo=1,
             q_hi=1, p_lo=8192, p_hi=65536, window=4096, sinks=4, lens=7),
        # prompt chunks under a window
        dict(name="window_chunk_h64", op="window", layout="paged", B=2, H=64, q_lo=777, q_hi=1024,
             p_lo=30000, p_hi=65536, window=1024, sinks=64, lens=8),
        # weights of a decode step, accumulated token by token
        dict(name="weights_token_batch_h64", op="weights", layout="paged", B=8, H=64, q_lo=1,
             q_hi=1, p_lo=1024, p_hi=65536, window=0, sinks=0, lens=9),
        # weights that a prompt's last tokens give to all keys before them
        dict(name="weights_chunk_h64_16k", op="weights", layout="paged", B=1, H=64, q_lo=256,
             q_hi=256, p_lo=16384, p_hi=16384, window=0, sinks=0, lens=10),
        # one small cache halved
        dict(name="evict_4k", op="evict", B=1, p_lo=4096, p_hi=4096, budget=2048, sinks=4,
             recent=128, lens=11),
        # a batch of long caches cut to one budget
        dict(name="evict_batch_200k", op="evict", B=64, p_lo=20000, p_hi=200000, budget=16384,
             sinks=4, recent=1024, lens=12),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "window", "window", "weights", "weights", "evict"])
    c = dict(op=op, lens=rng.randrange(1 << 30))
    if op == "evict":
        c["B"] = _log_uniform(rng, 1, 64)
        c["p_hi"] = _log_uniform(rng, 512, 200000)
        c["p_lo"] = max(1, int(c["p_hi"] * rng.uniform(0.1, 1.0)))
        c["budget"] = max(64, int(c["p_hi"] * rng.uniform(0.05, 0.8)))
        c["sinks"] = rng.choice([0, 1, 4, 64])
        c["recent"] = rng.randrange(0, c["budget"] - c["sinks"] + 1)
        return c
    c["layout"] = "paged" if op == "weights" else rng.choice(["paged", "paged", "contiguous"])
    c["H"] = rng.choice([1, 5, 8, 16, 24, 64, 64, 128])
    if rng.random() < 0.5:                       # a decode batch
        c["B"] = _log_uniform(rng, 1, 64)
        c["q_lo"] = c["q_hi"] = 1
    else:                                        # prompt chunks, ragged
        c["B"] = _log_uniform(rng, 1, 8)
        c["q_hi"] = _log_uniform(rng, 2, 2048)
        c["q_lo"] = rng.randrange(1, c["q_hi"] + 1)
    c["p_hi"] = _log_uniform(rng, 1, 200000)
    c["p_lo"] = rng.randrange(0, c["p_hi"] + 1)
    c["window"] = c["sinks"] = 0
    if op == "window" or (op == "weights" and rng.random() < 0.3):
        c["window"] = _log_uniform(rng, 1, 16384)
        c["sinks"] = rng.choice([0, 1, 4, 63, 64, 100])
    # no dearer than the largest listed case
    while True:
        w = work(c)
        if w["flops"] <= 0.9e12 and w["bytes"] <= 0.6e9:
            return c
        if c["q_hi"] > 1:
            c["q_hi"] = (c["q_hi"] + 1) // 2
            c["q_lo"] = min(c["q_lo"], c["q_hi"])
        elif c["B"] > 1:
            c["B"] = (c["B"] + 1) // 2
        else:
            c["p_hi"] //= 2
            c["p_lo"] = min(c["p_lo"], c["p_hi"])


def _lengths(case):
    """The requests' prefix lengths and numbers of new tokens."""
    rng = random.Random(case["lens"])
    B = case["B"]
    P = [rng.randint(case["p_lo"], case["p_hi"]) for _ in range(B)]
    n = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(B)] if "q_lo" in case else [0] * B
    return P, n


def _first(case, pos):
    """First key after the sinks that a token at position `pos` sees."""
    return max(0, pos - case["window"] + 1) if case["window"] > 0 else 0


def work(case):
    P, n = _lengths(case)
    if case["op"] == "evict":
        kept = [min(p, case["budget"]) for p in P]
        freed = sum(p - k for p, k in zip(P, kept))
        return {"bytes": 8 * sum(P) + 8 * sum(kept) + 4 * freed, "flops": sum(P)}
    pairs = keys = 0
    for p, m in zip(P, n):
        lo = _first(case, p)
        keys += p + m - lo + min(lo, case["sinks"])
        for pos in range(p, p + m):
            f = _first(case, pos)
            pairs += pos + 1 - f + min(f, case["sinks"])
    rows = sum(n) * case["H"]
    pairs *= case["H"]
    kv = keys * (D_QK * 2 + (4 if case["layout"] == "paged" else 0))
    if case["op"] == "weights":
        return {"bytes": rows * (D_QK * 2 + 4) + kv + 8 * sum(a + b for a, b in zip(P, n)),
                "flops": 2 * D_QK * pairs}
    return {"bytes": rows * (D_QK * 2 + D_V * 2 + 4) + kv, "flops": 2 * (D_QK + D_V) * pairs}


# ------------------------------------------------------------------ inputs

def _normal(shape, gen):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 1000003 + case["lens"] % 1000003)
    P, n = _lengths(case)
    B = case["B"]
    st = dict(case=case, P=P, n=n)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    lens = [a + b for a, b in zip(P, n)]
    total = sum(lens)
    base = [0]
    for v in lens:
        base.append(base[-1] + v)
    st["base"] = base
    pool_rows = total + total // 4 + 64 + 7 * B
    st["slots"] = torch.randperm(pool_rows, generator=gen, device=DEV)[:total].to(torch.int32)
    st["kv_indptr"] = i32(base)
    st["prefix_len"] = i32(P)

    if case["op"] == "evict":
        # totals of a softmax's weights: a few keys take most of it, and keys
        # that no token has looked at yet stand at zero
        w = torch.exp(2.0 * torch.randn(total, generator=gen, device=DEV)) / 64.0
        w[torch.rand(total, generator=gen, device=DEV) < 0.02] = 0.0
        st["weights"] = w
        freed = sum(max(0, p - case["budget"]) for p in P)
        st["free"] = torch.arange(pool_rows, pool_rows + freed + 32, dtype=torch.int32, device=DEV)
        st["head"] = i32([freed + 16])
        if own:
            import mla_speculative_decode_gb300 as va
            out = (torch.zeros_like(st["slots"]), torch.zeros_like(st["prefix_len"]),
                   torch.zeros_like(w), torch.zeros_like(st["head"]))
            st["call"] = va.prepare_kv_evict(
                st["slots"], st["kv_indptr"], st["prefix_len"], w, budget=case["budget"],
                sinks=case["sinks"], recent=case["recent"], free_slots=st["free"],
                free_head=st["head"], outputs=out)
            st["out"] = out
        return st

    H = case["H"]
    st["pool"] = _normal((pool_rows, D_QK), gen)
    st["q"] = _normal((sum(n), H, D_QK), gen)
    q_base = [0]
    for v in n:
        q_base.append(q_base[-1] + v)
    st["q_base"] = q_base
    st["q_indptr"] = i32(q_base)
    # contiguous requests lie one after the other, with a gap between them
    st["start"] = [base[b] + 7 * b for b in range(B)]
    st["kv_start"] = torch.tensor(st["start"], dtype=torch.int64, device=DEV)
    if case["op"] == "weights":
        # the attention call before gave the rows' lse; the totals so far
        st["lse"] = torch.cat([x.reshape(-1, H) for x in _plain_lse(st)])
        st["weights"] = torch.exp(torch.randn(total, generator=gen, device=DEV)) / 8.0
    if own:
        import mla_speculative_decode_gb300 as va
        kw = dict(sm_scale=SM_SCALE, window=case["window"], sinks=case["sinks"])
        if case["op"] == "weights":
            st["call"] = va.prepare_kv_weights(st["q"], st["pool"], st["slots"], st["kv_indptr"],
                                               st["prefix_len"], st["q_indptr"], st["lse"],
                                               st["weights"],
                                               weights_out=torch.empty_like(st["weights"]), **kw)
        elif case["layout"] == "paged":
            st["call"] = va.prepare_chunk_paged(st["q"], st["pool"], st["slots"], st["kv_indptr"],
                                                st["prefix_len"], st["q_indptr"], **kw)
        else:
            st["call"] = va.prepare_chunk_contiguous(st["q"], st["pool"], st["kv_start"],
                                                     st["prefix_len"], st["q_indptr"], **kw)
    return st


# -------------------------------------------------------------- plain form

def _keys(st, b, k0, k1):
    """Keys k0..k1-1 of request b: [k1 - k0, 576] in 32 bits."""
    if st["case"]["layout"] == "paged":
        rows = st["slots"][st["base"][b] + k0:st["base"][b] + k1].long()
        return st["pool"][rows].float()
    return st["pool"][st["start"][b] + k0:st["start"][b] + k1].float()


def _blocks(st):
    """(request, first token, past the last, pieces of keys) of the passes: the
    keys that a block of tokens can see, in one or two pieces (sinks, window)."""
    c = st["case"]
    for b, (p, m) in enumerate(zip(st["P"], st["n"])):
        step = max(1, min(m, (1 << 28) // max(1, (p + m) * c["H"])))
        for i0 in range(0, m, step):
            i1 = min(m, i0 + step)
            lo = _first(c, p + i0)
            s = min(lo, c["sinks"])
            yield b, i0, i1, [(0, s), (lo, p + i1)] if s else [(lo, p + i1)]


def _scores(st, b, i0, i1, pieces):
    """Scaled scores of the block's rows, hidden keys at -inf, and its keys."""
    c = st["case"]
    k = torch.cat([_keys(st, b, x, y) for x, y in pieces])
    j = torch.cat([torch.arange(x, y, device=k.device) for x, y in pieces])
    q = st["q"][st["q_base"][b] + i0:st["q_base"][b] + i1].float()
    s = (q.reshape(-1, D_QK) @ k.t()).mul_(SM_SCALE).view(i1 - i0, c["H"], -1)
    pos = st["P"][b] + torch.arange(i0, i1, device=k.device)[:, None]
    hidden = j[None, :] > pos
    if c["window"] > 0:
        hidden |= (j[None, :] <= pos - c["window"]) & (j[None, :] >= c["sinks"])
    return s.masked_fill_(hidden[:, None, :], -math.inf), k, j


def _plain_lse(st):
    for blk in _blocks(st):
        s, _, _ = _scores(st, *blk)
        top = s.amax(-1, keepdim=True)
        yield (top + torch.log(torch.exp(s - top).sum(-1, keepdim=True))).squeeze(-1)


def _attn_plain(st):
    outs, lses = [], []
    for blk in _blocks(st):
        s, k, _ = _scores(st, *blk)
        top = s.amax(-1, keepdim=True)
        e = torch.exp(s.sub_(top))
        l = e.sum(-1, keepdim=True)
        o = (e.view(-1, k.shape[0]) @ k[:, :D_V]).view(e.shape[0], e.shape[1], D_V)
        outs.append((o / l).to(torch.bfloat16))
        lses.append((top + torch.log(l)).squeeze(-1))
    return torch.cat(outs), torch.cat(lses)


def _weights_plain(st):
    w = st["weights"].clone()
    for blk in _blocks(st):
        b, i0, i1, _ = blk
        s, _, j = _scores(st, *blk)
        lse = st["lse"][st["q_base"][b] + i0:st["q_base"][b] + i1]
        w[st["base"][b] + j] += torch.exp(s.sub_(lse[:, :, None])).sum((0, 1))
    return w


def _evict_plain(st):
    c = st["case"]
    slots, w = torch.zeros_like(st["slots"]), torch.zeros_like(st["weights"])
    free, freed = st["free"].clone(), []
    for b, p in enumerate(st["P"]):
        x0 = st["base"][b]
        row, val = st["slots"][x0:x0 + p], st["weights"][x0:x0 + p]
        keep = torch.ones(p, dtype=torch.bool, device=row.device)
        if p > c["budget"]:
            lo, hi = c["sinks"], p - c["recent"]
            m = c["budget"] - c["sinks"] - c["recent"]
            order = torch.sort(val[lo:hi], descending=True, stable=True)[1]
            keep[lo:hi] = False
            keep[lo + order[:m]] = True
        k = min(p, c["budget"])
        slots[x0:x0 + k] = row[keep]
        w[x0:x0 + k] = val[keep]
        freed.append(row[~keep])
    freed = torch.cat(freed)
    head = st["head"] - freed.numel()
    free[head.long() + torch.arange(freed.numel(), device=free.device)] = freed
    return dict(slots=slots, prefix_len=st["prefix_len"].clamp(max=c["budget"]), weights=w,
                free=free, head=head)


def run(st):
    op = st["case"]["op"]
    if own:
        got = st["call"]()
        if op == "weights":
            return dict(weights=got)
        if op == "evict":
            slots, prefix_len, w, head = st["out"]
            return dict(slots=slots, prefix_len=prefix_len, weights=w, free=st["free"], head=head)
        return dict(out=got[0], lse=got[1])
    if op == "weights":
        return dict(weights=_weights_plain(st))
    if op == "evict":
        return _evict_plain(st)
    out, lse = _attn_plain(st)
    return dict(out=out, lse=lse)


# ------------------------------------------------------------ in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    P, n, B = st["P"], st["n"], case["B"]
    if case["op"] == "evict":
        slots, w = st["slots"].cpu().numpy(), st["weights"].cpu().numpy().astype(np.float64)
        o_slots, o_w = np.zeros_like(slots), np.zeros_like(w)
        free, freed = st["free"].cpu().numpy().copy(), []
        for b in range(B):
            x0, L = st["base"][b], P[b]
            rank = np.zeros(L)                      # 0: kept whatever its weight
            lo, hi = case["sinks"], L - case["recent"]
            if L > case["budget"]:
                # rank of a key among the keys between: by weight, then by index
                by = np.lexsort((np.arange(lo, hi), -w[x0 + lo:x0 + hi]))
                rank[lo + by] = 1 + np.arange(hi - lo)
                kept = rank <= case["budget"] - case["sinks"] - case["recent"]
            else:
                kept = rank == 0
            idx = np.flatnonzero(kept)
            o_slots[x0:x0 + len(idx)] = slots[x0 + idx]
            o_w[x0:x0 + len(idx)] = w[x0 + idx]
            freed.extend(slots[x0 + np.flatnonzero(~kept)].tolist())
        head = int(st["head"].item()) - len(freed)
        free[head:head + len(freed)] = freed
        return dict(slots=torch.from_numpy(o_slots),
                    prefix_len=torch.tensor([min(p, case["budget"]) for p in P],
                                            dtype=torch.int32),
                    weights=torch.from_numpy(o_w), free=torch.from_numpy(free),
                    head=torch.tensor([head], dtype=torch.int32))
    H = case["H"]
    outs, lses = [], []
    total = st["weights"].double() if case["op"] == "weights" else None
    for b in range(B):
        N = P[b] + n[b]
        rows = st["slots"][st["base"][b]:st["base"][b + 1]].long() if case["layout"] == "paged" \
            else torch.arange(st["start"][b], st["start"][b] + N, device=DEV)
        at = 0
        while at < n[b]:
            # 64-bit scores of a few tokens at a time over every key in reach
            end = min(n[b], at + max(1, (1 << 26) // (N * H)))
            lo = 0
            if case["window"] > 0:
                lo = max(0, P[b] + at + 1 - case["window"])
            j = torch.arange(P[b] + end, device=DEV)
            j = j[(j >= lo) | (j < case["sinks"])]
            K = st["pool"].index_select(0, rows[j]).double()
            q = st["q"][st["q_base"][b] + at:st["q_base"][b] + end].double()
            s = torch.einsum("ihd,jd->ihj", q, K) * SM_SCALE
            i = torch.arange(P[b] + at, P[b] + end, device=DEV)
            see = j[None] <= i[:, None]
            if case["window"] > 0:
                see &= (i[:, None] - j[None] < case["window"]) | (j[None] < case["sinks"])
            if total is not None:
                lse = st["lse"][st["q_base"][b] + at:st["q_base"][b] + end].double()
                e = torch.exp(s - lse[..., None]) * see[:, None]
                total.index_add_(0, st["base"][b] + j, e.sum(dim=(0, 1)))
            else:
                s = torch.where(see[:, None], s, torch.full_like(s, -math.inf))
                lse = torch.logsumexp(s, dim=-1)
                outs.append(torch.einsum("ihj,jd->ihd", torch.exp(s - lse[..., None]), K[:, :D_V]))
                lses.append(lse)
            at = end
    if total is not None:
        return dict(weights=total)
    return dict(out=torch.cat(outs), lse=torch.cat(lses))
