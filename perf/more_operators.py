"""Operators around the attention of a serving step, as a program calls them: what
prepares the new tokens for it, and what picks the next ones after it.

  rope     rotary positions of query (or key) heads: interleaved and half layouts,
           a part of the head, frequencies scaled for long contexts, and the
           inverse rotation (the gradient)
  append   the new tokens' rows of the latent cache: the 512 latent columns are
           RMS-normalised, the 64 rotary columns rotated, and the row goes to its
           slot of the pool; the same call rotates the queries' rotary columns
  sample   one token per row of logits: temperature, top-k, top-p and min-p, drawn
           by given random numbers
  accept   a draft tree accepted by sampling: every position's target token is
           drawn as above, and the tree is walked along the tokens drawn

Sampling: w_i = exp((l_i - max l) / temperature).  top-k keeps the k largest logits;
of those, top-p keeps the shortest run, largest first, that holds top_p of their
mass; min-p keeps w_i >= min_p.  Equal logits: the lower index first.  The token is
the first in index order at which the kept mass so far exceeds uniform * (kept mass).
"""
import math
import random

import numpy as np
import torch

own = False

D_QK, D_V, D_ROT = 576, 512, 64
EPS = 1e-6
DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# Frequency scalings: (name, factor, original length)
SCALINGS = {"none": ("none", 1.0, 0), "linear": ("linear", 4.0, 0), "ntk": ("ntk", 8.0, 0),
            "yarn": ("yarn", 40.0, 4096)}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one request decodes one token at 8 heads per rank: the smallest call.  The rotary
        # columns of the projected queries go behind the latent ones of the absorbed queries
        dict(name="rope_token_h8", op="rope", tokens=1, heads=8, width=64, off=0, rot=64, x_width=192,
             x_col=128, out_width=576, out_col=512, dtype="bf16", interleaved=True, inverse=False,
             scaling="yarn", pos_hi=200000),
        # a decode batch
        dict(name="rope_batch_h64", op="rope", tokens=64, heads=64, width=64, off=0, rot=64,
             x_width=192, x_col=128, out_width=576, out_col=512, dtype="bf16", interleaved=True,
             inverse=False, scaling="yarn", pos_hi=65536),
        # whole prompts, half layout
        dict(name="rope_prompt_h64", op="rope", tokens=4093, heads=64, width=64, off=0, rot=64,
             x_width=192, x_col=128, out_width=576, out_col=512, dtype="bf16", interleaved=False,
             inverse=False, scaling="none", pos_hi=4093),
        # gradient of whole heads of which a part is rotated, in 32 bits
        dict(name="rope_grad_part_f32", op="rope", tokens=2047, heads=32, width=128, off=0, rot=64,
             x_width=128, x_col=0, out_width=128, out_col=0, dtype="f32", interleaved=False,
             inverse=True, scaling="linear", pos_hi=8192),
        # a decode step's new rows and queries in one call
        dict(name="append_token_batch_h64", op="append", tokens=64, heads=64, dtype="bf16", norm=True,
             interleaved=True, scaling="yarn", pos_hi=65536, pad=0),
        # a chunk of a prompt, a few rows of padding behind it
        dict(name="append_chunk_h64", op="append", tokens=517, heads=64, dtype="bf16", norm=True,
             interleaved=True, scaling="yarn", pos_hi=16384, pad=5),
        # the rows of whole prompts, from a 32-bit projection; the queries are rotated elsewhere
        dict(name="append_prompt_f32", op="append", tokens=16381, heads=0, dtype="f32", norm=True,
             interleaved=False, scaling="none", pos_hi=16381, pad=0),
        # one request's next token
        dict(name="sample_token_32k", op="sample", rows=1, V=32000, dtype="f32", filters="top_p"),
        # a decode batch with every request's own settings, 16-bit logits
        dict(name="sample_batch64_129k_bf16", op="sample", rows=64, V=129280, dtype="bf16",
             filters="mixed"),
        # a large decode batch, 32-bit logits
        dict(name="sample_batch256_129k", op="sample", rows=256, V=129280, dtype="f32",
             filters="mixed"),
        # one request's draft tree
        dict(name="accept_tree16_129k", op="accept", B=1, T=16, V=129280, dtype="f32",
             filters="top_p"),
        # the trees of a batch
        dict(name="accept_batch8_tree16_129k", op="accept", B=8, T=16, V=129280, dtype="f32",
             filters="mixed"),
    ]


MAX_BYTES = 140e6      # of a drawn case: the largest listed one reads 132 MB


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "sample", "sample", "accept"])
    c = dict(op=op)
    if op in ("rope", "append"):
        c["tokens"] = _log_uniform(rng, 1, 16384)
        c["scaling"] = rng.choice(sorted(SCALINGS))
        c["pos_hi"] = _log_uniform(rng, 1, 1 << 20)
        c["interleaved"] = rng.random() < 0.5
        c["dtype"] = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "rope":
        c["heads"] = rng.choice([1, 5, 8, 16, 24, 64, 128])
        if rng.random() < 0.5:            # rotary columns of one tensor into another's
            c.update(width=64, off=0, rot=64, x_width=192, x_col=128, out_width=576, out_col=512)
        else:                             # whole heads, all or a part of them rotated
            width = rng.choice([64, 80, 96, 128, 192, 256])
            rot = rng.choice([r for r in (16, 32, 48, 64, 80, 96, 128, 192, 256) if r <= width])
            off = rng.choice([0, width - rot])
            c.update(width=width, off=off, rot=rot, x_width=width, x_col=0, out_width=width,
                     out_col=0)
        c["inverse"] = rng.random() < 0.3
    elif op == "append":
        c["heads"] = rng.choice([0, 1, 5, 8, 16, 64, 128])
        c["norm"] = rng.random() < 0.8
        c["pad"] = rng.choice([0, 0, 1, c["tokens"] // 3])
    else:
        c["V"] = _log_uniform(rng, 100, 262144)
        c["dtype"] = rng.choice(["f32", "f32", "bf16", "f16"])
        c["filters"] = rng.choice(["none", "top_k", "top_p", "min_p", "mixed", "mixed"])
        if op == "sample":
            c["rows"] = _log_uniform(rng, 1, 512)
        else:
            c["B"] = _log_uniform(rng, 1, 32)
            c["T"] = _log_uniform(rng, 1, 64)
    while work(c)["bytes"] > MAX_BYTES:   # no dearer than the largest listed case
        if op in ("rope", "append"):
            c["tokens"] = (c["tokens"] + 1) // 2
            c["pad"] = min(c.get("pad", 0), c["tokens"] // 3)
        elif op == "sample":
            c["rows"] = (c["rows"] + 1) // 2
        elif c["B"] > 1:
            c["B"] = (c["B"] + 1) // 2
        else:
            c["T"] = (c["T"] + 1) // 2
    return c


def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    if op == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * case["width"] * es + 4 * case["tokens"], "flops": 3 * n * case["rot"]}
    if op == "append":
        n, live = case["tokens"] * case["heads"], case["tokens"] - case["pad"]
        # queries read and written, new rows read, pool rows written, slots and positions
        return {"bytes": 4 * n * D_ROT + live * D_QK * (es + 2) + 8 * case["tokens"]
                + (D_V * es if case["norm"] else 0),
                "flops": 3 * n * D_ROT + live * (3 * D_ROT + 4 * D_V)}
    rows = case["rows"] if op == "sample" else case["B"] * (case["T"] + 1)
    out = 28 * rows if op == "sample" else 8 * rows + case["B"] * (16 + 20 * case["T"])
    return {"bytes": rows * case["V"] * es + out, "flops": 4 * rows * case["V"]}


# ------------------------------------------------------------------ inputs

def _frequencies(rot, scaling):
    """Radians per position of each pair, in 64 bits."""
    kind, factor, orig = SCALINGS[scaling]
    base = 10000.0
    if kind == "ntk":
        base *= factor ** (rot / max(rot - 2, 1))
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if kind == "linear":
        f = [x / factor for x in f]
    if kind == "yarn":
        # pairs that turn more than 32 times over the original length keep their frequency,
        # those that turn less than once are interpolated, those between are mixed
        def pair(turns):
            return rot * math.log(orig / (2 * math.pi * turns)) / (2 * math.log(base))
        lo, hi = max(0, math.floor(pair(32.0))), min(rot - 1, math.ceil(pair(1.0)))
        ramp = [min(1.0, max(0.0, (i - lo) / (max(hi - lo, 0.001)))) for i in range(rot // 2)]
        f = [x / factor * r + x * (1.0 - r) for x, r in zip(f, ramp)]
    return f


def _amplitude(scaling):
    return 0.1 * math.log(40.0) + 1.0 if scaling == "yarn" else 1.0


def _settings(case, n, gen):
    """Each request's temperature, top-k, top-p and min-p (None: not used by the batch)."""
    kind = case["filters"]

    def pick(values, dtype):
        i = torch.randint(0, len(values), (n,), generator=gen, device=DEV)
        return torch.tensor(values, dtype=dtype, device=DEV)[i]

    s = dict(temperature=pick([0.6, 0.8, 1.0, 1.0, 1.3], torch.float32), top_k=None, top_p=None,
             min_p=None)
    if kind == "mixed":       # some requests are greedy, some use no filter, some several
        s["temperature"] = pick([0.0, 0.6, 0.8, 1.0, 1.0, 1.3], torch.float32)
    if kind in ("top_k", "mixed"):
        s["top_k"] = pick([0, 0, 1, 20, 50, 500], torch.int32)
    if kind in ("top_p", "mixed"):
        s["top_p"] = pick([1.0, 0.8, 0.9, 0.95, 0.99], torch.float32)
    if kind in ("min_p", "mixed"):
        s["min_p"] = pick([0.0, 0.0, 0.02, 0.1], torch.float32)
    return s


def _logits(n, V, dtype, gen):
    """Rows of a model's logits: a broad tail, and a few dozen likely tokens, in some rows
    far ahead of it and in others hardly."""
    x = torch.randn(n, V, generator=gen, device=DEV) * 2.0
    k = min(V, 48)
    top = torch.randint(0, V, (n, k), generator=gen, device=DEV)
    lift = 9.0 + 3.0 * torch.randn(n, k, generator=gen, device=DEV)
    x.scatter_add_(1, top, lift)
    x *= 0.7 + 0.6 * torch.rand(n, 1, generator=gen, device=DEV)
    return x.to(DTYPES[dtype])


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 1000003 + 17)
    st = dict(case=case)
    op = case["op"]
    if own:
        import mla_speculative_decode_gb300 as va
    if op in ("rope", "append"):
        n, rot = case["tokens"], case["rot"] if op == "rope" else D_ROT
        dt = DTYPES[case["dtype"]]
        # a batch of runs of tokens, each at its own position
        start = torch.randint(0, case["pos_hi"], (n,), generator=gen, device=DEV)
        runs = (torch.arange(n, device=DEV) // 128) * 128
        pos = start[runs] + torch.arange(n, device=DEV) - runs
        st["pos"] = pos.to(torch.int32)
        st["inv_freq"] = _frequencies(rot, case["scaling"])
        st["freq"] = torch.tensor(st["inv_freq"], dtype=torch.float64, device=DEV)
        kw = dict(interleaved=case["interleaved"], amplitude=_amplitude(case["scaling"]))
    if op == "rope":
        buf = torch.randn(n, case["heads"], case["x_width"], generator=gen, device=DEV).to(dt)
        st["x"] = buf[..., case["x_col"]:case["x_col"] + case["width"]]
        out = torch.zeros(n, case["heads"], case["out_width"], dtype=dt, device=DEV)
        st["out"] = out[..., case["out_col"]:case["out_col"] + case["width"]]
        if own:
            st["call"] = va.prepare_rope(st["x"], st["pos"], st["inv_freq"], rot_offset=case["off"],
                                         inverse=case["inverse"], out=st["out"], **kw)
    elif op == "append":
        rows = n + n // 4 + 16
        st["pool"] = torch.randn(rows, D_QK, generator=gen, device=DEV).to(torch.bfloat16)
        st["kv"] = (torch.randn(n, D_QK, generator=gen, device=DEV) * 3.0).to(dt)
        st["slots"] = torch.randperm(rows, generator=gen, device=DEV)[:n].to(torch.int32)
        if case["pad"]:
            st["slots"][n - case["pad"]:] = -1
        st["norm"] = (1.0 + 0.2 * torch.randn(D_V, generator=gen, device=DEV)).to(dt) \
            if case["norm"] else None
        st["q_pe"] = st["q_out"] = None
        if case["heads"]:
            st["q_pe"] = torch.randn(n, case["heads"], 192, generator=gen, device=DEV) \
                .to(torch.bfloat16)[..., 128:]
            st["q_out"] = torch.zeros(n, case["heads"], D_QK, dtype=torch.bfloat16,
                                      device=DEV)[..., D_V:]
        if own:
            st["call"] = va.prepare_kv_append(st["pool"], st["kv"], st["slots"], st["pos"],
                                              st["inv_freq"], norm_weight=st["norm"], eps=EPS,
                                              q_pe=st["q_pe"], q_out=st["q_out"], **kw)
    elif op == "sample":
        n = case["rows"]
        st["logits"] = _logits(n, case["V"], case["dtype"], gen)
        st["set"] = _settings(case, n, gen)
        st["u"] = torch.rand(n, generator=gen, device=DEV)
        if own:
            st["call"] = va.prepare_sample(st["logits"], st["u"], **st["set"])
    else:
        B, T, V = case["B"], case["T"], case["V"]
        lg = _logits(B * (T + 1), V, case["dtype"], gen).view(B, T + 1, V)
        st["root"], st["logits"] = lg[:, 0].contiguous(), lg[:, 1:].contiguous()
        st["set"] = _settings(case, B, gen)
        st["u"] = torch.rand(B, T + 1, generator=gen, device=DEV)
        rng = random.Random(seed * 7919 + 3)
        par = [[rng.randrange(-1, i) if i else -1 for i in range(T)] for _ in range(B)]
        st["parent"] = torch.tensor(par, dtype=torch.int32, device=DEV)
        # the drafter proposes likely tokens: each node one of its parent's four best
        best = torch.topk(lg.float(), min(4, V), dim=-1)[1]
        at = st["parent"].long() + 1
        which = torch.randint(0, best.shape[-1], (B, T, 1), generator=gen, device=DEV)
        st["tokens"] = best.gather(1, at[..., None].expand(-1, -1, best.shape[-1])) \
            .gather(2, which).squeeze(-1).to(torch.int32)
        st["slots"] = torch.randperm(4 * B * T, generator=gen, device=DEV)[:B * T].view(B, T) \
            .to(torch.int32)
        if own:
            st["call"] = va.prepare_tree_accept_sampled(st["root"], st["logits"], st["tokens"],
                                                        st["parent"], st["u"],
                                                        draft_slots=st["slots"], **st["set"])
    return st


# -------------------------------------------------------------- plain form

def _rotate(x, st, inverse=False):
    """x [tokens, heads, rot] in 32 bits, rotated."""
    c = st["case"]
    ang = st["pos"].double()[:, None] * st["freq"]
    if inverse:
        ang = -ang
    amp = _amplitude(c["scaling"])
    cos, sin = (ang.cos() * amp).float()[:, None], (ang.sin() * amp).float()[:, None]
    if c["interleaved"]:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    half = x.shape[-1] // 2
    a, b = x[..., :half], x[..., half:]
    return torch.cat((a * cos - b * sin, a * sin + b * cos), -1)


def _rope_plain(st):
    c = st["case"]
    x = st["x"].float()
    lo, hi = c["off"], c["off"] + c["rot"]
    y = torch.cat((x[..., :lo], _rotate(x[..., lo:hi], st, c["inverse"]), x[..., hi:]), -1)
    st["out"].copy_(y.to(st["x"].dtype))
    return st["out"]


def _append_plain(st):
    kv = st["kv"].float()
    lat = kv[:, :D_V]
    if st["norm"] is not None:
        lat = lat * torch.rsqrt((lat * lat).mean(-1, keepdim=True) + EPS) * st["norm"].float()
    row = torch.cat((lat, _rotate(kv[:, None, D_V:], st)[:, 0]), -1).to(torch.bfloat16)
    live = st["slots"].shape[0] - st["case"]["pad"]
    st["pool"][st["slots"][:live].long()] = row[:live]
    out = dict(pool=st["pool"])
    if st["q_pe"] is not None:
        st["q_out"].copy_(_rotate(st["q_pe"].float(), st).to(torch.bfloat16))
        out["q"] = st["q_out"]
    return out


def _sample_plain(logits, u, temperature, top_k, top_p, min_p):
    """Tokens and log-probabilities of [n, V] logits; settings and u are [n]."""
    n, V = logits.shape
    greedy = temperature <= 0
    t = torch.where(greedy, torch.ones_like(temperature), temperature).double()[:, None]
    val, idx = torch.sort(logits.float(), dim=-1, descending=True, stable=True)
    w = torch.exp((val.double() - val[:, :1].double()) / t)
    keep = torch.ones_like(val, dtype=torch.bool)
    if top_k is not None:
        k = torch.where(top_k > 0, top_k, torch.full_like(top_k, V))[:, None]
        keep &= torch.arange(V, device=val.device) < k
    if top_p is not None:
        p = top_p.double()[:, None]
        cum = (w * keep).cumsum(-1)
        keep &= (p >= 1) | (cum - w < p * cum[:, -1:])
    if min_p is not None:
        keep &= w >= min_p.double()[:, None]
    keep[:, 0] = True
    kept = torch.zeros_like(w).scatter_(1, idx, w * keep)
    cum = kept.cumsum(-1)
    total = cum[:, -1:]
    tok = (cum <= u.double()[:, None] * total).sum(-1).clamp_(max=V - 1)
    tok = torch.where(greedy, idx[:, 0], tok)
    logp = torch.log(kept.gather(1, tok[:, None]) / total).squeeze(-1)
    logp = torch.where(greedy, torch.zeros_like(logp), logp)
    return tok.to(torch.int32), logp.float()


def _walk(tokens, drawn, parent, slots):
    """The path of each tree along the drawn tokens (position 0: the prefix)."""
    B, T = tokens.shape
    cur = torch.full((B,), -1, dtype=torch.int64, device=tokens.device)
    length = torch.zeros(B, dtype=torch.int32, device=tokens.device)
    nodes, acc = torch.full_like(tokens, -1), torch.full_like(tokens, -1)
    node = torch.arange(T, device=tokens.device).expand(B, T)
    bonus = drawn[:, 0].clone()
    alive = torch.ones(B, dtype=torch.bool, device=tokens.device)
    for step in range(T):
        hit = (parent == cur[:, None]) & (tokens == bonus[:, None])
        first = torch.where(hit, node, torch.full_like(node, T)).amin(-1)
        alive = alive & (first < T)
        at = first.clamp(max=T - 1)
        nodes[:, step] = torch.where(alive, at.to(torch.int32), nodes[:, step])
        acc[:, step] = torch.where(alive, slots.gather(1, at[:, None])[:, 0], acc[:, step])
        length += alive
        cur = torch.where(alive, at, cur)
        bonus = torch.where(alive, drawn.gather(1, at[:, None] + 1)[:, 0], bonus)
    return length, nodes, acc, bonus


def _accept_plain(st):
    B, T, V = st["logits"].shape
    each = {k: None if v is None else v.repeat_interleave(T + 1) for k, v in st["set"].items()}
    lg = torch.cat((st["root"][:, None], st["logits"]), 1).view(-1, V)
    tok, logp = _sample_plain(lg, st["u"].view(-1), **each)
    length, nodes, acc, bonus = _walk(st["tokens"], tok.view(B, T + 1), st["parent"], st["slots"])
    return dict(length=length, nodes=nodes, slots=acc, bonus=bonus, logprob=logp.view(B, T + 1))


def run(st):
    op = st["case"]["op"]
    if own:
        got = st["call"]()
        if op == "rope":
            return got
        if op == "append":
            return dict(pool=got[0]) if got[1] is None else dict(pool=got[0], q=got[1])
        if op == "sample":
            return dict(tokens=got[0], logprob=got[1])
        return dict(zip(("length", "nodes", "slots", "bonus", "logprob"), got))
    if op == "rope":
        return _rope_plain(st)
    if op == "append":
        return _append_plain(st)
    if op == "sample":
        tok, logp = _sample_plain(st["logits"], st["u"], **st["set"])
        return dict(tokens=tok, logprob=logp)
    return _accept_plain(st)


# ------------------------------------------------------------ in 64 bits

def _turn(x, st, sign=1.0):
    """x [tokens, heads, rot] in 64 bits, as complex numbers times a unit one."""
    c = st["case"]
    z = torch.view_as_complex(x.unflatten(-1, (-1, 2)).contiguous()) if c["interleaved"] \
        else torch.complex(*x.chunk(2, -1))
    ang = sign * torch.outer(st["pos"].double(), st["freq"])
    z = z * torch.polar(torch.full_like(ang, _amplitude(c["scaling"])), ang)[:, None]
    return torch.view_as_real(z).flatten(-2) if c["interleaved"] else torch.cat((z.real, z.imag), -1)


def _draw_exact(row, u, temperature, top_k, top_p, min_p):
    """One row's token and log-probability, from the definition."""
    row = row.astype(np.float64)
    V = len(row)
    if temperature <= 0:
        return int(np.argmax(row)), 0.0
    p = np.exp((row - row.max()) / temperature)
    p /= p.sum()
    order = np.argsort(-row, kind="stable")
    n = V if not top_k or top_k < 0 else min(V, int(top_k))
    order = order[:n]
    if top_p is not None and top_p < 1:
        mass = np.cumsum(p[order])
        # the shortest run of the largest whose mass reaches top_p of them all
        order = order[:max(1, int(np.searchsorted(mass, float(top_p) * mass[-1], side="left")) + 1)]
    if min_p is not None and min_p > 0:
        order = order[p[order] >= float(min_p) * p[order[0]]]
    idx = np.sort(order)
    mass = np.cumsum(p[idx])
    at = min(int(np.searchsorted(mass, u * mass[-1], side="right")), len(idx) - 1)
    return int(idx[at]), math.log(p[idx[at]] / mass[-1])


def _draw_rows(rows, u, settings):
    host = {k: None if v is None else v.cpu().numpy().astype(np.float64)
            for k, v in settings.items()}
    u = u.cpu().numpy().astype(np.float64)
    got = []
    for i in range(rows.shape[0]):
        got.append(_draw_exact(rows[i].float().cpu().numpy(), u[i],
                               *(None if host[k] is None else host[k][i]
                                 for k in ("temperature", "top_k", "top_p", "min_p"))))
    return [t for t, _ in got], [lp for _, lp in got]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        y = st["x"].double()
        lo, hi = case["off"], case["off"] + case["rot"]
        y[..., lo:hi] = _turn(y[..., lo:hi], st, -1.0 if case["inverse"] else 1.0)
        return y
    if op == "append":
        pool, kv = st["pool"].double(), st["kv"].double()
        if st["norm"] is not None:
            rms = torch.sqrt(kv[:, :D_V].pow(2).sum(-1, keepdim=True) / D_V + EPS)
            kv[:, :D_V] = kv[:, :D_V] / rms * st["norm"].double()
        kv[:, D_V:] = _turn(kv[:, None, D_V:], st)[:, 0]
        live = st["slots"] >= 0
        pool[st["slots"][live].long()] = kv[live]
        out = dict(pool=pool)
        if st["q_pe"] is not None:
            out["q"] = _turn(st["q_pe"].double(), st)
        return out
    if op == "sample":
        tok, logp = _draw_rows(st["logits"], st["u"], st["set"])
        return dict(tokens=torch.tensor(tok, dtype=torch.int32),
                    logprob=torch.tensor(logp, dtype=torch.float64))
    B, T, V = case["B"], case["T"], case["V"]
    out = dict(length=torch.zeros(B, dtype=torch.int32),
               nodes=torch.full((B, T), -1, dtype=torch.int32),
               slots=torch.full((B, T), -1, dtype=torch.int32),
               bonus=torch.zeros(B, dtype=torch.int32), logprob=[])
    par, tok, slot = (st[k].tolist() for k in ("parent", "tokens", "slots"))
    for b in range(B):
        each = {k: None if v is None else v[b:b + 1].expand(T + 1) for k, v in st["set"].items()}
        drawn, logp = _draw_rows(torch.cat((st["root"][b:b + 1], st["logits"][b])), st["u"][b], each)
        out["logprob"].append(logp)
        cur, n = -1, 0
        while True:
            kids = [i for i in range(T) if par[b][i] == cur and tok[b][i] == drawn[cur + 1]]
            if not kids:
                break
            cur = kids[0]
            out["nodes"][b, n], out["slots"][b, n] = cur, slot[b][cur]
            n += 1
        out["length"][b], out["bonus"][b] = n, drawn[cur + 1]
    out["logprob"] = torch.tensor(out["logprob"], dtype=torch.float64)
    return out
