"""A serving step from the new tokens' projections to the tokens drawn: rows normalised, rotated
and stored, attention over the cache, logits, sampling -- one token per request, and a draft
tree -- each captured in one CUDA graph and replayed; every step against the oracle (needs an
sm_103 GPU)."""
import numpy as np
import pytest
import torch

import oracle
import synth
from tests import _gpu, _tokens

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32
BOUND = 2.0 ** -17.8        # of a mass (see test_gpu_sample.py)


@pytest.fixture(scope="module")
def va():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mla_speculative_decode_gb300 as m
    m.build()
    m.init()
    return m


def drawn_as(row, token, u, temperature, top_k, top_p, min_p):
    want, _, margin = oracle.draw(row, u, temperature, top_k, top_p, min_p)
    return margin <= BOUND or want == token


def test_decode_steps_in_one_graph(va):
    """Tokens' projections come from tables by token: append and rotate -> attention -> logits ->
    sample -> the next step's token; lengths and positions advance on the device."""
    B, H, V, cap = 3, 16, 3001, 64
    g = torch.Generator().manual_seed(70)
    dev = "cuda"
    kv_of = torch.randn(V, 576, generator=g).to(BF16).to(dev)
    q_of = torch.randn(V, H, 192, generator=g).to(BF16).to(dev)
    lat_of = (torch.randn(V, H, 512, generator=g) * 0.3).to(BF16).to(dev)
    head = (torch.randn(H * 512, V, generator=g) * 0.6).to(dev)
    norm = (1 + 0.2 * torch.randn(512, generator=g)).to(BF16).to(dev)
    freq = va.rope_inv_freq(64, scaling="yarn", factor=8.0, original_len=64)
    P = [17, 5, 30]
    pool = torch.randn(B * cap + 9, 576, generator=g).to(BF16).to(dev)
    slots = torch.randperm(B * cap + 9, generator=g)[:B * cap].to(I32).to(dev)
    indptr = torch.tensor([b * cap for b in range(B + 1)], dtype=I32, device=dev)
    prefix = torch.tensor(P, dtype=I32, device=dev)
    q_ind = torch.arange(B + 1, dtype=I32, device=dev)
    token = torch.tensor([1, 500, 3000], dtype=I32, device=dev)
    uniforms = torch.rand(8, B, generator=g).to(dev)
    u = torch.zeros(B, device=dev)
    cfg = dict(temperature=[0.8, 1.0, 1.2], top_k=[50, 0, 400], top_p=[0.95, 0.9, 1.0],
               min_p=[0.0, 0.02, 0.0])
    dcfg = {k: torch.tensor(v, dtype=I32 if k == "top_k" else torch.float32, device=dev)
            for k, v in cfg.items()}
    kv = torch.empty(B, 576, dtype=BF16, device=dev)
    q_in = torch.empty(B, H, 192, dtype=BF16, device=dev)
    q = torch.empty(B, H, 576, dtype=BF16, device=dev)
    new_slot = torch.empty(B, dtype=I32, device=dev)
    status = torch.zeros(1, dtype=I32, device=dev)
    logits = torch.empty(B, V, device=dev)
    rows = torch.arange(B, device=dev) * cap
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    append = va.prepare_kv_append(pool, kv, new_slot, prefix, freq, norm_weight=norm,
                                  interleaved=True, q_pe=q_in[..., 128:], q_out=q[..., 512:],
                                  status=status, stream=st)
    attn = va.prepare_chunk_paged(q, pool, slots, indptr, prefix, q_ind, sm_scale=synth.SM_SCALE,
                                  stream=st)
    draw = va.prepare_sample(logits, u, tokens=token, status=status, stream=st, **dcfg)

    def step():
        t = token.long()
        kv.copy_(kv_of[t])
        q_in.copy_(q_of[t])
        q[..., :512].copy_(lat_of[t])
        new_slot.copy_(slots[rows + prefix])
        append()
        attn()
        torch.mm(attn.result[0].view(B, -1).float(), head, out=logits)
        draw()
        prefix.add_(1)

    with torch.cuda.stream(st):
        step()                                  # (set-up of the libraries)
    torch.cuda.synchronize()
    prefix.copy_(torch.tensor(P))
    token.copy_(torch.tensor([1, 500, 3000]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        step()
    lens = list(P)
    for k in range(6):
        tok = token.tolist()
        u.copy_(uniforms[k])
        before = pool.clone()
        graph.replay()
        torch.cuda.synchronize()
        at = np.array(lens)
        # the new rows, and no others
        kv64 = _tokens.f64(kv_of)[tok]
        want = oracle.latent_rows(kv64, at, freq, _tokens.f64(norm), 1e-6, True)
        where = [int(slots[b * cap + lens[b]]) for b in range(B)]
        err = np.abs(_tokens.f64(pool)[where] - want)
        assert np.all(err <= _tokens.row_bound(want, kv64, 32, norm=True, interleaved=True))
        before[where] = pool[where]
        assert torch.equal(before, pool)
        q64 = _tokens.f64(q_of)[tok][..., 128:]
        want = oracle.rope(q64, at, freq, 0, True)
        err = np.abs(_tokens.f64(q)[..., 512:] - want)
        assert np.all(err <= _tokens.rope_bound(want, q64, BF16, 32, interleaved=True))
        # attention over the cache as it now is
        keys = [slots[b * cap:b * cap + lens[b] + 1].cpu().numpy().astype(np.int64)
                for b in range(B)]
        o, lse, _, _ = oracle.chunk_attn(synth.as_u16(q.cpu()), synth.as_u16(pool.cpu()), keys,
                                         lens, list(range(B + 1)), synth.SM_SCALE)
        _gpu.compare(attn.result[0], attn.result[1], o.reshape(-1, 512), lse.reshape(-1))
        # and the tokens of its logits
        lg = logits.cpu().numpy()
        for b in range(B):
            assert drawn_as(lg[b], int(token[b]), float(u[b]), float(np.float32(cfg["temperature"][b])),
                            cfg["top_k"][b], float(np.float32(cfg["top_p"][b])),
                            float(np.float32(cfg["min_p"][b])))
        lens = [n + 1 for n in lens]
        assert prefix.tolist() == lens and int(status) == 0


def test_sampled_tree_step_in_one_graph(va):
    """Tree build -> the draft's rows and queries at their depths -> verify over two slot lists ->
    logits -> acceptance by sampling, on new inputs at every replay."""
    B, H, T, D, K, V = 2, 16, 12, 5, 4, 2500
    g = torch.Generator().manual_seed(80)
    rng = np.random.default_rng(81)
    dev = "cuda"
    P = [40, 73]
    pool = torch.randn(400, 576, generator=g).to(BF16).to(dev)
    perm = torch.randperm(400, generator=g).to(I32)
    prefix_slots = perm[:sum(P)].to(dev)
    indptr = torch.tensor([0, P[0], sum(P)], dtype=I32, device=dev)
    free = perm[sum(P):].contiguous().to(dev)
    head = torch.zeros(1, dtype=I32, device=dev)
    cand = torch.zeros(B, D, K, dtype=I32, device=dev)
    logp = torch.zeros(B, D, K, device=dev)
    kv = torch.zeros(B * T, 576, device=dev)
    q = torch.randn(B * T, H, 576, generator=g).to(BF16).to(dev)
    q_pe = torch.zeros(B * T, H, 64, dtype=BF16, device=dev)
    W = (torch.randn(H * 512, V, generator=g) * 0.3).to(dev)
    u = torch.zeros(B, T + 1, device=dev)
    root = torch.zeros(B, V, device=dev)
    lg = torch.zeros(B, T, V, device=dev)
    freq = va.rope_inv_freq(64)
    par, tok, depth = (torch.zeros(B, T, dtype=I32, device=dev) for _ in range(3))
    loc = torch.zeros(B * T, dtype=I32, device=dev)
    pos = torch.zeros(B * T, dtype=I32, device=dev)
    base = torch.tensor(P, dtype=I32, device=dev)[:, None]
    out = torch.empty(B * T, H, 512, dtype=BF16, device=dev)
    lse = torch.empty(B * T, H, device=dev)
    ws, ns = va.alloc_workspace(B, T, H)
    status = torch.zeros(1, dtype=I32, device=dev)
    temp = torch.tensor([0.7, 1.0], device=dev)
    top_p = torch.tensor([0.9, 0.95], device=dev)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    append = va.prepare_kv_append(pool, kv, loc, pos, freq, norm_weight=torch.ones(512, device=dev),
                                  q_pe=q_pe, q_out=q[..., 512:], status=status, stream=st)
    accept = va.prepare_tree_accept_sampled(root, lg, tok, par, u, temperature=temp, top_p=top_p,
                                            draft_slots=loc.view(B, T), stream=st)

    def step():
        va.tree_build(cand, logp, T, free, head, outputs=(par, tok, depth, loc), stream=st)
        torch.add(base, depth, out=pos.view(B, T))
        append()
        va.verify_attn_segmented(q, pool, prefix_slots, indptr, loc, tree_parent=par,
                                 sm_scale=synth.SM_SCALE, nsplit=ns, workspace=ws, out=out, lse=lse,
                                 stream=st)
        torch.mm(out.view(B * T, -1).float(), W, out=lg.view(B * T, V))
        # (likely draft tokens: their logits are raised at their parents)
        lg.scatter_add_(2, cand[:, 0, :].long()[:, None].expand(B, T, K), torch.full((B, T, K), 4.0,
                                                                                    device=dev))
        accept()

    with torch.cuda.stream(st):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        step()
    accepted = 0
    for k in range(4):
        c = rng.permuted(np.tile(np.arange(V), (B, D, 1)), axis=-1)[..., :K].astype(np.int32)
        c[:, 1:] = c[:, :1]                       # the same candidates at every depth
        lp = np.log(rng.dirichlet(np.ones(K), size=(B, D))).astype(np.float32)
        cand.copy_(torch.from_numpy(c))
        logp.copy_(torch.from_numpy(lp))
        kv.copy_(torch.randn(B * T, 576, generator=g))
        q_pe.copy_(torch.randn(B * T, H, 64, generator=g))
        u.copy_(torch.rand(B, T + 1, generator=g))
        r = torch.randn(B, V, generator=g)
        r.scatter_add_(1, torch.from_numpy(c[:, 0]).long(), torch.full((B, K), 8.0))
        root.copy_(r)
        head.zero_()
        status.zero_()
        graph.replay()
        torch.cuda.synchronize()
        par_w, tok_w, _, _ = oracle.tree_build(c, lp, T)
        np.testing.assert_array_equal(par.cpu().numpy(), par_w)
        kv64, p = _tokens.f64(kv), pos.cpu().numpy()
        np.testing.assert_array_equal(p.reshape(B, T), np.array(P)[:, None] + depth.cpu().numpy())
        want = oracle.latent_rows(kv64, p, freq, np.ones(512))
        got = _tokens.f64(pool)[loc.cpu().numpy()]
        assert np.all(np.abs(got - want) <= _tokens.row_bound(want, kv64, 32, norm=True))
        slots = np.concatenate([np.concatenate([prefix_slots.cpu().numpy()[sum(P[:b]):sum(P[:b + 1])],
                                                loc.cpu().numpy()[b * T:(b + 1) * T]])
                                for b in range(B)]).astype(np.int32)
        ind = np.array([0, P[0] + T, sum(P) + 2 * T], np.int32)
        bits, _ = oracle.tree_bits(par_w)
        ro, rl, _ = oracle.verify_attn(synth.as_u16(q.cpu()), synth.as_u16(pool.cpu()), slots, ind,
                                       np.array(P, np.int32), bits, synth.SM_SCALE)
        _gpu.compare(out, lse, ro, rl)
        # acceptance: each position's token, and the walk along them
        rows = torch.cat((root[:, None], lg), 1).cpu().numpy()
        alen, nodes, aslots, bonus, _ = (x.cpu().numpy() for x in accept.result)
        assert va.read_status(accept.workspace) == 0 and int(status) == 0
        for b in range(B):
            cur, t = -1, None
            for m in range(alen[b] + 1):
                here = rows[b, cur + 1]
                t = int(tok_w[b, nodes[b, m]]) if m < alen[b] else int(bonus[b])
                assert drawn_as(here, t, float(u[b, cur + 1]), float(temp[b]), 0, float(top_p[b]), 0.0)
                kids = [i for i in range(T) if par_w[b, i] == cur and tok_w[b, i] == t]
                assert (kids[:1] == [nodes[b, m]]) if m < alen[b] else not kids
                if m < alen[b]:
                    cur = int(nodes[b, m])
                    assert aslots[b, m] == loc[b * T + cur]
            accepted += int(alen[b])
    assert accepted > 0
