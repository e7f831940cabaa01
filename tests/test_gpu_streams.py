"""Memory that the binding takes for a call belongs to the stream the call runs on: when
the call's object goes while its kernels are still queued, no other stream's work gets
the memory (needs an sm_103 GPU)."""
import pytest
import torch

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


def prepare(va, what, stream):
    c = _chunk.make([700, 40], [30, 20], 32, seed=500,
                    layout="contiguous" if what == "contiguous" else "paged")
    if what != "weights":
        return _chunk.call(va, c, prepare=True, stream=stream)
    a = [c.dev(k) for k in ("q", "pool", "slot_idx", "kv_indptr", "prefix_len", "q_indptr")]
    lse = torch.full((50, 32), 30.0, device="cuda")
    return va.prepare_kv_weights(*a, lse, sm_scale=synth.SM_SCALE, stream=stream)


def taken(call):
    """(address, bytes) of the workspace and the outputs."""
    r = call.result if isinstance(call.result, tuple) else (call.result,)
    return [(t.data_ptr(), t.numel() * t.element_size()) for t in (call.workspace, *r)]


def overlaps(places, t):
    a, n = t.data_ptr(), t.numel()
    return any(a < p + m and p < a + n for p, m in places)


@pytest.mark.parametrize("what", ["paged", "contiguous", "weights"])
def test_a_given_stream_owns_the_memory(va, what):
    side = torch.cuda.Stream()
    prepare(va, what, side)()                # (the library's and the tests' own set-up)
    torch.cuda.synchronize()
    call = prepare(va, what, side)
    places = taken(call)
    del call
    new = [torch.empty(n, dtype=torch.uint8, device="cuda") for _, n in places]
    assert not any(overlaps(places, t) for t in new)


@pytest.mark.parametrize("what", ["paged", "contiguous", "weights"])
def test_a_call_on_another_current_stream_holds_the_memory(va, what):
    side = torch.cuda.Stream()
    call = prepare(va, what, None)
    call()
    torch.cuda.synchronize()
    places = taken(call)
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)       # 0.2 s
        call()
    keep = call._keep                        # (the inputs are the caller's to keep)
    keep = [t for t in keep[1:] if isinstance(t, torch.Tensor)
            and t.data_ptr() not in [p for p, _ in places]]
    del call
    new = [torch.empty(n, dtype=torch.uint8, device="cuda") for _, n in places]
    assert not any(overlaps(places, t) for t in new)
    assert not side.query()
    side.synchronize()
    assert keep


def test_results_used_and_dropped_on_the_current_stream(va):
    """The given stream's next call does not get the results' memory while the current
    stream still reads them."""
    side = torch.cuda.Stream()
    call = prepare(va, "paged", side)
    out = call()[0]
    side.synchronize()
    want = out.clone()
    place, n = out.data_ptr(), out.numel()
    torch.cuda._sleep(400_000_000)           # the current stream is busy for 0.2 s
    kept = out.clone()                       # ... and reads the result then
    del call, out
    with torch.cuda.stream(side):
        other = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    assert other.data_ptr() != place
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert torch.equal(kept, want)


@pytest.mark.parametrize("what", ["paged", "contiguous", "segmented", "accept", "build"])
def test_verify_and_tree_calls_on_a_given_stream(va, what, monkeypatch):
    """One call each on a stream that is busy: neither workspace nor results may be had
    by the current stream while the call is still queued."""
    s = synth.Spec("st", B=2, H=8, T=16, prefix=[900, 70], num_slots=1 << 12, seed=501,
                   layout="contiguous" if what == "contiguous" else "scattered")
    d = _gpu.to_device(synth.make(s))
    side = torch.cuda.Stream()
    places = []
    alloc = va.alloc_workspace

    def spy(*a, **k):
        ws, ns = alloc(*a, **k)
        places.append((ws.data_ptr(), ws.numel()))
        return ws, ns

    monkeypatch.setattr(va, "alloc_workspace", spy)
    kw = dict(sm_scale=s.sm_scale, stream=side)
    g = torch.Generator().manual_seed(502)
    pre = torch.cat([d["slot_idx"][int(d["kv_indptr"][b]):][:p] for b, p in enumerate(s.prefix)])
    loc = torch.cat([d["slot_idx"][int(d["kv_indptr"][b]) + p:][:s.T]
                     for b, p in enumerate(s.prefix)])
    ind = torch.tensor([0, 900, 970], dtype=torch.int32, device="cuda")
    root, lg = torch.randn(2, 999, generator=g).cuda(), torch.randn(2, 16, 999, generator=g).cuda()
    tok = torch.randint(0, 999, (2, 16), generator=g, dtype=torch.int32).cuda()
    ctok = torch.randint(0, 999, (2, 4, 4), generator=g, dtype=torch.int32).cuda()
    clp = torch.log_softmax(torch.randn(2, 4, 4, generator=g), -1).cuda()
    a = (d["prefix_len"], d["parents"])
    run = {"paged": lambda: va.verify_attn_paged(d["q"], d["kv_pool"], d["slot_idx"],
                                                 d["kv_indptr"], *a, **kw),
           "contiguous": lambda: va.verify_attn_contiguous(d["q"], d["kv_pool"], d["kv_start"], *a,
                                                           **kw),
           "segmented": lambda: va.verify_attn_segmented(d["q"], d["kv_pool"], pre, ind, loc,
                                                         tree_parent=d["parents"], **kw),
           "accept": lambda: va.tree_accept(root, lg, tok, d["parents"], stream=side),
           "build": lambda: va.tree_build(ctok, clp, 8, stream=side)}[what]
    run()
    torch.cuda.synchronize()
    places.clear()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)       # 0.2 s
    got = run()
    places += [(t.data_ptr(), t.numel() * t.element_size()) for t in got if t is not None]
    del got
    new = [torch.empty(n, dtype=torch.uint8, device="cuda") for _, n in places]
    assert not any(overlaps(places, t) for t in new)
    assert not side.query()
    side.synchronize()
