"""Memory that the binding takes for a call belongs to the stream the call runs on: when
the call's object goes while its kernels are still queued, no other stream's work gets
the memory (needs an sm_103 GPU)."""
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
