"""Batches whose lists hold nothing yet: the first step of a server, or one of idle requests
(needs an sm_103 GPU)."""
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def va():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mla_speculative_decode_gb300 as m
    m.build()
    m.init()
    return m


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("flags", [0, 1, 3])
@pytest.mark.parametrize("rows", [0, 3, 300])
def test_attention_and_weights_of_empty_lists(va, rows, flags):
    q = torch.ones(rows, 8, 576, dtype=torch.bfloat16, device="cuda")
    pool = torch.full((16, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    a = (q, pool, i32(), i32(0, 0, 0), i32(0, 0), i32(0, 0, 0))
    kw = dict(sm_scale=synth.SM_SCALE, flags=flags)
    # no request owns a row: nothing is written
    out = torch.full((rows, 8, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows, 8), 3.0, device="cuda")
    call = va.prepare_chunk_paged(*a, out=out, lse=lse, **kw)
    call()
    assert bool((out == 3).all()) and bool((lse == 3).all())
    assert va.read_status(call.workspace) == 0
    call = va.prepare_kv_weights(*a, lse, **kw)
    assert call().numel() == 0 and va.read_status(call.workspace) == 0
    # tokens without a key: empty rows, reported
    if rows:
        a = (*a[:5], i32(0, rows - 1, rows))
        call = va.prepare_chunk_paged(*a, out=out, lse=lse, **kw)
        call()
        assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
        assert va.read_status(call.workspace) == va.STATUS_BAD_INDPTR | va.STATUS_BAD_SLOT
        call = va.prepare_kv_weights(*a, lse, **kw)
        assert call().numel() == 0
        assert va.read_status(call.workspace) == va.STATUS_BAD_INDPTR


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("free", [False, True])
def test_eviction_of_empty_lists(va, free, inplace):
    slots, w, n, head = i32(), torch.empty(0, device="cuda"), i32(0, 0), i32(2)
    outs = None if inplace else (slots.clone(), i32(-1, -1), w.clone(), i32(-1))
    kw = dict(free_slots=i32(5, 6, 7), free_head=head) if free else {}
    status = i32(0)
    got = va.kv_evict(slots, i32(0, 0, 0), n, w, budget=4, outputs=outs, status=status, **kw)
    assert got[1].tolist() == [0, 0] and status.item() == 0
    assert got[3] is None if not free else got[3].item() == 2
    # lengths that the lists do not have are reported
    got = va.kv_evict(slots, i32(0, 0, 0), i32(9, 0), w, budget=4, outputs=outs, status=status,
                      **kw)
    assert got[1].tolist() == [0, 0] and status.item() == va.STATUS_BAD_INDPTR
