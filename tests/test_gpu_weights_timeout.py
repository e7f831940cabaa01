"""A weight call whose bounded wait runs out reports it and adds nothing to the totals.

The test build of the library makes the producer warps of the weight kernel wait on a
device flag that nothing sets; the wait gives up after about two seconds, every role
leaves through its abort path, and the context stays usable.  Nothing here faults, traps
or hangs."""
import ctypes
import time

import pytest
import torch

import synth
from tests import _chunk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def libs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mla_speculative_decode_gb300 as va
    from mla_speculative_decode_gb300 import _builder
    va.build()
    va.init()
    th = ctypes.CDLL(_builder.build(testhooks=True))
    th.va_init.argtypes = [ctypes.c_int]
    th.va_test_set_gate.argtypes = [ctypes.c_void_p]
    th.va_kv_weights_paged.argtypes = va.load().va_kv_weights_paged.argtypes
    assert th.va_init(torch.cuda.current_device()) == 0
    yield va, th
    th.va_test_set_gate(None)


# one token of 8 heads: one-SM products; 20 tokens: pairs
@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("inplace", [False, True])
def test_totals_stay_when_a_wait_runs_out(libs, n, inplace):
    va, th = libs
    c = _chunk.make([900, 70], [n, n], 8, seed=510)
    lse = _chunk.call(va, c)[1]
    a = [c.dev(k) for k in ("q", "pool", "slot_idx", "kv_indptr", "prefix_len", "q_indptr")]
    w = torch.rand(c.slot_idx.numel(), generator=torch.Generator().manual_seed(4)).cuda()
    before = w.clone()
    want = va.kv_weights(*a, lse, w, sm_scale=synth.SM_SCALE)
    out = w if inplace else torch.full_like(w, -1.0)
    need = va.load().va_kv_weights_workspace_bytes(2, 2 * n, 8, w.numel(), 0)
    # what an earlier call may have left in the workspace
    ws = torch.full((need // 4,), 1.0, device="cuda").view(torch.uint8)
    args = (*(t.data_ptr() for t in a[:2]), a[1].shape[0], a[1].stride(0),
            *(t.data_ptr() for t in a[2:]), lse.data_ptr(), w.data_ptr(), w.numel(), 2, 2 * n, 8,
            synth.SM_SCALE, 0, 0, 0, ws.data_ptr(), ws.numel(), out.data_ptr(),
            torch.cuda.current_stream().cuda_stream)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")      # nothing ever sets it
    assert th.va_test_set_gate(flag.data_ptr()) == 0
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    assert th.va_kv_weights_paged(*args) == 0
    status = va.read_status(ws)              # waits for the stream
    assert th.va_test_set_gate(None) == 0
    assert status == va.STATUS_TIMEOUT, hex(status)
    assert time.perf_counter() - t0 < 30.0
    assert torch.equal(out, before)
    # the next call is right
    assert th.va_kv_weights_paged(*args) == 0
    assert va.read_status(ws) == 0
    assert torch.equal(out, want)
