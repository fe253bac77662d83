"""The bounded waits of the losses' products, made to run out on purpose without faulting the GPU: the
stage barriers expect more bytes than the loads bring. The kernel must give up, report it through
relay_device_status() and leave the context usable, for one CTA a product (few rows) and two."""
import ctypes

import pytest
import torch

import objective_ref as ref
import pack_virtual_rank_gb300 as rv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [20, 200])
def test_waits_run_out_and_are_reported(tokens):
    L = rv.lib()
    rv.device_status()                                   # start from a clear fault word
    g = torch.Generator().manual_seed(1)
    h = torch.randn(tokens, 72, generator=g).bfloat16()
    w = (torch.randn(300, 72, generator=g) * 0.2).bfloat16()
    t = torch.randint(0, 300, (tokens,), generator=g, dtype=torch.int32)
    hc, wc, tc, loss = h.cuda(), w.cuda(), t.cuda(), torch.zeros(tokens, device="cuda")
    head = rv.make_head(hc, [wc])
    ws = rv.alloc_head_workspace(head, "cuda")

    def call(extra):
        st = L.relay_test_head_wait(ctypes.byref(head), tc.data_ptr(), loss.data_ptr(), ws.data_ptr(), ws.numel(),
                                    extra, None)
        assert st == rv.OK, L.relay_last_error()
        torch.cuda.synchronize()
    want = ref.head(h, [w], t[:, None], None, None, 1.0)
    call(0)
    rv.device_status()
    ref.close("loss", loss, want["loss"], want["loss_b"])
    call(16)
    assert L.relay_device_status() == rv.ERR_CUDA
    assert b"gave up" in L.relay_last_error()
    assert L.relay_device_status() == rv.OK             # reading cleared the word
    call(0)                                             # the context is still usable
    rv.device_status()
    ref.close("loss", loss, want["loss"], want["loss_b"])
