"""Calls of norm and rotation that the header allows beside those of test_gpu_rope."""
import ctypes

import pytest
import torch

from tests.test_gpu_rope import bpa, freqs, inputs  # noqa: F401

pytestmark = pytest.mark.gpu


def test_what_the_kernel_before_writes_is_read(bpa):  # noqa: F811
    """Weights, frequencies, positions and rows written late on the same stream, right in front of the call."""
    B, S, H, d = 1, 33, 6, 128
    want_q, want_w = inputs(1, B, S, H, d, torch.bfloat16).cuda(), torch.linspace(0.5, 1.5, d, device="cuda")
    want_pos, want_freq, dy = torch.arange(S, dtype=torch.int32, device="cuda")[None] * 7, freqs(d).cuda(), inputs(2, B, S, H, d, torch.bfloat16).cuda()
    good = bpa.bpa_rope_fwd(want_q, None, want_pos, want_freq, want_w)[0]
    back = bpa.bpa_rope_bwd(want_q, None, dy, None, want_pos, want_freq, want_w)
    torch.cuda.synchronize()
    for _ in range(20):
        q, w, pos, freq, g = (torch.zeros_like(t) for t in (want_q, want_w, want_pos, want_freq, dy))
        torch.cuda.synchronize()
        torch.cuda._sleep(200000)
        for x, y in ((pos, want_pos), (freq, want_freq), (g, dy), (q, want_q), (w, want_w)):
            x.copy_(y)
        got = bpa.bpa_rope_fwd(q, None, pos, freq, w)[0]
        w.zero_()
        w.copy_(want_w)
        grads = bpa.bpa_rope_bwd(q, None, g, None, pos, freq, w)
        torch.cuda.synchronize()
        assert torch.equal(got, good) and torch.equal(grads[0], back[0]) and torch.equal(grads[2], back[2])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,rot,inter", [(128, 128, False), (80, 32, True), (72, 36, False), (511, 510, True)])
def test_backward_without_norm_needs_no_inputs(bpa, d, rot, inter, dtype):  # noqa: F811
    """q and k NULL: the rotation's gradient does not read them."""
    B, S, Hq, Hkv = 2, 9, 3, 2
    q, k = inputs(1, B, S, Hq, d, dtype).cuda(), inputs(2, B, S, Hkv, d, dtype).cuda()
    dq_out, dk_out, freq = inputs(3, B, S, Hq, d, dtype).cuda(), inputs(4, B, S, Hkv, d, dtype).cuda(), freqs(rot).cuda()
    want = bpa.bpa_rope_bwd(q, k, dq_out, dk_out, None, freq, norm=False, interleaved=inter)
    D = bpa.make_rope_desc(q, k, None, freq, norm=False, interleaved=inter)
    D.q = D.k = None
    dq, dk = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    ws = torch.empty(bpa.bpa_rope_workspace_size(D), dtype=torch.uint8, device="cuda")
    L, s = bpa.lib(), torch.cuda.current_stream().cuda_stream
    assert L.bpa_rope_bwd(ctypes.byref(D), dq_out.data_ptr(), dk_out.data_ptr(), dq.data_ptr(), dk.data_ptr(), None, None, ws.data_ptr(),
                          ws.numel(), s) == 0, L.bpa_last_error()
    torch.cuda.synchronize()
    bpa.bpa_check(ws)
    assert torch.equal(dq, want[0]) and torch.equal(dk, want[1]) and want[2] is None and want[3] is None
