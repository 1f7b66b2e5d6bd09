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
