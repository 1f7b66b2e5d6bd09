"""Norm and rotation where what goes through them is far from 1: eps far above the squares that it joins, weights
far from 1 beside values far from 1.  Tolerances of test_gpu_rope; the 1e-38 beside them stands for results below
float32's normal numbers, which lose bits."""
import numpy as np
import pytest
import torch

from oracle import rope as ora
from tests.test_gpu_rope import U, bpa, f64, freqs, half, inputs, pair_sum  # noqa: F401

pytestmark = pytest.mark.gpu
SHAPES = [(128, 64, False), (80, 80, True), (72, 36, False), (511, 510, True)]     # two of 16-byte units, two of single elements


def check(x, dy, w, eps, rot, inter, out, dx, dw):
    """One side's results; x [1, S, H, d]."""
    angle = ora.angles(np.arange(x.shape[1])[None], freqs(rot).numpy())
    w64 = None if w is None else f64(w)
    want = ora.forward(f64(x), angle, w64, eps, inter)
    flat = ora.forward(f64(x), np.zeros_like(angle), w64, eps, inter)
    err, tol = np.abs(f64(out) - want), 24 * U * pair_sum(flat, rot, inter) + half(x.dtype) * np.abs(want) + 1e-38
    assert (err <= tol).all(), (float((err / tol).max()), np.argwhere(err > tol)[:3])
    want, want_w, _ = ora.backward(f64(x), f64(dy), angle, w64, eps, inter)
    r = 1 / np.sqrt((f64(x) ** 2).mean(-1, keepdims=True) + eps)
    ps, xh = pair_sum(f64(dy), rot, inter), np.abs(f64(x)) * r
    e = ps * (1.0 if w is None else np.abs(w64))
    err, tol = np.abs(f64(dx) - want), 96 * U * r * (e + xh * (e * xh).mean(-1, keepdims=True)) + half(x.dtype) * np.abs(want) + 1e-38
    assert (err <= tol).all(), (float((err / tol).max()), np.argwhere(err > tol)[:3])
    err, tol = np.abs(f64(dw) - want_w), (48 + 77) * U * (ps * xh).sum((0, 1, 2)) + U * np.abs(want_w) + 1e-38
    assert (err <= tol).all(), float((err / tol).max())


def both(bpa, x, dy, w, eps, rot, inter):  # noqa: F811
    kw = dict(eps=eps, interleaved=inter)
    dev = None if w is None else w.cuda()
    out, _ = bpa.bpa_rope_fwd(x.cuda(), None, None, freqs(rot).cuda(), dev, **kw)
    dx, _, dw, _ = bpa.bpa_rope_bwd(x.cuda(), None, dy.cuda(), None, None, freqs(rot).cuda(), dev, **kw)
    torch.cuda.synchronize()
    check(x, dy, w, float(np.float32(eps)), rot, inter, out, dx, dw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("eps", [1.1754944e-38, 1e-30, 1e-12, 1.0, 1e12, 1e30, 3.4e38])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_eps_of_any_size(bpa, shape, eps, dtype):  # noqa: F811
    """Heads far below and far above eps, in one warp: 1 / sqrt(mean + eps) is the larger one's."""
    d, rot, inter = shape
    x, dy = inputs(1, 1, 5, 9, d, dtype), inputs(2, 1, 5, 9, d, dtype)
    for h, f in enumerate((1.0, 1e-20, 0.0, 1e18, 1e-6, 1e6, 1e30, 1e-30, 1e15)):
        x[:, :, h] = (x[:, :, h].double() * f).to(dtype)
    both(bpa, x, dy, None, eps, rot, inter)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("value,weight", [(45, 90), (49, -100), (-49, 100), (-45, -90), (10, 110), (60, 95), (-60, -60), (0, 118)])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_weights_of_any_size(bpa, shape, value, weight, dtype):  # noqa: F811
    """Powers of two on the values and on the weights: the norm takes the first away, whatever their product is."""
    d, rot, inter = shape
    x, dy = inputs(1, 1, 5, 3, d, dtype), inputs(2, 1, 5, 3, d, dtype)
    x = (x.double() * 2.0 ** value).to(dtype)
    w = ((1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(3)).double()) * 2.0 ** weight).float()
    dy = (dy.double() * 2.0 ** -(weight // 2)).to(dtype)               # a gradient that leaves room for dx and dw
    both(bpa, x, dy, w, 1e-30, rot, inter)
