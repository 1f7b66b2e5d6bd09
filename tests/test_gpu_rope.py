"""Norm and rotation of q and k on the GPU against the 64-bit oracle.

Tolerances.  u = 2^-24, half a float32 step.  A head's 1 / sqrt(mean x^2 + eps): a lane adds at most 16 squares and
the lanes in 5 more steps, so the sum is off by at most 21 u and its root's inverse by half of that and
two steps, below 15 u; two more products (r x, w) and the rotation's (one rounding of each product and of the
sum) make 18 u of |a| + |b|, a and b the pair's values behind the norm.  The angle reaches sincospif as a
float32 of at most 1/4 (pi/4 u of a radian), whose sine and cosine are within two steps (4 u): 5 u more.
24 u (|a| + |b|) covers it; then the rounding to the result's type, eps / 2 of the value (bf16 2^-8).
Backward: e = w g and xh carry up to 24 u of their pairs' magnitudes each, their mean's product 21 u of
mean |e xh| beside that, and r 15 u: 96 u r (|e|_pair + |xh| mean |e|_pair |xh|) covers the products of them.  dw: each
term is off by up to 48 u of its magnitudes, and adding n terms in float32 by n u of them, n <= 64 + 13 here."""
import numpy as np
import pytest
import torch

from oracle import rope as ora

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def bpa():
    from ring_attention_gb300 import build
    build.build()
    from ring_attention_gb300 import bpa as mod
    return mod


def f64(t):
    return t.detach().double().cpu().numpy()


def pair_sum(x, rot, inter):
    """|a| + |b| of the pair that each channel belongs to, itself past the rotated ones."""
    x, n = np.abs(np.array(x, np.float64)), rot // 2
    y = x.copy()
    if inter:
        s = x[..., 0:rot:2] + x[..., 1:rot:2]
        y[..., 0:rot:2] = y[..., 1:rot:2] = s
    else:
        s = x[..., :n] + x[..., n:rot]
        y[..., :n] = y[..., n:rot] = s
    return y


def half(dtype):
    return torch.finfo(dtype).eps / 2


def inputs(seed, B, S, H, d, dtype, std=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, S, H, d, generator=g) * torch.exp2(torch.randn(1, 1, H, 1, generator=g)) * std
    return x.to(dtype)


def freqs(rot, theta=10000.0):
    return torch.tensor([theta ** (-i / max(rot // 2, 1)) for i in range(rot // 2)], dtype=torch.float32)


def check_forward(x, got, angle, w, eps, inter, there, before):
    rot = 2 * angle.shape[-1]
    want = ora.forward(f64(x), angle, None if w is None else f64(w), eps, inter)
    flat = ora.forward(f64(x), np.zeros_like(angle), None if w is None else f64(w), eps, inter)
    tol = 24 * U * pair_sum(flat, rot, inter) + half(x.dtype) * np.abs(want) + 1e-38
    err = np.abs(f64(got) - want)
    assert (err <= tol)[there].all(), float((err / tol)[there].max())
    assert np.array_equal(f64(got)[~there], before[~there])


def check_backward(x, dy, got, gw, angle, w, eps, inter, there):
    rot, w64 = 2 * angle.shape[-1], None if w is None else f64(w)
    g = np.where(there[:, :, None, None], f64(dy), 0.0)
    dx, dw, mag = ora.backward(f64(x), g, angle, w64, eps, inter)
    ps = pair_sum(g, rot, inter)
    if eps is None:
        tol = 24 * U * ps
    else:
        r = 1 / np.sqrt((f64(x) ** 2).mean(-1, keepdims=True) + eps)
        xh, e = np.abs(f64(x)) * r, ps * (1.0 if w is None else np.abs(w64))
        tol = 96 * U * r * (e + xh * (e * xh).mean(-1, keepdims=True))
        most = (48 + 77) * U * (ps * xh).sum((0, 1, 2)) + half(torch.float32) * np.abs(dw)
        err = np.abs(f64(gw) - dw)
        assert (err <= most + 1e-38).all(), float((err / (most + 1e-38)).max())
    tol = tol + half(x.dtype) * np.abs(dx) + 1e-38
    err = np.abs(f64(got) - dx)
    assert (err <= tol).all(), float((err / tol).max())


SHAPES = [  # B, S, Hq, Hkv, d, rot, interleaved, positions
    (1, 1, 1, 1, 1, 0, False, "none"), (1, 1, 1, 1, 2, 2, True, "far"), (2, 3, 2, 1, 33, 32, False, "none"),
    (1, 5, 3, 1, 24, 12, False, "skip"), (1, 7, 4, 2, 24, 12, True, "skip"), (2, 9, 4, 2, 64, 64, False, "none"),
    (1, 17, 6, 3, 72, 36, True, "far"), (3, 11, 4, 2, 80, 80, False, "skip"), (3, 11, 4, 2, 80, 32, True, "none"),
    (1, 67, 32, 8, 128, 128, False, "skip"), (1, 19, 8, 1, 128, 128, True, "far"), (2, 33, 5, 5, 96, 48, False, "far"),
    (1, 3, 2, 2, 192, 64, False, "none"), (1, 5, 2, 1, 256, 256, True, "skip"), (1, 6, 3, 1, 512, 512, False, "far"),
    (1, 6, 3, 1, 512, 64, True, "none"), (1, 4, 3, 2, 511, 510, False, "none"), (1, 300, 0, 3, 64, 32, False, "far"),
    (1, 300, 3, 0, 64, 16, True, "skip"), (1, 3, 70, 1, 16, 16, False, "none"),
]


def positions(kind, B, S, seed):
    if kind == "none":
        return None
    g = torch.Generator().manual_seed(seed)
    pos = torch.randint(0, 2 ** 31 - 1 if kind == "far" else 5000, (B, S), generator=g).to(torch.int32)
    if kind == "skip":
        pos[:, 1::3] = -1
        pos[:, -1] = -7
    return pos


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_forward_and_backward(bpa, shape, dtype, norm):
    B, S, Hq, Hkv, d, rot, inter, kind = shape
    eps = 1e-5 if norm else None
    pos, freq = positions(kind, B, S, 3), freqs(rot)
    angle = ora.angles(np.maximum(pos.numpy() if pos is not None else np.tile(np.arange(S), (B, 1)), 0), freq.numpy())
    there = np.ones((B, S), bool) if pos is None else pos.numpy() >= 0
    q, k = inputs(1, B, S, Hq, d, dtype), inputs(2, B, S, Hkv, d, dtype)
    dq, dk = inputs(4, B, S, Hq, d, dtype, 0.1), inputs(5, B, S, Hkv, d, dtype, 0.1)
    wq, wk = (1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(i)) for i in (6, 7))
    wq, wk = (wq if norm and Hq else None), (wk if norm and Hkv else None)
    dev = lambda t: None if t is None else t.cuda()                                               # noqa: E731
    some = lambda t: t.cuda() if t.shape[2] else None                                             # noqa: E731
    q_out, k_out = (torch.full(t.shape, 3.0, dtype=dtype, device="cuda") if t.shape[2] else None for t in (q, k))
    kw = dict(norm=norm, eps=1e-5, interleaved=inter)
    args = (dev(pos), dev(freq) if rot else None, dev(wq), dev(wk))
    out = bpa.bpa_rope_fwd(some(q), some(k), *args, q_out=q_out, k_out=k_out, **kw)
    got = bpa.bpa_rope_bwd(some(q), some(k), some(dq), some(dk), *args, **kw)
    torch.cuda.synchronize()
    for i, (x, dy, w) in enumerate(((q, dq, wq), (k, dk, wk))):
        if x.shape[2] == 0:
            assert out[i] is None and got[i] is None and got[2 + i] is None
            continue
        check_forward(x, out[i], angle, w, eps, inter, there, np.full(x.shape, 3.0))
        check_backward(x, dy, got[i], got[2 + i], angle, w, eps, inter, there)


@pytest.mark.parametrize("offset", [0, 1, 4])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_parts_of_one_buffer_packed_rows_and_alignment(bpa, dtype, offset):
    T, Hq, Hkv, d = 45, 4, 2, 64
    width = (Hq + 2 * Hkv) * d + (8 if offset else 0)
    raw = inputs(8, 1, T, 1, width, dtype)[0, :, 0]
    buf = raw.cuda().flatten()
    buf = torch.cat([buf, buf.new_zeros(16)])[offset:]

    def view(b, h0, h1):
        return b.as_strided((T, h1 - h0, d), (width, d, 1), b.storage_offset() + h0 * d)

    q, k = view(buf, 0, Hq), view(buf, Hq, Hq + Hkv)
    pos, freq = positions("skip", 1, T, 9)[0], freqs(64)
    angle, there = ora.angles(np.maximum(pos.numpy(), 0)[None], freq.numpy()), pos.numpy()[None] >= 0
    a, b = bpa.bpa_rope_fwd(q, k, pos.cuda(), freq.cuda(), eps=1e-5, q_out=torch.zeros(T, Hq, d, dtype=dtype, device="cuda"),
                            k_out=torch.zeros(T, Hkv, d, dtype=dtype, device="cuda"))
    for x, y in ((q, a), (k, b)):
        check_forward(x[None], y[None], angle, None, 1e-5, False, there, np.zeros((1,) + y.shape))
    # gradients into parts of one buffer: what lies between them stays
    grad = torch.full_like(buf, 7.0)
    dq, dk = view(grad, 0, Hq), view(grad, Hq, Hq + Hkv)
    dy = inputs(10, 1, T, Hq + Hkv, d, dtype)[0].cuda()
    got = bpa.bpa_rope_bwd(q, k, dy[:, :Hq], dy[:, Hq:], pos.cuda(), freq.cuda(), eps=1e-5, dq=dq, dk=dk)
    for x, g, o, w in ((q, dy[:, :Hq], got[0], got[2]), (k, dy[:, Hq:], got[1], got[3])):
        check_backward(x[None], g[None], o[None], w, angle, None, 1e-5, False, there)
    rest = grad.as_strided((T, width - (Hq + Hkv) * d), (width, 1), grad.storage_offset() + (Hq + Hkv) * d)
    assert (rest == 7).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,rot,inter", [(128, 64, False), (80, 40, True), (128, 128, False)])
def test_in_place(bpa, dtype, d, rot, inter):
    q, k = inputs(1, 2, 13, 4, d, dtype).cuda(), inputs(2, 2, 13, 2, d, dtype).cuda()
    dq, dk = inputs(3, 2, 13, 4, d, dtype).cuda(), inputs(4, 2, 13, 2, d, dtype).cuda()
    freq = freqs(rot).cuda()
    want = bpa.bpa_rope_fwd(q, k, None, freq, interleaved=inter)
    grads = bpa.bpa_rope_bwd(q, k, dq, dk, None, freq, interleaved=inter)
    over = [t.clone() for t in (dq, dk)]
    again = bpa.bpa_rope_bwd(q, k, *over, None, freq, interleaved=inter, dq=over[0], dk=over[1])
    assert again[0] is over[0] and all(torch.equal(x, y) for x, y in zip(grads, again))
    over = [t.clone() for t in (q, k)]
    again = bpa.bpa_rope_bwd(*over, dq, dk, None, freq, interleaved=inter, dq=over[0], dk=over[1])
    assert all(torch.equal(x, y) for x, y in zip(grads, again))
    over = [t.clone() for t in (q, k)]
    got = bpa.bpa_rope_fwd(*over, None, freq, interleaved=inter, q_out=over[0], k_out=over[1])
    assert got[0] is over[0] and all(torch.equal(x, y) for x, y in zip(want, got))


def test_values_at_the_ends_of_the_range(bpa):
    """Heads whose squares leave float32's range, of zeros, and with values that are not finite."""
    d, eps = 128, 1e-30
    x = inputs(1, 1, 8, 6, d, torch.float32)
    for h, f in enumerate((1e30, 1e-25, 0.0, 1.0, 3e38 / 8, 1e-37)):
        x[:, :, h] *= f / x[:, :, h].abs().amax() * 8 if h == 4 else f
    x[0, 3, 3, 17] = float("inf")
    x[0, 5, 3, 70] = float("nan")
    dy, freq = inputs(2, 1, 8, 6, d, torch.float32), freqs(64)
    angle = ora.angles(np.arange(8)[None], freq.numpy())
    out, _ = bpa.bpa_rope_fwd(x.cuda(), None, None, freq.cuda(), eps=eps)
    dx, _, dw, _ = bpa.bpa_rope_bwd(x.cuda(), None, dy.cuda(), None, None, freq.cuda(), eps=eps)
    clean = x.clone()
    clean[0, [3, 5], 3] = 1.0
    want = ora.forward(f64(clean), angle, None, eps)
    flat = ora.forward(f64(clean), np.zeros_like(angle), None, eps)
    ok = np.ones(x.shape[:3], bool)
    ok[0, [3, 5], 3] = False
    err, tol = np.abs(f64(out) - want), 24 * U * pair_sum(flat, 64, False) + U * np.abs(want) + 1e-38
    assert (err <= tol)[ok].all()
    # infinity: the others of its head become 0, it and its pair are lost (channels 17 and 49); NaN: the head is
    h3 = f64(out)[0, 3, 3]
    assert np.isnan(h3[[17, 49]]).all() and (np.delete(h3, [17, 49]) == 0).all() and np.isnan(f64(out)[0, 5, 3]).all()
    want, _, _ = ora.backward(f64(clean), f64(dy), angle, None, eps)
    r = 1 / np.sqrt((f64(clean) ** 2).mean(-1, keepdims=True) + eps)
    e, xh = pair_sum(f64(dy), 64, False), np.abs(f64(clean)) * r
    tol = 96 * U * r * (e + xh * (e * xh).mean(-1, keepdims=True)) + U * np.abs(want) + 1e-38
    assert (np.abs(f64(dx) - want) <= tol)[ok].all()
    assert np.isnan(f64(dw)).any()


def test_gradient_against_differences(bpa):
    """The kernel's gradient beside central differences of the 64-bit forward pass."""
    q, dy = inputs(1, 1, 6, 2, 64, torch.bfloat16), inputs(2, 1, 6, 2, 64, torch.bfloat16)
    w, freq = 1 + 0.2 * torch.randn(64, generator=torch.Generator().manual_seed(3)), freqs(64)
    angle = ora.angles(np.arange(6)[None], freq.numpy())
    dx, _, dw, _ = bpa.bpa_rope_bwd(q.cuda(), None, dy.cuda(), None, None, freq.cuda(), w.cuda(), eps=1e-3)
    f = lambda x, w: (ora.forward(x, angle, w, 1e-3) * f64(dy)).sum()                             # noqa: E731
    x, w64, h = f64(q), f64(w), 1e-6
    for at in [(0, 0, 0, 0), (0, 5, 1, 63), (0, 2, 0, 31), (0, 3, 1, 32)]:
        e = np.zeros_like(x)
        e[at] = h
        diff = (f(x + e, w64) - f(x - e, w64)) / (2 * h)
        assert abs(diff - f64(dx)[at]) <= 2.0 ** -8 * abs(diff) + 1e-5
    for c in (0, 33):
        e = np.zeros(64)
        e[c] = h
        assert abs((f(x, w64 + e) - f(x, w64 - e)) / (2 * h) - f64(dw)[c]) <= 1e-4


def test_heads_that_share_memory_and_repeated_calls(bpa):
    """An expanded input (stride 0) is read like any other; a call repeats itself bit for bit."""
    base = inputs(1, 1, 40, 1, 128, torch.bfloat16).cuda()
    q, freq = base.expand(1, 40, 8, 128), freqs(128).cuda()
    a, _ = bpa.bpa_rope_fwd(q, None, None, freq)
    b, _ = bpa.bpa_rope_fwd(q.contiguous(), None, None, freq)
    assert torch.equal(a, b)
    dy = inputs(2, 3, 700, 12, 128, torch.bfloat16).cuda()
    x = inputs(3, 3, 700, 12, 128, torch.bfloat16).cuda()
    first = bpa.bpa_rope_bwd(x, None, dy, None, None, freq)
    for _ in range(3):
        again = bpa.bpa_rope_bwd(x, None, dy, None, None, freq)
        assert torch.equal(first[0], again[0]) and torch.equal(first[2], again[2])


def test_captured_with_other_positions_and_streams(bpa):
    T, freq = 24, freqs(64).cuda()
    q, k = inputs(1, 1, T, 4, 64, torch.bfloat16)[0].cuda(), inputs(2, 1, T, 2, 64, torch.bfloat16)[0].cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    outs = [torch.zeros_like(q), torch.zeros_like(k)]
    grads = [torch.zeros_like(q), torch.zeros_like(k)]
    ws = torch.empty(bpa.bpa_rope_workspace_size(bpa.make_rope_desc(q, k, pos, freq)), dtype=torch.uint8, device="cuda")
    bpa.bpa_rope_fwd(q, k, pos, freq, q_out=outs[0], k_out=outs[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bpa.bpa_rope_fwd(q, k, pos, freq, q_out=outs[0], k_out=outs[1])
        _, _, dwq, dwk = bpa.bpa_rope_bwd(q, k, outs[0], outs[1], pos, freq, dq=grads[0], dk=grads[1], workspace_buf=ws)
    other = torch.cuda.Stream()
    for shift in (0, 1000, 123456789):
        pos.copy_(torch.arange(T, dtype=torch.int32) * 3 + shift)
        q.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        bpa.bpa_check(ws)
        with torch.cuda.stream(other):
            want = bpa.bpa_rope_fwd(q, k, pos, freq)
            back = bpa.bpa_rope_bwd(q, k, *want, pos, freq)
        same = bpa.bpa_rope_fwd(q, k, pos, freq, stream=other)
        torch.cuda.synchronize()
        for x, y, z in zip(outs, want, same):
            assert torch.equal(x, y) and torch.equal(x, z)
        for x, y in zip(grads + [dwq, dwk], back):
            assert torch.equal(x, y)


def test_no_rows(bpa):
    q, k, freq = torch.zeros(0, 4, 64, device="cuda"), torch.zeros(0, 2, 64, device="cuda"), freqs(64).cuda()
    a, b = bpa.bpa_rope_fwd(q, k, None, freq)
    assert a.shape == q.shape and b.shape == k.shape
    dq, dk, wq, wk = bpa.bpa_rope_bwd(q, k, a, b, None, freq)
    assert dq.shape == q.shape and (wq == 0).all() and (wk == 0).all()


def torch64(x, w, freq, eps, inter):
    """The forward pass in 64 bits on the GPU, positions 0, 1, .., for sizes that the oracle is slow at."""
    x = x.double()
    x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    t = torch.arange(x.shape[1], device="cuda").double()[:, None] * freq.double()
    c, s, n = t.cos()[:, None], t.sin()[:, None], freq.numel()
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if inter else (x[..., :n], x[..., n:2 * n])
    u, v = a * c - b * s, b * c + a * s
    return torch.cat([torch.stack([u, v], -1).flatten(-2) if inter else torch.cat([u, v], -1), x[..., 2 * n:]], -1)


@pytest.mark.parametrize("dtype,d,rot,inter", [(torch.bfloat16, 128, 128, False), (torch.bfloat16, 64, 32, True), (torch.bfloat16, 256, 64, False),
                                               (torch.float32, 80, 80, False), (torch.bfloat16, 72, 36, False)])
def test_many_rows_and_heads(bpa, dtype, d, rot, inter):
    """Rows and heads enough for chunks of several rounds and several items a warp; ragged ends of both."""
    q, k = inputs(1, 2, 2501, 37, d, dtype).cuda(), inputs(2, 2, 2501, 5, d, dtype).cuda()
    w, freq = (1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(6))).cuda(), freqs(rot).cuda()
    out = bpa.bpa_rope_fwd(q, k, None, freq, w, w, eps=1e-5, interleaved=inter)
    for x, got in zip((q, k), out):
        want = torch64(x, w, freq, 1e-5, inter)
        flat = torch64(x, w, freq * 0, 1e-5, inter).abs()
        n = rot // 2
        pair = flat.clone()
        if inter:
            pair[..., 0:rot:2] = pair[..., 1:rot:2] = flat[..., 0:rot:2] + flat[..., 1:rot:2]
        else:
            pair[..., :n] = pair[..., n:rot] = flat[..., :n] + flat[..., n:rot]
        assert ((got.double() - want).abs() <= 24 * U * pair + half(dtype) * want.abs() + 1e-38).all()
    dy = inputs(3, 2, 2501, 37, d, dtype, 0.1).cuda()
    x64, w64 = q.double().requires_grad_(), w.double().requires_grad_()
    want, want_w = torch.autograd.grad(torch64(x64, w64, freq, 1e-5, inter), [x64, w64], dy.double())
    dx, _, dw, _ = bpa.bpa_rope_bwd(q, None, dy, None, None, freq, w, eps=1e-5, interleaved=inter)
    r = 1 / (q.double().pow(2).mean(-1, keepdim=True) + 1e-5).sqrt()
    e, xh = dy.double().abs().amax(-1, keepdim=True) * 2 * w.double().abs(), q.double().abs() * r
    tol = 96 * U * r * (e + xh * (e * xh).mean(-1, keepdim=True)) + half(dtype) * want.abs() + 1e-38
    assert ((dx.double() - want).abs() <= tol).all()
    # a sum of n terms in float32, at most 1,024 of them one after the other in a lane, then 4 + 5 + 7 levels
    most = (48 + 1024 + 16) * U * (e * xh).sum((0, 1, 2)) + U * want_w.abs()
    assert ((dw.double() - want_w).abs() <= most).all()
