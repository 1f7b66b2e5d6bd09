"""Norm and rotation of q and k without a GPU: the descriptor's layout, the library's and the binding's
refusals, and pins of the 64-bit oracle that the GPU tests compare with."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from oracle import rope as ora

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def bpa():
    from ring_attention_gb300 import build
    build.build()
    from ring_attention_gb300 import bpa as mod
    return mod


def test_descriptor_layout_matches_c(tmp_path, bpa):
    cls = bpa.bpa_rope_desc
    fields = [f[0] for f in cls._fields_]
    body = "\n".join(f'printf("{f} %zu\\n", offsetof(bpa_rope_desc, {f}));' for f in fields)
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "bpa.h"\nint main(void){\n'
                   f'printf("size %zu\\n", sizeof(bpa_rope_desc));\n{body}\nreturn 0;}}\n')
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    got = dict(x.split() for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    assert int(got["size"]) == ctypes.sizeof(cls)
    for f in fields:
        assert int(got[f]) == getattr(cls, f).offset, f


def _desc(bpa, **over):
    D = bpa.bpa_rope_desc()
    D.struct_size, D.dtype = ctypes.sizeof(D), bpa.BPA_BF16
    D.B, D.S, D.Hq, D.Hkv, D.d, D.rot, D.norm, D.eps = 2, 5, 4, 2, 64, 32, 1, 1e-6
    D.q = D.k = D.inv_freq = 0x10000                 # never dereferenced by host checks
    for n in ("q_strides", "k_strides", "qo_strides", "ko_strides"):
        getattr(D, n)[:] = (5 * 4 * 64, 4 * 64, 64)
    for k, v in over.items():
        if isinstance(v, tuple):
            getattr(D, k)[:] = v
        else:
            setattr(D, k, v)
    return D


BAD = [(dict(struct_size=8), 1), (dict(dtype=7), 1), (dict(reserved=1), 1), (dict(B=0), 1), (dict(S=-1), 1),
       (dict(B=1 << 16, S=1 << 16), 1), (dict(Hq=-1), 1), (dict(Hq=0, Hkv=0), 1), (dict(Hkv=65536), 2), (dict(d=0), 1),
       (dict(d=513), 2), (dict(rot=-2), 1), (dict(rot=33), 1), (dict(rot=66), 1), (dict(eps=0.0), 1), (dict(eps=-1.0), 1),
       (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(eps=1e-40), 1), (dict(norm=0, q_weight=0x10000), 1),
       (dict(norm=0, k_weight=0x10000), 1), (dict(inv_freq=0), 1), (dict(q=0), 1), (dict(k=0), 1),
       (dict(q_strides=(-1, 256, 64)), 1), (dict(ko_strides=(1280, 256, -64)), 1)]


@pytest.mark.parametrize("over,status", BAD)
def test_both_directions_refuse(bpa, over, status):
    L, p = bpa.lib(), 0x40000
    D = ctypes.byref(_desc(bpa, **over))
    assert L.bpa_rope_fwd(D, p, p, None) == status, L.bpa_last_error()
    assert L.bpa_last_error() != b""
    assert L.bpa_rope_bwd(D, p, p, p, p, None, None, p, 1 << 40, None) == status


def test_outputs_over_one_another_and_null(bpa):
    L, p = bpa.lib(), 0x40000
    fwd = lambda D, q=p, k=p: L.bpa_rope_fwd(ctypes.byref(D), q, k, None)                          # noqa: E731
    bwd = lambda D, a=p, b=p, c=p, d=p, wq=None, ws=p, n=1 << 40: L.bpa_rope_bwd(                  # noqa: E731
        ctypes.byref(D), a, b, c, d, wq, None, ws, n, None)
    for st in ((0, 256, 64), (1280, 0, 64), (1280, 256, 0)):
        assert fwd(_desc(bpa, qo_strides=st)) == 1 and fwd(_desc(bpa, ko_strides=st)) == 1
        assert bwd(_desc(bpa, q_strides=st)) == 1 and bwd(_desc(bpa, k_strides=st)) == 1
    assert fwd(_desc(bpa), q=None) == 1 and fwd(_desc(bpa), k=None) == 1
    for name in "abcd":
        assert bwd(_desc(bpa), **{name: None}) == 1
    assert bwd(_desc(bpa, norm=0), wq=p) == 1
    D = _desc(bpa)
    need = L.bpa_rope_workspace_size(ctypes.byref(D))
    assert need >= 256 and need % 256 == 0
    assert bwd(D, ws=None) == 3 and bwd(D, ws=p + 16) == 3 and bwd(D, n=need - 1) == 3
    assert L.bpa_rope_workspace_size(ctypes.byref(_desc(bpa, d=0))) == 0


def test_no_rows_forward_is_a_call_without_work(bpa):
    L = bpa.lib()
    assert L.bpa_rope_fwd(ctypes.byref(_desc(bpa, S=0, q=0, k=0)), None, None, None) == 0


def _tensors(**kw):
    t = dict(q=torch.zeros(2, 5, 4, 64), k=torch.zeros(2, 5, 2, 64), positions=torch.zeros(2, 5, dtype=torch.int32),
             inv_freq=torch.zeros(16), q_weight=torch.ones(64), k_weight=torch.ones(64))
    t.update(kw)
    return t


@pytest.mark.parametrize("bad", [
    dict(k=torch.zeros(2, 4, 2, 64)), dict(k=torch.zeros(2, 5, 2, 32)), dict(k=torch.zeros(2, 5, 2, 64, dtype=torch.bfloat16)),
    dict(q=torch.zeros(5, 64), k=torch.zeros(5, 64)), dict(q=torch.zeros(2, 5, 64, 4).transpose(2, 3)),
    dict(positions=torch.zeros(2, 5)), dict(positions=torch.zeros(10, dtype=torch.int32)),
    dict(positions=torch.zeros(5, 2, dtype=torch.int32).T), dict(inv_freq=torch.zeros(16, dtype=torch.float64)),
    dict(inv_freq=torch.zeros(32)[::2]), dict(q_weight=torch.ones(32)), dict(k_weight=torch.ones(64, dtype=torch.bfloat16)),
    dict(q=None), dict(q=torch.zeros(2, 5, 4, 64, dtype=torch.float16), k=torch.zeros(2, 5, 2, 64, dtype=torch.float16)),
])
def test_binding_refuses(bpa, bad):
    with pytest.raises((ValueError, TypeError)):
        bpa.make_rope_desc(**_tensors(**bad))


def test_binding_fills_the_descriptor(bpa):
    buf = torch.zeros(7, 8, 64)
    D = bpa.make_rope_desc(buf[:, :4], buf[:, 4:6], None, torch.zeros(16), interleaved=True, eps=1e-5)
    assert (D.B, D.S, D.Hq, D.Hkv, D.d, D.rot, D.interleaved, D.norm) == (1, 7, 4, 2, 64, 32, 1, 1)
    assert list(D.q_strides) == list(D.k_strides) == [0, 512, 64] and D.k == buf.data_ptr() + 4 * 4 * 64
    assert list(D.qo_strides) == list(D.q_strides) and not D.positions and not D.q_weight
    alone = bpa.make_rope_desc(None, buf[:, 4:6], norm=False)
    assert (alone.Hq, alone.Hkv, alone.rot, alone.norm) == (0, 2, 0, 0)


def test_calls_refuse_tensors_of_the_cpu(bpa):
    t = _tensors()
    with pytest.raises(ValueError):
        bpa.bpa_rope_fwd(**t)
    with pytest.raises(ValueError):
        bpa.bpa_rope_bwd(t["q"], t["k"], t["q"], t["k"])
    with pytest.raises(ValueError):
        bpa.bpa_rope_fwd(None, None)
    with pytest.raises(ValueError):
        bpa.bpa_rope_fwd(t["q"], None, k_out=t["k"])
    with pytest.raises(ValueError):
        bpa.bpa_rope_bwd(t["q"], t["k"], t["q"], None)
    with pytest.raises(ValueError):
        bpa.bpa_rope_bwd(t["q"], None, t["q"], None, dq=torch.zeros(2, 5, 8, 64)[:, :, ::2])


# ---- the oracle -----------------------------------------------------------------------------------
def test_two_pi_and_angles():
    assert abs(ora.two_pi() / 2 ** ora.BITS - 2 * np.pi) < 1e-15
    got = ora.angles(np.array([0, 1, 7, 100000]), np.array([1.0, 0.25], np.float32))
    assert np.abs(np.cos(got) - np.cos(np.outer([0, 1, 7, 100000], [1.0, 0.25]))).max() < 1e-10


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_rotation_of_the_difference(interleaved):
    g = np.random.default_rng(1)
    freq = (10000.0 ** (-np.arange(4) / 4)).astype(np.float32)
    x, y = g.standard_normal((2, 1, 1, 1, 10))
    turn = lambda v, p: ora.rotate(v, ora.angles(np.array([[p]]), freq), interleaved)              # noqa: E731
    assert np.allclose((turn(x, 1234) ** 2).sum(), (x ** 2).sum())
    assert np.allclose((turn(x, 903) * turn(y, 900)).sum(), (turn(x, 3) * turn(y, 0)).sum(), atol=1e-9)
    assert np.array_equal(turn(x, 55)[..., 8:], x[..., 8:])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("eps", [None, 1e-3])
def test_gradients_against_differences(interleaved, eps):
    g = np.random.default_rng(2)
    x, dy = g.standard_normal((2, 2, 3, 2, 10))
    w = g.standard_normal(10) if eps is not None else None
    angle = ora.angles(np.arange(6).reshape(2, 3) * 5, np.array([1.0, 0.3, 0.01], np.float32))
    f = lambda x, w: (ora.forward(x, angle, w, eps, interleaved) * dy).sum()                       # noqa: E731
    dx, dw, _ = ora.backward(x, dy, angle, w, eps, interleaved)
    h = 1e-6
    for at in [(0, 0, 0, 0), (1, 2, 1, 4), (0, 1, 1, 9), (1, 0, 0, 3)]:
        e = np.zeros_like(x)
        e[at] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[at]) < 1e-7
    if eps is not None:
        for c in (0, 5, 9):
            e = np.zeros(10)
            e[c] = h
            assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[c]) < 1e-7
