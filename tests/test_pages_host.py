"""Trees, kept paths and shared pages without a GPU: the library's and the binding's refusals (each call here
fails its checks before anything touches a device) and pins of the 64-bit oracle."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import cache as ora
from tests.test_cache_host import _batch, _cache, _Fake, _Stream, streams  # noqa: F401


@pytest.fixture(scope="module")
def bpa():
    from ring_attention_gb300 import build
    build.build()
    from ring_attention_gb300 import bpa as mod
    return mod


P = 0x40000           # never dereferenced by host checks


# ---- the library's refusals ---------------------------------------------------------------------------
def test_attention_refuses_trees(bpa):
    L = bpa.lib()
    call = lambda **kw: L.bpa_cache_attn(ctypes.byref(_cache(bpa)), ctypes.byref(_batch(bpa, **kw)), P, P, P, P, 1 << 40, None)  # noqa: E731
    for bad in (dict(tree=P, tree_words=0), dict(tree=P, tree_words=33), dict(tree=P, tree_words=-1), dict(tree=P, tree_words=1, causal=0),
                dict(reserved=1)):
        assert call(**bad) == 1, bad
        assert L.bpa_cache_attn_workspace_size(ctypes.byref(_cache(bpa)), ctypes.byref(_batch(bpa, **bad))) == 0


def test_batches_of_before_the_tree_are_taken(bpa):
    L, B = bpa.lib(), bpa.bpa_cache_batch
    old = _batch(bpa, struct_size=B.tree.offset, tree=P, tree_words=99, reserved=5)      # not its fields
    new = _batch(bpa)
    size = lambda b: L.bpa_cache_attn_workspace_size(ctypes.byref(_cache(bpa)), ctypes.byref(b))      # noqa: E731
    assert size(old) == size(new) > 0
    assert size(_batch(bpa, struct_size=B.tree.offset + 4)) == 0


def test_tree_refuses(bpa):
    L = bpa.lib()
    base = dict(R=3, T=5, words=1, parents=P, kv=P, cu=P, tree=P, pos=P, ws=P, n=256)
    call = lambda **kw: L.bpa_cache_tree(*{**base, **kw}.values(), None)                              # noqa: E731
    for bad in (dict(R=0), dict(T=-1), dict(T=(1 << 30) + 1), dict(words=0), dict(words=33), dict(parents=None), dict(kv=None), dict(cu=None),
                dict(tree=None)):
        assert call(**bad) == 1, bad
    assert call(ws=None) == 3 and call(ws=P + 8) == 3 and call(n=255) == 3


def test_keep_refuses(bpa):
    L = bpa.lib()
    base = dict(R=3, T=5, max_pages=4, keep=P, max_keep=2, count=P, kv=P, cu=P, table=P, ws=P, n=256)

    def call(c=None, **kw):
        return L.bpa_cache_keep(ctypes.byref(c if c is not None else _cache(bpa)), *{**base, **kw}.values(), None)

    for bad in (dict(R=0), dict(T=-1), dict(max_keep=-1), dict(max_pages=0), dict(max_pages=1 << 27), dict(keep=None), dict(count=None),
                dict(kv=None), dict(cu=None), dict(table=None), dict(T=(1 << 30) + 1)):
        assert call(**bad) == 1, bad
    assert call(R=1 << 30) == 2 and call(ws=None) == 3 and call(n=255) == 3
    assert call(_cache(bpa, v_scale=0)) == 1 and call(_cache(bpa, page_size=0)) == 1
    flat = _cache(bpa)
    flat.v_cache_strides[2] = 0
    assert call(flat) == 1


def test_fork_and_release_refuse(bpa):
    L = bpa.lib()
    fork = dict(N=2, R=3, page=16, pages=9, width=4, src=P, dst=P, ctx=P, table=P, refs=P, free=P, count=P, a=P, b=P, out=P, left=P, ws=P, n=256)
    rel = dict(R=3, page=16, pages=9, width=4, ctx=P, keep=P, table=P, refs=P, free=P, count=P, out=P, left=P, ws=P, n=256)
    for f, base in ((L.bpa_cache_fork, fork), (L.bpa_cache_release, rel)):
        call = lambda **kw: f(*{**base, **kw}.values(), None)                                         # noqa: E731
        for bad in (dict(R=0), dict(page=0), dict(page=1025), dict(pages=0), dict(pages=1 << 27), dict(width=0), dict(width=1 << 27)):
            assert call(**bad) == 1, bad
        for name, v in base.items():
            if v == P and name != "ws":
                assert call(**{name: None}) == 1, name
        assert call(R=8193) == 2 and call(ws=None) == 3 and call(n=255) == 3 and call(ws=P + 4) == 3
    assert L.bpa_cache_fork(*{**fork, "N": -1}.values(), None) == 1 and L.bpa_cache_fork(*{**fork, "N": 8193}.values(), None) == 2


def test_copy_refuses(bpa):
    L = bpa.lib()
    call = lambda c=None, N=2, a=P, b=P, ws=P, n=256: L.bpa_cache_copy(                               # noqa: E731
        ctypes.byref(c if c is not None else _cache(bpa)), N, a, b, ws, n, None)
    assert call(N=-1) == 1 and call(a=None) == 1 and call(b=None) == 1 and call(N=1 << 29) == 2 and call(ws=None) == 3 and call(n=8) == 3
    assert call(_cache(bpa, k_cache=0)) == 1 and call(_cache(bpa, d=600)) == 2
    flat = _cache(bpa)
    flat.k_cache_strides[0] = 0
    assert call(flat) == 1


# ---- the binding ------------------------------------------------------------------------------------------
def _calls(bpa):
    i32 = lambda *s: _Fake(torch.zeros(*s, dtype=torch.int32))                                        # noqa: E731
    cache = dict(k_cache=_Fake(torch.zeros(9, 2, 16, 64, dtype=torch.uint8)), v_cache=_Fake(torch.zeros(9, 2, 16, 32, dtype=torch.uint8)),
                 k_scale=_Fake(torch.zeros(9, 2)), v_scale=_Fake(torch.zeros(9, 2)))
    args = {
        "tree": dict(parents=i32(5), kv_lens=i32(3), cu_q=i32(4), words=2),
        "keep": dict(keep=i32(3, 2), keep_count=i32(3), kv_lens=i32(3), cu_q=i32(4), page_table=i32(3, 4), **cache),
        "fork": dict(src=i32(2), dst=i32(2), ctx_lens=i32(3), page_table=i32(3, 4), page_refs=i32(9), free_pages=i32(9), free_count=i32(1),
                     page_size=16),
        "copy": dict(src=i32(2), dst=i32(2), **cache),
        "release": dict(ctx_lens=i32(3), keep_lens=i32(3), page_table=i32(3, 4), page_refs=i32(9), free_pages=i32(9), free_count=i32(1),
                        page_size=16),
    }
    return {n: (lambda f, a: lambda **kw: f(**{**a, **kw}))(getattr(bpa, "bpa_cache_" + n), a) for n, a in args.items()}, args


NAMES = ["tree", "keep", "fork", "copy", "release"]


@pytest.mark.parametrize("name", NAMES)
def test_streams_workspaces_and_devices(bpa, streams, name, monkeypatch):  # noqa: F811
    now, made, launched = streams
    call = _calls(bpa)[0][name]
    returned = call(stream=_Stream(0x20)) or ()
    assert launched == [("bpa_cache_" + name, 0x20)] and len(now) == 1
    assert made and all(t.made_on == 0x20 for t in made) and all(t.recorded == [0x10] for t in returned)
    made.clear()
    returned = call() or ()
    assert launched[-1][1] == 0x10 and all(t.made_on == 0x10 for t in made) and not any(t.recorded for t in made)
    for ptr in (0x10, 0x20):
        with pytest.raises(ValueError, match="stream"):
            call(stream=_Stream(ptr, 1))
    for bad in (torch.zeros(1024, dtype=torch.uint8), _Fake(torch.zeros(1, dtype=torch.uint8).expand(1024)),
                _Fake(torch.zeros(2048, dtype=torch.uint8)[::2]), _Fake(torch.zeros(1024, dtype=torch.int32))):
        with pytest.raises(ValueError, match="workspace"):
            call(workspace_buf=bad)
    assert len(launched) == 2

    def fails(*a, **kw):
        raise RuntimeError("out of memory")

    monkeypatch.setattr(bpa, "_empty", fails)
    with pytest.raises(RuntimeError):
        call(stream=_Stream(0x20))
    assert len(now) == 1 and len(launched) == 2


@pytest.mark.parametrize("name", NAMES)
def test_binding_refuses_shapes_and_types(bpa, streams, name):  # noqa: F811
    now, made, launched = streams
    calls, args = _calls(bpa)
    for key, t in args[name].items():
        if not isinstance(t, _Fake):
            continue
        longer = _Fake(torch.zeros(*(n + 1 for n in t.shape), dtype=t.dtype))
        for bad in (_Fake(t.t.to(torch.float64)), t.t, longer):
            if bad is longer and (name, key) in {("tree", "parents"), ("copy", "src")}:
                continue                      # they set the size
            with pytest.raises((ValueError, TypeError)):
                calls[name](**{key: bad})
    assert not launched


@pytest.mark.parametrize("name,kw", [("tree", dict(words=2 ** 31)), ("tree", dict(words=0)), ("tree", dict(words=33)),
                                     ("fork", dict(page_size=2 ** 32 + 16)), ("release", dict(page_size=2 ** 32 + 16))])
def test_binding_refuses_numbers(bpa, streams, name, kw):  # noqa: F811
    with pytest.raises(ValueError):
        _calls(bpa)[0][name](**kw)
    assert not streams[2]


@pytest.mark.parametrize("bad", [torch.zeros(5, 2), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(5, dtype=torch.int32),
                                 torch.zeros(2, 5, dtype=torch.int32).T])
def test_binding_refuses_trees_of_attention(bpa, bad):
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError, match="tree"):
        bpa.make_cache_batch(torch.zeros(5, 4, 64), torch.zeros(3, 4, **i32), torch.zeros(3, **i32), torch.zeros(4, **i32), tree=bad)
    got = bpa.make_cache_batch(torch.zeros(5, 4, 64), torch.zeros(3, 4, **i32), torch.zeros(3, **i32), torch.zeros(4, **i32),
                               tree=torch.zeros(5, 7, **i32))
    assert got.tree_words == 7 and got.tree


# ---- the oracle ---------------------------------------------------------------------------------------------
def test_oracle_tree_by_hand():
    tree, pos = ora.tree_masks([-1, 0, 0, 1, -1, -1, 0], [13, 7], [0, 5, 7], 1)
    assert tree[:, 0].tolist() == [1, 0b11, 0b101, 0b1011, 0b10000, 1, 0b11]
    assert pos.tolist() == [8, 9, 9, 10, 8, 5, 6]
    assert ora.tree_set([-2 ** 31, 3]) == {31, 32, 33}


def test_oracle_attention_under_a_chain_is_causal():
    rng = np.random.default_rng(1)
    kc, vc = rng.integers(0, 120, (3, 1, 4, 8)).astype(np.uint8), rng.integers(0, 120, (3, 1, 4, 8)).astype(np.uint8)
    s = np.full((3, 1), 0.125)
    q = rng.standard_normal((3, 2, 8))
    args = (q, kc, vc, s, s, np.array([[2, 0, 1]]), [9], [0, 3])
    tree, _ = ora.tree_masks([-1, 0, 1], [9], [0, 3], 1)
    for window in ((-1, -1), (8, -1)):
        for x, y in zip(ora.attention(*args, window=window, tree=tree), ora.attention(*args, window=window)):
            np.testing.assert_allclose(x, y)
    # a window is measured from the row's depth, and bounds the context alone
    o, m, l = ora.attention(*args, window=(2, -1), tree=tree)
    z = lambda i, k: ora.e4m3_values()[kc[[2, 0, 1][k // 4], 0, k % 4]] * 0.125 @ q[i, 0] / 8 ** 0.5   # noqa: E731
    for i, keys in enumerate(([4, 5, 6], [5, 6, 7], [6, 7, 8])):
        zs = np.array([z(i, k) for k in keys])
        assert np.isclose(m[0, i], zs.max()) and np.isclose(l[0, i], np.exp(zs - zs.max()).sum())


def test_oracle_keep_by_hand():
    codes = np.zeros((3, 1, 4, 1), np.uint8)
    codes[0, 0, :, 0], codes[1, 0, :, 0], codes[2, 0, :, 0] = [0x38, 0x40, 0x48, 0x50], [0x39, 0x41, 0x49, 0x51], [0x3A, 0x42, 0x4A, 0x52]
    scale = np.array([[1.0], [2.0], [0.5]])
    table = np.array([[0, 1, 2]])
    # ctx 2, ten new: tokens 1, 4, 7 (places 3, 6, 9) to places 2, 3, 4
    got, s = ora.keep(codes, scale, [[1, 4, 7]], [12], [0, 10], table)
    val = ora.e4m3_values()
    assert s[:, 0].tolist() == [2.0, 0.5, 0.5]
    np.testing.assert_array_equal(val[got[0, 0, :, 0]] * 2, [val[0x38], val[0x40], val[0x50], val[0x49] * 2])
    assert got[1, 0, 0, 0] == 0x42 and (got[2] == codes[2]).all()


def test_oracle_fork_and_release_by_hand():
    table = np.full((4, 3), -1)
    table[0, :3] = [5, 2, 7]
    a, b, ctx, table, refs, left = ora.fork([0, 0], [2, 3], [10, 0, 0, 0], table, np.zeros(8, int), [1, 3, 4, 6], 1, 4)
    assert a.tolist() == [7, -1] and b.tolist() == [1, -1] and ctx.tolist() == [10, 0, 10, 0] and left == 0
    assert table[2].tolist() == [5, 2, 1] and refs.tolist() == [0, 0, 1, 0, 0, 1, 0, 0]
    ctx, refs, free, left = ora.release(ctx, [0, 0, 8, 0], table, refs, [1, 3, 4, 6, 0, 0, 0, 0], 0, 4)
    assert refs.tolist() == [0] * 8 and free[:left].tolist() == [1, 7]
