"""Trees of drafted tokens under a sliding window, without a GPU: refusals, what the binding calls, and pins of the
64-bit oracle: a row under its mask sees what the last token of its path sees in plain causal attention."""
import numpy as np
import pytest
import torch

from oracle import cache as ora
from tests.test_cache_host import _Fake, streams  # noqa: F401
from tests.test_pages_host import P, _calls, bpa  # noqa: F401

WINDOWS = [0, 1, 3, 7, 8, 20]


def test_library_refuses(bpa):  # noqa: F811
    L = bpa.lib()
    base = dict(R=3, T=5, words=1, wl=3, parents=P, kv=P, cu=P, tree=P, pos=P, ws=P, n=256)
    call = lambda **kw: L.bpa_cache_tree_window(*{**base, **kw}.values(), None)                       # noqa: E731
    for bad in (dict(R=0), dict(T=-1), dict(T=(1 << 30) + 1), dict(words=0), dict(words=33), dict(wl=-2), dict(wl=-2 ** 31), dict(parents=None),
                dict(kv=None), dict(cu=None), dict(tree=None)):
        assert call(**bad) == 1, bad
    assert call(ws=None) == 3 and call(ws=P + 8) == 3 and call(n=255) == 3


@pytest.mark.parametrize("window,left", [(None, None), ((-1, -1), None), ((-1, 5), None), ((0, -1), 0), ((7, 0), 7), ((2 ** 31 - 1, -1), 2 ** 31 - 1)])
def test_binding_passes_the_left_bound(bpa, streams, monkeypatch, window, left):  # noqa: F811
    seen = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.append((name, a)) or 0

    monkeypatch.setattr(bpa, "lib", Lib)
    _calls(bpa)[0]["tree"](window=window)
    (name, a), = seen
    assert a[:3] == (3, 5, 2)
    assert (name, len(a)) == (("bpa_cache_tree", 11) if left is None else ("bpa_cache_tree_window", 12)) and (left is None or a[3] == left)


@pytest.mark.parametrize("window", [(-2, -1), (3, -2), (2 ** 31, -1), (0, -2 ** 40)])
def test_binding_refuses(bpa, streams, window):  # noqa: F811
    with pytest.raises(ValueError, match="window|2\\^31"):
        _calls(bpa)[0]["tree"](window=window)
    assert not streams[2]


def test_masks_by_hand():
    parents = [-1, 0, 0, 1, 3, -1, 4]                     # 0 - 1 - 3 - 4 - 6, 0 - 2, 5
    want = {0: [1, 2, 4, 8, 16, 32, 64], 1: [1, 3, 5, 10, 24, 32, 80], 2: [1, 3, 5, 11, 26, 32, 88], 3: [1, 3, 5, 11, 27, 32, 90],
            4: [1, 3, 5, 11, 27, 32, 91], -1: [1, 3, 5, 11, 27, 32, 91]}
    for wl, masks in want.items():
        tree, pos = ora.tree_masks(parents, [13], [0, 7], 1, wl)
        assert tree[:, 0].tolist() == masks and pos.tolist() == [6, 7, 7, 8, 9, 6, 10]
    far, _ = ora.tree_masks(list(range(-1, 69)), [70], [0, 70], 3, 33)
    assert [sorted(ora.tree_set(x)) for x in far] == [list(range(max(0, i - 33), i + 1)) for i in range(70)]


def _step(rng, ctx, n, P=4):
    pages = -(-(ctx + n) // P)
    kc, vc = (rng.integers(0, 120, (pages, 1, P, 8)).astype(np.uint8) for _ in range(2))
    return rng.standard_normal((n, 2, 8)), kc, vc, np.full((pages, 1), 0.05), rng.permutation(pages)


@pytest.mark.parametrize("wl", WINDOWS)
def test_oracle_chain_is_causal_attention_under_the_window(wl):
    q, kc, vc, s, ids = _step(np.random.default_rng(1), 20, 9)
    args = (q, kc, vc, s, s, ids[None], [29], [0, 9])
    tree, _ = ora.tree_masks(list(range(-1, 8)), [29], [0, 9], 1, wl)
    for x, y in zip(ora.attention(*args, window=(wl, -1), tree=tree), ora.attention(*args, window=(wl, -1))):
        np.testing.assert_allclose(x, y)


@pytest.mark.parametrize("wl", WINDOWS)
def test_oracle_every_path_is_causal_attention_under_the_window(wl):
    """Each row beside causal attention over the context and the row's path alone."""
    rng, ctx, n, P = np.random.default_rng(2), 5, 12, 4
    parents = [-1, 0, 1, 2, 3, 0, 5, 6, -1, 4, 9, 7]
    q, kc, vc, s, ids = _step(rng, ctx, n)
    at = lambda c, p: c[ids[p // P], 0, p % P]                                                         # noqa: E731
    tree, pos = ora.tree_masks(parents, [ctx + n], [0, n], 1, wl)
    got = ora.attention(q, kc, vc, s, s, ids[None], [ctx + n], [0, n], window=(wl, -1), tree=tree)
    for i in range(n):
        path, j = [], i
        while j >= 0:
            path.insert(0, j)
            j = parents[j]
        places = list(range(ctx)) + [ctx + j for j in path]
        assert pos[i] == len(places) - 1
        pages = -(-len(places) // P)
        k1, v1 = np.zeros((pages, 1, P, 8), np.uint8), np.zeros((pages, 1, P, 8), np.uint8)
        for to, p in enumerate(places):
            k1[to // P, 0, to % P], v1[to // P, 0, to % P] = at(kc, p), at(vc, p)
        one = ora.attention(q[i:i + 1], k1, v1, s[:pages], s[:pages], np.arange(pages)[None], [len(places)], [0, 1], window=(wl, -1))
        np.testing.assert_allclose(got[0][i], one[0][0])
        np.testing.assert_allclose(got[1][:, i], one[1][:, 0])
        np.testing.assert_allclose(got[2][:, i], one[2][:, 0])


def test_oracle_right_bound_says_nothing_under_a_tree():
    """Masks of the caller's own may name rows behind their own: the header's formula has no right bound there."""
    rng = np.random.default_rng(3)
    q, kc, vc, s, ids = _step(rng, 20, 9)
    args, tree = (q, kc, vc, s, s, ids[None], [29], [0, 9]), rng.integers(0, 2 ** 9, (9, 1))
    for wl in (-1, 4):
        for wr in (0, 3):
            for x, y in zip(ora.attention(*args, window=(wl, wr), tree=tree), ora.attention(*args, window=(wl, -1), tree=tree)):
                np.testing.assert_array_equal(x, y)
