"""GPU parity of trees of drafted tokens under a sliding window: masks equal to the definition, and attention under
them equal to plain causal attention under the same window (the 64-bit definition without a tree), with the
tolerances of test_gpu_cache."""
import numpy as np
import pytest
import torch

from oracle import cache as ora
from tests.test_gpu_cache import DTYPES, check_attention, i32, make_step, on_gpu
from tests.test_gpu_trees import bpa, grow, run_under_tree, takes_many_rows  # noqa: F401

pytestmark = pytest.mark.gpu


def run_masks(bpa, parents, kv, cu, words, wl):  # noqa: F811
    T, ws = len(parents), torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    tree, pos = torch.full((T, words), 99, dtype=torch.int32, device="cuda"), torch.full((T,), 99, dtype=torch.int32, device="cuda")
    bpa.bpa_cache_tree(i32(parents), i32(kv), i32(cu), words=words, window=(wl, -1), tree=tree, positions=pos, workspace_buf=ws)
    torch.cuda.synchronize()
    bpa.bpa_check(ws)
    return tree, pos


@pytest.mark.parametrize("wl", [-1, 0, 1, 3, 31, 32, 200, 2 ** 31 - 1])
@pytest.mark.parametrize("new,words,width", [([5, 0, 32, 7], 1, 3), ([33, 1, 64], 2, 2), ([200, 3], 7, 1)])
def test_masks_equal_the_definition(bpa, new, words, width, wl):  # noqa: F811
    rng = np.random.default_rng(sum(new))
    parents = sum((grow(rng, n, width) for n in new), []) + [-1] * 5
    cu, kv = np.concatenate([[0], np.cumsum(new)]), [n + int(rng.integers(0, 500)) for n in new]
    tree, pos = run_masks(bpa, parents, kv, cu, words, wl)
    want_tree, want_pos = ora.tree_masks(parents, kv, cu, words, wl)
    np.testing.assert_array_equal(tree.cpu().numpy(), want_tree)
    np.testing.assert_array_equal(pos.cpu().numpy(), want_pos)


SHAPES = {"few": ([200, 0, 63], [9, 1, 7], 4, 2, 64, 64, 16), "many": ([200, 0, 63, 140], [40, 60, 3, 33], 64, 16, 64, 64, 16),
          "any": ([200, 0, 63], [9, 1, 12], 4, 2, 40, 24, 20)}


@DTYPES
@pytest.mark.parametrize("wl", [0, 3, 20, 32])
@pytest.mark.parametrize("shape", SHAPES)
def test_a_chain_is_causal_attention_under_the_window(bpa, shape, wl, dtype):  # noqa: F811
    """The few-row kernel, the tensor cores (a table with room for more keys makes the choice) and the kernel for any shape."""
    rng = np.random.default_rng(31)
    case = SHAPES[shape]
    c, new, words = make_step(rng, *case, pad=2), case[1], -(-max(case[1]) // 32)
    parents = sum((list(range(-1, n - 1)) for n in new), []) + [-1] * 2
    tree, _ = run_masks(bpa, parents, c["kv"], c["cu"], words, wl)
    sink = torch.linspace(-2, 2, case[2], device="cuda")
    rooms = (0, 2 ** 18 // case[6]) if takes_many_rows(c, dtype) else (0,)
    assert (len(rooms) == 2) == (shape == "many" and dtype == torch.bfloat16)
    for room in rooms:
        t = on_gpu({**c, "table": np.concatenate([c["table"], np.full((len(new), room), -1)], 1)}, dtype)
        for s in (None, sink):
            o, m, l = bpa.bpa_cache_attn(*t, max_q=c["max_q"], window=(wl, -1), tree=tree, sink=s)
            torch.cuda.synchronize()
            check_attention(c, dtype, o, m, l, window=(wl, -1), sink=None if s is None else s.double().cpu().numpy())


@DTYPES
@pytest.mark.parametrize("shape", SHAPES)
def test_trees_under_windows_of_less_than_their_depth(bpa, shape, dtype):  # noqa: F811
    rng = np.random.default_rng(32)
    case = SHAPES[shape]
    c, new = make_step(rng, *case), case[1]
    parents = sum((grow(rng, n, 2) for n in new), [])
    for wl in (0, 2, 9):
        tree, _ = run_masks(bpa, parents, c["kv"], c["cu"], 2, wl)
        np.testing.assert_array_equal(tree.cpu().numpy(), ora.tree_masks(parents, c["kv"], c["cu"], 2, wl)[0])
        run_under_tree(bpa, c, dtype, tree.cpu().numpy(), window=(wl, -1))


@DTYPES
@pytest.mark.parametrize("shape", SHAPES)
def test_right_bounds_say_nothing_under_any_masks(bpa, shape, dtype):  # noqa: F811
    rng = np.random.default_rng(33)
    case = SHAPES[shape]
    c = make_step(rng, *case)
    tree = rng.integers(-2 ** 31, 2 ** 31, (c["q"].shape[0], 2))
    for window in ((-1, 0), (6, 3)):
        run_under_tree(bpa, c, dtype, tree, window=window)


def test_verified_rows_are_those_decoded_one_by_one(bpa):  # noqa: F811
    """Two paths of a tree of drafts, verified at once and decoded token by token under the same window: the same
    outputs.  Every row's largest key and value are alike, so pages keep one scale and codes are equal both ways; each side
    is then off by 2^-8 of the output and of the weighted values (at most 4) at most, and by a thousandth of that else."""
    Hq, Hkv, d, P, ctx, n, wl = 8, 2, 64, 16, 40, 24, 5
    g = torch.Generator().manual_seed(34)
    k, v = (torch.randn(ctx + n, Hkv, d, generator=g).clamp(-3, 3) for _ in range(2))
    k[..., 0], v[..., 0] = 4.0, 4.0
    k, v, q = (t.to(torch.bfloat16).cuda() for t in (k, v, torch.randn(n, Hq, d, generator=g)))
    pages = -(-(ctx + n) // P)
    parents = [-1] + [max(-1, i - 2) for i in range(1, n)]                    # two chains side by side from the context on

    def fresh():
        kc, vc = (torch.zeros(pages, Hkv, P, d, dtype=torch.uint8, device="cuda") for _ in range(2))
        cache = (kc, vc, torch.zeros(pages, Hkv, device="cuda"), torch.zeros(pages, Hkv, device="cuda"))
        bpa.bpa_cache_append(k[:ctx], v[:ctx], i32(range(ctx)), *cache)
        return cache

    cache, table = fresh(), i32(range(pages))[None]
    kv, cu = i32([ctx + n]), i32([0, n])
    bpa.bpa_cache_append(k[ctx:], v[ctx:], i32(range(ctx, ctx + n)), *cache)
    tree, pos = bpa.bpa_cache_tree(i32(parents), kv, cu, words=1, window=(wl, 0))
    at_once = bpa.bpa_cache_attn(q, *cache, table, kv, cu, max_q=n, window=(wl, 0), tree=tree)
    for leaf in (n - 1, n - 2):
        path, i = [], leaf
        while i >= 0:
            path.insert(0, i)
            i = parents[i]
        cache = fresh()
        for depth, i in enumerate(path):
            p = ctx + depth
            bpa.bpa_cache_append(k[ctx + i:ctx + i + 1], v[ctx + i:ctx + i + 1], i32([p]), *cache)
            o, m, l = bpa.bpa_cache_attn(q[i:i + 1], *cache, table, i32([p + 1]), i32([0, 1]), max_q=1, window=(wl, 0))
            torch.cuda.synchronize()
            assert int(pos[i]) == p
            assert (o[0].float() - at_once[0][i].float()).abs().max() <= 2 * 2.002 * 2.0 ** -8 * 4
            for a, b in ((m, at_once[1]), (l, at_once[2])):
                assert torch.allclose(a[:, 0], b[:, i], rtol=1e-4, atol=1e-4)
