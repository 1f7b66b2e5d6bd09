"""GPU parity of trees of drafted tokens over the paged 8-bit cache: masks from parents, attention under
them, accepted paths kept, and the steps of a speculating loop together.  Masks, positions, codes and
scales must be equal; attention is held to the tolerances of test_gpu_cache."""
import numpy as np
import pytest
import torch

from oracle import cache as ora
from oracle import rope as rope_ora
from tests.test_gpu_cache import DTYPES, as_dtype, check_attention, f64, i32, make_step, on_gpu, random_cache, slots_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bpa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from ring_attention_gb300 import build
    build.build()
    from ring_attention_gb300 import bpa as mod
    return mod


def grow(rng, n, width):
    """Parents of a random tree of n nodes; width 1: a chain."""
    return [-1 if i == 0 else int(rng.integers(max(-1 if width > 8 else 0, i - width), i)) for i in range(n)]


def run_tree(bpa, parents, kv, cu, words):
    T = len(parents)
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    tree, pos = torch.full((T, words), 99, dtype=torch.int32, device="cuda"), torch.full((T,), 99, dtype=torch.int32, device="cuda")
    bpa.bpa_cache_tree(i32(parents), i32(kv), i32(cu), words=words, tree=tree, positions=pos, workspace_buf=ws)
    torch.cuda.synchronize()
    return tree.cpu().numpy(), pos.cpu().numpy(), ws


# ---- masks -------------------------------------------------------------------------------------------
@pytest.mark.parametrize("new,words,width", [([1], 1, 1), ([5, 0, 32, 7], 1, 3), ([33, 1, 64], 2, 6), ([64], 2, 1), ([200, 3], 7, 20),
                                             ([1024, 17], 32, 1), ([1000], 32, 30)])
def test_masks_equal_the_definition(bpa, new, words, width):
    rng = np.random.default_rng(sum(new))
    parents = sum((grow(rng, n, width) for n in new), []) + [-1] * 5          # rows of no request
    cu = np.concatenate([[0], np.cumsum(new)])
    kv = [n + int(rng.integers(0, 500)) for n in new]
    tree, pos, ws = run_tree(bpa, parents, kv, cu, words)
    bpa.bpa_check(ws)
    want_tree, want_pos = ora.tree_masks(parents, kv, cu, words)
    np.testing.assert_array_equal(tree, want_tree)
    np.testing.assert_array_equal(pos, want_pos)


def test_masks_of_requests_that_wait_and_rows_in_front(bpa):
    rng = np.random.default_rng(1)
    cu, parents = [3, 8, 12, 12, 15], [7] * 3 + grow(rng, 5, 3) + grow(rng, 4, 3) + grow(rng, 3, 2) + [9, 9]
    kv = [0, 40, 6, 3]                                # the first waits
    tree, pos, ws = run_tree(bpa, parents, kv, cu, 1)
    bpa.bpa_check(ws)
    for got, want in zip((tree, pos), ora.tree_masks(parents, kv, cu, 1)):
        np.testing.assert_array_equal(got, want)


def test_masks_report_what_does_not_fit(bpa):
    chain = lambda n: list(range(-1, n - 1))                                  # noqa: E731
    good = chain(4) + chain(3)
    for at, value in ((5, 1), (5, 2), (5, -2), (4, 3), (6, 10 ** 6), (2, -2 ** 31)):
        bad = list(good)
        bad[at] = value
        tree, pos, ws = run_tree(bpa, bad, [10, 9], [0, 4, 7], 1)
        with pytest.raises(bpa.BpaError):
            bpa.bpa_check(ws)
        bad[at] = -1
        for got, want in zip((tree, pos), ora.tree_masks(bad, [10, 9], [0, 4, 7], 1)):
            np.testing.assert_array_equal(got, want)
    # more rows than tokens, more rows than bits: that request's rows see nothing
    for kv, cu, words, parents in (([10, 2], [0, 4, 7], 1, good), ([10, 60], [0, 4, 37], 1, chain(4) + chain(33))):
        tree, pos, ws = run_tree(bpa, parents, kv, cu, words)
        with pytest.raises(bpa.BpaError):
            bpa.bpa_check(ws)
        want_tree, want_pos = ora.tree_masks(parents[:4], kv[:1], cu[:2], words)
        np.testing.assert_array_equal(tree[:4], want_tree)
        assert (tree[4:] == 0).all() and (pos[4:] == -1).all() and (pos[:4] == want_pos).all()


# ---- attention under a tree ------------------------------------------------------------------------------
def takes_many_rows(c, dtype):
    """Whether the kernel for many rows takes these shapes, if the page table has room for enough keys."""
    (_, Hkv, P, d), dv, (T, Hq, _) = c["kc"].shape, c["vc"].shape[3], c["q"].shape
    return dtype == torch.bfloat16 and d % 16 == 0 and dv % 16 == 0 and max(d, dv) <= 128 and dv <= max(d, 64) and P % 16 == 0 and \
        c["max_q"] * Hq // Hkv > 32


def run_under_tree(bpa, c, dtype, tree, sink=None, nhd=False, max_q=None, **kw):
    """Once with a page table of just the pages, once (where that changes the kernel) with one of 2^18 tokens more."""
    out = attend_under_tree(bpa, c, dtype, tree, sink, nhd, max_q, **kw)
    if takes_many_rows(c, dtype) and max_q is None:
        more = 2 ** 18 // c["kc"].shape[2]
        roomy = {**c, "table": np.concatenate([c["table"], np.full((len(c["table"]), more), -1)], 1)}
        return attend_under_tree(bpa, roomy, dtype, tree, sink, nhd, max_q, **kw)
    return out


def attend_under_tree(bpa, c, dtype, tree, sink=None, nhd=False, max_q=None, **kw):
    t, marker = on_gpu(c, dtype, nhd), 77.0
    T, Hq = c["q"].shape[:2]
    o = torch.full((T, Hq, c["vc"].shape[3]), marker, dtype=dtype, device="cuda")
    m, l = (torch.full((Hq, T), marker, device="cuda") for _ in range(2))
    dev = {**kw, "tree": i32(tree), "max_q": c["max_q"] if max_q is None else max_q,
           "sink": None if sink is None else torch.from_numpy(sink.astype(np.float32)).cuda()}
    need = bpa.bpa_cache_attn_workspace_size(bpa.make_cache_desc(*t[1:5], dtype), bpa.make_cache_batch(t[0], *t[5:], **dev))
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    bpa.bpa_cache_attn(*t, o=o, m=m, l=l, workspace_buf=ws, **dev)
    torch.cuda.synchronize()
    bpa.bpa_check(ws)
    valid = check_attention(c, dtype, o, m, l, sink=sink, tree=tree, **kw)
    assert (o[~valid] == marker).all() and (m[:, ~valid] == marker).all() and (l[:, ~valid] == marker).all()
    return o, m, l


def masks_for(rng, c, new, width, words=None):
    words = words or max(1, -(-max(new) // 32))
    parents = sum((grow(rng, n, width) for n in new), []) + [-1] * (c["q"].shape[0] - sum(new))
    return ora.tree_masks(parents, c["kv"], c["cu"], words)[0]


TREES = [    # ctx, new, Hq, Hkv, d, dv, P: one row, few rows, items of many rows, shapes of every kernel, few requests
    ([0], [1], 1, 1, 64, 64, 16), ([700], [5], 32, 8, 128, 128, 64), ([0, 1, 63, 300], [3, 8, 1, 2], 8, 2, 128, 128, 64),
    ([15, 16, 511], [7, 16, 2], 8, 2, 64, 64, 16), ([40, 90], [26, 9], 16, 4, 128, 64, 32), ([130, 7], [11, 4], 7, 1, 80, 80, 16),
    ([260, 3], [5, 33], 6, 2, 192, 64, 128), ([300, 33], [9, 12], 4, 4, 256, 256, 16), ([90, 5], [10, 2], 3, 1, 33, 7, 5),
    ([9, 14], [3, 3], 2, 1, 512, 512, 8), ([500, 20], [64, 40], 8, 2, 128, 128, 64), ([64, 0], [33, 100], 8, 2, 64, 64, 32),
    ([1000, 130, 37], [64, 60, 3], 32, 8, 128, 128, 64), ([300, 5, 64, 127, 1], [17, 20, 64, 1, 129], 32, 8, 128, 64, 32),
    ([90, 0, 15], [130, 40, 257], 32, 16, 64, 64, 16), ([40, 200], [30, 2], 96, 16, 80, 112, 128),
]


@DTYPES
@pytest.mark.parametrize("width", [1, 4, 30])
@pytest.mark.parametrize("case", TREES, ids=lambda c: f"H{c[2]}_{c[3]}_d{c[4]}_{c[5]}_P{c[6]}_q{max(c[1])}")
def test_attention_under_trees(bpa, case, width, dtype):
    rng = np.random.default_rng(sum(case[0]) + case[4] + width)
    c = make_step(rng, *case, pad=2)
    run_under_tree(bpa, c, dtype, masks_for(rng, c, case[1], width))


MASKS = {"window": dict(window=(20, -1)), "window_0": dict(window=(0, -1)), "window_3": dict(window=(3, 0)), "scale": dict(scale=0.3),
         "wide": dict(window=(2 ** 31 - 1, 2 ** 31 - 1))}


@DTYPES
@pytest.mark.parametrize("shape", [([200, 0, 63], [9, 1, 4], 8, 2, 64, 64, 16), ([200, 0, 63, 140], [40, 65, 3, 20], 64, 16, 64, 64, 16),
                                   ([200, 0, 63], [9, 1, 4], 4, 2, 40, 24, 20)], ids=["few", "many", "any"])
@pytest.mark.parametrize("mask", MASKS)
def test_attention_under_trees_masks_and_sinks(bpa, mask, shape, dtype):
    rng = np.random.default_rng(8)
    c = make_step(rng, *shape, pad=2)
    tree = masks_for(rng, c, shape[1], 5)
    run_under_tree(bpa, c, dtype, tree, **MASKS[mask])
    run_under_tree(bpa, c, dtype, tree, sink=rng.standard_normal(shape[2]) * 3, **MASKS[mask])


@DTYPES
@pytest.mark.parametrize("shape", [([130, 0, 40], [9, 1, 4], 8, 2, 64, 64, 16), ([200, 0, 63, 140], [40, 65, 3, 20], 64, 16, 64, 64, 16),
                                   ([70, 0, 63], [9, 1, 4], 4, 2, 40, 24, 20)], ids=["few", "many", "any"])
def test_attention_under_any_masks(bpa, shape, dtype):
    """The caller's own masks: rows that do not see themselves or see later ones, rows that see nothing, bits past
    the request's rows, fewer words than rows; requests that wait, with fewer tokens than rows."""
    rng = np.random.default_rng(9)
    c = make_step(rng, *shape, pad=2)
    T, words = c["q"].shape[0], -(-max(shape[1]) // 32)
    tree = rng.integers(-2 ** 31, 2 ** 31, (T, words))
    tree[::3] = 0
    run_under_tree(bpa, c, dtype, tree)
    run_under_tree(bpa, c, dtype, tree[:, :1])
    run_under_tree(bpa, c, dtype, np.concatenate([tree, tree], 1), window=(5, -1))
    run_under_tree(bpa, c, dtype, tree, max_q=0)
    c["kv"] = c["kv"].copy()
    c["kv"][0], c["kv"][2] = 0, 2
    run_under_tree(bpa, c, dtype, tree)
    run_under_tree(bpa, c, dtype, tree, sink=rng.standard_normal(shape[2]))


@DTYPES
def test_a_chain_is_causal_attention(bpa, dtype):
    rng = np.random.default_rng(10)
    new = [20, 1, 33]
    c = make_step(rng, [200, 30, 77], new, 8, 2, 64, 64, 16)
    t, tree = on_gpu(c, dtype), i32(masks_for(rng, c, new, 1))
    for kw in ({}, dict(window=(50, -1))):
        a = bpa.bpa_cache_attn(*t, max_q=33, tree=tree, **kw)
        b = bpa.bpa_cache_attn(*t, max_q=33, **kw)
        tol = 2.0 ** -6 if dtype == torch.bfloat16 else 2.0 ** -16
        for x, y in zip(a, b):
            assert ((x.float() - y.float()).abs() <= tol * (y.float().abs() + 1)).all()


@pytest.mark.parametrize("shape", [([3000], [30], 8, 2, 128, 128, 64), ([5000, 9000], [64, 50], 8, 2, 64, 64, 16),
                                   ([2000] * 9, [48] * 9, 32, 8, 128, 128, 64)], ids=["one", "two", "batch"])
def test_attention_under_trees_long_contexts_and_repeats(bpa, shape):
    """Keys cut between blocks at any place; a call repeats itself bit for bit, also under a captured graph."""
    rng = np.random.default_rng(11)
    c = make_step(rng, *shape, pad=1)
    tree = masks_for(rng, c, shape[1], 6)
    c["table"] = np.concatenate([c["table"], np.full((len(c["table"]), 2 ** 14), -1)], 1)
    first = attend_under_tree(bpa, c, torch.bfloat16, tree)
    t, dt = on_gpu(c, torch.bfloat16), i32(tree)
    outs = [torch.full_like(x, 77.0) for x in first]
    graph = torch.cuda.CUDAGraph()
    call = lambda: bpa.bpa_cache_attn(*t, max_q=c["max_q"], tree=dt, o=outs[0], m=outs[1], l=outs[2])     # noqa: E731
    call()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        for x in outs:
            x.fill_(77.0)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(first, outs):
            assert torch.equal(x, y)


@pytest.mark.parametrize("dims", [(64, 64), (128, 64), (128, 128), (112, 96)], ids=lambda d: f"{d[0]}_{d[1]}")
def test_attention_under_trees_windows_of_many_rows(bpa, dims):
    rng = np.random.default_rng(13)
    new = [64, 33, 32, 60, 9]
    c = make_step(rng, [1200, 900, 1700, 3, 2100], new, 32, 8, *dims, 64)
    tree = masks_for(rng, c, new, 6)
    for kw in (dict(window=(1000, -1)), dict(window=(1100, -1), sink=rng.standard_normal(32) * 3)):
        run_under_tree(bpa, c, torch.bfloat16, tree, **kw)


MANY = ([300, 5, 640, 127], [40, 20, 64, 33], 32, 8, 128, 128, 32)


@pytest.mark.parametrize("first,later", [(1e-20, 1e15), (1e15, 1e-20), (1.0, 2.0 ** 45), (1.0, 2.0 ** -45)])
def test_attention_under_trees_value_scales_far_apart(bpa, first, later):
    rng = np.random.default_rng(14)
    c = make_step(rng, *MANY)
    tree = masks_for(rng, c, MANY[1], 4)
    c["vs"] = c["vs"].copy()
    for r in (0, 2):                              # the other requests' scales are alike
        pages = c["table"][r][c["table"][r] >= 0]
        c["vs"][pages[:4]] *= np.float32(first)
        c["vs"][pages[4:]] *= np.float32(later)
    run_under_tree(bpa, c, torch.bfloat16, tree)


def test_attention_under_trees_pages_of_zeros_and_nan(bpa):
    rng = np.random.default_rng(15)
    c = make_step(rng, *MANY)
    tree = masks_for(rng, c, MANY[1], 4)
    for r, j in ((0, 2), (2, 0), (2, 7)):
        page = c["table"][r, j]
        c["vc"][page], c["vs"][page] = 0, 0
    clean = run_under_tree(bpa, c, torch.bfloat16, tree)
    bad = {**c, "kc": c["kc"].copy(), "vc": c["vc"].copy()}
    bad["kc"][c["table"][0, 1], 1, 5, 7] = 0x7F       # a key of the context: every row of the request, kv head 1
    bad["vc"][c["table"][2, 3], 2, 9, 11] = 0x7F      # a value: channel 11 of the rows of that request, kv head 2
    bad["table"] = np.concatenate([bad["table"], np.full((4, 2 ** 14), -1)], 1)
    t = on_gpu(bad, torch.bfloat16)
    o, m, l = bpa.bpa_cache_attn(*t, max_q=64, tree=i32(tree))
    torch.cuda.synchronize()
    cu = c["cu"]
    lost = torch.zeros_like(o, dtype=torch.bool)
    lost[cu[0]:cu[1], 4:8] = True
    lost[cu[2]:cu[3], 8:12, 11] = True
    assert o[lost].isnan().all() and not o[~lost].isnan().any()
    assert (o[~lost].float() - clean[0][~lost].float()).abs().max() <= 2.0 ** -7 * clean[0].float().abs().max()
    assert l[4:8, cu[0]:cu[1]].isnan().all() and not l[:4].isnan().any()


def test_attention_under_trees_scores_of_any_size(bpa):
    rng = np.random.default_rng(16)
    for qmag in (1e-6, 30.0, 1e4):
        c = make_step(rng, *MANY, qmag=qmag)
        run_under_tree(bpa, c, torch.bfloat16, masks_for(rng, c, MANY[1], 4))


def test_attention_under_trees_odd_strides(bpa):
    """Rows of q and o that are parts of wider ones, not aligned to 16 or 32 bytes; a cache of [pages, tokens, heads]."""
    rng = np.random.default_rng(17)
    c = make_step(rng, *MANY)
    tree = masks_for(rng, c, MANY[1], 4)
    c["table"] = np.concatenate([c["table"], np.full((4, 2 ** 14), -1)], 1)
    want = attend_under_tree(bpa, c, torch.bfloat16, tree, nhd=True)[0]
    t = list(on_gpu(c, torch.bfloat16))
    T = t[0].shape[0]
    for pad, off in ((1, 1), (8, 8), (3, 2)):
        q = torch.zeros(T, 32, 128 + pad + off, dtype=torch.bfloat16, device="cuda")[..., off:off + 128]
        q.copy_(t[0])
        o = torch.zeros(T, 32, 128 + pad + off, dtype=torch.bfloat16, device="cuda")[..., off:off + 128]
        got = bpa.bpa_cache_attn(q, *t[1:], max_q=64, tree=i32(tree), o=o)[0]
        assert got is o and torch.equal(got, want)


GROUPS = [   # ctx, new, Hq, Hkv, d, dv, P: heads of their own, many heads to one, more requests than a warp looks at together
    ([300, 20, 700], [64, 33, 40], 6, 6, 64, 64, 16), ([200, 90], [9, 4], 64, 1, 128, 128, 64), ([100, 260], [5, 3], 128, 2, 64, 64, 32),
    ([int(x) for x in np.random.default_rng(18).integers(0, 150, 70)], [1 + (i * 7) % 40 for i in range(70)], 2, 1, 64, 64, 16),
]


@pytest.mark.parametrize("case", GROUPS, ids=lambda c: f"R{len(c[0])}_H{c[2]}_{c[3]}")
def test_attention_under_trees_groups_and_many_requests(bpa, case):
    rng = np.random.default_rng(19)
    c = make_step(rng, *case)
    run_under_tree(bpa, c, torch.bfloat16, masks_for(rng, c, case[1], 3))


def test_attention_under_trees_rows_in_front_of_the_first_request(bpa):
    rng = np.random.default_rng(22)
    c = make_step(rng, *MANY, pad=2)
    tree = masks_for(rng, c, MANY[1], 4)
    front = 5
    c["q"] = np.concatenate([rng.standard_normal((front,) + c["q"].shape[1:]), c["q"]])
    c["cu"] = c["cu"] + front
    tree = np.concatenate([np.full((front, tree.shape[1]), -1), tree])
    run_under_tree(bpa, c, torch.bfloat16, tree)


def test_two_calls_under_trees_at_once(bpa):
    """Two streams, a workspace each: the answers of calls made one after the other, on both kernels."""
    for room in (0, 2 ** 14):
        cs = [make_step(np.random.default_rng(23 + i), *MANY) for i in range(2)]
        trees = [i32(masks_for(np.random.default_rng(25), c, MANY[1], 4)) for c in cs]
        for c in cs:
            c["table"] = np.concatenate([c["table"], np.full((4, room), -1)], 1)
        ts = [on_gpu(c, torch.bfloat16) for c in cs]
        want = [bpa.bpa_cache_attn(*t, max_q=64, tree=m) for t, m in zip(ts, trees)]
        torch.cuda.synchronize()
        side = [torch.cuda.Stream() for _ in range(2)]
        for _ in range(20):
            got = [bpa.bpa_cache_attn(*t, max_q=64, tree=m, stream=s) for t, m, s in zip(ts, trees, side)]
            torch.cuda.synchronize()
            for x, y in zip(got, want):
                assert all(torch.equal(u, v) for u, v in zip(x, y))


def test_attention_under_trees_reports_bad_pages(bpa):
    for shape in (([200, 0], [9, 1], 8, 2, 64, 64, 16), ([200, 80], [40, 65], 64, 16, 64, 64, 16), ([70, 0], [9, 1], 4, 2, 40, 24, 20)):
        rng = np.random.default_rng(12)
        c = make_step(rng, *shape)
        tree = masks_for(rng, c, shape[1], 5)
        for bad in (-1, 10 ** 8, c["kc"].shape[0]):
            table = np.concatenate([c["table"], np.full((2, 2 ** 14), -1)], 1)
            table[0, 2] = bad
            t = on_gpu({**c, "table": table}, torch.bfloat16)
            need = bpa.bpa_cache_attn_workspace_size(bpa.make_cache_desc(*t[1:5], torch.bfloat16),
                                                     bpa.make_cache_batch(t[0], *t[5:], max_q=c["max_q"], tree=i32(tree)))
            ws = torch.empty(need, dtype=torch.uint8, device="cuda")
            o, m, l = bpa.bpa_cache_attn(*t, max_q=c["max_q"], tree=i32(tree), workspace_buf=ws)
            torch.cuda.synchronize()
            with pytest.raises(bpa.BpaError):
                bpa.bpa_check(ws)
            good = on_gpu(c, torch.bfloat16)
            a, _, _ = bpa.bpa_cache_attn(*good, max_q=c["max_q"], tree=i32(tree))
            assert torch.allclose(o[c["cu"][1]:].float(), a[c["cu"][1]:].float(), atol=2e-2)


# ---- accepted paths ---------------------------------------------------------------------------------------
def run_keep(bpa, paths, kv, cu, table, kc, vc, ks, vs, nhd=False, most=None):
    most = max(1, max(len(p) for p in paths)) if most is None else most
    keep = np.array([list(p) + [-5] * (most - len(p)) for p in paths], np.int64).reshape(len(paths), most)
    dk, dv = (torch.from_numpy(c).cuda() for c in (kc, vc))
    if nhd:
        dk, dv = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (dk, dv))
    sk, sv = (torch.from_numpy(c).cuda() for c in (ks, vs))
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    bpa.bpa_cache_keep(i32(keep), i32([len(p) for p in paths]), i32(kv), i32(cu), i32(table), dk, dv, sk, sv, workspace_buf=ws)
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in (dk, dv, sk, sv)], ws


def keep_case(rng, ctx, new, paths, Hkv, d, dv, P, spread=1.0):
    pages = sum(-(-(a + b) // P) for a, b in zip(ctx, new)) + 2
    _, table = slots_for(rng, ctx, new, P, pages)
    kc, ks = random_cache(rng, pages, Hkv, P, d, spread)
    vc, vs = random_cache(rng, pages, Hkv, P, dv, spread)
    return paths, np.add(ctx, new), np.concatenate([[0], np.cumsum(new)]), table, kc, vc, ks, vs


def check_keep(got, paths, kv, cu, table, kc, vc, ks, vs):
    for codes, scale, gc, gs in ((kc, ks, got[0], got[2]), (vc, vs, got[1], got[3])):
        wc, wsc = ora.keep(codes, scale, paths, kv, cu, table)
        np.testing.assert_array_equal(gs, wsc)
        np.testing.assert_array_equal(gc, wc)


KEEPS = {    # ctx, new, paths, Hkv, d, dv, P
    "one": ([5], [1], [[0]], 1, 64, 64, 16), "none": ([5, 0], [3, 2], [[], []], 2, 64, 64, 16), "in_place": ([5], [6], [[0, 1, 2]], 2, 64, 64, 16),
    "last": ([0], [40], [[39]], 2, 128, 128, 16), "across": ([13, 16, 30], [30, 20, 9], [[1, 4, 17, 29], [2, 3, 19], [0, 8]], 2, 128, 64, 16),
    "all": ([10], [50], [list(range(50))], 2, 80, 80, 16), "shifted": ([7], [60], [list(range(1, 60))], 2, 128, 128, 16),
    "every_second": ([31, 2], [100, 33], [list(range(1, 100, 2)), list(range(0, 33, 2))], 3, 96, 32, 8),
    "odd": ([4, 9], [12, 13], [[3, 5, 6, 11], [1, 2, 12]], 3, 33, 7, 5), "page_of_one": ([2, 3], [9, 4], [[2, 4, 8], [3]], 2, 16, 16, 1),
    "wide": ([20], [30], [[3, 4, 20]], 1, 512, 256, 16), "one_page": ([100], [64], [[0, 5, 9, 30, 31, 63]], 2, 128, 128, 256),
    "full_pages": ([16, 32], [32, 16], [[16, 17, 30], [0, 15]], 2, 64, 64, 16),
}


@pytest.mark.parametrize("spread", [0.0, 1.0, 8.0])
@pytest.mark.parametrize("nhd", [False, True], ids=["hnd", "nhd"])
@pytest.mark.parametrize("name", KEEPS)
def test_keep_equals_the_definition(bpa, name, nhd, spread):
    c = keep_case(np.random.default_rng(len(name)), *KEEPS[name], spread=spread)
    got, ws = run_keep(bpa, *c, nhd=nhd)
    bpa.bpa_check(ws)
    check_keep(got, *c)


def test_keep_of_many_random_trees(bpa):
    rng = np.random.default_rng(20)
    ctx, new = rng.integers(0, 70, 60), rng.integers(0, 65, 60)
    paths = [sorted(rng.choice(n, int(rng.integers(0, n + 1)), replace=False).tolist()) if n else [] for n in new]
    c = keep_case(rng, ctx, new, paths, 2, 64, 48, 16, spread=3.0)
    got, ws = run_keep(bpa, *c)
    bpa.bpa_check(ws)
    check_keep(got, *c)


def test_keep_scales_of_zero_and_nan(bpa):
    rng = np.random.default_rng(21)
    c = keep_case(rng, [10, 3], [30, 40], [[9, 20, 29], [2, 30, 39]], 2, 64, 64, 16)
    kc, ks, table = c[4], c[6], c[3]
    for page in (table[0, 0], table[1, 2]):
        ks[page], kc[page] = 0, 0                     # pages of zeros, one with NaN
    kc[table[1, 2], :, 1, 3] = 0x7F
    kc[table[0, 1], :, :, 5] = 0x7F
    got, ws = run_keep(bpa, *c)
    bpa.bpa_check(ws)
    wc, wsc = ora.keep(kc, ks, c[0], *c[1:4])
    np.testing.assert_array_equal(got[2], wsc)
    nan = (wc & 0x7F) == 0x7F
    np.testing.assert_array_equal((got[0] & 0x7F) == 0x7F, nan)
    val = ora.e4m3_values()
    np.testing.assert_array_equal(val[got[0]][~nan], val[wc][~nan])


@pytest.mark.parametrize("bad", [[[5, 2]], [[0, 0]], [[-1, 2]], [[3, 20]], [[1, 2 ** 31 - 1]], [[-7, -3]], [list(range(21))]])
def test_keep_reports_and_leaves_the_request(bpa, bad):
    rng = np.random.default_rng(22)
    paths = bad + [[1, 5]]
    c = keep_case(rng, [10, 12], [20, 9], paths, 2, 64, 64, 16)
    got, ws = run_keep(bpa, *c)
    with pytest.raises(bpa.BpaError):
        bpa.bpa_check(ws)
    check_keep(got, [[], [1, 5]], *c[1:])             # the other request is kept as it should be


def test_keep_reports_counts_lengths_and_pages(bpa):
    rng = np.random.default_rng(23)
    paths, kv, cu, table, *cache = keep_case(rng, [10, 12], [20, 9], [[3, 19], [1, 5]], 2, 64, 64, 16)
    far = table.copy()
    far[0, 1] = 10 ** 7
    short = table[:, :1].copy()
    for args in ((kv, cu, far), (np.array([10, kv[1]]), cu, table), (kv, cu, short)):
        got, ws = run_keep(bpa, paths, *args, *cache)
        with pytest.raises(bpa.BpaError):
            bpa.bpa_check(ws)
        # (a short table: neither request fits)
        check_keep(got, [[], [1, 5] if args[2].shape[1] > 1 else []], kv, cu, table, *cache)
    keep, dev = i32([[0, 1], [1, 5]]), [torch.from_numpy(x).cuda() for x in cache]
    for count in ([-1, 2], [3, 2], [2 ** 31 - 1, 2]):
        t = [x.clone() for x in dev]
        ws = torch.empty(256, dtype=torch.uint8, device="cuda")
        bpa.bpa_cache_keep(keep, i32(count), i32(kv), i32(cu), i32(table), *t, workspace_buf=ws)
        torch.cuda.synchronize()
        with pytest.raises(bpa.BpaError):
            bpa.bpa_check(ws)
        check_keep([x.cpu().numpy() for x in t], [[], [1, 5]], kv, cu, table, *cache)


# ---- the steps of a speculating loop -----------------------------------------------------------------------
def test_speculating_steps_together(bpa):
    """Norm and rotation, plan, append, masks, attention, keep and release, step after step in one captured
    graph: every state against the definitions run side by side."""
    rng = np.random.default_rng(30)
    dtype, R, Hq, Hkv, d, P, num, width, n = torch.bfloat16, 3, 8, 2, 64, 16, 40, 12, 11
    free, table, ctx, count, refs = rng.permutation(num), np.full((R, width), -1), np.zeros(R, int), num, np.zeros(num, int)
    kc, vc = np.zeros((num, Hkv, P, d), np.uint8), np.zeros((num, Hkv, P, d), np.uint8)
    ks, vs = np.zeros((num, Hkv), np.float32), np.zeros((num, Hkv), np.float32)
    T = R * n
    freq = torch.tensor([10000.0 ** (-i / 32) for i in range(32)], device="cuda")
    weight = torch.linspace(0.5, 1.5, d, device="cuda")
    dt, dctx, dfree, dcount, drefs = i32(table), i32(ctx), i32(free), i32([count]), i32(refs)
    cache = [torch.from_numpy(x).cuda() for x in (kc, vc, ks, vs)]
    qkv = torch.zeros(T, Hq + 2 * Hkv, d, dtype=dtype, device="cuda")
    new, parents, keep, kept = i32([n] * R), i32(np.zeros(T)), i32(np.zeros((R, n))), i32(np.zeros(R))

    def step():
        kv, cu, slots, _, after, _ = bpa.bpa_cache_plan(dctx, new, dt, dfree, dcount, page_size=P, T=T, ctx_lens_out=dctx,
                                                        free_count_out=dcount)
        tree, pos = bpa.bpa_cache_tree(parents, kv, cu, words=1)
        q, k = bpa.bpa_rope_fwd(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], pos, freq, weight, weight)
        bpa.bpa_cache_append(k, qkv[:, Hq + Hkv:], slots, *cache, max_new=n)
        o, m, l = bpa.bpa_cache_attn(q, *cache, dt, kv, cu, max_q=n, tree=tree)
        state = [x.clone() for x in (*cache, after, dcount)]
        bpa.bpa_cache_keep(keep, kept, kv, cu, dt, *cache)
        bpa.bpa_cache_release(after, after - n + kept, dt, drefs, dfree, dcount, page_size=P, ctx_lens_out=dctx,
                              free_count_out=dcount)
        return kv, cu, slots, tree, pos, q, k, o, m, l, state

    graph = outs = None
    for it in range(6):
        x = rng.standard_normal((T, Hq + 2 * Hkv, d)) * 2.0 ** (it % 3)
        par = sum((grow(rng, n, 4) for _ in range(R)), [])
        paths = []
        for r in range(R):
            i, path = int(rng.integers(0, n)), []
            while i >= 0:
                path.append(i)
                i = par[r * n + i]
            paths.append(path[::-1])
        tx, _ = as_dtype(x, dtype)
        qkv.copy_(tx)
        parents.copy_(i32(par))
        keep.copy_(i32([p + [-1] * (n - len(p)) for p in paths]))
        kept.copy_(i32([len(p) for p in paths]))
        torch.cuda.synchronize()
        if it == 0:
            outs = step()
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    outs = step()
            graph.replay()
        torch.cuda.synchronize()
        kv, cu, slots, _, ctx, table, count = ora.plan(ctx, [n] * R, table, free, count, P, T)
        tree, pos = ora.tree_masks(par, kv, cu, 1)
        for got, want in zip(outs[:5], (kv, cu, slots, tree, pos)):
            np.testing.assert_array_equal(got.cpu().numpy(), want)
        angle = rope_ora.angles(pos[None], freq.cpu().numpy())
        for got, src in ((outs[5], tx[:, :Hq]), (outs[6], tx[:, Hq:Hq + Hkv])):
            want = rope_ora.forward(f64(src)[None], angle, f64(weight), 1e-6)[0]
            assert (np.abs(f64(got) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * np.abs(want).max()).all()
        kc, ks = ora.append(f64(outs[6]), slots, kc, ks)
        vc, vs = ora.append(f64(tx[:, Hq + Hkv:]), slots, vc, vs)
        for got, want in zip(outs[10], (kc, vc, ks, vs, ctx, [count])):
            np.testing.assert_array_equal(got.cpu().numpy(), want)
        c = dict(q=f64(outs[5]), kc=kc, vc=vc, ks=ks, vs=vs, table=table, kv=kv, cu=cu)
        check_attention(c, dtype, *outs[7:10], tree=tree)
        kc, ks = ora.keep(kc, ks, paths, kv, cu, table)
        vc, vs = ora.keep(vc, vs, paths, kv, cu, table)
        ctx, refs, free, count = ora.release(ctx, [a - n + len(p) for a, p in zip(ctx, paths)], table, refs, free, count, P)
        for got, want in zip((*cache, dctx, drefs, dcount), (kc, vc, ks, vs, ctx, refs, [count])):
            np.testing.assert_array_equal(got.cpu().numpy(), want)
        np.testing.assert_array_equal(dfree.cpu().numpy(), free)
