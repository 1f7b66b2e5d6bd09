"""GPU parity of shared pages: forks, copies and releases.  Everything is whole numbers or copies and must
be equal to the definitions."""
import numpy as np
import pytest
import torch

from oracle import cache as ora
from tests.test_gpu_cache import check_attention, i32, make_plan, make_step, on_gpu, random_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bpa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from ring_attention_gb300 import build
    build.build()
    from ring_attention_gb300 import bpa as mod
    return mod


def state_of(rng, ctx, P, spare, rows=0):
    """Requests of ctx tokens and `rows` without any: ctx, table, refs, free, count."""
    c = make_plan(rng, list(ctx) + [0] * rows, [0] * (len(ctx) + rows), P, spare)
    return dict(ctx=c["ctx"], table=c["table"], refs=np.zeros(len(c["free"]), int), free=c["free"], count=c["count"], P=P)


def run_fork(bpa, src, dst, c, in_place=False):
    ctx, table, refs, count = i32(c["ctx"]), i32(c["table"]), i32(c["refs"]), i32([c["count"]])
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    kw = dict(ctx_lens_out=ctx, free_count_out=count) if in_place else {}
    a, b, out, left = bpa.bpa_cache_fork(i32(src), i32(dst), ctx, table, refs, i32(c["free"]), count, page_size=c["P"],
                                         workspace_buf=ws, **kw)
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in (a, b, out, table, refs)] + [int(left[0])], ws


def run_release(bpa, keep, c, in_place=False):
    ctx, refs, free, count = i32(c["ctx"]), i32(c["refs"]), i32(c["free"]), i32([c["count"]])
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    kw = dict(ctx_lens_out=ctx, free_count_out=count) if in_place else {}
    out, left = bpa.bpa_cache_release(ctx, i32(keep), i32(c["table"]), refs, free, count, page_size=c["P"], workspace_buf=ws, **kw)
    torch.cuda.synchronize()
    return [out.cpu().numpy(), refs.cpu().numpy(), free.cpu().numpy(), int(left[0])], ws


def same(got, want):
    for i, (g, w) in enumerate(zip(got, want)):
        np.testing.assert_array_equal(g, w, err_msg=str(i))


FORKS = {    # ctx, P, spare, src
    "one": ([37], 16, 3, [0]), "full": ([32], 16, 0, [0, 0]), "empty": ([0, 5], 16, 1, [0, 1]), "several": ([37, 16, 5, 100], 16, 9, [0, 3, 0, 1, 2, 0]),
    "none": ([9], 4, 2, []), "no_pages_left": ([33, 16, 5, 9], 16, 2, [0, 1, 2, 3, 1, 0]), "page_of_one": ([7, 3], 1, 0, [1, 0, 0]),
    "odd": ([50, 3], 7, 5, [1, 0, 1]),
}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name", FORKS)
def test_fork_equals_the_definition(bpa, name, in_place):
    ctx, P, spare, src = FORKS[name]
    c = state_of(np.random.default_rng(1), ctx, P, spare, len(src) + 1)
    dst = [len(ctx) + 1 + i for i in range(len(src))][::-1]
    got, ws = run_fork(bpa, src, dst, c, in_place)
    bpa.bpa_check(ws)
    same(got, ora.fork(src, dst, **c))


@pytest.mark.parametrize("R,N,hi,P,spare", [(300, 500, 700, 16, 450), (50, 2000, 90, 32, 3000), (4000, 4192, 40, 8, 100), (1, 8191, 3, 64, 9000)])
def test_fork_and_release_of_many(bpa, R, N, hi, P, spare):
    rng = np.random.default_rng(R)
    c = state_of(rng, rng.integers(0, hi, R), P, spare, N)
    src, dst = rng.integers(0, R, N), R + rng.permutation(N)
    got, ws = run_fork(bpa, src, dst, c)
    bpa.bpa_check(ws)
    want = ora.fork(src, dst, **c)
    same(got, want)
    c = dict(ctx=want[2], table=want[3], refs=want[4], free=c["free"], count=want[5], P=P)
    # some go on, some are over, some are cut: at a page's end, or inside one of their own
    keep = np.array(c["ctx"])
    for r in range(R + N):
        kind = int(rng.integers(0, 4))
        if kind == 1:
            keep[r] = 0
        elif kind == 2:
            keep[r] = keep[r] // P * int(rng.integers(0, 2)) * P
        elif kind == 3 and keep[r] % P:
            keep[r] -= int(rng.integers(0, keep[r] % P))
    got, ws = run_release(bpa, keep, c, in_place=R % 2 == 0)
    bpa.bpa_check(ws)
    same(got, ora.release(c["ctx"], keep, c["table"], c["refs"], c["free"], c["count"], P))


def test_release_small_and_large_pools(bpa):
    for num_spare, ctx, keep in ((0, [5], [0]), (0, [5], [5]), (3, [0, 17, 33], [0, 16, 1]), (300000, [100, 50], [33, 0]), (7, [16, 32], [0, 0])):
        c = state_of(np.random.default_rng(2), ctx, 16, num_spare)
        got, ws = run_release(bpa, keep, c)
        bpa.bpa_check(ws)
        same(got, ora.release(c["ctx"], keep, c["table"], c["refs"], c["free"], c["count"], 16))


def test_pages_given_up_by_all_of_their_holders_at_once(bpa):
    c = state_of(np.random.default_rng(3), [64, 40], 16, 4, 5)
    a = ora.fork([0, 0, 1, 0], [2, 3, 4, 5], **c)
    c = dict(ctx=a[2], table=a[3], refs=a[4], free=c["free"], count=a[5], P=16)
    keep = np.zeros(7, int)
    got, ws = run_release(bpa, keep, c)
    bpa.bpa_check(ws)
    same(got, ora.release(c["ctx"], keep, c["table"], c["refs"], c["free"], c["count"], 16))
    assert (got[1] == 0).all() and got[3] == len(c["free"])


@pytest.mark.parametrize("src,dst", [([0, 9], [4, 5]), ([0, -1], [4, 5]), ([0, 1], [4, 9]), ([0, 1], [4, -2]), ([0, 1], [4, 2]), ([0, 0, 0], [4, 5, 5]),
                                     ([0, 4], [4, 5]), ([0, 3], [4, 5])])
def test_fork_reports_and_does_not_grant(bpa, src, dst):
    c = state_of(np.random.default_rng(4), [40, 33, 20, 5], 16, 6, 3)
    c["ctx"] = c["ctx"].copy()
    c["ctx"][3] = 10 ** 6                            # does not fit the table
    got, ws = run_fork(bpa, src, dst, c)
    with pytest.raises(bpa.BpaError):
        bpa.bpa_check(ws)
    fine = [(s, d) for s, d in zip(src, dst) if 0 <= s < 3 and 4 <= d < 7 and dst.count(d) == 1 and s not in dst]
    want = ora.fork([s for s, _ in fine], [d for _, d in fine], **c)
    same(got[2:], want[2:])
    rest = [i for i, p in enumerate(zip(src, dst)) if p not in fine]
    assert (got[0][rest] == -1).all() and (got[1][rest] == -1).all()


def test_fork_reports_bad_ids(bpa):
    base = state_of(np.random.default_rng(5), [40, 33], 16, 6, 2)
    for where in ("table", "last", "free", "count"):
        c = {**base, "table": base["table"].copy(), "free": base["free"].copy()}
        if where == "table":
            c["table"][0, 0] = 10 ** 7
        elif where == "last":
            c["table"][0, 2] = -3
        elif where == "free":
            c["free"][c["count"] - 1] = 10 ** 7
        else:
            c["count"] = -4
        got, ws = run_fork(bpa, [0, 1], [2, 3], c)
        with pytest.raises(bpa.BpaError):
            bpa.bpa_check(ws)
        if where != "count":
            assert got[0][0] == (base["table"][0, 2] if where == "table" else -1) and got[0][1] == base["table"][1, 2]


def test_release_reports_and_keeps(bpa):
    base = state_of(np.random.default_rng(6), [40, 33, 64], 16, 6, 1)
    for r, keep in ((0, -1), (0, 41), (1, 10 ** 6), (2, -2 ** 31)):
        want_keep = [16, 0, 32, 0]
        bad = list(want_keep)
        bad[r] = keep
        got, ws = run_release(bpa, bad, base)
        with pytest.raises(bpa.BpaError):
            bpa.bpa_check(ws)
        want_keep[r] = base["ctx"][r]
        same(got, ora.release(base["ctx"], want_keep, base["table"], base["refs"], base["free"], base["count"], 16))
    # a cut inside a page that others hold
    a = ora.fork([2], [3], **base)
    c = dict(ctx=a[2], table=a[3], refs=a[4], free=base["free"], count=a[5], P=16)
    got, ws = run_release(bpa, [40, 0, 17, 64], c)
    with pytest.raises(bpa.BpaError):
        bpa.bpa_check(ws)
    same(got, ora.release(c["ctx"], [40, 0, 64, 64], c["table"], c["refs"], c["free"], c["count"], 16))
    # a bad id, a page given up too often, a count that leaves no room
    c = {**base, "table": base["table"].copy()}
    c["table"][1, 0], c["table"][0, 1] = 10 ** 8, c["table"][0, 2]
    got, ws = run_release(bpa, [0, 0, 64, 0], c)
    with pytest.raises(bpa.BpaError):
        bpa.bpa_check(ws)
    freed = sorted({base["table"][0, 0], base["table"][0, 2], base["table"][1, 1], base["table"][1, 2]})
    n = base["count"]
    assert got[3] == n + 4 and got[2][n:n + 4].tolist() == freed and (got[1] == 0).all()
    got, ws = run_release(bpa, [0, 0, 64, 0], {**base, "count": len(base["free"]) - 2})
    with pytest.raises(bpa.BpaError):
        bpa.bpa_check(ws)
    assert got[3] == len(base["free"])


@pytest.mark.parametrize("nhd", [False, True], ids=["hnd", "nhd"])
@pytest.mark.parametrize("shape", [(12, 2, 16, 64, 64), (9, 3, 5, 33, 7), (30, 8, 64, 128, 64), (6, 1, 1024, 512, 16), (8, 1, 1, 1, 1)])
def test_copy(bpa, shape, nhd):
    pages, Hkv, P, d, dv = shape
    rng = np.random.default_rng(pages)
    kc, ks = random_cache(rng, pages, Hkv, P, d)
    vc, vs = random_cache(rng, pages, Hkv, P, dv)
    kc[0, 0, 0, 0] = 0x7F
    ids = rng.permutation(pages)
    src, dst = np.array([ids[0], -1, ids[1], ids[0]]), np.array([ids[2], -1, ids[3], ids[4]])
    t = [torch.from_numpy(x).cuda() for x in (kc, vc, ks, vs)]
    if nhd:
        t[:2] = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in t[:2]]
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    bpa.bpa_cache_copy(i32(src), i32(dst), *t, workspace_buf=ws)
    torch.cuda.synchronize()
    bpa.bpa_check(ws)
    for x in (kc, vc, ks, vs):
        x[dst[[0, 2, 3]]] = x[src[[0, 2, 3]]]
    same([x.cpu().numpy() for x in t], (kc, vc, ks, vs))
    for a, b in (([0, pages], [1, 2]), ([0, 1], [2, -1]), ([-1, 0], [1, 2]), ([0, 2 ** 31 - 1], [1, 1]), ([0, -2], [1, -2])):
        got = [x.clone() for x in t]
        bpa.bpa_cache_copy(i32(a), i32(b), *got, workspace_buf=ws)
        torch.cuda.synchronize()
        with pytest.raises(bpa.BpaError):
            bpa.bpa_check(ws)
        want = [x.clone() for x in t]
        for x, y in zip(a, b):
            if 0 <= x < pages and 0 <= y < pages:
                for w in want:
                    w[y] = w[x]
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    bpa.bpa_cache_copy(i32([]), i32([]), *t, workspace_buf=ws)
    torch.cuda.synchronize()
    bpa.bpa_check(ws)


def test_forked_requests_go_on_by_themselves(bpa):
    """A prompt forked twice; all three append other tokens and attend; then they end: plan, append, attention, fork,
    copy and release together, pages and outputs against the definitions."""
    rng = np.random.default_rng(7)
    R, Hq, Hkv, d, P, num = 4, 4, 2, 64, 16, 20
    c = make_step(rng, [41], [1], Hq, Hkv, d, d, P)
    pages = c["kc"].shape[0]
    kc, vc = np.zeros((num, Hkv, P, d), np.uint8), np.zeros((num, Hkv, P, d), np.uint8)
    ks, vs = np.zeros((num, Hkv), np.float32), np.zeros((num, Hkv), np.float32)
    kc[:pages], vc[:pages], ks[:pages], vs[:pages] = c["kc"], c["vc"], c["ks"], c["vs"]
    table, ctx, refs = np.full((R, 5), -1), np.array([42, 0, 0, 0]), np.zeros(num, int)
    table[0, :3] = c["table"][0]
    rest = [i for i in rng.permutation(num) if i not in table[0, :3]]
    free, count = np.array(rest + [0] * 3), len(rest)
    dt, dctx, drefs, dfree, dcount = i32(table), i32(ctx), i32(refs), i32(free), i32([count])
    cache = [torch.from_numpy(x).cuda() for x in (kc, vc, ks, vs)]
    a, b, _, _ = bpa.bpa_cache_fork(i32([0, 0]), i32([3, 1]), dctx, dt, drefs, dfree, dcount, page_size=P, ctx_lens_out=dctx,
                                    free_count_out=dcount)
    bpa.bpa_cache_copy(a, b, *cache)
    src, dst, ctx, table, refs, count = ora.fork([0, 0], [3, 1], ctx, table, refs, free, count, P)
    for x in (kc, vc, ks, vs):
        x[dst] = x[src]
    for _ in range(3):
        new, T = np.array([3, 4, 0, 1]), 8
        q, k, v = (torch.randn(T, h, d, device="cuda").bfloat16() for h in (Hq, Hkv, Hkv))
        kv, cu, slots, *_ = bpa.bpa_cache_plan(dctx, i32(new), dt, dfree, dcount, page_size=P, T=T, ctx_lens_out=dctx, free_count_out=dcount)
        bpa.bpa_cache_append(k, v, slots, *cache, max_new=4)
        o, m, l = bpa.bpa_cache_attn(q, *cache, dt, kv, cu, max_q=4)
        wkv, wcu, wslots, _, ctx, table, count = ora.plan(ctx, new, table, free, count, P, T)
        kc, ks = ora.append(k.double().cpu().numpy(), wslots, kc, ks)
        vc, vs = ora.append(v.double().cpu().numpy(), wslots, vc, vs)
        torch.cuda.synchronize()
        same([x.cpu().numpy() for x in (*cache, dt, dctx)], (kc, vc, ks, vs, table, ctx))
        check_attention(dict(q=q.double().cpu().numpy(), kc=kc, vc=vc, ks=ks, vs=vs, table=table, kv=wkv, cu=wcu), torch.bfloat16, o, m, l)
    for keep in ([ctx[0], 0, 0, ctx[3]], [0, 0, 0, 32], [0, 0, 0, 0]):
        bpa.bpa_cache_release(dctx, i32(keep), dt, drefs, dfree, dcount, page_size=P, ctx_lens_out=dctx, free_count_out=dcount)
        ctx, refs, free, count = ora.release(ctx, keep, table, refs, free, count, P)
        torch.cuda.synchronize()
        same([x.cpu().numpy() for x in (dctx, drefs, dfree, dcount)], (ctx, refs, free, [count]))
    assert count == num and sorted(free.tolist()) == list(range(num))


def test_fork_copy_and_release_in_a_captured_graph(bpa):
    """A prompt sampled twice and both samples over, again and again in place: the pages come back each time."""
    rng = np.random.default_rng(8)
    P = 16
    c = state_of(rng, [41], P, 6, 2)
    kc, ks = random_cache(rng, len(c["free"]), 2, P, 32)
    t = [torch.from_numpy(x).cuda() for x in (kc, kc, ks, ks)]
    ctx, table, refs, free, count = i32(c["ctx"]), i32(c["table"]), i32(c["refs"]), i32(c["free"]), i32([c["count"]])
    src, dst, keep = i32([0, 0]), i32([1, 2]), i32([41, 0, 0])

    def step():
        a, b, after, _ = bpa.bpa_cache_fork(src, dst, ctx, table, refs, free, count, page_size=P, free_count_out=count)
        bpa.bpa_cache_copy(a, b, *t)
        bpa.bpa_cache_release(after, keep, table, refs, free, count, page_size=P, free_count_out=count)
        return a, b, after

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    state = dict(c)
    for _ in range(5):
        a, b, after, tab, r, left = ora.fork([0, 0], [1, 2], **state)
        for x in (kc, ks):
            x[b] = x[a]
        _, r, f, left = ora.release(after, [41, 0, 0], tab, r, state["free"], left, P)
        state = dict(state, table=tab, refs=r, free=f, count=left)
    same([x.cpu().numpy() for x in (*outs, table, refs, free, count)], (a, b, after, state["table"], state["refs"], state["free"], [state["count"]]))
    same([x.cpu().numpy() for x in t], (kc, kc, ks, ks))
