"""GPU parity of the paged 8-bit cache (plan, append, attention) against its 64-bit definitions.

Plans and appended codes and scales are whole numbers and powers of two: they must be equal.
Attention is compared element by element with a tolerance from arithmetic (``check_attention``):
with A = sum p |v| / l (the same attention over |v|) and Z = the largest sum_c |q_c k_c| * scale,
  * scores: exact products summed in float32 over d terms, at most d + 4 steps of 2^-23 of the
    partial sums (the tensor cores truncate): dz = (d + 4) 2^-23 Z, plus 2^-21 for the exponential;
  * each weight moves by dz relatively, in the numerator and in the denominator, and is rounded to
    16 bits for the product with v: half a bf16 step, 2^-8 (float32 paths keep two halves: 2^-21);
  * sums over n keys in float32: n 2^-23;
  * weights are fp16 numbers with the row's largest (weight times v scale, H) at 2^9 or more: fp16's
    smallest step is 2^-24, so each of the n weights is off by at most 2^-25 = 2^-34 of the largest,
    whatever its own size, times |v| <= 448: n 2^-34 448 H;
  * the output is rounded once: 2^-8 |o| in bf16, 2^-24 |o| in float32.
"""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import cache as ora

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bpa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from ring_attention_gb300 import build
    build.build()
    from ring_attention_gb300 import bpa as mod
    return mod


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().double().cpu().numpy()


# ---- plan ------------------------------------------------------------------------------------------
def make_plan(rng, ctx, new, P, spare, pad=0):
    ctx, new = np.asarray(ctx), np.asarray(new)
    have, total = -(-ctx // P), -(-(ctx + new) // P)
    num = max(1, int(total.sum()) + max(spare, -int((total - have).sum())))
    ids = rng.permutation(num)
    table = np.full((len(ctx), max(1, int(total.max()) + 1)), -1)
    at = 0
    for r, n in enumerate(have):
        table[r, :n] = ids[at:at + n]
        at += n
    free = np.zeros(num, int)
    free[:num - at] = ids[at:]
    return dict(ctx=ctx, new=new, table=table, free=free, count=num - at, P=P, T=int(new.sum()) + pad)


def run_plan(bpa, c, **kw):
    table = i32(c["table"])
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")     # stale: the call clears it
    got = bpa.bpa_cache_plan(i32(c["ctx"]), i32(c["new"]), table, i32(c["free"]), i32([c["count"]]), page_size=c["P"],
                             T=c["T"], workspace_buf=ws, **kw)
    torch.cuda.synchronize()
    kv, cu, slots, pos, ctx, left = (t.cpu().numpy() for t in got)
    return (kv, cu, slots, pos, ctx, table.cpu().numpy(), int(left[0])), ws


def check_plan(bpa, c):
    got, ws = run_plan(bpa, c)
    bpa.bpa_check(ws)
    for g, w, name in zip(got, ora.plan(**c), ("kv_lens", "cu_q", "slots", "positions", "ctx", "table", "count")):
        np.testing.assert_array_equal(g, w, err_msg=name)


PLANS = {
    "one": ([0], [1], 16, 0, 0), "one_idle": ([5], [0], 16, 3, 0), "page_full": ([16], [1], 16, 1, 0),
    "page_exact": ([15], [1], 16, 0, 2), "empty_rows": ([0, 0, 7], [0, 3, 0], 4, 2, 5),
    "page_of_one": ([2, 0, 9], [4, 1, 2], 1, 0, 1), "odd_page": ([2, 50, 9], [40, 1, 22], 7, 3, 0),
    "no_pages_left": ([3, 4, 0], [1, 1, 1], 4, -9, 0),     # only the first has room in its page
}


@pytest.mark.parametrize("name", PLANS)
def test_plan_small(bpa, name):
    check_plan(bpa, make_plan(np.random.default_rng(1), *PLANS[name]))


@pytest.mark.parametrize("R,hi,P,spare,pad", [(256, 1, 64, 10, 0), (1500, 4, 16, -100, 77), (61, 700, 16, 5, 100),
                                              (33, 900, 64, -40, 0), (8192, 2, 32, 0, 3)])
def test_plan_ragged(bpa, R, hi, P, spare, pad):
    rng = np.random.default_rng(R)
    check_plan(bpa, make_plan(rng, rng.integers(0, 500, R), rng.integers(0, hi + 1, R), P, spare, pad))


def test_plan_advances_in_place_under_a_graph(bpa):
    c = make_plan(np.random.default_rng(3), [0, 14, 31], [1, 1, 1], 16, 12)
    c["table"] = np.concatenate([c["table"], np.full((3, 4), -1)], 1)
    ctx, new, table, free, count = i32(c["ctx"]), i32(c["new"]), i32(c["table"]), i32(c["free"]), i32([c["count"]])
    kw = dict(page_size=16, T=3, ctx_lens_out=ctx, free_count_out=count)
    state = (c["ctx"], c["table"], c["count"])
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        outs = bpa.bpa_cache_plan(ctx, new, table, free, count, **kw)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs = bpa.bpa_cache_plan(ctx, new, table, free, count, **kw)
        for _ in range(4):
            g.replay()
    torch.cuda.synchronize()
    for _ in range(5):
        kv, cu, slots, pos, *rest = ora.plan(state[0], c["new"], state[1], c["free"], state[2], 16, 3)
        state = rest
    for got, want in zip(outs[:4] + (ctx, table, count), (kv, cu, slots, pos) + tuple(state)):
        np.testing.assert_array_equal(got.cpu().numpy().reshape(np.shape(want)), want)


def test_plan_reports_bad_inputs(bpa):
    base = make_plan(np.random.default_rng(4), [4, 9, 3], [2, 3, 1], 4, 3)
    good = ora.plan(**base)
    for field, r, value in (("ctx", 1, -3), ("new", 1, -1), ("new", 1, 4000)):
        c = {**base, field: np.array(base[field])}
        c[field][r] = value
        got, ws = run_plan(bpa, c)
        with pytest.raises(bpa.BpaError):
            bpa.bpa_check(ws)
        assert got[0][1] == 0 and got[4][1] == c["ctx"][1]       # the request waits
        assert got[0][0] == good[0][0]                           # the one before it does not
        np.testing.assert_array_equal(got[2][:2], good[2][:2])
    for T in (5, 4):                                             # too few rows: the last request waits
        got, ws = run_plan(bpa, {**base, "T": T})
        with pytest.raises(bpa.BpaError):
            bpa.bpa_check(ws)
        assert got[0][2] == 0 and got[1].max() <= T
    c = {**base, "free": np.full_like(base["free"], 10 ** 6)}
    got, ws = run_plan(bpa, c)
    with pytest.raises(bpa.BpaError):
        bpa.bpa_check(ws)
    assert got[5].max() < len(c["free"]) and got[2].max() < 4 * len(c["free"])


@pytest.mark.parametrize("R", [33, 1000, 1024, 2500])
def test_plan_reports_a_bad_length_anywhere(bpa, R):
    base = make_plan(np.random.default_rng(5), [3] * R, [1] * R, 4, R)
    for r in sorted({0, 31, R // 2, R - 1}):
        c = {**base, "ctx": np.array(base["ctx"])}
        c["ctx"][r] = -1
        for _ in range(10):
            got, ws = run_plan(bpa, c)
            with pytest.raises(bpa.BpaError):
                bpa.bpa_check(ws)
            assert got[0][r] == 0 and (got[0] > 0).sum() == R - 1


# ---- append ----------------------------------------------------------------------------------------
def random_cache(rng, pages, Hkv, P, c, spread=1.0):
    """Codes with the values +-[0, 448] and power-of-two scales, as append leaves them."""
    codes = rng.integers(0, 256, (pages, Hkv, P, c)).astype(np.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0
    x = rng.standard_normal((pages, Hkv, P, c))
    scale = np.exp2(np.round(rng.standard_normal((pages, Hkv)) * spread) - 7)
    codes = ora.e4m3_round(np.clip(x / scale[:, :, None, None], -448, 448))
    return codes, scale.astype(np.float32)


def slots_for(rng, ctx, new, P, pages):
    """(slots, table) of requests with pages of their own."""
    ids = rng.permutation(pages)
    width = max(1, max(-(-(a + b) // P) for a, b in zip(ctx, new)))
    table, at, slots = np.full((len(ctx), width), -1), 0, []
    for r, (a, b) in enumerate(zip(ctx, new)):
        n = -(-(a + b) // P)
        table[r, :n] = ids[at:at + n]
        at += n
        slots += [table[r, p // P] * P + p % P for p in range(a, a + b)]
    return np.array(slots, np.int64), table


def as_dtype(x, dtype):
    t = torch.from_numpy(np.asarray(x, np.float32)).to(dtype)
    return t.cuda(), t.double().numpy()


def run_append(bpa, k, v, slots, kc, vc, ks, vs, max_new=0, nhd=False):
    dk, dvv = (torch.from_numpy(c).cuda() for c in (kc, vc))
    if nhd:
        dk, dvv = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (dk, dvv))
    sk, sv = (torch.from_numpy(c).cuda() for c in (ks, vs))
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    bpa.bpa_cache_append(k, v, i32(slots), dk, dvv, sk, sv, max_new=max_new, workspace_buf=ws)
    torch.cuda.synchronize()
    return (dk.cpu().numpy(), sk.cpu().numpy(), dvv.cpu().numpy(), sv.cpu().numpy()), ws


def check_append(bpa, rng, ctx, new, Hkv, d, dv, P, dtype, *, mag=1.0, nhd=False, strided=False, max_new=None, pad=0):
    pages = sum(-(-(a + b) // P) for a, b in zip(ctx, new)) + 3
    slots, _ = slots_for(rng, ctx, new, P, pages)
    slots = np.concatenate([slots, np.full(pad, -1)])
    T = len(slots)
    kc, ks = random_cache(rng, pages, Hkv, P, d)
    vc, vs = random_cache(rng, pages, Hkv, P, dv)
    mags = np.exp2(rng.integers(-3, 4, (T, 1, 1))) * mag
    tk, xk = as_dtype(rng.standard_normal((T, Hkv, d)) * mags, dtype)
    tv, xv = as_dtype(rng.standard_normal((T, Hkv, dv)) * mags, dtype)
    if strided:       # rows of a fused [T, Hkv, d + dv + 5] projection
        both = torch.zeros(T, Hkv, d + dv + 5, dtype=dtype, device="cuda")
        both[:, :, :d], both[:, :, d:d + dv] = tk, tv
        tk, tv = both[:, :, :d], both[:, :, d:d + dv]
    got, ws = run_append(bpa, tk, tv, slots, kc, vc, ks, vs, max(new) if max_new is None else max_new, nhd)
    bpa.bpa_check(ws)
    for x, c, s, gc, gs in ((xk, kc, ks, got[0], got[1]), (xv, vc, vs, got[2], got[3])):
        wc, wsc = ora.append(x, slots, c, s)
        np.testing.assert_array_equal(gs, wsc)
        np.testing.assert_array_equal(gc, wc)


APPENDS = [   # ctx, new, Hkv, d, dv, P
    ([0], [1], 1, 64, 64, 16), ([15], [1], 2, 128, 128, 16), ([16, 3], [1, 1], 8, 128, 64, 16),
    ([0, 5, 60, 130], [70, 1, 9, 64], 2, 128, 128, 64), ([7, 0, 31], [40, 33, 0], 2, 80, 80, 32),
    ([1, 2], [300, 5], 1, 256, 64, 128), ([3, 0], [11, 25], 3, 33, 7, 5), ([0, 2], [9, 3], 2, 1, 1, 1),
    ([100, 0], [3, 1000], 2, 64, 512, 256),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", APPENDS, ids=lambda c: f"d{c[3]}_{c[4]}_P{c[5]}_T{sum(c[1])}")
def test_append_equals_the_definition(bpa, case, dtype):
    ctx, new, Hkv, d, dv, P = case
    check_append(bpa, np.random.default_rng(d + P), ctx, new, Hkv, d, dv, P, dtype)


@pytest.mark.parametrize("kw", [dict(nhd=True), dict(strided=True), dict(max_new=0), dict(max_new=1), dict(pad=9),
                                dict(mag=1e-30), dict(mag=1e30)],
                         ids=["nhd", "strided", "unknown_max", "wrong_max", "padded", "tiny", "huge"])
@pytest.mark.parametrize("new", [[1, 1, 1, 1], [90, 1, 17, 64]], ids=["step", "prompt"])
def test_append_layouts(bpa, kw, new):
    check_append(bpa, np.random.default_rng(5), [9, 0, 130, 64], new, 2, 128, 64, 64, torch.bfloat16, **kw)


@pytest.mark.parametrize("rows", [1, 20])
def test_append_zeros_infinities_and_nan(bpa, rows):
    rng = np.random.default_rng(6)
    kc, ks = random_cache(rng, 4, 2, 16, 32)
    ks[1] = 0                                     # a page of zeros so far
    kc[1] = 0
    x = rng.standard_normal((rows, 2, 32)).astype(np.float32)
    x[0, 0, :3] = [np.inf, -np.inf, np.nan]
    x[:, 1] = 0                                   # head 1: nothing but zeros
    slots = np.concatenate([np.arange(16 + 5, 32), np.arange(48, 64)])[:rows]
    (gc, gs, vc, vs), ws = run_append(bpa, torch.from_numpy(x).cuda(), torch.from_numpy(x).cuda(), slots, kc, kc, ks, ks)
    wc, wsc = ora.append(x.astype(np.float64), slots, kc, ks)
    np.testing.assert_array_equal(gs, wsc)
    nan = (wc & 0x7F) == 0x7F
    np.testing.assert_array_equal((gc & 0x7F) == 0x7F, nan)
    np.testing.assert_array_equal(gc[~nan], wc[~nan])
    np.testing.assert_array_equal(vc, gc)
    assert gs[1, 1] == 0 and (gc[1, 0, 5, :3] & 0x7F == 0x7F).all()


def test_append_skips_and_reports(bpa):
    rng = np.random.default_rng(7)
    kc, ks = random_cache(rng, 4, 1, 16, 16)
    x = torch.randn(4, 1, 16, device="cuda")
    slots = [-1, 3, 64, 2 ** 30]                  # two behind the cache's end
    (gc, gs, *_), ws = run_append(bpa, x, x, slots, kc, kc, ks, ks)
    with pytest.raises(bpa.BpaError):
        bpa.bpa_check(ws)
    wc, wsc = ora.append(f64(x), [-1, 3, -1, -1], kc, ks)
    np.testing.assert_array_equal(gc, wc)
    np.testing.assert_array_equal(gs, wsc)
    (gc, *_), ws = run_append(bpa, x[:0], x[:0], [], kc, kc, ks, ks)
    bpa.bpa_check(ws)
    np.testing.assert_array_equal(gc, kc)


# ---- attention ---------------------------------------------------------------------------------------
def make_step(rng, ctx, new, Hq, Hkv, d, dv, P, pad=0, spread=1.0, qmag=1.0):
    pages = sum(-(-(a + b) // P) for a, b in zip(ctx, new)) + 2
    slots, table = slots_for(rng, ctx, new, P, pages)
    kc, ks = random_cache(rng, pages, Hkv, P, d, spread)
    vc, vs = random_cache(rng, pages, Hkv, P, dv, spread)
    for r, (a, b) in enumerate(zip(ctx, new)):    # behind the last token: stale rows, NaN among them
        if (a + b) % P:
            last = table[r, (a + b) // P]
            kc[last, :, (a + b) % P:] = 0x7F
            vc[last, :, (a + b) % P:] = 0x7F
    return dict(q=rng.standard_normal((len(slots) + pad, Hq, d)) * qmag, kc=kc, vc=vc, ks=ks, vs=vs, table=table,
                kv=np.add(ctx, new), cu=np.concatenate([[0], np.cumsum(new)]), max_q=max(new))


def on_gpu(c, dtype, nhd=False):
    k, v = torch.from_numpy(c["kc"]).cuda(), torch.from_numpy(c["vc"]).cuda()
    if nhd:
        k, v = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v))
    return (as_dtype(c["q"], dtype)[0], k, v, torch.from_numpy(c["ks"]).cuda(), torch.from_numpy(c["vs"]).cuda(),
            i32(c["table"]), i32(c["kv"]), i32(c["cu"]))


def check_attention(c, dtype, o, m, l, rows=None, **kw):
    q = as_dtype(c["q"], dtype)[1]
    args = (c["kc"], c["vc"] & 0x7F, c["ks"], c["vs"], c["table"], c["kv"], c["cu"])
    A, _, _, H = ora.attention(q, *args, heaviest=True, **kw)
    wo, wm, wl = ora.attention(q, c["kc"], c["vc"], *args[2:], **kw)
    d, n = q.shape[2], int(max(c["kv"].max(), 1))
    scale = kw.get("scale") or d ** -0.5
    val = np.nan_to_num(np.abs(ora.e4m3_values()[c["kc"]])) * c["ks"][:, :, None, None]
    Z = max(np.abs(q[:, h]).max(0, initial=0) @ val[:, h // (q.shape[1] // val.shape[1])].max((0, 1))
            for h in range(q.shape[1])) * scale
    dz = (d + 4) * 2.0 ** -23 * Z + 2.0 ** -21
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    weight = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -21
    valid = ~np.isnan(wl[0])
    go, gm, gl = f64(o)[valid], f64(m)[:, valid], f64(l)[:, valid]
    wo, A, wm, wl = wo[valid], A[valid], wm[:, valid], wl[:, valid]
    off = (2 * dz + weight + n * 2.0 ** -23) * A + n * 2.0 ** -34 * 448 * H[valid]
    bad = ~(np.abs(go - wo) <= half * np.abs(wo) + off * (1 + half))
    assert not bad.any(), f"{bad.sum()} of {bad.size} outputs, the first {go[bad][0]} for {wo[bad][0]}, A {A[bad][0]}"
    np.testing.assert_array_equal(np.isneginf(gm), np.isneginf(wm))
    fin = np.isfinite(wm)
    assert (np.abs(gm[fin] - wm[fin]) <= dz + 2.0 ** -22 * np.abs(wm[fin])).all()
    assert (np.abs(gl - wl) <= (2 * dz + n * 2.0 ** -23 + 2.0 ** -21) * wl).all()
    return valid


def run_and_check(bpa, c, dtype, nhd=False, **kw):
    sink = kw.get("sink")
    t = on_gpu(c, dtype, nhd)
    T, Hq = c["q"].shape[:2]
    marker = 77.0
    o = torch.full((T, Hq, c["vc"].shape[3]), marker, dtype=dtype, device="cuda")
    m, l = (torch.full((Hq, T), marker, device="cuda") for _ in range(2))
    dev = {**kw, "sink": None if sink is None else torch.from_numpy(sink.astype(np.float32)).cuda()}
    need = bpa.bpa_cache_attn_workspace_size(
        bpa.make_cache_desc(*t[1:5], dtype), bpa.make_cache_batch(t[0], *t[5:], max_q=c["max_q"], **dev))
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    bpa.bpa_cache_attn(*t, max_q=c["max_q"], o=o, m=m, l=l, workspace_buf=ws, **dev)
    torch.cuda.synchronize()
    bpa.bpa_check(ws)
    valid = check_attention(c, dtype, o, m, l, **kw)
    assert (o[~valid] == marker).all() and (m[:, ~valid] == marker).all() and (l[:, ~valid] == marker).all()
    return o, m, l


DTYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])

SHAPES = [   # ctx, new, Hq, Hkv, d, dv, P
    ([0], [1], 1, 1, 64, 64, 16), ([700], [1], 32, 8, 128, 128, 64), ([0, 1, 63, 64, 300], [1] * 5, 8, 2, 128, 128, 64),
    ([15, 16, 17, 511], [1] * 4, 8, 2, 64, 64, 16), ([40, 90], [1, 1], 16, 1, 128, 64, 32),
    ([130, 7], [1, 1], 7, 1, 80, 80, 16), ([260, 3], [1, 1], 6, 2, 192, 64, 128), ([300, 33], [1, 1], 4, 4, 256, 256, 16),
    ([100, 0, 31], [3, 8, 1], 8, 2, 128, 128, 16), ([20, 200], [6, 2], 64, 4, 64, 64, 64),
    ([90, 5], [1, 2], 3, 1, 33, 7, 5), ([9, 14], [1, 1], 2, 1, 512, 512, 8), ([50, 0], [1, 2], 2, 2, 96, 112, 48),
    ([0, 100, 37], [70, 40, 1], 4, 2, 128, 128, 64), ([64, 0], [33, 130], 8, 2, 64, 64, 32),
]


@DTYPES
@pytest.mark.parametrize("case", SHAPES, ids=lambda c: f"H{c[2]}_{c[3]}_d{c[4]}_{c[5]}_P{c[6]}_q{max(c[1])}")
def test_attention_matches_the_definition(bpa, case, dtype):
    run_and_check(bpa, make_step(np.random.default_rng(sum(case[0]) + case[4]), *case), dtype)


MANY = [     # ctx, new, Hq, Hkv, d, dv, P: enough requests of more than 64 rows for the kernel for many rows,
             # beside others of few; row tiles half full, one row too many, of one token
    ([0, 130, 37, 250], [70, 1, 33, 9], 32, 8, 128, 128, 64), ([300, 5, 64, 127, 1], [17, 20, 64, 1, 129], 32, 8, 128, 64, 32),
    ([90, 0, 15], [130, 40, 257], 32, 16, 64, 64, 16), ([40, 200], [30, 2], 96, 16, 80, 112, 128), ([0, 60], [40, 41], 112, 16, 96, 48, 64),
    ([600, 1], [5, 6], 256, 16, 64, 64, 16),
]


@pytest.mark.parametrize("case", MANY, ids=lambda c: f"H{c[2]}_{c[3]}_d{c[4]}_{c[5]}_P{c[6]}_q{max(c[1])}")
def test_attention_many_rows_beside_few(bpa, case):
    run_and_check(bpa, make_step(np.random.default_rng(sum(case[1]) + case[4]), *case, pad=3), torch.bfloat16)


@DTYPES
@pytest.mark.parametrize("window", [(-1, -1), (200, -1)], ids=["all", "window"])
@pytest.mark.parametrize("few", [False, True], ids=["many_items", "few_items"])
def test_attention_requests_of_one_to_eight_tokens(bpa, few, window, dtype):
    # items of one, two and four row tiles whose keys are cut between CTAs at any place
    rng = np.random.default_rng(30 + few)
    n = 2 if few else 24
    new = [8, 1] if few else [1 + i % 8 for i in range(n)]
    ctx = [int(x) for x in rng.integers(0, 1500, n)]
    run_and_check(bpa, make_step(rng, ctx, new, 16, 2, 64, 64, 16), dtype, window=window)


MASKS = {"window": dict(window=(20, -1)), "window_0": dict(window=(0, -1)), "not_causal": dict(causal=False),
         "band": dict(causal=False, window=(10, 5)), "right": dict(causal=False, window=(-1, 0)),
         "scale": dict(scale=0.3), "wide": dict(window=(2 ** 31 - 1, 2 ** 31 - 1), causal=False)}


@DTYPES
@pytest.mark.parametrize("new", [[1, 1, 1], [5, 1, 0], [100, 3, 17]], ids=["step", "draft", "prompt"])
@pytest.mark.parametrize("mask", MASKS)
def test_attention_masks(bpa, mask, new, dtype):
    c = make_step(np.random.default_rng(8), [200, 0, 63], new, 8, 2, 64, 64, 16, pad=2)
    run_and_check(bpa, c, dtype, **MASKS[mask])


@pytest.mark.parametrize("mask", MASKS)
def test_attention_masks_many_rows(bpa, mask):
    c = make_step(np.random.default_rng(20), [200, 0, 63, 140], [40, 65, 3, 20], 64, 16, 64, 64, 16, pad=2)
    run_and_check(bpa, c, torch.bfloat16, **MASKS[mask])


def test_attention_many_rows_sinks_scales_and_ranges(bpa):
    rng = np.random.default_rng(21)
    sink = rng.standard_normal(64) * 3
    for qmag in (1e-6, 1.0, 30.0, 1e4):
        c = make_step(rng, [90, 0, 30, 1], [40, 20, 33, 50], 64, 16, 128, 128, 32, pad=3, qmag=qmag)
        c["kv"] = c["kv"].copy()
        c["kv"][1] = 0                            # a request that waits
        run_and_check(bpa, c, torch.bfloat16, sink=sink)
        c["kv"][0] = 5                            # fewer keys than rows
        run_and_check(bpa, c, torch.bfloat16, sink=sink)
        run_and_check(bpa, c, torch.bfloat16)
    c = make_step(rng, [150, 70], [60, 40], 64, 16, 64, 64, 16)
    c["vs"][:] = np.exp2(rng.integers(-30, 30, c["vs"].shape) - 7.0).astype(np.float32)
    for page in (c["table"][0, 0], c["table"][0, 2], c["table"][1, 1]):
        c["vs"][page] = 0
        c["vc"][page] = 0
    run_and_check(bpa, c, torch.bfloat16)
    run_and_check(bpa, c, torch.bfloat16, window=(3, -1))


@pytest.mark.parametrize("new", [[1, 1, 2], [40, 20, 33]], ids=["step", "prompt"])
@DTYPES
def test_attention_sink_of_minus_infinity_is_none(bpa, new, dtype):
    c = make_step(np.random.default_rng(26), [90, 0, 30], new, 32, 16, 64, 64, 16)
    c["kv"] = c["kv"].copy()
    c["kv"][1] = 0
    t = on_gpu(c, dtype)
    sink = torch.full((32,), -np.inf, device="cuda")
    for a, b in zip(bpa.bpa_cache_attn(*t, max_q=max(new), sink=sink), bpa.bpa_cache_attn(*t, max_q=max(new))):
        assert torch.equal(a, b)


def test_attention_of_no_rows(bpa):
    c = make_step(np.random.default_rng(27), [20, 3], [1, 1], 4, 2, 64, 64, 16)
    t = list(on_gpu(c, torch.bfloat16))
    t[0], t[7] = t[0][:0], torch.zeros_like(t[7])
    o, m, l = bpa.bpa_cache_attn(*t)
    assert o.shape == (0, 4, 64) and m.shape == (4, 0)
    t[0] = torch.zeros(5, 4, 64, dtype=torch.bfloat16, device="cuda")       # a padded batch of padding alone
    o = torch.full((5, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    bpa.bpa_cache_attn(*t, o=o)
    torch.cuda.synchronize()
    assert (o == 7).all()


def test_attention_without_statistics(bpa):
    c = make_step(np.random.default_rng(22), [90, 700, 30], [40, 1, 33], 32, 16, 128, 128, 32)
    for dtype in (torch.bfloat16, torch.float32):
        t = on_gpu(c, dtype)
        o, m, l = bpa.bpa_cache_attn(*t, max_q=40)
        got = torch.zeros_like(o)
        D, B = bpa.make_cache_desc(*t[1:5], dtype), bpa.make_cache_batch(t[0], *t[5:], max_q=40)
        B.o_strides[:] = o.stride()[:2]
        ws = torch.empty(bpa.bpa_cache_attn_workspace_size(D, B), dtype=torch.uint8, device="cuda")
        st = bpa.lib().bpa_cache_attn(ctypes.byref(D), ctypes.byref(B), got.data_ptr(), None, None, ws.data_ptr(),
                                      ws.numel(), torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert st == 0 and torch.equal(got, o)


@pytest.mark.parametrize("max_q", [0, 1, 10 ** 6], ids=["unknown", "too_small", "too_large"])
def test_attention_any_max_q(bpa, max_q):
    c = make_step(np.random.default_rng(23), [90, 0, 30, 5], [40, 1, 70, 0], 32, 16, 64, 64, 32)
    t = on_gpu(c, torch.bfloat16)
    o, m, l = bpa.bpa_cache_attn(*t, max_q=max_q)
    torch.cuda.synchronize()
    check_attention(c, torch.bfloat16, o, m, l)


def test_attention_one_token_of_many_heads(bpa):
    # 128 rows of one token, one kv head: the keys are shared out between CTAs all the same
    run_and_check(bpa, make_step(np.random.default_rng(24), [1500], [1], 128, 1, 128, 64, 64), torch.bfloat16)
    run_and_check(bpa, make_step(np.random.default_rng(25), [700, 3], [2, 1], 130, 1, 64, 64, 16), torch.float32)


@DTYPES
@pytest.mark.parametrize("new", [[1, 1, 1], [40, 3, 0]], ids=["step", "prompt"])
def test_attention_sink_and_empty_rows(bpa, new, dtype):
    rng = np.random.default_rng(9)
    for sink in (None, rng.standard_normal(4) * 3):
        c = make_step(rng, [90, 0, 30], new, 4, 2, 128, 128, 32, pad=3)
        c["kv"] = c["kv"].copy()
        c["kv"][1] = 0                            # a request that waits: its rows have no keys
        run_and_check(bpa, c, dtype, sink=sink)
        c["kv"][0] = min(5, new[0])               # fewer keys than rows: the first rows have none
        run_and_check(bpa, c, dtype, sink=sink)


@DTYPES
@pytest.mark.parametrize("new", [[1, 1], [60, 2]], ids=["step", "prompt"])
def test_attention_page_scales_far_apart(bpa, new, dtype):
    # scales from 2^-37 to 2^23 within a request; a page of zeros has scale 0
    c = make_step(np.random.default_rng(10), [150, 70], new, 4, 2, 64, 64, 16)
    c["ks"][:] = 2.0 ** -7
    c["vs"][:] = np.exp2(np.random.default_rng(11).integers(-30, 30, c["vs"].shape) - 7.0).astype(np.float32)
    c["vs"][c["table"][0, 2]] = 0
    c["vc"][c["table"][0, 2]] = 0
    run_and_check(bpa, c, dtype)
    # and the rows of one that is far below the others, alone behind a window
    run_and_check(bpa, c, dtype, window=(3, -1))


@DTYPES
@pytest.mark.parametrize("qmag", [1e-6, 30.0, 1e4], ids=str)
def test_attention_score_ranges(bpa, qmag, dtype):
    run_and_check(bpa, make_step(np.random.default_rng(12), [200, 65], [1, 2], 8, 2, 128, 128, 64, qmag=qmag), dtype)


@pytest.mark.parametrize("new", [[1, 1], [100, 30]], ids=["step", "prompt"])
def test_attention_layouts(bpa, new):
    c = make_step(np.random.default_rng(13), [130, 31], new, 8, 2, 128, 64, 64)
    want = run_and_check(bpa, c, torch.bfloat16)
    got = run_and_check(bpa, c, torch.bfloat16, nhd=True)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # q and o as slices of wider rows; k and v interleaved in one allocation
    t = on_gpu(c, torch.bfloat16)
    T = c["q"].shape[0]
    wide = torch.zeros(T, 8, 128 + 8, dtype=torch.bfloat16, device="cuda")
    wide[:, :, :128] = t[0]
    kv = torch.zeros(t[1].shape[0], 2, 64, 2 * 128, dtype=torch.uint8, device="cuda")
    kv[..., :128], kv[..., 128:192] = t[1], t[2]
    out = torch.zeros(T, 8, 72, dtype=torch.bfloat16, device="cuda")
    o, m, l = bpa.bpa_cache_attn(wide[:, :, :128], kv[..., :128], kv[..., 128:192], *t[3:], max_q=c["max_q"],
                                 o=out[:, :, :64])
    torch.cuda.synchronize()
    for a, b in zip((o, m, l), want):
        assert torch.equal(a, b)
    assert not out[:, :, 64:].any()


def test_attention_odd_strides_and_bases(bpa):
    # a cache whose rows start at odd bytes, q and o at odd elements: another path, the same answer
    c = make_step(np.random.default_rng(14), [130, 31], [2, 1], 4, 2, 64, 64, 16)
    t = on_gpu(c, torch.bfloat16)
    k = torch.zeros(t[1].shape[:3] + (65,), dtype=torch.uint8, device="cuda")
    k[..., 1:] = t[1]
    q = torch.zeros(t[0].shape[:2] + (65,), dtype=torch.bfloat16, device="cuda")
    q[..., 1:] = t[0]
    out = torch.zeros(t[0].shape[:2] + (65,), dtype=torch.bfloat16, device="cuda")
    o, m, l = bpa.bpa_cache_attn(q[..., 1:], k[..., 1:], *t[2:], max_q=2, o=out[..., 1:])
    torch.cuda.synchronize()
    check_attention(c, torch.bfloat16, o, m, l)


@pytest.mark.parametrize("new", [[1, 1], [40, 30]], ids=["step", "prompt"])
def test_attention_reports_bad_pages_and_lengths(bpa, new):
    rng = np.random.default_rng(15)
    for bad in (-1, 10 ** 6, "len"):
        c = make_step(rng, [130, 31], new, 4, 2, 64, 64, 16)
        good = c["table"].copy()
        if bad == "len":
            c["kv"] = c["kv"].copy()
            c["kv"][0] = 10 ** 6
        else:
            c["table"][0, 3] = bad
        t = on_gpu(c, torch.bfloat16)
        need = bpa.bpa_cache_attn_workspace_size(bpa.make_cache_desc(*t[1:5], torch.bfloat16),
                                                 bpa.make_cache_batch(t[0], *t[5:], max_q=max(new)))
        ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
        o, m, l = bpa.bpa_cache_attn(*t, max_q=max(new), workspace_buf=ws)
        torch.cuda.synchronize()
        with pytest.raises(bpa.BpaError):
            bpa.bpa_check(ws)
        # the other request is not touched by it
        c["table"], c["kv"] = good, np.add([130, 31], new)
        rows = slice(new[0], None)
        other = {**c, "q": c["q"][rows], "table": c["table"][1:], "kv": c["kv"][1:], "cu": c["cu"][1:] - new[0]}
        check_attention(other, torch.bfloat16, o[rows], m[:, rows], l[:, rows])


@pytest.mark.parametrize("bad", [-1, -2 ** 31, 10 ** 6, 2 ** 31 - 1])
@pytest.mark.parametrize("new", [[1] * 4, [70] * 4], ids=["step", "prompt"])
def test_attention_reports_bad_pages_of_every_kernel(bpa, new, bad):
    c = make_step(np.random.default_rng(16), [130, 31, 0, 63], new, 32, 8, 64, 64, 16)
    c["table"][3, 2] = bad
    t = on_gpu(c, torch.bfloat16)
    need = bpa.bpa_cache_attn_workspace_size(bpa.make_cache_desc(*t[1:5], torch.bfloat16),
                                             bpa.make_cache_batch(t[0], *t[5:], max_q=max(new)))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    o, m, l = bpa.bpa_cache_attn(*t, max_q=max(new), workspace_buf=ws)
    torch.cuda.synchronize()
    with pytest.raises(bpa.BpaError):
        bpa.bpa_check(ws)
    first = {**c, "q": c["q"][:sum(new[:3])], "table": c["table"][:3], "kv": c["kv"][:3], "cu": c["cu"][:4]}
    rows = slice(0, sum(new[:3]))
    check_attention(first, torch.bfloat16, o[rows], m[:, rows], l[:, rows])


def test_attention_cache_past_32_bits(bpa):
    # 5 GB of keys: pages whose bytes lie past 2^32
    c = make_step(np.random.default_rng(16), [600, 100], [1, 3], 4, 2, 128, 64, 64)
    t = on_gpu(c, torch.bfloat16)
    num = (5 << 30) // (2 * 64 * 128)
    ids = torch.randperm(num - 270000, device="cuda")[:t[1].shape[0]] + 270000
    big = [torch.empty(num, 2, 64, x.shape[3], dtype=torch.uint8, device="cuda") for x in t[1:3]]
    scales = [torch.zeros(num, 2, device="cuda") for _ in range(2)]
    for dst, src in zip(big + scales, t[1:5]):
        dst[ids] = src
    table = torch.where(t[5] >= 0, ids[t[5].long().clamp(min=0)].int(), t[5]).contiguous()
    assert int(ids.min()) * 2 * 64 * 128 > 1 << 32
    o, m, l = bpa.bpa_cache_attn(t[0], *big, *scales, table, *t[6:], max_q=3)
    torch.cuda.synchronize()
    check_attention(c, torch.bfloat16, o, m, l)


def test_attention_long_contexts_against_bpa_fwd(bpa):
    # codes times power-of-two scales are exact in bf16: the same attention without a cache
    g = torch.Generator(device="cuda").manual_seed(17)
    S, Hq, Hkv, d, P = 2048, 8, 2, 128, 64
    k, v = (torch.randn(1, S, Hkv, d, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    q = torch.randn(1, S, Hq, d, generator=g, device="cuda", dtype=torch.bfloat16)
    kc, vc = (torch.zeros(S // P + 1, Hkv, P, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(S // P + 1, Hkv, device="cuda") for _ in range(2))
    bpa.bpa_cache_append(k[0], v[0], torch.arange(S, dtype=torch.int32, device="cuda"), kc, vc, ks, vs, max_new=S)
    dk, dv = ((c[:-1].view(torch.float8_e4m3fn).float() * s[:-1, :, None, None]).transpose(1, 2).reshape(1, S, Hkv, d)
              .bfloat16() for c, s in ((kc, ks), (vc, vs)))
    want, wm, wl = bpa.bpa_fwd(q, dk.contiguous(), dv.contiguous(), causal=True)
    table = torch.arange(S // P, dtype=torch.int32, device="cuda")[None].contiguous()
    for rows in (1, 7, 300, S):
        o, m, l = bpa.bpa_cache_attn(q[0, S - rows:], kc, vc, ks, vs, table, i32([S]), i32([0, rows]), max_q=rows)
        torch.cuda.synchronize()
        # both round weights and outputs to bf16: |o| is at most 1 or so here, the sum of both sides' steps
        assert (o.float() - want[0, S - rows:].float()).abs().max() <= 2 * (2.0 ** -8 + 2.0 ** -8) * want[0].abs().max()
        assert torch.allclose(m, wm[0, :, S - rows:], atol=1e-4, rtol=1e-5)
        assert torch.allclose(l, wl[0, :, S - rows:], rtol=1e-3)
        assert (dk.double() - k.double()).abs().max() <= 2.0 ** -4 * k.abs().max()


# ---- the step of a serving loop ---------------------------------------------------------------------
@DTYPES
def test_serving_steps_together(bpa, dtype):
    """Prompts, then generated tokens: plan, append, attend on one stream, a captured graph from the
    third step on; every state and output against the definitions run side by side."""
    rng = np.random.default_rng(18)
    R, Hq, Hkv, d, dv, P, pages, width = 4, 8, 2, 64, 32, 16, 30, 9
    new = np.array([40, 1, 17, 33])
    table, ctx, count = np.full((R, width), -1), np.zeros(R, int), pages
    free = rng.permutation(pages)
    kc, vc = np.zeros((pages, Hkv, P, d), np.uint8), np.zeros((pages, Hkv, P, dv), np.uint8)
    ks, vs = np.zeros((pages, Hkv), np.float32), np.zeros((pages, Hkv), np.float32)
    dt, dctx, dfree, dcount = i32(table), i32(ctx), i32(free), i32([count])
    dk, dvv, dks, dvs = (torch.from_numpy(x).cuda() for x in (kc, vc, ks, vs))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = None
    for step in range(8):
        T = int(new.sum()) if step == 0 else R
        q, k, v = (rng.standard_normal((T, h, c)) * 2.0 ** (step % 3) for h, c in ((Hq, d), (Hkv, d), (Hkv, dv)))
        (tq, xq), (tk, xk), (tv, xv) = (as_dtype(x, dtype) for x in (q, k, v))

        def call(tq, tk, tv, tnew):
            plan = bpa.bpa_cache_plan(dctx, tnew, dt, dfree, dcount, page_size=P, T=tq.shape[0], ctx_lens_out=dctx,
                                      free_count_out=dcount)
            bpa.bpa_cache_append(tk, tv, plan[2], dk, dvv, dks, dvs, max_new=int(new.max()))
            return plan + bpa.bpa_cache_attn(tq, dk, dvv, dks, dvs, dt, plan[0], plan[1], max_q=int(new.max()))

        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            if step < 2:
                outs = call(tq, tk, tv, i32(new))
            elif graph is None:
                statics = [tq.clone(), tk.clone(), tv.clone(), i32(new)]
                graph = torch.cuda.CUDAGraph()
                torch.cuda.synchronize()
                with torch.cuda.graph(graph, stream=side):
                    outs = call(*statics)
                graph.replay()
            else:
                for a, b in zip(statics, (tq, tk, tv, i32(new))):
                    a.copy_(b)
                graph.replay()
        torch.cuda.synchronize()
        kv, cu, slots, pos, ctx, table, count = ora.plan(ctx, new, table, free, count, P, T)
        for got, want in zip(outs[:4] + (dctx, dt, dcount), (kv, cu, slots, pos, ctx, table, [count])):
            np.testing.assert_array_equal(got.cpu().numpy(), want)
        kc, ks = ora.append(xk, slots, kc, ks)
        vc, vs = ora.append(xv, slots, vc, vs)
        for got, want in ((dk, kc), (dvv, vc), (dks, ks), (dvs, vs)):
            np.testing.assert_array_equal(got.cpu().numpy(), want)
        c = dict(q=q, kc=kc, vc=vc, ks=ks, vs=vs, table=table, kv=kv, cu=cu)
        check_attention(c, dtype, *outs[6:])
        new = np.array([1, 1, 1, 1])


def test_two_calls_at_once(bpa):
    """Two streams, a workspace each: the answers of calls made one after the other."""
    cs = [make_step(np.random.default_rng(19 + i), [900, 300], [1, 2], 8, 2, 128, 128, 64) for i in range(2)]
    ts = [on_gpu(c, torch.bfloat16) for c in cs]
    want = [bpa.bpa_cache_attn(*t, max_q=2) for t in ts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        got = [bpa.bpa_cache_attn(*t, max_q=2, stream=s) for t, s in zip(ts, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


# ---- values that are not finite ----------------------------------------------------------------------
KERNELS = {   # ctx, new, Hq, Hkv, d, dv, P: 2 P + 1 and more tokens, so that a page of one token ends the first request
    "few_rows": ([128, 70], [1, 2], 8, 4, 128, 64, 64), "few_rows_pages_of_16": ([144, 31], [1, 3], 8, 2, 64, 64, 16),
    "many_rows": ([89, 20], [40, 30], 32, 16, 128, 128, 32), "any_shape": ([95, 30], [2, 1], 4, 2, 72, 40, 48),
}


def spoil(c, which, page_of, alone):
    """A copy of the step with NaN in channels 3 to 5 of kv head 1 of a request's token: (copy, clean copy with zeros
    in their place, the request, the token).  alone: the page's other values and so its scale are 0, as
    append leaves a page that has no finite value but 0."""
    r, token = page_of
    P = c["kc"].shape[2]
    page, off = c["table"][r, token // P], token % P
    bad = {**c, **{n: c[n].copy() for n in ("kc", "vc", "ks", "vs")}}
    for n in which:
        codes, scale = bad[n + "c"], bad[n + "s"]
        if alone:
            codes[page, 1], scale[page, 1] = 0, 0
        codes[page, 1, off, 3:6] = 0x7F
    clean = {**bad, **{n: bad[n].copy() for n in ("kc", "vc")}}
    for n in which:
        clean[n + "c"][page, 1, off, 3:6] = 0
    return bad, clean


@DTYPES
@pytest.mark.parametrize("alone", [True, False], ids=["alone", "among_others"])
@pytest.mark.parametrize("which", ["k", "v", "kv"])
@pytest.mark.parametrize("kernel", KERNELS)
def test_attention_keeps_what_is_not_finite(bpa, kernel, which, alone, dtype):
    case = KERNELS[kernel]
    c = make_step(np.random.default_rng(31), *case)
    end = c["kv"][0] - 1                               # the last token: only the last row of the request sees it
    T, Hq = c["q"].shape[:2]
    mine = np.arange(Hq) // (Hq // c["kc"].shape[1]) == 1
    for token in (end, 0, 37):
        bad, clean = spoil(c, which, (0, int(token)), alone)
        got, want = (bpa.bpa_cache_attn(*on_gpu(x, dtype), max_q=c["max_q"]) for x in (bad, clean))
        torch.cuda.synchronize()
        check_attention(clean, dtype, *want)
        p = c["kv"][0] - c["cu"][1] + np.arange(c["cu"][1])
        sees = np.zeros((T, Hq), bool)
        sees[:c["cu"][1]] = (p >= token)[:, None] & mine
        other = np.ones((T, Hq), bool)                 # rows of other requests and heads
        other[:c["cu"][1]] = ~mine
        wrong = torch.zeros(got[0].shape, dtype=torch.bool)
        wrong[torch.from_numpy(sees)] = True
        if which == "v":
            wrong[..., :3] = wrong[..., 6:] = False
        assert sees.any() and torch.isnan(got[0].cpu()[wrong]).all()
        assert torch.equal(got[0].cpu()[other], want[0].cpu()[other])
        assert torch.equal(got[1].T.cpu()[other], want[1].T.cpu()[other]) and torch.equal(got[2].T.cpu()[other], want[2].T.cpu()[other])
        if which == "v":                               # the weights and the other channels are what they were
            assert torch.equal(got[0][..., 6:], want[0][..., 6:])
            assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
        else:
            assert torch.isnan(got[2].T.cpu()[sees]).all()


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf], ids=str)
@pytest.mark.parametrize("kernel", KERNELS)
def test_append_then_attend_what_is_not_finite(bpa, kernel, value):
    # the first token of a fresh page has a value head without a finite value
    ctx, new, Hq, Hkv, d, dv, P = KERNELS[kernel]
    c = make_step(np.random.default_rng(32), ctx, new, Hq, Hkv, d, dv, P)
    end = int(c["kv"][0]) // P * P                     # a page's first token: the last one or one before it
    page = int(c["table"][0, end // P])
    t = on_gpu(c, torch.bfloat16)
    k, v = torch.randn(1, Hkv, d, device="cuda").bfloat16(), torch.randn(1, Hkv, dv, device="cuda").bfloat16()
    v[0, 1] = value
    bpa.bpa_cache_append(k, v, i32([page * P + end % P]), *t[1:5], max_new=1)
    o, m, l = bpa.bpa_cache_attn(*t, max_q=max(new))
    torch.cuda.synchronize()
    heads = slice(Hq // Hkv, 2 * Hq // Hkv)
    last = int(c["cu"][1]) - 1
    assert torch.isnan(o[last, heads]).all() and torch.isfinite(l[heads, last]).all()
    assert torch.isfinite(o[last, :Hq // Hkv]).all() and torch.isfinite(o[last + 1:]).all()


@DTYPES
@pytest.mark.parametrize("kernel", KERNELS)
def test_attention_scale_of_zero_stands_for_zeros(bpa, kernel, dtype):
    # pages whose codes are not zero although their scale is: whatever they hold counts as 0
    c = make_step(np.random.default_rng(33), *KERNELS[kernel])
    for n, pages in (("vs", (0, 2)), ("ks", (1, 2))):
        for j in pages:
            c[n][c["table"][0, min(j, (c["kv"][0] - 1) // c["kc"].shape[2])]] = 0
    run_and_check(bpa, c, dtype)
    c["vs"][:] = 0
    o, m, l = run_and_check(bpa, c, dtype)
    assert not o.any()


@DTYPES
@pytest.mark.parametrize("first,later", [(-100, 30), (-100, 110), (110, -100), (0, 60), (60, 0), (0, 40), (40, 0), (None, None), ("0", -90), ("0", 39)], ids=str)
@pytest.mark.parametrize("kernel", KERNELS)
def test_attention_value_scales_of_the_whole_range(bpa, kernel, first, later, dtype):
    # every scale that append writes, from 2^-100 to about 2^119, in any order within a request
    rng = np.random.default_rng(34)
    c = make_step(rng, *KERNELS[kernel])
    c["vs"][:] = np.exp2(rng.integers(-100, 110, c["vs"].shape) if first is None else np.full(c["vs"].shape, later)).astype(np.float32)
    for r in range(2):
        if first == "0":
            c["vs"][c["table"][r, 0]] = 0
        elif first is not None:
            c["vs"][c["table"][r, 0]] = 2.0 ** first
    run_and_check(bpa, c, dtype)
    run_and_check(bpa, c, dtype, window=(20, -1))
    run_and_check(bpa, c, dtype, sink=np.linspace(-2, 3, c["q"].shape[1]))


@pytest.mark.parametrize("name", ["plan", "append", "attn"])
def test_buffers_of_another_stream_are_not_the_current_ones(bpa, name):
    """Tensors dropped while the current stream has still to write them: a call on another stream, which is free
    at once, must not get their memory for its outputs and workspace."""
    t = on_gpu(make_step(np.random.default_rng(35), [900, 300], [1, 2], 8, 2, 128, 128, 64), torch.bfloat16)
    p = make_plan(np.random.default_rng(36), [3] * 300, [2] * 300, 16, 400)
    plan = (i32(p["ctx"]), i32(p["new"]), i32(p["table"]), i32(p["free"]), i32([p["count"]]))
    k, v, slots = torch.randn(3, 2, 128, device="cuda").bfloat16(), torch.randn(3, 2, 128, device="cuda").bfloat16(), i32([0, 1, 64])

    def call(stream=None):                        # the same again gives the same
        if name == "plan":
            return bpa.bpa_cache_plan(*plan, page_size=16, T=p["T"], stream=stream)
        if name == "append":
            bpa.bpa_cache_append(k, v, slots, *t[1:5], max_new=2, stream=stream)
            return t[1:5]
        return bpa.bpa_cache_attn(*t, max_q=2, stream=stream)

    want = [x.clone() for x in call()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    sizes = [256, 512, 1200, 2400, 4096, 6144] + [1 << n for n in range(13, 23)]
    junk = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(6)]
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                 # about ten milliseconds of the current stream
    for x in junk:
        x.fill_(0xFF)
    del junk, x
    got = call(stream=side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_plan_of_any_number_of_requests_in_a_fresh_process():
    # about 4,050 to 4,095 requests need more shared memory than a kernel has without asking for it, once its
    # static part is counted; an earlier plan of more requests in the process would have asked already
    body = """
import numpy as np, torch
from ring_attention_gb300 import bpa
from tests.test_gpu_cache import check_plan, make_plan
for R in (3900, 4049, 4050, 4051, 4095, 4096, 8192):
    rng = np.random.default_rng(R)
    check_plan(bpa, make_plan(rng, rng.integers(0, 40, R), rng.integers(0, 3, R), 16, 5))
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", body], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


WIDE = [     # head dims of 129 to 256 with more than 8 rows of a kv head, in one, two and four row tiles
    ([700], [1], 32, 2, 256, 256, 64), ([300, 33], [3, 5], 8, 2, 256, 256, 16), ([90, 0, 400], [20, 1, 7], 8, 2, 192, 128, 64),
    ([130], [1], 12, 1, 256, 64, 32), ([20, 250], [33, 2], 12, 4, 64, 192, 128), ([40, 10, 900], [9, 4, 2], 4, 2, 208, 240, 16),
    ([600, 31, 0], [1, 2, 1], 48, 2, 192, 128, 32), ([100, 5], [70, 131], 16, 4, 256, 256, 64), ([100, 5], [70, 131], 16, 4, 192, 112, 64),
]


@DTYPES
@pytest.mark.parametrize("case", WIDE, ids=lambda c: f"H{c[2]}_{c[3]}_d{c[4]}_{c[5]}_P{c[6]}_q{max(c[1])}")
def test_attention_many_rows_of_wide_heads(bpa, case, dtype):
    rng = np.random.default_rng(sum(case[0]) + case[5])
    c = make_step(rng, *case, pad=2)
    run_and_check(bpa, c, dtype)
    run_and_check(bpa, c, dtype, window=(70, -1), sink=rng.standard_normal(case[2]))
    c["kv"] = c["kv"].copy()
    c["kv"][-1] = 0
    c["vs"][:] = np.exp2(rng.integers(-30, 30, c["vs"].shape) - 7.0).astype(np.float32)
    run_and_check(bpa, c, dtype, causal=False)


@pytest.mark.parametrize("kernel", ["few_rows", "many_rows", "any_shape"])
@DTYPES
def test_attention_weights_keep_eleven_bits(bpa, kernel, dtype):
    """Two keys of scores delta and 0 with values 1 and -1: o = tanh(delta / 2), small beside A = 1, so the rounding of
    the weights shows.  Bound: the one of the module's text with n = 2, the weights' own part half a step of fp16,
    2^-11 (float32: two halves, 2^-21), and a largest weight of 2^7 at least: n 2^-32 448 H, H <= 1.
    Weights of bf16 would break it, which is checked first."""
    R, rows, Hq, Hkv, d, dv, P = {"few_rows": (20, 1, 64, 8, 64, 64, 16), "many_rows": (2, 40, 32, 16, 64, 64, 16),
                                  "any_shape": (4, 3, 32, 8, 72, 40, 8)}[kernel]
    T = R * rows
    q = np.zeros((T, Hq, d))
    q[..., 0] = np.linspace(0, 0.02, T * Hq).reshape(T, Hq)
    c = dict(q=q, kc=np.zeros((1, Hkv, P, d), np.uint8), vc=np.zeros((1, Hkv, P, dv), np.uint8),
             ks=np.ones((1, Hkv), np.float32), vs=np.ones((1, Hkv), np.float32), table=np.zeros((R, 1), int),
             kv=np.full(R, 2), cu=np.arange(R + 1) * rows, max_q=rows)
    c["kc"][:, :, 0, 0], c["vc"][:, :, 0], c["vc"][:, :, 1] = 0x38, 0x38, 0xB8      # 1, 1 and -1
    delta = as_dtype(q, dtype)[1][..., :1]
    want = np.tanh(delta / 2)
    half, weight = (2.0 ** -8, 2.0 ** -11) if dtype == torch.bfloat16 else (2.0 ** -24, 2.0 ** -21)
    dz = (d + 4) * 2.0 ** -23 * 0.02 + 2.0 ** -21
    bound = half * np.abs(want) + (2 * dz + weight + 2 * 2.0 ** -23 + 2 * 2.0 ** -32 * 448) * (1 + half)
    low = torch.from_numpy(np.exp(-delta)).to(torch.bfloat16).double().numpy()
    assert (np.abs((1 - low) / (1 + np.exp(-delta)) - want) > bound).any()
    o, m, l = bpa.bpa_cache_attn(*on_gpu(c, dtype), max_q=rows, causal=False, scale=1.0)
    torch.cuda.synchronize()
    assert (np.abs(f64(o) - want) <= bound).all()


@DTYPES
@pytest.mark.parametrize("kernel", KERNELS)
def test_attention_repeats_itself(bpa, kernel, dtype):
    ctx, new, *rest = KERNELS[kernel]
    c = make_step(np.random.default_rng(37), [900 + 13 * i for i in range(6)] + ctx, [1, 2, 1, 3, 1, 1] + new, *rest)
    t = on_gpu(c, dtype)
    first = bpa.bpa_cache_attn(*t, max_q=c["max_q"])
    for _ in range(20):
        for a, b in zip(bpa.bpa_cache_attn(*t, max_q=c["max_q"]), first):
            assert torch.equal(a, b)


@pytest.mark.parametrize("bad", [-2, -17, -2 ** 31])
def test_append_reports_slots_below_minus_one(bpa, bad):
    rng = np.random.default_rng(38)
    kc, ks = random_cache(rng, 4, 1, 16, 16)
    x = torch.randn(3, 1, 16, device="cuda")
    (gc, gs, *_), ws = run_append(bpa, x, x, [3, bad, -1], kc, kc, ks, ks)
    with pytest.raises(bpa.BpaError):
        bpa.bpa_check(ws)
    wc, wsc = ora.append(f64(x), [3, -1, -1], kc, ks)
    np.testing.assert_array_equal(gc, wc)
    np.testing.assert_array_equal(gs, wsc)


def test_attention_prompts_under_a_graph(bpa):
    """A captured call with requests of many and of few rows, replayed on other values: scales that send a request from
    one kernel to the other, a page that is no longer there, and back; the workspace is the same throughout."""
    rng = np.random.default_rng(39)
    cases = [make_step(rng, [130, 37, 250], [70, 1, 33], 32, 8, 128, 128, 64) for _ in range(4)]
    for c in cases[1:]:
        for n in ("table", "kv", "cu"):
            c[n] = cases[0][n]
    for c in cases:                                # the rows behind the last token of each
        for n in ("kc", "vc"):
            c[n][(c[n] & 0x7F) == 0x7F] = 0
    cases[1]["vs"][:] = np.exp2(rng.integers(-100, 100, cases[1]["vs"].shape)).astype(np.float32)
    cases[2]["kv"] = np.array([200, 0, 40])
    ts = [on_gpu(c, torch.bfloat16) for c in cases]
    t = [x.clone() for x in ts[0]]
    D, B = bpa.make_cache_desc(*t[1:5], torch.bfloat16), bpa.make_cache_batch(t[0], *t[5:], max_q=70)
    ws = torch.full((bpa.bpa_cache_attn_workspace_size(D, B),), 255, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        bpa.bpa_cache_attn(*t, max_q=70, workspace_buf=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            o, m, l = bpa.bpa_cache_attn(*t, max_q=70, workspace_buf=ws)
        for i in (0, 1, 2, 3, 1, 0):
            for dst, src in zip(t, ts[i]):
                dst.copy_(src)
            g.replay()
            s.synchronize()
            bpa.bpa_check(ws)
            check_attention(cases[i], torch.bfloat16, o, m, l)


@DTYPES
@pytest.mark.parametrize("kernel", KERNELS)
def test_attention_shared_pages_and_leading_rows(bpa, kernel, dtype):
    # two requests over the same first pages, one page twice in a row of the table, rows in front of the first request
    c = make_step(np.random.default_rng(40), *KERNELS[kernel])
    P = c["kc"].shape[2]
    n = min(c["kv"]) // P                          # whole pages of both
    c["table"] = c["table"].copy()
    c["table"][1, :n] = c["table"][0, :n]
    c["table"][0, 1] = c["table"][0, 0]
    c["q"] = np.concatenate([np.full((3,) + c["q"].shape[1:], np.nan), c["q"]])
    c["cu"] = c["cu"] + 3
    t = on_gpu(c, dtype)
    o = torch.full((len(c["q"]), t[0].shape[1], c["vc"].shape[3]), 77.0, dtype=dtype, device="cuda")
    _, m, l = bpa.bpa_cache_attn(*t, max_q=c["max_q"], o=o)
    torch.cuda.synchronize()
    check_attention({**c, "q": np.nan_to_num(c["q"])}, dtype, o, m, l)      # its bound takes every row's q
    assert (o[:3] == 77).all()


HEADS_ALONE = [([300, 0], [65, 200], 32, 32, 128, 128, 64), ([0, 129], [300, 1], 32, 32, 64, 64, 16), ([7], [513], 16, 16, 128, 64, 32)]


@pytest.mark.parametrize("case", HEADS_ALONE, ids=lambda c: f"d{c[4]}_{c[5]}_q{max(c[1])}")
def test_attention_many_rows_of_heads_of_their_own(bpa, case):
    c = make_step(np.random.default_rng(41), *case)
    run_and_check(bpa, c, torch.bfloat16)
    run_and_check(bpa, c, torch.bfloat16, window=(130, -1))


@pytest.mark.parametrize("rows", [1, 40])
def test_append_of_a_slot_twice_leaves_other_pages(bpa, rows):
    # what the page of the two rows holds is unspecified, everything else is not
    rng = np.random.default_rng(42)
    kc, ks = random_cache(rng, 9, 2, 16, 32)
    x = rng.standard_normal((rows + 3, 2, 32)).astype(np.float32)
    slots = np.concatenate([[5 * 16 + 3, 5 * 16 + 3, 5 * 16 + 3], np.arange(16, 16 + rows)])
    tx = torch.from_numpy(x).cuda()
    (gc, gs, vc, vs), ws = run_append(bpa, tx, tx, slots, kc, kc, ks, ks, max_new=rows)
    bpa.bpa_check(ws)
    wc, wsc = ora.append(x.astype(np.float64), np.concatenate([[-1] * 3, slots[3:]]), kc, ks)
    rest = np.arange(9) != 5
    for codes, scales in ((gc, gs), (vc, vs)):
        np.testing.assert_array_equal(codes[rest], wc[rest])
        np.testing.assert_array_equal(scales[rest], wsc[rest])
