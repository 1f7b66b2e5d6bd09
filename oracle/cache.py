"""Plain float64 definitions of the paged 8-bit cache's operators (numpy, loops over requests):
the step's plan, quantised append and attention.  They share nothing with the library."""
from __future__ import annotations

import numpy as np


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    out = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        x = np.nan if (e, f) == (15, 7) else f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        out[c] = -x if c & 128 else x
    return out


def e4m3_round(x: np.ndarray) -> np.ndarray:
    """Codes nearest to x, ties to the even code; infinities and NaN give 0x7f.  |x| <= 448 otherwise."""
    x = np.asarray(x, np.float64)
    pos = e4m3_values()[:127]                                  # ascending, codes 0..126
    a = np.abs(x)
    hi = np.searchsorted(pos, np.where(np.isfinite(a), a, 0.0)).clip(1, 126)
    lo = hi - 1
    v = np.where(np.isfinite(a), a, 0.0)
    dl, dh = v - pos[lo], pos[hi] - v
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi))).astype(np.uint8)
    code = np.where(np.signbit(x), code | 128, code).astype(np.uint8)
    return np.where(np.isfinite(x), code, 0x7F).astype(np.uint8)


def scale_for(amax: float) -> float:
    """The smallest power of two s >= 2^-100 with amax <= 448 s; 0 for amax 0."""
    if amax == 0:
        return 0.0
    s = 2.0 ** -100
    while amax > 448 * s:
        s *= 2
    return s


def plan(ctx, new, table, free, count, P, T):
    """One step: (kv_lens, cu_q, slots, positions, ctx_out, table, count_out) for valid inputs."""
    table = np.array(table)
    R = len(ctx)
    kv, out = np.zeros(R, np.int32), np.array(ctx, np.int32)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    slots, pos = np.full(T, -1, np.int32), np.full(T, -1, np.int32)
    left, wanted = count, 0
    for r in range(R):
        have, total = -(-ctx[r] // P), -(-(ctx[r] + new[r]) // P)
        wanted += total - have
        if total > have and wanted > count:
            continue
        for j in range(have, total):
            left -= 1
            table[r, j] = free[left]
        kv[r] = out[r] = ctx[r] + new[r]
        for i in range(new[r]):
            p = ctx[r] + i
            slots[cu[r] + i], pos[cu[r] + i] = table[r, p // P] * P + p % P, p
    return kv, cu, slots, pos, out, table, left


def append(x, slots, codes, scale):
    """Rows x [T, H, c] (float64) into codes [pages, H, P, c] (uint8) and scale [pages, H]; returns both."""
    codes, scale = codes.copy(), scale.astype(np.float64).copy()
    P, val, t, T = codes.shape[2], e4m3_values(), 0, len(slots)
    while t < T:
        if slots[t] < 0:
            t += 1
            continue
        n, (page, off) = 1, divmod(int(slots[t]), P)
        while t + n < T and off + n < P and slots[t + n] == slots[t] + n:
            n += 1
        for h in range(codes.shape[1]):
            rows = x[t:t + n, h]
            mags = np.abs(rows[np.isfinite(rows)])
            s = scale_for(float(mags.max()) if mags.size else 0.0)
            old = scale[page, h] if off else 0.0
            s = max(s, old)
            if off and s > old:
                codes[page, h, :off] = e4m3_round(val[codes[page, h, :off]] * (old / s))
            codes[page, h, off:off + n] = e4m3_round(rows / s if s > 0 else rows)
            scale[page, h] = s
        t += n
    return codes, scale


def tree_set(words):
    """The rows that a mask names."""
    return {32 * w + j for w, x in enumerate(np.asarray(words).astype(np.int64) & 0xFFFFFFFF) for j in range(32) if x >> j & 1}


def tree_masks(parents, kv_lens, cu_q, words, window_left=-1):
    """(tree [T, words] as int32 bits, positions [T]) for valid inputs; window_left >= 0: of a row's ancestors the
    nearest window_left alone."""
    T = len(parents)
    tree, pos = np.zeros((T, words), np.int64), np.full(T, -1)
    for r, L in enumerate(kv_lens):
        a, b = cu_q[r], cu_q[r + 1]
        if L == 0:
            continue
        for i in range(b - a):
            p = parents[a + i]
            if p >= 0:
                tree[a + i] = tree[a + p]
            tree[a + i, i // 32] |= 1 << i % 32
            if window_left >= 0:
                far = sorted(tree_set(tree[a + i]))[:-1 - window_left]           # ancestors stand in front of their rows
                for j in far:
                    tree[a + i, j // 32] &= ~(1 << j % 32)
            pos[a + i] = pos[a + p] + 1 if p >= 0 else L - (b - a)
    return np.where(tree >= 2 ** 31, tree - 2 ** 32, tree).astype(np.int32), pos.astype(np.int32)


def keep(codes, scale, paths, kv_lens, cu_q, table):
    """Tokens paths[r] (ascending indexes of request r's new rows) to the end of its context: (codes, scale)."""
    old, olds = codes, scale.astype(np.float64)
    codes, scale = codes.copy(), olds.copy()
    P, val = codes.shape[2], e4m3_values()
    for r, path in enumerate(paths):
        ctx = kv_lens[r] - (cu_q[r + 1] - cu_q[r])
        where = lambda p: (table[r][p // P], p % P)                                    # noqa: E731
        for j in range(ctx // P, -(-(ctx + len(path)) // P) if len(path) else 0):
            page = table[r][j]
            moves = [(where(ctx + x), i) for i, x in enumerate(path) if (ctx + i) // P == j]
            front = max(0, ctx - j * P)
            if not moves:
                continue
            for h in range(codes.shape[1]):
                s = max([olds[p, h] for (p, _), _ in moves] + ([olds[page, h]] if front else []))
                at = lambda c, o: c if o == s or s == 0 else e4m3_round(val[c] * (o / s))   # noqa: E731
                codes[page, h, :front] = at(old[page, h, :front], olds[page, h])
                for (p, t), i in moves:
                    codes[page, h, (ctx + i) % P] = at(old[p, h, t], olds[p, h])
                scale[page, h] = s
    return codes, scale


def fork(src, dst, ctx, table, refs, free, count, P):
    """(copy_src, copy_dst, ctx_out, table, refs, count_out) for valid inputs."""
    ctx, table, refs = np.array(ctx), np.array(table), np.array(refs)
    out, copies, wanted, left = ctx.copy(), [], 0, count
    for s, d in zip(src, dst):
        need = int(ctx[s] % P > 0)
        wanted += need
        pair = (-1, -1)
        if not need or wanted <= count:
            full = ctx[s] // P
            table[d, :full] = table[s, :full]
            np.add.at(refs, table[s, :full], 1)
            if need:
                left -= 1
                table[d, full] = free[left]
                pair = (table[s, full], free[left])
            out[d] = ctx[s]
        copies.append(pair)
    a = np.array(copies, np.int64).reshape(-1, 2)
    return a[:, 0], a[:, 1], out, table, refs, left


def release(ctx, keep_lens, table, refs, free, count, P):
    """(ctx_out, refs, free, count_out) for valid inputs."""
    refs, free = np.array(refs), np.array(free)
    for r, (n, k) in enumerate(zip(ctx, keep_lens)):
        for j in range(-(-k // P), -(-n // P)):
            refs[table[r][j]] -= 1
    for page in range(len(refs)):
        if refs[page] < 0:
            free[count] = page
            count += 1
            refs[page] = 0
    return np.array(keep_lens), refs, free, count


def attention(q, k_codes, v_codes, k_scale, v_scale, table, kv_lens, cu_q, *, causal=True, window=(-1, -1),
              scale=None, sink=None, heaviest=False, tree=None):
    """q [T, Hq, d] float64 over the cache.  Returns (o, m, l); rows behind cu_q[-1] are NaN.
    tree: [T, words] masks (32 bits each) over a request's own rows.
    heaviest: also the largest softmax weight times v scale of each row, [T, Hq, 1]."""
    T, Hq, d = q.shape
    Hkv, P, dv = k_codes.shape[1], k_codes.shape[2], v_codes.shape[3]
    val = e4m3_values()
    scale = d ** -0.5 if scale is None else scale
    o, m, l = np.full((T, Hq, dv), np.nan), np.full((Hq, T), np.nan), np.full((Hq, T), np.nan)
    heavy = np.zeros((T, Hq, 1))
    wl, wr = window
    for r in range(len(kv_lens)):
        L, a, b = int(kv_lens[r]), int(cu_q[r]), int(cu_q[r + 1])
        pages = table[r, :-(-L // P)]
        key = np.arange(L)
        for h in range(Hq):
            g = h // (Hq // Hkv)
            K = (val[k_codes[pages, g]] * k_scale[pages, g].astype(np.float64)[:, None, None]).reshape(-1, d)[:L]
            V = (val[v_codes[pages, g]] * v_scale[pages, g].astype(np.float64)[:, None, None]).reshape(-1, dv)[:L]
            for t in range(a, b):
                p = L - (b - a) + (t - a)
                ok = np.ones(L, bool)
                if tree is not None:
                    first, seen = L - (b - a), tree_set(tree[t])
                    depth = sum(j < t - a for j in seen)
                    ok = (key < first) & ((wl < 0) | (key >= first + depth - wl)) | np.isin(key - first, sorted(seen)) & (key >= first)
                elif causal:
                    ok &= key <= p
                if wl >= 0 and tree is None:
                    ok &= key >= p - wl
                if wr >= 0 and tree is None:
                    ok &= key <= p + wr
                z = (K[ok] @ q[t, h]) * scale
                top = max([z.max()] if z.size else [-np.inf])
                if sink is not None:
                    top = max(top, float(sink[h]))
                if top == -np.inf:
                    o[t, h], m[h, t], l[h, t] = 0, -np.inf, 0
                    continue
                w = np.exp(z - top)
                den = w.sum() + (np.exp(float(sink[h]) - top) if sink is not None else 0)
                o[t, h], m[h, t], l[h, t] = (w @ V[ok]) / den, top, den
                if w.size:
                    heavy[t, h] = (w * v_scale[pages, g].astype(np.float64).repeat(P)[:L][ok]).max() / den
    return (o, m, l, heavy) if heaviest else (o, m, l)
