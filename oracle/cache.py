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


def attention(q, k_codes, v_codes, k_scale, v_scale, table, kv_lens, cu_q, *, causal=True, window=(-1, -1),
              scale=None, sink=None, heaviest=False):
    """q [T, Hq, d] float64 over the cache.  Returns (o, m, l); rows behind cu_q[-1] are NaN.
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
                if causal:
                    ok &= key <= p
                if wl >= 0:
                    ok &= key >= p - wl
                if wr >= 0:
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
