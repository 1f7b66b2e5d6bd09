"""Cases of the operators around the attention calls: norms of q and k with the position rotation,
and what a serving loop that drafts trees of tokens does with its paged 8-bit cache.

* ``rope``  - RMS norm of each head of q and k, then the rotation by the token's position, one pass;
  its backward pass (gradients of q, k and of both norms' weights),
* ``tree``  - ancestor masks and positions of drafted trees from their parents, and the attention of
  the drafted rows over the cache under these masks,
* ``keep``  - the accepted path's keys and values moved to the end of the context, page scales joined,
* ``pages`` - requests forked (full pages shared, the last one copied), finished and cut ones released.

``run`` computes them in elementary torch operations in 32 bits (angles and long sums in 64) where
``own`` is false and calls the library where it is true.  ``exact`` is written from the definitions
in 64 bits.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-6


# ---- lengths, trees and sizes: from the case alone --------------------------------------------
def _spread(n, lo, hi):
    """n whole numbers from lo to hi, ragged, the same for every seed; the largest is hi."""
    if n == 1:
        return [hi]
    return [hi if i == n // 2 else lo + int((hi - lo + 1) * math.fmod(0.37 + i * 0.6180339887498949, 1.0))
            for i in range(n)]


def _lens(case):
    """Tokens that each request has in the cache before the step, and new ones."""
    return (_spread(case["R"], case["ctx_lo"], case["ctx_hi"]),
            _spread(case["R"], case["new_lo"], case["new_hi"]))


def _pages(n, P):
    return (n + P - 1) // P


def _parents(case):
    """Each request's drafted tree: the index of every node's parent, -1 for the first; a node hangs
    below one of the `width` nodes before it (width 1: a chain)."""
    out = []
    for r, n in enumerate(_lens(case)[1]):
        out.append([-1 if i == 0 else max(0, i - 1 - int(case["width"] * math.fmod(0.11 * r + i * 0.7548776662466927, 1.0)))
                    for i in range(n)])
    return out


def _paths(case):
    """Each request's accepted path: a node and its ancestors, ascending."""
    out = []
    for r, par in enumerate(_parents(case)):
        path, i = [], int(len(par) * math.fmod(0.29 + r * 0.5698402909980532, 1.0)) if par else -1
        while i >= 0:
            path.append(i)
            i = par[i]
        out.append(path[::-1])
    return out


def listed():
    G = {"Hq": 32, "Hkv": 8, "d": 128}
    C = {**G, "dv": 128, "P": 64}
    return [
        # one generation step: a row per request, far positions, q and k inside one projection's output
        {"name": "rope_decode", "op": "rope", "way": "fwd", "B": 1, "S": 64, "pad_rows": 3, **G, "rot": 128,
         "inter": False, "norm": True, "fused": True, "theta": 500000.0, "pos_hi": 131071, "dtype": "bfloat16"},
        # a forward pass over long training sequences of many query heads
        {"name": "rope_forward", "op": "rope", "way": "fwd", "B": 2, "S": 4096, "Hq": 128, "Hkv": 8, "d": 128, "rot": 128,
         "inter": False, "norm": True, "fused": False, "theta": 10000.0, "pos_hi": 0, "dtype": "bfloat16"},
        # the backward pass of a training step
        {"name": "rope_backward", "op": "rope", "way": "bwd", "B": 2, "S": 4096, **G, "rot": 128,
         "inter": False, "norm": True, "fused": True, "theta": 10000.0, "pos_hi": 0, "dtype": "bfloat16"},
        # the 32-bit shape: an odd length, a part of the head rotated in neighbouring pairs
        {"name": "rope_backward_fp32", "op": "rope", "way": "bwd", "B": 3, "S": 333, "Hq": 4, "Hkv": 2, "d": 80, "rot": 32,
         "inter": True, "norm": True, "fused": False, "theta": 10000.0, "pos_hi": 0, "dtype": "float32"},
        # one conversation with a drafted tree: the latency of a single step
        {"name": "tree_one", "op": "tree", "R": 1, "ctx_lo": 1500, "ctx_hi": 1500, "new_lo": 26, "new_hi": 26, "width": 5,
         **C, "dtype": "bfloat16", "wl": -1, "sink": False},
        # a batch of conversations of mixed lengths, trees of mixed sizes
        {"name": "tree_batch", "op": "tree", "R": 32, "ctx_lo": 200, "ctx_hi": 8191, "new_lo": 8, "new_hi": 64, "width": 7,
         **C, "dtype": "bfloat16", "wl": -1, "sink": False},
        # few requests with very long contexts
        {"name": "tree_long", "op": "tree", "R": 2, "ctx_lo": 100000, "ctx_hi": 131007, "new_lo": 40, "new_hi": 64, "width": 9,
         **C, "dtype": "bfloat16", "wl": -1, "sink": False},
        # small trees under a sliding window and with a sink, small pages, a padded batch
        {"name": "tree_window", "op": "tree", "R": 33, "ctx_lo": 1, "ctx_hi": 8000, "new_lo": 1, "new_hi": 15, "width": 4,
         "Hq": 64, "Hkv": 8, "d": 64, "dv": 64, "P": 16, "dtype": "bfloat16", "wl": 1024, "sink": True, "pad_rows": 9},
        # after a verified step of a small batch
        {"name": "keep_small", "op": "keep", "R": 4, "ctx_lo": 700, "ctx_hi": 1500, "new_lo": 20, "new_hi": 26, "width": 5,
         "Hkv": 8, "d": 128, "dv": 128, "P": 64},
        # ... of a large one: deep trees over small pages, narrower values
        {"name": "keep_batch", "op": "keep", "R": 256, "ctx_lo": 0, "ctx_hi": 900, "new_lo": 0, "new_hi": 64, "width": 3,
         "Hkv": 8, "d": 128, "dv": 64, "P": 16},
        # a request sampled four times from here on, another one over
        {"name": "pages_small", "op": "pages", "N": 3, "parents": 1, "ends": 2, "ctx_lo": 900, "ctx_hi": 1500, "Hkv": 8,
         "d": 128, "dv": 128, "P": 64},
        # many samples of long prompts begin while a large batch ends or gives rejected tokens back
        {"name": "pages_large", "op": "pages", "N": 256, "parents": 32, "ends": 256, "ctx_lo": 100, "ctx_hi": 2000, "Hkv": 8,
         "d": 128, "dv": 128, "P": 32},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "tree", "tree", "keep", "pages"])
    d = rng.choice([64, 80, 96, 128, 128, 192, 256])
    if op == "rope":
        dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
        Hkv = rng.choice([1, 2, 3, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
        d = rng.choice([d, d, d, 24, 72])
        B = rng.choice([1, 1, 2, 3])
        S = _log_int(rng, 1, 2 * 4096 * 40 * 128 // (B * (Hq + Hkv) * d))
        far = B == 1 and rng.random() < 0.5
        return {"op": op, "way": rng.choice(["fwd", "bwd"]), "B": B, "S": S, "pad_rows": rng.choice([0, 5]) if far else 0,
                "Hq": Hq, "Hkv": Hkv, "d": d, "rot": rng.choice([d, d, d // 2, d // 4 * 2]), "inter": rng.random() < 0.3,
                "norm": rng.random() < 0.8, "fused": rng.random() < 0.5, "theta": rng.choice([1e4, 5e5]),
                "pos_hi": _log_int(rng, 10, 1000000) if far else 0, "dtype": dtype}
    Hkv = rng.choice([1, 2, 4, 8])
    dv = rng.choice([d, d, d, 64])
    P = rng.choice([16, 32, 64, 128])
    if op == "pages":
        return {"op": op, "N": _log_int(rng, 1, 200), "parents": rng.randint(1, 20), "ends": _log_int(rng, 1, 200),
                "ctx_lo": 1, "ctx_hi": _log_int(rng, 1, 2500), "Hkv": Hkv, "d": d, "dv": dv, "P": P}
    width = rng.choice([1, 2, 4, 8, 20])
    if op == "keep":
        return {"op": op, "R": _log_int(rng, 1, 250), "ctx_lo": 0, "ctx_hi": _log_int(rng, 1, 900), "new_lo": rng.randint(0, 1),
                "new_hi": _log_int(rng, 1, 64), "width": width, "Hkv": Hkv, "d": d, "dv": dv, "P": P}
    c = {"op": op, "Hkv": Hkv, "Hq": Hkv * rng.choice([1, 2, 3, 4, 7, 8, 16]), "d": d, "dv": dv, "P": P,
         "dtype": rng.choice(["bfloat16", "bfloat16", "bfloat16", "float32"]), "wl": rng.choice([-1, -1, -1, 3, 200, 1500]),
         "sink": rng.random() < 0.25, "ctx_lo": rng.randint(0, 1), "pad_rows": rng.choice([0, 0, 3]), "width": width,
         "new_lo": rng.randint(0, 1), "new_hi": _log_int(rng, 1, 100)}
    c["R"] = _log_int(rng, 1, 50)
    c["ctx_hi"] = _log_int(rng, 1, max(1, min(100000, 8000000 // (c["R"] * c["new_hi"] * c["Hq"] // 8 + 1))))
    return c


# ---- what a user's program has in hand -------------------------------------------------------
def _scale_for(amax):
    """The smallest power of two s with amax <= 448 s."""
    return torch.exp2(torch.ceil(torch.log2(amax.double() / E4M3_MAX)).clamp(-100, 127)).float()


def _filled_pages(num, H, P, d, gen):
    """Pages as earlier steps left them: e4m3 codes and a power of two for each page and head."""
    x = torch.randn(num, H, P, d, generator=gen, device="cuda")
    x *= torch.exp2(torch.randn(num, H, 1, 1, generator=gen, device="cuda"))
    s = _scale_for(x.abs().amax((2, 3)))
    x /= s[:, :, None, None]
    return x.clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), s


def _table(counts, spare, gen):
    """Tables of `counts` pages each, taken at random from the pool, the ids left and the pool's size."""
    used = sum(counts)
    ids = torch.randperm(used + spare, generator=gen, device="cuda").to(torch.int32)
    have = torch.tensor(counts, device="cuda")
    table = torch.full((len(counts), max(1, max(counts))), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(table.shape[1], device="cuda")[None] < have[:, None]] = ids[:used]
    return table, ids[used:].contiguous(), used + spare


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _prepare_rope(c, gen):
    B, S, Hq, Hkv, d = c["B"], c["S"] + c.get("pad_rows", 0), c["Hq"], c["Hkv"], c["d"]
    dt, s = getattr(torch, c["dtype"]), {"case": c}

    def pair(std, fused):      # q and k (or their gradients): parts of one buffer [B, S, Hq + 2 Hkv, d], or two tensors
        H = Hq + 2 * Hkv if fused else Hq + Hkv
        x = torch.randn(B, S, H, d, generator=gen, device="cuda")
        x *= std * torch.exp2(torch.randn(1, 1, H, 1, generator=gen, device="cuda"))
        x = x.to(dt)
        if fused:
            return x[:, :, :Hq], x[:, :, Hq:Hq + Hkv]
        return x[:, :, :Hq].contiguous(), x[:, :, Hq:].contiguous()

    s["q"], s["k"] = pair(1.0, c["fused"])
    s["wq"] = 1 + 0.2 * torch.randn(d, generator=gen, device="cuda") if c["norm"] else None
    s["wk"] = 1 + 0.2 * torch.randn(d, generator=gen, device="cuda") if c["norm"] else None
    i = torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda")
    s["inv_freq"] = torch.pow(c["theta"], -i / c["rot"]).float()
    s["pos"] = None
    if c["pos_hi"]:
        s["pos"] = torch.randint(0, c["pos_hi"] + 1, (B, S), generator=gen, device="cuda").to(torch.int32)
        s["pos"][:, c["S"]:] = -1                     # rows behind the last sequence
    if c["way"] == "fwd":
        s["q_out"] = torch.zeros(B, S, Hq, d, dtype=dt, device="cuda")     # skipped rows stay
        s["k_out"] = torch.zeros(B, S, Hkv, d, dtype=dt, device="cuda")
        return s
    s["dq_out"], s["dk_out"] = pair(0.01, False)
    if c["fused"]:
        buf = torch.zeros(B, S, Hq + 2 * Hkv, d, dtype=dt, device="cuda")  # the projection's gradient
        s["dq"], s["dk"] = buf[:, :, :Hq], buf[:, :, Hq:Hq + Hkv]
    else:
        s["dq"], s["dk"] = torch.zeros_like(s["q"]), torch.zeros_like(s["k"])
    return s


def _prepare_pages(c, gen):
    P, A, N, E = c["P"], c["parents"], c["N"], c["ends"]
    ctx = _spread(A + E, c["ctx_lo"], c["ctx_hi"])
    table, left, num = _table([_pages(n, P) for n in ctx], N + 3, gen)
    R, width = A + E + N, table.shape[1]
    s = {"case": c, "P": P}
    s["table"] = torch.cat([table, torch.full((N, width), -1, dtype=torch.int32, device="cuda")])
    refs = torch.zeros(num, dtype=torch.int32, device="cuda")
    keep = ctx[:A] + [0 if i % 3 else max(0, n - 1 - i % 70) for i, n in enumerate(ctx[A:])]
    # every fourth of the ending requests shares its full pages with a fork that goes on elsewhere
    for i in range(0, E, 4):
        full = ctx[A + i] // P
        refs[table[A + i, :full].long()] = 1
        keep[A + i] = 0
    src = [i % A for i in range(N)]
    s["src"], s["dst"] = _i32(src), _i32([A + E + i for i in range(N)])
    s["ctx"], s["keep_lens"] = _i32(ctx + [0] * N), _i32(keep + [ctx[i] for i in src])
    s["refs"], s["count"] = refs, _i32([left.numel()])
    s["free"] = torch.zeros(num, dtype=torch.int32, device="cuda")
    s["free"][:left.numel()] = left
    s["k_cache"], s["k_scale"] = _filled_pages(num, c["Hkv"], P, c["d"], gen)
    s["v_cache"], s["v_scale"] = _filled_pages(num, c["Hkv"], P, c["dv"], gen)
    return s


def prepare(case, seed):
    c, gen = case, torch.Generator(device="cuda").manual_seed(seed)
    if c["op"] == "rope":
        return _prepare_rope(c, gen)
    if c["op"] == "pages":
        return _prepare_pages(c, gen)
    ctx, new = _lens(c)
    P, T = c["P"], sum(new) + c.get("pad_rows", 0)
    table, _, num = _table([_pages(a + b, P) for a, b in zip(ctx, new)], 7, gen)
    s = {"case": c, "P": P, "T": T, "table": table}
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["cu_q"], s["kv_lens"] = _i32(cu), _i32([a + b for a, b in zip(ctx, new)])
    s["k_cache"], s["k_scale"] = _filled_pages(num, c["Hkv"], P, c["d"], gen)
    s["v_cache"], s["v_scale"] = _filled_pages(num, c["Hkv"], P, c["dv"], gen)
    s["max_q"], s["max_kv"] = c["new_hi"], max(a + b for a, b in zip(ctx, new))
    if c["op"] == "keep":
        paths = _paths(c)
        most = max(1, max(len(p) for p in paths))
        s["keep"] = _i32([p + [-1] * (most - len(p)) for p in paths])
        s["keep_count"] = _i32([len(p) for p in paths])
        return s
    s["words"] = max(1, _pages(c["new_hi"], 32))
    s["parents"] = _i32([p for par in _parents(c) for p in par] + [-1] * (T - cu[-1]))
    s["q"] = torch.randn(T, c["Hq"], c["d"], generator=gen, device="cuda").to(getattr(torch, c["dtype"]))
    s["sink"] = torch.randn(c["Hq"], generator=gen, device="cuda") if c["sink"] else None
    s["o"] = torch.zeros(T, c["Hq"], c["dv"], dtype=s["q"].dtype, device="cuda")   # rows behind the last sequence stay
    s["m"], s["l"] = torch.zeros(c["Hq"], T, device="cuda"), torch.zeros(c["Hq"], T, device="cuda")
    return s


# ---- the plain forms ---------------------------------------------------------------------------
def _rotation(s, B, S):
    """(cos, sin) [B, S, 1, rot / 2] and which rows there are, [B, S, 1, 1]; angles in 64 bits."""
    pos = torch.arange(S, device="cuda")[None].expand(B, S) if s["pos"] is None else s["pos"]
    angle = pos.double()[:, :, None, None] * s["inv_freq"].double()
    return angle.cos().float(), angle.sin().float(), (pos >= 0)[:, :, None, None]


def _rotated(x, c, cos, sin):
    """The rotation of the first rot channels of x [B, S, H, d], float32."""
    rot = c["rot"]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if c["inter"] else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, v = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([u, v], -1).flatten(-2) if c["inter"] else torch.cat([u, v], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _rope(s):
    c = s["case"]
    B, S = s["q"].shape[:2]
    cos, sin, there = _rotation(s, B, S)
    out = []
    for x, w, y in ((s["q"], s["wq"], s["q_out"]), (s["k"], s["wk"], s["k_out"])):
        x = x.float()
        if c["norm"]:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
        out.append(y.copy_(torch.where(there, _rotated(x, c, cos, sin).to(y.dtype), y)))
    return {"q_out": out[0], "k_out": out[1]}


def _rope_backward(s):
    c = s["case"]
    B, S = s["q"].shape[:2]
    cos, sin, there = _rotation(s, B, S)
    out = {}
    for n in "qk":
        x, w, g = s[n].float(), s["w" + n], _rotated(s[f"d{n}_out"].float(), c, cos, -sin)
        g = torch.where(there, g, torch.zeros_like(g))
        if c["norm"]:
            r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
            xh = x * r
            out["w" + n] = (g * xh).sum((0, 1, 2), dtype=torch.float64).float()
            g = g * w
            g = (g - xh * (g * xh).mean(-1, keepdim=True)) * r
        out["d" + n] = s["d" + n].copy_(g)
    return out


def _tree_masks(s):
    """(tree [T, words] int32, positions [T] int32) from the parents."""
    T, words, cu, kv = s["T"], s["words"], s["cu_q"].long(), s["kv_lens"].long()
    t = torch.arange(T, device="cuda")
    r = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=kv.numel() - 1)
    there = t < cu[-1]
    anc = torch.where(there, t - cu[r], torch.full_like(t, -1))
    masks = torch.zeros(T + 1, words * 32, dtype=torch.bool, device="cuda")
    depth = torch.full_like(t, -1)
    par = s["parents"].long()
    for _ in range(s["max_q"]):
        masks[torch.where(anc >= 0, t, torch.full_like(t, T)), anc.clamp(min=0)] = True
        depth += anc >= 0
        anc = torch.where(anc >= 0, par[(cu[r] + anc).clamp(0, T - 1)], anc)
    bits = masks[:T].view(T, words, 32).long() << torch.arange(32, device="cuda")
    tree = bits.sum(-1)
    tree = torch.where(tree >= 2 ** 31, tree - 2 ** 32, tree).to(torch.int32)
    pos = kv[r] - (cu[r + 1] - cu[r]) + depth
    return tree, torch.where(there, pos, torch.full_like(pos, -1)).to(torch.int32), masks[:T], depth


def _tree(s):
    c, P, T = s["case"], s["P"], s["T"]
    R, Hq, Hkv, d, dv = c["R"], c["Hq"], c["Hkv"], c["d"], c["dv"]
    tree, positions, masks, depth = _tree_masks(s)
    G, Lq, Lk = Hq // Hkv, s["max_q"], s["max_kv"]
    table = s["table"].long().clamp(min=0)
    kv, cu = s["kv_lens"].long(), s["cu_q"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(Lq, device="cuda")
    row = torch.where(i[None] < n[:, None], cu[:-1, None] + i[None], torch.full_like(n, T)[:, None])    # [R, Lq]
    masks = torch.cat([masks, masks.new_zeros(1, masks.shape[1])])[row]                                # [R, Lq, bits]
    depth = torch.cat([depth, depth.new_zeros(1)])[row]
    k = s["k_cache"][table].float() * s["k_scale"][table][..., None, None]      # [R, pages, Hkv, P, d]
    k = k.transpose(1, 2).reshape(R, Hkv, -1, d)[:, :, :Lk]
    q = torch.cat([s["q"], s["q"].new_zeros(1, Hq, d)])[row].float()            # [R, Lq, Hq, d]
    q = q.view(R, Lq, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(R, Hkv, Lq * G, d)
    z = (q @ k.transpose(2, 3)).mul_(d ** -0.5).view(R, Hkv, Lq, G, Lk)
    del k
    key, ctx = torch.arange(Lk, device="cuda"), kv - n
    allowed = (key[None] < ctx[:, None])[:, None].expand(R, Lq, Lk)
    if c["wl"] >= 0:
        allowed = allowed & (key[None, None] >= (ctx[:, None] + depth - c["wl"])[..., None])
    j = key[None] - ctx[:, None]
    own_tokens = (j >= 0) & (key[None] < kv[:, None])
    at = j.clamp(0, masks.shape[2] - 1)[:, None].expand(R, Lq, Lk)
    allowed = allowed | (own_tokens[:, None] & masks.gather(2, at))
    z.masked_fill_(~allowed[:, None, :, None], -math.inf)
    m = z.amax(-1)
    if s["sink"] is not None:
        sink = s["sink"].view(1, Hkv, 1, G)
        m = torch.maximum(m, sink)
    w = z.sub_(torch.where(m > -math.inf, m, torch.zeros_like(m))[..., None]).exp_()
    l = w.sum(-1)
    if s["sink"] is not None:
        l = l + (sink - m).exp()
    v = s["v_cache"][table].float() * s["v_scale"][table][..., None, None]
    v = v.transpose(1, 2).reshape(R, Hkv, -1, dv)[:, :, :Lk]
    v = v.masked_fill((key[None] >= kv[:, None])[:, None, :, None], 0)
    o = w.view(R, Hkv, Lq * G, Lk) @ v
    o = o.view(R, Hkv, Lq, G, dv) / torch.where(l > 0, l, torch.ones_like(l))[..., None]
    dest = row.reshape(-1)
    out = torch.cat([s["o"], s["o"].new_zeros(1, Hq, dv)])
    out[dest] = o.permute(0, 2, 1, 3, 4).reshape(-1, Hq, dv).to(out.dtype)
    stats = torch.cat([torch.stack([s["m"], s["l"]]), s["m"].new_zeros(2, Hq, 1)], 2)
    stats[:, :, dest] = torch.stack([m, l]).permute(0, 2, 4, 1, 3).reshape(2, Hq, -1)
    return {"tree": tree, "positions": positions, "o": out[:T], "m": stats[0, :, :T], "l": stats[1, :, :T]}


def _keep_one(cache, scale, src, dst, there, head_pages, heads):
    """Tokens at slots src to slots dst (where `there`), pages in front of them rescaled."""
    num, H, P, _ = cache.shape
    pages = cache.view(torch.uint8)
    sp, dp = src // P, dst // P
    # a page's scale becomes the largest of what it holds: its own, where tokens in front of the moved
    # ones stay in it, and those of the pages that its kept tokens come from
    hit = torch.zeros(num + 1, dtype=torch.bool, device="cuda")
    hit[torch.where(there, dp, torch.full_like(dp, num))] = True
    top = torch.full((num + 1, H), -1.0, device="cuda")
    at = torch.where(there, dp, torch.full_like(dp, num))[:, None].expand(-1, H)
    top.scatter_reduce_(0, at, torch.where(there[:, None], scale[sp], torch.zeros_like(scale[sp])), "amax")
    staying = torch.zeros(num + 1, dtype=torch.long, device="cuda")
    staying[head_pages] = heads
    top[:num] = torch.where((staying[:num] > 0)[:, None], torch.maximum(top[:num], scale), top[:num])
    new = torch.where(hit[:num, None], top[:num], scale)
    codes = cache[sp, :, src % P].float()                                                  # [tokens, H, c]
    ratio = torch.where(new[dp] > 0, scale[sp] / new[dp], torch.ones_like(new[dp]))
    moved = (codes * ratio[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    hp = torch.where(hit[head_pages], head_pages, torch.zeros_like(head_pages))
    ratio = torch.where(new[hp] > 0, scale[hp] / new[hp], torch.ones_like(new[hp]))
    rows = (cache[hp].float() * ratio[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    front = (torch.arange(P, device="cuda")[None] < heads[:, None]) & (hit[head_pages] & (heads > 0))[:, None]
    r, t = torch.meshgrid(torch.arange(hp.numel(), device="cuda"), torch.arange(P, device="cuda"), indexing="ij")
    pick = front.reshape(-1)
    pages[hp[r.reshape(-1)[pick]], :, t.reshape(-1)[pick]] = rows.transpose(1, 2).reshape(-1, *rows.shape[1:2], rows.shape[3])[pick]
    pages[dp[there], :, (dst % P)[there]] = moved[there]
    scale.copy_(new)


def _keep(s):
    P, kv, cu = s["P"], s["kv_lens"].long(), s["cu_q"].long()
    ctx = kv - (cu[1:] - cu[:-1])
    table, most = s["table"].long().clamp(min=0), s["keep"].shape[1]
    i = torch.arange(most, device="cuda")[None]
    there = (i < s["keep_count"].long()[:, None])
    src, dst = ctx[:, None] + s["keep"].long().clamp(min=0), ctx[:, None] + i
    last = table.shape[1] - 1
    slot = lambda p: table.gather(1, (p // P).clamp(max=last)) * P + p % P                 # noqa: E731
    src, dst = slot(src).reshape(-1), slot(dst).reshape(-1)
    head_pages, heads = table.gather(1, (ctx // P).clamp(max=last)[:, None])[:, 0], ctx % P
    some = s["keep_count"] > 0
    head_pages, heads = head_pages[some], heads[some]
    for n in "kv":
        _keep_one(s[n + "_cache"], s[n + "_scale"], src, dst, there.reshape(-1), head_pages, heads)
    return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _pages_pass(s):
    P, src, dst, table, free = s["P"], s["src"].long(), s["dst"].long(), s["table"], s["free"]
    num = free.numel()
    ctx, count = s["ctx"].long(), s["count"].long()
    col = torch.arange(table.shape[1], device="cuda")[None]
    # fork: full pages are shared, the last one is copied to a page from the end of the free list
    n = ctx[src]
    need = (n % P > 0).long()
    upto = need.cumsum(0)
    ok = (need == 0) | (upto <= count)
    fresh = free[(count - upto).clamp(min=0)]
    rows = table[src]
    shared = (col < (n // P)[:, None]) & ok[:, None]
    s["refs"].index_add_(0, rows.clamp(min=0).reshape(-1).long(), shared.reshape(-1).to(torch.int32))
    last = rows.gather(1, (n // P).clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    none = torch.full_like(last, -1)
    copies = ok & (need > 0)
    copy_src, copy_dst = torch.where(copies, last, none), torch.where(copies, fresh, none)
    new = torch.where(shared, rows, table[dst])
    new = torch.where((col == (n // P)[:, None]) & copies[:, None], fresh[:, None], new)
    table[dst] = new
    ctx = ctx.index_copy(0, dst, torch.where(ok, n, torch.zeros_like(n)))
    count = count - torch.where(ok, need, torch.zeros_like(need)).sum()
    # the copied pages of one layer
    a, b = copy_src[copies].long(), copy_dst[copies].long()
    for x in ("k_cache", "v_cache"):
        s[x].view(torch.uint8)[b] = s[x].view(torch.uint8)[a]
    for x in ("k_scale", "v_scale"):
        s[x][b] = s[x][a]
    # release: pages that no request holds any more go to the end of the free list, ascending
    keep = s["keep_lens"].long()
    out = (col >= _pages(keep, P)[:, None]) & (col < _pages(ctx, P)[:, None])
    s["refs"].index_add_(0, table.clamp(min=0).reshape(-1).long(), -out.reshape(-1).to(torch.int32))
    gone = s["refs"] < 0
    s["refs"].clamp_(min=0)
    at = torch.where(gone, count + gone.long().cumsum(0) - 1, torch.full_like(gone, num, dtype=torch.long))
    ids = torch.arange(num, device="cuda", dtype=torch.int32)
    longer = torch.cat([free, free[:1]])
    longer[at] = ids
    free.copy_(longer[:num])
    count = (count + gone.sum()).to(torch.int32)
    return {"copy_src": copy_src, "copy_dst": copy_dst, "ctx": keep.to(torch.int32), "table": table, "refs": s["refs"],
            "free": free, "count": count, "k_cache": s["k_cache"], "v_cache": s["v_cache"], "k_scale": s["k_scale"],
            "v_scale": s["v_scale"]}


def _own(s):
    from ring_attention_gb300 import bpa
    c = s["case"]
    if c["op"] == "rope":
        kw = dict(norm=c["norm"], eps=EPS, interleaved=c["inter"])
        if c["way"] == "fwd":
            q, k = bpa.bpa_rope_fwd(s["q"], s["k"], s["pos"], s["inv_freq"], s["wq"], s["wk"], q_out=s["q_out"],
                                    k_out=s["k_out"], **kw)
            return {"q_out": q, "k_out": k}
        dq, dk, wq, wk = bpa.bpa_rope_bwd(s["q"], s["k"], s["dq_out"], s["dk_out"], s["pos"], s["inv_freq"], s["wq"],
                                          s["wk"], dq=s["dq"], dk=s["dk"], **kw)
        return {"wq": wq, "dq": dq, "wk": wk, "dk": dk} if c["norm"] else {"dq": dq, "dk": dk}
    cache = [s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")]
    if c["op"] == "tree":
        tree, pos = bpa.bpa_cache_tree(s["parents"], s["kv_lens"], s["cu_q"], words=s["words"])
        o, m, l = bpa.bpa_cache_attn(s["q"], *cache, s["table"], s["kv_lens"], s["cu_q"], max_q=s["max_q"], causal=True,
                                     window=(c["wl"], -1), sink=s["sink"], tree=tree, o=s["o"], m=s["m"], l=s["l"])
        return {"tree": tree, "positions": pos, "o": o, "m": m, "l": l}
    if c["op"] == "keep":
        bpa.bpa_cache_keep(s["keep"], s["keep_count"], s["kv_lens"], s["cu_q"], s["table"], *cache)
        return dict(zip(("k_cache", "v_cache", "k_scale", "v_scale"), cache))
    copy_src, copy_dst, ctx, count = bpa.bpa_cache_fork(s["src"], s["dst"], s["ctx"], s["table"], s["refs"], s["free"],
                                                        s["count"], page_size=s["P"])
    bpa.bpa_cache_copy(copy_src, copy_dst, *cache)
    ctx, count = bpa.bpa_cache_release(ctx, s["keep_lens"], s["table"], s["refs"], s["free"], count, page_size=s["P"])
    return {"copy_src": copy_src, "copy_dst": copy_dst, "ctx": ctx, "table": s["table"], "refs": s["refs"], "free": s["free"],
            "count": count, "k_cache": cache[0], "v_cache": cache[1], "k_scale": cache[2], "v_scale": cache[3]}


def run(s):
    if own:
        return _own(s)
    c = s["case"]
    if c["op"] == "rope":
        return _rope(s) if c["way"] == "fwd" else _rope_backward(s)
    return {"tree": _tree, "keep": _keep, "pages": _pages_pass}[c["op"]](s)


# ---- the definitions in 64 bits -----------------------------------------------------------------
def _exact_rope_of(x, w, c, turn):
    """Norm and rotation of x [B, S, H, d] in 64 bits; turn [B, S, 1, rot / 2], complex of modulus 1."""
    if c["norm"]:
        x = w * x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / c["d"] + EPS)
    rot, head = c["rot"], x[..., :c["rot"]]
    pairs = head.unflatten(-1, (rot // 2, 2)) if c["inter"] else head.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    y = y.flatten(-2) if c["inter"] else y.transpose(-1, -2).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _exact_rope(s):
    c = s["case"]
    B, S = s["q"].shape[:2]
    pos = s["pos"].double() if s["pos"] is not None else torch.arange(S, device="cuda").double().repeat(B, 1)
    there = (pos >= 0)[..., None, None]
    angle = pos[..., None, None] * s["inv_freq"].double()
    turn = torch.polar(torch.ones_like(angle), angle)
    out = {}
    for n in "qk":
        w = s["w" + n].double().requires_grad_() if c["norm"] else None
        if c["way"] == "fwd":
            with torch.no_grad():
                out[n + "_out"] = torch.where(there, _exact_rope_of(s[n].double(), w, c, turn), s[n + "_out"].double())
            continue
        x = s[n].double().requires_grad_()
        y = _exact_rope_of(x, w, c, turn)
        dy = torch.where(there, s[f"d{n}_out"].double(), 0.0)
        got = torch.autograd.grad(y, [x, w] if c["norm"] else [x], dy)
        out["d" + n] = got[0]
        if c["norm"]:
            out["w" + n] = got[1]
    return out


def _exact_tree(s):
    c, P = s["case"], s["P"]
    Hq, Hkv, d, dv = c["Hq"], c["Hkv"], c["d"], c["dv"]
    G, t = Hq // Hkv, 0
    o, m, l = s["o"].double().clone(), s["m"].double().clone(), s["l"].double().clone()
    sinks = s["sink"].double() if s["sink"] is not None else None
    for r, (a, n, par) in enumerate(zip(*_lens(c), _parents(c))):
        if n == 0:
            continue
        L = a + n
        sees, depth = torch.zeros(n, n, dtype=torch.bool), [0] * n
        for i in range(n):
            if par[i] >= 0:
                sees[i] = sees[par[i]]
                depth[i] = depth[par[i]] + 1
            sees[i, i] = True
        off = torch.zeros(n, L, dtype=torch.bool, device="cuda")
        off[:, a:] = ~sees.cuda()
        if c["wl"] >= 0:
            first = torch.tensor([a + x - c["wl"] for x in depth], device="cuda")
            off[:, :a] = torch.arange(a, device="cuda")[None] < first[:, None]
        pages = s["table"][r, :_pages(L, P)].long()
        for g in range(Hkv):
            K = (s["k_cache"][pages, g].double() * s["k_scale"][pages, g].double()[:, None, None]).reshape(-1, d)[:L]
            V = (s["v_cache"][pages, g].double() * s["v_scale"][pages, g].double()[:, None, None]).reshape(-1, dv)[:L]
            for h in range(g * G, (g + 1) * G):
                z = (s["q"][t:t + n, h].double() @ K.T) / math.sqrt(d)
                z[off] = -math.inf
                top = z.amax(1)
                if sinks is not None:
                    top = torch.maximum(top, sinks[h])
                w = torch.exp(z - top[:, None])
                den = w.sum(1) + (torch.exp(sinks[h] - top) if sinks is not None else 0)
                o[t:t + n, h] = (w @ V) / den[:, None]
                m[h, t:t + n], l[h, t:t + n] = top, den
        t += n
    return {"tree": None, "positions": None, "o": o, "m": m, "l": l}


def _round_e4m3(x):
    """To the nearest e4m3 number, ties to even; |x| <= 448."""
    _, e = torch.frexp(x.abs().clamp(min=2.0 ** -6))
    step = torch.exp2((e - 4).double())              # three bits behind the leading one
    return torch.round(x / step) * step


def _exact_keep(s):
    P, out, tables = s["P"], {}, s["table"].tolist()
    for n in "kv":
        code, scale = s[n + "_cache"].double(), s[n + "_scale"].double()
        before, olds = code.clone(), scale.clone()
        for r, (a, path) in enumerate(zip(_lens(s["case"])[0], _paths(s["case"]))):
            for first in range(a // P * P, a + len(path) if path else 0, P):
                page = tables[r][first // P]
                moves = [(i, a + i - first) for i in range(len(path)) if 0 <= a + i - first < P]
                front = max(0, a - first)
                froms = [(tables[r][(a + path[i]) // P], (a + path[i]) % P, to) for i, to in moves]
                if not froms:
                    continue
                all_scales = [olds[p] for p, _, _ in froms] + ([olds[page]] if front else [])
                new = torch.stack(all_scales).amax(0)
                per = torch.where(new > 0, 1 / new, torch.ones_like(new))
                if front:
                    code[page, :, :front] = _round_e4m3(before[page, :, :front] * (olds[page] * per)[:, None, None])
                fp, ft, to = (torch.tensor(x, device="cuda") for x in zip(*froms))
                code[page, :, to] = _round_e4m3(before[fp, :, ft] * (olds[fp] * per)[..., None]).transpose(0, 1)
                scale[page] = new
        out[n + "_cache"], out[n + "_scale"] = code, scale
    return out


def _exact_pages(s):
    """The cache with each child's last page as its parent's; the rest is whole numbers."""
    P, ctx, table, free, left = s["P"], s["ctx"].tolist(), s["table"].tolist(), s["free"].tolist(), s["count"].item()
    out = {n: s[n].double() for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
    for parent in s["src"].tolist():
        if ctx[parent] % P:
            left -= 1
            for x in out.values():
                x[free[left]] = x[table[parent][ctx[parent] // P]]
    return {**dict.fromkeys(("copy_src", "copy_dst", "ctx", "table", "refs", "free", "count")), **out}


def exact(case, seed):
    if case["op"] == "tree" and work(case)["flops"] > 1e12:
        return None
    s = prepare(case, seed)
    return {"rope": _exact_rope, "tree": _exact_tree, "keep": _exact_keep, "pages": _exact_pages}[case["op"]](s)


def work(case):
    c = case
    if c["op"] == "rope":
        rows, heads, e = c["B"] * c["S"], c["Hq"] + c["Hkv"], 2 if c["dtype"] == "bfloat16" else 4
        n, each = rows * heads * c["d"], 2 if c["way"] == "fwd" else 3
        # rows in (backward: the gradients too) and out; positions, frequencies, weights and their gradients
        return {"bytes": n * e * each + 4 * rows * (c["pos_hi"] > 0) + 2 * c["rot"] + 8 * c["d"] * (each - 1) * c["norm"],
                "flops": n * (7 if c["way"] == "fwd" else 14)}
    P, Hkv, per = c["P"], c["Hkv"], c["d"] + c["dv"]
    if c["op"] == "pages":
        A, N, E = c["parents"], c["N"], c["ends"]
        ctx = _spread(A + E, c["ctx_lo"], c["ctx_hi"])
        kids = [ctx[i % A] for i in range(N)]
        copied = sum(n % P > 0 for n in kids)
        shared = sum(n // P for n in kids)
        out = sum(_pages(n, P) - _pages(0 if i % 3 or i % 4 == 0 else max(0, n - 1 - i % 70), P) for i, n in enumerate(ctx[A:]))
        # pages copied with their scales; ids read, written and counted; ids given up; lengths
        return {"bytes": copied * 2 * (Hkv * P * per + 8 * Hkv + 4) + 16 * shared + 16 * out + 16 * (A + N + E), "flops": 0}
    ctx, new = _lens(c)
    if c["op"] == "keep":
        moved = sum(sum(p != i for i, p in enumerate(path)) for path in _paths(c))
        kept = sum(len(path) for path in _paths(c))
        # moved tokens in and out; a scale in and out for each, head and tensor; the paths and lengths
        return {"bytes": 2 * moved * Hkv * per + 4 * kept + 16 * moved // P * Hkv + 12 * c["R"], "flops": moved * Hkv * per}
    esize, Hq, wl = 2 if c["dtype"] == "bfloat16" else 4, c["Hq"], c["wl"]
    pairs = keys = pages = 0
    T = sum(new)
    for a, n, par in zip(ctx, new, _parents(c)):
        depth = []
        for p in par:
            depth.append(0 if p < 0 else depth[p] + 1)
        lo = max(0, a - wl) if wl >= 0 else 0
        if n:
            keys += a + n - lo
            pages += _pages(a + n, P) - lo // P
        pairs += sum(x + 1 + (a if wl < 0 else min(a, max(0, wl - x))) for x in depth)
    words = max(1, _pages(c["new_hi"], 32))
    return {"bytes": keys * Hkv * per + pages * (8 * Hkv + 4) + T * Hq * (per * esize + 8) + T * (8 + 4 * words) + 8 * c["R"],
            "flops": 2 * pairs * Hq * per}
