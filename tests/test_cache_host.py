"""The paged 8-bit cache without a GPU: descriptor layouts, the library's refusals (each call here
fails its checks before anything touches a device), the binding's refusals, and pins of the
64-bit oracle that the GPU tests compare with."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from oracle import cache as ora

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def bpa():
    from ring_attention_gb300 import build
    build.build()
    from ring_attention_gb300 import bpa as mod
    return mod


@pytest.mark.parametrize("name", ["bpa_cache_desc", "bpa_cache_batch"])
def test_descriptor_layouts_match_c(tmp_path, bpa, name):
    cls = getattr(bpa, name)
    fields = [f[0] for f in cls._fields_]
    body = "\n".join(f'printf("{f} %zu\\n", offsetof({name}, {f}));' for f in fields)
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "bpa.h"\nint main(void){\n'
                   f'printf("size %zu\\n", sizeof({name}));\n{body}\nreturn 0;}}\n')
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    got = dict(x.split() for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                                 check=True).stdout.splitlines())
    assert int(got["size"]) == ctypes.sizeof(cls)
    for f in fields:
        assert int(got[f]) == getattr(cls, f).offset, f


def _cache(bpa, **over):
    D = bpa.bpa_cache_desc()
    D.struct_size, D.dtype = ctypes.sizeof(D), bpa.BPA_BF16
    D.Hkv, D.d, D.dv, D.page_size, D.num_pages = 2, 64, 64, 16, 100
    D.k_cache = D.v_cache = D.k_scale = D.v_scale = 0x10000      # never dereferenced by host checks
    D.k_cache_strides[:] = D.v_cache_strides[:] = (2 * 16 * 64, 16 * 64, 64)
    for k, v in over.items():
        setattr(D, k, v)
    return D


def _batch(bpa, **over):
    B = bpa.bpa_cache_batch()
    B.struct_size = ctypes.sizeof(B)
    B.R, B.T, B.Hq, B.max_pages = 3, 5, 4, 10
    B.q = B.page_table = B.kv_lens = B.cu_q = 0x20000
    B.q_strides[:] = B.o_strides[:] = (4 * 64, 64)
    B.causal, B.window_left, B.window_right = 1, -1, -1
    for k, v in over.items():
        setattr(B, k, v)
    return B


@pytest.mark.parametrize("cache,batch,status", [
    (dict(struct_size=8), {}, 1), (dict(dtype=5), {}, 1), (dict(reserved=1), {}, 1), (dict(Hkv=0), {}, 1),
    (dict(d=0), {}, 1), (dict(d=513), {}, 2), (dict(dv=513), {}, 2), (dict(page_size=0), {}, 1),
    (dict(page_size=1025), {}, 1), (dict(num_pages=0), {}, 1), (dict(num_pages=1 << 27), {}, 1),
    (dict(k_cache=0), {}, 1), (dict(v_scale=0), {}, 1),
    ({}, dict(struct_size=4), 1), ({}, dict(R=0), 1), ({}, dict(T=-1), 1), ({}, dict(T=(1 << 30) + 1), 1),
    ({}, dict(Hq=3), 1), ({}, dict(max_pages=0), 1), ({}, dict(max_pages=1 << 27), 1), ({}, dict(max_q=-1), 1),
    ({}, dict(window_left=-2), 1), ({}, dict(q=0), 1), ({}, dict(cu_q=0), 1), ({}, dict(page_table=0), 1),
])
def test_attention_refuses(bpa, cache, batch, status):
    L, p = bpa.lib(), 0x40000
    st = L.bpa_cache_attn(ctypes.byref(_cache(bpa, **cache)), ctypes.byref(_batch(bpa, **batch)), p, p, p, p, 1 << 40,
                          None)
    assert st == status, L.bpa_last_error()
    assert L.bpa_last_error() != b""


def test_attention_workspace_and_statistics(bpa):
    L, p = bpa.lib(), 0x40000
    c, b = _cache(bpa), _batch(bpa)
    need = L.bpa_cache_attn_workspace_size(ctypes.byref(c), ctypes.byref(b))
    assert need >= 256 and need % 256 == 0
    assert L.bpa_cache_attn_workspace_size(ctypes.byref(_cache(bpa, d=0)), ctypes.byref(b)) == 0
    call = lambda m, l, ws, n: L.bpa_cache_attn(ctypes.byref(c), ctypes.byref(b), p, m, l, ws, n, None)  # noqa: E731
    assert call(p, p, None, need) == 3 and call(p, p, p + 16, need) == 3 and call(p, p, p, need - 1) == 3
    assert call(p, None, p, need) == 1 and call(None, p, p, need) == 1


def test_append_refuses(bpa):
    L, p = bpa.lib(), 0x40000
    s2 = (ctypes.c_int64 * 2)(128, 64)
    neg = (ctypes.c_int64 * 2)(-128, 64)
    call = lambda c, T=4, new=0, k=p, slots=p, ks=s2, ws=p, n=256: L.bpa_cache_append(  # noqa: E731
        ctypes.byref(c), k, p, ks, s2, slots, T, new, ws, n, None)
    assert call(_cache(bpa, page_size=2000)) == 1
    assert call(_cache(bpa, k_scale=0)) == 1
    assert call(_cache(bpa, d=600)) == 2
    for bad in (dict(T=-1), dict(new=-1), dict(k=None), dict(slots=None), dict(ks=neg)):
        assert call(_cache(bpa), **bad) == 1, bad
    assert call(_cache(bpa), n=255) == 3 and call(_cache(bpa), ws=None) == 3
    assert call(_cache(bpa), T=1 << 30) == 2
    flat = _cache(bpa)
    flat.k_cache_strides[1] = 0                  # heads over one another: read at most, never written
    assert call(flat) == 1


def test_plan_refuses(bpa):
    L, p = bpa.lib(), 0x40000

    def call(R=2, T=8, P=16, pages=10, width=4, ptrs=None, ws=p, n=256):
        return L.bpa_cache_plan(R, T, P, pages, width, *(ptrs or [p] * 11), ws, n, None)

    for bad, status in ((dict(R=0), 1), (dict(R=8193), 2), (dict(T=-1), 1), (dict(T=(1 << 30) + 1), 1), (dict(P=0), 1),
                        (dict(P=1025), 1), (dict(pages=0), 1), (dict(pages=1 << 27), 1), (dict(width=0), 1),
                        (dict(width=1 << 27), 1), (dict(ws=None), 3), (dict(ws=p + 8), 3), (dict(n=255), 3)):
        assert call(**bad) == status, bad
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 9, 10):     # every buffer but positions
        ptrs = [p] * 11
        ptrs[i] = None
        assert call(ptrs=ptrs) == 1, i


# ---- the binding's own checks ------------------------------------------------------------------
def _tensors(R=3, T=5, Hq=4, Hkv=2, d=64, dv=32, P=16, pages=20, dtype=torch.bfloat16):
    return dict(q=torch.zeros(T, Hq, d, dtype=dtype), k_cache=torch.zeros(pages, Hkv, P, d, dtype=torch.uint8),
                v_cache=torch.zeros(pages, Hkv, P, dv, dtype=torch.uint8), k_scale=torch.ones(pages, Hkv),
                v_scale=torch.ones(pages, Hkv), page_table=torch.zeros(R, 4, dtype=torch.int32),
                kv_lens=torch.ones(R, dtype=torch.int32), cu_q=torch.zeros(R + 1, dtype=torch.int32))


def test_descriptors_from_tensors(bpa):
    t = _tensors()
    D = bpa.make_cache_desc(t["k_cache"], t["v_cache"], t["k_scale"], t["v_scale"], torch.bfloat16)
    assert (D.Hkv, D.d, D.dv, D.page_size, D.num_pages) == (2, 64, 32, 16, 20)
    assert tuple(D.k_cache_strides) == (2 * 16 * 64, 16 * 64, 64)
    nhd = torch.zeros(20, 16, 2, 64, dtype=torch.float8_e4m3fn).transpose(1, 2)
    D = bpa.make_cache_desc(nhd, t["v_cache"], t["k_scale"], t["v_scale"], torch.float32)
    assert tuple(D.k_cache_strides) == (16 * 2 * 64, 64, 2 * 64) and D.dtype == bpa.BPA_FP32
    B = bpa.make_cache_batch(t["q"], t["page_table"], t["kv_lens"], t["cu_q"], max_q=2, window=(7, -1), scale=0.5)
    assert (B.R, B.T, B.Hq, B.max_pages, B.max_q, B.causal) == (3, 5, 4, 4, 2, 1)
    assert (B.window_left, B.window_right, B.scale) == (7, -1, 0.5)


@pytest.mark.parametrize("bad", [
    dict(k_cache=torch.zeros(20, 2, 16, 64, dtype=torch.int8)), dict(k_cache=torch.zeros(20, 2, 64, dtype=torch.uint8)),
    dict(v_cache=torch.zeros(20, 2, 32, 32, dtype=torch.uint8)), dict(k_scale=torch.ones(20, 2, dtype=torch.float64)),
    dict(v_scale=torch.ones(2, 20).T), dict(k_scale=torch.ones(19, 2)), dict(kv_lens=torch.ones(3, dtype=torch.int64)),
    dict(cu_q=torch.zeros(3, dtype=torch.int32)), dict(page_table=torch.zeros(3, 8, dtype=torch.int32)[:, ::2]),
    dict(q=torch.zeros(5, 4, 32, dtype=torch.bfloat16)), dict(q=torch.zeros(5, 64, 4, dtype=torch.bfloat16).transpose(1, 2)),
    dict(sink=torch.zeros(3)), dict(m=torch.zeros(5, 4)), dict(o=torch.zeros(5, 4, 64, dtype=torch.bfloat16)),
    dict(),     # all well but on the CPU
], ids=["k_int8", "k_3d", "v_page", "scale_f64", "scale_strided", "scale_rows", "lens_i64", "cu_len", "table_strided",
        "q_dim", "q_strided", "sink_len", "m_shape", "o_dim", "cpu"])
def test_binding_refuses_attention(bpa, bad):
    t = {**_tensors(), **bad}
    with pytest.raises(ValueError):
        bpa.bpa_cache_attn(t.pop("q"), **t)


def test_binding_refuses_types(bpa):
    t = _tensors(dtype=torch.float16)
    with pytest.raises(TypeError):
        bpa.bpa_cache_attn(t.pop("q"), **t)


@pytest.mark.parametrize("bad", [dict(v=torch.zeros(5, 2, 32)), dict(v=torch.zeros(4, 2, 32, dtype=torch.bfloat16)),
                                 dict(k=torch.zeros(5, 3, 64, dtype=torch.bfloat16)),
                                 dict(slot_map=torch.zeros(5, dtype=torch.int64)), dict()],
                         ids=["v_type", "v_rows", "k_heads", "slots_i64", "cpu"])
def test_binding_refuses_append(bpa, bad):
    t = _tensors()
    a = dict(k=torch.zeros(5, 2, 64, dtype=torch.bfloat16), v=torch.zeros(5, 2, 32, dtype=torch.bfloat16),
             slot_map=torch.zeros(5, dtype=torch.int32), **{n: t[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")})
    with pytest.raises(ValueError):
        bpa.bpa_cache_append(**{**a, **bad})


@pytest.mark.parametrize("bad", [dict(new_lens=torch.zeros(2, dtype=torch.int32)), dict(free_count=torch.zeros(2, dtype=torch.int32)),
                                 dict(page_table=torch.zeros(2, 4, dtype=torch.int32)),
                                 dict(slot_map=torch.zeros(7, dtype=torch.int32)),
                                 dict(free_pages=torch.zeros(9, dtype=torch.int64)), dict()],
                         ids=["new_len", "count_len", "table_rows", "slots_len", "free_i64", "cpu"])
def test_binding_refuses_plan(bpa, bad):
    i32 = dict(dtype=torch.int32)
    a = dict(ctx_lens=torch.zeros(3, **i32), new_lens=torch.zeros(3, **i32), page_table=torch.zeros(3, 4, **i32),
             free_pages=torch.zeros(9, **i32), free_count=torch.zeros(1, **i32), page_size=16, T=8)
    with pytest.raises(ValueError):
        bpa.bpa_cache_plan(**{**a, **bad})


# ---- pins of the oracle ----------------------------------------------------------------------------
def test_oracle_codes():
    v = ora.e4m3_values()
    assert v[0x7E] == 448 and v[1] == 2.0 ** -9 and v[0x38] == 1 and np.isnan(v[0x7F]) and v[0xB8] == -1
    fin = np.arange(256)[np.isfinite(v)]
    np.testing.assert_array_equal(ora.e4m3_round(v[fin]), fin)
    np.testing.assert_array_equal(v, torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy())
    mid = (v[:126] + v[1:127]) / 2                       # ties go to the even code
    np.testing.assert_array_equal(ora.e4m3_round(mid) % 2, 0)
    x = np.random.default_rng(0).standard_normal(20000).astype(np.float32) * 40
    np.testing.assert_array_equal(ora.e4m3_round(x),
                                  torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_oracle_scales():
    assert ora.scale_for(0.0) == 0 and ora.scale_for(448.0) == 1 and ora.scale_for(448.1) == 2
    assert ora.scale_for(1.75) == 2.0 ** -8 and ora.scale_for(1e-38) == 2.0 ** -100


def test_oracle_plan_by_hand():
    table = np.full((3, 3), -1)
    table[1, 0] = 7
    kv, cu, slots, pos, ctx, table, left = ora.plan([0, 3, 0], [5, 2, 9], table, [10, 11, 12], 3, 4, 17)
    # request 0 takes 12, 11; request 1 takes 10 for its fifth token; request 2 has to wait
    assert kv.tolist() == [5, 5, 0] and ctx.tolist() == [5, 5, 0] and left == 0 and cu.tolist() == [0, 5, 7, 16]
    assert table.tolist() == [[12, 11, -1], [7, 10, -1], [-1, -1, -1]]
    assert slots.tolist() == [48, 49, 50, 51, 44, 31, 40] + [-1] * 10
    assert pos.tolist() == [0, 1, 2, 3, 4, 3, 4] + [-1] * 10


def test_oracle_append_rescales():
    codes, scale = np.zeros((1, 1, 4, 1), np.uint8), np.zeros((1, 1))
    codes, scale = ora.append(np.full((1, 1, 1), 1.0), [0], codes, scale)
    assert scale[0, 0] == 2.0 ** -8 and ora.e4m3_values()[codes[0, 0, 0, 0]] == 256
    codes, scale = ora.append(np.full((1, 1, 1), 3.0), [1], codes, scale)
    assert scale[0, 0] == 2.0 ** -7 and ora.e4m3_values()[codes[0, 0, :2, 0]].tolist() == [128, 384]


def test_oracle_attention_closed_forms():
    # equal keys: the mean of the values that the mask leaves; rows without keys are empty
    rng = np.random.default_rng(1)
    k = np.full((2, 1, 4, 8), 0x38, np.uint8)
    v = rng.integers(0, 0x7E, (2, 1, 4, 8)).astype(np.uint8)
    s = np.array([[0.5], [2.0]])
    val = ora.e4m3_values()[v] * s[:, :, None, None]
    val = np.concatenate([val[1, 0], val[0, 0]])
    q = rng.standard_normal((3, 1, 8))
    o, m, l = ora.attention(q * 0, k, v, s, s, np.array([[1, 0], [0, 0]]), [6, 0], [0, 2, 3], window=(3, -1))
    np.testing.assert_allclose(o[0, 0], val[1:5].mean(0))
    np.testing.assert_allclose(o[1, 0], val[2:6].mean(0))
    assert l[0].tolist() == [4, 4, 0] and m[0, 2] == -np.inf and not o[2].any()


# ---- calls on another stream than torch's current one --------------------------------------------------
class _Fake:
    """A CPU tensor that says it is on GPU 0 and remembers the stream that was current when it was made."""

    def __init__(self, t, made_on=None):
        self.t, self.made_on, self.recorded = t, made_on, []

    def get_device(self):
        return 0

    def record_stream(self, s):
        self.recorded.append(s.cuda_stream)

    def __getattr__(self, name):
        return getattr(self.t, name)


class _Stream:
    def __init__(self, ptr, index=0):
        self.cuda_stream, self.device = ptr, torch.device("cuda", index)


@pytest.fixture
def streams(bpa, monkeypatch):
    """The binding over a library and an allocator that note streams: (current stream, made tensors, launches)."""
    now, made, launched = [_Stream(0x10)], [], []

    class Enter:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            now.append(self.s)

        def __exit__(self, *_):
            now.pop()

    def empty(shape, dtype=None, device=None):
        made.append(_Fake(torch.empty(shape, dtype=dtype), now[-1].cuda_stream))
        return made[-1]

    class Lib:
        bpa_cache_attn_workspace_size = staticmethod(lambda *a: 512)

        def __getattr__(self, name):
            return lambda *a: launched.append((name, a[-1])) or 0

    monkeypatch.setattr(bpa, "_empty", empty)
    monkeypatch.setattr(bpa, "_current_device", lambda: 0)
    monkeypatch.setattr(bpa, "lib", Lib)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: now[-1].cuda_stream, raising=False)
    monkeypatch.setattr(torch.cuda, "stream", Enter)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: now[-1])
    return now, made, launched


def _cache_calls(bpa):
    f = {n: _Fake(x) for n, x in _tensors().items()}
    i32 = dict(dtype=torch.int32)
    rows = dict(k=_Fake(torch.zeros(5, 2, 64, dtype=torch.bfloat16)), v=_Fake(torch.zeros(5, 2, 32, dtype=torch.bfloat16)),
                slot_map=_Fake(torch.zeros(5, **i32)), **{n: f[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")})
    plan = dict(ctx_lens=_Fake(torch.zeros(3, **i32)), new_lens=_Fake(torch.zeros(3, **i32)),
                page_table=_Fake(torch.zeros(3, 4, **i32)), free_pages=_Fake(torch.zeros(9, **i32)),
                free_count=_Fake(torch.zeros(1, **i32)), page_size=16, T=8)
    return {"plan": lambda **kw: bpa.bpa_cache_plan(**plan, **kw), "append": lambda **kw: bpa.bpa_cache_append(**rows, **kw),
            "attn": lambda **kw: bpa.bpa_cache_attn(**f, **kw)}


@pytest.mark.parametrize("name", ["plan", "append", "attn"])
def test_buffers_are_made_on_the_stream_that_uses_them(bpa, streams, name):
    # memory that the current stream may still be writing must not be handed to another stream's kernels
    now, made, launched = streams
    call = _cache_calls(bpa)[name]
    returned = call(stream=_Stream(0x20)) or ()
    assert [p for _, p in launched] == [0x20] and len(now) == 1
    assert made and all(t.made_on == 0x20 for t in made)
    assert all(t.recorded == [0x10] for t in returned)      # they may be used, and dropped, on the current one
    made.clear()
    returned = call() or ()
    assert launched[-1][1] == 0x10 and all(t.made_on == 0x10 for t in made)
    assert not any(t.recorded for t in made)


@pytest.mark.parametrize("name", ["plan", "append", "attn"])
def test_streams_of_another_device_are_refused(bpa, streams, name):
    now, made, launched = streams
    for ptr in (0x10, 0x20):
        with pytest.raises(ValueError, match="stream"):
            _cache_calls(bpa)[name](stream=_Stream(ptr, 1))
    assert not launched and not made and len(now) == 1


def test_a_failed_call_leaves_the_other_stream(bpa, streams, monkeypatch):
    now, made, launched = streams

    def fails(*a, **kw):
        raise RuntimeError("out of memory")

    monkeypatch.setattr(bpa, "_empty", fails)
    for call in _cache_calls(bpa).values():
        with pytest.raises(RuntimeError):
            call(stream=_Stream(0x20))
    assert len(now) == 1 and not launched


# ---- sizes past 32 bits --------------------------------------------------------------------------------
def test_rows_of_a_kv_head_past_two_to_the_30(bpa):
    """Kernels that number a request's rows (tokens times q heads of a kv head) in 32 bits are left to calls of at most
    2^30; the kernel for any shape, which numbers tokens and heads apart, takes the rest: its workspace is
    the header alone."""
    L = bpa.lib()

    def need(T, Hq, Hkv):
        return L.bpa_cache_attn_workspace_size(ctypes.byref(_cache(bpa, Hkv=Hkv)), ctypes.byref(_batch(bpa, T=T, Hq=Hq)))

    assert need(1 << 20, 1 << 10, 1) > 256 and need(1 << 27, 64, 8) > 256
    assert need((1 << 20) + 1, 1 << 10, 1) == 256 and need(1 << 30, 2, 1) == 256 and need(1 << 16, 65535, 1) == 256


# ---- arguments that would reach memory that is not theirs ----------------------------------------------
@pytest.mark.parametrize("name", ["plan", "append", "attn"])
def test_binding_refuses_workspaces_that_are_not_memory_of_the_device(bpa, streams, name):
    now, made, launched = streams
    call = _cache_calls(bpa)[name]
    for bad in (torch.zeros(1024, dtype=torch.uint8),                             # the CPU's
                _Fake(torch.zeros(1, dtype=torch.uint8).expand(1024)),            # one byte
                _Fake(torch.zeros(2048, dtype=torch.uint8)[::2]), _Fake(torch.zeros(1024, dtype=torch.int32))):
        with pytest.raises(ValueError, match="workspace"):
            call(workspace_buf=bad)
    assert not launched and not made
    call(workspace_buf=_Fake(torch.zeros(1024, dtype=torch.uint8)))
    assert len(launched) == 1


def test_attention_refuses_outputs_that_lie_over_one_another(bpa):
    # strides of 0 (a descriptor whose o_strides were never filled in): rows would overwrite one another
    L, p = bpa.lib(), 0x40000

    def call(row, head, **over):
        b = _batch(bpa, **over)
        b.o_strides[:] = (row, head)
        return L.bpa_cache_attn(ctypes.byref(_cache(bpa)), ctypes.byref(b), p, p, p, p, 256, None)

    assert call(0, 64) == 1 and b"o_strides" in L.bpa_last_error()
    assert call(256, 0) == 1 and b"o_strides" in L.bpa_last_error()
    assert call(256, 64) == 3                            # past that check: the workspace is too small
    assert call(0, 64, T=1) == 3                         # a single row never steps


# ---- numbers that 32 bits do not hold --------------------------------------------------------------------
@pytest.mark.parametrize("name,kw", [("plan", dict(T=(1 << 32) + 8)), ("plan", dict(page_size=(1 << 32) + 16)), ("plan", dict(T=-(1 << 32) + 8)),
                                     ("append", dict(max_new=1 << 32)), ("attn", dict(max_q=1 << 32)),
                                     ("attn", dict(window=(1 << 31, -1))), ("attn", dict(window=(-1, -(1 << 33))))],
                         ids=["T", "page_size", "T_negative", "max_new", "max_q", "left", "right"])
def test_binding_refuses_numbers_past_32_bits(bpa, streams, name, kw):
    now, made, launched = streams
    f = {n: _Fake(x) for n, x in _tensors().items()}
    i32 = dict(dtype=torch.int32)
    args = {"plan": dict(ctx_lens=_Fake(torch.zeros(3, **i32)), new_lens=_Fake(torch.zeros(3, **i32)), page_table=_Fake(torch.zeros(3, 4, **i32)),
                         free_pages=_Fake(torch.zeros(9, **i32)), free_count=_Fake(torch.zeros(1, **i32)), page_size=16, T=8),
            "append": dict(k=_Fake(torch.zeros(5, 2, 64, dtype=torch.bfloat16)), v=_Fake(torch.zeros(5, 2, 32, dtype=torch.bfloat16)),
                           slot_map=_Fake(torch.zeros(5, **i32)), **{n: f[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}),
            "attn": f}[name]
    with pytest.raises(ValueError, match="2\\^31"):
        getattr(bpa, "bpa_cache_" + name)(**{**args, **kw})
    assert not launched and not made
