"""Weights of the attention under trees keep eleven bits: the bound of test_gpu_cache's test of the calls without trees
(its text has the arithmetic), on each kernel."""
import numpy as np
import pytest
import torch

from oracle import cache as ora
from tests.test_gpu_cache import DTYPES, as_dtype, f64, i32, on_gpu
from tests.test_gpu_trees import bpa  # noqa: F401

pytestmark = pytest.mark.gpu

KERNELS = {  # R, rows, Hq, Hkv, d, dv, P, whether the table has room for the keys that the tensor cores are worth
    "few_rows": (20, 1, 64, 8, 64, 64, 64, False), "more_rows": (3, 40, 32, 16, 128, 64, 64, False),
    "half_a_tile": (2, 40, 32, 16, 64, 64, 64, True), "whole_tiles": (2, 60, 64, 16, 128, 128, 64, True), "any_shape": (4, 3, 32, 8, 72, 40, 8, False)}


@DTYPES
@pytest.mark.parametrize("own", [False, True], ids=["context", "masks"])
@pytest.mark.parametrize("kernel", KERNELS)
def test_weights_keep_eleven_bits(bpa, kernel, own, dtype):  # noqa: F811
    """Two keys of scores delta and 0 with values 1 and -1, in front of the step's tokens (masks of nothing) or its first
    two (masks of 3): o = tanh(delta / 2).  The weights' own part is half a step of fp16, 2^-11 (float32: two halves,
    2^-21); weights of bf16 would break the bound, which is checked first."""
    R, rows, Hq, Hkv, d, dv, P, room = KERNELS[kernel]
    T, ctx = R * rows, 0 if own else 2
    if own and rows < 2:
        ctx, rows, R = 0, 2, R // 2
        T = R * rows
    pages = -(-(ctx + rows) // P)
    q = np.zeros((T, Hq, d))
    q[..., 0] = np.linspace(0, 0.02, T * Hq).reshape(T, Hq)
    c = dict(q=q, kc=np.zeros((pages, Hkv, P, d), np.uint8), vc=np.zeros((pages, Hkv, P, dv), np.uint8), ks=np.ones((pages, Hkv), np.float32),
             vs=np.ones((pages, Hkv), np.float32), table=np.tile(np.arange(pages), (R, 1)), kv=np.full(R, ctx + rows), cu=np.arange(R + 1) * rows)
    c["kc"][0, :, 0, 0], c["vc"][0, :, 0], c["vc"][0, :, 1] = 0x38, 0x38, 0xB8      # 1, 1 and -1
    tree = np.zeros((T, 2), int)
    tree[:, 0] = 3 if own else 0
    delta = as_dtype(q, dtype)[1][..., :1]
    want = np.tanh(delta / 2)
    exact = ora.attention(as_dtype(q, dtype)[1], *(c[n] for n in ("kc", "vc", "ks", "vs", "table", "kv", "cu")), scale=1.0, tree=tree)[0]
    np.testing.assert_allclose(exact, np.broadcast_to(want, exact.shape), atol=1e-12)
    half, weight = (2.0 ** -8, 2.0 ** -11) if dtype == torch.bfloat16 else (2.0 ** -24, 2.0 ** -21)
    dz = (d + 4) * 2.0 ** -23 * 0.02 + 2.0 ** -21
    bound = half * np.abs(want) + (2 * dz + weight + 2 * 2.0 ** -23 + 2 * 2.0 ** -32 * 448) * (1 + half)
    low = torch.from_numpy(np.exp(-delta)).to(torch.bfloat16).double().numpy()
    assert (np.abs((1 - low) / (1 + np.exp(-delta)) - want) > bound).any()
    if room:
        c["table"] = np.concatenate([c["table"], np.full((R, 2 ** 18 // P), -1)], 1)
    o, m, l = bpa.bpa_cache_attn(*on_gpu(c, dtype), max_q=rows, scale=1.0, tree=i32(tree))
    torch.cuda.synchronize()
    assert (np.abs(f64(o) - want) <= bound).all()
