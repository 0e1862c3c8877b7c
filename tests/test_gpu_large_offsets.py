"""Tensors whose element offsets pass 32 bits: the last rows against the same rows on their own."""
import pytest

from gpu_util import cuda_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]


@pytest.fixture(scope="module")
def nv():
    import nvfp4_bit_precision_b200 as nv
    return nv


def _normal(torch, shape, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    return x.normal_(generator=g)


def test_norm(nv):
    import torch
    rows, cols = 270000, 8192                       # 2.2e9 elements
    x, w = _normal(torch, (rows, cols), 0), _normal(torch, (cols,), 1)
    f = nv.rmsnorm(x, w, x, mx=True, rstd=True, mx_sf_layout=nv.NVFP4_SF_MMA)
    last = x[-256:].clone()                         # (270000 is 112 past a multiple of 128)
    g = nv.rmsnorm(last, w, last, mx=True, rstd=True)
    for a, b in ((f["y"], g["y"]), (f["h"], g["h"]), (f["mx"][0], g["mx"][0]), (f["rstd"], g["rstd"])):
        assert torch.equal(a[-256:], b)
    k32 = cols // 32
    r = torch.arange(rows - 256, rows, device="cuda")[:, None]
    b = torch.arange(k32, device="cuda")[None, :]
    at = ((r // 128) * (k32 // 4) + b // 4) * 512 + (r % 32) * 16 + ((r % 128) // 32) * 4 + b % 4
    assert torch.equal(f["mx"][1][at], g["mx"][1])
    del f
    dx, _ = nv.rmsnorm_backward(x, x, w, nv.rmsnorm(x, w, rstd=True)["rstd"])
    rs = nv.rmsnorm(last, w, rstd=True)["rstd"]
    assert torch.equal(dx[-256:], nv.rmsnorm_backward(last, last, w, rs)[0])


def test_combine(nv):
    import torch
    tokens, k, cols = 67000, 4, 8200                # 2.2e9 elements of rows
    rows = _normal(torch, (tokens * k, cols), 2)
    slot = torch.arange(tokens * k, dtype=torch.int32, device="cuda").flip(0).reshape(tokens, k).contiguous()
    w = torch.rand((tokens, k), device="cuda")
    out = nv.combine(rows, slot, w)
    few = nv.combine(rows[-40:].clone(), slot[:10] - (tokens * k - 40), w[:10].contiguous())
    assert torch.equal(out[:10], few)
    dr, dw = nv.combine_backward(out, rows, slot, w, torch.tensor([0, tokens * k], dtype=torch.int32, device="cuda"))
    a, b = nv.combine_backward(out[:10].contiguous(), rows[-40:].clone(), slot[:10] - (tokens * k - 40),
                               w[:10].contiguous())
    assert torch.equal(dr[-40:], a) and torch.equal(dw[:10], b)


def test_grouped_products(nv):
    import torch
    G, n, k = 160, 8192, 4096                       # 2.7e9 bytes of codes
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    u8 = dict(dtype=torch.uint8, device="cuda")
    q = torch.randint(0, 256, (G, n, k // 2), generator=g, **u8)
    sf = torch.randint(0x30, 0x40, (G, nv.nvfp4_sf_mma_bytes(n, k)), generator=g, **u8)
    gs = torch.rand(G, device="cuda") + 0.5
    x = _normal(torch, (3, k), 4)
    off = torch.zeros(G + 1, dtype=torch.int32)
    off[1:] = 1
    off[G - 1:] = 2
    off[G] = 3
    y = nv.grouped_gemv(off.cuda(), x, q, sf, gs, n, None, nv.NVFP4_OUT_F32)
    for row, e in ((0, 0), (1, G - 2), (2, G - 1)):
        w = nv.dequantize(nv.NVFP4Tensor(q[e], sf[e], gs[e:e + 1], n, k, nv.NVFP4_SF_MMA)).double()
        ref, size = w @ x[row].double(), w.abs() @ x[row].double().abs()
        # the sums as in test_gpu_gemv.py: 8 accumulations of 17 truncated additions, two additions for each of 16
        # steps and 19 more; the dequantised weight's own rounding is another half step of FP32
        assert bool(((y[row].double() - ref).abs() <= ((8 * 17 + 2 * 16 + 19) * 2.0 ** -23 + 2.0 ** -24) * size).all())
