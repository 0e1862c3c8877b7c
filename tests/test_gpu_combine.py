"""The combine and its gradients on the GPU against 64-bit restatements.  A sum of k products and a base in
FP32 is off by (k + 1) 2^-24 of the terms' magnitudes, a dot product of n columns by (n / 8 + 16) 2^-24 at
most (each thread adds its columns, then a tree); one rounding to bf16 adds 2^-8 of the value."""
import numpy as np
import pytest

import moe_ref as R
import workloads as W
from gpu_util import cuda_available, host, to_dev

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]

B = 2.0 ** -8
U = 2.0 ** -24


def bits(rng, shape, std=1.0):
    return W.f32_to_bf16_bits(rng.standard_normal(shape).astype(np.float32) * np.float32(std))


def val(b):
    return W.bf16_bits_to_f32(b).astype(np.float64)


def f64(t):
    return val(host(t)) if t.dtype.itemsize == 2 else host(t).astype(np.float64)


def make(rng, tokens, k, cols, f32, drop=0.0):
    """Rows, an injective slot_row with some slots dropped, and weights."""
    import torch
    n = tokens * k
    rows = rng.standard_normal((n, cols)).astype(np.float32) if f32 else None
    b = None if f32 else bits(rng, (n, cols))
    rd = torch.from_numpy(rows).cuda() if f32 else to_dev(b)
    slot = rng.permutation(n).astype(np.int32).reshape(tokens, k)
    slot[rng.random((tokens, k)) < drop] = -1
    w = rng.standard_normal((tokens, k)).astype(np.float32)
    return (rows.astype(np.float64) if f32 else val(b)), rd, slot, w


@pytest.mark.parametrize("tokens,k,cols", [(1, 1, 8), (1, 4, 4096), (3, 2, 264), (17, 5, 1000), (130, 8, 128),
                                           (2, 64, 32), (700, 3, 64), (9, 4, 8200)])
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("base", [True, False])
@pytest.mark.parametrize("drop", [0.0, 0.4])
def test_forward_and_backward(tokens, k, cols, f32, base, drop):
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(tokens * 11 + cols)
    rows, rd, slot, w = make(rng, tokens, k, cols, f32, drop)
    bb = bits(rng, (tokens, cols)) if base else None
    sd, wd = torch.from_numpy(slot).cuda(), torch.from_numpy(w).cuda()
    out = nv.combine(rd, sd, wd, to_dev(bb) if base else None)
    ref = R.combine(rows, slot, w, val(bb) if base else None)
    mag = R.combine(np.abs(rows), slot, np.abs(w), np.abs(val(bb)) if base else None)
    assert np.all(np.abs(f64(out) - ref) <= B * np.abs(ref) + (k + 1) * U * mag + 2.0 ** -134)
    dout = bits(rng, (tokens, cols), 1e-2)
    ws = torch.empty(nv.nvfp4_combine_backward_workspace_size(rows.shape[0]), dtype=torch.uint8, device="cuda")
    dr, dw = nv.combine_backward(to_dev(dout), rd, sd, wd, workspace=ws)
    rr, rw = R.combine_backward(val(dout), rows, slot, w)
    assert dr.dtype == rd.dtype and nv.nvfp4_workspace_status(ws) == 0
    assert np.all(np.abs(f64(dr) - rr) <= ((0 if f32 else B) + U) * np.abs(rr) + 2.0 ** -134)
    _, mw = R.combine_backward(np.abs(val(dout)), np.abs(rows), slot, w)
    assert np.all(np.abs(f64(dw) - rw) <= (cols / 8 + 16) * U * mw)


def test_formula_against_differences():
    rng = np.random.default_rng(2)
    rows, slot = rng.standard_normal((6, 5)), np.array([[0, 3], [5, -1]])
    w, dout = rng.standard_normal((2, 2)), rng.standard_normal((2, 5))
    dr, dw = R.combine_backward(dout, rows, slot, w)
    u, v, d = rng.standard_normal(rows.shape), rng.standard_normal(w.shape), 1e-5
    loss = lambda a, b: float((R.combine(a, slot, b) * dout).sum())
    num = (loss(rows + d * u, w + d * v) - loss(rows - d * u, w - d * v)) / (2 * d)
    assert abs(num - ((dr * u).sum() + (dw * v).sum())) <= 1e-8


def test_bad_indexes():
    """A row past the end is left out and reported; a row that two slots name is, in the backward pass."""
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(3)
    rows, rd, _, _ = make(rng, 4, 2, 64, False)
    slot = np.array([[0, 8], [1, 2], [3, 2147483647], [-5, 4]], dtype=np.int32)
    w = rng.standard_normal((4, 2)).astype(np.float32)
    sd, wd = torch.from_numpy(slot).cuda(), torch.from_numpy(w).cuda()
    ws = torch.zeros(512, dtype=torch.uint8, device="cuda")
    out = nv.combine(rd, sd, wd, workspace=ws)
    assert nv.nvfp4_workspace_status(ws) == 8
    ref = R.combine(rows, slot, w)
    assert np.all(np.abs(f64(out) - ref) <= B * np.abs(ref) + 3 * U * R.combine(np.abs(rows), slot, np.abs(w)))
    dout = to_dev(bits(rng, (4, 64)))
    nv.combine_backward(dout, rd, sd, wd, workspace=ws)
    assert nv.nvfp4_workspace_status(ws) == 8
    twice = torch.tensor([[0, 1], [2, 3], [4, 5], [6, 1]], dtype=torch.int32, device="cuda")
    dr, dw = nv.combine_backward(dout, rd, twice, wd, workspace=ws)
    assert nv.nvfp4_workspace_status(ws) == 8
    assert nv.nvfp4_workspace_status(ws) == 0
    ok = torch.tensor([[0, 1], [2, 3], [4, 5], [6, 7]], dtype=torch.int32, device="cuda")
    nv.combine_backward(dout, rd, ok, wd, workspace=ws)
    assert nv.nvfp4_workspace_status(ws) == 0


def test_rows_behind_the_last_one():
    """With the routing's offsets the tail's gradient is zero, whatever the buffer held."""
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(4)
    rd = to_dev(bits(rng, (12, 64)))
    slot = torch.tensor([[0, 1], [2, -1], [3, 4]], dtype=torch.int32, device="cuda")
    w = torch.ones((3, 2), device="cuda")
    off = torch.tensor([0, 3, 5], dtype=torch.int32, device="cuda")
    dout = to_dev(bits(rng, (3, 64)))
    dr = torch.full((12, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.empty((3, 2), device="cuda")
    ws = torch.empty(512, dtype=torch.uint8, device="cuda")
    nv.nvfp4_combine_backward(dout, rd, nv.NVFP4_OUT_BF16, 12, 64, slot, w, 3, 2, off.data_ptr() + 8, dr, dw, ws, 512)
    assert bool((dr[5:] == 0).all()) and torch.equal(dr[:5], dout[[0, 0, 1, 2, 2]])
    a, _ = nv.combine_backward(dout, rd, slot, w, off)
    b, _ = nv.combine_backward(dout, rd, slot, w)
    assert torch.equal(a, dr) and torch.equal(b, dr)


def test_no_tokens():
    import torch
    import nvfp4_bit_precision_b200 as nv
    e = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    w = torch.empty((0, 2), device="cuda")
    rows = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda")
    assert nv.combine(rows, e, w).shape == (0, 64)
    dr, dw = nv.combine_backward(rows[:0], rows, e, w)
    assert bool((dr == 0).all()) and dw.shape == (0, 2)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert bool((nv.combine_backward(rows[:0], rows, e, w, off)[0] == 0).all())
