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


@pytest.mark.parametrize("tokens,k,cols", [(3, 2, 8), (40, 4, 264), (700, 3, 64), (5000, 4, 128), (9, 4, 8200)])
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("checked", [True, False])
def test_slots_dropped_after_routing(tokens, k, cols, f32, checked):
    """Rows below the routing's last one whose slots were taken out, or that a bad index left out, get a zero
    gradient, whatever the buffer held: here NaN, and numbers of slots that name other rows or none."""
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(tokens + cols)
    rows, rd, slot, w = make(rng, tokens, k, cols, f32, 0.3)
    n = tokens * k
    slot[0, 0], slot[-1, -1] = 2147483647, -7
    dout = bits(rng, (tokens, cols), 1e-2)
    sd, wd, dd = torch.from_numpy(slot).cuda(), torch.from_numpy(w).cuda(), to_dev(dout)
    off = torch.tensor([0, n // 2, n], dtype=torch.int32, device="cuda")
    rr, rw = R.combine_backward(val(dout), rows, slot, w)
    named = np.zeros(n, dtype=bool)
    named[slot[(slot >= 0) & (slot < n)]] = True
    assert not named.all()
    ws = torch.empty(nv.nvfp4_combine_backward_workspace_size(n), dtype=torch.uint8, device="cuda") if checked else None
    for fill in ("nan", "numbers"):
        dr = torch.full_like(rd, float("nan"))
        if fill == "numbers":  # a 64-bit number at the head of each row
            head = dr.view(torch.int64).view(n, -1)
            head[:, 0] = torch.from_numpy(rng.integers(-2, n + 2, n)).cuda()
        dw = torch.full((tokens, k), float("nan"), device="cuda")
        nv.nvfp4_combine_backward(dd, rd, nv.NVFP4_OUT_F32 if f32 else nv.NVFP4_OUT_BF16, n, cols, sd, wd, tokens, k,
                                  off.data_ptr() + 8, dr, dw, ws, 0 if ws is None else ws.numel())
        assert bool((dr[torch.from_numpy(~named).cuda()] == 0).all())
        assert np.all(np.abs(f64(dr) - rr) <= ((0 if f32 else B) + U) * np.abs(rr) + 2.0 ** -134)
        assert checked is False or nv.nvfp4_workspace_status(ws) == 8
    spoil = torch.full_like(rd, float("nan"))
    del spoil                                   # the wrapper's buffer is likely this memory
    a, b = nv.combine_backward(dd, rd, sd, wd, off, workspace=ws)
    assert torch.equal(a, dr) and torch.equal(b, dw)
    a, b = nv.combine_backward(dd, rd, sd, wd)
    assert torch.equal(a, dr) and torch.equal(b, dw)


def test_rows_named_twice_and_dropped():
    """The check and the zeroing together: the row two slots name has the gradient of one of them."""
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(8)
    rd, dout = to_dev(bits(rng, (8, 64))), to_dev(bits(rng, (4, 64)))
    slot = torch.tensor([[0, 1], [2, -1], [4, 5], [6, 1]], dtype=torch.int32, device="cuda")
    w = torch.ones((4, 2), device="cuda")
    off = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    ws = torch.empty(nv.nvfp4_combine_backward_workspace_size(8), dtype=torch.uint8, device="cuda")
    spoil = torch.full_like(rd, float("nan"))
    del spoil
    dr, dw = nv.combine_backward(dout, rd, slot, w, off, workspace=ws)
    assert nv.nvfp4_workspace_status(ws) == 8
    assert torch.equal(dr[[0, 2, 4, 5, 6]], dout[[0, 1, 2, 2, 3]]) and bool((dr[[3, 7]] == 0).all())
    assert torch.equal(dr[1], dout[0]) or torch.equal(dr[1], dout[3])


def test_gradients_of_a_routing_with_dropped_slots():
    """Through autograd, with the slots past an expert's capacity taken out of the routing."""
    import dataclasses
    import torch
    import nvfp4_bit_precision_b200 as nv
    from nvfp4_bit_precision_b200.moe import moe_combine
    rng = np.random.default_rng(9)
    tokens, experts, cols, capacity = 300, 8, 256, 60
    r = nv.route(torch.from_numpy(rng.standard_normal((tokens, experts)).astype(np.float32)).cuda(), 2)
    first = r.group_offsets[r.expert.long()]
    slot = torch.where(r.slot_row - first < capacity, r.slot_row, torch.full_like(r.slot_row, -1))
    assert bool((slot < 0).any())
    rows = to_dev(bits(rng, (2 * tokens, cols))).requires_grad_()
    dout = to_dev(bits(rng, (tokens, cols)))
    spoil = torch.full_like(rows, float("nan"))
    del spoil
    moe_combine(rows, dataclasses.replace(r, slot_row=slot)).backward(dout)
    rr, _ = R.combine_backward(f64(dout), f64(rows.detach()), host(slot), host(r.weight))
    assert np.all(np.abs(f64(rows.grad) - rr) <= (B + U) * np.abs(rr) + 2.0 ** -134)


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("what,spare", [("rows", 0), ("weight", 0), ("weight", 5)])
def test_gradients_in_place(f32, what, spare):
    """drows over rows, or dweight over weight, with slots left out and rows behind the last slot's."""
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(12)
    tokens, k, cols = 50, 3, 136
    rows, rd, slot, w = make(rng, tokens, k, cols, f32, 0.3)
    n = tokens * k + spare
    rd = torch.cat([rd, rd[:spare]])
    dout = to_dev(bits(rng, (tokens, cols)))
    sd, wd = torch.from_numpy(slot).cuda(), torch.from_numpy(w).cuda()
    off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    want = nv.combine_backward(dout, rd, sd, wd, off)
    dr = rd.clone() if what == "rows" else torch.full_like(rd, float("nan"))
    dw = wd.clone() if what == "weight" else torch.full_like(wd, float("nan"))
    nv.nvfp4_combine_backward(dout, dr if what == "rows" else rd, nv.NVFP4_OUT_F32 if f32 else nv.NVFP4_OUT_BF16, n, cols,
                              sd, dw if what == "weight" else wd, tokens, k, off.data_ptr() + 4, dr, dw)
    assert torch.equal(dr, want[0]) and torch.equal(dw, want[1])


def test_more_rows_than_slots():
    """Rows past the places that dweight has for the slots' numbers, named and not."""
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(13)
    rd, dout = to_dev(bits(rng, (1000, 64))), to_dev(bits(rng, (3, 64)))
    slot = torch.tensor([[999, 2], [5, 600], [-1, 6]], dtype=torch.int32, device="cuda")
    w = torch.ones((3, 2), device="cuda")
    off = torch.tensor([0, 1000], dtype=torch.int32, device="cuda")
    for poison in (float("nan"), 0.0):
        spoil = torch.full_like(rd, poison)
        del spoil
        dr, dw = nv.combine_backward(dout, rd, slot, w, off)
        ref = torch.zeros_like(rd)
        ref[[999, 2, 5, 600, 6]] = dout[[0, 0, 1, 1, 2]]
        assert torch.equal(dr, ref) and float(dw[2, 0]) == 0.0
