"""Refusals of the norm, routing, combine and few-token product calls, on the host: the C entry points return
their status before any device work, and the wrappers raise before they call them.  CPU only."""
import ctypes

import pytest

FAKE = 1 << 20  # a 16-byte aligned non-null address that validation never dereferences
OK, ARG, SHAPE, ALIGN, WORKSPACE = 0, 1, 2, 3, 7


@pytest.fixture(scope="module")
def nv():
    import nvfp4_bit_precision_b200 as nv
    return nv


def norm(nv, **kw):
    a = dict(x=FAKE, ldx=256, r=None, ldr=256, w=FAKE, wdt=1, eps=1e-6, rows=4, cols=256, h=None, ldh=256, y=FAKE,
             ldy=256, rstd=None, amax=None, q=None, sf=None, layout=0)
    a.update(kw)
    return nv._lib.nvfp4_rmsnorm(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), ARG), (dict(w=None), ARG), (dict(y=None), ARG), (dict(wdt=2), ARG), (dict(eps=-1.0), ARG),
    (dict(eps=float("nan")), ARG), (dict(r=FAKE), ARG), (dict(h=FAKE), ARG), (dict(q=FAKE), ARG), (dict(sf=FAKE), ARG),
    (dict(y=None, q=FAKE, sf=FAKE, amax=FAKE), ARG), (dict(q=FAKE, sf=FAKE, layout=2), ARG),
    (dict(cols=252), SHAPE), (dict(cols=0), SHAPE), (dict(rows=-1), SHAPE), (dict(ldx=248), SHAPE),
    (dict(cols=32776, ldx=32776, ldy=32776), SHAPE), (dict(ldy=128), SHAPE), (dict(r=FAKE, h=FAKE, ldr=64), SHAPE),
    (dict(q=FAKE, sf=FAKE, cols=40), SHAPE), (dict(q=FAKE, sf=FAKE, cols=96, layout=1), SHAPE),
    (dict(x=FAKE + 8), ALIGN), (dict(ldx=260), ALIGN), (dict(w=FAKE + 2), ALIGN), (dict(y=FAKE + 8), ALIGN),
    (dict(q=FAKE + 8, sf=FAKE), ALIGN), (dict(q=FAKE, sf=FAKE + 2), ALIGN), (dict(rstd=FAKE + 2), ALIGN)])
def test_norm_argument_errors(nv, change, status):
    assert norm(nv, **change) == status


def back(nv, **kw):
    a = dict(dy=FAKE, lddy=256, h=FAKE, ldh=256, dh=None, lddh=0, w=FAKE, wdt=0, rstd=FAKE, rows=4, cols=256, dx=FAKE,
             lddx=256, dw=FAKE, ws=FAKE, n=1 << 20)
    a.update(kw)
    return nv._lib.nvfp4_rmsnorm_backward(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(dy=None), ARG), (dict(h=None), ARG), (dict(rstd=None), ARG), (dict(dx=None), ARG), (dict(wdt=7), ARG),
    (dict(cols=100), SHAPE), (dict(lddx=128), SHAPE), (dict(dh=FAKE, lddh=8), SHAPE), (dict(lddy=260), ALIGN),
    (dict(dh=FAKE + 8, lddh=256), ALIGN), (dict(ws=None), WORKSPACE), (dict(n=300), WORKSPACE)])
def test_norm_backward_argument_errors(nv, change, status):
    assert back(nv, **change) == status


def route(nv, tokens=200, experts=64, ld=None, dt=0, logits=FAKE, bias=None, outs=(FAKE,) * 5, ws=FAKE, n=1 << 20, **kw):
    p = dict(top_k=4, score=0, groups=1, topk_groups=1, group_top=2, renormalize=1, scale=1.0)
    p.update(kw)
    return nv._lib.nvfp4_route(logits, dt, experts if ld is None else ld, bias, tokens, experts,
                               ctypes.byref(nv.RouteParams(**p)), *outs, ws, n, None)


@pytest.mark.parametrize("change,status", [
    (dict(logits=None), ARG), (dict(dt=3), ARG), (dict(score=2), ARG), (dict(group_top=3), ARG),
    (dict(group_top=0), ARG), (dict(renormalize=2), ARG), (dict(outs=(FAKE, None, FAKE, FAKE, FAKE)), ARG),
    (dict(outs=(FAKE, FAKE, None, FAKE, FAKE)), ARG),
    (dict(top_k=0), SHAPE), (dict(top_k=33), SHAPE), (dict(experts=3), SHAPE), (dict(experts=513), SHAPE),
    (dict(ld=63), SHAPE), (dict(tokens=-1), SHAPE), (dict(tokens=1 << 30), SHAPE), (dict(groups=0), SHAPE),
    (dict(groups=5), SHAPE), (dict(groups=64, topk_groups=64), SHAPE), (dict(groups=4, topk_groups=5), SHAPE),
    (dict(groups=32, topk_groups=1), SHAPE),
    (dict(logits=FAKE + 2), ALIGN), (dict(logits=FAKE + 1, dt=1), ALIGN), (dict(bias=FAKE + 2), ALIGN),
    (dict(ws=None), WORKSPACE), (dict(n=256), WORKSPACE), (dict(ws=FAKE + 4), WORKSPACE)])
def test_route_argument_errors(nv, change, status):
    assert route(nv, **change) == status


def test_route_backward_argument_errors(nv):
    def call(dw=FAKE, logits=FAKE, dt=0, ld=64, ids=FAKE, tokens=4, experts=64, d=FAKE, ldd=64, **kw):
        p = nv.RouteParams(**{**dict(top_k=4, score=0, renormalize=1, scale=1.0), **kw})
        return nv._lib.nvfp4_route_backward(dw, logits, dt, ld, ids, tokens, experts, ctypes.byref(p), d, ldd, None)
    assert call(dw=None) == ARG and call(d=None) == ARG and call(ids=None) == ARG and call(dt=5) == ARG
    assert call(score=9) == ARG and call(renormalize=4) == ARG
    assert call(ldd=60) == SHAPE and call(top_k=0) == SHAPE and call(experts=600, ld=600, ldd=600) == SHAPE
    assert call(d=FAKE + 2) == ALIGN and call(logits=FAKE + 3, dt=1) == ALIGN
    assert call(tokens=0) == OK


def test_combine_argument_errors(nv):
    def call(rows=FAKE, dt=1, n=8, cols=64, slot=FAKE, w=FAKE, t=4, k=2, base=None, out=FAKE, ws=None, wn=0):
        return nv._lib.nvfp4_combine(rows, dt, n, cols, slot, w, t, k, base, out, ws, wn, None)
    assert call(rows=None) == ARG and call(dt=2) == ARG and call(k=0) == ARG and call(k=65) == ARG
    assert call(slot=None) == ARG and call(w=None) == ARG and call(out=None) == ARG
    assert call(cols=60) == SHAPE and call(n=-1) == SHAPE and call(t=-1) == SHAPE and call(n=1 << 31) == SHAPE
    assert call(rows=FAKE + 8) == ALIGN and call(base=FAKE + 8) == ALIGN and call(slot=FAKE + 2) == ALIGN
    assert call(ws=FAKE, wn=8) == WORKSPACE and call(ws=FAKE + 8, wn=256) == WORKSPACE

    def back(dout=FAKE, rows=FAKE, dt=1, n=8, cols=64, slot=FAKE, w=FAKE, t=4, k=2, used=None, dr=FAKE, dw=FAKE,
             ws=FAKE, wn=512):
        return nv._lib.nvfp4_combine_backward(dout, rows, dt, n, cols, slot, w, t, k, used, dr, dw, ws, wn, None)
    assert back(dout=None) == ARG and back(dr=None) == ARG and back(dw=None) == ARG
    assert back(cols=4) == SHAPE and back(dr=FAKE + 4) == ALIGN and back(used=FAKE + 1) == ALIGN
    assert back(ws=FAKE + 8) == WORKSPACE and back(wn=256) == WORKSPACE
    assert back(ws=None, wn=0) not in (ARG, SHAPE, ALIGN, WORKSPACE)   # the check is optional (no GPU here)
    assert nv.nvfp4_combine_backward_workspace_size(33) == 256 + 8


def test_gemv_argument_errors(nv):
    def call(x=FAKE, ldx=128, rows=2, q=FAKE, sf=FAKE, g=FAKE, n=128, k=128, dt=1, d=FAKE, ldd=128):
        return nv._lib.nvfp4_gemv(x, ldx, rows, q, sf, g, n, k, dt, d, ldd, None)
    assert call(x=None) == ARG and call(q=None) == ARG and call(sf=None) == ARG and call(g=None) == ARG
    assert call(d=None) == ARG and call(dt=2) == ARG
    assert call(n=100, ldd=100) == SHAPE and call(k=96) == SHAPE and call(ldx=64) == SHAPE and call(ldd=64) == SHAPE
    assert call(rows=-1) == SHAPE and call(n=0) == SHAPE
    assert call(x=FAKE + 8) == ALIGN and call(ldx=132) == ALIGN and call(q=FAKE + 8) == ALIGN
    assert call(sf=FAKE + 4) == ALIGN and call(d=FAKE + 1) == ALIGN and call(g=FAKE + 2) == ALIGN

    def grouped(G=4, off=FAKE, total=8, x=FAKE, ldx=128, src=8, idx=None, n=128, k=128, d=FAKE, ws=None, wn=0):
        return nv._lib.nvfp4_grouped_gemv(G, off, total, x, ldx, src, idx, FAKE, FAKE, FAKE, n, k, 1, d, n, ws, wn,
                                          None)
    assert grouped(G=0) == ARG and grouped(G=257) == ARG and grouped(off=None) == ARG and grouped(src=0, idx=FAKE) == ARG
    assert grouped(n=64) == SHAPE and grouped(src=7) == SHAPE and grouped(off=FAKE + 2) == ALIGN
    assert grouped(ws=FAKE, wn=4) == WORKSPACE


def test_wrappers_refuse(nv):
    """Tensors off the GPU, of the wrong type, shape or strides."""
    import torch
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    f = lambda *s: torch.zeros(s)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensors expected"):
        nv.rmsnorm(b(2, 64), b(64))
    with pytest.raises(ValueError, match="CUDA tensors expected"):
        nv.rmsnorm_backward(b(2, 64), b(2, 64), b(64), f(2))
    with pytest.raises(ValueError, match="CUDA tensors expected"):
        nv.route(f(2, 8), 2)
    with pytest.raises(ValueError, match="CUDA tensors expected"):
        nv.combine(b(4, 64), i(2, 2), f(2, 2))
    with pytest.raises(ValueError, match="CUDA tensors expected"):
        nv.combine_backward(b(2, 64), b(4, 64), i(2, 2), f(2, 2))
    w = nv.NVFP4Tensor(torch.zeros((128, 32), dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), f(1), 128, 64,
                       nv.NVFP4_SF_MMA)
    with pytest.raises(ValueError, match="CUDA tensors expected"):
        nv.gemv(b(1, 64), w)
    with pytest.raises(ValueError, match="CUDA tensors expected"):
        nv.grouped_gemv(i(2), b(1, 64), w.q[None], w.sf, w.g, 128)


def test_wrappers_refuse_types_shapes_and_devices(nv, monkeypatch):
    """The same checks past the device's, with a stand-in for it."""
    import torch
    monkeypatch.setattr(nv, "_one_device", lambda name, *t: t[0].device)
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    f = lambda *s: torch.zeros(s)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    for call, match in [
            (lambda: nv.rmsnorm(f(2, 64), b(64)), "bfloat16 matrix"),
            (lambda: nv.rmsnorm(b(2, 64), b(32)), "weight"),
            (lambda: nv.rmsnorm(b(2, 64), b(64).half()), "bfloat16 or float32"),
            (lambda: nv.rmsnorm(b(2, 64), b(64), b(3, 64)), "expected"),
            (lambda: nv.rmsnorm(b(64, 2).t(), b(64)), "contiguous"),
            (lambda: nv.rmsnorm(b(2, 64), b(64), y=False), "neither"),
            (lambda: nv.rmsnorm(b(2, 64), b(64), y=False, mx=True, amax=True), "amax"),
            (lambda: nv.rmsnorm_backward(b(2, 64), b(2, 32), b(64), f(2)), "expected"),
            (lambda: nv.rmsnorm_backward(b(2, 64), b(2, 64), b(64), f(3)), "rstd"),
            (lambda: nv.route(f(2, 8).half(), 2), "bfloat16 or float32"),
            (lambda: nv.route(f(2, 8, 1), 2), "logits"),
            (lambda: nv.route(f(8, 2).t(), 2), "contiguous"),
            (lambda: nv.route(f(2, 8), 2, bias=f(7)), "bias"),
            (lambda: nv.route(f(2, 8), 0), "top_k"),
            (lambda: nv.combine(b(4, 64), i(2, 2), f(2, 3)), "weight"),
            (lambda: nv.combine(b(4, 64), f(2, 2), f(2, 2)), "slot_row"),
            (lambda: nv.combine(b(4, 64), i(2, 2), f(2, 2), f(2, 64)), "base"),
            (lambda: nv.combine(b(64, 4).t(), i(2, 2), f(2, 2)), "contiguous rows"),
            (lambda: nv.combine_backward(b(3, 64), b(4, 64), i(2, 2), f(2, 2)), "dout"),
            (lambda: nv.combine_backward(b(2, 64), b(4, 64), i(2, 2), f(2, 2), i(1)), "group_offsets"),
            (lambda: nv.grouped_gemv(i(3), b(2, 64), torch.zeros((1, 128, 32), dtype=torch.uint8), i(4), f(1), 128), "qb")]:
        with pytest.raises(ValueError, match=match):
            call()


def test_one_device_refuses_the_wrong_current_device(nv, monkeypatch):
    import torch

    class T:
        def __init__(self, d):
            self.device = torch.device(d)

        def get_device(self):
            return self.device.index

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    assert nv._one_device("op", T("cuda:0"), None, T("cuda:0")).index == 0
    with pytest.raises(ValueError, match="current device"):
        nv._one_device("op", T("cuda:1"), T("cuda:1"))
    with pytest.raises(ValueError, match="cuda:0 and cuda:1"):
        nv._one_device("op", T("cuda:0"), T("cuda:1"))


def test_autograd_forms_refuse():
    """moe's functions check before they launch; a captured gradient is refused (with a stand-in for capture)."""
    import torch
    from nvfp4_bit_precision_b200 import moe
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensors expected"):
        moe.rms_norm(x, x[0])
    with pytest.raises(ValueError, match="differ"):
        moe.rms_norm(x, x[0], x[:1])
    with pytest.raises(ValueError, match="CUDA tensors expected"):
        moe.moe_route(torch.zeros((2, 8)), 2)
    assert moe.RMSNorm(64).weight.dtype == torch.bfloat16


def test_captured_gradients_refused_on_the_host(monkeypatch):
    import torch
    from nvfp4_bit_precision_b200 import moe
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    x = torch.zeros((2, 64), dtype=torch.bfloat16, requires_grad=True)
    with pytest.raises(RuntimeError, match="CUDA graph"):
        moe.rms_norm(x, x[0])
    with pytest.raises(RuntimeError, match="CUDA graph"):
        moe.moe_route(torch.zeros((2, 8), requires_grad=True), 2)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA tensors expected"):
        moe.rms_norm(x, x[0])


def test_combine_backward_refuses_gradients_over_the_rows(nv):
    """With used_rows the slots' numbers pass through drows, where dweight has no place for them, before rows is
    read."""
    at, w = 1 << 30, 1 << 34

    def back(rows, dr, used=FAKE, dt=1, n=8, dw=1 << 35):
        return nv._lib.nvfp4_combine_backward(FAKE, rows, dt, n, 64, FAKE, w, 4, 2, used, dr, dw, None, 0, None)
    for more in (dict(n=9), dict(dw=w), dict(dw=w + 28), dict(dw=w - 28)):
        assert back(at, at, **more) == ARG and back(at, at + 896, **more) == ARG and back(at + 896, at, **more) == ARG
        assert back(at, at + 1152, dt=0, **more) == ARG
    import torch
    if not torch.cuda.is_available():  # nothing is launched
        for status in (back(at, at), back(at, at, used=None, n=9), back(at, at + 1152, n=9), back(at, at + 2304, dt=0, n=9),
                       back(at, at + 1024, dw=w), back(at, at, dw=w + 32)):
            assert status not in (ARG, SHAPE, ALIGN, WORKSPACE)


def test_stand_in_addresses_stay_off_a_gpu(monkeypatch):
    import pathlib
    import torch
    import conftest

    class Item:
        def __init__(self, name):
            self.path, self.marks = pathlib.Path(name), []

        def add_marker(self, mark):
            self.marks.append(mark.name)

    for gpu in (True, False):
        monkeypatch.setattr(torch.cuda, "is_available", lambda: gpu)
        items = [Item(__file__), Item("tests/test_gpu_norm.py")]
        conftest.pytest_collection_modifyitems(items)
        assert [i.marks for i in items] == [["skip"] if gpu else [], []]


def test_gemv_refuses_sizes_whose_product_overflows(nv):
    """rows x tiles x steps past 2^31 and past 2^63 alike, before anything is asked of a device."""
    def dense(rows, n, k):
        return nv._lib.nvfp4_gemv(FAKE, k, rows, FAKE, FAKE, FAKE, n, k, 1, FAKE, n, None)

    def grouped(rows, n, k):
        return nv._lib.nvfp4_grouped_gemv(4, FAKE, rows, FAKE, k, rows, None, FAKE, FAKE, FAKE, n, k, 1, FAKE, n, None,
                                          0, None)
    for call in (dense, grouped):
        for rows, n, k in ((2 ** 31 - 1, 2 ** 30, 45056), (2 ** 31 - 1, 2 ** 30, 64 * 512), (2 ** 31 - 1, 2 ** 30, 64),
                           (2 ** 28, 128, 64), (2 ** 20, 2 ** 14, 1024), (1, 128, 45120 + 64)):
            assert call(rows, n, k) == SHAPE, (rows, n, k)


@pytest.mark.parametrize("change", [dict(ws=FAKE + 2), dict(ws=FAKE + 4), dict(ws=FAKE + 8), dict(n=8), dict(n=0)])
def test_norm_backward_checks_a_workspace_without_dweight(nv, change):
    """Its status word is cleared whether or not dweight is asked for."""
    assert back(nv, dw=None, **change) == WORKSPACE
    assert back(nv, dw=None, rows=0, **change) == WORKSPACE


def test_products_refuse_scales_of_other_types(nv, monkeypatch):
    """The matrix scale is one FP32 number and the block scales are bytes; others would be read as if they were."""
    import torch
    monkeypatch.setattr(nv, "_one_device", lambda name, *t: t[0].device)
    monkeypatch.setattr(nv, "_raw_stream", lambda dev: None)   # nothing gets as far as a launch
    called = []
    monkeypatch.setattr(nv, "_lib", type("Lib", (), {n: staticmethod(lambda *a: called.append(a) or 0)
                                                    for n in ("nvfp4_gemv", "nvfp4_grouped_gemv")}
                                         | {"nvfp4_sf_mma_bytes": nv._lib.nvfp4_sf_mma_bytes}))
    x, q, sf = torch.zeros((1, 64), dtype=torch.bfloat16), torch.zeros((128, 32), dtype=torch.uint8), \
        torch.zeros(512, dtype=torch.uint8)
    off = torch.zeros(2, dtype=torch.int32)
    dense = lambda g, s: nv.gemv(x, nv.NVFP4Tensor(q, s, g, 128, 64, nv.NVFP4_SF_MMA))
    grouped = lambda g, s: nv.grouped_gemv(off, x, q[None], s, g, 128)
    one = torch.ones(1)
    for g in (one.bfloat16(), one.double(), one.half(), one.int(), torch.ones(0), torch.ones(2)):
        with pytest.raises(ValueError, match="w.g"):
            dense(g, sf)
        with pytest.raises(ValueError, match="gb"):
            grouped(g, sf)
    for s in (sf.int(), sf.float(), sf.bfloat16()):
        with pytest.raises(ValueError, match="w.sf"):
            dense(one, s)
        with pytest.raises(ValueError, match="sfb"):
            grouped(one, s)
    assert not called
    for g, s in ((one, sf), (one, sf.view(torch.float8_e4m3fn)), (one, torch.zeros(2048, dtype=torch.int8))):
        dense(g, s)
        grouped(g, s)
    dense(torch.tensor(1.0), sf)
    assert len(called) == 7


def test_import_leaves_torch_to_first_use():
    """Importing the package brings no torch along; the first call that needs it does."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = ("import sys, nvfp4_bit_precision_b200 as nv\n"
            "assert nv.nvfp4_version() >= 300 and nv.nvfp4_sf_mma_bytes(128, 64) == 512\n"
            "assert nv.nvfp4_rmsnorm_backward_workspace_size(4, 256) > 256\n"
            "assert 'torch' not in sys.modules\n"
            "import torch\n"
            "try:\n    nv.rmsnorm(torch.zeros((2, 64), dtype=torch.bfloat16), torch.zeros(64))\n"
            "except ValueError as e:\n    assert 'CUDA tensors expected' in str(e)\n"
            "else:\n    raise AssertionError\n"
            "assert nv._matrix(torch.device('cpu'), torch.uint8, 2, 3).shape == (2, 3) and nv.torch is torch\n")
    subprocess.run([sys.executable, "-c", code], cwd=root, check=True)


def test_combine_backward_counts_slots_in_31_bits(nv):
    def back(t, used=FAKE, k=2):
        return nv._lib.nvfp4_combine_backward(FAKE, FAKE, 1, 8, 64, FAKE, FAKE, t, k, used, 1 << 32, 1 << 35, None, 0, None)
    assert back(1 << 30) == SHAPE and back((1 << 62) - 1) == SHAPE and back(1 << 28, k=8) == SHAPE
