"""The norm and its gradients on the GPU against 64-bit restatements.

Tolerances.  An FP32 operation is off by 2^-24 of its result at most, so y, which is a sum of squares
(at most 64 additions deep, and halved by the root), a quotient, a sum, a root and two products, is off by
less than 2^-17; rounding to bf16 adds 2^-8 of the value, and the smallest bf16 numbers half a step (2^-134)."""
import numpy as np
import pytest

import moe_ref as R
import workloads as W
from gpu_util import cuda_available, host, to_dev

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]

F = 2.0 ** -17     # FP32 arithmetic, see above
B = 2.0 ** -8      # one rounding to bf16
TINY = 2.0 ** -134
EPS = 1e-6


def bits(rng, shape, std=1.0):
    return W.f32_to_bf16_bits(rng.standard_normal(shape).astype(np.float32) * np.float32(std))


def val(b):
    return W.bf16_bits_to_f32(b).astype(np.float64)


def f64(t):
    return val(host(t)) if t.dtype.itemsize == 2 else host(t).astype(np.float64)


def check_mx(codes, e8, y):
    """codes, e8 [rows, cols/32] against the float64 norm y: the scale is the block's unless its largest
    magnitude is within the arithmetic's error of a power of two, and each code is as near as the best."""
    e = e8.astype(np.int64) - 127
    ref = R.mx_exponent(y)
    top = np.abs(y).reshape(y.shape[0], -1, 32).max(2)
    near = (R.mx_exponent(y * (1 + F)) != ref) | (R.mx_exponent(y * (1 - F)) != ref)
    assert np.all((e == ref) | (near & (np.abs(e - ref) == 1))), (e, ref, top)
    s = y.reshape(y.shape[0], -1, 32) * np.ldexp(1.0, -e)[..., None]
    got = R.e4m3_value(codes).reshape(s.shape)
    best = np.abs(R.e4m3_nearest(s) - s)
    # a value at a border of two codes may take either: it is then F |s| off the border at most
    assert np.all(np.abs(got - s) <= best + 2 * F * np.abs(s))


@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 5120), (3, 32), (7, 264), (33, 1032), (130, 2048), (5, 2056),
                                       (17, 8192), (4, 8200), (2, 16384), (3, 32768), (700, 512)])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("w32", [False, True])
def test_forward(rows, cols, residual, w32):
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(rows * 131 + cols)
    x, r = bits(rng, (rows, cols)), bits(rng, (rows, cols), 3.0) if residual else None
    w = rng.uniform(0.5, 1.5, cols).astype(np.float32) * rng.choice([-1, 1], cols).astype(np.float32)
    if not w32:
        w = W.bf16_bits_to_f32(W.f32_to_bf16_bits(w))
    wd = torch.from_numpy(w).cuda() if w32 else to_dev(W.f32_to_bf16_bits(w))
    f = nv.rmsnorm(to_dev(x), wd, to_dev(r) if residual else None, EPS, amax=True, rstd=True)
    h, rstd, y = R.rmsnorm(val(x), val(r) if residual else None, w.astype(np.float64), EPS)
    np.testing.assert_array_equal(f64(f["h"]), h)
    assert np.all(np.abs(f64(f["rstd"]) - rstd) <= F * rstd)
    got = f64(f["y"])
    assert np.all(np.abs(got - y) <= (B + F) * np.abs(y) + TINY)
    assert float(f["amax"]) == np.abs(got).max()


@pytest.mark.parametrize("rows,cols,tiled", [(1, 32, False), (5, 96, False), (1, 128, True), (129, 128, True),
                                             (127, 256, True), (300, 5120, True), (33, 5120, False),
                                             (2, 32768, True), (9, 4128, False)])
@pytest.mark.parametrize("both", [False, True])
def test_mxfp8(rows, cols, tiled, both):
    """Codes and scales, with and without y beside them; the tiled layout's padding rows are zeroed."""
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(rows + cols)
    x, r, w = bits(rng, (rows, cols)), bits(rng, (rows, cols)), bits(rng, cols, 0.3)
    x[:, :7] = W.f32_to_bf16_bits(val(x[:, :7]).astype(np.float32) * 100)   # outlier columns
    if cols >= 96:
        w[32:64] = 0                                                         # blocks of zeros
    layout = nv.NVFP4_SF_MMA if tiled else nv.NVFP4_SF_ROWMAJOR
    f = nv.rmsnorm(to_dev(x), to_dev(w), to_dev(r), EPS, y=both, mx=True, mx_sf_layout=layout)
    _, _, y = R.rmsnorm(val(x), val(r), val(w), EPS)
    q, sf = host(f["mx"][0]), host(f["mx"][1])
    if tiled:
        rm = R.untile(sf, rows, cols // 32)
        np.testing.assert_array_equal(R.tile(rm), sf)
    else:
        rm = sf
    check_mx(q, rm, y)
    assert (f["y"] is not None) == both


def test_mxfp8_feeds_the_gemm():
    """The codes and tiled scales are what the MXFP8 GEMM reads."""
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(4)
    x, w, b = bits(rng, (64, 256)), bits(rng, 256, 0.3), bits(rng, (48, 256), 0.1)
    f = nv.rmsnorm(to_dev(x), to_dev(w), y=False, mx=True, mx_sf_layout=nv.NVFP4_SF_MMA)
    bq = nv.quantize(to_dev(W.f32_to_bf16_bits(val(b).astype(np.float32))), rowwise=False,
                     mx_outputs=nv.NVFP4_ROWWISE, mx_sf_layout=nv.NVFP4_SF_MMA)["mx_row"]
    D = f64(nv.mx_gemm(f["mx"][0], f["mx"][1], bq[0], bq[1], nv.NVFP4_OUT_F32))
    A = R.e4m3_value(host(f["mx"][0])) * np.repeat(np.ldexp(1.0, R.untile(host(f["mx"][1]), 64, 8).astype(int) - 127), 32, 1)
    Bm = R.e4m3_value(host(bq[0])) * np.repeat(np.ldexp(1.0, R.untile(host(bq[1]), 48, 8).astype(int) - 127), 32, 1)
    assert np.all(np.abs(D - A @ Bm.T) <= 1e-3 * (np.abs(A) @ np.abs(Bm).T))


def test_amax_skips_the_quantisers_pass():
    """y and its amax give the NVFP4 codes that quantising y gives."""
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(5)
    f = nv.rmsnorm(to_dev(bits(rng, (48, 256))), to_dev(bits(rng, 256, 0.3)), amax=True)
    given = nv.quantize(f["y"], amax=torch.cat([f["amax"], f["amax"]]))["row"]
    plain = nv.quantize(f["y"])["row"]
    for a, b in ((given.q, plain.q), (given.sf, plain.sf), (given.g, plain.g)):
        np.testing.assert_array_equal(host(a), host(b))


def test_sums_of_any_bit_patterns():
    """h is the FP32 sum rounded to bf16 for any finite numbers: every exponent, subnormals, overflow, signed zeros,
    addends of one size, 2^-7 to 2^-18 apart, and of any."""
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(16)
    x = rng.integers(0, 1 << 16, (512, 4096)).astype(np.uint16)
    r = rng.integers(0, 1 << 16, (512, 4096)).astype(np.uint16)
    x[:, :256] &= 0x80FF                                             # subnormals and the smallest normal numbers
    r[:, :256] &= 0x80FF
    far = (x[:, 256:2048].astype(np.int32) & 0x7F80) - (rng.integers(0, 19, (512, 1792)) << 7)
    r[:, 256:2048] = (r[:, 256:2048] & 0x807F) | np.maximum(far, 0).astype(np.uint16)
    for b in (x, r):
        b[(b & 0x7F80) == 0x7F80] &= 0x807F                          # no infinities and NaN
    h = host(nv.rmsnorm(to_dev(x), to_dev(bits(rng, 4096)), to_dev(r))["h"])
    with np.errstate(over="ignore"):
        want = W.f32_to_bf16_bits(W.bf16_bits_to_f32(x) + W.bf16_bits_to_f32(r))
    np.testing.assert_array_equal(h, want)


def test_extremes():
    """Rows of zeros, of one value, of subnormals and of large values; NaN and inf stay in their rows."""
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(6)
    cols = 512
    v = val(bits(rng, (8, cols)))
    v[0] = 0.0
    v[1] = 7.0
    v[2] = 2.0 ** -130
    v[3] *= 2.0 ** 60
    v[4, 5] = np.nan
    v[5, 6] = np.inf
    x = W.f32_to_bf16_bits(v.astype(np.float32))
    x[4, 5] = 0x7FC0
    w = bits(rng, cols, 0.5)
    f = nv.rmsnorm(to_dev(x), to_dev(w), eps=EPS, mx=True, rstd=True)
    y = f64(f["y"])
    ok = [0, 1, 2, 3, 6, 7]
    _, _, ref = R.rmsnorm(val(x)[ok], None, val(w), EPS)
    assert np.all(np.abs(y[ok] - ref) <= (B + F) * np.abs(ref) + TINY)
    check_mx(host(f["mx"][0])[ok], host(f["mx"][1])[ok], ref)
    assert np.isnan(y[4]).all() and np.isnan(y[5, 6]) and np.all(y[5][np.arange(cols) != 6] == 0)


@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 4096), (5, 264), (37, 1032), (300, 512), (2000, 256), (9, 8192),
                                       (6, 8200), (3, 32768), (513, 5120)])
@pytest.mark.parametrize("dh", [False, True])
@pytest.mark.parametrize("w32", [False, True])
def test_backward(rows, cols, dh, w32):
    """dx: FP32 arithmetic on its terms; dw: a sum of `rows` products in FP32, then one rounding."""
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(rows * 7 + cols)
    x, dy = bits(rng, (rows, cols), 2.0), bits(rng, (rows, cols), 1e-3)
    g = bits(rng, (rows, cols), 1e-3) if dh else None
    w = bits(rng, cols)
    wd = torch.from_numpy(W.bf16_bits_to_f32(w)).cuda() if w32 else to_dev(w)
    f = nv.rmsnorm(to_dev(x), wd, eps=EPS, rstd=True)
    dx, dw = nv.rmsnorm_backward(to_dev(dy), f["h"], wd, f["rstd"], to_dev(g) if dh else None)
    rx, rw = R.rmsnorm_backward(val(dy), val(x), val(w), EPS, val(g) if dh else None)
    _, rstd, _ = R.rmsnorm(val(x), None, val(w), EPS)
    n = val(x) * rstd[:, None]
    t = np.abs(val(dy) * val(w))
    terms = rstd[:, None] * (t + np.abs(n) * (t * np.abs(n)).mean(1, keepdims=True)) + (np.abs(val(g)) if dh else 0)
    assert np.all(np.abs(f64(dx) - rx) <= B * np.abs(rx) + F * terms + TINY)
    assert dw.dtype == wd.dtype
    add = (rows + 64) * 2.0 ** -24 + F
    assert np.all(np.abs(f64(dw) - rw) <= (0 if w32 else B) * np.abs(rw) + add * np.abs(val(dy) * n).sum(0) + TINY)
    again = nv.rmsnorm_backward(to_dev(dy), f["h"], wd, f["rstd"], to_dev(g) if dh else None)
    assert torch.equal(again[1], dw) and torch.equal(again[0], dx)
    only = nv.rmsnorm_backward(to_dev(dy), f["h"], wd, f["rstd"], to_dev(g) if dh else None, dweight=False)
    assert only[1] is None and torch.equal(only[0], dx)


def test_formula_against_differences():
    """The 64-bit gradient the kernel is held to, against central differences of the 64-bit norm."""
    rng = np.random.default_rng(8)
    h, w, dy = rng.standard_normal((3, 16)), rng.standard_normal(16), rng.standard_normal((3, 16))
    dx, dw = R.rmsnorm_backward(dy, h, w, EPS)
    loss = lambda a, b: float((R.rmsnorm(a, None, b, EPS)[2] * dy).sum())
    d = 1e-5
    for _ in range(20):
        u, v = rng.standard_normal(h.shape), rng.standard_normal(16)
        num = (loss(h + d * u, w + d * v) - loss(h - d * u, w - d * v)) / (2 * d)
        assert abs(num - ((dx * u).sum() + (dw * v).sum())) <= 1e-7 * (1 + abs(num))


def test_strided_and_in_place():
    """Column slices of wider tensors in, and what lies beside the outputs left as it was."""
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(9)
    wide = to_dev(bits(rng, (19, 1024)))
    x, r = wide[:, 64:64 + 320], wide[:, 512:512 + 320]
    w = to_dev(bits(rng, 320))
    a = nv.rmsnorm(x, w, r, rstd=True)
    b = nv.rmsnorm(x.contiguous(), w, r.contiguous(), rstd=True)
    assert torch.equal(a["y"], b["y"]) and torch.equal(a["h"], b["h"])
    ga, gb = nv.rmsnorm_backward(x, r, w, a["rstd"], x), nv.rmsnorm_backward(x.contiguous(), r.contiguous(), w,
                                                                           a["rstd"], x.contiguous())
    assert torch.equal(ga[0], gb[0]) and torch.equal(ga[1], gb[1])
    # h in place of the residual, y into a slice of a wider tensor
    out = torch.full((19, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    res = r.contiguous()
    nv.nvfp4_rmsnorm(x, 1024, res, 320, w, nv.NVFP4_OUT_BF16, 1e-6, 19, 320, res, 320, out[:, 64:], 512, None, None,
                     None, None, 0)
    assert torch.equal(res, b["h"]) and torch.equal(out[:, 64:384], b["y"])
    assert bool((out[:, :64] == 3).all()) and bool((out[:, 384:] == 3).all())
    # dx in place of dh
    dh = r.contiguous()
    ws = torch.empty(nv.nvfp4_rmsnorm_backward_workspace_size(19, 320), dtype=torch.uint8, device="cuda")
    dw = torch.empty_like(w)
    nv.nvfp4_rmsnorm_backward(x, 1024, r, 1024, dh, 320, w, nv.NVFP4_OUT_BF16, a["rstd"], 19, 320, dh, 320, dw, ws,
                              ws.numel())
    assert torch.equal(dh, nv.rmsnorm_backward(x, r, w, a["rstd"], r)[0])
    assert nv.nvfp4_workspace_status(ws) == 0


def test_no_rows():
    import torch
    import nvfp4_bit_precision_b200 as nv
    x = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    f = nv.rmsnorm(x, w, x, mx=True, amax=True, rstd=True, mx_sf_layout=nv.NVFP4_SF_MMA)
    assert f["y"].shape == (0, 256) and float(f["amax"]) == 0.0
    dx, dw = nv.rmsnorm_backward(x, x, w, f["rstd"])
    assert dx.shape == (0, 256) and bool((dw == 0).all())
