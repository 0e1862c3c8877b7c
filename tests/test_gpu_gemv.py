"""Few-token products with NVFP4 matrices against float64 products of the same values.

Tolerance.  An accumulation of 16 products by the tensor cores may truncate each of its 17 additions:
17 * 2^-23 of the magnitudes; of 256 columns two chains of 8 of them run side by side, then come two sums
for every 256 columns, up to 16 over the warps and the products with the scales.  x is exact or within
2^-40 of its row's largest magnitude."""
import numpy as np
import pytest

import moe_ref as R
import workloads as W
from gpu_util import cuda_available, host, to_dev

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]


def bits(rng, shape, std=1.0):
    return W.f32_to_bf16_bits(rng.standard_normal(shape).astype(np.float32) * np.float32(std))


def val(b):
    return W.bf16_bits_to_f32(b).astype(np.float64)


def f64(t):
    return val(host(t)) if t.dtype.itemsize == 2 else host(t).astype(np.float64)


def bound(x, w, ref, f32):
    k = x.shape[1]
    c = (8 * 17 + 2 * -(-k // 256) + 19) * 2.0 ** -23
    top = np.abs(x).max(1, keepdims=True) * np.ones_like(x)
    return c * (np.abs(x) @ np.abs(w).T) + 2.0 ** -40 * (top @ np.abs(w).T) + (0 if f32 else 2.0 ** -8) * np.abs(ref) + 1e-44


def upload(nv, q, sf, g):
    import torch
    return nv.NVFP4Tensor(torch.from_numpy(q).cuda(), torch.from_numpy(R.tile(sf)).cuda(),
                          torch.tensor([g], dtype=torch.float32, device="cuda"), q.shape[0], q.shape[1] * 2,
                          nv.NVFP4_SF_MMA)


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 16, 17, 33])
@pytest.mark.parametrize("n,k", [(16, 64), (144, 192), (128, 1088), (272, 2048), (2048, 576)])
@pytest.mark.parametrize("f32", [True, False])
def test_dense(rows, n, k, f32):
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(rows + n + k)
    q, sf, g = R.random_nvfp4(rng, n, k, extreme=True)
    x = bits(rng, (rows, k))
    y = nv.gemv(to_dev(x), upload(nv, q, sf, g), nv.NVFP4_OUT_F32 if f32 else nv.NVFP4_OUT_BF16)
    w = R.nvfp4_matrix(q, sf, g)
    ref = val(x) @ w.T
    assert np.all(np.abs(f64(y) - ref) <= bound(val(x), w, ref, f32))


def test_every_code_and_scale():
    """One-hot x reads single elements: every code under every finite scale byte, exactly."""
    import torch
    import nvfp4_bit_precision_b200 as nv
    n, k = 128, 64
    q = np.empty((n, k // 2), dtype=np.uint8)
    q[:] = (np.arange(k // 2) % 8 * 2) | ((np.arange(k // 2) % 8 * 2 + 1) << 4)  # all 16 codes in each block
    sf = np.repeat(np.arange(n)[:, None], k // 16, axis=1).astype(np.uint8)
    sf[127] = 0
    x = W.f32_to_bf16_bits(np.eye(k, dtype=np.float32))
    y = nv.gemv(to_dev(x), upload(nv, q, sf, np.float32(1.0)), nv.NVFP4_OUT_F32)
    np.testing.assert_array_equal(f64(y).T, R.nvfp4_matrix(q, sf, 1.0))


def test_range_of_x():
    """Token after token of its own size, from 2^-120 to 2^110; zeros; huge spreads within 128 columns."""
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(7)
    n, k = 128, 512
    q, sf, g = R.random_nvfp4(rng, n, k)
    v = rng.standard_normal((13, k))
    v *= np.ldexp(1.0, [-120, -60, -20, -5, 0, 5, 20, 60, 110, 0, 0, 0, -126])[:, None]
    v[9] = 0
    v[10, ::3] *= 2.0 ** 40
    v[11, 128:256] = 0
    v[11, 5] = 2.0 ** 100
    x = W.f32_to_bf16_bits(v.astype(np.float32))
    w = R.nvfp4_matrix(q, sf, g)
    ref = val(x) @ w.T
    y = nv.gemv(to_dev(x), upload(nv, q, sf, g), nv.NVFP4_OUT_F32)
    assert np.all(np.abs(f64(y) - ref) <= bound(val(x), w, ref, True))


def test_small_x_and_g():
    """x near the smallest numbers under a small g: the result keeps FP32's precision where it is a normal number."""
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(17)
    q, sf, _ = R.random_nvfp4(rng, 128, 256)
    for g, exponent in ((2.0 ** -20, -100), (2.0 ** -30, -110), (2.0 ** -3, -124)):
        x = W.f32_to_bf16_bits((rng.standard_normal((3, 256)) * 2.0 ** exponent * 2.0 ** 14).astype(np.float32))
        w = R.nvfp4_matrix(q, sf, np.float32(g))
        ref = val(x) @ w.T
        y = nv.gemv(to_dev(x), upload(nv, q, sf, np.float32(g)), nv.NVFP4_OUT_F32)
        # (the two products' roundings are half of 2^-149 where they leave the normal numbers)
        assert np.all(np.abs(f64(y) - ref) <= bound(val(x), w, ref, True))


def test_non_finite_tokens_stay_alone():
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(8)
    q, sf, g = R.random_nvfp4(rng, 128, 256)
    x = bits(rng, (5, 256))
    x[1, 3], x[3, 77] = 0x7F80, 0x7FC0
    y = f64(nv.gemv(to_dev(x), upload(nv, q, sf, g)))
    clean = f64(nv.gemv(to_dev(x[[0, 2, 4]]), upload(nv, q, sf, g)))
    np.testing.assert_array_equal(y[[0, 2, 4]], clean)
    assert np.isnan(y[3]).all() and not np.isfinite(y[1]).any()


def test_strided_x_and_out():
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(9)
    q, sf, g = R.random_nvfp4(rng, 144, 320)
    w = upload(nv, q, sf, g)
    wide = to_dev(bits(rng, (11, 1024)))
    x = wide[:, 128:128 + 320]
    out = torch.full((11, 200), 5.0, device="cuda")
    nv.gemv(x, w, nv.NVFP4_OUT_F32, out[:, 17:17 + 144])
    assert torch.equal(out[:, 17:161], nv.gemv(x.contiguous(), w, nv.NVFP4_OUT_F32))
    assert bool((out[:, :17] == 5).all()) and bool((out[:, 161:] == 5).all())
    assert nv.gemv(x[:0], w).shape == (0, 144)


def test_quantised_weight_serves_both():
    """The weight that nvfp4_gemm reads, unchanged: both products of x values that FP4 holds exactly agree."""
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(10)
    w = nv.quantize(to_dev(bits(rng, (256, 512), 0.02)), sf_layout=nv.NVFP4_SF_MMA)["row"]
    x = rng.choice([0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], (16, 512)) * rng.choice([-1, 1], (16, 512))
    x[:, ::16] = 6.0
    xd = to_dev(W.f32_to_bf16_bits(x.astype(np.float32)))
    xq = nv.quantize(xd, sf_layout=nv.NVFP4_SF_MMA)["row"]
    # g = 6 / 2688 is rounded to FP32 (2^-24 of it) and so is its product with the exact codes (2^-24)
    assert np.all(np.abs(f64(nv.dequantize(xq)) - x) <= 2.0 ** -23 * np.abs(x))
    a, b = f64(nv.gemv(xd, w, nv.NVFP4_OUT_F32)), f64(nv.gemm(xq, w, nv.NVFP4_OUT_F32))
    wf = f64(nv.dequantize(w))
    assert np.all(np.abs(a - b) <= 2 * bound(x, wf, x @ wf.T, True) + 1e-3 * (np.abs(x) @ np.abs(wf).T))
    assert np.all(np.abs(a - x @ wf.T) <= bound(x, wf, x @ wf.T, True) + 2.0 ** -24 * (np.abs(x) @ np.abs(wf).T))


@pytest.mark.parametrize("counts", [[1], [0, 3, 0, 1, 12, 0], [0, 0, 5], [9, 0, 0, 0], [1] * 40, [0] * 255 + [4],
                                    [20, 35, 2]])
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("k,f32", [(64, True), (320, False), (1152, True)])
def test_grouped(counts, gather, k, f32):
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(sum(counts) + k)
    G, n, total = len(counts), 128, sum(counts)
    few = min(G, 8)  # matrices repeat, so that many groups stay small
    mats = [R.random_nvfp4(rng, n, k) for _ in range(few)]
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    src = 6 if gather else total
    x = bits(rng, (src, k))
    idx = rng.integers(0, src, total).astype(np.int32) if gather else None
    qb = torch.from_numpy(np.stack([mats[e % few][0] for e in range(G)])).cuda()
    sfb = torch.from_numpy(np.concatenate([R.tile(mats[e % few][1]) for e in range(G)])).cuda()
    gb = torch.tensor([mats[e % few][2] for e in range(G)], dtype=torch.float32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    y = nv.grouped_gemv(torch.from_numpy(off).cuda(), to_dev(x), qb, sfb, gb, n,
                        torch.from_numpy(idx).cuda() if gather else None,
                        nv.NVFP4_OUT_F32 if f32 else nv.NVFP4_OUT_BF16, workspace=ws)
    assert nv.nvfp4_workspace_status(ws) == 0
    xs = val(x)[idx] if gather else val(x)
    got = f64(y)
    for e in range(G):
        s = slice(off[e], off[e + 1])
        if counts[e] == 0:
            continue
        w = R.nvfp4_matrix(*mats[e % few])
        ref = xs[s] @ w.T
        assert np.all(np.abs(got[s] - ref) <= bound(xs[s], w, ref, f32))


@pytest.mark.parametrize("G,n,k", [(40, 1024, 1152), (64, 512, 320), (6, 4096, 704), (3, 2176, 2560)])
def test_many_tiles(G, n, k):
    """CTAs and warps that begin and end inside tiles and segments; a matrix with more rows than fit at once."""
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(G)
    counts = rng.integers(0, 4, G)
    counts[0], counts[G // 2] = 21, 9
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    mats = [R.random_nvfp4(rng, n, k) for _ in range(3)]
    x = bits(rng, (off[-1], k))
    qb = torch.from_numpy(np.stack([mats[e % 3][0] for e in range(G)])).cuda()
    sfb = torch.from_numpy(np.concatenate([R.tile(mats[e % 3][1]) for e in range(G)])).cuda()
    gb = torch.tensor([mats[e % 3][2] for e in range(G)], dtype=torch.float32, device="cuda")
    y = nv.grouped_gemv(torch.from_numpy(off).cuda(), to_dev(x), qb, sfb, gb, n, None, nv.NVFP4_OUT_F32)
    again = nv.grouped_gemv(torch.from_numpy(off).cuda(), to_dev(x), qb, sfb, gb, n, None, nv.NVFP4_OUT_F32)
    assert torch.equal(y, again)
    got, w = f64(y), [R.nvfp4_matrix(*m) for m in mats]
    for e in range(G):
        if counts[e]:
            s = slice(off[e], off[e + 1])
            ref = val(x[s]) @ w[e % 3].T
            assert np.all(np.abs(got[s] - ref) <= bound(val(x[s]), w[e % 3], ref, True))


@pytest.mark.parametrize("rows,k", [(3, 20480), (9, 12288), (2, 45056)])
def test_long_rows(rows, k):
    """Rows of which few fit into shared memory at a time."""
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(k)
    q, sf, g = R.random_nvfp4(rng, 272, k)
    x = bits(rng, (rows, k))
    y = nv.gemv(to_dev(x), upload(nv, q, sf, g), nv.NVFP4_OUT_F32)
    w = R.nvfp4_matrix(q, sf, g)
    ref = val(x) @ w.T
    assert np.all(np.abs(f64(y) - ref) <= bound(val(x), w, ref, True))


def test_grouped_rows_outside_groups_and_bad_indexes():
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(12)
    q, sf, g = R.random_nvfp4(rng, 128, 128)
    qb, sfb = torch.from_numpy(q[None]).cuda(), torch.from_numpy(R.tile(sf)).cuda()
    gb = torch.tensor([g], device="cuda")
    x = to_dev(bits(rng, (4, 128)))
    off = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    out = torch.full((5, 128), 7.0, device="cuda")
    idx = torch.tensor([2, 9, -1, 0, 0], dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    nv.grouped_gemv(off, x, qb, sfb, gb, 128, idx, nv.NVFP4_OUT_F32, out, workspace=ws)
    assert nv.nvfp4_workspace_status(ws) == 8
    assert bool((out[3:] == 7).all()) and bool((out[1:3] == 0).all())
    one = nv.gemv(x[2:3], nv.NVFP4Tensor(qb[0], sfb, gb, 128, 128, nv.NVFP4_SF_MMA), nv.NVFP4_OUT_F32)
    assert torch.equal(out[:1], one)


# Rows of which not all fit go in panels of columns.  The bound above holds for them: a panel's chain of sums is
# shorter than the whole row's by two for every 256 columns of the others, and the panels' sums add one each.

@pytest.mark.parametrize("rows", [4, 8, 9, 13, 16, 17, 24, 33])
@pytest.mark.parametrize("n,k", [(16, 45056), (272, 5888), (144, 11328), (2448, 8256)])
def test_panels(rows, n, k):
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(rows + k)
    q, sf, g = R.random_nvfp4(rng, n, k, extreme=True)
    x = bits(rng, (rows, k))
    wide = torch.full((rows + 1, n + 16), 5.0, device="cuda")
    y = nv.gemv(to_dev(x), upload(nv, q, sf, g), nv.NVFP4_OUT_F32, wide[:rows, :n])
    w = R.nvfp4_matrix(q, sf, g)
    ref = val(x) @ w.T
    assert np.all(np.abs(f64(y) - ref) <= bound(val(x), w, ref, True))
    assert bool((wide[rows] == 5).all()) and bool((wide[:, n:] == 5).all())
    half = nv.gemv(to_dev(x), upload(nv, q, sf, g), nv.NVFP4_OUT_BF16)
    assert np.all(np.abs(f64(half) - ref) <= bound(val(x), w, ref, False))


def test_panels_of_different_size():
    """Columns of one panel far larger or smaller than the others', panels of zeros, small and large g."""
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(21)
    n, k = 128, 12288
    q, sf, _ = R.random_nvfp4(rng, n, k)
    v = rng.standard_normal((8, k))
    v[0, :512] *= 2.0 ** 90
    v[1, -512:] *= 2.0 ** 90
    v[2] *= 2.0 ** 110
    v[3] *= 2.0 ** -100
    v[4, 256:] = 0
    v[5, :-256] = 0
    v[6] = 0
    x = W.f32_to_bf16_bits(v.astype(np.float32))
    for g in (2.0 ** -20, 2.0 ** -3):
        w = R.nvfp4_matrix(q, sf, np.float32(g))
        ref = val(x) @ w.T
        y = f64(nv.gemv(to_dev(x), upload(nv, q, sf, np.float32(g)), nv.NVFP4_OUT_F32))
        assert np.all(np.abs(y - ref) <= bound(val(x), w, ref, True))
        assert (y[6] == 0).all()


def test_panels_non_finite_tokens_stay_alone():
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(22)
    n, k = 128, 12288
    q, sf, g = R.random_nvfp4(rng, n, k)
    x = bits(rng, (8, k))
    clean = f64(nv.gemv(to_dev(x), upload(nv, q, sf, g)))
    x[1, 3], x[3, 6000], x[6, k - 1] = 0x7F80, 0x7FC0, 0xFF80
    y = f64(nv.gemv(to_dev(x), upload(nv, q, sf, g)))
    np.testing.assert_array_equal(y[[0, 2, 4, 5, 7]], clean[[0, 2, 4, 5, 7]])
    assert np.isnan(y[3]).all() and not np.isfinite(y[[1, 6]]).any()


@pytest.mark.parametrize("rows", [8, 13])
def test_panels_more_tiles_than_sums_kept(rows):
    """So many matrix rows that a multiprocessor goes over the panels more than once."""
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(23)
    k, copies = 5888, 470
    q, sf, g = R.random_nvfp4(rng, 128, k)
    x = bits(rng, (rows, k))
    y = f64(nv.gemv(to_dev(x), upload(nv, np.tile(q, (copies, 1)), np.tile(sf, (copies, 1)), g), nv.NVFP4_OUT_F32))
    w = R.nvfp4_matrix(q, sf, g)
    ref = val(x) @ w.T
    assert np.all(np.abs(y.reshape(rows, copies, 128) - ref[:, None]) <= bound(val(x), w, ref, True)[:, None])


@pytest.mark.parametrize("counts", [[9, 0, 17, 8], [33], [0, 40, 1, 30]])
def test_panels_grouped(counts):
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(sum(counts))
    G, n, k, total = len(counts), 256, 8256, sum(counts)
    mats = [R.random_nvfp4(rng, n, k) for _ in range(G)]
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    src = bits(rng, (11, k))
    idx = rng.integers(0, 11, total + 2).astype(np.int32)
    out = torch.full((total + 2, n), 7.0, device="cuda")
    nv.grouped_gemv(torch.from_numpy(off).cuda(), to_dev(src), torch.from_numpy(np.stack([m[0] for m in mats])).cuda(),
                    torch.from_numpy(np.concatenate([R.tile(m[1]).reshape(-1) for m in mats])).cuda(),
                    torch.tensor([m[2] for m in mats], dtype=torch.float32, device="cuda"), n,
                    torch.from_numpy(idx).cuda(), nv.NVFP4_OUT_F32, out)
    got = f64(out)
    assert (got[total:] == 7).all()
    for e in range(G):
        s = slice(off[e], off[e + 1])
        xe, w = val(src[idx[s]]), R.nvfp4_matrix(*mats[e])
        if len(xe):
            ref = xe @ w.T
            assert np.all(np.abs(got[s] - ref) <= bound(xe, w, ref, True))


def test_panels_are_repeatable_in_a_graph():
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(24)
    q, sf, g = R.random_nvfp4(rng, 2048, 8256)
    x, w = to_dev(bits(rng, (8, 8256))), upload(nv, q, sf, g)
    first = nv.gemv(x, w, nv.NVFP4_OUT_F32)
    out = torch.empty_like(first)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.gemv(x, w, nv.NVFP4_OUT_F32, out)
    for _ in range(5):
        out.fill_(3.0)
        graph.replay()
        assert torch.equal(out, first)


@pytest.mark.parametrize("rows,n,k", [(5003, 48, 128), (1301, 16, 5888), (700, 128, 1024), (300, 1040, 320)])
def test_more_segments_than_multiprocessors(rows, n, k):
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(rows)
    q, sf, g = R.random_nvfp4(rng, n, k)
    x = bits(rng, (rows, k))
    y = nv.gemv(to_dev(x), upload(nv, q, sf, g), nv.NVFP4_OUT_F32)
    w = R.nvfp4_matrix(q, sf, g)
    ref = val(x) @ w.T
    assert np.all(np.abs(f64(y) - ref) <= bound(val(x), w, ref, True))


@pytest.mark.parametrize("rows,n,k", [(5, 128, 256), (13, 272, 512), (8, 128, 12288), (5, 2048, 64)])
@pytest.mark.parametrize("grouped", [True, False])
def test_infinities_beside_large_values(rows, n, k, grouped):
    """An infinite entry decides its row's sums; the finite ones beside it, beyond FP16's range or not, do not make
    them NaN.  Two infinities of opposite signs, and one under a weight of zero, do."""
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(k)
    q, sf, g = R.random_nvfp4(rng, n, k)
    q = (rng.integers(1, 8, (n, k // 2)) | rng.integers(1, 8, (n, k // 2)) << 4).astype(np.uint8)  # positive weights
    q[::5, 3] = 0
    if grouped and n % 128:
        n, q, sf = 256, q[:256], sf[:256]
    v = rng.standard_normal((rows, k))
    v[0], v[1], v[2] = -np.abs(v[0]) * 2.0 ** 125, np.abs(v[1]) * 1e6, np.abs(v[2]) * 2.0 ** -120
    v[0, k - 1], v[1, 6], v[2, 11] = np.inf, -np.inf, np.inf
    v[3, 1], v[3, k - 2] = np.inf, -np.inf
    x = W.f32_to_bf16_bits(v.astype(np.float32))
    if grouped:
        off = torch.tensor([0, 2, 2, rows], dtype=torch.int32, device="cuda")
        y = nv.grouped_gemv(off, to_dev(x), torch.from_numpy(np.stack([q] * 3)).cuda(),
                            torch.from_numpy(np.concatenate([R.tile(sf)] * 3)).cuda(),
                            torch.full((3,), float(g), device="cuda"), n, None, nv.NVFP4_OUT_F32)
    else:
        y = nv.gemv(to_dev(x), upload(nv, q, sf, g), nv.NVFP4_OUT_F32)
    w = R.nvfp4_matrix(q, sf, g)
    with np.errstate(invalid="ignore"):
        ref = val(x) @ w.T
    assert (ref[0] == np.inf).all() and (ref[1, ::5] != ref[1, ::5]).all() and (ref[1, 1::5] == -np.inf).all()
    np.testing.assert_array_equal(f64(y)[:4], ref[:4])
    finite = np.abs(f64(y)[4:] - ref[4:]) <= bound(val(x)[4:], w, ref[4:], True)
    assert finite.all()
