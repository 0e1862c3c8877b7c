"""The MoE block's operators together, as a model uses them: norm, routing, experts, combine; their autograd
forms; CUDA graphs, streams and concurrent calls.  The pieces' own tolerances are in their own tests: here each
stage is checked from the stage before it as the GPU computed it."""
import numpy as np
import pytest

import moe_ref as R
import workloads as W
from gpu_util import check_gemm, cuda_available, grouped_padded_rows, host, sf_mma_to_rowmajor, to_dev

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]

B = 2.0 ** -8


def bits(rng, shape, std=1.0):
    return W.f32_to_bf16_bits(rng.standard_normal(shape).astype(np.float32) * np.float32(std))


def val(b):
    return W.bf16_bits_to_f32(b).astype(np.float64)


def f64(t):
    return val(host(t)) if t.dtype.itemsize == 2 else host(t.detach()).astype(np.float64)


@pytest.fixture(scope="module")
def nv():
    import nvfp4_bit_precision_b200 as nv
    return nv


def experts(nv, rng, E, n, k):
    import torch
    from nvfp4_bit_precision_b200.moe import ExpertWeights
    t = [nv.quantize(to_dev(bits(rng, (n, k), 0.05)), sf_layout=nv.NVFP4_SF_MMA)["row"] for _ in range(E)]
    w = ExpertWeights(torch.stack([a.q for a in t]), torch.cat([a.sf for a in t]), torch.cat([a.g for a in t]), n)
    return w, [f64(nv.dequantize(a)) for a in t]


@pytest.mark.parametrize("tokens,masked", [(1, False), (5, True), (24, False)])
def test_decoding_step(nv, tokens, masked):
    """norm with the residual -> router -> the experts of a few tokens -> combine onto the residual stream."""
    import torch
    from nvfp4_bit_precision_b200.moe import expert_gemv, moe_route, rms_norm
    rng = np.random.default_rng(tokens)
    hidden, ffn, E, k = 256, 384, 8, 2
    up, up_w = experts(nv, rng, E, ffn, hidden)
    down, down_w = experts(nv, rng, E, hidden, ffn)
    x, res = to_dev(bits(rng, (tokens, hidden))), to_dev(bits(rng, (tokens, hidden)))
    w, router = to_dev(bits(rng, hidden, 0.5)), torch.from_numpy(rng.standard_normal((E, hidden)).astype(np.float32)).cuda()
    y, h = rms_norm(x, w, res)
    logits = y.float() @ router.t()
    if masked:
        logits[2] = -float("inf")
    r = moe_route(logits, k)
    out = expert_gemv(y, r, up, down, base=h)
    ids, wts = R.route(f64(logits), k)
    np.testing.assert_array_equal(host(r.expert), ids)
    ref, mag = f64(h).copy(), np.abs(f64(h))
    yy = f64(y)
    for t in range(tokens):
        for j in range(k):
            e = ids[t, j]
            if e < 0:
                continue
            mid = up_w[e] @ yy[t]
            ref[t] += wts[t, j] * (down_w[e] @ mid)
            # the bf16 rounding of the rows between the two products, and FP32 sums (below 2^-15 of the terms)
            mag[t] += wts[t, j] * (np.abs(down_w[e]) @ (B * np.abs(mid) + 2.0 ** -15 * (np.abs(up_w[e]) @ np.abs(yy[t])))) / 2 ** -15
    assert np.all(np.abs(f64(out) - ref) <= B * np.abs(ref) + 2.0 ** -15 * mag)
    if masked:
        assert torch.equal(out[2], h[2])


def test_routing_feeds_the_grouped_gemm(nv):
    """The plan's arrays are the ones that dispatch and grouped product read, for many tokens."""
    import torch
    rng = np.random.default_rng(3)
    tokens, hidden, n, E, k = 64, 256, 128, 6, 2
    w, wd = experts(nv, rng, E, n, hidden)
    x = to_dev(bits(rng, (tokens, hidden)))
    r = nv.route(torch.from_numpy(rng.standard_normal((tokens, E)).astype(np.float32)).cuda(), k)
    xq = nv.quantize(x, sf_layout=nv.NVFP4_SF_MMA)["row"]
    A = nv.gather_rows(xq, r.row_index, r.group_offsets)
    D = f64(nv.grouped_gemm(r.group_offsets, A, w.q, w.sf, w.g, n, nv.NVFP4_OUT_F32))
    off, idx, xr = host(r.group_offsets), host(r.row_index), f64(nv.dequantize(xq))
    ref, mag = np.empty_like(D), np.empty_like(D)
    for e in range(E):
        s = slice(off[e], off[e + 1])
        ref[s], mag[s] = xr[idx[s]] @ wd[e].T, np.abs(xr[idx[s]]) @ np.abs(wd[e]).T
    check_gemm(D, ref, mag, bf16_out=False)
    # and the same rows through the few-token product, which does not quantise x
    y = f64(nv.grouped_gemv(r.group_offsets, x, w.q, w.sf, w.g, n, r.row_index, nv.NVFP4_OUT_F32))
    for e in range(E):
        s = slice(off[e], off[e + 1])
        a = f64(x)[idx[s]]
        assert np.all(np.abs(y[s] - a @ wd[e].T) <= 2.0 ** -15 * (np.abs(a) @ np.abs(wd[e]).T))


def test_autograd_is_the_backward_calls(nv):
    """Gradients through autograd are those of the package's backward calls, bit for bit, also from an upstream
    gradient that is not contiguous and from a sum's broadcast one."""
    import torch
    from nvfp4_bit_precision_b200.moe import moe_combine, moe_route, rms_norm
    rng = np.random.default_rng(4)
    x, res = to_dev(bits(rng, (3, 10, 128))).requires_grad_(), to_dev(bits(rng, (3, 10, 128))).requires_grad_()
    w = to_dev(bits(rng, 128, 0.5)).requires_grad_()
    y, h = rms_norm(x, w, res)
    dy, dh = to_dev(bits(rng, (3, 10, 256)))[..., ::2], to_dev(bits(rng, (3, 10, 128)))
    torch.autograd.backward([y, h], [dy, dh])
    f = nv.rmsnorm(x.detach().reshape(30, 128), w.detach(), res.detach().reshape(30, 128), rstd=True)
    dx, dw = nv.rmsnorm_backward(dy.reshape(30, 128).contiguous(), f["h"], w.detach(), f["rstd"], dh.reshape(30, 128))
    assert torch.equal(x.grad.reshape(30, 128), dx) and torch.equal(res.grad, x.grad) and torch.equal(w.grad, dw)
    # only the sum used; only y used; no residual
    x2 = x.detach().clone().requires_grad_()
    rms_norm(x2, w.detach(), res.detach())[1].backward(dh)
    assert torch.equal(x2.grad, dh)
    x3, w3 = x.detach().clone().requires_grad_(), w.detach().clone().requires_grad_()
    rms_norm(x3, w3).sum().backward()
    g = nv.rmsnorm(x3.detach().reshape(30, 128), w3.detach(), rstd=True)
    dx, dw = nv.rmsnorm_backward(torch.ones((30, 128), dtype=torch.bfloat16, device="cuda"), g["h"], w3.detach(), g["rstd"])
    assert torch.equal(x3.grad.reshape(30, 128), dx) and torch.equal(w3.grad, dw)

    logits = torch.from_numpy(rng.standard_normal((30, 8)).astype(np.float32)).cuda().requires_grad_()
    rows = to_dev(bits(rng, (60, 128))).requires_grad_()
    base = to_dev(bits(rng, (30, 128))).requires_grad_()
    r = moe_route(logits, 2, score=nv.NVFP4_SIGMOID, scale=1.5)
    out = moe_combine(rows, r, base)
    dout = to_dev(bits(rng, (30, 128)))
    out.backward(dout)
    p = nv.route(logits.detach(), 2, score=nv.NVFP4_SIGMOID, scale=1.5)
    dr, dwt = nv.combine_backward(dout, rows.detach(), p.slot_row, p.weight, p.group_offsets)
    assert torch.equal(rows.grad, dr) and torch.equal(base.grad, dout)
    assert torch.equal(logits.grad, nv.route_backward(dwt, logits.detach(), p))


@pytest.mark.parametrize("same", [True, False])
def test_training_chain_against_64_bits(nv, same):
    """norm -> router and rows -> combine, differentiated end to end; the reference is torch autograd in float64 on
    the experts that the GPU chose.  At most six bf16 roundings lie between the loss and any leaf: 6 * 2^-8.

    With `same` a token's rows are all its own norm.  The weights' gradients <dout, row> of its slots are then one
    number g, and q_j (g_j - sum g q) vanishes: the router's gradient is nothing but FP32 arithmetic, at most 2^-17 of
    sum |g| for each logit (test_gpu_route.py), and is held to that.  Otherwise each expert scales its rows."""
    import torch
    from nvfp4_bit_precision_b200.moe import moe_combine, moe_route, rms_norm
    rng = np.random.default_rng(5)
    T, H, E, k = 40, 128, 6, 2
    leaf = lambda b: to_dev(b).requires_grad_()
    x, res, w = leaf(bits(rng, (T, H))), leaf(bits(rng, (T, H))), leaf(bits(rng, H, 0.5))
    router = torch.from_numpy(rng.standard_normal((E, H)).astype(np.float32) * 0.1).cuda().requires_grad_()
    dout = to_dev(bits(rng, (T, H)))
    factor = torch.ones(E, dtype=torch.bfloat16, device="cuda") if same else \
        torch.tensor([0.5, -1.0, 2.0, 1.0, -0.25, 4.0], dtype=torch.bfloat16, device="cuda")  # exact in bf16
    y, h = rms_norm(x, w, res)
    r = moe_route(y.float() @ router.t(), k)
    which = torch.repeat_interleave(torch.arange(E, device="cuda"), (r.group_offsets[1:] - r.group_offsets[:-1]).long())
    out = moe_combine(y[r.row_index.long()] * factor[which].unsqueeze(1), r, h)
    out.backward(dout)
    d = [t.detach().double().requires_grad_() for t in (x, res, w, router)]
    hh = d[0] + d[1]
    hq = hh + (h.detach().double() - hh).detach()     # the stored sum's value, the sum's gradient
    yy = hq * torch.rsqrt((hq * hq).mean(1, keepdim=True) + 1e-6) * d[2]
    lg = (yy @ d[3].t()).gather(1, r.expert.long())
    mix = torch.softmax(lg, 1) * factor.double()[r.expert.long()]
    ref = hq + (mix.unsqueeze(2) * yy.unsqueeze(1)).sum(1)
    ref.backward(dout.double())
    for got, want in zip((x, res, w) if same else (x, res, w, router), d):
        err = (got.grad.double() - want.grad).norm() / want.grad.norm()
        assert float(err) <= 6 * B, float(err)
    if same:
        g = k * (dout.double() * yy.detach()).sum(1, keepdim=True).abs()          # sum |g| of a token
        noise = torch.zeros((T, E), dtype=torch.float64, device="cuda").scatter_(1, r.expert.long(), g.expand(T, k))
        assert bool((router.grad.double().abs() <= 2.0 ** -16 * (noise.t() @ yy.detach().abs())).all())


def test_graphs(nv):
    """The block's calls captured once and replayed on new inputs, two graphs in turn, against eager calls."""
    import torch
    from nvfp4_bit_precision_b200.moe import expert_gemv
    rng = np.random.default_rng(6)
    hidden, E = 256, 8
    up, _ = experts(nv, rng, E, 128, hidden)
    down, _ = experts(nv, rng, E, hidden, 128)
    w = to_dev(bits(rng, hidden))

    def block(x, res, logits, dy):
        f = nv.rmsnorm(x, w, res, mx=True, amax=True, rstd=True, mx_sf_layout=nv.NVFP4_SF_MMA)
        r = nv.route(logits, 2)
        out = expert_gemv(f["y"], r, up, down, base=f["h"])
        dx, dw = nv.rmsnorm_backward(dy, f["h"], w, f["rstd"], dy)
        rows = f["y"][r.row_index.long()]
        dr, dwt = nv.combine_backward(dy, rows, r.slot_row, r.weight, r.group_offsets)
        return [f["y"], f["h"], f["mx"][0], f["mx"][1], f["amax"], out, dx, dw, dr, dwt, r.expert, r.row_index,
                nv.route_backward(dwt, logits, r)]

    def inputs(tokens):
        return [to_dev(bits(rng, (tokens, hidden))), to_dev(bits(rng, (tokens, hidden))),
                torch.from_numpy(rng.standard_normal((tokens, E)).astype(np.float32)).cuda(), to_dev(bits(rng, (tokens, hidden)))]

    made = []
    for tokens in (4, 300):
        static = inputs(tokens)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            block(*static)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = block(*static)
        made.append((g, static, outs))
    for _ in range(3):
        fresh = [inputs(s[0].shape[0]) for _, s, _ in made]
        want = [block(*f) for f in fresh]
        for (g, static, _), f in zip(made, fresh):
            for a, b in zip(static, f):
                a.copy_(b)
            g.replay()
        torch.cuda.synchronize()
        for (_, _, outs), ref in zip(made, want):
            for a, b in zip(outs, ref):
                assert torch.equal(a, b)


def test_streams_and_concurrent_calls(nv):
    """Calls given a stream, and two streams at once, give what the current stream gives."""
    import torch
    rng = np.random.default_rng(7)
    W1, _ = experts(nv, rng, 4, 1024, 512)
    x = to_dev(bits(rng, (6, 512)))
    wn = to_dev(bits(rng, 512))
    logits = [torch.from_numpy(rng.standard_normal((n, 4)).astype(np.float32)).cuda() for n in (3, 700)]
    plan = nv.route(logits[0], 2)
    ref = [nv.route(l, 2) for l in logits]
    ref_y = nv.grouped_gemv(plan.group_offsets, x, W1.q, W1.sf, W1.g, 1024, plan.row_index)
    ref_n = nv.rmsnorm(x, wn, x, rstd=True)
    ref_b = nv.rmsnorm_backward(x, ref_n["h"], wn, ref_n["rstd"])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(20):
        got = []
        for s in streams:
            given = s.cuda_stream if s is streams[0] else s
            got.append(([nv.route(l, 2, stream=given) for l in logits],
                        nv.grouped_gemv(plan.group_offsets, x, W1.q, W1.sf, W1.g, 1024, plan.row_index, stream=given),
                        nv.rmsnorm_backward(x, ref_n["h"], wn, ref_n["rstd"], stream=given),
                        nv.combine(ref_y, plan.slot_row, plan.weight, stream=given)))
        torch.cuda.synchronize()
        c = nv.combine(ref_y, plan.slot_row, plan.weight)
        for r, y, b, o in got:
            for p, q in zip(r, ref):
                assert torch.equal(p.expert, q.expert) and torch.equal(p.row_index, q.row_index)
                assert torch.equal(p.weight, q.weight) and torch.equal(p.group_offsets, q.group_offsets)
            assert torch.equal(y, ref_y) and torch.equal(b[0], ref_b[0]) and torch.equal(b[1], ref_b[1])
            assert torch.equal(o, c)


def test_captured_gradients_are_refused(nv):
    """Through autograd, while a stream captures; the package's calls are the way (see test_graphs)."""
    import torch
    from nvfp4_bit_precision_b200.moe import moe_combine, moe_route, rms_norm
    x = torch.ones((16, 128), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    logits = torch.zeros((16, 8), device="cuda", requires_grad=True)
    r = nv.route(logits.detach(), 2)
    rows = torch.zeros((32, 128), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for call in (lambda: rms_norm(x, w), lambda: moe_route(logits, 2), lambda: moe_combine(rows, r)):
            with pytest.raises(RuntimeError, match="CUDA graph"):
                call()
        with torch.no_grad():
            y = rms_norm(x, w)
    g.replay()
    torch.cuda.synchronize()
    assert bool((y == 1).all())


def test_gradients_that_begin_anywhere(nv):
    """An upstream gradient that is a piece of a larger tensor, off the 16-byte boundary that the kernels read from."""
    import torch
    from nvfp4_bit_precision_b200.moe import moe_combine, moe_route, rms_norm
    rng = np.random.default_rng(10)
    leaf = lambda *s: to_dev(bits(rng, s)).requires_grad_()
    x, res, w, rows, base = leaf(5, 128), leaf(5, 128), leaf(128), leaf(10, 128), leaf(5, 128)
    logits = torch.from_numpy(rng.standard_normal((5, 8)).astype(np.float32)).cuda().requires_grad_()
    leaves = (x, res, w, rows, base, logits)
    head = torch.zeros(3, dtype=torch.bfloat16, device="cuda")
    up = [to_dev(bits(rng, 3 + 5 * 128)) for _ in range(3)]

    def grads(apart):
        for t in leaves:
            t.grad = None
        y, h = rms_norm(x, w, res)
        out = moe_combine(rows, moe_route(logits, 2), base)
        if apart:
            torch.autograd.backward([y, h, out], [u[3:].clone().view(5, 128) for u in up])
        else:
            torch.autograd.backward([torch.cat([head, t.reshape(-1)]) for t in (y, h, out)], up)
        return [t.grad.clone() for t in leaves]

    for a, b in zip(grads(True), grads(False)):
        assert torch.equal(a, b)


def test_stream_numbers(nv, monkeypatch):
    """A stream given as its address, 0 for the default stream as torch gives it."""
    import torch
    rng = np.random.default_rng(11)
    x, w = to_dev(bits(rng, (4, 128))), to_dev(bits(rng, 128))
    side = torch.cuda.Stream()
    used, raw = [], nv._raw_stream
    monkeypatch.setattr(nv, "_raw_stream", lambda dev: used.append(raw(dev)) or used[-1])
    assert torch.cuda.default_stream().cuda_stream == 0
    with torch.cuda.stream(side):
        for s in (0, torch.cuda.default_stream(), side.cuda_stream, side, None):
            nv.rmsnorm(x, w, stream=s)
    nv.rmsnorm(x, w, stream=torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert used == [0, 0, side.cuda_stream, side.cuda_stream, side.cuda_stream, 0]


@pytest.mark.parametrize("shape", [(6, 128), (2, 3, 128), (128,)])
def test_gradients_accumulate_apart(nv, shape):
    """x and residual have one gradient, but two leaves do not share its memory: two backward passes give each of
    them twice the gradient, and leave the tensors that were handed in as they were."""
    import torch
    from nvfp4_bit_precision_b200.moe import rms_norm
    rng = np.random.default_rng(12)
    x, res, w = (to_dev(bits(rng, s)).requires_grad_() for s in (shape, shape, 128))
    dy, dh = to_dev(bits(rng, shape)), to_dev(bits(rng, shape))
    kept = dh.clone()

    def twice(outputs, grads):
        out = []
        for n in range(2):
            y, h = rms_norm(x, w, res)
            torch.autograd.backward([(y, h)[i] for i in outputs], grads)
            out.append([t.grad.clone() for t in (x, res)])
            assert x.grad.data_ptr() != res.grad.data_ptr()
        x.grad = res.grad = w.grad = None
        return out

    for outputs, grads in (((0, 1), [dy, dh]), ((0,), [dy]), ((1,), [dh])):
        (a, b), (a2, b2) = twice(outputs, grads)
        assert torch.equal(a, b) and torch.equal(a2, 2 * a) and torch.equal(b2, 2 * b)   # (doubling is exact)
        assert torch.equal(dh, kept)


def test_norm_of_strided_inputs_and_changed_outputs(nv):
    """Views with gaps go in and out; y may be changed in place, and a change of the sum or of x that the backward
    pass reads is reported."""
    import torch
    from nvfp4_bit_precision_b200.moe import rms_norm
    rng = np.random.default_rng(13)
    wide, w = to_dev(bits(rng, (4, 6, 256))), to_dev(bits(rng, 128)).requires_grad_()
    a, b = wide[:, ::2, :128], wide[:, 1::2, 128:]
    xs, rs = (t.detach().clone().requires_grad_() for t in (a, b))
    xv, rv = (torch.empty(4, 3, 256, dtype=torch.bfloat16, device="cuda")[..., :128].copy_(t).requires_grad_() for t in (a, b))
    dy = to_dev(bits(rng, (4, 3, 128)))
    for p, q in ((xs, rs), (xv, rv)):
        y, h = rms_norm(p, w, q)
        y.mul_(2.0)
        torch.autograd.backward([y, h], [dy, dy])
    assert torch.equal(xs.grad, xv.grad) and torch.equal(rs.grad, rv.grad) and torch.equal(xs.grad, rs.grad)
    y, h = rms_norm(xs, w, rs)
    h.add_(1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    y = rms_norm(xs, w)
    with torch.no_grad():
        xs.add_(1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
