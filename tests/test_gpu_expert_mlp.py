"""A few tokens' experts, activation inside, against float64.

Tolerance.  A product's sum over k columns is off by (8 * 17 + 2 ceil(k / 256) + 19) 2^-23 of the magnitudes, as the
few-token products' own tests derive.  silu(z) u: |silu'| <= 1.1, the exponential and the division 2^-20; h is rounded
to bf16, 2^-8 of it; the last product carries what h is off by, and rounds its own sums; the weighted sum in FP32 adds
(k + 1) 2^-24 and the result's rounding 2^-8."""
import numpy as np
import pytest

import moe_ref as R
import workloads as W
from gpu_util import cuda_available, host, to_dev

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]


@pytest.fixture(scope="module")
def nv():
    import nvfp4_bit_precision_b200 as nv
    return nv


def bits(rng, shape, std=1.0):
    return W.f32_to_bf16_bits(rng.standard_normal(shape).astype(np.float32) * np.float32(std))


def val(b):
    return W.bf16_bits_to_f32(b).astype(np.float64)


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def matrices(rng, G, n, k, size=1.0):
    import torch
    from nvfp4_bit_precision_b200.moe import ExpertWeights
    made = [R.random_nvfp4(rng, n, k) for _ in range(G)]
    g = [np.float32(size / np.sqrt(k) / np.abs(R.nvfp4_matrix(q, sf, 1.0)).std()) for q, sf, _ in made]
    w = ExpertWeights(dev(np.stack([q for q, _, _ in made])), dev(np.concatenate([R.tile(sf) for _, sf, _ in made])),
                      dev(np.array(g, np.float32)), n)
    return w, [R.nvfp4_matrix(q, sf, s) for (q, sf, _), s in zip(made, g)]


def routing(nv, ids, weight, G):
    import torch
    off, row_index, slot_row = R.plan(ids, G)
    return nv.Routing(dev(ids.astype(np.int32)), dev(weight), dev(off.astype(np.int32)), dev(row_index.astype(np.int32)),
                      dev(slot_row.astype(np.int32)), None)


def products(x, w):
    c = (8 * 17 + 2 * -(-x.shape[1] // 256) + 19) * 2.0 ** -23
    return x @ w.T, c * (np.abs(x) @ np.abs(w).T) + 2.0 ** -40 * np.abs(x).max(1, keepdims=True) * np.abs(w).sum(1)


def reference(x, ids, weight, up, down, gate, base):
    out = np.zeros((x.shape[0], down[0].shape[0])) if base is None else base.copy()
    err = np.zeros_like(out)
    mags = np.abs(out)
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = ids[t, j]
            if e < 0:
                continue
            u, du = products(x[t:t + 1], up[e])
            if gate is not None:
                z, dz = products(x[t:t + 1], gate[e])
                s = z / (1 + np.exp(-z))
                h, dh = s * u, np.abs(s) * du + 1.1 * dz * (np.abs(u) + du) + 2.0 ** -20 * np.abs(s * u)
            else:
                p = np.maximum(u, 0)
                h, dh = p * p, 2 * p * du + du * du + 2.0 ** -23 * p * p
            dh = dh + 2.0 ** -8 * (np.abs(h) + dh)
            y, dy = products(h, down[e])
            dy = dy + dh @ np.abs(down[e]).T * (1 + 2.0 ** -12)
            out[t] += weight[t, j] * y[0]
            err[t] += np.abs(weight[t, j]) * dy[0]
            mags[t] += np.abs(weight[t, j] * y[0])
    return out, err + (ids.shape[1] + 2) * 2.0 ** -24 * mags + 2.0 ** -8 * np.abs(out) + 2.0 ** -7 * err


def compare(got, ref, bound):
    err = np.abs(val(host(got)) - ref)
    assert np.all(err <= bound), float(np.max(err / bound))


@pytest.mark.parametrize("tokens,top_k,G", [(1, 1, 1), (1, 4, 8), (7, 2, 5), (16, 3, 4), (33, 2, 3), (24, 1, 60)])
@pytest.mark.parametrize("hidden,ffn", [(128, 128), (384, 256), (640, 896), (1024, 640)])
@pytest.mark.parametrize("gated", [True, False])
def test_experts(nv, tokens, top_k, G, hidden, ffn, gated):
    from nvfp4_bit_precision_b200 import moe
    if top_k > G:
        top_k = G
    rng = np.random.default_rng(tokens + G + hidden + ffn)
    up, upw = matrices(rng, G, ffn, hidden)
    down, downw = matrices(rng, G, hidden, ffn)
    gate, gatew = matrices(rng, G, ffn, hidden) if gated else (None, None)
    ids = np.stack([rng.permutation(G)[:top_k] for _ in range(tokens)])
    if tokens > 4:
        ids[2] = -1                                    # a token without experts, one with fewer
        ids[4, top_k - 1:] = -1
    weight = rng.random((tokens, top_k)).astype(np.float32) - np.float32(0.2)
    x, base = bits(rng, (tokens, hidden)), bits(rng, (tokens, hidden)) if tokens % 2 else None
    r = routing(nv, ids, weight, G)
    got = moe.expert_mlp(to_dev(x), r, up, down, gate, None if base is None else to_dev(base))
    compare(got, *reference(val(x), ids, weight, upw, downw, gatew, None if base is None else val(base)))


def test_many_rows_of_one_expert(nv):
    """Every token at the same expert: its rows are cut into segments; a wide hidden size fits few rows at a time."""
    from nvfp4_bit_precision_b200 import moe
    rng = np.random.default_rng(1)
    for tokens, hidden, ffn in ((70, 256, 384), (20, 8192, 128)):
        up, upw = matrices(rng, 3, ffn, hidden)
        down, downw = matrices(rng, 3, hidden, ffn)
        gate, gatew = matrices(rng, 3, ffn, hidden)
        ids, weight = np.full((tokens, 1), 1), np.ones((tokens, 1), np.float32)
        x = bits(rng, (tokens, hidden))
        got = moe.expert_mlp(to_dev(x), routing(nv, ids, weight, 3), up, down, gate)
        compare(got, *reference(val(x), ids, weight, upw, downw, gatew, None))


@pytest.mark.parametrize("gated", [True, False])
def test_large_and_small_products(nv, gated):
    """Gates far below zero give nothing, far above their product; tokens of different sizes side by side."""
    from nvfp4_bit_precision_b200 import moe
    rng = np.random.default_rng(2)
    hidden = ffn = 256
    up, upw = matrices(rng, 2, ffn, hidden)
    down, downw = matrices(rng, 2, hidden, ffn)
    gate, gatew = matrices(rng, 2, ffn, hidden, 60.0) if gated else (None, None)
    x = val(bits(rng, (6, hidden))) * np.array([1, 2.0 ** -20, 8, 0, 3, 2.0 ** 6])[:, None]
    xb = W.f32_to_bf16_bits(x.astype(np.float32))
    ids, weight = np.array([[0, 1]] * 6), np.ones((6, 2), np.float32)
    got = moe.expert_mlp(to_dev(xb), routing(nv, ids, weight, 2), up, down, gate)
    compare(got, *reference(val(xb), ids, weight, upw, downw, gatew, None))


def test_non_finite_tokens_stay_alone(nv):
    import torch
    from nvfp4_bit_precision_b200 import moe
    rng = np.random.default_rng(3)
    up, _ = matrices(rng, 2, 128, 256)
    down, _ = matrices(rng, 2, 256, 128)
    x = to_dev(bits(rng, (5, 256)))
    ids, weight = np.array([[0, 1]] * 5), np.ones((5, 2), np.float32)
    r = routing(nv, ids, weight, 2)
    for gate in (None, matrices(rng, 2, 128, 256)[0]):
        want = moe.expert_mlp(x, r, up, down, gate)
        bad = x.clone()
        bad[1, 3], bad[3, 200] = float("nan"), float("inf")
        got = moe.expert_mlp(bad, r, up, down, gate)
        assert torch.equal(got[[0, 2, 4]], want[[0, 2, 4]])
        assert torch.isnan(got[1].float()).all() and not torch.isfinite(got[3].float()).any()


def test_rows_without_an_expert_and_bad_indexes(nv):
    """Rows behind the last expert's are not computed; a bad row of x counts as zeros; bad slots are left out."""
    import torch
    from nvfp4_bit_precision_b200 import moe
    rng = np.random.default_rng(4)
    hidden, ffn, G = 256, 128, 4
    up, _ = matrices(rng, G, ffn, hidden)
    down, _ = matrices(rng, G, hidden, ffn)
    gate, _ = matrices(rng, G, ffn, hidden)
    x, base = to_dev(bits(rng, (6, hidden))), to_dev(bits(rng, (6, hidden)))
    ids, weight = np.stack([rng.permutation(G)[:2] for _ in range(6)]), rng.random((6, 2)).astype(np.float32)
    r = routing(nv, ids, weight, G)
    ws = torch.zeros(nv.nvfp4_expert_mlp_workspace_size(12, hidden, ffn), dtype=torch.uint8, device="cuda")
    want = nv.expert_mlp(x, r, up, down, gate, base, workspace=ws)
    assert nv.nvfp4_workspace_status(ws) == 0
    # what an earlier call left in the workspace does not matter
    ws.fill_(0xFF)
    assert torch.equal(nv.expert_mlp(x, r, up, down, gate, base, workspace=ws), want)
    # an empty routing
    none = nv.Routing(torch.full_like(r.expert, -1), r.weight, torch.zeros_like(r.group_offsets), torch.full_like(r.row_index, -1),
                      torch.full_like(r.slot_row, -1), None)
    assert torch.equal(nv.expert_mlp(x, none, up, down, gate, base, workspace=ws), base)
    assert not nv.expert_mlp(x, none, up, down, gate).any()
    # a row of x that does not exist: the token's slot gives nothing
    for bad in (-3, 6, 2 ** 31 - 1):
        index = r.row_index.clone()
        index[int(r.slot_row[2, 1])] = bad
        got = nv.expert_mlp(x, nv.Routing(r.expert, r.weight, r.group_offsets, index, r.slot_row, None), up, down, gate, base, workspace=ws)
        assert nv.nvfp4_workspace_status(ws) == 8
        slots = r.slot_row.clone()
        slots[2, 1] = -1
        left = nv.Routing(r.expert, r.weight, r.group_offsets, r.row_index, slots, None)
        assert torch.equal(got, nv.expert_mlp(x, left, up, down, gate, base, workspace=ws))
        assert nv.nvfp4_workspace_status(ws) == 0
    slots[2, 1] = 12
    assert torch.equal(nv.expert_mlp(x, left, up, down, gate, base, workspace=ws), got)
    assert nv.nvfp4_workspace_status(ws) == 8
    # no tokens at all
    empty = nv.Routing(*(t[:0] for t in (r.expert, r.weight)), torch.zeros_like(r.group_offsets), r.row_index[:0], r.slot_row[:0], None)
    assert nv.expert_mlp(x[:0], empty, up, down, gate).shape == (0, hidden)


def test_same_results_again(nv):
    """Twice, on two streams at once, captured and replayed with other tokens; x as a piece of a wider matrix."""
    import torch
    rng = np.random.default_rng(5)
    hidden, ffn, G = 512, 384, 16
    up, _ = matrices(rng, G, ffn, hidden)
    down, _ = matrices(rng, G, hidden, ffn)
    gate, _ = matrices(rng, G, ffn, hidden)
    wide = to_dev(bits(rng, (9, 2 * hidden)))
    x = wide[:, hidden:]
    ids, weight = np.stack([rng.permutation(G)[:3] for _ in range(9)]), rng.random((9, 3)).astype(np.float32)
    r = routing(nv, ids, weight, G)
    want = nv.expert_mlp(x, r, up, down, gate)
    assert torch.equal(nv.expert_mlp(x.contiguous(), r, up, down, gate), want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [nv.expert_mlp(x, r, up, down, gate, stream=streams[i % 2]) for i in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = nv.expert_mlp(x, r, up, down, gate)
    wide.mul_(0.5)
    for _ in range(3):
        graph.replay()
    assert torch.equal(out, nv.expert_mlp(x, r, up, down, gate))


def test_routings_that_change_behind_an_empty_one(nv):
    """The routing's tensors are written anew as soon as a call that had no rows is behind: neither call sees the
    other's, eager or captured (a call ends only when all its kernels have)."""
    import torch
    rng = np.random.default_rng(6)
    hidden, ffn, G, tokens = 256, 128, 4, 6
    up, _ = matrices(rng, G, ffn, hidden)
    down, _ = matrices(rng, G, hidden, ffn)
    gate, _ = matrices(rng, G, ffn, hidden)
    x, base = to_dev(bits(rng, (tokens, hidden))), to_dev(bits(rng, (tokens, hidden)))
    r = routing(nv, np.stack([rng.permutation(G)[:2] for _ in range(tokens)]), rng.random((tokens, 2)).astype(np.float32), G)
    none = [torch.full_like(r.expert, -1), r.weight, torch.zeros_like(r.group_offsets), torch.full_like(r.row_index, -1),
            torch.full_like(r.slot_row, -1)]
    full = [r.expert, r.weight, r.group_offsets, r.row_index, r.slot_row]
    want = nv.expert_mlp(x, r, up, down, gate, base)
    now = [t.clone() for t in none]
    live = nv.Routing(*now, None)
    ws = torch.zeros(nv.nvfp4_expert_mlp_workspace_size(2 * tokens, hidden, ffn), dtype=torch.uint8, device="cuda")

    def turn():
        a = nv.expert_mlp(x, live, up, down, gate, base, workspace=ws)
        torch._foreach_copy_(now, full)
        b = nv.expert_mlp(x, live, up, down, gate, base, workspace=ws)
        torch._foreach_copy_(now, none)
        return a, b

    outs = [turn() for _ in range(100)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs.append(turn())
    graph.replay()
    for a, b in outs:
        assert torch.equal(a, base) and torch.equal(b, want)
    assert nv.nvfp4_workspace_status(ws) == 0


@pytest.mark.parametrize("gated", [True, False])
def test_slots_behind_the_routed_rows(nv, gated):
    """A slot that names a row behind group_offsets[G], which no product writes, is left out and reported, whatever
    the workspace held there."""
    import torch
    rng = np.random.default_rng(7)
    hidden, ffn, G, tokens = 256, 128, 3, 9
    up, _ = matrices(rng, G, ffn, hidden)
    down, _ = matrices(rng, G, hidden, ffn)
    gate = matrices(rng, G, ffn, hidden)[0] if gated else None
    x, base = to_dev(bits(rng, (tokens, hidden))), to_dev(bits(rng, (tokens, hidden)))
    ids = np.stack([rng.permutation(G)[:2] for _ in range(tokens)])
    ids[4], ids[7, 1] = -1, -1                                  # three slots without an expert: 15 routed rows of 18
    r = routing(nv, ids, rng.random((tokens, 2)).astype(np.float32), G)
    size = nv.nvfp4_expert_mlp_workspace_size(2 * tokens, hidden, ffn)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    want = nv.expert_mlp(x, r, up, down, gate, base, workspace=ws)
    assert nv.nvfp4_workspace_status(ws) == 0 and int(r.group_offsets[-1]) == 15
    for row in (15, 17):
        slots = r.slot_row.clone()
        slots[4, 0] = slots[7, 1] = row
        for left in (0x00, 0x3F, 0xFF):
            ws.fill_(left)
            got = nv.expert_mlp(x, nv.Routing(r.expert, r.weight, r.group_offsets, r.row_index, slots, None), up, down, gate, base, workspace=ws)
            assert nv.nvfp4_workspace_status(ws) == 8
            assert torch.equal(got, want)


def reference_by_expert(x, ids, weight, up, down, gate, base):
    """``reference``, all rows of an expert at once (its bounds are those of each row)."""
    out = base.copy()
    err, mags = np.zeros_like(out), np.abs(out)
    for e in range(len(up)):
        t, j = np.nonzero(ids == e)
        if not t.size:
            continue
        u, du = products(x[t], up[e])
        if gate is not None:
            z, dz = products(x[t], gate[e])
            s = z / (1 + np.exp(-z))
            h, dh = s * u, np.abs(s) * du + 1.1 * dz * (np.abs(u) + du) + 2.0 ** -20 * np.abs(s * u)
        else:
            p = np.maximum(u, 0)
            h, dh = p * p, 2 * p * du + du * du + 2.0 ** -23 * p * p
        dh = dh + 2.0 ** -8 * (np.abs(h) + dh)
        y, dy = products(h, down[e])
        dy = dy + dh @ np.abs(down[e]).T * (1 + 2.0 ** -12)
        w = weight[t, j][:, None].astype(np.float64)
        np.add.at(out, t, w * y)
        np.add.at(err, t, np.abs(w) * dy)
        np.add.at(mags, t, np.abs(w * y))
    return out, err + (ids.shape[1] + 2) * 2.0 ** -24 * mags + 2.0 ** -8 * np.abs(out) + 2.0 ** -7 * err


@pytest.mark.parametrize("tokens,top_k,G,hidden,ffn", [(96, 2, 12, 640, 4096), (40, 1, 6, 1024, 6272), (16, 8, 128, 256, 128), (5, 8, 256, 128, 256),
                                                       (200, 2, 256, 128, 128)])
@pytest.mark.parametrize("gated", [True, False])
def test_wide_experts_and_many(nv, tokens, top_k, G, hidden, ffn, gated):
    """Down products of which a CTA's segments do not fit at once (rows of h of 8 and 12 KB); as many experts as are
    taken, most of them without a row."""
    from nvfp4_bit_precision_b200 import moe
    rng = np.random.default_rng(tokens + G + hidden + ffn)
    up, upw = matrices(rng, G, ffn, hidden)
    down, downw = matrices(rng, G, hidden, ffn)
    gate, gatew = matrices(rng, G, ffn, hidden) if gated else (None, None)
    ids = np.stack([rng.permutation(G)[:top_k] for _ in range(tokens)])
    weight = rng.random((tokens, top_k)).astype(np.float32) - np.float32(0.2)
    x, base = bits(rng, (tokens, hidden)), bits(rng, (tokens, hidden))
    got = moe.expert_mlp(to_dev(x), routing(nv, ids, weight, G), up, down, gate, to_dev(base))
    compare(got, *reference_by_expert(val(x), ids, weight, upw, downw, gatew, val(base)))


@pytest.mark.parametrize("tokens", [1, 20])
@pytest.mark.parametrize("gated", [True, False])
def test_what_h_is_rounded_to(nv, gated, tokens):
    """h enters the last product in FP16 at a power of two a row: 2^-11 of itself, 2^-38 of the row's largest.  Down
    matrices that hand h through, a base that takes most of it away again."""
    import torch
    from nvfp4_bit_precision_b200 import moe
    rng = np.random.default_rng(8)
    hidden = ffn = 384
    up, upw = matrices(rng, 1, ffn, hidden)
    gate, gatew = matrices(rng, 1, ffn, hidden, 4.0) if gated else (None, None)
    q = np.zeros((1, hidden, ffn // 2), np.uint8)
    at = np.arange(hidden)
    q[0, at, at // 2] = np.where(at % 2, 0x20, 0x02)                                     # 1.0
    down = moe.ExpertWeights(dev(q), torch.full((hidden * ffn // 16,), 0x38, dtype=torch.uint8, device="cuda"), torch.ones(1, device="cuda"), hidden)
    x = val(bits(rng, (tokens, hidden))) * np.exp2(rng.integers(-12, 12, (tokens, 1)))
    xb = W.f32_to_bf16_bits(x.astype(np.float32))
    u, du = products(val(xb), upw[0])
    if gated:
        z, dz = products(val(xb), gatew[0])
        s = z / (1 + np.exp(-z))
        h, dh = s * u, np.abs(s) * du + 1.1 * dz * (np.abs(u) + du) + 2.0 ** -20 * np.abs(s * u)
    else:
        p = np.maximum(u, 0)
        h, dh = p * p, 2 * p * du + du * du + 2.0 ** -23 * p * p
    base = W.f32_to_bf16_bits(-h.astype(np.float32))
    got = moe.expert_mlp(to_dev(xb), routing(nv, np.zeros((tokens, 1), int), np.ones((tokens, 1), np.float32), 1), up, down, gate, to_dev(base))
    ref = val(base) + h
    dh = dh + 2.0 ** -11 * (np.abs(h) + dh) + 2.0 ** -38 * np.abs(h).max(1, keepdims=True)
    # (the last product's sum of one number and zeros, its factors and the weighted sum: 8 roundings to FP32)
    compare(got, ref, dh * (1 + 2.0 ** -7) + 2.0 ** -20 * np.abs(h) + 2.0 ** -8 * np.abs(ref))
