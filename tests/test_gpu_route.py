"""Routing on the GPU against a token-by-token restatement in 64 bits: the chosen experts, the offsets and
both row orders are equal; weights and gradients are within FP32 arithmetic.

Tolerance of a weight: exp is off by 2 ulp (2^-22) and by half an ulp of its argument for each unit of it
(|argument| <= 30 here: 30 * 2^-24), numerator and denominator each, and the sum of up to 512 terms is 25
additions deep: less than 2^-17 in all."""
import numpy as np
import pytest

import moe_ref as R
import workloads as W
from gpu_util import cuda_available, host

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]

F = 2.0 ** -17
B = 2.0 ** -8


def draw(rng, tokens, experts, bf16, std=1.5):
    l = (rng.standard_normal((tokens, experts)) * std).astype(np.float32)
    return W.bf16_bits_to_f32(W.f32_to_bf16_bits(l)) if bf16 else l


def dev(l, bf16):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(l)).cuda()
    return t.to(torch.bfloat16) if bf16 else t


def check(l, bf16, top_k, softmax=True, bias=None, groups=1, topk_groups=1, group_top=2, renorm=True, scale=1.0,
          logits=None):
    import torch
    import nvfp4_bit_precision_b200 as nv
    x = dev(l, bf16) if logits is None else logits
    b = None if bias is None else torch.from_numpy(bias).cuda()
    r = nv.route(x, top_k, score=nv.NVFP4_SOFTMAX if softmax else nv.NVFP4_SIGMOID, bias=b, groups=groups,
                 topk_groups=topk_groups, group_top=group_top, renormalize=renorm, scale=scale)
    ids, wts = R.route(l, top_k, softmax, bias, groups, topk_groups, group_top, renorm, scale)
    np.testing.assert_array_equal(host(r.expert), ids)
    got = host(r.weight).astype(np.float64)
    assert np.all(np.abs(got - wts) <= F * np.abs(wts) + 2.0 ** -126), np.abs(got - wts).max()
    off, row, slot = R.plan(ids, l.shape[1])
    np.testing.assert_array_equal(host(r.group_offsets), off)
    np.testing.assert_array_equal(host(r.row_index), row)
    np.testing.assert_array_equal(host(r.slot_row), slot)
    return r, x, ids


SHAPES = [(1, 1, 1), (1, 8, 8), (2, 5, 3), (16, 64, 4), (17, 64, 4), (31, 33, 4), (127, 64, 4), (128, 64, 4), (129, 64, 4), (300, 60, 6),
          (515, 256, 8), (1185, 24, 3), (257, 160, 32), (40, 300, 7), (140, 512, 12)]


@pytest.mark.parametrize("tokens,experts,top_k", SHAPES)
@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("renorm", [True, False])
def test_plain_choice(tokens, experts, top_k, softmax, bf16, renorm):
    rng = np.random.default_rng(tokens * 3 + experts)
    check(draw(rng, tokens, experts, bf16), bf16, top_k, softmax, renorm=renorm, scale=1.0 if renorm else 2.5)


@pytest.mark.parametrize("tokens,experts,top_k,groups,topk_groups", [
    (5, 8, 2, 4, 2), (130, 256, 8, 8, 4), (64, 60, 5, 4, 1), (33, 96, 6, 32, 7), (200, 512, 9, 16, 3),
    (7, 6, 2, 6, 2), (90, 64, 4, 4, 4)])
@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("group_top", [1, 2])
def test_groups_and_bias(tokens, experts, top_k, groups, topk_groups, softmax, biased, group_top):
    rng = np.random.default_rng(experts + groups)
    bias = (rng.standard_normal(experts) * 0.05).astype(np.float32) if biased else None
    check(draw(rng, tokens, experts, True), True, top_k, softmax, bias, groups, topk_groups, group_top)


@pytest.mark.parametrize("softmax", [True, False])
def test_bias_alone(softmax):
    rng = np.random.default_rng(3)
    bias = (rng.standard_normal(64) * 0.3).astype(np.float32)
    check(draw(rng, 400, 64, False), False, 6, softmax, bias)
    check(draw(rng, 100, 64, False), False, 6, softmax, bias * 100)   # the bias decides


@pytest.mark.parametrize("softmax", [True, False])
def test_differences_below_fp32(softmax):
    """Biased scores that FP32 cannot tell apart are ranked as the exact ones; equal ones by index."""
    rng = np.random.default_rng(11)
    tokens, experts = 200, 32
    l = (rng.standard_normal((tokens, experts)) * 0.5).astype(np.float32)
    s = np.stack([R.scores(row.astype(np.float64), softmax) for row in l[:1]])[0]
    l[:] = l[0]
    bias = (1.0 - s).astype(np.float32)       # every biased score is 1 within FP32's rounding of the bias
    for t in range(tokens):                   # and the tokens' logits differ in the last bits
        l[t] = np.nextafter(l[t], np.float32(10.0 if t % 2 else -10.0))
    check(l, False, 8, softmax, bias)
    check(l, False, 8, softmax, bias, groups=8, topk_groups=3)
    same = np.zeros((150, experts), dtype=np.float32)
    check(same, False, 5, softmax, np.zeros(experts, dtype=np.float32))
    check(same, False, 5, softmax, np.zeros(experts, dtype=np.float32), groups=4, topk_groups=2)
    check(same, False, 5, softmax)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("tokens", [50, 300])
def test_masks(bf16, softmax, biased, tokens):
    """-inf, the types' lowest values, tokens that keep fewer experts than slots, tokens that keep none."""
    rng = np.random.default_rng(21)
    l = draw(rng, tokens, 64, bf16)
    low = [-np.inf, R.MASKED] + ([] if bf16 else [np.finfo(np.float32).min])
    for t in range(tokens):
        out = rng.random(64) < (0.5 if t % 3 else 0.97)
        l[t, out] = rng.choice(low, out.sum())
    l[7] = -np.inf
    l[8] = R.MASKED
    l[tokens - 1] = -np.inf
    bias = (rng.standard_normal(64)).astype(np.float32) if biased else None
    r, x, ids = check(l, bf16, 6, softmax, bias)
    assert (ids[7] == -1).all()
    check(l, bf16, 6, softmax, bias, groups=4, topk_groups=2)
    check(l, bf16, 6, softmax, bias, renorm=False)
    gradients(x, l, r, ids, softmax, True, 1.0, bf16)


def test_nan_and_infinite_logits():
    """A NaN ranks last and leaves the choice among the others alone; every index stays in range."""
    rng = np.random.default_rng(22)
    l = draw(rng, 64, 16, False)
    l[3, 2] = np.nan
    l[4] = np.nan
    l[5, 9] = np.inf
    import torch
    import nvfp4_bit_precision_b200 as nv
    r = nv.route(dev(l, False), 4)
    ids = host(r.expert)
    clean = l.copy()
    clean[3, 2] = -1e30
    ref, _ = R.route(clean[:4], 4)
    np.testing.assert_array_equal(ids[:4], ref)
    np.testing.assert_array_equal(ids[4], [0, 1, 2, 3])
    assert ids[5, 0] == 9 and ids.min() >= 0 and ids.max() < 16
    b = nv.route(dev(l, False), 4, bias=torch.zeros(16, device="cuda"), groups=4, topk_groups=2)
    assert int(b.expert.max()) < 16 and int(b.group_offsets[-1]) == 64 * 4


def test_far_negative_logits_keep_their_ratio():
    """Renormalised sigmoid and softmax weights of logits whose scores underflow."""
    rng = np.random.default_rng(23)
    l = draw(rng, 40, 32, False) - np.float32(300.0)
    check(l, False, 4, False)
    check(l, False, 4, True)


@pytest.mark.parametrize("softmax", [True, False])
def test_scores_near_the_smallest_numbers(softmax):
    """Groups ranked by scores that FP32 flushes to zero, or almost."""
    rng = np.random.default_rng(24)
    l = np.full((60, 16), -87.0, dtype=np.float32) - np.float32(4.0) * rng.random((60, 16)).astype(np.float32)
    if softmax:
        l[:, 5] = 0.0
    check(l, False, 4, softmax, groups=4, topk_groups=2)
    check(l, False, 4, softmax, groups=4, topk_groups=2, group_top=1)


def gradients(x, l, r, ids, softmax, renorm, scale, bf16):
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(5)
    dw = (rng.standard_normal(ids.shape) * 0.1).astype(np.float32)
    got = nv.route_backward(torch.from_numpy(dw).cuda(), x, r)
    assert got.dtype == x.dtype and got.shape == x.shape
    g = W.bf16_bits_to_f32(host(got)).astype(np.float64) if bf16 else host(got).astype(np.float64)
    ref = R.route_backward(dw, l, ids, softmax, renorm, scale)
    # each entry is a product with a difference of terms up to scale * sum |dw| (times the entry's own score)
    size = scale * np.abs(dw).sum(1, keepdims=True)
    assert np.all(np.abs(g - ref) <= (B if bf16 else 0) * np.abs(ref) + F * size)
    assert np.all(g[l <= R.MASKED] == 0)


@pytest.mark.parametrize("tokens,experts,top_k", SHAPES)
@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("bf16", [True, False])
def test_backward(tokens, experts, top_k, softmax, renorm, bf16):
    rng = np.random.default_rng(tokens + experts)
    l = draw(rng, tokens, experts, bf16)
    r, x, ids = check(l, bf16, top_k, softmax, renorm=renorm, scale=2.5)
    gradients(x, l, r, ids, softmax, renorm, 2.5, bf16)


def test_formula_against_differences():
    rng = np.random.default_rng(31)
    l = rng.standard_normal((4, 12))
    dw = rng.standard_normal((4, 3))
    for softmax in (True, False):
        for renorm in (True, False):
            ids, _ = R.route(l, 3, softmax, renorm=renorm, scale=1.5)
            d = R.route_backward(dw, l, ids, softmax, renorm, 1.5)
            u = rng.standard_normal(l.shape)
            step = 1e-6
            loss = lambda a: float((R.route(a, 3, softmax, renorm=renorm, scale=1.5)[1] * dw).sum())
            num = (loss(l + step * u) - loss(l - step * u)) / (2 * step)
            assert abs(num - (d * u).sum()) <= 1e-7 * (1 + abs(num))


def test_strided_logits_and_no_tokens():
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(41)
    wide = draw(rng, 150, 100, False)
    x = torch.from_numpy(wide).cuda()[:, 3:67]
    r, _, ids = check(np.ascontiguousarray(wide[:, 3:67]), False, 4, logits=x)
    gradients(x, np.ascontiguousarray(wide[:, 3:67]), r, ids, True, True, 1.0, False)
    e = nv.route(torch.empty((0, 64), device="cuda"), 4)
    assert e.expert.shape == (0, 4) and bool((e.group_offsets == 0).all())
    assert nv.route_backward(torch.empty((0, 4), device="cuda"), torch.empty((0, 64), device="cuda"), e).shape == (0, 64)


def test_many_tokens():
    """16384 tokens: the order of the rows against numpy's stable sort, and the same answer twice."""
    import torch
    import nvfp4_bit_precision_b200 as nv
    rng = np.random.default_rng(43)
    l = draw(rng, 16384, 64, False)
    x = dev(l, False)
    r = nv.route(x, 4)
    order = np.argsort(-l.astype(np.float64), axis=1, kind="stable")[:, :4]
    np.testing.assert_array_equal(host(r.expert), order)
    rows = np.argsort(order.reshape(-1), kind="stable")
    np.testing.assert_array_equal(host(r.row_index), rows // 4)
    slot = np.empty(rows.size, dtype=np.int64)
    slot[rows] = np.arange(rows.size)
    np.testing.assert_array_equal(host(r.slot_row), slot.reshape(-1, 4))
    again = nv.route(x, 4)
    for a, b in ((r.expert, again.expert), (r.weight, again.weight), (r.row_index, again.row_index)):
        assert torch.equal(a, b)


def cancelled(softmax, experts, where, small, rest):
    """41 tokens with expert `where`'s score cancelled by its bias but for its rounding, the logit in steps of one
    unit in the last place: the biased score is a small number that only the score's own digits tell, next to the
    biases `small` {expert: value} of experts with scores of 1e-17 (whose FP32 errors are far smaller), all others
    at the bias `rest`."""
    l = np.full((41, experts), -40.0, dtype=np.float32)
    l[:, where] = np.float32(0.4) + np.arange(-20, 21).astype(np.float32) * np.float32(2.0 ** -25)
    l[:, experts - 1] = 0.0                      # (softmax: the other half of the sum)
    bias = np.full(experts, rest, dtype=np.float32)
    bias[where] = -np.float32(R.scores(l[20].astype(np.float64), softmax)[where])
    for e, v in small.items():
        bias[e] = v
    return l, bias


@pytest.mark.parametrize("softmax", [True, False])
def test_a_third_score_within_its_error(softmax):
    """The best two FP32 scores are told apart by their own errors; a third one, with a larger error, is the best."""
    l, bias = cancelled(softmax, 8, 2, {0: 2e-9, 1: 1e-9}, -4.0)
    for k in (1, 2, 3):
        check(l, False, k, softmax, bias, renorm=False)
    l, bias = cancelled(softmax, 256, 200, {0: 2e-9, 1: 1e-9, 2: -1e-8}, -4.0)
    for k in (1, 2, 5):
        check(l, False, k, softmax, bias, renorm=False)


def test_a_third_softmax_score_of_many():
    """As above among 512 experts, the largest score not the winner of the FP32 order."""
    l = np.full((2, 512), -100.0, dtype=np.float32)
    l[:, 0], l[:, 1:16], l[:, 200:202] = 0.0, -16.54, -60.0
    p = R.scores(l[0].astype(np.float64), True)[0]
    bias = np.zeros(512, dtype=np.float32)
    bias[200], bias[201] = p - 2.4e-7, p - 6.0e-7
    check(l, False, 1, True, bias)
    check(l, False, 2, True, bias)


GROUPS = [(5, 4), (8, 4), (7, 3), (32, 4), (20, 5)]  # ranked by lanes, or one after the other


@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("groups,size", GROUPS)
def test_groups_within_a_third_ones_error(softmax, groups, size):
    """Group 1 has the cancelled score, groups 0 and 2 values whose errors tell those two apart: it is left out, kept
    last or kept first."""
    a, b, c = 0, size, 2 * size
    l, bias = cancelled(softmax, groups * size, b, {a: 2e-9, c: 1e-9}, -5.0)
    for topk_groups in (1, 2):
        check(l, False, 1, softmax, bias, groups, topk_groups, 1, renorm=False)
    # sums of the best two: 2e-9, the cancelled one, 1e-9
    l, bias = cancelled(softmax, groups * size, b, {a: 1e-9, a + 1: 1e-9, b + 1: 0.0, c: 5e-10, c + 1: 5e-10}, -5.0)
    for topk_groups in (1, 2):
        check(l, False, 2, softmax, bias, groups, topk_groups, 2, renorm=False)


@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("groups,size", GROUPS)
def test_a_member_of_a_group_within_its_error(softmax, groups, size):
    """The group's best scores in FP32 are not its best ones: a member with a larger error is."""
    b, c = size, 2 * size
    l, bias = cancelled(softmax, groups * size, b, {b + 1: 2e-9, c: 2.5e-9}, -5.0)
    check(l, False, 1, softmax, bias, groups, 1, 1, renorm=False)
    l, bias = cancelled(softmax, groups * size, b, {b + 1: 2e-9, b + 2: 1e-9, c: 2.5e-9, c + 1: 1e-9}, -5.0)
    check(l, False, 2, softmax, bias, groups, 1, 2, renorm=False)
