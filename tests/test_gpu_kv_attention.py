"""Attention over a paged NVFP4 cache against float64, with the bounds that kv_ref derives."""
import numpy as np
import pytest

import kv_ref as K
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


def i32(a):
    return dev(np.asarray(a, dtype=np.int32))


def filled(nv, rng, pages, kv, page, dim, amax=(8.0, 4.0), std=(1.0, 1.0)):
    """A cache of normal numbers (quantised by the plain form) and the page's unused part of any finite bytes."""
    c = nv.kv_cache(pages, kv, page, dim, *amax)
    q, sf = np.empty(tuple(c.q.shape), np.uint8), np.empty(tuple(c.sf.shape), np.uint8)
    for w in (0, 1):
        q[w], sf[w] = K.quantise((rng.standard_normal((pages, kv, page, dim)) * std[w]).astype(np.float32), amax[w])
    c.q.copy_(dev(q))
    c.sf.copy_(dev(sf))
    return c, q, sf


def sequence_of(q, sf, g, table, length, page):
    """One sequence's keys or values, float64 [kv, length, dim]."""
    n = -(-length // page)
    v = K.decode(q[table[:n]], sf[table[:n]], g)          # [pages, kv, page, dim]
    return v.transpose(1, 0, 2, 3).reshape(v.shape[1], -1, v.shape[3])[:, :length]


def check(nv, cache, q, sf, qb, table, lengths, page, window=0, scale=None, qd=None, td=None):
    g = host(cache.g)
    dim = qb.shape[3]
    qd, td = to_dev(qb) if qd is None else qd, i32(table) if td is None else td
    out, lse = nv.kv_attention(qd, cache, td, i32(lengths), window=window, scale=scale, lse=True)
    only = nv.kv_attention(qd, cache, td, i32(lengths), window=window, scale=scale)
    np.testing.assert_array_equal(host(only), host(out))
    got, sums = val(host(out)), host(lse).astype(np.float64)
    for s, n in enumerate(lengths):
        k, v = (sequence_of(q[w], sf[w], g[w], table[s], n, page) for w in (0, 1))
        ref, l, ob, lb = K.attend(val(qb[s]), k, v, n, np.float32(dim ** -0.5 if scale is None else scale).astype(np.float64), window)
        assert np.all(np.abs(got[s] - ref) <= ob + 2.0 ** -8 * np.abs(ref)), (s, n, np.max(np.abs(got[s] - ref) / (ob + 2.0 ** -8 * np.abs(ref) + 1e-30)))
        nothing = np.isneginf(l)
        np.testing.assert_array_equal(np.isneginf(sums[s]), nothing)
        assert np.all(np.abs(sums[s][~nothing] - l[~nothing]) <= lb[~nothing])
        assert not got[s][nothing].any()
    return out


@pytest.mark.parametrize("dim,kv,group", [(128, 2, 4), (128, 1, 1), (128, 2, 5), (128, 1, 16), (128, 1, 17), (64, 3, 2), (64, 1, 9), (256, 2, 2),
                                          (256, 1, 12)])
@pytest.mark.parametrize("page", [16, 32, 128])
@pytest.mark.parametrize("new,window", [(1, 0), (3, 0), (1, 50), (4, 33)])
def test_ragged(nv, dim, kv, group, page, new, window):
    rng = np.random.default_rng(dim + 7 * kv + group + page + new + window)
    lengths = [0, 1, 2, 15, 16, 17, 31, 33, 64, 127, 128, 129, 300, 517]
    most = -(-517 // page)
    pages = len(lengths) * most + 2
    cache, q, sf = filled(nv, rng, pages, kv, page, dim)
    table = rng.permutation(pages)[:len(lengths) * most].reshape(len(lengths), most)
    check(nv, cache, q, sf, bits(rng, (len(lengths), new, kv * group, dim), 1.5), table, lengths, page, window)


@pytest.mark.parametrize("n,lengths", [(1, [5000]), (3, [9000, 1, 700]), (200, None)])
def test_cut_lengths(nv, n, lengths):
    """Long sequences are cut into parts that several CTAs take; many short ones share a CTA."""
    rng = np.random.default_rng(n)
    dim, kv, page = 128, 2, 64
    lengths = lengths or list(rng.integers(0, 260, n))
    most = -(-max(lengths) // page)
    pages = n * most
    cache, q, sf = filled(nv, rng, pages, kv, page, dim)
    table = rng.permutation(pages).reshape(n, most)
    check(nv, cache, q, sf, bits(rng, (n, 1, 6, dim), 2.0), table, lengths, page)


@pytest.mark.parametrize("heads,new", [(3, 1), (9, 1), (9, 3)])
def test_more_items_than_workers(nv, heads, new):
    """Short sequences by the hundred, a few long ones among them, the first and the last too."""
    rng = np.random.default_rng(heads + new)
    n, dim, kv, page = 700, 64, 3, 16
    lengths = rng.integers(0, 60, n)
    lengths[[0, 137, 138, 500, 699]] = [700, 1024, 3, 1000, 650]
    pages = int(sum(-(-lengths // page))) + 1
    cache, q, sf = filled(nv, rng, pages, kv, page, dim)
    table, at = np.full((n, 64), -1), 0
    order = rng.permutation(pages)
    for i, m in enumerate(-(-lengths // page)):
        table[i, :m] = order[at:at + m]
        at += m
    check(nv, cache, q, sf, bits(rng, (n, new, heads, dim)), table, [int(x) for x in lengths], page)


@pytest.mark.parametrize("n", [129, 300])
def test_more_sequences_than_threads(nv, n):
    rng = np.random.default_rng(n)
    cache, q, sf = filled(nv, rng, n, 1, 16, 64)
    table = rng.permutation(n)[:, None]
    check(nv, cache, q, sf, bits(rng, (n, 1, 2, 64)), table, list(rng.integers(0, 17, n)), 16)


@pytest.mark.parametrize("spread", [1.0, 30.0, 1e-20, 1e20])
def test_sharp_and_flat(nv, spread):
    """Scores from all but equal to one that takes all; queries of any size, each row on its own."""
    rng = np.random.default_rng(9)
    dim, page = 128, 32
    cache, q, sf = filled(nv, rng, 40, 1, page, dim, (1e3, 1e-3), (100.0, 1e-4))
    qb = bits(rng, (2, 1, 5, dim), 0.01)
    qb[0, 0, 1] = 0
    qb[1] = bits(rng, (1, 5, dim), 0.01 * spread)
    scale = dim ** -0.5 if spread < 1e10 else 1e-21
    check(nv, cache, q, sf, qb, rng.permutation(40).reshape(2, 20), [640, 601], page, scale=scale)


def test_negative_scale_and_growing_scores(nv):
    """The maximum rises with every token, then only falls."""
    rng = np.random.default_rng(10)
    dim, page, n = 64, 16, 800
    cache, q, sf = filled(nv, rng, n // page, 1, page, dim, (64.0, 4.0))
    ramp = np.linspace(0.0, 40.0, n).astype(np.float32)
    k = np.zeros((n // page, 1, page, dim), np.float32)
    k[:, 0, :, 0] = ramp.reshape(-1, page)
    q[0], sf[0] = K.quantise(k, 64.0)
    cache.q[0].copy_(dev(q[0]))
    cache.sf[0].copy_(dev(sf[0]))
    qb = np.zeros((1, 1, 2, dim), np.uint16)
    qb[..., 0] = W.f32_to_bf16_bits(np.array([[[1.0, -1.0]]], np.float32))
    for scale in (1.0, -1.0, 0.0):
        check(nv, cache, q, sf, qb, np.arange(n // page)[None], [n], page, scale=scale)


def test_windows(nv):
    """A window as long as the table or longer is none; one of a token leaves each query its own."""
    import torch
    rng = np.random.default_rng(16)
    cache, q, sf = filled(nv, rng, 12, 1, 16, 64)
    table, lengths = rng.permutation(12).reshape(2, 6), [96, 33]
    qb = bits(rng, (2, 3, 2, 64))
    whole = check(nv, cache, q, sf, qb, table, lengths, 16)
    for window in (96, 97, 2 ** 31 - 1, 2 ** 31, 2 ** 62):
        assert torch.equal(nv.kv_attention(to_dev(qb), cache, i32(table), i32(lengths), window=window), whole)
    for window in (1, 2, 16, 95):
        check(nv, cache, q, sf, qb, table, lengths, 16, window)


def test_strides(nv):
    """Queries as a piece of a projection's output, a table as a piece of a larger one."""
    import torch
    rng = np.random.default_rng(11)
    dim, page, kv, n, new, heads = 128, 32, 2, 5, 2, 6
    cache, q, sf = filled(nv, rng, 30, kv, page, dim)
    wide = bits(rng, (n, new, heads + 2 * kv, dim))
    big = rng.permutation(30).reshape(5, 6)
    check(nv, cache, q, sf, wide[:, :, :heads], big, [100, 3, 128, 77, 150], page, qd=to_dev(wide)[:, :, :heads],
          td=torch.cat([i32(big), i32(np.full((5, 3), 99))], 1)[:, :6])


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_masked_tokens_do_not_matter(nv, dim):
    """NaN scales behind the end of a sequence, in its pages and in the table's other pages, before the window and
    among the later of the query tokens: what does not see them stays as it was; what does is NaN."""
    import torch
    rng = np.random.default_rng(12 + dim)
    page, kv, new, n = 32, 2, 3, 83
    cache, q, sf = filled(nv, rng, 8, kv, page, dim)
    table, qd = i32([[5, 2, 7, 1]]), to_dev(bits(rng, (1, new, 2 * kv, dim)))
    for window in (0, 40):
        want, wl = nv.kv_attention(qd, cache, table, i32([n]), window=window, lse=True)
        bad = nv.KVCache(cache.q.clone(), cache.sf.clone(), cache.amax, cache.g)
        for w in (0, 1):
            bad.sf[w, 7, :, n - 64:] = 0x7F
            bad.sf[w, [1, 0, 3, 4, 6]] = 0xFF
            if window:
                bad.sf[w, 5, :, :n - 2 - window] = 0x7F
        got, gl = nv.kv_attention(qd, bad, table, i32([n]), window=window, lse=True)
        assert torch.equal(got, want) and torch.equal(gl, wl)
        # the last token, seen by the last query alone: one block of its value
        bad.sf[1, 7, 0, n - 1 - 64, 1] = 0x7F
        got = nv.kv_attention(qd, bad, table, i32([n]), window=window)
        assert torch.equal(got[:, :2], want[:, :2]) and torch.equal(got[:, 2, 2:], want[:, 2, 2:])
        nan = torch.isnan(got[0, 2, :2].float())
        assert nan[:, 16:32].all() and not nan[:, :16].any() and not nan[:, 32:].any()
        # and of its key: the whole row
        bad.sf[1, 7, 0, n - 1 - 64, 1] = 1
        bad.sf[0, 7, 1, n - 1 - 64, 0] = 0x7F
        got = nv.kv_attention(qd, bad, table, i32([n]), window=window)
        assert torch.equal(got[:, :2], want[:, :2]) and torch.isnan(got[0, 2, 2:].float()).all()
        # a value that all see
        bad.sf[0, 7, 1, n - 1 - 64, 0] = 1
        bad.sf[1, 2, 0, 20, 0] = 0x7F
        got = nv.kv_attention(qd, bad, table, i32([n]), window=window)
        assert torch.isnan(got[0, :, :2, :16].float()).all() and not torch.isnan(got[0, :, 2:].float()).any()


def test_non_finite_queries_stay_alone(nv):
    import torch
    rng = np.random.default_rng(13)
    cache, q, sf = filled(nv, rng, 8, 1, 64, 128)
    qd = to_dev(bits(rng, (2, 2, 4, 128)))
    table, lengths = i32([[0, 1, 2, 3], [4, 5, 6, 7]]), i32([200, 256])
    want = nv.kv_attention(qd, cache, table, lengths)
    qd[0, 1, 2, 5] = float("nan")
    qd[1, 0, 0, 7] = float("inf")
    got = nv.kv_attention(qd, cache, table, lengths)
    assert torch.isnan(got[0, 1, 2].float()).all() and torch.isnan(got[1, 0, 0].float()).all()
    keep = torch.ones((2, 2, 4), dtype=torch.bool, device="cuda")
    keep[0, 1, 2] = keep[1, 0, 0] = False
    assert torch.equal(got[keep], want[keep])


def test_bad_pages_and_lengths(nv):
    """A page outside the cache counts as zeros, a length outside the table as its end; both are reported."""
    import torch
    rng = np.random.default_rng(14)
    dim, page = 128, 32
    cache, q, sf = filled(nv, rng, 6, 1, page, dim)
    qd = to_dev(bits(rng, (2, 1, 4, dim)))
    size = nv.nvfp4_kv_attention_workspace_size(2, 1, 4, 1, dim, 96)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    good = nv.kv_attention(qd, cache, i32([[0, 1, 2], [3, 4, 5]]), i32([96, 0]), workspace=ws)
    assert nv.nvfp4_workspace_status(ws) == 0
    got = nv.kv_attention(qd, cache, i32([[0, 1, 2], [3, 4, 5]]), i32([2 ** 31 - 1, -7]), workspace=ws)
    assert nv.nvfp4_workspace_status(ws) == 8
    assert torch.equal(got, good)
    zero = nv.KVCache(torch.cat([cache.q, torch.zeros_like(cache.q[:, :1])], 1), torch.cat([cache.sf, torch.zeros_like(cache.sf[:, :1])], 1),
                      cache.amax, cache.g)
    want = nv.kv_attention(qd, zero, i32([[0, 6, 2], [3, 4, 6]]), i32([80, 96]), workspace=ws)
    assert nv.nvfp4_workspace_status(ws) == 0
    for bad in (-1, 6, 2 ** 31 - 1, -2 ** 31):
        got = nv.kv_attention(qd, cache, i32([[0, bad, 2], [3, 4, bad]]), i32([80, 96]), workspace=ws)
        assert nv.nvfp4_workspace_status(ws) == 8
        assert torch.equal(got, want)
    # entries past a sequence's length are not read
    got = nv.kv_attention(qd, cache, i32([[0, 1, -1], [3, 99, 99]]), i32([64, 32]), workspace=ws)
    assert nv.nvfp4_workspace_status(ws) == 0


def test_no_sequences_and_no_pages(nv):
    import torch
    cache = nv.kv_cache(2, 1, 16, 64)
    q = torch.zeros((0, 1, 2, 64), dtype=torch.bfloat16, device="cuda")
    assert nv.kv_attention(q, cache, torch.zeros((0, 3), dtype=torch.int32, device="cuda"), i32([])).shape == (0, 1, 2, 64)
    q = torch.ones((3, 2, 2, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = nv.kv_attention(q, cache, torch.zeros((3, 0), dtype=torch.int32, device="cuda"), i32([0, 0, 0]), lse=True)
    assert not out.any() and torch.isneginf(lse).all()


def test_same_results_again(nv):
    """Twice, on another stream, captured and replayed, and two calls at once on two streams."""
    import torch
    rng = np.random.default_rng(15)
    dim, page = 128, 64
    cache, q, sf = filled(nv, rng, 80, 2, page, dim)
    qd, table, lengths = to_dev(bits(rng, (2, 2, 10, dim))), i32(rng.permutation(80).reshape(2, 40)), i32([2560, 999])
    want = nv.kv_attention(qd, cache, table, lengths)
    assert torch.equal(nv.kv_attention(qd, cache, table, lengths), want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [nv.kv_attention(qd, cache, table, lengths, stream=streams[i % 2]) for i in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = nv.kv_attention(qd, cache, table, lengths)
    lengths.fill_(700)
    graph.replay()
    assert torch.equal(out, nv.kv_attention(qd, cache, table, lengths))


# ------------------------------------------------------------------------------------------ wide tables
def kernels_of(call):
    """The (mangled) names of the kernels that a call launches, from its captured graph."""
    import os
    import tempfile
    import warnings
    import torch
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    graph.enable_debug_mode()
    with torch.cuda.graph(graph):
        call()
    with tempfile.TemporaryDirectory() as d, warnings.catch_warnings():
        warnings.simplefilter("ignore")  # (torch announces the dump as one)
        graph.debug_dump(os.path.join(d, "graph.dot"))
        with open(os.path.join(d, "graph.dot")) as f:
            return f.read()


def widened(table, lengths, page, tokens):
    """The table as wide as `tokens` tokens, with no page behind a sequence's last."""
    wide = np.full((len(lengths), tokens // page), -1, dtype=np.int64)
    for s, n in enumerate(lengths):
        m = -(-int(n) // page)
        wide[s, :m] = table[s, :m]
    return wide


WIDE = 1 << 20  # tokens of a table that a serving program allocates for its longest context


@pytest.mark.parametrize("dim,step", [(64, 64), (128, 64), (256, 32)])
def test_steps_go_by_the_tables_width(nv, dim, step):
    """Narrow tables take steps of 32 tokens, wide ones of 64 for heads of up to 128: the tests below run what they say."""
    import torch
    cache = nv.kv_cache(4, 2, 16, dim)
    q = torch.zeros((3, 1, 4, dim), dtype=torch.bfloat16, device="cuda")
    names = []
    for table in (np.zeros((3, 4)), np.zeros((3, WIDE // 16))):
        args = (q, cache, i32(table), i32([5, 0, 64]))
        nv.kv_attention(*args)
        names.append(kernels_of(lambda: nv.kv_attention(*args)))  # noqa: B023
    for text, want in zip(names, (32, step)):
        assert f"attend_kernelILi{dim}ELi{want}E" in text, text[:2000]


@pytest.mark.parametrize("dim,kv,group", [(128, 2, 4), (128, 1, 17), (128, 3, 1), (64, 3, 2), (64, 1, 9), (256, 2, 3)])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 1024])
@pytest.mark.parametrize("new,window", [(1, 0), (3, 0), (1, 50), (4, 33), (6, 64)])
def test_ragged_in_a_wide_table(nv, dim, kv, group, page, new, window):
    rng = np.random.default_rng(dim + 7 * kv + group + page + new + window)
    lengths = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 300, 517]
    most = -(-517 // page)
    pages = len(lengths) * most + 2
    cache, q, sf = filled(nv, rng, pages, kv, page, dim)
    table = rng.permutation(pages)[:len(lengths) * most].reshape(len(lengths), most)
    check(nv, cache, q, sf, bits(rng, (len(lengths), new, kv * group, dim), 1.5), table, lengths, page, window,
          td=i32(widened(table, lengths, page, WIDE)))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n,lengths", [(1, [9000]), (3, [20000, 1, 700]), (200, None)])
def test_cut_lengths_in_a_wide_table(nv, dim, n, lengths):
    rng = np.random.default_rng(n + dim)
    kv, page = 2, 64
    lengths = lengths or list(rng.integers(0, 400, n))
    most = -(-max(lengths) // page)
    cache, q, sf = filled(nv, rng, n * most, kv, page, dim)
    table = rng.permutation(n * most).reshape(n, most)
    check(nv, cache, q, sf, bits(rng, (n, 1, 6, dim), 2.0), table, [int(x) for x in lengths], page,
          td=i32(widened(table, lengths, page, 1 << 18 if n > 3 else WIDE * 8)))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_masked_tokens_do_not_matter_in_a_wide_table(nv, dim, page):
    """NaN scales behind the end of a sequence, in pages of others, before the window and among the later of the query
    tokens, in steps of 64 tokens."""
    import torch
    rng = np.random.default_rng(dim + page)
    kv, new, n = 2, 3, 200
    most = -(-n // page)
    cache, q, sf = filled(nv, rng, 2 * most, kv, page, dim)
    own = rng.permutation(2 * most)[:most]
    others = np.setdiff1d(np.arange(2 * most), own)
    table = i32(widened(own[None], [n], page, WIDE * 8))
    qd = to_dev(bits(rng, (1, new, 2 * kv, dim)))

    def spoil(c, which, token, head=slice(None), block=slice(None), byte=0x7F):
        c.sf[which, int(own[token // page]), head, token % page, block] = byte

    for window in (0, 70):
        want, wl = nv.kv_attention(qd, cache, table, i32([n]), window=window, lse=True)
        bad = nv.KVCache(cache.q.clone(), cache.sf.clone(), cache.amax, cache.g)
        for w in (0, 1):
            bad.sf[w, others] = 0xFF
            for token in range(n, most * page):
                spoil(bad, w, token)
            for token in range(n - 2 - window if window else 0):
                spoil(bad, w, token)
        got, gl = nv.kv_attention(qd, bad, table, i32([n]), window=window, lse=True)
        assert torch.equal(got, want) and torch.equal(gl, wl)
        # the last token, seen by the last query alone: one block of its value
        spoil(bad, 1, n - 1, 0, 1)
        got = nv.kv_attention(qd, bad, table, i32([n]), window=window)
        assert torch.equal(got[:, :2], want[:, :2]) and torch.equal(got[:, 2, 2:], want[:, 2, 2:])
        nan = torch.isnan(got[0, 2, :2].float())
        assert nan[:, 16:32].all() and not nan[:, :16].any() and not nan[:, 32:].any()
        # its key in the other head: the whole row
        spoil(bad, 1, n - 1, 0, 1, 1)
        spoil(bad, 0, n - 1, 1, 0)
        got = nv.kv_attention(qd, bad, table, i32([n]), window=window)
        assert torch.equal(got[:, :2], want[:, :2]) and torch.isnan(got[0, 2, 2:].float()).all()
        # a value that all see
        spoil(bad, 0, n - 1, 1, 0, 1)
        spoil(bad, 1, n - 10, 0, 0)
        got = nv.kv_attention(qd, bad, table, i32([n]), window=window)
        assert torch.isnan(got[0, :, :2, :16].float()).all() and not torch.isnan(got[0, :, 2:].float()).any()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_bad_pages_in_a_wide_table(nv, dim, page):
    """A page outside the cache counts as zeros, wherever it lies in a step of 64 tokens, and is reported."""
    import torch
    rng = np.random.default_rng(dim + page)
    n = 400
    most = -(-n // page)
    cache, q, sf = filled(nv, rng, most, 1, page, dim)
    zero = nv.KVCache(torch.cat([cache.q, torch.zeros_like(cache.q[:, :1])], 1), torch.cat([cache.sf, torch.zeros_like(cache.sf[:, :1])], 1),
                      cache.amax, cache.g)
    qd = to_dev(bits(rng, (1, 1, 4, dim)))
    own = rng.permutation(most)
    ws = torch.zeros(nv.nvfp4_kv_attention_workspace_size(1, 1, 4, 1, dim, WIDE * 8), dtype=torch.uint8, device="cuda")
    for at in ([0], [most - 1], [most // 2], list(range(0, most, 2)), list(range(most))):
        entry = lambda x: i32(widened(np.where(np.isin(np.arange(most), at), x, own)[None], [n], page, WIDE * 8))  # noqa: B023, E731
        want = nv.kv_attention(qd, zero, entry(most), i32([n]), workspace=ws)
        assert nv.nvfp4_workspace_status(ws) == 0
        for bad in (-1, most, 2 ** 31 - 1):
            got = nv.kv_attention(qd, cache, entry(bad), i32([n]), workspace=ws)
            assert nv.nvfp4_workspace_status(ws) == 8
            assert torch.equal(got, want)


# ------------------------------------------------------------------------------------------ many queries
@pytest.mark.parametrize("dim,kv,group,page", [(64, 1, 2, 16), (128, 2, 1, 64), (256, 1, 3, 32)])
@pytest.mark.parametrize("new,window", [(33, 0), (128, 0), (128, 40), (1000, 0), (1000, 77)])
def test_a_prompts_queries(nv, dim, kv, group, page, new, window):
    """More queries than a block has rows: of a sequence that is longer, as long, and (its first queries see nothing)
    shorter."""
    rng = np.random.default_rng(dim + new + window)
    lengths = [new + 77, new, new // 2 + 1, 0]
    most = -(-lengths[0] // page)
    cache, q, sf = filled(nv, rng, 4 * most, kv, page, dim)
    table = rng.permutation(4 * most).reshape(4, most)
    check(nv, cache, q, sf, bits(rng, (4, new, kv * group, dim), 1.5), table, lengths, page, window)


@pytest.mark.parametrize("dim,wide", [(64, False), (64, True), (128, False), (128, True), (256, False)])
@pytest.mark.parametrize("page", [16, 32, 64])
def test_pages_before_the_window_are_not_read(nv, dim, wide, page):
    """A program that gives back the pages which no query's window reaches any more has no page there: that is no
    error, and what the queries see is as it was.  A missing page that one query sees is reported."""
    import torch
    rng = np.random.default_rng(dim + page + wide)
    tokens = WIDE * 8 if wide else 512
    lengths = [500, 333, 77, 16, 0]
    most = -(-max(lengths) // page)
    cache, q, sf = filled(nv, rng, len(lengths) * most, 2, page, dim)
    table = rng.permutation(len(lengths) * most).reshape(len(lengths), most)
    full = widened(table, lengths, page, tokens)
    size = nv.nvfp4_kv_attention_workspace_size(len(lengths), 3, 4, 2, dim, tokens)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for new, window in ((1, 1), (1, 17), (3, 33), (2, 100), (3, 64)):
        qd = to_dev(bits(rng, (len(lengths), new, 4, dim)))
        want, wl = nv.kv_attention(qd, cache, i32(full), i32(lengths), window=window, lse=True)
        left = full.copy()
        for s, n in enumerate(lengths):
            left[s, :max(0, n - new + 1 - window) // page] = -1
        got, gl = nv.kv_attention(qd, cache, i32(left), i32(lengths), window=window, lse=True, workspace=ws)
        assert nv.nvfp4_workspace_status(ws) == 0, (new, window)
        assert torch.equal(got, want) and torch.equal(gl, wl)
        left[0, max(0, lengths[0] - new + 1 - window) // page] = -1
        nv.kv_attention(qd, cache, i32(left), i32(lengths), window=window, workspace=ws)
        assert nv.nvfp4_workspace_status(ws) == 8, (new, window)


@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 20, 2.0 ** 27, 2.0 ** 40, 2.0 ** 90])
@pytest.mark.parametrize("dim,wide", [(64, False), (64, True), (128, False), (128, True), (256, False)])
def test_scores_of_any_size(nv, dim, wide, size):
    """Products that lie far above or below zero and far apart: the token of the largest has it all, in a whole sequence,
    among parts that are joined, behind a maximum that rises at every token and one that falls."""
    rng = np.random.default_rng(dim + wide)
    page, n = 16, 2400
    pages = n // page
    cache, q, sf = filled(nv, rng, pages, 1, page, dim, (2688.0, 4.0))
    # keys of one element, 1 to 6 times a block scale of 2^-2 to 2^3: rising, the last 16-block of tokens the largest twice over
    k = np.zeros((n, dim), np.float32)
    k[:, 0] = np.exp2(np.linspace(-2, 1, n)).astype(np.float32)
    k[n // 2, 0] = 12.0
    for order in (np.arange(n), np.arange(n)[::-1], rng.permutation(n)):
        kq, ksf = K.quantise(k[order].reshape(pages, 1, page, dim), 2688.0)
        q[0], sf[0] = kq, ksf
        cache.q[0].copy_(dev(q[0]))
        cache.sf[0].copy_(dev(sf[0]))
        keys = K.decode(kq, ksf, host(cache.g)[0])[:, 0].reshape(n, dim)[:, 0]
        v = K.decode(q[1], sf[1], host(cache.g)[1])[:, 0].reshape(n, dim)
        qb = np.zeros((1, 1, 2, dim), np.uint16)
        qb[..., 0] = W.f32_to_bf16_bits(np.array([[[size, -size]]], np.float32))
        table = np.arange(pages)[None]
        td = i32(widened(table, [n], page, WIDE * 8)) if wide else i32(table)
        out, lse = nv.kv_attention(to_dev(qb), cache, td, i32([n]), scale=64.0, lse=True)
        got, sums = val(host(out))[0, 0], host(lse)[0, 0].astype(np.float64)
        x = 64.0 * size * keys
        for row, score in ((0, x), (1, -x)):
            top = score.max()
            p = np.where(score == top, 1.0, 0.0)                    # (the next is 64 size 2^-6 below)
            assert (top - np.unique(score)[-2]) >= 2.0 ** 7
            ref = p @ v / p.sum()
            assert np.all(np.abs(got[row] - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -12) * (p @ np.abs(v)) / p.sum())
            assert abs(sums[row] - top - np.log(p.sum())) <= 2.0 ** -20 * (1 + abs(top))
