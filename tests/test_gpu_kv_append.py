"""Append to a paged NVFP4 cache, bit for bit against the plain form."""
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


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def i32(a):
    return dev(np.asarray(a, dtype=np.int32))


def random_cache(nv, rng, pages, kv, page, dim, amax=(8.0, 4.0)):
    c = nv.kv_cache(pages, kv, page, dim, *amax)
    c.q.copy_(dev(rng.integers(0, 256, c.q.shape, dtype=np.uint8)))
    c.sf.copy_(dev(rng.integers(0, 127, c.sf.shape, dtype=np.uint8)))
    return c


def place(held, table, position, sequence, values, page):
    """values [tokens, heads, ...] into held [pages, heads, page, ...]."""
    for t in range(len(position)):
        if position[t] >= 0 and sequence[t] >= 0:
            held[table[sequence[t], position[t] // page], :, position[t] % page] = values[t]


@pytest.mark.parametrize("dim,page,kv,heads", [(128, 64, 8, 32), (64, 16, 1, 3), (256, 32, 2, 10), (128, 128, 3, 0), (64, 1024, 5, 5)])
@pytest.mark.parametrize("rot,neighbours", [(0, False), (32, False), (32, True), (-1, False), (-1, True)])
def test_appended(nv, dim, page, kv, heads, rot, neighbours):
    """Ragged sequences, some tokens left out, keys and values as pieces of one projection's output."""
    rng = np.random.default_rng(dim + page + kv + rot)
    rot = dim if rot < 0 else rot
    heads = heads if rot else 0
    counts, starts = [1, 0, 37, 5], [page - 1, 3, 11, 0]
    sequence = np.repeat(np.arange(4), counts)
    position = np.concatenate([np.arange(s, s + n) for s, n in zip(starts, counts)])
    order = rng.permutation(len(position))
    sequence, position = sequence[order], position[order]
    position[3], sequence[7] = -1, -5
    most = 48 // page + 2
    pages = 4 * most + 3
    table = rng.permutation(pages)[:4 * most].reshape(4, most)
    cache = random_cache(nv, rng, pages, kv, page, dim)
    cq, csf = host(cache.q).copy(), host(cache.sf).copy()
    tokens = len(position)
    qkv = bits(rng, (tokens, heads + 2 * kv, dim), 2.0)
    d = to_dev(qkv)
    q, k, v = d[:, :heads], d[:, heads:heads + kv], d[:, heads + kv:]
    cos, sin = K.tables(rot, 48 + page) if rot else (None, None)
    ws = cache.q.new_zeros(256)
    got = nv.kv_append(cache, k, v, i32(table), i32(position), i32(sequence), cos=dev(cos) if rot else None,
                       sin=dev(sin) if rot else None, interleaved=neighbours, q=q if heads else None, workspace=ws)
    assert nv.nvfp4_workspace_status(ws) == 0
    kb = qkv[:, heads:heads + kv]
    at = np.maximum(position, 0)
    if rot:
        kb = K.turn(kb, cos, sin, at, rot, neighbours)
    for which, b in ((0, kb), (1, qkv[:, heads + kv:])):
        codes, scales = K.quantise(W.bf16_bits_to_f32(b), host(cache.amax)[which])
        place(cq[which], table, position, sequence, codes, page)
        place(csf[which], table, position, sequence, scales, page)
    np.testing.assert_array_equal(host(cache.q), cq)
    np.testing.assert_array_equal(host(cache.sf), csf)
    if heads:
        want = K.turn(qkv[:, :heads], cos, sin, at, rot, neighbours)
        there = (position >= 0) & (sequence >= 0)
        np.testing.assert_array_equal(host(got)[there], want[there])
    for which, t in ((0, cache.keys()), (1, cache.values())):
        mine = K.decode(cq[which].reshape(-1, dim // 2), csf[which].reshape(-1, dim // 16), host(cache.g)[which])
        np.testing.assert_allclose(host(nv.dequantize(t)), mine, rtol=2.0 ** -23)


@pytest.mark.parametrize("tokens", [1, 4000])
def test_one_token_each(nv, tokens):
    """Without `sequence` token t belongs to sequence t; many tokens take several heads a thread."""
    rng = np.random.default_rng(tokens)
    dim, page, kv, heads = 128, 16, 4, 40
    cache = random_cache(nv, rng, tokens + 1, kv, page, dim)
    cq, csf = host(cache.q).copy(), host(cache.sf).copy()
    table, position = rng.permutation(tokens + 1)[:tokens, None], rng.integers(0, 16, tokens)
    q, k, v = bits(rng, (tokens, heads, dim)), bits(rng, (tokens, kv, dim), 3.0), bits(rng, (tokens, kv, dim))
    cos, sin = K.tables(dim, 16)
    dq = to_dev(q)
    got = nv.kv_append(cache, to_dev(k), to_dev(v), i32(table), i32(position), cos=dev(cos), sin=dev(sin), q=dq, q_out=dq)
    assert got is dq
    np.testing.assert_array_equal(host(got), K.turn(q, cos, sin, position, dim, False))
    for which, b in ((0, K.turn(k, cos, sin, position, dim, False)), (1, v)):
        codes, scales = K.quantise(W.bf16_bits_to_f32(b), host(cache.amax)[which])
        place(cq[which], table, position, np.arange(tokens), codes, page)
        place(csf[which], table, position, np.arange(tokens), scales, page)
    np.testing.assert_array_equal(host(cache.q), cq)
    np.testing.assert_array_equal(host(cache.sf), csf)


def test_the_librarys_quantisation(nv):
    """The values' bits are those of nvfp4_quantize from the same amax."""
    import torch
    rng = np.random.default_rng(1)
    dim, page, kv, tokens = 128, 64, 2, 64
    for amax in (5.5, 1e-3, 2688.0, 0.0):
        cache = nv.kv_cache(1, kv, page, dim, 1.0, amax)
        v = to_dev(bits(rng, (tokens, kv, dim), max(amax, 1e-3) / 3))
        nv.kv_append(cache, v, v, i32([[0]]), i32(np.arange(tokens)), i32(np.zeros(tokens)))
        want = nv.quantize(v.transpose(0, 1).reshape(kv * tokens, dim).contiguous(), amax=torch.tensor([amax, amax], device="cuda"))["row"]
        assert torch.equal(cache.values().q, want.q) and torch.equal(cache.values().sf, want.sf)
        assert torch.equal(cache.values().g, want.g)


@pytest.mark.parametrize("neighbours", [False, True])
def test_rounding_borders(nv, neighbours):
    """Numbers whose turned value lies on or next to the middle of two bf16 numbers, large and tiny ones, zeros of both
    signs, large parts that cancel."""
    rng = np.random.default_rng(2)
    dim, n = 64, 512
    half = dim // 2
    cos = np.ones((n, half), dtype=np.float32)
    sin = np.ones((n, half), dtype=np.float32)
    eps = np.float32(2.0 ** -8)
    cos[0::8] = 1 + eps                                                  # exact middles
    cos[1::8] = np.nextafter(1 + eps, np.float32(2))
    cos[2::8] = np.nextafter(1 + eps, np.float32(0))
    sin[0::8], sin[1::8], sin[2::8] = 2.0 ** -30, 0, -2.0 ** -45
    sin[3::8] = np.float32(1 / 3)
    cos[4::8], sin[4::8] = 1, 1                                          # equal parts cancel
    cos[5::8], sin[5::8] = np.nextafter(np.float32(1), np.float32(0)), 1
    cos[6::8], sin[6::8] = 2.0 ** -60, 2.0 ** -66
    cos[7::8], sin[7::8] = rng.standard_normal((2, n // 8, half))
    x = bits(rng, (n, 1, dim))
    x[:, :, 5] = 0
    x[:, :, half + 5] = 0x8000
    x[4::8, :, half:] = x[4::8, :, :half]
    x[4::8, :, 1::2] = x[4::8, :, 0::2]
    x[6::8] = bits(rng, (n // 8, 1, dim), 2.0 ** -70)
    x[6::16] = (x[6::16] & 0x8007)                                        # the smallest numbers
    cache = nv.kv_cache(n // 16, 1, 16, dim, 4.0, 4.0)
    got = nv.kv_append(cache, to_dev(x), to_dev(x), i32(np.arange(n // 16)[None]), i32(np.arange(n)), i32(np.zeros(n)), cos=dev(cos),
                       sin=dev(sin), interleaved=neighbours, q=to_dev(x))
    np.testing.assert_array_equal(host(got), K.turn(x, cos, sin, np.arange(n), dim, neighbours))


def test_tokens_without_a_place(nv):
    """Bad pages, places, sequences and angles are left out and reported; everything else is as it would be."""
    rng = np.random.default_rng(3)
    dim, page, kv = 64, 16, 2
    table = np.array([[1, 2], [7, 0], [-1, 3]])
    cos, sin = K.tables(dim, 30)
    good = dict(position=[0, 31 - 2], sequence=[0, 0])
    for bad in (dict(position=[32], sequence=[0]), dict(position=[3], sequence=[3]), dict(position=[0], sequence=[1]),
                dict(position=[0], sequence=[2]), dict(position=[30], sequence=[0]), dict(position=[2 ** 31 - 1], sequence=[0])):
        cache = random_cache(nv, rng, 4, kv, page, dim)
        other = nv.KVCache(cache.q.clone(), cache.sf.clone(), cache.amax, cache.g)
        k, v = to_dev(bits(rng, (3, kv, dim))), to_dev(bits(rng, (3, kv, dim)))
        ws = cache.q.new_zeros(256)
        nv.kv_append(cache, k, v, i32(table), i32(good["position"] + bad["position"]), i32(good["sequence"] + bad["sequence"]),
                     cos=dev(cos), sin=dev(sin), workspace=ws)
        assert nv.nvfp4_workspace_status(ws) == 8
        nv.kv_append(other, k[:2], v[:2], i32(table), i32(good["position"]), i32(good["sequence"]), cos=dev(cos), sin=dev(sin),
                     workspace=ws)
        assert nv.nvfp4_workspace_status(ws) == 0
        np.testing.assert_array_equal(host(cache.q), host(other.q))
        np.testing.assert_array_equal(host(cache.sf), host(other.sf))


def test_two_tokens_at_one_place(nv):
    """Each block of eight codes and each scale byte there is one of theirs; the places beside it are as they were."""
    rng = np.random.default_rng(6)
    dim, page, kv = 128, 16, 2
    cache = random_cache(nv, rng, 2, kv, page, dim)
    cq, csf = host(cache.q).copy(), host(cache.sf).copy()
    k, v = bits(rng, (2, kv, dim)), bits(rng, (2, kv, dim))
    nv.kv_append(cache, to_dev(k), to_dev(v), i32([[1]]), i32([5, 5]), i32([0, 0]))
    gq, gsf = host(cache.q), host(cache.sf)
    for which, b in ((0, k), (1, v)):
        codes, scales = K.quantise(W.bf16_bits_to_f32(b), host(cache.amax)[which])
        got, gots = gq[which, 1, :, 5].reshape(kv, -1, 4), gsf[which, 1, :, 5]
        codes = codes.reshape(2, kv, -1, 4)
        assert np.all((got == codes[0]).all(-1) | (got == codes[1]).all(-1))
        assert np.all((gots == scales[0]) | (gots == scales[1]))
    gq[:, 1, :, 5], gsf[:, 1, :, 5] = cq[:, 1, :, 5], csf[:, 1, :, 5]
    np.testing.assert_array_equal(gq, cq)
    np.testing.assert_array_equal(gsf, csf)


def test_streams_and_graphs(nv):
    """On another stream, captured and replayed with other tokens at other places."""
    import torch
    rng = np.random.default_rng(7)
    dim, page, kv, heads, n = 64, 16, 2, 4, 3
    cos, sin = (dev(a) for a in K.tables(dim, 64))
    a, b = (nv.kv_cache(12, kv, page, dim, 4.0, 4.0) for _ in range(2))
    table = i32(rng.permutation(12).reshape(n, 4))
    qkv, place = to_dev(bits(rng, (n, heads + 2 * kv, dim))), i32([0, 3, 40])
    call = lambda c, **kw: nv.kv_append(c, qkv[:, heads:heads + kv], qkv[:, heads + kv:], table, place, cos=cos, sin=sin,  # noqa: E731
                                        q=qkv[:, :heads], **kw)
    want = call(a)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(b, stream=stream)
    stream.synchronize()
    assert torch.equal(got, want) and torch.equal(a.q, b.q) and torch.equal(a.sf, b.sf)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(b)
    for i in range(5):
        qkv.copy_(to_dev(bits(rng, tuple(qkv.shape))))
        place += 1
        graph.replay()
        assert torch.equal(out, call(a)) and torch.equal(a.q, b.q) and torch.equal(a.sf, b.sf)


def test_nothing_to_append(nv):
    import torch
    cache = nv.kv_cache(1, 2, 16, 64)
    k = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    assert nv.kv_append(cache, k, k, i32([[0]]), i32([]), i32([])) is None
    assert not cache.q.any()


def test_no_tokens_with_queries(nv):
    """An empty batch is one like any other: queries without a token come back as they are."""
    import torch
    cache = nv.kv_cache(1, 2, 16, 64)
    cos, sin = (dev(a) for a in K.tables(64, 4))
    k, q = (torch.empty((0, n, 64), dtype=torch.bfloat16, device="cuda") for n in (2, 8))
    for out in (None, q):
        got = nv.kv_append(cache, k, k, i32([[0]]), i32([]), i32([]), cos=cos, sin=sin, q=q, q_out=out)
        assert got.shape == (0, 8, 64)
    assert not cache.q.any()


def test_offsets_past_32_bits(nv):
    """A cache of 5 GiB of keys' codes: its last page, and the values' behind it."""
    import torch
    rng = np.random.default_rng(5)
    dim, page, kv, pages = 256, 1024, 8, 5200
    cache = nv.KVCache(torch.empty((2, pages, kv, page, dim // 2), dtype=torch.uint8, device="cuda"),
                       torch.empty((2, pages, kv, page, dim // 16), dtype=torch.uint8, device="cuda"),
                       torch.tensor([4.0, 4.0], device="cuda"), torch.tensor([4.0, 4.0], device="cuda") / 2688)
    small = nv.kv_cache(1, kv, page, dim, 4.0, 4.0)
    cache.q[:, -1], cache.sf[:, -1] = 0, 0
    k, v = to_dev(bits(rng, (page, kv, dim))), to_dev(bits(rng, (page, kv, dim)))
    pos, seq = i32(np.arange(page)), i32(np.zeros(page))
    nv.kv_append(cache, k, v, i32([[pages - 1]]), pos, seq)
    nv.kv_append(small, k, v, i32([[0]]), pos, seq)
    assert torch.equal(cache.q[:, -1], small.q[:, 0]) and torch.equal(cache.sf[:, -1], small.sf[:, 0])
    q = to_dev(bits(rng, (1, 2, 16, dim)))
    a, b = (nv.kv_attention(q, c, i32([[p]]), i32([page - 3])) for c, p in ((cache, pages - 1), (small, 0)))
    assert torch.equal(a, b)


@pytest.mark.parametrize("dim,page,kv,heads,rot,neighbours,tokens", [
    (64, 16, 4, 16, 32, True, 3003), (64, 64, 3, 7, 64, False, 20000), (128, 64, 5, 0, 0, False, 9000), (128, 128, 2, 3, 64, True, 6000),
    (256, 32, 2, 6, 256, True, 2600), (256, 32, 2, 5, 32, False, 5000)])
def test_many_tokens(nv, dim, page, kv, heads, rot, neighbours, tokens):
    """Several heads a thread, most of them not a divisor of all heads: ragged prompts, their tokens in any order and some
    left out, the queries turned in place in a piece of the projection's output."""
    import torch
    rng = np.random.default_rng(dim + kv + heads + tokens)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert tokens * (heads + 2 * kv) * (dim // 16) >= 2 * 768 * sms  # (a thread for each head would be more than are at once)
    n = 7
    counts = rng.multinomial(tokens, np.full(n, 1 / n))
    starts = rng.integers(0, 40, n)
    sequence = np.repeat(np.arange(n), counts)
    position = np.concatenate([np.arange(s, s + c) for s, c in zip(starts, counts)])
    order = rng.permutation(tokens)
    sequence, position = sequence[order], position[order]
    position[5::97], sequence[9::101] = -1, -2
    most = -(-int((starts + counts).max()) // page)
    table = rng.permutation(n * most + 1)[:n * most].reshape(n, most)
    cache = random_cache(nv, rng, n * most + 1, kv, page, dim)
    cq, csf = host(cache.q).copy(), host(cache.sf).copy()
    qkv = bits(rng, (tokens, heads + 2 * kv, dim), 2.0)
    d = to_dev(qkv)
    q, k, v = d[:, :heads], d[:, heads:heads + kv], d[:, heads + kv:]
    cos, sin = K.tables(rot, most * page) if rot else (None, None)
    ws = cache.q.new_zeros(256)
    got = nv.kv_append(cache, k, v, i32(table), i32(position), i32(sequence), cos=dev(cos) if rot else None, sin=dev(sin) if rot else None,
                       interleaved=neighbours, q=q if heads else None, q_out=q if heads else None, workspace=ws)
    assert nv.nvfp4_workspace_status(ws) == 0
    there = (position >= 0) & (sequence >= 0)
    at = np.maximum(position, 0)
    want = qkv.copy()
    if rot:
        want[there] = K.turn(qkv[there], cos, sin, at[there], rot, neighbours)
    p, s = position[there], sequence[there]
    pages, slots = table[s, p // page], p % page
    for which, b in ((0, want[there, heads:heads + kv]), (1, qkv[there, heads + kv:])):
        codes, scales = K.quantise(W.bf16_bits_to_f32(b), host(cache.amax)[which])
        cq[which][pages, :, slots], csf[which][pages, :, slots] = codes, scales
    np.testing.assert_array_equal(host(cache.q), cq)
    np.testing.assert_array_equal(host(cache.sf), csf)
    if heads:
        assert got is q
        np.testing.assert_array_equal(host(d)[:, :heads], want[:, :heads])
    np.testing.assert_array_equal(host(d)[:, heads:], qkv[:, heads:])


@pytest.mark.parametrize("neighbours", [False, True])
def test_non_finite_numbers_stay_in_their_blocks(nv, neighbours):
    """What is not finite spoils the blocks of its own pair and no other byte, and no other pair of the queries."""
    rng = np.random.default_rng(8)
    dim, page, kv, heads, n = 64, 16, 2, 3, 6
    cos, sin = (dev(a) for a in K.tables(dim, 16))
    good = bits(rng, (n, heads + 2 * kv, dim))
    one, two = (18, 19) if neighbours else (18, 18 + dim // 2)  # a pair's places
    for bad in (0x7F80, 0xFF80, 0x7FC0):
        qkv = good.copy()
        for h in (1, heads + 1, heads + kv):                    # of token 2: a query, a key, a value
            qkv[2, h, 18] = bad
        held, turned = [], []
        for x in (good, qkv):
            c = nv.kv_cache(1, kv, page, dim, 4.0, 4.0)
            d = to_dev(x)
            turned.append(host(nv.kv_append(c, d[:, heads:heads + kv], d[:, heads + kv:], i32([[0]]), i32(np.arange(n)), i32(np.zeros(n)),
                                            cos=cos, sin=sin, interleaved=neighbours, q=d[:, :heads])))
            held.append((host(c.q)[:, 0].reshape(2, kv, page, dim // 16, 8), host(c.sf)[:, 0].copy()))
        same = np.ones((2, kv, page, dim // 16), bool)
        same[0, 1, 2, [one // 16, two // 16]] = same[1, 0, 2, 18 // 16] = False
        np.testing.assert_array_equal(held[1][0][same], held[0][0][same])
        np.testing.assert_array_equal(held[1][1][same], held[0][1][same])
        same = np.ones((n, heads, dim), bool)
        same[2, 1, [one, two]] = False
        np.testing.assert_array_equal(turned[1][same], turned[0][same])
        assert not np.isfinite(W.bf16_bits_to_f32(turned[1][~same])).any()


@pytest.mark.parametrize("rows,cols", [(30011, 112), (5, 16), (1001, 2416)])
def test_read_back(nv, rows, cols):
    """Row-major NVFP4 bytes of any kind in both output types; the largest with several steps a thread and a last one that
    is not full."""
    import torch
    rng = np.random.default_rng(rows)
    q = rng.integers(0, 256, (rows, cols // 2), dtype=np.uint8)
    sf = rng.integers(0, 256, (rows, cols // 16), dtype=np.uint8)
    sf[(sf & 127) == 127] = 5
    g = np.float32(0.0123)
    t = nv.NVFP4Tensor(dev(q), dev(sf), torch.tensor([g], device="cuda"), rows, cols, nv.NVFP4_SF_ROWMAJOR)
    want = K.decode(q, sf, 1.0).astype(np.float32) * g  # (the first product has six bits, the second is rounded once)
    np.testing.assert_array_equal(host(nv.dequantize(t)), want)
    np.testing.assert_array_equal(host(nv.dequantize(t, nv.NVFP4_OUT_BF16)), W.f32_to_bf16_bits(want))
