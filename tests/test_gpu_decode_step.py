"""A decoding step of one block as a model runs it: norm, the query, key and value products, append with rotation,
attention over the 4-bit cache, the output product, norm with the residual, routing, the experts.  Each stage is
checked from the stage before it as the GPU computed it; the pieces' own tolerances are in their own tests."""
import numpy as np
import pytest

import kv_ref as K
import moe_ref as R
import test_gpu_expert_mlp as E
import workloads as W
from gpu_util import cuda_available, host, to_dev

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]

HIDDEN, HEADS, KV, DIM, PAGE, FFN, EXPERTS, TOP = 512, 8, 2, 64, 16, 256, 8, 2


@pytest.fixture(scope="module")
def nv():
    import nvfp4_bit_precision_b200 as nv
    return nv


def bits(rng, shape, std=1.0):
    return W.f32_to_bf16_bits(rng.standard_normal(shape).astype(np.float32) * np.float32(std))


def val(t):
    return W.bf16_bits_to_f32(host(t)).astype(np.float64)


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Block:
    def __init__(self, nv, rng):
        import torch
        self.nv = nv
        q = lambda n, k: nv.quantize(to_dev(bits(rng, (n, k), 1 / np.sqrt(k))), sf_layout=nv.NVFP4_SF_MMA)["row"]  # noqa: E731
        self.qkv, self.out = q((HEADS + 2 * KV) * DIM, HIDDEN), q(HIDDEN, HEADS * DIM)
        self.norm1, self.norm2 = to_dev(bits(rng, HIDDEN)), to_dev(bits(rng, HIDDEN))
        self.router = torch.from_numpy(rng.standard_normal((EXPERTS, HIDDEN)).astype(np.float32)).cuda()
        self.up, self.up_w = E.matrices(rng, EXPERTS, FFN, HIDDEN)
        self.gate, self.gate_w = E.matrices(rng, EXPERTS, FFN, HIDDEN)
        self.down, self.down_w = E.matrices(rng, EXPERTS, HIDDEN, FFN)
        self.cos_np, self.sin_np = K.tables(DIM, 128)
        self.cos, self.sin = dev(self.cos_np), dev(self.sin_np)

    def step(self, x, cache, table, lengths):
        """x [sequences, hidden]: the next token of each; lengths with it."""
        import torch
        from nvfp4_bit_precision_b200 import moe
        nv, s = self.nv, {}
        n = x.shape[0]
        s["y"] = moe.rms_norm(x, self.norm1)
        s["qkv"] = nv.gemv(s["y"], self.qkv).view(n, HEADS + 2 * KV, DIM)
        q, k, v = s["qkv"].split((HEADS, KV, KV), 1)
        s["q"] = nv.kv_append(cache, k, v, table, lengths - 1, cos=self.cos, sin=self.sin, q=q)
        s["a"] = nv.kv_attention(s["q"][:, None], cache, table, lengths)
        s["o"] = nv.gemv(s["a"].view(n, HEADS * DIM), self.out)
        s["z"], s["h"] = moe.rms_norm(s["o"], self.norm2, x)
        s["r"] = moe.moe_route(s["z"].float() @ self.router.t(), TOP)
        s["out"] = moe.expert_mlp(s["z"], s["r"], self.up, self.down, self.gate, base=s["h"])
        return s


def test_steps(nv):
    """Forty tokens of five sequences, two of which begin later; every tenth step is checked stage by stage, and at
    the end the cache holds what one append of all tokens leaves."""
    import torch
    rng = np.random.default_rng(0)
    b = Block(nv, rng)
    n, pages = 5, 20
    cache, whole = (nv.kv_cache(pages, KV, PAGE, DIM, 6.0, 6.0) for _ in range(2))
    table = dev(rng.permutation(pages).reshape(n, 4).astype(np.int32))
    start = np.array([0, 0, 7, 0, 33])
    keys, values, places, owners = [], [], [], []
    for t in range(40):
        lengths = np.maximum(t + 1 - start, 0).astype(np.int32)
        x = to_dev(bits(rng, (n, HIDDEN)))
        s = b.step(x, cache, table, dev(lengths))
        live = lengths > 0
        for i in np.nonzero(live)[0]:
            places.append(lengths[i] - 1)
            owners.append(i)
            keys.append(s["qkv"][i, HEADS:HEADS + KV])
            values.append(s["qkv"][i, HEADS + KV:])
        if t % 10 != 9:
            continue
        q_ref = K.turn(host(s["qkv"])[:, :HEADS], b.cos_np, b.sin_np, np.maximum(lengths - 1, 0), DIM, False)
        np.testing.assert_array_equal(host(s["q"])[live], q_ref[live])
        g, cq, csf, tab = host(cache.g), host(cache.q), host(cache.sf), host(table)
        for i in range(n):
            m = -(-int(lengths[i]) // PAGE)
            k, v = (K.decode(cq[w][tab[i, :m]], csf[w][tab[i, :m]], g[w]).transpose(1, 0, 2, 3).reshape(KV, -1, DIM)[:, :lengths[i]]
                    for w in (0, 1))
            ref, _, ob, _ = K.attend(val(s["q"])[i:i + 1], k, v, int(lengths[i]), np.float64(np.float32(DIM ** -0.5)))
            assert np.all(np.abs(val(s["a"])[i] - ref) <= ob + 2.0 ** -8 * np.abs(ref))
        ids, wts = R.route(host(s["z"].float() @ b.router.t()).astype(np.float64), TOP)
        np.testing.assert_array_equal(host(s["r"].expert), ids)
        E.compare(s["out"], *E.reference(val(s["z"]), ids, host(s["r"].weight), b.up_w, b.down_w, b.gate_w, val(s["h"])))
    as_i32 = lambda a: dev(np.array(a, dtype=np.int32))  # noqa: E731
    nv.kv_append(whole, torch.stack(keys), torch.stack(values), table, as_i32(places), as_i32(owners), cos=b.cos, sin=b.sin)
    assert torch.equal(cache.q, whole.q) and torch.equal(cache.sf, whole.sf)


def test_captured_step(nv):
    """The step captured once, with the lengths counted up inside, replayed token after token, against eager steps."""
    import torch
    rng = np.random.default_rng(1)
    b = Block(nv, rng)
    n, pages = 3, 12
    caches = [nv.kv_cache(pages, KV, PAGE, DIM, 6.0, 6.0) for _ in range(2)]
    table = dev(rng.permutation(pages).reshape(n, 4).astype(np.int32))
    lengths = [dev(np.array([0, 15, 30], dtype=np.int32)) for _ in range(2)]
    x = torch.empty((n, HIDDEN), dtype=torch.bfloat16, device="cuda")
    x.copy_(to_dev(bits(rng, (n, HIDDEN))))
    b.step(x, caches[0], table, lengths[0] + 1)              # (libraries that initialise at their first call)
    caches[0].q.zero_()
    caches[0].sf.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lengths[0] += 1
        captured = b.step(x, caches[0], table, lengths[0])
    for _ in range(20):
        x.copy_(to_dev(bits(rng, (n, HIDDEN))))
        graph.replay()
        lengths[1] += 1
        eager = b.step(x, caches[1], table, lengths[1])
        for name in ("q", "a", "out"):
            assert torch.equal(captured[name], eager[name]), name
    assert torch.equal(caches[0].q, caches[1].q) and torch.equal(caches[0].sf, caches[1].sf)


def test_drafts_are_single_steps(nv):
    """Five tokens attended at once see what five single steps see."""
    import torch
    rng = np.random.default_rng(2)
    cache = nv.kv_cache(8, KV, PAGE, DIM, 4.0, 4.0)
    table = dev(rng.permutation(8).reshape(1, 8).astype(np.int32))
    total, new = 100, 5
    kv = to_dev(bits(rng, (total, 2 * KV, DIM)))
    at = torch.arange(total, dtype=torch.int32, device="cuda")
    nv.kv_append(cache, kv[:, :KV], kv[:, KV:], table, at, torch.zeros_like(at))
    q = to_dev(bits(rng, (1, new, HEADS, DIM)))
    for window in (0, 20):
        both, lse = nv.kv_attention(q, cache, table, at[total - 1:] + 1, window=window, lse=True)
        for i in range(new):
            one, l1 = nv.kv_attention(q[:, i:i + 1], cache, table, at[total - new + i:total - new + i + 1] + 1, window=window, lse=True)
            # (the maximum that exponentials are taken from may be another: their roundings, 2^-11 each, twice)
            np.testing.assert_allclose(val(both)[:, i], val(one)[:, 0], rtol=2.0 ** -7, atol=2.0 ** -9 * float(np.abs(val(kv)).max()))
            np.testing.assert_allclose(host(lse)[:, i], host(l1)[:, 0], rtol=0, atol=2.0 ** -14)
