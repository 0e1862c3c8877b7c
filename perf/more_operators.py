"""The operators of a decoding step that keep their operands in NVFP4: what is measured of them, their plain forms,
and their values in 64 bits.

  append   keys and values of new tokens into a paged cache held in NVFP4 (4-bit codes, an E4M3 scale per 16
           elements along the head dimension, one FP32 scale each for keys and values), the keys (and the queries,
           which are returned) turned by their position on the way.  What the cache then holds is returned whole.
  attend   attention of a few query tokens per sequence over such a cache: causal among the query tokens,
           optionally over a window of positions, query heads in groups that share a key and value head
  experts  the experts of a mixture-of-experts layer for a few tokens: each routed row through its expert's gate
           and up matrices, silu(gate) * up (or relu(up)^2 without a gate), the down matrix, and the weighted sum
           per token on top of the residual; all matrices in NVFP4, the tokens in bf16
"""
import math

import torch

if not torch.cuda.is_available():  # the file can be read, listed and drawn from on a machine without a GPU
    DEVICE = "cpu"
else:
    DEVICE = "cuda"

own = False


def listed():
    return [
        # the next token of one sequence, 4096 = 32 heads of 128: latency
        dict(name="append_one_token", op="append", sequences=1, new=1, past=777, heads=32, kv_heads=8, dim=128, rot=128,
             interleaved=False, page=64),
        # the next tokens of 64 sequences, 5120 = 40 heads of 128
        dict(name="append_64_tokens", op="append", sequences=64, new=1, past=500, heads=40, kv_heads=8, dim=128, rot=128,
             interleaved=False, page=64),
        # a prompt chunk's 1001 tokens a sequence, small heads of which half is turned, in neighbouring pairs
        dict(name="append_chunks", op="append", sequences=3, new=1001, past=37, heads=16, kv_heads=4, dim=64, rot=32,
             interleaved=True, page=16),
        # prompts of 16384 tokens in all
        dict(name="append_prompts", op="append", sequences=8, new=2048, past=0, heads=32, kv_heads=8, dim=128, rot=128,
             interleaved=False, page=64),
        # the next token of one sequence over a short cache: latency
        dict(name="attend_one_short", op="attend", sequences=1, new=1, longest=1000, heads=32, kv_heads=8, dim=128,
             window=0, page=64, lse=False),
        # 64 sequences of ragged lengths, five query heads to a key head
        dict(name="attend_64_ragged", op="attend", sequences=64, new=1, longest=8192, heads=40, kv_heads=8, dim=128,
             window=0, page=64, lse=False),
        # four long contexts
        dict(name="attend_4_long", op="attend", sequences=4, new=1, longest=131072, heads=32, kv_heads=8, dim=128,
             window=0, page=128, lse=False),
        # five drafted tokens to check at once, over a window, with the sums' logarithms
        dict(name="attend_drafts", op="attend", sequences=16, new=5, longest=6001, heads=16, kv_heads=4, dim=64,
             window=4096, page=16, lse=True),
        # wide heads
        dict(name="attend_wide_heads", op="attend", sequences=8, new=2, longest=16384, heads=16, kv_heads=4, dim=256,
             window=0, page=32, lse=False),
        # one token through its four of 64 experts: latency
        dict(name="experts_one_token", op="experts", tokens=1, hidden=4096, ffn=1536, experts=64, top_k=4, gate=True),
        # the next tokens of 8 sequences
        dict(name="experts_8_tokens", op="experts", tokens=8, hidden=4096, ffn=1536, experts=64, top_k=4, gate=True),
        # the next tokens of 32 sequences, experts without a gate
        dict(name="experts_32_tokens", op="experts", tokens=32, hidden=4096, ffn=1536, experts=64, top_k=4, gate=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "experts"])
    if op == "append":
        dim = rng.choice([64, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8])
        sequences = _log_int(rng, 1, 128)
        tokens = _log_int(rng, 1, 16384 * 1024 // (kv_heads * dim * sequences))
        return dict(op=op, sequences=sequences, new=max(1, min(tokens, 4096)), past=rng.randint(0, 600),
                    heads=kv_heads * rng.randint(1, 4), kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([r for r in (0, 32, 64, 128, 256) if r <= dim]), interleaved=rng.random() < 0.4,
                    page=rng.choice([16, 32, 64, 128]))
    if op == "attend":
        dim = rng.choice([64, 128, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8])
        sequences = _log_int(rng, 1, 128)
        longest = _log_int(rng, 1, min(131072, 131072 * 4 * 1024 // (8 * sequences * kv_heads * dim)))
        return dict(op=op, sequences=sequences, new=rng.choice([1, 1, 1, 2, 3, 4, 6]), longest=longest,
                    heads=kv_heads * rng.randint(1, 8), kv_heads=kv_heads, dim=dim,
                    window=rng.choice([0, 0, _log_int(rng, 16, 8192)]), page=rng.choice([16, 32, 64, 128]),
                    lse=rng.random() < 0.4)
    return dict(op=op, tokens=_log_int(rng, 1, 32), hidden=128 * _log_int(rng, 4, 32), ffn=128 * _log_int(rng, 2, 12),
                experts=rng.choice([8, 16, 60, 64]), top_k=rng.randint(1, 4), gate=rng.random() < 0.6)


# ------------------------------------------------------------------------------------------ inputs
def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device=DEVICE) * std).to(dtype)


def _codes(y):
    """E2M1 codes nearest to y, ties to the even code: the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6."""
    a = y.abs()
    c = (a > 0.25).to(torch.uint8)
    c += a >= 0.75
    c += a > 1.25
    c += a >= 1.75
    c += a > 2.5
    c += a >= 3.5
    c += a > 5.0
    return c + torch.signbit(y).to(torch.uint8) * 8


def _to_nvfp4(x, amax):
    """Codes [..., d/2] and scale bytes [..., d/16] of x [..., d] for the largest magnitude amax [1] in 32 bits:
    S = 2688 / amax, the scale byte E4M3(blockmax / 6 * S), the codes those of x * (S / scale)."""
    blocks = x.float().unflatten(-1, (-1, 16))
    up = torch.full_like(amax, 2688.0) / amax   # (a tensor over a number would be multiplied by its reciprocal)
    scale = (blocks.abs().amax(-1) / torch.full_like(amax, 6.0) * up).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = scale.float()
    by = torch.where(d > 0, up / d, 0.0)
    c = _codes(blocks * by.unsqueeze(-1)).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), scale.view(torch.uint8)


def _values():
    v = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEVICE)
    return torch.cat([v, -v])


def _from_nvfp4(q, sf):
    """code * block scale in 32 bits: q [..., d/2] bytes, sf [..., d/16] E4M3 bytes."""
    both = torch.stack([q & 15, q >> 4], dim=-1)
    v = _values().index_select(0, both.reshape(-1).int()).view(*q.shape[:-1], -1, 16)
    return (v * sf.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)


def _pages(g, sequences, each, page):
    """A page table [sequences, pages of the longest], the pages in random order; each: tokens that a sequence holds."""
    most = -(-each // page)
    return torch.randperm(sequences * most, generator=g, device=DEVICE).int().view(sequences, most), sequences * most


def _nvfp4_weights(g, matrices, n, k):
    """`matrices` weights [n, k] ~ N(0, 0.02) in NVFP4: codes [matrices, n, k/2], tiled scale bytes
    [matrices, n*k/16], FP32 scales [matrices]."""
    grid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEVICE)
    codes = torch.empty((matrices, n, k // 2), dtype=torch.uint8, device=DEVICE)
    scales = torch.empty((matrices, n * k // 16), dtype=torch.uint8, device=DEVICE)
    glob = torch.empty(matrices, dtype=torch.float32, device=DEVICE)
    for e in range(matrices):
        w = torch.randn((n, k // 16, 16), generator=g, device=DEVICE).mul_(0.02)
        block = w.abs().amax(2)
        glob[e] = block.amax() / 2688.0
        byte = (block / (6.0 * glob[e])).to(torch.float8_e4m3fn)
        w /= (byte.float() * glob[e]).clamp_min(1e-30).unsqueeze(2)
        c = torch.bucketize(w.abs(), grid, out_int32=True)
        c += (w < 0).int() * 8
        c = c.to(torch.uint8).reshape(n, k // 2, 2)
        codes[e] = c[..., 0] | (c[..., 1] << 4)
        scales[e] = byte.view(torch.uint8).view(n // 128, 4, 32, k // 64, 4).permute(0, 3, 2, 1, 4).reshape(-1)
    return codes, scales, glob


def _routing(g, tokens, experts, top_k):
    """top_k distinct experts for each token, the experts' popularity falling as rank^-1.1 (Gumbel top-k), and the
    routed rows in expert order: offsets, the rows' tokens, the slots' rows, the slots' weights."""
    rank = torch.randperm(experts, generator=g, device=DEVICE).float() + 1.0
    u = torch.rand((tokens, experts), generator=g, device=DEVICE).clamp_(1e-6, 1 - 1e-6)
    chosen = (-1.1 * rank.log() - (-u.log()).log()).topk(top_k, dim=1).indices
    flat = chosen.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    slot_row = torch.empty_like(order)
    slot_row[order] = torch.arange(order.numel(), device=flat.device)
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device=flat.device)
    offsets[1:] = torch.bincount(flat, minlength=experts).cumsum(0)
    return dict(expert=chosen.int(), offsets=offsets.int(), row_index=(order // top_k).int(),
                slot_row=slot_row.view(tokens, top_k).int(),
                weight=torch.softmax(torch.randn((tokens, top_k), generator=g, device=DEVICE), 1))


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    c, s = case, {"case": case}
    if c["op"] == "append":
        n, new, heads, kv, dim, page = c["sequences"], c["new"], c["heads"], c["kv_heads"], c["dim"], c["page"]
        # the projection's output, of which q, k and v are pieces
        qkv = _normal(g, (n * new, heads + 2 * kv, dim))
        qkv[:, heads:heads + kv, ::16] *= 6.0   # keys have large channels
        s["q"], s["k"], s["v"] = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
        # sequences that hold up to `past` tokens go on; the first of them is as long as that
        past = torch.randint(0, c["past"] + 1, (n,), generator=g, device=DEVICE)
        past[0] = c["past"]
        s["position"] = (past.unsqueeze(1) + torch.arange(new, device=DEVICE)).reshape(-1).int()
        s["sequence"] = torch.arange(n, device=DEVICE).repeat_interleave(new).int()
        s["table"], pages = _pages(g, n, c["past"] + new, page)
        s["codes"] = torch.randint(0, 256, (2, pages, kv, page, dim // 2), generator=g, device=DEVICE, dtype=torch.uint8)
        s["scales"] = torch.randint(1, 0x70, (2, pages, kv, page, dim // 16), generator=g, device=DEVICE, dtype=torch.uint8)
        s["amax"] = torch.tensor([40.0, 5.5], device=DEVICE)
        s["g"] = s["amax"] / torch.full_like(s["amax"], 2688.0)
        s["cos"] = s["sin"] = None
        if c["rot"]:
            f = 10000.0 ** (-torch.arange(0, c["rot"], 2, device=DEVICE, dtype=torch.float64) / c["rot"])
            angle = torch.arange(c["past"] + new, device=DEVICE, dtype=torch.float64).unsqueeze(1) * f
            s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    elif c["op"] == "attend":
        n, new, heads, kv, dim, page = c["sequences"], c["new"], c["heads"], c["kv_heads"], c["dim"], c["page"]
        s["q"] = _normal(g, (n, new, heads, dim), 1.5)
        # lengths from a quarter of the longest on; the first is the longest
        low = max(1, c["longest"] // 4)
        s["lengths"] = torch.randint(low, c["longest"] + 1, (n,), generator=g, device=DEVICE).int()
        s["lengths"][0] = c["longest"]
        s["table"], pages = _pages(g, n, c["longest"], page)
        s["amax"] = torch.tensor([32.0, 6.0], device=DEVICE)
        s["g"] = s["amax"] / torch.full_like(s["amax"], 2688.0)
        s["codes"] = torch.empty((2, pages, kv, page, dim // 2), dtype=torch.uint8, device=DEVICE)
        s["scales"] = torch.empty((2, pages, kv, page, dim // 16), dtype=torch.uint8, device=DEVICE)
        step = max(1, (1 << 26) // (kv * page * dim))
        for i in range(0, pages, step):
            m = min(step, pages - i)
            for which in (0, 1):
                x = _normal(g, (m, kv, page, dim))
                if which == 0:
                    x[..., ::16] *= 4.0
                s["codes"][which, i:i + m], s["scales"][which, i:i + m] = _to_nvfp4(x, s["amax"][which:which + 1])
    else:
        t, h, f, e = c["tokens"], c["hidden"], c["ffn"], c["experts"]
        s["x"] = _normal(g, (t, h))
        s["base"] = _normal(g, (t, h))
        s |= _routing(g, t, e, c["top_k"])
        s["gate"] = _nvfp4_weights(g, e, f, h) if c["gate"] else None
        s["up"] = _nvfp4_weights(g, e, f, h)
        s["down"] = _nvfp4_weights(g, e, h, f)
    return s


# ------------------------------------------------------------------------------------------ plain forms
def _to_bf16(x):
    """64 bits to bf16 in one rounding: 32 bits between two bf16 values are moved off the middle first."""
    f = x.float()
    bits = f.view(torch.int32)
    lost = x.abs() - f.double().abs()
    step = torch.where(((bits & 0xFFFF) == 0x8000) & torch.isfinite(x), torch.sign(lost), 0.0).int()
    return (bits + step).view(torch.float32).to(torch.bfloat16)


def _turned(s, x):
    """x [tokens, heads, dim] turned by its position, in 64 bits up to the one rounding to bf16 (the keys' rounding
    to 4 bits looks at which side of a border a value lies on)."""
    c = s["case"]
    if not c["rot"]:
        return x
    at = s["position"].long()
    cos, sin = s["cos"][at].double().unsqueeze(1), s["sin"][at].double().unsqueeze(1)
    y = x.double()
    r = y[..., :c["rot"]]
    if c["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = r.chunk(2, dim=-1)
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return _to_bf16(torch.cat([turned, y[..., c["rot"]:]], dim=-1))


def _plain_append(s):
    c = s["case"]
    at = s["position"].long()
    page, slot = s["table"][s["sequence"].long(), at // c["page"]].long(), at % c["page"]
    out = {"q": _turned(s, s["q"])} if c["rot"] else {}
    for which, (name, x) in enumerate((("k", _turned(s, s["k"])), ("v", s["v"]))):
        codes, scales = _to_nvfp4(x, s["amax"][which:which + 1])
        s["codes"][which][page, :, slot] = codes
        s["scales"][which][page, :, slot] = scales
        held = _from_nvfp4(s["codes"][which], s["scales"][which]) * s["g"][which]
        out[name] = held.to(torch.bfloat16).view(-1, c["dim"])
    return out


def _plain_attend(s):
    c = s["case"]
    n, new, kv, dim = c["sequences"], c["new"], c["kv_heads"], c["dim"]
    table = s["table"].long()
    k, v = (_from_nvfp4(s["codes"][i][table], s["scales"][i][table]).transpose(1, 2).reshape(n, kv, -1, dim)
            for i in (0, 1))
    group = c["heads"] // kv
    q = s["q"].float().view(n, new, kv, group, dim).permute(0, 2, 1, 3, 4).reshape(n, kv, new * group, dim)
    score = q @ k.transpose(2, 3) * (s["g"][0] / math.sqrt(dim))
    score = score.view(n, kv, new, group, -1)
    place = torch.arange(score.shape[-1], device=DEVICE)
    last = s["lengths"].long().unsqueeze(1) - new + torch.arange(new, device=DEVICE)    # [n, new]
    seen = place <= last.unsqueeze(2)
    if c["window"]:
        seen = seen & (place > last.unsqueeze(2) - c["window"])
    score = torch.where(seen[:, None, :, None, :], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - torch.where(top > -math.inf, top, 0.0)).exp()
    total = p.sum(-1, keepdim=True)
    o = p.view(n, kv, new * group, -1) @ v
    o = o.view(n, kv, new, group, dim) / torch.where(total > 0, total, 1.0) * s["g"][1]
    out = {"out": o.permute(0, 2, 1, 3, 4).reshape(n, new, c["heads"], dim).to(torch.bfloat16)}
    if c["lse"]:
        out["lse"] = (total.log() + top).squeeze(-1).permute(0, 2, 1, 3).reshape(n, new, c["heads"])
    return out


def _plain_matrix(w, which, n, k):
    """The matrices `which` [rows] in 32 bits, without their FP32 scales: [rows, n, k]."""
    q, sf, _ = w
    m = which.shape[0]
    scale = sf[which].view(m, n // 128, k // 64, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(m, n, k // 16)
    return _from_nvfp4(q[which], scale)


def _plain_experts(s):
    c = s["case"]
    h, f, t = c["hidden"], c["ffn"], c["tokens"]
    row = torch.arange(t * c["top_k"], device=DEVICE)
    which = torch.searchsorted(s["offsets"][1:].contiguous().long(), row, right=True)
    x = s["x"].float()[s["row_index"].long()].unsqueeze(2)
    u = torch.bmm(_plain_matrix(s["up"], which, f, h), x) * s["up"][2][which].view(-1, 1, 1)
    if c["gate"]:
        z = torch.bmm(_plain_matrix(s["gate"], which, f, h), x) * s["gate"][2][which].view(-1, 1, 1)
        a = z / (1.0 + (-z).exp()) * u
    else:
        a = u.clamp_min(0.0) * u.clamp_min(0.0)
    y = torch.bmm(_plain_matrix(s["down"], which, h, f), a).squeeze(2) * s["down"][2][which].unsqueeze(1)
    acc = (y[s["slot_row"].long()] * s["weight"].unsqueeze(2)).sum(1) + s["base"].float()
    return {"out": acc.to(torch.bfloat16)}


# ------------------------------------------------------------------------------------------ the framework's
def _own(s):
    import nvfp4_bit_precision_b200 as nv
    from nvfp4_bit_precision_b200 import moe
    c = s["case"]
    if c["op"] == "experts":
        routing = nv.Routing(s["expert"], s["weight"], s["offsets"], s["row_index"], s["slot_row"], None)
        gate = moe.ExpertWeights(*s["gate"], c["ffn"]) if c["gate"] else None
        return {"out": moe.expert_mlp(s["x"], routing, moe.ExpertWeights(*s["up"], c["ffn"]),
                                      moe.ExpertWeights(*s["down"], c["hidden"]), gate=gate, base=s["base"])}
    cache = nv.KVCache(s["codes"], s["scales"], s["amax"], s["g"])
    if c["op"] == "append":
        q = nv.kv_append(cache, s["k"], s["v"], s["table"], s["position"], s["sequence"], cos=s["cos"], sin=s["sin"],
                         interleaved=c["interleaved"], q=s["q"] if c["rot"] else None)
        out = {"k": nv.dequantize(cache.keys(), nv.NVFP4_OUT_BF16),
               "v": nv.dequantize(cache.values(), nv.NVFP4_OUT_BF16)}
        return {"q": q, **out} if c["rot"] else out
    got = nv.kv_attention(s["q"], cache, s["table"], s["lengths"], window=c["window"], lse=c["lse"])
    return {"out": got[0], "lse": got[1]} if c["lse"] else {"out": got}


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "attend": _plain_attend, "experts": _plain_experts}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------ cost
def work(case):
    c = case
    if c["op"] == "append":
        t, d = c["sequences"] * c["new"], c["dim"]
        pool = 2 * c["sequences"] * -(-(c["past"] + c["new"]) // c["page"]) * c["page"] * c["kv_heads"] * d
        b = t * d * 2 * ((2 * c["heads"] if c["rot"] else 0) + 2 * c["kv_heads"])   # q in and out, k, v in
        b += t * c["kv_heads"] * d * 2 * 9 // 16 + 8 * t + 8 * (c["past"] + c["new"]) * (c["rot"] // 2)
        b += pool * 9 // 16 + pool * 2                               # what the cache holds, read back in bf16
        return {"bytes": b, "flops": 3 * t * c["rot"] * (c["heads"] + c["kv_heads"])}
    if c["op"] == "attend":
        mean = (max(1, c["longest"] // 4) + c["longest"]) / 2
        held = c["longest"] + (c["sequences"] - 1) * mean
        if c["window"]:
            held = min(held, c["sequences"] * (c["window"] + c["new"] - 1.0))
        rows = c["sequences"] * c["new"] * c["heads"]
        b = held * c["kv_heads"] * c["dim"] * 2 * 9 / 16 + rows * c["dim"] * 4 + (4 * rows if c["lse"] else 0)
        return {"bytes": int(b), "flops": int(4 * held * c["new"] * c["heads"] * c["dim"])}
    t, h, f, k = c["tokens"], c["hidden"], c["ffn"], c["top_k"]
    # experts that some token is expected to choose
    p = [r ** -1.1 for r in range(1, c["experts"] + 1)]
    used = sum(1.0 - (1.0 - min(1.0, k * v / sum(p))) ** t for v in p)
    matrices = 3 if c["gate"] else 2
    return {"bytes": int(used * matrices * h * f * 9 / 16 + 6 * t * h + 12 * t * k),
            "flops": 2 * t * k * matrices * h * f}


# ------------------------------------------------------------------------------------------ 64 bits
def _decoded(q, sf):
    """code * scale of NVFP4 bytes in 64 bits, from the fields of both formats."""
    nib = torch.empty((*q.shape[:-1], 2 * q.shape[-1]), dtype=torch.uint8, device=q.device)
    nib[..., 0::2] = q % 16
    nib[..., 1::2] = q // 16
    e, m = nib % 8 // 2, nib % 2
    mag = torch.where(e == 0, m * 0.5, (1.0 + 0.5 * m.double()) * torch.exp2(e.double() - 1.0))
    mag = torch.where(nib >= 8, -mag, mag)
    ex, fr = (sf // 8).double(), (sf % 8).double()
    d = torch.where(ex == 0, fr * 2.0 ** -9, (1.0 + fr / 8.0) * torch.exp2(ex - 7.0))
    return mag * d.repeat_interleave(16, -1)


def _round32(x):
    return x.float().double()


def _nearest_held(x, amax):
    """What the format keeps of x [..., d] (64 bits holding bf16 values), the steps that it defines in 32 bits rounded
    to those: scale = E4M3(amax_block / 6 * S), value = E2M1(x * (S / scale)) * scale."""
    b = x.unflatten(-1, (-1, 16))
    up = _round32(torch.full_like(amax, 2688.0, dtype=torch.float64) / amax.double())
    s = _round32(_round32(b.abs().amax(-1) / torch.full_like(b[..., 0], 6.0)) * up)
    _, e = torch.frexp(s)
    step = torch.ldexp(torch.ones_like(s), (e - 1).clamp_min(-6) - 3)
    d = (torch.round(s / step) * step).clamp(max=448.0)
    y = _round32(b * torch.where(d > 0, _round32(up / d.clamp_min(2.0 ** -9)), torch.zeros_like(d)).unsqueeze(-1))
    a = y.abs()
    grid = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0)).double()
    v = torch.copysign((torch.round(a / grid) * grid).clamp(max=6.0), y)
    return (v * d.unsqueeze(-1)).flatten(-2)


def _exact_turn(c, s, x):
    x = x.double().clone()
    half = c["rot"] // 2
    if half:
        i = torch.arange(half, device=x.device)
        one, two = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
        z = torch.complex(x[..., one], x[..., two])
        at = s["position"].long()
        z = z * torch.complex(s["cos"].double(), s["sin"].double())[at][:, None]
        x[..., one], x[..., two] = z.real, z.imag
    return x


def _exact_append(c, s):
    out = {"q": _exact_turn(c, s, s["q"])} if c["rot"] else {}
    at = s["position"].long()
    row = s["table"][s["sequence"].long(), at // c["page"]].long()[:, None] * c["kv_heads"]
    row = (row + torch.arange(c["kv_heads"], device=row.device)) * c["page"] + (at % c["page"])[:, None]
    for which, name in enumerate(("k", "v")):
        held = _decoded(s["codes"][which], s["scales"][which]).view(-1, c["dim"])
        x = s["v"].double()
        if which == 0:  # the keys in bf16: eight bits of the fraction that frexp gives
            m, e = torch.frexp(_exact_turn(c, s, s["k"]))
            x = torch.ldexp(torch.round(m * 256.0), e - 8)
        held[row.flatten()] = _nearest_held(x, s["amax"][which]).flatten(0, 1)
        out[name] = held * s["g"][which].double()
    return out


def _exact_attend(c, s):
    n, new, heads, kv, dim = c["sequences"], c["new"], c["heads"], c["kv_heads"], c["dim"]
    out = torch.zeros((n, new, heads, dim), dtype=torch.float64, device=DEVICE)
    lse = torch.full((n, new, heads), -math.inf, dtype=torch.float64, device=DEVICE)
    for b, length in enumerate(s["lengths"].tolist()):
        pages = s["table"][b, :-(-length // c["page"])].long()
        for h in range(kv):
            k = _decoded(s["codes"][0][pages, h], s["scales"][0][pages, h]).flatten(0, 1)[:length] * s["g"][0].double()
            v = _decoded(s["codes"][1][pages, h], s["scales"][1][pages, h]).flatten(0, 1)[:length] * s["g"][1].double()
            mine = slice(h * (heads // kv), (h + 1) * (heads // kv))
            for i in range(new):
                end = length - new + 1 + i
                begin = max(0, end - c["window"]) if c["window"] else 0
                if end <= begin:
                    continue
                z = torch.mm(s["q"][b, i, mine].double(), k[begin:end].t()) * dim ** -0.5
                lse[b, i, mine] = torch.logsumexp(z, 1)
                out[b, i, mine] = torch.mm(torch.exp(z - lse[b, i, mine, None]), v[begin:end])
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}


def _exact_matrix(w, e, n, k):
    """Matrix e in 64 bits, by the place of each scale byte in the tiled order."""
    r = torch.arange(n, device=w[0].device)[:, None]
    b = torch.arange(k // 16, device=w[0].device)[None, :]
    sf = w[1][e][(r // 128 * (k // 64) + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4]
    return _decoded(w[0][e], sf) * w[2][e].double()


def _exact_experts(c, s):
    h, f = c["hidden"], c["ffn"]
    out = s["base"].double()
    for e in sorted(set(s["expert"].flatten().tolist())):
        token, slot = torch.nonzero(s["expert"] == e, as_tuple=True)
        x = s["x"][token].double()
        u = torch.mm(x, _exact_matrix(s["up"], e, f, h).t())
        if c["gate"]:
            z = torch.mm(x, _exact_matrix(s["gate"], e, f, h).t())
            a = u * z * torch.sigmoid(z)
        else:
            a = torch.square(torch.relu(u))
        y = torch.mm(a, _exact_matrix(s["down"], e, h, f).t())
        out[token] += y * s["weight"][token, slot].double()[:, None]
    return {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "experts": _exact_experts}[case["op"]](case, s)
