"""The operators around the experts of a mixture-of-experts block and around the linear layers: what is
measured of them, their plain forms, and their values in 64 bits.

  norm     h = bf16(x + residual); y = h * rsqrt(mean(h^2) + eps) * w, in bf16 or as MXFP8 codes with one
           E8M0 scale per 32 elements (the operand of the MXFP8 GEMM); with "train" also the gradients of
           x (and residual) and w from those of y and h
  route    expert scores (softmax or sigmoid of the logits), a bias that only steers the choice, expert
           groups, top-k, renormalised weights, and the order of the routed rows that the grouped
           products read; with "train" also the logits' gradient
  combine  out[t] = base[t] + sum_j weight[t, j] * rows[slot_row[t, j]]; with "train" also the gradients
           of the rows and of the weights
  gemv     a few bf16 tokens times an NVFP4 matrix (4-bit codes, an E4M3 scale per 16 elements in the
           tensor cores' tiled order, one FP32 scale), dense or one matrix per expert
"""
import math

import torch

if not torch.cuda.is_available():  # the file can be read, listed and drawn from on a machine without a GPU
    DEVICE = "cpu"
else:
    DEVICE = "cuda"

own = False

EPS = 1e-6


def listed():
    return [
        # one token of a decoding step through the dense layer's norm: latency
        dict(name="norm_one_token", op="norm", rows=1, cols=5120, residual=True, out="mx", tiled=False, train=False),
        # the dense layer's 16384 tokens, the sum with the residual and the MXFP8 operand in one pass
        dict(name="norm_mx_prefill", op="norm", rows=16384, cols=5120, residual=True, out="mx", tiled=True, train=False),
        # a training step's norm, forward and backward, a ragged token count
        dict(name="norm_train", op="norm", rows=8191, cols=4096, residual=True, out="bf16", tiled=False, train=True),
        # eight sequences' next tokens over 64 experts
        dict(name="route_decode", op="route", tokens=8, experts=64, top_k=4, score="softmax", bias=False, groups=1,
             topk_groups=1, renorm=True, scale=1.0, bf16=False, train=False),
        # the training step's 16384 tokens over 64 experts, with the logits' gradient
        dict(name="route_train", op="route", tokens=16384, experts=64, top_k=4, score="softmax", bias=False, groups=1,
             topk_groups=1, renorm=True, scale=1.0, bf16=False, train=True),
        # a wide router: sigmoid scores, a balancing bias, four of eight groups, bf16 logits, a ragged count
        dict(name="route_groups", op="route", tokens=4099, experts=256, top_k=8, score="sigmoid", bias=True, groups=8,
             topk_groups=4, renorm=True, scale=2.5, bf16=True, train=False),
        # a decoding step's expert outputs back to their tokens, added to the residual stream
        dict(name="combine_decode", op="combine", tokens=8, cols=4096, top_k=4, base=True, f32=True, train=False),
        # the training step's 65536 routed rows, forward and backward
        dict(name="combine_train", op="combine", tokens=16384, cols=4096, top_k=4, base=False, f32=False, train=True),
        # one token through the dense layer's weight
        dict(name="gemv_one_token", op="gemv", tokens=1, n=20480, k=5120, experts=0, top_k=0, gather=False, f32=False),
        # thirteen sequences' tokens (a ragged few) through a square projection
        dict(name="gemv_13_tokens", op="gemv", tokens=13, n=4096, k=4096, experts=0, top_k=0, gather=False, f32=False),
        # eight tokens through their four experts' up matrices: the rows gathered from the tokens
        dict(name="experts_up_8", op="gemv", tokens=8, n=1536, k=4096, experts=64, top_k=4, gather=True, f32=False),
        # thirty-two tokens through the experts' down matrices, rows in expert order, FP32 for the combine
        dict(name="experts_down_32", op="gemv", tokens=32, n=4096, k=1536, experts=64, top_k=4, gather=False, f32=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "route", "combine", "gemv"])
    if op == "norm":
        out = rng.choice(["mx", "bf16"])
        train = out == "bf16" and rng.random() < 0.6
        return dict(op=op, rows=_log_int(rng, 1, 8191 if train else 16384),
                    cols=128 * _log_int(rng, 2, 32 if train else 40), residual=rng.random() < 0.7, out=out,
                    tiled=out == "mx" and rng.random() < 0.5, train=train)
    if op == "route":
        experts = rng.choice([8, 16, 24, 60, 64, 96, 128, 160, 256])
        groups = rng.choice([1, 1, 2, 4]) if experts % 4 == 0 else 1
        topk_groups = rng.randint(1, groups)
        top_k = min(rng.randint(1, 8), experts // groups * topk_groups)
        return dict(op=op, tokens=_log_int(rng, 1, 16384), experts=experts, top_k=top_k,
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                    topk_groups=topk_groups, renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]),
                    bf16=rng.random() < 0.4, train=rng.random() < 0.5)
    if op == "combine":
        cols, top_k, f32 = 64 * _log_int(rng, 2, 64), rng.randint(1, 5), rng.random() < 0.3
        most = min(16384, 65536 * 4096 // (cols * top_k * (2 if f32 else 1)))
        return dict(op=op, tokens=_log_int(rng, 1, most), cols=cols, top_k=top_k, base=rng.random() < 0.5, f32=f32,
                    train=rng.random() < 0.5)
    if rng.random() < 0.5:
        return dict(op=op, tokens=_log_int(rng, 1, 40), n=16 * _log_int(rng, 8, 1280), k=64 * _log_int(rng, 4, 80),
                    experts=0, top_k=0, gather=False, f32=rng.random() < 0.5)
    return dict(op=op, tokens=_log_int(rng, 1, 32), n=128 * _log_int(rng, 2, 24), k=64 * _log_int(rng, 8, 32),
                experts=rng.choice([8, 16, 60, 64]), top_k=rng.randint(1, 4), gather=rng.random() < 0.5,
                f32=rng.random() < 0.5)


# ------------------------------------------------------------------------------------------ inputs
def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device=DEVICE) * std).to(dtype)


def _grad(g, shape, std, dtype=torch.bfloat16):
    """Gradient-like: a normal draw over a square root, heavy tails."""
    a = torch.randn(shape, generator=g, device=DEVICE)
    b = torch.rand(shape, generator=g, device=DEVICE).clamp_(1e-3)
    return (a * b.rsqrt() * std).to(dtype)


def _choose(g, tokens, experts, top_k):
    """top_k distinct experts for each token, the experts' popularity falling as rank^-1.1 (Gumbel top-k)."""
    rank = torch.randperm(experts, generator=g, device=DEVICE).float() + 1.0
    u = torch.rand((tokens, experts), generator=g, device=DEVICE).clamp_(1e-6, 1 - 1e-6)
    return (-1.1 * rank.log() - (-u.log()).log()).topk(top_k, dim=1).indices


def _grouped(chosen, experts):
    """Rows in expert order, by (token, slot) within an expert: offsets, the rows' tokens, the slots' rows."""
    flat = chosen.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    slot_row = torch.empty_like(order)
    slot_row[order] = torch.arange(order.numel(), device=flat.device)
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device=flat.device)
    offsets[1:] = torch.bincount(flat, minlength=experts).cumsum(0)
    return (offsets.int(), (order // chosen.shape[1]).int(), slot_row.reshape(chosen.shape).int())


def _nvfp4_weights(g, matrices, n, k):
    """`matrices` weights [n, k] ~ N(0, 0.02) in NVFP4: codes [matrices, n, k/2], tiled scale bytes
    [matrices, ceil(n/128)*128*k/16], FP32 scales [matrices]."""
    grid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEVICE)
    codes = torch.empty((matrices, n, k // 2), dtype=torch.uint8, device=DEVICE)
    pad = -(-n // 128) * 128
    scales = torch.empty((matrices, pad * k // 16), dtype=torch.uint8, device=DEVICE)
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
        rows = torch.zeros((pad, k // 16), dtype=torch.uint8, device=DEVICE)
        rows[:n] = byte.view(torch.uint8)
        scales[e] = rows.view(pad // 128, 4, 32, k // 64, 4).permute(0, 3, 2, 1, 4).reshape(-1)
    return codes, scales, glob


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    c, s = case, {"case": case}
    if c["op"] == "norm":
        shape = (c["rows"], c["cols"])
        s["x"] = _normal(g, shape)
        s["residual"] = _normal(g, shape, 2.0) if c["residual"] else None
        s["w"] = (1.0 + 0.2 * torch.randn(c["cols"], generator=g, device=DEVICE)).to(torch.bfloat16)
        if c["train"]:
            s["dy"] = _grad(g, shape, 1e-3)
            s["dh"] = _grad(g, shape, 1e-3)
    elif c["op"] == "route":
        t, e = c["tokens"], c["experts"]
        s["logits"] = _normal(g, (t, e), 1.5, torch.bfloat16 if c["bf16"] else torch.float32)
        s["bias"] = torch.randn(e, generator=g, device=DEVICE) * 0.05 if c["bias"] else None
        if c["train"]:
            s["dweight"] = _grad(g, (t, c["top_k"]), 1e-2, torch.float32)
    elif c["op"] == "combine":
        t, k, n = c["tokens"], c["top_k"], c["cols"]
        dt = torch.float32 if c["f32"] else torch.bfloat16
        s["rows"] = _normal(g, (t * k, n), 0.5, dt)
        s["offsets"], _, s["slot_row"] = _grouped(_choose(g, t, 64, k), 64)
        s["weight"] = torch.softmax(torch.randn((t, k), generator=g, device=DEVICE), 1)
        s["base"] = _normal(g, (t, n)) if c["base"] else None
        if c["train"]:
            s["dout"] = _grad(g, (t, n), 1e-3)
    else:
        n, k, t = c["n"], c["k"], c["tokens"]
        s["q"], s["sf"], s["g"] = _nvfp4_weights(g, max(1, c["experts"]), n, k)
        s["offsets"] = s["row_index"] = None
        rows = t
        if c["experts"]:
            s["offsets"], row_index, _ = _grouped(_choose(g, t, c["experts"], c["top_k"]), c["experts"])
            s["row_index"] = row_index if c["gather"] else None
            rows = t if c["gather"] else t * c["top_k"]
        s["x"] = _normal(g, (rows, k))
    return s


# ------------------------------------------------------------------------------------------ plain forms
def _plain_norm(s):
    c = s["case"]
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(torch.bfloat16)
    hf, w = h.float(), s["w"].float()
    r = 1.0 / torch.sqrt((hf * hf).mean(1, keepdim=True) + EPS)
    n = hf * r
    y = n * w
    out = {"h": h}
    if c["out"] == "bf16":
        out["y"] = y.to(torch.bfloat16)
    else:
        blocks = y.view(c["rows"], -1, 32)
        e = torch.frexp(blocks.abs().amax(2)).exponent - 9  # floor(log2 amax) - 8
        e = e.clamp(-127, 127)
        v = torch.ldexp(blocks, -e.unsqueeze(2)).clamp(-448.0, 448.0)
        out["codes"] = v.to(torch.float8_e4m3fn).view(c["rows"], c["cols"])
        byte = (e + 127).to(torch.uint8)
        if c["tiled"]:
            pad = -(-c["rows"] // 128) * 128
            full = torch.zeros((pad, c["cols"] // 32), dtype=torch.uint8, device=byte.device)
            full[:c["rows"]] = byte
            byte = full.view(pad // 128, 4, 32, -1, 4).permute(0, 3, 2, 1, 4).reshape(-1)
        out["scales"] = byte.view(torch.float8_e8m0fnu)
    if c["train"]:
        dy = s["dy"].float()
        gy = dy * w
        dx = r * (gy - n * (gy * n).mean(1, keepdim=True)) + s["dh"].float()
        out["dx"] = dx.to(torch.bfloat16)
        out["dw"] = (dy * n).sum(0).to(torch.bfloat16)
    return out


def _scores(case, logits):
    if case["score"] == "softmax":
        z = (logits - logits.amax(1, keepdim=True)).exp()
        return z / z.sum(1, keepdim=True)
    return 1.0 / (1.0 + (-logits).exp())


def _plain_route(s):
    c = s["case"]
    t, e, k = c["tokens"], c["experts"], c["top_k"]
    # the choice goes by values next to one another: 64 bits, ties to the lowest index
    key = s["logits"].double()
    if c["bias"] or c["groups"] > 1:
        key = _scores(c, key)
    if c["bias"]:
        key = key + s["bias"].double()
    if c["groups"] > 1:
        per = key.view(t, c["groups"], e // c["groups"])
        two = torch.sort(per, dim=2, descending=True).values[:, :, :2].sum(2)
        keep = torch.sort(two, dim=1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        mask = torch.zeros((t, c["groups"]), dtype=torch.bool, device=key.device).scatter_(1, keep, True)
        key = torch.where(mask.unsqueeze(2), per, -math.inf).view(t, e)
    chosen = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    p = _scores(c, s["logits"].float())
    at = p.gather(1, chosen)
    total = at.sum(1, keepdim=True)
    w = at / total * c["scale"] if c["renorm"] else at * c["scale"]
    offsets, row_index, slot_row = _grouped(chosen, e)
    out = {"expert": chosen.int(), "weight": w, "offsets": offsets, "row_index": row_index, "slot_row": slot_row}
    if c["train"]:
        d = s["dweight"] * c["scale"]
        if c["renorm"]:
            d = (d - (d * at / total).sum(1, keepdim=True)) / total
        dp = torch.zeros_like(p).scatter_(1, chosen, d)
        if c["score"] == "softmax":
            dl = p * (dp - (dp * p).sum(1, keepdim=True))
        else:
            dl = dp * p * (1.0 - p)
        out["dlogits"] = dl.to(s["logits"].dtype)
    return out


def _plain_combine(s):
    c = s["case"]
    at = s["slot_row"].long()
    rows = s["rows"].float()[at]
    acc = (rows * s["weight"].unsqueeze(2)).sum(1)
    if s["base"] is not None:
        acc = acc + s["base"].float()
    out = {"out": acc.to(torch.bfloat16)}
    if c["train"]:
        d = s["dout"].float().unsqueeze(1)
        out["dweight"] = (rows * d).sum(2)
        drows = torch.empty_like(s["rows"])
        drows[at.reshape(-1)] = (s["weight"].unsqueeze(2) * d).to(s["rows"].dtype).reshape(-1, c["cols"])
        out["drows"] = drows
    return out


def _plain_gemv(s):
    c = s["case"]
    n, k = c["n"], c["k"]
    values = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEVICE)
    values = torch.cat([values, -values])
    if c["experts"]:
        row = torch.arange(int(c["tokens"] * c["top_k"]), device=DEVICE)
        which = torch.searchsorted(s["offsets"][1:].contiguous().long(), row, right=True)
        q, sf, g = s["q"][which], s["sf"][which], s["g"][which]
        x = s["x"].float()[s["row_index"].long()] if c["gather"] else s["x"].float()
    else:
        q, sf, g, x = s["q"], s["sf"], s["g"], s["x"].float()
    m = q.shape[0]
    both = torch.stack([q & 15, q >> 4], dim=3).view(-1).int()
    w = values.index_select(0, both).view(m, n, k // 16, 16)
    pad = -(-n // 128) * 128
    scale = sf.view(m, pad // 128, k // 64, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(m, pad, k // 16)[:, :n]
    w = (w * scale.contiguous().view(torch.float8_e4m3fn).float().unsqueeze(3)).view(m, n, k)
    if c["experts"]:
        y = torch.bmm(w, x.unsqueeze(2)).squeeze(2) * g.unsqueeze(1)
    else:
        y = (x @ w[0].t()) * g
    return {"y": y if c["f32"] else y.to(torch.bfloat16)}


# ------------------------------------------------------------------------------------------ the framework's
def _own(s):
    import nvfp4_bit_precision_b200 as nv
    c = s["case"]
    if c["op"] == "norm":
        mx = c["out"] == "mx"
        f = nv.rmsnorm(s["x"], s["w"], s["residual"], EPS, y=not mx, mx=mx, rstd=c["train"],
                       mx_sf_layout=nv.NVFP4_SF_MMA if c["tiled"] else nv.NVFP4_SF_ROWMAJOR)
        out = {"h": f["h"]}
        if mx:
            out["codes"] = f["mx"][0].view(torch.float8_e4m3fn)
            out["scales"] = f["mx"][1].view(torch.float8_e8m0fnu)
        else:
            out["y"] = f["y"]
        if c["train"]:
            out["dx"], out["dw"] = nv.rmsnorm_backward(s["dy"], f["h"], s["w"], f["rstd"], s["dh"])
        return out
    if c["op"] == "route":
        r = nv.route(s["logits"], c["top_k"], bias=s["bias"], groups=c["groups"], topk_groups=c["topk_groups"],
                     score=nv.NVFP4_SOFTMAX if c["score"] == "softmax" else nv.NVFP4_SIGMOID,
                     renormalize=c["renorm"], scale=c["scale"])
        out = {"expert": r.expert, "weight": r.weight, "offsets": r.group_offsets, "row_index": r.row_index,
               "slot_row": r.slot_row}
        if c["train"]:
            out["dlogits"] = nv.route_backward(s["dweight"], s["logits"], r)
        return out
    if c["op"] == "combine":
        out = {"out": nv.combine(s["rows"], s["slot_row"], s["weight"], s["base"])}
        if c["train"]:
            out["drows"], out["dweight"] = nv.combine_backward(s["dout"], s["rows"], s["slot_row"], s["weight"],
                                                               s["offsets"])
        return out
    dt = nv.NVFP4_OUT_F32 if c["f32"] else nv.NVFP4_OUT_BF16
    if c["experts"]:
        return {"y": nv.grouped_gemv(s["offsets"], s["x"], s["q"], s["sf"], s["g"], c["n"], s["row_index"], dt)}
    w = nv.NVFP4Tensor(s["q"][0], s["sf"][0], s["g"], c["n"], c["k"], nv.NVFP4_SF_MMA)
    return {"y": nv.gemv(s["x"], w, dt)}


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "route": _plain_route, "combine": _plain_combine,
            "gemv": _plain_gemv}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------ cost
def work(case):
    c = case
    if c["op"] == "norm":
        m = c["rows"] * c["cols"]
        b = m * 2 * (3 if c["residual"] else 1) + 2 * c["cols"]      # x, residual in, h out
        b += m * 2 if c["out"] == "bf16" else m + m // 32
        f = 6 * m
        if c["train"]:                                               # h, dy, dh in, dx out
            b += m * 2 * 4 + 4 * c["cols"]
            f += 10 * m
        return {"bytes": b, "flops": f}
    if c["op"] == "route":
        t, e, k = c["tokens"], c["experts"], c["top_k"]
        el = 2 if c["bf16"] else 4
        b = t * e * el + (4 * e if c["bias"] else 0) + 16 * t * k + 4 * (e + 1)
        if c["train"]:                                               # logits, dweight, expert in, dlogits out
            b += 2 * t * e * el + 8 * t * k
        return {"bytes": b, "flops": 5 * t * e}
    if c["op"] == "combine":
        t, n, k = c["tokens"], c["cols"], c["top_k"]
        el = 4 if c["f32"] else 2
        b = t * k * n * el + 8 * t * k + 2 * t * n * (2 if c["base"] else 1)
        f = 2 * t * k * n
        if c["train"]:                                               # rows, dout in, drows, dweight out
            b += 2 * t * k * n * el + 2 * t * n + 12 * t * k
            f += 3 * t * k * n
        return {"bytes": b, "flops": f}
    n, k, t = c["n"], c["k"], c["tokens"]
    rows = t * max(1, c["top_k"])
    used = 1
    if c["experts"]:                                                 # experts that some token is expected to choose
        p = [r ** -1.1 for r in range(1, c["experts"] + 1)]
        used = sum(1.0 - (1.0 - min(1.0, c["top_k"] * v / sum(p))) ** t for v in p)
    b = used * n * k * 9 / 16 + (t if c["gather"] else rows) * k * 2 + rows * n * (4 if c["f32"] else 2)
    return {"bytes": int(b), "flops": 2 * rows * n * k}


# ------------------------------------------------------------------------------------------ 64 bits
def _e4m3(v):
    """The E4M3 value nearest v (ties to even, saturating), by its grid: 3 fraction bits, smallest step 2^-9."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp_min(-6) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _exact_norm(c, s):
    out = {}
    h = s["x"].double()
    if s["residual"] is not None:
        h = (h + s["residual"].double()).to(torch.bfloat16).double()
    out["h"] = h
    w = s["w"].double()
    rstd = (h.square().sum(1) / c["cols"] + EPS).pow(-0.5)
    y = torch.einsum("rc,r,c->rc", h, rstd, w)
    if c["out"] == "bf16":
        out["y"] = y
    else:
        b = y.unflatten(1, (-1, 32))
        e = torch.floor(torch.log2(b.abs().amax(-1))) - 8
        e = torch.where(torch.isfinite(e), e.clamp(-127, 127), torch.full_like(e, -127))
        out["codes"] = _e4m3(b * torch.exp2(-e)[..., None]).flatten(1)
        if c["tiled"]:
            r = torch.arange(c["rows"], device=h.device)[:, None]
            k = torch.arange(c["cols"] // 32, device=h.device)[None, :]
            at = (r // 128 * (c["cols"] // 128) + k // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + k % 4
            flat = torch.full((-(-c["rows"] // 128) * 4 * c["cols"],), 2.0 ** -127, dtype=torch.float64, device=h.device)
            flat[at.flatten()] = torch.exp2(e).flatten()
            out["scales"] = flat
        else:
            out["scales"] = torch.exp2(e)
    if c["train"]:
        # d/dh of sum(dy * y): the Jacobian diag(w) rstd (I - h h^T rstd^2 / n), transposed and applied
        u = s["dy"].double() * w
        hu = (h * u).sum(1) * rstd.pow(3) / c["cols"]
        out["dx"] = u * rstd[:, None] - h * hu[:, None] + s["dh"].double()
        out["dw"] = torch.einsum("rc,rc,r->c", s["dy"].double(), h, rstd)
    return out


def _exact_route(c, s):
    l = s["logits"].double()
    t, e = l.shape
    if c["score"] == "softmax":
        p = torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
    else:
        p = torch.sigmoid(l)
    pick = p if s["bias"] is None else p + s["bias"].double()
    if s["bias"] is None and c["groups"] == 1:
        pick = l
    if c["groups"] > 1:
        per = pick.unflatten(1, (c["groups"], -1))
        a = per.amax(2)
        if per.shape[2] > 1:
            a = a + per.kthvalue(per.shape[2] - 1, dim=2).values
        order = torch.argsort(-a, dim=1, stable=True)
        rank = torch.argsort(order, dim=1)
        pick = per.masked_fill((rank >= c["topk_groups"])[..., None], -math.inf).flatten(1)
    order = torch.argsort(-pick, dim=1, stable=True)[:, :c["top_k"]]
    hot = torch.nn.functional.one_hot(order, e).double()             # [tokens, slot, expert]
    at = torch.einsum("tke,te->tk", hot, p)
    norm = at.sum(1, keepdim=True) if c["renorm"] else torch.ones_like(at[:, :1])
    w = c["scale"] * at / norm
    out = {"expert": None, "weight": w, "offsets": None, "row_index": None, "slot_row": None}
    if c["train"]:
        d = s["dweight"].double()
        dat = c["scale"] * d / norm
        if c["renorm"]:
            dat = dat - (d * w).sum(1, keepdim=True) / norm
        dp = torch.einsum("tke,tk->te", hot, dat)
        if c["score"] == "softmax":
            out["dlogits"] = p * dp - p * torch.einsum("te,te->t", p, dp)[:, None]
        else:
            out["dlogits"] = dp * p * torch.sigmoid(-l)
    return out


def _exact_combine(c, s):
    t, k, n = c["tokens"], c["top_k"], c["cols"]
    acc = torch.zeros((t, n), dtype=torch.float64, device=DEVICE) if s["base"] is None else s["base"].double()
    out = {}
    if c["train"]:
        out["dweight"] = torch.empty((t, k), dtype=torch.float64, device=DEVICE)
        out["drows"] = torch.empty((t * k, n), dtype=torch.float64, device=DEVICE)
    for j in range(k):
        at = s["slot_row"][:, j].long()
        row = s["rows"].index_select(0, at).double()
        wj = s["weight"][:, j].double()
        acc = acc + row * wj[:, None]
        if c["train"]:
            d = s["dout"].double()
            out["dweight"][:, j] = torch.einsum("tn,tn->t", row, d)
            out["drows"][at] = d * wj[:, None]
    out["out"] = acc
    return out


def _exact_matrix(q, sf, g, n, k):
    """One NVFP4 matrix in 64 bits, by the place of each scale byte in the tiled order."""
    nib = torch.empty((n, k), dtype=torch.int64, device=q.device)
    nib[:, 0::2] = q.long() % 16
    nib[:, 1::2] = q.long() // 16
    e, m = nib % 8 // 2, nib % 2
    mag = torch.where(e == 0, m * 0.5, (1.0 + 0.5 * m.double()) * torch.exp2((e - 1).double()))
    r = torch.arange(n, device=q.device)[:, None]
    b = torch.arange(k // 16, device=q.device)[None, :]
    byte = sf[(r // 128 * (k // 64) + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4].long()
    ex, fr = byte // 8, (byte % 8).double()
    d = torch.where(ex == 0, fr * 2.0 ** -9, (1.0 + fr / 8.0) * torch.exp2((ex - 7).double()))
    return (mag * torch.where(nib >= 8, -1.0, 1.0)) * d.repeat_interleave(16, 1) * g.double()


def _exact_gemv(c, s):
    n, k = c["n"], c["k"]
    if not c["experts"]:
        return {"y": torch.mm(s["x"].double(), _exact_matrix(s["q"][0], s["sf"][0], s["g"][0], n, k).t())}
    x = s["x"].double()
    if c["gather"]:
        x = x[s["row_index"].long()]
    y = torch.empty((x.shape[0], n), dtype=torch.float64, device=DEVICE)
    off = s["offsets"].tolist()
    for e in range(c["experts"]):
        if off[e] < off[e + 1]:
            w = _exact_matrix(s["q"][e], s["sf"][e], s["g"][e], n, k)
            y[off[e]:off[e + 1]] = torch.mm(x[off[e]:off[e + 1]], w.t())
    return {"y": y}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "route": _exact_route, "combine": _exact_combine,
            "gemv": _exact_gemv}[case["op"]](case, s)
