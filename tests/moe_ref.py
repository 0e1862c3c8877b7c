"""64-bit restatements of the MoE block's operators, in numpy: the norm, the MXFP8 rule, routing, the
combine and the few-token products, with the gradients.  They share nothing with the package."""
import numpy as np

MASKED = -3.38953138925153547590e+38  # the lowest finite bf16 value


def bf16_round(a):
    """Nearest bf16 value (ties to even) of float64 data whose FP32 rounding is exact or irrelevant."""
    u = np.asarray(a, dtype=np.float32).view(np.uint32)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & np.uint32(0xFFFF0000)
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


# ------------------------------------------------------------------------------------ norm
def rmsnorm(x, r, w, eps):
    """h (bf16 values), rstd, y in float64; the sum x + r is rounded through FP32, as two bf16 values' is."""
    h = x if r is None else bf16_round((x.astype(np.float32) + r.astype(np.float32)).astype(np.float64))
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h, rstd, h * rstd[:, None] * w[None, :]


def rmsnorm_backward(dy, h, w, eps, dh=None):
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    n = h * rstd[:, None]
    g = dy * w[None, :]
    dx = rstd[:, None] * (g - n * (g * n).mean(1, keepdims=True))
    if dh is not None:
        dx = dx + dh
    return dx, (dy * n).sum(0)


def e4m3_nearest(v):
    """Nearest E4M3 value, ties to even, saturating at 448."""
    _, e = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.clip(np.round(v / step) * step, -448.0, 448.0)


def e4m3_value(codes):
    c = codes.astype(np.int64)
    e, m = (c >> 3) & 15, (c & 7).astype(np.float64)
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * np.ldexp(1.0, e - 7))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v)


def mx_exponent(y):
    """floor(log2 amax) - 8 of each 32-block, clamped to [-127, 127]; -127 for a block of zeros."""
    b = np.abs(y).reshape(y.shape[0], -1, 32).max(2)
    _, e = np.frexp(b)
    return np.clip(np.where(b == 0, -127, e - 1 - 8), -127, 127)


def untile(sf, rows, blocks):
    """Tiled scale bytes -> [rows, blocks] (128 x 4 atoms of 512 bytes)."""
    r = np.arange(rows)[:, None]
    b = np.arange(blocks)[None, :]
    return sf.reshape(-1)[((r // 128) * (blocks // 4) + b // 4) * 512 + (r % 32) * 16 + ((r % 128) // 32) * 4 + b % 4]


def tile(sf):
    """[rows, blocks] scale bytes -> tiled, padded rows zero."""
    rows, blocks = sf.shape
    out = np.zeros(-(-rows // 128) * 128 * blocks, dtype=np.uint8)
    r = np.arange(rows)[:, None]
    b = np.arange(blocks)[None, :]
    out[((r // 128) * (blocks // 4) + b // 4) * 512 + (r % 32) * 16 + ((r % 128) // 32) * 4 + b % 4] = sf
    return out


# ------------------------------------------------------------------------------------ routing
def scores(l, softmax):
    """Scores of one token's logits; masked experts 0."""
    live = ~(l <= MASKED)
    with np.errstate(invalid="ignore", over="ignore"):
        if softmax:
            top = np.nanmax(l[live]) if live.any() and not np.isnan(l[live]).all() else 0.0
            z = np.where(live, np.exp(l - top), 0.0)
            return z / z.sum() if live.any() else z
        return np.where(live, 1.0 / (1.0 + np.exp(-l)), 0.0)


def route(logits, top_k, softmax=True, bias=None, groups=1, topk_groups=1, group_top=2, renorm=True, scale=1.0):
    """expert ids [tokens, k] (-1 = none) and weights, token by token, from the definition."""
    T, E = logits.shape
    ids = np.full((T, top_k), -1, dtype=np.int64)
    wts = np.zeros((T, top_k))
    for t in range(T):
        l = logits[t].astype(np.float64)
        live = ~(l <= MASKED)
        s = scores(l, softmax)
        if bias is None and (groups == 1 or topk_groups == groups):
            key = l.copy()
        else:
            key = s + (0.0 if bias is None else bias.astype(np.float64))
        key = np.where(np.isnan(key), -np.inf, key)  # NaN ranks last among the live ones
        cand = [e for e in range(E) if live[e]]
        if groups > 1 and topk_groups < groups:
            size = E // groups
            rank = []
            for g in range(groups):
                mine = sorted((key[e] for e in cand if e // size == g), reverse=True)[:group_top]
                if mine:
                    rank.append((-sum(mine), g))
            keep = {g for _, g in sorted(rank)[:topk_groups]}
            cand = [e for e in cand if e // size in keep]
        chosen = sorted(cand, key=lambda e: (-key[e], e))[:top_k]
        ids[t, :len(chosen)] = chosen
        if not chosen:
            continue
        if renorm:
            lc = l[chosen]
            if softmax:
                v = np.exp(lc - lc.max())
            else:  # log-sigmoid, so that very negative logits keep their ratio
                v = -np.logaddexp(0.0, -lc)
                v = np.exp(v - v.max())
            v = v / v.sum()
        else:
            v = s[chosen]
        wts[t, :len(chosen)] = scale * v
    return ids, wts


def plan(ids, experts):
    """group offsets, row_index and slot_row of the routed rows, by expert and then (token, slot)."""
    T, k = ids.shape
    flat = ids.reshape(-1)
    rows = [s for e in range(experts) for s in np.nonzero(flat == e)[0]]
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[flat >= 0], minlength=experts))])
    row_index = np.full(T * k, -1, dtype=np.int64)
    slot_row = np.full(T * k, -1, dtype=np.int64)
    for i, s in enumerate(rows):
        row_index[i] = s // k
        slot_row[s] = i
    return offsets, row_index, slot_row.reshape(T, k)


def route_backward(dw, logits, ids, softmax, renorm, scale):
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        l = logits[t].astype(np.float64)
        on = ids[t] >= 0
        if not on.any():
            continue
        e, g = ids[t][on], dw[t][on].astype(np.float64)
        if renorm:
            lc = l[e]
            v = np.exp(lc - lc.max()) if softmax else np.exp(-np.logaddexp(0, -lc) - (-np.logaddexp(0, -lc)).max())
            q = v / v.sum()
            d = scale * q * (g - (g * q).sum())
            if not softmax:
                d = d / (1.0 + np.exp(lc))
            np.add.at(out[t], e, d)
        elif softmax:
            p = scores(l, True)
            dp = np.zeros(E)
            np.add.at(dp, e, scale * g)
            out[t] = p * (dp - (p * dp).sum())
        else:
            s = 1.0 / (1.0 + np.exp(-l[e]))
            np.add.at(out[t], e, scale * g * s / (1.0 + np.exp(l[e])))
    return out


# ------------------------------------------------------------------------------------ combine
def combine(rows, slot_row, weight, base=None):
    T, k = slot_row.shape
    out = np.zeros((T, rows.shape[1])) if base is None else base.astype(np.float64).copy()
    for t in range(T):
        for j in range(k):
            if 0 <= slot_row[t, j] < rows.shape[0]:
                out[t] += weight[t, j].astype(np.float64) * rows[slot_row[t, j]]
    return out


def combine_backward(dout, rows, slot_row, weight):
    drows = np.zeros_like(rows)
    dw = np.zeros(slot_row.shape)
    for t in range(slot_row.shape[0]):
        for j in range(slot_row.shape[1]):
            r = slot_row[t, j]
            if 0 <= r < rows.shape[0]:
                drows[r] = weight[t, j].astype(np.float64) * dout[t]
                dw[t, j] = dout[t] @ rows[r]
    return drows, dw


# ------------------------------------------------------------------------------------ NVFP4 matrices
def random_nvfp4(rng, n, k, extreme=False):
    """Codes [n, k/2], scale bytes [n, k/16], g: a random NVFP4 matrix; `extreme` draws every scale byte
    up to 0x7E (subnormal ones and 0 among them)."""
    q = rng.integers(0, 256, (n, k // 2), dtype=np.uint8)
    sf = rng.integers(0, 0x7F, (n, k // 16)) if extreme else rng.integers(0x28, 0x40, (n, k // 16))
    return q, sf.astype(np.uint8), np.float32(rng.uniform(0.5, 2.0) * 2.0 ** -7)


def nvfp4_matrix(q, sf, g):
    nib = np.empty((q.shape[0], q.shape[1] * 2), dtype=np.int64)
    nib[:, 0::2], nib[:, 1::2] = q & 15, q >> 4
    values = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6])
    return values[nib] * np.repeat(e4m3_value(sf), 16, axis=1) * np.float64(g)
