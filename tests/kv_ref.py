"""A paged NVFP4 cache, its append and the attention over it in plain NumPy with 64 bits, for the tests."""
import numpy as np

import workloads as W

MAG = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
E2M1 = np.concatenate([MAG, -MAG])


def e4m3_table():
    b = np.arange(256)
    e, m = b >> 3 & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    v[(b & 127) == 127] = np.nan
    return np.where(b >= 128, -v, v)


E4M3 = e4m3_table()


def decode(q, sf, g):
    """Codes [..., d/2], scale bytes [..., d/16] -> float64 [..., d]."""
    d = 2 * q.shape[-1]
    v = np.empty(q.shape[:-1] + (d,))
    v[..., 0::2], v[..., 1::2] = E2M1[q & 15], E2M1[q >> 4]
    return v * np.repeat(E4M3[sf], 16, axis=-1) * float(g)


def quantise(x, amax):
    """bf16 values in float32 [..., d] -> (codes, scale bytes) by the format's steps in binary32."""
    one = np.float32
    amax = one(amax)
    S = one(1) if amax == 0 else one(2688) / amax
    b = x.astype(np.float32).reshape(x.shape[:-1] + (-1, 16))
    s = (np.abs(b).max(-1) / one(6)) * S
    # E4M3, nearest with ties to even, saturating
    s64 = np.minimum(s.astype(np.float64), 1e9)
    _, e = np.frexp(s64)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    d = np.minimum(np.rint(s64 / step) * step, 448.0)
    byte = np.searchsorted(E4M3[:127], d).astype(np.uint8)
    assert np.array_equal(E4M3[byte], d)
    with np.errstate(divide="ignore"):
        r = np.where(d > 0, S / d.astype(np.float32), one(0)).astype(np.float32)
    y = b * r[..., None]
    a = np.abs(y)
    c = ((a > 0.25).astype(np.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)).astype(np.uint8)
    c += np.signbit(b).astype(np.uint8) * 8
    c = c.reshape(x.shape)
    return c[..., 0::2] | c[..., 1::2] << 4, byte


def bf16_of(d):
    """float64 -> bf16 bits in one rounding, ties to even."""
    f = d.astype(np.float32)
    u = f.view(np.uint32).astype(np.int64)
    tie = ((u & 0xFFFF) == 0x8000) & np.isfinite(d)
    lost = np.abs(d) - np.abs(f.astype(np.float64))
    u = (u + np.where(tie, np.sign(lost), 0).astype(np.int64)).astype(np.uint32)
    return W.f32_to_bf16_bits(u.view(np.float32))


def turn(x, cos, sin, position, rot, neighbours):
    """bf16 bits [tokens, heads, dim] turned by position -> bf16 bits."""
    y = W.bf16_bits_to_f32(x).astype(np.float64)
    c, s = cos[position][:, None].astype(np.float64), sin[position][:, None].astype(np.float64)
    one = np.arange(0, rot, 2) if neighbours else np.arange(rot // 2)
    two = one + 1 if neighbours else one + rot // 2
    a, b = y[..., one].copy(), y[..., two].copy()
    y[..., one], y[..., two] = a * c - b * s, b * c + a * s
    return bf16_of(y)


def tables(rot, angles, base=10000.0):
    f = base ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(angles)[:, None] * f
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def attend(q, k, v, length, scale, window=0):
    """One sequence: q [queries, heads, dim], k, v [kv_heads, tokens, dim] float64 -> out, lse, and the bounds of both
    on what a kernel may differ by (without the result's own rounding)."""
    new, heads, dim = q.shape
    kv = k.shape[0]
    group = heads // kv
    out, lse = np.zeros((new, heads, dim)), np.full((new, heads), -np.inf)
    obound, lbound = np.zeros((new, heads, dim)), np.zeros((new, heads))
    for i in range(new):
        end = length - new + 1 + i
        begin = max(0, end - window) if window else 0
        if end <= begin:
            continue
        for h in range(heads):
            K, V = k[h // group, begin:end], v[h // group, begin:end]
            x = (K @ q[i, h]) * scale
            top = x.max()
            p = np.exp(x - top)
            lse[i, h] = top + np.log(p.sum())
            p /= p.sum()
            out[i, h] = p @ V
            # A score: the tensor cores' sums over dim may truncate each addition, 2^-23 of the magnitudes, and the
            # products with the scale and the factors' roundings are 2^-22 of it; in base 2, 2^-23 of the largest
            # for the difference from the maximum.
            mags = (np.abs(K) @ np.abs(q[i, h])) * abs(scale)
            e = ((17 * (dim // 16) + 8) * 2.0 ** -23 * mags).max() + 2.0 ** -20 * (1 + np.abs(x).max())
            n = end - begin
            lbound[i, h] = e + (n + 64) * 2.0 ** -24 + 2.0 ** -22 * (1 + abs(lse[i, h]))
            # An exponential in FP16: half a step, 2^-11 of it, or, where it is below FP16's normal numbers, 2^-25; they are
            # taken times 2^9 or more at the largest, so that this is 2^-34 of it; both sums.
            obound[i, h] = (p @ np.abs(V)) * (2.0 ** -11 + 2 * e + (17 * (n // 16 + 8) + n + 64) * 2.0 ** -23) + \
                2.0 ** -34 * np.abs(V).sum(0)
    return out, lse, obound, lbound
