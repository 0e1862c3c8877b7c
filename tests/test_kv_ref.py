"""The cache's plain forms against the oracle: the bits that a cache holds are those of the library's quantisation
from a given amax.  CPU only."""
import numpy as np
import pytest

import kv_ref as K
import workloads as W


@pytest.mark.parametrize("amax", [1.0, 5.5, 448.0, 1e-3])
def test_quantise_is_the_oracles(orc, amax):
    rng = np.random.default_rng(3)
    x = W.f32_to_bf16_bits((rng.standard_normal((32, 128)) * amax / 3).astype(np.float32))
    x[5] = 0
    x[6, :16] = 0x8000
    q, sf, g = orc.nvfp4_quantize(x, 0, amax=(amax, amax))[:3]
    mine = K.quantise(W.bf16_bits_to_f32(x), amax)
    np.testing.assert_array_equal(mine[0], q)
    np.testing.assert_array_equal(mine[1], sf)
    assert np.float32(g) == np.float32(amax) / np.float32(2688)
    np.testing.assert_array_equal(K.decode(q, sf, g), orc.nvfp4_dequant(q, sf, g))


def test_one_rounding():
    assert K.bf16_of(np.array([1 + 2.0 ** -8 + 2.0 ** -40]))[0] == 0x3F81   # above the middle, which FP32 would hit
    assert K.bf16_of(np.array([1 + 2.0 ** -8]))[0] == 0x3F80
    assert K.bf16_of(np.array([-(1 + 3 * 2.0 ** -8) + 2.0 ** -40]))[0] == 0xBF81


def test_turn_keeps_lengths():
    rng = np.random.default_rng(4)
    x = W.f32_to_bf16_bits(rng.standard_normal((5, 2, 64)).astype(np.float32))
    cos, sin = K.tables(32, 9)
    for neighbours in (False, True):
        y = W.bf16_bits_to_f32(K.turn(x, cos, sin, np.arange(5), 32, neighbours))
        np.testing.assert_allclose((y ** 2).sum(-1), (W.bf16_bits_to_f32(x) ** 2).sum(-1), rtol=2.0 ** -7)
        np.testing.assert_array_equal(y[0], W.bf16_bits_to_f32(x)[0])
        np.testing.assert_array_equal(y[..., 32:], W.bf16_bits_to_f32(x)[..., 32:])


def test_attend_sees_what_it_may():
    rng = np.random.default_rng(5)
    q, k, v = rng.standard_normal((3, 2, 4)), rng.standard_normal((1, 9, 4)), rng.standard_normal((1, 9, 4))
    a = K.attend(q, k, v, 9, 0.5)
    k2, v2 = k.copy(), v.copy()
    k2[:, 8], v2[:, 8] = 7, np.nan
    b = K.attend(q, k2, v2, 9, 0.5)
    np.testing.assert_array_equal(a[0][:2], b[0][:2])
    assert np.isnan(b[0][2]).all()
    c = K.attend(q, k, v, 2, 0.5)
    assert (c[0][0] == 0).all() and np.isneginf(c[1][0]).all() and np.isfinite(c[1][1:]).all()
    d = K.attend(q, k, v, 9, 0.5, window=1)
    np.testing.assert_allclose(d[0][1], np.broadcast_to(v[0, 7], (2, 4)))
