"""Pins of the oracle of the single-token and 4-bit operators (oracle/tokens.py) against facts that do
not depend on its code."""
import numpy as np
import pytest

from oracle import attention as OA, layer as OL, tokens as OT
from oracle.formats import bf16_bits_to_f32, bf16_rne

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def _bits(rng, *shape, scale=1.0):
    return bf16_rne((rng.standard_normal(shape) * scale).astype(np.float32))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("is_v", [0, 1])
def test_places_are_a_permutation(dim, is_v):
    codes, scales = OT._places(dim, is_v)
    assert np.array_equal(np.sort(codes.ravel()), np.arange(32 * dim))
    assert np.array_equal(np.sort(scales.ravel()), np.arange(2 * dim))


def test_a_block_written_out_by_hand():
    x = np.zeros((1, 32), np.float32)
    x[0, :8] = [7.0, -6.0, 5.0, 2.5, 0.25, -0.25, 0.26, -0.0]    # max 7: exponent 0, 7 saturates
    codes, scales = OT.quantise(x)
    assert scales.tolist() == [[127]]
    assert codes[0, :4].tolist() == [0x7 | 0xF << 4, 0x6 | 0x4 << 4, 0x0 | 0x8 << 4, 0x1 | 0x8 << 4]
    assert OT.dequantise(codes, scales)[0, :7].tolist() == [6, -6, 4, 2, 0, 0, 0.5]
    c4, s4 = OT.quantise(x * 4)
    assert np.array_equal(c4, codes) and s4.tolist() == [[129]]


def test_every_value_is_nearest_and_blocks_are_independent():
    rng = np.random.default_rng(0)
    x = bf16_bits_to_f32(_bits(rng, 50, 128)) * np.exp(3 * rng.standard_normal((50, 128))).astype(np.float32)
    x = bf16_bits_to_f32(bf16_rne(x))
    codes, scales = OT.quantise(x)
    v = OT.dequantise(codes, scales)
    unit = np.ldexp(1.0, scales.astype(int) - 127).repeat(32, axis=1)
    grid = np.concatenate([-GRID[::-1], GRID])
    best = np.abs(np.clip(x / unit, -6, 6)[..., None] - grid).min(axis=-1)
    assert np.allclose(np.abs(np.clip(x / unit, -6, 6) - v / unit), best, atol=0, rtol=0)
    a = np.abs(x).reshape(50, 4, 32).max(-1)
    u = np.ldexp(1.0, scales.astype(int) - 127)
    assert np.all((4 * u <= a) & (a < 8 * u))
    one = OT.quantise(x[:, 32:64])
    assert np.array_equal(one[0], codes[:, 16:32]) and np.array_equal(one[1], scales[:, 1:2])


def test_limits_of_the_exponent_and_bad_values():
    x = np.zeros((6, 32), np.float32)
    x[1, 0], x[2, 0], x[3, 0], x[4, 0], x[5, 0] = 3e38, 2.0 ** -120, np.inf, np.nan, -3e38
    codes, scales = OT.quantise(x)
    assert scales.ravel().tolist() == [17, 212, 17, 255, 255, 212]
    v = OT.dequantise(codes, scales)
    assert v[1, 0] == 6 * 2.0 ** 85 and v[5, 0] == -6 * 2.0 ** 85 and np.all(v[2] == 0)
    assert np.all(np.isnan(v[3:5])) and np.all(codes[3:5] == 0)


def test_cache_of_tokens_in_any_order():
    rng = np.random.default_rng(1)
    dim, n = 64, 150
    K, V = _bits(rng, n, 2 * dim), _bits(rng, n, 2 * dim)
    table = np.array([[3, 0, 2]])
    whole, parts = OT.new_cache(4, 2, dim, 0x5A), OT.new_cache(4, 2, dim, 0x5A)
    OT.kv_write(whole, K, V, table, [0, n], [0])
    for a, b in ((100, 150), (0, 37), (37, 100)):
        OT.kv_write(parts, K[a:b], V[a:b], table, [0, b - a], [a])
    for k in ("kc", "vc", "ks", "vs"):
        assert np.array_equal(whole[k], parts[k])
        assert np.all(whole[k][1] == 0x5A)
    for h in range(2):
        got, ok = OT.kv_values(whole, table[0], n, h, 1)
        x = bf16_bits_to_f32(V[:, h * dim:(h + 1) * dim])
        assert ok.all() and np.array_equal(got, OT.dequantise(*OT.quantise(x)))
        assert np.linalg.norm(got - x) < 0.14 * np.linalg.norm(x)


def test_attention_of_one_token_and_of_equal_keys():
    rng = np.random.default_rng(2)
    dim = 64
    c = OT.new_cache(2, 1, dim)
    V = _bits(rng, 70, dim)
    OT.kv_write(c, np.zeros_like(V), V, np.array([[1, 0]]), [0, 70], [0])
    v, _ = OT.kv_values(c, np.array([1, 0]), 70, 0, 1)
    q = rng.standard_normal((3, 1, dim))
    o = OT.attention(q, c, np.array([[1, 0]]), [0, 3], [70], 0.1, False)
    assert np.allclose(o["O"][:, 0], v.mean(axis=0)) and np.allclose(o["lse"], np.log(70))
    o = OT.attention(q, c, np.array([[1, 0]]), [0, 3], [1], 0.1, True)
    assert np.all(np.isneginf(o["lse"][:2])) and np.all(o["O"][:2] == 0)
    assert np.allclose(o["O"][2, 0], v[0])


def test_qk_norm_rope_by_hand():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((4, 3, 32))
    freq, pos = np.array([0.3, 0.2, 0.1, 0.5, 0.0, 1.0, 2.0, 3.0]), rng.integers(-9, 9, (4, 1))
    g = bf16_rne(np.full(32, 2.0, np.float32))
    y, z = OT.qk_norm_rope(x, 2, g, None, 1e-30, pos, freq, [16], True)
    assert np.allclose((z ** 2).mean(-1), [[4, 4, 1]] * 4) and np.allclose((y ** 2).sum(-1), (z ** 2).sum(-1))
    assert np.array_equal(y[..., 16:], z[..., 16:])
    w = (z[..., 0:16:2] + 1j * z[..., 1:16:2]) * np.exp(1j * pos[:, :, None] * freq)
    assert np.allclose(y[..., 0:16:2], w.real) and np.allclose(y[..., 1:16:2], w.imag)
    y2, _ = OT.qk_norm_rope(1000 * x, 2, g, None, 1e-30, pos, freq, [16], True)
    assert np.allclose(y, y2)
    assert np.allclose(OT.qk_norm_rope(x, 2, None, None, 1e-30, 0 * pos, freq, [16], False)[0],
                       x / np.sqrt((x ** 2).mean(-1, keepdims=True)))


@pytest.mark.parametrize("fmt", ["nvfp4", "int4", "mxfp4"])
def test_gemv_rebuilds_the_layer(fmt):
    """Weight values by loops; and with the residual and both factors the product of the weight."""
    rng = np.random.default_rng(4)
    N, K, r = 6, 256, 8
    W, X = _bits(rng, N, K, scale=K ** -0.5), _bits(rng, 3, K)
    lam = np.exp(0.5 * rng.standard_normal(K)).astype(np.float32)
    down, up = _bits(rng, r, K, scale=0.05), _bits(rng, N, r, scale=0.05)
    wt = OL.prepare_weight(W, lam, down, up, fmt)
    w = OT.weight_values(wt["codes"], wt["scales"], wt["g"], fmt)
    n = dict(nvfp4=16, int4=64, mxfp4=32)[fmt]
    for i, k in ((0, 0), (2, 77), (5, 255), (3, 128)):
        nib = int(wt["codes"][i, k // 2]) >> (4 * (k % 2)) & 15
        s = wt["scales"][i, k // n]
        if fmt == "int4":
            want = (nib - 16 if nib > 7 else nib) * float(s)
        else:
            want = GRID[nib & 7] * (-1 if nib & 8 else 1)
            want *= 2.0 ** (int(s) - 127) if fmt == "mxfp4" else \
                (((8 + (s & 7)) * 2.0 ** ((s >> 3) - 10)) if s >> 3 else (s & 7) * 2.0 ** -9) * float(wt["g"])
        assert w[i, k] == want
    y, a = OT.gemv(X, lam, down, up, w)
    assert np.all(np.abs(y) <= a)
    full = w + bf16_bits_to_f32(up).astype(np.float64) @ bf16_bits_to_f32(down)
    xh = bf16_bits_to_f32(bf16_rne(bf16_bits_to_f32(X) / lam))
    assert np.allclose(y, xh @ full.T, atol=1e-2)
    y0, _ = OT.gemv(X, None, None, None, w)
    assert np.allclose(y0, bf16_bits_to_f32(X).astype(np.float64) @ w.T)


def test_planted_mistakes_are_seen():
    """A wrong pair order, a scale of the next token or a floor rule off by one fails the pins above:
    their effect is larger than what those allow."""
    rng = np.random.default_rng(5)
    x = bf16_bits_to_f32(_bits(rng, 64, 64))
    codes, scales = OT.quantise(x)
    v = OT.dequantise(codes, scales)
    swapped = (codes >> 4) | (codes << 4).astype(np.uint8)
    assert not np.array_equal(OT.dequantise(swapped, scales), v)
    assert not np.array_equal(OT.dequantise(codes, np.roll(scales, 1, axis=0)), v)
    assert np.linalg.norm(OT.dequantise(codes, scales + 1) - x) > 0.5 * np.linalg.norm(x)
    assert OA.PAGE == OT.PAGE == 64
