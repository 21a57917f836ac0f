"""Pins of the oracle of the attention half (norm, rotary positions, 8-bit cache, attention)
against facts that do not depend on its code."""
import numpy as np
import pytest

from oracle import attention as OA, mx
from oracle.formats import bf16_bits_to_f32, bf16_rne, e4m3_decode


def _bits(rng, *shape, scale=1.0):
    return bf16_rne((rng.standard_normal(shape) * scale).astype(np.float32))


def test_norm_of_a_constant_row_is_one_and_scales_away():
    x = np.full((1, 256), 3.0, np.float32)
    o = OA.rmsnorm_quant(bf16_rne(x), None, None, 1e-12, None, None)
    assert np.all(o["xhat"] == 1.0) and np.all(o["H"] == bf16_rne(x))
    assert np.all(mx.mx_dequantize(o["codes"], o["scales"], "e4m3") == 1.0)
    # the norm does not change with the row's scale; gamma and 1/λ multiply it
    rng = np.random.default_rng(0)
    b = _bits(rng, 3, 512)
    four = bf16_rne(bf16_bits_to_f32(b) * 4)
    p, q = (OA.rmsnorm_quant(v, None, None, 1e-30, None, None) for v in (b, four))
    assert np.array_equal(p["codes"], q["codes"]) and np.array_equal(p["scales"], q["scales"])
    g, lam = np.full(512, 2.0, np.float32), np.full(512, 4.0, np.float32)
    r = OA.rmsnorm_quant(b, None, bf16_rne(g), 1e-30, lam, None)
    assert np.array_equal(r["xhat"], p["xhat"] / 2)
    rms = np.sqrt(np.mean(p["xhat"].astype(np.float64) ** 2, axis=1))
    assert np.all(np.abs(rms - 1) < 1e-6)


def test_rope_keeps_lengths_and_relative_positions():
    rng = np.random.default_rng(1)
    dims, freq = [4, 6, 6], np.concatenate([100.0 ** (-np.arange(0, d, 2) / d) for d in (4, 6, 6)])
    x = rng.standard_normal((5, 2, 32))
    pos = rng.integers(-1000, 1000, (5, 3))
    for inter in (True, False):
        y = OA.rope(x, pos, freq, dims, inter, False)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        assert np.array_equal(y[..., 16:], x[..., 16:])
        assert np.allclose(OA.rope(y, pos, freq, dims, inter, True), x)
        # q·k depends on the difference of the positions only
        q, k = rng.standard_normal((2, 1, 1, 16))
        at = lambda v, p: OA.rope(v, np.array([p]), freq, dims, inter, False).ravel()  # noqa: E731
        d0 = at(q, [7, 5, -3]) @ at(k, [4, 9, 1])
        d1 = at(q, [107, 55, -33]) @ at(k, [104, 59, -29])
        assert abs(d0 - d1) < 1e-9
    one = OA.rope(np.array([[[1.0, 0.0]]]), np.array([[3]]), np.array([0.5]), [2], True, False)
    assert np.allclose(one.ravel(), [np.cos(1.5), np.sin(1.5)])


@pytest.mark.parametrize("dim", [64, 128])
def test_cache_places_cover_the_page_once(dim):
    for is_v in (0, 1):
        assert np.array_equal(np.sort(OA._place(dim, is_v).ravel()), np.arange(64 * dim))


def test_page_exponent_is_the_smallest():
    for a in (1e-30, 0.1, 1.0, 447.9, 448.0, 448.1, 896.0, 1e30):
        e = OA.page_exponent(np.float32(a))
        assert np.float64(np.float32(a)) <= 448.0 * 2.0 ** e
        assert np.float64(np.float32(a)) > 448.0 * 2.0 ** (e - 1)
    assert OA.page_exponent(0.0) == -110


def test_cache_append_grows_the_scale_and_keeps_the_rest():
    rng = np.random.default_rng(2)
    dim = 64
    c = OA.new_cache(3, 2, dim, fill=0x3C)
    table = np.array([[2, 0]])
    first, big = _bits(rng, 10, 2 * dim), _bits(rng, 60, 2 * dim, scale=500.0)
    OA.kv_write(c, first, first, table, np.array([0, 10]), np.array([0]))
    v0, _ = OA.kv_values(c, table[0], 10, 1, 0)
    x0 = bf16_bits_to_f32(first).reshape(10, 2, dim)[:, 1]
    assert np.all(np.abs(v0 - x0) <= np.abs(x0) * 2.0 ** -4 + 2.0 ** -10 * np.abs(x0).max())
    OA.kv_write(c, big, big, table, np.array([0, 60]), np.array([10]))
    v1, ok = OA.kv_values(c, table[0], 70, 1, 1)
    assert ok.all()
    x1 = bf16_bits_to_f32(big).reshape(60, 2, dim)[:, 1]
    top = np.abs(x1[:54]).max()
    assert np.all(np.abs(v1[10:64] - x1[:54]) <= np.abs(x1[:54]) * 2.0 ** -4 + top * 2.0 ** -18)
    # the earlier tokens lost only what the new scale's smallest step cannot hold
    assert np.all(np.abs(v1[:10] - v0) <= 448 * 2.0 ** (int(c["vs"][2, 1]) - 127) * 2.0 ** -18)
    # untouched: page 1 and the slots behind the last token
    assert np.all(c["kc"][1] == 0x3C) and np.all(c["ks"][1] == 0x3C)
    assert np.all(c["vc"][0][:, OA._place(dim, 1)[6:]] == 0x3C)
    # codes that stay normal keep their value exactly when the scale doubles
    assert np.all(e4m3_decode(np.array([0x10], np.uint8)) * 0.5 == e4m3_decode(np.array([8], np.uint8)))


def test_attention_against_closed_forms():
    rng = np.random.default_rng(3)
    dim = 64
    c = OA.new_cache(4, 1, dim)
    kv = _bits(rng, 100, dim)
    table = np.array([[3, 1]])
    OA.kv_write(c, kv, kv, table, np.array([0, 100]), np.array([0]))
    v, _ = OA.kv_values(c, table[0], 100, 0, 1)
    cu, ln = np.array([0, 3]), np.array([100])
    z = OA.attention(np.zeros((3, 2, dim)), c, table, cu, ln, 0.125, False)   # equal weights
    assert np.allclose(z["O"], v.mean(0)) and np.allclose(z["lse"], np.log(100))
    q = rng.standard_normal((3, 2, dim))
    a = OA.attention(q, c, table, cu, ln, 0.125, True)
    # the causal row i is the plain attention over its own prefix
    for i in range(3):
        one = OA.attention(q[i:i + 1], c, table, np.array([0, 1]), np.array([98 + i]), 0.125, False)
        assert np.allclose(a["O"][i], one["O"][0]) and np.allclose(a["lse"][i], one["lse"][0])
    # more rows than tokens: the first rows see nothing
    e = OA.attention(q, c, table, cu, np.array([1]), 0.125, True)
    assert np.all(e["O"][:2] == 0) and np.all(np.isneginf(e["lse"][:2]))
    assert np.allclose(e["O"][2], v[0])
    # a missing page is masked
    m = OA.attention(q, c, np.array([[3, 9]]), cu, ln, 0.125, False)
    f = OA.attention(q, c, table, cu, np.array([64]), 0.125, False)
    assert np.allclose(m["O"], f["O"])
