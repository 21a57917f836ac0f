"""GPU parity of svdq_rope_axes against the float64 oracle.  Tolerance: half a bf16 step of the
result (2^-8 relative) plus the fp32 rotation: cos and sin of the reduced fraction of a turn within
2^-22 (two units in the last place) and 2^-23 from rounding the fraction (2π·2^-26), the products
and their sum within 2^-23 each — together below 2^-20·(|u| + |v|)."""
import numpy as np
import pytest

from oracle import attention as OA
from oracle.formats import bf16_bits_to_f32, bf16_rne
from tests.gpu_common import dev, dev_bf16, host_bits, torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from w4a4_quantized_dit_amd import _lib, layer
    _lib.load()
    return layer


def _run(L, M, heads, dim, axes, inter, inverse, pos=None, pad=0, tail=0, in_place=False, seed=0):
    torch = torch_mod()
    rng = np.random.default_rng(seed)
    wide = (heads + tail) * dim + pad
    bits = bf16_rne(rng.standard_normal((M, wide)).astype(np.float32))
    if pos is None:
        pos = rng.integers(-50, 5000, (M, len(axes)))
    pos = pos.astype(np.int32)
    from w4a4_quantized_dit_amd import _lib
    freq = _lib.svdq_rope_frequencies(axes, 10000.0)
    buf = dev_bf16(bits)
    X = buf[:, :heads * dim]
    Y = L.rope(X, dev(pos), dev(freq), axes, dim, interleaved=inter, inverse=inverse,
               out=X if in_place else None)
    torch.cuda.synchronize()
    x = bf16_bits_to_f32(bits[:, :heads * dim]).reshape(M, heads, dim)
    want = OA.rope(x, pos, freq, axes, inter, inverse)
    got = bf16_bits_to_f32(host_bits(Y.contiguous())).reshape(M, heads, dim).astype(np.float64)
    rot = sum(axes)
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    mag = np.zeros_like(want)
    mag[:, :, a] = mag[:, :, b] = np.abs(x[:, :, a].astype(np.float64)) + np.abs(x[:, :, b])
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * mag)
    assert np.array_equal(got[..., rot:], x[..., rot:])
    if in_place:   # the other columns of the packed rows stay as they were
        assert np.array_equal(host_bits(buf)[:, heads * dim:], bits[:, heads * dim:])
    else:
        assert np.array_equal(host_bits(buf), bits)


@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("inverse", [True, False])
@pytest.mark.parametrize("dim,axes", [(128, [44, 42, 42]), (128, [16, 56, 56]), (64, [16, 24, 24]),
                                      (128, [64]), (16, [16]), (96, [32, 32, 16]), (48, [0, 16]),
                                      (256, [64, 64, 64, 64]), (240, [100, 60, 64])])
def test_axes_and_layouts(L, dim, axes, inter, inverse):
    _run(L, 13, 5, dim, axes, inter, inverse)


@pytest.mark.parametrize("M,heads", [(1, 1), (1, 80), (3, 2), (700, 17), (5000, 3), (2, 200), (21000, 50)])
@pytest.mark.parametrize("inter", [True, False])
def test_row_and_head_counts(L, M, heads, inter):
    _run(L, M, heads, 128, [44, 42, 42], inter, False, seed=M)


@pytest.mark.parametrize("inter", [True, False])
def test_in_place_inside_packed_rows(L, inter):
    _run(L, 77, 6, 64, [16, 24, 24], inter, False, tail=3, pad=8, in_place=True)
    _run(L, 77, 6, 64, [24, 24], inter, False, tail=3, in_place=True)


def test_far_positions_keep_their_angle(L):
    """Positions near ±2^31: θ is reduced in float64, where it is good to 2^31·2^-52 radians."""
    top = 2 ** 31 - 1
    pos = np.array([[top, -top - 1, 0], [top - 7, 12345678, -99999999], [2 ** 24 + 1, 2 ** 25 + 3, 1]])
    _run(L, 3, 4, 128, [44, 42, 42], True, False, pos=pos)
    _run(L, 3, 4, 128, [44, 42, 42], False, True, pos=pos)


def test_inverse_is_the_gradient(L):
    """d(rope(x)·w)/dx = rope(w, inverse), checked against differences of the oracle."""
    torch = torch_mod()
    rng = np.random.default_rng(9)
    axes, freq = [16, 24, 24], None
    from w4a4_quantized_dit_amd import _lib
    freq = _lib.svdq_rope_frequencies(axes, 100.0)
    pos = rng.integers(0, 50, (2, 3)).astype(np.int32)
    x, w = rng.standard_normal((2, 2, 1, 64))
    wb = bf16_rne(w.astype(np.float32).reshape(2, 64))
    w = bf16_bits_to_f32(wb).reshape(2, 1, 64).astype(np.float64)
    g = L.rope(dev_bf16(wb), dev(pos), dev(freq), axes, 64, inverse=True)
    torch.cuda.synchronize()
    got = bf16_bits_to_f32(host_bits(g)).astype(np.float64)
    f = lambda v: np.sum(OA.rope(v, pos, freq, axes, True, False) * w)  # noqa: E731
    for i in range(2):
        for j in range(64):
            e = np.zeros_like(x)
            e[i, 0, j] = 0.5
            diff = f(x + e) - f(x - e)          # linear: exact up to float64 rounding
            assert abs(got[i, j] - diff) <= 2.0 ** -8 * abs(diff) + 2.0 ** -20 * 8


def test_more_rows_than_blocks(L):
    """2^21 + 5 rows: the blocks take a second row each."""
    torch = torch_mod()
    from w4a4_quantized_dit_amd import _lib
    M, n = (1 << 21) + 5, 64
    freq = _lib.svdq_rope_frequencies([16], 1000.0)
    g = torch.Generator(device="cuda").manual_seed(3)
    X = torch.randn(M, 16, generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.randint(-1000, 1000, (M, 1), generator=g, device="cuda", dtype=torch.int32)
    Y = L.rope(X, pos, dev(freq), [16], 16)
    torch.cuda.synchronize()
    for rows in (slice(0, n), slice(M - n, M)):
        x = X[rows].float().cpu().numpy().reshape(n, 1, 16).astype(np.float64)
        want = OA.rope(x, pos[rows].cpu().numpy(), freq, [16], True, False)
        got = Y[rows].float().cpu().numpy().reshape(n, 1, 16)
        mag = np.repeat(np.abs(x[..., 0::2]) + np.abs(x[..., 1::2]), 2, axis=-1)
        assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * mag)
