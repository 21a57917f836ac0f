"""GPU parity of svdq_qk_norm_rope against the float64 oracle.  Tolerance: half a bf16 step of the
result (2^-8 relative) plus fp32: the sum of at most 256 squares in chains of 16 and 4 exchanges, 20
roundings of 2^-24 (half of that reaches the root), the root and two products, 2^-22 together; and the
rotation of test_gpu_rope.py, 2^-20·(|u| + |v|) of the normed pair.  Together below 2^-19·(|u| + |v|)."""
import numpy as np
import pytest

from oracle import tokens as OT
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


def _pair_sums(z, axes, inter):
    rot = sum(axes)
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    mag = np.abs(z).copy()
    mag[:, :, a] = mag[:, :, b] = np.abs(z[:, :, a]) + np.abs(z[:, :, b])
    return mag


def _run(L, M, Hq, Hk, dim, axes, inter, pos=None, pad=0, tail=0, in_place=False, seed=0, spread=None,
         gammas=(True, True), eps=1e-6, x=None):
    torch = torch_mod()
    from w4a4_quantized_dit_amd import _lib
    rng = np.random.default_rng(seed)
    H = Hq + Hk
    wide = (H + tail) * dim + pad
    if x is None:
        x = rng.standard_normal((M, wide)) * (1.0 if spread is None else spread)
    bits = bf16_rne(x.astype(np.float32))
    if pos is None:
        pos = rng.integers(-50, 5000, (M, len(axes)))
    pos = pos.astype(np.int32)
    g = [bf16_rne((1 + 0.3 * rng.standard_normal(dim)).astype(np.float32)) if w else None for w in gammas]
    freq = _lib.svdq_rope_frequencies(axes, 10000.0)
    buf = dev_bf16(bits)
    X = buf[:, :H * dim]
    Y = L.qk_norm_rope(X, dev(pos), dev(freq), axes, dim, Hq, *[dev_bf16(v) if v is not None else None
                                                               for v in g],
                       eps=eps, interleaved=inter, out=X if in_place else None)
    torch.cuda.synchronize()
    xf = bf16_bits_to_f32(bits[:, :H * dim]).reshape(M, H, dim)
    want, z = OT.qk_norm_rope(xf, Hq, g[0], g[1], eps, pos, freq, axes, inter)
    got = bf16_bits_to_f32(host_bits(Y.contiguous())).reshape(M, H, dim).astype(np.float64)
    bad = np.abs(got - want) > 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * _pair_sums(z, axes, inter) + 1e-38
    assert not (bad & ~np.isnan(want)).any()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    if in_place:   # the other columns of the packed rows stay as they were
        assert np.array_equal(host_bits(buf)[:, H * dim:], bits[:, H * dim:])
    else:
        assert np.array_equal(host_bits(buf), bits)


@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("dim,axes", [(128, [44, 42, 42]), (128, [16, 56, 56]), (64, [16, 24, 24]),
                                      (128, [64]), (16, [16]), (32, [32]), (96, [32, 32, 16]),
                                      (48, [0, 16]), (256, [64, 64, 64, 64]), (240, [100, 60, 64]),
                                      (112, [96])])
def test_axes_and_layouts(L, dim, axes, inter):
    _run(L, 13, 4, 3, dim, axes, inter)


@pytest.mark.parametrize("M,Hq,Hk", [(1, 1, 0), (1, 0, 1), (1, 40, 8), (3, 1, 2), (32, 40, 8), (700, 16, 1),
                                     (5000, 2, 1), (2, 150, 50), (21000, 32, 18), (1, 500, 3)])
@pytest.mark.parametrize("inter", [True, False])
def test_row_and_head_counts(L, M, Hq, Hk, inter):
    _run(L, M, Hq, Hk, 128, [44, 42, 42], inter, seed=M)


@pytest.mark.parametrize("gammas", [(True, False), (False, True), (False, False)])
def test_without_weights(L, gammas):
    _run(L, 9, 3, 2, 64, [16, 24, 24], True, gammas=gammas)


@pytest.mark.parametrize("inter", [True, False])
def test_in_place_inside_packed_rows(L, inter):
    _run(L, 77, 4, 2, 64, [16, 24, 24], inter, tail=3, pad=8, in_place=True)
    _run(L, 77, 4, 2, 64, [24, 24], inter, tail=3, in_place=True)
    _run(L, 3000, 4, 2, 128, [64, 64], inter, tail=2, in_place=True)


def test_far_positions_keep_their_angle(L):
    top = 2 ** 31 - 1
    pos = np.array([[top, -top - 1, 0], [top - 7, 12345678, -99999999], [2 ** 24 + 1, 2 ** 25 + 3, 1]])
    _run(L, 3, 2, 2, 128, [44, 42, 42], True, pos=pos)
    _run(L, 3, 2, 2, 128, [44, 42, 42], False, pos=pos)


@pytest.mark.parametrize("dim", [64, 96, 128])
def test_sizes_from_the_smallest_to_the_largest(L, dim):
    """Heads of zeros, of subnormals, of squares below and past fp32's range, side by side in a wave."""
    size = np.array([0.0, 1e-39, 1e-30, 1e-19, 1e-10, 1.0, 1e10, 1e18, 3e19, 1e30, 2e37, 1e38])
    rng = np.random.default_rng(3)
    x = rng.uniform(-1, 1, (4, 12, dim)) * size[None, :, None]
    _run(L, 4, 7, 5, dim, [48], False, x=x.reshape(4, -1))
    _run(L, 4, 7, 5, dim, [48], True, x=x.reshape(4, -1), eps=1e-12)
    _run(L, 4, 7, 5, dim, [48], True, x=np.full((4, 12 * dim), 3.3e38))
    _run(L, 4, 7, 5, dim, [48], True, x=1e-3 * x.reshape(4, -1).clip(-1, 1), eps=1e-30)
    _run(L, 4, 7, 5, dim, [48], True, x=x.reshape(4, -1).clip(-1, 1), eps=1e5)


def test_infinities_and_nan_stay_in_their_head(L):
    rng = np.random.default_rng(4)
    x = rng.standard_normal((3, 6, 64))
    x[0, 1, 5], x[1, 2, 60], x[2, 5, 0], x[2, 0, 33] = np.inf, np.nan, -np.inf, np.nan
    with np.errstate(invalid="ignore"):
        _run(L, 3, 4, 2, 64, [16, 24, 24], True, x=x.reshape(3, -1))
        _run(L, 3, 4, 2, 64, [48], False, x=x.reshape(3, -1))


def test_agrees_with_the_rotation_of_normed_rows(L):
    """With unit weights on rows of unit mean square it is the rotation alone."""
    torch = torch_mod()
    rng = np.random.default_rng(5)
    x = rng.choice([-1.0, 1.0], (50, 6 * 64)).astype(np.float32)
    pos = dev(rng.integers(0, 999, (50, 3)).astype(np.int32))
    freq = L.rope_frequencies([16, 24, 24])
    X = dev_bf16(bf16_rne(x))
    a = L.qk_norm_rope(X, pos, freq, [16, 24, 24], 64, 4, None, None, eps=1e-30)
    b = L.rope(X, pos, freq, [16, 24, 24], 64)
    torch.cuda.synchronize()
    # the root of 1 is 1 to 2^-22: at most the other neighbour of a value at a rounding border
    assert torch.all((a.float() - b.float()).abs() <= 2.0 ** -7 * b.float().abs())
    assert (a != b).float().mean() < 0.01


def test_more_rows_than_blocks(L):
    """2^21 + 5 rows: the blocks take a second row each."""
    torch = torch_mod()
    from w4a4_quantized_dit_amd import _lib
    M, n = (1 << 21) + 5, 64
    freq = _lib.svdq_rope_frequencies([16], 1000.0)
    g = torch.Generator(device="cuda").manual_seed(3)
    X = torch.randn(M, 32, generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.randint(-1000, 1000, (M, 1), generator=g, device="cuda", dtype=torch.int32)
    Y = L.qk_norm_rope(X, pos, dev(freq), [16], 16, 1, None, None)
    torch.cuda.synchronize()
    for rows in (slice(0, n), slice(M - n, M)):
        x = X[rows].float().cpu().numpy().reshape(n, 2, 16)
        want, z = OT.qk_norm_rope(x, 1, None, None, 1e-6, pos[rows].cpu().numpy(), freq, [16], True)
        got = Y[rows].float().cpu().numpy().reshape(n, 2, 16)
        assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * _pair_sums(z, [16], True))


@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("M,Hq,Hk,dim,axes", [(1537, 2, 1, 64, [64]), (3085, 5, 2, 96, [32, 32, 16]),
                                              (6151, 1, 0, 48, [0, 16]), (12293, 1, 1, 64, [16, 24, 24]),
                                              (24580, 1, 0, 16, [16]), (3073, 20, 1, 128, [64]),
                                              (12291, 1, 1, 240, [100, 60, 64])])
def test_several_rows_a_block(L, M, Hq, Hk, dim, axes, inter):
    """Many rows of few heads, the last block's rows fewer than the others'."""
    _run(L, M, Hq, Hk, dim, axes, inter, seed=M, tail=1, pad=8, in_place=inter)


@pytest.mark.parametrize("M,heads,dim", [((1 << 20) + 21, 2, 16), ((1 << 16) + 5, 513, 16)])
def test_more_blocks_than_a_grid_has(L, M, heads, dim):
    """The blocks take a second turn, of several rows or of one."""
    torch = torch_mod()
    from w4a4_quantized_dit_amd import _lib
    n = 40
    freq = _lib.svdq_rope_frequencies([16], 1000.0)
    g = torch.Generator(device="cuda").manual_seed(3)
    X = torch.randn(M, heads * dim, generator=g, device="cuda", dtype=torch.bfloat16)
    pos = torch.randint(-1000, 1000, (M, 1), generator=g, device="cuda", dtype=torch.int32)
    Y = L.qk_norm_rope(X, pos, dev(freq), [16], dim, 1, None, None)
    torch.cuda.synchronize()
    for rows in (slice(0, n), slice(M - n, M)):
        x = X[rows].float().cpu().numpy().reshape(n, heads, dim)
        want, z = OT.qk_norm_rope(x, 1, None, None, 1e-6, pos[rows].cpu().numpy(), freq, [16], True)
        got = Y[rows].float().cpu().numpy().reshape(n, heads, dim)
        assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * _pair_sums(z, [16], True))
