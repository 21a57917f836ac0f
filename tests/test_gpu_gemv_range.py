"""GPU tests of svdq_w4a16_gemv at the ends of fp32's range and of the branch's 24 bits: what the float64
formula gives is finite, exact or infinite there, and so is the result."""
import numpy as np
import pytest

from oracle.formats import bf16_bits_to_f32, bf16_rne
from tests.gpu_common import dev, dev_bf16, torch_mod
from tests.test_gpu_gemv import FMTS, L, run  # noqa: F401

pytestmark = pytest.mark.gpu


SIZES = [(f, 1e35, 1.0) for f in FMTS] + [(f, 1e36, 1.0) for f in FMTS]   # (int4's scales are fp16)
SIZES += [(f, *s) for f in ("nvfp4", "mxfp4") for s in ((1e36, 1e-20), (1e-33, 1e18), (1e4, 1e32))]


@pytest.mark.parametrize("fmt,size,spread", SIZES)
@pytest.mark.parametrize("r", [0, 16])
def test_results_at_the_ends_of_the_range(L, fmt, r, size, spread):  # noqa: F811
    """Results up to 1e37 from rows and weights of any size: no sum on the way is infinite where the products
    and their sums are not (NVFP4's tensor scale is 2e-5 of the weight's and smaller)."""
    rng = np.random.default_rng(31)
    M, N, K = 18, 40, 768
    X = bf16_rne((rng.standard_normal((M, K)) * size).astype(np.float32))
    got = run(L, fmt, M, N, K, r, X=X, spread=spread)
    assert np.isfinite(got).all() and np.abs(got).max() > 0.1 * size * min(spread, 1.0)


def plain_weight(L, fmt, codes, r, up):  # noqa: F811
    """A prepared weight of these codes, all its scales 1."""
    N, K = codes.shape[0], 2 * codes.shape[1]
    block = dict(nvfp4=16, int4=64, mxfp4=32)[fmt]
    if fmt == "int4":
        scales = np.ones((N, K // block), np.float16)
    else:
        scales = np.full((N, K // block), 0x38 if fmt == "nvfp4" else 127, np.uint8)
    code = dict(nvfp4=L.NVFP4, int4=L.INT4_G64, mxfp4=L.MXFP4)[fmt]
    return L.PreparedWeight(code, N, K, r, dev(codes), dev(scales),
                            dev(np.ones(1, np.float32)) if fmt == "nvfp4" else None, dev_bf16(bf16_rne(up)))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 17, 64])
@pytest.mark.parametrize("r", [8, 32, 128])
def test_the_branch_keeps_24_bits(L, fmt, M, r):  # noqa: F811
    """Outputs that are the last eight of D's 24 bits: rank 2 i is a·2^16 + b·2^8 + c, rank 2 i + 1 the same
    without c, and the up factor takes their difference.  Every sum on the way is a whole number of the
    row's power of two below 2^24 of it, so the result is exact."""
    torch = torch_mod()
    rng = np.random.default_rng(32)
    N, K = 2 * r + 3, 1536
    a, b, c = (2 * rng.integers(64, 128, r // 2) + 1 for _ in range(3))
    down = np.zeros((r, K), np.float32)
    down[0::2, 5], down[0::2, 600], down[0::2, 1100] = a * 65536.0, b * 256.0, c
    down[1::2, 5], down[1::2, 600] = a * 65536.0, b * 256.0
    up = np.zeros((N, r), np.float32)
    pair, u = rng.integers(0, r // 2, N), 2.0 ** rng.integers(-4, 5, N)
    pair[:r // 2] = np.arange(r // 2)
    up[np.arange(N), 2 * pair], up[np.arange(N), 2 * pair + 1] = u, -u
    X = np.zeros((M, K), np.float32)
    size = 2.0 ** rng.integers(-20, 21, M)
    X[:, [5, 600, 1100]] = size[:, None]
    pw = plain_weight(L, fmt, np.zeros((N, K // 2), np.uint8), r, up)
    Y = L.gemv(dev_bf16(bf16_rne(X)), pw, None, dev_bf16(bf16_rne(down)))
    torch.cuda.synchronize()
    assert np.array_equal(Y.float().cpu().numpy(), size[:, None] * (c[pair] * u)[None])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_the_branch_up_to_the_largest_number(L, fmt, sign):  # noqa: F811
    """D between bf16's largest number and fp32's: 2^128 − 2^118."""
    torch = torch_mod()
    K, N, r = 512, 20, 8
    top = bf16_bits_to_f32(np.array([0x7F7F], np.uint16))[0]
    down = np.zeros((r, K), np.float32)
    down[3, [7, 300]] = 1.0
    X = np.zeros((2, K), np.float32)
    X[0, 7], X[0, 300] = sign * top, sign * 1.5 * 2.0 ** 119
    X[1, 7] = 1.0
    up = np.zeros((N, r), np.float32)
    up[:, 3] = 2.0 ** -np.arange(1, N + 1)
    Y = L.gemv(dev_bf16(bf16_rne(X)), plain_weight(L, fmt, np.zeros((N, K // 2), np.uint8), r, up), None,
               dev_bf16(bf16_rne(down)))
    torch.cuda.synchronize()
    want = np.array([sign * (2.0 ** 128 - 2.0 ** 118), 1.0])[:, None] * up[:, 3].astype(np.float64)
    assert np.all(np.abs(Y.float().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [2, 20, 50])
@pytest.mark.parametrize("r", [0, 8, 64, 128])
@pytest.mark.parametrize("smooth", [False, True])
def test_an_infinity_among_positive_numbers_is_the_result(L, fmt, M, r, smooth):  # noqa: F811
    """Every weight, factor and channel positive: the row of the infinity is infinite, not NaN, and the
    others are what they are without it."""
    torch = torch_mod()
    rng = np.random.default_rng(33)
    N, K = 40, 1024
    codes = (rng.integers(1, 8, (N, K // 2)) | rng.integers(1, 8, (N, K // 2)) << 4).astype(np.uint8)
    X = np.exp(rng.standard_normal((M, K))).astype(np.float32)
    down, up = (np.exp(rng.standard_normal(s)).astype(np.float32) for s in ((r, K), (N, r)))
    lam = dev(np.exp(rng.standard_normal(K)).astype(np.float32)) if smooth else None
    pw = plain_weight(L, fmt, codes, r, up)
    d = dev_bf16(bf16_rne(down)) if r else None
    clean = L.gemv(dev_bf16(bf16_rne(X)), pw, lam, d)
    for at in (0, 129, 700, K - 1):
        Z = X.copy()
        Z[M - 1, at] = np.inf
        Y = L.gemv(dev_bf16(bf16_rne(Z)), pw, lam, d)
        torch.cuda.synchronize()
        assert torch.equal(Y[:M - 1], clean[:M - 1]) and torch.isposinf(Y[M - 1]).all(), at
