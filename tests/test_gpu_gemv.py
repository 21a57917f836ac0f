"""GPU parity of svdq_w4a16_gemv against the float64 oracle.  Tolerance, per element, A the sum of the
magnitudes of its products: half a bf16 step of the result, 2^-8·|y|; the products are exact in fp32
(x̂ has 8 bits, a weight value 6, 3 before its scale) and every addition loses at most a whole step,
2^-23, of a partial sum: at most K products in a row where K is not split, fewer where it is (and a
group of 64 is multiplied by its scale); the low-rank branch adds K of its own, r products with the up
factor whose D is taken to 16 bits and more in two bf16 (2^-17)."""
import numpy as np
import pytest

from oracle import layer as OL, tokens as OT
from oracle.formats import bf16_bits_to_f32, bf16_rne
from tests.gpu_common import dev, dev_bf16, host_bits, torch_mod

pytestmark = pytest.mark.gpu
FMTS = ["nvfp4", "int4", "mxfp4"]


@pytest.fixture(scope="module")
def L():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from w4a4_quantized_dit_amd import _lib, layer
    _lib.load()
    return layer


def case(rng, fmt, N, K, r, smooth=True, spread=1.0):
    """Oracle weight and its device form."""
    W = bf16_rne((rng.standard_normal((N, K)) * K ** -0.5 * spread).astype(np.float32))
    lam = np.exp(0.5 * rng.standard_normal(K)).astype(np.float32) if smooth else None
    down = bf16_rne((0.05 * rng.standard_normal((r, K))).astype(np.float32)) if r else None
    up = bf16_rne((0.1 * rng.standard_normal((N, r))).astype(np.float32)) if r else None
    one = np.ones(K, np.float32)
    wt = OL.prepare_weight(W, lam if smooth else one, down if r else np.zeros((0, K), np.uint16),
                           up if r else np.zeros((N, 0), np.uint16), fmt)
    return wt, lam, down, up


def device_weight(L, fmt, wt, up, N, K, r):
    code = dict(nvfp4=L.NVFP4, int4=L.INT4_G64, mxfp4=L.MXFP4)[fmt]
    g = dev(np.array([wt["g"]], np.float32)) if fmt == "nvfp4" else None
    return L.PreparedWeight(code, N, K, r, dev(wt["codes"]), dev(wt["scales"]), g,
                            dev_bf16(up) if r else None)


def tolerance(y, a, K, r):
    steps = K + 32 + (K + 64 + r if r else 0)
    return 2.0 ** -8 * np.abs(y) + steps * 2.0 ** -23 * a + 1e-37


def run(L, fmt, M, N, K, r, smooth=True, pad=0, seed=0, X=None, ypad=0, spread=1.0):
    torch = torch_mod()
    rng = np.random.default_rng(seed)
    wt, lam, down, up = case(rng, fmt, N, K, r, smooth, spread)
    if X is None:
        X = bf16_rne((rng.standard_normal((M, K)) * np.exp(0.75 * rng.standard_normal(K))).astype(np.float32))
    pw = device_weight(L, fmt, wt, up, N, K, r)
    wide = dev_bf16(np.concatenate([X, np.full((M, pad), 0x7FC0, np.uint16)], 1))
    out = torch.full((M + 1, N + ypad), 7.0, dtype=torch.bfloat16, device="cuda")
    Y = L.gemv(wide[:, :K], pw, dev(lam) if smooth else None, dev_bf16(down) if r else None,
               out=out[:M, :N])
    torch.cuda.synchronize()
    y, a = OT.gemv(X, lam, down, up, OT.weight_values(wt["codes"], wt["scales"], wt["g"], fmt))
    got = Y.float().cpu().numpy().astype(np.float64)
    bad = np.abs(got - y) > tolerance(y, a, K, r)
    assert not bad.any(), (int(bad.sum()), np.abs(got - y)[bad].max(), np.argwhere(bad)[:5].tolist())
    assert torch.all(out[M:] == 7.0) and torch.all(out[:, N:] == 7.0)
    return got


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 32, 33, 48, 49, 64])
def test_rows(L, fmt, M):
    run(L, fmt, M, 40, 512, 16, seed=M)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("N", [1, 7, 8, 15, 16, 17, 31, 32, 33, 250])
@pytest.mark.parametrize("M", [1, 20])
def test_outputs(L, fmt, N, M):
    run(L, fmt, M, N, 256, 8, seed=N, ypad=3)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("K", [256, 768, 1024, 1280, 2304, 5120, 13824])
@pytest.mark.parametrize("r", [0, 32])
def test_channels(L, fmt, K, r):
    run(L, fmt, 3, 24, K, r, seed=K)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("r", [0, 8, 24, 64, 120, 128])
@pytest.mark.parametrize("smooth", [False, True])
@pytest.mark.parametrize("M", [1, 40])
def test_ranks(L, fmt, r, smooth, M):
    run(L, fmt, M, 33, 768, r, smooth=smooth, seed=r)


@pytest.mark.parametrize("fmt", FMTS)
def test_strided_rows(L, fmt):
    run(L, fmt, 5, 40, 512, 16, pad=8)
    run(L, fmt, 40, 40, 512, 0, smooth=False, pad=264, ypad=1)
    run(L, fmt, 1, 40, 512, 0, smooth=False, pad=8)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 20, 64])
def test_wide_outputs(L, fmt, M):
    """Enough outputs that a block takes two tiles, the last one ragged."""
    run(L, fmt, M, 16384 + 24, 256, 8)


@pytest.mark.parametrize("fmt", FMTS)
def test_every_code_and_place(L, fmt):
    """Unit rows: output n of row k is the weight w[n, k] itself, every channel in turn."""
    torch = torch_mod()
    rng = np.random.default_rng(5)
    N, K = 17, 256
    wt, _, _, _ = case(rng, fmt, N, K, 0, False)
    wt["codes"] = rng.integers(0, 256, wt["codes"].shape).astype(np.uint8)
    pw = device_weight(L, fmt, wt, None, N, K, 0)
    w = OT.weight_values(wt["codes"], wt["scales"], wt["g"], fmt)
    for k0 in range(0, K, 64):
        X = np.zeros((64, K), np.float32)
        X[np.arange(64), k0 + np.arange(64)] = 1.0
        Y = L.gemv(dev_bf16(bf16_rne(X)), pw, None, None)
        torch.cuda.synchronize()
        got = Y.float().cpu().numpy().T
        # one product, one rounding (and with a tensor scale one more in fp32)
        assert np.all(np.abs(got - w[:, k0:k0 + 64]) <= 2.0 ** -8 * (1 + 2.0 ** -15) * np.abs(w[:, k0:k0 + 64]))


@pytest.mark.parametrize("fmt", FMTS)
def test_extremes(L, fmt):
    """Zero weights and rows; rows of very different sizes; infinities and NaN stay in their row."""
    torch = torch_mod()
    rng = np.random.default_rng(6)
    N, K = 24, 512
    X = (rng.standard_normal((6, K)) * np.array([1e-30, 1.0, 1e30, 0.0, 1.0, 1.0])[:, None])
    got = run(L, fmt, 6, N, K, 16, X=bf16_rne(X.astype(np.float32)))
    assert np.all(got[3] == 0)
    assert np.all(run(L, fmt, 3, N, K, 0, spread=0.0) == 0)
    wt, lam, down, up = case(rng, fmt, N, K, 16)
    pw = device_weight(L, fmt, wt, up, N, K, 16)
    X[4, 100], X[5, 7] = np.inf, np.nan
    Y = L.gemv(dev_bf16(bf16_rne(X.astype(np.float32))), pw, dev(lam), dev_bf16(down))
    clean = L.gemv(dev_bf16(bf16_rne(X[:4].astype(np.float32))), pw, dev(lam), dev_bf16(down))
    torch.cuda.synchronize()
    assert torch.equal(Y[:4], clean) and not torch.isfinite(Y[4:]).any()


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_do_not_depend_on_each_other(L, fmt):
    """A row's result is the same bits alone and among others: the sums' order is fixed."""
    torch = torch_mod()
    rng = np.random.default_rng(7)
    N, K = 100, 1280
    wt, lam, down, up = case(rng, fmt, N, K, 32)
    pw = device_weight(L, fmt, wt, up, N, K, 32)
    X = dev_bf16(bf16_rne(rng.standard_normal((64, K)).astype(np.float32)))
    whole = L.gemv(X, pw, dev(lam), dev_bf16(down))
    for rows in ([0], [63], list(range(3, 20)), list(range(30))):
        part = L.gemv(X[rows], pw, dev(lam), dev_bf16(down))
        torch.cuda.synchronize()
        assert torch.equal(part, whole[rows])


@pytest.mark.parametrize("fmt", FMTS)
def test_prepared_weight_of_the_library(L, fmt):
    """The weight that prepare_weight makes, beside forward() with its quantised activations, and
    leading dimensions."""
    torch = torch_mod()
    rng = np.random.default_rng(8)
    M, N, K, r = 12, 256, 512, 16
    _, lam, down, up = case(rng, fmt, 8, K, r)
    up = bf16_rne((0.1 * rng.standard_normal((N, r))).astype(np.float32))
    W = bf16_rne((rng.standard_normal((N, K)) * K ** -0.5).astype(np.float32))
    code = dict(nvfp4=L.NVFP4, int4=L.INT4_G64, mxfp4=L.MXFP4)[fmt]
    pw = L.prepare_weight(dev_bf16(W), dev(lam), dev_bf16(down), dev_bf16(up), code)
    X = dev_bf16(bf16_rne(rng.standard_normal((3, 4, K)).astype(np.float32)))
    Y = L.gemv(X, pw, dev(lam), dev_bf16(down))
    full = L.forward(X, pw, None, dev(lam), dev_bf16(down))
    torch.cuda.synchronize()
    assert Y.shape == full.shape == (3, 4, N)
    x = X.float().cpu().numpy().reshape(M, K).astype(np.float64)
    ref = x @ bf16_bits_to_f32(W).astype(np.float64).T
    err = lambda t: np.linalg.norm(t.float().cpu().numpy().reshape(M, N) - ref) / np.linalg.norm(ref)  # noqa: E731
    assert err(Y) < err(full)              # without the activations' error
    w = OT.weight_values(pw.codes.cpu().numpy(), pw.scales.cpu().numpy(),
                         pw.g.cpu().numpy()[0] if pw.g is not None else None, fmt)
    y, a = OT.gemv(host_bits(X).reshape(M, K), lam, down, up, w)
    assert np.all(np.abs(Y.float().cpu().numpy().reshape(M, N) - y) <= tolerance(y, a, K, r))


def test_workspace_of_the_caller(L):
    torch = torch_mod()
    from w4a4_quantized_dit_amd import _lib
    rng = np.random.default_rng(9)
    wt, lam, down, up = case(rng, "int4", 40, 512, 16)
    pw = device_weight(L, "int4", wt, up, 40, 512, 16)
    X = dev_bf16(bf16_rne(rng.standard_normal((20, 512)).astype(np.float32)))
    want = L.gemv(X, pw, dev(lam), dev_bf16(down))
    n = _lib.svdq_w4a16_gemv_workspace_bytes(20, 40, 512, 16)
    buf = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    off = (-buf.data_ptr()) % 256
    got = L.gemv(X, pw, dev(lam), dev_bf16(down), workspace=buf[off:off + n])
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert torch.all(buf[:off] == 0xA5) and torch.all(buf[off + n:] == 0xA5)
    assert L.gemv_workspace(20, pw).numel() == n


def test_rows_far_apart(L):
    """The largest leading dimension: the last row starts two gigabytes behind the first."""
    torch = torch_mod()
    rng = np.random.default_rng(14)
    N, K, ld = 24, 512, 1 << 24
    wt, lam, down, up = case(rng, "nvfp4", N, K, 8)
    pw = device_weight(L, "nvfp4", wt, up, N, K, 8)
    X = dev_bf16(bf16_rne(rng.standard_normal((64, K)).astype(np.float32)))
    wide = torch.empty(64, ld, dtype=torch.bfloat16, device="cuda")[:, :K]
    wide.copy_(X)
    a, b = L.gemv(wide, pw, dev(lam), dev_bf16(down)), L.gemv(X, pw, dev(lam), dev_bf16(down))
    torch.cuda.synchronize()
    assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", FMTS)
def test_the_longest_rows(L, fmt):
    """K of 2^22: units in a few channels from the first to the last, in a row each and all in one; every
    partial sum is of at most nine values, and the factors' sums of units are exact."""
    torch = torch_mod()
    rng = np.random.default_rng(15)
    N, K, r, M = 17, 1 << 22, 128, 10
    at = np.array([0, 255, 256, 4097, 1 << 20, (1 << 21) + 77, 3 << 20, K - 257, K - 1])
    block = dict(nvfp4=16, int4=64, mxfp4=32)[fmt]
    codes = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    if fmt == "int4":
        scales = (2.0 ** rng.integers(-9, 3, (N, K // block))).astype(np.float16)
    else:
        scales = rng.integers(0x30, 0x48, (N, K // block)).astype(np.uint8) + np.uint8(80 if fmt == "mxfp4" else 0)
    g = np.float32(0.5) if fmt == "nvfp4" else None
    down = np.zeros((r, K), np.float32)
    down[:, at] = rng.integers(-8, 9, (r, len(at)))
    up = rng.integers(-2, 3, (N, r)).astype(np.float32) / 64
    w = np.stack([OT.weight_values(codes[:, c // 256 * 128:c // 256 * 128 + 128],
                                   scales[:, c // 256 * (256 // block):(c // 256 + 1) * (256 // block)],
                                   g, fmt)[:, c % 256] for c in at], 1)
    x = np.zeros((M, len(at)))
    x[:len(at)] = np.eye(len(at))
    x[-1] = 1.0
    X = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    X[:, torch.as_tensor(at)] = torch.as_tensor(x, dtype=torch.bfloat16, device="cuda")
    code = dict(nvfp4=L.NVFP4, int4=L.INT4_G64, mxfp4=L.MXFP4)[fmt]
    pw = L.PreparedWeight(code, N, K, r, dev(codes), dev(scales), dev(np.array([g])) if g else None,
                          dev_bf16(bf16_rne(up)))
    Y = L.gemv(X, pw, None, dev_bf16(bf16_rne(down)))
    torch.cuda.synchronize()
    D = x @ down[:, at].T.astype(np.float64)
    y, a = x @ w.T + D @ up.T.astype(np.float64), np.abs(x) @ np.abs(w.T) + np.abs(D) @ np.abs(up.T)
    # half a bf16 step, and 9 + 128 additions and the tensor's scale in fp32
    assert np.all(np.abs(Y.float().cpu().numpy() - y) <= 2.0 ** -8 * np.abs(y) + 140 * 2.0 ** -23 * a)


@pytest.mark.parametrize("fmt", FMTS)
def test_small_channels_beside_a_large_one(L, fmt):
    """A channel that the weight ignores beside one up to 2^40 times smaller: NVFP4 and int4 take x̂ in
    fp16 with the largest of 256 channels in [2^14, 2^15), off by less than 2^-24 there, 2^-38 of it."""
    torch = torch_mod()
    rng = np.random.default_rng(16)
    N, K = 40, 512
    wt, _, _, _ = case(rng, fmt, N, K, 0, False)
    wt["codes"][:, 0] &= 0xF0   # channel 0 in the low nibble
    pw = device_weight(L, fmt, wt, None, N, K, 0)
    w = OT.weight_values(wt["codes"], wt["scales"], wt["g"], fmt)
    assert np.all(w[:, 0] == 0)
    v = 1.9921875 * 2.0 ** -np.arange(0, 41)
    X = np.zeros((41, K), np.float32)
    X[:, 0], X[:, 201] = 1.5, v
    Y = L.gemv(dev_bf16(bf16_rne(X)), pw, None, None)
    torch.cuda.synchronize()
    y = v[:, None] * w[:, 201]
    exact = 2.0 ** -8 * np.abs(y) * (1 + 2.0 ** -15)
    lost = 0.0 if fmt == "mxfp4" else np.where(v[:, None] < 2.0 ** -29, 2.0 ** -37 * np.abs(w[:, 201]), 0.0)
    assert np.all(np.abs(Y.float().cpu().numpy() - y) <= exact + lost)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("K", [256, 768, 1024])
@pytest.mark.parametrize("M", [1, 40])
def test_scales_that_are_no_numbers_stay_in_their_output(L, fmt, K, M):
    """Channels end inside a chunk of four pieces: the next row's scales lie where the load goes on.
    (NVFP4's are at most 0x7E, 448, as the library makes them; 0x7F counts on as 480 in this layer.)"""
    torch = torch_mod()
    rng = np.random.default_rng(17)
    N = 21
    wt, _, _, _ = case(rng, fmt, N, K, 0, False)
    X = dev_bf16(bf16_rne(rng.standard_normal((M, K)).astype(np.float32)))
    want = L.gemv(X, device_weight(L, fmt, wt, None, N, K, 0), None, None)
    bad = [1, 6, 16, 20]
    wt["scales"] = wt["scales"].copy()
    wt["scales"][bad] = np.float16(np.nan) if fmt == "int4" else 0x7F if fmt == "nvfp4" else 0xFF
    got = L.gemv(X, device_weight(L, fmt, wt, None, N, K, 0), None, None)
    torch.cuda.synchronize()
    good = [n for n in range(N) if n not in bad]
    assert torch.isnan(got[:, bad]).all() or fmt == "nvfp4"
    assert torch.equal(got[:, good], want[:, good])
