"""GPU parity of svdq_rmsnorm_quant_act: H, codes and scales bit-exact to the oracle (the sum of
squares is exact in fp64 for these inputs, every other step is one IEEE operation), D within the
fp32 accumulation's tolerance (gpu_common)."""
import numpy as np
import pytest

from oracle import attention as OA
from oracle.formats import bf16_rne
from tests.gpu_common import dev, dev_bf16, host_bits, check_d, torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from w4a4_quantized_dit_amd import _lib, layer
    _lib.load()
    return layer


def _case(M, K, r, residual, gamma, smooth, seed=0, pad=0):
    rng = np.random.default_rng(seed)
    f = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    prof = np.exp(0.75 * f(K))
    c = dict(X=bf16_rne(f(M, K + pad) * 0.5), res=bf16_rne(f(M, K + pad) * np.exp(0.5 * f(K + pad)))
             if residual else None, gamma=bf16_rne(1 + 0.2 * f(K)) if gamma else None,
             lam=prof if smooth else None, down=bf16_rne(0.05 * f(r, K)) if r else None)
    return c


def _check(L, c, K, eps=1e-6, in_place=None):
    torch = torch_mod()
    X, res = dev_bf16(c["X"])[:, :K], None
    if c["res"] is not None:
        res = dev_bf16(c["res"])[:, :K]
    out = {None: None, "X": X, "res": res}[in_place]
    want = OA.rmsnorm_quant(c["X"][:, :K], None if res is None else c["res"][:, :K], c["gamma"], eps,
                            c["lam"], c["down"])
    d = lambda v, f: None if v is None else f(v)  # noqa: E731
    codes, scales, D, H = L.norm_quantize_activation(
        X, d(c["gamma"], dev_bf16), d(c["lam"], dev), d(c["down"], dev_bf16), eps=eps, residual=res,
        out_residual=out)
    torch.cuda.synchronize()
    if out is not None:
        assert H is out
    assert np.array_equal(host_bits(H.contiguous()), want["H"])
    assert np.array_equal(scales.cpu().numpy(), want["scales"])
    assert np.array_equal(codes.cpu().numpy(), want["codes"])
    if want["D"] is not None:
        check_d(D.cpu().numpy(), want["D"])
    else:
        assert D is None


@pytest.mark.parametrize("M", [1, 2, 15, 17, 65, 600, 4200])
@pytest.mark.parametrize("r", [0, 8, 128])
def test_rows_and_ranks(L, M, r):
    _check(L, _case(M, 512, r, True, True, True, seed=M), 512)


@pytest.mark.parametrize("K", [256, 768, 2048, 2304, 5120, 5376, 6400, 8448, 16640, 32768])
@pytest.mark.parametrize("r", [0, 32])
def test_row_lengths(L, K, r):
    _check(L, _case(19, K, r, True, True, True, seed=K), K)


@pytest.mark.parametrize("r", [16, 24, 40, 64, 72, 96, 112, 120])
@pytest.mark.parametrize("M", [33, 1500, 20500])
def test_every_rank_tile(L, r, M):
    K = 1280 if M == 33 else 256
    _check(L, _case(M, K, r, True, True, True, seed=r), K)


@pytest.mark.parametrize("r", [8, 24, 40, 64, 72, 96, 112, 128])
@pytest.mark.parametrize("K", [256, 768])
def test_every_rank_tile_between_few_and_many_rows(L, r, K):
    _check(L, _case(8500, K, r, True, True, True, seed=r), K)


@pytest.mark.parametrize("gamma,smooth", [(False, True), (True, False), (False, False)])
@pytest.mark.parametrize("M", [2100, 17000])
def test_many_rows_without_factors(L, gamma, smooth, M):
    _check(L, _case(M, 256, 128, False, gamma, smooth, seed=9), 256)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("gamma", [False, True])
@pytest.mark.parametrize("smooth", [False, True])
@pytest.mark.parametrize("r", [0, 16])
def test_optional_operands(L, residual, gamma, smooth, r):
    _check(L, _case(21, 1024, r, residual, gamma, smooth, seed=3), 1024)


@pytest.mark.parametrize("r", [0, 8])
def test_padded_strides(L, r):
    _check(L, _case(37, 512, r, True, True, True, seed=4, pad=24), 512)


@pytest.mark.parametrize("K", [512, 16640])
@pytest.mark.parametrize("r", [0, 8])
@pytest.mark.parametrize("where", ["X", "res"])
def test_in_place_residual(L, r, where, K):
    _check(L, _case(37, K, r, True, True, True, seed=5), K, in_place=where)


@pytest.mark.parametrize("r", [0, 8])
def test_zero_rows_large_and_tiny_values(L, r):
    c = _case(8, 512, r, True, True, True, seed=6)
    c["X"][0], c["res"][0] = 0, 0                                   # a row of zeros
    c["X"][1], c["res"][1] = 0, 0x8000                              # negative zeros
    c["X"][2, 1:], c["res"][2] = 0, 0                               # one live channel
    c["X"][3] = bf16_rne(np.full(512, 1e30, np.float32))
    c["X"][4] = bf16_rne(np.full(512, 1e-30, np.float32))
    c["res"][3:5] = 0
    c["X"][5, :32] = bf16_rne(np.full(32, 1000.0, np.float32))      # one loud block
    _check(L, c, 512)


def test_feeds_the_mxfp8_product(L):
    """Codes, scales and D go into the MXFP8 GEMM as svdq_quant_act_lowrank_down's do."""
    torch = torch_mod()
    from oracle import gemm as OG, layer as OL
    from tests.gpu_common import check_y
    M, K, N, r = 70, 512, 256, 16
    c = _case(M, K, r, True, True, True, seed=7)
    rng = np.random.default_rng(8)
    W = bf16_rne((rng.standard_normal((N, K)) * K ** -0.5).astype(np.float32))
    up = bf16_rne((rng.standard_normal((N, r)) * 0.1).astype(np.float32))
    wt = OL.prepare_weight(W, c["lam"], c["down"], up, "mxfp8")
    o = OA.rmsnorm_quant(c["X"], c["res"], c["gamma"], 1e-6, c["lam"], c["down"])
    _, y = OG.linear_mx(o["codes"], o["scales"], wt["codes"], wt["scales"], o["D"], up, "e4m3")
    pw = L.prepare_weight(dev_bf16(W), dev(c["lam"]), dev_bf16(c["down"]), dev_bf16(up), L.MXFP8)
    codes, scales, D, _ = L.norm_quantize_activation(dev_bf16(c["X"]), dev_bf16(c["gamma"]),
                                                     dev(c["lam"]), dev_bf16(c["down"]),
                                                     residual=dev_bf16(c["res"]))
    Y = L.gemm(codes, scales, None, D, pw, M)
    torch.cuda.synchronize()
    check_y(host_bits(Y), y)


@pytest.mark.parametrize("r", [0, 8])
def test_more_rows_than_blocks(L, r):
    """2^21 + 5 rows: two launches of the row kernel."""
    torch = torch_mod()
    M, K, n = (1 << 21) + 5, 256, 96
    g = torch.Generator(device="cuda").manual_seed(4)
    X = torch.randn(M, K, generator=g, device="cuda", dtype=torch.bfloat16)
    c = _case(1, K, r, False, True, True, seed=9)
    codes, scales, D, _ = L.norm_quantize_activation(X, dev_bf16(c["gamma"]), dev(c["lam"]),
                                                     dev_bf16(c["down"]) if r else None)
    torch.cuda.synchronize()
    for rows in (slice(0, n), slice(M - n, M)):
        want = OA.rmsnorm_quant(host_bits(X[rows]), None, c["gamma"], 1e-6, c["lam"], c["down"])
        assert np.array_equal(codes[rows].cpu().numpy(), want["codes"])
        assert np.array_equal(scales[rows].cpu().numpy(), want["scales"])
        if r:
            check_d(D[rows].cpu().numpy(), want["D"])
