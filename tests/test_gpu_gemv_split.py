"""GPU parity of svdq_w4a16_gemv on the launches of the wide layers: several groups of outputs, the last one
ragged, times several parts of K, the last one short, each of more than eight pieces of 128 channels, so
that a block's loads go round more than once.  The weight is any codes; the float64 forms run on the
device.

Tolerance, per element, A the sum of the magnitudes of the products: half a bf16 step of the result,
2^-8·|y|; every product is exact in fp32 and every addition loses at most a whole step, 2^-23, of a
partial sum.  An element of A takes part in at most 256 additions within its pair of pieces, one for each
pair of its part, one for each part, and the tensor's scale; through the branch in at most 512 within its
part of D (four pieces), one for the halves of that, one for each part, and 3·r + 1 with the up factor
(three exact parts of D)."""
import numpy as np
import pytest

from oracle import tokens as OT
from tests.gpu_common import torch_mod
from tests.test_gpu_gemv import FMTS, L  # noqa: F401

pytestmark = pytest.mark.gpu
# N, K, pieces of a part, parts.  39 whole groups of 128 outputs and one of 8; 107 and one of 120.
SHAPES = [(5000, 7936, 12, 6), (13816, 2304, 12, 2), (5000, 13568, 20, 6)]
GROUP = dict(nvfp4=16, int4=64, mxfp4=32)


class Case:
    def __init__(self, L, fmt, N, K, r=128):  # noqa: F811
        torch = torch_mod()
        rng = torch.Generator(device="cuda").manual_seed(N + K)
        f = lambda *s: torch.randn(*s, device="cuda", generator=rng)  # noqa: E731
        ints = lambda lo, hi, *s: torch.randint(lo, hi, s, device="cuda", dtype=torch.uint8, generator=rng)  # noqa: E731
        self.N, self.K, self.r, self.fmt, self.L = N, K, r, fmt, L
        self.codes = ints(0, 256, N, K // 2)
        n = K // GROUP[fmt]
        self.g = None
        if fmt == "int4":
            self.scales = (torch.rand(N, n, device="cuda", generator=rng) * 0.01 + 1e-3).half()
        elif fmt == "nvfp4":
            self.scales, self.g = ints(0x20, 0x7F, N, n), torch.full((1,), 2.3e-5, device="cuda")
        else:
            self.scales = ints(112, 120, N, n)
        self.down, self.up = (0.05 * f(r, K)).bfloat16(), (0.05 * f(N, r)).bfloat16()
        self.lam = torch.exp(0.5 * f(K))
        self.X = (f(64, K) * torch.exp(0.75 * f(K))).bfloat16()
        # float64 values, by the oracle's tables
        nib = torch.stack([self.codes & 15, self.codes >> 4], -1).reshape(N, K).long()
        every = np.arange(256, dtype=np.uint8)
        if fmt == "int4":
            v = torch.as_tensor(np.r_[np.arange(8), np.arange(-8, 0)].astype(np.float64)).cuda()[nib]
            s = self.scales.double()
        else:
            v = torch.as_tensor(OT.e2m1_decode(np.arange(16, dtype=np.uint8)).astype(np.float64)).cuda()[nib]
            if fmt == "nvfp4":
                table = OT.e4m3_decode(np.arange(0x7F, dtype=np.uint8)).astype(np.float64)
                s = torch.as_tensor(table).cuda()[self.scales.long()] * self.g.double()
            else:
                s = torch.as_tensor(np.ldexp(1.0, every.astype(np.int64) - 127)).cuda()[self.scales.long()]
        self.w = (v.view(N, n, -1) * s[..., None]).view(N, K)

    def weight(self, r):
        L = self.L  # noqa: F811
        code = dict(nvfp4=L.NVFP4, int4=L.INT4_G64, mxfp4=L.MXFP4)[self.fmt]
        return L.PreparedWeight(code, self.N, self.K, r, self.codes, self.scales, self.g,
                                self.up[:, :r].contiguous() if r else None)


@pytest.fixture(scope="module", params=[(f, s) for f in FMTS for s in SHAPES],
                ids=lambda p: f"{p[0]}-{p[1][0]}x{p[1][1]}")
def case(request, L):  # noqa: F811
    fmt, (N, K, each, parts) = request.param
    from w4a4_quantized_dit_amd import _lib
    # (the launches are what the docstring says: the workspace without a rank is a sum for each part)
    assert _lib.svdq_w4a16_gemv_workspace_bytes(4, N, K, 0) == parts * N * 16
    pieces = K // 128
    assert each > 8 and (pieces + each - 1) // each == parts and 0 < pieces % each < each and N % 128
    return Case(L, fmt, N, K), each, parts


@pytest.mark.parametrize("M", [1, 5, 16, 17, 32, 33, 48, 64])
@pytest.mark.parametrize("r,smooth", [(0, False), (32, True), (128, True)])
def test_dense(case, M, r, smooth):
    torch = torch_mod()
    c, each, parts = case
    X, lam = c.X[:M], c.lam if smooth else None
    out = torch.full((M + 1, c.N + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    down = c.down[:r].contiguous()
    Y = c.L.gemv(X, c.weight(r), lam, down if r else None, out=out[:M, :c.N])
    torch.cuda.synchronize()
    assert torch.all(out[M:] == 7.0) and torch.all(out[:, c.N:] == 7.0)
    x = X.float()
    if smooth:
        x = (x * (1.0 / lam)).bfloat16()
    x = x.double()
    y, a = x @ c.w.T, x.abs() @ c.w.abs().T
    tol = (256 + each // 2 + parts + 1) * 2.0 ** -23 * a
    if r:
        d, u = down.double(), c.up[:, :r].double()
        y, a = y + (x @ d.T) @ u.T, (x.abs() @ d.abs().T) @ u.abs().T
        tol += (512 + 1 + (c.K // 128 + 3) // 4 + 3 * r + 1) * 2.0 ** -23 * a
    tol += 2.0 ** -8 * y.abs()
    bad = (Y.double() - y).abs() > tol
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:5].tolist())


@pytest.mark.parametrize("M", [16, 32, 64])
def test_every_channel_of_every_output(case, M):
    """Unit rows: output n of row k is w[n, k] itself, one product and one rounding (and in fp32 the
    tensor's scale), for every channel in turn."""
    torch = torch_mod()
    c, _, _ = case
    pw = c.weight(0)
    bad = torch.zeros((), dtype=torch.bool, device="cuda")
    for k in range(0, c.K, M):
        X = torch.zeros(M, c.K, dtype=torch.bfloat16, device="cuda")
        X[:, k:k + M].fill_diagonal_(1.0)
        n = min(M, c.K - k)
        w = c.w[:, k:k + n].T
        Y = c.L.gemv(X, pw, None, None)
        bad |= ((Y[:n].double() - w).abs() > 2.0 ** -8 * (1 + 2.0 ** -15) * w.abs()).any() | (Y[n:] != 0).any()
    assert not bool(bad)


def test_rows_do_not_depend_on_each_other(case):
    torch = torch_mod()
    c, _, _ = case
    pw = c.weight(32)
    down = c.down[:32].contiguous()
    whole = c.L.gemv(c.X, pw, c.lam, down)
    for rows in ([0], [63], list(range(5)), list(range(3, 20)), list(range(20, 60))):
        part = c.L.gemv(c.X[rows], pw, c.lam, down)
        torch.cuda.synchronize()
        assert torch.equal(part, whole[rows]), rows
