"""GPU tests of svdq_w4a16_gemv at the ends of fp32's range: what the float64 formula gives is finite there,
and so is the result."""
import numpy as np
import pytest

from oracle.formats import bf16_rne
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
