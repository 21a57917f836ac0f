"""GPU parity of the paged 8-bit cache: every byte of the cache (codes, scales, and what must stay
untouched) and every value read back equal to the oracle's."""
import numpy as np
import pytest

from oracle import attention as OA
from oracle.formats import bf16_rne
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


def device_cache(L, c):
    return L.KVCache(dev(c["kc"]), dev(c["vc"]), dev(c["ks"]), dev(c["vs"]), c["dim"])


def same(kv, c):
    for got, want in ((kv.k_scales, "ks"), (kv.v_scales, "vs"), (kv.k_codes, "kc"),
                      (kv.v_codes, "vc")):
        assert np.array_equal(got.cpu().numpy(), c[want]), want


def i32(v):
    return dev(np.asarray(v, np.int32))


def _write(L, c, kv, K, V, table, cu, start, pad=0):
    """On both sides; K and V as strided columns of one packed buffer."""
    wide = np.concatenate([K, V, np.zeros((len(K), pad), np.uint16)], 1)
    buf = dev_bf16(wide)
    w = K.shape[1]
    n = max(1, int(np.max(np.diff(cu))))
    L.kv_write(kv, buf[:, :w], buf[:, w:2 * w], i32(table), i32(cu), i32(start), n)
    OA.kv_write(c, K, V, np.asarray(table), cu, start)


def _rand(rng, rows, width, spread=1.0):
    return bf16_rne((rng.standard_normal((rows, width)) * spread).astype(np.float32))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads", [1, 3])
@pytest.mark.parametrize("start,n", [(0, 1), (0, 63), (0, 64), (0, 65), (5, 1), (63, 1), (63, 2),
                                     (64, 64), (1, 63), (17, 200), (130, 129), (0, 0)])
def test_one_sequence(L, dim, heads, start, n):
    torch = torch_mod()
    rng = np.random.default_rng(start * 1000 + n)
    c = OA.new_cache(9, heads, dim, fill=0xFF)          # NaN codes wherever nothing is written
    kv = device_cache(L, c)
    table = [[4, 0, 7, 2, 8]]
    if start:
        _write(L, c, kv, _rand(rng, start, heads * dim), _rand(rng, start, heads * dim), table,
               [0, start], [0])
    K, V = _rand(rng, n, heads * dim, 3.0), _rand(rng, n, heads * dim, 0.01)
    _write(L, c, kv, K, V, table, [0, n], [start], pad=8)
    torch.cuda.synchronize()
    same(kv, c)
    total = start + n
    if total:
        k, v = L.kv_read(kv, i32(table), i32([0, total]), i32([0]), total, total)
        torch.cuda.synchronize()
        for got, is_v in ((k, 0), (v, 1)):
            for h in range(heads):
                want, _ = OA.kv_values(c, np.array(table[0]), total, h, is_v)
                g = got[:, h * dim:(h + 1) * dim].float().cpu().numpy()
                assert np.array_equal(g, want)


@pytest.mark.parametrize("dim", [64, 128])
def test_token_by_token_with_growing_and_shrinking_values(L, dim):
    """70 single appends whose size rises and falls: the scale only grows within a page, and
    earlier codes are rounded again when it does."""
    torch = torch_mod()
    rng = np.random.default_rng(11)
    c = OA.new_cache(3, 2, dim, fill=0x7F)
    kv = device_cache(L, c)
    table = [[2, 1]]
    for t in range(70):
        spread = 2.0 ** (t % 13 - 4) * (1 + t / 10)
        K, V = _rand(rng, 1, 2 * dim, spread), _rand(rng, 1, 2 * dim, 1 / spread)
        if t == 20:
            K[:], V[:] = 0, 0x8000                      # zeros, and negative zeros
        _write(L, c, kv, K, V, table, [0, 1], [t])
    torch.cuda.synchronize()
    same(kv, c)


def test_extreme_magnitudes(L):
    torch = torch_mod()
    dim = 64
    c = OA.new_cache(6, 1, dim)
    kv = device_cache(L, c)
    vals = [3.0e38, 1e-38, 448.0, 449.0, 0.0, 2.0 ** -100]
    for p, v in enumerate(vals):
        K = bf16_rne(np.full((64, dim), v, np.float32) * np.linspace(-1, 1, dim, dtype=np.float32))
        _write(L, c, kv, K, K[::-1].copy(), [[p]], [0, 64], [0])
    # tiny codes under a huge new token
    K = bf16_rne(np.full((1, dim), 1e30, np.float32))
    _write(L, c, kv, K, K, [[1]], [0, 1], [40])
    torch.cuda.synchronize()
    same(kv, c)


@pytest.mark.parametrize("start,n,bound", [(0, 64, 1), (10, 100, 60), (63, 10, 1), (64, 200, 65)])
def test_rows_past_the_bound_are_left(L, start, n, bound):
    """max_rows below a sequence's rows: the rows past it are neither written nor read, within the
    last page that the others reach too."""
    torch = torch_mod()
    rng = np.random.default_rng(15)
    dim, rows = 64, 2 * n
    c = OA.new_cache(12, 1, dim, fill=0x33)
    kv = device_cache(L, c)
    table = [[4, 0, 7, 2, 8], [9, 1, 3, 10, 6]]
    before = _rand(rng, 2 * start, dim)
    if start:
        _write(L, c, kv, before, before, table, [0, start, 2 * start], [0, 0])
    K, V = _rand(rng, rows, dim), _rand(rng, rows, dim)
    L.kv_write(kv, dev_bf16(K), dev_bf16(V), i32(table), i32([0, n, rows]), i32([start, start]), bound)
    at = np.r_[0:bound, n:n + bound]
    OA.kv_write(c, K[at], V[at], np.asarray(table), [0, bound, 2 * bound], [start, start])
    torch.cuda.synchronize()
    same(kv, c)
    out = [torch.full((rows, dim), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    L.kv_read(kv, i32(table), i32([0, n, rows]), i32([start, start]), rows, bound, out=out)
    torch.cuda.synchronize()
    for o in out:
        left = np.setdiff1d(np.arange(rows), at)
        assert torch.all(o[dev(left)] == 5.0) and torch.all((o[dev(at)] != 5.0).any(dim=1))


@pytest.mark.parametrize("dim", [64, 128])
def test_infinities_and_nan(L, dim):
    """They are stored as the NaN code and read back as NaN; the page's scale and the other tokens'
    codes are those without them, also where a later token raises the scale over them."""
    torch = torch_mod()
    rng = np.random.default_rng(14)
    H = 2
    odd = np.array([0x7F80, 0xFF80, 0x7FC0, 0xFFC1, 0x7F81, 0x7F7F, 0xFF7F], np.uint16)
    for start, n, later in ((0, 64, 0), (0, 40, 3), (10, 130, 2), (63, 1, 0), (0, 1, 1)):
        for only in (False, True):                      # some values, or every one
            c = OA.new_cache(5, H, dim, fill=0x55)
            kv = device_cache(L, c)
            table = [[3, 1, 4]]
            if start:
                _write(L, c, kv, _rand(rng, start, H * dim), _rand(rng, start, H * dim), table,
                       [0, start], [0])
            X = [_rand(rng, n, H * dim) for _ in range(2)]
            for x in X:
                hit = rng.random(x.shape) < (1.1 if only else 0.02)
                x[hit] = rng.choice(odd[:5] if only else odd[:rng.choice([5, 7])], int(hit.sum()))
            _write(L, c, kv, X[0], X[1], table, [0, n], [start])
            if later:
                _write(L, c, kv, _rand(rng, later, H * dim, 1e6), _rand(rng, later, H * dim, 30.0),
                       table, [0, later], [start + n])
            torch.cuda.synchronize()
            same(kv, c)
            total = start + n + later
            got = L.kv_read(kv, i32(table), i32([0, total]), i32([0]), total, total)
            torch.cuda.synchronize()
            for is_v in range(2):
                for h in range(H):
                    want, _ = OA.kv_values(c, np.array(table[0]), total, h, is_v)
                    g = got[is_v][:, h * dim:(h + 1) * dim].float().cpu().numpy()
                    assert np.array_equal(g, want, equal_nan=True)


@pytest.mark.parametrize("dim", [64, 128])
def test_ragged_batch(L, dim):
    """Sequences of other lengths and starts, one without rows, rows behind the last sequence."""
    torch = torch_mod()
    rng = np.random.default_rng(12)
    H = 2
    c = OA.new_cache(24, H, dim, fill=0xAA)
    kv = device_cache(L, c)
    table = rng.permutation(24)[:20].reshape(4, 5)
    prior = [10, 0, 64, 199]
    cu = np.concatenate([[0], np.cumsum(prior)])
    _write(L, c, kv, _rand(rng, cu[-1], H * dim), _rand(rng, cu[-1], H * dim), table, cu, [0] * 4)
    cu = np.array([0, 70, 70, 71, 150])
    rows = 160                                          # ten rows of no sequence
    K, V = _rand(rng, rows, H * dim), _rand(rng, rows, H * dim)
    _write(L, c, kv, K, V, table, cu, prior)
    torch.cuda.synchronize()
    same(kv, c)
    out = [torch.full((rows, H * dim), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    L.kv_read(kv, i32(table), i32(cu), i32(prior), rows, 80, out=out)
    torch.cuda.synchronize()
    assert torch.all(out[0][150:] == 5.0) and torch.all(out[1][150:] == 5.0)
    for b in range(4):
        n = cu[b + 1] - cu[b]
        for h in range(H):
            want, _ = OA.kv_values(c, table[b], prior[b] + n, h, 1)
            got = out[1][cu[b]:cu[b + 1], h * dim:(h + 1) * dim].float().cpu().numpy()
            assert np.array_equal(got, want[prior[b]:])


def test_bad_pages_are_skipped(L):
    """Entries outside the cache, a table too short, rows outside the tensors: nothing is written
    for them and nothing else changes."""
    torch = torch_mod()
    rng = np.random.default_rng(13)
    dim, H = 64, 1
    c = OA.new_cache(4, H, dim, fill=0x11)
    kv = device_cache(L, c)
    K, V = _rand(rng, 200, dim), _rand(rng, 200, dim)
    _write(L, c, kv, K, V, [[1, -1], [99, 3]], [0, 140, 200], [0, 60])
    torch.cuda.synchronize()
    same(kv, c)
    before = {k: v.copy() for k, v in c.items() if k != "dim"}
    L.kv_write(kv, dev_bf16(K), dev_bf16(V), i32([[1, 2]]), i32([0, 500]), i32([0]), 500)
    L.kv_write(kv, dev_bf16(K), dev_bf16(V), i32([[1, 2]]), i32([0, 100]), i32([-5]), 100)
    L.kv_write(kv, dev_bf16(K), dev_bf16(V), i32([[1, 2]]), i32([50, 20]), i32([0]), 100)
    torch.cuda.synchronize()
    for k, v in before.items():
        assert np.array_equal(c[k], v)
    same(kv, c)


def test_refusals_of_the_binding(L):
    torch = torch_mod()
    kv = L.kv_cache(2, 2, 64)
    X = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    good = (i32([[0]]), i32([0, 4]), i32([0]), 4)
    L.kv_write(kv, X, X, *good)
    for bad in (X[:, :64], X.float(), X.cpu()):
        with pytest.raises((ValueError, TypeError)):
            L.kv_write(kv, bad, X, *good)
    with pytest.raises(ValueError):
        L.kv_write(kv, X, X, i32([[0]]), i32([0]), i32([0]), 4)        # cu_rows too short
    with pytest.raises(ValueError):
        L.kv_write(kv, X, X, i32([0]), i32([0, 4]), i32([0]), 4)       # block_table not 2-D
    with pytest.raises(ValueError):
        L.kv_write(L.KVCache(kv.k_codes, kv.v_codes, kv.k_scales[:1], kv.v_scales, 64), X, X, *good)
    torch.cuda.synchronize()


def test_large_read_back(L):
    """Outputs past 256 MB are stored past the caches: the same values."""
    torch = torch_mod()
    n, H, dim = 4300, 128, 128
    g = torch.Generator(device="cuda").manual_seed(5)
    X = [torch.randn(n, H * dim, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    pages = (n + 63) // 64
    kv = L.kv_cache(pages, H, dim)
    table = torch.randperm(pages, generator=g, device="cuda").int()[None]
    L.kv_write(kv, X[0], X[1], table, i32([0, n]), i32([0]), n)
    whole = L.kv_read(kv, table, i32([0, n]), i32([0]), n, n)
    parts = [L.kv_read(kv, table, i32([0, 1075]), i32([a]), 1075, 1075) for a in range(0, n, 1075)]
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(whole[i], torch.cat([p[i] for p in parts]))
        err = (whole[i].float() - X[i].float()).abs()
        # half a step of E4M3, or of its smallest step under the page's scale
        assert torch.all(err <= 2.0 ** -4 * X[i].float().abs() + 2.0 ** -10 * 8 / 448)
