"""GPU parity of the paged 4-bit cache: every byte of the cache (codes, scales, and what must stay
untouched) and every value read back equal to the oracle's."""
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


def device_cache(L, c):
    return L.KVCache(dev(c["kc"]), dev(c["vc"]), dev(c["ks"]), dev(c["vs"]), c["dim"], bits=4)


def same(kv, c):
    for got, want in ((kv.k_scales, "ks"), (kv.v_scales, "vs"), (kv.k_codes, "kc"),
                      (kv.v_codes, "vc")):
        assert np.array_equal(got.cpu().numpy(), c[want]), want


def i32(v):
    return dev(np.asarray(v, np.int32))


def _write(L, c, kv, K, V, table, cu, start, pad=0, bound=None):
    """On both sides; K and V as strided columns of one packed buffer."""
    wide = np.concatenate([K, V, np.zeros((len(K), pad), np.uint16)], 1)
    buf = dev_bf16(wide)
    w = K.shape[1]
    n = max(1, int(np.max(np.diff(cu)))) if bound is None else bound
    L.kv_write(kv, buf[:, :w], buf[:, w:2 * w], i32(table), i32(cu), i32(start), n)
    OT.kv_write(c, K, V, np.asarray(table), cu, start)


def _rand(rng, rows, width, spread=1.0):
    return bf16_rne((rng.standard_normal((rows, width)) * spread).astype(np.float32))


def _same_rows(got, c, table_row, first, total, heads, dim):
    """Rows of K and V read back are the oracle's tokens first .. total, bit for bit (NaN as NaN)."""
    for t, is_v in zip(got, (0, 1)):
        g = t.float().cpu().numpy()
        for h in range(heads):
            want, _ = OT.kv_values(c, table_row, total, h, is_v)
            assert np.array_equal(g[:, h * dim:(h + 1) * dim], want[first:], equal_nan=True)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads", [1, 3])
@pytest.mark.parametrize("start,n", [(0, 1), (0, 63), (0, 64), (0, 65), (5, 1), (6, 3), (63, 1), (63, 2),
                                     (64, 64), (1, 63), (17, 200), (130, 129), (0, 0), (3, 6)])
def test_one_sequence(L, dim, heads, start, n):
    torch = torch_mod()
    rng = np.random.default_rng(start * 1000 + n)
    c = OT.new_cache(9, heads, dim, fill=0xFF)          # NaN blocks wherever nothing is written
    kv = device_cache(L, c)
    table = [[4, 0, 7, 2, 8]]
    if start:
        _write(L, c, kv, _rand(rng, start, heads * dim), _rand(rng, start, heads * dim), table,
               [0, start], [0])
    K, V = _rand(rng, n, heads * dim, 3.0), _rand(rng, n, heads * dim, 0.01)
    _write(L, c, kv, K, V, table, [0, n], [start], pad=8)
    torch.cuda.synchronize()
    same(kv, c)
    for first, total in ((0, start + n), (start, start + n), (min(7, start + n), start + n)):
        if total > first:
            got = L.kv_read(kv, i32(table), i32([0, total - first]), i32([first]), total - first,
                            total - first)
            torch.cuda.synchronize()
            _same_rows(got, c, np.array(table[0]), first, total, heads, dim)


@pytest.mark.parametrize("dim", [64, 128])
def test_token_by_token(L, dim):
    """70 single appends whose sizes differ: each keeps its own scale, the others their bytes."""
    torch = torch_mod()
    rng = np.random.default_rng(11)
    c = OT.new_cache(3, 2, dim, fill=0x7F)
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


@pytest.mark.parametrize("start", [0, 3])
def test_every_bf16_value(L, start):
    """All 65536 bit patterns as keys, reversed as values, in blocks of neighbours and of strangers."""
    torch = torch_mod()
    bits = np.arange(65536, dtype=np.uint16).reshape(1024, 64)
    mixed = np.random.default_rng(1).permutation(bits.ravel()).reshape(1024, 64)
    for K in (bits, mixed):
        c = OT.new_cache(18, 1, 64)
        kv = device_cache(L, c)
        table = np.arange(18)[None, ::-1].copy()
        _write(L, c, kv, K, K[::-1].copy(), table, [0, 1024], [start])
        torch.cuda.synchronize()
        same(kv, c)
        got = L.kv_read(kv, i32(table), i32([0, 1024]), i32([start]), 1024, 1024)
        torch.cuda.synchronize()
        _same_rows(got, c, table[0], start, start + 1024, 1, 64)


@pytest.mark.parametrize("dim", [64, 128])
def test_infinities_and_nan_make_their_block_nan(L, dim):
    torch = torch_mod()
    rng = np.random.default_rng(2)
    for n, start in ((64, 0), (50, 9)):
        K, V = _rand(rng, n, 2 * dim), _rand(rng, n, 2 * dim)
        K[3, 5], K[10, dim + 33], V[3, 40], V[20, 0], V[21, 2 * dim - 1] = (0x7F80, 0x7FC0, 0xFF80, 0xFFFF,
                                                                           0x7F81)
        c = OT.new_cache(2, 2, dim)
        kv = device_cache(L, c)
        _write(L, c, kv, K, V, [[1]], [0, n], [start])
        torch.cuda.synchronize()
        same(kv, c)
        assert (c["ks"] == 255).sum() == 2 and (c["vs"] == 255).sum() == 3
        got = L.kv_read(kv, i32([[1]]), i32([0, n]), i32([start]), n, n)
        torch.cuda.synchronize()
        _same_rows(got, c, np.array([1]), start, start + n, 2, dim)
        assert int(torch.isnan(got[0]).sum()) == 64 and int(torch.isnan(got[1]).sum()) == 96


@pytest.mark.parametrize("dim", [64, 128])
def test_ragged_batch_with_missing_pages(L, dim):
    """Entries outside the cache and past the table are skipped, empty sequences too."""
    torch = torch_mod()
    rng = np.random.default_rng(4)
    lens, start = [100, 0, 1, 300, 64], [10, 5, 191, 0, 64]
    cu = np.concatenate([[0], np.cumsum(lens)])
    table = np.array([[0, 1, 2], [3, 3, 3], [4, 5, 6], [7, -1, 8], [9, 99, 10]])
    c = OT.new_cache(11, 2, dim, fill=0xAA)
    kv = device_cache(L, c)
    K, V = _rand(rng, cu[-1], 2 * dim), _rand(rng, cu[-1], 2 * dim)
    _write(L, c, kv, K, V, table, cu, start, pad=16)
    torch.cuda.synchronize()
    same(kv, c)
    out = [torch.full((cu[-1], 2 * dim), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    L.kv_read(kv, i32(table), i32(cu), i32(start), int(cu[-1]), 300, out=out)
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        for t, is_v in zip(out, (0, 1)):
            g = t[cu[b]:cu[b + 1]].float().cpu().numpy()
            for h in range(2):
                want, ok = OT.kv_values(c, table[b], start[b] + n, h, is_v)
                want = np.where(ok[:, None], want, 7.0)[start[b]:]
                assert np.array_equal(g[:, h * dim:(h + 1) * dim], want)


def test_sequences_that_share_a_page(L):
    """Two sequences write other tokens of one page in one call: every token has bytes of its own."""
    torch = torch_mod()
    rng = np.random.default_rng(5)
    for dim in (64, 128):
        for cut in (1, 30, 33):
            c = OT.new_cache(2, 3, dim, fill=0x33)
            kv = device_cache(L, c)
            K, V = _rand(rng, 60, 3 * dim), _rand(rng, 60, 3 * dim)
            _write(L, c, kv, K, V, [[1], [1]], [0, cut, 60], [0, cut])
            torch.cuda.synchronize()
            same(kv, c)


@pytest.mark.parametrize("start,n,bound", [(0, 64, 1), (10, 100, 60), (63, 10, 1), (64, 200, 65)])
def test_rows_past_the_bound_are_left(L, start, n, bound):
    torch = torch_mod()
    rng = np.random.default_rng(15)
    dim, rows = 64, 2 * n
    K, V = _rand(rng, rows, dim), _rand(rng, rows, dim)
    table = np.arange(10).reshape(2, 5)
    c = OT.new_cache(10, 1, dim, fill=0x11)
    kv = device_cache(L, c)
    L.kv_write(kv, dev_bf16(K), dev_bf16(V), i32(table), i32([0, n, rows]), i32([start, start]), bound)
    for b in range(2):
        at = slice(b * n, b * n + min(n, bound))
        OT.kv_write(c, K[at], V[at], table[b:b + 1], [0, at.stop - at.start], [start])
    out = [torch.full((rows, dim), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    L.kv_read(kv, i32(table), i32([0, n, rows]), i32([start, start]), rows, bound, out=out)
    torch.cuda.synchronize()
    same(kv, c)
    for b in range(2):
        for t, is_v in zip(out, (0, 1)):
            want, _ = OT.kv_values(c, table[b], start + min(n, bound), 0, is_v)
            g = t[b * n:(b + 1) * n].float().cpu().numpy()
            assert np.array_equal(g[:bound], want[start:]) and np.all(g[bound:] == 7.0)


def test_bad_rows_are_skipped(L):
    """cu_rows that leave the rows, and negative starts: nothing is written for them."""
    torch = torch_mod()
    rng = np.random.default_rng(16)
    dim = 64
    K = _rand(rng, 20, dim)
    c = OT.new_cache(3, 1, dim, fill=0x22)
    kv = device_cache(L, c)
    for cu, start in (([0, 30], [0]), ([-5, 10], [0]), ([0, 10], [-1]), ([10, 5], [0])):
        L.kv_write(kv, dev_bf16(K), dev_bf16(K), i32([[0, 1, 2]]), i32(cu), i32(start), 20)
    torch.cuda.synchronize()
    same(kv, c)


def test_large_write_and_read(L):
    """Past the caches' size on the way back: the nontemporal stores, every value."""
    torch = torch_mod()
    g = torch.Generator(device="cuda").manual_seed(5)
    n, H, dim = 16500, 40, 128
    K, V = (torch.randn(n, H * dim, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    pages = (n + 63) // 64
    kv = L.kv_cache(pages, H, dim, bits=4)
    table = torch.randperm(pages, generator=g, device="cuda").int().reshape(1, pages)
    cu, zero = i32([0, n]), i32([0])
    L.kv_write(kv, K, V, table, cu, zero, n)
    k, v = L.kv_read(kv, table, cu, zero, n, n)
    torch.cuda.synchronize()
    for got, x in ((k, K), (v, V)):
        for rows in (slice(0, 70), slice(8000, 8070), slice(n - 70, n)):
            want = OT.dequantise(*OT.quantise(x[rows].float().cpu().numpy()))
            assert np.array_equal(got[rows].float().cpu().numpy(), want)
        err = (got.float() - x.float()).norm() / x.float().norm()
        assert float(err) < 0.13     # MXFP4 of normal values: 0.115
    assert host_bits(k).shape == (n, H * dim) and bf16_bits_to_f32(host_bits(k[:1])).shape == (1, H * dim)
