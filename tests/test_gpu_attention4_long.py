"""GPU parity of svdq_attn_kv4 where one block walks many pages, so that it looks its page numbers up again
on the way: every 61 pages where many rows share a page, every 256 where 17 rows to 512 do (a page for each
of a block's four waves), every 64 a wave up to 16 rows.  (The bound of the cached tokens sizes the split
only: a small one leaves the pages in one block, and each test asserts that.)

The weight lies on the pages around those places, with keys that rise there page by page or stand alike;
each page's values have a mean and a scale of their own, so that one page taken for its neighbour moves
the result by more than the tolerance; some of these pages are missing.  Oracle and tolerances are
test_gpu_attention4's."""
import numpy as np
import pytest

from oracle import tokens as OT
from oracle.formats import bf16_bits_to_f32, bf16_rne
from tests.gpu_common import dev_bf16, torch_mod
from tests.test_gpu_attention4 import L, check, device_cache, fill, i32  # noqa: F401
from tests.test_gpu_attention_long import heavy_pages, queries

pytestmark = pytest.mark.gpu

MANY, FEW = 61, 256


def long_case(rng, kv_lens, dim, rising, every):
    """Cache of ragged sequences on shuffled pages, the direction u of their heavy keys; every other byte
    belongs to a NaN block."""
    need = [max(1, (n + 63) // 64) for n in kv_lens]
    pages = sum(need) + 3
    c = OT.new_cache(pages, 1, dim, fill=0xFF)
    order = rng.permutation(pages)
    table = np.full((len(kv_lens), max(need)), -1)
    u = rng.choice([-1.0, 1.0], dim)
    K, V = [], []
    for b, n in enumerate(kv_lens):
        table[b, :need[b]] = order[sum(need[:b]):sum(need[:b + 1])]
        k = 0.5 * rng.standard_normal((n, dim))
        v = np.repeat(rng.standard_normal((need[b], dim)), 64, axis=0)[:n]
        v = v + 0.5 * rng.standard_normal((n, dim))
        heavy = heavy_pages(need[b], every) if need[b] > every else []
        for i, p in enumerate(heavy):
            k[64 * p:64 * p + 64] += u * (0.25 * (i % 7) if rising else 0.75)
        v *= np.repeat(2.0 ** rng.integers(-2, 3, need[b]), 64)[:n, None]
        K.append(k), V.append(v)
    K, V = (bf16_rne(np.concatenate(x).astype(np.float32)) for x in (K, V))
    fill(c, K, V, table, kv_lens)
    return c, table, u


def run_long(L, q_lens, kv_lens, G, dim, causal, max_kv, every, rising, missing):  # noqa: F811
    torch = torch_mod()
    rng = np.random.default_rng(sum(kv_lens) + sum(q_lens))
    c, table, u = long_case(rng, kv_lens, dim, rising, every)
    if missing:
        for i, p in enumerate((every - 1, every + 1, 2 * every)):
            if p < table.shape[1]:
                table[:, p] = -1 if i % 2 else len(c["ks"])
    cu = np.concatenate([[0], np.cumsum(q_lens)])
    bits = queries(rng, int(cu[-1]), G, dim, u)
    O, lse = L.attention(dev_bf16(bits), device_cache(L, c), i32(table), i32(cu), i32(kv_lens),
                         max(q_lens), max_kv, causal=causal, return_lse=True)
    torch.cuda.synchronize()
    want = OT.attention(bf16_bits_to_f32(bits).reshape(-1, G, dim), c, table, cu, kv_lens,
                        float(np.float32(dim ** -0.5)), causal)
    check(want, O.float().cpu().numpy().reshape(-1, G, dim).astype(np.float64),
          lse.cpu().numpy().astype(np.float64), max(kv_lens))


def splits(q, B, G, dim, rows, max_kv):
    from w4a4_quantized_dit_amd import _lib
    return _lib.svdq_attn_kv4_workspace_bytes(rows, G, 1, dim, B, q, max_kv) // (rows * G * (dim + 2) * 4)


HOW = [(False, False, False), (False, True, True), (True, True, False), (True, False, True)]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q,kv,G", [(600, 9600, 1), (200, 9001, 3)])
@pytest.mark.parametrize("causal,rising,missing", HOW)
def test_many_rows_many_pages(L, q, kv, G, dim, causal, rising, missing):  # noqa: F811
    """600 rows of a key head over 141 and 150 pages: lookups at 61 and 122."""
    assert splits(q, 1, G, dim, q, 10) == 0
    run_long(L, [q], [kv], G, dim, causal, 10, MANY, rising, missing)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q,G", [(20, 1), (4, 8)])
@pytest.mark.parametrize("kv", [16384, 16385, 33500])
@pytest.mark.parametrize("causal,rising,missing", HOW)
def test_few_rows_many_pages(L, q, kv, G, dim, causal, rising, missing):  # noqa: F811
    """20 and 32 rows of a key head over 256, 257 and 524 pages."""
    assert splits(q, 1, G, dim, q, 10) == 0
    run_long(L, [q], [kv], G, dim, causal, 10, FEW, rising, missing)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q,G", [(1, 1), (2, 8)])
@pytest.mark.parametrize("causal,rising,missing", HOW[1:])
def test_sixteen_rows_many_pages(L, q, G, dim, causal, rising, missing):  # noqa: F811
    """Eight waves a block, which take 64 pages each from a lookup: the second one at page 512."""
    assert splits(q, 1, G, dim, q, 10) == 0
    run_long(L, [q], [33500], G, dim, causal, 10, 512, rising, missing)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal,rising,missing", HOW[1:])
def test_neighbouring_blocks_of_few_rows_many_pages(L, dim, causal, rising, missing):  # noqa: F811
    """40 rows of 128 sequences, two of them long: 262 pages in each of two splits, so that the lookups
    are at pages 256 and 262 + 256, both within three pages of a multiple of 259."""
    B, q, kv = 128, 40, 33500
    assert splits(q, B, 1, dim, B * q, kv) == 2
    kv_lens = [kv, 33400] + [1 + 7 * b for b in range(B - 2)]
    run_long(L, [q] * B, kv_lens, 1, dim, causal, kv, 259, rising, missing)
