"""GPU parity of svdq_attn_kv8 where one block walks many pages, so that it looks its page numbers and
exponents up again on the way: every 61 pages where many rows share a page, every 256 where a few do.
(The bound of the cached tokens sizes the split only: a small one leaves the pages in one block.)

The weight lies on the pages around those places, with keys that rise there page by page or stand
alike; each page's values have a mean and a scale of their own, so that one page or exponent taken for
its neighbour's moves the result by more than the tolerance; some of these pages are missing.  Oracle
and tolerances are test_gpu_attention's."""
import numpy as np
import pytest

from oracle import attention as OA
from oracle.formats import bf16_bits_to_f32, bf16_rne
from tests.gpu_common import dev_bf16, torch_mod
from tests.test_gpu_attention import L, check, device_cache, i32  # noqa: F401

pytestmark = pytest.mark.gpu

MANY, FEW = 61, 256


def heavy_pages(pages, every):
    """The pages that carry the weight: those on both sides of each place, 64 pages being a wave's."""
    at = np.concatenate([np.arange(e, pages, e) for e in (every, 64 if every < 64 else every)])
    return np.unique(np.clip((at[:, None] + np.arange(-3, 4)).ravel(), 0, pages - 1))


def long_case(rng, kv_lens, heads, dim, rising, every):
    """Cache of ragged sequences on shuffled pages, the direction u of their heavy keys; every
    other byte is a NaN code."""
    need = [max(1, (n + 63) // 64) for n in kv_lens]
    pages = sum(need) + 3
    c = OA.new_cache(pages, heads, dim, fill=0xFF)
    order = rng.permutation(pages)
    table = np.full((len(kv_lens), max(need)), -1)
    u = rng.choice([-1.0, 1.0], dim)
    K, V = [], []
    for b, n in enumerate(kv_lens):
        table[b, :need[b]] = order[sum(need[:b]):sum(need[:b + 1])]
        k = 0.5 * rng.standard_normal((n, heads, dim))
        v = np.repeat(rng.standard_normal((need[b], heads, dim)), 64, axis=0)[:n]
        v = v + 0.5 * rng.standard_normal((n, heads, dim))
        heavy = heavy_pages(need[b], every) if need[b] > every else []
        for i, p in enumerate(heavy):
            k[64 * p:64 * p + 64] += u * (0.25 * (i % 7) if rising else 0.75)
        v *= np.repeat(2.0 ** rng.integers(-2, 3, need[b]), 64)[:n, None, None]
        K.append(k), V.append(v)
    cu = np.concatenate([[0], np.cumsum(kv_lens)])
    K, V = (bf16_rne(np.concatenate(x).reshape(-1, heads * dim).astype(np.float32)) for x in (K, V))
    OA.kv_write(c, K, V, table, cu, [0] * len(kv_lens))
    return c, table, u


def queries(rng, rows, Hq, dim, u):
    q = 0.5 * rng.standard_normal((rows, Hq, dim)) + 2 * u
    return bf16_rne(q.reshape(rows, -1).astype(np.float32))


def run_long(L, q_lens, kv_lens, G, dim, causal, max_kv, every, rising, missing):  # noqa: F811
    torch = torch_mod()
    rng = np.random.default_rng(sum(kv_lens) + sum(q_lens))
    c, table, u = long_case(rng, kv_lens, 1, dim, rising, every)
    if missing:
        for i, p in enumerate((every - 1, every + 1, 2 * every)):
            if p < table.shape[1]:
                table[:, p] = -1 if i % 2 else len(c["ks"])
    cu = np.concatenate([[0], np.cumsum(q_lens)])
    bits = queries(rng, int(cu[-1]), G, dim, u)
    O, lse = L.attention(dev_bf16(bits), device_cache(L, c), i32(table), i32(cu), i32(kv_lens),
                         max(q_lens), max_kv, causal=causal, return_lse=True)
    torch.cuda.synchronize()
    want = OA.attention(bf16_bits_to_f32(bits).reshape(-1, G, dim), c, table, cu, kv_lens,
                        float(np.float32(dim ** -0.5)), causal)
    check(want, O.float().cpu().numpy().reshape(-1, G, dim).astype(np.float64),
          lse.cpu().numpy().astype(np.float64), max(kv_lens))


def splits(q, B, G, dim, rows, max_kv):
    from w4a4_quantized_dit_amd import _lib
    return _lib.svdq_attn_kv8_workspace_bytes(rows, G, 1, dim, B, q, max_kv) // (rows * G * (dim + 2) * 4)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q,kv,G", [(600, 4200, 1), (600, 8300, 1), (200, 17000, 3), (4200, 4200, 1)])
@pytest.mark.parametrize("causal,rising,missing", [(False, False, False), (False, True, True),
                                                   (True, True, False), (True, False, True)])
def test_many_rows_many_pages(L, q, kv, G, dim, causal, rising, missing):  # noqa: F811
    assert splits(q, 1, G, dim, q, 10) == 0
    run_long(L, [q], [kv], G, dim, causal, 10, MANY, rising, missing)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q,G", [(1, 1), (1, 8), (5, 3)])
@pytest.mark.parametrize("kv", [16384, 16385, 33500])
@pytest.mark.parametrize("causal,rising,missing", [(False, False, False), (False, True, False),
                                                   (True, False, True)])
def test_few_rows_many_pages(L, q, kv, G, dim, causal, rising, missing):  # noqa: F811
    assert splits(q, 1, G, dim, q, 10) == 0
    run_long(L, [q], [kv], G, dim, causal, 10, FEW, rising, missing)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal,rising,missing", [(False, False, False), (False, True, False),
                                                   (True, False, True)])
def test_neighbouring_blocks_of_few_rows_many_pages(L, dim, causal, rising, missing):  # noqa: F811
    """40 rows of 128 sequences, two of them long: 262 pages in each of two splits, so that the lookups
    are at pages 256 and 262 + 256, both within three pages of a multiple of 259."""
    B, q, kv = 128, 40, 33500
    assert splits(q, B, 1, dim, B * q, kv) == 2
    kv_lens = [kv, 33400] + [1 + 7 * b for b in range(B - 2)]
    run_long(L, [q] * B, kv_lens, 1, dim, causal, kv, 259, rising, missing)
