"""GPU parity of svdq_attn_kv8 against the float64 oracle, and the attention half run as one chain.

Tolerance of O (derived, per element; A = Σ p|v|, the magnitude the weights' errors act on):
  - each weight is rounded to bf16 once, at most half a step:            2^-8·A
  - the result is rounded to bf16 once:                                  2^-8·|O|
  - scores: up to 128 products, each exact in fp32 (8 bits times 4), summed with at most a whole step,
    2^-23, lost an addition, and four more steps for c and the exponent's argument: dz = 132·2^-23·Z
    with Z = scale·max_t Σ|q k|; a weight moves by that, in numerator and denominator:
                                                                         2·dz·(A + |O|)
  - exponential, fp32 sums: 2^-21 + tokens·2^-24, twice, of A
lse: the score's error, plus the relative error of the sum."""
import numpy as np
import pytest

from oracle import attention as OA
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


def i32(v):
    return dev(np.asarray(v, np.int32))


def make_cache(rng, lens, heads, dim, spread=1.0, extra=3, garbage=0xFF):
    """Cache with `lens` tokens a sequence on shuffled pages, every other byte `garbage`."""
    blocks = max(1, max((n + 63) // 64 for n in lens))
    pages = len(lens) * blocks + extra
    c = OA.new_cache(pages, heads, dim, fill=garbage)
    table = rng.permutation(pages)[:len(lens) * blocks].reshape(len(lens), blocks)
    cu = np.concatenate([[0], np.cumsum(lens)])
    w = heads * dim
    K = bf16_rne((rng.standard_normal((cu[-1], w)) * spread).astype(np.float32))
    V = bf16_rne((rng.standard_normal((cu[-1], w)) * np.exp(rng.standard_normal((cu[-1], 1))))
                 .astype(np.float32))
    OA.kv_write(c, K, V, table, cu, [0] * len(lens))
    return c, table


def device_cache(L, c):
    return L.KVCache(dev(c["kc"]), dev(c["vc"]), dev(c["ks"]), dev(c["vs"]), c["dim"])


def check(want, O, lse, tokens, what=""):
    A, W = want["absO"], np.abs(want["O"])
    dz = want["absz"] * 132 * 2.0 ** -23
    tol = 2.0 ** -8 * (A + W) * (1 + 2.0 ** -7) + (2 * np.expm1(dz)[..., None] + 2.0 ** -20
                                                  + tokens * 2.0 ** -23) * (A + W) + 1e-37
    bad = np.abs(O - want["O"]) > tol
    assert not bad.any(), (what, int(bad.sum()), np.abs(O - want["O"])[bad].max(),
                           np.argwhere(bad)[:5].tolist())
    live = np.isfinite(want["lse"])
    assert np.array_equal(np.isneginf(lse), ~live), what
    err = np.abs(lse - np.where(live, want["lse"], 0))[live]
    lim = (dz + 2.0 ** -20 + tokens * 2.0 ** -24 + 2.0 ** -22 * np.abs(
        np.where(live, want["lse"], 0)))[live]
    assert np.all(err <= lim), (what, (err - lim).max())


def run(L, q_lens, kv_lens, Hq, Hkv, dim, causal, seed=0, spread=1.0, scale=None, q_spread=1.0,
        tail=0, pad=0, max_kv=None):
    torch = torch_mod()
    rng = np.random.default_rng(seed)
    c, table = make_cache(rng, kv_lens, Hkv, dim, spread)
    cu = np.concatenate([[0], np.cumsum(q_lens)])
    rows = int(cu[-1]) + tail
    bits = bf16_rne((rng.standard_normal((rows, Hq * dim + pad)) * q_spread).astype(np.float32))
    Q = dev_bf16(bits)[:, :Hq * dim]
    scale = dim ** -0.5 if scale is None else scale
    out = torch.full((rows, Hq * dim + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    O, lse = L.attention(Q, device_cache(L, c), i32(table), i32(cu), i32(kv_lens), max(q_lens),
                         max(kv_lens) if max_kv is None else max_kv, scale=scale, causal=causal,
                         out=out[:, :Hq * dim], return_lse=True)
    torch.cuda.synchronize()
    q = bf16_bits_to_f32(bits[:, :Hq * dim]).reshape(rows, Hq, dim)
    want = OA.attention(q, c, table, cu, kv_lens, float(np.float32(scale)), causal)
    n = int(cu[-1])
    got = out[:n, :Hq * dim].float().cpu().numpy().reshape(n, Hq, dim).astype(np.float64)
    check({k: v[:n] for k, v in want.items()}, got, lse[:n].cpu().numpy().astype(np.float64),
          max(kv_lens), f"{q_lens} {kv_lens}")
    assert torch.all(out[n:] == 7.0) and torch.all(out[:, Hq * dim:] == 7.0)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kv", [0, 1, 31, 32, 33, 63, 64, 65, 127, 130, 700])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 2), (5, 1), (40, 1)])
def test_single_tokens(L, dim, kv, Hq, Hkv):
    run(L, [1], [kv], Hq, Hkv, dim, True, seed=kv)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q,kv", [(1, 1), (2, 1), (33, 33), (64, 64), (127, 300), (128, 128),
                                  (129, 65), (200, 1000), (257, 257), (520, 70), (600, 600),
                                  (700, 1000)])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("G", [1, 3])
def test_many_rows(L, dim, q, kv, causal, G):
    """Causal with more rows than tokens leaves the first rows empty."""
    run(L, [q], [kv], 2 * G, 2, dim, causal, seed=q + kv)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q", [1, 20, 150, 400])
@pytest.mark.parametrize("causal", [False, True])
def test_long_cache_is_split(L, dim, q, causal):
    """Few blocks over a long cache: the page range is split and joined."""
    from w4a4_quantized_dit_amd import _lib
    assert _lib.svdq_attn_kv8_workspace_bytes(q, 2, 1, dim, 1, q, 5000) > 0
    run(L, [q], [5000], 2, 1, dim, causal, seed=q)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("q_lens,kv_lens", [
    ([1, 1, 1, 1], [5, 0, 64, 900]),
    ([3, 0, 70, 1], [300, 20, 70, 4]),
    ([130, 5, 400], [130, 2000, 300]),
    ([1, 17], [2500, 1]),
])
def test_ragged_batches(L, dim, causal, q_lens, kv_lens):
    run(L, q_lens, kv_lens, 4, 2, dim, causal, tail=3, seed=len(q_lens))


def test_strided_rows(L):
    run(L, [40], [200], 4, 2, 64, True, pad=24)
    run(L, [1], [200], 4, 2, 128, True, pad=8)
    run(L, [600], [700], 4, 2, 128, True, pad=8)


@pytest.mark.parametrize("q", [1, 100, 600])
def test_peaked_and_flat_scores(L, q):
    """Scores over a wide range (the running maximum rises often), nearly equal ones, and a
    bound on kv_len that is too small (it sizes the split only)."""
    run(L, [q], [900], 2, 1, 128, False, spread=4.0, q_spread=4.0)
    run(L, [q], [900], 2, 1, 64, False, spread=1e-3, q_spread=1e-3)
    run(L, [q], [900], 2, 1, 64, False, scale=3.0)
    run(L, [q], [900], 2, 1, 64, True, max_kv=10)


@pytest.mark.parametrize("q", [1, 70, 600])
def test_rising_scores_every_page(L, q):
    """Keys aligned with the query and growing page by page: every page raises the maximum."""
    torch = torch_mod()
    dim, n = 64, 1000
    rng = np.random.default_rng(5)
    u = rng.standard_normal(dim).astype(np.float32)
    K = bf16_rne(u[None] * np.linspace(-3, 12, n, dtype=np.float32)[:, None])
    V = bf16_rne(rng.standard_normal((n, dim)).astype(np.float32))
    c = OA.new_cache(16, 1, dim)
    table = np.arange(16)[None]
    OA.kv_write(c, K, V, table, np.array([0, n]), [0])
    bits = bf16_rne(np.tile(u, (q, 1)) * np.linspace(0.1, 1, q, dtype=np.float32)[:, None])
    O, lse = L.attention(dev_bf16(bits), device_cache(L, c), i32(table), i32([0, q]), i32([n]), q, n,
                         return_lse=True)
    torch.cuda.synchronize()
    qf = bf16_bits_to_f32(bits).reshape(q, 1, dim)
    want = OA.attention(qf, c, table, np.array([0, q]), [n], 0.125, False)
    check(want, O.float().cpu().numpy().reshape(q, 1, dim).astype(np.float64),
          lse.cpu().numpy().astype(np.float64), n)


@pytest.mark.parametrize("q", [1, 50, 600])
def test_zero_rows_and_zero_pages(L, q):
    """All-zero queries weigh every token alike; pages of zeros (smallest exponent) beside pages of
    large values keep their weight in the sum."""
    torch = torch_mod()
    dim = 64
    rng = np.random.default_rng(6)
    V = rng.standard_normal((192, dim)).astype(np.float32) * 1000
    V[64:128] = 0
    K = V.copy()
    K[:64] = 0
    c = OA.new_cache(3, 1, dim)
    table = np.array([[0, 1, 2]])
    OA.kv_write(c, bf16_rne(K), bf16_rne(V), table, np.array([0, 192]), [0])
    bits = bf16_rne(np.zeros((q, dim), np.float32))
    O, lse = L.attention(dev_bf16(bits), device_cache(L, c), i32(table), i32([0, q]), i32([192]), q,
                         192, return_lse=True)
    torch.cuda.synchronize()
    qf = np.zeros((q, 1, dim), np.float32)
    want = OA.attention(qf, c, table, np.array([0, q]), [192], 0.125, False)
    check(want, O.float().cpu().numpy().reshape(q, 1, dim).astype(np.float64),
          lse.cpu().numpy().astype(np.float64), 192)


@pytest.mark.parametrize("q", [1, 64, 600])
def test_missing_pages_are_masked(L, q):
    torch = torch_mod()
    rng = np.random.default_rng(7)
    dim = 64
    c, table = make_cache(rng, [400], 1, dim)
    bad = table.copy()
    bad[0, 1], bad[0, 3] = -1, 10 ** 6
    bits = bf16_rne(rng.standard_normal((q, dim)).astype(np.float32))
    for t, kv in ((bad, 400), (np.full_like(table, -1), 400), (table, 10 ** 6)):
        O, lse = L.attention(dev_bf16(bits), device_cache(L, c), i32(t), i32([0, q]), i32([kv]), q,
                             400, return_lse=True)
        torch.cuda.synchronize()
        if kv > 400:     # kv_len past the table is limited to it; its last page holds garbage
            continue
        qf = bf16_bits_to_f32(bits).reshape(q, 1, dim)
        want = OA.attention(qf, c, t, np.array([0, q]), [kv], 0.125, False)
        check(want, O.float().cpu().numpy().reshape(q, 1, dim).astype(np.float64),
              lse.cpu().numpy().astype(np.float64), kv)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q,kv", [(1, 400), (70, 400), (3, 5000), (150, 5000), (600, 400),
                                  (600, 5000)])
@pytest.mark.parametrize("causal", [False, True])
def test_missing_pages_beside_a_garbage_page(L, q, kv, dim, causal):
    """Page 0, which no sequence owns, holds NaN codes: nothing of it shows where pages are missing."""
    torch = torch_mod()
    rng = np.random.default_rng(17)
    c, table = make_cache(rng, [kv], 1, dim)
    for name in ("kc", "vc", "ks", "vs"):     # page 0 <-> the one that holds nothing
        free = next(p for p in range(len(c[name])) if p not in table) if 0 in table else 0
        c[name][[0, free]] = c[name][[free, 0]]
    table = np.where(table == 0, free, table)
    assert np.all(c["vc"][0] == 0xFF)
    for miss in ([0], [1, 3], [table.shape[1] - 1], list(range(table.shape[1]))):
        t = table.copy()
        t[0, miss] = -1
        bits = bf16_rne(rng.standard_normal((q, dim)).astype(np.float32))
        O, lse = L.attention(dev_bf16(bits), device_cache(L, c), i32(t), i32([0, q]), i32([kv]), q,
                             kv, causal=causal, return_lse=True)
        torch.cuda.synchronize()
        assert torch.isfinite(O.float()).all()
        qf = bf16_bits_to_f32(bits).reshape(q, 1, dim)
        want = OA.attention(qf, c, t, np.array([0, q]), [kv], float(np.float32(dim ** -0.5)), causal)
        check(want, O.float().cpu().numpy().reshape(q, 1, dim).astype(np.float64),
              lse.cpu().numpy().astype(np.float64), kv)


def check_with_nan(want, O, lse, tokens, what=""):
    """NaN exactly where the oracle has it, the rest as in `check`."""
    assert np.array_equal(np.isnan(O), np.isnan(want["O"])), what
    assert np.array_equal(np.isnan(lse), np.isnan(want["lse"])), what
    clean = {k: np.nan_to_num(v, nan=0.0, neginf=-np.inf) for k, v in want.items()}
    check(clean, np.nan_to_num(O), np.nan_to_num(lse, neginf=-np.inf), tokens, what)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("G", [1, 2])
@pytest.mark.parametrize("q,kv", [(1, 70), (1, 5000), (3, 130), (15, 4100), (64, 64), (70, 300),
                                  (150, 5000), (300, 300), (600, 700), (600, 5000)])
@pytest.mark.parametrize("causal", [False, True])
def test_nan_in_seen_and_hidden_tokens(L, q, kv, G, dim, causal):
    """Infinities and NaN in keys, values and queries: they show where they are seen, and a row that
    does not see a token has nothing of it, in the pages that its block shares with later rows too."""
    torch = torch_mod()
    rng = np.random.default_rng(q + kv)
    B, H, Hq = 2, 1, G
    for where in ("v", "k", "q", "all"):
        pages = (kv + 63) // 64
        c = OA.new_cache(2 * pages + 1, H, dim, fill=0xFF)
        table = rng.permutation(2 * pages + 1)[:2 * pages].reshape(2, pages)
        K, V = (bf16_rne(rng.standard_normal((2 * kv, H * dim)).astype(np.float32)) for _ in range(2))
        bits = bf16_rne(rng.standard_normal((2 * q, Hq * dim)).astype(np.float32))
        late = max(0, kv - q) + rng.integers(0, min(q, kv), 3)     # tokens that some rows see
        if where in ("v", "all"):
            V[late, rng.integers(0, dim, 3)] = [0x7FC0, 0x7F80, 0xFF80]
            V[kv - 1, dim - 1] = 0x7FC0
        if where in ("k", "all"):
            K[kv + late[:1], rng.integers(0, dim, 1)] = 0x7FC0     # the second sequence's
        if where in ("q", "all"):
            bits[[q // 2, 2 * q - 1], [3, Hq * dim - 1]] = [0x7FC0, 0xFF80]
        OA.kv_write(c, K, V, table, np.array([0, kv, 2 * kv]), [0, 0])
        cu = np.array([0, q, 2 * q])
        O, lse = L.attention(dev_bf16(bits), device_cache(L, c), i32(table), i32(cu), i32([kv, kv]),
                             q, kv, causal=causal, return_lse=True)
        torch.cuda.synchronize()
        qf = bf16_bits_to_f32(bits).reshape(2 * q, Hq, dim)
        with np.errstate(invalid="ignore"):
            want = OA.attention(qf, c, table, cu, [kv, kv], float(np.float32(dim ** -0.5)), causal)
        assert np.isnan(want["O"]).any()
        check_with_nan(want, O.float().cpu().numpy().reshape(2 * q, Hq, dim).astype(np.float64),
                       lse.cpu().numpy().astype(np.float64), kv, where)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q", [1, 32, 300, 600])
def test_scores_are_summed_in_fp32(L, q, dim):
    """One token: lse is the score itself.  Channels from 1 down to 2^-14 side by side, of both signs,
    so that a sum aligned to its largest product with fewer bits than fp32 shows."""
    torch = torch_mod()
    rng = np.random.default_rng(dim + q)
    K = rng.choice([-1.0, 1.0], (1, dim)) * 2.0 ** -rng.integers(0, 15, (1, dim))
    Q = rng.standard_normal((q, dim))
    c = OA.new_cache(1, 1, dim)
    OA.kv_write(c, bf16_rne(K.astype(np.float32)), bf16_rne(K.astype(np.float32)), np.array([[0]]),
                np.array([0, 1]), [0])
    bits = bf16_rne(Q.astype(np.float32))
    O, lse = L.attention(dev_bf16(bits), device_cache(L, c), i32([[0]]), i32([0, q]), i32([1]), q, 1,
                         scale=1.0, return_lse=True)
    torch.cuda.synchronize()
    k, _ = OA.kv_values(c, np.array([0]), 1, 0, 0)
    qf = bf16_bits_to_f32(bits).astype(np.float64)
    # at most a whole step, 2^-23, of a partial sum an addition, and two for lse itself
    lim = (dim + 2) * 2.0 ** -23 * (np.abs(qf) @ np.abs(k).T)
    assert np.all(np.abs(lse.cpu().numpy() - qf @ k.T) <= lim)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q", [1, 40, 600])
@pytest.mark.parametrize("sign", [1, -1])
def test_very_large_scores(L, q, dim, sign):
    """Scores of one sign up to 2^26, exact in fp32 (one channel, powers of two and their sums of few
    bits): the largest takes the whole weight, and lse is that score."""
    torch = torch_mod()
    n = 200
    K = np.zeros((n, dim), np.float32)
    K[:, 5] = sign * 2.0 ** 13 * (1 + (np.arange(n) * 37 % n) / n)
    V = np.random.default_rng(3).standard_normal((n, dim)).astype(np.float32)
    Q = np.zeros((q, dim), np.float32)
    Q[:, 5] = 2.0 ** 12
    c = OA.new_cache(4, 1, dim)
    table = np.array([[2, 0, 3, 1]])
    OA.kv_write(c, bf16_rne(K), bf16_rne(V), table, np.array([0, n]), [0])
    bits = bf16_rne(Q)
    O, lse = L.attention(dev_bf16(bits), device_cache(L, c), i32(table), i32([0, q]), i32([n]), q, n,
                         scale=1.0, return_lse=True)
    torch.cuda.synchronize()
    qf = bf16_bits_to_f32(bits).reshape(q, 1, dim)
    want = OA.attention(qf, c, table, np.array([0, q]), [n], 1.0, False)
    got = O.float().cpu().numpy().reshape(q, 1, dim)
    # weights that are equal (the codes of several keys are) or 0: only the roundings of the weights
    # and of the result are left, 2^-8 each, of Σ p|v|
    assert np.all(np.abs(got - want["O"]) <= 2.0 ** -6 * want["absO"])
    # lse = (scale / c)·(c·z): c·z rounded (made up for by the sum), the last product: 2^-23 and room
    assert np.all(np.abs(lse.cpu().numpy() - want["lse"]) <= 2.0 ** -22 * np.abs(want["lse"]))


@pytest.mark.parametrize("q,kv,bound", [(3, 100, 1), (20, 5000, 7), (300, 300, 130), (150, 5000, 129),
                                        (400, 400, 330), (400, 5000, 270)])
def test_rows_past_the_bound_are_left(L, q, kv, bound):
    """max_rows below a sequence's rows: the rows past it stay as they were, with a split too, and
    the others see what they see without the bound (causal by the true number of rows)."""
    torch = torch_mod()
    rng = np.random.default_rng(9)
    c, table = make_cache(rng, [kv, kv], 1, 64)
    kvc, t = device_cache(L, c), i32(table)
    Q = dev_bf16(bf16_rne(rng.standard_normal((2 * q, 2 * 64)).astype(np.float32)))
    cu, ln = i32([0, q, 2 * q]), i32([kv, kv])
    whole = L.attention(Q, kvc, t, cu, ln, q, kv, causal=True)
    out = torch.full_like(whole, 7.0)
    L.attention(Q, kvc, t, cu, ln, bound, kv, causal=True, out=out)
    torch.cuda.synchronize()
    for b in range(2):
        got, want = out[b * q:(b + 1) * q].float(), whole[b * q:(b + 1) * q].float()
        assert torch.all(got[bound:] == 7.0)
        # another split of the pages may round each result the other way
        assert torch.all((got[:bound] - want[:bound]).abs() <= 2.0 ** -6 * want[:bound].abs() + 1e-2)


@pytest.mark.parametrize("q,kv", [(1, 3000), (150, 3000), (300, 300), (700, 3000)])
def test_repeats_bit_for_bit(L, q, kv):
    torch = torch_mod()
    rng = np.random.default_rng(8)
    c, table = make_cache(rng, [kv], 2, 128)
    kvc, t = device_cache(L, c), i32(table)
    Q = dev_bf16(bf16_rne(rng.standard_normal((q, 4 * 128)).astype(np.float32)))
    a = [L.attention(Q, kvc, t, i32([0, q]), i32([kv]), q, kv, causal=True, return_lse=True)
         for _ in range(3)]
    torch.cuda.synchronize()
    for o, l in a[1:]:
        assert torch.equal(o, a[0][0]) and torch.equal(l, a[0][1])


# ------------------------------------------------------------------------------------------
# the chain
# ------------------------------------------------------------------------------------------

class Block:
    """The attention half: norm with MXFP8 output -> q|k|v projection -> rotary positions -> cache
    -> attention -> output projection, on small sizes (K = 512, 4 query and 2 key heads of 64)."""
    K, Hq, Hkv, dim, r = 512, 4, 2, 64, 16
    axes = [16, 24, 24]

    def __init__(self, L, seed=0):
        rng = np.random.default_rng(seed)
        f = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
        K, r = self.K, self.r
        n_qkv = (self.Hq + 2 * self.Hkv) * self.dim
        self.L = L
        self.lam = np.exp(0.5 * f(K))
        self.gamma = bf16_rne(1 + 0.1 * f(K))
        self.down, self.up = bf16_rne(0.05 * f(r, K)), bf16_rne(0.05 * f(n_qkv, r))
        self.W = bf16_rne(f(n_qkv, K) * K ** -0.5)
        self.Wo = bf16_rne(f(512, self.Hq * self.dim) * 0.06)
        self.d = dict(lam=dev(self.lam), gamma=dev_bf16(self.gamma), down=dev_bf16(self.down))
        self.pw = L.prepare_weight(dev_bf16(self.W), self.d["lam"], self.d["down"],
                                   dev_bf16(self.up), L.MXFP8)
        self.pwo = L.prepare_weight(dev_bf16(self.Wo), None, None, None, L.MXFP8)
        self.freq = L.rope_frequencies(self.axes)

    def step(self, kv, x, res, pos, table, cu, start, length, n, kv_max, workspace=None):
        L, w = self.L, self.dim
        codes, scales, D, H = L.norm_quantize_activation(x, self.d["gamma"], self.d["lam"],
                                                         self.d["down"], residual=res)
        qkv = L.gemm(codes, scales, None, D, self.pw, x.shape[0])
        qk = qkv[:, :(self.Hq + self.Hkv) * w]
        L.rope(qk, pos, self.freq, self.axes, w, out=qk)
        K = qkv[:, self.Hq * w:(self.Hq + self.Hkv) * w]
        V = qkv[:, (self.Hq + self.Hkv) * w:]
        L.kv_write(kv, K, V, table, cu, start, n)
        O = L.attention(qkv[:, :self.Hq * w], kv, table, cu, length, n, kv_max, causal=True,
                        workspace=workspace)
        Y = L.forward(O, self.pwo, None, None, None)
        return H, qkv, O, Y


def _chain_inputs(rng, rows, K):
    x = bf16_rne(rng.standard_normal((rows, K)).astype(np.float32) * 0.5)
    res = bf16_rne(rng.standard_normal((rows, K)).astype(np.float32))
    pos = rng.integers(0, 40, (rows, 3)).astype(np.int32)
    return x, res, pos


def test_chain_prompt_then_tokens(L):
    """Two ragged prompts, then single tokens.  Each stage against the oracle on the bf16 rows the
    stage before wrote: the chain's own values, not a re-derivation that rounding could part."""
    torch = torch_mod()
    from oracle import gemm as OG, layer as OL
    from tests.gpu_common import check_y
    rng = np.random.default_rng(21)
    blk = Block(L)
    w, Hq, Hkv = blk.dim, blk.Hq, blk.Hkv
    c = OA.new_cache(9, Hkv, w, fill=0xFF)
    kv = device_cache(L, c)
    table = rng.permutation(9)[:6].reshape(2, 3)
    wt = OL.prepare_weight(blk.W, blk.lam, blk.down, blk.up, "mxfp8")
    freq = blk.freq.cpu().numpy()
    have = np.array([0, 0])
    for lens in ([100, 37], [1, 1], [1, 1], [30, 1]):
        cu = np.concatenate([[0], np.cumsum(lens)])
        x, res, pos = _chain_inputs(rng, cu[-1], blk.K)
        H, qkv, O, Y = blk.step(kv, dev_bf16(x), dev_bf16(res), dev(pos), i32(table), i32(cu),
                                i32(have), i32(have + lens), max(lens), 192)
        torch.cuda.synchronize()
        o = OA.rmsnorm_quant(x, res, blk.gamma, 1e-6, blk.lam, blk.down)
        assert np.array_equal(host_bits(H), o["H"])
        y64, yb = OG.linear_mx(o["codes"], o["scales"], wt["codes"], wt["scales"], o["D"], blk.up,
                               "e4m3")
        got = host_bits(qkv)
        check_y(np.ascontiguousarray(got[:, (Hq + Hkv) * w:]), yb[:, (Hq + Hkv) * w:], "V columns")
        # rope of the product's bf16 rows: its one rounding on top of the product's
        q = bf16_bits_to_f32(got[:, :(Hq + Hkv) * w]).reshape(-1, Hq + Hkv, w)
        want = OA.rope(bf16_bits_to_f32(yb[:, :(Hq + Hkv) * w]).reshape(q.shape), pos, freq, blk.axes,
                       True, False)
        rms = np.sqrt(np.mean(want ** 2))
        assert np.all(np.abs(q - want) <= 2.0 ** -6 * np.abs(want) + 2.0 ** -6 * rms)
        OA.kv_write(c, got[:, Hq * w:(Hq + Hkv) * w], got[:, (Hq + Hkv) * w:], table, cu, have)
        assert np.array_equal(kv.k_codes.cpu().numpy(), c["kc"])
        assert np.array_equal(kv.v_codes.cpu().numpy(), c["vc"])
        have = have + lens
        qf = q[:, :Hq].astype(np.float32)
        a = OA.attention(qf, c, table, cu, have, w ** -0.5, True)
        check(a, O.float().cpu().numpy().reshape(-1, Hq, w).astype(np.float64), a["lse"], 192)
        wto = OL.prepare_weight(blk.Wo, np.ones(Hq * w, np.float32), np.zeros((0, Hq * w), np.uint16),
                                np.zeros((512, 0), np.uint16), "mxfp8")
        acto = OL.prepare_activation(host_bits(O), np.ones(Hq * w, np.float32), None,
                                     np.zeros((0, Hq * w), np.uint16), "mxfp8")
        _, yo = OL.forward(acto, wto, np.zeros((512, 0), np.uint16), "mxfp8")
        check_y(host_bits(Y), yo, "output projection")


def test_chain_captured_and_replayed(L):
    """The single-token chain in a graph, replayed on new inputs with eager work in between, equals
    the eager chain bit for bit, cache included; two graphs with a workspace each do not mix."""
    torch = torch_mod()
    rng = np.random.default_rng(22)
    blk = Block(L, 1)
    w = blk.dim
    c0, table = make_cache(rng, [2000, 1500], blk.Hkv, w)
    t = i32(table)
    cu = i32([0, 1, 2])
    x, res = (torch.zeros(2, blk.K, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pos = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    start, length = i32([1990, 1480]), i32([1991, 1481])
    graphs = []
    for _ in range(2):
        kv = device_cache(L, c0)
        ws = L.attention_workspace(2, blk.Hq, blk.Hkv, w, 2, 1, 2048)
        assert ws is not None
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            blk.step(kv, x, res, pos, t, cu, start, length, 1, 2048, ws)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        kv0 = device_cache(L, c0)
        for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
            getattr(kv, name).copy_(getattr(kv0, name))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = blk.step(kv, x, res, pos, t, cu, start, length, 1, 2048, ws)
        graphs.append((g, kv, out, ws))   # the workspace lives as long as its graph
    ref = device_cache(L, c0)
    for i in range(4):
        xb, rb, pb = _chain_inputs(rng, 2, blk.K)
        x.copy_(dev_bf16(xb)), res.copy_(dev_bf16(rb)), pos.copy_(dev(pb))
        start.copy_(i32([1990 + i, 1480 + i])), length.copy_(i32([1991 + i, 1481 + i]))
        want = blk.step(ref, x, res, pos, t, cu, start, length, 1, 2048)
        torch.cuda.synchronize()
        for g, kv, out, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for g, kv, out, _ in graphs:
            for a, b in zip(out, want):
                assert torch.equal(a, b), i
            assert torch.equal(kv.k_codes, ref.k_codes) and torch.equal(kv.v_codes, ref.v_codes)
            assert torch.equal(kv.k_scales, ref.k_scales) and torch.equal(kv.v_scales, ref.v_scales)


def test_calls_on_another_stream(L):
    """Two calls at once on streams of their own equal the same calls one after the other."""
    torch = torch_mod()
    rng = np.random.default_rng(23)
    c, table = make_cache(rng, [3000], 2, 128)
    kv, t = device_cache(L, c), i32(table)
    Q = [dev_bf16(bf16_rne(rng.standard_normal((q, 512)).astype(np.float32))) for q in (1, 140)]
    cu, ln = [i32([0, 1]), i32([0, 140])], i32([3000])
    want = [L.attention(Q[i], kv, t, cu[i], ln, Q[i].shape[0], 3000) for i in range(2)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [None, None]
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            got[i] = L.attention(Q[i], kv, t, cu[i], ln, Q[i].shape[0], 3000)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_empty_batches(L):
    torch = torch_mod()
    kv = L.kv_cache(2, 1, 64)
    Q = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    O = L.attention(Q, kv, i32([[0]]), i32([0, 0]), i32([5]), 0, 5)
    assert O.shape == (0, 64)
    L.kv_write(kv, Q, Q, i32([[0]]), i32([0, 0]), i32([0]), 0)
    k, v = L.kv_read(kv, i32([[0]]), i32([0, 0]), i32([0]), 0, 0)
    assert k.shape == (0, 64)
    torch.cuda.synchronize()
