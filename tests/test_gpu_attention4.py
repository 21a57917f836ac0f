"""GPU parity of svdq_attn_kv4 against the float64 oracle.

Tolerance of O (derived, per element; A = Σ p|v|, the magnitude the weights' errors act on):
  - each weight is rounded to bf16 once, at most half a step:            2^-8·A
  - the result is rounded to bf16 once:                                  2^-8·|O|
  - scores: up to 128 products, each exact in fp32 (8 bits times 3), summed with at most a whole step,
    2^-23, lost an addition, and four more steps for c and the exponent's argument: dz = 132·2^-23·Z
    with Z = scale·max_t Σ|q k|; a weight moves by that, in numerator and denominator:
                                                                         2·dz·(A + |O|)
  - exponential, fp32 sums: 2^-21 + tokens·2^-24, twice, of A
lse: the score's error, plus the relative error of the sum."""
import numpy as np
import pytest

from oracle import tokens as OT
from oracle.formats import bf16_bits_to_f32, bf16_rne
from tests.gpu_common import dev, dev_bf16, torch_mod

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


def fill(c, K, V, table, lens):
    """The oracle's kv_write of whole sequences, a page at a time."""
    dim, heads = c["dim"], c["ks"].shape[1]
    cu = np.concatenate([[0], np.cumsum(lens)])
    for is_v, bits, codes, scales in ((0, K, c["kc"], c["ks"]), (1, V, c["vc"], c["vs"])):
        q, s = OT.quantise(bf16_bits_to_f32(bits).reshape(-1, heads, dim))
        at_c, at_s = OT._places(dim, is_v)
        for b, n in enumerate(lens):
            for p in range((n + 63) // 64):
                m = min(64, n - 64 * p)
                rows = slice(cu[b] + 64 * p, cu[b] + 64 * p + m)
                for h in range(heads):
                    codes[table[b, p], h, at_c[:m]] = q[rows, h]
                    scales[table[b, p], h, at_s[:m]] = s[rows, h]


def make_cache(rng, lens, heads, dim, spread=1.0, extra=3, garbage=0xFF):
    """Cache with `lens` tokens a sequence on shuffled pages, every other byte `garbage`."""
    blocks = max(1, max((n + 63) // 64 for n in lens))
    pages = len(lens) * blocks + extra
    c = OT.new_cache(pages, heads, dim, fill=garbage)
    table = rng.permutation(pages)[:len(lens) * blocks].reshape(len(lens), blocks)
    w = heads * dim
    K = bf16_rne((rng.standard_normal((sum(lens), w)) * spread).astype(np.float32))
    V = bf16_rne((rng.standard_normal((sum(lens), w)) * np.exp(rng.standard_normal((sum(lens), 1))))
                 .astype(np.float32))
    fill(c, K, V, table, lens)
    return c, table


def device_cache(L, c):
    return L.KVCache(dev(c["kc"]), dev(c["vc"]), dev(c["ks"]), dev(c["vs"]), c["dim"], bits=4)


def check(want, O, lse, tokens, what=""):
    """NaN exactly where the oracle has it, the rest within the tolerance."""
    assert np.array_equal(np.isnan(O), np.isnan(want["O"])), what
    assert np.array_equal(np.isnan(lse), np.isnan(want["lse"])), what
    want = {k: np.nan_to_num(v, nan=0.0, neginf=-np.inf) for k, v in want.items()}
    O, lse = np.nan_to_num(O), np.nan_to_num(lse, neginf=-np.inf)
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


def attend(L, c, table, cu, kv_lens, bits, Hq, dim, causal, max_q, max_kv, scale=None, what=""):
    """One call against the oracle."""
    torch = torch_mod()
    scale = dim ** -0.5 if scale is None else scale
    O, lse = L.attention(dev_bf16(bits), device_cache(L, c), i32(table), i32(cu), i32(kv_lens), max_q,
                         max_kv, scale=scale, causal=causal, return_lse=True)
    torch.cuda.synchronize()
    rows = len(bits)
    q = bf16_bits_to_f32(bits).reshape(rows, Hq, dim)
    with np.errstate(invalid="ignore"):
        want = OT.attention(q, c, np.asarray(table), cu, kv_lens, float(np.float32(scale)), causal)
    check(want, O.float().cpu().numpy().reshape(rows, Hq, dim).astype(np.float64),
          lse.cpu().numpy().astype(np.float64), max(kv_lens), what)
    return O, lse, want


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
    want = OT.attention(q, c, table, cu, kv_lens, float(np.float32(scale)), causal)
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
    assert _lib.svdq_attn_kv4_workspace_bytes(q, 2, 1, dim, 1, q, 5000) > 0
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


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q", [1, 70, 600])
def test_rising_scores_every_page(L, q, dim):
    """Keys aligned with the query and growing page by page: every page raises the maximum."""
    n = 1000
    rng = np.random.default_rng(5)
    u = rng.standard_normal(dim).astype(np.float32)
    K = bf16_rne(u[None] * np.linspace(-3, 12, n, dtype=np.float32)[:, None])
    V = bf16_rne(rng.standard_normal((n, dim)).astype(np.float32))
    c = OT.new_cache(16, 1, dim)
    table = np.arange(16)[None]
    fill(c, K, V, table, [n])
    bits = bf16_rne(np.tile(u, (q, 1)) * np.linspace(0.1, 1, q, dtype=np.float32)[:, None])
    attend(L, c, table, np.array([0, q]), [n], bits, 1, dim, False, q, n)


@pytest.mark.parametrize("q", [1, 50, 600])
def test_zero_rows_and_blocks_of_every_size(L, q):
    """All-zero queries weigh every token alike; tokens and channel blocks from the smallest exponent to
    large values side by side keep their place in the sum."""
    dim, n = 128, 192
    rng = np.random.default_rng(6)
    size = 2.0 ** rng.integers(-130, 20, (n, dim // 32))
    V = (rng.standard_normal((n, dim // 32, 32)) * size[..., None]).reshape(n, dim).astype(np.float32)
    V[64:100] = 0
    K = rng.standard_normal((n, dim)).astype(np.float32)
    K[:64] = 0
    c = OT.new_cache(3, 1, dim)
    table = np.array([[0, 1, 2]])
    fill(c, bf16_rne(K), bf16_rne(V), table, [n])
    attend(L, c, table, np.array([0, q]), [n], bf16_rne(np.zeros((q, dim), np.float32)), 1, dim, False, q, n)
    bits = bf16_rne(rng.standard_normal((q, dim)).astype(np.float32))
    attend(L, c, table, np.array([0, q]), [n], bits, 1, dim, True, q, n)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q", [1, 50, 600])
def test_one_token_and_one_channel_at_a_time(L, q, dim):
    """Values that tell tokens and channels apart, one token seen with all the weight: O is that token's
    row, bit for bit up to one rounding, wherever it lies in its page."""
    torch = torch_mod()
    n = 150
    rng = np.random.default_rng(7)
    V = rng.choice([0.5, 1, 1.5, 2, 3, 4, 6], (n, dim)) * rng.choice([-1, 1], (n, dim)) \
        * 2.0 ** rng.integers(-3, 4, (n, dim // 32)).repeat(32, axis=1)
    V = V.astype(np.float32)
    c = OT.new_cache(3, 1, dim)
    table = np.array([[2, 0, 1]])
    for t in (0, 1, 5, 8, 15, 31, 32, 63, 64, 100, 149):
        K = np.zeros((n, dim), np.float32)
        K[t, t % dim] = 6.0
        fill(c, bf16_rne(K), bf16_rne(V), table, [n])
        bits = np.zeros((q, dim), np.float32)
        bits[:, t % dim] = 64.0
        O = L.attention(dev_bf16(bf16_rne(bits)), device_cache(L, c), i32(table), i32([0, q]), i32([n]), q, n,
                        scale=1.0)
        torch.cuda.synchronize()
        want, _ = OT.kv_values(c, table[0], n, 0, 1)
        assert np.array_equal(O.float().cpu().numpy(), np.tile(want[t], (q, 1))), t


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q,kv", [(1, 400), (70, 400), (3, 5000), (150, 5000), (600, 400),
                                  (600, 5000)])
@pytest.mark.parametrize("causal", [False, True])
def test_missing_pages_beside_a_garbage_page(L, q, kv, dim, causal):
    """Page 0, which no sequence owns, is all NaN blocks: nothing of it shows where pages are missing."""
    torch = torch_mod()
    rng = np.random.default_rng(17)
    c, table = make_cache(rng, [kv], 1, dim)
    free = next(p for p in range(len(c["kc"])) if p not in table) if 0 in table else 0
    for name in ("kc", "vc", "ks", "vs"):     # page 0 <-> the one that holds nothing
        c[name][[0, free]] = c[name][[free, 0]]
    table = np.where(table == 0, free, table)
    assert np.all(c["vs"][0] == 0xFF)
    for miss in ([0], [1, 3], [table.shape[1] - 1], list(range(table.shape[1]))):
        t = table.copy()
        t[0, miss] = [-1, 10 ** 6][len(miss) % 2]
        bits = bf16_rne(rng.standard_normal((q, dim)).astype(np.float32))
        O, _, _ = attend(L, c, t, np.array([0, q]), [kv], bits, 1, dim, causal, q, kv, what=str(miss))
        assert torch.isfinite(O.float()).all()


def test_length_past_the_table_is_limited_to_it(L):
    rng = np.random.default_rng(18)
    for q, causal in ((1, True), (70, False), (600, False)):
        c, table = make_cache(rng, [448], 2, 64)     # whole pages: every slot of the table holds a token
        bits = bf16_rne(rng.standard_normal((q, 2 * 64)).astype(np.float32))
        attend(L, c, table, np.array([0, q]), [10 ** 6], bits, 2, 64, causal, q, 448)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("G", [1, 2])
@pytest.mark.parametrize("q,kv", [(1, 70), (1, 5000), (3, 130), (15, 4100), (64, 64), (70, 300),
                                  (150, 5000), (300, 300), (600, 700), (600, 5000)])
@pytest.mark.parametrize("causal", [False, True])
def test_nan_in_seen_and_hidden_tokens(L, q, kv, G, dim, causal):
    """Infinities and NaN in keys, values and queries: they show where they are seen, and a row that
    does not see a token has nothing of it, in the pages that its block shares with later rows too."""
    rng = np.random.default_rng(q + kv)
    for where in ("v", "k", "q", "all"):
        pages = (kv + 63) // 64
        c = OT.new_cache(2 * pages + 1, 1, dim, fill=0xFF)
        table = rng.permutation(2 * pages + 1)[:2 * pages].reshape(2, pages)
        K, V = (bf16_rne(rng.standard_normal((2 * kv, dim)).astype(np.float32)) for _ in range(2))
        bits = bf16_rne(rng.standard_normal((2 * q, G * dim)).astype(np.float32))
        late = max(0, kv - q) + rng.integers(0, min(q, kv), 3)     # tokens that some rows see
        if where in ("v", "all"):
            V[late, rng.integers(0, dim, 3)] = [0x7FC0, 0x7F80, 0xFF80]
            V[kv - 1, dim - 1] = 0x7FC0
        if where in ("k", "all"):
            K[kv + late[:1], rng.integers(0, dim, 1)] = 0x7FC0     # the second sequence's
        if where in ("q", "all"):
            bits[[q // 2, 2 * q - 1], [3, G * dim - 1]] = [0x7FC0, 0xFF80]
        fill(c, K, V, table, [kv, kv])
        _, _, want = attend(L, c, table, np.array([0, q, 2 * q]), [kv, kv], bits, G, dim, causal, q, kv,
                            what=where)
        assert np.isnan(want["O"]).any()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q", [1, 32, 300, 600])
def test_scores_are_summed_in_fp32(L, q, dim):
    """One token: lse is the score itself.  Channels over 2^14 side by side, of both signs, so that a sum
    aligned to its largest product with fewer bits than fp32 shows."""
    torch = torch_mod()
    rng = np.random.default_rng(dim + q)
    K = rng.choice([-1.0, 1.0], (1, dim)) * 2.0 ** -rng.integers(0, 3, (1, dim)) \
        * 2.0 ** -(6 * np.arange(dim // 32)).repeat(32)
    Q = rng.standard_normal((q, dim)) * 2.0 ** -rng.integers(0, 8, (q, dim))
    c = OT.new_cache(1, 1, dim)
    fill(c, bf16_rne(K.astype(np.float32)), bf16_rne(K.astype(np.float32)), np.array([[0]]), [1])
    bits = bf16_rne(Q.astype(np.float32))
    _, lse = L.attention(dev_bf16(bits), device_cache(L, c), i32([[0]]), i32([0, q]), i32([1]), q, 1,
                         scale=1.0, return_lse=True)
    torch.cuda.synchronize()
    k, _ = OT.kv_values(c, np.array([0]), 1, 0, 0)
    qf = bf16_bits_to_f32(bits).astype(np.float64)
    # at most a whole step, 2^-23, of a partial sum an addition, and two for lse itself
    lim = (dim + 2) * 2.0 ** -23 * (np.abs(qf) @ np.abs(k).T)
    assert np.all(np.abs(lse.cpu().numpy() - qf @ k.T) <= lim)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q", [1, 40, 600])
@pytest.mark.parametrize("sign", [1, -1])
def test_very_large_scores(L, q, dim, sign):
    """Scores of one sign up to 2^26, exact in fp32: the largest takes the whole weight (or all that
    are as large), and lse is that score."""
    torch = torch_mod()
    n = 200
    K = np.zeros((n, dim), np.float32)
    K[:, 5] = sign * 2.0 ** 13 * (1 + (np.arange(n) * 37 % n) / n)
    V = np.random.default_rng(3).standard_normal((n, dim)).astype(np.float32)
    Q = np.zeros((q, dim), np.float32)
    Q[:, 5] = 2.0 ** 12
    c = OT.new_cache(4, 1, dim)
    table = np.array([[2, 0, 3, 1]])
    fill(c, bf16_rne(K), bf16_rne(V), table, [n])
    bits = bf16_rne(Q)
    O, lse = L.attention(dev_bf16(bits), device_cache(L, c), i32(table), i32([0, q]), i32([n]), q, n,
                         scale=1.0, return_lse=True)
    torch.cuda.synchronize()
    qf = bf16_bits_to_f32(bits).reshape(q, 1, dim)
    want = OT.attention(qf, c, table, np.array([0, q]), [n], 1.0, False)
    got = O.float().cpu().numpy().reshape(q, 1, dim)
    # weights that are equal (the codes of several keys are) or 0: only the roundings of the weights
    # and of the result are left, 2^-8 each, of Σ p|v|
    assert np.all(np.abs(got - want["O"]) <= 2.0 ** -6 * want["absO"])
    # lse = (scale / c)·(c·z): c·z rounded (made up for by the sum), the last product: 2^-23 and room
    assert np.all(np.abs(lse.cpu().numpy() - want["lse"]) <= 2.0 ** -22 * np.abs(want["lse"]))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q", [1, 40, 600])
def test_the_largest_values_that_the_cache_holds(L, q, dim):
    """Every value saturated at 6·2^85: the weighted sum stays finite and is that value; tokens of the
    smallest exponent: their mean."""
    torch = torch_mod()
    n = 5000
    rng = np.random.default_rng(4)
    for value in (3e38, 2.0 ** -108):
        V = np.full((n, dim), value, np.float32)
        K = rng.standard_normal((n, dim)).astype(np.float32)
        c = OT.new_cache(79, 1, dim)
        table = np.arange(79)[None]
        fill(c, bf16_rne(K), bf16_rne(V), table, [n])
        bits = bf16_rne((4 * rng.standard_normal((q, dim))).astype(np.float32))
        O = L.attention(dev_bf16(bits), device_cache(L, c), i32(table), i32([0, q]), i32([n]), q, n)
        torch.cuda.synchronize()
        want = OT.kv_values(c, table[0], 1, 0, 1)[0][0, 0]
        # each weight rounded to bf16 against the unrounded sum, the result once more
        assert np.all(np.abs(O.float().cpu().numpy() - want) <= 2.0 ** -7 * want * (1 + 2.0 ** -7))


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


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q,kv", [(40, 40000), (1, 60000)])
def test_more_pages_than_a_block_looks_up_at_once(L, q, kv, dim):
    """Page numbers are looked up 61 (many rows) or 256 (few) at a time: longer walks, with missing
    pages, in the order of the table."""
    rng = np.random.default_rng(10)
    for heads in (1, 8):
        if heads == 8 and q == 1:
            continue
        c, table = make_cache(rng, [kv], 1, dim, garbage=0x55)
        t = table.copy()
        t[0, [5, 62, 300]] = -1
        Hq = 4 * heads
        bits = bf16_rne(rng.standard_normal((q, Hq * dim)).astype(np.float32))
        attend(L, c, t, np.array([0, q]), [kv], bits, Hq, dim, True, q, kv)


@pytest.mark.parametrize("dim", [64, 128])
def test_a_block_walks_hundreds_of_pages(L, dim):
    """Enough heads and sequences that nothing is split: each block walks its whole sequence."""
    from w4a4_quantized_dit_amd import _lib
    rng = np.random.default_rng(11)
    heads, B, kv = 64, 8, 17000
    assert _lib.svdq_attn_kv4_workspace_bytes(B, heads, heads, dim, B, 1, kv) == 0
    blocks = (kv + 63) // 64
    c, table = make_cache(rng, [kv], 1, dim, garbage=0x55)
    big = OT.new_cache(len(c["kc"]), 1, dim)
    for k in ("kc", "vc", "ks", "vs"):
        big[k] = np.repeat(c[k], heads, axis=1)
    t = np.repeat(table, B, axis=0)
    torch = torch_mod()
    one = bf16_rne(rng.standard_normal((1, dim)).astype(np.float32))
    Q = np.tile(one, (B, heads))
    O, lse = L.attention(dev_bf16(Q), device_cache(L, big), i32(t), i32(np.arange(B + 1)), i32([kv] * B), 1, kv,
                         causal=True, return_lse=True)
    torch.cuda.synchronize()
    want = OT.attention(bf16_bits_to_f32(one).reshape(1, 1, dim), c, table, [0, 1], [kv],
                        float(np.float32(dim ** -0.5)), True)
    O = O.float().cpu().numpy().reshape(B * heads, 1, dim).astype(np.float64)
    assert np.all(O == O[:1])
    check(want, O[:1], lse.cpu().numpy().reshape(-1)[:1, None].astype(np.float64), kv)
    assert blocks > 256


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
    kv = L.kv_cache(2, 1, 64, bits=4)
    Q = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    O = L.attention(Q, kv, i32([[0]]), i32([0, 0]), i32([5]), 0, 5)
    assert O.shape == (0, 64)
    L.kv_write(kv, Q, Q, i32([[0]]), i32([0, 0]), i32([0]), 0)
    k, v = L.kv_read(kv, i32([[0]]), i32([0, 0]), i32([0]), 0, 0)
    assert k.shape == (0, 64) and v.shape == (0, 64)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("G,q_lens", [(1, [1] * 6), (5, [1] * 6), (16, [1] * 6), (4, [4, 1, 2, 3, 4, 0]),
                                      (1, [16, 3, 1, 16, 7, 2])])
@pytest.mark.parametrize("max_kv", [5000, 300000, 64])
def test_sixteen_rows_over_ragged_splits(L, dim, causal, G, q_lens, max_kv):
    """Splits of one length: shorter sequences have fewer, the empty one none, whatever the bound says."""
    run(L, q_lens, [5000, 3, 0, 700, 513, 4999], 2 * G, 2, dim, causal, seed=G, tail=2, max_kv=max_kv)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_sixteen_rows_of_many_heads(L, dim, causal):
    """More sequences and heads than compute units."""
    kv = np.random.default_rng(12).integers(0, 400, 44)
    run(L, [1] * 22 + [3, 2] * 11, [int(v) for v in kv], 24, 6, dim, causal, seed=4)


@pytest.mark.parametrize("dim", [64, 128])
def test_eight_waves_walk_hundreds_of_pages(L, dim):
    """As many heads and sequences as compute units: one block each, which looks page numbers up twice."""
    from w4a4_quantized_dit_amd import _lib
    rng = np.random.default_rng(13)
    heads, B, kv = 64, 4, 33000
    assert _lib.svdq_attn_kv4_workspace_bytes(B, heads, heads, dim, B, 1, kv) == 0
    c, table = make_cache(rng, [kv], 1, dim, garbage=0x55)
    table = table.copy()
    table[0, [5, 62, 514]] = -1
    big = OT.new_cache(len(c["kc"]), 1, dim)
    for k in ("kc", "vc", "ks", "vs"):
        big[k] = np.repeat(c[k], heads, axis=1)
    torch = torch_mod()
    one = bf16_rne(rng.standard_normal((1, dim)).astype(np.float32))
    O, lse = L.attention(dev_bf16(np.tile(one, (B, heads))), device_cache(L, big),
                         i32(np.repeat(table, B, axis=0)), i32(np.arange(B + 1)), i32([kv] * B), 1, kv,
                         causal=True, return_lse=True)
    torch.cuda.synchronize()
    want = OT.attention(bf16_bits_to_f32(one).reshape(1, 1, dim), c, table, [0, 1], [kv],
                        float(np.float32(dim ** -0.5)), True)
    O = O.float().cpu().numpy().reshape(B * heads, 1, dim).astype(np.float64)
    assert np.all(O == O[:1])
    check(want, O[:1], lse.cpu().numpy().reshape(-1)[:1, None].astype(np.float64), kv)
