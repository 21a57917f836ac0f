"""GPU tests of svdq_attn_kv8 at the limits of its host bounds (oracle and tolerances of
test_gpu_attention)."""
import numpy as np
import pytest

from oracle import attention as OA
from oracle.formats import bf16_bits_to_f32, bf16_rne
from tests.gpu_common import dev, dev_bf16, host_bits, torch_mod
from tests.test_gpu_attention import (Block, L, _chain_inputs, check, device_cache,  # noqa: F401
                                      i32, make_cache)

pytestmark = pytest.mark.gpu


def test_loose_bounds_of_rows_and_tokens(L):  # noqa: F811
    """max_rows = 2^26 + 128 and max_kv = 2^20 for 1000 rows over 300 tokens: the page range is split
    for the bounds' sake, and a block of the joining kernel for each row of the bound would be more
    than a launch holds."""
    from w4a4_quantized_dit_amd import _lib
    torch = torch_mod()
    dim, rows, kv, bound = 64, 1000, 300, (1 << 26) + 128
    assert _lib.svdq_attn_kv8_workspace_bytes(rows, 1, 1, dim, 1, bound, 1 << 20) > 0
    rng = np.random.default_rng(31)
    c, table = make_cache(rng, [kv], 1, dim)
    bits = bf16_rne(rng.standard_normal((rows, dim)).astype(np.float32))
    for causal in (False, True):
        O, lse = L.attention(dev_bf16(bits), device_cache(L, c), i32(table), i32([0, rows]),
                             i32([kv]), bound, 1 << 20, causal=causal, return_lse=True)
        torch.cuda.synchronize()
        want = OA.attention(bf16_bits_to_f32(bits).reshape(rows, 1, dim), c, table,
                            np.array([0, rows]), [kv], 0.125, causal)
        check(want, O.float().cpu().numpy().reshape(rows, 1, dim).astype(np.float64),
              lse.cpu().numpy().astype(np.float64), kv)


def test_more_rows_than_the_join_has_blocks_for(L):  # noqa: F811
    """2^22 + 200 rows with a split: the joining kernel's blocks take a second sweep."""
    from w4a4_quantized_dit_amd import _lib
    torch = torch_mod()
    dim, rows, kv, n = 64, (1 << 22) + 200, 100, 300
    assert _lib.svdq_attn_kv8_workspace_bytes(rows, 1, 1, dim, 1, rows, 1 << 18) > 0
    rng = np.random.default_rng(32)
    c, table = make_cache(rng, [kv], 1, dim)
    g = torch.Generator(device="cuda").manual_seed(6)
    Q = torch.randn(rows, dim, generator=g, device="cuda").to(torch.bfloat16)
    O, lse = L.attention(Q, device_cache(L, c), i32(table), i32([0, rows]), i32([kv]), rows, 1 << 18,
                         return_lse=True)
    torch.cuda.synchronize()
    for part in (slice(0, n), slice((1 << 22) - n, (1 << 22) + 200)):
        q = bf16_bits_to_f32(host_bits(Q[part])).reshape(-1, 1, dim)
        want = OA.attention(q, c, table, np.array([0, len(q)]), [kv], 0.125, False)
        check(want, O[part].float().cpu().numpy().reshape(-1, 1, dim).astype(np.float64),
              lse[part].cpu().numpy().astype(np.float64), kv)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q,kv,G", [(1, 2, 1), (1, 130, 4), (40, 130, 1), (600, 200, 1), (3, 5000, 1),
                                    (150, 5000, 1)])
@pytest.mark.parametrize("causal", [False, True])
def test_values_near_the_caches_largest(L, q, kv, G, dim, causal):  # noqa: F811
    """Values to 2.9e38: the weighted sum passes fp32's range unless it is scaled, the average does
    not.  Equal weights (zero queries), and weights over a wide range."""
    torch = torch_mod()
    rng = np.random.default_rng(q + kv)
    pages = (kv + 63) // 64
    c = OA.new_cache(pages + 1, 1, dim, fill=0xFF)
    table = rng.permutation(pages + 1)[:pages][None]
    K = bf16_rne(rng.standard_normal((kv, dim)).astype(np.float32))
    V = bf16_rne((rng.uniform(1.9e38, 2.9e38, (kv, dim)) * rng.choice([-1, 1], (1, dim)))
                 .astype(np.float32))
    OA.kv_write(c, K, V, table, np.array([0, kv]), [0])
    for spread in (0.0, 3.0):
        bits = bf16_rne((rng.standard_normal((q, G * dim)) * spread).astype(np.float32))
        O, lse = L.attention(dev_bf16(bits), device_cache(L, c), i32(table), i32([0, q]), i32([kv]),
                             q, kv, causal=causal, return_lse=True)
        torch.cuda.synchronize()
        assert torch.isfinite(O.float()).all()
        want = OA.attention(bf16_bits_to_f32(bits).reshape(q, G, dim), c, table, np.array([0, q]),
                            [kv], float(np.float32(dim ** -0.5)), causal)
        check(want, O.float().cpu().numpy().reshape(q, G, dim).astype(np.float64),
              lse.cpu().numpy().astype(np.float64), kv)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q,kv", [(1, 130), (40, 130), (600, 200), (3, 5000)])
def test_values_near_the_caches_smallest(L, q, kv, dim):  # noqa: F811
    """Values from 2^-119 on: right but for what may count as 0, 2^-110 of the weights' whole."""
    torch = torch_mod()
    rng = np.random.default_rng(q + kv)
    pages = (kv + 63) // 64
    c = OA.new_cache(pages, 1, dim, fill=0xFF)
    table = rng.permutation(pages)[None]
    K = bf16_rne(rng.standard_normal((kv, dim)).astype(np.float32))
    V = bf16_rne((rng.uniform(1, 2, (kv, dim)) * 2.0 ** rng.integers(-119, -95, (kv, dim)))
                 .astype(np.float32))
    OA.kv_write(c, K, V, table, np.array([0, kv]), [0])
    bits = bf16_rne(rng.standard_normal((q, dim)).astype(np.float32))
    O, lse = L.attention(dev_bf16(bits), device_cache(L, c), i32(table), i32([0, q]), i32([kv]), q, kv,
                         return_lse=True)
    torch.cuda.synchronize()
    want = OA.attention(bf16_bits_to_f32(bits).reshape(q, 1, dim), c, table, np.array([0, q]), [kv],
                        float(np.float32(dim ** -0.5)), False)
    got = O.float().cpu().numpy().reshape(q, 1, dim).astype(np.float64)
    up = 2.0 ** 60     # (the shared check allows 1e-37 on its own)
    err = np.abs(got - want["O"]) * up
    dz = want["absz"] * 132 * 2.0 ** -23
    A, W = want["absO"] * up, np.abs(want["O"]) * up
    tol = 2.0 ** -8 * (A + W) * (1 + 2.0 ** -7) + (2 * np.expm1(dz)[..., None] + 2.0 ** -20
                                                  + kv * 2.0 ** -23) * (A + W) + 2.0 ** -110 * up
    assert np.all(err <= tol)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q", [1, 64, 600])
@pytest.mark.parametrize("causal", [False, True])
def test_length_past_the_page_table(L, q, dim, causal):  # noqa: F811
    """kv_len is limited to the table's 64·max_blocks tokens, the causal mask's last row sees them all;
    a negative one counts as none."""
    torch = torch_mod()
    rng = np.random.default_rng(33)
    c, table = make_cache(rng, [448, 448, 448], 1, dim)
    bits = bf16_rne(rng.standard_normal((3 * q, dim)).astype(np.float32))
    cu, lens = np.array([0, q, 2 * q, 3 * q]), [10 ** 6, 2 ** 31 - 1, -5]
    O, lse = L.attention(dev_bf16(bits), device_cache(L, c), i32(table), i32(cu), i32(lens), q, 448,
                         causal=causal, return_lse=True)
    torch.cuda.synchronize()
    qf = bf16_bits_to_f32(bits).reshape(3 * q, 1, dim)
    want = OA.attention(qf, c, table, cu, [448, 448, 0], float(np.float32(dim ** -0.5)), causal)
    check(want, O.float().cpu().numpy().reshape(3 * q, 1, dim).astype(np.float64),
          lse.cpu().numpy().astype(np.float64), 448)


def test_lse_of_the_chain(L):  # noqa: F811
    """The attention half as it is used, prompts and then single tokens: the lse that the attention
    gives there, against the oracle on the rows that the stages before it wrote."""
    torch = torch_mod()

    class Noted:
        """The layer, with the lse of its attention kept."""
        def __getattr__(self, name):
            return getattr(L, name)

        def attention(self, *a, **k):
            O, self.lse = L.attention(*a, return_lse=True, **k)
            return O

    rng = np.random.default_rng(34)
    noted = Noted()
    blk = Block(noted)
    w, Hq, Hkv = blk.dim, blk.Hq, blk.Hkv
    c = OA.new_cache(9, Hkv, w, fill=0xFF)
    kv = device_cache(L, c)
    table = rng.permutation(9)[:6].reshape(2, 3)
    have = np.array([0, 0])
    for lens in ([100, 37], [1, 1], [30, 1]):
        cu = np.concatenate([[0], np.cumsum(lens)])
        x, res, pos = _chain_inputs(rng, cu[-1], blk.K)
        _, qkv, O, _ = blk.step(kv, dev_bf16(x), dev_bf16(res), dev(pos), i32(table), i32(cu),
                                i32(have), i32(have + lens), max(lens), 192)
        torch.cuda.synchronize()
        have = have + lens
        got = host_bits(qkv)
        for name, t in (("kc", kv.k_codes), ("vc", kv.v_codes), ("ks", kv.k_scales), ("vs", kv.v_scales)):
            c[name] = t.cpu().numpy()
        want = OA.attention(bf16_bits_to_f32(got[:, :Hq * w]).reshape(-1, Hq, w), c, table, cu, have,
                            w ** -0.5, True)
        check(want, O.float().cpu().numpy().reshape(-1, Hq, w).astype(np.float64),
              noted.lse.cpu().numpy().astype(np.float64), 192)
