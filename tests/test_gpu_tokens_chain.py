"""The single-token path of a block as it is used: projection of a few rows -> norm of the query and key
heads with rotary positions -> 4-bit cache -> attention over it -> output projection."""
import numpy as np
import pytest

from oracle import layer as OL, tokens as OT
from oracle.formats import bf16_bits_to_f32, bf16_rne
from tests.gpu_common import dev, dev_bf16, host_bits, torch_mod
from tests.test_gpu_attention4 import check as check_attention, device_cache, i32, make_cache
from tests.test_gpu_gemv import tolerance as gemv_tolerance

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from w4a4_quantized_dit_amd import _lib, layer
    _lib.load()
    return layer


class Block:
    """K = 512 channels, 4 query and 2 key heads of 64."""
    K, Hq, Hkv, dim, r = 512, 4, 2, 64, 16
    axes = [16, 24, 24]

    def __init__(self, L, fmt="nvfp4", seed=0):
        rng = np.random.default_rng(seed)
        f = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
        K, r, n = self.K, self.r, (self.Hq + 2 * self.Hkv) * self.dim
        self.L, self.fmt = L, fmt
        self.lam = np.exp(0.5 * f(K))
        self.down, self.up = bf16_rne(0.05 * f(r, K)), bf16_rne(0.05 * f(n, r))
        self.W, self.Wo = bf16_rne(f(n, K) * K ** -0.5), bf16_rne(f(512, self.Hq * self.dim) * 0.06)
        self.gq, self.gk = bf16_rne(1 + 0.1 * f(self.dim)), bf16_rne(1 + 0.1 * f(self.dim))
        self.d = dict(lam=dev(self.lam), down=dev_bf16(self.down), gq=dev_bf16(self.gq),
                      gk=dev_bf16(self.gk))
        code = dict(nvfp4=L.NVFP4, int4=L.INT4_G64, mxfp4=L.MXFP4)[fmt]
        self.pw = L.prepare_weight(dev_bf16(self.W), self.d["lam"], self.d["down"], dev_bf16(self.up), code)
        self.pwo = L.prepare_weight(dev_bf16(self.Wo), None, None, None, code)
        self.freq = L.rope_frequencies(self.axes)

    def step(self, kv, x, pos, table, cu, start, length, n, kv_max, ws=(None, None)):
        L, w, Hq, Hkv = self.L, self.dim, self.Hq, self.Hkv
        qkv = L.gemv(x, self.pw, self.d["lam"], self.d["down"], workspace=ws[0])
        raw = qkv.clone()
        qk = qkv[:, :(Hq + Hkv) * w]
        L.qk_norm_rope(qk, pos, self.freq, self.axes, w, Hq, self.d["gq"], self.d["gk"], out=qk)
        L.kv_write(kv, qkv[:, Hq * w:(Hq + Hkv) * w], qkv[:, (Hq + Hkv) * w:], table, cu, start, n)
        O = L.attention(qkv[:, :Hq * w], kv, table, cu, length, n, kv_max, causal=True, workspace=ws[1])
        return raw, qkv, O, L.gemv(O, self.pwo, None, None)


def _inputs(rng, rows, K):
    return bf16_rne(rng.standard_normal((rows, K)).astype(np.float32)), \
        rng.integers(0, 40, (rows, 3)).astype(np.int32)


@pytest.mark.parametrize("fmt", ["nvfp4", "int4", "mxfp4"])
def test_chain_prompt_then_tokens(L, fmt):
    """A short ragged prompt, then single tokens.  Each stage against the oracle on the bf16 rows that the
    stage before wrote."""
    torch = torch_mod()
    rng = np.random.default_rng(21)
    blk = Block(L, fmt)
    w, Hq, Hkv = blk.dim, blk.Hq, blk.Hkv
    c = OT.new_cache(9, Hkv, w, fill=0xFF)
    kv = device_cache(L, c)
    table = rng.permutation(9)[:6].reshape(2, 3)
    wt = OL.prepare_weight(blk.W, blk.lam, blk.down, blk.up, fmt)
    W = OT.weight_values(wt["codes"], wt["scales"], wt["g"], fmt)
    one, none = np.ones(Hq * w, np.float32), np.zeros((0, Hq * w), np.uint16)
    wto = OL.prepare_weight(blk.Wo, one, none, np.zeros((512, 0), np.uint16), fmt)
    Wo = OT.weight_values(wto["codes"], wto["scales"], wto["g"], fmt)
    freq = blk.freq.cpu().numpy()
    have = np.array([0, 0])
    for lens in ([40, 23], [1, 1], [1, 1], [30, 1]):
        cu = np.concatenate([[0], np.cumsum(lens)])
        x, pos = _inputs(rng, cu[-1], blk.K)
        raw, qkv, O, Y = blk.step(kv, dev_bf16(x), dev(pos), i32(table), i32(cu), i32(have),
                                  i32(have + lens), max(lens), 192)
        torch.cuda.synchronize()
        y, a = OT.gemv(x, blk.lam, blk.down, blk.up, W)
        f = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
        assert np.all(np.abs(f(raw) - y) <= gemv_tolerance(y, a, blk.K, blk.r))
        heads = f(raw)[:, :(Hq + Hkv) * w].reshape(-1, Hq + Hkv, w)
        want, z = OT.qk_norm_rope(heads, Hq, blk.gq, blk.gk, 1e-6, pos, freq, blk.axes, True)
        got = f(qkv)[:, :(Hq + Hkv) * w].reshape(heads.shape)
        assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * np.abs(z).max())
        bits = host_bits(qkv)
        OT.kv_write(c, bits[:, Hq * w:(Hq + Hkv) * w], bits[:, (Hq + Hkv) * w:], table, cu, have)
        for name, t in (("kc", kv.k_codes), ("vc", kv.v_codes), ("ks", kv.k_scales), ("vs", kv.v_scales)):
            assert np.array_equal(t.cpu().numpy(), c[name])
        have = have + lens
        want = OT.attention(got[:, :Hq], c, table, cu, have, w ** -0.5, True)
        check_attention(want, f(O).reshape(-1, Hq, w), want["lse"], 192)
        y, a = OT.gemv(host_bits(O), None, None, None, Wo)
        assert np.all(np.abs(f(Y) - y) <= gemv_tolerance(y, a, Hq * w, 0))


def test_chain_captured_and_replayed(L):
    """The single-token chain in a graph, replayed on new inputs with eager work in between, equals
    the eager chain bit for bit, cache included; two graphs with workspaces of their own do not mix."""
    torch = torch_mod()
    rng = np.random.default_rng(22)
    blk = Block(L, "int4", 1)
    w = blk.dim
    c0, table = make_cache(rng, [2000, 1500], blk.Hkv, w)
    t, cu = i32(table), i32([0, 1, 2])
    x = torch.zeros(2, blk.K, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    start, length = i32([1990, 1480]), i32([1991, 1481])
    names = ("k_codes", "v_codes", "k_scales", "v_scales")
    graphs = []
    for _ in range(2):
        kv = device_cache(L, c0)
        ws = (L.gemv_workspace(2, blk.pw), L.attention_workspace(2, blk.Hq, blk.Hkv, w, 2, 1, 2048, bits=4))
        assert ws[0] is not None and ws[1] is not None
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            blk.step(kv, x, pos, t, cu, start, length, 1, 2048, ws)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        kv0 = device_cache(L, c0)
        for name in names:
            getattr(kv, name).copy_(getattr(kv0, name))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = blk.step(kv, x, pos, t, cu, start, length, 1, 2048, ws)
        graphs.append((g, kv, out, ws))   # the workspaces live as long as their graph
    ref = device_cache(L, c0)
    for i in range(4):
        xb, pb = _inputs(rng, 2, blk.K)
        x.copy_(dev_bf16(xb)), pos.copy_(dev(pb))
        start.copy_(i32([1990 + i, 1480 + i])), length.copy_(i32([1991 + i, 1481 + i]))
        want = blk.step(ref, x, pos, t, cu, start, length, 1, 2048)
        torch.cuda.synchronize()
        for g, kv, out, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for g, kv, out, _ in graphs:
            for a, b in zip(out, want):
                assert torch.equal(a, b), i
            for name in names:
                assert torch.equal(getattr(kv, name), getattr(ref, name))


def test_chain_on_two_streams(L):
    """Two chains at once, each with its cache, on streams of their own."""
    torch = torch_mod()
    rng = np.random.default_rng(24)
    blk = Block(L, "mxfp4", 2)
    c0, table = make_cache(rng, [900, 700], blk.Hkv, blk.dim)
    t, cu, start, length = i32(table), i32([0, 1, 2]), i32([890, 690]), i32([891, 691])
    data = []
    for _ in range(2):
        x, pos = _inputs(rng, 2, blk.K)
        data.append((dev_bf16(x), dev(pos)))
    want = [blk.step(device_cache(L, c0), x, p, t, cu, start, length, 1, 1024) for x, p in data]
    caches = [device_cache(L, c0) for _ in range(2)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [None, None]
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            got[i] = blk.step(caches[i], *data[i], t, cu, start, length, 1, 1024)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for u, v in zip(a, b):
            assert torch.equal(u, v)


def test_cache_of_four_bits_beside_one_of_eight(L):
    """The same calls on both caches: what 4 bits cost is the quantisation's error, and the tensors are a
    little over half."""
    torch = torch_mod()
    rng = np.random.default_rng(25)
    n, H, dim = 700, 4, 128
    K, V = (dev_bf16(bf16_rne(rng.standard_normal((n, H * dim)).astype(np.float32))) for _ in range(2))
    Q = dev_bf16(bf16_rne(rng.standard_normal((50, 2 * H * dim)).astype(np.float32)))
    table, out, size = i32([list(range(11))]), {}, {}
    for bits in (8, 4):
        kv = L.kv_cache(11, H, dim, bits=bits)
        L.kv_write(kv, K, V, table, i32([0, n]), i32([0]), n)
        out[bits] = L.attention(Q, kv, table, i32([0, 50]), i32([n]), 50, n, causal=True).float()
        size[bits] = sum(t.numel() for t in (kv.k_codes, kv.v_codes, kv.k_scales, kv.v_scales))
    torch.cuda.synchronize()
    assert size[4] < 0.54 * size[8]
    # values within 0.116 (MXFP4 of normal values), weights within exp of scores that are as much off
    rel = float((out[4] - out[8]).norm() / out[8].norm())
    assert rel < 0.25
    assert bf16_bits_to_f32(host_bits(Q)).shape == (50, 2 * H * dim)
