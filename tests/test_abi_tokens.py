"""CPU tests of the refusals of the single-token and 4-bit entry points (nothing is enqueued for an
invalid call) and of the binding's checks of their tensors."""
import ctypes

import pytest
import torch

from w4a4_quantized_dit_amd import _lib, layer

OK, INVALID, SHAPE, NULLP = 0, 1, 2, 3
P = 1 << 20          # a fake, aligned, non-NULL "device pointer" (never dereferenced)
MIS = P + 4
BF, I32, U8 = torch.bfloat16, torch.int32, torch.uint8


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def _err(lib):
    return lib.svdq_last_error().decode()


def _dims(*v):
    return ctypes.cast((ctypes.c_int64 * max(1, len(v)))(*v), ctypes.c_void_p)


def test_qk_norm_rope_refusals(lib):
    def call(**kw):
        a = dict(X=P, M=4, ldx=384, hq=2, hk=1, dim=128, gq=P, gk=P, eps=1e-6, pos=P, freq=P, n=3,
                 dims=_dims(32, 48, 48), Y=P, ldy=384)
        a.update(kw)
        return lib.svdq_qk_norm_rope(a["X"], a["M"], a["ldx"], a["hq"], a["hk"], a["dim"], a["gq"],
                                     a["gk"], a["eps"], a["pos"], a["freq"], a["n"], a["dims"], 1,
                                     a["Y"], a["ldy"], None)
    for k in ("X", "pos", "freq", "dims", "Y"):
        assert call(**{k: None}) == NULLP, k
    for k in ("X", "Y", "gq", "gk"):
        assert call(**{k: MIS}) == SHAPE and "aligned" in _err(lib), k
    assert call(M=0) == SHAPE and call(M=(1 << 28) + 1) == SHAPE
    assert call(hq=0, hk=0) == SHAPE and call(hq=-1) == SHAPE and call(hk=-1) == SHAPE
    assert call(hq=(1 << 20) + 1) == SHAPE and call(hk=(1 << 20) + 1) == SHAPE
    for dim in (0, 8, 100, 272):
        assert call(dim=dim) == SHAPE, dim
    assert call(n=0) == SHAPE and call(n=5, dims=_dims(16, 16, 16, 16, 16)) == SHAPE
    assert call(dims=_dims(33, 47, 48)) == SHAPE               # odd
    assert call(dims=_dims(44, 44, 48)) == SHAPE               # 136 > dim
    assert call(dims=_dims(2, 2, 2)) == SHAPE                  # 6, not a multiple of 16
    assert call(ldx=376, ldy=376) == SHAPE and call(ldx=392) == INVALID
    for eps in (0.0, -1.0, 1e-31, 1e30, float("inf"), float("nan")):
        assert call(eps=eps) == INVALID, eps


@pytest.mark.parametrize("name", ["svdq_kv4_write", "svdq_kv4_read"])
def test_cache_refusals(lib, name):
    f = getattr(lib, name)

    def call(**kw):
        a = dict(K=P, ldk=256, V=P, ldv=256, rows=4, h=2, dim=128, cu=P, start=P, B=1, mr=4, bt=P,
                 mb=3, n=5, kc=P, vc=P, ks=P, vs=P)
        a.update(kw)
        return f(a["K"], a["ldk"], a["V"], a["ldv"], a["rows"], a["h"], a["dim"], a["cu"],
                 a["start"], a["B"], a["mr"], a["bt"], a["mb"], a["n"], a["kc"], a["vc"], a["ks"],
                 a["vs"], None)
    for k in ("K", "V", "cu", "start", "bt", "kc", "vc", "ks", "vs"):
        assert call(**{k: None}) == NULLP and name in _err(lib), k
    for k in ("K", "V", "kc", "vc", "ks", "vs"):
        assert call(**{k: MIS}) == SHAPE, k
    for dim in (0, 32, 96, 256):
        assert call(dim=dim) == SHAPE, dim
    assert call(h=0) == SHAPE and call(h=65536) == SHAPE
    assert call(B=0) == SHAPE and call(B=65536) == SHAPE
    assert call(rows=-1) == SHAPE and call(mr=-1) == SHAPE
    assert call(mb=0) == SHAPE and call(n=0) == SHAPE
    assert call(ldk=248) == SHAPE and call(ldv=260) == SHAPE
    assert call(rows=0) == OK and call(mr=0) == OK             # nothing to do


def test_attention_refusals(lib):
    def call(**kw):
        a = dict(Q=P, ldq=512, rows=4, hq=4, hk=2, dim=128, cu=P, kl=P, B=1, mr=4, mkv=100, bt=P,
                 mb=3, n=5, kc=P, vc=P, ks=P, vs=P, scale=0.1, O=2 * P, ldo=512, lse=P, ws=None,
                 wb=0)
        a.update(kw)
        return lib.svdq_attn_kv4(a["Q"], a["ldq"], a["rows"], a["hq"], a["hk"], a["dim"], a["cu"],
                                 a["kl"], a["B"], a["mr"], a["mkv"], a["bt"], a["mb"], a["n"],
                                 a["kc"], a["vc"], a["ks"], a["vs"], a["scale"], 1, a["O"],
                                 a["ldo"], a["lse"], a["ws"], a["wb"], None)
    for k in ("Q", "O", "cu", "kl", "bt", "kc", "vc", "ks", "vs"):
        assert call(**{k: None}) == NULLP and "svdq_attn_kv4" in _err(lib), k
    for k in ("Q", "O", "kc", "vc", "ks", "vs", "lse"):
        assert call(**{k: MIS}) == SHAPE, k
    assert call(dim=96) == SHAPE and call(hq=3) == SHAPE and call(hq=1) == SHAPE
    assert call(hk=0) == SHAPE and call(ldq=504) == SHAPE and call(ldo=516) == SHAPE
    assert call(mkv=-1) == INVALID and call(O=P) == INVALID
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=s) == INVALID
    assert call(rows=0) == OK and call(mr=0) == OK
    assert call(rows=(1 << 28) + 1) == SHAPE and call(rows=1 << 28, mr=1 << 28) == SHAPE
    need = lib.svdq_attn_kv4_workspace_bytes(4, 4, 2, 128, 1, 4, 20000)
    assert need > 0 and need % (4 * 4 * 130 * 4) == 0
    big = dict(mkv=20000, mb=400)
    assert call(**big) == NULLP and "workspace" in _err(lib)
    assert call(ws=P, wb=need - 1, **big) == SHAPE
    assert call(ws=P + 16, wb=need, **big) == SHAPE
    for bad in ((4, 3, 2, 128, 1, 4, 9), (4, 4, 2, 96, 1, 4, 9), (4, 4, 0, 64, 1, 4, 9),
                (-1, 4, 2, 64, 1, 4, 9), (4, 4, 2, 64, 0, 4, 9), (4, 4, 2, 64, 1, 4, -9)):
        assert lib.svdq_attn_kv4_workspace_bytes(*bad) == -1, bad
    assert lib.svdq_attn_kv4_workspace_bytes(4, 4, 2, 128, 1, 4, 64) == 0


def test_gemv_refusals(lib):
    def call(**kw):
        a = dict(fmt=0, X=P, M=4, K=512, ldx=512, lam=P, down=P, r=8, c=P, s=P, g=P, up=P, N=24,
                 Y=2 * P, ldy=24, ws=3 * P, wb=1 << 20)
        a.update(kw)
        return lib.svdq_w4a16_gemv(a["fmt"], a["X"], a["M"], a["K"], a["ldx"], a["lam"], a["down"],
                                   a["r"], a["c"], a["s"], a["g"], a["up"], a["N"], a["Y"], a["ldy"],
                                   a["ws"], a["wb"], None)
    for k in ("X", "down", "c", "s", "g", "up", "Y", "ws"):
        assert call(**{k: None}) == NULLP, k
    for k in ("X", "lam", "down", "c", "s", "up"):
        assert call(**{k: MIS}) == SHAPE and "aligned" in _err(lib), k
    assert call(fmt=4) == INVALID and call(fmt=3) == INVALID and call(fmt=-1) == INVALID
    for M in (0, -1, 65, 1 << 40):
        assert call(M=M) == SHAPE, M
    for K in (0, 128, 300, (1 << 22) + 256):
        assert call(K=K, ldx=1 << 23) == SHAPE, K
    assert call(ldx=(1 << 24) + 8) == SHAPE
    assert call(N=0) == SHAPE and call(N=(1 << 28) + 1, ldy=1 << 29) == SHAPE
    assert call(ldx=504) == SHAPE and call(ldx=516) == SHAPE and call(ldy=23) == SHAPE
    assert call(r=4) == SHAPE and call(r=136) == SHAPE and call(r=-8) == SHAPE
    need = lib.svdq_w4a16_gemv_workspace_bytes(4, 24, 512, 8)
    assert need >= 4 * 24 * 4 + 4 * 8 * 4
    assert call(wb=need - 1) == SHAPE and call(ws=3 * P + 16) == SHAPE
    assert 0 < lib.svdq_w4a16_gemv_workspace_bytes(4, 24, 512, 0) < need
    for bad in ((0, 24, 512, 8), (65, 24, 512, 8), (4, 24, 500, 8), (4, 24, 0, 8), (4, 24, 512, 4),
                (4, 24, 512, 136), (4, 24, 512, -8), (4, 24, (1 << 22) + 256, 8), (4, 0, 512, 8),
                (4, (1 << 28) + 1, 512, 8)):
        assert lib.svdq_w4a16_gemv_workspace_bytes(*bad) == -1, bad


def _calls(device):
    """One good call of each operator, with every tensor on `device`."""
    z = lambda dt, *s: torch.zeros(*s, dtype=dt, device=device)  # noqa: E731
    X = z(BF, 4, 256)
    kv = layer.KVCache(z(U8, 3, 2, 2048), z(U8, 3, 2, 2048), z(U8, 3, 2, 128), z(U8, 3, 2, 128), 64, 4)
    table, cu, seq = z(I32, 1, 3), z(I32, 2), z(I32, 1)
    return {
        "qk": lambda: layer.qk_norm_rope(X, z(I32, 4, 3), z(torch.float64, 32), [16, 24, 24], 64, 3,
                                         z(BF, 64), None, out=z(BF, 4, 256)),
        "write": lambda: layer.kv_write(kv, X[:, :128], X[:, 128:], table, cu, seq, 4),
        "read": lambda: layer.kv_read(kv, table, cu, seq, 4, 4, out=[z(BF, 4, 128)] * 2),
        "attention": lambda: layer.attention(X, kv, table, cu, seq, 4, 64, causal=True,
                                             out=z(BF, 4, 256)),
        "gemv": lambda: layer.gemv(X, layer.PreparedWeight(layer.INT4_G64, 8, 256, 0, z(U8, 8, 128),
                                                           z(torch.float16, 8, 4), None, None),
                                   None, None, out=z(BF, 4, 8)),
    }


@pytest.mark.parametrize("device", ["cpu", "meta"])
@pytest.mark.parametrize("op", ["qk", "write", "read", "attention", "gemv"])
def test_tensors_that_are_not_on_a_device_are_refused(op, device, monkeypatch):
    def enqueue(*a):
        raise AssertionError("the call went on")
    monkeypatch.setattr(_lib._Args, "call", enqueue)
    with pytest.raises(ValueError, match="must be a device tensor"):
        _calls(device)[op]()


@pytest.fixture
def on_device(monkeypatch):
    """Host tensors pass for device tensors; the entry points' names are collected instead of called."""
    names = []

    def at(self, t, name):
        self.dev = 0
        return P
    monkeypatch.setattr(_lib._Args, "_at", at)
    monkeypatch.setattr(_lib._Args, "call", lambda self, name, *a: names.append(name))
    return names


def test_the_calls_above_are_good_ones(on_device):
    for f in _calls("cpu").values():
        f()
    assert on_device == ["svdq_qk_norm_rope", "svdq_kv4_write", "svdq_kv4_read", "svdq_attn_kv4",
                         "svdq_w4a16_gemv"]


def test_shapes_and_types_are_checked(on_device):
    z = lambda dt, *s: torch.zeros(*s, dtype=dt)  # noqa: E731
    X = z(BF, 4, 256)
    pos, freq = z(I32, 4, 3), z(torch.float64, 32)
    qk = lambda **k: layer.qk_norm_rope(**{**dict(  # noqa: E731
        X=X, pos=pos, freq=freq, axis_dims=[16, 24, 24], dim=64, q_heads=3, gamma_q=z(BF, 64),
        gamma_k=None), **k})
    qk()
    for bad, err in ((dict(X=X.float()), TypeError), (dict(pos=pos[:, :2]), ValueError),
                     (dict(freq=freq[:31]), ValueError), (dict(freq=freq.float()), TypeError),
                     (dict(gamma_q=z(BF, 63)), ValueError), (dict(gamma_k=z(torch.float32, 64)), TypeError),
                     (dict(out=z(BF, 3, 256)), ValueError), (dict(pos=pos[:3]), ValueError)):
        with pytest.raises(err):
            qk(**bad)
    kv = layer.kv_cache(3, 2, 64, device="cpu", bits=4)
    table, cu, seq = z(I32, 1, 3), z(I32, 2), z(I32, 1)
    layer.kv_write(kv, X[:, :128], X[:, 128:], table, cu, seq, 4)
    for bits in (8, 3):     # the 4-bit tensors are no cache of 8 bits
        with pytest.raises(ValueError):
            layer.kv_write(layer.KVCache(kv.k_codes, kv.v_codes, kv.k_scales, kv.v_scales, 64, bits),
                           X[:, :128], X[:, 128:], table, cu, seq, 4)
    with pytest.raises(ValueError):
        layer.kv_write(layer.KVCache(kv.k_codes, kv.v_codes, kv.k_scales[..., :64], kv.v_scales, 64, 4),
                       X[:, :128], X[:, 128:], table, cu, seq, 4)
    with pytest.raises(ValueError):
        layer.kv_cache(3, 2, 64, device="cpu", bits=2)
    pw = layer.PreparedWeight(layer.NVFP4, 8, 256, 8, z(U8, 8, 128), z(U8, 8, 16), z(torch.float32, 1),
                              z(BF, 8, 8))
    down, lam = z(BF, 8, 256), z(torch.float32, 256)
    ws = z(U8, 4096)
    layer.gemv(X, pw, lam, down, workspace=ws)
    assert layer.gemv(X.reshape(2, 2, 256), pw, lam, down, workspace=ws).shape == (2, 2, 8)
    bad = [dict(X=X[:, :128]), dict(lam=lam[:100]), dict(lora_down=down[:4]), dict(out=z(BF, 4, 7))]
    for b in bad:
        with pytest.raises((ValueError, TypeError)):
            layer.gemv(**{**dict(X=X, pw=pw, lam=lam, lora_down=down, workspace=ws), **b})
    with pytest.raises(ValueError, match="64"):
        layer.gemv(z(BF, 65, 256), pw, lam, down)
    with pytest.raises(ValueError):
        layer.gemv(X, layer.PreparedWeight(layer.NVFP4, 9, 256, 0, pw.codes, pw.scales, pw.g, None), lam,
                   None, workspace=ws)
