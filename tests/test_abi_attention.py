"""CPU tests of the refusals of the attention half's entry points (nothing is enqueued for an
invalid call) and of their host functions."""
import ctypes

import numpy as np
import pytest

from w4a4_quantized_dit_amd import _lib

OK, INVALID, SHAPE, NULLP = 0, 1, 2, 3
P = 1 << 20          # a fake, aligned, non-NULL "device pointer" (never dereferenced)
MIS = P + 4


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def _err(lib):
    return lib.svdq_last_error().decode()


def _dims(*v):
    return ctypes.cast((ctypes.c_int64 * max(1, len(v)))(*v), ctypes.c_void_p)


def test_norm_refusals(lib):
    def call(**kw):
        a = dict(X=P, M=4, K=256, ldx=256, res=P, ldr=256, H=P, ldh=256, g=P, eps=1e-6, lam=P,
                 down=P, r=8, c=P, s=P, D=P)
        a.update(kw)
        return lib.svdq_rmsnorm_quant_act(a["X"], a["M"], a["K"], a["ldx"], a["res"], a["ldr"],
                                          a["H"], a["ldh"], a["g"], a["eps"], a["lam"], a["down"],
                                          a["r"], a["c"], a["s"], a["D"], None)
    for k in ("X", "H", "down", "c", "s", "D"):
        assert call(**{k: None}) == NULLP, k
    for k in ("X", "res", "H", "g", "lam", "down", "c", "D"):
        assert call(**{k: MIS}) == SHAPE and "aligned" in _err(lib), k
    assert call(M=0) == SHAPE and call(M=(1 << 28) + 1) == SHAPE
    assert call(K=128) == SHAPE and call(K=0) == SHAPE
    assert call(K=33024, ldx=33024, ldr=33024, ldh=33024) == SHAPE
    for k in ("ldx", "ldr", "ldh"):
        assert call(**{k: 255}) == SHAPE and call(**{k: 260}) == SHAPE, k
    for eps in (0.0, -1.0, float("inf"), float("nan")):
        assert call(eps=eps) == INVALID
    assert call(r=4) == SHAPE and call(r=136) == SHAPE and call(r=-8) == SHAPE
    assert call(X=P, H=P, ldh=512, res=2 * P) == INVALID       # in place with another stride


def test_rope_refusals(lib):
    def call(**kw):
        a = dict(X=P, M=4, ldx=256, h=2, dim=128, pos=P, freq=P, n=3, dims=_dims(32, 48, 48), Y=P,
                 ldy=256)
        a.update(kw)
        return lib.svdq_rope_axes(a["X"], a["M"], a["ldx"], a["h"], a["dim"], a["pos"], a["freq"],
                                  a["n"], a["dims"], 1, 0, a["Y"], a["ldy"], None)
    for k in ("X", "pos", "freq", "dims", "Y"):
        assert call(**{k: None}) == NULLP, k
    assert call(X=MIS) == SHAPE and call(Y=MIS) == SHAPE
    assert call(M=0) == SHAPE and call(h=0) == SHAPE
    for dim in (0, 8, 100, 272):
        assert call(dim=dim) == SHAPE, dim
    assert call(n=0) == SHAPE and call(n=5, dims=_dims(16, 16, 16, 16, 16)) == SHAPE
    assert call(dims=_dims(33, 47, 48)) == SHAPE               # odd
    assert call(dims=_dims(-2, 66, 64)) == SHAPE
    assert call(dims=_dims(44, 44, 48)) == SHAPE               # 136 > dim
    assert call(dims=_dims(2, 2, 2)) == SHAPE                  # 6, not a multiple of 16
    assert call(dims=_dims(0, 0, 0)) == SHAPE
    assert call(ldx=248, ldy=248) == SHAPE and call(ldx=264) == INVALID


def test_rope_frequencies(lib):
    f = _lib.svdq_rope_frequencies([4, 0, 6], 100.0)
    assert np.allclose(f, [1, 0.1, 1, 100 ** (-1 / 3), 100 ** (-2 / 3)], rtol=1e-15)
    for dims, theta in (([3], 10.0), ([], 10.0), ([4], 1.0), ([4], float("nan")), ([4], float("inf"))):
        with pytest.raises(_lib.SvdqError):
            _lib.svdq_rope_frequencies(dims, theta)


@pytest.mark.parametrize("name", ["svdq_kv_write", "svdq_kv_read"])
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
        assert call(**{k: None}) == NULLP, k
    for k in ("K", "V", "kc", "vc"):
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
        return lib.svdq_attn_kv8(a["Q"], a["ldq"], a["rows"], a["hq"], a["hk"], a["dim"], a["cu"],
                                 a["kl"], a["B"], a["mr"], a["mkv"], a["bt"], a["mb"], a["n"],
                                 a["kc"], a["vc"], a["ks"], a["vs"], a["scale"], 1, a["O"],
                                 a["ldo"], a["lse"], a["ws"], a["wb"], None)
    for k in ("Q", "O", "cu", "kl", "bt", "kc", "vc", "ks", "vs"):
        assert call(**{k: None}) == NULLP, k
    for k in ("Q", "O", "kc", "vc", "lse"):
        assert call(**{k: MIS}) == SHAPE, k
    assert call(dim=96) == SHAPE and call(hq=3) == SHAPE and call(hq=1) == SHAPE
    assert call(hk=0) == SHAPE and call(ldq=504) == SHAPE and call(ldo=516) == SHAPE
    assert call(mkv=-1) == INVALID and call(O=P) == INVALID
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=s) == INVALID
    assert call(rows=0) == OK and call(mr=0) == OK
    assert call(rows=(1 << 28) + 1) == SHAPE and call(rows=1 << 28, mr=1 << 28) == SHAPE
    # a long cache is split: the workspace is checked
    need = lib.svdq_attn_kv8_workspace_bytes(4, 4, 2, 128, 1, 4, 20000)
    assert need > 0 and need % (4 * 4 * 130 * 4) == 0
    big = dict(mkv=20000, mb=400)
    assert call(**big) == NULLP and "workspace" in _err(lib)
    assert call(ws=P, wb=need - 1, **big) == SHAPE
    assert call(ws=P + 16, wb=need, **big) == SHAPE
    for bad in ((4, 3, 2, 128, 1, 4, 9), (4, 4, 2, 96, 1, 4, 9), (4, 4, 0, 64, 1, 4, 9),
                (-1, 4, 2, 64, 1, 4, 9), (4, 4, 2, 64, 0, 4, 9), (4, 4, 2, 64, 1, 4, -9)):
        assert lib.svdq_attn_kv8_workspace_bytes(*bad) == -1, bad
    assert lib.svdq_attn_kv8_workspace_bytes(4, 4, 2, 128, 1, 4, 64) == 0
