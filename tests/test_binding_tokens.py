"""CPU tests of the binding and the layer API of the single-token and 4-bit operators: what is refused and
what is answered without a launch."""
import pytest
import torch

from w4a4_quantized_dit_amd import _lib, layer

BF, I32, U8 = torch.bfloat16, torch.int32, torch.uint8


@pytest.mark.parametrize("bits", [0, 2, 5, 16, None, "8"])
def test_workspace_of_a_cache_that_is_none(bits):
    """Neither 4 nor 8 bits: refused as kv_cache() refuses it."""
    with pytest.raises(ValueError, match="must be 4 or 8"):
        layer.attention_workspace(4, 4, 2, 64, 1, 4, 64, device="cpu", bits=bits)
    with pytest.raises(ValueError, match="must be 4 or 8"):
        layer.kv_cache(3, 2, 64, device="cpu", bits=bits)


@pytest.mark.parametrize("bits", [4, 8])
def test_workspace_of_either_cache(bits):
    assert layer.attention_workspace(4, 4, 2, 64, 1, 4, 64, device="cpu", bits=bits) is None
    ws = layer.attention_workspace(4, 4, 2, 64, 1, 4, 20000, device="cpu", bits=bits)
    assert ws.data_ptr() % 256 == 0 and ws.numel() % (4 * 4 * 66 * 4) == 0


@pytest.fixture
def on_device(monkeypatch):
    """Host tensors pass for device tensors; the entry points' names are collected instead of called."""
    names = []

    def at(self, t, name):
        self.dev = 0
        return t.data_ptr()
    monkeypatch.setattr(_lib._Args, "_at", at)
    monkeypatch.setattr(_lib._Args, "call", lambda self, name, *a: names.append(name))
    return names


def test_no_rows_at_all(on_device):
    """An empty batch goes through the chain of the single-token path without a launch; what is checked of
    the other operands is checked all the same."""
    z = lambda dt, *s: torch.zeros(*s, dtype=dt)  # noqa: E731
    pw = layer.PreparedWeight(layer.NVFP4, 256, 512, 8, z(U8, 256, 256), z(U8, 256, 32), z(torch.float32, 1),
                              z(BF, 256, 8))
    lam, down = z(torch.float32, 512), z(BF, 8, 512)
    for lead in ((0,), (0, 3), (2, 0)):
        Y = layer.gemv(z(BF, *lead, 512), pw, lam, down)
        assert Y.shape == (*lead, 256) and Y.dtype == BF
    out = z(BF, 0, 256)
    assert layer.gemv(z(BF, 0, 512), pw, lam, down, out=out) is out
    pos, freq = z(I32, 0, 3), z(torch.float64, 32)
    qkv = z(BF, 0, 256)
    assert layer.qk_norm_rope(qkv, pos, freq, [16, 24, 24], 64, 2, None, None).shape == (0, 256)
    qk = qkv[:, :192]
    layer.qk_norm_rope(qk, pos, freq, [16, 24, 24], 64, 2, z(BF, 64), None, out=qk)
    kv = layer.kv_cache(3, 1, 64, device="cpu", bits=4)
    table, cu, seq = z(I32, 1, 3), z(I32, 2), z(I32, 1)
    layer.kv_write(kv, qkv[:, 128:192], qkv[:, 192:], table, cu, seq, 1)
    O = layer.attention(qkv[:, :128], kv, table, cu, seq, 1, 100, causal=True)
    assert O.shape == (0, 128) and on_device == []
    with pytest.raises(ValueError):
        layer.gemv(z(BF, 0, 256), pw, lam, down)
    with pytest.raises(TypeError):
        layer.gemv(z(torch.float32, 0, 512), pw, lam, down)
    with pytest.raises(ValueError):
        layer.qk_norm_rope(qkv, pos, freq[:31], [16, 24, 24], 64, 2, None, None)
    with pytest.raises(ValueError, match="0 rows"):
        layer.gemv_workspace(0, pw)
