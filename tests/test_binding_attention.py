"""CPU tests of the binding's checks of the attention half: tensors that are not on a device are
refused before anything is enqueued, whichever operand comes first (the library takes addresses, and
a kernel would read the host's)."""
import pytest
import torch

from w4a4_quantized_dit_amd import _lib, layer

BF, I32, U8 = torch.bfloat16, torch.int32, torch.uint8


def _kv(device):
    z = lambda *s: torch.zeros(*s, dtype=U8, device=device)  # noqa: E731
    return layer.KVCache(z(3, 2, 64 * 64), z(3, 2, 64 * 64), z(3, 2), z(3, 2), 64)


def _calls(device):
    """One good call of each operator, with every tensor on `device`."""
    z = lambda dt, *s: torch.zeros(*s, dtype=dt, device=device)  # noqa: E731
    X, kv = z(BF, 4, 256), _kv(device)
    table, cu, seq = z(I32, 1, 3), z(I32, 2), z(I32, 1)
    axes = [16, 24, 24]
    return {
        "norm": lambda: _lib.svdq_rmsnorm_quant_act(X, X, z(BF, 4, 256), None, 1e-6, None, None, 0,
                                                    z(U8, 4, 256), z(U8, 4, 8), None),
        "rope": lambda: _lib.svdq_rope_axes(X, 4, 64, z(I32, 4, 3), z(torch.float64, 32), axes, True,
                                            False, z(BF, 4, 256)),
        "write": lambda: layer.kv_write(kv, X[:, :128], X[:, 128:], table, cu, seq, 4),
        "read": lambda: layer.kv_read(kv, table, cu, seq, 4, 4, out=[z(BF, 4, 128)] * 2),
        "attention": lambda: _lib.svdq_attn_kv8(X, 64, cu, seq, 4, 64, table, kv.k_codes, kv.v_codes,
                                                kv.k_scales, kv.v_scales, 0.125, True,
                                                z(BF, 4, 256)),
    }


@pytest.mark.parametrize("device", ["cpu", "meta"])
@pytest.mark.parametrize("op", ["norm", "rope", "write", "read", "attention"])
def test_tensors_that_are_not_on_a_device_are_refused(op, device, monkeypatch):
    def enqueue(*a):
        raise AssertionError("the call went on")
    monkeypatch.setattr(_lib._Args, "call", enqueue)
    with pytest.raises(ValueError, match="must be a device tensor"):
        _calls(device)[op]()


class _On:
    """What the binding asks of a tensor, on a device of its own choosing."""
    def __init__(self, t, dev):
        self._t, self._dev = t, dev

    def get_device(self):
        return self._dev

    def __getattr__(self, name):
        return getattr(self._t, name)


@pytest.mark.parametrize("where", [(-1, 0, 0), (0, -1, 0), (0, 0, -1), (0, 0, 1), (1, 0, 0), (-1, -1, -1)])
def test_every_operand_has_to_be_on_the_calls_device(where):
    x = torch.zeros(4, 256, dtype=BF)
    a = _lib._Args()
    with pytest.raises(ValueError, match="device"):
        for i, dev in enumerate(where):
            t = _On(x, dev)
            a.mat(t, 4, 256, (BF,), "X") if i % 2 else a.vec(t, 0, BF, "Y")
    for dev in (0, 3):
        a = _lib._Args()
        for i in range(3):
            a.vec(_On(x, dev), 0, BF, "X")
        assert a.dev == dev


def test_the_calls_above_are_good_ones():
    """The refusals come from the device: on a device the same operands reach the entry point."""
    names = []

    def on_device(self, t, name):
        self.dev = 0
        return 1 << 20

    mp = pytest.MonkeyPatch()
    try:
        mp.setattr(_lib._Args, "_at", on_device)
        mp.setattr(_lib._Args, "call", lambda self, name, *a: names.append(name))
        for f in _calls("cpu").values():
            f()
    finally:
        mp.undo()
    assert names == ["svdq_rmsnorm_quant_act", "svdq_rope_axes", "svdq_kv_write", "svdq_kv_read",
                     "svdq_attn_kv8"]
