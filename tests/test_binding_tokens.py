"""CPU tests of the binding and the layer API of the single-token and 4-bit operators: what is refused and
what is answered without a launch."""
import pytest

from w4a4_quantized_dit_amd import layer


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
