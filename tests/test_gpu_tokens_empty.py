"""An empty batch through the single-token path on the device: no rows come back, and the cache is left."""
import pytest

from tests.gpu_common import torch_mod
from tests.test_gpu_tokens_chain import Block, L, i32  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["nvfp4", "int4", "mxfp4"])
def test_chain_without_rows(L, fmt):  # noqa: F811
    torch = torch_mod()
    blk = Block(L, fmt)
    kv = L.kv_cache(3, blk.Hkv, blk.dim, bits=4)
    for t in (kv.k_codes, kv.v_codes, kv.k_scales, kv.v_scales):
        t.fill_(0xA5)
    x = torch.zeros(0, blk.K, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    _, qkv, O, Y = blk.step(kv, x, pos, i32([[0, 1, 2]]), i32([0, 0]), i32([0]), i32([0]), 1, 64)
    torch.cuda.synchronize()
    assert qkv.shape == (0, (blk.Hq + 2 * blk.Hkv) * blk.dim) and O.shape == (0, blk.Hq * blk.dim)
    assert Y.shape == (0, 512) and Y.is_cuda
    for t in (kv.k_codes, kv.v_codes, kv.k_scales, kv.v_scales):
        assert bool((t == 0xA5).all())
