"""Blocks so small that their fp32 scale is 0: kv_append_q4 and the weights'
quantizer store the same bits, codes of 8, as for a block of zeros (GPU)."""
import pytest
import torch

from gpu_common import lib

pytestmark = pytest.mark.gpu
LEAST = 2.0 ** -149  # of fp32; an eighth of up to four of it rounds to 0


def rows(dtype):
    """[rows, 64]: a block of tiny elements of both signs, and one beside it
    that has a scale."""
    x = torch.zeros(10, 64, dtype=torch.float64)
    unit = LEAST if dtype == torch.float32 else 2.0 ** -133  # least bfloat16: its eighth is not 0
    for i, top in enumerate((1, -1, 2, -3, 4, -4, 5, -5, 12, 40)):
        x[i, 3], x[i, 9], x[i, 20], x[i, 31] = top * unit, -unit, unit, -top * unit
        x[i, 32:] = torch.linspace(-1, 1, 32) * (i + 1)
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_codes_and_scales_equal_the_quantizers(dtype):
    q4 = lib()
    x = rows(dtype)
    n = len(x)
    qkv = torch.cat([x, x, x], 1).cuda()
    cache = q4.kv_cache_q4(2, 1, 16, 64)
    batch = (torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
             torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.tensor([n], dtype=torch.int32, device="cuda"))
    q4.kv_append_q4(qkv, torch.zeros(16, 0, device="cuda"), cache, *batch, q_heads=1)
    assert q4.device_error() == q4.OK
    blocks = q4.quantize(x.float().cuda()).view(n, 2, 18)
    for codes, scales in (cache[:2], cache[2:]):
        assert torch.equal(codes[0, 0, :n].view(n, 2, 16), blocks[..., 2:])
        assert torch.equal(scales[0, 0, :n].contiguous().view(torch.uint8).view(n, 2, 2), blocks[..., :2])
        if dtype == torch.float32:
            assert (codes[0, 0, :6, :16] == 0x88).all()
            assert (codes[0, 0, 6:8, :16] != 0x88).any(1).all()
        assert (codes[0, 0, :n, 16:] != 0x88).any(1).all()
    k, v = q4.kv_read_q4(cache, *batch, rows=n, out_dtype=torch.float32)
    assert (k[:, 0, :32] == 0).all() and torch.equal(k, v)
