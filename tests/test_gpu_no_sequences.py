"""A batch without a sequence, all of whose rows belong to none (GPU)."""
import pytest
import torch

from gpu_common import lib

pytestmark = pytest.mark.gpu


def test_rows_without_any_sequence():
    q4 = lib()
    ints = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")  # noqa: E731
    k = torch.randn(3, 2, 16, 64, device="cuda").bfloat16()
    v, batch = k.clone(), (ints(0, 5), ints(1), ints(0))
    out = torch.full((4, 6, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    before = k.clone()
    q = q4.kv_append(torch.randn(4, 10 * 64, device="cuda"), torch.ones(9, 64, device="cuda"), k, v, *batch, q_heads=6,
                     out=out)
    a = q4.attention(q, k, v, *batch, max_q_len=4, out=out)
    torch.cuda.synchronize()
    assert a is out and (out == 7).all() and torch.equal(k, before) and torch.equal(v, before)
    assert q4.device_error() == q4.OK
