"""q4_0_kv_append without a rotation needs no table (GPU)."""
import pytest
import torch

import serving_ref as ref
from gpu_common import lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("table_rows", [0, 1, 3])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_past_the_table_are_appended(table_rows, given, dtype):
    q4 = lib()
    b = ref.Batch([1, 5, 33], [60, 5, 70], 16, 2, 64, seed=8)
    k, v, *rest = b.cuda()
    qkv = torch.randn(b.rows, (4 + 2 * 2) * 64, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    positions = torch.full((b.rows,), 10 ** 6, dtype=torch.int32, device="cuda") if given else None
    q = q4.kv_append(qkv, torch.zeros(table_rows, 0, device="cuda"), k, v, *rest, q_heads=4, positions=positions)
    assert q4.device_error() == q4.OK
    x = qkv.view(b.rows, 8, 64).bfloat16()
    assert torch.equal(q, x[:, :4])
    k_want, v_want = torch.zeros_like(k), torch.zeros_like(v)
    for s, n in enumerate(b.new):
        for i in range(n):
            page, off = b.place(s, b.kv[s] - n + i)
            k_want[page, :, off], v_want[page, :, off] = x[int(b.q_start[s]) + i].split([4, 2, 2])[1:]
    assert torch.equal(k, k_want) and torch.equal(v, v_want)
