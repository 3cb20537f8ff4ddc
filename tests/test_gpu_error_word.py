"""Two reports in the device error word (GPU): one of skipped indices does not
hide one of an output left incomplete."""
import ctypes

import pytest
import torch

from gpu_common import lib

pytestmark = pytest.mark.gpu


def token_out_of_range(q4):
    q4.token_logprobs(torch.zeros(1, 10, device="cuda"), torch.tensor([10], device="cuda"))


def page_out_of_range(q4):
    cache = torch.zeros(2, 1, 8, 64, dtype=torch.bfloat16, device="cuda")
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    q4.kv_append(torch.zeros(1, 3 * 64, device="cuda"), torch.zeros(8, 0, device="cuda"), cache, cache.clone(),
                 ints(2)[None], ints(0, 1), ints(1), q_heads=1)


def page_out_of_range_read(q4):
    cache = torch.zeros(2, 1, 8, 64, dtype=torch.bfloat16, device="cuda")
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    q4.attention(torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda"), cache, cache.clone(), ints(2)[None],
                 ints(0, 1), ints(1), max_q_len=1)


@pytest.mark.parametrize("bad", [token_out_of_range, page_out_of_range, page_out_of_range_read])
@pytest.mark.parametrize("timeout_first", [True, False])
def test_a_wait_that_was_given_up_is_reported_first(bad, timeout_first):
    q4 = lib()
    assert q4.device_error() == q4.OK
    bad(q4)
    assert q4.device_error() == q4.ERR_DEVICE_INDEX
    if not timeout_first:
        bad(q4)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert q4.lib().q4_0_selftest_wait_timeout(20000, stream) == q4.OK
    if timeout_first:
        bad(q4)
    assert q4.device_error() == q4.ERR_DEVICE_TIMEOUT
    assert q4.device_error() == q4.OK
