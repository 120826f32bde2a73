"""Calls of the paged cache that the documentation allows: hints far off, captures, strides,
infinities."""
import pytest
import torch

import sparse_kv_prefetch_gb300 as dd
from paged_util import Cache, check_attention, run_attention

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,q4", [(BF, False), (BF, True), (F32, False)])
def test_a_length_hint_beyond_the_call_costs_nothing(dtype, q4):
    """The grid follows the call's tokens where max_q_len is larger: with a place for each of 2^31
    rows the call below would have 33 million CTAs."""
    c = Cache([1, 0] * 32, [3 + b for b in range(64)], 8, 8, 64, 16, dtype, q4)
    out, lse = run_attention(c, max_q=2 ** 31 - 1)
    check_attention(c, out, lse)
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    run_attention(c, max_q=2 ** 31 - 1)
    b.record()
    b.synchronize()
    assert a.elapsed_time(b) < 20
    dd.check_device()
