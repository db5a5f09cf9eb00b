"""Both forms of the kernels' bounded waits end after their time, not after a count of tries."""
from __future__ import annotations

import pytest
import torch

import attention_lightning_indexer_b200 as dsa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("limit_us", [100, 2000, 10000])
def test_bounded_waits_last_their_time(limit_us):
    dsa.dsa_check_device_errors()
    dsa.dsa_selftest_bounded_wait(1)
    with pytest.raises(dsa.DsaError):
        dsa.dsa_check_device_errors()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    dsa.dsa_selftest_bounded_wait(limit_us)
    end.record()
    with pytest.raises(dsa.DsaError) as e:
        dsa.dsa_check_device_errors()
    assert e.value.code == 5             # timeouts, and no wait that ended early (which would be 6)
    # two waits; the clock steps by about a microsecond.  An upper bound: three rounds of 4096 tries
    # beyond the limit, at no more than 10 us a try
    assert 2 * limit_us - 10 <= 1000 * begin.elapsed_time(end) <= 2 * limit_us + 3 * 4096 * 10
    dsa.dsa_check_device_errors()
