"""The device status word of all units of the library (GPU)."""
import pytest
import torch

import gated_delta_rule_85_b200 as kda

pytestmark = pytest.mark.gpu
BOTH = kda.DEV_WAIT_TIMEOUT | kda.DEV_BAD_SLOT


def _flag_both():
    """A wait that runs out in one unit, an entry outside the pool in another."""
    kda.debug_wait_timeout(100_000)
    x = torch.zeros(1, 2, 64, device="cuda")
    pool = torch.zeros(1, 2, 64, 64, device="cuda")
    kda.la_recurrent_step_slots(x, x, x, torch.zeros(2, device="cuda"), pool, torch.tensor([5], dtype=torch.int32, device="cuda"))


def test_flags_of_all_units_are_read_and_cleared_together():
    assert kda.device_status() == 0
    _flag_both()
    assert kda.device_status(clear=False) == BOTH
    assert kda.device_status(clear=False) == BOTH   # reading does not lose them
    assert kda.device_status() == BOTH
    assert kda.device_status() == 0
    _flag_both()
    assert kda.device_status() == BOTH and kda.device_status() == 0


def test_status_takes_one_copy():
    """One device-to-host copy and one wait a call, however many units the library has."""
    kda.device_status()
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CPU, torch.profiler.ProfilerActivity.CUDA]) as p:
        kda.device_status()
    names = [e.name for e in p.events()]
    copies = [n for n in names if n.startswith("cudaMemcpy")]
    waits = [n for n in names if n == "cudaStreamSynchronize"]
    assert len(copies) == 1 and len(waits) == 1, names
