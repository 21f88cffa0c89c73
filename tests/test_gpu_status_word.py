"""The status word holds what the calls on a handle met: the handle's creation is
complete when it returns, and reading the word waits for the device, whichever
streams the calls ran on."""
import pytest
import torch

import compressed_kv_cache_turboquant_b200 as tq

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
DEV = "cuda"
D, ROWS = 64, 8
LONG = 400_000_000                                            # cycles: about 0.2 s


class Arrays:
    """One token whose slot lies outside the cache: a call that sets TQ_STATUS_RANGE."""

    def __init__(self):
        self.k = torch.randn(1, 1, D, device=DEV)
        self.slots = torch.tensor([[ROWS]], device=DEV)
        self.codes, self.scales = torch.zeros(ROWS, D, dtype=torch.int8, device=DEV), torch.zeros(ROWS, device=DEV)

    def write(self, h, stream=None):
        tq.tq_quant_kv8(h, self.k, None, self.slots, self.codes, self.scales, stream=stream)


def test_a_handle_is_ready_when_its_creation_returns():
    a, side = Arrays(), torch.cuda.Stream()
    a.write(tq.tq_create_kv8(D), side)                        # all is loaded
    torch.cuda._sleep(1)
    torch.cuda.synchronize()
    torch.cuda._sleep(LONG)                                   # the default stream is busy for a while
    h = tq.tq_create_kv8(D)
    a.write(h, side)
    side.synchronize()
    torch.cuda.synchronize()
    assert tq.tq_device_status(h) == tq.TQ_STATUS_RANGE


def test_reading_the_word_waits_for_work_on_other_streams():
    a, side = Arrays(), torch.cuda.Stream()
    h = tq.tq_create_kv8(D)
    a.write(h, side)
    side.synchronize()
    assert tq.tq_device_status(h) == tq.TQ_STATUS_RANGE
    assert tq.tq_device_status(h) == 0
    with torch.cuda.stream(side):
        torch.cuda._sleep(LONG)
    a.write(h, side)
    assert tq.tq_device_status(h) == tq.TQ_STATUS_RANGE
    assert tq.tq_device_status(h) == 0
