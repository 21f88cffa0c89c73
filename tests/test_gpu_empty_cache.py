"""A cache of no rows, whose arrays have no address: every page id lies
outside it."""
import math

import pytest
import torch

from test_gpu_attn_tree import BF, DEV, HF, Case

import compressed_kv_cache_turboquant_b200 as tq

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def no_rows(d):
    return [torch.empty(0, d, dtype=torch.int8, device=DEV), torch.empty(0, device=DEV)] * 2


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n,Hq,Hkv,d", [(1, 8, 2, 128), (16, 8, 2, 64), (3, 2, 1, 256), (12, 8, 2, 128), (40, 8, 2, 64)])
def test_attention_over_it_sees_nothing(n, Hq, Hkv, d, dtype):
    c = Case([300, 0, 9], n, Hq, Hkv, d, 16, dtype)
    c.kcodes, c.kscales, c.vcodes, c.vscales = no_rows(d)
    c.run()
    assert (c.out == 0).all() and (c.lse == -math.inf).all()
    assert tq.tq_device_status(c.h) == tq.TQ_STATUS_RANGE


def test_fewer_rows_than_a_page():
    c = Case([30], 2, 4, 2, 64, 16, BF)
    c.kcodes, c.vcodes, c.kscales, c.vscales = c.kcodes[:15], c.vcodes[:15], c.kscales[:15], c.vscales[:15]
    c.run()
    assert (c.out == 0).all() and (c.lse == -math.inf).all()
    assert tq.tq_device_status(c.h) == tq.TQ_STATUS_RANGE
