"""A cache of no rows, whose arrays have no address: every slot and every page id
lies outside it."""
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


def test_writes_are_left_out_and_reads_give_zeros():
    d = 64
    h = tq.tq_create_kv8(d)
    k = torch.randn(3, 2, d, device=DEV)
    cache = no_rows(d)
    slots = torch.full((3, 2), -1, device=DEV)
    tq.tq_quant_kv8(h, k, k, slots, *cache)
    assert tq.tq_device_status(h) == 0                        # padding is no event
    slots[1, 0] = 0
    tq.tq_quant_kv8(h, k, k, slots, *cache)
    assert tq.tq_device_status(h) == tq.TQ_STATUS_RANGE
    ko, vo = torch.full((6, d), 7.0, device=DEV), torch.full((6, d), 7.0, device=DEV)
    tq.tq_dequant_kv8(h, slots, *cache, ko, vo)
    assert (ko == 0).all() and (vo == 0).all()
    assert tq.tq_device_status(h) == tq.TQ_STATUS_RANGE
    tq.tq_quant_kv8(h, k, None, slots, *cache[:2])
    tq.tq_dequant_kv8(h, slots, *cache[:2], None, None, ko)
    assert (ko == 0).all() and tq.tq_device_status(h) == tq.TQ_STATUS_RANGE
