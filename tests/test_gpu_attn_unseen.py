"""Drafted tokens do not feel what keys they cannot see hold: scales of NaN and of
either infinity, codes of -128.  Each kernel masks in its own way, so the shapes
reach all of them: blocks of 8, 16 and 32 rows on mma.sync (d = 64, 128, 256), and
one or two tiles of 128 rows on tcgen05."""
import pytest
import torch

from test_gpu_attn_tree import BF, DEV, HF, Case

import compressed_kv_cache_turboquant_b200 as tq

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
ODD = [float("nan"), float("inf"), -float("inf")]

SHAPES = [  # n, Hq, Hkv, d
    (2, 8, 2, 128), (4, 8, 2, 128), (8, 8, 2, 128), (5, 4, 4, 64), (16, 2, 2, 64), (4, 8, 2, 256), (40, 2, 1, 256),
    (12, 8, 2, 128), (64, 4, 2, 64), (40, 8, 2, 128), (70, 8, 2, 64)]


def case(n, Hq, Hkv, d, dtype):
    c = Case([70, 0, 300], n, Hq, Hkv, d, 16, dtype, seed=n + d, drafts=[n, n // 2, n - 1], mask="any")
    c.bits[0, n - 1, 0] = True                                # a drafted token that one sees and another does not
    c.set_mask(c.bits)
    return c


def rows_nobody_sees(c):
    """Cache rows of the pages' places behind the drafts and of drafted tokens that no token sees."""
    rows = []
    T = c.table.shape[1] * c.page
    for b in range(c.B):
        m = c.drafts[b]
        dead = torch.ones(T, dtype=torch.bool, device=DEV)
        dead[:c.ctx[b]] = False
        dead[c.ctx[b]:c.ctx[b] + m] = ~c.bits[b, :m, :m].any(0)
        for h in range(c.Hkv):
            rows.append(c.rows_of(b, h, T)[dead])
    return torch.cat(rows)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n,Hq,Hkv,d", SHAPES)
def test_rows_that_nobody_sees_may_hold_anything(n, Hq, Hkv, d, dtype):
    c = case(n, Hq, Hkv, d, dtype)
    c.run()
    c.check()
    want, want_lse = c.out.clone(), c.lse.clone()
    dead = rows_nobody_sees(c)
    c.kcodes[dead], c.vcodes[dead] = -128, -128
    odd = torch.tensor(ODD, device=DEV)[torch.arange(len(dead), device=DEV) % 3]
    for kscales, vscales in ((odd, odd.roll(1)), (torch.ones_like(odd), odd), (odd, torch.ones_like(odd))):
        c.kscales[dead], c.vscales[dead] = kscales, vscales
        c.run()
        assert torch.equal(c.out, want) and torch.equal(c.lse, want_lse)
    assert tq.tq_device_status(c.h) == 0


@pytest.mark.parametrize("bad", ODD)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n,Hq,Hkv,d", SHAPES)
def test_a_scale_reaches_only_who_sees_it(n, Hq, Hkv, d, dtype, bad):
    """One drafted token of the first sequence, the value's scale alone and the key's alone."""
    c = case(n, Hq, Hkv, d, dtype)
    c.run()
    want, want_lse = c.out.clone(), c.lse.clone()
    G, h = Hq // Hkv, Hkv - 1
    j = int((c.bits[0].any(0) & ~c.bits[0].all(0)).nonzero()[0])
    r = c.rows_of(0, h, c.ctx[0] + n)[c.ctx[0] + j]
    hit = torch.zeros(c.B, n, Hq, dtype=torch.bool, device=DEV)
    hit[0, :, h * G:(h + 1) * G] = c.bits[0, :, j][:, None]
    for scales in (c.vscales, c.kscales):
        old = scales[r].clone()
        scales[r] = bad
        c.run()
        assert torch.equal(c.out[~hit], want[~hit]) and torch.equal(c.lse[~hit], want_lse[~hit])
        if scales is c.vscales:
            assert not torch.isfinite(c.out[hit]).any()     # a weight times it, in every channel
            assert torch.equal(c.lse, want_lse)
        scales[r] = old
    c.run()
    assert torch.equal(c.out, want)
