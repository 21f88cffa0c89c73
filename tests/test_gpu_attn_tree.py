"""Attention of drafted tokens over the 8-bit paged cache against the definition in
64 bits (the cache's codes and scales taken as given).

Tolerance of an output element, by arithmetic: with A = sum_t w_t |v_t| and
u = eps / 2 of the type, rounding the weights (the value's scale in them) to the
type costs at most u A, rounding the result u |out|; the logits (d products in
float32, then scaled) are off by at most
  delta = scale (d + 2) 2^-24 max_t sum_i |q_i k_ti| + 2^-22 max_t |logit_t|
each, which moves a weight by 2 delta relative at most, and float32
exponentials, sums and the merge of parts add under 2^-20; a float16 result
below 2^-14 rounds by up to 2^-25.  A weight below 2^-126 of the largest is not
a normal float32 and may count as 0: at most T 2^-126 max |v|.  The log-sum is off by delta + 2^-20 and a
float32 rounding of itself."""
import math

import pytest
import torch

import compressed_kv_cache_turboquant_b200 as tq

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
DEV = "cuda"
BF, HF = torch.bfloat16, torch.float16


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


class Case:
    """A paged cache with everything a call needs; pages of all sequences shuffled in one pool."""

    def __init__(self, ctx, n, Hq, Hkv, d, page, dtype, seed=0, drafts=None, mask="tree", spare=3):
        g = self.g = gen(seed)
        self.B, self.n, self.Hq, self.Hkv, self.d, self.page, self.dtype = len(ctx), n, Hq, Hkv, d, page, dtype
        self.h = tq.tq_create_kv8(d)
        B = self.B
        self.drafts = [n] * B if drafts is None else list(drafts)
        self.ctx = list(ctx)
        self.ctx_lens = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        self.draft_lens = None if drafts is None else torch.tensor(drafts, dtype=torch.int32, device=DEV)
        pages = max(1, max(-(-(c + m) // page) for c, m in zip(self.ctx, self.drafts)))
        pool = B * Hkv * pages + spare
        self.table = torch.randperm(pool, generator=g, device=DEV)[: B * Hkv * pages].reshape(B * Hkv, pages).to(torch.int32)
        rows = pool * page
        self.kcodes, self.vcodes = (torch.randint(-127, 128, (rows, d), generator=g, device=DEV, dtype=torch.int32).to(torch.int8)
                                    for _ in range(2))
        self.kscales, self.vscales = ((torch.randn(rows, generator=g, device=DEV) * 0.7).exp() / 60 for _ in range(2))
        self.q = torch.randn(B, n, Hq, d, generator=g, device=DEV).to(dtype)
        if mask == "tree":
            bits = torch.rand(B, n, n, generator=g, device=DEV) < 0.4
            bits &= torch.ones(n, n, dtype=torch.bool, device=DEV).tril()
            bits |= torch.eye(n, dtype=torch.bool, device=DEV)
        elif mask == "any":                                  # any bits at all, rows that see no drafted token among them
            bits = torch.rand(B, n, n, generator=g, device=DEV) < 0.2
            bits[:, 0] = False
        else:
            bits = None
        self.set_mask(bits)
        self.scale = 1 / math.sqrt(d)
        self.out = torch.full_like(self.q, 77)
        self.lse = torch.full((B, n, Hq), 77.0, device=DEV)

    def set_mask(self, bits):
        self.bits, self.mask = bits, None
        if bits is None:
            self.bits = torch.ones(self.n, self.n, dtype=torch.bool, device=DEV).tril().expand(self.B, -1, -1)
            return
        words = (self.n + 31) // 32
        wide = torch.zeros(self.B, self.n, words * 32, dtype=torch.int64, device=DEV)
        wide[..., :self.n] = bits
        packed = (wide.reshape(self.B, self.n, words, 32) << torch.arange(32, device=DEV)).sum(-1)
        self.mask = torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed).to(torch.int32)

    def run(self, **kw):
        a = dict(lse=self.lse, mask=self.mask, draft_lens=self.draft_lens) | kw
        tq.tq_attn_tree(self.h, self.q, self.Hkv, self.ctx_lens, self.table, self.page, self.kcodes, self.kscales,
                        self.vcodes, self.vscales, self.scale, self.out, **a)
        return self.out, self.lse

    def rows_of(self, b, h, T):
        t = torch.arange(T, device=DEV)
        return self.table[b * self.Hkv + h].long()[t // self.page] * self.page + t % self.page

    def check(self, absent=None, sample=None):
        """absent(b, h) -> bool [T]: keys that count as not there."""
        G, u = self.Hq // self.Hkv, torch.finfo(self.dtype).eps / 2
        for b in range(self.B) if sample is None else sample:
            c, m = self.ctx[b], self.drafts[b]
            T = c + m
            assert (self.out[b, m:] == 77).all() and (self.lse[b, m:] == 77).all()
            if m == 0:
                continue
            sees0 = torch.ones(m, T, dtype=torch.bool, device=DEV)
            sees0[:, c:] = self.bits[b, :m, :m]
            for h in range(self.Hkv):
                r = self.rows_of(b, h, T)
                K = self.kcodes[r].double() * self.kscales[r].double()[:, None]
                V = self.vcodes[r].double() * self.vscales[r].double()[:, None]
                sees = sees0 if absent is None else sees0 & ~absent(b, h)[None, :]
                unseen = ~sees.any(0)
                K[unseen], V[unseen] = 0, 0
                for x in range(h * G, h * G + G):
                    q = self.q[b, :m, x].double()
                    z = (self.scale * (q @ K.T)).masked_fill(~sees, -math.inf)
                    lse = torch.logsumexp(z, 1)
                    empty = ~sees.any(1)
                    w = torch.exp(z - torch.where(empty, torch.zeros_like(lse), lse)[:, None])
                    want, A = w @ V, w @ V.abs()
                    mags = self.scale * (q.abs() @ K.abs().T).masked_fill(~sees, 0).amax(1)
                    delta = (self.d + 2) * 2.0 ** -24 * mags + 2.0 ** -22 * z.masked_fill(~sees, 0).abs().amax(1)
                    tol = (u + 2 * delta[:, None] + 2.0 ** -20) * A + u * want.abs() + T * 2.0 ** -126 * V.abs().amax()
                    if self.dtype == HF:
                        tol = tol + 2.0 ** -25
                    got, gl = self.out[b, :m, x].double(), self.lse[b, :m, x].double()
                    err = (got - want).abs()
                    assert (err <= tol).all(), (b, x, float((err / tol.clamp(min=1e-30)).max()))
                    assert (got[empty] == 0).all() and (gl[empty] == -math.inf).all()
                    tl = delta + 2.0 ** -20 + 2.0 ** -23 * lse.abs()
                    el = (gl - lse).abs()[~empty]
                    assert (el <= tl[~empty]).all(), (b, x, float((el / tl[~empty]).max()))


SHAPES = [  # context lengths, n, Hq, Hkv, d, page
    ([1], 1, 1, 1, 16, 8), ([0], 1, 4, 1, 64, 16), ([1000], 1, 32, 8, 128, 16), ([63, 64, 65, 0], 1, 8, 2, 128, 64),
    ([15, 129, 500], 4, 8, 2, 128, 16), ([200, 7], 3, 5, 5, 64, 8), ([333], 9, 7, 1, 80, 24), ([40, 900, 0], 16, 8, 2, 128, 64),
    ([100, 256], 33, 4, 1, 128, 32), ([77], 64, 8, 2, 64, 16), ([130], 5, 32, 1, 96, 256), ([300, 300], 8, 3, 1, 256, 16),
    ([513], 1, 16, 1, 256, 64), ([90], 100, 2, 2, 48, 8), ([5000, 1], 2, 28, 4, 128, 16), ([20], 256, 2, 1, 32, 40),
    ([6000], 61, 16, 4, 64, 64), ([259], 13, 128, 1, 128, 8),
]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("ctx,n,Hq,Hkv,d,page", SHAPES)
def test_trees_over_ragged_contexts(ctx, n, Hq, Hkv, d, page, dtype):
    c = Case(ctx, n, Hq, Hkv, d, page, dtype, seed=len(ctx) + n)
    c.run()
    c.check()
    assert tq.tq_device_status(c.h) == 0


@pytest.mark.parametrize("dtype", [BF, HF])
def test_draft_lengths_and_empty_sequences(dtype):
    c = Case([0, 50, 0, 1200, 64, 31], 20, 8, 2, 128, 16, dtype, drafts=[1, 0, 0, 20, 13, 7])
    c.run()
    c.check()
    assert tq.tq_device_status(c.h) == 0


def test_a_chain_without_a_mask():
    c = Case([100, 0, 700], 10, 8, 2, 128, 32, BF, mask=None, drafts=[10, 10, 3])
    c.run()
    c.check()


@pytest.mark.parametrize("n", [3, 40])
def test_any_mask_and_rows_that_see_nothing(n):
    c = Case([0, 0, 90], n, 8, 2, 64, 16, BF, mask="any")
    c.run()
    c.check()
    assert (c.out[0, 0] == 0).all() and (c.lse[0, 0] == -math.inf).all()


@pytest.mark.parametrize("Hkv,n", [(8, 1), (1, 16), (2, 64)])
def test_a_long_context(Hkv, n):
    c = Case([40001, 3], n, 4 * Hkv, Hkv, 128, 64, BF, seed=7)
    c.run()
    c.check()
    assert tq.tq_device_status(c.h) == 0


def test_many_short_sequences():
    g = torch.Generator().manual_seed(1)
    ctx = torch.randint(0, 40, (700,), generator=g).tolist()
    c = Case(ctx, 2, 4, 2, 64, 8, BF, drafts=torch.randint(0, 3, (700,), generator=g).tolist())
    c.run()
    c.check(sample=range(0, 700, 23))
    assert tq.tq_device_status(c.h) == 0


def test_sharp_logits_and_values_of_very_different_sizes():
    c = Case([700, 90], 6, 8, 2, 128, 16, BF)
    c.scale = 3.0
    at = torch.arange(len(c.vscales), device=DEV)
    c.vscales *= 10.0 ** ((at % 13).float() - 6)
    c.run()
    c.check()
    c = Case([700, 90], 6, 8, 2, 128, 16, HF)
    c.vscales *= 10.0 ** ((torch.arange(len(c.vscales), device=DEV) % 7).float() - 6)
    c.run()
    c.check()


def test_zero_scales_of_values_and_keys():
    c = Case([300], 4, 8, 2, 64, 16, BF)
    c.vscales[::2] = 0
    c.kscales[::3] = 0
    c.run()
    c.check()
    c.vscales.zero_()
    c.run()
    assert (c.out == 0).all() and torch.isfinite(c.lse).all()


def test_what_is_not_seen_may_hold_anything():
    c = Case([70, 0, 300], 12, 8, 2, 128, 16, BF, drafts=[12, 5, 9], mask="any")
    c.run()
    want, want_lse = c.out.clone(), c.lse.clone()
    c.check()
    for b in range(3):
        seen = c.bits[b, :c.drafts[b], :c.drafts[b]].any(0)
        for h in range(2):
            T = c.table.shape[1] * 16
            r = c.rows_of(b, h, T)
            dead = torch.ones(T, dtype=torch.bool, device=DEV)
            dead[:c.ctx[b]] = False
            dead[c.ctx[b]:c.ctx[b] + c.drafts[b]] = ~seen
            c.kscales[r[dead]] = float("nan")
            c.vscales[r[dead]] = float("inf")
            c.kcodes[r[dead]] = -128
            c.vcodes[r[dead]] = -128
    # a drafted token that some see and others do not spoils only those that see it
    c.run()
    assert torch.equal(c.out, want) and torch.equal(c.lse, want_lse)
    j = int(c.bits[0, :, :].any(0).nonzero()[0])
    r = c.rows_of(0, 1, 82)[70 + j]
    c.vscales[r] = float("nan")
    c.kscales[r] = float("nan")
    c.run()
    hit = torch.zeros(3, 12, 8, dtype=torch.bool, device=DEV)
    hit[0, :, 4:] = c.bits[0, :, j][:, None]
    assert torch.isnan(c.out[hit]).all()
    assert torch.equal(c.out[~hit], want[~hit]) and torch.equal(c.lse[~hit], want_lse[~hit])


def test_page_ids_outside_the_cache_are_absent_keys():
    c = Case([500, 40], 3, 8, 2, 128, 16, BF)
    pool = c.kcodes.shape[0] // 16
    bad = torch.zeros(4, c.table.shape[1], dtype=torch.bool, device=DEV)
    bad[0, 3] = bad[1, 0] = bad[1, 31] = bad[2, 1] = True
    good = c.table.clone()
    c.table = torch.where(bad, torch.tensor([-1, pool, 2 ** 31 - 1, -(2 ** 31)], device=DEV, dtype=torch.int32)[:, None], good)
    c.run()
    assert tq.tq_device_status(c.h) == tq.TQ_STATUS_RANGE
    c.table = good
    c.check(absent=lambda b, h: bad[b * 2 + h][torch.arange(c.ctx[b] + 3, device=DEV) // 16])


def test_lengths_outside_the_block_table():
    c = Case([100, 30, 64], 4, 8, 2, 64, 16, BF, drafts=[4, 4, 4])
    c.run()
    want = c.out.clone()
    assert tq.tq_device_status(c.h) == 0
    cap = c.table.shape[1] * 16
    c.ctx_lens[0] = 2 ** 31 - 1                               # everything in its pages counts as context
    c.ctx_lens[1] = -7                                        # no context
    c.draft_lens[2] = 99                                      # n of them
    c.run()
    assert tq.tq_device_status(c.h) == tq.TQ_STATUS_RANGE
    assert torch.equal(c.out[2], want[2])
    c.ctx[0], c.drafts[0] = cap, 4
    all_seen = Case([cap - 4, 0, 64], 4, 8, 2, 64, 16, BF)
    for k in ("q", "kcodes", "kscales", "vcodes", "vscales", "table"):
        setattr(all_seen, k, getattr(c, k))
    bits = c.bits.clone()
    bits[0] = True
    all_seen.set_mask(bits)
    all_seen.run()
    assert torch.allclose(all_seen.out[:2].float(), c.out[:2].float(), rtol=2.0 ** -6, atol=2.0 ** -6)
    assert torch.allclose(all_seen.lse[:2], c.lse[:2], rtol=1e-5, atol=1e-5)


def test_queries_of_a_fused_projection():
    c = Case([200, 31], 5, 8, 2, 128, 16, BF)
    c.run()
    want = c.out.clone()
    wide = torch.zeros(2, 5, 12 * 128, dtype=BF, device=DEV)
    wide[..., :1024] = c.q.reshape(2, 5, 1024)
    c.q = wide[..., :1024].view(2, 5, 8, 128)
    c.out = torch.empty(2, 5, 8, 128, dtype=BF, device=DEV)
    c.run()
    assert torch.equal(c.out, want)


def test_the_same_twice_and_without_lse():
    c = Case([9000, 300, 12], 7, 32, 8, 128, 64, BF)
    c.run()
    first, lse = c.out.clone(), c.lse.clone()
    for _ in range(3):
        c.run(lse=None)
        assert torch.equal(c.out, first)
    c.run()
    assert torch.equal(c.lse, lse)


def test_a_captured_step_replays_with_other_lengths_and_pages():
    c = Case([1000, 400], 4, 8, 2, 128, 16, BF, drafts=[4, 4])
    c.run()
    graph = torch.cuda.CUDAGraph()
    ws = torch.empty(max(1, tq.tq_attn_tree_workspace(c.h, 2, 4, 8, 2)), dtype=torch.uint8, device=DEV)
    with torch.cuda.graph(graph):
        c.run(workspace=ws)
    for ctx, drafts, seed in (([7, 1000], [4, 2], 1), ([0, 0], [1, 4], 2), ([1003, 500], [1, 4], 3)):
        c.ctx_lens.copy_(torch.tensor(ctx))
        c.draft_lens.copy_(torch.tensor(drafts))
        c.table.copy_(c.table.reshape(-1)[torch.randperm(c.table.numel(), generator=gen(seed), device=DEV)].reshape(c.table.shape))
        c.ctx, c.drafts = ctx, drafts
        c.out.fill_(77)
        c.lse.fill_(77)
        graph.replay()
        torch.cuda.synchronize()
        c.check()
    assert tq.tq_device_status(c.h) == 0


def test_two_graphs_that_share_a_workspace():
    cases = [Case([3000, 5], 4, 8, 2, 128, 16, BF, seed=1), Case([10, 2000], 4, 8, 2, 128, 16, BF, seed=2)]
    ws = torch.empty(max(1, tq.tq_attn_tree_workspace(cases[0].h, 2, 4, 8, 2)), dtype=torch.uint8, device=DEV)
    graphs = []
    for c in cases:
        c.run(workspace=ws)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c.run(workspace=ws)
    for order in ((0, 1, 0), (1, 1, 0)):
        for c in cases:
            c.out.fill_(77)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for c in cases:
            c.check()


def test_two_streams_at_once():
    cases = [Case([3000, 700], 8, 8, 2, 128, 16, BF, seed=i) for i in range(2)]
    for c in cases:
        c.run()
    want = [c.out.clone() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        for c, s in zip(cases, streams):
            c.run(stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(c.out, w) for c, w in zip(cases, want))


def test_a_cache_past_32_bits_of_bytes():
    c = Case([300], 2, 4, 1, 256, 64, BF)
    pages = 2 ** 32 // (256 * 64) + 100
    big = torch.zeros(pages * 64, 256, dtype=torch.int8, device=DEV)
    bigv = torch.zeros_like(big)
    scales = torch.zeros(2, pages * 64, device=DEV)
    old = c.rows_of(0, 0, c.table.shape[1] * 64)
    c.table = (pages - 1 - 3 * torch.arange(c.table.shape[1], device=DEV)).to(torch.int32).reshape(1, -1)
    new = c.rows_of(0, 0, c.table.shape[1] * 64)
    big[new], bigv[new] = c.kcodes[old], c.vcodes[old]
    scales[0][new], scales[1][new] = c.kscales[old], c.vscales[old]
    c.kcodes, c.vcodes, c.kscales, c.vscales = big, bigv, scales[0], scales[1]
    c.run()
    c.check()


def test_refusals_of_the_binding():
    c = Case([30], 2, 4, 2, 64, 16, BF)
    for name, value in (("q", c.q.float()), ("q", c.q[..., :32]), ("ctx_lens", c.ctx_lens.long()), ("table", c.table[:1]),
                        ("table", c.table.long()), ("kcodes", c.kcodes[:5]), ("kscales", c.kscales.double()),
                        ("vcodes", c.vcodes.to(torch.int16)), ("mask", c.mask[:, :1]), ("out", c.out[:, :1]),
                        ("page", 12), ("page", 0), ("scale", float("inf")), ("scale", -1.0), ("q", c.q.cpu())):
        old = getattr(c, name)
        setattr(c, name, value)
        with pytest.raises((ValueError, tq.TQError)):
            c.run()
        setattr(c, name, old)
    c.run()
    c.check()
