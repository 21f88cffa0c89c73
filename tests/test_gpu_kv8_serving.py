"""The 8-bit cache and the two attention calls as a server uses them together:
prompts attend to their exact keys and values and are written, drafted tokens are
written and verified, the accepted branch is read back and moved into place, the
next token decodes, and old rows go on into a TurboQuant cache.  Every step is
held to its own definition in 64 bits, on what the steps before it wrote; then
the whole step runs again as one captured graph.  Behind it: calls at the borders
between the kernels that carry them out."""
import math

import numpy as np
import pytest
import torch

from cases import Instance, assert_status_clean, compare_codes, rel_err, words_u32
from test_gpu_attn_prompt import check as check_prompt
from test_gpu_attn_tree import Case

import compressed_kv_cache_turboquant_b200 as tq

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
DEV = "cuda"
BF, HF = torch.bfloat16, torch.float16


def written(x):
    """Codes and scales of rows x [n][d] by the definition."""
    x = x.float()
    m = x.abs().amax(-1)
    s = m / torch.full_like(m, 127)                          # (a quotient by a Python number is a product by its reciprocal)
    # the quotient in 64 bits decides every rounding but an exact tie, and a tie is exact there
    c = torch.round(x.double() / s.double()[..., None].clamp(min=2.0 ** -1000)).clamp(-127, 127)
    return c.to(torch.int8), s


class Server:
    """Prompts of the given lengths, one projection of q, k and v side by side, a
    pool of pages with room for the drafts."""

    def __init__(self, lens, n, Hq, Hkv, d, page, dtype, seed):
        self.lens, self.n, self.Hq, self.Hkv, self.d, self.page, self.dtype = lens, n, Hq, Hkv, d, page, dtype
        self.c = c = Case(lens, n, Hq, Hkv, d, page, dtype, seed=seed)
        self.h, self.g = c.h, c.g
        c.kcodes.zero_(), c.vcodes.zero_(), c.kscales.zero_(), c.vscales.zero_()
        total = sum(lens)
        self.fused = torch.randn(total, (Hq + 2 * Hkv) * d, generator=self.g, device=DEV).to(dtype)
        self.q, self.k, self.v = self.split(self.fused, total)
        self.cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)
        self.out = torch.full((total, Hq, d), 77.0, dtype=dtype, device=DEV)
        self.lse = torch.full((total, Hq), 77.0, device=DEV)
        self.slots = torch.cat([self.slots_of(b, 0, m) for b, m in enumerate(lens)])
        self.draft = torch.randn(c.B * n, (Hq + 2 * Hkv) * d, generator=self.g, device=DEV).to(dtype)
        dq, self.dk, self.dv = self.split(self.draft, c.B * n)
        c.q = dq.unflatten(0, (c.B, n))
        self.draft_slots = torch.cat([self.slots_of(b, m, n) for b, m in enumerate(lens)])

    def split(self, fused, total):
        Hq, Hkv, d = self.Hq, self.Hkv, self.d
        a, b = Hq * d, (Hq + Hkv) * d
        return (fused[:, :a].unflatten(1, (Hq, d)), fused[:, a:b].unflatten(1, (Hkv, d)), fused[:, b:].unflatten(1, (Hkv, d)))

    def slots_of(self, b, first, m):
        """[m][Hkv] cache rows of tokens first .. of sequence b."""
        t = torch.arange(first, first + m, device=DEV)
        pages = self.c.table[b * self.Hkv:(b + 1) * self.Hkv].long()
        return (pages[:, t // self.page] * self.page + t % self.page).T.contiguous()

    def write(self, k, v, slots):
        c = self.c
        tq.tq_quant_kv8(self.h, k, v, slots, c.kcodes, c.kscales, c.vcodes, c.vscales)

    def step(self):
        tq.tq_attn_prompt(self.h, self.q, self.k, self.v, self.cu, self.c.scale, self.out, lse=self.lse)
        self.write(self.k, self.v, self.slots)
        self.write(self.dk, self.dv, self.draft_slots)
        self.c.run()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lens,n,Hq,Hkv,d,page", [([70, 1, 300], 6, 8, 2, 128, 16), ([200, 129], 12, 4, 1, 64, 32)])
def test_prompts_drafts_acceptance_and_decode(lens, n, Hq, Hkv, d, page, dtype):
    s = Server(lens, n, Hq, Hkv, d, page, dtype, seed=5)
    c = s.c
    s.step()
    check_prompt(s.q, s.k, s.v, s.cu, c.scale, s.out, s.lse)
    c.check()
    for x, codes, scales in ((s.k, c.kcodes, c.kscales), (s.v, c.vcodes, c.vscales)):
        want, ws = written(x)
        assert torch.equal(codes[s.slots], want) and torch.equal(scales[s.slots], ws)
    before = [t.clone() for t in (s.out, s.lse, c.out, c.lse, c.kcodes, c.vcodes, c.kscales, c.vscales)]

    # the branch 0, 2, .. of each tree is accepted: its rows are read and moved behind the context
    keep = list(range(0, n, 2))
    src = torch.cat([s.slots_of(b, m, n)[keep] for b, m in enumerate(lens)])
    dst = torch.cat([s.slots_of(b, m, len(keep)) for b, m in enumerate(lens)])
    moved = [torch.empty(src.numel(), d, dtype=torch.float32, device=DEV) for _ in range(2)]
    tq.tq_dequant_kv8(s.h, src, c.kcodes, c.kscales, c.vcodes, c.vscales, *moved)
    for x, codes, scales in ((moved[0], c.kcodes, c.kscales), (moved[1], c.vcodes, c.vscales)):
        assert torch.equal(x, codes[src.flatten()].float() * scales[src.flatten()][:, None])
    s.write(moved[0].view(-1, Hkv, d), moved[1].view(-1, Hkv, d), dst)
    for x, codes, scales in ((moved[0], c.kcodes, c.kscales), (moved[1], c.vcodes, c.vscales)):
        want, ws = written(x)
        assert torch.equal(codes[dst.flatten()], want) and torch.equal(scales[dst.flatten()], ws)

    # the next token of each sequence: a row behind the accepted ones, then one step of decode
    nxt = Case([m + len(keep) for m in lens], 1, Hq, Hkv, d, page, dtype, seed=6)
    nxt.table, nxt.kcodes, nxt.kscales, nxt.vcodes, nxt.vscales = c.table, c.kcodes, c.kscales, c.vcodes, c.vscales
    new = torch.randn(2, c.B, Hkv, d, generator=s.g, device=DEV).to(dtype)
    s.write(new[0], new[1], torch.cat([s.slots_of(b, m + len(keep), 1) for b, m in enumerate(lens)]))
    nxt.run()
    nxt.check()

    # the oldest rows go on into a TurboQuant cache
    old = s.slots_of(0, 0, min(lens[0], 64)).flatten()
    rows = torch.empty(old.numel(), d, dtype=torch.float32, device=DEV)
    tq.tq_dequant_kv8(s.h, old, c.kcodes, c.kscales, None, None, rows)
    inst = Instance(d, 4, tq.TQ_MSE, seed=3)
    kept = inst.alloc_outputs(c.kcodes.shape[0])
    tq.tq_quant_paged(inst.h, rows, old, kept["codes"], kept["norms"])
    torch.cuda.synchronize()
    at = old.cpu().numpy()
    ref = inst.oracle_quant(rows.double().cpu().numpy())
    compare_codes(words_u32(kept["codes"])[at], ref["idx"], ref["y"], inst.t_o, d, inst.bm)
    assert np.max(rel_err(kept["norms"].cpu().numpy()[at], ref["norms"])) <= 1e-5
    assert_status_clean(inst)

    # the same step as one graph, replayed on other numbers and back
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            s.step()
    torch.cuda.current_stream().wait_stream(stream)
    first = s.fused.clone()
    s.fused.copy_(torch.randn(s.fused.shape, generator=s.g, device=DEV).to(dtype))
    graph.replay()
    check_prompt(s.q, s.k, s.v, s.cu, c.scale, s.out, s.lse)
    c.check()
    s.fused.copy_(first)
    graph.replay()
    torch.cuda.synchronize()
    for got, want in zip((s.out, s.lse, c.out, c.lse), before):
        assert torch.equal(got, want)
    for t, want in ((c.kcodes, before[4]), (c.vcodes, before[5]), (c.kscales, before[6]), (c.vscales, before[7])):
        named = torch.cat([s.slots.flatten(), s.draft_slots.flatten()])
        assert torch.equal(t[named], want[named])
    assert tq.tq_device_status(s.h) == 0
    del graph


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n,Hq,Hkv,d", [
    (1, 7, 1, 128), (1, 8, 1, 128), (1, 9, 1, 128), (4, 4, 1, 64), (17, 1, 1, 64), (8, 4, 1, 128), (11, 3, 1, 128),
    (2, 4, 1, 256), (9, 1, 1, 256), (2, 130, 1, 64), (1, 129, 1, 128), (3, 40, 1, 96)])
def test_rows_beside_the_borders_of_a_block(n, Hq, Hkv, d, dtype):
    """7 to 390 rows of a kv-head, with contexts that end inside a tile and a mask that leaves rows empty."""
    c = Case([0, 61, 700], n, Hq, Hkv, d, 16, dtype, seed=n + Hq, drafts=[n, max(n - 1, 0), n], mask="any")
    c.run()
    c.check()
    assert tq.tq_device_status(c.h) == 0


def test_logits_of_minus_infinity():
    """A key of -infinity is seen with weight 0; a token that sees no other has no weights."""
    d, n = 64, 200
    h = tq.tq_create_kv8(d)
    g = torch.Generator(device=DEV).manual_seed(2)
    q, k, v = (torch.randn(n, 2, d, generator=g, device=DEV).to(BF) for _ in range(3))
    q[:, :, 7] = q[:, :, 7].abs() + 1
    k[0, :, 7] = -math.inf
    out, lse = torch.full_like(q, 77), torch.full((n, 2), 77.0, device=DEV)
    tq.tq_attn_prompt(h, q, k, v, torch.tensor([0, n], dtype=torch.int32, device=DEV), 0.1, out, lse=lse)
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all()
    check_prompt(q[1:], k[1:], v[1:], torch.tensor([0, n - 1]), 0.1, out[1:], lse[1:])
    assert tq.tq_device_status(h) == 0


@pytest.mark.parametrize("n", [1, 64])
def test_workspaces_that_are_too_small_are_refused(n):
    c = Case([3000], n, 8, 2, 128, 16, BF)
    need = tq.tq_attn_tree_workspace(c.h, 1, n, 8, 2)
    assert need > 0
    with pytest.raises(tq.TQError):
        c.run(workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))
    c.run(workspace=torch.empty(need, dtype=torch.uint8, device=DEV))
    c.check()


@pytest.mark.parametrize("d", [8, 24, 72, 120])
def test_prompts_of_a_compressed_cache_handle(d):
    """Prompt attention takes the handle that compresses the same heads, whose dimension is any multiple of 8."""
    h = Instance(d, 3, tq.TQ_MSE, seed=4).h
    g = torch.Generator(device=DEV).manual_seed(d)
    q = torch.randn(333, 6, d, generator=g, device=DEV).to(BF)
    k, v = (torch.randn(333, 2, d, generator=g, device=DEV).to(BF) for _ in range(2))
    cu = torch.tensor([0, 3, 3, 200, 333], dtype=torch.int32, device=DEV)
    out, lse = torch.full_like(q, 77), torch.full((333, 6), 77.0, device=DEV)
    tq.tq_attn_prompt(h, q, k, v, cu, d ** -0.5, out, lse=lse)
    check_prompt(q, k, v, cu, d ** -0.5, out, lse)
    assert tq.tq_device_status(h) == 0


def test_prompt_graphs_that_share_a_workspace():
    """Two captured calls with a list of items (more of them than blocks) and one workspace, replayed in turn."""
    Hq, Hkv, d, scale = 32, 8, 64, 0.125
    h = tq.tq_create_kv8(d)
    g = torch.Generator(device=DEV).manual_seed(9)
    calls = []
    sizes = ([700, 1, 2300, 64], [5, 1500, 1500])
    ws = torch.empty(max(tq.tq_attn_prompt_workspace(h, len(x), sum(x), Hq, Hkv) for x in sizes), dtype=torch.uint8, device=DEV)
    assert ws.numel() > 0
    for lens in sizes:
        n = sum(lens)
        q = torch.randn(n, Hq, d, generator=g, device=DEV).to(HF)
        k, v = (torch.randn(n, Hkv, d, generator=g, device=DEV).to(HF) for _ in range(2))
        cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)
        out = torch.zeros_like(q)
        args = (h, q, k, v, cu, scale, out)
        tq.tq_attn_prompt(*args, workspace=ws)
        want = out.clone()
        check_prompt(q, k, v, cu, scale, out, None, rows=[(0, 3), (640, 650), (1490, 1500), (2290, 2300)])
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            tq.tq_attn_prompt(*args, workspace=ws)
        calls.append((graph, out, want, args))
    for _ in range(3):
        for graph, out, want, _ in calls:
            out.zero_()
            graph.replay()
        for _, out, want, _ in calls:
            assert torch.equal(out, want)
    assert tq.tq_device_status(h) == 0
