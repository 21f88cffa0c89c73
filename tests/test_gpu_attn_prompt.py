"""Causal attention over packed prompts against the definition in 64 bits.

Tolerance of an output element, by arithmetic: with A = sum_t w_t |v_t| the
exact sum of magnitudes and u = eps / 2 of the type, rounding the weights to the
type costs at most u A, rounding the result u |out|; the logits (d products in
float32, then scaled) are off by at most
  delta = scale (d + 2) 2^-24 max_t sum_i |q_i k_ti| + 2^-22 max_t |logit_t|
each, which moves a weight by 2 delta relative at most (it and their sum), and
float32 exponentials and sums add under 2^-20.  float16 weights below 2^-14
round by up to 2^-25 absolute, n of them; weights below 2^-126, which are not
normal float32, may count as 0.  The log-sum is off by delta + 2^-20
and a float32 rounding of itself."""
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


def handle(d):
    return tq.tq_create_kv8(d)


def inputs(total, Hq, Hkv, d, dtype, seed, size=1.0):
    g = gen(seed)
    q = (torch.randn(total, Hq, d, generator=g, device=DEV) * size).to(dtype)
    k, v = (torch.randn(total, Hkv, d, generator=g, device=DEV).to(dtype) for _ in range(2))
    return q, k, v


def cu_of(lens, start=0):
    cu = [start]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def rows_exact(q, K, V, first, scale):
    """Exact out, lse and their tolerances of rows q [m][d] (positions first ..) over K, V [n][d]."""
    q, K, V = q.double(), K.double(), V.double()
    z = scale * (q @ K.T)
    sees = torch.arange(K.shape[0], device=DEV)[None, :] <= (first + torch.arange(q.shape[0], device=DEV))[:, None]
    z = z.masked_fill(~sees, -math.inf)
    lse = torch.logsumexp(z, 1)
    w = torch.exp(z - lse[:, None])
    A = w @ V.abs()
    mags = scale * (q.abs() @ K.abs().T).masked_fill(~sees, 0).amax(1)
    zmax = z.masked_fill(~sees, 0).abs().amax(1)
    delta = (q.shape[1] + 2) * 2.0 ** -24 * mags + 2.0 ** -22 * zmax
    return w @ V, lse, A, delta


def check_rows(out, lse, want, want_lse, A, delta, dtype, n):
    u = torch.finfo(dtype).eps / 2
    tol = (u + 2 * delta[:, None] + 2.0 ** -20) * A + u * want.abs() + n * 2.0 ** -126 * A.amax()
    if dtype == HF:
        tol = tol + n * 2.0 ** -25 * A.amax() + 2.0 ** -25
    err = (out.double() - want).abs()
    assert torch.isfinite(out).all()
    assert (err <= tol).all(), float((err / tol).max())
    if lse is not None:
        tl = delta + 2.0 ** -20 + 2.0 ** -23 * want_lse.abs()
        assert ((lse.double() - want_lse).abs() <= tl).all(), float(((lse.double() - want_lse).abs() / tl).max())


def check(q, k, v, cu, scale, out, lse, rows=None):
    """Every row of every sequence (or the rows named) against the exact one."""
    Hq, Hkv = q.shape[1], k.shape[1]
    G = Hq // Hkv
    bounds = cu.tolist()
    for a, b in zip(bounds, bounds[1:]):
        if b <= a:
            continue
        for h in range(Hq):
            for i0, i1 in rows or [(0, b - a)]:
                i1 = min(i1, b - a)
                if i0 >= i1:
                    continue
                want, wl, A, delta = rows_exact(q[a + i0:a + i1, h], k[a:a + i1, h // G], v[a:a + i1, h // G], i0, scale)
                check_rows(out[a + i0:a + i1, h], None if lse is None else lse[a + i0:a + i1, h], want, wl, A, delta,
                           q.dtype, i1)


def run(h, q, k, v, cu, scale, **kw):
    out = torch.full(q.shape, 77.0, dtype=q.dtype, device=DEV)
    lse = torch.full(q.shape[:2], 77.0, device=DEV)
    tq.tq_attn_prompt(h, q, k, v, cu, scale, out, lse=lse, **kw)
    return out, lse


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lens,Hq,Hkv,d", [
    ([1], 1, 1, 128), ([1], 32, 8, 128), ([2, 1, 0, 5], 8, 2, 64), ([127], 4, 4, 128), ([128], 4, 1, 128),
    ([129], 2, 2, 64), ([255, 256, 257], 8, 2, 128), ([64, 0, 1, 63, 65, 0], 32, 8, 128), ([300, 17, 511], 6, 2, 128),
    ([33, 400], 10, 2, 64), ([200, 1, 90], 7, 1, 80), ([385], 16, 1, 128), ([97, 3], 32, 1, 64), ([150], 128, 1, 16),
    ([70, 260], 96, 2, 32), ([140], 48, 1, 128), ([513, 640, 12], 4, 2, 96), ([131, 259], 3, 3, 8), ([1100], 2, 1, 112),
])
def test_packed_prompts(lens, Hq, Hkv, d, dtype):
    if d % 16:
        import numpy as np
        h = tq.tq_create(d, 4, tq.TQ_MSE, np.eye(d))       # any handle gives d; an 8-bit one takes multiples of 16
    else:
        h = handle(d)
    total = sum(lens)
    q, k, v = inputs(total, Hq, Hkv, d, dtype, total + Hq)
    cu = cu_of(lens)
    out, lse = run(h, q, k, v, cu, 1 / math.sqrt(d))
    check(q, k, v, cu, 1 / math.sqrt(d), out, lse)
    assert tq.tq_device_status(h) == 0


@pytest.mark.parametrize("dtype", [BF, HF])
def test_long_prompt_sampled(dtype):
    n, Hq, Hkv, d = 9001, 8, 2, 128
    h = handle(d)
    q, k, v = inputs(n, Hq, Hkv, d, dtype, 3, size=3.0)
    cu = cu_of([n])
    out, lse = run(h, q, k, v, cu, 1 / math.sqrt(d))
    check(q, k, v, cu, 1 / math.sqrt(d), out, lse, rows=[(0, 40), (250, 260), (4090, 4103), (8990, 9001)])
    assert torch.isfinite(out).all()
    assert tq.tq_device_status(h) == 0


def test_many_sequences_of_up_to_three_tokens():
    lens = [(7 * i) % 4 for i in range(4096)]
    d = 64
    h = handle(d)
    q, k, v = inputs(sum(lens), 2, 1, d, BF, 4)
    cu = cu_of(lens)
    out, lse = run(h, q, k, v, cu, 0.125)
    # all sequences at once: dense over the neighbourhood of three tokens
    start = torch.repeat_interleave(cu[:-1].long(), torch.tensor(lens, device=DEV))
    at = torch.arange(len(start), device=DEV)
    for hq in range(2):
        z = torch.full((len(at), 3), -math.inf, dtype=torch.float64, device=DEV)
        for j in range(3):
            src = at - j
            ok = src >= start
            z[ok, j] = 0.125 * (q[at[ok], hq].double() * k[src[ok], 0].double()).sum(-1)
        w = torch.softmax(z, 1)
        src = (at[:, None] - torch.arange(3, device=DEV)).clamp(min=0)
        want = (w[..., None] * v[src, 0].double()).sum(1)
        A = (w[..., None] * v[src, 0].double().abs()).sum(1)
        mags = 0.125 * 3 * d * torch.ones(len(at), device=DEV, dtype=torch.float64)   # |q||k| of normal values: well below
        check_rows(out[:, hq], lse[:, hq], want, torch.logsumexp(z, 1), A, (d + 2) * 2.0 ** -24 * mags, BF, 3)
    assert tq.tq_device_status(h) == 0


@pytest.mark.parametrize("d,Hq,Hkv", [(128, 8, 2), (64, 2, 2)])
def test_tokens_of_no_sequence_are_left_alone(d, Hq, Hkv):
    h = handle(d)
    total, a, lens = 500, 37, [100, 0, 201]
    q, k, v = inputs(total, Hq, Hkv, d, BF, 5)
    for t in (q, k, v):                                     # what lies outside may hold anything
        t[:a] = float("nan")
        t[a + sum(lens):] = float("inf")
    cu = cu_of(lens, a)
    out, lse = run(h, q, k, v, cu, 0.1)
    check(q, k, v, cu, 0.1, out, lse)
    assert (out[:a] == 77).all() and (out[a + sum(lens):] == 77).all()
    assert (lse[:a] == 77).all() and (lse[a + sum(lens):] == 77).all()
    assert tq.tq_device_status(h) == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("place", [0, 130, 299])
def test_a_bad_value_or_key_reaches_only_who_sees_it(bad, place):
    d, n, Hq, Hkv = 64, 300, 4, 2
    h = handle(d)
    q, k, v = inputs(2 * n, Hq, Hkv, d, BF, 6)
    cu = cu_of([n, n])
    clean, clean_lse = run(h, q, k, v, cu, 0.125)
    v2 = v.clone()
    v2[place, 0, 5] = bad
    out, lse = run(h, q, k, v2, cu, 0.125)
    assert torch.equal(lse, clean_lse)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[place:n, 0:2, 5] = True                             # the tokens from it on, heads of its group, its channel
    assert not torch.isfinite(out[hit]).any()
    if bad == bad:
        first = out[place, 0, 5].float()
        assert first == bad                                 # a positive weight times an infinity
    assert torch.equal(out[~hit], clean[~hit])
    k2 = k.clone()
    k2[place, 1, 9] = float("nan")
    out, lse = run(h, q, k2, v, cu, 0.125)
    hit = torch.zeros(2 * n, Hq, dtype=torch.bool, device=DEV)
    hit[place:n, 2:4] = True
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])
    assert tq.tq_device_status(h) == 0


@pytest.mark.parametrize("scale", [0.0, 1e-3, 6.0])
def test_flat_and_sharp_softmax(scale):
    d, lens = 128, [200, 77]
    h = handle(d)
    q, k, v = inputs(sum(lens), 4, 2, d, BF, 7)
    cu = cu_of(lens)
    out, lse = run(h, q, k, v, cu, scale)
    check(q, k, v, cu, scale, out, lse)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_rising_and_falling_logits(dtype):
    # keys whose logits climb (the running maximum moves at every tile) or fall by hundreds
    d, n = 64, 700
    h = handle(d)
    q, k, v = inputs(n, 2, 2, d, dtype, 8)
    ramp = torch.linspace(-40, 40, n, device=DEV)
    q[:] = 0
    q[:, :, 0] = 4
    k[:, 0, 0] = ramp.to(dtype)
    k[:, 1, 0] = ramp.flip(0).to(dtype)
    cu = cu_of([n])
    out, lse = run(h, q, k, v, cu, 1.0)
    check(q, k, v, cu, 1.0, out, lse)


def test_slices_of_a_fused_projection():
    d, Hq, Hkv, lens = 128, 8, 2, [70, 200]
    h = handle(d)
    total = sum(lens)
    qkv = torch.randn(total, (Hq + 2 * Hkv) * d + 8, generator=gen(9), device=DEV).to(BF)
    q = qkv[:, :Hq * d].view(total, Hq, d)
    k = qkv[:, Hq * d:(Hq + Hkv) * d].view(total, Hkv, d)
    v = qkv[:, (Hq + Hkv) * d:(Hq + 2 * Hkv) * d].view(total, Hkv, d)
    cu = cu_of(lens)
    out, lse = run(h, q, k, v, cu, 0.09)
    check(q, k, v, cu, 0.09, out, lse)
    plain, _ = run(h, q.contiguous(), k.contiguous(), v.contiguous(), cu, 0.09)
    assert torch.equal(out, plain)


def test_without_lse_and_the_same_twice():
    d, lens = 128, [1000, 3, 513]
    h = handle(d)
    q, k, v = inputs(sum(lens), 32, 8, d, BF, 10)
    cu = cu_of(lens)
    a, _ = run(h, q, k, v, cu, 0.1)
    b = torch.empty_like(a)
    tq.tq_attn_prompt(h, q, k, v, cu, 0.1, b)
    assert torch.equal(a, b)


@pytest.mark.parametrize("cu,means", [([0, 50, 30, 90], [0, 50, 50, 90]), ([-5, 20, 90], [0, 20, 90]),
                                      ([0, 40, 2 ** 31 - 1], [0, 40, 90]), ([80, 10, 5, 60], [80, 80, 80, 80]),
                                      ([2 ** 30, 5, 9], [90, 90, 90]), ([-(2 ** 31), -3, 70], [0, 0, 70])])
def test_bounds_out_of_order_or_out_of_range(cu, means):
    d = 64
    h = handle(d)
    q, k, v = inputs(90, 4, 2, d, BF, 11)
    out, lse = run(h, q, k, v, torch.tensor(cu, dtype=torch.int32, device=DEV), 0.125)
    want, want_lse = run(h, q, k, v, torch.tensor(means, dtype=torch.int32, device=DEV), 0.125)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_nothing_to_do():
    d = 64
    h = handle(d)
    e = torch.empty(0, 4, d, dtype=BF, device=DEV)
    tq.tq_attn_prompt(h, e, e[:, :2], e[:, :2], torch.zeros(3, dtype=torch.int32, device=DEV), 0.1, e.clone())
    q, k, v = inputs(5, 4, 2, d, BF, 1)
    out, _ = run(h, q, k, v, torch.zeros(1, dtype=torch.int32, device=DEV), 0.1)
    assert (out == 77).all()
    out, _ = run(h, q, k, v, torch.zeros(9, dtype=torch.int32, device=DEV), 0.1)
    assert (out == 77).all()


def test_a_captured_call_replays_with_other_lengths():
    d, total = 128, 600
    h = handle(d)
    q, k, v = inputs(total, 8, 2, d, BF, 12)
    cu = cu_of([200, 200, 200])
    out, lse = run(h, q, k, v, cu, 0.1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.tq_attn_prompt(h, q, k, v, cu, 0.1, out, lse=lse)
    for lens in ([600, 0, 0], [1, 598, 1], [100, 400, 0], [128, 256, 127]):
        cu.copy_(cu_of(lens))
        out.fill_(77)
        graph.replay()
        torch.cuda.synchronize()
        check(q, k, v, cu, 0.1, out, lse)
        assert (out[sum(lens):] == 77).all()
    assert tq.tq_device_status(h) == 0


def test_two_streams_at_once():
    d, lens = 128, [700, 900]
    h = handle(d)
    sets = [inputs(sum(lens), 8, 2, d, BF, 20 + i) for i in range(2)]
    cu = cu_of(lens)
    want = [run(h, *s, cu, 0.1)[0] for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [torch.empty_like(w) for w in want]
    for _ in range(5):
        for s, st, o in zip(sets, streams, got):
            tq.tq_attn_prompt(h, *s, cu, 0.1, o, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert tq.tq_device_status(h) == 0


def test_refusals_of_the_binding():
    d = 64
    h = handle(d)
    q, k, v = inputs(10, 4, 2, d, BF, 1)
    cu, out = cu_of([10]), torch.empty_like(q)
    bad = [dict(q=q.float()), dict(k=k.to(HF)), dict(v=v[:9]), dict(cu=cu.long()), dict(out=out[:, :2]),
           dict(out=out.float()), dict(q=q.transpose(0, 1)), dict(k=k[..., ::2]), dict(cu=cu.cpu()), dict(k=k[:, :, :32])]
    for b in bad:
        a = dict(q=q, k=k, v=v, cu=cu, out=out) | b
        with pytest.raises((ValueError, TypeError, tq.TQError)):
            tq.tq_attn_prompt(h, a["q"], a["k"], a["v"], a["cu"], 0.1, a["out"])
    with pytest.raises(tq.TQError):
        tq.tq_attn_prompt(h, q, k[:, :1].expand(10, 3, d).contiguous(), k[:, :1].expand(10, 3, d).contiguous(), cu, 0.1, out)
    with pytest.raises(tq.TQError):
        tq.tq_attn_prompt(h, q, k, v, cu, float("nan"), out)
    with pytest.raises(tq.TQError):
        tq.tq_attn_prompt(tq.tq_create_kv8(144), *(torch.zeros(2, 1, 144, dtype=BF, device=DEV),) * 3, cu_of([2]), 0.1,
                          torch.zeros(2, 1, 144, dtype=BF, device=DEV))
