"""Prompt attention where the weights of a row lie far apart: what the 16-bit
weights of the value product may lose, against the definition in 64 bits.

Tolerance, by arithmetic, beside that of float32 logits and sums (delta, 2^-20): a
weight is kept to u = eps / 2 of the type relative to itself; a float16 one below
2^-14 of what the row's reference weighs in the kernel (2^7 float16 units: 2^-21 of
the reference, which no weight passes by more than 2^8) to half the last place of
a subnormal, 2^-25 of those units, so 2^-32 of the reference.  The reference is one
of the row's weights, so with w_t the true weights (their sum is 1) this is at most
n 2^-32 max_t |v_t| for n keys.  Rounding the result costs u |out|."""
import math

import pytest
import torch

import compressed_kv_cache_turboquant_b200 as tq

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
DEV = "cuda"
BF, HF = torch.bfloat16, torch.float16


def check_last_row(q, k, v, out, lse):
    """The last token, which sees all n keys, of head 0 (logit scale 1)."""
    n, d = k.shape[0], k.shape[2]
    u = torch.finfo(q.dtype).eps / 2
    q, K, V = q[-1, 0].double(), k[:, 0].double(), v[:, 0].double()
    z = K @ q
    want_lse = torch.logsumexp(z, 0)
    w = torch.exp(z - want_lse)
    want, A = w @ V, w @ V.abs()
    delta = (d + 2) * 2.0 ** -24 * (K.abs() @ q.abs()).amax() + 2.0 ** -22 * z.abs().amax()
    tol = (u + 2 * delta + 2.0 ** -20) * A + u * want.abs() + n * 2.0 ** -32 * V.abs().amax(0) + 2.0 ** -25
    err = (out[-1, 0].double() - want).abs()
    assert (err <= tol).all(), float((err / tol).max())
    assert (lse[-1, 0].double() - want_lse).abs() <= delta + 2.0 ** -20 + 2.0 ** -23 * want_lse.abs()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,place", [(131072, 0), (131072, 131071), (40000, 20000)])
def test_one_dominant_key_and_a_long_tail(n, place, d, dtype):
    """The tail's keys weigh 2^-25.2 of the dominant one each: together they are 2^-8.2 of the row at 131072."""
    g = torch.Generator(device=DEV).manual_seed(d)
    h = tq.tq_create_kv8(d)
    q, k = (torch.zeros(n, 1, d, dtype=dtype, device=DEV) for _ in range(2))
    q[:, 0, 0] = 1
    k[:, 0, 0] = 8 - 25.2 * math.log(2)
    k[place, 0, 0] = 8
    v = (1 + 0.1 * torch.randn(n, 1, d, generator=g, device=DEV)).to(dtype)
    v[place] = 0                                              # the result is the tail's alone
    out, lse = torch.full_like(q, 77), torch.full((n, 1), 77.0, device=DEV)
    tq.tq_attn_prompt(h, q, k, v, torch.tensor([0, n], dtype=torch.int32, device=DEV), 1.0, out, lse=lse)
    check_last_row(q, k, v, out, lse)
    assert tq.tq_device_status(h) == 0


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
def test_weights_far_above_the_rows_reference(d, dtype):
    """Logits that climb by just under 2^8 after the first tile: the reference stays, the weights are the largest there are."""
    n = 1000
    g = torch.Generator(device=DEV).manual_seed(d)
    h = tq.tq_create_kv8(d)
    q, k = (torch.zeros(n, 1, d, dtype=dtype, device=DEV) for _ in range(2))
    q[:, 0, 0] = 1
    k[128:, 0, 0] = 5.53                                      # 2^7.98
    v = torch.randn(n, 1, d, generator=g, device=DEV).to(dtype)
    out, lse = torch.full_like(q, 77), torch.full((n, 1), 77.0, device=DEV)
    tq.tq_attn_prompt(h, q, k, v, torch.tensor([0, n], dtype=torch.int32, device=DEV), 1.0, out, lse=lse)
    check_last_row(q, k, v, out, lse)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 12.5, 2.0 ** 13])
def test_logits_beyond_the_exact_integers_stay_finite(size, dtype):
    """Logits of 2^24 and more, whose own float32 roundings are whole powers of two of a weight: the result is
    still a mean of values."""
    n, d = 400, 64
    g = torch.Generator(device=DEV).manual_seed(1)
    h = tq.tq_create_kv8(d)
    q = (size * (1 + torch.rand(n, 2, d, generator=g, device=DEV) * 2.0 ** -6)).to(dtype)
    k = (size / d * (1 + torch.rand(n, 2, d, generator=g, device=DEV) * 2.0 ** -6)).to(dtype)
    v = torch.rand(n, 2, d, generator=g, device=DEV).to(dtype)
    out, lse = torch.full_like(q, 77), torch.full((n, 2), 77.0, device=DEV)
    tq.tq_attn_prompt(h, q, k, v, torch.tensor([0, n], dtype=torch.int32, device=DEV), 1.0, out, lse=lse)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    assert (out >= 0).all() and (out <= 1.01).all()
