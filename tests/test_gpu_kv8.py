"""The 8-bit paged cache through the binding: rows quantized on write and read
back, against the definition in 64 bits.  Codes, scales and values read back
have one right answer each, so every comparison here is exact."""
import pytest
import torch

import compressed_kv_cache_turboquant_b200 as tq

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
DEV = "cuda"
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def quantized(x):
    """codes, scales of the rows of x by the definition, in 64 bits."""
    a = x.double()
    bad = ~torch.isfinite(a).all(-1)
    s = (torch.where(bad[..., None], torch.zeros_like(a), a).abs().amax(-1) / 127).float()
    c = torch.where((s > 0)[..., None] & ~bad[..., None], a / s.double()[..., None], torch.zeros_like(a))
    c = c.round().clamp(-127, 127).to(torch.int8)
    return c, torch.where(bad, torch.full_like(s, float("nan")), s)


def same(a, b):
    return torch.equal(torch.nan_to_num(a.double(), nan=1e300), torch.nan_to_num(b.double(), nan=1e300))


def cache(rows, d):
    return [torch.full((rows, d), 7, dtype=torch.int8, device=DEV), torch.full((rows,), 3.0, device=DEV),
            torch.full((rows, d), 9, dtype=torch.int8, device=DEV), torch.full((rows,), 5.0, device=DEV)]


def write_and_check(h, k, v, rows, seed):
    n, H, d = k.shape
    slots = torch.randperm(rows, generator=gen(seed), device=DEV)[: n * H].reshape(n, H)
    c = cache(rows, d)
    tq.tq_quant_kv8(h, k, v, slots, *c)
    want = cache(rows, d)
    for x, i in ((k, 0), (v, 2)):
        codes, scales = quantized(x)
        want[i][slots.reshape(-1)] = codes.reshape(-1, d)
        want[i + 1][slots.reshape(-1)] = scales.reshape(-1)
    for got, ref in zip(c, want):
        assert same(got, ref)
    assert tq.tq_device_status(h) == 0
    return c, slots


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,H,d", [(1, 1, 16), (3, 5, 48), (65, 2, 64), (37, 3, 80), (130, 8, 128), (9, 1, 256), (1000, 7, 112)])
def test_rows_are_written_as_defined_and_read_back(dtype, n, H, d):
    h = tq.tq_create_kv8(d)
    g = gen(n)
    k = (torch.randn(n, H, d, generator=g, device=DEV) * (torch.randn(n, H, 1, generator=g, device=DEV) * 3).exp()).to(dtype)
    v = torch.randn(n, H, d, generator=g, device=DEV).to(dtype)
    rows = n * H + 13
    c, slots = write_and_check(h, k, v, rows, n)
    for out_type in TYPES:
        ko = torch.empty(n * H, d, dtype=out_type, device=DEV)
        vo = torch.empty_like(ko)
        tq.tq_dequant_kv8(h, slots, *c, ko, vo)
        at = slots.reshape(-1)
        # an input row with an infinity (float16 overflows here) reads back as NaN
        assert same(ko, (c[0][at].float() * c[1][at][:, None]).to(out_type))
        assert same(vo, (c[2][at].float() * c[3][at][:, None]).to(out_type))


@pytest.mark.parametrize("dtype", TYPES)
def test_quotients_on_and_beside_a_border(dtype):
    # rows whose scale is a power of two, so that halves (ties) are hit exactly, and
    # whole ranges of 16-bit values, whose quotients crowd around the borders
    d = 128
    h = tq.tq_create_kv8(d)
    half = (torch.arange(d, device=DEV) - 64.0) * 0.5
    ties = torch.stack([half.clone() * 2.0 ** e for e in range(-3, 4)])
    ties[:, 0] = 127 * 2.0 ** torch.arange(-3.0, 4.0, device=DEV)
    g = gen(3)
    bits = torch.randint(-(2 ** 15), 2 ** 15, (4096, d), generator=g, device=DEV, dtype=torch.int32).to(torch.int16)
    crowd = bits.view(torch.bfloat16 if dtype != torch.float16 else torch.float16).to(dtype)
    narrow = (torch.randint(0, 255, (4096, d), generator=g, device=DEV).float() / 2 * 1.001).to(dtype)
    for x in (ties.to(dtype), crowd, narrow):
        k = x.reshape(-1, 1, d)
        write_and_check(h, k, k.flip(0), k.shape[0] + 1, 5)


@pytest.mark.parametrize("dtype", TYPES)
def test_zeros_tiny_huge_and_non_finite_rows(dtype):
    d = 64
    h = tq.tq_create_kv8(d)
    g = gen(9)
    x = torch.randn(12, d, generator=g, device=DEV).to(dtype)
    tiny = torch.finfo(dtype).smallest_normal
    x[0] = 0
    x[1] = (x[1].float() * tiny).to(dtype)                       # the scale is subnormal in float32 for bf16 and f32
    x[2] = 0
    x[2, 5] = torch.finfo(dtype).max
    x[3, 7] = float("inf")
    x[4, 0] = -float("inf")
    x[5, 63] = float("nan")
    x[6] = -0.0
    x[7] = 0
    x[7, 1] = tiny / 64 if dtype != torch.float16 else 2.0 ** -24  # a single subnormal value
    x[8] = (torch.arange(d, device=DEV).float() * tiny * 2.0 ** -6).to(dtype)
    k = x.reshape(12, 1, d)
    write_and_check(h, k, k.flip(0), 20, 1)


def test_a_bad_row_spoils_only_itself():
    d = 128
    h = tq.tq_create_kv8(d)
    k = torch.randn(6, 1, d, generator=gen(1), device=DEV)
    k[2, 0, 3] = float("nan")
    c = cache(6, d)
    slots = torch.arange(6, device=DEV)
    tq.tq_quant_kv8(h, k, None, slots.reshape(6, 1), c[0], c[1])
    out = torch.empty(6, d, device=DEV)
    tq.tq_dequant_kv8(h, slots, c[0], c[1], None, None, out)
    bad = torch.isnan(out).all(1)
    assert bad.tolist() == [False, False, True, False, False, False]
    assert torch.isfinite(out[~bad]).all()
    assert torch.equal(c[2], cache(6, d)[2]) and torch.equal(c[3], cache(6, d)[3])   # keys only: the values' arrays stay


def test_slices_of_a_fused_projection_and_one_token():
    d, Hq, Hkv, n = 128, 8, 2, 33
    h = tq.tq_create_kv8(d)
    qkv = torch.randn(n, (Hq + 2 * Hkv) * d, generator=gen(2), device=DEV).to(torch.bfloat16)
    k = qkv[:, Hq * d:(Hq + Hkv) * d].view(n, Hkv, d)
    v = qkv[:, (Hq + Hkv) * d:].view(n, Hkv, d)
    write_and_check(h, k, v, 100, 3)
    write_and_check(h, k[:1], v[:1], 9, 4)
    with pytest.raises(ValueError):
        tq.tq_quant_kv8(h, k.transpose(0, 1), None, torch.zeros(Hkv, n, dtype=torch.int64, device=DEV), *cache(4, d)[:2])


def test_padding_and_slots_outside_the_cache():
    d, rows = 64, 10
    h = tq.tq_create_kv8(d)
    k = torch.randn(5, 1, d, generator=gen(4), device=DEV)
    slots = torch.tensor([[3], [-1], [9], [-(2 ** 40)], [0]], device=DEV)
    c = cache(rows, d)
    tq.tq_quant_kv8(h, k, k, slots, *c)
    assert tq.tq_device_status(h) == 0                            # padding is no event
    codes, scales = quantized(k.reshape(5, d))
    want = cache(rows, d)
    for i in (0, 2, 4):
        want[0][slots[i, 0]], want[1][slots[i, 0]] = codes[i], scales[i]
        want[2][slots[i, 0]], want[3][slots[i, 0]] = codes[i], scales[i]
    assert all(same(a, b) for a, b in zip(c, want))
    slots[1], slots[3] = rows, 2 ** 40
    tq.tq_quant_kv8(h, k, k, slots, *c)
    assert tq.tq_device_status(h) == tq.TQ_STATUS_RANGE
    assert all(same(a, b) for a, b in zip(c, want))
    out = torch.full((5, d), 8.0, device=DEV)
    tq.tq_dequant_kv8(h, slots, *c[:2], None, None, out)
    assert tq.tq_device_status(h) == tq.TQ_STATUS_RANGE
    assert (out[1] == 0).all() and (out[3] == 0).all() and (out[0] != 0).any()


def test_nothing_to_do_and_a_second_stream():
    d = 128
    h = tq.tq_create_kv8(d)
    c = cache(300, d)
    empty = torch.empty(0, 2, d, device=DEV)
    tq.tq_quant_kv8(h, empty, empty, torch.empty(0, 2, dtype=torch.int64, device=DEV), *c)
    tq.tq_dequant_kv8(h, torch.empty(0, dtype=torch.int64, device=DEV), *c, torch.empty(0, d, device=DEV))
    k = torch.randn(100, 2, d, generator=gen(6), device=DEV)
    slots = torch.arange(200, device=DEV).reshape(100, 2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    tq.tq_quant_kv8(h, k, k, slots, *c, stream=side)
    out = torch.empty(200, d, device=DEV)
    tq.tq_dequant_kv8(h, slots, *c, out, stream=side.cuda_stream)
    side.synchronize()
    codes, scales = quantized(k.reshape(-1, d))
    assert torch.equal(out, codes.float() * scales[:, None])


def test_a_captured_write_and_read_replay_on_new_values():
    d = 64
    h = tq.tq_create_kv8(d)
    c = cache(64, d)
    k = torch.zeros(16, 2, d, device=DEV, dtype=torch.bfloat16)
    slots = torch.arange(32, device=DEV).reshape(16, 2)
    out = torch.empty(32, d, device=DEV)
    tq.tq_quant_kv8(h, k, k, slots, *c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.tq_quant_kv8(h, k, k, slots, *c)
        tq.tq_dequant_kv8(h, slots, *c, out)
    for seed in (1, 2):
        k.copy_(torch.randn(16, 2, d, generator=gen(seed), device=DEV))
        slots.copy_(torch.randperm(64, generator=gen(seed + 7), device=DEV)[:32].reshape(16, 2))
        graph.replay()
        torch.cuda.synchronize()
        codes, scales = quantized(k.reshape(-1, d))
        assert torch.equal(out, codes.float() * scales[:, None])


def test_rows_past_32_bits_of_bytes():
    # 17 million rows of 256: the last row's byte offset is above 2^32
    d, rows = 256, 17_000_000
    h = tq.tq_create_kv8(d)
    codes = torch.zeros(rows, d, dtype=torch.int8, device=DEV)
    scales = torch.zeros(rows, device=DEV)
    k = torch.randn(3, 1, d, generator=gen(8), device=DEV)
    slots = torch.tensor([[rows - 1], [rows - 2], [16_777_216]], device=DEV)
    tq.tq_quant_kv8(h, k, None, slots, codes, scales)
    c, s = quantized(k.reshape(3, d))
    at = slots.reshape(-1)
    assert torch.equal(codes[at], c) and torch.equal(scales[at], s)
    out = torch.empty(3, d, device=DEV)
    tq.tq_dequant_kv8(h, slots, codes, scales, None, None, out)
    assert torch.equal(out, c.float() * s[:, None])
