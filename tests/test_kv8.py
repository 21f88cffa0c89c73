"""The 8-bit cache's calls refuse bad arguments before any GPU work (no GPU needed)."""
import ctypes

import pytest
import torch

tq = pytest.importorskip("compressed_kv_cache_turboquant_b200")
from compressed_kv_cache_turboquant_b200 import _lib  # noqa: E402

L = _lib.lib
P, Q = ctypes.c_void_p(4096), ctypes.c_void_p(4104)      # an aligned and a misaligned address; never read


def handle_of(d, variant=_lib.TQ_KV8):
    """The head of a handle (d, b, variant, mse bits): all that the checks of arguments look at."""
    return (ctypes.c_int * 1024)(d, 8, variant, 8)


def test_create_refuses_unsupported_dimensions():
    h = ctypes.c_void_p()
    for d in (0, 8, 24, 120, 264, 272, -16):
        assert L.tq_create_kv8(ctypes.byref(h), d) == _lib.TQ_EUNSUPPORTED
    assert L.tq_create_kv8(None, 128) == _lib.TQ_EINVAL


def quant(h=None, k=P, v=P, dtype=_lib.TQ_BF16, n=4, Hkv=2, ks=256, vs=256, slots=P, kc=P, ksc=P, vc=P, vsc=P, rows=64):
    h = handle_of(128) if h is None else h
    return L.tq_quant_kv8(h, k, v, dtype, n, Hkv, ks, vs, slots, kc, ksc, vc, vsc, rows, None)


def test_quant_refusals():
    E, U, A = _lib.TQ_EINVAL, _lib.TQ_EUNSUPPORTED, _lib.TQ_EALIGN
    assert L.tq_quant_kv8(None, P, P, 1, 4, 2, 256, 256, P, P, P, P, P, 64, None) == E
    for variant in (_lib.TQ_MSE, _lib.TQ_PROD, _lib.TQ_POLAR):
        assert quant(h=handle_of(128, variant)) == E
    assert quant(dtype=3) == U and quant(dtype=-1) == U
    assert quant(n=-1) == E and quant(Hkv=0) == E and quant(rows=-1) == E
    assert quant(n=1 << 30, Hkv=2) == U                                   # 2^31 rows
    assert quant(ks=248) == E and quant(ks=260) == E and quant(vs=255) == E
    assert quant(ks=258, dtype=_lib.TQ_F32) == E                          # 8 bytes off a 16-byte unit
    for name in ("k", "slots", "kc", "ksc", "vc", "vsc"):
        assert quant(**{name: None}) == E, name
    for name in ("k", "v", "slots", "kc", "ksc", "vc", "vsc"):
        assert quant(**{name: Q}) == A, name
    assert b"aligned" in L.tq_last_error()
    assert quant(n=0, k=None) == _lib.TQ_OK                               # nothing to do


def dequant(h=None, n=4, slots=P, kc=P, ksc=P, vc=P, vsc=P, rows=64, k=P, v=P, dtype=_lib.TQ_BF16):
    h = handle_of(128) if h is None else h
    return L.tq_dequant_kv8(h, n, slots, kc, ksc, vc, vsc, rows, k, v, dtype, None)


def test_dequant_refusals():
    E, U, A = _lib.TQ_EINVAL, _lib.TQ_EUNSUPPORTED, _lib.TQ_EALIGN
    assert L.tq_dequant_kv8(None, 4, P, P, P, P, P, 64, P, P, 1, None) == E
    assert dequant(h=handle_of(128, _lib.TQ_MSE)) == E
    assert dequant(dtype=9) == U and dequant(n=-1) == E and dequant(n=1 << 31) == U and dequant(rows=-5) == E
    for name in ("slots", "kc", "ksc", "vc", "vsc", "k"):
        assert dequant(**{name: None}) == E, name
    for name in ("slots", "kc", "ksc", "vc", "vsc", "k", "v"):
        assert dequant(**{name: Q}) == A, name
    assert dequant(n=0, k=None) == _lib.TQ_OK


def test_calls_of_the_other_caches_refuse_an_8_bit_handle():
    h = handle_of(128)
    E = _lib.TQ_EINVAL
    assert L.tq_quant_mse(h, P, 1, 4, 128, P, P, 1, None) == E
    assert L.tq_quant_prod(h, P, 1, 4, 128, P, P, P, P, 1, None) == E
    assert L.tq_dequant_mse(h, P, P, 4, P, 0, None) == E
    assert L.tq_ip_scores(h, P, 1, P, P, P, P, 4, P, 0, None, None, P, 1 << 20, None) == E
    assert L.tq_quant_gather(h, P, 1, 4, 128, P, P, P, P, P, 1, None) == E
    assert L.tq_quant_paged(h, P, 1, 4, 128, None, P, P, P, P, P, 0, None) == E
    assert L.tq_quant_polar(h, P, 1, 4, 128, P, P, 1, None) == E
    assert L.tq_dequant_polar(h, P, P, 4, P, 0, None) == E
    one = (ctypes.c_void_p * 1)(ctypes.addressof(h))
    ptrs = (ctypes.c_void_p * 1)(4096)
    assert L.tq_quant_gather_groups(one, 1, P, 1, 4, 128, P, ptrs, ptrs, ptrs, ptrs, 1, None) == E
    assert L.tq_attn_logits(one, 1, None, P, 1, 128, 1, 8, 2, 4, 4, ptrs, ptrs, ptrs, ptrs, ctypes.c_float(1), P, P,
                            1 << 20, None) == E
    f = ctypes.c_float(0.1)
    assert L.tq_attn_decode(h, h, P, 1, 1, 8, 2, 4, 4, P, P, P, P, P, P, f, P, P, 1 << 30, None) == E
    assert L.tq_attn_prefill(h, h, P, 1, 1, 4, 8, 2, 4, 4, P, P, P, P, P, P, f, P, P, 1 << 30, None) == E
    assert L.tq_attn_merge(h, P, 2, 4, P, None) == E


def test_binding_refuses_cpu_tensors():
    t = torch.zeros(2, 1, 16)
    h = tq.api.Handle(0, 16, 8, tq.TQ_KV8)
    with pytest.raises(ValueError):
        tq.tq_quant_kv8(h, t, t, torch.zeros(2, 1, dtype=torch.int64), torch.zeros(4, 16, dtype=torch.int8), torch.zeros(4))
    with pytest.raises(ValueError):
        tq.tq_dequant_kv8(h, torch.zeros(2, dtype=torch.int64), torch.zeros(4, 16, dtype=torch.int8), torch.zeros(4), None,
                          None, torch.zeros(2, 16))
