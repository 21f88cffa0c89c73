"""Prompt and drafted-token attention refuse bad arguments before any GPU work
(no GPU needed)."""
import ctypes

import pytest

tq = pytest.importorskip("compressed_kv_cache_turboquant_b200")
from compressed_kv_cache_turboquant_b200 import _lib, api  # noqa: E402

L = _lib.lib
P, Q = ctypes.c_void_p(4096), ctypes.c_void_p(4104)      # an aligned and a misaligned address; never read
E, U, A, W = _lib.TQ_EINVAL, _lib.TQ_EUNSUPPORTED, _lib.TQ_EALIGN, _lib.TQ_EWORKSPACE
BIG = 1 << 50


def handle_of(d, variant=_lib.TQ_KV8):
    """The head of a handle (d, b, variant, mse bits): all that the checks of arguments look at."""
    return (ctypes.c_int * 1024)(d, 8, variant, 8)


def prompt(d=128, q=P, k=P, v=P, dtype=_lib.TQ_BF16, cu=P, nseq=3, total=100, Hq=8, Hkv=2, qs=1024, ks=256, vs=256,
           scale=0.1, out=P, lse=P, ws=P, ws_bytes=0):
    return L.tq_attn_prompt(handle_of(d), q, k, v, dtype, cu, nseq, total, Hq, Hkv, qs, ks, vs, scale, out, lse, ws,
                            ws_bytes, None)


def test_prompt_refusals():
    assert L.tq_attn_prompt(None, P, P, P, 1, P, 1, 9, 8, 2, 1024, 256, 256, 0.1, P, P, P, 0, None) == E
    assert prompt(d=144) == U and prompt(dtype=_lib.TQ_F32) == U and prompt(dtype=7) == U
    assert prompt(nseq=-1) == E and prompt(total=-1) == E and prompt(Hq=-8) == E and prompt(Hkv=0) == E
    assert prompt(Hq=9) == E                                              # not whole groups
    assert prompt(Hq=129, Hkv=1, qs=129 * 128) == U
    assert prompt(nseq=_lib.TQ_MAX_SEQS + 1) == U and prompt(total=1 << 25) == U
    for scale in (-0.5, float("inf"), float("nan")):
        assert prompt(scale=scale) == E
    assert prompt(qs=1016) == E and prompt(ks=248) == E and prompt(vs=260) == E and prompt(ks=0) == E
    for name in ("q", "k", "v", "cu", "out"):
        assert prompt(**{name: None}) == E, name
    for name in ("q", "k", "v", "cu", "out", "lse", "ws"):
        assert prompt(**{name: Q}) == A, name
    assert b"aligned" in L.tq_last_error()
    for nothing in (dict(nseq=0), dict(total=0), dict(Hq=0)):
        assert prompt(q=None, **nothing) == _lib.TQ_OK


def test_prompt_workspace():
    h = handle_of(128)
    need = L.tq_attn_prompt_workspace(h, 3, 100000, 8, 2)
    assert need >= 100000 // 64 * 16                                      # a record for every two row tiles of 32 tokens
    assert prompt(total=100000, ws=None, ws_bytes=BIG) == W and prompt(total=100000, ws_bytes=need - 1) == W
    assert L.tq_attn_prompt_workspace(None, 3, 100, 8, 2) == 0
    for args in ((-1, 100, 8, 2), (3, -1, 8, 2), (3, 100, -1, 2), (3, 100, 8, 0), (0, 100, 8, 2), (3, 0, 8, 2), (3, 100, 0, 2)):
        assert L.tq_attn_prompt_workspace(h, *args) == 0


def tree(d=128, variant=_lib.TQ_KV8, q=P, dtype=_lib.TQ_BF16, qs=1024, B=3, n=5, Hq=8, Hkv=2, ctx=P, drafts=P, mask=P,
         table=P, max_pages=9, page=16, kc=P, ks=P, vc=P, vs=P, rows=4096, scale=0.1, out=P, lse=P, ws=P, ws_bytes=0):
    return L.tq_attn_tree(handle_of(d, variant), q, dtype, qs, B, n, Hq, Hkv, ctx, drafts, mask, table, max_pages, page, kc,
                          ks, vc, vs, rows, scale, out, lse, ws, ws_bytes, None)


def test_tree_refusals():
    assert L.tq_attn_tree(None, P, 1, 1024, 3, 5, 8, 2, P, P, P, P, 9, 16, P, P, P, P, 4096, 0.1, P, P, P, 0, None) == E
    for variant in (_lib.TQ_MSE, _lib.TQ_PROD, _lib.TQ_POLAR):
        assert tree(variant=variant) == E
    assert tree(dtype=_lib.TQ_F32) == U
    assert tree(B=-1) == E and tree(n=-1) == E and tree(Hq=-8) == E and tree(Hkv=0) == E and tree(Hq=9) == E
    assert tree(n=_lib.TQ_MAX_DRAFT + 1) == U and tree(B=_lib.TQ_MAX_SEQS + 1) == U
    assert tree(B=4096, n=256, Hq=64) == U                                # B n Hq rows of the result
    for page in (0, -8, 4, 12):
        assert tree(page=page) == E, page
    assert tree(max_pages=0) == E and tree(max_pages=1 << 28) == E
    assert tree(rows=-1) == E and tree(rows=2 ** 31 - 4096) == U
    for scale in (-0.5, float("inf"), float("nan")):
        assert tree(scale=scale) == E
    assert tree(qs=1016) == E and tree(qs=1028) == E and tree(qs=-1024) == E
    for name in ("q", "ctx", "table", "kc", "ks", "vc", "vs", "out"):
        assert tree(**{name: None}) == E, name
    for name in ("q", "ctx", "drafts", "mask", "table", "kc", "ks", "vc", "vs", "out", "lse", "ws"):
        assert tree(**{name: Q}) == A, name
    for nothing in (dict(B=0), dict(n=0), dict(Hq=0)):
        assert tree(q=None, **nothing) == _lib.TQ_OK


def test_binding_refuses_tensors_of_another_device_than_the_handle():
    class On:                                                             # where a tensor is: all that this check looks at
        def __init__(self, i):
            self.device = f"cuda:{i}"
            self.get_device = lambda: i

    h = tq.api.Handle(0, 128, 8, tq.TQ_KV8)
    h.device = 0
    api._same_device(h, On(0), None, On(0))
    for tensors in ((On(1), On(1)), (On(0), On(1)), (On(0), None, On(-1)), (On(-1),)):
        with pytest.raises(ValueError):
            api._same_device(h, *tensors)
    with pytest.raises(TypeError):
        api._same_device(h, None)
