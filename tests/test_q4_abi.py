"""CPU checks of the entry points of the cache in 4 bits: bad arguments are refused on the host before any launch."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def S():
    from speculative_decoding_verify_05_gb300.build import build
    build()
    from speculative_decoding_verify_05_gb300 import binding
    return binding


FAKE, OTHER, ODD = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 21), ctypes.c_void_p((1 << 20) + 8)


def norm_args(S, **kw):
    a = dict(Q=FAKE, ldq=1024, Qout=OTHER, ldqo=1024, K=FAKE, ldk=256, Kout=OTHER, ldko=256, wq=FAKE, wk=FAKE, eps=1e-6,
             cs=FAKE, M=5, Hq=8, Hkv=2, D=128)
    a.update(kw)
    return S._lib.spec_qk_norm_rope(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), "SPEC_EINVAL"), (dict(Hq=-1), "SPEC_EINVAL"), (dict(Hkv=-1), "SPEC_EINVAL"), (dict(D=64), "SPEC_EUNSUPPORTED"),
    (dict(Q=None), "SPEC_EINVAL"), (dict(Qout=None), "SPEC_EINVAL"), (dict(K=None), "SPEC_EINVAL"),
    (dict(Kout=None), "SPEC_EINVAL"), (dict(wq=None), "SPEC_EINVAL"), (dict(wk=None), "SPEC_EINVAL"),
    (dict(Q=ODD), "SPEC_EINVAL"), (dict(Qout=ODD), "SPEC_EINVAL"), (dict(K=ODD), "SPEC_EINVAL"), (dict(Kout=ODD), "SPEC_EINVAL"),
    (dict(wq=ODD), "SPEC_EINVAL"), (dict(wk=ODD), "SPEC_EINVAL"), (dict(cs=ODD), "SPEC_EINVAL"),
    (dict(ldq=1016), "SPEC_EINVAL"), (dict(ldqo=1028), "SPEC_EINVAL"), (dict(ldk=248), "SPEC_EINVAL"),
    (dict(ldko=260), "SPEC_EINVAL"), (dict(Qout=FAKE, ldqo=1032), "SPEC_EINVAL"), (dict(Kout=FAKE, ldko=264), "SPEC_EINVAL"),
    (dict(eps=-1.0), "SPEC_EINVAL"), (dict(eps=float("nan")), "SPEC_EINVAL"), (dict(eps=float("inf")), "SPEC_EINVAL"),
])
def test_norm_refusals(S, kw, code):
    assert norm_args(S, **kw) == getattr(S, code)
    assert S._lib.spec_last_error() and S._lib.spec_launches() == 0


def append_args(S, **kw):
    a = dict(Q=FAKE, ldq=1024, Qrot=FAKE, ldqr=1024, K=FAKE, V=FAKE, ldkv=256, wq=FAKE, wk=FAKE, eps=1e-6, cs=FAKE, cu=FAKE,
             ctx=FAKE, B=2, M=5, Kp=FAKE, Vp=FAKE, num_pages=4, table=FAKE, max_pages=2, Hq=8, Hkv=2, D=128)
    a.update(kw)
    return S._lib.spec_kv_append_paged_q4(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), "SPEC_EINVAL"), (dict(M=-1), "SPEC_EINVAL"), (dict(D=64), "SPEC_EUNSUPPORTED"),
    (dict(K=None), "SPEC_EINVAL"), (dict(V=None), "SPEC_EINVAL"), (dict(V=ODD), "SPEC_EINVAL"),
    (dict(cu=None), "SPEC_EINVAL"), (dict(ctx=None), "SPEC_EINVAL"), (dict(table=None), "SPEC_EINVAL"),
    (dict(Kp=None), "SPEC_EINVAL"), (dict(Vp=ODD), "SPEC_EINVAL"), (dict(num_pages=0), "SPEC_EINVAL"),
    (dict(max_pages=0), "SPEC_EINVAL"), (dict(max_pages=1 << 24), "SPEC_EINVAL"), (dict(Hkv=0), "SPEC_EINVAL"),
    (dict(ldkv=248), "SPEC_EINVAL"), (dict(ldkv=260), "SPEC_EINVAL"), (dict(ldq=1016), "SPEC_EINVAL"),
    (dict(ldqr=1028), "SPEC_EINVAL"), (dict(ldqr=1032), "SPEC_EINVAL"), (dict(Hq=0), "SPEC_EINVAL"),
    (dict(cs=None, wq=None, wk=None), "SPEC_EINVAL"), (dict(cs=ODD), "SPEC_EINVAL"), (dict(Q=ODD), "SPEC_EINVAL"),
    (dict(Q=None), "SPEC_EINVAL"), (dict(Q=None, Qrot=None), "SPEC_EINVAL"), (dict(Qrot=None), "SPEC_EINVAL"),
    (dict(wq=None), "SPEC_EINVAL"), (dict(wk=None), "SPEC_EINVAL"), (dict(wk=ODD), "SPEC_EINVAL"),
    (dict(eps=-1.0), "SPEC_EINVAL"), (dict(eps=float("nan")), "SPEC_EINVAL"), (dict(M=(1 << 22) + 1), "SPEC_EUNSUPPORTED"),
    (dict(B=1 << 29), "SPEC_EUNSUPPORTED"),
])
def test_append_refusals(S, kw, code):
    assert append_args(S, **kw) == getattr(S, code)
    assert S._lib.spec_last_error() and S._lib.spec_launches() == 0


def read_args(S, **kw):
    a = dict(Kp=FAKE, Vp=FAKE, num_pages=4, table=FAKE, max_pages=2, cu=FAKE, ctx=FAKE, B=2, M=5, K=FAKE, V=FAKE, ldkv=256,
             Hkv=2, D=128)
    a.update(kw)
    return S._lib.spec_kv_read_paged_q4(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), "SPEC_EINVAL"), (dict(M=-1), "SPEC_EINVAL"), (dict(D=64), "SPEC_EUNSUPPORTED"),
    (dict(K=None), "SPEC_EINVAL"), (dict(V=None), "SPEC_EINVAL"), (dict(K=ODD), "SPEC_EINVAL"), (dict(V=ODD), "SPEC_EINVAL"),
    (dict(cu=None), "SPEC_EINVAL"), (dict(ctx=None), "SPEC_EINVAL"), (dict(table=None), "SPEC_EINVAL"),
    (dict(Kp=ODD), "SPEC_EINVAL"), (dict(Vp=None), "SPEC_EINVAL"), (dict(num_pages=0), "SPEC_EINVAL"),
    (dict(max_pages=0), "SPEC_EINVAL"), (dict(max_pages=1 << 24), "SPEC_EINVAL"), (dict(Hkv=0), "SPEC_EINVAL"),
    (dict(ldkv=248), "SPEC_EINVAL"), (dict(ldkv=260), "SPEC_EINVAL"), (dict(B=1 << 29), "SPEC_EUNSUPPORTED"),
    (dict(num_pages=1 << 30), "SPEC_EINVAL"),
])
def test_read_refusals(S, kw, code):
    assert read_args(S, **kw) == getattr(S, code)
    assert S._lib.spec_last_error() and S._lib.spec_launches() == 0


def test_empty_calls_are_no_ops(S):
    assert norm_args(S, M=0, Q=None) == 0 and norm_args(S, Hq=0, Hkv=0, Q=None, K=None) == 0
    assert append_args(S, B=0, K=None) == 0 and append_args(S, M=0, K=None) == 0
    assert read_args(S, B=0, K=None) == 0 and read_args(S, M=0, K=None) == 0
    assert S._lib.spec_launches() == 0


def test_binding_refuses_before_the_library(S):
    """Types, shapes and strides, on the CPU: nothing here is a CUDA tensor, and that is what is said first."""
    bf, u8, i32 = torch.bfloat16, torch.uint8, torch.int32
    cu, ctx, table = torch.zeros(2, dtype=i32), torch.zeros(1, dtype=i32), torch.zeros((1, 1), dtype=i32)
    pool = torch.zeros((1, 1, S.Q4_PAGE_BYTES), dtype=u8)
    k = torch.zeros((1, 128), dtype=bf)
    for call in (lambda: S.spec_kv_append_paged_q4(k, k, cu, ctx, pool, pool, table),
                 lambda: S.spec_kv_read_paged_q4(cu, ctx, pool, pool, table, 1),
                 lambda: S.spec_qk_norm_rope(k, k, k[0], k[0])):
        with pytest.raises(TypeError):
            call()
    assert S.q4_pool(3, 5, "cpu").shape == (3, 5, 8704) and S.Q4_PAGE_BYTES == 8704


def attn_args(S, **kw):
    a = dict(Q=FAKE, ldq=1024, cu=FAKE, ctx=FAKE, B=2, M=5, max_rows=3, Kp=FAKE, Vp=FAKE, num_pages=4, table=FAKE, max_pages=2,
             Hq=8, Hkv=2, D=128, scale=0.1, O=FAKE, ldo=1024, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return S._lib.spec_chunk_attention_paged_q4(*a.values(), None)


@pytest.mark.parametrize("most", [3, 1000])
@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), "SPEC_EINVAL"), (dict(M=-1), "SPEC_EINVAL"), (dict(D=64), "SPEC_EUNSUPPORTED"),
    (dict(Q=None), "SPEC_EINVAL"), (dict(O=None), "SPEC_EINVAL"), (dict(Q=ODD), "SPEC_EINVAL"),
    (dict(O=ODD), "SPEC_EINVAL"), (dict(cu=None), "SPEC_EINVAL"), (dict(ctx=None), "SPEC_EINVAL"),
    (dict(table=None), "SPEC_EINVAL"), (dict(Kp=ODD), "SPEC_EINVAL"), (dict(Vp=None), "SPEC_EINVAL"),
    (dict(num_pages=0), "SPEC_EINVAL"), (dict(max_pages=0), "SPEC_EINVAL"), (dict(Hq=7), "SPEC_EINVAL"),
    (dict(Hq=0), "SPEC_EINVAL"), (dict(Hq=258), "SPEC_EUNSUPPORTED"), (dict(ldq=1016), "SPEC_EINVAL"),
    (dict(ldo=1028), "SPEC_EINVAL"), (dict(scale=float("nan")), "SPEC_EINVAL"), (dict(scale=float("inf")), "SPEC_EINVAL"),
    (dict(scale=-0.1), "SPEC_EINVAL"), (dict(ws_bytes=16), "SPEC_EINVAL"), (dict(ws=None, ws_bytes=0), "SPEC_EINVAL"),
    (dict(ws=ODD), "SPEC_EINVAL"), (dict(M=(1 << 22) + 1), "SPEC_EUNSUPPORTED"),
])
def test_attention_refusals(S, kw, code, most):
    assert attn_args(S, **{"max_rows": most, **kw}) == getattr(S, code)
    assert S._lib.spec_last_error() and S._lib.spec_launches() == 0


def test_attention_workspace(S):
    assert attn_args(S, max_rows=0) == attn_args(S, max_rows=-1) == S.SPEC_EINVAL
    for most in (1, 16, 17, 5000):
        n = S.spec_chunk_attention_q4_workspace_bytes(8, 5000, most, 32, 8, 128, 64)
        assert n > 64 * 1024
        assert attn_args(S, max_rows=most, M=5000, Hq=32, Hkv=8, ldq=4096, ldo=4096, ws_bytes=n - 1) == S.SPEC_EINVAL
        assert b"workspace" in S._lib.spec_last_error()
    assert S.spec_chunk_attention_q4_workspace_bytes(8, 1000, 0, 32, 8, 128, 64) == 0
    assert attn_args(S, B=0, Q=None) == 0 and attn_args(S, M=0, Q=None) == 0 and S._lib.spec_launches() == 0
