"""CPU checks of the prompt-side entry points: bad arguments are refused on the host before any launch."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def S():
    from speculative_decoding_verify_05_gb300.build import build
    build()
    from speculative_decoding_verify_05_gb300 import binding
    return binding


FAKE, ODD = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 8)


def table_args(S, **kw):
    a = dict(pos=FAKE, ldpos=4, axes=3, M=4, D=128, theta=1e6, sections=[16, 24, 24], interleaved=0, cs=FAKE)
    a.update(kw)
    sec = a["sections"]
    a["sections"] = None if sec is None else (ctypes.c_int32 * len(sec))(*sec)
    return S._lib.spec_rope_table_axes(*a.values(), None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(axes=0), "SPEC_EUNSUPPORTED", b"axes"), (dict(axes=9), "SPEC_EUNSUPPORTED", b"axes"),
    (dict(D=127), "SPEC_EUNSUPPORTED", b"even"), (dict(D=258), "SPEC_EUNSUPPORTED", b"256"),
    (dict(theta=0.0), "SPEC_EINVAL", b"theta"), (dict(theta=float("inf")), "SPEC_EINVAL", b"theta"),
    (dict(theta=float("nan")), "SPEC_EINVAL", b"theta"), (dict(sections=None), "SPEC_EINVAL", b"sections"),
    (dict(sections=[16, 24, 23]), "SPEC_EINVAL", b"sum to 63"), (dict(sections=[70, -3, -3]), "SPEC_EINVAL", b"< 0"),
    (dict(sections=[16, 24, 24], interleaved=1), "SPEC_EINVAL", b"past"), (dict(interleaved=2), "SPEC_EINVAL", b"0 or 1"),
    (dict(ldpos=3), "SPEC_EINVAL", b"ldpos"), (dict(pos=None), "SPEC_EINVAL", b"NULL"),
    (dict(cs=None), "SPEC_EINVAL", b"NULL"), (dict(M=-1), "SPEC_EINVAL", b"M="),
])
def test_table_refusals(S, kw, code, word):
    assert table_args(S, **kw) == getattr(S, code)
    assert word in S._lib.spec_last_error() and S._lib.spec_launches() == 0


def test_empty_calls_are_no_ops(S):
    assert table_args(S, M=0, pos=None, cs=None) == 0
    assert append_args(S, B=0, K=None) == 0 and append_args(S, M=0, K=None) == 0
    assert attn_args(S, B=0, Q=None) == 0 and attn_args(S, M=0, Q=None) == 0
    assert S._lib.spec_launches() == 0


def append_args(S, **kw):
    a = dict(Q=FAKE, ldq=1024, Qrot=FAKE, ldqr=1024, K=FAKE, V=FAKE, ldkv=256, cs=FAKE, cu=FAKE, ctx=FAKE, B=2, M=5,
             Kp=FAKE, Vp=FAKE, num_pages=4, table=FAKE, max_pages=2, Hq=8, Hkv=2, D=128)
    a.update(kw)
    return S._lib.spec_kv_append_paged(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), "SPEC_EINVAL"), (dict(M=-1), "SPEC_EINVAL"), (dict(D=64), "SPEC_EUNSUPPORTED"),
    (dict(K=None), "SPEC_EINVAL"), (dict(V=None), "SPEC_EINVAL"), (dict(V=ODD), "SPEC_EINVAL"),
    (dict(cu=None), "SPEC_EINVAL"), (dict(ctx=None), "SPEC_EINVAL"), (dict(table=None), "SPEC_EINVAL"),
    (dict(Kp=None), "SPEC_EINVAL"), (dict(Vp=ODD), "SPEC_EINVAL"), (dict(num_pages=0), "SPEC_EINVAL"),
    (dict(max_pages=0), "SPEC_EINVAL"), (dict(max_pages=1 << 24), "SPEC_EINVAL"), (dict(Hkv=0), "SPEC_EINVAL"),
    (dict(ldkv=248), "SPEC_EINVAL"), (dict(ldkv=260), "SPEC_EINVAL"), (dict(ldq=1016), "SPEC_EINVAL"),
    (dict(ldqr=1028), "SPEC_EINVAL"), (dict(ldqr=1032), "SPEC_EINVAL"), (dict(Hq=0), "SPEC_EINVAL"),
    (dict(cs=None), "SPEC_EINVAL"), (dict(cs=ODD), "SPEC_EINVAL"), (dict(Q=ODD), "SPEC_EINVAL"),
    (dict(Q=None), "SPEC_EINVAL"), (dict(Qrot=None), "SPEC_EINVAL"),
])
def test_append_refusals(S, kw, code):
    assert append_args(S, **kw) == getattr(S, code)
    assert S._lib.spec_last_error() and S._lib.spec_launches() == 0


def attn_args(S, **kw):
    a = dict(Q=FAKE, ldq=1024, cu=FAKE, ctx=FAKE, B=2, M=5, Kp=FAKE, Vp=FAKE, num_pages=4, table=FAKE, max_pages=2,
             Hq=8, Hkv=2, D=128, scale=0.1, O=FAKE, ldo=1024, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return S._lib.spec_chunk_attention_paged(*a.values(), None)


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
def test_attention_refusals(S, kw, code):
    assert attn_args(S, **kw) == getattr(S, code)
    assert S._lib.spec_last_error() and S._lib.spec_launches() == 0


def test_workspace_query_is_host_only(S):
    n = S.spec_chunk_attention_workspace_bytes(8, 1000, 32, 8, 128, 64)
    assert n > 64 * 1024
    # a batch with more rows or sequences never needs less
    assert S.spec_chunk_attention_workspace_bytes(9, 1000, 32, 8, 128, 64) >= n
    assert S.spec_chunk_attention_workspace_bytes(8, 2000, 32, 8, 128, 64) >= n
    assert S.spec_chunk_attention_workspace_bytes(0, 1000, 32, 8, 128, 64) == 0


def test_workspace_follows_the_grid(S):
    """The attention's workspace is that of its CTAs (two slots of 256 rows each, fp32 outputs, references and sums) behind the
    counters, whatever the batch; one that was sized for fewer CTAs is refused."""
    size = lambda: S.spec_chunk_attention_workspace_bytes(2, 5, 8, 2, 128, 2)
    of = lambda ctas: 64 * 1024 + ctas * 2 * 256 * (128 * 4 + 16)
    try:
        for ctas in (1, 37, 600):
            S.spec_set_option("persistent_grid", ctas)
            assert size() == of(ctas) == S.spec_chunk_attention_workspace_bytes(900, 100000, 40, 8, 128, 64)
            assert attn_args(S, ws_bytes=of(ctas) - 1) == S.SPEC_EINVAL
            assert b"workspace" in S._lib.spec_last_error()
        S.spec_set_option("persistent_grid", 4096)
        assert size() == of(1024)                        # (the most CTAs that the counters have room for)
    finally:
        S.spec_set_option("persistent_grid", 0)
    assert size() > 64 * 1024
