"""CPU: arguments that the header says are ignored, and ranges that it gives, of the cache in 4 bits.  (Every call here is
refused on the host before any launch; which refusal it is says what was looked at.)"""
import pytest

from test_prompt_abi import attn_args as chunk_args
from test_q4_abi import ODD, S, append_args, attn_args, norm_args  # noqa: F401  (S: fixture)


@pytest.mark.parametrize("eps", [-1.0, float("nan"), float("inf")])
def test_append_without_weights_ignores_eps(S, eps):  # noqa: F811
    for kw in (dict(Q=None, Qrot=None), dict()):
        kw = dict(kw, wq=None, wk=None, M=(1 << 22) + 1)
        assert append_args(S, eps=eps, **kw) == append_args(S, **kw) == S.SPEC_EUNSUPPORTED
        assert b"rows" in S._lib.spec_last_error()
    assert append_args(S, eps=eps) == append_args(S, Q=None, Qrot=None, wq=None, eps=eps) == S.SPEC_EINVAL
    assert S._lib.spec_launches() == 0


def test_norm_without_queries_or_keys_ignores_theirs(S):  # noqa: F811
    """Refused for what comes after the ignored pointers' place in the checks: the other side's leading dimension, eps."""
    for kw, said in ((dict(Hq=0, Q=ODD, Qout=ODD, wq=ODD, ldq=-3, ldk=248), b"ldk"), (dict(Hq=0, wq=ODD, Q=None, eps=-1.0), b"eps"),
                     (dict(Hkv=0, K=ODD, Kout=ODD, wk=ODD, ldk=-3, ldq=1016), b"ldq"), (dict(Hkv=0, wk=ODD, K=None, eps=-1.0), b"eps")):
        assert norm_args(S, **kw) == S.SPEC_EINVAL and said in S._lib.spec_last_error(), kw
    assert S._lib.spec_launches() == 0


@pytest.mark.parametrize("most", [3, 1000])
def test_attention_scale_range(S, most):  # noqa: F811
    """The kernels' factor, scale * log2(e) * 2^19, has to be a float (2^128 / (2^19 log2(e)) is 4.5e32): beyond, the scale is
    refused; up to it, it is not (the call is refused for its workspace)."""
    for scale, said in ((0.0, b"workspace"), (4e32, b"workspace"), (4.6e32, b"scale"), (3.4e38, b"scale")):
        assert attn_args(S, max_rows=most, scale=scale, ws_bytes=16) == S.SPEC_EINVAL
        assert said in S._lib.spec_last_error(), scale
    assert S._lib.spec_launches() == 0


def test_chunk_attention_scale_range(S):  # noqa: F811
    """Over bf16 pages the factor is scale * log2(e)."""
    for scale, said in ((2e38, b"workspace"), (3e38, b"scale")):
        assert chunk_args(S, scale=scale, ws_bytes=16) == S.SPEC_EINVAL
        assert said in S._lib.spec_last_error(), scale
    assert S._lib.spec_launches() == 0
