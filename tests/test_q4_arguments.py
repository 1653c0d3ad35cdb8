"""CPU: arguments that the header says are ignored, and ranges that it gives, of the cache in 4 bits.  (Every call here is
refused on the host before any launch; which refusal it is says what was looked at.)"""
import pytest

from test_q4_abi import ODD, S, append_args, norm_args  # noqa: F401  (S: fixture)


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
