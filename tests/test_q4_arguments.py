"""CPU: arguments that the header says are ignored, and ranges that it gives, of the cache in 4 bits.  (Every call here is
refused on the host before any launch; which refusal it is says what was looked at.)"""
import pytest

from test_q4_abi import S, append_args  # noqa: F401  (S: fixture)


@pytest.mark.parametrize("eps", [-1.0, float("nan"), float("inf")])
def test_append_without_weights_ignores_eps(S, eps):  # noqa: F811
    for kw in (dict(Q=None, Qrot=None), dict()):
        kw = dict(kw, wq=None, wk=None, M=(1 << 22) + 1)
        assert append_args(S, eps=eps, **kw) == append_args(S, **kw) == S.SPEC_EUNSUPPORTED
        assert b"rows" in S._lib.spec_last_error()
    assert append_args(S, eps=eps) == append_args(S, Q=None, Qrot=None, wq=None, eps=eps) == S.SPEC_EINVAL
    assert S._lib.spec_launches() == 0
