"""What the failure-path checks of attention over all keys refuse, on a machine without a GPU."""
import ctypes

import pytest

from block_sparse_top_fvattn_b200 import _lib
from test_around_abi import CAPACITY, INVALID, P, UNSUPPORTED, dense


def both(lib, s, status=P, step=0, polls=4, n=1 << 40):
    sp = ctypes.byref(s)
    return (lib.fvattn_dense_attn_timeout_check(P, P, P, sp, None, P, None, P, P, n, status, step, polls, None),
            lib.fvattn_dense_attn_bwd_timeout_check(P, P, P, P, P, None, P, sp, None, P, P, P, P, n, status, step, polls,
                                                    None))


@pytest.mark.parametrize("shape,kw,code", [
    ({}, dict(polls=0), INVALID), ({}, dict(status=None), INVALID), (dict(dtype=1), {}, UNSUPPORTED),
    (dict(Sk=0), {}, INVALID), (dict(d=96), {}, UNSUPPORTED)])
def test_timeout_checks_reject_on_the_host(lib, shape, kw, code):
    assert both(lib, dense(**shape), **kw) == (code, code)


def test_timeout_checks_need_the_workspace(lib):
    assert both(lib, dense(Sq=40, Sk=100000), n=0) == (CAPACITY, CAPACITY)
