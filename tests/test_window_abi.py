"""Refusals of the windowed calls, on the CPU: a bad argument is refused with
its code before anything is queued, and the cache is left as it was."""
import ctypes

import pytest

from bit_quantized_evicted_b200 import minikv as mk
from tests.test_abi import _bound_cache

P = 1 << 24


@pytest.mark.parametrize("window,n_sink,code", [(0, 0, mk.ERR_INVALID_ARG), (-1, 4, mk.ERR_INVALID_ARG),
                                                (4, -1, mk.ERR_INVALID_ARG)])
def test_window_decode_refusals(window, n_sink, code):
    L, c = mk.lib(), _bound_cache()
    assert L.minikv_decode_attn_window(ctypes.byref(c), P, P, P, 2, window, n_sink, 0.1, P, P, 1 << 20, None) == code
    assert b"window" in L.minikv_last_error_string()
    assert (c.n_packed, c.n_res, c.res_start) == (0, 0, 0)


def test_window_decode_refuses_what_decode_attn_refuses():
    L, c = mk.lib(), _bound_cache()
    call = lambda q=P, Hq=2, out=P, ws=P: L.minikv_decode_attn_window(  # noqa: E731
        ctypes.byref(c), q, P, P, Hq, 8, 2, 0.1, out, ws, 1 << 20, None)
    assert call(Hq=3) == mk.ERR_INVALID_ARG
    assert call(Hq=10) == mk.ERR_UNSUPPORTED
    assert call(q=P + 2) == mk.ERR_INVALID_ARG
    assert call(out=None) == mk.ERR_INVALID_ARG
    assert call(ws=None) == mk.ERR_INVALID_ARG
    assert call(ws=P + 8) == mk.ERR_INVALID_ARG
    c.n_packed, c.n_res = c.cap, c.R + c.G - 1
    assert call() == mk.ERR_CAPACITY
    assert (c.n_packed, c.n_res) == (c.cap, c.R + c.G - 1)
