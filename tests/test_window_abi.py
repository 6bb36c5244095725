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


@pytest.mark.parametrize("change,code", [
    (dict(q=None), mk.ERR_INVALID_ARG), (dict(ws=None), mk.ERR_INVALID_ARG), (dict(o=P + 8), mk.ERR_INVALID_ARG),
    (dict(k=P + 2), mk.ERR_INVALID_ARG), (dict(Hq=5), mk.ERR_INVALID_ARG), (dict(B=0), mk.ERR_INVALID_ARG),
    (dict(Tq=0), mk.ERR_INVALID_ARG), (dict(Tq=513), mk.ERR_INVALID_ARG), (dict(D=64), mk.ERR_UNSUPPORTED),
    (dict(window=0), mk.ERR_INVALID_ARG), (dict(n_sink=-1), mk.ERR_INVALID_ARG), (dict(scale=0.0), mk.ERR_INVALID_ARG),
    (dict(scale=float("nan")), mk.ERR_INVALID_ARG), (dict(scale=float("inf")), mk.ERR_INVALID_ARG),
    (dict(B=20000, Hq=4, Hkv=4), mk.ERR_UNSUPPORTED), (dict(Tk=2 ** 31 - 1), mk.ERR_UNSUPPORTED),
    (dict(ws_bytes=4), mk.ERR_INVALID_ARG),
])
def test_window_prefill_refusals(change, code):
    a = dict(q=P, k=P, v=P, B=1, Hq=4, Hkv=2, Tq=512, Tk=512, D=128, window=64, n_sink=4, scale=0.1, o=P, ws=P,
             ws_bytes=1 << 20)
    a.update(change)
    L = mk.lib()
    assert L.minikv_window_prefill(a["q"], a["k"], a["v"], a["B"], a["Hq"], a["Hkv"], a["Tq"], a["Tk"], a["D"],
                                   a["window"], a["n_sink"], a["scale"], a["o"], a["ws"], a["ws_bytes"], None) == code
    assert L.minikv_last_error_string()


def test_window_prefill_workspace_and_status_refusals():
    # a word a query tile: 4 tiles of 128 rows of each head, in 256-byte units
    assert mk.workspace_size(mk.OP_WINDOW_PREFILL, 2, 6, 2, 500) == 256
    assert mk.workspace_size(mk.OP_WINDOW_PREFILL, 4, 32, 8, 4096) == 4 * 32 * 32 * 4
    assert mk.workspace_size(mk.OP_WINDOW_PREFILL, 1, 5, 2, 500) == 0
    L, st = mk.lib(), ctypes.c_uint(0)
    assert L.minikv_window_prefill_status(None, 256, 1, 4, 2, 512, None, ctypes.byref(st)) == mk.ERR_INVALID_ARG
    assert L.minikv_window_prefill_status(P, 256, 1, 4, 2, 512, None, None) == mk.ERR_INVALID_ARG
    assert L.minikv_window_prefill_status(P, 255, 1, 4, 2, 512, None, ctypes.byref(st)) == mk.ERR_INVALID_ARG
    assert L.minikv_window_prefill_status(P, 256, 1, 5, 2, 512, None, ctypes.byref(st)) == mk.ERR_INVALID_ARG
