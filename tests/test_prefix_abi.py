"""Refusals of the shared-prefix step, on the CPU."""
import ctypes

import pytest

from bit_quantized_evicted_b200 import minikv as mk
from tests.test_abi import _bound_cache

P = 1 << 24
WS = 1 << 24


def _prefix(**kw):
    c = _bound_cache(**{**dict(B=1, Hkv=2, cap=256), **kw})
    L, n = mk.lib(), mk.lib().minikv_cache_bytes(c.B, c.Hkv, 128, c.G, c.Gv, c.R, c.cap)
    assert L.minikv_cache_bind(ctypes.byref(c), 1 << 28, n, c.B, c.Hkv, 128, c.G, c.Gv, c.R, c.cap) == 0
    return c


def _call(c, p, shared=None, q=P, Hq=4, scale=0.1, out=P, ws=P, ws_bytes=WS):
    return mk.lib().minikv_decode_attn_prefix(ctypes.byref(c), ctypes.byref(p), shared, q, P, P, Hq, scale, out, ws,
                                              ws_bytes, None)


@pytest.mark.parametrize("prefix,code", [(dict(B=2), mk.ERR_INVALID_ARG), (dict(Hkv=1), mk.ERR_INVALID_ARG),
                                         (dict(Gv=32), mk.ERR_UNSUPPORTED)])
def test_prefix_shape_refusals(prefix, code):
    c = _bound_cache()
    assert _call(c, _prefix(**prefix)) == code
    assert b"prefix" in mk.lib().minikv_last_error_string()


def test_prefix_state_refusals():
    c, p = _bound_cache(), _prefix()
    p.dseq = 1 << 20
    assert _call(c, p) == mk.ERR_UNSUPPORTED
    p.dseq = None
    p.n_packed = 17
    assert _call(c, p) == mk.ERR_INVALID_ARG
    assert _call(c, c) == mk.ERR_INVALID_ARG            # the batch's own memory
    assert mk.lib().minikv_decode_attn_prefix(ctypes.byref(c), None, None, P, P, P, 4, 0.1, P, P, WS,
                                              None) == mk.ERR_INVALID_ARG


@pytest.mark.parametrize("change,code", [
    (dict(q=None), mk.ERR_INVALID_ARG), (dict(q=P + 2), mk.ERR_INVALID_ARG), (dict(out=None), mk.ERR_INVALID_ARG),
    (dict(Hq=3), mk.ERR_INVALID_ARG), (dict(Hq=10), mk.ERR_UNSUPPORTED), (dict(scale=0.0), mk.ERR_INVALID_ARG),
    (dict(scale=float("nan")), mk.ERR_INVALID_ARG), (dict(ws=None), mk.ERR_INVALID_ARG),
    (dict(ws=P + 8), mk.ERR_INVALID_ARG), (dict(ws_bytes=1 << 12), mk.ERR_INVALID_ARG),
])
def test_prefix_argument_refusals(change, code):
    c, p = _bound_cache(), _prefix()
    p.n_packed = 64
    assert _call(c, p, **change) == code
    assert (c.n_packed, c.n_res) == (0, 0)


def test_prefix_capacity_and_flag_refusals():
    c, p = _bound_cache(), _prefix()
    c.n_packed, c.n_res = c.cap, c.R + c.G - 1
    assert _call(c, p) == mk.ERR_CAPACITY
    big = _bound_cache(B=mk.MAX_RAGGED_SEQS + 1, cap=64)
    assert _call(big, p, shared=mk.shared_rows([1] * big.B), ws_bytes=1 << 30) == mk.ERR_UNSUPPORTED


def test_prefix_workspace_and_status_refusals():
    size = lambda B, Hq, Hkv: mk.workspace_size(mk.OP_DECODE_ATTN_PREFIX, B, Hq, Hkv, 1000)  # noqa: E731
    assert size(4, 5, 2) == 0 and size(0, 4, 2) == 0
    # 4 rows a KV head: 16-row tiles, 148 + 2 partial states
    assert size(4, 2, 2) >= mk.workspace_size(mk.OP_DECODE_ATTN, 4, 2, 2, 1000) + 150 * 16 * 132 * 4
    L, st = mk.lib(), ctypes.c_uint(0)
    assert L.minikv_decode_attn_prefix_status(None, 1 << 24, 4, 2, 2, None, ctypes.byref(st)) == mk.ERR_INVALID_ARG
    assert L.minikv_decode_attn_prefix_status(P, 1 << 24, 4, 2, 2, None, None) == mk.ERR_INVALID_ARG
    assert L.minikv_decode_attn_prefix_status(P, 1 << 10, 4, 2, 2, None, ctypes.byref(st)) == mk.ERR_INVALID_ARG
    assert L.minikv_decode_attn_prefix_status(P, 1 << 24, 4, 3, 2, None, ctypes.byref(st)) == mk.ERR_INVALID_ARG
