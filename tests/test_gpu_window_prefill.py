"""minikv_window_prefill on the GPU against a plain 64-bit form.

Tolerance of an output value o = sum p v / sum p: half an fp16 step of o
(2^-11 |o|); P rounded to fp16 before the product, half a step of each p, so
2^-11 sum p |v| / sum p, and 2^-25 a key where p is below fp16's normal range
(against a sum of at least 1), so n 2^-25 max |v| for n visible keys; scores from
fp32 sums of 128 products in 8 steps of magnitude up to 300, 300 * 8 * 2^-23 *
2^-3.5 = 2.5e-5 in a score, 5e-5 sum p |v| / sum p in o (numerator and sum).
"""
import math

import pytest
import torch

from bit_quantized_evicted_b200 import minikv as mk
from bit_quantized_evicted_b200 import synth
from bit_quantized_evicted_b200.build import WAIT_PROBE_LIB
from tests.plain64 import attend

pytestmark = pytest.mark.gpu

TAU = 1.0 / math.sqrt(128.0)
DEV = "cuda"


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mk.lib()


def _qkv(B, Hq, Hkv, Tq, Tk, seed=900):
    return (synth.normal_fp16((B, Hq, Tq, 128), synth.seed_of(seed, Tk, synth.T_Q), DEV),
            synth.keys_fp16((B, Hkv, Tk, 128), synth.seed_of(seed, Tk, synth.T_K), DEV),
            synth.normal_fp16((B, Hkv, Tk, 128), synth.seed_of(seed, Tk, synth.T_V), DEV))


def _seen(Tq, Tk, window, n_sink, device=DEV):
    p = torch.arange(Tk - Tq, Tk, device=device)[:, None]
    j = torch.arange(Tk, device=device)[None]
    return (j <= p) & ((p - j < window) | (j < n_sink))


def _check(o, q, k, v, window, n_sink, rows=None):
    B, Hq, Tq, _ = q.shape
    g, Tk = Hq // k.shape[1], k.shape[2]
    seen = _seen(Tq, Tk, window, n_sink)
    rows = slice(None) if rows is None else rows
    for b in range(B):
        for h in range(Hq):
            kk, vv = k[b, h // g].double(), v[b, h // g].double()
            ref = attend(q[b, h, rows], kk, vv, TAU, seen[rows])
            mean = attend(q[b, h, rows], kk, vv.abs(), TAU, seen[rows])
            n = seen[rows].sum(-1, keepdim=True).double()
            tol = 2 ** -11 * ref.abs() + (2 ** -11 + 5e-5) * mean + n * 2 ** -25 * vv.abs().max() + 2 ** -25
            err = (o[b, h, rows].double() - ref).abs()
            assert torch.isfinite(o[b, h, rows]).all(), (b, h)
            assert (err <= tol).all(), (b, h, float((err - tol).max()), int((err - tol).argmax()) // 128)


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (7, 3), (128, 0), (129, 4), (300, 128), (511, 130),
                                           (2 ** 31 - 1, 0), (3, 2 ** 31 - 1)])
@pytest.mark.parametrize("B,Hq,Hkv,Tq,Tk", [(1, 1, 1, 1, 1), (1, 2, 1, 1, 700), (2, 3, 1, 129, 129), (1, 4, 2, 128, 500),
                                            (1, 7, 1, 300, 1001), (3, 2, 2, 257, 640), (1, 8, 1, 1100, 1100)])
def test_window_prefill(B, Hq, Hkv, Tq, Tk, window, n_sink):
    q, k, v = _qkv(B, Hq, Hkv, Tq, Tk)
    ws = torch.full((mk.workspace_size(mk.OP_WINDOW_PREFILL, B, Hq, Hkv, Tq),), 255, dtype=torch.uint8, device=DEV)
    o = mk.window_prefill(q, k, v, window, n_sink, ws=ws)
    _check(o, q, k, v, window, n_sink)
    assert mk.window_prefill_status(ws, B, Hq, Hkv, Tq) == 0


def test_window_prefill_long():
    """A long prompt (rows of every part of it), in whole and as its last chunk."""
    q, k, v = _qkv(1, 4, 1, 9001, 9001)
    o = mk.window_prefill(q, k, v, 2000, 21)
    rows = torch.tensor([0, 1, 127, 128, 1999, 2000, 2020, 2021, 2022, 2176, 5003, 8959, 8960, 9000], device=DEV)
    _check(o, q, k, v, 2000, 21, rows)
    part = mk.window_prefill(q[:, :, 7700:].contiguous(), k, v, 2000, 21)
    _check(part, q[:, :, 7700:], k, v, 2000, 21, torch.tensor([0, 5, 300, 1300], device=DEV))


def test_window_over_everything_is_causal():
    """window = Tk: the result of select_prefill, to the tolerance of both."""
    q, k, v = _qkv(1, 8, 2, 1000, 1000)
    o, _ = mk.select_prefill(q, k, v, 32)
    torch.testing.assert_close(mk.window_prefill(q, k, v, 1000).float(), o.float(), rtol=2 ** -9, atol=2e-3)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -65504.0])
@pytest.mark.parametrize("Hq,Hkv,Tq,Tk,window,n_sink", [(2, 2, 400, 400, 100, 5), (4, 1, 200, 700, 60, 0), (3, 1, 300, 300, 300, 0)])
def test_hidden_keys_may_hold_anything(bad, Hq, Hkv, Tq, Tk, window, n_sink):
    """A row's hidden keys and values may be NaN, infinite or the type's largest: poison from a position on (a padded
    batch) and before the band, and look at the rows that see none of it."""
    q, k, v = _qkv(1, Hq, Hkv, Tq, Tk)
    end = Tk - 77                       # keys from here on belong to nobody's text
    gone = max(n_sink, Tk - Tq - window - 30)   # [n_sink, gone): before the band of every row
    k2, v2 = k.clone(), v.clone()
    k2[:, :, end:], v2[:, :, end:] = bad, bad
    k2[:, :, n_sink:gone], v2[:, :, n_sink:gone] = bad, bad
    one = gone + 50                     # a single bad key inside the band: rows past it by `window` see it no more
    k2[:, :, one], v2[:, :, one] = bad, bad
    o = mk.window_prefill(q, k2, v2, window, n_sink)
    p = torch.arange(Tk - Tq, Tk, device=DEV)
    rows = torch.nonzero((p < end) & ((p < one) | (p - one >= window)))[:, 0]
    assert len(rows) >= 50              # rows before the single bad key
    _check(o, q, k, v, window, n_sink, rows)
    if bad != bad:
        sees = torch.nonzero((p < end) & (p >= one) & (p - one < window))[:, 0]
        assert torch.isnan(o[:, :, sees].float()).all()


def test_masks_of_the_lowest_value_and_large_scores():
    """Scores up to the fp16 products' limit: the softmax is one key's value, not NaN."""
    q, k, v = _qkv(1, 2, 1, 300, 300)
    q, k = (q.float() * 2000).half(), (k.float() * 500).clamp(-60000, 60000).half()
    _check(mk.window_prefill(q, k, v, 90, 4), q, k, v, 90, 4)


def test_window_prefill_captured_and_on_another_stream():
    q, k, v = _qkv(1, 4, 2, 333, 600)
    ref = mk.window_prefill(q, k, v, 200, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(_on(side, q, k, v), ref)
    o, ws = torch.zeros_like(q), torch.empty(mk.workspace_size(mk.OP_WINDOW_PREFILL, 1, 4, 2, 333), dtype=torch.uint8,
                                             device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mk.window_prefill(q, k, v, 200, 4, o=o, ws=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, ref)


def _on(stream, q, k, v):
    o = mk.window_prefill(q, k, v, 200, 4, stream=stream)
    stream.synchronize()
    return o


def test_rows_outside_the_call_are_left_alone():
    """Output planes lie side by side: a tile that ends past Tq writes nothing of the next plane's rows."""
    q, k, v = _qkv(2, 2, 1, 130, 200)
    pool = torch.full((3, 2, 130, 128), 7.0, dtype=torch.float16, device=DEV)
    mk.window_prefill(q[:1].contiguous(), k[:1].contiguous(), v[:1].contiguous(), 50, 2, o=pool[1:2])
    assert (pool[0] == 7).all() and (pool[2] == 7).all()
    _check(pool[1:2], q[:1], k[:1], v[:1], 50, 2)


def test_expired_waits_are_reported():
    """A build whose waits give up at once: the call returns, its status is set, and the context goes on."""
    import ctypes
    probe = ctypes.CDLL(WAIT_PROBE_LIB)
    for name, (res, args) in mk._SIGS.items():
        f = getattr(probe, name)
        f.restype, f.argtypes = res, args
    q, k, v = _qkv(1, 4, 2, 1000, 1000)
    ws = torch.zeros(mk.workspace_size(mk.OP_WINDOW_PREFILL, 1, 4, 2, 1000), dtype=torch.uint8, device=DEV)
    mk.window_prefill(q, k, v, 300, 4, ws=ws, library=probe)
    assert mk.window_prefill_status(ws, 1, 4, 2, 1000, library=probe) == 1
    o = mk.window_prefill(q, k, v, 300, 4, ws=ws)
    assert mk.window_prefill_status(ws, 1, 4, 2, 1000) == 0
    _check(o, q, k, v, 300, 4, torch.arange(0, 1000, 37, device=DEV))


def test_nan_stays_with_the_rows_that_see_it():
    """A NaN query row spoils itself alone; a value that is not finite the rows that see its key, in its channel."""
    T, window, n_sink, row, key, ch = 700, 150, 3, 300, 400, 17
    q, k, v = _qkv(1, 4, 2, T, T, seed=901)
    clean, q0, v0 = mk.window_prefill(q, k, v, window, n_sink), q.clone(), v.clone()
    q[0, 1, row] = float("nan")
    v[0, 1, key, ch] = float("inf")
    o = mk.window_prefill(q, k, v, window, n_sink)
    assert torch.isnan(o[0, 1, row]).all()
    o[0, 1, row] = clean[0, 1, row]
    assert torch.equal(o[0, :2], clean[0, :2])
    seen = _seen(T, T, window, n_sink)[:, key]
    assert not torch.isfinite(o[0, 2:, seen, ch]).any()
    o[0, 2:, seen, ch] = clean[0, 2:, seen, ch]
    _check(o, q0, k, v0, window, n_sink)   # (rows that share a block with the value are computed again)


@pytest.mark.parametrize("window,n_sink", [(70, 3), (2000, 0), (129, 200)])
def test_rows_beside_padding_of_nan(window, n_sink):
    """Prompts padded behind their ends with NaN: the rows before the padding, some beside it in a block, are right."""
    T, end = 900, 777
    q, k, v = _qkv(1, 6, 2, T, T, seed=902)
    k0, v0 = k.clone(), v.clone()
    for t in (k, v, q):
        t[:, :, end:] = float("nan")
    o = mk.window_prefill(q, k, v, window, n_sink)
    q[:, :, end:] = 0
    _check(o, q, k0, v0, window, n_sink, rows=slice(0, end))


@pytest.mark.parametrize("n_sink", [15, 16, 31, 32, 33, 127, 128, 129])
@pytest.mark.parametrize("Hq,Hkv,Tq,Tk,window", [(2, 1, 600, 600, 64), (3, 1, 140, 1000, 200)])
def test_sizes_of_the_sink_block(Hq, Hkv, Tq, Tk, window, n_sink):
    """Sinks that take part of a block, a whole one or more; the rest of the block may hold anything."""
    q, k, v = _qkv(1, Hq, Hkv, Tq, Tk, seed=903)
    o = mk.window_prefill(q, k, v, window, n_sink)
    _check(o, q, k, v, window, n_sink)
    first = max(0, n_sink + window + 1 - (Tk - Tq))   # rows from here on see nothing between the sinks and n_sink + 1
    k[:, :, n_sink:n_sink + 1] = float("nan")
    v[:, :, n_sink:n_sink + 1] = float("nan")
    bad = mk.window_prefill(q, k, v, window, n_sink)
    k[:, :, n_sink:n_sink + 1] = 0
    v[:, :, n_sink:n_sink + 1] = 0
    _check(bad, q, k, v, window, n_sink, rows=slice(first, Tq))
