"""minikv_decode_attn_window on the GPU against a plain 64-bit form: the newest
`window` tokens and the first `n_sink` of each sequence.

Tolerance of an output value: half an fp16 step of it (2^-11 relative), plus
2e-4 of the largest |v|.  The second part: a packed score is a sum of 128
products of a code (at most 3) and a 16-bit hi / lo pair whose lo part is off by
at most 2^-25 before the code's factor 2^8, so at most 128 * 3 * 2^-17 * scale =
2.6e-4 if all agreed in sign, 2.3e-5 at the 1 sigma of independent ones (four
times that is allowed: 1e-4 relative in a probability); the value side rounds p * scale
the same way, 3 * 2^-25 a token against a sum of probabilities of at least 1,
1e-4 for 1100 tokens of one sign.
"""
import math

import pytest
import torch

from bit_quantized_evicted_b200 import minikv as mk
from bit_quantized_evicted_b200 import synth
from tests.plain64 import attend, cache_rows, window_seen

pytestmark = pytest.mark.gpu

TAU = 1.0 / math.sqrt(128.0)
DEV = "cuda"
MODES = ["uniform", "ragged", "device"]


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mk.lib()


@pytest.fixture
def deterministic():
    mk.set_deterministic(True)
    try:
        yield
    finally:
        mk.set_deterministic(False)


def _load(lengths, Hq, Hkv, G, R, mode, steps=4, seed=300):
    cap = (max(lengths) // G + steps // G + 2) * G
    cache = mk.MiniKVCache(len(lengths), Hkv, cap, G=G, R=R, Hq=Hq)
    if mode == "ragged":
        cache.set_ragged()
    elif mode == "device":
        cache.set_device_state()
    k = [synth.keys_fp16((Hkv, n, 128), synth.seed_of(seed, b, synth.T_K), DEV) for b, n in enumerate(lengths)]
    v = [synth.normal_fp16((Hkv, n, 128), synth.seed_of(seed, b, synth.T_V), DEV) for b, n in enumerate(lengths)]
    if mode == "uniform":
        mk.quant_pack(cache, torch.stack(k), torch.stack(v))
    else:
        for b in range(len(lengths)):
            mk.quant_pack_seq(cache, b, k[b], v[b])
    return cache


def _inputs(B, Hq, Hkv, step, seed=301):
    return (synth.normal_fp16((B, Hq, 128), synth.seed_of(seed, 0, synth.T_QDEC, step), DEV),
            synth.keys_fp16((B, Hkv, 128), synth.seed_of(seed, 0, synth.T_KNEW, step), DEV),
            synth.normal_fp16((B, Hkv, 128), synth.seed_of(seed, 0, synth.T_VNEW, step), DEV))


def _expected(cache, q, kn, vn, window, n_sink):
    """Before the step: [B, Hq, 128] in float64, and the largest |v|."""
    B, Hq = q.shape[:2]
    g = Hq // cache.Hkv
    out, top = torch.empty((B, Hq, 128), dtype=torch.float64), 0.0
    for b in range(B):
        for h in range(cache.Hkv):
            k, v = cache_rows(cache, b, h)
            k, v = torch.cat([k, kn[b, h:h + 1].double().cpu()]), torch.cat([v, vn[b, h:h + 1].double().cpu()])
            top = max(top, float(v.abs().max()))
            out[b, h * g:(h + 1) * g] = attend(q[b, h * g:(h + 1) * g].cpu(), k, v, TAU,
                                               window_seen(len(k), window, n_sink))
    return out, top


def _check(got, ref, top):
    err = (got.double().cpu() - ref).abs() - ref.abs() * 2 ** -11
    assert torch.isfinite(got).all()
    assert float(err.max()) <= 2e-4 * top, float(err.max())


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (5, 3), (33, 0), (64, 32), (100, 45), (257, 4), (2000, 0),
                                           (2 ** 31 - 1, 2 ** 31 - 1), (40, 900)])
@pytest.mark.parametrize("n,Hq,Hkv,G,R", [(700, 8, 2, 32, 32), (451, 3, 1, 64, 64), (130, 4, 4, 32, 128),
                                          (600, 2, 1, 128, 0), (0, 2, 1, 32, 32)])
def test_window_decode(n, Hq, Hkv, G, R, window, n_sink, mode):
    cache = _load([n, n], Hq, Hkv, G, R, mode)
    for step in range(2):
        q, kn, vn = _inputs(2, Hq, Hkv, step)
        ref, top = _expected(cache, q, kn, vn, window, n_sink)
        _check(mk.decode_attn_window(cache, q, kn, vn, window, n_sink), ref, top)


@pytest.mark.parametrize("mode", ["ragged", "device"])
def test_window_decode_ragged_across_flushes(mode):
    """Unequal sequences, among them empty ones and one shorter than the window, over two flushes; the cache ends
    as decode_attn leaves it."""
    lengths, Hq, Hkv, G, R = (0, 1, 95, 1500, 333, 64), 4, 2, 32, 32
    cache, other = (_load(lengths, Hq, Hkv, G, R, mode, steps=70) for _ in range(2))
    for step in range(70):
        q, kn, vn = _inputs(len(lengths), Hq, Hkv, step)
        if step % 9 == 0:
            ref, top = _expected(cache, q, kn, vn, 120, 7)
            _check(mk.decode_attn_window(cache, q, kn, vn, 120, 7), ref, top)
        else:
            mk.decode_attn_window(cache, q, kn, vn, 120, 7)
        mk.decode_attn(other, q, kn, vn)
    for b in range(len(lengths)):
        assert cache.seq_state(b) == other.seq_state(b)
    a, c = cache.arrays(), other.arrays()
    for name in a:
        assert torch.equal(a[name], c[name]), name
    assert cache.status() == [0] * len(lengths)


@pytest.mark.parametrize("mode", MODES)
def test_window_over_everything_is_decode_attn(mode, deterministic):
    cache, other = (_load([777, 777, 777], 8, 2, 32, 64, mode) for _ in range(2))
    q, kn, vn = _inputs(3, 8, 2, 0)
    top = max(float(cache_rows(cache, b, h)[1].abs().max()) for b in range(3) for h in range(2))
    top = max(top, float(vn.abs().max()))
    got, other_got = mk.decode_attn_window(cache, q, kn, vn, 778), mk.decode_attn(other, q, kn, vn)
    # each within the tolerance above of the exact value
    tol = 2 ** -10 * other_got.double().abs() + 4e-4 * top
    assert ((got.double() - other_got.double()).abs() <= tol).all()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 65504.0])
def test_hidden_tokens_may_hold_anything(mode, bad, deterministic):
    """NaN, infinities and the largest value in hidden tokens: the same bits as without them."""
    n, window, n_sink, G, R = 900, 70, 20, 32, 32
    for length, sink in ((n, n_sink), (60, 45)):   # the second: no packed token, the sinks inside the residual
        outs = []
        for poison in (False, True):
            cache = _load([length], 4, 2, G, R, mode)
            nq, r, start = cache.seq_state(0)
            w = window if length == n else 5
            if poison:
                a = cache.arrays()
                lo = length + 1 - w
                end = min(lo, nq)
                if end > sink:
                    a["v_scale"][:, :, sink:end] = bad
                    a["v_zero"][:, :, sink:end] = bad
                    a["k_scale"][:, :, -(-sink // G):end // G] = bad
                    a["k_zero"][:, :, -(-sink // G):end // G] = bad
                for i in range(r):
                    if sink <= nq + i < lo:
                        a["k_res"][:, :, (start + i) % (R + G)] = bad
                        a["v_res"][:, :, (start + i) % (R + G)] = bad
            q, kn, vn = _inputs(1, 4, 2, 0)
            outs.append(mk.decode_attn_window(cache, q, kn, vn, w, sink))
        assert torch.isfinite(outs[0]).all() and torch.equal(outs[0], outs[1])


def test_window_decode_captured_and_replayed():
    """Device state: one captured step, replayed across a flush, against eager steps of another cache."""
    lengths, Hq, Hkv = (300, 40, 1000), 8, 2
    cache, other = (_load(lengths, Hq, Hkv, 32, 32, "device", steps=40) for _ in range(2))
    q, kn, vn = _inputs(3, Hq, Hkv, 0)
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        mk.decode_attn_window(cache, q, kn, vn, 90, 6, out=out)
    for step in range(36):
        for dst, src in zip((q, kn, vn), _inputs(3, Hq, Hkv, step)):
            dst.copy_(src)
        graph.replay()
        ref = mk.decode_attn_window(other, q, kn, vn, 90, 6)
        torch.testing.assert_close(out.float(), ref.float(), rtol=2 ** -10, atol=5e-4)
    assert [cache.seq_state(b) for b in range(3)] == [other.seq_state(b) for b in range(3)]
    a, c = cache.arrays(), other.arrays()
    for name in a:
        assert torch.equal(a[name], c[name]), name


def test_window_decode_on_another_stream():
    cache = _load([500, 500], 8, 2, 32, 32, "uniform")
    q, kn, vn = _inputs(2, 8, 2, 0)
    ref, top = _expected(cache, q, kn, vn, 77, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = mk.decode_attn_window(cache, q, kn, vn, 77, 5, stream=side)
    side.synchronize()
    _check(out, ref, top)
