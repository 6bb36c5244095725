"""The windowed and shared-prefix operators as a server uses them: a prompt, its
packing, then decode steps; layers of both kinds one after another without a
wait between them; two streams at once; captured.

Prompt outputs: the tolerance of the window prefill's own tests.  Decode steps:
that of the shared-prefix step's tests for sharing rows, 2^-11 |o| + 4e-4 max |v|
otherwise (the sequence's own tokens, 2e-4 max |v|, twice for the two partial
states of a split unit and their merge).
"""
import ctypes
import math

import pytest
import torch

from bit_quantized_evicted_b200 import minikv as mk
from bit_quantized_evicted_b200 import synth
from bit_quantized_evicted_b200.build import WAIT_PROBE_LIB
from tests.plain64 import attend, cache_rows, window_seen
from tests.test_gpu_prefix import _batch, _expected, _inputs, _prefix
from tests.test_gpu_prefix import _check as _check_prefix
from tests.test_gpu_window_prefill import _check as _check_prompt
from tests.test_gpu_window_prefill import _qkv

pytestmark = pytest.mark.gpu

TAU = 1.0 / math.sqrt(128.0)
DEV = "cuda"


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


def _window_ref(cache, q, kn, vn, window, n_sink):
    """Before the step: the output in float64 and its tolerance."""
    B, Hq = q.shape[:2]
    g = Hq // cache.Hkv
    out, tol = (torch.empty((B, Hq, 128), dtype=torch.float64) for _ in range(2))
    for b in range(B):
        for h in range(cache.Hkv):
            k, v = cache_rows(cache, b, h)
            k, v = torch.cat([k, kn[b, h:h + 1].double().cpu()]), torch.cat([v, vn[b, h:h + 1].double().cpu()])
            rows = slice(h * g, (h + 1) * g)
            out[b, rows] = attend(q[b, rows].double().cpu(), k, v, TAU, window_seen(len(k), window, n_sink))
            tol[b, rows] = 2 ** -11 * out[b, rows].abs() + 4e-4 * v.abs().max()
    return out, tol


def _check_step(got, ref):
    out, tol = ref
    err = (got.double().cpu() - out).abs()
    assert torch.isfinite(got).all()
    assert (err <= tol).all(), (float((err / tol).max()), int((err / tol).argmax()))


@pytest.mark.parametrize("mode", ["uniform", "ragged", "device"])
def test_windowed_prompt_then_steps(mode):
    """A windowed layer: the prompt's attention, its packing, and steps across two flushes."""
    T, Hq, Hkv, window, n_sink = 421, 8, 2, 100, 4
    q, k, v = _qkv(2, Hq, Hkv, T, T, seed=910)
    cache = mk.MiniKVCache(2, Hkv, 640, G=32, R=32, Hq=Hq)
    o = mk.window_prefill(q, k, v, window, n_sink)
    if mode == "uniform":
        mk.quant_pack(cache, k, v)
    else:
        cache.set_ragged() if mode == "ragged" else cache.set_device_state()
        for b in range(2):
            mk.quant_pack_seq(cache, b, k[b], v[b])
    _check_prompt(o, q, k, v, window, n_sink)
    for step in range(70):
        x = _inputs(2, Hq, Hkv, step, seed=911)
        ref = _window_ref(cache, *x, window, n_sink) if step % 9 == 0 else None
        got = mk.decode_attn_window(cache, *x, window, n_sink)
        if ref:
            _check_step(got, ref)


def test_prompt_in_chunks_is_the_prompt():
    """Chunks of odd lengths against everything before them: each row's block order is the whole prompt's up to
    where its tile begins, so the results agree to the rounding of P and O (twice the tolerance)."""
    T, window, n_sink = 700, 190, 5
    q, k, v = _qkv(1, 6, 2, T, T, seed=912)
    parts, a = [], 0
    for n in (1, 130, 127, 257, 185):
        parts.append(mk.window_prefill(q[:, :, a:a + n].contiguous(), k[:, :, :a + n].contiguous(),
                                       v[:, :, :a + n].contiguous(), window, n_sink))
        a += n
    assert a == T
    _check_prompt(torch.cat(parts, 2), q, k, v, window, n_sink)


def _layers(B, Hq, Hkv, T):
    """The caches of a layer behind a shared prefix and of a windowed layer, loaded from prompts."""
    shared = _batch([60] * B, Hq, Hkv, "device", steps=80, seed=920)
    local = _batch([200] * B, Hq, Hkv, "device", steps=80, seed=930)
    return shared, local, _prefix(Hkv, T, seed=940)


def test_layers_of_both_kinds_captured_and_replayed(deterministic):
    """A step of two layers, queued without a wait in between, eager and as a replayed graph: the same bits, and
    the plain form's values."""
    B, Hq, Hkv, T = 6, 8, 2, 1500
    flags = [1, 1, 0, 1, 0, 1]
    runs = []
    for captured in (False, True):
        shared, local, prefix = _layers(B, Hq, Hkv, T)
        x = [t.clone() for t in _inputs(B, Hq, Hkv, 0, seed=950)]
        o1, o2 = torch.empty_like(x[0]), torch.empty_like(x[0])
        ws = torch.zeros(mk.workspace_size(mk.OP_DECODE_ATTN_PREFIX, B, Hq, Hkv, shared.cap + 64), dtype=torch.uint8,
                         device=DEV)

        def step():
            mk.decode_attn_prefix(shared, prefix, *x, shared=flags, out=o1, ws=ws)
            mk.decode_attn_window(local, o1, x[1], x[2], 70, 4, out=o2)   # the next layer's queries

        if captured:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        got = []
        for i in range(40):
            for dst, src in zip(x, _inputs(B, Hq, Hkv, i, seed=950)):
                dst.copy_(src)
            if not captured and i % 13 == 0:
                ref1 = _expected(shared, prefix, flags, *x)
                step()
                _check_prefix(o1, ref1)
            else:
                graph.replay() if captured else step()
            got.append((o1.clone(), o2.clone()))
        runs.append(got)
        assert mk.decode_attn_prefix_status(ws, B, Hq, Hkv) == 0
    for i, (a, b) in enumerate(zip(*runs)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), i


def test_two_streams_at_once(deterministic):
    """Steps and prompts on two streams, each with its own workspaces and caches, mixed."""
    B, Hq, Hkv = 20, 8, 2
    prefix = _prefix(Hkv, 6000)
    q, k, v = _qkv(1, 8, 2, 1500, 1500, seed=960)
    ref_o = mk.window_prefill(q, k, v, 300, 4)
    x = _inputs(B, Hq, Hkv, 0, seed=961)
    ref = mk.decode_attn_prefix(_batch([100] * B, Hq, Hkv, "uniform"), prefix, *x)
    streams = [torch.cuda.Stream() for _ in range(2)]
    caches = [[_batch([100] * B, Hq, Hkv, "uniform") for _ in range(6)] for _ in streams]
    torch.cuda.synchronize()
    outs = []
    for i in range(6):
        for s, c in zip(streams, caches):
            outs.append((mk.decode_attn_prefix(c[i], prefix, *x, stream=s), ref))
            outs.append((mk.window_prefill(q, k, v, 300, 4, stream=s), ref_o))
    torch.cuda.synchronize()
    for i, (got, want) in enumerate(outs):
        assert torch.equal(got, want), i


def test_default_workspace_belongs_to_the_calls_stream():
    """The workspace of a call queued on another stream is not handed out again before the call has run."""
    q, k, v = _qkv(1, 2, 1, 256, 256, seed=970)
    mk.window_prefill(q, k, v, 50, 2)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    o = torch.zeros_like(q)
    mk.window_prefill(q, k, v, 50, 2, o=o, stream=side)
    mine = [torch.full((256,), 7, dtype=torch.uint8, device=DEV) for _ in range(64)]
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in mine)
    _check_prompt(o, q, k, v, 50, 2)


def test_first_captured_call_needs_a_workspace():
    cache, prefix = _batch([50], 4, 2, "device"), _prefix(2, 100)
    x = _inputs(1, 4, 2, 0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one = x[0] + 1
        with pytest.raises(RuntimeError, match="before the capture"):
            mk.decode_attn_prefix(cache, prefix, *x)
    graph.replay()
    assert torch.equal(one, x[0] + 1)
    mk.decode_attn_prefix(cache, prefix, *x)


def test_status_is_of_the_last_call():
    """A short prefix after a long one whose waits gave up: fewer CTAs report, and none of the old words is seen."""
    probe = ctypes.CDLL(WAIT_PROBE_LIB)
    for name, (res, args) in mk._SIGS.items():
        f = getattr(probe, name)
        f.restype, f.argtypes = res, args
    cache, long_, short = _batch([100] * 4, 8, 2, "uniform"), _prefix(2, 20000), _prefix(2, 40)
    x = _inputs(4, 8, 2, 0)
    ws = torch.zeros(mk.workspace_size(mk.OP_DECODE_ATTN_PREFIX, 4, 8, 2, cache.cap + 64), dtype=torch.uint8, device=DEV)
    mk.decode_attn_prefix(cache, long_, *x, ws=ws, library=probe)
    assert mk.decode_attn_prefix_status(ws, 4, 8, 2) == 1
    ref = _expected(cache, short, None, *x)
    _check_prefix(mk.decode_attn_prefix(cache, short, *x, ws=ws), ref)
    assert mk.decode_attn_prefix_status(ws, 4, 8, 2) == 0


def test_more_sequences_than_a_flag_table_holds():
    """A uniform batch above the ragged limit: three tiles of 128 rows, the last in part empty."""
    B, Hq, Hkv = 300, 1, 1
    cache, prefix = _batch([40] * 1, Hq, Hkv, "uniform"), _prefix(Hkv, 333)
    k, v = (synth.normal_fp16((B, Hkv, 40, 128), synth.seed_of(980, i, synth.T_K), DEV) for i in range(2))
    cache = mk.MiniKVCache(B, Hkv, 64, G=32, R=32, Hq=Hq)
    mk.quant_pack(cache, k, v)
    x = _inputs(B, Hq, Hkv, 0, seed=981)
    ref = _expected(cache, prefix, None, *x)
    _check_prefix(mk.decode_attn_prefix(cache, prefix, *x), ref)


def test_output_in_the_queries_place():
    q, k, v = _qkv(2, 6, 2, 300, 500, seed=990)
    ref = mk.window_prefill(q, k, v, 100, 3)
    mk.window_prefill(q, k, v, 100, 3, o=q)
    assert torch.equal(q, ref)


def test_a_prompt_and_steps_without_a_wait():
    """Prompt, packing and steps queued back to back: each reads what the one before wrote."""
    T, Hq, Hkv = 1111, 8, 2
    q, k, v = _qkv(1, Hq, Hkv, T, T, seed=991)
    p, batch = mk.MiniKVCache(1, Hkv, 1280, G=32, R=32, Hq=Hq), _batch([70] * 3, Hq, Hkv, "ragged")
    x = _inputs(3, Hq, Hkv, 0, seed=992)
    mk.decode_attn_prefix(batch, p, *x)   # (makes the workspace)
    torch.cuda.synchronize()
    o = mk.window_prefill(q, k, v, T, 0)   # the shared text: causal over all of it
    mk.quant_pack(p, k, v)
    got = [mk.decode_attn_prefix(batch, p, *_inputs(3, Hq, Hkv, 1 + i, seed=992)) for i in range(3)]
    again = _batch([70] * 3, Hq, Hkv, "ragged")
    mk.decode_attn(again, *x)
    for i in range(3):
        y = _inputs(3, Hq, Hkv, 1 + i, seed=992)
        _check_prefix(got[i], _expected(again, p, None, *y))
        mk.decode_attn(again, *y)
    _check_prompt(o, q, k, v, T, 0)


@pytest.mark.parametrize("mode", ["uniform", "device"])
def test_large_values(mode):
    """Values up to fp16's limit and scores that grow along the cache: nothing overflows on the way."""
    B, Hq, Hkv, n = 2, 8, 2, 3000
    gen = torch.Generator(device=DEV).manual_seed(995)

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    def load(n, B, cap):
        c = mk.MiniKVCache(B, Hkv, cap, G=32, R=32, Hq=Hq)
        k = (rand(B, Hkv, n, 128) * torch.linspace(0.2, 2, n, device=DEV)[:, None]).half()
        v = (rand(B, Hkv, n, 128) * 15000).clamp(-65504, 65504).half()
        if mode == "device" and B > 1:
            c.set_device_state()
            for b in range(B):
                mk.quant_pack_seq(c, b, k[b], v[b])
        else:
            mk.quant_pack(c, k, v)
        return c, k, v

    x = rand(B, Hq, 128).half(), rand(B, Hkv, 128).half(), rand(B, Hkv, 128).half()
    cache, k, v = load(n, B, n + 8)
    ref = _window_ref(cache, *x, 2500, 4)
    _check_step(mk.decode_attn_window(cache, *x, 2500, 4), ref)
    cache, prefix = load(n, B, n + 8)[0], load(1500, 1, 1600)[0]
    ref = _expected(cache, prefix, None, *x)
    _check_prefix(mk.decode_attn_prefix(cache, prefix, *x), ref)
    q = rand(B, Hq, n, 128).half()
    _check_prompt(mk.window_prefill(q, k, v, 500, 4), q, k, v, 500, 4)


@pytest.mark.parametrize("n,shared", [(0, None), (300, [0, 0, 0])])
def test_nobody_attends_to_the_prefix_captured(n, shared, deterministic):
    """An empty prefix, or one that no sequence shares: steps queued without a wait, eager and replayed, are
    decode_attn's."""
    cache, other = (_batch([100, 40, 300], 8, 2, "device", steps=40) for _ in range(2))
    prefix = _prefix(2, n) if n else mk.MiniKVCache(1, 2, 64, R=32)
    x = [t.clone() for t in _inputs(3, 8, 2, 0, seed=996)]
    out = torch.empty_like(x[0])
    mk.decode_attn_prefix(cache, prefix, *x, shared=shared, out=out)
    mk.decode_attn(other, *x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mk.decode_attn_prefix(cache, prefix, *x, shared=shared, out=out)
        mk.decode_attn_prefix(cache, prefix, out, x[1], x[2], shared=shared, out=out)
    for i in range(20):
        for dst, src in zip(x, _inputs(3, 8, 2, i, seed=996)):
            dst.copy_(src)
        graph.replay()
        ref = mk.decode_attn(other, mk.decode_attn(other, *x), x[1], x[2])
        assert torch.equal(out, ref), i
    assert [cache.seq_state(b) for b in range(3)] == [other.seq_state(b) for b in range(3)]
