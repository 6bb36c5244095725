"""minikv_decode_attn_prefix on the GPU against a plain 64-bit form: every
sharing sequence attends to the prefix cache's tokens and its own.

Tolerance of an output value o = sum p v / sum p: half an fp16 step of o
(2^-11 |o|), and for the prefix's tokens what fp16 operands of the two products
would cost (the kernel's own key and value operands are exact, only P is
rounded, so it has room to spare):
  * P and the dequantized value each rounded once, half a step each: 2^-10 mean,
    mean = sum p |v| / sum p; 2^-25 max |v| a token below fp16's normal range
    (against a sum of at least 1);
  * the dequantized key rounded once: each of the 128 products q k^ is off by at
    most 2^-11 of itself, so a score by e = 2^-11 scale sum |q k^|, o by 2 e mean.
    The worst row's e is used (about 5 times what independent roundings give).
The sequence's own tokens: as for the decode kernel, 2e-4 max |v|.
"""
import math

import pytest
import torch

from bit_quantized_evicted_b200 import minikv as mk
from bit_quantized_evicted_b200 import synth
from bit_quantized_evicted_b200.build import WAIT_PROBE_LIB
from tests.plain64 import attend, cache_rows

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


def _kv(Hkv, n, seed):
    return (synth.keys_fp16((Hkv, n, 128), synth.seed_of(seed, n, synth.T_K), DEV),
            synth.normal_fp16((Hkv, n, 128), synth.seed_of(seed, n, synth.T_V), DEV))


def _prefix(Hkv, n, G=32, R=32, seed=500, rotate=0):
    """A prefix cache of n tokens; its ring starts `rotate` slots in (as after decode steps)."""
    p = mk.MiniKVCache(1, Hkv, (n // G + 1) * G, G=G, R=R)
    k, v = _kv(Hkv, n, seed)
    mk.quant_pack(p, k[None], v[None])
    if rotate:
        a = p.arrays()
        for name in ("k_res", "v_res"):
            a[name].copy_(torch.roll(a[name], rotate, 2))
        p.c.res_start = rotate
    return p


def _batch(lengths, Hq, Hkv, mode, G=32, R=32, steps=2, seed=600):
    cache = mk.MiniKVCache(len(lengths), Hkv, (max(lengths) // G + steps // G + 2) * G, G=G, R=R, Hq=Hq)
    kv = [_kv(Hkv, n, seed + b) for b, n in enumerate(lengths)]
    if mode == "uniform":
        mk.quant_pack(cache, torch.stack([k for k, _ in kv]), torch.stack([v for _, v in kv]))
        return cache
    cache.set_ragged() if mode == "ragged" else cache.set_device_state()
    for b, (k, v) in enumerate(kv):
        mk.quant_pack_seq(cache, b, k, v)
    return cache


def _inputs(B, Hq, Hkv, step, seed=601):
    return (synth.normal_fp16((B, Hq, 128), synth.seed_of(seed, 0, synth.T_QDEC, step), DEV),
            synth.keys_fp16((B, Hkv, 128), synth.seed_of(seed, 0, synth.T_KNEW, step), DEV),
            synth.normal_fp16((B, Hkv, 128), synth.seed_of(seed, 0, synth.T_VNEW, step), DEV))


def _expected(cache, prefix, shared, q, kn, vn):
    """Before the step: the output in float64 and its tolerance."""
    B, Hq = q.shape[:2]
    g = Hq // cache.Hkv
    out, tol = (torch.empty((B, Hq, 128), dtype=torch.float64) for _ in range(2))
    for h in range(cache.Hkv):
        pk, pv = cache_rows(prefix, 0, h)
        for b in range(B):
            rows = slice(h * g, (h + 1) * g)
            k, v = cache_rows(cache, b, h)
            k, v = torch.cat([k, kn[b, h:h + 1].double().cpu()]), torch.cat([v, vn[b, h:h + 1].double().cpu()])
            qq = q[b, rows].double().cpu()
            if shared is None or shared[b]:
                k, v = torch.cat([pk, k]), torch.cat([pv, v])
                e = 2 ** -11 * TAU * float((qq.abs() @ pk.abs().T).max()) if len(pk) else 0.0
                low = 2 ** -25 * len(pk)
            else:
                e, low = 0.0, 0.0
            out[b, rows] = attend(qq, k, v, TAU)
            mean = attend(qq, k, v.abs(), TAU) if e else 0.0
            tol[b, rows] = 2 ** -11 * out[b, rows].abs() + (2 ** -10 + 2 * e) * mean + (low + 2e-4) * v.abs().max()
    return out, tol


def _check(got, ref):
    out, tol = ref
    err = (got.double().cpu() - out).abs()
    assert torch.isfinite(got).all()
    assert (err <= tol).all(), (float((err / tol).max()), int((err / tol).argmax()))


@pytest.mark.parametrize("mode", ["uniform", "ragged", "device"])
@pytest.mark.parametrize("B,Hq,Hkv", [(1, 1, 1), (2, 8, 2), (5, 3, 1), (8, 4, 4), (9, 8, 2), (17, 4, 1), (33, 4, 2)])
@pytest.mark.parametrize("n,G,R,rotate", [(1, 32, 32, 0), (31, 32, 0, 0), (129, 32, 32, 5), (160, 64, 64, 0),
                                          (700, 128, 128, 77), (3001, 32, 128, 159)])
def test_prefix_decode(B, Hq, Hkv, n, G, R, rotate, mode):
    cache, prefix = _batch([90] * B, Hq, Hkv, mode), _prefix(Hkv, n, G, R, rotate=rotate)
    before = {k: v.clone() for k, v in prefix.arrays().items()}
    ws = torch.zeros(mk.workspace_size(mk.OP_DECODE_ATTN_PREFIX, B, Hq, Hkv, cache.cap + 64), dtype=torch.uint8, device=DEV)
    for step in range(2):
        q, kn, vn = _inputs(B, Hq, Hkv, step)
        ref = _expected(cache, prefix, None, q, kn, vn)
        _check(mk.decode_attn_prefix(cache, prefix, q, kn, vn, ws=ws), ref)
    assert mk.decode_attn_prefix_status(ws, B, Hq, Hkv) == 0
    for name, t in prefix.arrays().items():
        assert torch.equal(t, before[name]), name


@pytest.mark.parametrize("mode", ["ragged", "device"])
@pytest.mark.parametrize("shared", [(1, 0, 1, 1, 0, 1), (0, 0, 0, 0, 0, 1), (0, 0, 0, 0, 0, 0), None])
def test_some_sequences_share(shared, mode):
    """Unequal sequences (one empty), some of which do not share; across a flush, the cache ends as decode_attn's."""
    lengths, Hq, Hkv = (0, 300, 33, 1000, 64, 5), 8, 2
    cache, other = (_batch(lengths, Hq, Hkv, mode, steps=40) for _ in range(2))
    prefix = _prefix(Hkv, 515)
    for step in range(40):
        q, kn, vn = _inputs(6, Hq, Hkv, step)
        if step % 13 == 0:
            ref = _expected(cache, prefix, shared, q, kn, vn)
            _check(mk.decode_attn_prefix(cache, prefix, q, kn, vn, shared), ref)
        else:
            mk.decode_attn_prefix(cache, prefix, q, kn, vn, shared)
        mk.decode_attn(other, q, kn, vn)
    a, c = cache.arrays(), other.arrays()
    for name in a:
        assert torch.equal(a[name], c[name]), name
    assert [cache.seq_state(b) for b in range(6)] == [other.seq_state(b) for b in range(6)]


def test_empty_prefix_is_decode_attn(deterministic):
    cache, other = (_batch([300] * 3, 8, 2, "uniform") for _ in range(2))
    q, kn, vn = _inputs(3, 8, 2, 0)
    empty = mk.MiniKVCache(1, 2, 64, R=32)
    assert torch.equal(mk.decode_attn_prefix(cache, empty, q, kn, vn), mk.decode_attn(other, q, kn, vn))


def test_rows_that_do_not_share_meet_nothing_of_the_prefix(deterministic):
    """A prefix of NaN and infinities: the sequences without it come out as decode_attn's, bit for bit; those with it
    are NaN."""
    cache, other = (_batch((100, 200, 300, 50), 4, 2, "ragged") for _ in range(2))
    prefix = _prefix(2, 400)
    a = prefix.arrays()
    a["k_scale"][:, :, 2] = float("nan")
    a["v_zero"][:, :, 77] = float("inf")
    q, kn, vn = _inputs(4, 4, 2, 0)
    out = mk.decode_attn_prefix(cache, prefix, q, kn, vn, (0, 1, 0, 1))
    ref = mk.decode_attn(other, q, kn, vn)
    assert torch.equal(out[[0, 2]], ref[[0, 2]])
    assert torch.isnan(out[[1, 3]].float()).all()


def test_what_lies_behind_the_prefix_is_not_seen(deterministic):
    """Garbage in the prefix cache behind its tokens (capacity, ring) changes no bit."""
    outs = []
    for poison in (False, True):
        cache, prefix = _batch([40] * 6, 8, 2, "uniform"), _prefix(2, 401)
        if poison:
            a, n, r = prefix.arrays(), prefix.n_packed, prefix.n_res
            for name in ("k_codes", "v_codes"):
                a[name][:, :, n:] = -1
            for name in ("v_scale", "v_zero"):
                a[name][:, :, n:] = float("nan")
            for name in ("k_scale", "k_zero"):
                a[name][:, :, n // 32:] = float("inf")
            for name in ("k_res", "v_res"):
                a[name][:, :, r:] = float("nan")
        q, kn, vn = _inputs(6, 8, 2, 0)
        outs.append(mk.decode_attn_prefix(cache, prefix, q, kn, vn))
    assert torch.isfinite(outs[0]).all() and torch.equal(outs[0], outs[1])


def test_growing_scores_move_the_reference():
    """Keys whose scores grow along the prefix, so that every tile moves the running maximum, and a last token that
    takes all the weight."""
    Hkv, n = 1, 1500
    k, v = _kv(Hkv, n, 510)
    k = (k.float() * torch.linspace(0.2, 6.0, n, device=DEV)[:, None]).half()
    prefix = mk.MiniKVCache(1, Hkv, 1536, R=32)
    mk.quant_pack(prefix, k[None], v[None])
    cache = _batch([40] * 6, 4, Hkv, "uniform")
    q, kn, vn = _inputs(6, 4, Hkv, 0)
    ref = _expected(cache, prefix, None, q, kn, vn)
    _check(mk.decode_attn_prefix(cache, prefix, q, kn, vn), ref)


def test_same_inputs_same_bits(deterministic):
    outs = []
    for _ in range(2):
        cache, prefix = _batch([200] * 20, 8, 2, "uniform"), _prefix(2, 5000)
        q, kn, vn = _inputs(20, 8, 2, 0)
        outs.append(mk.decode_attn_prefix(cache, prefix, q, kn, vn))
    assert torch.equal(outs[0], outs[1])


def test_prefix_decode_captured_and_replayed():
    lengths, Hq, Hkv = (300, 40, 1000), 8, 2
    cache, other = (_batch(lengths, Hq, Hkv, "device", steps=40) for _ in range(2))
    prefix = _prefix(Hkv, 1111)
    q, kn, vn = _inputs(3, Hq, Hkv, 0)
    out = torch.empty_like(q)
    ws = torch.zeros(mk.workspace_size(mk.OP_DECODE_ATTN_PREFIX, 3, Hq, Hkv, cache.cap + 64), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mk.decode_attn_prefix(cache, prefix, q, kn, vn, out=out, ws=ws)
    for step in range(36):
        for dst, src in zip((q, kn, vn), _inputs(3, Hq, Hkv, step)):
            dst.copy_(src)
        graph.replay()
        ref = mk.decode_attn_prefix(other, prefix, q, kn, vn)
        torch.testing.assert_close(out.float(), ref.float(), rtol=2 ** -10, atol=5e-4)
    assert [cache.seq_state(b) for b in range(3)] == [other.seq_state(b) for b in range(3)]


def test_expired_waits_are_reported():
    """A build whose waits give up at once: the call returns, its status is set, and the context goes on."""
    import ctypes
    probe = ctypes.CDLL(WAIT_PROBE_LIB)
    for name, (res, args) in mk._SIGS.items():
        f = getattr(probe, name)
        f.restype, f.argtypes = res, args
    cache, prefix = _batch([200] * 20, 8, 2, "uniform"), _prefix(2, 5000)
    q, kn, vn = _inputs(20, 8, 2, 0)
    ws = torch.zeros(mk.workspace_size(mk.OP_DECODE_ATTN_PREFIX, 20, 8, 2, cache.cap + 64), dtype=torch.uint8, device=DEV)
    state = cache.seq_state(0)
    mk.decode_attn_prefix(cache, prefix, q, kn, vn, ws=ws, library=probe)
    assert mk.decode_attn_prefix_status(ws, 20, 8, 2, library=probe) == 1
    cache.c.n_packed, cache.c.n_res, cache.c.res_start = state
    ref = _expected(cache, prefix, None, q, kn, vn)
    _check(mk.decode_attn_prefix(cache, prefix, q, kn, vn, ws=ws), ref)
    assert mk.decode_attn_prefix_status(ws, 20, 8, 2) == 0


@pytest.mark.parametrize("B,Hq,Hkv,n", [(2, 8, 8, 60000), (12, 8, 4, 100001), (32, 16, 4, 100000)])
def test_many_tiles_a_cta(B, Hq, Hkv, n):
    """More than 20 tiles a CTA: every buffer and barrier goes round several times (16, 32 and 128 rows)."""
    cache, prefix = _batch([40] * B, Hq, Hkv, "uniform"), _prefix(Hkv, n, 128, 128)
    q, kn, vn = _inputs(B, Hq, Hkv, 0)
    some = sorted({0, B // 2, B - 1})
    g = Hq // Hkv
    own = {(b, h): cache_rows(cache, b, h) for b in some for h in range(Hkv)}
    out = mk.decode_attn_prefix(cache, prefix, q, kn, vn)
    for h in range(Hkv):
        pk, pv = cache_rows(prefix, 0, h)
        for b in some:
            k, v = (torch.cat([p, o, x[b, h:h + 1].double().cpu()]) for p, o, x in
                    ((pk, own[b, h][0], kn), (pv, own[b, h][1], vn)))
            qq = q[b, h * g:(h + 1) * g].double().cpu()
            ref = attend(qq, k, v, TAU)
            e = 2 ** -11 * TAU * float((qq.abs() @ pk.abs().T).max())
            mean = attend(qq, k, v.abs(), TAU)
            tol = 2 ** -11 * ref.abs() + (2 ** -10 + 2 * e) * mean + (2 ** -25 * n + 2e-4) * v.abs().max()
            _check(out[b, h * g:(h + 1) * g], (ref, tol))
