"""Decode steps over values up to fp16's limit, with scores that grow along the
cache: a probability may be 2^8 under the lazy reference, and its product with a
value scale of 2^8 or more does not fit fp16.  Every call of the decode body; and
sequences that hold NaN beside sound ones.

Tolerance of an output value: half an fp16 step of it (2^-11 relative), plus
4e-4 of the largest |v|: 2e-4 for scores and probabilities (as in the tests of
the windowed step), 2e-4 for the value sums, whose code operands cost up to 1e-4
of sum p (max - min), at most twice the largest |v|.
"""
import math

import pytest
import torch

from bit_quantized_evicted_b200 import minikv as mk
from tests.plain64 import attend, cache_rows

pytestmark = pytest.mark.gpu

TAU = 1.0 / math.sqrt(128.0)
DEV = "cuda"
B, HQ, HKV, N = 2, 8, 2, 3000


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mk.lib()


def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _load(mode, scale, seed=995):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    k = (_rand(gen, B, HKV, N, 128) * torch.linspace(0.2, 2, N, device=DEV)[:, None]).half()
    v = (_rand(gen, B, HKV, N, 128) * scale).clamp(-65504, 65504).half()
    cache = mk.MiniKVCache(B, HKV, N + 8, G=32, R=32, Hq=HQ)
    if mode == "uniform":
        mk.quant_pack(cache, k, v)
    else:
        cache.set_ragged() if mode == "ragged" else cache.set_device_state()
        for b in range(B):
            mk.quant_pack_seq(cache, b, k[b], v[b])
    return cache, (_rand(gen, B, HQ, 128).half(), _rand(gen, B, HKV, 128).half(), _rand(gen, B, HKV, 128).half())


def _check(cache, got, x, before):
    q, kn, vn = x
    g = HQ // HKV
    for (b, h), (k, v) in before.items():
        k, v = torch.cat([k, kn[b, h:h + 1].double().cpu()]), torch.cat([v, vn[b, h:h + 1].double().cpu()])
        ref = attend(q[b, h * g:(h + 1) * g].double().cpu(), k, v, TAU)
        o = got[b, h * g:(h + 1) * g].double().cpu()
        assert torch.isfinite(o).all(), (b, h)
        assert ((o - ref).abs() <= 2 ** -11 * ref.abs() + 4e-4 * v.abs().max()).all(), (b, h)


@pytest.mark.parametrize("mode", ["uniform", "ragged", "device"])
@pytest.mark.parametrize("call", ["decode_attn", "decode_attn_mass", "decode_attn_static", "decode_attn_window"])
@pytest.mark.parametrize("scale", [100.0, 500.0, 15000.0])
def test_large_value_scales(call, mode, scale):
    cache, x = _load(mode, scale)
    before = {(b, h): cache_rows(cache, b, h) for b in range(B) for h in range(HKV)}
    if call == "decode_attn_mass":
        mass = torch.zeros((B, HKV, cache.cap + cache.R + cache.G), dtype=torch.float32, device=DEV)
        ws = torch.zeros(mk.workspace_size(mk.OP_DECODE_ATTN_MASS, B, HQ, HKV, cache.cap + cache.R + cache.G),
                         dtype=torch.uint8, device=DEV)
        got = mk.decode_attn_mass(cache, *x, mass, ws=ws)
        # a token's probabilities over the group's heads add up to the number of heads
        torch.testing.assert_close(mass.double().sum(-1), torch.full((B, HKV), HQ / HKV, dtype=torch.float64, device=DEV),
                                   rtol=1e-3, atol=0)
    elif call == "decode_attn_window":
        got = mk.decode_attn_window(cache, *x, N + 1)
    else:
        got = getattr(mk, call)(cache, *x)
    _check(cache, got, x, before)


@pytest.mark.parametrize("mode", ["uniform", "ragged", "device"])
def test_steps_with_large_values_across_a_flush(mode):
    """The flush packs what it packs after any other step, and the steps after it are right."""
    cache, x = _load(mode, 15000.0)
    other, _ = _load(mode, 15000.0)
    for step in range(40):
        mk.decode_attn(cache, *x)
        mk.decode_attn_window(other, *x, 5)
    for name, t in cache.arrays().items():
        assert torch.equal(t, other.arrays()[name]), name
    assert [cache.seq_state(b) for b in range(B)] == [other.seq_state(b) for b in range(B)]
    before = {(b, h): cache_rows(cache, b, h) for b in range(B) for h in range(HKV)}
    _check(cache, mk.decode_attn(cache, *x), x, before)


@pytest.mark.parametrize("mode", ["uniform", "ragged", "device"])
def test_what_is_not_finite_stays_with_its_sequence(mode):
    """NaN and an infinity in one sequence's values: its outputs in their channels are not finite, all others are sound."""
    cache, x = _load(mode, 1.0)
    before = {(b, h): cache_rows(cache, b, h) for b in range(B) for h in range(HKV)}
    a = cache.arrays()
    a["v_zero"][0, 0, 700] = float("nan")
    a["v_res"][0, 1, 3, 9] = float("inf")
    got = mk.decode_attn(cache, *x).float()
    g = HQ // HKV
    assert torch.isnan(got[0, :g]).all()
    assert not torch.isfinite(got[0, g:, 9]).any()
    got[0, g:, 9] = 0
    q, kn, vn = x
    for (b, h), (k, v) in before.items():
        if (b, h) == (0, 0):
            continue
        k, v = torch.cat([k, kn[b, h:h + 1].double().cpu()]), torch.cat([v, vn[b, h:h + 1].double().cpu()])
        ref = attend(q[b, h * g:(h + 1) * g].double().cpu(), k, v, TAU)
        if b == 0:
            ref[:, 9] = 0
        assert ((got[b, h * g:(h + 1) * g].double().cpu() - ref).abs() <= 2 ** -11 * ref.abs() + 4e-4 * v.abs().max()).all()
