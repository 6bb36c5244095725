"""Steps behind a shared prefix in which every tile of 128 tokens counts: a lost,
doubled or stale tile moves outputs far beyond the tolerance, at any length, and
at a few thousand tokens a single lost token does.

Values: 1.5 times a random sign a (tile, channel), the same for a tile's tokens,
which the 2-bit cache holds exactly.  Keys and queries are N(0, 1), so that the
scores are too and no token has much of the weight.  Against the outputs of a
sound step, a tile that is missing among n tokens moves each channel by about
128 / n (1.5 - o); a token 1.5 / n.

Tolerance of an output o = sum p v / sum p, from 64 bits:
  * its own rounding, 2^-11 |o|;
  * P's, independent, each off by at most 2^-11: the sum by 2^-11 / sqrt(3)
    sqrt(sum p^2 (v - o)^2) / sum p at one sigma of the widest spread, seven of
    them (4 2^-11) allowed;
  * sums in fp32: 8 steps a tile and CTA and a few for the merge, each off by at
    most 2^-23 of a running sum, at most max |2 V'| = 2: (8 tiles + 16) 2^-22;
  * scores of 128 products in fp32, off by e = 2^-20 sum |q k| scale: 1.5 e;
  * the own tokens, as in the decode kernel's tests: 2e-4 max |v| of their share
    of the weight.
The mistakes are planted in the plain form, on the CPU: each has to be seen.
"""
import math

import pytest
import torch

from bit_quantized_evicted_b200 import minikv as mk
from tests.plain64 import cache_rows
from tests.test_gpu_prefix import _batch

TAU = 1.0 / math.sqrt(128.0)
DEV = "cuda"
SMS = 148


def _random(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def _tiles(n, n_packed):
    """The prefix pass's tile of each token: the packed ones from 0, the others after them."""
    t = torch.arange(n)
    return torch.where(t < n_packed, t // 128, -(-n_packed // 128) + (t - n_packed) // 128)


def _marked(n, n_packed, seed):
    """Values [n, 128] that mark their tiles."""
    tile = _tiles(n, n_packed)
    return 1.5 * torch.where(_random((int(tile[-1]) + 1, 128), seed) < 0, -1.0, 1.0)[tile]


def _split(n, G, R):
    return 0 if n < R else (n - R) // G * G


def _attend(q, k, v, tiles, own):
    """Outputs and tolerances of rows q [m, 128] over k, v [n, 128] (float64), the last `own` tokens the sequence's."""
    x = (q @ k.T) * TAU
    p = torch.softmax(x, -1)
    o = p @ v
    square = (p ** 2 @ v ** 2) - 2 * o * (p ** 2 @ v) + o ** 2 * (p ** 2).sum(-1, keepdim=True)
    tol = 2 ** -11 * o.abs() + 4 * 2 ** -11 * square.clamp(min=0).sqrt() + (8 * tiles + 16) * 2 ** -22
    tol = tol + 1.5 * 2 ** -20 * TAU * (q.abs() @ k.abs().T).amax(-1, keepdim=True)
    tol = tol + 2e-4 * float(v[-own:].abs().max()) * p[:, -own:].sum(-1, keepdim=True)
    return o, tol


def _case(B, Hq, Hkv, n, G, R, q_scale, seed):
    """Keys, values of the prefix, queries and the new token, float32 on the CPU."""
    packed = _split(n, G, R)
    k = _random((Hkv, n, 128), seed)
    v = torch.stack([_marked(n, packed, seed + 7 * h + 1) for h in range(Hkv)])
    q = _random((B, Hq, 128), seed + 100) * q_scale
    return k, v, q, _random((B, Hkv, 128), seed + 101), _random((B, Hkv, 128), seed + 102)


def _run(B, Hq, Hkv, n, G, R, q_scale, rotate=0, some=None, seed=700):
    k, v, q, kn, vn = _case(B, Hq, Hkv, n, G, R, q_scale, seed)
    prefix = mk.MiniKVCache(1, Hkv, (n // G + 1) * G, G=G, R=R)
    mk.quant_pack(prefix, k[None].half().to(DEV), v[None].half().to(DEV))
    if rotate:
        a = prefix.arrays()
        for name in ("k_res", "v_res"):
            a[name].copy_(torch.roll(a[name], rotate, 2))
        prefix.c.res_start = rotate
    cache = _batch([40] * B, Hq, Hkv, "uniform", seed=seed)
    q, kn, vn = (t.half().to(DEV) for t in (q, kn, vn))
    some = range(B) if some is None else some
    own = {(b, h): cache_rows(cache, b, h) for b in some for h in range(Hkv)}
    out = mk.decode_attn_prefix(cache, prefix, q, kn, vn)
    g = Hq // Hkv
    rows = 16
    while rows < min(B * g, 128):
        rows *= 2
    total = -(-B * g // rows) * Hkv * (-(-prefix.n_packed // 128) + -(-prefix.n_res // 128))
    for h in range(Hkv):
        pk, pv = (t.to(DEV) for t in cache_rows(prefix, 0, h))
        assert torch.equal(pv.cpu(), v[h].double())   # exactly what was put in
        for b in some:
            ok, ov = own[b, h]
            kk, vv = torch.cat([pk, ok.to(DEV), kn[b, h:h + 1].double()]), torch.cat([pv, ov.to(DEV), vn[b, h:h + 1].double()])
            ref, tol = _attend(q[b, h * g:(h + 1) * g].double(), kk, vv, -(-total // SMS), len(ov) + 1)
            err = (out[b, h * g:(h + 1) * g].double() - ref).abs()
            assert (err <= tol).all(), (b, h, float((err / tol).max()))


@pytest.fixture
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mk.lib()


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,n", [(2, 8, 8, 60000), (12, 8, 4, 100001), (32, 16, 4, 100000), (24, 4, 2, 131000)])
@pytest.mark.parametrize("q_scale", [0.0, 1.0])
def test_every_tile_of_a_long_prefix_counts(gpu, B, Hq, Hkv, n, q_scale):
    """Tens of tiles a CTA: every buffer and barrier goes round many times (16, 32, 64 and 128 rows)."""
    _run(B, Hq, Hkv, n, 128, 128, q_scale, some=sorted({0, B // 2, B - 1}))


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv", [(1, 2, 1), (6, 8, 2), (16, 3, 1), (33, 4, 2)])
@pytest.mark.parametrize("n,G,R,rotate", [(1, 32, 32, 0), (33, 32, 0, 0), (127, 32, 32, 0), (128, 32, 0, 0), (129, 32, 64, 90),
                                          (255, 64, 64, 100), (257, 128, 32, 1), (700, 32, 128, 159), (3001, 128, 128, 200)])
def test_every_token_of_a_prefix_counts(gpu, B, Hq, Hkv, n, G, R, rotate):
    _run(B, Hq, Hkv, n, G, R, 1.0, rotate)


def _sound(n, G, R, m, seed=720):
    """One KV head's rows on the CPU: q, k, v with 41 own tokens at the end, the prefix's tiles, outputs, tolerances."""
    k, v, q, _, _ = _case(m, 1, 1, n, G, R, 1.0, seed)
    own_k, own_v = _random((41, 128), seed + 300).double(), _random((41, 128), seed + 301).double()
    q, k, v = q[:, 0].double(), torch.cat([k[0].double(), own_k]), torch.cat([v[0].double(), own_v])
    tile = torch.cat([_tiles(n, _split(n, G, R)), torch.full((41,), -1)])
    # as many tiles a CTA as the tests above have at most
    return q, k, v, tile, *_attend(q, k, v, 26 if n > 50000 else 2, 41)


def _seen(o, tol, q, k, v, x=None, keep=None):
    x = (q @ k.T) * TAU if x is None else x
    if keep is not None:
        x = x + keep.log()
    return bool(((torch.softmax(x, -1) @ v - o).abs() > tol).any())


@pytest.mark.parametrize("n", [3001, 60000, 131000])
@pytest.mark.parametrize("at", [0, 1, 2, 0.3, 0.7, -2, -1])
def test_a_planted_tile_is_seen(n, at):
    """A tile that is missing, counted twice, or meets the keys or the values of the tile two before it."""
    q, k, v, tile, o, tol = _sound(n, 128, 128, 8)
    last = int(tile.max())
    j = last + 1 + at if at < 0 else at if isinstance(at, int) else int(at * last)
    here = tile == j
    assert not _seen(o, tol, q, k, v)
    for weight in (0.0, 2.0):
        assert _seen(o, tol, q, k, v, keep=torch.where(here, weight, 1.0).double()), weight
    if j >= 2:
        i = torch.nonzero(here)[:, 0]
        stale = torch.nonzero(tile == j - 2)[:, 0][:len(i)]
        if len(stale) == len(i):
            other = v.clone()
            other[i] = v[stale]
            assert _seen(o, tol, q, k, other), "values"
            x = (q @ k.T) * TAU
            x[:, i] = x[:, stale]
            assert _seen(o, tol, q, k, v, x=x), "keys"


@pytest.mark.parametrize("n,G,R", [(129, 32, 64), (700, 32, 128), (3001, 128, 128)])
def test_a_planted_token_is_seen(n, G, R):
    """The first or the last token, or one at an edge of the packed part, that is missing or counted twice."""
    q, k, v, _, o, tol = _sound(n, G, R, 8)
    packed = _split(n, G, R)
    for t in {0, 31, packed - 1, packed, n - 1}:
        for weight in (0.0, 2.0):
            keep = torch.ones(len(k), dtype=torch.float64)
            keep[t] = weight
            assert _seen(o, tol, q, k, v, keep=keep), (t, weight)
