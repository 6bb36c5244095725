"""Precision of the steps behind a shared prefix, against 64 bits: what a
sequence's own tokens and the prefix's tokens each add to the rounding of the
output.

The relative norm of the error is made of two roundings to fp16, the output's and
P's (over the prefix's tokens), each off by at most 2^-11 and spread evenly at the
widest, independent: 2^-11 sqrt(1/3) = 2.82e-4 the first, as much the second if
all the weight is on the prefix, 4.0e-4 together.  Where the weight is on the own
tokens (4000 of 4090) the first remains, with a few percent for the prefix's part:
2.9e-4; sums of subnormal value codes made it 3.7e-4 to 4.9e-4 there
(groups of four).  Rounding the dequantized keys to fp16 would give 0.7e-3 to 1.5e-3.
"""
import math

import pytest
import torch

from bit_quantized_evicted_b200 import minikv as mk
from tests.plain64 import attend, cache_rows
from tests.test_gpu_prefix import _batch, _inputs, _prefix

pytestmark = pytest.mark.gpu

TAU = 1.0 / math.sqrt(128.0)


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mk.lib()


def _reference(cache, prefix, q, kn, vn):
    """Before the step: the output in float64."""
    B, Hq = q.shape[:2]
    g = Hq // cache.Hkv
    out = torch.empty((B, Hq, 128), dtype=torch.float64)
    for h in range(cache.Hkv):
        shared = cache_rows(prefix, 0, h)
        for b in range(B):
            k, v = (torch.cat([p, own, x[b, h:h + 1].double().cpu()])
                    for p, own, x in zip(shared, cache_rows(cache, b, h), (kn, vn)))
            out[b, h * g:(h + 1) * g] = attend(q[b, h * g:(h + 1) * g].double().cpu(), k, v, TAU)
    return out


@pytest.mark.parametrize("B,Hq,Hkv", [(3, 8, 2), (5, 2, 2), (20, 4, 1), (40, 8, 2)])
@pytest.mark.parametrize("own,n,bound", [(90, 700, 4.0e-4), (90, 3001, 4.0e-4), (2000, 2000, 4.0e-4), (4000, 90, 2.9e-4),
                                         (6000, 1, 2.9e-4)])
def test_error_is_that_of_the_roundings(B, Hq, Hkv, own, n, bound):
    cache, prefix = _batch([own] * B, Hq, Hkv, "uniform"), _prefix(Hkv, n, 32, 128, rotate=5)
    x = _inputs(B, Hq, Hkv, 0)
    ref = _reference(cache, prefix, *x)
    err = mk.decode_attn_prefix(cache, prefix, *x).double().cpu() - ref
    assert float(err.norm() / ref.norm()) <= bound, float(err.norm() / ref.norm())


def test_sequences_without_the_prefix_keep_their_bits():
    """Among sharing sequences: the others come out as minikv_decode_attn's, bit for bit, whatever their length."""
    mk.set_deterministic(True)
    try:
        lengths, Hq, Hkv, flags = (5000, 300, 2500, 40), 8, 2, (0, 1, 0, 1)
        for mode in ("ragged", "device"):
            cache, other = (_batch(lengths, Hq, Hkv, mode) for _ in range(2))
            x = _inputs(4, Hq, Hkv, 0)
            out = mk.decode_attn_prefix(cache, _prefix(Hkv, 1000), *x, flags)
            assert torch.equal(out[[0, 2]], mk.decode_attn(other, *x)[[0, 2]])
    finally:
        mk.set_deterministic(False)
