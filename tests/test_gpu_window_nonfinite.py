"""Values that are not finite in the window prefill: a channel whose visible values
hold a NaN, or infinities of both signs, is NaN, one with infinities of a sign
that infinity (every weight is positive), and all others are as if the rest held
numbers, whatever hidden keys hold.  And what a few of them cost.

Finite channels: the tolerance of the window prefill's own tests.
"""
import math

import pytest
import torch

from bit_quantized_evicted_b200 import minikv as mk
from tests.plain64 import attend
from tests.test_gpu_window_prefill import _qkv, _seen

pytestmark = pytest.mark.gpu

TAU = 1.0 / math.sqrt(128.0)
DEV = "cuda"
NAN, INF = float("nan"), float("inf")


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mk.lib()


def _check(o, q, k, v, window, n_sink):
    """o against the plain form: classes of what is not finite, and the finite channels."""
    B, Hq, Tq, _ = q.shape
    g, Tk = Hq // k.shape[1], k.shape[2]
    seen = _seen(Tq, Tk, window, n_sink)
    sees = lambda what: (seen.float() @ what.float()) > 0  # noqa: E731
    n = seen.sum(-1, keepdim=True).double()
    for b in range(B):
        for h in range(Hq):
            vv, got = v[b, h // g], o[b, h].double()
            up, down = sees(vv == INF), sees(vv == -INF)
            none = sees(vv.isnan()) | (up & down)
            up, down = up & ~none, down & ~none
            assert got[none].isnan().all(), (b, h)
            assert (got[up] == INF).all() and (got[down] == -INF).all(), (b, h)
            clean = torch.where(vv.isfinite(), vv, 0).double()
            kk = k[b, h // g].double()
            ref, mean = (attend(q[b, h], kk, x, TAU, seen) for x in (clean, clean.abs()))
            tol = 2 ** -11 * ref.abs() + (2 ** -11 + 5e-5) * mean + n * 2 ** -25 * clean.abs().max() + 2 ** -25
            fine = ~(none | up | down)
            assert ((got - ref).abs()[fine] <= tol[fine]).all(), (b, h, float(((got - ref).abs() - tol)[fine].max()))


@pytest.mark.parametrize("Hq,Hkv,Tq,Tk,window,n_sink", [(2, 2, 700, 700, 150, 3), (4, 2, 500, 900, 130, 40), (3, 1, 300, 300, 300, 0),
                                                        (2, 1, 260, 1500, 700, 200), (7, 1, 129, 129, 1000, 0),
                                                        (1, 1, 1, 400, 90, 5)])
@pytest.mark.parametrize("some", ["nan", "plus", "minus", "both", "mixed", "all"])
def test_classes(Hq, Hkv, Tq, Tk, window, n_sink, some):
    q, k, v = _qkv(1, Hq, Hkv, Tq, Tk, seed=940)
    gen = torch.Generator().manual_seed(941)

    def put(x, times):
        for _ in range(times):
            j, c = int(torch.randint(Tk, (1,), generator=gen)), int(torch.randint(128, (1,), generator=gen))
            v[:, int(torch.randint(Hkv, (1,), generator=gen)), j, c] = x

    for x, names in ((NAN, ("nan", "mixed")), (INF, ("plus", "both", "mixed")), (-INF, ("minus", "both", "mixed"))):
        if some in names:
            put(x, 6)
    if some == "both":
        v[:, :, Tk // 2, 5], v[:, :, Tk // 2 + 9, 5] = INF, -INF
    if some == "mixed" and n_sink:
        v[:, 0, n_sink - 1, 77] = -INF
    if some == "all":
        v[:, :, Tk // 3:2 * Tk // 3] = NAN
    _check(mk.window_prefill(q, k, v, window, n_sink), q, k, v, window, n_sink)


def test_infinite_value_of_a_key_without_weight():
    """The weight of the key is far below fp16's range, and fp32's smallest: the sum is infinite all the same."""
    q, k, v = _qkv(1, 2, 1, 300, 300, seed=942)
    q[..., 0], k[..., 0] = 40.0, 40.0
    k[:, :, 17, 0] = -40.0
    v[:, :, 17, 3] = INF
    _check(mk.window_prefill(q, k, v, 100, 0), q, k, v, 100, 0)


def test_one_bad_value_that_every_row_sees_costs_little():
    """A NaN or an infinity in a sink of a long prompt: no row is computed again.  (One pass over the values a warp,
    a few of the call's own time; a row at a time it was 140 times.)"""
    q, k, v = _qkv(1, 8, 2, 8192, 8192, seed=943)
    ws = torch.empty(mk.workspace_size(mk.OP_WINDOW_PREFILL, 1, 8, 2, 8192), dtype=torch.uint8, device=DEV)
    o = torch.empty_like(q)

    def ms():
        mk.window_prefill(q, k, v, 4096, 4, o=o, ws=ws)
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        for _ in range(3):
            mk.window_prefill(q, k, v, 4096, 4, o=o, ws=ws)
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b) / 3

    clean = ms()
    for x in (NAN, INF):
        v[:, :, 2, 7] = x
        assert ms() <= 20 * clean, (x, clean)
        assert not torch.isfinite(o[:, :, 2:, 7]).any() and torch.isfinite(o[..., 8:]).all()
