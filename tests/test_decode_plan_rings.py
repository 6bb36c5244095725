"""The cut of a cache's next decode step depends on that cache alone: two caches
of the same state whose rings differ are planned in both orders, on host threads
of their own (each has its own memory of earlier plans).  On the CPU."""
import threading

import pytest

from bit_quantized_evicted_b200 import minikv as mk
from tests.test_decode_plan import _bound


def _plans(*caches):
    """The plans of the caches, in order, on a host thread that has planned nothing before."""
    out = []
    thread = threading.Thread(target=lambda: out.extend(mk.decode_plan(c) for c in caches))
    thread.start()
    thread.join()
    return out


@pytest.mark.parametrize("B,Hkv,n_packed", [(1, 2, 0), (1, 4, 512), (1, 8, 2048), (12, 8, 512), (3, 32, 96), (16, 16, 1024)])
def test_plans_do_not_depend_on_what_was_planned_before(B, Hkv, n_packed):
    short, long_ = _bound(B, Hkv, 4096, 32, 0), _bound(B, Hkv, 4096, 32, 128)   # rings of 32 and 160 tokens
    for c in (short, long_):
        c.n_packed, c.n_res = n_packed, 31
    a, b = _plans(short)[0], _plans(long_)[0]
    assert _plans(short, long_) == [a, b]
    assert _plans(long_, short) == [b, a]
