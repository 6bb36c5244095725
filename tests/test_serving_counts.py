"""Windows and sink counts that pass 32 bits reach the library as its largest
int (every key is visible), those below zero as a negative one (refused).  On the
CPU, with a library that records what it is given."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

from bit_quantized_evicted_b200 import minikv as mk

MAX = 2 ** 31 - 1


class _On(torch.Tensor):
    """A tensor that says it is on CUDA device 0."""
    is_cuda, device = True, torch.device("cuda", 0)

    def get_device(self):
        return 0


@pytest.fixture
def seen(monkeypatch):
    got = []

    def record(*at):
        return lambda *args: got.append([ctypes.c_int(args[i]).value for i in at]) or 0   # as ctypes converts them

    lib = SimpleNamespace(minikv_window_prefill=record(9, 10),
                          minikv_decode_attn_window=record(5, 6))
    monkeypatch.setattr(mk, "lib", lambda: lib)
    monkeypatch.setattr(mk, "_cuda_device", lambda: 0)
    monkeypatch.setattr(mk, "_current_stream", lambda device: 0)
    return got


@pytest.mark.parametrize("given,value", [(1, 1), (MAX, MAX), (2 ** 31, MAX), (2 ** 32 + 5, MAX), (2 ** 63 - 1, MAX),
                                         (0, 0), (-1, -1), (-2 ** 31 - 5, -1), (-2 ** 32 + 7, -1)])
def test_counts(seen, given, value):
    def fake(*shape, dtype=torch.float16):
        return torch.empty(shape, dtype=dtype).as_subclass(_On)

    q, k = fake(1, 2, 9, 128), fake(1, 2, 9, 128)
    ws = fake(256, dtype=torch.uint8)
    mk.window_prefill(q, k, k, given, given, o=q, ws=ws)
    cache = SimpleNamespace(c=mk.CacheStruct(B=1, Hkv=2, D=128), device=torch.device("cuda", 0), ws=ws)
    row = fake(1, 2, 128)
    mk.decode_attn_window(cache, row, row, row, given, given, out=row)
    assert seen == [[value, value], [value, value]]
