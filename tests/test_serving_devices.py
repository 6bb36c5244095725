"""Caches and streams of another GPU than the call's tensors: refused by the
binding before the library sees a pointer.  On the CPU, with stand-ins."""
from types import SimpleNamespace

import pytest
import torch

from bit_quantized_evicted_b200 import minikv as mk


class _On(torch.Tensor):
    """A tensor that says it is on CUDA device 1."""
    is_cuda, device = True, "cuda:1"

    def get_device(self):
        return 1


class _NoLibrary:
    def __getattr__(self, name):
        raise AssertionError(f"{name} was called")


def _fake(*shape):
    return torch.empty(shape, dtype=torch.float16).as_subclass(_On)


def _cache(device, B=2):
    return SimpleNamespace(c=SimpleNamespace(B=B, Hkv=2, D=128), Hkv=2, device=torch.device("cuda", device), ws=None)


@pytest.fixture
def step(monkeypatch):
    monkeypatch.setattr(mk, "lib", lambda: _NoLibrary())
    monkeypatch.setattr(mk, "_cuda_device", lambda: 1)
    return _fake(2, 8, 128), _fake(2, 2, 128), _fake(2, 2, 128)


def test_window_step_on_a_cache_of_another_device(step):
    for ws in (None, _fake(64)):
        with pytest.raises(ValueError, match="cache is on cuda:0, other tensors on cuda:1"):
            mk.decode_attn_window(_cache(0), *step, 8, ws=ws)


@pytest.mark.parametrize("cache,prefix,match", [(0, 1, "cache is on cuda:0"), (1, 0, "prefix is on cuda:0"),
                                                (1, 2, "prefix is on cuda:2")])
def test_prefix_step_on_caches_of_another_device(step, cache, prefix, match):
    for ws in (None, _fake(64)):
        with pytest.raises(ValueError, match=match):
            mk.decode_attn_prefix(_cache(cache), _cache(prefix, 1), *step, ws=ws, library=_NoLibrary())


def test_streams_of_another_device(step):
    stream = SimpleNamespace(device=torch.device("cuda", 0), cuda_stream=7)
    q, kn, vn = step
    k = _fake(2, 2, 9, 128)
    for call in (lambda: mk.decode_attn_window(_cache(1), *step, 8, stream=stream),
                 lambda: mk.decode_attn_prefix(_cache(1), _cache(1, 1), *step, stream=stream, library=_NoLibrary()),
                 lambda: mk.window_prefill(_fake(2, 8, 9, 128), k, k, 4, stream=stream, library=_NoLibrary())):
        with pytest.raises(ValueError, match="stream is on cuda:0, tensors on cuda:1"):
            call()
