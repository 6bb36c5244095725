"""Calls whose waits give up while their copies are in flight (the wait-probe
build gives up at the first poll): prompts of one to three key blocks, where the
producer queues every load without waiting for anyone, and the other roles may
leave at any time after.  Every call returns, reports what happened, and the
context goes on; loads that outlived their CTA would show in the next one's
shared memory.
"""
import ctypes

import pytest
import torch

from bit_quantized_evicted_b200 import minikv as mk
from bit_quantized_evicted_b200.build import WAIT_PROBE_LIB
from tests.test_gpu_window_prefill import _check, _qkv

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mk.lib()


@pytest.fixture
def probe():
    lib = ctypes.CDLL(WAIT_PROBE_LIB)
    for name, (res, args) in mk._SIGS.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    return lib


@pytest.mark.parametrize("B,Hq,Hkv,T,window,n_sink", [(1, 4, 2, 100, 50, 0), (40, 8, 4, 128, 128, 0), (8, 6, 2, 256, 40, 4),
                                                      (2, 32, 8, 384, 100, 130), (4, 8, 8, 200, 2000, 0)])
def test_short_window_prompts(probe, B, Hq, Hkv, T, window, n_sink):
    q, k, v = _qkv(B, Hq, Hkv, T, T, seed=930)
    ws = torch.zeros(mk.workspace_size(mk.OP_WINDOW_PREFILL, B, Hq, Hkv, T), dtype=torch.uint8, device=DEV)
    ref = mk.window_prefill(q, k, v, window, n_sink, ws=ws)
    for _ in range(10):
        mk.window_prefill(q, k, v, window, n_sink, ws=ws, library=probe)
        assert mk.window_prefill_status(ws, B, Hq, Hkv, T, library=probe) == 1
        assert torch.equal(mk.window_prefill(q, k, v, window, n_sink, ws=ws), ref)
        assert mk.window_prefill_status(ws, B, Hq, Hkv, T) == 0
    _check(ref[:1], q[:1], k[:1], v[:1], window, n_sink)


@pytest.mark.parametrize("B,H,T", [(1, 2, 100), (40, 4, 128), (8, 4, 256), (4, 8, 384)])
def test_short_prompts(probe, B, H, T):
    q, k, v = _qkv(B, H, H, T, T, seed=931)
    W = 16
    ws = torch.zeros(mk.workspace_size(mk.OP_SELECT_PREFILL, B, H, H, T, 128, W), dtype=torch.uint8, device=DEV)
    ref, scores = mk.select_prefill(q, k, v, W, ws=ws)
    o, sc = torch.empty_like(ref), torch.empty_like(scores)
    for _ in range(10):
        assert probe.minikv_select_prefill(q.data_ptr(), k.data_ptr(), v.data_ptr(), B, H, H, T, 128, W, 128 ** -0.5,
                                           o.data_ptr(), sc.data_ptr(), ws.data_ptr(), ws.numel(),
                                           torch.cuda.current_stream().cuda_stream) == mk.OK
        assert mk.select_prefill_status(ws, B, H, W, library=probe) == 1
        again = mk.select_prefill(q, k, v, W, ws=ws)
        assert torch.equal(again[0], ref) and torch.equal(again[1], scores)
        assert mk.select_prefill_status(ws, B, H, W) == 0
    _check(ref[:1], q[:1], k[:1], v[:1], T, 0)
