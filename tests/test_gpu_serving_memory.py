"""Default workspaces that captured graphs hold: a later call on the same cache
with more query heads needs a larger one, and must leave the graph its own."""
import weakref

import pytest
import torch

from bit_quantized_evicted_b200 import minikv as mk
from tests.test_gpu_prefix import _batch, _inputs, _prefix

pytestmark = pytest.mark.gpu

DEV = "cuda"
B, HKV = 9, 2   # (9 rows a KV head take tiles of 16, the 36 of four times the heads tiles of 64)


@pytest.fixture(autouse=True)
def _deterministic():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mk.set_deterministic(True)
    try:
        yield
    finally:
        mk.set_deterministic(False)


@pytest.mark.parametrize("call", ["prefix", "mass"])
def test_a_graph_keeps_the_workspace_it_was_given(call):
    prefix = _prefix(HKV, 700)

    def step(cache, x, mass, out=None):
        if call == "prefix":
            return mk.decode_attn_prefix(cache, prefix, *x, out=out)
        return mk.decode_attn_mass(cache, *x, mass, out=out)

    few, many = _inputs(B, HKV, HKV, 0), _inputs(B, 4 * HKV, HKV, 1)
    runs = []
    for captured in (False, True):
        cache = _batch([200] * B, 4 * HKV, HKV, "device", steps=40)
        mass = torch.zeros((B, HKV, cache.cap + cache.R + cache.G), dtype=torch.float32, device=DEV)
        out = torch.empty_like(few[0])
        step(cache, few, mass, out)
        ws = weakref.ref(getattr(cache, "ws_" + call))
        if captured:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step(cache, few, mass, out)
        got = []
        for _ in range(3):
            got.append(step(cache, many, mass).clone())
            assert ws() is not None, "the first workspace is gone"
            junk = [torch.full((ws().numel(),), 255, dtype=torch.uint8, device=DEV) for _ in range(4)]
            graph.replay() if captured else step(cache, few, mass, out)
            got.append(out.clone())
            del junk
        runs.append([*got, mass])
    for a, b in zip(*runs):
        assert torch.equal(a, b)
