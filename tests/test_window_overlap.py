"""An output of the window prefill that shares memory with its inputs in part is
refused (on the CPU); one right beside them is not (on the GPU).
"""
import pytest
import torch

from bit_quantized_evicted_b200 import minikv as mk

Q, K, V = 1 << 24, 2 << 24, 3 << 24
ROWS = 4 * 512 * 256     # bytes of q and o: 4 heads
KEYS = 2 * 512 * 256     # of k and v: 2 heads


def _call(o, **at):
    a = dict(q=Q, k=K, v=V, **at)
    rc = mk.lib().minikv_window_prefill(a["q"], a["k"], a["v"], 1, 4, 2, 512, 512, 128, 64, 4, 0.1, o, 4 << 24, 1 << 20, None)
    return rc, mk.lib().minikv_last_error_string().decode()


@pytest.mark.parametrize("o", [K, V, K + 256, K + KEYS - 256, K - ROWS + 256, V + 4096, V - 16, V + KEYS - 16])
def test_over_keys_or_values(o):
    rc, why = _call(o)
    assert rc == mk.ERR_INVALID_ARG and "over k or v" in why


@pytest.mark.parametrize("o", [Q + 256, Q - 256, Q + ROWS - 16, Q - ROWS + 16])
def test_over_part_of_the_queries(o):
    rc, why = _call(o)
    assert rc == mk.ERR_INVALID_ARG and "part of q" in why


@pytest.mark.gpu
def test_beside_the_inputs():
    """q, o, k, v of one buffer without a gap: o is written between them, and nothing else."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    n = 4 * 130 * 128
    buf = torch.randn(4 * n, device="cuda").half()
    q, o, k, v = (buf[i * n:(i + 1) * n].view(1, 4, 130, 128) for i in range(4))
    before = buf.clone()
    want = mk.window_prefill(q.clone(), k.clone(), v.clone(), 40, 2)
    mk.window_prefill(q, k, v, 40, 2, o=o)
    assert torch.equal(o, want)
    assert torch.equal(buf[:n], before[:n]) and torch.equal(buf[2 * n:], before[2 * n:])
