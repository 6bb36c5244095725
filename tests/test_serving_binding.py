"""What the Python binding refuses before the windowed and shared-prefix calls
reach the library, on the CPU."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

from bit_quantized_evicted_b200 import minikv as mk

P = 1 << 24
CACHE = SimpleNamespace(c=SimpleNamespace(B=3, Hkv=2, D=128))


def _step(q=(3, 8, 128), k=(3, 2, 128), v=(3, 2, 128), out=(3, 8, 128)):
    mk._check_step(CACHE, *(torch.empty(s, dtype=torch.float16) for s in (q, k, v)),
                   None if out is None else torch.empty(out, dtype=torch.float16))


def test_step_shapes():
    _step()
    _step(out=None)


@pytest.mark.parametrize("change", [dict(q=(2, 8, 128)), dict(q=(3, 8, 64)), dict(k=(3, 1, 128)), dict(k=(2, 2, 128)),
                                    dict(v=(3, 2, 64)), dict(v=(3, 2, 1, 128)), dict(out=(3, 4, 128)),
                                    dict(out=(2, 8, 128))])
def test_step_shape_refusals(change):
    with pytest.raises(ValueError):
        _step(**change)


class _Fake(torch.Tensor):
    """A tensor that says it is on CUDA device 1."""
    is_cuda, device = True, "cuda:1"

    def get_device(self):
        return 1


def test_tensors_of_two_devices_are_refused():
    t = torch.empty(4, dtype=torch.float16).as_subclass(_Fake)
    assert mk._at(t, torch.float16, 1, "k") == t.data_ptr()
    with pytest.raises(ValueError, match="k is on cuda:1, other tensors on cuda:0"):
        mk._at(t, torch.float16, 0, "k")
    with pytest.raises(TypeError, match="k must be torch.float16"):
        mk._at(t.float(), torch.float16, 1, "k")
    with pytest.raises(TypeError, match="CUDA tensor"):
        mk._at(torch.empty(4, dtype=torch.float16), torch.float16, 0, "k")


def test_tensors_of_the_cpu_are_refused():
    q, k = torch.empty((1, 4, 9, 128), dtype=torch.float16), torch.empty((1, 2, 9, 128), dtype=torch.float16)
    with pytest.raises(TypeError, match="CUDA tensor"):
        mk.window_prefill(q, k, k, 4)


@pytest.mark.parametrize("q,k,v,o", [
    ((1, 4, 9, 128), (1, 2, 9, 128), (1, 2, 8, 128), None), ((2, 4, 9, 128), (1, 2, 9, 128), (1, 2, 9, 128), None),
    ((1, 4, 9, 128), (1, 2, 9, 64), (1, 2, 9, 64), None), ((1, 4, 9, 128), (1, 2, 9, 128), (1, 2, 9, 128), (1, 4, 8, 128))])
def test_window_prefill_shape_refusals(q, k, v, o):
    t = [torch.empty(s, dtype=torch.float16) for s in (q, k, v)]
    with pytest.raises(ValueError):
        mk.window_prefill(*t, 4, o=None if o is None else torch.empty(o, dtype=torch.float16))


def test_flags_of_another_type_are_converted():
    """A ctypes array of bytes is not read as one of ints."""
    flags = mk.shared_rows((ctypes.c_byte * 3)(1, 0, 1))
    assert flags._type_ is ctypes.c_int and list(flags) == [1, 0, 1]
    assert list(mk.shared_rows([True, False, 2])) == [1, 0, 1]


@pytest.mark.parametrize("over", [dict(o=P), dict(o=2 * P)])
def test_output_over_keys_or_values_is_refused(over):
    a = dict(q=3 * P, k=P, v=2 * P, **over)
    assert mk.lib().minikv_window_prefill(a["q"], a["k"], a["v"], 1, 4, 2, 512, 512, 128, 64, 4, 0.1, a["o"], 4 * P,
                                          1 << 20, None) == mk.ERR_INVALID_ARG
    assert b"over k or v" in mk.lib().minikv_last_error_string()
