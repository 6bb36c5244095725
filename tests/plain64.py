"""Plain 64-bit forms of the cache's attention, for the parity tests: what a
cache holds in order of arrival, and softmax attention over chosen tokens."""
import numpy as np
import torch


def cache_rows(cache, b: int, h: int):
    """Keys and values [n, 128] (float64, CPU) of sequence b and KV head h, in order of arrival."""
    a = cache.arrays()
    n, r, start = cache.seq_state(b)
    bits = torch.arange(0, 32, 2, device=cache.device)

    def codes(words):
        return ((words[:n].long()[..., None] >> bits) & 3).reshape(n, 128).double()

    group = torch.arange(n, device=cache.device) // cache.G
    k = codes(a["k_codes"][b, h]) * a["k_scale"][b, h].double()[group] + a["k_zero"][b, h].double()[group]
    v = codes(a["v_codes"][b, h]) * a["v_scale"][b, h, :n].double() + a["v_zero"][b, h, :n].double()
    slot = (start + torch.arange(r, device=cache.device)) % (cache.R + cache.G)
    return (torch.cat([k, a["k_res"][b, h][slot].double()]).cpu(), torch.cat([v, a["v_res"][b, h][slot].double()]).cpu())


def attend(q, k, v, scale: float, seen=None):
    """softmax(scale q k^T) v in float64: q [m, 128], k, v [n, 128], seen [m, n] or [n] (None: all)."""
    x = (q.double() @ k.T) * scale
    if seen is not None:
        x = x.masked_fill(~seen, -np.inf)
    return torch.softmax(x, -1) @ v


def window_seen(n: int, window: int, n_sink: int):
    """Tokens the newest of n sees."""
    t = torch.arange(n)
    return (t < n_sink) | (t >= n - window)
