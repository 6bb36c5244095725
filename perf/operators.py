"""Attention with a sliding window and sinks, and decoding behind a shared prefix: cases, inputs, plain forms, 64-bit values.

Three operators of the 2-bit KV cache library (head size 128, fp16 tensors):

* ``window_prefill``: prompt attention in which a query at position p sees the keys j <= p with
  p - j < window, and the first ``n_sink`` keys.  The queries are the last Tq of Tk positions.
* ``decode_attn_window``: one decode step over the 2-bit cache under the same mask; positions are
  the order in which tokens entered the cache.
* ``decode_attn_prefix``: one decode step of a batch whose sequences (all, or those marked) also
  attend to one shared prefix, held once in a 2-bit cache of its own.

A cache's tensors: codes [B, Hkv, cap, 8] (16 two-bit codes a word), key scale and zero per channel
and group of G tokens, value scale and zero per token, and a ring of R + G fp16 rows for the newest
tokens.  A decode step appends its token to the ring.
"""
import math

import torch

own = False

D = 128
DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a short system message through a layer with a small window: a call of a few microseconds
        dict(name="prefill 512", op="prefill", B=1, Hq=4, Hkv=4, Tq=512, Tk=512, window=128, sink=4),
        # a chat prompt of a Mistral-7B layer (32 query heads over 8 KV heads, window 4096)
        dict(name="prefill 8K", op="prefill", B=1, Hq=32, Hkv=8, Tq=8192, Tk=8192, window=4096, sink=4),
        # two prompts of odd length through a LLaMA2-7B layer (32 heads, no grouping)
        dict(name="prefill 3001 x2", op="prefill", B=2, Hq=32, Hkv=32, Tq=3001, Tk=3001, window=1000, sink=17),
        # one chunk of a long prompt against everything before it
        dict(name="prefill chunk", op="prefill", B=1, Hq=32, Hkv=8, Tq=2048, Tk=20011, window=4096, sink=64),
        # the longest prompt of the benchmark's contexts
        dict(name="prefill 32K", op="prefill", B=1, Hq=32, Hkv=8, Tq=32768, Tk=32768, window=4096, sink=4),
        # one user's token: latency
        dict(name="window decode 1", op="window", B=1, Hq=32, Hkv=8, G=32, R=128, lo=2500, hi=2500, window=512, sink=4),
        # a serving batch whose prompts were longer than the window
        dict(name="window decode 16", op="window", B=16, Hq=32, Hkv=8, G=32, R=128, lo=6553, hi=6553, window=4096, sink=4),
        # a large batch of unequal prompts, some shorter than the window, without grouping
        dict(name="window decode 48", op="window", B=48, Hq=32, Hkv=32, G=32, R=128, lo=300, hi=9000, window=2048, sink=33),
        # a few users of one short system prompt: latency
        dict(name="prefix 4 x 1K", op="prefix", B=4, Hq=32, Hkv=8, G=32, R=128, lo=150, hi=400, prefix=1100, skip=0),
        # a LLaMA2-7B batch (no grouping) behind a page of instructions; every fifth request has another prompt
        dict(name="prefix 24 x 4K", op="prefix", B=24, Hq=32, Hkv=32, G=32, R=128, lo=200, hi=900, prefix=4321, skip=5),
        # a Mistral-7B serving batch behind a long document
        dict(name="prefix 16 x 32K", op="prefix", B=16, Hq=32, Hkv=8, G=32, R=128, lo=300, hi=1000, prefix=32768, skip=0),
        # the largest: many readers of one very long document
        dict(name="prefix 96 x 128K", op="prefix", B=96, Hq=32, Hkv=8, G=32, R=128, lo=200, hi=700, prefix=131000, skip=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "window", "prefix"])
    if op == "prefill":
        Hkv = rng.choice([1, 2, 3, 4, 8])
        g = rng.choice([1, 2, 3, 4, 7, 8])
        Tk = _log(rng, 1, 20000)
        Tq = Tk if rng.random() < 0.6 else _log(rng, 1, Tk)
        B = rng.randint(1, 3) if Tk < 4096 else 1
        return dict(op=op, B=B, Hq=g * Hkv if g * Hkv <= 32 else Hkv, Hkv=Hkv, Tq=Tq, Tk=Tk,
                    window=_log(rng, 1, 5000), sink=rng.choice([0, 1, 4, _log(rng, 1, 300)]))
    g = rng.choice([1, 2, 3, 4])
    Hkv = rng.choice([1, 2, 5, 8, 16])
    G = rng.choice([32, 32, 64, 128])
    R = rng.choice([32, 64, 128])
    B = _log(rng, 1, 64)
    lo, hi = sorted((_log(rng, 1, 6000), _log(rng, 1, 6000)))
    if op == "window":
        return dict(op=op, B=B, Hq=g * Hkv, Hkv=Hkv, G=G, R=R, lo=lo, hi=hi, window=_log(rng, 1, 6000),
                    sink=rng.choice([0, 1, 4, _log(rng, 1, 300)]))
    return dict(op=op, B=B, Hq=g * Hkv, Hkv=Hkv, G=G, R=R, lo=min(lo, 1500), hi=min(hi, 1500),
                prefix=_log(rng, 1, 60000), skip=rng.choice([0, 0, 2, 3]))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(shape, g):
    return torch.randn(shape, generator=g, device=DEV).half()


def _keys(shape, g):
    """Keys with four outlier channels, as the cache's per-channel quantization meets them."""
    x = torch.randn(shape, generator=g, device=DEV)
    x[..., :4] *= 10.0
    return x.half()


def _split(n, R, G):
    """Tokens of an n-token sequence that are (packed, in the ring), with room for one more in the ring."""
    if n < R:
        return 0, n
    r = R + (n - R) % G
    r -= r == R + G - 1
    return (n - R) // G * G, r


def _quantize(x, groups, dim):
    """2-bit codes of x (fp32), split along dim into groups; (codes, scale, zero) with the group axis reduced."""
    y = x.unflatten(dim, (groups, -1))
    zero, top = y.amin(dim + 1), y.amax(dim + 1)
    scale = ((top - zero) / 3).half()
    s = scale.float().unsqueeze(dim + 1)
    code = ((y - zero.unsqueeze(dim + 1)) / torch.where(s == 0, torch.ones_like(s), s)).round().clamp(0, 3)
    return code.flatten(dim, dim + 1).int(), scale, zero.half()


def _words(code):
    c = code.unflatten(-1, (8, 16)) << (2 * torch.arange(16, device=DEV, dtype=torch.int32))
    return c.sum(-1).int()      # 16 codes in 32 bits; the top code's sign bit wraps


def _cache(B, Hkv, G, R, lens, g):
    """A cache after prefill and some steps: sequence b holds lens[b] tokens (fp16 rows, quantized here)."""
    state = [_split(n, R, G) for n in lens]
    cap = max(max(p for p, _ in state) + G, G)
    ring = R + G
    kc, ks, kz = _quantize(_keys((B, Hkv, cap, D), g).float(), cap // G, 2)
    k_codes = _words(kc)
    del kc
    vc, vs, vz = _quantize(_normal((B, Hkv, cap, D), g).float(), 1, 3)
    arrays = dict(k_codes=k_codes, v_codes=_words(vc), k_scale=ks, k_zero=kz, v_scale=vs, v_zero=vz,
                  k_res=_keys((B, Hkv, ring, D), g), v_res=_normal((B, Hkv, ring, D), g))
    n_packed = [p for p, _ in state]
    n_res = [r for _, r in state]
    start = [(7 * b + 3) % ring if lens[0] != lens[-1] else 3 % ring for b in range(B)]
    t = lambda v: torch.tensor(v, device=DEV)  # noqa: E731
    return dict(arrays, B=B, Hkv=Hkv, G=G, R=R, cap=cap, ring=ring, state=(n_packed, n_res, start),
                n_packed=t(n_packed), n_res=t(n_res), start=t(start))


def _lens(case):
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [lo + (hi - lo) * b // max(B - 1, 1) for b in range(B)]


def _shared(case):
    return [not case["skip"] or b % case["skip"] != case["skip"] - 1 for b in range(case["B"])]


def _inputs(case, seed):
    g = _gen(seed)
    if case["op"] == "prefill":
        B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
        return dict(q=_normal((B, Hq, case["Tq"], D), g), k=_keys((B, Hkv, case["Tk"], D), g),
                    v=_normal((B, Hkv, case["Tk"], D), g))
    B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
    s = dict(cache=_cache(B, Hkv, case["G"], case["R"], _lens(case), g), q=_normal((B, Hq, D), g),
             k_new=_keys((B, Hkv, D), g), v_new=_normal((B, Hkv, D), g))
    if case["op"] == "prefix":
        s["prefix"] = _cache(1, Hkv, case["G"], case["R"], [case["prefix"]], g)
        s["shared"] = _shared(case)
        s["shared_t"] = torch.tensor(s["shared"], device=DEV)
    return s


def _handle(c, Hq, mk):
    """The library's cache with these contents, as a program that serves has it."""
    h = mk.MiniKVCache(c["B"], c["Hkv"], c["cap"], G=c["G"], R=c["R"], Hq=Hq)
    for name, dst in h.arrays().items():
        dst.copy_(c[name])
    n_packed, n_res, start = c["state"]
    if len(set(zip(n_packed, n_res, start))) > 1:
        h.set_ragged()
    return h


def _rewind(h, state):
    """Put the host-side lengths back, so that the same step can be run again."""
    n_packed, n_res, start = state
    if h.ragged:
        for b in range(h.B):
            h._seq[3 * b], h._seq[3 * b + 1], h._seq[3 * b + 2] = n_packed[b], n_res[b], start[b]
    else:
        h.c.n_packed, h.c.n_res, h.c.res_start = n_packed[0], n_res[0], start[0]


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    s["scale"] = 1.0 / math.sqrt(D)
    if own:
        from bit_quantized_evicted_b200 import minikv as mk
        s["mk"] = mk
        B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
        if case["op"] == "prefill":
            s["o"] = torch.empty_like(s["q"])
            s["ws"] = torch.empty(mk.workspace_size(mk.OP_WINDOW_PREFILL, B, Hq, Hkv, case["Tq"]), dtype=torch.uint8,
                                  device=DEV)
            return s
        s["out"] = torch.empty_like(s["q"])
        s["handle"] = h = _handle(s["cache"], Hq, mk)
        a = h.arrays()
        s["rings"] = (a["k_res"], a["v_res"])
        _rewind(h, s["cache"]["state"])
        if case["op"] == "prefix":
            s["prefix_handle"] = p = _handle(s["prefix"], Hq, mk)
            _rewind(p, s["prefix"]["state"])
            s["ws"] = torch.zeros(mk.workspace_size(mk.OP_DECODE_ATTN_PREFIX, B, Hq, Hkv, h.cap + h.R + h.G),
                                  dtype=torch.uint8, device=DEV)
            s["share"] = mk.shared_rows(s["shared"]) if not all(s["shared"]) else None
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    if own:
        mk = s["mk"]
        if case["op"] == "prefill":
            return mk.window_prefill(s["q"], s["k"], s["v"], case["window"], case["sink"], s["scale"], o=s["o"],
                                     ws=s["ws"])
        h = s["handle"]
        _rewind(h, s["cache"]["state"])
        if case["op"] == "window":
            out = mk.decode_attn_window(h, s["q"], s["k_new"], s["v_new"], case["window"], case["sink"], s["scale"],
                                        out=s["out"])
        else:
            out = mk.decode_attn_prefix(h, s["prefix_handle"], s["q"], s["k_new"], s["v_new"], s["share"], s["scale"],
                                        out=s["out"], ws=s["ws"])
        return [out, *s["rings"]]
    if case["op"] == "prefill":
        return _plain_prefill(s["q"], s["k"], s["v"], case["window"], case["sink"], s["scale"])
    return _plain_decode(s)


def _plain_prefill(q, k, v, window, sink, scale):
    """Blocks of 128 queries against their band of keys (one gathered view), and the sinks before the band."""
    B, Hq, Tq, _ = q.shape
    Hkv, Tk = k.shape[1], k.shape[2]
    g, bs = Hq // Hkv, min(128, Tq)
    nb = -(-Tq // bs)
    back = min(window, Tk) - 1                     # keys before a query's own
    first = Tk - Tq                                # position of query 0
    qb = torch.nn.functional.pad(q.float(), (0, 0, 0, nb * bs - Tq)).view(B, Hkv, g, nb, bs, D)
    qb = qb.permute(0, 1, 3, 2, 4, 5).reshape(B, Hkv, nb, g * bs, D)
    pad = lambda x: torch.nn.functional.pad(x.float(), (0, 0, back, nb * bs - Tq))[:, :, first:]  # noqa: E731
    kb = pad(k).unfold(2, back + bs, bs)           # [B, Hkv, nb, D, back + bs]
    vb = pad(v).unfold(2, back + bs, bs).transpose(-1, -2)
    pos = first + torch.arange(nb * bs, device=q.device).view(nb, 1, bs, 1)
    j = first - back + bs * torch.arange(nb, device=q.device).view(nb, 1, 1, 1) + torch.arange(back + bs, device=q.device)
    seen = (j >= 0) & (j < Tk) & (j <= pos) & (pos - j < window)
    x = torch.matmul(qb, kb).view(B, Hkv, nb, g, bs, -1).mul_(scale).masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    n = min(sink, Tk)
    if n:
        js = torch.arange(n, device=q.device)
        seen = (js <= pos) & (pos - js >= window)
        y = torch.matmul(qb, k[:, :, None, :n].float().transpose(-1, -2)).view(B, Hkv, nb, g, bs, n)
        y = y.mul_(scale).masked_fill_(~seen, -math.inf)
        top = torch.maximum(top, y.amax(-1, keepdim=True))
        y = y.sub_(top).exp_()
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, Hkv, nb, g * bs, -1), vb).view(B, Hkv, nb, g, bs, D)
    if n:
        total = total + y.sum(-1, keepdim=True)
        o = o + torch.matmul(y.view(B, Hkv, nb, g * bs, n), v[:, :, None, :n].float()).view(B, Hkv, nb, g, bs, D)
    o = (o / total).permute(0, 1, 3, 2, 4, 5).reshape(B, Hq, nb * bs, D)
    return o[:, :, :Tq].half()


def _unpack(words):
    return ((words.unsqueeze(-1) >> (2 * torch.arange(16, device=DEV, dtype=torch.int32))) & 3).flatten(-2)


def _dequant(c):
    """fp32 keys and values of the packed tokens, [B, Hkv, cap, D]."""
    groups = c["cap"] // c["G"]
    k = _unpack(c["k_codes"]).float().unflatten(2, (groups, c["G"]))
    k = k.mul_(c["k_scale"].float().unsqueeze(3)).add_(c["k_zero"].float().unsqueeze(3)).flatten(2, 3)
    v = _unpack(c["v_codes"]).float().mul_(c["v_scale"].float()).add_(c["v_zero"].float())
    return k, v


def _tokens(c, extra):
    """Keys, values [B, Hkv, cap + ring, D] and each one's place in order of arrival (-1: none) [B, cap + ring]."""
    k, v = _dequant(c)
    t = torch.arange(c["cap"], device=DEV)[None]
    i = (torch.arange(c["ring"], device=DEV)[None] - c["start"][:, None]) % c["ring"]
    place = torch.cat([torch.where(t < c["n_packed"][:, None], t, -1),
                       torch.where(i < c["n_res"][:, None] + extra, c["n_packed"][:, None] + i, -1)], 1)
    return torch.cat([k, c["k_res"].float()], 2), torch.cat([v, c["v_res"].float()], 2), place


def _plain_decode(s):
    case, c = s["case"], s["cache"]
    B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
    g = Hq // Hkv
    rows = torch.arange(B, device=DEV)
    slot = (c["start"] + c["n_res"]) % c["ring"]
    c["k_res"][rows, :, slot] = s["k_new"]
    c["v_res"][rows, :, slot] = s["v_new"]
    k, v, place = _tokens(c, 1)
    q = s["q"].float().view(B, Hkv, g, D)
    seen = place >= 0
    if case["op"] == "window":
        n = (c["n_packed"] + c["n_res"] + 1)[:, None]
        seen = seen & ((place < case["sink"]) | (n - 1 - place < case["window"]))
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]).masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    if case["op"] == "prefix":
        pk, pv, at = _tokens(s["prefix"], 0)
        seen = (at >= 0) & s["shared_t"][:, None]                                  # [B, P]
        y = torch.matmul(q.permute(1, 0, 2, 3).reshape(Hkv, B * g, D), pk[0].transpose(-1, -2)).view(Hkv, B, g, -1)
        y = y.mul_(s["scale"]).masked_fill_(~seen[None, :, None], -math.inf)
        top = torch.maximum(top, y.amax(-1, keepdim=True).transpose(0, 1))
        y = y.sub_(top.transpose(0, 1)).exp_()
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v)
    if case["op"] == "prefix":
        total = total + y.sum(-1, keepdim=True).transpose(0, 1)
        o = o + torch.matmul(y.view(Hkv, B * g, -1), pv[0]).view(Hkv, B, g, D).transpose(0, 1)
    return [(o / total).view(B, Hq, D).half(), c["k_res"], c["v_res"]]


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
    if case["op"] == "prefill":
        Tq, Tk, w, n = case["Tq"], case["Tk"], case["window"], case["sink"]
        pairs = sum(min(p + 1, w) + min(n, max(0, p + 1 - w)) for p in range(Tk - Tq, Tk))
        first = max(0, Tk - Tq - w + 1)            # keys from here on are read, and the sinks before
        keys = Tk - first + min(n, first)
        return {"bytes": 2 * D * B * (2 * Hq * Tq + 2 * Hkv * keys), "flops": 4 * D * B * Hq * pairs}
    G, R = case["G"], case["R"]
    token = 2 * (D // 4) + 4 * D / G + 4           # packed: codes, its share of the group's scale and zero, its own
    nbytes, pairs = 2 * D * B * (2 * Hq + 4 * Hkv), 0

    def add(n, r, times):
        nonlocal nbytes, pairs
        nbytes += Hkv * (n * token + r * 4 * D)
        pairs += (n + r) * times

    for length in _lens(case):
        n, r = _split(length, R, G)
        if case["op"] == "window":
            seen_r = min(r, case["window"] - 1)
            seen_n = min(n, case["window"] - 1 - seen_r)
            seen_n += min(n - seen_n, case["sink"])
            n, r = seen_n, seen_r
        add(n, r, 1)
        pairs += 1
    if case["op"] == "prefix":
        add(*_split(case["prefix"], R, G), sum(_shared(case)))
    return {"bytes": nbytes, "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------ the same from the definition, in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
    g = Hq // Hkv
    scale = 1.0 / math.sqrt(D)
    if case["op"] == "prefill":
        Tq, Tk, w, n = case["Tq"], case["Tk"], case["window"], case["sink"]
        o = torch.empty((B, Hq, Tq, D), dtype=torch.float64, device=DEV)
        for b in range(B):
            for h in range(Hq):
                k, v = s["k"][b, h // g].double(), s["v"][b, h // g].double()
                for i0 in range(0, Tq, 1024):
                    i1 = min(i0 + 1024, Tq)
                    p = torch.arange(Tk - Tq + i0, Tk - Tq + i1, device=DEV)[:, None]
                    lo, hi = max(0, int(p[0]) - w + 1), int(p[-1]) + 1
                    j = torch.cat([torch.arange(min(n, lo), device=DEV), torch.arange(lo, hi, device=DEV)])[None]
                    hidden = (j > p) | ((p - j >= w) & (j >= n))
                    x = (s["q"][b, h, i0:i1].double() @ k[j[0]].T) * scale
                    o[b, h, i0:i1] = torch.softmax(x.masked_fill(hidden, -math.inf), -1) @ v[j[0]]
        return o

    def rows(c, b, h, end):
        """Keys and values of one sequence and KV head in order of arrival."""
        n, r, st = (x[b] for x in c["state"])
        bits = torch.arange(0, 32, 2, device=DEV)
        code = lambda words: ((words[:n].long()[..., None] >> bits) & 3).reshape(n, D).double()  # noqa: E731
        grp = torch.arange(n, device=DEV) // c["G"]
        k = code(c["k_codes"][b, h]) * c["k_scale"][b, h].double()[grp] + c["k_zero"][b, h].double()[grp]
        v = code(c["v_codes"][b, h]) * c["v_scale"][b, h, :n].double() + c["v_zero"][b, h, :n].double()
        at = (st + torch.arange(r, device=DEV)) % c["ring"]
        return (torch.cat([k, c["k_res"][b, h][at].double()] + ([end[0][b, h:h + 1].double()] if end else [])),
                torch.cat([v, c["v_res"][b, h][at].double()] + ([end[1][b, h:h + 1].double()] if end else [])))

    c = s["cache"]
    o = torch.empty((B, Hq, D), dtype=torch.float64, device=DEV)
    for h in range(Hkv):
        pk, pv = rows(s["prefix"], 0, h, None) if case["op"] == "prefix" else (None, None)
        for b in range(B):
            k, v = rows(c, b, h, (s["k_new"], s["v_new"]))
            if case["op"] == "window":
                t = torch.arange(len(k), device=DEV)
                t = t[(t < case["sink"]) | (t >= len(k) - case["window"])]
                k, v = k[t], v[t]
            elif s["shared"][b]:
                k, v = torch.cat([pk, k]), torch.cat([pv, v])
            o[b, h * g:(h + 1) * g] = torch.softmax(s["q"][b, h * g:(h + 1) * g].double() @ k.T * scale, -1) @ v
    k_ring, v_ring = c["k_res"].double(), c["v_res"].double()
    for b in range(B):
        slot = (c["state"][2][b] + c["state"][1][b]) % c["ring"]
        k_ring[b, :, slot], v_ring[b, :, slot] = s["k_new"][b].double(), s["v_new"][b].double()
    return [o, k_ring, v_ring]
