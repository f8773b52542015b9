"""Cases of the paged key/value cache operators and their plain forms.

Three operators: ``cache_write`` (rows of new tokens into pages, copied or
quantised), ``cache_read`` (pages back into dense [B, Hkv, T, d] tensors) and
``sdpa_paged`` (attention of each sequence's newest tokens over its cache).

With ``own`` false, ``run`` computes them in elementary torch operations in 32
bits, rounded once at the end; with ``own`` true it calls this package.
``exact`` computes the same outputs from the definitions in 64 bits.

A cache holds keys and values as [pages, Hkv, page, d]; an 8-bit one holds
codes and one f32 scale per (token, head), [pages, Hkv, page]:

    scale = max(f32(amax / Q), 2^-30), Q = 448 (e4m3) or 127 (int8)
    code  = round_to_type(f32(x / scale))        value = code * scale

Sequence b has lens[b] tokens in the cache, the last n_b of them new.  Query i
of it stands at pos = lens[b] - n_b + i and sees the keys j <= pos (with a
window: j > pos - window as well); its scores are x = scale q.k, capped to
softcap tanh(x / softcap) where a cap is given, plus slope_h (j - pos) where
slopes are given.
"""
import math
import random

import torch

own = False

_TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
_BYTES = {"f32": 4, "bf16": 2, "e4m3": 1, "int8": 1}
_QMAX = {"e4m3": 448.0, "int8": 127.0}
_FLOOR = 2.0 ** -30


def _case(kind, name=None, *, io="bf16", cache="bf16", B=1, Hq=32, Hkv=8, d=128, page=16, q=(1, 1), kv=(1, 1),
          window=0, softcap=0.0, slopes=False, lens=0):
    c = dict(kind=kind, io=io, cache=cache, B=B, Hq=Hq, Hkv=Hkv, d=d, page=page, q_lo=q[0], q_hi=q[1], kv_lo=kv[0],
             kv_hi=kv[1], window=window, softcap=softcap, slopes=slopes, lens=lens)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decode step's new rows of eight sequences: as small as a write gets
        _case("write", "write_token", B=8, q=(1, 1), kv=(20, 3000), lens=1),
        # chunks of four prompts into a quantised cache, read back for a dense call
        _case("write_read", "write_read_e4m3", cache="e4m3", B=4, q=(101, 512), kv=(300, 2048), lens=2),
        # a whole long prompt at once, narrow heads
        _case("write_read", "write_read_int8", cache="int8", B=1, Hq=12, Hkv=12, d=64, page=64, q=(8190, 8190),
              kv=(8190, 8190), lens=3),
        # a batch's cache brought back as dense tensors
        _case("read", "read_e4m3", cache="e4m3", B=16, page=64, kv=(1000, 8192), lens=4),
        # one short conversation decoding alone: latency
        _case("attend", "decode_one", B=1, kv=(131, 131), lens=5),
        # a decoding batch of ragged lengths, bf16 cache
        _case("attend", "decode_bf16", B=32, kv=(200, 8192), lens=6),
        # a large decoding batch with long contexts over a quantised cache
        _case("attend", "decode_e4m3", cache="e4m3", B=64, page=64, kv=(1000, 16384), lens=7),
        # unshared narrow heads, capped scores in a sliding window
        _case("attend", "decode_int8_window_cap", cache="int8", B=24, Hq=12, Hkv=12, d=64, page=32, kv=(500, 8192),
              window=1024, softcap=30.0, lens=8),
        # 32-bit throughout
        _case("attend", "decode_f32", io="f32", cache="f32", B=4, Hq=12, Hkv=12, d=64, page=16, kv=(100, 1024), lens=9),
        # a few drafted tokens of every sequence checked in one step
        _case("attend", "draft_e4m3", cache="e4m3", B=16, page=32, q=(2, 5), kv=(500, 8192), lens=10),
        # a chunk of a long prompt behind its context
        _case("attend", "chunk_bf16", B=1, page=64, q=(2048, 2048), kv=(8192, 8192), lens=11),
        # prompts and single tokens mixed in one step, bias by distance
        _case("attend", "mixed_e4m3_slopes", cache="e4m3", B=8, page=32, q=(1, 1024), kv=(1024, 4096), slopes=True,
              lens=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = [max(work(c)[x] for c in listed()) for x in ("bytes", "flops")]
    while True:
        case = _draw(rng)
        w = work(case)
        if w["bytes"] <= most[0] and w["flops"] <= most[1]:
            return case


def _draw(rng):
    kind = rng.choice(("write", "write_read", "read", "attend", "attend", "attend", "attend"))
    d = rng.choice((64, 128))
    Hkv = rng.choice((1, 2, 4, 8, 12) if d == 64 else (1, 2, 4, 8))
    G = rng.choice((1, 2, 3, 4, 7, 8))
    io = "bf16" if rng.random() < 0.9 else "f32"
    cache = rng.choice((io, "e4m3", "int8"))
    page = rng.choice((16, 32, 64, 128))
    lens = rng.randrange(1 << 30)
    if kind != "attend":
        io = cache if cache in ("f32", "bf16") else io
        if kind == "write" and cache in _QMAX:
            kind = "write_read"  # codes are returned as what they stand for
        B = _log_int(rng, 1, 24)
        kv_hi = _log_int(rng, 40, 8192)
        q_hi = _log_int(rng, 1, kv_hi)
        return _case(kind, io=io, cache=cache, B=B, Hq=Hkv * G, Hkv=Hkv, d=d, page=page, q=(max(1, q_hi // 3), q_hi),
                     kv=(max(q_hi, kv_hi // 5), kv_hi), lens=lens)
    shape = rng.choice(("decode", "decode", "draft", "chunk", "mixed"))
    window = rng.choice((0, 0, 0, 128, 1000))
    softcap = rng.choice((0.0, 0.0, 30.0, 50.0))
    slopes = rng.random() < 0.25
    if io == "f32":
        shape, cap = rng.choice(("decode", "draft")), 1024
    else:
        cap = 16384 if shape == "decode" else 8192
    kv_hi = _log_int(rng, 20, cap)
    if shape == "decode":
        B, q = _log_int(rng, 1, 4 if io == "f32" else 64), (1, 1)
    elif shape == "draft":
        B, q = _log_int(rng, 1, 4 if io == "f32" else 32), (1, rng.randint(2, 8))
    elif shape == "chunk":
        n = _log_int(rng, 20, min(2048, kv_hi))
        B, q = 1, (n, n)
    else:
        B, q = _log_int(rng, 2, 8), (1, _log_int(rng, 20, min(1024, kv_hi)))
    kv_hi = max(kv_hi, q[1])
    return _case("attend", io=io, cache=cache, B=B, Hq=Hkv * G, Hkv=Hkv, d=d, page=page, q=q,
                 kv=(max(q[1], kv_hi // 6), kv_hi), window=window, softcap=softcap, slopes=slopes, lens=lens)


def _lengths(case):
    """(tokens in the cache, new tokens) of each sequence; the first has the longest of both."""
    rng = random.Random(case["lens"])
    kv = [case["kv_hi"]] + [rng.randint(case["kv_lo"], case["kv_hi"]) for _ in range(case["B"] - 1)]
    n = [case["q_hi"]] + [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(case["B"] - 1)]
    return kv, [min(a, b) for a, b in zip(n, kv)]


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import attention_sdpa_fwd_b200 as S
        s["cache"] = S.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    return s


def _inputs(case, seed):
    kv, n = _lengths(case)
    B, Hkv, d, page = case["B"], case["Hkv"], case["d"], case["page"]
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    pages = [-(-x // page) for x in kv]
    total, width = sum(pages), max(pages)
    pool = total + 3  # a few pages belong to nobody
    perm = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(B, width, dtype=torch.int32, device=dev)
    at = 0
    for b, m in enumerate(pages):
        table[b, :m] = perm[at:at + m]
        at += m
    io = _TORCH[case["io"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = dict(case=case, kv=kv, n=n, table=table, lens=torch.tensor(kv, dtype=torch.int32, device=dev),
             max_q=max(n), T=max(kv), k_scale=None, v_scale=None)
    s["cu"] = None if max(n) == 1 else torch.tensor([sum(n[:i]) for i in range(B + 1)], dtype=torch.int32, device=dev)
    # channels of a key differ in size, as do the values of different tokens
    chan = torch.exp(0.4 * normal(Hkv, 1, d))
    ct = _TORCH[case["cache"]]
    for x in ("k", "v"):
        y = normal(pool, Hkv, page, d)
        y = y * chan if x == "k" else y * torch.exp(0.4 * normal(pool, Hkv, page, 1))
        if case["cache"] in _QMAX:
            y, scale = _quantise(y, case["cache"])
            s[x + "_scale"] = scale
        s[x] = y.to(ct)
    if case["kind"] in ("write", "write_read"):
        s["k_new"] = (normal(sum(n), Hkv, d) * chan[:, 0]).to(io)
        s["v_new"] = (normal(sum(n), Hkv, d) * torch.exp(0.4 * normal(sum(n), Hkv, 1))).to(io)
    if case["kind"] in ("read", "write_read"):
        s["k_out"] = torch.zeros(B, Hkv, s["T"], d, dtype=io, device=dev)
        s["v_out"] = torch.zeros(B, Hkv, s["T"], d, dtype=io, device=dev)
    if case["kind"] == "attend":
        s["q"] = normal(sum(n), case["Hq"], d).to(io)
        s["slopes"] = None
        if case["slopes"]:
            s["slopes"] = torch.exp2(-8.0 * torch.arange(1, case["Hq"] + 1, device=dev) / case["Hq"])
    return s


# ------------------------------------------------------------------ plain forms
def _quantise(x, kind):
    """Codes (as the type) and scales of the rows of x, in 32 bits."""
    x = x.float()
    scale = (x.abs().amax(-1) / _QMAX[kind]).clamp_min(_FLOOR)
    y = x / scale[..., None]
    if kind == "int8":
        return y.round().clamp(-127, 127).to(torch.int8), scale
    return y.clamp(-448, 448).to(torch.float8_e4m3fn), scale


def _slots(s, b, lo, hi):
    """(page, offset) of tokens lo .. hi - 1 of sequence b."""
    t = torch.arange(lo, hi, device=s["table"].device)
    return s["table"][b].long()[t // s["case"]["page"]], t % s["case"]["page"]


def _tokens(s, x, b, lo, hi):
    """Keys or values of tokens lo .. hi - 1 of sequence b: [Hkv, tokens, d] in 32 bits."""
    p, o = _slots(s, b, lo, hi)
    y = s[x][p, :, o].float()
    if s[x + "_scale"] is not None:
        y = y * s[x + "_scale"][p, :, o][..., None]
    return y.transpose(0, 1)


def _write(s):
    at = 0
    for b, (L, n) in enumerate(zip(s["kv"], s["n"])):
        p, o = _slots(s, b, L - n, L)
        for x in ("k", "v"):
            rows = s[x + "_new"][at:at + n]
            if s[x + "_scale"] is None:
                s[x][p, :, o] = rows.to(s[x].dtype)
            else:
                c, scale = _quantise(rows, s["case"]["cache"])
                s[x].view(torch.uint8)[p, :, o] = c.view(torch.uint8)
                s[x + "_scale"][p, :, o] = scale
        at += n


def _read(s):
    for b, L in enumerate(s["kv"]):
        for x in ("k", "v"):
            s[x + "_out"][b, :, :L] = _tokens(s, x, b, 0, L).to(s[x + "_out"].dtype)
    return s["k_out"], s["v_out"]


def _attend(s):
    case = s["case"]
    G, d = case["Hq"] // case["Hkv"], case["d"]
    out = torch.empty_like(s["q"])
    at = 0
    for b, (L, n) in enumerate(zip(s["kv"], s["n"])):
        lo = max(0, L - n - case["window"] + 1) if case["window"] else 0
        k, v = _tokens(s, "k", b, lo, L), _tokens(s, "v", b, lo, L)
        q = s["q"][at:at + n].float().view(n, case["Hkv"], G, d).permute(1, 2, 0, 3)
        x = torch.matmul(q, k[:, None].transpose(2, 3)) * (1.0 / math.sqrt(d))
        if case["softcap"]:
            x = case["softcap"] * torch.tanh(x / case["softcap"])
        back = torch.arange(lo, L, device=x.device) - torch.arange(L - n, L, device=x.device)[:, None]
        if s["slopes"] is not None:
            x = x + s["slopes"].view(case["Hkv"], G, 1, 1) * back
        hidden = back > 0
        if case["window"]:
            hidden = hidden | (back <= -case["window"])
        x = x.masked_fill(hidden, float("-inf"))
        p = torch.exp(x - x.amax(-1, keepdim=True))
        y = torch.matmul(p, v[:, None]) / p.sum(-1, keepdim=True)
        out[at:at + n] = y.permute(2, 0, 1, 3).reshape(n, case["Hq"], d).to(out.dtype)
        at += n
    return out


def run(state):
    s = state
    kind = s["case"]["kind"]
    if own:
        import attention_sdpa_fwd_b200 as S
        if kind == "attend":
            c = s["case"]
            return S.sdpa_paged(s["q"], s["cache"], s["table"], s["lens"], s["cu"], max_q=s["max_q"], window=c["window"],
                                softcap=c["softcap"], slopes=s["slopes"])
        if kind in ("write", "write_read"):
            S.cache_write(s["cache"], s["k_new"], s["v_new"], s["table"], s["lens"], s["cu"], max_q=s["max_q"])
        if kind in ("read", "write_read"):
            return S.cache_read(s["cache"], s["table"], s["lens"], s["k_out"], s["v_out"])
    else:
        if kind == "attend":
            return _attend(s)
        if kind in ("write", "write_read"):
            _write(s)
        if kind in ("read", "write_read"):
            return _read(s)
    return s["k"], s["v"]


# ------------------------------------------------------------------ in 64 bits
def _to_grid(y, kind):
    """y (64 bits) to the nearest value of the 8-bit type, ties to even."""
    if kind == "int8":
        return torch.round(y).clamp(-127, 127)
    _, e = torch.frexp(y)                       # |y| in [2^(e-1), 2^e)
    step = torch.ldexp(torch.ones_like(y), (e - 1).clamp_min(-6) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def exact(case, seed):
    s = _inputs(case, seed)
    wide = {}
    for x in ("k", "v"):
        y = s[x].double()
        if s[x + "_scale"] is not None:
            y = y * s[x + "_scale"].double()[..., None]
        wide[x] = y
    page = case["page"]

    def rows(b, lo, hi):
        j = torch.arange(lo, hi, device="cuda")
        return s["table"][b, j // page].long(), j % page

    if case["kind"] in ("write", "write_read"):
        at = 0
        for b in range(case["B"]):
            L, n = s["kv"][b], s["n"][b]
            p, o = rows(b, L - n, L)
            for x in ("k", "v"):
                y = s[x + "_new"][at:at + n].double()
                if case["cache"] in _QMAX:
                    # scale and quotient are rounded to 32 bits by definition
                    sc = torch.clamp((y.abs().amax(-1, keepdim=True) / _QMAX[case["cache"]]).float().double(), min=_FLOOR)
                    y = _to_grid((y / sc).float().double(), case["cache"]) * sc
                wide[x][p, :, o] = y
            at += n
    if case["kind"] == "write":
        return wide["k"], wide["v"]
    if case["kind"] in ("read", "write_read"):
        res = []
        for x in ("k", "v"):
            z = torch.zeros(case["B"], case["Hkv"], s["T"], case["d"], dtype=torch.float64, device="cuda")
            for b in range(case["B"]):
                p, o = rows(b, 0, s["kv"][b])
                z[b, :, :s["kv"][b]] = wide[x][p, :, o].permute(1, 0, 2)
            res.append(z)
        return tuple(res)
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    out = torch.zeros(sum(s["n"]), Hq, d, dtype=torch.float64, device="cuda")
    at = 0
    for b in range(case["B"]):
        L, n = s["kv"][b], s["n"][b]
        first = 0 if not case["window"] else max(0, L - n + 1 - case["window"])
        p, o = rows(b, first, L)
        pos = torch.arange(L - n, L, device="cuda", dtype=torch.float64)[:, None]
        j = torch.arange(first, L, device="cuda", dtype=torch.float64)[None]
        seen = j <= pos
        if case["window"]:
            seen &= j > pos - case["window"]
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            x = (s["q"][at:at + n, h].double() / math.sqrt(d)) @ wide["k"][p, hk, o].T
            if case["softcap"]:
                x = torch.tanh(x / case["softcap"]) * case["softcap"]
            if s["slopes"] is not None:
                x = x + s["slopes"][h].double() * (j - pos)
            w = torch.softmax(torch.where(seen, x, -math.inf), dim=-1)
            out[at:at + n, h] = w @ wide["v"][p, hk, o]
        at += n
    return out


# ------------------------------------------------------------------ what a pass needs
def work(case):
    kv, n = _lengths(case)
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    io, ch = _BYTES[case["io"]], _BYTES[case["cache"]]
    row = 2 * Hkv * (d * ch + (4 if ch == 1 else 0))  # one token's keys and values in the cache
    new = 2 * Hkv * d * io
    pages = sum(-(-x // case["page"]) for x in kv)
    nbytes, flops = 4 * (pages + 2 * case["B"]), 0
    if case["kind"] in ("write", "write_read"):
        nbytes += sum(n) * (new + row)
        flops += 4 * sum(n) * 2 * Hkv * d
    if case["kind"] in ("read", "write_read"):
        nbytes += sum(kv) * (row + new)
        flops += sum(kv) * 2 * Hkv * d
    if case["kind"] == "attend":
        w = case["window"]
        pairs = keys = 0
        for L, m in zip(kv, n):
            first, last = L - m + 1, L  # keys the first and the last query see without a window
            if w:
                short = max(0, min(last, w) - first + 1)  # queries that see fewer than w keys, or w exactly
                pairs += short * (first + first + short - 1) // 2 + (m - short) * w
                keys += min(L, m - 1 + w)
            else:
                pairs += m * (first + last) // 2
                keys += L
        nbytes += 2 * sum(n) * Hq * d * io + keys * row
        flops += 4 * d * Hq * pairs
    return {"bytes": nbytes, "flops": flops}
