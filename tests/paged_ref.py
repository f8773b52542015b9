"""The paged cache operators in 64 bits on the CPU, from their definitions, and
the bounds their tests hold the kernels to."""
from __future__ import annotations

import math

import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
QMAX = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}


def quantise(x, dtype):
    """(codes as 64-bit numbers, scales) of the rows of x; the scale and the
    quotient are rounded to 32 bits by definition, the code to the type."""
    x = x.double()
    s = torch.clamp((x.abs().amax(-1) / QMAX[dtype]).float().double(), min=2.0 ** -30)
    y = (x / s[..., None]).float().double()
    if dtype == torch.int8:
        return torch.round(y).clamp(-127, 127), s
    _, e = torch.frexp(y)
    step = torch.ldexp(torch.ones_like(y), (e - 1).clamp_min(-6) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448), s


class Pool:
    """A batch's cache on the CPU: values in 64 bits, pages in random order,
    every row the batch's tokens do not cover filled with NaN (INT8: NaN
    scales)."""

    def __init__(self, dtype, Hkv, d, page, kv, seed=0, spare=2, garbage=True):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.Hkv, self.d, self.page, self.kv = dtype, Hkv, d, page, list(kv)
        pages = [-(-x // page) for x in kv]
        n = sum(pages) + spare
        order = torch.randperm(n, generator=g).int()
        self.table = torch.full((len(kv), max(pages + [1])), -1, dtype=torch.int32)
        live = torch.zeros(n, page, dtype=torch.bool)
        at = 0
        for b, m in enumerate(pages):
            self.table[b, :m] = order[at:at + m]
            at += m
            for i in range(m):
                live[self.table[b, i].long(), :kv[b] - i * page] = True
        k = torch.randn(n, Hkv, page, d, generator=g) * torch.exp(0.5 * torch.randn(Hkv, 1, d, generator=g))
        v = torch.randn(n, Hkv, page, d, generator=g) * torch.exp(torch.randn(n, Hkv, page, 1, generator=g))
        live4 = live[:, None, :, None]
        self.raw = []      # what the device cache holds
        self.scales = []
        self.val = []      # what it stands for, 64 bits
        for x in (k, v):
            if dtype in QMAX:
                c, s = quantise(x, dtype)
                self.val.append(c * s[..., None])
                c = c.float()
                s = s.float()
                if garbage:
                    if dtype == torch.float8_e4m3fn:
                        c = torch.where(live4, c, torch.full((), math.nan))
                    s = torch.where(live[:, None], s, torch.full((), math.nan))
                self.raw.append(c.to(dtype))
                self.scales.append(s)
            else:
                r = x.to(dtype)
                self.val.append(r.double())
                if garbage:
                    r = torch.where(live4, r, torch.full((), math.nan, dtype=dtype))
                self.raw.append(r)
        self.lens = torch.tensor(self.kv, dtype=torch.int32)

    def cache(self, layout="hnd"):
        """The device cache; "nhd" keeps it as [pages, page, Hkv, d]."""
        import attention_sdpa_fwd_b200 as S

        def put(t):
            if layout == "nhd":
                raw = t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
                r = raw.transpose(1, 2).contiguous().cuda().transpose(1, 2)
                return r.view(t.dtype) if t.dtype == torch.float8_e4m3fn else r
            return t.cuda()
        return S.KVCache(*(put(t) for t in self.raw + self.scales))

    def tokens(self, which, b, hi=None):
        """[Hkv, tokens, d] in 64 bits."""
        j = torch.arange(self.kv[b] if hi is None else hi)
        return self.val[which][self.table[b, j // self.page].long(), :, j % self.page].transpose(0, 1)


def attend(pool, q, n, *, scale=None, window=0, softcap=0.0, slopes=None, u_p=0.0, p_floor=0.0, u_kv=0.0):
    """(out, lse, bound on |out|'s error without its own rounding, bound on
    lse's) in 64 bits for packed rows q [sum n, Hq, d].

    The bound: a score's error e is that of d fp32 products and sums (taken as
    twice a rounding each: tensor cores may cut instead of rounding), of
    the few operations behind them and of exp2 (2^-22); a weight is off by a
    factor e^(+-e) and by u_p where P is rounded; the value sum adds its own
    accumulation, one rounding per 8 keys and a few.

    p_floor: where P is f16 a weight below f16's normal range is off by half
    its smallest number whatever its size.  In units of P that is 2^-25, with
    the largest P at 2^12 or more: 2^-37 of the largest.  P there stands for
    2^t, t_j = x_j log2 e + log2 vs_j, and multiplies codes c_j, so the sum of
    p_j c_j is off by at most p_floor 2^tmax sum |c_j|; it is divided by sum
    2^t_j / vs_j >= 2^tmax / vs_(argmax t): p_floor vs_(argmax t) sum |c_j|.

    u_kv: where dequantised keys and values are rounded to f16 (codes times a
    scale relative to a power of two of 32 keys).  A score is off by u_kv scale
    sum |q k| more, the value sum by u_kv sum p |v|.  P then multiplies
    v_j 2^-ev_j, with 2^ev_j at most the largest scale of j's 32 keys / 64 and
    at least vs_j / 128, so the floor's share is at most p_floor 2^ev sum |v_j|
    2^-ev_j <= p_floor (max vs / 64) sum 128 |c_j| = 2 p_floor max vs sum |c_j|.
    (A value below 2^-30 of its 32 keys' largest is off by 2^-40 of that largest
    at most, which the fp32 terms cover.)"""
    T, Hq, d = q.shape
    q = q.double()
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    G = Hq // pool.Hkv
    out = torch.zeros(T, Hq, d, dtype=torch.float64)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    tol = torch.zeros(T, Hq, d, dtype=torch.float64)
    ltol = torch.zeros(T, Hq, dtype=torch.float64)
    at = 0
    for b, m in enumerate(n):
        L = pool.kv[b]
        if m and L:
            k, v = pool.tokens(0, b), pool.tokens(1, b)
            pos = torch.arange(L - m, L)[:, None]
            j = torch.arange(L)[None]
            hidden = j > pos
            if window:
                hidden = hidden | (j <= pos - window)
            for h in range(Hq):
                kk, vv = k[h // G], v[h // G]
                qq = q[at:at + m, h]
                x = qq @ kk.T * scale
                size = (qq.abs() @ kk.abs().T) * abs(scale)
                if softcap:
                    x = softcap * torch.tanh(x / softcap)
                if slopes is not None:
                    x = x + slopes[h].double() * (j - pos)
                e = u_kv * size + 2.0 ** -23 * ((d + 8) * size + 8 * x.abs() + 4 * softcap + 4)
                x = x.masked_fill(hidden, -math.inf)
                top = x.amax(-1, keepdim=True)
                ok = torch.isfinite(top[:, 0])
                p = torch.exp(x - torch.where(torch.isfinite(top), top, torch.zeros(())))
                den = p.sum(-1, keepdim=True)
                p = torch.where(ok[:, None], p / den, torch.zeros(()))
                out[at:at + m, h] = p @ vv
                lse[at:at + m, h] = torch.where(ok, top[:, 0] + den[:, 0].log(), torch.full((), -math.inf))
                pe = p * (2 * e)
                acc = (L / 8 + 64) * 2.0 ** -23
                tol[at:at + m, h] = (pe + (u_p + u_kv + acc) * p) @ vv.abs() + (pe.sum(-1, keepdim=True) + acc) * out[at:at + m, h].abs()
                if p_floor:
                    vs = pool.scales[1].double()[pool.table[b, j[0] // pool.page].long(), h // G, j[0] % pool.page]
                    t = x / math.log(2.0) + vs.log2()
                    size_c = (~hidden).double() @ (vv / vs[:, None]).abs()
                    top_vs = 2 * vs.max() if u_kv else vs[t.argmax(-1)][:, None]
                    tol[at:at + m, h] += p_floor * top_vs * size_c
                ltol[at:at + m, h] = pe.sum(-1) + acc + 2.0 ** -22 * lse[at:at + m, h].abs().nan_to_num(posinf=0)
        at += m
    return out, lse, tol, ltol


def check(got, want, tol, dtype, what=""):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    bound = tol + U[dtype] * (want.abs() + tol) + 1e-30
    worst = ((got - want).abs() / bound).max().item() if got.numel() else 0.0
    assert worst <= 1.0, f"{what}: error {worst:.2f} times the bound, {(got - want).abs().max().item():.3e} at most"
    return worst


def check_lse(got, want, tol, what=""):
    got = got.double().cpu()
    dead = torch.isinf(want)
    assert torch.equal(got[dead], want[dead]), f"{what}: rows without keys"
    assert ((got - want).abs()[~dead] <= tol[~dead] + 1e-6).all(), f"{what}: lse"
