"""Soft caps of every size: c tanh(x / c) against its value in 64 bits on each
kernel family, from caps far above the scores (tanh is all but the identity)
to caps far below them (a sign).

The bound: a score's own error is that of ``paged_ref.attend``'s formula
without its cap term.  The cap multiplies it by at most 1 (its slope) and adds
its evaluation.  Where c <= 128 that is c - 2 c / (1 + 2^w): the exponential is
off by 2^-22 and by w's three roundings, the reciprocal by 2^-23, the sum by
2^-24, a reciprocal shared by four by six roundings more; the term is at most
c there, so 2^-19 c holds them.  Above 128 it is a polynomial where |x| <= c / 3
(2^-22.7 cut off, a few roundings) and that formula beyond, c < 3.2 of what
comes out: 2^-19 |c tanh(x / c)| holds both.
"""
from __future__ import annotations

import itertools
import math

import pytest
import torch

import attention_sdpa_fwd_b200 as S
import paged_ref as R

pytestmark = pytest.mark.gpu

F32, BF16, E4M3, INT8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn, torch.int8
CAPS = [1e-40, 1e-30, 1e-3, 30.0, 128.0, 128.5, 1e3, 1e4, 1e6, 1e30, 3e38]


def attend(pool, q, n, cap, slopes, u_p, p_floor, u_kv):
    """(out, lse, bounds on both), as paged_ref.attend with the cap's own bound."""
    T, Hq, d = q.shape
    q, scale, G = q.double(), 1.0 / math.sqrt(d), Hq // pool.Hkv
    out, tol = (torch.zeros(T, Hq, d, dtype=torch.float64) for _ in range(2))
    lse, ltol = (torch.zeros(T, Hq, dtype=torch.float64) for _ in range(2))
    at = 0
    for b, m in enumerate(n):
        L = pool.kv[b]
        k, v = pool.tokens(0, b), pool.tokens(1, b)
        pos, j = torch.arange(L - m, L)[:, None], torch.arange(L)
        hidden = j > pos
        for h in range(Hq):
            rows = slice(at, at + m)
            kk, vv = k[h // G], v[h // G]
            size = (q[rows, h].abs() @ kk.abs().T) * scale
            raw = q[rows, h] @ kk.T * scale
            x = cap * torch.tanh(raw / cap)
            e = u_kv * size + 2.0 ** -23 * ((d + 8) * size + 8 * raw.abs() + 4)
            # no error of a score moves a capped one by more than the cap's width
            e = e.clamp_max(2 * cap) + 2.0 ** -19 * (cap if cap <= 128 else x.abs())
            if slopes is not None:
                x = x + slopes[h].double() * (j - pos)
                e = e + 2.0 ** -23 * 8 * x.abs()
            x = x.masked_fill(hidden, -math.inf)
            top = x.amax(-1, keepdim=True)
            p = torch.exp(x - top)
            den = p.sum(-1, keepdim=True)
            p = p / den
            e = e + 2.0 ** -22 * (x - top).abs().nan_to_num(posinf=0) + 2.0 ** -21
            out[rows, h] = p @ vv
            lse[rows, h] = top[:, 0] + den[:, 0].log()
            pe = p * (2 * e)
            acc = (L / 8 + 64) * 2.0 ** -23
            tol[rows, h] = (pe + (u_p + u_kv + acc) * p) @ vv.abs() + (pe.sum(-1, keepdim=True) + acc) * out[rows, h].abs()
            if p_floor:
                vs = pool.scales[1].double()[pool.table[b, j // pool.page].long(), h // G, j % pool.page]
                t = x / math.log(2.0) + vs.log2()
                top_vs = 2 * vs.max() if u_kv else vs[t.argmax(-1)][:, None]
                tol[rows, h] += p_floor * top_vs * ((~hidden).double() @ (vv / vs[:, None]).abs())
            ltol[rows, h] = pe.sum(-1) + acc + 2.0 ** -22 * lse[rows, h].abs()
        at += m
    return out, lse, tol, ltol


PATHS = [("exact", F32, F32), ("exact", BF16, BF16), ("exact", E4M3, BF16)] + \
    list(itertools.product(("decode", "tcgen05"), (BF16, E4M3, INT8), (BF16,)))


@pytest.mark.parametrize("cap", CAPS, ids=str)
@pytest.mark.parametrize("path,cdt,io", PATHS, ids=str)
@pytest.mark.parametrize("d", [64, 128])
def test_caps_of_every_size(d, path, cdt, io, cap):
    """Scores of a few, and of some hundred (past c / 3 of the middle caps); one
    key, a few, several tiles; a row of zeros."""
    kv, n = [1, 9, 300, 130], [1, 3, 4, 4]
    pool = R.Pool(cdt, 2, d, 16, kv, seed=d)
    sl = torch.tensor([0.0, 0.5, -0.01, 0.25])
    codes = cdt in R.QMAX
    rounded = path != "exact"
    for std, slopes in ((1.0, None), (60.0, None), (1.0, sl)):
        q = (torch.randn(sum(n), 4, d, generator=torch.Generator().manual_seed(int(std))) * std)
        q[2] = 0
        q = q.to(io)
        lse = torch.empty(sum(n), 4, device="cuda")
        cu = torch.tensor([0] + list(itertools.accumulate(n)), dtype=torch.int32, device="cuda")
        out = S.sdpa_paged(q.cuda(), pool.cache(), pool.table.cuda(), pool.lens.cuda(), cu, max_q=4, softcap=cap, lse=lse,
                           slopes=None if slopes is None else slopes.cuda(), path=path)
        torch.cuda.synchronize()
        assert S.sdpa_last_device_error(torch.cuda.current_stream().cuda_stream) == 0
        want, wlse, tol, ltol = attend(pool, q, n, cap, slopes, R.U[torch.float16 if codes else BF16] if rounded else 0.0,
                                       2.0 ** -37 if rounded and codes else 0.0,
                                       R.U[torch.float16] if codes and path == "tcgen05" else 0.0)
        what = f"{path} {cdt} d{d} cap {cap} std {std} slopes {slopes is not None}"
        R.check(out, want, tol, io, what)
        R.check_lse(lse, wlse, ltol, what)
