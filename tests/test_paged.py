"""The paged cache operators on the GPU against their definitions in 64 bits."""
from __future__ import annotations

import itertools
import math

import pytest
import torch

import attention_sdpa_fwd_b200 as S
import paged_ref as R

pytestmark = pytest.mark.gpu

F32, BF16, E4M3, INT8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn, torch.int8


def device_error():
    torch.cuda.synchronize()
    return S.sdpa_last_device_error(torch.cuda.current_stream().cuda_stream)


def cu(n):
    return torch.tensor([0] + list(itertools.accumulate(n)), dtype=torch.int32, device="cuda")


def bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]).cpu()


# ------------------------------------------------------------------ write and read
WRITES = [  # cache, io, Hkv, d, page, tokens, new rows (None: one each, without cu_q)
    (BF16, BF16, 8, 128, 16, [20, 1, 300], None),
    (BF16, BF16, 1, 64, 5, [7, 64, 1], [7, 3, 1]),
    (F32, F32, 3, 16, 16, [33, 16], [17, 0]),
    (E4M3, BF16, 8, 128, 32, [500, 31, 1], [100, 0, 1]),
    (E4M3, F32, 2, 64, 7, [40, 9], [40, 9]),
    (INT8, BF16, 12, 64, 64, [129, 4], [66, 4]),
    (INT8, F32, 1, 16, 1, [11], [5]),
    (E4M3, BF16, 2, 16, 128, [1000], [999]),
]


@pytest.mark.parametrize("layout", ["hnd", "nhd"])
@pytest.mark.parametrize("cdt,io,Hkv,d,page,kv,n", WRITES)
def test_write_then_read(cdt, io, Hkv, d, page, kv, n, layout):
    pool = R.Pool(cdt, Hkv, d, page, kv, seed=3)
    cache = pool.cache(layout)
    before = [bits(t).clone() for t in (cache.k, cache.v)]
    rows = n if n is not None else [1] * len(kv)
    g = torch.Generator().manual_seed(9)
    new = [(torch.randn(sum(rows) + 2, Hkv, d, generator=g) * 3).to(io) for _ in range(2)]  # two rows belong to nobody
    new[0][0] = 0
    if sum(rows) > 2:
        new[1][1] *= 1e-12   # below the floor of the scale
        new[1][2] *= 1e12
    dev = [x.cuda() for x in new]
    if n is None:
        dev = [x[:-2] for x in dev]
    S.cache_write(cache, dev[0], dev[1], pool.table.cuda(), pool.lens.cuda(), None if n is None else cu(n),
                  max_q=max(rows))
    assert device_error() == 0
    for w, (raw, old) in enumerate(zip((cache.k, cache.v), before)):
        got = bits(raw)
        touched = torch.zeros(got.shape[0], page, dtype=torch.bool)
        at = 0
        for b, m in enumerate(rows):
            for i in range(m):
                j = kv[b] - m + i
                p, o = pool.table[b, j // page].long(), j % page
                touched[p, o] = True
                x = new[w][at + i]
                if cdt in R.QMAX:
                    c, s = R.quantise(x, cdt)
                    assert torch.equal(bits(c.float().to(cdt)), got[p, :, o]) or \
                        torch.equal(c, raw[p, :, o].cpu().double()), "codes"
                    sc = (cache.k_scale, cache.v_scale)[w][p, :, o].cpu()
                    assert torch.equal(sc, s.float()), "scales"
                else:
                    assert torch.equal(bits(x.to(cdt)), got[p, :, o])
            at += m
        keep = ~touched[:, None, :, None].expand_as(got)
        assert torch.equal(got[keep], old[keep]), "rows of other tokens changed"
    # read back: values of the codes, one rounding; rows past the tokens kept
    out = F32 if cdt in R.QMAX and io == F32 else (cdt if cdt not in R.QMAX else BF16)
    T = max(kv) + 3
    if layout == "nhd":
        ko, vo = (torch.full((len(kv), T, Hkv, d), 7.0, dtype=out, device="cuda").transpose(1, 2) for _ in range(2))
    else:
        ko, vo = (torch.full((len(kv), Hkv, T, d), 7.0, dtype=out, device="cuda") for _ in range(2))
    S.cache_read(cache, pool.table.cuda(), pool.lens.cuda(), ko, vo)
    assert device_error() == 0
    for raw, sc, o in ((cache.k, cache.k_scale, ko), (cache.v, cache.v_scale, vo)):
        full = raw.cpu().float()
        if sc is not None:
            full = full * sc.cpu()[..., None]
        for b, L in enumerate(kv):
            j = torch.arange(L)
            want = full[pool.table[b, j // page].long(), :, j % page].transpose(0, 1).to(out)
            got = o[b, :, :L].cpu()
            assert torch.equal(bits(want.contiguous()), bits(got.contiguous())) or \
                torch.equal(want.nan_to_num(), got.nan_to_num())
            assert (o[b, :, L:] == 7).all()


def test_write_odd_strides_and_infinities():
    """Sources and pools that no 16-byte access fits; NaN and infinities in a row."""
    pool = R.Pool(INT8, 2, 64, 16, [30], seed=1)
    base = torch.zeros(4, 2 * 2 * 64 + 1, dtype=BF16, device="cuda")
    k = torch.as_strided(base, (4, 2, 64), (base.stride(0), 64, 1), 1)
    k.copy_(torch.randn(4, 2, 64))
    v = torch.randn(4, 2, 64, device="cuda").to(BF16)
    v[1, 0, 3] = math.inf
    v[2, 1, 5] = math.nan
    cache = pool.cache()
    wide = torch.zeros(cache.k.shape[0], 2, 16, 65, dtype=INT8, device="cuda")
    cache = S.KVCache(wide[..., :64], cache.v, cache.k_scale, cache.v_scale)
    S.cache_write(cache, k, v, pool.table.cuda(), pool.lens.cuda(), cu([4]), max_q=4)
    assert device_error() == 0
    for i in range(4):
        p, o = pool.table[0, (26 + i) // 16].long(), (26 + i) % 16
        c, s = R.quantise(k[i].cpu(), INT8)
        assert torch.equal(cache.k[p, :, o].cpu().double(), c)
        assert (wide[p, :, o, 64] == 0).all()
    p, o = pool.table[0, 27 // 16].long(), 27 % 16
    assert torch.isinf(cache.v_scale[p, 0, o]) and (cache.v[p, 0, o] == 0).all()
    p, o = pool.table[0, 28 // 16].long(), 28 % 16
    x = v[2, 1].cpu().clone()
    x[5] = 0
    c, s = R.quantise(x, INT8)
    assert torch.equal(cache.v[p, 1, o].cpu().double(), c) and cache.v_scale[p, 1, o].item() == s.item()


# ------------------------------------------------------------------ attention
def run_case(path, cdt, io, Hq, Hkv, d, page, kv, n, *, layout="hnd", window=0, softcap=0.0, slopes=False, seed=0,
             scale=None, qstd=1.0, **kw):
    pool = R.Pool(cdt, Hkv, d, page, kv, seed=seed)
    rows = n if n is not None else [1] * len(kv)
    g = torch.Generator().manual_seed(seed + 100)
    q = (torch.randn(sum(rows), Hq, d, generator=g) * qstd).to(io)
    sl = 2.0 ** (-8.0 * torch.arange(1, Hq + 1) / Hq) if slopes else None
    lse = torch.empty(sum(rows), Hq, device="cuda")
    out = S.sdpa_paged(q.cuda(), pool.cache(layout), pool.table.cuda(), pool.lens.cuda(), None if n is None else cu(n),
                       scale, max_q=max(rows + [0]), window=window, softcap=softcap,
                       slopes=None if sl is None else sl.cuda(), lse=lse, path=path, **kw)
    assert device_error() == 0
    codes = cdt in R.QMAX
    rounded = path != "exact" and io == BF16  # P is f16 beside codes, else bf16
    want, wlse, tol, ltol = R.attend(pool, q, rows, scale=scale, window=window, softcap=softcap, slopes=sl,
                                     u_p=R.U[torch.float16 if codes else BF16] if rounded else 0.0,
                                     p_floor=2.0 ** -37 if rounded and codes else 0.0,
                                     u_kv=R.U[torch.float16] if codes and path in ("tcgen05", "auto") and io == BF16 else 0.0)
    what = f"{path} {cdt} {Hq}/{Hkv} d{d} page {page} kv {kv} n {n} w{window} c{softcap} s{slopes}"
    R.check(out, want, tol, io, what)
    R.check_lse(lse, wlse, ltol, what)
    return out


TYPES = [(F32, F32), (BF16, BF16), (E4M3, BF16), (INT8, BF16), (E4M3, F32), (INT8, F32)]


@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("cdt,io", TYPES)
def test_exact_every_type(cdt, io, d):
    run_case("exact", cdt, io, 6, 2, d, 16, [1, 17, 200, 33], [1, 5, 2, 33], seed=d)
    run_case("exact", cdt, io, 3, 3, d, 7, [40, 1, 130], None, seed=d + 1, layout="nhd")


@pytest.mark.parametrize("kw", [dict(window=1), dict(window=20), dict(window=1000), dict(softcap=5.0),
                                dict(slopes=True), dict(window=30, softcap=20.0, slopes=True),
                                dict(scale=0.0), dict(scale=-0.3), dict(qstd=30.0)])
@pytest.mark.parametrize("cdt", [BF16, E4M3])
def test_exact_options(cdt, kw):
    run_case("exact", cdt, BF16, 4, 2, 64, 16, [100, 31, 64], [10, 31, 1], **kw)


def test_exact_more_rows_than_tokens():
    """New rows in front of the sequence's first token see nothing: zero, -inf."""
    run_case("exact", BF16, BF16, 4, 2, 64, 16, [3, 0, 20], [5, 2, 4])


# lengths around the tiles (64 or 128 keys to a CTA's tile, 16 or 32 to a warp's step), one sequence and many
DECODE_LENS = [[1], [2, 15, 16, 17], [31, 33, 63, 64, 65], [127, 128, 129, 500], [3000, 1, 0, 777], [9000]]


@pytest.mark.parametrize("kv", DECODE_LENS, ids=str)
@pytest.mark.parametrize("cdt", [BF16, E4M3, INT8])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_lengths(d, cdt, kv):
    run_case("decode", cdt, BF16, 8, 2, d, 16, kv, None, seed=len(kv))


@pytest.mark.parametrize("Hq,Hkv,n", [(1, 1, [1, 1, 1]), (32, 1, [1, 1, 1]), (7, 1, [2, 1, 2]), (12, 12, [9, 1, 16]),
                                      (24, 3, [4, 2, 3]), (6, 2, [5, 0, 10]), (16, 1, [1, 2, 1]), (32, 2, [1, 0, 1])])
@pytest.mark.parametrize("cdt", [BF16, E4M3, INT8])
@pytest.mark.parametrize("d,page,layout", [(128, 48, "hnd"), (64, 32, "nhd")])
def test_decode_rows(d, page, layout, cdt, Hq, Hkv, n):
    run_case("decode", cdt, BF16, Hq, Hkv, d, page, [700, 20, 260], n, layout=layout, seed=Hq)


OPTIONS = [dict(window=1), dict(window=17), dict(window=100), dict(window=100000), dict(softcap=5.0), dict(slopes=True),
           dict(window=200, softcap=20.0, slopes=True), dict(scale=0.0), dict(scale=-0.3), dict(qstd=30.0)]


@pytest.mark.parametrize("kw", OPTIONS, ids=str)
@pytest.mark.parametrize("n", [[1, 1, 1], [6, 3, 8]], ids=str)
@pytest.mark.parametrize("cdt", [BF16, E4M3, INT8])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_options(d, cdt, n, kw):
    run_case("decode", cdt, BF16, 8, 4, d, 16, [1000, 131, 64], n, seed=d, **kw)


def test_decode_many_sequences():
    """More sequences than a CTA has threads, most of them empty or short."""
    kv = [(i * 37) % 90 if i % 3 else 0 for i in range(300)]
    run_case("decode", BF16, BF16, 4, 2, 64, 16, kv, [1 if i % 5 else 0 for i in range(300)])


def test_decode_more_rows_than_tokens():
    run_case("decode", E4M3, BF16, 4, 2, 64, 16, [3, 0, 200], [5, 2, 4])


@pytest.mark.parametrize("cdt", [BF16, INT8])
def test_decode_equals_itself_and_any_split(cdt):
    """The same call twice gives the same bits."""
    a = run_case("decode", cdt, BF16, 8, 2, 128, 16, [5000, 300], None)
    b = run_case("decode", cdt, BF16, 8, 2, 128, 16, [5000, 300], None)
    assert torch.equal(a, b)


# ------------------------------------------------------------------ chunks on the tensor cores
CHUNKS = [([1], [1]), ([128], [128]), ([129, 300], [129, 1]), ([1000], [100]), ([257, 40, 0, 640], [200, 40, 0, 3]),
          ([2000], [17]), ([513], [513])]


@pytest.mark.parametrize("kv,n", CHUNKS, ids=str)
@pytest.mark.parametrize("cdt", [BF16, E4M3, INT8])
@pytest.mark.parametrize("d", [64, 128])
def test_chunk_lengths(d, cdt, kv, n):
    run_case("tcgen05", cdt, BF16, 8, 2, d, 32, kv, n, seed=len(kv))


@pytest.mark.parametrize("Hq,Hkv,page,layout", [(2, 2, 16, "hnd"), (3, 1, 48, "nhd"), (12, 4, 256, "hnd"), (7, 1, 128, "hnd"),
                                                (8, 1, 64, "nhd"), (40, 1, 80, "hnd"), (100, 1, 16, "hnd"), (128, 1, 32, "hnd")])
@pytest.mark.parametrize("cdt", [BF16, E4M3, INT8])
@pytest.mark.parametrize("d", [64, 128])
def test_chunk_heads_and_pages(d, cdt, Hq, Hkv, page, layout):
    run_case("tcgen05", cdt, BF16, Hq, Hkv, d, page, [300, 77], [150, 30], layout=layout, seed=Hq)


@pytest.mark.parametrize("kw", OPTIONS, ids=str)
@pytest.mark.parametrize("cdt", [BF16, E4M3, INT8])
@pytest.mark.parametrize("d", [64, 128])
def test_chunk_options(d, cdt, kw):
    run_case("tcgen05", cdt, BF16, 8, 4, d, 16, [1000, 131, 400], [200, 131, 30], seed=d, **kw)


@pytest.mark.parametrize("cdt", [BF16, E4M3])
def test_chunk_more_rows_than_tokens(cdt):
    run_case("tcgen05", cdt, BF16, 4, 2, 64, 16, [3, 0, 200], [150, 20, 220])


@pytest.mark.parametrize("cdt", [BF16, E4M3, INT8])
@pytest.mark.parametrize("d", [64, 128])
def test_auto_mixed(d, cdt):
    """Single tokens, drafts and chunks of one batch: two kernels share it."""
    run_case("auto", cdt, BF16, 8, 2, d, 16, [700, 65, 0, 300, 128, 1000], [1, 5, 0, 120, 128, 9], seed=7)


# ------------------------------------------------------------------ what the kernels check
def bad_batch(path, *, table=None, lens=None, cuq=None, max_q=2):
    pool = R.Pool(BF16, 2, 64, 16, [100, 60], seed=2, garbage=False)
    q = torch.randn(4, 8, 64, device="cuda").to(BF16)
    t, l, c = pool.table.clone(), pool.lens.clone(), torch.tensor([0, 2, 4], dtype=torch.int32)
    for x, change in ((t, table), (l, lens), (c, cuq)):
        for at, v in (change or {}).items():
            x[at] = v
    S.sdpa_paged(q, pool.cache(), t.cuda(), l.cuda(), c.cuda(), max_q=max_q, path=path)
    return device_error()


@pytest.mark.parametrize("path", ["exact", "decode", "tcgen05"])
@pytest.mark.parametrize("kw", [dict(table={(0, 1): 10 ** 6}), dict(table={(1, 3): -5}), dict(lens={0: -1}),
                                dict(lens={1: 10 ** 9}), dict(cuq={1: 5}), dict(cuq={1: -1}), dict(cuq={2: 1}),
                                dict(cuq={2: 400}), dict(max_q=1)], ids=str)
def test_bad_device_values_are_reported(path, kw):
    """Pages, lengths and ranges only the kernels see: an error word, nothing else."""
    assert bad_batch(path) == 0
    assert bad_batch(path, **kw) == -7
    assert bad_batch(path) == 0


@pytest.mark.parametrize("cdt", [BF16, E4M3, INT8])
@pytest.mark.parametrize("path", ["decode", "tcgen05"])
def test_tiny_and_huge_rows(path, cdt):
    """Rows of q at the ends of the range, an all-zero one, a tiny scale, masked
    keys beside them; a window no sequence can leave, and the largest."""
    pool = R.Pool(cdt, 2, 64, 16, [70, 140], seed=11)
    n = [3, 2]
    q = torch.randn(5, 8, 64, generator=torch.Generator().manual_seed(5))
    q[0] *= 1e-37
    q[1] = 0
    q[2] *= 3e4
    q = q.to(BF16)
    codes = cdt in R.QMAX
    for kw in (dict(), dict(scale=1e-38), dict(window=2 ** 31 - 1), dict(window=140), dict(window=139)):
        out = S.sdpa_paged(q.cuda(), pool.cache(), pool.table.cuda(), pool.lens.cuda(), cu(n), max_q=3, path=path, **kw)
        assert device_error() == 0
        want, _, tol, _ = R.attend(pool, q, n, u_p=R.U[torch.float16 if codes else BF16],
                                   p_floor=2.0 ** -37 if codes else 0.0,
                                   u_kv=R.U[torch.float16] if codes and path == "tcgen05" else 0.0, **kw)
        R.check(out, want, tol, BF16, f"{path} {cdt} {kw}")


def test_entries_past_the_tokens_are_not_read():
    """Table entries behind a sequence's tokens, and in front of its window, may be anything."""
    for path in ("exact", "decode", "tcgen05"):
        for cdt in (BF16, E4M3):
            pool = R.Pool(cdt, 2, 64, 16, [1000], seed=4)
            q = torch.randn(3, 4, 64, generator=torch.Generator().manual_seed(1)).to(BF16)
            a = S.sdpa_paged(q.cuda(), pool.cache(), pool.table.cuda(), pool.lens.cuda(), cu([3]), max_q=3, window=50, path=path)
            t = torch.full((1, 90), -7, dtype=torch.int32)
            first = (1000 - 3 + 1 - 50) // 16
            t[0, first:63] = pool.table[0, first:63]
            b = S.sdpa_paged(q.cuda(), pool.cache(), t.cuda(), pool.lens.cuda(), cu([3]), max_q=3, window=50, path=path)
            assert device_error() == 0
            u_p = 0.0 if path == "exact" else R.U[torch.float16 if cdt == E4M3 else BF16]
            want, _, tol, _ = R.attend(pool, q, [3], window=50, u_p=u_p, p_floor=2.0 ** -37 if cdt == E4M3 else 0.0,
                                       u_kv=2.0 ** -11 if cdt == E4M3 else 0.0)
            R.check(a, want, tol, BF16, f"{path} {cdt}")
            R.check(b, want, tol, BF16, f"{path} {cdt} with freed pages")


def test_bad_write_and_read_are_reported():
    pool = R.Pool(E4M3, 2, 64, 16, [100, 60], seed=2, garbage=False)
    x = torch.randn(4, 2, 64, device="cuda").to(BF16)
    for change in (lambda t, l, c: t.__setitem__((0, 6), 99), lambda t, l, c: l.__setitem__(1, 1),
                   lambda t, l, c: l.__setitem__(0, 10 ** 6), lambda t, l, c: c.__setitem__(2, 9)):
        t, l, c = pool.table.clone(), pool.lens.clone(), torch.tensor([0, 2, 4], dtype=torch.int32)
        change(t, l, c)
        S.cache_write(pool.cache(), x, x, t.cuda(), l.cuda(), c.cuda(), max_q=2)
        assert device_error() == -7
    t = pool.table.clone()
    t[0, 2] = -1
    S.cache_read(pool.cache(), t.cuda(), pool.lens.cuda(), T=100)
    assert device_error() == -7


# ------------------------------------------------------------------ together, as they are used
@pytest.mark.parametrize("cdt", [BF16, E4M3, INT8])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_then_decode_equals_dense(d, cdt):
    """A prompt written in two chunks, then token by token, attended at each
    step, against dense causal attention (``sdpa``) of what the cache holds,
    read back; 8-bit caches and the dense call round keys, values and weights
    each their own way: 2^-8 for every bf16 rounding there is."""
    Hq, Hkv, page, n = 8, 2, 16, [150, 61]
    g = torch.Generator().manual_seed(3)
    total = [x + 5 for x in n]
    k, v, q = (torch.randn(2, max(total), h, d, generator=g).to(BF16).cuda() for h in (Hkv, Hkv, Hq))
    cache = S.KVCache.empty(40, page, Hkv, d, cdt)
    table = torch.randperm(40, generator=g).int()[:24].view(2, 12).cuda()
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    got = torch.zeros(2, max(total), Hq, d, dtype=BF16, device="cuda")
    done = [0, 0]
    steps = [[100, 20], [50, 41]] + [[1, 1]] * 5
    for step in steps:
        rows = [slice(a, a + m) for a, m in zip(done, step)]
        cat = lambda t: torch.cat([t[b, r] for b, r in enumerate(rows)])
        lens += torch.tensor(step, dtype=torch.int32, device="cuda")
        single = step == [1, 1]
        args = (table, lens, None if single else cu(step))
        S.cache_write(cache, cat(k), cat(v), *args, max_q=max(step))
        out = S.sdpa_paged(cat(q), cache, *args, max_q=max(step))
        at = 0
        for b, (r, m) in enumerate(zip(rows, step)):
            got[b, r] = out[at:at + m]
            at += m
            done[b] += m
    kd, vd = S.cache_read(cache, table, lens, T=max(total))
    want = S.sdpa(q.transpose(1, 2), kd, vd, mask_kind=S.MASK_CAUSAL).transpose(1, 2)
    assert device_error() == 0
    size = S.sdpa(q.transpose(1, 2), kd, vd.abs(), mask_kind=S.MASK_CAUSAL).transpose(1, 2).float()
    for b in range(2):
        a, w, z = got[b, :total[b]].float(), want[b, :total[b]].float(), size[b, :total[b]]
        # two outputs rounded (|w|, |a|), P rounded twice, K (its score error bounded by 2^-8 of sum |q k| scale,
        # below 8 for these sizes) and V rounded by the read, size itself off by two roundings
        tol = 2.0 ** -8 * (2 * w.abs() + (3 + 2 * 8 * (cdt != BF16)) * z) * 1.02
        assert ((a - w).abs() <= tol + 1e-6).all()


def test_f32_chain():
    pool_kv = [0, 0]
    cache = S.KVCache.empty(8, 8, 2, 16, F32)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    g = torch.Generator().manual_seed(1)
    k, v, q = (torch.randn(2, 20, h, 16, generator=g).cuda() for h in (2, 2, 4))
    lens = torch.tensor([20, 13], dtype=torch.int32, device="cuda")
    cat = lambda t: torch.cat([t[0], t[1, :13]])
    S.cache_write(cache, cat(k), cat(v), table, lens, cu([20, 13]))
    out = S.sdpa_paged(cat(q), cache, table, lens, cu([20, 13]))
    kd, vd = S.cache_read(cache, table, lens, T=20)
    want = S.sdpa(q.transpose(1, 2), kd, vd, mask_kind=S.MASK_CAUSAL).transpose(1, 2)
    assert device_error() == 0 and pool_kv == [0, 0]
    assert torch.equal(kd[0].transpose(0, 1), k[0]) and (kd[1, :, 13:] == 0).all()
    assert (out[:20] - want[0]).abs().max() < 1e-4 and (out[20:] - want[1, :13]).abs().max() < 1e-4


def decode_setup(cdt=BF16, d=64, kv=(700, 300, 64)):
    pool = R.Pool(cdt, 2, d, 16, list(kv), seed=6, garbage=False)
    q = torch.randn(len(kv), 8, d, generator=torch.Generator().manual_seed(2)).to(BF16).cuda()
    k, v = (torch.randn(len(kv), 2, d, generator=torch.Generator().manual_seed(3 + i)).to(BF16).cuda() for i in range(2))
    return pool, q, k, v, pool.table.cuda(), pool.lens.cuda()


@pytest.mark.parametrize("cdt", [BF16, E4M3])
def test_graph_replays_with_new_lengths(cdt):
    """A captured step replays with what lengths, tables and rows hold then."""
    pool, q, k, v, table, lens = decode_setup(cdt)
    cache = pool.cache()
    step = lambda: S.sdpa_paged(q, S.cache_write(cache, k, v, table, lens), table, lens)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for new in ([5, 300, 1], [700, 64, 17], [699, 0, 64]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        if 0 in new:
            lens[1] = 16
        q.normal_()
        k.normal_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, step()) and device_error() == 0


def test_two_graphs_and_two_streams_do_not_share_scratch():
    """Calls whose kernels overlap keep to their own workspaces: two captured
    graphs and eager calls on two streams at once."""
    sets = [decode_setup(BF16, 64, kv) for kv in ((4000, 900, 64), (3000, 2500, 1))]
    caches = [s[0].cache() for s in sets]
    plain = [S.sdpa_paged(s[1], c, s[4], s[5]).clone() for s, c in zip(sets, caches)]
    chunk = [torch.randn(200, 8, 64, device="cuda").to(BF16) for _ in range(2)]
    cuq = [cu([100, 50, 50]), cu([180, 20, 0])]
    plain2 = [S.sdpa_paged(x, c, s[4], s[5], u, max_q=180).clone() for x, c, s, u in zip(chunk, caches, sets, cuq)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append((S.sdpa_paged(sets[i][1], caches[i], sets[i][4], sets[i][5]),
                         S.sdpa_paged(chunk[i], caches[i], sets[i][4], sets[i][5], cuq[i], max_q=180)))
        graphs.append(g)
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    eager = []
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                eager.append((i, S.sdpa_paged(sets[i][1], caches[i], sets[i][4], sets[i][5])))
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i][0], plain[i]) and torch.equal(outs[i][1], plain2[i])
    for i, o in eager:
        assert torch.equal(o, plain[i])
    assert device_error() == 0


def test_stream_argument():
    pool, q, k, v, table, lens = decode_setup(E4M3)
    cache = pool.cache()
    want = S.sdpa_paged(q, cache, table, lens)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    busy = torch.zeros(1 << 26, device="cuda")
    with torch.cuda.stream(st):
        busy.add_(1)
    got = S.sdpa_paged(q, cache, table, lens, stream=st)
    S.cache_read(cache, table, lens, T=10, stream=st)
    st.synchronize()
    assert torch.equal(got, want)


def test_strided_rows_and_padding_rows():
    """q and out as slices of wider tensors, rows behind the last sequence kept."""
    for path, cdt in itertools.product(("exact", "auto", "tcgen05"), (BF16, INT8)):
        pool = R.Pool(cdt, 2, 64, 32, [70, 200], seed=8)
        n = [3, 90]
        wide = torch.randn(100, 8 + 4, 64, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
        q, out = wide[:, :8], torch.full((100, 10, 64), 7.0, dtype=BF16, device="cuda")
        S.sdpa_paged(q, pool.cache(), pool.table.cuda(), pool.lens.cuda(), cu(n), max_q=90, out=out[:, 1:9], path=path)
        assert device_error() == 0
        codes = cdt == INT8
        u_p = 0.0 if path == "exact" else R.U[torch.float16 if codes else BF16]
        want, _, tol, _ = R.attend(pool, q[:93].cpu(), n, u_p=u_p, p_floor=2.0 ** -37 if codes else 0.0,
                                   u_kv=2.0 ** -11 if codes else 0.0)
        R.check(out[:93, 1:9], want, tol, BF16, f"{path} {cdt}")
        assert (out[93:] == 7).all() and (out[:, 0] == 7).all() and (out[:, 9] == 7).all()


@pytest.mark.parametrize("cdt", [BF16, E4M3])
def test_auto_takes_odd_layouts(cdt):
    """A page size and strides that only the exact kernel takes."""
    run_case("auto", cdt, BF16, 8, 2, 64, 20, [100, 31], [40, 3])
    pool = R.Pool(cdt, 2, 64, 16, [100], seed=5)
    q = torch.randn(1, 8, 65, device="cuda").to(BF16)[:, :, :64]
    out = S.sdpa_paged(q, pool.cache(), pool.table.cuda(), pool.lens.cuda())
    want, _, tol, _ = R.attend(pool, q.cpu(), [1])
    R.check(out, want, tol, BF16)


def test_large_offsets():
    """A pool whose last pages lie past 2^31 elements."""
    pages, page, Hkv, d = 70000, 128, 2, 128
    k = torch.zeros(pages, Hkv, page, d, dtype=torch.int8, device="cuda")
    assert (pages - 1) * Hkv * page * d > 2 ** 31
    cache = S.KVCache(k, torch.zeros_like(k), *(torch.ones(pages, Hkv, page, device="cuda") for _ in range(2)))
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32, device="cuda")
    kv, n = 300, 150
    g = torch.Generator().manual_seed(1)
    kn, vn = (torch.randn(kv, Hkv, d, generator=g).to(BF16).cuda() for _ in range(2))
    lens = torch.tensor([kv], dtype=torch.int32, device="cuda")
    S.cache_write(cache, kn, vn, table, lens, cu([kv]))
    kd, vd = S.cache_read(cache, table, lens, T=kv)
    c, s = R.quantise(kn.cpu(), INT8)
    assert torch.equal(kd[0].transpose(0, 1).cpu(), (c * s[..., None]).to(BF16))
    q = torch.randn(n, 8, d, generator=g).to(BF16).cuda()
    outs = [S.sdpa_paged(q, cache, table, lens, cu([n]), path=p) for p in ("exact", "tcgen05")]
    one = [S.sdpa_paged(q[-1:], cache, table, lens, path=p) for p in ("exact", "decode")]
    assert device_error() == 0
    # both within 2^-8 of rounding and (codes) 2^-11 of P, K and V of one another's sums
    for a, b in (outs, one):
        assert (a.float() - b.float()).abs().max() < 2.0 ** -5 and (a.float() - b.float()).abs().mean() < 2.0 ** -9
    assert torch.isfinite(outs[0]).all()


@pytest.mark.parametrize("cdt", [BF16, E4M3, INT8])
def test_decode_whole_units(cdt):
    """A unit for every SM and short reaches: no unit is split (a window inside long caches, drafts)."""
    run_case("decode", cdt, BF16, 32, 16, 64, 16, [900] * 5 + [0, 1, 33, 2000, 64], None, window=300)
    run_case("decode", cdt, BF16, 16, 16, 128, 32, [(97 * i) % 700 for i in range(10)],
             [min(4, (97 * i) % 700) for i in range(10)])


@pytest.mark.parametrize("window", [1, 200, 600, 1500, 2999, 3000])
def test_chunk_windows_on_long_tables(window):
    """How a chunk's keys are split, and the scratch for it, go by the window."""
    run_case("auto", BF16, BF16, 4, 1, 64, 16, [3000], [200], window=window)
    run_case("auto", E4M3, BF16, 4, 2, 128, 32, [3000, 900], [40, 1], window=window)


def test_window_past_32_bits():
    """A window wider than a C int is no window, and a negative one is refused whatever its low bits."""
    pool, q, _, _, table, lens = decode_setup()
    cache = pool.cache()
    want = S.sdpa_paged(q, cache, table, lens)
    for window in (2 ** 31, 2 ** 32 + 1, 2 ** 40):
        assert torch.equal(S.sdpa_paged(q, cache, table, lens, window=window), want)
    for window in (-1, -2 ** 32 + 1):
        with pytest.raises(S.SdpaError):
            S.sdpa_paged(q, cache, table, lens, window=window)


@pytest.mark.parametrize("kw", [{}, dict(window=40), dict(softcap=5.0), dict(slopes=True)], ids=str)
@pytest.mark.parametrize("path,kv,n", [("exact", [300, 90], [5, 2]), ("exact", [40], [1]), ("decode", [300, 90, 2500], [5, 1, 2]),
                                       ("tcgen05", [300, 90], [200, 64]), ("tcgen05", [2500], [130])], ids=str)
@pytest.mark.parametrize("cdt", [BF16, E4M3])
@pytest.mark.parametrize("d", [64, 128])
def test_nan_in_a_key_reaches_the_rows_that_see_it(d, cdt, path, kv, n, kw):
    """NaN in a key (one, then every one of a sequence) or a query makes NaN of
    the rows whose scores it is in, their log-sum-exp too, and nothing else."""
    kw = dict(kw)
    pool = R.Pool(cdt, 2, d, 16, kv, seed=4)
    Hq, T = 4, sum(n)
    q = torch.randn(T, Hq, d, generator=torch.Generator().manual_seed(5)).to(BF16).cuda()
    if kw.pop("slopes", False):
        kw["slopes"] = torch.tensor([-0.5, 0.0, 0.25, 0.01], device="cuda")
    cache, table, lens = pool.cache(), pool.table.cuda(), pool.lens.cuda()

    def run(q):
        lse = torch.empty(T, Hq, device="cuda")
        out = S.sdpa_paged(q, cache, table, lens, cu(n), max_q=max(n), lse=lse, path=path, **kw)
        assert device_error() == 0
        return out, lse

    clean, clean_lse = run(q)
    assert torch.isfinite(clean).all() and torch.isfinite(clean_lse).all()
    b, at = 0, kv[0] - max(2, n[0] // 2)  # between the new rows where there are several
    pos = torch.arange(n[b]) + kv[b] - n[b]
    w = kw.get("window") or 1 << 30
    for keys in ([at], list(range(kv[b]))):
        kept = cache.k.clone()
        for j in keys:
            cache.k[int(pool.table[b, j // 16]), 1, j % 16, 3] = math.nan
        bad = torch.zeros(T, Hq, dtype=torch.bool)
        for j in keys:
            bad[:n[b], 2:] |= ((pos >= j) & (pos - w < j))[:, None]
        out, lse = run(q)
        bad = bad.cuda()
        assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
        assert torch.equal(out[~bad], clean[~bad]) and torch.equal(lse[~bad], clean_lse[~bad])
        cache.k.copy_(kept)
    q2 = q.clone()
    q2[T - 1, 1, 7] = math.nan
    out, lse = run(q2)
    bad = torch.zeros(T, Hq, dtype=torch.bool, device="cuda")
    bad[T - 1, 1] = True
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    assert torch.equal(out[~bad], clean[~bad]) and torch.equal(lse[~bad], clean_lse[~bad])


@pytest.mark.parametrize("path", ["exact", "decode", "tcgen05", "auto"])
def test_no_new_rows_announced(path):
    """max_q 0: sequences that bring rows all the same are reported, rows that
    belong to nobody are kept."""
    assert bad_batch(path, max_q=0) == -7
    pool = R.Pool(BF16, 2, 64, 16, [100, 60], seed=2)
    out = torch.full((4, 8, 64), 7.0, dtype=BF16, device="cuda")
    S.sdpa_paged(torch.zeros_like(out), pool.cache(), pool.table.cuda(), pool.lens.cuda(), cu([0, 0]), max_q=0, out=out,
                 path=path)
    assert device_error() == 0 and (out == 7).all()


def test_scratch_goes_by_the_call():
    """What a call allocates is what sdpa_fwd_paged_workspace asks for it,
    whatever ran on the cache before."""
    pool, q, _, _, table, lens = decode_setup(BF16, 64, (4000, 900, 64))
    cache, short, few = pool.cache(), table[:, :8].contiguous(), lens.clamp(max=100)
    chunk = torch.randn(200, 8, 64, device="cuda").to(BF16)

    def taken(q, table, lens, n, most):
        out = torch.empty_like(q)
        cuq = None if n is None else cu(n)
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        S.sdpa_paged(q, cache, table, lens, cuq, max_q=most, out=out)
        got = torch.cuda.max_memory_allocated() - before
        b = S.paged._batch(cache, table, lens, cuq, q.shape[0], most)
        need = S.sdpa_fwd_paged_workspace(cache.descriptor(), b, q.data_ptr(), None, out.data_ptr(), None, S.SDPA_BF16, 8, 0, 0)
        assert device_error() == 0 and need <= got <= need + 511, (got, need)  # the allocator's granule
        return need

    calls = [(q, short, few, None, 1), (q, table, lens, None, 1), (chunk, table, lens, [100, 50, 50], 100)]
    first = [taken(*c) for c in calls]
    assert first[0] == 0 < first[1] < first[2]
    for i in (0, 1, 0, 2, 2, 0):
        assert taken(*calls[i]) == first[i]


@pytest.mark.parametrize("cdt,io", [(BF16, BF16), (E4M3, BF16), (INT8, F32)])
def test_back_to_back_calls_read_what_the_last_one_wrote(cdt, io):
    """Calls that feed one another with nothing between them: a step's rows are
    another call's output, its cache is written, attended by single tokens and
    by a chunk, read back, and the rows read are written again."""
    n = [400, 30, 260]
    caches = [S.KVCache.empty(80, 16, 2, 64, cdt) for _ in range(2)]
    table = torch.randperm(80, generator=torch.Generator().manual_seed(1)).int().cuda()[:78].view(3, 26)
    lens = torch.tensor(n, dtype=torch.int32, device="cuda")
    rows = torch.randn(2, sum(n), 2, 64, device="cuda").to(io)

    def steps(wait):
        outs = []
        for t in (x for c in caches for x in (c.k, c.v, c.k_scale, c.v_scale) if x is not None):
            t.zero_()
        k, v = rows[0].clone(), rows[1].clone()
        torch.cuda.synchronize()
        for i in range(6):
            a, b = caches[i % 2], caches[1 - i % 2]
            S.cache_write(a, k, v, table, lens, cu_n, max_q=400)
            wait()
            one = S.sdpa_paged(q1, a, table, lens)
            wait()
            S.sdpa_paged(one, a, table, lens, out=q1b)
            wait()
            many = S.sdpa_paged(qn, a, table, lens, cu_n, max_q=400)
            wait()
            kd, vd = S.cache_read(a, table, lens, k_out, v_out)
            wait()
            # 64 tokens of sequence 0, straight from what was read, into the other cache
            S.cache_write(b, kd[0].transpose(0, 1)[:64], vd[0].transpose(0, 1)[:64], table[:1], l64, cu64, max_q=64)
            wait()
            # and over rows this cache holds: the chunk call behind it sees the new ones
            S.cache_write(a, many[:64, :2], many[64:128, 2:4], table[:1], l64, cu64, max_q=64)
            wait()
            last = S.sdpa_paged(qn[:64], a, table[:1], l64, cu64, max_q=64)
            wait()
            outs += [one.clone(), q1b.clone(), many, kd.clone(), vd.clone(), last]
        return outs

    cu_n, cu64, l64 = cu(n), cu([64]), torch.tensor([64], dtype=torch.int32, device="cuda")
    q1, q1b = torch.randn(3, 4, 64, device="cuda").to(io), torch.empty(3, 4, 64, device="cuda", dtype=io)
    qn = torch.randn(sum(n), 4, 64, device="cuda").to(io)
    k_out, v_out = (torch.zeros(3, 2, 400, 64, device="cuda", dtype=io) for _ in range(2))
    want = steps(torch.cuda.synchronize)
    for _ in range(5):
        for a, b in zip(want, steps(lambda: None)):
            assert torch.equal(a, b)
    assert device_error() == 0


@pytest.mark.parametrize("path,kv,n", [("exact", [300, 90], [5, 2]), ("decode", [300, 90, 2500], [5, 1, 2]),
                                       ("tcgen05", [300, 90], [200, 64]), ("tcgen05", [2500], [130])], ids=str)
@pytest.mark.parametrize("cdt", [BF16, E4M3, INT8])
@pytest.mark.parametrize("d", [64, 128])
def test_values_that_are_not_finite(d, cdt, path, kv, n):
    """A NaN or an infinity in a value (INT8: an infinite scale) makes every row
    that sees it not finite, and touches no other sequence or kv head; in front
    of every row's window, or behind the sequence's tokens, it touches nothing."""
    pool = R.Pool(cdt, 2, d, 16, kv, seed=4)
    T = sum(n)
    q = torch.randn(T, 4, d, generator=torch.Generator().manual_seed(5)).to(BF16).cuda()
    cache, table, lens = pool.cache(), pool.table.cuda(), pool.lens.cuda()

    def run(window=0):
        lse = torch.empty(T, 4, device="cuda")
        out = S.sdpa_paged(q, cache, table, lens, cu(n), max_q=max(n), window=window, lse=lse, path=path)
        assert device_error() == 0
        return out, lse

    def spoil(j, x):
        p, o = int(pool.table[0, j // 16]), j % 16
        if cdt == INT8:
            cache.v_scale[p, 1, o] = math.inf
        else:
            row = cache.v[p, 1, o].float()
            row[3] = x
            cache.v[p, 1, o] = row.to(cdt)

    first = kv[0] - n[0]
    clean, clean_lse = run()
    for j, x in ((0, math.nan), (first, math.nan), (first + 1, math.inf), (kv[0] - 1, math.inf)):
        if cdt == E4M3 and x == math.inf:
            x = math.nan  # the type has no infinity
        kept = [t.clone() for t in (cache.v, cache.v_scale) if t is not None]
        spoil(j, x)
        out, lse = run()
        see = torch.arange(n[0]) + first >= j
        assert not torch.isfinite(out[:n[0]][see.cuda(), 2:, 3]).any()
        assert torch.equal(out[:, :2], clean[:, :2]) and torch.equal(out[n[0]:], clean[n[0]:])
        if cdt != INT8:  # an infinite scale is in the weights' sum too
            assert torch.equal(lse, clean_lse)
        for t, old in zip((cache.v, cache.v_scale), kept):
            t.copy_(old)
    # in front of the window of the first new row, in its tile and far from it
    window = 20
    clean, clean_lse = run(window)
    for j in (0, first - window, max(0, first - window - 15)):
        spoil(j, math.nan)
    out, lse = run(window)
    assert torch.isfinite(out).all() and torch.equal(out, clean) and torch.equal(lse, clean_lse)


@pytest.mark.parametrize("path,kv,n", [("exact", [300, 90], [5, 2]), ("decode", [300, 90, 2500], [5, 1, 2]),
                                       ("tcgen05", [300, 90], [200, 64]), ("tcgen05", [2500], [130])], ids=str)
@pytest.mark.parametrize("cdt", [E4M3, INT8])
@pytest.mark.parametrize("d", [64, 128])
def test_infinite_key_reaches_the_rows_that_see_it(d, cdt, path, kv, n):
    """A key written with an infinity (its scale is infinite) makes NaN of the
    rows that see it; those in front of it keep every bit."""
    pool = R.Pool(cdt, 2, d, 16, kv, seed=4)
    T = sum(n)
    q = torch.randn(T, 4, d, generator=torch.Generator().manual_seed(5)).to(BF16).cuda()
    cache, table, lens = pool.cache(), pool.table.cuda(), pool.lens.cuda()

    def run():
        lse = torch.empty(T, 4, device="cuda")
        out = S.sdpa_paged(q, cache, table, lens, cu(n), max_q=max(n), lse=lse, path=path)
        assert device_error() == 0
        return out, lse

    clean, clean_lse = run()
    at = kv[0] - max(2, n[0] // 2)  # between the new rows
    p, o = int(pool.table[0, at // 16]), at % 16
    cache.k[p, 1, o] = 0
    cache.k_scale[p, 1, o] = math.inf  # what cache_write makes of an infinity (an E4M3 one's own code is NaN)
    bad = torch.zeros(T, 4, dtype=torch.bool, device="cuda")
    bad[:n[0], 2:] = (torch.arange(n[0]) + kv[0] - n[0] >= at)[:, None].cuda()
    out, lse = run()
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    assert torch.equal(out[~bad], clean[~bad]) and torch.equal(lse[~bad], clean_lse[~bad])


@pytest.mark.parametrize("cdt", [BF16, INT8])
def test_calls_follow_their_stream(cdt):
    """Every operator called with ``stream=`` sees what was queued on that stream
    in front of it: the inputs are filled there behind a long kernel."""
    pool, q, k, v, table, lens = decode_setup(cdt)
    new_q, new_k, new_v = (torch.randn_like(x) for x in (q, k, v))
    new_lens = torch.tensor([650, 17, 64], dtype=torch.int32, device="cuda")

    def steps(cache, q, k, v, lens, **kw):
        S.cache_write(cache, k, v, table, lens, **kw)
        return (S.sdpa_paged(q, cache, table, lens, **kw),) + S.cache_read(cache, table, lens, T=700, **kw)

    want = steps(pool.cache(), new_q, new_k, new_v, new_lens)
    old = steps(pool.cache(), q, k, v, lens)
    assert all(not torch.equal(a, b) for a, b in zip(want, old))
    st, busy = torch.cuda.Stream(), torch.zeros(1 << 28, device="cuda")
    first = [x.clone() for x in (q, k, v, lens)]
    for _ in range(5):  # until the calls were all made while the stream was still busy (a first try may allocate)
        cache = pool.cache()
        for x, y in zip((q, k, v, lens), first):
            x.copy_(y)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            for _ in range(60):
                busy.add_(1)  # 20 ms or so in all
            for x, y in ((q, new_q), (k, new_k), (v, new_v), (lens, new_lens)):
                x.copy_(y)
        got = steps(cache, q, k, v, lens, stream=st)
        early = not st.query()
        st.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got)) and device_error() == 0
        if early:
            return
    pytest.fail("the stream was always done before the calls: nothing was tested")


@pytest.mark.parametrize("cdt", [BF16, E4M3])
def test_decode_sequence_in_any_batch(cdt):
    """One sequence beside different others: its keys are cut elsewhere each
    time, its result stays within the bound."""
    kv = [5000, 300, 2900, 1, 700, 64]
    pool = R.Pool(cdt, 2, 128, 16, kv, seed=3)
    q = torch.randn(6, 8, 128, generator=torch.Generator().manual_seed(4)).to(BF16)
    codes = cdt == E4M3
    want, wlse, tol, ltol = R.attend(pool, q, [1] * 6, u_p=R.U[torch.float16 if codes else BF16],
                                     p_floor=2.0 ** -37 if codes else 0.0)
    cache, bits_seen = pool.cache(), set()
    for batch in ([0], [0, 1], [2, 0], [0, 1, 2, 3, 4, 5], [5, 4, 3, 2, 1, 0], [2] * 40 + [0] + [4] * 30, [0] * 7):
        lse = torch.empty(len(batch), 8, device="cuda")
        out = S.sdpa_paged(q[batch].cuda(), cache, pool.table[batch].cuda(), pool.lens[batch].cuda(), lse=lse, path="decode")
        assert device_error() == 0
        R.check(out, want[batch], tol[batch], BF16, f"{cdt} {batch}")
        R.check_lse(lse, wlse[batch], ltol[batch], f"{cdt} {batch}")
        bits_seen.add(lse[batch.index(0)].cpu().numpy().tobytes())
    assert len(bits_seen) > 1, "every batch cut the sequence alike: nothing was tested"


@pytest.mark.parametrize("cdt", [E4M3, INT8])
def test_codes_of_every_scale(cdt):
    """Rows whose scale has all ones in its significand, the one kind of divisor
    whose reciprocal does not give the rounded quotient, and scales of every size."""
    Q = R.QMAX[cdt]
    s = torch.cat([torch.tensor([2.0 ** e], dtype=F32).view(torch.int32) - 1 for e in range(-29, 116)]).view(F32)
    near = (s.double() * Q).float().view(torch.int32)[:, None] + torch.arange(-3, 4, dtype=torch.int32)
    near = near.view(F32)
    hit = (near.double() / Q).float() == s[:, None]  # the quotients of maxima that round to it
    assert hit.any(1).all()
    top = near[torch.arange(len(s)), hit.int().argmax(1)]
    g = torch.Generator().manual_seed(3)
    top = torch.cat([top, torch.exp(torch.empty(2000).uniform_(-60, 80, generator=g))])
    d, T = 128, len(top)
    x = torch.empty(T, 2, d).uniform_(-1, 1, generator=g) * top[:, None, None]
    x[:, :, 5] = top[:, None]
    # halfway between two codes and next to it
    step = (x[:, 1, 6:40] / top[:, None] * Q).round() + 0.5
    x[:, 1, 6:40] = (step.clamp(-Q + 0.5, Q - 0.5).double() / Q * top[:, None].double()).float()
    cache = S.KVCache.empty(-(-T // 16), 16, 2, d, cdt)
    table = torch.arange(-(-T // 16), dtype=torch.int32, device="cuda")[None]
    S.cache_write(cache, x.cuda(), x.flip(1).cuda(), table, torch.tensor([T], dtype=torch.int32, device="cuda"), cu([T]))
    assert device_error() == 0
    c, want = R.quantise(x, cdt)
    assert ((want.float().view(torch.int32) & 0x7fffff) == 0x7fffff).sum() >= 2 * len(s)
    flat = lambda t: t.transpose(1, 2).flatten(0, 1)[:T].cpu()
    for raw, sc, ref, refs in ((cache.k, cache.k_scale, c, want), (cache.v, cache.v_scale, c.flip(1), want.flip(1))):
        assert torch.equal(flat(raw.float()).double(), ref) and torch.equal(flat(sc), refs.float())


@pytest.mark.parametrize("path", ["exact", "auto", "tcgen05"])
@pytest.mark.parametrize("cdt", [BF16, INT8])
def test_many_sequences_of_every_kind(cdt, path):
    """More sequences than any block has threads, new rows from none to a chunk,
    tables wider than their rows' pages and sliced from a wider tensor; rows of
    nobody in front of the first sequence and behind the last keep out and lse."""
    kv = [(i * 53) % 120 for i in range(1200)]
    n = [0 if i % 4 == 0 else min(kv[i], 1 + (i * 7) % (90 if i % 100 == 3 else 5)) for i in range(1200)]
    pool = R.Pool(cdt, 1, 64, 16, kv, seed=2)
    front, T = 3, sum(n)
    q = torch.randn(front + T + 4, 4, 64, generator=torch.Generator().manual_seed(3)).to(BF16)
    wide = torch.full((1200, pool.table.shape[1] + 9), -3, dtype=torch.int32)
    wide[:, 2:2 + pool.table.shape[1]] = pool.table
    out = torch.full((front + T + 4, 4, 64), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((front + T + 4, 4), 7.0, device="cuda")
    S.sdpa_paged(q.cuda(), pool.cache(), wide.cuda()[:, 2:-5], pool.lens.cuda(), cu(n) + front, max_q=max(n), out=out, lse=lse,
                 path=path)
    assert device_error() == 0
    mine = slice(front, front + T)
    codes = cdt in R.QMAX
    want, wlse, tol, ltol = R.attend(pool, q[mine], n, u_p=0.0 if path == "exact" else R.U[torch.float16 if codes else BF16],
                                     p_floor=2.0 ** -37 if path != "exact" and codes else 0.0,
                                     u_kv=R.U[torch.float16] if path != "exact" and codes else 0.0)
    R.check(out[mine], want, tol, BF16, f"{path} {cdt}")
    R.check_lse(lse[mine], wlse, ltol, f"{path} {cdt}")
    for t in (out, lse):
        assert (t[:front] == 7).all() and (t[front + T:] == 7).all()


@pytest.mark.parametrize("path", ["exact", "decode", "tcgen05"])
def test_tables_without_pages(path):
    """A batch whose table has no pages: every row sees nothing, and a write says so."""
    cache = R.Pool(BF16, 2, 64, 16, [20]).cache()
    table, lens = (torch.zeros(*s, dtype=torch.int32, device="cuda") for s in ((3, 0), (3,)))
    lse = torch.zeros(6, 4, device="cuda")
    out = S.sdpa_paged(torch.ones(6, 4, 64, dtype=BF16, device="cuda"), cache, table, lens, cu([1, 2, 3]), max_q=3, lse=lse, path=path)
    assert device_error() == 0 and (out == 0).all() and (lse == -math.inf).all()
    k, v = S.cache_read(cache, table, lens, T=5)
    assert device_error() == 0 and (k == 0).all() and (v == 0).all()
    x = torch.ones(3, 2, 64, dtype=BF16, device="cuda")
    S.cache_write(cache, x, x, table, lens)
    assert device_error() == -7


@pytest.mark.parametrize("cdt", [F32, BF16, E4M3, INT8])
def test_read_of_the_first_tokens(cdt):
    """T below the sequences' lengths, odd, one, and past the longest."""
    kv = [300, 0, 1, 77]
    pool = R.Pool(cdt, 3, 64, 16, kv, seed=8)
    io = F32 if cdt == F32 else BF16
    cache, table, lens = pool.cache(), pool.table.cuda(), pool.lens.cuda()
    for T in (1, 2, 33, 64, 77, 299, 300, 301):
        got = S.cache_read(cache, table, lens, T=T)
        assert device_error() == 0
        for which, x in enumerate(got):
            assert x.shape == (4, 3, T, 64) and x.dtype == io
            for b, L in enumerate(kv):
                m = min(L, T)
                want = pool.tokens(which, b, m).float() if m else torch.zeros(3, 0, 64)
                assert torch.equal(x[b, :, :m].cpu(), want.to(io)) and (x[b, :, m:] == 0).all()


def test_threads_call_at_once():
    """Several host threads, each with its stream, on one cache and on their own."""
    import threading
    sets = [decode_setup(BF16 if i % 2 else E4M3, 64, (2000 + 100 * i, 900, 64)) for i in range(4)]
    caches = [s[0].cache() for s in sets]
    chunks = [torch.randn(150, 8, 64, device="cuda").to(BF16) for _ in sets]
    cuq = cu([100, 30, 20])
    step = lambda i: (S.sdpa_paged(sets[i][1], caches[i], sets[i][4], sets[i][5]),
                      S.sdpa_paged(chunks[i], caches[i], sets[i][4], sets[i][5], cuq, max_q=100))
    want = [step(i) for i in range(4)]
    torch.cuda.synchronize()
    bad = []

    def work(t):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for j in range(30):
                    i = (t + j) % 4 if j % 3 else 0  # one cache for all, or one each
                    got = step(i)
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                        bad.append((t, j))
        except Exception as e:  # reported by the main thread
            bad.append(e)

    threads = [threading.Thread(target=work, args=(t,)) for t in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and device_error() == 0


@pytest.mark.parametrize("Tq,T", [(900, 20), (300, 200), (8, 2000)])
def test_narrow_heads_read_back_for_dense_calls(Tq, T):
    """Rows written, read back and attended densely at head_dim 16 with nothing
    between the calls, each reading what the one before it wrote."""
    cache = S.KVCache.empty(260, 16, 2, 16, BF16)
    table = torch.randperm(260, generator=torch.Generator().manual_seed(1)).int().cuda()[:250].view(2, 125)
    lens = torch.tensor([T, T], dtype=torch.int32, device="cuda")
    rows = torch.randn(8, 2 * T, 2, 16, device="cuda").to(BF16)
    q = torch.randn(2, 4, Tq, 16, device="cuda").to(BF16)
    k_out, v_out = (torch.zeros(2, 2, T, 16, dtype=BF16, device="cuda") for _ in range(2))
    x, y = torch.empty_like(q), torch.empty_like(q)

    def steps(wait):
        outs = []
        for i in range(4):
            S.cache_write(cache, rows[2 * i], rows[2 * i + 1], table, lens, cuq, max_q=T)
            wait()
            S.cache_read(cache, table, lens, k_out, v_out)
            wait()
            S.sdpa(q, k_out, v_out, out=x)
            wait()
            S.sdpa(x, k_out, v_out, out=y)
            wait()
            outs += [x.clone(), y.clone()]
        return outs

    cuq = cu([T, T])
    want = steps(torch.cuda.synchronize)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(want, steps(lambda: None)))
    assert device_error() == 0
