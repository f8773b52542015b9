"""What the paged cache operators refuse, before anything touches a GPU."""
import ctypes

import pytest
import torch

import attention_sdpa_fwd_b200 as S
from attention_sdpa_fwd_b200 import build
from attention_sdpa_fwd_b200.paged import _strides

BF16, F32 = S.SDPA_BF16, S.SDPA_F32
# distinct fake device addresses, far apart (never dereferenced: validation comes first)
K, V, KS, VS, Q, O, W, TAB, LEN, CU, LSE = (0x10000000 * i for i in range(1, 12))


@pytest.fixture(scope="module", autouse=True)
def L():
    build.build()
    return S.lib()


def cache(**kw):
    d, ps, h = kw.get("d", 64), kw.get("page_size", 16), kw.get("Hkv", 2)
    st = S.sdpa_strides_t(h * ps * d, ps * d, d)
    sc = S.sdpa_strides_t(h * ps, ps, 1)
    a = dict(k=K, v=V, k_scale=KS, v_scale=VS, dtype=S.paged.CACHE_BF16, num_pages=8, page_size=ps, Hkv=h, d=d,
             k_strides=st, v_strides=st, k_scale_strides=sc, v_scale_strides=sc)
    a.update(kw)
    return S.sdpa_cache_t(**a)


def batch(**kw):
    a = dict(page_table=TAB, table_stride=4, max_pages=4, kv_lens=LEN, cu_q=CU, B=2, total_q=6, max_q=4)
    a.update(kw)
    return S.sdpa_batch_t(**a)


def paged(c=None, b=None, **kw):
    a = dict(q=Q, qs=None, out=O, os=None, dtype=BF16, Hq=4, scale=0.1, window=0, softcap=0.0, slopes=None, lse=None,
             path=0, ws=None, ws_bytes=0)
    a.update(kw)
    return S.sdpa_fwd_paged(a["q"], a["qs"], c or cache(), b or batch(), a["out"], a["os"], a["dtype"], a["Hq"], a["scale"],
                            a["window"], a["softcap"], a["slopes"], a["lse"], a["path"], a["ws"], a["ws_bytes"], None)


def write(c=None, b=None, k=Q, v=O, ks=None, vs=None, dtype=BF16):
    return S.sdpa_cache_write(c or cache(), b or batch(), k, ks, v, vs, dtype, None)


def read(c=None, b=None, k=Q, v=O, ks=None, vs=None, dtype=BF16, T=10):
    return S.sdpa_cache_read(c or cache(), b or batch(), k, ks, v, vs, dtype, T, None)


E4 = S.paged.CACHE_E4M3
BAD_CACHES = [(dict(dtype=4), -1), (dict(dtype=-1), -1), (dict(d=32), -2), (dict(d=80), -2), (dict(num_pages=0), -1),
              (dict(page_size=0), -1), (dict(Hkv=0), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(k=K + 1), -3),
              (dict(k_strides=S.sdpa_strides_t(0, 64, 64)), -1), (dict(v_strides=S.sdpa_strides_t(64, -1, 64)), -1),
              (dict(v_strides=S.sdpa_strides_t(64, 64, (1 << 40) + 1)), -1), (dict(dtype=E4, k_scale=None), -1),
              (dict(dtype=E4, v_scale=VS + 2), -3), (dict(dtype=E4, k_scale_strides=S.sdpa_strides_t(1, 0, 1)), -1)]
BAD_BATCHES = [(dict(B=-1), -1), (dict(max_pages=-1), -1), (dict(table_stride=3), -1), (dict(kv_lens=None), -1),
               (dict(page_table=None), -1), (dict(page_table=TAB + 2), -3), (dict(kv_lens=LEN + 1), -3),
               (dict(max_pages=1 << 28, table_stride=1 << 28), -2)]
BAD_ROWS = [(dict(total_q=(1 << 30) + 1), -2), (dict(total_q=-1), -1), (dict(max_q=-1), -1), (dict(cu_q=None), -1), (dict(B=0), -1), (dict(cu_q=CU + 1), -3)]


@pytest.mark.parametrize("call", [paged, write, read])
@pytest.mark.parametrize("kw,code", BAD_CACHES, ids=str)
def test_bad_cache(call, kw, code):
    assert call(cache(**kw)) == code


@pytest.mark.parametrize("call", [paged, write, read])
@pytest.mark.parametrize("kw,code", BAD_BATCHES, ids=str)
def test_bad_batch(call, kw, code):
    assert call(None, batch(**kw)) == code


@pytest.mark.parametrize("call", [paged, write])
@pytest.mark.parametrize("kw,code", BAD_ROWS, ids=str)
def test_bad_rows(call, kw, code):
    assert call(None, batch(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), -1), (dict(Hq=3), -1), (dict(Hq=0), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(softcap=-1.0), -1), (dict(softcap=float("inf")), -1), (dict(window=-1), -1), (dict(q=None), -1),
    (dict(out=None), -1), (dict(q=Q + 1), -3), (dict(out=O + 1), -3), (dict(lse=LSE + 2), -3), (dict(slopes=W + 1), -3),
    (dict(out=Q + 64), -1), (dict(out=K + 64), -1), (dict(out=V), -1), (dict(lse=O), -1), (dict(lse=Q + 4), -1),
    (dict(lse=K), -1), (dict(path=-1), -1), (dict(path=4), -1), (dict(dtype=F32), -2),
    (dict(qs=S.sdpa_rows_t(0, 64)), -1), (dict(os=S.sdpa_rows_t(256, -64)), -1),
    (dict(ws=None), -6), (dict(ws=W, ws_bytes=64), -6), (dict(ws=W + 8, ws_bytes=1 << 30), -3),
    (dict(path=2, Hq=64), -2),                                # 4 x 32 rows: not few
    (dict(path=2, qs=S.sdpa_rows_t(260, 65)), -3), (dict(path=3, os=S.sdpa_rows_t(260, 65)), -3),
], ids=str)
def test_bad_attention(kw, code):
    b = batch(page_table=TAB, max_pages=64, table_stride=64)
    assert paged(None, b, **kw) == code


@pytest.mark.parametrize("path", [2, 3])
@pytest.mark.parametrize("kw,dtype,code", [(dict(d=16), BF16, -2), (dict(page_size=24), BF16, -2),
                                           (dict(dtype=S.paged.CACHE_F32), F32, -2), (dict(dtype=E4), F32, -2),
                                           (dict(k=K + 2), BF16, -3), (dict(v_strides=S.sdpa_strides_t(2052, 1024, 65)), BF16, -3)],
                         ids=str)
def test_forced_path_refuses_layout(path, kw, dtype, code):
    assert paged(cache(**kw), path=path, dtype=dtype) == code


def test_bf16_and_f32_do_not_mix():
    assert write(dtype=F32) == -2 and read(dtype=F32) == -2
    assert write(cache(dtype=S.paged.CACHE_F32), dtype=BF16) == -2


@pytest.mark.parametrize("kw,code", [(dict(k=None), -1), (dict(v=None), -1), (dict(k=Q + 1), -3), (dict(k=K), -1),
                                     (dict(v=V + 128), -1), (dict(ks=S.sdpa_rows_t(0, 1)), -1)], ids=str)
def test_bad_write(kw, code):
    assert write(**kw) == code


@pytest.mark.parametrize("kw,code", [(dict(k=None), -1), (dict(k=Q + 1), -3), (dict(v=K), -1), (dict(T=-1), -1),
                                     (dict(ks=S.sdpa_strides_t(0, 1, 1)), -1)], ids=str)
def test_bad_read(kw, code):
    assert read(**kw) == code


def test_nothing_to_do():
    b = batch(B=0, total_q=0, page_table=None, kv_lens=None, cu_q=None)
    assert paged(None, b, q=None, out=None) == 0
    assert write(None, b, k=None, v=None) == 0
    assert read(None, b, k=None, v=None) == 0
    assert paged(None, batch(total_q=0)) == 0 and read(T=0, k=None, v=None) == 0


def workspace(c=None, b=None, Hq=4, path=0, dtype=BF16, window=0):
    return S.sdpa_fwd_paged_workspace(c or cache(), b or batch(), Q, None, O, None, dtype, Hq, window, path)


def test_workspace_sizes():
    long = batch(max_pages=512, table_stride=512)
    assert workspace() == 0                                     # short caches are not split
    assert workspace(b=long) > 0
    assert workspace(b=long, path=1) == 0 and workspace(b=long, dtype=7) == -1 and workspace(b=long, path=9) == -1
    assert workspace(b=batch(total_q=0)) == 0
    assert workspace(b=long, window=64) == 0 and workspace(b=long, window=-1) == -1
    # a window changes how chunks are split: what is asked for is what the call wants
    for window in (0, 200, 600, 1500, 5000, 9000):
        b = batch(B=1, max_pages=600, table_stride=600, total_q=200, max_q=200)
        need = workspace(b=b, window=window)
        assert paged(None, b, window=window, ws=W, ws_bytes=need - 1) == -6 if need else True
        assert need >= 0
    # both kernels of a mixed batch have their share
    mixed = batch(max_pages=512, table_stride=512, total_q=400, max_q=300)
    assert workspace(b=mixed) > workspace(b=mixed, path=3) > 0


def test_binding_refuses():
    c = S.KVCache.empty(4, 16, 2, 64, torch.bfloat16, device="cpu")
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: S.cache_write(c, x, x, table, lens), lambda: S.cache_read(c, table, lens, T=4),
                 lambda: S.sdpa_paged(x, c, table, lens)):
        with pytest.raises(ValueError):
            call()  # no CPU path
    with pytest.raises(TypeError):
        S.KVCache.empty(4, 16, 2, 64, torch.float16, device="cpu")
    with pytest.raises(ValueError):
        S.KVCache(c.k, c.v[:2])
    with pytest.raises(ValueError):
        S.KVCache(c.k.transpose(2, 3), c.v.transpose(2, 3))
    with pytest.raises(ValueError):
        S.KVCache(c.k, c.v, torch.zeros(4, 2, 16), torch.zeros(4, 2, 16))
    q8 = torch.zeros(4, 2, 16, 64, dtype=torch.int8)
    with pytest.raises(ValueError):
        S.KVCache(q8, q8)
    with pytest.raises(AttributeError):
        c.k = None


def test_strides_of_one_element_axes():
    t = torch.zeros(1, 2, 1, 64)[:, :, :, :].expand(1, 2, 1, 64)
    s = _strides(t.as_strided((1, 2, 1, 64), (0, 64, 0, 1)))
    assert (s.b, s.h, s.t) == (1, 64, 1)
    assert ctypes.sizeof(S.sdpa_strides_t) == 24


def test_read_refuses_rows_past_the_longest_sequence():
    one = S.sdpa_strides_t(64, 64, 64)
    for T in ((1 << 30) + 1, (1 << 31) - 32, (1 << 31) - 1):
        assert read(cache(Hkv=1), batch(B=1), T=T) == -2
        assert read(cache(Hkv=1), batch(B=1), ks=one, vs=one, T=T) == -2


@pytest.mark.parametrize("where", ["ks", "vs", "inside"])
def test_scales_are_not_overwritten(where):
    """An 8-bit cache's scales are as much of it as its codes."""
    c = cache(dtype=E4)
    at = {"ks": KS, "vs": VS, "inside": KS + 256}[where]
    assert paged(c, out=at) == -1 and paged(c, lse=at) == -1
    assert write(c, k=at) == -1 and write(c, v=at) == -1
    assert read(c, k=at) == -1 and read(c, v=at) == -1


@pytest.mark.parametrize("which", ["k_strides", "v_strides", "k_scale_strides", "v_scale_strides"])
def test_pools_past_the_address_space(which):
    """(num_pages - 1) times the page stride is 2^64: as 64 bits it would be 0
    and an overlap behind the first page unseen."""
    st = dict.fromkeys(("k_strides", "v_strides", "k_scale_strides", "v_scale_strides"), S.sdpa_strides_t(1, 1024, 64))
    st[which] = S.sdpa_strides_t(1 << 40, 1024, 64)
    c = cache(dtype=E4, num_pages=(1 << 24) + 1, **st)
    for call in (paged, write, read):
        assert call(c) == -1


def test_rows_past_the_address_space():
    far, b = S.sdpa_rows_t(1 << 40, 64), batch(total_q=(1 << 24) + 1)
    assert paged(None, b, qs=far) == -1 and paged(None, b, os=far) == -1
    assert write(None, b, ks=far) == -1 and write(None, b, vs=far) == -1
    far, b = S.sdpa_strides_t(1 << 40, 640, 64), batch(B=(1 << 24) + 1)
    assert read(None, b, ks=far) == -1 and read(None, b, vs=far) == -1


def test_outputs_are_not_the_batch():
    """What the kernels read of a batch, and the slopes, are not written over."""
    for at in (TAB, LEN, LEN + 4, CU, CU + 8):
        assert paged(None, None, out=at) == -1 and paged(None, None, lse=at) == -1
        assert write(cache(k=at)) == -1 and write(cache(dtype=E4, v_scale=at)) == -1
    for at in (TAB, LEN + 4):
        assert read(k=at) == -1 and read(v=at) == -1
    assert paged(None, None, slopes=W, out=W) == -1 and paged(None, None, slopes=W + 12, lse=W) == -1


def test_read_outputs_are_two():
    assert read(k=Q, v=Q) == -1 and read(k=Q, v=Q + 126) == -1 and read(k=Q + 64, v=Q) == -1
