"""The 8-bit paged cache without a GPU: refusals before any launch, and the plain quantiser of the GPU
tests pinned by its definition."""
import ctypes
import struct

import pytest
import torch

from _q8_util import FORMATS, quantise_ref, values_ref


@pytest.fixture(scope="module")
def tvlib():
    import __graft_entry__
    __graft_entry__.build()
    import speculative_decoding_tree_tv_gb300 as tv
    return tv


P = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails its checks first
ODD = ctypes.c_void_p(0x1008)


def cache(tv, **kw):
    from speculative_decoding_tree_tv_gb300._lib import Q8_CACHE_FORMAT
    f = dict(k=0x1000, v=0x1000, ks=0x1000, vs=0x1000, page_stride=16 * 64 * 2, head_stride=16 * 64, row_stride=64,
             num_pages=10, page_size=16, Hkv=2, D=64, format=0, dtype=0)
    f.update(kw)
    return struct.pack(Q8_CACHE_FORMAT, *f.values())


@pytest.mark.parametrize("kw,code", [
    (dict(num_pages=0), 1), (dict(Hkv=0), 1), (dict(D=0), 1), (dict(D=24), 3), (dict(D=1040), 3), (dict(dtype=2), 3),
    (dict(format=2), 3), (dict(format=-1), 3), (dict(page_size=24), 3), (dict(page_size=4), 3),
    (dict(page_size=512), 3), (dict(k=0), 1), (dict(v=0x1008), 1), (dict(ks=0), 1), (dict(vs=0), 1),
    (dict(vs=0x1004), 1), (dict(row_stride=72), 1), (dict(head_stride=-64), 1), (dict(head_stride=8), 1),
    (dict(page_stride=8), 1)])
def test_bad_caches_are_refused(tvlib, kw, code):
    lib, c = tvlib.lib, cache(tvlib, **kw)
    assert lib.tv_paged_append_q8(P, P, 128, 64, P, 4, c, P, None) == code
    assert lib.tv_paged_read_q8(c, P, P, P, 1, 4, 4, P, P, P, None) == code
    assert lib.tv_commit_paged_q8(c, P, P, P, P, 1, 4, 4, ctypes.c_void_p(0x2000), P, None) == code
    assert lib.tv_paged_append_q8(P, P, 128, 64, P, 4, None, P, None) == 1


def test_arguments_are_checked(tvlib):
    lib, c = tvlib.lib, cache(tvlib)
    ap = lambda **k: lib.tv_paged_append_q8(k.get("k", P), k.get("v", P), k.get("t", 128), k.get("h", 64),  # noqa: E731
                                            k.get("slots", P), k.get("T", 4), c, None, None)
    for kw in (dict(T=-1), dict(k=None), dict(v=None), dict(slots=None), dict(t=3), dict(h=-8), dict(k=ODD)):
        assert ap(**kw) == tvlib.TV_ERR_INVALID_ARG, kw
    assert ap(T=2**30) == tvlib.TV_ERR_UNSUPPORTED
    assert ap(T=0) == tvlib.TV_OK

    def rd(table=P, q=P, s=P, B=1, T=4, Pg=4, k=P, v=P):
        return lib.tv_paged_read_q8(c, table, q, s, B, T, Pg, k, v, P, None)
    for kw in (dict(B=-1), dict(T=-1), dict(Pg=0), dict(table=None), dict(q=None), dict(s=None), dict(k=None),
               dict(v=ODD)):
        assert rd(**kw) == tvlib.TV_ERR_INVALID_ARG, kw
    for kw in (dict(B=4097), dict(Pg=2**28), dict(B=4096, Pg=2**20)):
        assert rd(**kw) == tvlib.TV_ERR_UNSUPPORTED, kw
    assert rd(B=0) == tvlib.TV_OK
    other = ctypes.c_void_p(0x2000)

    def cm(table=P, kv=P, path=P, acc=P, B=1, N=4, Pg=4, new=other, st=P):
        return lib.tv_commit_paged_q8(c, table, kv, path, acc, B, N, Pg, new, st, None)
    for kw in (dict(B=-1), dict(N=0), dict(N=513), dict(Pg=0), dict(table=None), dict(kv=None), dict(path=None),
               dict(acc=None), dict(new=None), dict(st=None), dict(new=P)):
        assert cm(**kw) == tvlib.TV_ERR_INVALID_ARG, kw
    for kw in (dict(Pg=2**28), dict(B=2**31 - 1)):
        assert cm(**kw) == tvlib.TV_ERR_UNSUPPORTED, kw
    assert cm(B=0) == tvlib.TV_OK


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_plain_quantiser(fmt, dt):
    """The scale is the least that holds the row, each code is the nearest of all the format has, and torch's own
    rounding agrees."""
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(200, 16, generator=g) * torch.exp2(torch.randn(200, 1, generator=g) * 3)).to(dt)
    kind, most = FORMATS[fmt]
    codes, scale = quantise_ref(x, fmt)
    top, e = x.double().abs().amax(1), scale.double() - 127
    assert bool((top <= most * 2.0**e).all()) and bool((top > most * 2.0**(e - 1)).all())
    every = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(kind).float().double()
    every = every[torch.isfinite(every) & (every.abs() <= most)]
    y = x.double() * 2.0**-e[:, None]
    near = (y[..., None] - every).abs()
    assert torch.equal((codes - y).abs(), near.amin(-1))
    again = y.float().to(kind) if fmt == "e4m3" else torch.round(y.float())
    assert torch.equal(again.float().double(), codes)
    assert torch.equal(values_ref(codes, scale).bfloat16().double(), values_ref(codes, scale))


def paged_cache(tv, **kw):
    from speculative_decoding_tree_tv_gb300._lib import PAGED_CACHE_FORMAT
    f = dict(k=0x1000, v=0x1000, page_stride=16 * 64 * 2, head_stride=16 * 64, row_stride=64, num_pages=10,
             page_size=16, Hkv=2, D=64, dtype=0)
    f.update(kw)
    return struct.pack(PAGED_CACHE_FORMAT, *f.values())


ATTN = [(dict(B=-1), 1), (dict(T=-1), 1), (dict(Pg=0), 1), (dict(Hq=0), 1), (dict(Hq=3), 1), (dict(max_q=0), 1),
        (dict(window=-1), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(softcap=-2.0), 1),
        (dict(B=5000), 3), (dict(Hq=2 * 130), 3), (dict(T=2**30), 3), (dict(Pg=2**28), 3),
        (dict(anc=P, max_q=513), 3), (dict(q=None), 1), (dict(out=None), 1), (dict(table=None), 1),
        (dict(q_start=None), 1), (dict(kv_len=None), 1), (dict(q=ODD), 1), (dict(out=ODD), 1), (dict(qt=100), 1),
        (dict(qh=-64), 1), (dict(), 7), (dict(ws=None, n=2**30), 7), (dict(B=0), 0)]


def args(**kw):
    a = dict(q=P, qt=256, qh=64, table=P, q_start=P, kv_len=P, anc=None, slopes=None, B=1, T=4, Pg=4, Hq=4, max_q=4,
             scale=0.0, softcap=0.0, window=0, out=P, lse=None, status=None, ws=P, n=0)
    a.update(kw)
    return a


def tail(a):
    return (a["table"], a["q_start"], a["kv_len"], a["anc"], a["slopes"], a["B"], a["T"], a["Pg"], a["Hq"], a["max_q"],
            a["scale"], a["softcap"], a["window"], a["out"], a["lse"], a["status"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,code", ATTN)
def test_attention_arguments_are_checked(tvlib, kw, code):
    a = args(**kw)
    assert tvlib.lib.tv_attn_paged_q8(a["q"], a["qt"], a["qh"], cache(tvlib), *tail(a)) == code
    assert tvlib.lib.tv_attn_paged_prefix(a["q"], a["qt"], a["qh"], paged_cache(tvlib), P, P, P, 1, 4, *tail(a)) == code


@pytest.mark.parametrize("d", [32, 48, 96, 256])
def test_attention_head_sizes(tvlib, d):
    a = args()
    assert tvlib.lib.tv_attn_paged_q8(a["q"], a["qt"], a["qh"], cache(tvlib, D=d), *tail(a)) == 3
    assert tvlib.lib.tv_attn_paged_prefix(a["q"], a["qt"], a["qh"], paged_cache(tvlib, D=d), P, P, P, 1, 4, *tail(a)) == 3


def test_prefix_arguments_are_checked(tvlib):
    def call(table=P, length=P, start=P, groups=1, prefix_P=4, **kw):
        a = args(**kw)
        return tvlib.lib.tv_attn_paged_prefix(a["q"], a["qt"], a["qh"], paged_cache(tvlib), table, length, start, groups,
                                              prefix_P, *tail(a))
    for kw in (dict(groups=-1), dict(prefix_P=0), dict(table=None), dict(length=None), dict(start=None)):
        assert call(**kw) == tvlib.TV_ERR_INVALID_ARG, kw
    for kw in (dict(groups=4097), dict(groups=4096, prefix_P=2**20), dict(prefix_P=2**27), dict(prefix_P=2**26, Pg=2**26)):
        assert call(**kw) == tvlib.TV_ERR_UNSUPPORTED, kw
    assert call(groups=0, table=None, length=None, start=None) == tvlib.TV_ERR_WORKSPACE  # (as tv_attn_paged)
    assert call(B=0) == tvlib.TV_OK


def test_workspace_sizes(tvlib):
    f = tvlib.lib.tv_attn_paged_prefix_workspace_size
    one = tvlib.lib.tv_attn_paged_workspace_size(1, 8, 2, 64)
    assert f(1, 64, 0, 8, 2, 64) == one
    # both passes' parts, and a 32-bit row with its maximum and sum for each query row
    assert f(1, 64, 1, 8, 2, 64) >= one + 64 * 8 * (64 * 4 + 8)
    for bad in ((0, 64, 1, 8, 2, 64), (1, -1, 1, 8, 2, 64), (1, 64, -1, 8, 2, 64), (1, 64, 1, 7, 2, 64), (1, 64, 1, 8, 2, 80)):
        assert f(*bad) == 0
    g = tvlib.lib.tv_attn_paged_q8_workspace_size
    assert g(1, 8, 2, 64) > 0 and g(1, 8, 2, 80) == 0 and g(0, 8, 2, 64) == 0
