"""Paged-cache entry points without a GPU: refusals before any launch, and the
plain page map of the GPU tests pinned by its own invariants."""
import ctypes
import random
import struct

import pytest

from _paged_util import page_map_ref


@pytest.fixture(scope="module")
def tvlib():
    import __graft_entry__
    __graft_entry__.build()
    import speculative_decoding_tree_tv_gb300 as tv
    return tv


D = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails its checks first
ODD = ctypes.c_void_p(0x1008)


def cache(tv, **kw):
    from speculative_decoding_tree_tv_gb300._lib import PAGED_CACHE_FORMAT
    f = dict(k=0x1000, v=0x1000, page_stride=16 * 64 * 2, head_stride=16 * 64, row_stride=64, num_pages=10,
             page_size=16, Hkv=2, D=64, dtype=0)
    f.update(kw)
    f["k"] = f["k"] or 0
    return struct.pack(PAGED_CACHE_FORMAT, *f.values())


BAD_CACHES = [(dict(num_pages=0), 1), (dict(Hkv=0), 1), (dict(D=0), 1), (dict(dtype=2), 3),
              (dict(page_size=24), 3), (dict(page_size=4), 3), (dict(page_size=512), 3),
              (dict(page_size=0), 3), (dict(page_size=-16), 3), (dict(k=None), 1), (dict(v=0x1008), 1),
              (dict(row_stride=60), 1), (dict(head_stride=-64), 1), (dict(page_stride=1), 1)]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_bad_caches_are_refused(tvlib, kw, code):
    lib, c = tvlib.lib, cache(tvlib, **kw)
    assert lib.tv_paged_append(D, D, 128, 64, D, 4, c, D, None) == code
    assert lib.tv_commit_paged(c, D, D, D, D, 1, 4, 4, D, D, None) == code
    assert attn(lib, c) == code
    assert lib.tv_paged_append(D, D, 128, 64, D, 4, None, D, None) == 1


def attn(lib, c, **kw):
    a = dict(q=D, qt=256, qh=64, table=D, q_start=D, kv_len=D, anc=None, slopes=None, B=1, T=4, P=4, Hq=4,
             max_q=4, scale=0.0, softcap=0.0, window=0, out=D, lse=None, status=None, ws=D, n=0)
    a.update(kw)
    return lib.tv_attn_paged(a["q"], a["qt"], a["qh"], c, a["table"], a["q_start"], a["kv_len"], a["anc"],
                             a["slopes"], a["B"], a["T"], a["P"], a["Hq"], a["max_q"], a["scale"], a["softcap"],
                             a["window"], a["out"], a["lse"], a["status"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), 1), (dict(T=-1), 1), (dict(P=0), 1), (dict(Hq=0), 1), (dict(Hq=3), 1), (dict(max_q=0), 1),
    (dict(window=-1), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(softcap=-2.0), 1),
    (dict(softcap=float("inf")), 1), (dict(B=5000), 3), (dict(Hq=2 * 130), 3), (dict(T=2**30), 3),
    (dict(P=2**28), 3), (dict(anc=D, max_q=513), 3), (dict(q=None), 1), (dict(out=None), 1), (dict(table=None), 1),
    (dict(q_start=None), 1), (dict(kv_len=None), 1), (dict(q=ODD), 1), (dict(out=ODD), 1), (dict(qt=100), 1),
    (dict(qh=-64), 1), (dict(B=0), 0)])
def test_attention_arguments_are_checked(tvlib, kw, code):
    assert attn(tvlib.lib, cache(tvlib), **kw) == code


@pytest.mark.parametrize("d", [32, 96, 256])
def test_attention_head_sizes(tvlib, d):
    assert attn(tvlib.lib, cache(tvlib, D=d)) == 3


def test_page_map_arguments_are_checked(tvlib):
    f = tvlib.lib.tv_page_map

    def call(q_start=D, kv_len=D, B=1, T=4, P=4, page=16, pool=8, table=D, n_pages=D, free=D, n_free=D, slots=D,
             status=D):
        return f(q_start, kv_len, B, T, P, page, pool, table, n_pages, free, n_free, slots, status, None)
    for kw in (dict(B=-1), dict(T=-1), dict(P=0), dict(pool=0), dict(q_start=None), dict(kv_len=None),
               dict(table=None), dict(n_pages=None), dict(free=None), dict(n_free=None), dict(slots=None),
               dict(status=None)):
        assert call(**kw) == tvlib.TV_ERR_INVALID_ARG, kw
    for kw in (dict(page=12), dict(page=4), dict(page=512), dict(B=4097), dict(P=2**28, page=8),
               dict(B=4096, P=2**20), dict(T=2**31 - 1)):
        assert call(**kw) == tvlib.TV_ERR_UNSUPPORTED, kw
    assert call(B=0, T=0) == tvlib.TV_OK


def test_append_and_commit_arguments_are_checked(tvlib):
    lib, c = tvlib.lib, cache(tvlib)
    ap = lambda **k: lib.tv_paged_append(k.get("k", D), k.get("v", D), k.get("t", 128), k.get("h", 64),  # noqa: E731
                                         k.get("slots", D), k.get("T", 4), k.get("c", c), None, None)
    for kw in (dict(T=-1), dict(k=None), dict(v=None), dict(slots=None), dict(t=3), dict(h=-8), dict(k=ODD)):
        assert ap(**kw) == tvlib.TV_ERR_INVALID_ARG, kw
    for kw in (dict(c=cache(tvlib, D=12)), dict(c=cache(tvlib, D=1032)), dict(T=2**30)):
        assert ap(**kw) == tvlib.TV_ERR_UNSUPPORTED, kw
    assert ap(T=0) == tvlib.TV_OK
    other = ctypes.c_void_p(0x2000)

    def cm(c=c, table=D, kv=D, path=D, acc=D, B=1, N=4, P=4, new=other, st=D):
        return lib.tv_commit_paged(c, table, kv, path, acc, B, N, P, new, st, None)
    for kw in (dict(B=-1), dict(N=0), dict(N=513), dict(P=0), dict(table=None), dict(kv=None), dict(path=None),
               dict(acc=None), dict(new=None), dict(st=None), dict(new=D)):
        assert cm(**kw) == tvlib.TV_ERR_INVALID_ARG, kw
    for kw in (dict(c=cache(tvlib, D=12)), dict(P=2**28), dict(B=2**31 - 1)):
        assert cm(**kw) == tvlib.TV_ERR_UNSUPPORTED, kw
    assert cm(B=0) == tvlib.TV_OK


def test_status_string(tvlib):
    assert tvlib.TV_ERR_NO_PAGES == 8
    assert tvlib.status_string(8) == "TV_ERR_NO_PAGES"


def test_binding_refuses_cpu_tensors(tvlib):
    import torch
    i = torch.zeros(1, dtype=torch.int32)
    kv = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        tvlib.page_map(i, i, i[None], i, i, i, 16, 1)
    with pytest.raises(ValueError, match="CUDA"):
        tvlib.paged_append(kv[0], kv[0], torch.zeros(1, dtype=torch.int64), kv, kv)
    with pytest.raises(ValueError, match="CUDA"):
        tvlib.attn_paged(kv[0], kv, kv, i[None], i, i, 1)
    with pytest.raises(ValueError, match="CUDA"):
        tvlib.commit_paged(kv, kv, i[None], i, i[None], i)


@pytest.mark.parametrize("seed", range(30))
def test_plain_page_map_keeps_every_page_once(seed):
    """Pages are neither lost nor held twice, slots are distinct, and releasing
    everything fills the pool."""
    rng = random.Random(seed)
    B, page, P = rng.randint(1, 9), rng.choice([8, 16, 64]), rng.randint(1, 12)
    pool = rng.randint(1, B * P + 3)
    free = list(range(pool))
    rng.shuffle(free)
    table, held, n_free = [[-1] * P for _ in range(B)], [0] * B, pool
    for _ in range(12):
        kv = [rng.randint(0, P * page) for _ in range(B)]
        new = [rng.randint(0, P * page - L) for L in kv]
        q = [0]
        for n in new:
            q.append(q[-1] + n)
        slots, status, n_free = page_map_ref(q, kv, table, held, free, n_free, page, q[-1] + 2)
        everyone = free[:n_free] + [p for b in range(B) for p in table[b][:held[b]]]
        assert sorted(everyone) == list(range(pool))
        got = [s for s in slots if s >= 0]
        assert len(set(got)) == len(got) and slots[-2:] == [-1, -1]
        for b in range(B):
            assert status[b] in (0, 8)
            if status[b] == 0:
                assert held[b] == -(-(kv[b] + new[b]) // page)
            mine = slots[q[b]:q[b + 1]]
            assert all((s < 0) == (status[b] != 0) for s in mine)
    _, status, n_free = page_map_ref([0] * (B + 1), [0] * B, table, held, free, n_free, page, 0)
    assert n_free == pool and status == [0] * B


def test_a_torch_without_the_private_names(tvlib):
    """The package imports, and takes stream and device by torch's public names."""
    import os
    import subprocess
    import sys
    code = ("import torch\n"
            "for name in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, name): delattr(torch._C, name)\n"
            "from speculative_decoding_tree_tv_gb300 import api\n"
            "class Stream: cuda_stream = 77\n"
            "torch.cuda.current_stream = lambda device=None: Stream\n"
            "assert api._raw_stream(0) == 77 and api._current_device is torch.cuda.current_device\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))), timeout=300)
    assert r.returncode == 0, r.stderr


def test_the_workspace_is_sized_for_its_device(tvlib, monkeypatch):
    import torch
    from speculative_decoding_tree_tv_gb300 import api
    inside = []

    class On:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            inside.append(self.device)

        def __exit__(self, *_):
            inside.pop()

    monkeypatch.setattr(api, "_current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(api.lib, "tv_attn_paged_workspace_size", lambda *a: 100 + len(inside))
    assert [tvlib.attn_paged_workspace_size(1, 8, 2, 64, d) for d in (None, "cuda:0", "cuda", "cuda:1")] == \
        [100, 100, 100, 101]
