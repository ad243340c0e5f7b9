"""The 8-bit paged cache on the GPU: its writes, reads and commits against plain forms in whole
numbers and 64-bit floats."""
import math
import random

import numpy as np
import pytest
import torch

from _gpu_util import i32, np_
from _paged_util import DTYPES
from _q8_util import FORMATS, cache, quantise_ref, raw, values_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tv():
    import speculative_decoding_tree_tv_gb300 as m
    return m


def starts(new):
    return [0] + list(np.cumsum(new))


# --------------------------------------------------------------------- write
def written(nk, nv, slots, before, fmt):
    """The cache's bytes after the write, from the definition."""
    k, v, ks, vs = (raw(x).clone().cpu() for x in before)
    page, limit = k.shape[2], k.shape[0] * k.shape[2]
    for x, codes, scales in ((nk, k, ks), (nv, v, vs)):
        c, s = quantise_ref(x, fmt)
        c8 = c.float().to(FORMATS[fmt][0])
        for t, at in enumerate(slots.tolist()):
            if 0 <= at < limit:
                codes[at // page, :, at % page] = c8[t].view(torch.uint8)
                scales[at // page, :, at % page] = s[t].to(torch.uint8)
    return k, v, ks, vs


def same_codes(got, want, fmt):
    """Bytes equal, but for the sign of an e4m3 zero."""
    got, want = raw(got).cpu(), want.clone()
    if fmt == "e4m3":
        zero = (got & 0x7f == 0) & (want & 0x7f == 0)
        want[zero] = got[zero]
    return torch.equal(got, want)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("T,Hkv,D,page,dtype,layout", [
    (1, 1, 64, 8, "bf16", "heads"), (33, 8, 128, 16, "fp16", "rows"), (700, 3, 64, 32, "bf16", "both"),
    (5, 5, 48, 16, "bf16", "heads"), (3000, 8, 128, 64, "bf16", "rows"), (9, 2, 1024, 256, "fp16", "heads"),
    (7, 3, 16, 8, "fp16", "both"), (6, 1, 528, 8, "bf16", "rows")])
@pytest.mark.parametrize("fused", [False, True])
def test_append_writes_the_slots_and_nothing_else(tv, fmt, T, Hkv, D, page, dtype, layout, fused):
    dt, g = DTYPES[dtype], torch.Generator().manual_seed(T)
    pool = -(-T // page) + 3
    before = cache(fmt, pool, Hkv, page, D, layout)
    size = torch.exp2(torch.randn(T, 1, 1, generator=g) * 4)
    x = (torch.randn(T, 3 * Hkv if fused else 2 * Hkv, D, generator=g) * size).to(dt).to("cuda:0")
    nk, nv = x[:, -2 * Hkv:-Hkv], x[:, -Hkv:]
    if not fused:
        nk, nv = nk.contiguous(), nv.contiguous()
    slots = torch.randperm(pool * page, generator=g)[:T]
    bad = torch.rand(T, generator=g)
    slots[bad < 0.1] = -1
    slots[bad > 0.95] = pool * page + (slots[bad > 0.95] % 3) * 2**33
    want = written(nk, nv, slots, before, fmt)
    status = torch.full((T,), 9, dtype=torch.int32, device="cuda:0")
    tv.paged_append_q8(nk, nv, slots.to("cuda:0"), *before, status)
    torch.cuda.synchronize()
    assert same_codes(before[0], want[0], fmt) and same_codes(before[1], want[1], fmt)
    assert torch.equal(before[2].cpu(), want[2]) and torch.equal(before[3].cpu(), want[3])
    assert np_(status).tolist() == [1 if s >= pool * page else 0 for s in slots.tolist()]


def edge_rows(dt, most):
    """Rows [n, 64] at the borders of scales and codes."""
    fin = torch.finfo(dt)
    g = torch.Generator().manual_seed(5)
    rows = [torch.zeros(64), -torch.zeros(64)]
    step = 1.0 + fin.eps
    for e in (-9, -3, 0, 3):  # largest magnitudes just below, at and just above M 2^e
        for f in (1.0, step, 2.0 - step):
            x = torch.randn(64, generator=g).clamp(-1, 1)
            x[7] = -most * 2.0**e * f
            rows.append(x)
    ties = torch.arange(64).float() * 0.5 - 15.75  # codes halfway between whole numbers
    ties[0] = most
    rows.append(ties)
    small = torch.exp2(-torch.arange(64).float() / 4)  # down through an e4m3 row's smallest codes
    small[0] = most / 2**4
    rows += [small, small * fin.tiny * 2, torch.full((64,), fin.smallest_normal * fin.eps)]
    for big in (fin.max, -fin.max):
        x = torch.randn(64, generator=g)
        x[63] = big
        rows.append(x)
    for odd in (math.inf, -math.inf, math.nan):
        x = torch.randn(64, generator=g)
        x[31] = odd
        rows.append(x)
    return torch.stack(rows).to(dt)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_rows_at_the_edges(tv, fmt, dtype):
    x = edge_rows(DTYPES[dtype], FORMATS[fmt][1])[:, None].to("cuda:0")
    T = x.shape[0]
    before = cache(fmt, -(-T // 8), 1, 8, 64)
    want = written(x, -x, torch.arange(T), before, fmt)
    tv.paged_append_q8(x, -x, torch.arange(T, device="cuda:0"), *before)
    assert same_codes(before[0], want[0], fmt) and same_codes(before[1], want[1], fmt)
    assert torch.equal(before[2].cpu(), want[2]) and torch.equal(before[3].cpu(), want[3])
    table = torch.arange(before[0].shape[0], dtype=torch.int32, device="cuda:0")[None]
    k, v, status = tv.paged_read_q8(*before, table, i32([0, T]), i32([0]), T, dtype=DTYPES[dtype])
    assert np_(status).tolist() == [0]
    val = values_ref(want[0].view(FORMATS[fmt][0]), want[2]).transpose(1, 2).reshape(-1, 1, 64)[:T]
    check_read(k, val, DTYPES[dtype])
    check_read(v, -val, DTYPES[dtype])


# ---------------------------------------------------------------------- read
def check_read(got, val, dt):
    """Values rounded to nearest once, the type's largest past it, NaN for NaN."""
    most = torch.finfo(dt).max
    want = val.clamp(-most, most).to(dt)  # (64 bits to 16: nearest, ties to even)
    nan = torch.isnan(val)
    got = got.cpu()
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("lens,Hkv,D,page,layout", [
    ([(0, 1)], 1, 64, 8, "heads"), ([(3, 40), (0, 0), (17, 1), (0, 130)], 8, 128, 16, "rows"),
    ([(0, 3000)], 3, 48, 64, "both"), ([(5, 2)] * 40 + [(0, 0)] * 3, 2, 64, 32, "heads"),
    ([(100, 20), (250, 6)], 1, 1024, 256, "heads")])
def test_read_gives_the_values(tv, fmt, dtype, lens, Hkv, D, page, layout):
    dt, pad = DTYPES[dtype], 5
    held = [-(-(a + n) // page) for a, n in lens]
    pool = sum(held) + 2
    c = cache(fmt, pool, Hkv, page, D, layout, seed=D)
    ids = list(range(pool))
    random.Random(1).shuffle(ids)
    P = max(held) + 1
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-1] * (P - h))
        at += h
    q_start = starts([n for _, n in lens])
    T = q_start[-1] + pad
    k, v = (torch.full((T, Hkv, D), 7.0, dtype=dt, device="cuda:0") for _ in range(2))
    _, _, status = tv.paged_read_q8(*c, i32(table), i32(q_start), i32([a for a, _ in lens]), T, k=k, v=v)
    torch.cuda.synchronize()
    assert np_(status).tolist() == [0] * len(lens)
    val = [values_ref(c[i], c[2 + i]) for i in range(2)]
    for b, (a, n) in enumerate(lens):
        pos = np.arange(a, a + n)
        pages = np.array(table[b])[pos // page]
        for got, w in ((k, val[0]), (v, val[1])):
            check_read(got[q_start[b]:q_start[b] + n], w[pages, :, pos % page], dt)
    assert bool((k[T - pad:] == 7).all()) and bool((v[T - pad:] == 7).all())


def test_read_bad_sequences(tv):
    page, D = 8, 64
    c = cache("int8", 20, 2, page, D)
    table = torch.arange(20, dtype=torch.int32).view(5, 4).to("cuda:0")
    table[3, 1] = 10**6
    lens = [4, 4, 4, 20, 4]
    start = [-1, 29, 28, 0, 2**31 - 2]
    q_start = starts(lens)
    k, v = (torch.full((40, 2, D), 7.0, dtype=torch.bfloat16, device="cuda:0") for _ in range(2))
    _, _, status = tv.paged_read_q8(*c, table, i32(q_start), i32(start), 40, k=k, v=v)
    assert np_(status).tolist() == [1, 1, 0, 1, 1]
    for x in (k, v):
        assert bool((x[:8] == 0).all())          # outside the table
        assert bool((x[20:28] == 0).all())       # the page that is none
        assert bool((x[32:36] == 0).all()) and bool((x[36:] == 7).all())
    # starts that descend: a status, and nothing out of place
    k.fill_(7)
    _, _, status = tv.paged_read_q8(*c, table, i32([0, 9, 4, 50, 50, 50]), i32([0] * 5), 40, k=k, v=v)
    assert np_(status).tolist() == [0, 1, 1, 1, 1]
    assert bool((k[9:] == 7).all())
    tv.paged_read_q8(*c, table[:0], i32([0]), i32([]), 40, k=k, v=v)
    k2, _, status = tv.paged_read_q8(*c, table, i32([0] * 6), i32([0] * 5), 0)
    assert k2.shape == (0, 2, D) and np_(status).tolist() == [0] * 5


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_what_is_read_is_written_back_as_it_was(tv, fmt):
    """A code's value is a bf16 number, so reading rounds nothing, and writing the values again keeps them."""
    T, Hkv, D, page = 300, 4, 128, 16
    g = torch.Generator().manual_seed(2)
    x = (torch.randn(T, 2 * Hkv, D, generator=g) * torch.exp2(torch.randn(T, 1, 1, generator=g) * 3)).bfloat16().cuda()
    c = cache(fmt, 19, Hkv, page, D)
    slots = torch.arange(T, device="cuda:0")
    table = torch.arange(19, dtype=torch.int32, device="cuda:0")[None]
    tv.paged_append_q8(x[:, :Hkv], x[:, Hkv:], slots, *c)
    k, v, _ = tv.paged_read_q8(*c, table, i32([0, T]), i32([0]), T)
    d = cache(fmt, 19, Hkv, page, D, seed=3)
    tv.paged_append_q8(k, v, slots, *d)
    k2, v2, _ = tv.paged_read_q8(*d, table, i32([0, T]), i32([0]), T)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    # and a value is off by half a step at most
    e = torch.from_numpy(quantise_ref(x[:, :Hkv], fmt)[1].numpy() - 127.0)[..., None]
    off, val = (k.cpu().double() - x[:, :Hkv].cpu().double()).abs(), k.cpu().double().abs()
    tol = torch.exp2(e - 1).expand_as(off) if fmt == "int8" else torch.maximum(val * 2.0**-4, torch.exp2(e - 10))
    assert bool((off <= tol).all())


def test_offsets_past_32_bits(tv):
    """Slots whose codes lie past 4 GiB, whose scales past 2^31 elements are not needed for that."""
    Hkv, D, page, pool = 8, 128, 256, 18000
    k, v = (torch.empty(pool, Hkv, page, D, dtype=torch.int8, device="cuda:0") for _ in range(2))
    ks, vs = (torch.zeros(pool, Hkv, page, dtype=torch.uint8, device="cuda:0") for _ in range(2))
    x = torch.randn(4, 2 * Hkv, D, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    slots = torch.tensor([0, pool * page - 1, pool * page - 300, 9000 * page + 5], device="cuda:0")
    tv.paged_append_q8(x[:, :Hkv], x[:, Hkv:], slots, k, v, ks, vs)
    table = torch.tensor([[pool - 1, 0], [pool - 2, 0], [9000, 0]], dtype=torch.int32, device="cuda:0")
    gk, gv, status = tv.paged_read_q8(k, v, ks, vs, table, i32([0, 1, 2, 3]), i32([255, 256 - 44, 5]), 3)
    assert np_(status).tolist() == [0, 0, 0]
    for got, want in ((gk, x[:, :Hkv]), (gv, x[:, Hkv:])):
        check_read(got, values_ref(*quantise_ref(want[1:], "int8")), torch.bfloat16)


# -------------------------------------------------------------------- commit
@pytest.mark.parametrize("B,N,Hkv,D,page,fmt,layout", [
    (1, 2, 1, 64, 8, "e4m3", "heads"), (5, 60, 8, 128, 16, "e4m3", "rows"), (3, 512, 2, 128, 64, "int8", "both"),
    (4, 33, 3, 48, 32, "int8", "heads"), (2, 100, 1, 1024, 256, "e4m3", "heads"), (3, 512, 1, 16, 8, "int8", "heads")])
def test_commit_moves_codes_and_scales(tv, B, N, Hkv, D, page, fmt, layout):
    rng = random.Random(N)
    lens = [rng.randint(0, 3 * page) for _ in range(B)]
    held = [-(-(L + N) // page) for L in lens]
    c = cache(fmt, sum(held) + 2, Hkv, page, D, layout)
    ids = list(range(sum(held) + 2))
    rng.shuffle(ids)
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-1] * (max(held) - h))
        at += h
    acc = [rng.randint(0, min(N - 1, 40)) for _ in range(B)]
    if B > 1:
        acc[0], acc[1] = 0, N - 1
    if B > 2:
        acc[2] = N - 9
    paths = [[0] + sorted(rng.sample(range(1, N), a)) for a in acc]
    want = [raw(x).clone() for x in c]
    for x in want:
        for b, L in enumerate(lens):
            at = lambda i: (table[b][(L + i) // page], slice(None), (L + i) % page)  # noqa: E731
            rows = [x[at(p)].clone() for p in paths[b]]
            for d, r in enumerate(rows):
                x[at(d)] = r
    new_len, status = tv.commit_paged_q8(*c, i32(table), i32(lens), i32([p + [-1] * (N - len(p)) for p in paths]),
                                         i32(acc))
    torch.cuda.synchronize()
    assert np_(status).tolist() == [0] * B
    assert np_(new_len).tolist() == [L + a + 1 for L, a in zip(lens, acc)]
    assert all(torch.equal(raw(x), w) for x, w in zip(c, want))


def test_commit_bad_sequences_move_nothing(tv):
    N, page, B = 8, 8, 9
    c = cache("e4m3", 3 * B, 2, page, 64)
    table = torch.arange(2 * B, dtype=torch.int32).view(B, 2).to("cuda:0")
    good = [0, 2, 3, 5] + [-1] * 4
    path = [list(good) for _ in range(B)]
    acc, kv = [3] * B, [5] * B
    path[0][0] = 1                    # not from node 0
    path[1][2] = 2                    # not ascending
    path[2][3] = N                    # outside the tree
    acc[3], acc[4] = -1, N            # outside [0, N)
    kv[5], kv[6] = -2, 10**9          # a negative length, one past the table
    table[7, 1] = 10**6               # the page of rows 8 and up
    before = [raw(x).clone() for x in c]
    new_len, status = tv.commit_paged_q8(*c, table, i32(kv), i32(path), i32(acc))
    assert np_(status).tolist() == [1] * 8 + [0]
    assert np_(new_len).tolist() == kv[:8] + [9]
    for x, was in zip(c, before):
        assert torch.equal(raw(x)[:16], was[:16]) and torch.equal(raw(x)[18:], was[18:])
        assert not torch.equal(raw(x), was)


# ------------------------------------------------------------------ together
def test_write_commit_read_in_a_graph_on_another_stream(tv):
    T, Hkv, D, page, N = 24, 2, 64, 16, 10
    g = torch.Generator().manual_seed(4)
    c = cache("e4m3", 4, Hkv, page, D)
    x = torch.zeros(T, 2 * Hkv, D, dtype=torch.float16, device="cuda:0")
    table = i32([[2, 0, 3]])
    slots = torch.tensor([table[0, t // page].item() * page + t % page for t in range(T)], device="cuda:0")
    path, acc, kv = i32([[0] * N]), i32([0]), i32([T - N])

    def step():
        tv.paged_append_q8(x[:, :Hkv], x[:, Hkv:], slots, *c)
        new_len, _ = tv.commit_paged_q8(*c, table, kv, path, acc)
        k, v, _ = tv.paged_read_q8(*c, table, i0, kv0, T, dtype=torch.float16)
        return new_len, k, v
    i0, kv0 = i32([0, T]), i32([0])
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            new_len, k, v = step()
        for seed in range(3):
            a = 2 + seed
            p = [0] + sorted(random.Random(seed).sample(range(1, N), a))
            x.copy_(torch.randn(T, 2 * Hkv, D, generator=g))
            path.copy_(i32([p + [-1] * (N - a - 1)]))
            acc.fill_(a)
            graph.replay()
            stream.synchronize()
            assert int(new_len) == T - N + a + 1
            order = list(range(T))
            order[T - N:T - N + a + 1] = [T - N + i for i in p]
            for got, side in ((k, x[:, :Hkv]), (v, x[:, Hkv:])):
                check_read(got, values_ref(*quantise_ref(side, "e4m3"))[order], torch.float16)


def test_refusals_of_the_binding(tv):
    k, v, ks, vs = cache("e4m3", 3, 2, 16, 64)
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda:0")
    slots = torch.arange(4, device="cuda:0")
    table, q_start, start = i32([[0, 1]]), i32([0, 4]), i32([0])
    tv.paged_append_q8(x, x, slots, k, v, ks, vs)
    for bad in ((k.view(torch.uint8), v.view(torch.uint8), ks, vs), (k, v.view(torch.int8), ks, vs),
                (k, v, ks.int(), vs), (None, v, ks, vs)):
        with pytest.raises(TypeError):
            tv.paged_append_q8(x, x, slots, *bad)
    for bad in ((k, v[:2], ks, vs), (k, v, ks[:2], vs), (k, v, ks, vs.transpose(1, 2)), (k, v, ks.cpu(), vs),
                (k.cpu(), v.cpu(), ks, vs), (k[..., ::2], v[..., ::2], ks, vs)):
        with pytest.raises(ValueError):
            tv.paged_append_q8(x, x, slots, *bad)
    with pytest.raises(TypeError):
        tv.paged_append_q8(x.float(), x.float(), slots, k, v, ks, vs)
    with pytest.raises(TypeError):
        tv.paged_append_q8(x, x.half(), slots, k, v, ks, vs)
    with pytest.raises(ValueError):
        tv.paged_append_q8(x[:3], x, slots, k, v, ks, vs)
    with pytest.raises(TypeError):
        tv.paged_read_q8(k, v, ks, vs, table, q_start, start, 4, dtype=torch.float32)
    with pytest.raises(ValueError):
        tv.paged_read_q8(k, v, ks, vs, table, q_start, start, -1)
    with pytest.raises(ValueError):
        tv.paged_read_q8(k, v, ks, vs, table, q_start, start, 4, k=x[:3])
    with pytest.raises(ValueError):
        tv.commit_paged_q8(k, v, ks, vs, table, start, i32([[0], [0]]), i32([0]))
    # strides that are no multiples of 16 bytes, and pages of no power of two
    wide = torch.zeros(2, 3, 2, 16, 72, dtype=torch.int8, device="cuda:0")[..., :64]
    with pytest.raises(tv.TVError):
        tv.paged_append_q8(x, x, slots, wide[0], wide[1], ks, vs)
    with pytest.raises(tv.TVError):
        tv.paged_append_q8(x, x, slots, *cache("int8", 3, 2, 24, 64))


def test_outputs_that_do_not_fit_are_refused(tv):
    c = cache("int8", 3, 2, 16, 64)
    table, q_start, start = i32([[0, 1]]), i32([0, 4]), i32([0])
    x = torch.zeros(4, 2, 64, dtype=torch.float16, device="cuda:0")
    for kw in (dict(k=[0.0]), dict(v=[0.0]), dict(v=x), dict(k=x.float()), dict(k=x, v=x.bfloat16()),
               dict(status=x)):
        with pytest.raises(TypeError):
            tv.paged_read_q8(*c, table, q_start, start, 4, **kw)
    for kw in (dict(k=x.cpu()), dict(k=x[:, :1]), dict(k=x, v=x.transpose(0, 1)), dict(status=i32([0, 0]))):
        with pytest.raises(ValueError):
            tv.paged_read_q8(*c, table, q_start, start, 4, **kw)
    k, v, _ = tv.paged_read_q8(*c, table, q_start, start, 4, k=x)
    assert k is x and v.dtype == torch.float16


def test_read_beside_malformed_starts(tv):
    """Sequences are judged by their own starts, wherever others' lie: rows of one with status 0 are there."""
    page, D, T = 8, 64, 40
    c = cache("e4m3", 20, 2, page, D)
    c[2].clamp_(0, 250)
    c[3].clamp_(0, 250)
    for side in c[:2]:
        side.view(torch.uint8).bitwise_and_(0x3f)  # (codes that are numbers)
    for q_start in ([0, 2, 100, 4, 6], [6, 7, 0, 4, 4], [30, 31, 5, 9, 9], [-3, 2, 5, 30, 30], [0, 9, 4, 9, 12],
                    [0, 50, 50, 3, 8]):
        B = len(q_start) - 1
        table = torch.arange(20, dtype=torch.int32).view(5, 4)[:B].to("cuda:0")
        start = [3, 0, 7, 2][:B]
        k, v = (torch.full((T, 2, D), 7.0, dtype=torch.bfloat16, device="cuda:0") for _ in range(2))
        _, _, status = tv.paged_read_q8(*c, table, i32(q_start), i32(start), T, k=k, v=v)
        status = np_(status).tolist()
        val = [values_ref(c[i], c[2 + i]) for i in range(2)]
        written = torch.zeros(T, dtype=torch.bool)
        spans = [range(a, b) if 0 <= a <= b <= T else range(0) for a, b in zip(q_start, q_start[1:])]
        for b in range(B):
            a, e = q_start[b], q_start[b + 1]
            if not 0 <= a <= e <= T:
                assert status[b] == 1, (q_start, status)
                continue
            alone = not any(set(spans[b]) & set(spans[o]) for o in range(B) if o != b)
            assert status[b] == 0 or not alone, (q_start, status)
            written[a:e] = True
            if status[b] == 0:
                pos = np.arange(start[b], start[b] + e - a)
                pages = np_(table)[b][pos // page]
                for got, w in ((k, val[0]), (v, val[1])):
                    check_read(got[a:e], w[pages, :, pos % page], torch.bfloat16)
        assert bool((k[~written.cuda()] == 7).all()) and bool((v[~written.cuda()] == 7).all())
