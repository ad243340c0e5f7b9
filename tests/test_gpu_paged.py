"""The paged KV cache on the GPU: page map, append, attention and commit against
plain implementations in integers and 64-bit floats, their refusals, and a
verify step of all of them together."""
import math
import random

import numpy as np
import pytest
import torch

from _gpu_util import i32, np_
from _paged_util import DTYPES, attn_ref, check_attn, make, page_map_ref, tree_masks

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tv():
    import speculative_decoding_tree_tv_gb300 as m
    return m


def starts(new):
    return [0] + list(np.cumsum(new))


# ------------------------------------------------------------------ page map
class Pool:
    """Tables of a serving loop, on the GPU and as python lists."""

    def __init__(self, seed, B, P, pool, page):
        rng = random.Random(seed)
        self.page = page
        self.free = list(range(pool))
        rng.shuffle(self.free)
        self.table, self.held, self.n_free = [[-1] * P for _ in range(B)], [0] * B, pool
        self.gpu = dict(table=i32(self.table), held=i32(self.held), free=i32(self.free), n_free=i32([pool]))

    def step(self, tv, q_start, kv_len, T):
        g = self.gpu
        slots, status = tv.page_map(i32(q_start), i32(kv_len), g["table"], g["held"], g["free"], g["n_free"],
                                    self.page, T)
        ref_slots, ref_status, self.n_free = page_map_ref(q_start, kv_len, self.table, self.held, self.free,
                                                          self.n_free, self.page, T)
        assert np_(status).tolist() == ref_status
        owners = [1] * T
        if sorted(q_start) != list(q_start):
            owners = [sum(a <= t < b for a, b in zip(q_start, q_start[1:])) for t in range(T)]
        got = np_(slots).tolist()  # a descending q_start gives some tokens two owners: either's slot
        assert [s for s, n in zip(got, owners) if n < 2] == [s for s, n in zip(ref_slots, owners) if n < 2]
        assert int(g["n_free"]) == self.n_free
        assert np_(g["held"]).tolist() == self.held
        assert np_(g["table"]).tolist() == self.table
        assert np_(g["free"]).tolist() == self.free
        return ref_status


@pytest.mark.parametrize("B,P,page,scarce", [(1, 1, 8, 1.0), (1, 40, 16, 1.0), (7, 12, 8, 0.5), (64, 20, 16, 0.6),
                                             (300, 9, 32, 0.9), (600, 5, 256, 0.4), (1030, 3, 64, 0.7),
                                             (4096, 4, 8, 0.5)])
def test_page_map_follows_the_plain_one(tv, B, P, page, scarce):
    rng = random.Random(B)
    pool = Pool(B, B, P, max(1, int(B * P * scarce)), page)
    seen = set()
    for it in range(6):
        kv = [rng.randint(0, P * page) for _ in range(B)]
        most = [P * page, 3, 40, 1, page, 0][it]
        new = [rng.randint(0, min(most, P * page - L)) for L in kv]
        if B > 1000 and it == 0:
            new = [min(n, 60) for n in new]
        seen |= set(pool.step(tv, starts(new), kv, sum(new) + rng.choice([0, 5])))
    assert 0 in seen
    pool.step(tv, [0] * (B + 1), [0] * B, 0)
    assert pool.n_free == len(pool.free)


def test_page_map_many_tokens(tv):
    """More tokens than one cluster maps (the wide slot launch)."""
    B, P, page = 40, 70, 16
    pool = Pool(3, B, P, B * P - 100, page)
    rng = random.Random(5)
    new = [rng.randint(0, P * page) for _ in range(B)]
    st = pool.step(tv, starts(new), [0] * B, sum(new) + 1500)
    assert set(st) <= {0, 8}


def test_page_map_bad_sequences(tv):
    """Malformed ranges, lengths and page counts are reported and left alone; their
    neighbours are served."""
    B, P, page = 6, 4, 16
    pool = Pool(1, B, P, 30, page)
    pool.step(tv, starts([20] * B), [0] * B, 120)
    pool.step(tv, starts([10, 10, 0, 10, 10, 10]), [20, -3, 20, 100, 20, 60], 50)   # negative, above P pages
    pool.step(tv, [0, 5, 10, 8, 20, 30, 70], [20] * B, 60)      # descending; past T
    pool.step(tv, [-4, 5, 10, 12, 20, 30, 40], [20] * B, 60)    # negative start
    pool.held[2] = -1
    pool.held[3] = P + 1
    pool.gpu["held"].copy_(i32(pool.held))
    pool.step(tv, starts([5] * B), [20] * B, 30)


@pytest.mark.parametrize("n_free", [-1, 31, 29])
def test_page_map_bad_free_count_changes_nothing(tv, n_free):
    B, P, page = 3, 4, 16
    pool = Pool(1, B, P, 30, page)
    pool.step(tv, starts([40] * B), [0] * B, 120)  # 9 pages out, 21 free
    pool.n_free = n_free                           # 29 + the 9 that would come back pass 30
    pool.gpu["n_free"].fill_(n_free)
    assert pool.step(tv, [0] * (B + 1), [0] * B, 4) == [1] * B


def test_page_map_empty_batch(tv):
    z = torch.zeros(0, dtype=torch.int32, device="cuda:0")
    slots, status = tv.page_map(i32([0]), z, z.reshape(0, 4), z, i32([0, 1]), i32([2]), 16, 7)
    assert np_(slots).tolist() == [-1] * 7 and status.numel() == 0


def test_page_map_in_a_graph(tv):
    """A captured step replayed on new lengths in the same buffers."""
    B, P, page, T = 5, 8, 16, 64
    pool = Pool(2, B, P, 30, page)
    g = pool.gpu
    q, kv = i32([0] * (B + 1)), i32([0] * B)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        tv.page_map(q, kv, g["table"], g["held"], g["free"], g["n_free"], page, T)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        slots, status = tv.page_map(q, kv, g["table"], g["held"], g["free"], g["n_free"], page, T)
    rng = random.Random(9)
    for _ in range(4):
        kv_h = [rng.randint(0, 90) for _ in range(B)]
        q_h = starts([rng.randint(0, 12) for _ in range(B)])
        q.copy_(i32(q_h))
        kv.copy_(i32(kv_h))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ref, st, pool.n_free = page_map_ref(q_h, kv_h, pool.table, pool.held, pool.free, pool.n_free, page, T)
        assert np_(slots).tolist() == ref and np_(status).tolist() == st
        assert np_(g["table"]).tolist() == pool.table and int(g["n_free"]) == pool.n_free


# -------------------------------------------------------------------- append
@pytest.mark.parametrize("T,Hkv,D,page,dtype,layout", [
    (1, 1, 64, 8, "bf16", "heads"), (33, 8, 128, 16, "fp16", "rows"), (700, 3, 64, 32, "bf16", "both"),
    (5, 5, 40, 16, "bf16", "heads"), (3000, 8, 128, 64, "bf16", "rows"), (9, 2, 1024, 256, "fp16", "heads")])
@pytest.mark.parametrize("fused", [False, True])
def test_append_writes_the_slots_and_nothing_else(tv, T, Hkv, D, page, dtype, layout, fused):
    dt, g = DTYPES[dtype], torch.Generator().manual_seed(T)
    pool = -(-T // page) + 3
    kv = torch.randn(2, pool, Hkv, page, D, generator=g).to(dt).to("cuda:0")
    if layout == "heads":
        k, v = kv[0], kv[1]
    elif layout == "rows":
        kv = kv.view(2, pool, page, Hkv, D)
        k, v = kv[0].transpose(1, 2), kv[1].transpose(1, 2)
    else:
        kv = kv.view(pool, 2, Hkv, page, D)
        k, v = kv[:, 0], kv[:, 1]
    x = torch.randn(T, 3 * Hkv if fused else 2 * Hkv, D, generator=g).to(dt).to("cuda:0")
    nk, nv = x[:, -2 * Hkv:-Hkv], x[:, -Hkv:]
    if not fused:
        nk, nv = nk.contiguous(), nv.contiguous()
    slots = torch.randperm(pool * page, generator=g)[:T]
    bad = torch.rand(T, generator=g)
    slots[bad < 0.1] = -1
    slots[bad > 0.95] = pool * page + (slots[bad > 0.95] % 3) * 2**33
    ek, ev = k.clone(), v.clone()
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pool * page:
            ek[s // page, :, s % page] = nk[t]
            ev[s // page, :, s % page] = nv[t]
    status = torch.full((T,), 9, dtype=torch.int32, device="cuda:0")
    tv.paged_append(nk, nv, slots.to("cuda:0"), k, v, status)
    torch.cuda.synchronize()
    assert torch.equal(k, ek) and torch.equal(v, ev)
    assert np_(status).tolist() == [1 if s >= pool * page else 0 for s in slots.tolist()]


def test_append_without_tokens(tv):
    k = torch.ones(2, 1, 16, 64, dtype=torch.bfloat16, device="cuda:0")
    x = torch.zeros(0, 1, 64, dtype=torch.bfloat16, device="cuda:0")
    tv.paged_append(x, x, torch.zeros(0, dtype=torch.int64, device="cuda:0"), k, k.clone())
    torch.cuda.synchronize()
    assert bool((k == 1).all())


# -------------------------------------------------------------------- commit
@pytest.mark.parametrize("B,N,Hkv,D,page,dtype,layout", [
    (1, 2, 1, 64, 8, "bf16", "heads"), (5, 60, 8, 128, 16, "bf16", "rows"), (3, 512, 2, 128, 64, "fp16", "both"),
    (4, 33, 3, 40, 32, "bf16", "heads"), (2, 100, 1, 1024, 256, "bf16", "heads")])
def test_commit_moves_the_branch(tv, B, N, Hkv, D, page, dtype, layout):
    rng = random.Random(N)
    lens = [(rng.randint(0, 3 * page), N) for _ in range(B)]
    c = make(N, lens, Hkv, Hkv, D, page, dtype, layout=layout)
    acc = [rng.randint(0, min(N - 1, 40)) for _ in range(B)]
    if B > 1:
        acc[0], acc[1] = 0, N - 1
    paths = [[0] + sorted(rng.sample(range(1, N), a)) for a in acc]
    path = [p + [-1] * (N - len(p)) for p in paths]
    ek, ev = c["k"].clone(), c["v"].clone()
    table = np_(c["table"]).tolist()
    for x in (ek, ev):
        for b, (L, _) in enumerate(lens):
            at = lambda i: (table[b][(L + i) // page], slice(None), (L + i) % page)  # noqa: E731
            rows = [x[at(p)].clone() for p in paths[b]]
            for d, r in enumerate(rows):
                x[at(d)] = r
    new_len, status = tv.commit_paged(c["k"], c["v"], c["table"], c["kv_len"], i32(path), i32(acc))
    torch.cuda.synchronize()
    assert np_(status).tolist() == [0] * B
    assert np_(new_len).tolist() == [L + a + 1 for (L, _), a in zip(lens, acc)]
    for got, want in ((c["k"], ek), (c["v"], ev)):
        assert torch.equal(got.contiguous().view(torch.int16), want.contiguous().view(torch.int16))


def test_commit_bad_sequences_move_nothing(tv):
    N, page = 8, 8
    lens = [(5, N)] * 9
    c = make(3, lens, 2, 2, 64, page)
    good = [0, 2, 3, 5] + [-1] * 4
    path = [list(good) for _ in lens]
    acc, kv = [3] * 9, [5] * 9
    path[0][0] = 1                    # not from node 0
    path[1][2] = 2                    # not ascending
    path[2][3] = N                    # outside the tree
    acc[3], acc[4] = -1, N            # outside [0, N)
    kv[5], kv[6] = -2, 10**9          # a negative length, one past the table
    table = c["table"].clone()
    table[7, 1] = table[7, 1] + 10**6  # the page of rows 8 and up
    before = c["k"].clone().view(torch.int16), c["v"].clone().view(torch.int16)
    new_len, status = tv.commit_paged(c["k"], c["v"], table, i32(kv), i32(path), i32(acc))
    torch.cuda.synchronize()
    assert np_(status).tolist() == [1] * 8 + [0]
    assert np_(new_len).tolist() == kv[:8] + [9]
    mine = set(np_(c["table"])[8].tolist())
    for got, was in zip((c["k"], c["v"]), before):
        for p in range(got.shape[0]):
            if p not in mine:
                assert torch.equal(got[p].view(torch.int16), was[p])
    assert not torch.equal(c["k"].view(torch.int16), before[0])


def test_commit_path_that_leaves_the_table_before_it_falls(tv):
    """A node past the table's end in the middle of a path that then falls: a status, and no entry
    behind the table is looked at (the checked build records one that is)."""
    N, page, L = 8, 8, 9
    c = make(5, [(L, 7)], 2, 2, 64, page)
    table = c["table"][:, :2].contiguous()
    before = [c[x].clone().view(torch.int16) for x in "kv"]
    path = [0, 7, 2] + [-1] * 5
    new_len, status = tv.commit_paged(c["k"], c["v"], table, i32([L]), i32([path]), i32([2]))
    torch.cuda.synchronize()
    assert np_(status).tolist() == [1] and np_(new_len).tolist() == [L]
    assert all(torch.equal(c[x].view(torch.int16), was) for x, was in zip("kv", before))


# ----------------------------------------------------------------- attention
def run(tv, c, pad=0, **kw):
    T, Hq, D = c["q"].shape
    out = torch.full((T, Hq, D), 7.0, dtype=c["q"].dtype, device="cuda:0")
    lse = torch.full((T, Hq), 7.0, device="cuda:0")
    out, lse, status = tv.attn_paged(c["q"], c["k"], c["v"], c["table"], c["q_start"], c["kv_len"], c["max_q"],
                                     anc_mask=c["anc"], out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    n = c["T"]
    assert bool((out[n:] == 7).all()) and bool((lse[n:] == 7).all())  # rows of nobody
    return out[:n], lse[:n], np_(status).tolist()


def agree(tv, c, Hq, Hkv, D, dtype, what="", **kw):
    out, lse, status = run(tv, c, **kw)
    assert status == [0] * len(c["lens"])
    check_attn(out, lse, attn_ref(c, Hq, Hkv, D, **kw), dtype, what)
    return out, lse


DECODE = [[(0, 1)], [(1, 1)], [(63, 1), (64, 1), (65, 1), (0, 1)], [(2500, 1), (3, 1), (0, 1), (700, 1)],
          [(127, 1), (128, 1), (4100, 1)]]


@pytest.mark.parametrize("lens", DECODE)
@pytest.mark.parametrize("Hq,Hkv,D,page,dtype", [(8, 2, 128, 16, "bf16"), (4, 4, 64, 8, "fp16"),
                                                 (7, 1, 128, 256, "bf16"), (16, 1, 64, 64, "bf16"),
                                                 (32, 1, 128, 32, "fp16"), (100, 2, 64, 128, "bf16")])
def test_decode(tv, lens, Hq, Hkv, D, page, dtype):
    c = make(len(lens), lens, Hq, Hkv, D, page, dtype)
    agree(tv, c, Hq, Hkv, D, dtype)


CHUNKS = [[(0, 2)], [(0, 129)], [(200, 33), (0, 0), (5, 64), (130, 1)], [(64, 200), (700, 3)],
          [(1000, 5), (1, 4), (33, 8)], [(0, 1), (0, 0), (2000, 127)]]


@pytest.mark.parametrize("lens", CHUNKS)
@pytest.mark.parametrize("Hq,Hkv,D,page,dtype", [(8, 2, 128, 16, "bf16"), (3, 3, 64, 8, "bf16"),
                                                 (10, 2, 128, 128, "fp16"), (7, 1, 64, 256, "bf16"),
                                                 (64, 1, 128, 32, "bf16")])
def test_causal_chunks(tv, lens, Hq, Hkv, D, page, dtype):
    c = make(len(lens) + 10, lens, Hq, Hkv, D, page, dtype, pad=3)
    agree(tv, c, Hq, Hkv, D, dtype)


TREES = [[(0, 1)], [(100, 4), (0, 3)], [(300, 64), (17, 60), (0, 5), (64, 1)], [(190, 65)], [(40, 300), (0, 7)]]


@pytest.mark.parametrize("lens", TREES)
@pytest.mark.parametrize("Hq,Hkv,D,page,dtype", [(8, 2, 128, 16, "bf16"), (4, 4, 64, 64, "fp16"),
                                                 (8, 1, 64, 8, "bf16")])
def test_trees(tv, lens, Hq, Hkv, D, page, dtype):
    c = make(len(lens) + 20, lens, Hq, Hkv, D, page, dtype, tree=True, pad=2)
    agree(tv, c, Hq, Hkv, D, dtype)


def slopes_of(Hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], device="cuda:0")


KINDS = [dict(softcap=5.0), dict(softcap=50.0, scale=0.7), dict(window=1), dict(window=70), dict(window=10**6),
         dict(slopes=True), dict(slopes=True, softcap=20.0, window=150)]


@pytest.mark.parametrize("kw", KINDS)
@pytest.mark.parametrize("lens,tree", [([(900, 1), (0, 1), (150, 1)], False), ([(300, 200), (0, 40), (77, 1)], False),
                                       ([(260, 70), (0, 9), (129, 1)], True), ([(500, 3), (64, 4)], True)])
@pytest.mark.parametrize("Hq,Hkv,D,page,dtype", [(8, 2, 128, 16, "bf16"), (4, 4, 64, 32, "fp16")])
def test_score_kinds(tv, kw, lens, tree, Hq, Hkv, D, page, dtype):
    kw = dict(kw)
    if kw.get("slopes"):
        kw["slopes"] = slopes_of(Hq)
    c = make(5, lens, Hq, Hkv, D, page, dtype, tree=tree, q_mag=3.0)
    agree(tv, c, Hq, Hkv, D, dtype, **kw)


@pytest.mark.parametrize("window", [33, 128, 300, 700])
@pytest.mark.parametrize("tree", [False, True])
def test_windows_over_many_units(tv, window, tree):
    """Units whose first and last key tiles both hold rows that nobody sees, many to a CTA."""
    lens = [(1500, 90), (130, 250), (0, 400), (777, 40), (255, 129), (5, 33)] * 3
    c = make(window, lens, 16, 8, 64, 16, tree=tree)
    agree(tv, c, 16, 8, 64, "bf16", window=window)


@pytest.mark.parametrize("layout", ["heads", "rows", "both"])
@pytest.mark.parametrize("lens", [[(700, 1), (90, 1)], [(300, 90), (20, 5)]])
def test_cache_layouts(tv, layout, lens):
    """[pages, heads, rows, D], [pages, rows, heads, D] and K, V side by side."""
    c = make(1, lens, 8, 2, 128, 16, layout=layout)
    agree(tv, c, 8, 2, 128, "bf16")


@pytest.mark.parametrize("lens", [[(3000, 1)] * 3, [(2900, 90), (1, 2)], [(0, 1500)]])
def test_same_result_every_time(tv, lens):
    """The split of the key ranges depends on the lengths alone and nothing is added
    in an order that can change."""
    c = make(8, lens, 8, 2, 128, 16)
    a = run(tv, c)
    for _ in range(3):
        b = run(tv, c)
        assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


def test_lengths_do_not_depend_on_the_hint(tv):
    """Chunks longer than max_q says are served too."""
    c = make(4, [(100, 70), (0, 3), (40, 200)], 8, 2, 128, 16)
    want = attn_ref(c, 8, 2, 128)
    for hint in (1, 3, 8, 64, 4000):
        c["max_q"] = hint
        out, lse, status = run(tv, c)
        assert status == [0, 0, 0]
        check_attn(out, lse, want, "bf16", f"max_q {hint}")


@pytest.mark.parametrize("new", [1, 6])
@pytest.mark.parametrize("B", [33, 700])
def test_many_short_sequences(tv, B, new):
    """More sequences than a CTA has threads; some without tokens."""
    rng = random.Random(B)
    lens = [(rng.randint(0, 90), new if rng.random() < 0.9 else 0) for _ in range(B)]
    c = make(B, lens, 8, 2, 64, 16, pad=2)
    agree(tv, c, 8, 2, 64, "bf16")


@pytest.mark.parametrize("lens", [[(70000, 1)], [(30000, 40), (5, 3)]])
def test_long_contexts(tv, lens):
    c = make(2, lens, 4, 1, 64, 64)
    agree(tv, c, 4, 1, 64, "bf16")


def test_the_widest_group(tv):
    """128 query heads of one kv head: a token fills a row block."""
    c = make(3, [(150, 5), (0, 2), (300, 1)], 128, 1, 64, 32)
    agree(tv, c, 128, 1, 64, "bf16")


def test_one_head_and_one_page(tv):
    """Dimensions of extent one, with strides that no one reads."""
    c = make(3, [(3, 2)], 1, 1, 64, 16, spare=0)
    assert c["k"].shape[:2] == (1, 1)
    c["k"], c["v"] = (x.as_strided(x.shape, (7, 3, 64, 1)) for x in (c["k"], c["v"]))
    c["q"] = c["q"].as_strided(c["q"].shape, (c["q"].stride(0), 5, 1))
    agree(tv, c, 1, 1, 64, "bf16")
    slots = torch.tensor([3], device="cuda:0")
    x = torch.randn(1, 1, 64, device="cuda:0").bfloat16().as_strided((1, 1, 64), (9, 11, 1))
    tv.paged_append(x, x, slots, c["k"], c["v"])
    torch.cuda.synchronize()
    assert torch.equal(c["k"][0, 0, 3], x[0, 0]) and torch.equal(c["v"][0, 0, 3], x[0, 0])


def test_offsets_past_32_bits(tv):
    """Pages two billion elements apart."""
    L, n, page, D, Hkv = 20, 6, 16, 64, 2
    c = make(9, [(L, n)], 4, Hkv, D, page, spare=0)
    far = 2**31 + page * D
    flat = [torch.empty(far + page * Hkv * D, dtype=torch.bfloat16, device="cuda:0") for _ in range(2)]
    wide = [f.as_strided((2, Hkv, page, D), (far, page * D, D, 1)) for f in flat]
    for w, x in zip(wide, (c["k"], c["v"])):
        w.copy_(x)
    c["k"], c["v"] = wide
    agree(tv, c, 4, Hkv, D, "bf16")
    d = dict(c, q=c["q"][:1], lens=[(L, 1)], q_start=i32([0, 1]), max_q=1, T=1,
             rows=[tuple(r[:L + 1] for r in c["rows"][0])])
    agree(tv, d, 4, Hkv, D, "bf16")
    x = torch.randn(1, Hkv, D, device="cuda:0").bfloat16()
    last = int(c["table"][0, 1])
    tv.paged_append(x, x, torch.tensor([last * page + 12], device="cuda:0"), *wide)
    # rows 16 .. : the branch [0, 2] moves row 18 to row 17
    before = wide[0][last, :, 2].clone()
    new_len, status = tv.commit_paged(*wide, c["table"], i32([16]), i32([[0, 2, -1]]), i32([1]))
    torch.cuda.synchronize()
    assert np_(status).tolist() == [0] and np_(new_len).tolist() == [18]
    assert torch.equal(wide[0][last, :, 12], x[0]) and torch.equal(wide[0][last, :, 1], before)


def test_large_scores(tv):
    """Rows whose scores differ by hundreds: the running maximum moves far and often."""
    for lens in ([(1500, 1)], [(700, 100)]):
        c = make(6, lens, 4, 1, 128, 16, q_mag=30.0)
        agree(tv, c, 4, 1, 128, "bf16")


def test_values_of_the_types_edge(tv):
    """V near the largest half: sums of weights times values stay in 32 bits."""
    c = make(6, [(300, 40), (500, 1)], 4, 1, 64, 16, "fp16")
    for x in c["rows"]:
        x[1].mul_(8000.0)
    c["v"].mul_(8000.0)
    agree(tv, c, 4, 1, 64, "fp16")


def test_bad_sequences(tv):
    """Lengths that do not fit are reported and zeroed, malformed ranges left alone;
    their neighbours are served."""
    lens = [(40, 3), (20, 3), (60, 3), (10, 3)]
    for extra in (0, 60):  # single-token and many-token kernels
        lens = [(L, n + extra) for L, n in lens]
        c = make(2, lens, 8, 2, 128, 16)
        ref = attn_ref(c, 8, 2, 128)
        n = lens[0][1]
        c["kv_len"][0] = -1
        c["kv_len"][2] = 10**6
        out, lse, status = run(tv, c)
        assert status == [1, 0, 1, 0]
        for b in (0, 2):
            assert bool((out[b * n:(b + 1) * n] == 0).all()) and bool((lse[b * n:(b + 1) * n] == 0).all())
        for b in (1, 3):
            part = tuple(r[b * n:(b + 1) * n] for r in ref)
            check_attn(out[b * n:(b + 1) * n], lse[b * n:(b + 1) * n], part, "bf16")
        c = make(2, lens, 8, 2, 128, 16)
        c["q_start"][2] = c["q_start"][1] - 1   # sequence 1 descends, sequence 2 overlaps sequence 0
        out, lse, status = run(tv, c)
        assert status[1] == 1
        last = tuple(r[3 * n:] for r in ref)
        check_attn(out[3 * n:], lse[3 * n:], last, "bf16")
        c = make(2, lens, 8, 2, 128, 16)
        c["q_start"][4] += 1                    # past T
        out, lse, status = run(tv, c)
        assert status == [0, 0, 0, 1] and bool((out[3 * n:] == 7).all())


@pytest.mark.parametrize("new", [1, 50])
@pytest.mark.parametrize("page", [8, 32, 128, 256])
def test_bad_pages_are_hidden_and_reported(tv, new, page):
    lens = [(600, new), (600, new), (90, new)]
    c = make(3, lens, 8, 2, 128, page)
    c["table"][0, 1] = -5
    c["table"][2, 0] = 10**7
    hidden = {0: set(range(page, min(2 * page, 600 + new))), 2: set(range(min(page, 90 + new)))}
    out, lse, status = run(tv, c)
    assert status == [1, 0, 1]
    ref = attn_ref(c, 8, 2, 128, hidden=hidden)
    check_attn(out, lse, ref, "bf16")


@pytest.mark.parametrize("new", [1, 40])
def test_pages_behind_the_window_may_be_gone(tv, new):
    c = make(3, [(500, new), (100, new)], 4, 2, 64, 16)
    ref = attn_ref(c, 4, 2, 64, window=100)
    gone = (500 - 100 + 1) // 16
    ids = np_(c["table"])[0, :gone].tolist()
    c["table"][0, :gone] = -1
    c["k"][ids] = float("nan")
    c["v"][ids] = float("inf")
    edge = int(c["table"][0, gone])           # rows in front of the window, in its first page
    front = (500 - 100 + 1) % 16
    c["k"][edge, :, :front] = float("nan")
    c["v"][edge, :, :front] = float("nan")
    out, lse, status = run(tv, c, window=100)
    assert status == [0, 0]
    check_attn(out, lse, ref, "bf16")


def test_empty_masks(tv):
    """The masks of an invalid tree: nothing of the tree is seen."""
    c = make(3, [(0, 6), (30, 6)], 4, 2, 64, 16, tree=True)
    c["anc"].zero_()
    out, lse, status = run(tv, c)
    assert status == [0, 0]
    assert bool((out[:6] == 0).all()) and bool((lse[:6] == -math.inf).all())
    assert bool(torch.isfinite(lse[6:]).all()) and bool((out[6:] != 0).any())
    for i in range(6):  # the same prefix for every node: only its query differs
        d = make(3, [(0, 6), (30, 6)], 4, 2, 64, 16)
        q = d["q"][6 + i:7 + i].clone()
        one, lse1, _ = tv.attn_paged(q, d["k"], d["v"], d["table"][1:], i32([0, 1]), i32([29]), 1)
        assert (one.float() - out[6 + i:7 + i].float()).abs().max() <= 2 * 2.0**-8 * 4
        assert (lse1 - lse[6 + i:7 + i]).abs().max() <= 1e-4


def test_no_tokens(tv):
    c = make(3, [(40, 0), (0, 0)], 4, 2, 64, 16, pad=4)
    out, lse, status = run(tv, c)
    assert status == [0, 0] and out.numel() == 0
    q = c["q"][:0]
    out, lse, status = tv.attn_paged(q, c["k"], c["v"], c["table"], c["q_start"], c["kv_len"], 1)
    torch.cuda.synchronize()
    assert out.shape == (0, 4, 64) and np_(status).tolist() == [0, 0]


# (decode tokens; few units, joined by the merge kernel; many, joined by their CTAs; short ones, whole)
@pytest.mark.parametrize("lens", [[(300, 1), (2000, 1)], [(300, 80), (2000, 9)],
                                  [(700 + 40 * i, 64) for i in range(45)], [(90, 1), (70, 1)]])
def test_other_stream_and_graphs(tv, lens):
    """On a stream of its own, and two captured calls replayed at the same time on new
    inputs in the same buffers."""
    cs = [make(s, lens, 8, 2, 128, 16) for s in (1, 2)]
    refs = [attn_ref(c, 8, 2, 128) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    graphs, outs = [], []
    for c, s in zip(cs, streams):
        with torch.cuda.stream(s):
            got = tv.attn_paged(c["q"], c["k"], c["v"], c["table"], c["q_start"], c["kv_len"], c["max_q"])
        s.synchronize()
        check_attn(got[0], got[1], refs[len(graphs)], "bf16")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(tv.attn_paged(c["q"], c["k"], c["v"], c["table"], c["q_start"], c["kv_len"], c["max_q"]))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(5):
        for o in outs:
            o[0].zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, r in zip(outs, refs):
            check_attn(o[0], o[1], r, "bf16")


def test_refusals_of_the_binding(tv):
    c = make(1, [(40, 3)], 4, 2, 64, 16)
    ok = (c["q"], c["k"], c["v"], c["table"], c["q_start"], c["kv_len"], 3)

    def bad(i, x, err, **kw):
        a = list(ok)
        a[i] = x
        with pytest.raises(err):
            tv.attn_paged(*a, **kw)
    bad(0, c["q"].float(), TypeError)
    bad(0, c["q"].half(), TypeError)
    bad(0, c["q"][..., :32], ValueError)
    bad(0, c["q"].transpose(1, 2).contiguous().transpose(1, 2), ValueError)
    bad(0, c["q"][0], ValueError)
    bad(1, c["k"].float(), TypeError)
    bad(2, c["v"].half(), TypeError)
    bad(2, c["v"][:-1], ValueError)
    bad(2, c["v"].transpose(1, 2).contiguous().transpose(1, 2), ValueError)
    bad(3, c["table"].long(), TypeError)
    bad(3, c["table"][0], ValueError)
    bad(4, c["q_start"][:1], ValueError)
    bad(5, c["kv_len"].cpu(), ValueError)
    bad(6, 0, tv.TVError)
    bad(6, 3, ValueError, anc_mask=torch.zeros(2, 1, dtype=torch.int64, device="cuda:0"))
    bad(6, 3, ValueError, slopes=torch.zeros(3, device="cuda:0"))
    bad(6, 3, tv.TVError, softcap=-1.0)
    bad(6, 3, tv.TVError, window=-1)
    bad(6, 3, ValueError, ws=torch.zeros(10, dtype=torch.uint8))
    bad(6, 3, tv.TVError, ws=torch.zeros(256, dtype=torch.uint8, device="cuda:0"))
    bad(6, 3, TypeError, out=torch.zeros(3, 4, 64, device="cuda:0"))
    odd = torch.zeros(c["q"].numel() + 1, dtype=torch.bfloat16, device="cuda:0")[1:].view(c["q"].shape)
    bad(0, odd, tv.TVError)
    torch.cuda.synchronize()


# ------------------------------------------------------------------ together
def test_verify_steps_of_a_paged_batch_equal_the_dense_ones(tv):
    """Speculative steps over the paged cache (page map, append, tree attention,
    greedy acceptance, commit) against the dense entry points on the same rows."""
    B, N, Hq, Hkv, D, page, V = 3, 20, 8, 2, 128, 16, 500
    rng, g = random.Random(4), torch.Generator().manual_seed(4)
    prompt = [37, 5, 130]
    Lcap, P = 320, 20
    pool = Pool(6, B, P, 2 * B * P // 3, page)
    t = pool.gpu
    kp, vp = (torch.full((len(pool.free), Hkv, page, D), float("nan"), dtype=torch.bfloat16, device="cuda:0")
              for _ in range(2))
    kd, vd = (torch.zeros(B, Hkv, Lcap, D, dtype=torch.bfloat16, device="cuda:0") for _ in range(2))
    randn = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to("cuda:0")  # noqa: E731

    def write(kv_len, new, k, v, q_start):
        slots, status = tv.page_map(i32(q_start), kv_len, t["table"], t["held"], t["free"], t["n_free"], page,
                                    q_start[-1])
        assert np_(status).tolist() == [0] * B
        tv.paged_append(k, v, slots, kp, vp)
        for b, L in enumerate(np_(kv_len).tolist()):
            kd[b, :, L:L + new[b]] = k[q_start[b]:q_start[b + 1]].transpose(0, 1)
            vd[b, :, L:L + new[b]] = v[q_start[b]:q_start[b + 1]].transpose(0, 1)

    def close(a, b, u):
        a, b = a.float(), b.float()
        assert (a - b).abs().max() <= 2 * u * b.abs().max().clamp_min(1.0)

    # the prompts in one ragged chunk: each token against its causal prefix
    q0 = starts(prompt)
    kv_len = i32([0] * B)
    write(kv_len, prompt, randn(q0[-1], Hkv, D), randn(q0[-1], Hkv, D), q0)
    q = randn(q0[-1], Hq, D)
    out, lse, status = tv.attn_paged(q, kp, vp, t["table"], i32(q0), kv_len, max(prompt))
    assert np_(status).tolist() == [0] * B
    for b in range(B):
        for i in {0, prompt[b] // 2, prompt[b] - 1}:
            one = torch.ones(1, 1, 1, dtype=torch.int64, device="cuda:0")
            do, dl, _ = tv.attn_verify(q[q0[b] + i].view(1, 1, Hq, D), kd[b:b + 1], vd[b:b + 1], i32([i]), one)
            close(out[q0[b] + i], do[0, 0], 2.0**-8)
            assert (lse[q0[b] + i] - dl[0, 0]).abs().max() <= 1e-4
    kv_len = i32(prompt)
    for step in range(3):
        parent = i32([[-1] + [rng.randrange(max(0, i - 6), i) for i in range(1, N)] for _ in range(B)])
        depth, anc, st = tv.tree_build(parent)
        q1 = starts([N] * B)
        write(kv_len, [N] * B, randn(B * N, Hkv, D), randn(B * N, Hkv, D), q1)
        q = randn(B * N, Hq, D)
        out, lse, status = tv.attn_paged(q, kp, vp, t["table"], i32(q1), kv_len, N, anc_mask=anc.view(B * N, -1))
        dout, dlse, _ = tv.attn_verify(q.view(B, N, Hq, D), kd, vd, kv_len, anc)
        close(out.view(B, N, Hq, D), dout, 2.0**-8)
        assert (lse.view(B, N, Hq) - dlse).abs().max() <= 1e-4
        tokens = torch.randint(0, V, (B, N), generator=g, dtype=torch.int32).to("cuda:0")
        logits = torch.randn(B, N, V, generator=g).to("cuda:0")
        for b in range(B):      # the target agrees with a branch
            node = rng.randrange(N // 2, N)
            while node > 0:
                up = int(parent[b, node])
                logits[b, up, int(tokens[b, node])] = 50.0
                node = up
        acc = tv.accept_greedy(logits, tokens, parent, depth)
        dnew, _ = tv.commit_path(kd, vd, kv_len, acc["path"], acc["accept_len"])
        pnew, status = tv.commit_paged(kp, vp, t["table"], kv_len, acc["path"], acc["accept_len"])
        assert np_(status).tolist() == [0] * B
        assert torch.equal(dnew, pnew) and int(acc["accept_len"].max()) > 0
        kv_len = pnew
        table, lens = np_(t["table"]).tolist(), np_(kv_len).tolist()
        for b in range(B):
            for pos in range(lens[b]):
                p, r = table[b][pos // page], pos % page
                assert torch.equal(kp[p, :, r], kd[b, :, pos]) and torch.equal(vp[p, :, r], vd[b, :, pos])
    # one plain decode token each, then everything is released
    q1 = starts([1] * B)
    write(kv_len, [1] * B, randn(B, Hkv, D), randn(B, Hkv, D), q1)
    q = randn(B, Hq, D)
    out, lse, _ = tv.attn_paged(q, kp, vp, t["table"], i32(q1), kv_len, 1)
    one = torch.ones(B, 1, 1, dtype=torch.int64, device="cuda:0")
    dout, dlse, _ = tv.attn_verify(q.view(B, 1, Hq, D), kd, vd, kv_len, one)
    close(out, dout[:, 0], 2.0**-8)
    assert (lse - dlse[:, 0]).abs().max() <= 1e-4
    tv.page_map(i32([0] * (B + 1)), i32([0] * B), t["table"], t["held"], t["free"], t["n_free"], page, 0)
    assert int(t["n_free"]) == len(pool.free)
    assert sorted(np_(t["free"]).tolist()) == list(range(len(pool.free)))


@pytest.mark.parametrize("G", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("tree,kw", [(False, {}), (True, {}), (True, dict(window=4, slopes=True)),
                                     (False, dict(window=200, softcap=9.0))])
@pytest.mark.parametrize("ctx,page", [(150, 16), (1500, 64)])
def test_small_units_of_either_height(tv, G, tree, kw, ctx, page):
    """1 to 16 rows a unit: both heights of the small units, whole and split."""
    kw = dict(kw)
    if kw.get("slopes"):
        kw["slopes"] = slopes_of(2 * G)
    for n in sorted({1, 8 // G, 8 // G + 1, 16 // G}):
        c = make(G + n, [(ctx, n), (0, max(1, n - 1)), (ctx // 3, n)], 2 * G, 2, 128 if G % 2 else 64, page, tree=tree)
        agree(tv, c, 2 * G, 2, 128 if G % 2 else 64, "bf16", **kw)


def test_two_calls_at_once(tv):
    """Calls that overlap on two streams, each with its own workspace, eager and as two replayed graphs:
    whole, split and joined in the launch, split and merged."""
    cases = [make(i, lens, 8, 2, 128, 16) for i, lens in enumerate(
        [[(700, 64)] * 40, [(3000, 64)], [(900, 1)] * 30, [(100, 1)] * 3, [(50, 300), (2000, 90)] * 8, [(2500, 2)] * 2])]
    call = lambda c: tv.attn_paged(c["q"], c["k"], c["v"], c["table"], c["q_start"], c["kv_len"],  # noqa: E731
                                   c["max_q"])
    bits = lambda r: (r[0].view(torch.int16), r[1])  # noqa: E731
    want = [bits(call(c)) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]

    def same(i, r):
        return all(torch.equal(a, b) for a, b in zip(bits(r), want[i])) and not bool(r[2].any())

    for i in range(0, len(cases), 2):
        got = ([], [])
        for _ in range(8):
            for j, s in enumerate(streams):
                with torch.cuda.stream(s):
                    got[j].append(call(cases[i + j]))
        torch.cuda.synchronize()
        for j in range(2):
            assert all(same(i + j, r) for r in got[j])
        graphs, outs = [], []
        for j, s in enumerate(streams):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[j], stream=s):
                outs.append([call(cases[i + j]) for _ in range(3)])
        for _ in range(5):
            for j, s in enumerate(streams):
                with torch.cuda.stream(s):
                    graphs[j].replay()
        torch.cuda.synchronize()
        for j in range(2):
            assert all(same(i + j, r) for r in outs[j])


def tail_ref(c, b, m, Hq, Hkv, D, **kw):
    """Token range and attn_ref of the last m tokens of sequence b alone."""
    L, n = c["lens"][b]
    end = sum(n for _, n in c["lens"][:b + 1])
    part = dict(c, lens=[(L + n - m, m)], rows=[c["rows"][b]], q=c["q"][end - m:end])
    return slice(end - m, end), attn_ref(part, Hq, Hkv, D, **kw)


# (joined by their CTAs, and by the merge kernel)
@pytest.mark.parametrize("good,bad,rest", [([(100, 20), (700, 64)] * 20, (0, 64), []),
                                           ([(300, 9)] * 3, (0, 70), [(20000, 20)])])
def test_bad_sequences_between_units_of_one_cta(tv, good, bad, rest):
    """A CTA whose share goes from a unit with rows to clear (a ragged last tile) to the many units
    without tiles of a sequence that does not fit: its neighbours are served and no wait runs out."""
    lens = [x for s in good for x in (s, bad)] + rest
    Hq, Hkv, D = 32, 8, 64
    c = make(7, lens, Hq, Hkv, D, 16)
    wrong = set(range(1, 2 * len(good), 2))
    for b in wrong:
        c["kv_len"][b] = 10**6
    out, lse, status = run(tv, c)
    assert status == [int(b in wrong) for b in range(len(lens))]
    at = 0
    for b, (_, n) in enumerate(lens):
        if b in wrong:
            assert bool((out[at:at + n] == 0).all()) and bool((lse[at:at + n] == 0).all())
        elif b < 8 or b >= len(lens) - 2:
            where, ref = tail_ref(c, b, min(n, 9), Hq, Hkv, D)
            check_attn(out[where], lse[where], ref, "bf16", f"sequence {b}")
        at += n


@pytest.mark.parametrize("nodes", [1, 3, 40, 100])
@pytest.mark.parametrize("D,kw", [(64, {}), (128, dict(slopes=True))])
@pytest.mark.parametrize("last", [True, False])
def test_pages_behind_a_trees_window_may_be_gone(tv, nodes, D, kw, last):
    """Row kv_len - window is the first that the root does not see: its page may be gone where it is
    the page's last row, and it may hold NaN where its page stays."""
    L, page = 500, 16
    window = L - (6 * page + 15 if last else 6 * page + 4)
    kw = dict(kw, window=window)
    if kw.get("slopes"):
        kw["slopes"] = slopes_of(4)
    c = make(nodes, [(L, nodes), (30, 2)], 4, 2, D, page, tree=True)
    ref = attn_ref(c, 4, 2, D, **kw)
    ids = np_(c["table"])[0].tolist()
    whole = 7 if last else 6
    c["table"][0, :whole] = -1
    c["k"][ids[:whole]] = float("nan")
    c["v"][ids[:whole]] = float("inf")
    if not last:
        c["k"][ids[6], :, :5] = float("nan")
        c["v"][ids[6], :, :5] = float("nan")
    out, lse, status = run(tv, c, **kw)
    assert status == [0, 0]
    check_attn(out, lse, ref, "bf16")


@pytest.mark.parametrize("nodes", [3, 40])
def test_empty_masks_reach_as_far_as_the_root(tv, nodes):
    """A node whose mask is empty sits at the root's depth: what it sees of the prefix under a
    window is what a token at the prefix's end sees under one that is a row shorter."""
    L, window = 90, 50
    c = make(3, [(L, nodes)], 4, 2, 64, 16, tree=True)
    c["anc"].zero_()
    out, lse, status = run(tv, c, window=window)
    assert status == [0]
    for i in {0, 1, nodes - 1}:
        part = dict(c, lens=[(L - 1, 1)], rows=[tuple(r[:L] for r in c["rows"][0])], q=c["q"][i:i + 1], anc=None)
        check_attn(out[i:i + 1], lse[i:i + 1], attn_ref(part, 4, 2, 64, window=window - 1), "bf16")


@pytest.mark.parametrize("nodes", [20, 90])
@pytest.mark.parametrize("kw", [dict(slopes=True), dict(window=4), dict(slopes=True, window=6, softcap=9.0)])
@pytest.mark.parametrize("Hq", [1, 4])
def test_a_bad_page_inside_a_tree(tv, nodes, kw, Hq):
    """Hidden nodes still count for the depth of those behind them (both kernels: 20 nodes of one head
    are handed to the small one by the hint below)."""
    L, page = 37, 8
    kw = dict(kw)
    if kw.get("slopes"):
        kw["slopes"] = -8 * slopes_of(Hq)  # (what lies far back matters)
    c = make(nodes, [(L, nodes), (50, 3)], Hq, 1, 64, page, tree=True)
    W = (nodes + 63) // 64
    c["max_q"] = min(nodes, 16) if Hq == 1 and W == 1 else nodes
    c["table"][0, 5] = -1
    hidden = {0: set(range(5 * page, 6 * page))}
    out, lse, status = run(tv, c, **kw)
    assert status == [1, 0]
    check_attn(out, lse, attn_ref(c, Hq, 1, 64, hidden=hidden, **kw), "bf16")


# (small units, whole and split; larger ones whole, merged, and joined by their CTAs)
NAN_LENS = [[(90, 1), (128, 1)], [(300, 1), (2048, 1), (64, 1)], [(50, 40), (120, 9)], [(300, 80), (2040, 9)],
            [(700 + 40 * i, 64) for i in range(45)]]


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


@pytest.mark.parametrize("lens", NAN_LENS)
@pytest.mark.parametrize("kw", [{}, dict(softcap=30.0), dict(window=40)])
def test_nan_in_a_query_row(tv, lens, kw):
    """The row's out and lse are NaN, whichever way its unit is cut; no other row changes."""
    c = make(3, lens, 8, 2, 128, 16)
    want = run(tv, c, **kw)
    last = [s - 1 for s in starts([n for _, n in lens])[1:]]
    c["q"] = c["q"].clone()
    for b, t in enumerate(last):
        c["q"][t, b % 8, 5] = float("nan")
    out, lse, status = run(tv, c, **kw)
    assert status == [0] * len(lens)
    for b, t in enumerate(last):
        assert bool(out[t, b % 8].isnan().all()) and bool(lse[t, b % 8].isnan())
        out[t, b % 8], lse[t, b % 8] = want[0][t, b % 8], want[1][t, b % 8]
    assert same_bits(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("lens", NAN_LENS)
@pytest.mark.parametrize("kw", [{}, dict(softcap=30.0), dict(window=40)])
@pytest.mark.parametrize("where", ["last", "middle", "first"])
def test_nan_in_a_key(tv, lens, kw, where):
    """Tokens that see the key get NaN (alone in its tile or not, in one part of a unit or another);
    tokens that do not are as they were."""
    c = make(4, lens, 8, 2, 128, 16)
    want = run(tv, c, **kw)
    sees, at = [], 0
    table = np_(c["table"])
    for b, (L, n) in enumerate(lens):
        j = dict(last=L + n - 1, middle=L + n // 2, first=0)[where]
        c["k"][table[b, j // 16], :, j % 16, 3] = float("nan")
        sees += [L + i >= j and L + i - j < kw.get("window", 10**9) for i in range(n)]
    out, lse, status = run(tv, c, **kw)
    assert status == [0] * len(lens)
    sees = torch.tensor(sees, device="cuda:0")
    assert bool(out[sees].isnan().all()) and bool(lse[sees].isnan().all())
    assert same_bits(out[~sees], want[0][~sees]) and torch.equal(lse[~sees], want[1][~sees])


@pytest.mark.parametrize("softcap", [1e-42, 1e-30, 1e-7, 9e3, 1e5, 1e8, 1e30, 3.4e38])
@pytest.mark.parametrize("lens", [[(300, 1), (5, 1)], [(200, 40)]])
def test_caps_of_any_size(tv, softcap, lens):
    """A large cap leaves scores as they are, a small one makes them equal.  attn_ref's bound on a score
    holds 8 roundings of the cap, which say nothing for a large one: without them it is the bound of the
    uncapped scores, and the cubic's 2^-22 and its seven roundings of the score (below 8 * 2^-23 of
    the terms' magnitudes, of which the bound has D + 4 = 68) make it 9 / 8 of that at most."""
    c = make(3, lens, 4, 1, 64, 16, q_mag=3.0)
    c["q"] = c["q"].clone()
    c["q"][0, 0] = 0
    out, lse, status = run(tv, c, softcap=softcap)
    assert status == [0] * len(lens)
    ref, plain = attn_ref(c, 4, 1, 64, softcap=softcap), attn_ref(c, 4, 1, 64)
    check_attn(out, lse, ref[:3] + (plain[3] * 1.125 if softcap > 1 else ref[3],) + ref[4:], "bf16")


@pytest.mark.parametrize("lens", [[(200, 37)], [(500, 35), (0, 33)]])
@pytest.mark.parametrize("Hq,D", [(8, 64), (10, 128)])
def test_capped_rows_do_not_depend_on_rows_past_the_unit(tv, lens, Hq, D):
    """What the rows behind a unit's tokens hold (the query box reaches over them) changes no bit."""
    got = []
    for fill in (0.0, 1000.0, float("nan")):
        c = make(3, lens, Hq, 2, D, 16, pad=40)
        c["q"] = c["q"].clone()
        c["q"][c["T"]:] = fill
        got.append(run(tv, c, softcap=9.0))
        assert got[-1][2] == [0] * len(lens)
    for g in got[1:]:
        assert same_bits(g[0], got[0][0]) and torch.equal(g[1], got[0][1])


# (small units, whole and merged; larger ones whole, merged, and joined by their CTAs; more sequences
# than a CTA has threads)
@pytest.mark.parametrize("lens", [[(90, 1), (0, 0), (128, 1)], [(300, 1), (0, 0), (2048, 1), (64, 1)],
                                  [(50, 40), (9, 0), (120, 9)], [(300, 80), (7, 0), (2040, 9)],
                                  [(700 + 40 * i, 64) for i in range(45)] + [(5, 0)],
                                  [(60, 2)] * 450 + [(3, 0)], [(40, 20)] * 450])
def test_a_wait_that_runs_out_is_reported(tv, lens):
    """Failure detection without a fault: with a limit of 0 the tiles that a CTA waits for never come.
    Every sequence with tokens says so, and no other; the next call is right."""
    c = make(5, lens, 8, 2, 64, 16)
    call = lambda: tv.attn_paged(c["q"], c["k"], c["v"], c["table"], c["q_start"], c["kv_len"],  # noqa: E731
                                 c["max_q"])
    want = call()
    torch.cuda.synchronize()
    try:
        assert tv.lib.tv_debug_set_wait_limit(0) == tv.TV_OK
        late = call()
        torch.cuda.synchronize()
    finally:
        assert tv.lib.tv_debug_set_wait_limit(tv.TV_WAIT_LIMIT_DEFAULT) == tv.TV_OK
    assert np_(late[2]).tolist() == [tv.TV_ERR_TIMEOUT if n else 0 for _, n in lens]
    got = call()
    torch.cuda.synchronize()
    assert np_(got[2]).tolist() == [0] * len(lens)
    assert same_bits(got[0], want[0]) and torch.equal(got[1], want[1])
    if tv.CHECKED:  # (this build records the site of a wait that gave up)
        tv.check_take()


def test_strides_of_extent_one_may_differ(tv):
    """One token from two projections, and a cache of one page whose K and V are cut from different pools."""
    g = torch.Generator().manual_seed(2)
    randn = lambda *s: torch.randn(*s, generator=g).bfloat16().to("cuda:0")  # noqa: E731
    qkv, v = randn(1, 12, 64), randn(1, 2, 64)
    k = qkv[:, 8:10]
    pool = randn(3, 2, 2, 16, 64)
    kp, vp = pool[1:2, 0], randn(1, 2, 16, 64)
    assert k.stride() != v.stride() and kp.stride() != vp.stride()
    tv.paged_append(k, v, torch.tensor([5], device="cuda:0"), kp, vp)
    out, lse, status = tv.attn_paged(qkv[:, :8], kp, vp, i32([[0]]), i32([0, 1]), i32([5]), 1)
    c = dict(lens=[(5, 1)], rows=[tuple(x[0, :, :6].transpose(0, 1).cpu() for x in (kp, vp))], q=qkv[:, :8], anc=None)
    torch.cuda.synchronize()
    assert torch.equal(kp[0, :, 5], k[0]) and torch.equal(vp[0, :, 5], v[0]) and int(status) == 0
    check_attn(out, lse, attn_ref(c, 8, 2, 64), "bf16")
    with pytest.raises(ValueError, match="same strides"):
        tv.paged_append(qkv.repeat(2, 1, 1)[:, 8:10], v.repeat(2, 1, 1), torch.tensor([5, 6], device="cuda:0"), kp, vp)
    with pytest.raises(ValueError, match="contiguous"):
        wide = randn(1, 2, 16, 128)[..., ::2]
        tv.paged_append(k, v, torch.tensor([5], device="cuda:0"), wide, wide)
    with pytest.raises(ValueError, match="contiguous"):
        tv.paged_append(randn(1, 2, 128)[..., ::2], v, torch.tensor([5], device="cuda:0"), kp, vp)


def test_page_map_refuses_other_free_lists(tv):
    z = i32([0])
    for free, err in (([0, 1], TypeError), (i32([[0, 1]]), ValueError), (torch.zeros(2, device="cuda:0"), TypeError),
                      (torch.zeros(2, dtype=torch.int32), ValueError)):
        with pytest.raises(err, match="free_list"):
            tv.page_map(i32([0, 0]), z, i32([[0]]), z, free, z, 16, 0)


@pytest.mark.parametrize("T", [40, 20000])
def test_page_map_serves_sequences_behind_a_descent(tv, T):
    """Sequence 1 descends; the tokens of those behind it belong to them alone and get their slots."""
    B, P, page = 6, 8, 16
    pool = Pool(4, B, P, 44, page)
    pool.step(tv, starts([20] * B), [0] * B, 120)
    assert pool.step(tv, [20, 30, 5, 10, 12, 12, 19], [20, 7, 20, 90, 3, 33], T) == [0, 1, 0, 0, 0, 0]
    assert pool.step(tv, [T - 3, T, 0, 2, 1, 9, 9], [20] * B, T) == [0, 1, 0, 1, 0, 0]


@pytest.mark.parametrize("N", [5, 40])
def test_verify_steps_as_a_replayed_graph(tv, N):
    """The whole step (tree, page map, append, attention, acceptance, commit, the next lengths) captured once
    and replayed on new inputs in the same buffers: every bit as in eager steps."""
    B, Hq, Hkv, D, page, V, P, pool = 3, 8, 2, 128, 16, 300, 9, 24
    g, rng = torch.Generator().manual_seed(N), random.Random(N)
    randn = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to("cuda:0")  # noqa: E731
    free = list(range(pool))
    rng.shuffle(free)

    def state():
        return dict(kp=torch.zeros(pool, Hkv, page, D, dtype=torch.bfloat16, device="cuda:0"),
                    vp=torch.zeros(pool, Hkv, page, D, dtype=torch.bfloat16, device="cuda:0"),
                    table=i32([[-1] * P] * B), held=i32([0] * B), free=i32(free), n_free=i32([pool]),
                    kv_len=i32([0] * B), q_start=i32(starts([N] * B)))

    def inputs():
        parent = [[-1] + [rng.randrange(max(0, i - 4), i) for i in range(1, N)] for _ in range(B)]
        logits = torch.randn(B, N, V, generator=g)
        tokens = torch.randint(0, V, (B, N), generator=g, dtype=torch.int32)
        for b in range(B):  # the target agrees with a branch
            node = rng.randrange(N)
            while node > 0:
                logits[b, parent[b][node], int(tokens[b, node])] = 50.0
                node = parent[b][node]
        return dict(q=randn(B * N, Hq, D), k=randn(B * N, Hkv, D), v=randn(B * N, Hkv, D), parent=i32(parent),
                    logits=logits.to("cuda:0"), tokens=tokens.to("cuda:0"))

    def step(s, x):
        depth, anc, st0 = tv.tree_build(x["parent"])
        slots, st1 = tv.page_map(s["q_start"], s["kv_len"], s["table"], s["held"], s["free"], s["n_free"], page, B * N)
        tv.paged_append(x["k"], x["v"], slots, s["kp"], s["vp"])
        out, lse, st2 = tv.attn_paged(x["q"], s["kp"], s["vp"], s["table"], s["q_start"], s["kv_len"], N,
                                      anc_mask=anc.view(B * N, -1))
        acc = tv.accept_greedy(x["logits"], x["tokens"], x["parent"], depth)
        new_len, st3 = tv.commit_paged(s["kp"], s["vp"], s["table"], s["kv_len"], acc["path"], acc["accept_len"])
        s["kv_len"].copy_(new_len)
        return out, lse, slots, acc["accept_len"], torch.stack([st0, st1, st2, st3])

    a, b, buf = state(), state(), inputs()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step(state(), buf)  # (the workspaces that are kept)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = step(b, buf)
    moved = 0
    for _ in range(6):
        x = inputs()
        want = step(a, x)
        for name, t in x.items():
            buf[name].copy_(t)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert not bool(want[4].any()) and all(torch.equal(p, q) for p, q in zip(want, got))
        assert all(torch.equal(a[n], b[n]) for n in a)
        moved += int(want[3].sum())
    assert moved > 0


def test_sizes_past_an_int_are_not_cut(tv):
    """No argument loses its upper bits on the way to the library."""
    c = make(1, [(40, 3)], 4, 2, 64, 16)
    want = run(tv, c)
    for window in (2**31, 2**32 + 5, 2**63 - 1):
        got = run(tv, c, window=window)
        assert same_bits(got[0], want[0]) and torch.equal(got[1], want[1])
    wide = torch.zeros((0, 2**32 + 4), dtype=torch.int32, device="cuda:0")
    z = i32([0])
    for bad in (lambda: tv.page_map(i32([0, 0]), z, c["table"], z, z, z, 16, 2**32),
                lambda: tv.page_map(i32([0, 0]), z, c["table"], z, z, z, 16, -1),
                lambda: tv.page_map(i32([0, 0]), z, c["table"], z, z, z, 2**32 + 16, 0),
                lambda: tv.page_map(i32([0]), z[:0], wide, z[:0], z, z, 16, 0),
                lambda: tv.attn_paged(c["q"], c["k"], c["v"], c["table"], c["q_start"], c["kv_len"], 2**32 + 3),
                lambda: tv.attn_paged(c["q"], c["k"], c["v"], wide, i32([0]), z[:0], 3),
                lambda: tv.commit_paged(c["k"], c["v"], wide, z[:0], wide[:, :3].contiguous(), z[:0])):
        with pytest.raises(ValueError, match="2\\^31"):
            bad()


@pytest.mark.parametrize("kw", [{}, dict(slopes=True, window=120)])
def test_chunks_and_tokens_among_trees(tv, kw):
    """In a call with masks a chunk is a chain and a decode token a tree of one node."""
    kw = dict(kw)
    if kw.get("slopes"):
        kw["slopes"] = slopes_of(8)
    lens = [(300, 64), (100, 130), (50, 1), (0, 40)]
    c = make(3, lens, 8, 2, 64, 16, tree=True)
    c["parents"][1] = list(range(-1, 129))
    W = (130 + 63) // 64
    words, c["depth"] = tree_masks(c["parents"], W)
    c["anc"] = torch.tensor(words, dtype=torch.int64, device="cuda:0")
    out, lse = agree(tv, c, 8, 2, 64, "bf16", **kw)
    for b in (1, 2):  # as without masks
        L, n = lens[b]
        t = sum(m for _, m in lens[:b])
        part = dict(c, lens=[lens[b]], rows=[c["rows"][b]], q=c["q"][t:t + n], anc=None)
        check_attn(out[t:t + n], lse[t:t + n], attn_ref(part, 8, 2, 64, **kw), "bf16")


@pytest.mark.parametrize("lens,tree", [([(300, 1), (5, 1), (900, 1)], False), ([(200, 80), (30, 3)], False),
                                       ([(200, 20), (30, 3)], True)])
def test_tables_as_wide_as_the_longest_permitted_sequence(tv, lens, tree):
    """A server's block table: most of a row is never held."""
    c = make(3, lens, 8, 2, 64, 16, tree=tree)
    c["table"] = torch.nn.functional.pad(c["table"], (0, 8192), value=-1)
    agree(tv, c, 8, 2, 64, "bf16")


@pytest.mark.parametrize("lens", [[(300, 1), (20, 1)], [(200, 80), (30, 3)], [(700 + 40 * i, 64) for i in range(45)]])
def test_output_rows_between_sectors(tv, lens):
    """out on a 16-byte boundary that is no 32-byte one, written into a larger buffer."""
    c = make(3, lens, 8, 2, 64, 16)
    want = tv.attn_paged(c["q"], c["k"], c["v"], c["table"], c["q_start"], c["kv_len"], c["max_q"])[0]
    flat = torch.full((want.numel() + 16,), 7.0, dtype=torch.bfloat16, device="cuda:0")
    out = flat[8:-8].view(want.shape)
    assert out.data_ptr() % 32 == 16
    tv.attn_paged(c["q"], c["k"], c["v"], c["table"], c["q_start"], c["kv_len"], c["max_q"], out=out)
    torch.cuda.synchronize()
    assert same_bits(out, want) and bool((flat[:8] == 7).all()) and bool((flat[-8:] == 7).all())


@pytest.mark.parametrize("lens", [[(300, 1), (20, 1)], [(200, 80), (30, 3)]])
def test_pages_inside_heads(tv, lens):
    """A [heads, pages, rows, D] cache, the fourth order of the outer dimensions."""
    c = make(3, lens, 8, 4, 128, 32)
    for x in "kv":
        c[x] = c[x].transpose(0, 1).contiguous().transpose(0, 1)
    assert c["k"].stride(1) > c["k"].stride(0)
    agree(tv, c, 8, 4, 128, "bf16")


@pytest.mark.parametrize("lens", [[(300, 1), (20, 1)], [(200, 80), (30, 3)]])
def test_tokens_before_the_first_sequence(tv, lens):
    """q_start need not begin at 0: the tokens in front belong to nobody."""
    c = make(3, lens, 8, 2, 64, 16)
    front = 5
    c["q"] = torch.cat([torch.full_like(c["q"][:1], float("nan")).repeat(front, 1, 1), c["q"]])
    q_start = c["q_start"] + front
    out = torch.full(c["q"].shape, 7.0, dtype=torch.bfloat16, device="cuda:0")
    out, lse, status = tv.attn_paged(c["q"], c["k"], c["v"], c["table"], q_start, c["kv_len"], c["max_q"], out=out)
    torch.cuda.synchronize()
    assert np_(status).tolist() == [0] * len(lens) and bool((out[:front] == 7).all())
    c["q"] = c["q"][front:]
    check_attn(out[front:], lse[front:], attn_ref(c, 8, 2, 64), "bf16")


@pytest.mark.parametrize("lens", [[(1500, 1), (40, 1)], [(700, 100)]])
def test_negative_slopes(tv, lens):
    """What lies far back weighs most: the maximum moves with every tile."""
    c = make(6, lens, 4, 1, 64, 16)
    agree(tv, c, 4, 1, 64, "bf16", slopes=-slopes_of(4))


def test_the_most_sequences(tv):
    rng = random.Random(1)
    lens = [(rng.randint(0, 40), int(rng.random() < 0.8)) for _ in range(4096)]
    c = make(1, lens, 2, 1, 64, 8, pad=3)
    agree(tv, c, 2, 1, 64, "bf16")
    pool = Pool(2, 4096, 6, 4096 * 6, 8)
    pool.step(tv, starts([n for _, n in lens]), [L for L, _ in lens], c["T"])


@pytest.mark.parametrize("lens", [[(300, 1), (75, 1), (1000, 1)], [(70, 1), (30, 1)], [(90, 2), (700, 1)],
                                  [(200, 37), (500, 33)], [(70, 9), (3000, 40)]])
@pytest.mark.parametrize("Hq,D", [(8, 64), (16, 128)])
@pytest.mark.parametrize("window", [0, 41])
def test_capped_rows_do_not_depend_on_rows_nobody_sees(tv, lens, Hq, D, window):
    """What cache rows behind a sequence's end and in front of its window hold changes no bit."""
    got = []
    for fill in (0.0, 1000.0, float("nan")):
        c = make(3, lens, Hq, 2, D, 16)
        for x in "kv":
            c[x] = torch.where(c[x].isnan(), torch.full_like(c[x], fill), c[x])
        if window:
            table = np_(c["table"])
            for b, (L, n) in enumerate(lens):
                for j in range(max(0, L - window + 1)):
                    c["k"][table[b, j // 16], :, j % 16] = fill
                    c["v"][table[b, j // 16], :, j % 16] = fill
        got.append(run(tv, c, softcap=9.0, window=window))
        assert got[-1][2] == [0] * len(lens)
    assert bool(torch.isfinite(got[0][0]).all())
    for g in got[1:]:
        assert same_bits(g[0], got[0][0]) and torch.equal(g[1], got[0][1])
