"""Attention of sequences that share prefixes, on the GPU against 64-bit floats over each sequence's whole rows:
chunks, trees, groups of all kinds, score kinds, bad data, and a serving loop."""
import math
import random

import numpy as np
import pytest
import torch

from _gpu_util import i32, np_
from _paged_util import attn_ref, check_attn, make, random_tree, tree_masks

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tv():
    import speculative_decoding_tree_tv_gb300 as m
    return m


def starts(new):
    return [0] + list(np.cumsum(new))


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


def shared(seed, groups, Hq, Hkv, D, page, dtype="bf16", first=(), last=(), **kw):
    """A case of groups [(prefix rows, [(own cached, new), ..]), ..]; `first` and `last` are sequences outside of
    them.  c["full"]: the case of the sequences with their prefixes in front of their own rows, for attn_ref."""
    own = list(first) + [s for _, seqs in groups for s in seqs] + list(last)
    G = len(groups)
    c = make(seed, [(S, 0) for S, _ in groups] + own, Hq, Hkv, D, page, dtype, **kw)
    c["pre_table"], c["table"] = c["table"][:G].contiguous(), c["table"][G:].contiguous()
    c["pre_len"], c["kv_len"] = c["kv_len"][:G].contiguous(), c["kv_len"][G:].contiguous()
    c["q_start"] = c["q_start"][G:].contiguous()
    bounds = [len(first) + x for x in starts([len(seqs) for _, seqs in groups])]
    c["group_start"] = i32(bounds)
    of = [-1] * len(first) + [g for g, (_, seqs) in enumerate(groups) for _ in seqs] + [-1] * len(last)
    full = dict(c)
    full["lens"] = [(L + (groups[g][0] if g >= 0 else 0), n) for g, (L, n) in zip(of, own)]
    full["rows"] = [tuple(torch.cat([c["rows"][g][i], c["rows"][G + b][i]]) if g >= 0 else c["rows"][G + b][i]
                          for i in range(2)) for b, g in enumerate(of)]
    if c["anc"] is not None:
        full["parents"] = c["parents"][G:]
    c["own"], c["of"], c["full"] = own, of, full
    return c


def run(tv, c, **kw):
    T, Hq, D = c["q"].shape
    out = torch.full((T, Hq, D), 7.0, dtype=c["q"].dtype, device="cuda:0")
    lse = torch.full((T, Hq), 7.0, device="cuda:0")
    out, lse, status = tv.attn_paged_prefix(c["q"], c["k"], c["v"], c["pre_table"], c["pre_len"], c["group_start"],
                                            c["table"], c["q_start"], c["kv_len"], c["max_q"], anc_mask=c["anc"],
                                            out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    n = c["T"]
    assert bool((out[n:] == 7).all()) and bool((lse[n:] == 7).all())  # rows of nobody
    return out[:n], lse[:n], np_(status).tolist()


def agree(tv, c, Hq, Hkv, D, dtype, **kw):
    out, lse, status = run(tv, c, **kw)
    assert status == [0] * len(c["own"])
    if c["T"] == 0:  # (attn_ref wants a token)
        return out, lse
    check_attn(out, lse, attn_ref(c["full"], Hq, Hkv, D, **kw), dtype)
    return out, lse


SHAPES = [(8, 2, 128, 16, "bf16"), (4, 4, 64, 8, "fp16"), (7, 1, 128, 256, "bf16"), (16, 1, 64, 64, "bf16"),
          (32, 1, 128, 32, "fp16"), (3, 3, 64, 128, "bf16")]
DECODE = [[(1, [(0, 1)])], [(500, [(5, 1), (60, 1), (17, 1)])], [(128, [(0, 1)] * 9), (0, [(300, 1), (2, 1)])],
          [(3000, [(i, 1) for i in range(40)]), (127, [(90, 1)]), (64, [])], [(4000, [(1500, 1), (3, 1)])]]
CHUNKS = [[(200, [(0, 33), (5, 64), (130, 1)])], [(64, [(0, 2), (0, 0), (700, 3)]), (129, [(1, 200)])],
          [(1000, [(20, 5), (1, 4), (33, 8)]), (0, [(0, 40)])], [(2000, [(40, 9)] * 12)], [(100, [(0, 0)]), (7, [])]]


@pytest.mark.parametrize("groups", DECODE + CHUNKS)
@pytest.mark.parametrize("Hq,Hkv,D,page,dtype", SHAPES)
def test_causal(tv, groups, Hq, Hkv, D, page, dtype):
    c = shared(len(groups), groups, Hq, Hkv, D, page, dtype, pad=3)
    agree(tv, c, Hq, Hkv, D, dtype)


@pytest.mark.parametrize("groups", [[(300, [(40, 4), (0, 3), (9, 7)])], [(1500, [(17, 60), (0, 5), (64, 1)]), (33, [(5, 64)])],
                                    [(70, [(190, 65)])], [(260, [(40, 300), (0, 7)])], [(900, [(20, 1)] * 5)]])
@pytest.mark.parametrize("Hq,Hkv,D,page,dtype", SHAPES[:3])
def test_trees(tv, groups, Hq, Hkv, D, page, dtype):
    c = shared(len(groups) + 20, groups, Hq, Hkv, D, page, dtype, tree=True, pad=2)
    agree(tv, c, Hq, Hkv, D, dtype)


def slopes_of(Hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], device="cuda:0")


KINDS = [dict(softcap=5.0), dict(softcap=50.0, scale=0.7), dict(window=1), dict(window=70), dict(window=400),
         dict(window=10**6), dict(slopes=True), dict(slopes=True, softcap=20.0, window=150)]


@pytest.mark.parametrize("kw", KINDS)
@pytest.mark.parametrize("groups,tree", [([(300, [(9, 1), (0, 1), (150, 1)]), (90, [(600, 1)])], False),
                                         ([(200, [(30, 90), (0, 40), (77, 1)])], False),
                                         ([(260, [(60, 70), (0, 9), (129, 1)]), (40, [(3, 20)])], True),
                                         ([(500, [(64, 4), (2, 3)])], True)])
@pytest.mark.parametrize("Hq,Hkv,D,page,dtype", [(8, 2, 128, 16, "bf16"), (4, 4, 64, 32, "fp16")])
def test_score_kinds(tv, kw, groups, tree, Hq, Hkv, D, page, dtype):
    kw = dict(kw)
    if kw.get("slopes"):
        kw["slopes"] = slopes_of(Hq)
    c = shared(9, groups, Hq, Hkv, D, page, dtype, tree=tree)
    agree(tv, c, Hq, Hkv, D, dtype, **kw)


@pytest.mark.parametrize("kw", [{}, dict(window=120)])
@pytest.mark.parametrize("n", [1, 30])
def test_sequences_outside_the_groups(tv, kw, n):
    c = shared(4, [(400, [(20, n), (3, n)]), (150, [(0, n)])], 8, 2, 64, 16, first=[(200, n), (0, n)], last=[(33, n)])
    agree(tv, c, 8, 2, 64, "bf16", **kw)


@pytest.mark.parametrize("lens", [[(300, 1), (75, 1)], [(200, 37), (500, 33)]])
def test_without_groups_it_is_attn_paged(tv, lens):
    c = shared(3, [], 8, 2, 64, 16, first=lens)
    assert c["pre_table"].shape[0] == 0
    out, lse, status = run(tv, c)
    want = tv.attn_paged(c["q"], c["k"], c["v"], c["table"], c["q_start"], c["kv_len"], c["max_q"])
    assert status == [0, 0] and same_bits(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("groups", [[(3000, [(50, 1)] * 30)], [(1500, [(30, 60)] * 6)], [(100, [(5, 1)] * 3)]])
def test_same_result_every_time(tv, groups):
    c = shared(8, groups, 8, 2, 128, 64)
    a = run(tv, c)
    for _ in range(3):
        b = run(tv, c)
        assert same_bits(a[0], b[0]) and torch.equal(a[1], b[1])


def test_lengths_do_not_depend_on_the_hint(tv):
    c = shared(4, [(300, [(100, 70), (0, 3), (40, 120)])], 8, 2, 128, 16)
    want = attn_ref(c["full"], 8, 2, 128)
    for hint in (1, 3, 64, 4000):
        c["max_q"] = hint
        out, lse, status = run(tv, c)
        assert status == [0, 0, 0]
        check_attn(out, lse, want, "bf16", f"max_q {hint}")


@pytest.mark.parametrize("B,per", [(300, 1), (500, 7), (700, 700)])
def test_many_sequences_and_groups(tv, B, per):
    rng = random.Random(B)
    seqs = [(rng.randint(0, 60), int(rng.random() < 0.9)) for _ in range(B)]
    groups = [(rng.randint(0, 200), seqs[i:i + per]) for i in range(0, B, per)]
    c = shared(B, groups, 4, 1, 64, 16, pad=2)
    agree(tv, c, 4, 1, 64, "bf16")


def test_layouts_and_fused_queries(tv):
    for layout in ("rows", "both"):
        for groups in ([(700, [(90, 1), (4, 1)])], [(300, [(20, 90), (5, 5)])]):
            c = shared(5, groups, 8, 2, 64, 16, layout=layout, pad=3)
            agree(tv, c, 8, 2, 64, "bf16")


@pytest.mark.parametrize("n", [1, 40])
def test_large_scores_and_long_prefixes(tv, n):
    agree(tv, shared(6, [(1500, [(200, n), (3, n)])], 4, 1, 128, 16, q_mag=30.0), 4, 1, 128, "bf16")
    agree(tv, shared(6, [(20000, [(200, n), (3, n)])], 4, 1, 64, 64), 4, 1, 64, "bf16")


def part(ref, a, b):
    return tuple(r[a:b] for r in ref)


@pytest.mark.parametrize("n", [1, 40])
def test_bad_data(tv, n):
    groups = [(200, [(10, n), (20, n)]), (100, [(5, n), (60, n)])]
    mk = lambda: shared(2, groups, 8, 2, 128, 16)  # noqa: E731
    c = mk()
    ref = attn_ref(c["full"], 8, 2, 128)
    own = dict(c, anc=None, lens=c["own"], rows=c["rows"][2:])
    alone = attn_ref(own, 8, 2, 128)
    # a prefix length that does not fit: hidden, and said by its sequences
    for L in (-1, 10**8):
        c = mk()
        c["pre_len"][0] = L
        out, lse, status = run(tv, c)
        assert status == [1, 1, 0, 0]
        check_attn(out[:2 * n], lse[:2 * n], part(alone, 0, 2 * n), "bf16")
        check_attn(out[2 * n:], lse[2 * n:], part(ref, 2 * n, 4 * n), "bf16")
    # an own length that does not fit
    c = mk()
    c["kv_len"][1] = -1
    out, lse, status = run(tv, c)
    assert status == [0, 1, 0, 0]
    assert bool((out[n:2 * n] == 0).all()) and bool((lse[n:2 * n] == 0).all())
    check_attn(out[:n], lse[:n], part(ref, 0, n), "bf16")
    check_attn(out[2 * n:], lse[2 * n:], part(ref, 2 * n, 4 * n), "bf16")
    # a page of a prefix that is none: its rows are hidden
    c = mk()
    c["pre_table"][1, 2] = 10**7
    hidden = {b: set(range(32, 48)) for b in (2, 3)}
    out, lse, status = run(tv, c)
    assert status == [0, 0, 1, 1]
    check_attn(out, lse, attn_ref(c["full"], 8, 2, 128, hidden=hidden), "bf16")
    # groups that are none: their sequences say so
    for bad, want in (([0, -1, 4], {0, 1, 2, 3}), ([0, 2, 9], {2, 3}), ([0, 3, 2], {0, 1, 2, 3})):
        c = mk()
        c["group_start"] = i32(bad)
        out, lse, status = run(tv, c)
        assert {b for b, s in enumerate(status) if s} <= want and (status[2] == 1 or bad == [0, 3, 2])
        assert bool(torch.isfinite(out).all())
    # starts that descend inside a group
    c = mk()
    c["q_start"][2] = c["q_start"][1] - 1
    out, lse, status = run(tv, c)
    assert status[1] == 1 and status[3] == 0
    check_attn(out[3 * n:], lse[3 * n:], part(ref, 3 * n, 4 * n), "bf16")


@pytest.mark.parametrize("n", [1, 40])
def test_pages_behind_the_window_may_be_gone(tv, n):
    c = shared(3, [(500, [(10, n), (30, n)])], 4, 2, 64, 16)
    ref = attn_ref(c["full"], 4, 2, 64, window=100)
    gone = (510 - 100 + 1) // 16
    ids = np_(c["pre_table"])[0, :gone].tolist()
    c["pre_table"][0, :gone] = -1
    c["k"][ids] = float("nan")
    c["v"][ids] = float("inf")
    edge = int(c["pre_table"][0, gone])           # rows in front of the window, in its first page
    front = (510 - 100 + 1) % 16
    c["k"][edge, :, :front] = float("nan")
    c["v"][edge, :, :front] = 0                   # (rows of a unit's range that no token sees are finite)
    out, lse, status = run(tv, c, window=100)
    assert status == [0, 0]
    check_attn(out, lse, ref, "bf16")


def test_empty_masks_see_the_prefix(tv):
    for n in (6, 40):
        c = shared(3, [(30, [(0, n), (5, n)])], 4, 2, 64, 16, tree=True)
        c["anc"].zero_()
        out, lse, status = run(tv, c)
        assert status == [0, 0] and bool(torch.isfinite(lse).all())
        assert bool((out != 0).any())
        c = shared(3, [(0, [(0, n), (5, n)])], 4, 2, 64, 16, tree=True)
        c["anc"].zero_()
        out, lse, status = run(tv, c)
        assert bool((out[:n] == 0).all()) and bool((lse[:n] == -math.inf).all())


@pytest.mark.parametrize("groups", [[(300, [(9, 1), (70, 1)]), (1500, [(3, 1)])], [(70, [(5, 30), (500, 40)])]])
@pytest.mark.parametrize("kw", [{}, dict(softcap=30.0)])
def test_nan_in_queries_and_prefix_keys(tv, groups, kw):
    c = shared(3, groups, 8, 2, 128, 16)
    want = run(tv, c, **kw)
    last = [s - 1 for s in starts([n for _, n in c["own"]])[1:]]
    c["q"] = c["q"].clone()
    for b, t in enumerate(last):
        c["q"][t, b % 8, 5] = float("nan")
    out, lse, status = run(tv, c, **kw)
    assert not any(status)
    for b, t in enumerate(last):
        assert bool(out[t, b % 8].isnan().all()) and bool(lse[t, b % 8].isnan())
        out[t, b % 8], lse[t, b % 8] = want[0][t, b % 8], want[1][t, b % 8]
    assert same_bits(out, want[0]) and torch.equal(lse, want[1])
    for j in (0, groups[0][0] - 1):
        c = shared(3, groups, 8, 2, 128, 16)
        c["k"][c["pre_table"][0, j // 16], :, j % 16, 3] = float("nan")
        out, lse, status = run(tv, c, **kw)
        n = sum(m for _, m in groups[0][1])
        assert bool(out[:n].isnan().all()) and bool(lse[:n].isnan().all())
        assert same_bits(out[n:], want[0][n:]) and torch.equal(lse[n:], want[1][n:])


@pytest.mark.parametrize("groups", [[(300, [(9, 1), (70, 1)])], [(2000, [(9, 1)] * 40)], [(700, [(40, 64)] * 12)],
                                    [(90, [(5, 1)] * 2)]])
def test_other_stream_and_graphs(tv, groups):
    """On a stream of its own, and two captured calls replayed at the same time."""
    cs = [shared(s, groups, 8, 2, 128, 64) for s in (1, 2)]
    want = [run(tv, c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    graphs, outs = [], []
    call = lambda c: tv.attn_paged_prefix(c["q"], c["k"], c["v"], c["pre_table"], c["pre_len"], c["group_start"],  # noqa: E731
                                          c["table"], c["q_start"], c["kv_len"], c["max_q"])
    for c, s in zip(cs, streams):
        with torch.cuda.stream(s):
            got = call(c)
        s.synchronize()
        assert same_bits(got[0], want[len(graphs)][0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(call(c))
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
        for o, w in zip(outs, want):
            assert same_bits(o[0], w[0]) and torch.equal(o[1], w[1])


@pytest.mark.parametrize("groups", [[(300, [(9, 1), (0, 0), (70, 1)])], [(2000, [(9, 1)] * 40), (50, [])],
                                    [(700, [(40, 64)] * 12), (9, [(3, 0)])], [(90, [(5, 1)] * 2)],
                                    [(0, [(700 + 40 * i, 64) for i in range(45)])]])
def test_a_wait_that_runs_out_is_reported(tv, groups):
    c = shared(5, groups, 8, 2, 64, 16)
    want = run(tv, c)
    try:
        assert tv.lib.tv_debug_set_wait_limit(0) == tv.TV_OK
        late = run(tv, c)
    finally:
        assert tv.lib.tv_debug_set_wait_limit(tv.TV_WAIT_LIMIT_DEFAULT) == tv.TV_OK
    assert late[2] == [tv.TV_ERR_TIMEOUT if n else 0 for _, n in c["own"]]
    got = run(tv, c)
    assert not any(got[2]) and same_bits(got[0], want[0]) and torch.equal(got[1], want[1])
    if tv.CHECKED:  # (this build records the site of a wait that gave up)
        tv.check_take()


def test_refusals_of_the_binding(tv):
    c = shared(1, [(40, [(3, 2)])], 4, 2, 64, 16)
    ok = (c["q"], c["k"], c["v"], c["pre_table"], c["pre_len"], c["group_start"], c["table"], c["q_start"], c["kv_len"], 2)

    def bad(i, x, err, **kw):
        a = list(ok)
        a[i] = x
        with pytest.raises(err):
            tv.attn_paged_prefix(*a, **kw)
    bad(0, c["q"].float(), TypeError)
    bad(3, c["pre_table"].long(), TypeError)
    bad(3, c["pre_table"][0], ValueError)
    bad(4, c["pre_len"].cpu(), ValueError)
    bad(4, None, TypeError)
    bad(5, c["group_start"][:1], ValueError)
    bad(6, c["table"][0], ValueError)
    bad(9, 0, tv.TVError)
    bad(9, 2, tv.TVError, ws=torch.zeros(256, dtype=torch.uint8, device="cuda:0"))


# ------------------------------------------------------------------ together
def test_a_serving_loop_behind_one_prompt(tv):
    """A prompt written once as a sequence of its own; requests behind it take verify steps; all pages
    come back when the requests and the prompt are released, each once."""
    rng, g = random.Random(3), torch.Generator().manual_seed(3)
    B, Hq, Hkv, D, page, P, S, N = 4, 8, 2, 64, 16, 30, 210, 12
    pool = 200
    k, v = (torch.full((pool, Hkv, page, D), float("nan"), dtype=torch.bfloat16, device="cuda:0") for _ in range(2))
    # row 0 of the table is the prompt's, the others the requests'
    table, held = i32([[-1] * P] * (B + 1)), i32([0] * (B + 1))
    free, n_free = i32(list(range(pool))), i32([pool])
    rows = [(torch.zeros(0, Hkv, D), torch.zeros(0, Hkv, D)) for _ in range(B + 1)]
    group_start = i32([0, B])
    for step in range(4):
        lens = [r[0].shape[0] for r in rows]
        new = [S if step == 0 else 0] + [0 if step == 0 else rng.randint(3, 40) if step == 1 else N] * B
        if step == 1:
            new = [0] + [rng.randint(3, 40) for _ in range(B)]
        T, q_start = sum(new), starts(new)
        x = torch.randn(T, Hq + 2 * Hkv, D, generator=g).bfloat16().cuda()
        slots, st = tv.page_map(i32(q_start), i32(lens), table, held, free, n_free, page, T)
        assert not bool(st.any())
        nk, nv = x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        tv.paged_append(nk, nv, slots, k, v)
        rows = [tuple(torch.cat([r[i], t[q_start[b]:q_start[b + 1]].cpu().float()]) for i, t in enumerate((nk, nv)))
                for b, r in enumerate(rows)]
        if step == 0:
            continue
        case = dict(anc=None)
        if step > 1:
            parents = [random_tree(rng, N) for _ in range(B)]
            words, depth = tree_masks(parents, 1)
            case = dict(anc=torch.tensor(words, dtype=torch.int64, device="cuda:0"), parents=parents, depth=depth)
        out, lse, st = tv.attn_paged_prefix(x[:, :Hq], k, v, table[:1], i32([S]), group_start, table[1:],
                                            i32(q_start[1:]), i32(lens[1:]), max(new), anc_mask=case["anc"])
        assert not bool(st.any())
        case.update(lens=[(S + L, n) for L, n in zip(lens[1:], new[1:])], q=x[:, :Hq],
                    rows=[tuple(torch.cat([rows[0][i], rows[b + 1][i]]) for i in range(2)) for b in range(B)])
        check_attn(out, lse, attn_ref(case, Hq, Hkv, D), "bf16")
        if step > 1:
            path = [[0] + sorted(rng.sample(range(1, N), rng.randint(0, 6))) for _ in range(B)]
            new_len, st = tv.commit_paged(k, v, table[1:], i32(lens[1:]), i32([p + [-1] * (N - len(p)) for p in path]),
                                          i32([len(p) - 1 for p in path]))
            assert not bool(st.any())
            rows[1:] = [tuple(torch.cat([r[:L], r[[L + i for i in p]]]) for r in rows[b + 1])
                        for b, (L, p) in enumerate(zip(lens[1:], path))]
            assert np_(new_len).tolist() == [r[0].shape[0] for r in rows[1:]]
    zero = i32([0] * (B + 2))
    tv.page_map(zero, zero[1:], table, held, free, n_free, page, 0)
    assert int(n_free) == pool and sorted(np_(free).tolist()) == list(range(pool))


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("own", [(10, 30), (120, 150), (99, 300), (98, 0)])
@pytest.mark.parametrize("tree", [False, True])
def test_prefix_rows_that_no_window_reaches_may_hold_anything(tv, n, own, tree):
    """The window reaches back from a sequence's own rows: what is ahead of all of a group's is not read."""
    window, S = 100, 500
    c = shared(3, [(S, [(own[0], n), (2, 0), (own[1], n)])], 4, 2, 64, 16, tree=tree)
    ref = attn_ref(c["full"], 4, 2, 64, window=window)
    for fill in (float("nan"), float("inf")):
        for j in range(min(S, S + min(own) - window + 1)):
            page = int(c["pre_table"][0, j // 16])
            c["k"][page, :, j % 16] = fill
            c["v"][page, :, j % 16] = fill
        out, lse, status = run(tv, c, window=window)
        assert status == [0, 0, 0]
        check_attn(out, lse, ref, "bf16")


@pytest.mark.parametrize("n", [1, 40])
def test_groups_that_descend(tv, n):
    """The first malformed group and those behind it have no prefix, and sequences from its start on say so."""
    groups = [(200, [(10, n), (20, n)]), (100, [(5, n)]), (60, [(60, n)])]
    for bounds, good, status in (([0, 3, 2, 4], 1, [0, 0, 0, 1]), ([0, 2, 1, 4], 1, [0, 0, 1, 1]),
                                 ([2, 1, 3, 4], 0, [1, 1, 1, 1]), ([0, 1, 9, 4], 1, [0, 1, 1, 1]),
                                 ([0, 1, 3, 1], 2, [0, 0, 0, 1]), ([1, 2, 3, 4], 3, [0, 0, 0, 0]),
                                 ([0, 3, 2], 1, [0, 0, 0, 1]), ([5, 6, 7, 8], 0, [1, 1, 1, 1])):
        c = shared(2, groups, 8, 2, 128, 16)
        c["group_start"] = i32(bounds)
        c["pre_table"], c["pre_len"] = c["pre_table"][:len(bounds) - 1], c["pre_len"][:len(bounds) - 1]
        # the groups that count, and what their sequences see
        of = [max([g for g in range(good) if bounds[g] <= b < bounds[g + 1]], default=-1) for b in range(4)]
        full = dict(c["full"])
        full["lens"] = [(L + (groups[g][0] if g >= 0 else 0), m) for g, (L, m) in zip(of, c["own"])]
        full["rows"] = [tuple(torch.cat([c["rows"][g][i], c["rows"][3 + b][i]]) if g >= 0 else c["rows"][3 + b][i]
                              for i in range(2)) for b, g in enumerate(of)]
        out, lse, got = run(tv, c)
        assert got == status, bounds
        check_attn(out, lse, attn_ref(full, 8, 2, 128), "bf16", f"{bounds}")
        again = run(tv, c)
        assert same_bits(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("first", [2**31 - 1, 2**31 - 2, 2**31 - 300, -2**31, 303, 304])
def test_whatever_the_workspace_held(tv, n, first):
    """Tokens of nobody, whose entries in the workspace are old or anything."""
    groups = [(3000, [(50, n)] * 20)]
    c = shared(8, groups, 8, 2, 128, 64, pad=40)
    want = run(tv, c)
    T, Hq, D = c["q"].shape
    size = tv.attn_paged_prefix_workspace_size(c["max_q"], T, 1, Hq, 2, D)
    for parts, token, of in ((3, c["T"], 0), (2**31 - 1, c["T"] - 1, 0), (2, 2**31 - 1, 2**31 - 1),
                             (2, -2**31, -1), (9, c["T"] + 39, 19)):
        words = torch.tensor([first, parts, token, of], dtype=torch.int64).to(torch.int32)
        ws = words.repeat(-(-size // 16)).to("cuda:0").view(torch.uint8)[:size]
        out, lse, status = run(tv, c, ws=ws)
        assert not any(status)
        assert same_bits(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (7, 1)])
def test_other_groups_queries_change_no_bit(tv, Hq, Hkv):
    """Rows of a block that are another group's or sequence's, whatever their size."""
    groups = [(300, [(40, 20), (7, 3)]), (500, [(20, 30)])]
    c = shared(3, groups, Hq, Hkv, 128, 16)
    want = run(tv, c)
    c["q"] = c["q"].clone()
    for size in (2.0**30, 2.0**100):
        c["q"][23:] = torch.randn(c["q"][23:].shape, generator=torch.Generator().manual_seed(1)).to(c["q"]) * size
        out, lse, status = run(tv, c)
        assert not any(status)
        assert same_bits(out[:23], want[0][:23]) and torch.equal(lse[:23], want[1][:23])
