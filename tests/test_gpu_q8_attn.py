"""Attention over the 8-bit paged cache on the GPU against 64-bit floats over the values that its codes
stand for: chunks, trees, masks, score kinds, layouts, bad data, and a loop of steps with the other calls."""
import math
import random

import numpy as np
import pytest
import torch

from _gpu_util import i32, np_
from _paged_util import attn_ref
from _q8_util import cache, check_attn_q8, check_seen, make_q8, quantise_ref, raw, set_rows, values_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tv():
    import speculative_decoding_tree_tv_gb300 as m
    return m


def starts(new):
    return [0] + list(np.cumsum(new))


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


def run(tv, c, **kw):
    T, Hq, D = c["q"].shape
    out = torch.full((T, Hq, D), 7.0, dtype=c["q"].dtype, device="cuda:0")
    lse = torch.full((T, Hq), 7.0, device="cuda:0")
    out, lse, status = tv.attn_paged_q8(c["q"], *c["q8"], c["table"], c["q_start"], c["kv_len"], c["max_q"],
                                        anc_mask=c["anc"], out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    n = c["T"]
    assert bool((out[n:] == 7).all()) and bool((lse[n:] == 7).all())  # rows of nobody
    return out[:n], lse[:n], np_(status).tolist()


def agree(tv, c, Hq, Hkv, D, dtype, **kw):
    out, lse, status = run(tv, c, **kw)
    assert status == [0] * len(c["lens"])
    check_attn_q8(out, lse, attn_ref(c, Hq, Hkv, D, **kw), c, dtype, Hkv, kw.get("scale", 0.0))
    return out, lse


SHAPES = [(8, 2, 128, 16, "e4m3", "bf16", "heads"), (4, 4, 64, 8, "int8", "fp16", "rows"),
          (7, 1, 128, 256, "int8", "bf16", "both"), (10, 2, 64, 64, "e4m3", "bf16", "rows"),
          (16, 1, 128, 32, "e4m3", "fp16", "heads"), (3, 3, 64, 128, "e4m3", "bf16", "both"),
          (64, 1, 128, 32, "int8", "bf16", "rows"), (8, 2, 64, 16, "e4m3", "fp16", "rows")]
DECODE = [[(0, 1)], [(1, 1)], [(63, 1), (64, 1), (127, 1), (0, 1), (128, 1)], [(1500, 1), (3, 1), (0, 1), (700, 1)]]
CHUNKS = [[(0, 2)], [(0, 129)], [(200, 33), (0, 0), (5, 64), (130, 1)], [(64, 200), (700, 3)],
          [(1000, 5), (1, 4), (33, 8)]]
TREES = [[(0, 1)], [(100, 4), (0, 3)], [(300, 64), (17, 60), (0, 5), (64, 1)], [(190, 65)], [(40, 300), (0, 7)]]


@pytest.mark.parametrize("lens", DECODE + CHUNKS)
@pytest.mark.parametrize("Hq,Hkv,D,page,fmt,dtype,layout", SHAPES)
def test_causal(tv, lens, Hq, Hkv, D, page, fmt, dtype, layout):
    c = make_q8(len(lens), lens, Hq, Hkv, D, page, fmt, dtype, layout, pad=3)
    agree(tv, c, Hq, Hkv, D, dtype)


@pytest.mark.parametrize("lens", TREES)
@pytest.mark.parametrize("Hq,Hkv,D,page,fmt,dtype,layout", SHAPES[:4])
def test_trees(tv, lens, Hq, Hkv, D, page, fmt, dtype, layout):
    c = make_q8(len(lens) + 20, lens, Hq, Hkv, D, page, fmt, dtype, layout, tree=True, pad=2)
    agree(tv, c, Hq, Hkv, D, dtype)


def slopes_of(Hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], device="cuda:0")


KINDS = [dict(softcap=5.0), dict(softcap=50.0, scale=0.7), dict(window=1), dict(window=70), dict(window=10**6),
         dict(slopes=True), dict(slopes=True, softcap=20.0, window=150)]


@pytest.mark.parametrize("kw", KINDS)
@pytest.mark.parametrize("lens,tree", [([(900, 1), (0, 1), (150, 1)], False), ([(300, 200), (0, 40), (77, 1)], False),
                                       ([(260, 70), (0, 9), (129, 1)], True), ([(500, 3), (64, 4)], True)])
@pytest.mark.parametrize("Hq,Hkv,D,page,fmt,dtype", [(8, 2, 128, 16, "e4m3", "bf16"), (4, 4, 64, 32, "int8", "fp16")])
def test_score_kinds(tv, kw, lens, tree, Hq, Hkv, D, page, fmt, dtype):
    kw = dict(kw)
    if kw.get("slopes"):
        kw["slopes"] = slopes_of(Hq)
    c = make_q8(9, lens, Hq, Hkv, D, page, fmt, dtype, tree=tree)
    agree(tv, c, Hq, Hkv, D, dtype, **kw)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("tree,kw", [(False, {}), (True, dict(window=4, slopes=True)),
                                     (False, dict(window=200, softcap=9.0))])
@pytest.mark.parametrize("ctx,page", [(150, 16), (1500, 64)])
def test_units_of_either_height(tv, G, tree, kw, ctx, page):
    """1 to 17 rows a unit, whole and split."""
    kw = dict(kw)
    if kw.get("slopes"):
        kw["slopes"] = slopes_of(2 * G)
    D = 128 if G % 2 else 64
    for n in sorted({1, 8 // G, 8 // G + 1, 16 // G, 16 // G + 1}):
        c = make_q8(G + n, [(ctx, n), (0, max(1, n - 1)), (ctx // 3, n)], 2 * G, 2, D, page, "e4m3", tree=tree)
        agree(tv, c, 2 * G, 2, D, "bf16", **kw)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("lens", [[(900, 1), (40, 1)], [(300, 90)]])
@pytest.mark.parametrize("dtype,spread,q_mag", [("bf16", 0.0, 30.0), ("bf16", 12.0, 1e-3), ("fp16", 3.0, 20.0),
                                                ("bf16", 25.0, 1e-7)])
def test_rows_of_very_different_sizes(tv, fmt, lens, dtype, spread, q_mag):
    """Scores that differ by hundreds, and rows (of K and V alike) many powers of two apart."""
    c = make_q8(6, lens, 4, 1, 128, 16, fmt, dtype, spread=spread, q_mag=q_mag)
    agree(tv, c, 4, 1, 128, dtype)


@pytest.mark.parametrize("lens", [[(500, 1), (30, 1)], [(200, 40)]])
def test_sizes_at_the_ends_of_the_scale(tv, lens):
    """Values near the largest and the smallest bf16 numbers."""
    for e in (230, 12):
        c = make_q8(6, lens, 4, 1, 64, 16, "int8", spread=0.5)
        # (V alone: K of that size has no finite scores)
        s = c["q8"][3]
        moved = (s.int() + e - 120).clamp(1, 248)
        s.copy_(torch.where(s == 255, s.int(), moved).to(torch.uint8))
        f = 2.0 ** (e - 120)
        c["rows"] = [(k, v * f) for k, v in c["rows"]]
        out, lse, status = run(tv, c)
        ref = attn_ref(c, 4, 1, 64)
        # (check_attn_q8 at the values' own size: outputs by 2^-e, exactly)
        c["rows"] = [(k, v / f) for k, v in c["rows"]]
        back = (out.double() / f).cpu()
        want = attn_ref(c, 4, 1, 64)
        u = 2.0**-8
        n = max(L + m for L, m in lens)
        vmax = max(v.abs().max().item() for _, v in c["rows"])
        tol = want[2] * (2.0**-11 + 2 * want[3][..., None] + 2.0**-19) + u * want[0].abs() * 1.01 + 2.0**-29 * n * vmax
        assert bool(((back - want[0]).abs() <= tol).all())
        assert torch.isfinite(out).all() and ref[0].shape == out.shape


@pytest.mark.parametrize("lens", [[(3000, 1)] * 3, [(1500, 90), (1, 2)], [(700, 64)] * 45])
def test_same_result_every_time(tv, lens):
    c = make_q8(8, lens, 8, 2, 128, 64, "e4m3")
    a = run(tv, c)
    for _ in range(3):
        b = run(tv, c)
        assert same_bits(a[0], b[0]) and torch.equal(a[1], b[1])


def test_lengths_do_not_depend_on_the_hint(tv):
    c = make_q8(4, [(100, 70), (0, 3), (40, 200)], 8, 2, 128, 16, "int8")
    want = attn_ref(c, 8, 2, 128)
    for hint in (1, 3, 8, 64, 4000):
        c["max_q"] = hint
        out, lse, status = run(tv, c)
        assert status == [0, 0, 0]
        check_attn_q8(out, lse, want, c, "bf16", 2)


@pytest.mark.parametrize("new", [1, 20])
@pytest.mark.parametrize("B", [33, 500])
def test_many_short_sequences(tv, B, new):
    rng = random.Random(B)
    lens = [(rng.randint(0, 90), new if rng.random() < 0.9 else 0) for _ in range(B)]
    c = make_q8(B, lens, 8, 2, 64, 16, "e4m3", pad=2)
    agree(tv, c, 8, 2, 64, "bf16")


@pytest.mark.parametrize("lens", [[(30000, 1)], [(12000, 40), (5, 3)]])
def test_long_contexts(tv, lens):
    c = make_q8(2, lens, 4, 1, 64, 64, "int8")
    agree(tv, c, 4, 1, 64, "bf16")


def test_the_widest_group(tv):
    c = make_q8(3, [(150, 5), (0, 2), (300, 1)], 128, 1, 64, 32, "e4m3")
    agree(tv, c, 128, 1, 64, "bf16")


def test_offsets_past_32_bits(tv):
    """A sequence in the last pages of codes of more than 4 GiB a side."""
    Hkv, D, page, pool = 8, 128, 256, 18000
    q8 = [torch.zeros(pool, Hkv, page, D, dtype=torch.int8, device="cuda:0") for _ in range(2)]
    q8 += [torch.zeros(pool, Hkv, page, dtype=torch.uint8, device="cuda:0") for _ in range(2)]
    for n in (1, 40):
        lens = [(600, n)]
        c = make_q8(n, lens, 8, Hkv, D, page, "int8")
        ids = np_(c["table"])[0]
        table = [pool - 1, 0, pool - 2] + [9000] * (len(ids) - 3)
        for big, small in zip(q8, c["q8"]):
            for i in range(3):
                big[table[i]] = small[int(ids[i])]
        c["q8"], c["table"] = tuple(q8), i32([table])
        agree(tv, c, 8, Hkv, D, "bf16")


def test_bad_sequences(tv):
    """Lengths that do not fit are reported and zeroed, malformed ranges left alone; their neighbours are served."""
    lens = [(40, 3), (20, 3), (60, 3), (10, 3)]
    for extra in (0, 60):
        lens = [(L, n + extra) for L, n in lens]
        c = make_q8(2, lens, 8, 2, 128, 16, "e4m3")
        want = run(tv, c)
        n = lens[0][1]
        c["kv_len"][0] = -1
        c["kv_len"][2] = 10**6
        out, lse, status = run(tv, c)
        assert status == [1, 0, 1, 0]
        for b in (0, 2):
            assert bool((out[b * n:(b + 1) * n] == 0).all()) and bool((lse[b * n:(b + 1) * n] == 0).all())
        for b in (1, 3):
            assert (out[b * n:(b + 1) * n].float() - want[0][b * n:(b + 1) * n].float()).abs().max() < 0.1
        c = make_q8(2, lens, 8, 2, 128, 16, "e4m3")
        c["q_start"][4] += 1                    # past T
        out, lse, status = run(tv, c)
        assert status == [0, 0, 0, 1] and bool((out[3 * n:] == 7).all())


@pytest.mark.parametrize("new", [1, 50])
@pytest.mark.parametrize("page", [8, 32, 128, 256])
def test_bad_pages_are_hidden_and_reported(tv, new, page):
    lens = [(600, new), (600, new), (90, new)]
    c = make_q8(3, lens, 8, 2, 128, page, "e4m3")
    c["table"][0, 1] = -5
    c["table"][2, 0] = 10**7
    hidden = {0: set(range(page, min(2 * page, 600 + new))), 2: set(range(min(page, 90 + new)))}
    out, lse, status = run(tv, c)
    assert status == [1, 0, 1]
    check_attn_q8(out, lse, attn_ref(c, 8, 2, 128, hidden=hidden), c, "bf16", 2)


@pytest.mark.parametrize("new", [1, 40])
def test_pages_behind_the_window_may_be_gone(tv, new):
    c = make_q8(3, [(500, new), (100, new)], 4, 2, 64, 16, "int8")
    ref = attn_ref(c, 4, 2, 64, window=100)
    gone = (500 - 100 + 1) // 16
    ids = np_(c["table"])[0, :gone].tolist()
    c["table"][0, :gone] = -1
    edge = int(c["table"][0, gone])           # rows in front of the window, in its first page
    front = (500 - 100 + 1) % 16
    for x in c["q8"][2:]:
        x[ids] = 255
        x[edge, :, :front] = 255
    out, lse, status = run(tv, c, window=100)
    assert status == [0, 0]
    check_attn_q8(out, lse, ref, c, "bf16", 2)


def test_empty_masks(tv):
    for n in (6, 40):
        c = make_q8(3, [(0, n), (30, n)], 4, 2, 64, 16, "e4m3", tree=True)
        c["anc"].zero_()
        out, lse, status = run(tv, c)
        assert status == [0, 0]
        assert bool((out[:n] == 0).all()) and bool((lse[:n] == -math.inf).all())
        assert bool(torch.isfinite(lse[n:]).all()) and bool((out[n:] != 0).any())


def test_no_tokens(tv):
    c = make_q8(3, [(40, 0), (0, 0)], 4, 2, 64, 16, "int8", pad=4)
    out, lse, status = run(tv, c)
    assert status == [0, 0] and out.numel() == 0


NAN_LENS = [[(90, 1), (300, 1), (1500, 1)], [(70, 30), (500, 90)]]


@pytest.mark.parametrize("lens", NAN_LENS)
@pytest.mark.parametrize("kw", [{}, dict(softcap=30.0), dict(window=40)])
def test_nan_in_a_query_row(tv, lens, kw):
    c = make_q8(3, lens, 8, 2, 128, 16, "e4m3")
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
@pytest.mark.parametrize("side", ["k", "v"])
def test_a_row_that_is_no_number(tv, lens, kw, where, side):
    """Tokens that see the row get NaN (its lse too, if it is a key); tokens that do not are as they were: a V
    row that one token sees and another does not may be NaN here."""
    c = make_q8(4, lens, 8, 2, 128, 16, "e4m3")
    want = run(tv, c, **kw)
    sees, at = [], 0
    table = np_(c["table"])
    for b, (L, n) in enumerate(lens):
        j = dict(last=L + n - 1, middle=L + n // 2, first=0)[where]
        k, v, ks, vs = c["q8"]
        page, row = int(table[b, j // 16]), j % 16
        (k if side == "k" else v).view(torch.uint8)[page, :, row] = 0
        (ks if side == "k" else vs)[page, :, row] = 255
        sees += [L + i >= j and L + i - j < kw.get("window", 10**9) for i in range(n)]
    out, lse, status = run(tv, c, **kw)
    assert status == [0] * len(lens)
    sees = torch.tensor(sees, device="cuda:0")
    assert bool(out[sees].isnan().all())
    if side == "k":
        assert bool(lse[sees].isnan().all())
    else:
        assert torch.equal(lse, want[1])
    assert torch.equal(lse[~sees], want[1][~sees])
    # (scales of a warp's V rows decide how far its sums are scaled: the same but for the NaN row's own)
    assert (out[~sees].float() - want[0][~sees].float()).abs().max().item() <= 0.05 if bool((~sees).any()) else True
    assert bool(torch.isfinite(out[~sees]).all())


@pytest.mark.parametrize("lens", [[(300, 1), (75, 1), (1000, 1)], [(70, 1), (30, 1)], [(90, 2), (700, 1)],
                                  [(200, 37), (500, 33)], [(70, 9), (1000, 40)]])
@pytest.mark.parametrize("softcap", [0.0, 9.0])
@pytest.mark.parametrize("window", [0, 41])
def test_rows_that_nobody_sees_change_no_bit(tv, lens, softcap, window):
    got = []
    for fill in (0, 0x7f, 0xff, 200):
        c = make_q8(3, lens, 8, 2, 64, 16, "e4m3")
        table = np_(c["table"])
        for x in c["q8"]:
            x = x.view(torch.uint8)
            for b, (L, n) in enumerate(lens):
                for j in list(range(max(0, L - window + 1) if window else 0)) + list(range(L + n, -(-(L + n) // 16) * 16)):
                    x[table[b, j // 16], :, j % 16] = fill
        got.append(run(tv, c, softcap=softcap, window=window))
        assert got[-1][2] == [0] * len(lens)
    assert bool(torch.isfinite(got[0][0]).all())
    for g in got[1:]:
        assert same_bits(g[0], got[0][0]) and torch.equal(g[1], got[0][1])


@pytest.mark.parametrize("lens", [[(300, 1), (2000, 1)], [(300, 80), (2000, 9)],
                                  [(700 + 40 * i, 64) for i in range(45)], [(90, 1), (70, 1)]])
def test_other_stream_and_graphs(tv, lens):
    """On a stream of its own, and two captured calls replayed at the same time."""
    cs = [make_q8(s, lens, 8, 2, 128, 64, "int8") for s in (1, 2)]
    want = [run(tv, c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    graphs, outs = [], []
    call = lambda c: tv.attn_paged_q8(c["q"], *c["q8"], c["table"], c["q_start"], c["kv_len"], c["max_q"])  # noqa: E731
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


@pytest.mark.parametrize("lens", [[(90, 1), (0, 0), (128, 1)], [(300, 1), (0, 0), (2048, 1), (64, 1)],
                                  [(50, 40), (9, 0), (120, 9)], [(300, 80), (7, 0), (2040, 9)],
                                  [(700 + 40 * i, 64) for i in range(45)] + [(5, 0)], [(60, 2)] * 450 + [(3, 0)]])
def test_a_wait_that_runs_out_is_reported(tv, lens):
    c = make_q8(5, lens, 8, 2, 64, 16, "e4m3")
    call = lambda: tv.attn_paged_q8(c["q"], *c["q8"], c["table"], c["q_start"], c["kv_len"], c["max_q"])  # noqa: E731
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


def test_refusals_of_the_binding(tv):
    c = make_q8(1, [(40, 3)], 4, 2, 64, 16, "e4m3")
    ok = (c["q"], *c["q8"], c["table"], c["q_start"], c["kv_len"], 3)

    def bad(i, x, err, **kw):
        a = list(ok)
        a[i] = x
        with pytest.raises(err):
            tv.attn_paged_q8(*a, **kw)
    bad(0, c["q"].float(), TypeError)
    bad(0, None, ValueError)
    bad(0, c["q"][..., :32], ValueError)
    bad(1, c["q8"][0].view(torch.int8), TypeError)
    bad(3, c["q8"][2][:-1], ValueError)
    bad(5, c["table"].long(), TypeError)
    bad(6, c["q_start"][:1], ValueError)
    bad(7, c["kv_len"].cpu(), ValueError)
    bad(8, 0, tv.TVError)
    bad(8, 3, tv.TVError, softcap=-1.0)
    bad(8, 3, tv.TVError, ws=torch.zeros(256, dtype=torch.uint8, device="cuda:0"))
    bad(8, 3, TypeError, out=torch.zeros(3, 4, 64, dtype=torch.float16, device="cuda:0"))
    wide = cache("int8", c["q8"][0].shape[0], 2, 16, 48)
    with pytest.raises(tv.TVError):  # D 64 or 128
        tv.attn_paged_q8(c["q"][..., :48].contiguous(), *wide, c["table"], c["q_start"], c["kv_len"], 3)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("fmt,N", [("e4m3", 5), ("int8", 40)])
def test_steps_of_a_serving_loop(tv, fmt, N):
    """Page map, quantised writes, tree attention, commit, and the next step: the cache's values follow the
    rows that were accepted, and attention over them is the formula's."""
    rng = random.Random(N)
    B, Hq, Hkv, D, page, P = 3, 8, 2, 64, 16, 40
    pool = B * P
    q8 = cache(fmt, pool, Hkv, page, D)
    table, held = i32([[-1] * P] * B), i32([0] * B)
    free, n_free = i32(list(range(pool))), i32([pool])
    g = torch.Generator().manual_seed(1)
    kept = [(torch.zeros(0, Hkv, D), torch.zeros(0, Hkv, D)) for _ in range(B)]  # 64-bit values per sequence
    kept = [tuple(x.double() for x in k) for k in kept]
    for step in range(4):
        lens = [k[0].shape[0] for k in kept]
        new = [rng.randint(30, 200) if step == 0 else N for _ in range(B)]
        T, q_start, kv_len = sum(new), starts(new), i32(lens)
        x = torch.randn(T, Hq + 2 * Hkv, D, generator=g).bfloat16().cuda()
        slots, st = tv.page_map(i32(q_start), kv_len, table, held, free, n_free, page, T)
        assert not bool(st.any())
        nk, nv = x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        tv.paged_append_q8(nk, nv, slots, *q8)
        vals = [values_ref(*quantise_ref(t, fmt)) for t in (nk, nv)]
        if step == 0:  # prompts
            out, lse, st = tv.attn_paged_q8(x[:, :Hq], *q8, table, i32(q_start), kv_len, max(new))
            case = dict(anc=None)
        else:
            from _paged_util import random_tree, tree_masks
            parents = [random_tree(rng, N) for _ in range(B)]
            words, depth = tree_masks(parents, (N + 63) // 64)
            anc = torch.tensor(words, dtype=torch.int64, device="cuda:0")
            out, lse, st = tv.attn_paged_q8(x[:, :Hq], *q8, table, i32(q_start), kv_len, N, anc_mask=anc)
            case = dict(anc=anc, parents=parents, depth=depth)
        assert not bool(st.any())
        rows = [tuple(torch.cat([kept[b][i], vals[i][q_start[b]:q_start[b + 1]]]) for i in range(2)) for b in range(B)]
        case.update(lens=list(zip(lens, new)), rows=rows, q=x[:, :Hq])
        check_attn_q8(out, lse, attn_ref(case, Hq, Hkv, D), case, "bf16", Hkv)
        if step == 0:
            kept = rows
            continue
        path = [[0] + sorted(rng.sample(range(1, N), rng.randint(0, min(N - 1, 9)))) for _ in range(B)]
        new_len, st = tv.commit_paged_q8(*q8, table, kv_len, i32([p + [-1] * (N - len(p)) for p in path]),
                                         i32([len(p) - 1 for p in path]))
        assert not bool(st.any())
        kept = [tuple(torch.cat([r[:L], r[[L + i for i in p]]]) for r in rows[b]) for b, (L, p) in enumerate(zip(lens, path))]
        assert np_(new_len).tolist() == [k[0].shape[0] for k in kept]
    lens = [k[0].shape[0] for k in kept]
    k, v, st = tv.paged_read_q8(*q8, table, i32(starts(lens)), i32([0] * B), sum(lens))
    for i, got in enumerate((k, v)):
        assert torch.equal(got.cpu().double(), torch.cat([s[i] for s in kept]))
    assert raw(q8[0]).numel() == pool * Hkv * page * D


ZERO_LENS = [([(300, 1), (40, 1)], False), ([(300, 60), (0, 40)], False), ([(190, 60), (5, 40)], True),
             ([(1500, 40)], False)]


@pytest.mark.parametrize("lens,tree", ZERO_LENS)
@pytest.mark.parametrize("fmt,dtype", [("e4m3", "bf16"), ("int8", "bf16"), ("e4m3", "fp16")])
@pytest.mark.parametrize("kw", [{}, dict(window=33), dict(softcap=7.0)])
def test_zero_and_tiny_rows(tv, lens, tree, fmt, dtype, kw):
    """Queries of zeros and tiny ones, keys of zeros, small ones and both: scores of 0, no less finite for that."""
    for zero_q, zero_k, size in ((True, False, 1.0), (False, True, 1.0), (True, True, 1.0), (True, False, 2.0**-30),
                                 (False, True, 2.0**-22)):
        c = make_q8(7, lens, 8, 2, 128, 16, fmt, dtype, tree=tree)
        c["q"] = c["q"].clone() * (size if not zero_q else 1.0)
        if zero_q:
            c["q"][::2] = 0
        for b, (L, n) in enumerate(lens):
            if zero_k:  # (whole tiles of them, and the new tokens)
                set_rows(c, b, 0, k=torch.zeros(min(L + n, 256), 2, 128))
                set_rows(c, b, L, k=torch.zeros(n, 2, 128))
            elif size != 1.0:
                set_rows(c, b, 0, k=c["rows"][b][0] * size)
        out, lse, status = run(tv, c, **kw)
        assert not any(status)
        check_seen(out, lse, c, 2, what=f"{zero_q} {zero_k} {size}", **kw)


@pytest.mark.parametrize("new", [1, 40])
def test_tiny_queries_beside_pages_that_are_none(tv, new):
    c = make_q8(3, [(600, new), (300, new)], 8, 2, 128, 128, "e4m3")
    c["q"] = c["q"].clone() * 2.0**-22
    c["q"][::3] = 0
    c["table"][0, 1] = -5
    hidden = {0: set(range(128, 256))}
    out, lse, status = run(tv, c)
    assert status == [1, 0]
    check_seen(out, lse, c, 2, hidden=hidden)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("scale_byte", [0, 1])
def test_a_call_on_zeros_gives_the_mean_of_v(tv, new, scale_byte):
    c = make_q8(3, [(300, new), (0, new)], 8, 2, 64, 16, "int8")
    c["q"] = torch.zeros_like(c["q"])
    c["q8"][0].view(torch.uint8).zero_()
    c["q8"][2].fill_(scale_byte)
    c["rows"] = [(torch.zeros_like(k), v) for k, v in c["rows"]]
    out, lse, status = run(tv, c)
    assert status == [0, 0]
    check_seen(out, lse, c, 2)


@pytest.mark.parametrize("new", [1, 40])
def test_large_rows_at_right_angles(tv, new):
    """Products of 0 between rows whose sizes' product is past the 32-bit range are scores of 0."""
    c = make_q8(3, [(300, new)], 8, 2, 128, 16, "e4m3")
    c["q"] = torch.zeros_like(c["q"])
    c["q"][..., 0] = 2.0**100
    k = torch.zeros(300 + new, 2, 128)
    k[..., 1] = 2.0**60
    set_rows(c, 0, 0, k=k)
    out, lse, status = run(tv, c)
    assert not any(status)
    same = dict(c, q=torch.zeros_like(c["q"]))  # (what a score may be off by goes by the sizes: none here)
    check_seen(out, lse, same, 2)


@pytest.mark.parametrize("lens", [[(90, 1), (300, 1)], [(70, 30), (300, 40)]])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_a_key_that_is_no_number_beside_the_largest_ones(tv, lens, fmt):
    """Tokens that see it get NaN, whatever the size of the keys beside it."""
    c = make_q8(4, lens, 8, 2, 128, 16, fmt, spread=0.5, q_mag=2.0**-118)
    c["q8"][2].copy_((c["q8"][2].int() + 122).clamp(0, 247).to(torch.uint8))
    c["rows"] = [(k * 2.0**122, v) for k, v in c["rows"]]
    out, lse, status = run(tv, c)
    assert not any(status)
    check_seen(out, lse, c, 2)
    want, sees = (out, lse), []
    table = np_(c["table"])
    for b, (L, n) in enumerate(lens):
        j = L + n // 2
        c["q8"][0].view(torch.uint8)[table[b, j // 16], :, j % 16] = 0
        c["q8"][2][table[b, j // 16], :, j % 16] = 255
        sees += [L + i >= j for i in range(n)]
    out, lse, status = run(tv, c)
    sees = torch.tensor(sees, device="cuda:0")
    assert not any(status) and bool(out[sees].isnan().all()) and bool(lse[sees].isnan().all())
    assert torch.equal(lse[~sees], want[1][~sees]) and same_bits(out[~sees], want[0][~sees])


@pytest.mark.parametrize("lens", [[(0, 1), (2, 1), (6, 1)], [(0, 20)], [(3, 30), (0, 40)]])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_values_up_to_the_largest_bf16_number(tv, lens, fmt):
    """Means of values near 2^128, which are bf16 numbers, are finite."""
    c = make_q8(6, lens, 8, 2, 64, 16, fmt)
    g = torch.Generator().manual_seed(3)
    for b, (L, n) in enumerate(lens):
        big = (1.0 + 0.9 * torch.rand(L + n, 2, 64, generator=g)) * 2.0**127
        big[..., ::3] *= -0.5
        set_rows(c, b, 0, v=big.bfloat16())
        assert bool((c["rows"][b][1].abs() < 2.0**128).all())
    out, lse, status = run(tv, c)
    assert not any(status)
    check_seen(out, lse, c, 2)


APART = [([(60, 4), (1500, 3)], True), ([(60, 40), (700, 64)], True), ([(60, 4), (1500, 3)], False),
         ([(60, 40), (700, 64)], False), ([(2000, 70)] * 3, True)]


@pytest.mark.parametrize("lens,tree", APART)
@pytest.mark.parametrize("Hq,D,fmt", [(8, 128, "e4m3"), (4, 64, "int8"), (2, 128, "int8")])
@pytest.mark.parametrize("bits", [12, 28, 100])
@pytest.mark.parametrize("side", ["k", "v"])
def test_large_rows_that_a_token_does_not_see(tv, lens, tree, Hq, D, fmt, bits, side):
    """A rejected node's or a later token's row, far larger than the others, costs those that do not see it nothing."""
    for where in ("last", "middle"):
        c = make_q8(5, lens, Hq, 2, D, 16, fmt, tree=tree, spread=0.7)
        for b, (L, n) in enumerate(lens):
            i = n - 1 if where == "last" else n // 2
            row = c["rows"][b][0 if side == "k" else 1][L + i:L + i + 1] * 2.0**bits
            set_rows(c, b, L + i, **{side: row})
        out, lse, status = run(tv, c)
        assert not any(status)
        check_seen(out, lse, c, 2, what=where)


@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("bits", [28, 100])
@pytest.mark.parametrize("side", ["k", "v"])
def test_large_rows_that_the_window_left(tv, n, bits, side):
    lens = [(300, n), (77, n)]
    c = make_q8(5, lens, 8, 2, 128, 16, "e4m3", spread=0.7)
    for b, (L, _) in enumerate(lens):
        j = L - 40 + n // 2 + 1  # (seen by about half of the tokens)
        row = c["rows"][b][0 if side == "k" else 1][j:j + 1] * 2.0**bits
        set_rows(c, b, j, **{side: row})
    out, lse, status = run(tv, c, window=40)
    assert not any(status)
    check_seen(out, lse, c, 2, window=40)


@pytest.mark.parametrize("lens", [[(40, 1)], [(900, 1), (300, 2)], [(40, 40)], [(900, 33)], [(3000, 64)]])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("nats,bits", [(10.0, 15), (30.0, 44), (60.0, 90)])
@pytest.mark.parametrize("at", [0, -1, 3])
def test_values_of_all_sizes_with_weights_that_make_up_for_them(tv, lens, fmt, nats, bits, at):
    """A key whose probability is e^-nats of the others' and whose value is 2^bits of theirs counts like them."""
    H, D = 2, 128
    c = make_q8(5, lens, H, H, D, 16, fmt, spread=0.5)
    q = c["q"][:1].clone()
    c["q"] = q.expand(c["T"], H, D).contiguous()
    for b, (L, n) in enumerate(lens):
        j = at % L if at < 0 else at  # (the last row that all tokens see, or one of the first)
        k = -nats * D**0.5 * q.cpu().double() / (q.cpu().double()**2).sum(2, keepdim=True)
        set_rows(c, b, j, k=k, v=c["rows"][b][1][j:j + 1] * 2.0**bits)
    out, lse, status = run(tv, c)
    assert not any(status)
    check_seen(out, lse, c, H)


@pytest.mark.parametrize("lens", [[(600, 1)], [(900, 40)]])
@pytest.mark.parametrize("spread,kw", [(2.5, {}), (12.0, {}), (25.0, dict(window=300)), (12.0, dict(softcap=9.0))])
@pytest.mark.parametrize("fmt,D", [("e4m3", 128), ("int8", 64)])
def test_values_many_powers_of_two_apart(tv, lens, spread, kw, fmt, D):
    """Each output is off by little of what its token's largest weighed value is."""
    c = make_q8(6, lens, 4, 1, D, 16, fmt, spread=0.5)
    g = torch.Generator().manual_seed(2)
    for b, (L, n) in enumerate(lens):
        set_rows(c, b, 0, v=c["rows"][b][1] * torch.exp2(torch.randn(L + n, 1, 1, generator=g) * spread))
    out, lse, status = run(tv, c, **kw)
    assert not any(status)
    check_seen(out, lse, c, 1, **kw)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("n", [1, 40])
def test_a_value_that_is_no_number_beside_scales_of_any_size(tv, fmt, n):
    """A V row that is no number has no say in the outputs of tokens that do not see it."""
    for byte in [1, 2, 60] + list(range(120, 136)) + [200, 240]:
        c = make_q8(4, [(300, n), (70, n)], 4, 2, 64, 16, fmt, spread=0.0)
        c["q8"][3].fill_(byte)
        want, sees = run(tv, c), []
        table = np_(c["table"])
        for b, (L, _) in enumerate(c["lens"]):
            j = L + n // 2
            c["q8"][1].view(torch.uint8)[table[b, j // 16], :, j % 16] = 0
            c["q8"][3][table[b, j // 16], :, j % 16] = 255
            sees += [L + i >= j for i in range(n)]
        out, lse, status = run(tv, c)
        sees = torch.tensor(sees, device="cuda:0")
        assert not any(status) and torch.equal(lse, want[1])
        assert bool(out[sees].isnan().all()) and same_bits(out[~sees], want[0][~sees]), byte


@pytest.mark.parametrize("kw", KINDS)
@pytest.mark.parametrize("lens,tree", [([(200, 1), (0, 1), (150, 4)], False), ([(300, 90), (0, 40), (77, 1)], False),
                                       ([(260, 70), (0, 9), (129, 1)], True), ([(500, 3), (64, 4)], True)])
@pytest.mark.parametrize("Hq,Hkv,D,fmt,dtype", [(8, 2, 128, "e4m3", "bf16"), (4, 4, 64, "int8", "bf16")])
@pytest.mark.parametrize("side", ["k", "v", "both"])
def test_score_kinds_over_rows_of_all_sizes(tv, kw, lens, tree, Hq, Hkv, D, fmt, dtype, side):
    """Rows that some tokens see and others do not, 2^40 of the others, and tiny ones among them."""
    kw = dict(kw)
    if kw.get("slopes"):
        kw["slopes"] = slopes_of(Hq)
    c = make_q8(9, lens, Hq, Hkv, D, 16, fmt, dtype, tree=tree, spread=0.7)
    for b, (L, n) in enumerate(lens):
        for j, bits in ((L + n - 1, 40), (max(0, L - 60), 40), (L // 2, -30), (L // 3, -30)):
            k, v = (r[j:j + 1] * 2.0**bits for r in c["rows"][b])
            set_rows(c, b, j, k=k if side != "v" else None, v=v if side != "k" else None)
    out, lse, status = run(tv, c, **kw)
    assert not any(status)
    check_seen(out, lse, c, Hkv, **kw)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("n", [1, 3, 40])
@pytest.mark.parametrize("side", ["k", "v"])
def test_rows_at_the_ends_of_what_shares_a_power_of_two(tv, fmt, n, side):
    """Rows of the other tiles some powers of two above or below those of the last."""
    for bits in (-17, -16, -15, -14, -10, -9, -8, -7, -6, -5, -4, 1, 2, 3, 4, 5, 6, 8, 9, 10, 12):
        c = make_q8(5, [(700, n), (390, n)], 4, 2, 128, 16, fmt, spread=0.0, q_mag=0.1 if bits < 6 else 2.0**-bits)
        for b, (L, _) in enumerate(c["lens"]):
            r = c["rows"][b][0 if side == "k" else 1]
            set_rows(c, b, 0, **{side: torch.cat([r[:L - 200] * 2.0**bits, r[L - 200:]])})
        out, lse, status = run(tv, c)
        assert not any(status)
        check_seen(out, lse, c, 2, what=f"{bits}")


@pytest.mark.parametrize("lens", [[(300, 40), (50, 30)], [(300, 70), (700, 9), (20, 33)]])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (7, 1)])
def test_other_sequences_queries_change_no_bit(tv, lens, dtype, Hq, Hkv):
    """Rows of a block that are another sequence's, whatever their size."""
    c = make_q8(3, lens, Hq, Hkv, 128, 16, "e4m3", dtype)
    want = run(tv, c)
    n = lens[0][1]
    c["q"] = c["q"].clone()
    for size in (2.0**30, 2.0**100) if dtype == "bf16" else (2.0**13,):
        c["q"][n:] = torch.randn(c["q"][n:].shape, generator=torch.Generator().manual_seed(1)).to(c["q"]) * size
        if dtype == "fp16":
            c["q"][n:] = c["q"][n:].clamp(-6e4, 6e4)
        out, lse, status = run(tv, c, scale=0.0)
        assert not any(status)
        assert same_bits(out[:n], want[0][:n]) and torch.equal(lse[:n], want[1][:n])


def test_rows_of_all_sizes_where_ctas_join_units_themselves(tv):
    lens = [(500 + 23 * i, 64) for i in range(45)]
    c = make_q8(5, lens, 8, 2, 64, 64, "e4m3", tree=True, spread=0.7)
    for b, (L, n) in enumerate(lens):
        k, v = c["rows"][b]
        set_rows(c, b, L + n - 1, v=v[L + n - 1:] * 2.0**40)
        set_rows(c, b, L // 2, k=k[L // 2:L // 2 + 1] * 2.0**-30, v=v[L // 2:L // 2 + 1] * 2.0**-30)
    out, lse, status = run(tv, c)
    assert not any(status)
    check_seen(out, lse, c, 2)
