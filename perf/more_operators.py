"""Operators of an 8-bit paged KV cache and of shared prefixes: the quantising cache write, reading
rows back, the commit of an accepted branch, attention of ragged chunks over the 8-bit pages, and
attention of sequences that share a long prefix, which is read once for all of them.

An 8-bit cache row (one token, one kv head, K or V) is D codes, e4m3 or int8, and one scale byte s: the
row's values are code * 2^(s - 127).  s - 127 is the smallest exponent e >= -126 with
max|x| <= M * 2^e (M = 448 or 127), codes are x * 2^-e to the nearest, ties to even; a row with an
infinity or a NaN has s = 255 and codes 0.

`listed()` names the measured cases and says what each stands for, `draw(rng)` gives more of the
same ranges, `prepare` makes a case's inputs, `run` makes one pass (elementary torch operations, or
the library's calls where `own` is true), `exact` computes the same outputs in 64 bits, and `work`
counts the bytes and operations a pass cannot do without.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
FORMATS = {"e4m3": (torch.float8_e4m3fn, 448.0), "int8": (torch.int8, 127.0)}


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


# --------------------------------------------------------------------- cases
def listed():
    attn = dict(op="attn", fmt="e4m3", dtype="bf16", page=16, Hq=32, Hkv=8, D=128, mask="causal",
                cap=0.0, window=0, alibi=False)
    pre = {k: v for k, v in dict(attn, op="prefix").items() if k != "fmt"}
    return [
        # cache write of one decode step
        dict(name="write 64 tokens", op="write", fmt="e4m3", dtype="bf16", page=16, tokens=64, Hkv=8, D=128,
             packed=True),
        # cache write of a prefill chunk, k and v views of one fused projection
        dict(name="write 8192 tokens", op="write", fmt="int8", dtype="bf16", page=16, tokens=8192, Hkv=8,
             D=128, packed=True),
        # one short sequence handed to a 16-bit consumer
        dict(name="read one of 300", op="read", fmt="int8", dtype="fp16", page=16, B=1, Hkv=8, D=128, ctx_lo=0,
             ctx_hi=0, new_lo=300, new_hi=300),
        # a batch of sequences leaving the 8-bit cache
        dict(name="read 16 sequences", op="read", fmt="e4m3", dtype="bf16", page=16, B=16, Hkv=8, D=128,
             ctx_lo=0, ctx_hi=0, new_lo=512, new_hi=8192),
        # the accepted branch of one 60-node spine tree
        dict(name="commit spine tree", op="commit", fmt="e4m3", page=16, B=1, N=60, Hkv=8, D=128, acc_lo=12,
             acc_hi=12, ctx_lo=2048, ctx_hi=2048),
        # the accepted branches of a large batch of 64-node trees
        dict(name="commit 128 trees", op="commit", fmt="int8", page=32, B=128, N=64, Hkv=8, D=128, acc_lo=0,
             acc_hi=8, ctx_lo=500, ctx_hi=2000),
        # decode of a few short sequences: latency
        dict(attn, name="attn decode of 4 short", B=4, ctx_lo=300, ctx_hi=700, new_lo=1, new_hi=1),
        # decode of a serving batch: the cache is read once
        dict(attn, name="attn decode of 64", B=64, ctx_lo=512, ctx_hi=8192, new_lo=1, new_hi=1),
        # tree verification of a ragged batch, 64 nodes a sequence
        dict(attn, name="attn 16 trees of 64", fmt="int8", mask="tree", B=16, ctx_lo=512, ctx_hi=8192, new_lo=64,
             new_hi=64),
        # a few requests just behind one system prompt: latency
        dict(pre, name="prefix decode of 3 short", groups=1, per_lo=3, per_hi=3, pre_lo=500, pre_hi=500,
             ctx_lo=5, ctx_hi=60, new_lo=1, new_hi=1),
        # decode of many requests behind one long document
        dict(pre, name="prefix decode of 64", groups=1, per_lo=64, per_hi=64, pre_lo=8000, pre_hi=8000,
             ctx_lo=30, ctx_hi=600, new_lo=1, new_hi=1),
        # draft trees of requests behind several system prompts, narrow heads
        dict(pre, name="prefix trees behind 4", dtype="fp16", page=32, Hq=16, Hkv=4, D=64, mask="tree", groups=4,
             per_lo=3, per_hi=5, pre_lo=1500, pre_hi=5000, ctx_lo=40, ctx_hi=700, new_lo=16, new_hi=48),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "commit", "attn", "attn", "attn", "prefix", "prefix"])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    dtype, fmt = rng.choice(["bf16", "fp16"]), rng.choice(["e4m3", "int8"])
    D = rng.choice([64, 128])
    if op == "write":
        return dict(op=op, fmt=fmt, dtype=dtype, page=page, tokens=_log_int(rng, 1, 8192),
                    Hkv=rng.choice([1, 2, 3, 5, 8]), D=D, packed=rng.random() < 0.5)
    if op == "read":
        hi = _log_int(rng, 1, 8192)
        ctx = rng.choice([0, _log_int(rng, 1, 1000)])
        return dict(op=op, fmt=fmt, dtype=dtype, page=page, B=_log_int(rng, 1, 16), Hkv=rng.choice([1, 2, 3, 8]),
                    D=D, ctx_lo=0, ctx_hi=ctx, new_lo=rng.randint(1, hi), new_hi=hi)
    if op == "commit":
        N = _log_int(rng, 2, 512)
        ctx = _log_int(rng, 1, 2000)
        return dict(op=op, fmt=fmt, page=page, B=_log_int(rng, 1, 128), N=N, Hkv=rng.choice([1, 2, 4, 8]), D=D,
                    acc_lo=0, acc_hi=min(N - 1, rng.randint(0, 16)), ctx_lo=ctx // 2, ctx_hi=ctx)
    Hkv = rng.choice([1, 2, 4, 8])
    G = min(rng.choice([1, 2, 4, 5, 7, 8]), 32 // Hkv)
    case = dict(op=op, dtype=dtype, page=page, Hq=Hkv * G, Hkv=Hkv, D=D, mask=rng.choice(["causal", "causal", "tree"]),
                cap=rng.choice([0.0, 0.0, 0.0, 20.0, 50.0]), window=rng.choice([0, 0, 0, 512, 1111]),
                alibi=rng.random() < 0.25)
    if op == "attn":
        kind = rng.choice(["one", "one", "few", "many"])
        B = _log_int(rng, 1, 48)
        if kind == "one" and case["mask"] == "causal":
            new_lo, new_hi, ctx = 1, 1, _log_int(rng, 1, 8192)
        elif kind == "many" and case["mask"] == "causal":
            B = min(B, 4)
            new_hi, ctx = _log_int(rng, 65, 500), _log_int(rng, 1, 2048)
            new_lo = rng.randint(1, new_hi)
        else:
            B = min(B, 12)
            new_lo, new_hi, ctx = 1, _log_int(rng, 2, 90), _log_int(rng, 1, 6000)
        return dict(case, fmt=fmt, B=B, ctx_lo=ctx // rng.choice([1, 2, 9]), ctx_hi=ctx, new_lo=new_lo, new_hi=new_hi)
    pre, ctx = _log_int(rng, 1, 8192), _log_int(rng, 1, 800)
    per, new = _log_int(rng, 1, 24), rng.choice([1, 1, _log_int(rng, 2, 40)])
    per = min(per, max(1, 200 // new))
    return dict(case, groups=rng.choice([1, 1, 2, 3]), per_lo=rng.randint(1, per), per_hi=per,
                pre_lo=pre // rng.choice([1, 2, 9]), pre_hi=pre, ctx_lo=ctx // rng.choice([1, 3]), ctx_hi=ctx,
                new_lo=1, new_hi=new)


def _lengths(case):
    """Prefix and new-token lengths of a case's sequences: fixed by the case, so that the shapes are."""
    rng = random.Random("%d %d %d" % (case["B"], case["ctx_hi"], case["new_hi"]))
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["B"])]
    return ctx, new


def _groups(case):
    """(shared prefix lengths, sequences of each group, own cached lengths, new tokens)."""
    rng = random.Random("%d %d %d %d" % (case["groups"], case["pre_hi"], case["ctx_hi"], case["new_hi"]))
    per = [rng.randint(case["per_lo"], case["per_hi"]) for _ in range(case["groups"])]
    pre = [rng.randint(case["pre_lo"], case["pre_hi"]) for _ in per]
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(sum(per))]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in ctx]
    return pre, per, ctx, new


def _commit_plan(case):
    """Prefix lengths and accepted branches [B][1 + accepted], node ids strictly increasing from 0."""
    rng = random.Random("%d %d %d" % (case["B"], case["N"], case["ctx_hi"]))
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    paths = [[0] + sorted(rng.sample(range(1, case["N"]), rng.randint(case["acc_lo"], case["acc_hi"])))
             for _ in range(case["B"])]
    return ctx, paths


def _ceil(a, b):
    return -(-a // b)


# -------------------------------------------------------------------- inputs
def _gen(seed, dev):
    return torch.Generator(device=dev).manual_seed(seed)


def _randn(g, dev, dtype, *shape):
    return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dtype)


def _i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _starts(new):
    out = [0]
    for n in new:
        out.append(out[-1] + n)
    return out


def _tables(lens, page, seed, dev):
    """Shuffled pages for sequences of these lengths: (table [B, P] with -1 past a sequence's pages,
    number of pages in the pool)."""
    held = [_ceil(n, page) for n in lens]
    pool = sum(held) + 7
    ids = list(range(pool))
    random.Random(seed).shuffle(ids)
    P = max(max(held), 1)
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-1] * (P - h))
        at += h
    return _i32(table, dev), pool


def _codes(g, dev, fmt, pool, Hkv, page, D):
    """Codes and scale bytes of a filled 8-bit cache: rows of about unit size, whose largest codes lie in
    the format's upper binade, as quantised rows' do."""
    shape = (pool, Hkv, page, D)
    x = torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)
    codes = x.mul_(110.0).clamp_(-448.0, 448.0) if fmt == "e4m3" else x.mul_(31.0).round_().clamp_(-127.0, 127.0)
    first = 119 if fmt == "e4m3" else 121
    scale = torch.randint(first, first + 3, shape[:3], generator=g, device=dev, dtype=torch.uint8)
    return codes.to(FORMATS[fmt][0]), scale


def _tree_masks(new, seed, dev):
    """Ancestor-or-self bit masks [T, W] of random topological trees, one per sequence, and depths [T]."""
    rng = random.Random(seed)
    W = _ceil(max(new), 64)
    rows, depth = [], []
    for n in new:
        anc, dep = [], []
        for i in range(n):
            p = rng.randrange(max(0, i - 6), i) if i else -1
            anc.append((1 << i) | (anc[p] if i else 0))
            dep.append(dep[p] + 1 if i else 0)
        depth += dep
        for a in anc:
            words = [(a >> (64 * w)) & (2**64 - 1) for w in range(W)]
            rows.append([w - 2**64 if w >= 2**63 else w for w in words])
    return torch.tensor(rows, dtype=torch.int64, device=dev), torch.tensor(depth, device=dev)


def prepare(case, seed):
    dev = _device()
    g = _gen(seed, dev)
    op, page, Hkv, D = case["op"], case["page"], case["Hkv"], case["D"]
    st = dict(case=case)
    if op == "write":
        T, dt = case["tokens"], DTYPES[case["dtype"]]
        pool = _ceil(T, page) + 5
        # rows of different sizes, and a few channels that stand out, as projections give them
        size = torch.exp2(torch.randn(T, 1, 1, generator=g, device=dev))
        channel = 1.0 + 7.0 * (torch.rand(1, 1, D, generator=g, device=dev) < 0.03).float()
        if case["packed"]:  # views of a fused projection's output
            qkv = (_randn(g, dev, torch.float32, T, 3 * Hkv, D) * size * channel).to(dt)
            k, v = qkv[:, Hkv:2 * Hkv], qkv[:, 2 * Hkv:]
        else:
            k = (_randn(g, dev, torch.float32, T, Hkv, D) * size * channel).to(dt)
            v = (_randn(g, dev, torch.float32, T, Hkv, D) * size).to(dt)
        kc, ks = _codes(g, dev, case["fmt"], pool, Hkv, page, D)
        vc, vs = _codes(g, dev, case["fmt"], pool, Hkv, page, D)
        # consecutive positions of one sequence in shuffled pages; a few padding tokens have no slot
        order = torch.randperm(pool, generator=g, device=dev)
        t = torch.arange(T, device=dev)
        slots = order[t // page] * page + t % page
        slots[T - T // 16:] = -1
        st.update(k=k, v=v, kc=kc, vc=vc, ks=ks, vs=vs, slots=slots)
    elif op == "read":
        ctx, new = _lengths(case)
        table, pool = _tables([c + n for c, n in zip(ctx, new)], page, seed, dev)
        kc, ks = _codes(g, dev, case["fmt"], pool, Hkv, page, D)
        vc, vs = _codes(g, dev, case["fmt"], pool, Hkv, page, D)
        st.update(table=table, kc=kc, vc=vc, ks=ks, vs=vs, q_start=_i32(_starts(new), dev), start=_i32(ctx, dev),
                  T=sum(new))
    elif op == "commit":
        ctx, paths = _commit_plan(case)
        N = case["N"]
        table, pool = _tables([c + N for c in ctx], page, seed, dev)
        kc, ks = _codes(g, dev, case["fmt"], pool, Hkv, page, D)
        vc, vs = _codes(g, dev, case["fmt"], pool, Hkv, page, D)
        st.update(table=table, kc=kc, vc=vc, ks=ks, vs=vs, kv_len=_i32(ctx, dev),
                  path=_i32([p + [-1] * (N - len(p)) for p in paths], dev),
                  acc=_i32([len(p) - 1 for p in paths], dev), most=max(len(p) for p in paths))
    else:
        Hq, dt = case["Hq"], DTYPES[case["dtype"]]
        if op == "attn":
            ctx, new = _lengths(case)
            table, pool = _tables([c + n for c, n in zip(ctx, new)], page, seed, dev)
            kc, ks = _codes(g, dev, case["fmt"], pool, Hkv, page, D)
            vc, vs = _codes(g, dev, case["fmt"], pool, Hkv, page, D)
            st.update(kc=kc, vc=vc, ks=ks, vs=vs)
        else:
            # the prefixes' pages and the sequences' own come from one pool
            pre, per, ctx, new = _groups(case)
            both, pool = _tables(pre + [c + n for c, n in zip(ctx, new)], page, seed, dev)
            table = both[len(pre):].contiguous()
            st.update(pre_table=both[:len(pre)].contiguous(), pre_len=_i32(pre, dev),
                      group_start=_i32(_starts(per), dev), most_group=max(_starts(new)[b] - _starts(new)[a]
                                                                       for a, b in zip(_starts(per), _starts(per)[1:])),
                      kp=_randn(g, dev, dt, pool, Hkv, page, D), vp=_randn(g, dev, dt, pool, Hkv, page, D))
        st.update(q=_randn(g, dev, dt, sum(new), Hq, D), table=table, q_start=_i32(_starts(new), dev),
                  kv_len=_i32(ctx, dev), max_q=max(new), anc=None, depth=None, slopes=None)
        if case["mask"] == "tree":
            st["anc"], st["depth"] = _tree_masks(new, seed, dev)
        if case["alibi"]:  # the geometric series of slopes
            st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)],
                                        dtype=torch.float32, device=dev)
    return st


# ---------------------------------------------------------------------- runs
def run(st):
    return {"write": _run_write, "read": _run_read, "commit": _run_commit, "attn": _run_attn,
            "prefix": _run_prefix}[st["case"]["op"]](st)


def _quantise(x, fmt):
    """Codes [.., D] and scale bytes [..] of rows x [.., D]."""
    kind, most = FORMATS[fmt]
    x = x.float()
    top = x.abs().amax(-1)
    fine = torch.isfinite(top)
    m, e = torch.frexp(torch.where(fine, top, torch.ones_like(top)) / most)  # m 2^e, m in [1/2, 1)
    e = torch.where(m == 0.5, e - 1, e).clamp_min(-126)
    e = torch.where(top == 0, torch.full_like(e, -126), e)
    y = x * ((127 - e) << 23).view(torch.float32)[..., None]  # x 2^-e
    y = torch.where(fine[..., None], y, torch.zeros_like(y))
    codes = y.to(kind) if fmt == "e4m3" else torch.round(y).to(kind)
    return codes, torch.where(fine, e + 127, torch.full_like(e, 255)).to(torch.uint8)


def _values(codes, scale):
    """The 32-bit values that codes [.., D] of any format with scale bytes [..] stand for."""
    f = (scale.to(torch.int32) << 23).view(torch.float32)
    f = torch.where(scale == 255, torch.full_like(f, float("nan")), f)
    return codes.float() * f[..., None]


def _rows(codes, scale, page, row):
    """Codes and scales of rows `row` of pages `page` (index arrays of one shape): [.., Hkv, D], [.., Hkv]."""
    return codes.view(torch.uint8)[page, :, row].view(codes.dtype), scale[page, :, row]


def _run_write(st):
    if own:
        import speculative_decoding_tree_tv_gb300 as tv
        tv.paged_append_q8(st["k"], st["v"], st["slots"], st["kc"], st["vc"], st["ks"], st["vs"])
    else:
        page, slots, fmt = st["case"]["page"], st["slots"], st["case"]["fmt"]
        keep = slots >= 0
        # a token without a slot writes what the last token with one writes
        last = torch.where(keep, torch.arange(len(slots), device=slots.device), 0).amax()
        t = torch.where(keep, torch.arange(len(slots), device=slots.device), last)
        p, r = slots[t] // page, slots[t] % page
        kc, ks = _quantise(st["k"], fmt)
        vc, vs = _quantise(st["v"], fmt)
        st["kc"].view(torch.uint8)[p, :, r] = kc.view(torch.uint8)[t]
        st["vc"].view(torch.uint8)[p, :, r] = vc.view(torch.uint8)[t]
        st["ks"][p, :, r] = ks[t]
        st["vs"][p, :, r] = vs[t]
    return dict(k=st["kc"], v=st["vc"], ks=st["ks"], vs=st["vs"])


def _run_read(st):
    dt = DTYPES[st["case"]["dtype"]]
    if own:
        import speculative_decoding_tree_tv_gb300 as tv
        k, v, status = tv.paged_read_q8(st["kc"], st["vc"], st["ks"], st["vs"], st["table"], st["q_start"],
                                        st["start"], st["T"], dtype=dt)
        return dict(k=k, v=v, status=status)
    page, q_start = st["case"]["page"], st["q_start"].long()
    t = torch.arange(st["T"], device=q_start.device)
    b = torch.searchsorted(q_start[1:], t, right=True)
    pos = st["start"].long()[b] + t - q_start[b]
    p, r = st["table"].long()[b, pos // page], pos % page
    most = torch.finfo(dt).max
    k = _values(*_rows(st["kc"], st["ks"], p, r)).clamp(-most, most)
    v = _values(*_rows(st["vc"], st["vs"], p, r)).clamp(-most, most)
    return dict(k=k.to(dt), v=v.to(dt), status=torch.zeros_like(st["start"]))


def _run_commit(st):
    if own:
        import speculative_decoding_tree_tv_gb300 as tv
        new_len, status = tv.commit_paged_q8(st["kc"], st["vc"], st["ks"], st["vs"], st["table"], st["kv_len"],
                                             st["path"], st["acc"])
    else:
        page, table, kv_len, acc = st["case"]["page"], st["table"].long(), st["kv_len"].long(), st["acc"].long()
        d = torch.arange(st["most"], device=table.device)
        path = st["path"][:, :st["most"]].long()
        path = torch.where(d <= acc[:, None], path, torch.zeros_like(path))  # rows past the branch:
        to = torch.where(d <= acc[:, None], d, torch.zeros_like(d))          # the root's once more
        src, dst = kv_len[:, None] + path, kv_len[:, None] + to
        sp, dp = table.gather(1, src // page), table.gather(1, dst // page)
        kc, vc = st["kc"].view(torch.uint8), st["vc"].view(torch.uint8)
        kc[dp, :, dst % page] = kc[sp, :, src % page]
        vc[dp, :, dst % page] = vc[sp, :, src % page]
        st["ks"][dp, :, dst % page] = st["ks"][sp, :, src % page]
        st["vs"][dp, :, dst % page] = st["vs"][sp, :, src % page]
        new_len, status = st["kv_len"] + st["acc"] + 1, torch.zeros_like(st["acc"])
    return dict(k=st["kc"], v=st["vc"], ks=st["ks"], vs=st["vs"], new_len=new_len, status=status)


def _attend(case, st, tok, k, v, pos_q, pos_k, seen):
    """Unnormalised attention of padded query tokens tok [X, M] over k, v [X, Hkv, L, D] in 32 bits, with
    positions pos_q [X, M], pos_k [X, 1, L] or [L] and visibility [X, M, L]: outputs, sums and maxima."""
    (X, M), Hkv, L, D = tok.shape, k.shape[1], k.shape[2], k.shape[3]
    G = case["Hq"] // Hkv
    q = st["q"][tok].float().view(X, M, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(X, Hkv, G * M, D)
    s = torch.matmul(q, k.transpose(2, 3)).mul_(1.0 / math.sqrt(D)).view(X, Hkv, G, M, L)
    if case["cap"]:
        s = s.div_(case["cap"]).tanh_().mul_(case["cap"])
    dist = pos_q[:, :, None] - pos_k
    if case["window"]:
        seen = seen & (dist < case["window"])
    if st["slopes"] is not None:
        s = s - st["slopes"].view(1, Hkv, G, 1, 1) * dist[:, None, None].float()
    s = s.masked_fill_(~seen[:, None, None], float("-inf"))
    top = s.amax(-1, keepdim=True)
    low = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    s = s.sub_(low).exp_()
    return torch.matmul(s.view(X, Hkv, G * M, L), v).view(X, Hkv, G, M, D), s.sum(-1, keepdim=True), top


def _finish(st, o, total, top):
    """Rows [T, Hq, ..] of the joined sums: out and lse."""
    T, Hq, D = st["q"].shape
    o = torch.where(total == 0, torch.zeros_like(o), o / total)
    return o.reshape(T, Hq, D).to(st["q"].dtype), (top + total.log()).reshape(T, Hq)


def _own_keys(case, st, k, v):
    """_attend over the sequences' own rows, k, v [B, P, Hkv, page, D]: results as rows [T, Hkv, G, ..]."""
    q_start, kv_len, dev = st["q_start"].long(), st["kv_len"].long(), st["q"].device
    T, B, n, Hkv, D = len(st["q"]), len(kv_len), st["max_q"], case["Hkv"], case["D"]
    k = k.permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    v = v.permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    L = k.shape[2]
    i = torch.arange(n, device=dev)
    tok = (q_start[:-1, None] + i).clamp_max(T - 1)
    j = torch.arange(L, device=dev)
    a = j - kv_len[:, None]  # the chunk's own slots
    inside = (a >= 0) & (a < (q_start[1:] - q_start[:-1])[:, None])
    if st["anc"] is None:
        pos_q, pos_k = kv_len[:, None] + i, j
        seen = j <= pos_q[:, :, None]
    else:
        pos_q = kv_len[:, None] + st["depth"][tok]
        aa = a.clamp(0, n - 1)
        pos_k = torch.where(inside, kv_len[:, None] + st["depth"][(q_start[:-1, None] + aa).clamp_max(T - 1)],
                            j)[:, None]
        words = st["anc"][tok].gather(2, (aa // 64)[:, None, :].expand(B, n, L))
        seen = (a < 0)[:, None, :] | (inside[:, None, :] & ((words >> (aa % 64)[:, None, :]) & 1).bool())
    o, total, top = _attend(case, st, tok, k, v, pos_q, pos_k, seen)
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(q_start[1:], t, right=True)
    r = t - q_start[b]
    return o[b, :, :, r], total[b, :, :, r], top[b, :, :, r], b, pos_q[b, r]


def _run_attn(st):
    case = st["case"]
    if own:
        import speculative_decoding_tree_tv_gb300 as tv
        out, lse, status = tv.attn_paged_q8(st["q"], st["kc"], st["vc"], st["ks"], st["vs"], st["table"],
                                            st["q_start"], st["kv_len"], st["max_q"], anc_mask=st["anc"],
                                            softcap=case["cap"], window=case["window"], slopes=st["slopes"])
        return dict(out=out, lse=lse, status=status)
    table = st["table"].long().clamp_min(0)
    k = _values(st["kc"].view(torch.uint8)[table].view(st["kc"].dtype), st["ks"][table])
    v = _values(st["vc"].view(torch.uint8)[table].view(st["vc"].dtype), st["vs"][table])
    o, total, top, _, _ = _own_keys(case, st, k, v)
    out, lse = _finish(st, o, total, top)
    return dict(out=out, lse=lse, status=torch.zeros_like(st["kv_len"]))


def _run_prefix(st):
    case = st["case"]
    if own:
        import speculative_decoding_tree_tv_gb300 as tv
        out, lse, status = tv.attn_paged_prefix(st["q"], st["kp"], st["vp"], st["pre_table"], st["pre_len"],
                                                st["group_start"], st["table"], st["q_start"], st["kv_len"],
                                                st["max_q"], anc_mask=st["anc"], softcap=case["cap"],
                                                window=case["window"], slopes=st["slopes"])
        return dict(out=out, lse=lse, status=status)
    table, T, dev = st["table"].long().clamp_min(0), len(st["q"]), st["q"].device
    o1, l1, m1, b, pos = _own_keys(case, st, st["kp"][table].float(), st["vp"][table].float())
    # the prefixes' rows, each group's against all of its tokens
    starts = st["q_start"].long()[st["group_start"].long()]
    pre_len, Hkv, D = st["pre_len"].long(), case["Hkv"], case["D"]
    table = st["pre_table"].long().clamp_min(0)
    k = st["kp"][table].permute(0, 2, 1, 3, 4).reshape(len(pre_len), Hkv, -1, D).float()
    v = st["vp"][table].permute(0, 2, 1, 3, 4).reshape(len(pre_len), Hkv, -1, D).float()
    tok = (starts[:-1, None] + torch.arange(st["most_group"], device=dev)).clamp_max(T - 1)
    j = torch.arange(k.shape[2], device=dev)
    seen = (j < pre_len[:, None])[:, None].expand(-1, tok.shape[1], -1)
    o, total, top = _attend(case, st, tok, k, v, pre_len[:, None] + pos[tok], j, seen)
    t = torch.arange(T, device=dev)
    g = torch.searchsorted(starts[1:], t, right=True)
    r = t - starts[g]
    o2, l2, m2 = o[g, :, :, r], total[g, :, :, r], top[g, :, :, r]
    m = torch.maximum(m1, m2)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    f1, f2 = (m1 - m).exp(), (m2 - m).exp()
    out, lse = _finish(st, o1 * f1 + o2 * f2, l1 * f1 + l2 * f2, m)
    return dict(out=out, lse=lse, status=torch.zeros_like(st["kv_len"]))


# --------------------------------------------------------------------- exact
def _pow2(e):
    """2^e in 64 bits for whole e (a pow may be off by a last bit, which would break ties)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_row_codes(x, fmt):
    """Codes as 64-bit values, by the definition: exponents from base-2 logarithms put right by comparison,
    the code's step from its own binade."""
    x = x.double()
    most = FORMATS[fmt][1]
    top = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top / most)).clamp_min(-126.0).nan_to_num(neginf=-126.0)
    e = torch.where(top > most * _pow2(e), e + 1, e)
    e = torch.where((top <= most * _pow2(e - 1)) & (e > -126), e - 1, e)
    y = x * _pow2(-e)
    if fmt == "int8":
        return torch.round(y)
    b = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6)))
    step = _pow2(torch.where(y.abs() >= _pow2(b + 1), b + 1, torch.where(y.abs() < _pow2(b.clamp_min(-6)), b - 1, b)
                             ).clamp_min(-6) - 3)
    return torch.round(y / step) * step


def _exact_values(codes, scale):
    return codes.double() * _pow2(scale.to(torch.int64) - 127)[..., None]


def exact(case, seed):
    st = prepare(case, seed)
    page = case["page"]
    if case["op"] == "write":
        if case["fmt"] == "int8":
            return None  # whole numbers and nothing else
        kc, vc = st["kc"].double(), st["vc"].double()
        k, v = _exact_row_codes(st["k"], case["fmt"]), _exact_row_codes(st["v"], case["fmt"])
        for t, s in enumerate(st["slots"].tolist()):
            if s >= 0:
                kc[s // page, :, s % page] = k[t]
                vc[s // page, :, s % page] = v[t]
        return dict(k=kc, v=vc, ks=None, vs=None)
    if case["op"] == "read":
        ctx, new = _lengths(case)
        ks, vs = [], []
        for b, (c, n) in enumerate(zip(ctx, new)):
            pos = torch.arange(c, c + n, device=st["table"].device)
            ids = st["table"][b][pos // page].long()
            both = [_exact_values(codes.to(torch.float32)[ids, :, pos % page], scale[ids, :, pos % page])
                    for codes, scale in ((st["kc"], st["ks"]), (st["vc"], st["vs"]))]
            ks.append(both[0])
            vs.append(both[1])
        return dict(k=torch.cat(ks), v=torch.cat(vs), status=None)
    if case["op"] == "commit":
        if case["fmt"] == "int8":
            return None  # whole numbers and nothing else
        table = st["table"].tolist()
        ctx, paths = _commit_plan(case)
        out = []
        for pages in (st["kc"].double(), st["vc"].double()):
            for b, path in enumerate(paths):
                rows = [pages[table[b][(ctx[b] + p) // page], :, (ctx[b] + p) % page].clone() for p in path]
                for d, r in enumerate(rows):
                    pages[table[b][(ctx[b] + d) // page], :, (ctx[b] + d) % page] = r
            out.append(pages)
        return dict(k=out[0], v=out[1], ks=None, vs=None, new_len=None, status=None)
    return _exact_attn(case, st)


def _exact_attn(case, st):
    """Sequence by sequence and head by head, over the rows that the tables name, a shared prefix's first."""
    if case["op"] == "attn":
        ctx, new = _lengths(case)
        shared, group = [0] * len(ctx), [None] * len(ctx)
    else:
        pre, per, ctx, new = _groups(case)
        group = [g for g, n in enumerate(per) for _ in range(n)]
        shared = [pre[g] for g in group]
    Hq, Hkv, D, page, dev = case["Hq"], case["Hkv"], case["D"], case["page"], st["q"].device
    out = torch.zeros(sum(new), Hq, D, dtype=torch.float64, device=dev)
    lse = torch.full((sum(new), Hq), -math.inf, dtype=torch.float64, device=dev)

    def gather(table, n):
        """64-bit K and V [n, Hkv, D] of a table row's first n positions."""
        at = torch.arange(n, device=dev)
        ids = table[at // page].long()
        if case["op"] == "prefix":
            return [x[ids, :, at % page].double() for x in (st["kp"], st["vp"])]
        raw = [x.view(torch.uint8)[ids, :, at % page].view(x.dtype).to(torch.float32) for x in (st["kc"], st["vc"])]
        return [_exact_values(c, s[ids, :, at % page]) for c, s in zip(raw, (st["ks"], st["vs"]))]

    start = 0
    for b, (L, n, S) in enumerate(zip(ctx, new, shared)):
        keys, vals = gather(st["table"][b], L + n)
        if S:
            pk, pv = gather(st["pre_table"][group[b]], S)
            keys, vals = torch.cat([pk, keys]), torch.cat([pv, vals])
        seen_by_all = S + L
        kpos = torch.arange(S + L + n, device=dev)
        qpos = seen_by_all + torch.arange(n, device=dev)
        if case["mask"] == "tree":
            nodes = torch.arange(n, device=dev)
            bits = (st["anc"][start:start + n][:, nodes >> 6] >> (nodes & 63)) & 1
            up = bits.sum(1) - 1  # ancestors of each node: its depth
            qpos = seen_by_all + up
            kpos[seen_by_all:] = seen_by_all + up
            visible = torch.cat([torch.ones(n, seen_by_all, dtype=torch.bool, device=dev), bits == 1], 1)
        else:
            visible = kpos[None] <= qpos[:, None]
        away = (qpos[:, None] - kpos[None]).double()
        if case["window"] > 0:
            visible &= away < case["window"]
        for h in range(Hq):
            kh = h // (Hq // Hkv)
            x = st["q"][start:start + n, h].double() @ keys[:, kh].T / math.sqrt(D)
            if case["cap"] > 0:
                x = case["cap"] * torch.tanh(x / case["cap"])
            if case["alibi"]:
                x = x - float(st["slopes"][h]) * away
            x = torch.where(visible, x, torch.full_like(x, -math.inf))
            z = torch.logsumexp(x, 1)
            lse[start:start + n, h] = z
            p = torch.exp(x - z[:, None])
            out[start:start + n, h] = torch.where(torch.isfinite(z)[:, None], p @ vals[:, kh],
                                                  torch.zeros_like(vals[:1, kh]))
        start += n
    return dict(out=out, lse=lse, status=None)


# ---------------------------------------------------------------------- work
def work(case):
    op, Hkv, D, page = case["op"], case["Hkv"], case["D"], case["page"]
    row = Hkv * (D + 1)  # bytes of a token's codes and scales in K or V
    if op == "write":
        rows = case["tokens"] - case["tokens"] // 16
        return dict(bytes=8 * case["tokens"] + 2 * rows * (2 * Hkv * D + row), flops=0)
    if op == "read":
        ctx, new = _lengths(case)
        return dict(bytes=2 * sum(new) * (2 * Hkv * D + row) + 4 * _ceil(sum(new), page) + 12 * len(new), flops=0)
    if op == "commit":
        ctx, paths = _commit_plan(case)
        rows = sum(sum(p != d for d, p in enumerate(path)) for path in paths)
        return dict(bytes=2 * 2 * rows * row + 4 * sum(map(len, paths)) + 16 * case["B"], flops=0)
    win, tree = case["window"] or 1 << 40, case["mask"] == "tree"
    if op == "attn":
        ctx, new = _lengths(case)
        shared, once = [0] * len(ctx), 0
    else:
        pre, per, ctx, new = _groups(case)
        shared = [s for s, n in zip(pre, per) for _ in range(n)]
        ends = _starts(per)
        # a prefix is read once, as far as the furthest reaching window of its sequences
        once = sum(max(min(s, max(0, win - 1 - c)) for c in ctx[a:b]) for s, a, b in zip(pre, ends, ends[1:]))
        row = 2 * Hkv * D
    keys = once + sum(c + n - max(0, c - win + 1) for c, n in zip(ctx, new) if n)
    # a tree node sees the prefix, and about log-many ancestors: counted as the prefix and itself
    pairs = sum(sum(min(win, s + c + (1 if tree else i + 1)) for i in range(n)) for s, c, n in zip(shared, ctx, new))
    T = sum(new)
    return dict(bytes=2 * keys * row + 2 * 2 * T * case["Hq"] * D + 4 * T * case["Hq"] + 4 * _ceil(keys, page),
                flops=4 * D * case["Hq"] * pairs)
