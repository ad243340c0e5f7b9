"""Operators of the paged KV cache: page allocation with slot maps, the cache write, attention of
ragged chunks of new tokens (causal or tree-masked, one token to thousands, capped, windowed or
distance-biased scores) over the pages, and the commit of an accepted branch.

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


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


# --------------------------------------------------------------------- cases
def listed():
    attn = dict(op="attn", dtype="bf16", page=16, Hq=32, Hkv=8, D=128, mask="causal", cap=0.0,
                window=0, alibi=False)
    return [
        # one decode step of a serving batch: a page or none per sequence, pages back after it
        dict(name="pages, decode step of 64", op="pages", B=64, page=16, ctx_lo=512, ctx_hi=8192,
             new_lo=1, new_hi=1),
        # admission of a batch of prompts: every page is new, and all go back when they finish
        dict(name="pages, 200 prompts", op="pages", B=200, page=16, ctx_lo=0, ctx_hi=0,
             new_lo=40, new_hi=2000),
        # cache write of one decode step
        dict(name="append, 64 tokens", op="append", dtype="bf16", page=16, tokens=64, Hkv=8, D=128,
             packed=True),
        # cache write of a prefill chunk, k and v views of one fused projection
        dict(name="append, 8192 tokens", op="append", dtype="bf16", page=16, tokens=8192, Hkv=8,
             D=128, packed=True),
        # the accepted branch of one 60-node spine tree
        dict(name="commit, spine tree", op="commit", dtype="bf16", page=16, B=1, N=60, Hkv=8, D=128,
             acc_lo=12, acc_hi=12, ctx_lo=2048, ctx_hi=2048),
        # the accepted branches of a large batch of 64-node trees
        dict(name="commit, 128 trees", op="commit", dtype="fp16", page=32, B=128, N=64, Hkv=8, D=128,
             acc_lo=0, acc_hi=8, ctx_lo=500, ctx_hi=2000),
        # decode of a few short sequences: latency
        dict(attn, name="attn, decode of 4 short", B=4, ctx_lo=300, ctx_hi=700, new_lo=1, new_hi=1),
        # decode of a serving batch: the cache is read once
        dict(attn, name="attn, decode of 64", B=64, ctx_lo=512, ctx_hi=8192, new_lo=1, new_hi=1),
        # tree verification of a ragged batch, 64 nodes a sequence
        dict(attn, name="attn, 16 trees of 64", mask="tree", B=16, ctx_lo=512, ctx_hi=8192,
             new_lo=64, new_hi=64),
        # one chunk of a long prompt behind a cached prefix
        dict(attn, name="attn, chunk of 2048", page=64, B=1, ctx_lo=6100, ctx_hi=6100, new_lo=2048,
             new_hi=2048),
        # prefill chunks and short continuations in one batch, capped scores in a local window
        dict(attn, name="attn, mixed capped window", dtype="fp16", page=32, Hq=16, Hkv=8, D=128, B=12,
             ctx_lo=0, ctx_hi=4000, new_lo=1, new_hi=700, cap=50.0, window=1024),
        # prompts from empty caches, heads of their own keys, distance bias, narrow heads
        dict(attn, name="attn, prompts with bias", page=128, Hq=12, Hkv=12, D=64, B=5, ctx_lo=0,
             ctx_hi=0, new_lo=200, new_hi=1500, alibi=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pages", "append", "commit", "attn", "attn", "attn"])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    dtype = rng.choice(["bf16", "fp16"])
    D = rng.choice([64, 128])
    if op == "pages":
        hi = _log_int(rng, 1, 2000)
        ctx = rng.choice([0, _log_int(rng, 1, 8192)])
        return dict(op=op, B=_log_int(rng, 1, 300), page=page, ctx_lo=ctx // 3, ctx_hi=ctx,
                    new_lo=rng.randint(0, hi), new_hi=hi)
    if op == "append":
        return dict(op=op, dtype=dtype, page=page, tokens=_log_int(rng, 1, 8192),
                    Hkv=rng.choice([1, 2, 3, 5, 8]), D=D, packed=rng.random() < 0.5)
    if op == "commit":
        N = _log_int(rng, 2, 512)
        ctx = _log_int(rng, 1, 2000)
        return dict(op=op, dtype=dtype, page=page, B=_log_int(rng, 1, 128), N=N,
                    Hkv=rng.choice([1, 2, 4, 8]), D=D, acc_lo=0, acc_hi=min(N - 1, rng.randint(0, 16)),
                    ctx_lo=ctx // 2, ctx_hi=ctx)
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 5, 7, 8])
    G = min(G, 32 // Hkv)
    mask = rng.choice(["causal", "causal", "tree"])
    kind = rng.choice(["one", "few", "many"])
    B = _log_int(rng, 1, 48)
    if kind == "one" and mask == "causal":
        new_lo, new_hi, ctx = 1, 1, _log_int(rng, 1, 8192)
    elif kind == "many" and mask == "causal":
        B = min(B, 6)
        new_hi, ctx = _log_int(rng, 65, 1500), _log_int(rng, 1, 4096)
        new_lo = rng.randint(1, new_hi)
    else:
        B = min(B, 16)
        new_lo, new_hi, ctx = 1, _log_int(rng, 2, 100 if mask == "causal" else 300), _log_int(rng, 1, 6000)
    return dict(op="attn", dtype=dtype, page=page, Hq=Hkv * G, Hkv=Hkv, D=D, mask=mask,
                cap=rng.choice([0.0, 0.0, 20.0, 50.0]), window=rng.choice([0, 0, 512, 1111]),
                alibi=rng.random() < 0.3, B=B, ctx_lo=ctx // rng.choice([1, 2, 9]), ctx_hi=ctx,
                new_lo=new_lo, new_hi=new_hi)


def _lengths(case):
    """Prefix and new-token lengths of a case's sequences: fixed by the case, so that the shapes are."""
    rng = random.Random("%d %d %d" % (case["B"], case["ctx_hi"], case.get("new_hi", 0)))
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["B"])]
    return ctx, new


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
    pages held [B], number of pages in the pool, the pool's other pages)."""
    held = [_ceil(n, page) for n in lens]
    pool = sum(held) + 7
    ids = list(range(pool))
    random.Random(seed).shuffle(ids)
    P = max(max(held), 1)
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-1] * (P - h))
        at += h
    return _i32(table, dev), held, pool, ids[at:]


def _pages(g, dev, dtype, pool, Hkv, page, D):
    return (_randn(g, dev, dtype, pool, Hkv, page, D), _randn(g, dev, dtype, pool, Hkv, page, D))


def _tree_masks(case, new, seed, dev):
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
    op, page = case["op"], case["page"]
    st = dict(case=case)
    if op == "pages":
        # a pool that holds every sequence's pages with its new tokens, and some more
        ctx, new = _lengths(case)
        P = max(1, max(_ceil(c + n, page) for c, n in zip(ctx, new)))
        pool = sum(_ceil(c + n, page) for c, n in zip(ctx, new)) + 11
        ids = list(range(pool))
        random.Random(seed).shuffle(ids)
        held = [_ceil(c, page) for c in ctx]
        table, at = [], 0
        for h in held:
            table.append(ids[at:at + h] + [-1] * (P - h))
            at += h
        free = ids[at:]
        st.update(q_start=_i32(_starts(new), dev), none=_i32([0] * (len(new) + 1), dev), kv_len=_i32(ctx, dev),
                  table=_i32(table, dev), n_pages=_i32(held, dev),
                  free=_i32(free + [-1] * (pool - len(free)), dev), n_free=_i32([len(free)], dev),
                  T=sum(new), pool=pool)
    elif op == "append":
        T, Hkv, D, dt = case["tokens"], case["Hkv"], case["D"], DTYPES[case["dtype"]]
        pool = _ceil(T, page) + 5
        if case["packed"]:  # views of a fused projection's output
            qkv = _randn(g, dev, dt, T, 3 * Hkv, D)
            k, v = qkv[:, Hkv:2 * Hkv], qkv[:, 2 * Hkv:]
        else:
            k, v = _randn(g, dev, dt, T, Hkv, D), _randn(g, dev, dt, T, Hkv, D)
        kp, vp = _pages(g, dev, dt, pool, Hkv, page, D)
        # consecutive positions of one sequence in shuffled pages; a few padding tokens have no slot
        order = torch.randperm(pool, generator=g, device=dev)
        t = torch.arange(T, device=dev)
        slots = order[t // page] * page + t % page
        slots[T - T // 16:] = -1
        st.update(k=k, v=v, kp=kp, vp=vp, slots=slots)
    elif op == "commit":
        ctx, paths = _commit_plan(case)
        Hkv, D, dt, N = case["Hkv"], case["D"], DTYPES[case["dtype"]], case["N"]
        table, _, pool, _ = _tables([c + N for c in ctx], page, seed, dev)
        kp, vp = _pages(g, dev, dt, pool, Hkv, page, D)
        st.update(table=table, kp=kp, vp=vp, kv_len=_i32(ctx, dev),
                  path=_i32([p + [-1] * (N - len(p)) for p in paths], dev),
                  acc=_i32([len(p) - 1 for p in paths], dev), most=max(len(p) for p in paths))
    else:
        ctx, new = _lengths(case)
        Hq, Hkv, D, dt = case["Hq"], case["Hkv"], case["D"], DTYPES[case["dtype"]]
        T = sum(new)
        table, _, pool, _ = _tables([c + n for c, n in zip(ctx, new)], page, seed, dev)
        kp, vp = _pages(g, dev, dt, pool, Hkv, page, D)
        st.update(q=_randn(g, dev, dt, T, Hq, D), kp=kp, vp=vp, table=table, q_start=_i32(_starts(new), dev),
                  kv_len=_i32(ctx, dev), max_q=max(new), anc=None, depth=None, slopes=None)
        if case["mask"] == "tree":
            st["anc"], st["depth"] = _tree_masks(case, new, seed, dev)
        if case["alibi"]:  # the geometric series of slopes
            st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)],
                                        dtype=torch.float32, device=dev)
    return st


# ---------------------------------------------------------------------- runs
def run(st):
    return {"pages": _run_pages, "append": _run_append, "commit": _run_commit,
            "attn": _run_attn}[st["case"]["op"]](st)


def _run_pages(st):
    """A step: the tables grow by the new tokens, and go back to the cached lengths behind it."""
    page = st["case"]["page"]
    if own:
        import speculative_decoding_tree_tv_gb300 as tv
        args = (st["kv_len"], st["table"], st["n_pages"], st["free"], st["n_free"], page)
        slots, status = tv.page_map(st["q_start"], *args, st["T"])
        grown = st["table"].clone()
        _, status2 = tv.page_map(st["none"], *args, 0)
    else:
        slots, status = _plain_page_map(st, st["q_start"], st["T"])
        grown = st["table"].clone()
        _, status2 = _plain_page_map(st, st["none"], 0)
    return dict(slots=slots, status=status, status2=status2, grown=grown, table=st["table"],
                n_pages=st["n_pages"], free=st["free"], n_free=st["n_free"])


def _plain_page_map(st, q_start, T):
    """Table entries past a sequence's pages, and free-list entries past n_free, keep their values."""
    page, kv_len, table, held = st["case"]["page"], st["kv_len"].long(), st["table"], st["n_pages"].long()
    free, n_free, dev = st["free"], st["n_free"].long(), st["table"].device
    P = table.shape[1]
    new = (q_start[1:] - q_start[:-1]).long()
    target = (kv_len + new + page - 1) // page
    need, back = (target - held).clamp_min(0), (held - target).clamp_min(0)
    # freed pages on top of the stack, in (sequence, page) order
    j = torch.arange(P, device=dev)
    old = table.clone()
    freed_at = n_free + back.cumsum(0)[:, None] - back[:, None] + (j - target[:, None])
    is_freed = (j >= target[:, None]) & (j < held[:, None])
    stack = torch.cat([free, torch.zeros(P * len(new) + 1, dtype=torch.int32, device=dev)])
    stack[torch.where(is_freed, freed_at, torch.full_like(freed_at, stack.numel() - 1))] = old
    size = n_free + back.sum()
    # the granted sequences take theirs from the top
    granted = (need.cumsum(0) <= size) | (need == 0)
    take = torch.where(granted, need, torch.zeros_like(need))
    taken_at = size - 1 - (take.cumsum(0) - take)[:, None] - (j - held[:, None])
    is_taken = (j >= held[:, None]) & (j < (held + take)[:, None])
    table.copy_(torch.where(is_taken, stack[taken_at.clamp(0, stack.numel() - 1)], old))
    left = size - take.sum()
    i = torch.arange(free.numel(), device=dev)
    free.copy_(torch.where((i >= n_free) & (i < left), stack[:free.numel()], free))
    st["n_free"].copy_(left)
    st["n_pages"].copy_(torch.where(granted, target, held))
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(q_start[1:].long(), t, right=True).clamp_max(len(new) - 1)
    pos = kv_len[b] + t - q_start[b]
    slots = table[b, (pos // page).clamp_max(P - 1)].long() * page + pos % page
    ok = granted[b] & (t < q_start[-1])
    return torch.where(ok, slots, torch.full_like(slots, -1)), torch.where(granted, 0, 8).to(torch.int32)


def _run_append(st):
    if own:
        import speculative_decoding_tree_tv_gb300 as tv
        tv.paged_append(st["k"], st["v"], st["slots"], st["kp"], st["vp"])
    else:
        page, slots = st["case"]["page"], st["slots"]
        keep = slots >= 0
        # a token without a slot writes what the last token with one writes
        last = torch.where(keep, torch.arange(len(slots), device=slots.device), 0).amax()
        t = torch.where(keep, torch.arange(len(slots), device=slots.device), last)
        s = slots[t]
        st["kp"][s // page, :, s % page] = st["k"][t]
        st["vp"][s // page, :, s % page] = st["v"][t]
    return dict(k=st["kp"], v=st["vp"])


def _run_commit(st):
    if own:
        import speculative_decoding_tree_tv_gb300 as tv
        new_len, status = tv.commit_paged(st["kp"], st["vp"], st["table"], st["kv_len"], st["path"], st["acc"])
    else:
        page, table, kv_len, acc = st["case"]["page"], st["table"].long(), st["kv_len"].long(), st["acc"].long()
        d = torch.arange(st["most"], device=table.device)
        path = st["path"][:, :st["most"]].long()
        path = torch.where(d <= acc[:, None], path, d)  # rows past the branch stay
        path = torch.where(d <= acc[:, None], path, torch.zeros_like(path))
        to = torch.where(d <= acc[:, None], d, torch.zeros_like(d))
        src, dst = kv_len[:, None] + path, kv_len[:, None] + to
        sp, dp = table.gather(1, src // page), table.gather(1, dst // page)
        st["kp"][dp, :, dst % page] = st["kp"][sp, :, src % page]
        st["vp"][dp, :, dst % page] = st["vp"][sp, :, src % page]
        new_len, status = st["kv_len"] + st["acc"] + 1, torch.zeros_like(st["acc"])
    return dict(k=st["kp"], v=st["vp"], new_len=new_len, status=status)


def _run_attn(st):
    case = st["case"]
    if own:
        import speculative_decoding_tree_tv_gb300 as tv
        out, lse, status = tv.attn_paged(st["q"], st["kp"], st["vp"], st["table"], st["q_start"], st["kv_len"],
                                         st["max_q"], anc_mask=st["anc"], softcap=case["cap"],
                                         window=case["window"], slopes=st["slopes"])
        return dict(out=out, lse=lse, status=status)
    q_start, kv_len, dev = st["q_start"].long(), st["kv_len"].long(), st["q"].device
    T, Hq, D = st["q"].shape
    Hkv, B, n = case["Hkv"], len(kv_len), st["max_q"]
    G = Hq // Hkv
    # [B, n] padded chunks, [B, Hkv, L, D] gathered caches
    i = torch.arange(n, device=dev)
    tok = (q_start[:-1, None] + i).clamp_max(T - 1)
    q = st["q"][tok].float().view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    table = st["table"].long().clamp_min(0)
    k = st["kp"][table].permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D).float()
    v = st["vp"][table].permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D).float()
    L = k.shape[2]
    s = torch.matmul(q, k.transpose(2, 3)).mul_(1.0 / math.sqrt(D)).view(B, Hkv, G, n, L)
    if case["cap"]:
        s = s.div_(case["cap"]).tanh_().mul_(case["cap"])
    # positions and visibility [B, n, L]
    j = torch.arange(L, device=dev)
    a = j - kv_len[:, None]  # the chunk's own slots
    inside = (a >= 0) & (a < (q_start[1:] - q_start[:-1])[:, None])
    if st["anc"] is None:
        pos_q = kv_len[:, None] + i
        pos_k = j.expand(B, L)
        seen = j <= pos_q[:, :, None]
    else:
        pos_q = kv_len[:, None] + st["depth"][tok]
        aa = a.clamp(0, n - 1)
        pos_k = torch.where(inside, kv_len[:, None] + st["depth"][(q_start[:-1, None] + aa).clamp_max(T - 1)], j)
        words = st["anc"][tok].gather(2, (aa // 64)[:, None, :].expand(B, n, L))
        seen = (a < 0)[:, None, :] | (inside[:, None, :] & ((words >> (aa % 64)[:, None, :]) & 1).bool())
    dist = pos_q[:, :, None] - pos_k[:, None, :]
    if case["window"]:
        seen = seen & (dist < case["window"])
    if st["slopes"] is not None:
        s = s - st["slopes"].view(1, Hkv, G, 1, 1) * dist[:, None, None].float()
    s = s.masked_fill_(~seen[:, None, None], float("-inf"))
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    s = s.sub_(top).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(B, Hkv, G * n, L), v).view(B, Hkv, G, n, D) / total
    o = torch.where(total == 0, torch.zeros_like(o), o)
    lse = (top + total.log())[..., 0]
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(q_start[1:], t, right=True)
    r = t - q_start[b]
    return dict(out=o[b, :, :, r].reshape(T, Hq, D).to(st["q"].dtype), lse=lse[b, :, :, r].reshape(T, Hq),
                status=torch.zeros(B, dtype=torch.int32, device=dev))


# --------------------------------------------------------------------- exact
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "pages":
        return None  # whole numbers and nothing else
    if case["op"] == "append":
        kp, vp, page = st["kp"].double(), st["vp"].double(), case["page"]
        for t, s in enumerate(st["slots"].tolist()):
            if s >= 0:
                kp[s // page, :, s % page] = st["k"][t].double()
                vp[s // page, :, s % page] = st["v"][t].double()
        return dict(k=kp, v=vp)
    if case["op"] == "commit":
        page, table = case["page"], st["table"].tolist()
        ctx, paths = _commit_plan(case)
        out = []
        for pages in (st["kp"].double(), st["vp"].double()):
            for b, path in enumerate(paths):
                rows = [pages[table[b][(ctx[b] + p) // page], :, (ctx[b] + p) % page].clone() for p in path]
                for d, r in enumerate(rows):
                    pages[table[b][(ctx[b] + d) // page], :, (ctx[b] + d) % page] = r
            out.append(pages)
        return dict(k=out[0], v=out[1], new_len=None, status=None)
    return _exact_attn(case, st)


def _exact_attn(case, st):
    """Sequence by sequence and head by head, over the rows the block table names."""
    ctx, new = _lengths(case)
    Hq, Hkv, D, page, dev = case["Hq"], case["Hkv"], case["D"], case["page"], st["q"].device
    out = torch.zeros(sum(new), Hq, D, dtype=torch.float64, device=dev)
    lse = torch.full((sum(new), Hq), -math.inf, dtype=torch.float64, device=dev)
    start = 0
    for b, (L, n) in enumerate(zip(ctx, new)):
        slot = torch.arange(L + n, device=dev)
        ids = st["table"][b][slot // page].long()
        qpos = torch.arange(L, L + n, device=dev)
        kpos = slot.clone()
        if case["mask"] == "tree":
            bits = st["anc"][start:start + n]
            own_slots = torch.arange(n, device=dev)
            sees = (bits[:, own_slots >> 6] >> (own_slots & 63)) & 1
            up = sees.sum(1) - 1  # ancestors of each node: its depth
            qpos = L + up
            kpos[L:] = L + up
            visible = torch.cat([torch.ones(n, L, dtype=torch.bool, device=dev), sees == 1], 1)
        else:
            visible = slot[None] <= qpos[:, None]
        away = (qpos[:, None] - kpos[None]).double()
        if case["window"] > 0:
            visible &= away < case["window"]
        for h in range(Hq):
            kh = h // (Hq // Hkv)
            keys = st["kp"][ids, kh, slot % page].double()
            vals = st["vp"][ids, kh, slot % page].double()
            x = st["q"][start:start + n, h].double() @ keys.T / math.sqrt(D)
            if case["cap"] > 0:
                x = case["cap"] * torch.tanh(x / case["cap"])
            if case["alibi"]:
                x = x - float(st["slopes"][h]) * away
            x = torch.where(visible, x, torch.full_like(x, -math.inf))
            z = torch.logsumexp(x, 1)
            lse[start:start + n, h] = z
            p = torch.exp(x - z[:, None])
            out[start:start + n, h] = torch.where(torch.isfinite(z)[:, None], p @ vals, torch.zeros_like(vals[:1]))
        start += n
    return dict(out=out, lse=lse, status=None)


# ---------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "pages":
        ctx, new = _lengths(case)
        B, T, page = case["B"], sum(new), case["page"]
        moved = sum(_ceil(c + n, page) - _ceil(c, page) for c, n in zip(ctx, new))
        # lengths, starts and held pages in, held pages out; every moved page read and written, both ways
        return dict(bytes=2 * (4 * (4 * B + 2) + 4 * B) + 16 * moved + 8 * T, flops=0)
    if op == "append":
        rows = case["tokens"] - case["tokens"] // 16
        return dict(bytes=8 * case["tokens"] + 2 * 2 * rows * case["Hkv"] * case["D"] * 2, flops=0)
    if op == "commit":
        ctx, paths = _commit_plan(case)
        rows = sum(sum(p != d for d, p in enumerate(path)) for path in paths)
        return dict(bytes=2 * 2 * rows * case["Hkv"] * case["D"] * 2 + 4 * sum(map(len, paths)) + 16 * case["B"], flops=0)
    ctx, new = _lengths(case)
    D, win = case["D"], case["window"] or 1 << 40
    tree = case["mask"] == "tree"
    keys = sum(c + n - max(0, c - win + 1) for c, n in zip(ctx, new) if n)
    # a tree node sees the prefix, and about log-many ancestors: counted as the prefix and itself
    pairs = sum(sum(min(win, c + (1 if tree else i + 1)) for i in range(n)) for c, n in zip(ctx, new))
    T = sum(new)
    return dict(bytes=2 * 2 * keys * case["Hkv"] * D + 2 * 2 * T * case["Hq"] * D + 4 * T * case["Hq"]
                + 4 * _ceil(keys, case["page"]), flops=4 * D * case["Hq"] * pairs)
