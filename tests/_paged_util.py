"""Plain implementations of the paged-cache operators (python integers and 64-bit
floats) and inputs for their tests."""
import math
import random

import torch

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ page map
def page_map_ref(q_start, kv_len, table, n_pages, free_list, n_free, page, T):
    """tv_page_map on python lists; `table`, `n_pages` and `free_list` are changed
    in place.  Returns (slots, status, n_free)."""
    B, P, pool = len(kv_len), len(table[0]) if table else 0, len(free_list)
    status = [0] * B
    target = [0] * B
    for b in range(B):
        t0, t1 = q_start[b], q_start[b + 1]
        target[b] = -(-(kv_len[b] + t1 - t0) // page)
        if not (0 <= t0 <= t1 <= T) or kv_len[b] < 0 or not 0 <= n_pages[b] <= P or target[b] > P:
            status[b] = 1
    back = sum(max(0, n_pages[b] - target[b]) for b in range(B) if not status[b])
    if not 0 <= n_free <= pool or n_free + back > pool:
        return [-1] * T, [1] * B, n_free
    stack = list(free_list[:n_free])
    for b in range(B):
        if not status[b] and n_pages[b] > target[b]:
            stack += table[b][target[b]:n_pages[b]]
            n_pages[b] = target[b]
    size, asked = len(stack), 0
    for b in range(B):
        if not status[b] and target[b] > n_pages[b]:
            asked += target[b] - n_pages[b]
            if asked > size:
                status[b] = 8
                continue
            while n_pages[b] < target[b]:
                table[b][n_pages[b]] = stack.pop()
                n_pages[b] += 1
    for i in range(n_free, len(stack)):
        free_list[i] = stack[i]
    slots = [-1] * T
    for b in range(B):
        for t in range(max(q_start[b], 0), min(q_start[b + 1], T)):
            if not status[b]:
                pos = kv_len[b] + t - q_start[b]
                slots[t] = table[b][pos // page] * page + pos % page
    return slots, status, len(stack)


# ----------------------------------------------------------------- attention
def random_tree(rng, n):
    """parent[] of a random topological tree."""
    return [-1] + [rng.randrange(max(0, i - 5), i) for i in range(1, n)]


def tree_masks(parents, W):
    """Masks [T][W] as signed 64-bit words, and depths, of one tree per sequence."""
    rows, depth = [], []
    for parent in parents:
        anc, dep = [], []
        for i, p in enumerate(parent):
            anc.append((1 << i) | (anc[p] if i else 0))
            dep.append(dep[p] + 1 if i else 0)
        depth += dep
        for a in anc:
            words = [(a >> (64 * w)) & (2**64 - 1) for w in range(W)]
            rows.append([w - 2**64 if w >= 2**63 else w for w in words])
    return rows, depth


def make(seed, lens, Hq, Hkv, D, page, dtype="bf16", tree=False, layout="heads", pad=0, device="cuda:0",
         spare=3, q_mag=1.0):
    """Inputs of tv.attn_paged for sequences of `lens` = [(cached, new), ...].
    Cache rows past a sequence's tokens and the pool's spare pages hold NaN."""
    rng = random.Random(seed)
    g = torch.Generator().manual_seed(seed)
    dt = DTYPES[dtype]
    held = [-(-(L + n) // page) for L, n in lens]
    pool = sum(held) + spare
    ids = list(range(pool))
    rng.shuffle(ids)
    P = max(held + [1]) + 1
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-1] * (P - h))
        at += h
    T = sum(n for _, n in lens)
    if layout == "heads":       # [pages, Hkv, page, D]
        kv = torch.full((2, pool, Hkv, page, D), float("nan"), dtype=dt)
        k, v = kv[0], kv[1]
    elif layout == "rows":      # [pages, page, Hkv, D]
        kv = torch.full((2, pool, page, Hkv, D), float("nan"), dtype=dt)
        k, v = kv[0].transpose(1, 2), kv[1].transpose(1, 2)
    else:                       # K and V interleaved page by page
        kv = torch.full((pool, 2, Hkv, page, D), float("nan"), dtype=dt)
        k, v = kv[:, 0], kv[:, 1]
    rows = []
    for b, (L, n) in enumerate(lens):
        kr = torch.randn(L + n, Hkv, D, generator=g).to(dt)
        vr = torch.randn(L + n, Hkv, D, generator=g).to(dt)
        rows.append((kr, vr))
        for j in range(held[b]):
            m = min(page, L + n - j * page)
            k[table[b][j], :, :m] = kr[j * page:j * page + m].transpose(0, 1)
            v[table[b][j], :, :m] = vr[j * page:j * page + m].transpose(0, 1)
    wide = (torch.randn(T + pad, Hq + 2 * Hkv, D, generator=g) * q_mag).to(dt)  # a fused projection
    starts = [0]
    for _, n in lens:
        starts.append(starts[-1] + n)
    kv = kv.to(device)
    if layout == "heads":
        k, v = kv[0], kv[1]
    elif layout == "rows":
        k, v = kv[0].transpose(1, 2), kv[1].transpose(1, 2)
    else:
        k, v = kv[:, 0], kv[:, 1]
    wide = wide.to(device)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=device)  # noqa: E731
    max_q = max([n for _, n in lens] + [1])
    case = dict(lens=lens, rows=rows, q=wide[:, :Hq], k=k, v=v, table=i32(table), q_start=i32(starts),
                kv_len=i32([L for L, _ in lens]), max_q=max_q, anc=None, depth=None, T=T, page=page)
    if tree:
        W = (max_q + 63) // 64
        case["parents"] = [random_tree(rng, n) if n else [] for _, n in lens]
        words, case["depth"] = tree_masks(case["parents"], W)
        case["words"] = words
        words = words + [[-1] * W] * pad
        case["anc"] = torch.tensor(words, dtype=torch.int64, device=device).reshape(T + pad, W)
    return case


def attn_ref(case, Hq, Hkv, D, softcap=0.0, window=0, slopes=None, scale=0.0, hidden=None):
    """(out, lse, spread, xerr, vsum) in 64 bits: spread = sum_j p_j |v_j|, xerr = a bound
    on the absolute error of a score taken in 32 bits, vsum = sum_j |v_j| over the visible
    rows.  `hidden` = {b: set of positions} treated as not visible."""
    scale = scale or 1.0 / math.sqrt(D)
    G = Hq // Hkv
    outs, lses, spreads, xerrs, vsums = [], [], [], [], []
    at = 0
    for b, (L, n) in enumerate(case["lens"]):
        if n == 0:
            continue
        kr, vr = (r.double() for r in case["rows"][b])
        q = case["q"][at:at + n].cpu().double()
        slot = torch.arange(L + n)
        see = torch.ones(n, L + n, dtype=torch.bool)
        if case["anc"] is None:
            qpos, kpos = torch.arange(L, L + n), slot.clone()
            see = slot[None] <= qpos[:, None]
        else:
            par = case["parents"][b]
            dep = torch.tensor(case["depth"][at:at + n])
            see[:, L:] = False
            for i in range(n):
                j = i
                while j >= 0:
                    see[i, L + j] = True
                    j = par[j]
            qpos, kpos = L + dep, slot.clone()
            kpos[L:] = L + dep
        dist = qpos[:, None] - kpos[None]
        if window:
            see &= dist < window
        if hidden and b in hidden:
            for j in hidden[b]:
                see[:, j] = False
        kh = kr[:, torch.arange(Hq) // G].transpose(0, 1)    # [Hq, L + n, D]
        vh = vr[:, torch.arange(Hq) // G].transpose(0, 1)
        qh = q.transpose(0, 1)
        x = scale * qh @ kh.transpose(1, 2)
        mag = (scale * qh.abs() @ kh.abs().transpose(1, 2)).amax(2)
        if softcap:
            x = softcap * torch.tanh(x / softcap)
        if slopes is not None:
            x = x - slopes.double().cpu()[:, None, None] * dist.double()
        x = torch.where(see, x, torch.full_like(x, -math.inf))
        lse = torch.logsumexp(x, 2)
        p = torch.exp(x - torch.where(torch.isfinite(lse), lse, torch.zeros_like(lse))[..., None])
        outs.append((p @ vh).transpose(0, 1))
        spreads.append((p @ vh.abs()).transpose(0, 1))
        vsums.append((see.double() @ vh.abs()).transpose(0, 1))
        lses.append(lse.T)
        # a D-term dot product in 32 bits (mag bounds the sum of |terms|, each product
        # and sum rounded), then scale, cap and bias: a few roundings of what they hold.
        # The bias of the keys that matter is not above what the scores range over.
        top = torch.where(see, x.abs(), torch.zeros_like(x)).amax(2)
        near = torch.minimum(top, 2 * mag + 40)
        xerrs.append((2.0**-23 * ((D + 4) * mag + 4 * near + 8 * softcap)).T)
        at += n
    return tuple(torch.cat(z) for z in (outs, lses, spreads, xerrs, vsums))


def check_attn(got_out, got_lse, ref, dtype, what=""):
    """Outputs against 64 bits.  A probability is rounded to the cache's type once
    (eps / 2 of it: at most eps / 2 of spread in the output), carries the error of its
    score (xerr, and as much again in the normaliser, plus a few 2^-22 of the
    exponential and the sums: 2^-19), and the output is rounded once more.  Halves below
    2^-14 are rounded to a multiple of 2^-24: each probability (its row's largest is
    at least 1 before the division) by 2^-25, and the output."""
    out, lse, spread, xerr, vsum = ref
    u = torch.finfo(DTYPES[dtype]).eps / 2
    got = got_out.cpu().double()
    tol = spread * (u + 2 * xerr[..., None] + 2.0**-19) + u * (out.abs() + u * spread) + 1e-30
    if dtype == "fp16":
        tol = tol + 2.0**-25 * (vsum + 1)
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    worst = ((got - out).abs() / tol).max().item() if got.numel() else 0.0
    assert worst <= 1.0, f"{what}: output {worst:.3g} of its tolerance"
    if got_lse is not None:
        g = got_lse.cpu().double()
        fin = torch.isfinite(lse)
        assert torch.equal(fin, torch.isfinite(g)), f"{what}: lse finiteness"
        assert bool((g[~fin] == -math.inf).all()), f"{what}: lse of an empty row"
        ltol = 2 * xerr + 2.0**-21 + 2.0**-21 * torch.where(fin, lse.abs(), torch.zeros_like(lse))
        bad = ((g - lse).abs() / ltol)[fin]
        assert bad.numel() == 0 or bad.max().item() <= 1.0, f"{what}: lse {bad.max().item():.3g}"
    return worst
