"""Plain forms of the 8-bit paged cache (64-bit floats and whole numbers), and its tests' inputs."""
import numpy as np
import torch

from _paged_util import make

FORMATS = {"e4m3": (torch.float8_e4m3fn, 448.0), "int8": (torch.int8, 127.0)}
NAN_SCALE = 255


def quantise_ref(x, fmt):
    """(codes as 64-bit values [.., D], scale bytes [..]) of rows x [.., D], from the definition."""
    x = x.double().cpu().numpy()
    most = FORMATS[fmt][1]
    top = np.abs(x).max(-1)
    fine = np.isfinite(top)
    m, e = np.frexp(np.where(fine, top, 1.0) / most)  # (a quotient that is no power of two is 2^-11 from one)
    e = np.maximum(np.where(top == 0, -126, np.where(m == 0.5, e - 1, e)), -126)
    y = np.ldexp(np.where(fine[..., None], x, 0.0), -e[..., None])
    if fmt == "int8":
        codes = np.rint(y)
    else:
        b = np.maximum(np.frexp(y)[1] - 1, -6)  # the code's binade; below 2^-6 steps stay 2^-9
        codes = np.ldexp(np.rint(np.ldexp(y, 3 - b)), b - 3)
    return torch.from_numpy(codes + 0.0), torch.from_numpy(np.where(fine, e + 127, NAN_SCALE))


def values_ref(codes, scale):
    """64-bit values of codes (any type) [.., D] and scale bytes [..]."""
    c, s = codes.cpu().to(torch.float32).double().numpy(), scale.cpu().long().numpy()
    v = np.ldexp(c, s[..., None] - 127)
    return torch.from_numpy(np.where((s == NAN_SCALE)[..., None], np.nan, v))


def cache(fmt, pool, Hkv, page, D, layout="heads", seed=1, device="cuda:0"):
    """k, v codes and scales of a cache whose every byte is set (codes of e4m3 NaN and of -128 among them)."""
    g = torch.Generator().manual_seed(seed)
    raw = torch.randint(0, 256, (2, pool, Hkv, page, D), generator=g, dtype=torch.uint8).to(device)
    if layout == "heads":
        k, v = raw[0], raw[1]
    elif layout == "rows":
        raw = raw.view(2, pool, page, Hkv, D)
        k, v = raw[0].transpose(1, 2), raw[1].transpose(1, 2)
    else:
        raw = raw.view(pool, 2, Hkv, page, D)
        k, v = raw[:, 0], raw[:, 1]
    s = torch.randint(0, 256, (2, pool, Hkv, page), generator=g, dtype=torch.uint8).to(device)
    t = FORMATS[fmt][0]
    return k.view(t), v.view(t), s[0], s[1]


def raw(x):
    return x.contiguous().view(torch.uint8)


def make_q8(seed, lens, Hq, Hkv, D, page, fmt, dtype="bf16", layout="heads", spread=2.0, **kw):
    """_paged_util.make's case over an 8-bit cache: `rows` hold the quantised values (64 bits), and c["q8"] the four
    cache tensors.  Rows differ in size by powers of two; what no token sees is any byte."""
    c = make(seed, lens, Hq, Hkv, D, page, dtype, **kw)
    pool = c["k"].shape[0]
    g = torch.Generator().manual_seed(seed + 1)
    sides = [t.cpu() for t in cache(fmt, pool, Hkv, page, D, layout, seed, "cpu")]
    table = c["table"].cpu().tolist()
    rows = []
    for b, both in enumerate(c["rows"]):
        new = []
        for side, x in enumerate(both):
            n = x.shape[0]
            size = torch.exp2(torch.randn(n, Hkv, 1, generator=g) * spread)
            codes, scale = quantise_ref((x.float() * size).to(x.dtype), fmt)
            for p in range(-(-n // page)):
                m = min(page, n - p * page)
                at = table[b][p]
                raw8 = codes[p * page:p * page + m].float().to(FORMATS[fmt][0]).view(torch.uint8)
                sides[side].view(torch.uint8)[at, :, :m] = raw8.transpose(0, 1)
                sides[2 + side][at, :, :m] = scale[p * page:p * page + m].to(torch.uint8).T
            new.append(values_ref(codes, scale))
        rows.append(tuple(new))
    dev = c["q"].device
    c["rows"] = rows
    moved = []
    for t in sides[:2]:
        perm = {"heads": t, "rows": t.transpose(1, 2), "both": t}[layout].contiguous().to(dev)
        moved.append(perm.transpose(1, 2) if layout == "rows" else perm)
    if layout == "both":  # K and V interleaved page by page
        both = torch.stack([raw(m) for m in moved], 1)
        moved = [both[:, 0].view(FORMATS[fmt][0]), both[:, 1].view(FORMATS[fmt][0])]
    c["q8"] = (moved[0], moved[1], sides[2].to(dev), sides[3].to(dev))
    c["fmt"] = fmt
    return c


def check_attn_q8(got_out, got_lse, ref, case, dtype, Hkv, scale=0.0, what=""):
    """Outputs against 64 bits (ref: attn_ref's).  Beside what attn_ref bounds:
    q, scaled by a power of two to [1, 2) at its largest, is rounded to fp16 below 2^-14 of that (2^-25 of the
    row's largest at most, times sum |k| in a score; elsewhere it is exact); a probability times its V row's scale is rounded
    to fp16 (2^-11 of it) or, far below the largest V scale, to a multiple of 2^-30 of it, 2^-31 off: a row's
    largest value is above half of what its scale can hold, the kept scale at most twice the largest and a row's
    sum at least 1, so that is below 2^-29 of the largest |v| a row; and the output is rounded once.  Larger units
    hold a tile's K over the power of two of its largest row, so an element is off by 2^-25 of that, which is below 2^-30
    of the largest |k| (127 codes are the fewest that reach half of a scale), and V likewise, in the bound above."""
    out, lse, spread, xerr, _ = ref
    D = case["q"].shape[2]
    u = torch.finfo(got_out.dtype).eps / 2
    scale = scale or D**-0.5
    qerr, far, at = [], [], 0
    for b, (L, n) in enumerate(case["lens"]):
        if n == 0:
            continue
        kr, vr = case["rows"][b]
        q = case["q"][at:at + n].cpu().double()
        ksum = kr.abs().nan_to_num(0.0).sum(2).amax(0).repeat_interleave(q.shape[1] // Hkv)
        kmax = kr.abs().nan_to_num(0.0).amax((0, 2)).repeat_interleave(q.shape[1] // Hkv)
        qerr.append(scale * (2.0**-25 * q.abs().nan_to_num(0.0).amax(2) * ksum
                             + 2.0**-30 * q.abs().nan_to_num(0.0).sum(2) * kmax))
        vmax = vr.abs().nan_to_num(0.0).amax((0, 2)).repeat_interleave(q.shape[1] // Hkv)
        far.append((2.0**-29 * (L + n) * vmax).expand(n, -1))
        at += n
    xerr = xerr + torch.cat(qerr)
    got = got_out.cpu().double()
    tol = (spread * (2.0**-11 + 2 * xerr[..., None] + 2.0**-19) + torch.cat(far)[..., None]
           + u * (out.abs() + 2.0**-11 * spread) + 1e-30)
    if got_out.dtype == torch.float16:
        tol = tol + 2.0**-25
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    worst = ((got - out).abs() / tol).max().item() if got.numel() else 0.0
    assert worst <= 1.0, f"{what}: output {worst:.3g} of its tolerance"
    if got_lse is not None:
        g = got_lse.cpu().double()
        fin = torch.isfinite(lse)
        assert torch.equal(fin, torch.isfinite(g)), f"{what}: lse finiteness"
        assert bool((g[~fin] == -float("inf")).all()), f"{what}: lse of an empty row"
        ltol = 2 * xerr + 2.0**-21 + 2.0**-21 * torch.where(fin, lse.abs(), torch.zeros_like(lse))
        bad = ((g - lse).abs() / ltol)[fin]
        assert bad.numel() == 0 or bad.max().item() <= 1.0, f"{what}: lse {bad.max().item():.3g}"
    return worst


def set_rows(c, b, j, k=None, v=None):
    """Rows j, j + 1, .. of sequence b of a make_q8 case become the quantised rows of k, v [n, Hkv, D]."""
    table, page = c["table"].cpu().tolist(), c["page"]
    for side, x in enumerate((k, v)):
        if x is None:
            continue
        codes, scale = quantise_ref(x, c["fmt"])
        raw8 = codes.float().to(FORMATS[c["fmt"]][0]).view(torch.uint8)
        pos = np.arange(j, j + len(x))
        at, row = torch.tensor(np.array(table[b])[pos // page]), torch.from_numpy(pos % page)
        c["q8"][side].view(torch.uint8)[at, :, row] = raw8.to(c["q"].device)
        c["q8"][2 + side][at, :, row] = scale.to(torch.uint8).to(c["q"].device)
        c["rows"][b][side][j:j + len(x)] = values_ref(codes, scale)


def visible(c, b, at, window=0, hidden=None):
    """Which rows [n, L + n] the tokens of sequence b (the first is token `at`) see, and how far they are."""
    L, n = c["lens"][b]
    slot = torch.arange(L + n)
    if c["anc"] is None:
        qpos, kpos = torch.arange(L, L + n), slot.clone()
        see = slot[None] <= qpos[:, None]
    else:
        see = torch.ones(n, L + n, dtype=torch.bool)
        see[:, L:] = False
        for i in range(n):
            j = i
            while j >= 0:
                see[i, L + j] = True
                j = c["parents"][b][j]
        dep = torch.tensor(c["depth"][at:at + n])
        qpos, kpos = L + dep, slot.clone()
        kpos[L:] = L + dep
    if window:
        see &= qpos[:, None] - kpos[None] < window
    for j in (hidden or {}).get(b, ()):
        see[:, j] = False
    return see, qpos[:, None] - kpos[None]


def check_seen(got_out, got_lse, c, Hkv, window=0, softcap=0.0, slopes=None, scale=0.0, hidden=None, what=""):
    """Outputs against 64 bits, held to what each token sees: rows that it does not see have no say in its bound,
    whatever their size.  As check_attn_q8 has it, with keys exact (a key is held over no other's size), and
    p_j 2^t_j, a probability (its row's largest is 1) times its V row's power of two, is rounded to fp16 times 2^6, so
    far below what it is held over to a multiple of 2^-30 of that, 2^-31 off.  V rows within 2^9 of one another are held over
    the largest's power of two, so over 2^9 of that of the row whose probability is 1, at most; others over the largest
    p_j 2^t_j, rounded up.  A row's largest value is above half of what its scale can hold: 2^-21 of the largest p_j |v_j|
    for each visible row."""
    Hq, D = c["q"].shape[1:]
    scale = scale or D**-0.5
    u = torch.finfo(got_out.dtype).eps / 2
    heads = torch.arange(Hq) // (Hq // Hkv)
    at, worst = 0, 0.0
    for b, (L, n) in enumerate(c["lens"]):
        if n == 0:
            continue
        see, dist = visible(c, b, at, window, hidden)
        kh, vh = (r.double()[:, heads].transpose(0, 1) for r in c["rows"][b])
        q = c["q"][at:at + n].cpu().double().transpose(0, 1)
        x = scale * q @ kh.transpose(1, 2)
        mag = (see * (scale * q.abs() @ kh.abs().transpose(1, 2))).amax(2)
        if softcap:
            x = softcap * torch.tanh(x / softcap)
        if slopes is not None:
            x = x - slopes.double().cpu()[:, None, None] * dist.double()
        x = torch.where(see, x, torch.full_like(x, -float("inf")))
        lse = torch.logsumexp(x, 2)
        p = torch.exp(x - torch.where(torch.isfinite(lse), lse, torch.zeros_like(lse))[..., None])
        out, spread = p @ vh, p @ vh.abs()
        top = torch.where(see, x.abs(), torch.zeros_like(x)).amax(2)
        xerr = (2.0**-23 * ((D + 4) * mag + 4 * torch.minimum(top, 2 * mag + 40) + 8 * softcap)
                + scale * 2.0**-25 * q.abs().amax(2) * (see * kh.abs().sum(2)[:, None]).amax(2))
        if slopes is not None:  # (a key's bias is counted on from its tile's first key, up to 127 on: three roundings of that)
            xerr = xerr + 3 * 2.0**-24 * 128 * slopes.double().cpu()[:, None]
        vmax = vh.abs().amax(2)[:, None]
        far = see.sum(1) * 2.0**-21 * (p * vmax).amax(2)
        tol = (spread * (2.0**-11 + 2 * xerr[..., None] + 2.0**-19) + far[..., None]
               + u * (out.abs() + 2.0**-11 * spread) + 1e-30)
        if got_out.dtype == torch.float16:
            tol = tol + 2.0**-25
        got = got_out[at:at + n].cpu().double().transpose(0, 1)
        assert torch.isfinite(got).all(), f"{what}: non-finite output"
        worst = max(worst, ((got - out).abs() / tol).max().item())
        assert worst <= 1.0, f"{what}: output {worst:.3g} of its tolerance"
        fin = torch.isfinite(lse)
        g = got_lse[at:at + n].cpu().double().T
        assert torch.equal(fin, torch.isfinite(g)), f"{what}: lse finiteness"
        ltol = 2 * xerr + 2.0**-21 + 2.0**-21 * torch.where(fin, lse.abs(), torch.zeros_like(lse))
        bad = ((g - lse).abs() / ltol)[fin]
        assert bad.numel() == 0 or bad.max().item() <= 1.0, f"{what}: lse {bad.max().item():.3g}"
        at += n
    return worst
