"""Problems of groups of requests that share their first tokens, and their plain 64-bit
attention, request by request as if nothing were shared, with the bounds of the kernels'
distance from it."""
import math

import torch


def problem(seed, groups, Hkv, G, D, P, fp8, sinks=False, lead=0, tail=0, wide=0, spread=3):
    """groups: (shared tokens, lengths of its requests, 0 for an idle one).  Full shared pages
    are one and the same, a partly shared one is a copy in each row.  Slots that no request
    sees hold NaN, and so do scales of unused pages; unused entries are -1.  lead and tail:
    padding rows around the groups'."""
    g = torch.Generator().manual_seed(seed)
    lens, cu, shared, rows, pool = [7] * lead, [lead], [], [[]] * lead, 0
    copies, copied = [], set()
    for S, Ls in groups:
        full = min(S, max(Ls, default=0)) // P
        head = list(range(pool, pool + full))
        pool += full
        first = None
        for L in Ls:
            n = max(0, -(-L // P) - full) if L else 0
            mine = list(range(pool, pool + n))
            pool += n
            rows.append((head + mine)[:-(-L // P)])
            if L and S % P and L > full * P:
                part = min(S, L) - full * P
                if first is None or first[2] < part:
                    first = (rows[-1][full], len(rows), part)
                copies.append((first, rows[-1][full], part))
            lens.append(L)
        cu.append(len(lens))
        shared.append(S)
    lens += [9] * tail
    rows += [[]] * tail
    order = torch.randperm(pool + 4, generator=g)
    table = torch.full((len(lens), max(1, max(map(len, rows))) + wide), -1, dtype=torch.int32)
    for b, r in enumerate(rows):
        table[b, :len(r)] = order[torch.tensor(r, dtype=torch.int64)].int() if r else table[b, :0]
    x = torch.randn(pool + 4, Hkv, P, 2 * D, generator=g)
    seen = torch.zeros(pool + 4, P, dtype=torch.bool)
    for b, r in enumerate(rows):
        for j, page in enumerate(r):
            seen[order[page], :min(P, lens[b] - j * P)] = True
    for first, page, part in copies:  # the longest of a group's copies came first, or replaced it
        x[order[page], :, :part] = x[order[first[0]], :, :part]
    scale = None
    if fp8:
        size = torch.exp2(torch.randint(-spread, spread + 1, (pool + 4, Hkv, 2), generator=g).float())
        for first, page, part in copies:
            size[order[page]] = size[order[first[0]]]
        codes = (x * 60).to(torch.float8_e4m3fn)
        kv = torch.where(seen[:, None, :, None], codes.view(torch.uint8),
                         torch.tensor(0x7f, dtype=torch.uint8)).view(torch.float8_e4m3fn)
        scale = torch.where(seen.any(1)[:, None, None], size / 60, torch.tensor(math.nan))
    else:
        kv = torch.where(seen[:, None, :, None], x, torch.tensor(math.nan)).bfloat16()
    return dict(q=torch.randn(len(lens), Hkv * G, D, generator=g).bfloat16(), kv=kv, sc=scale, bt=table,
                sl=torch.tensor(lens, dtype=torch.int32), cu=torch.tensor(cu, dtype=torch.int32),
                shared=torch.tensor(shared, dtype=torch.int32),
                sinks=torch.randn(Hkv * G, generator=g) * 2 if sinks else None,
                scale=1 / math.sqrt(D), P=P, fp8=fp8, lead=lead, tail=tail)


def decode(pr, device="cpu"):
    """out, lse in double, and elementwise bounds: weights rounded once to bf16 (2^-8), N of
    them and D products added in 32 bits, the output rounded to bf16 (2^-8)."""
    q, kv, P = pr["q"].to(device).double(), pr["kv"].to(device), pr["P"]
    table = pr["bt"].to(device).long()
    sc = None if pr["sc"] is None else pr["sc"].to(device).double()
    B, Hq, D = q.shape
    Hkv = kv.shape[1]
    zero = torch.zeros((), dtype=torch.float64, device=device)
    out, tol = torch.zeros(2, B, Hq, D, dtype=torch.float64, device=device)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=device)
    lse_tol = torch.zeros(B, Hq, dtype=torch.float64, device=device)
    for b, N in enumerate(pr["sl"].tolist()):
        if N <= 0:
            continue
        pos = torch.arange(N, device=device)
        page = table[b][pos // P]
        ok = ((page >= 0) & (page < kv.shape[0]))[:, None, None]
        page = page.clamp(0, kv.shape[0] - 1)
        raw = kv.view(torch.uint8 if pr["fp8"] else torch.bfloat16)
        row = raw[page, :, pos % P].view(kv.dtype).double()  # [N, Hkv, 2D]
        k, v = row[..., :D], row[..., D:]
        if sc is not None:
            k, v = k * sc[page][..., :1], v * sc[page][..., 1:]
        k, v = torch.where(ok, k, zero).transpose(0, 1), torch.where(ok, v, zero).transpose(0, 1)
        qb = q[b].view(Hkv, -1, D)
        x = pr["scale"] * (qb @ k.mT)  # [Hkv, G, N]
        dx = (D + 4) * 2.0 ** -24 * abs(pr["scale"]) * (qb.abs() @ k.abs().mT).amax(-1) \
            + 2.0 ** -22 * (1 + x.abs().amax(-1))
        total = torch.logsumexp(x, -1)
        lse[b] = total.view(Hq)
        lse_tol[b] = (dx + N * 2.0 ** -24 + 2.0 ** -22 * (1 + total.abs())).view(Hq)
        if pr["sinks"] is not None:
            total = torch.logaddexp(total, pr["sinks"].to(device).double().view(Hkv, -1))
        w = torch.exp(x - total[..., None])
        o = w @ v
        sums = (2.0 ** -8 + 2 * dx + (N + 16) * 2.0 ** -24)[..., None]
        out[b] = o.view(Hq, D)
        tol[b] = (2.0 ** -8 * o.abs() + sums * (w @ v.abs())).view(Hq, D)
    return out, lse, tol, lse_tol
