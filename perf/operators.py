"""Cases and plain forms of the 8-bit paged cache and what works on it.

Four operators of a paged-attention server, each as a user calls it:

* ``append``  writes new tokens into an e4m3 cache that keeps one fp32 scale for each
  (page, kv head) of K and one of V;
* ``attn8``   one decode token per request over that cache, optionally with a sliding window
  and first tokens that stay visible, and sink logits in the denominator;
* ``window``  the same visibility (window and first tokens) over a bf16 cache;
* ``fork``, ``compact``, ``turnover``  the cache's pages: forking requests (shared full pages,
  a copied partial one), compacting the pool, releasing and reserving pages.

``run`` computes them with elementary torch operations while ``own`` is false, and through the
package's entry points while it is true.
"""
import math
import random

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
MIN_EXP = -100  # scales are powers of two, 2^-100 at least


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # four short requests on one kv head: the smallest decode call, all latency
        attn_case("attn8", B=4, Hq=8, Hkv=1, D=128, P=16, lengths="uniform", lo=1, hi=300,
                  window=0, first=0, sinks=False, pick=1, name="attn8_tiny"),
        # a served batch of mixed lengths with sink logits, full attention
        attn_case("attn8", B=64, Hq=64, Hkv=8, D=128, P=16, lengths="loguniform", lo=1, hi=32768,
                  window=0, first=0, sinks=True, pick=2, name="attn8_batch"),
        # a few requests of very long context on larger pages
        attn_case("attn8", B=8, Hq=64, Hkv=8, D=128, P=32, lengths="const", lo=131072, hi=131072,
                  window=0, first=0, sinks=False, pick=3, name="attn8_long"),
        # 16 query heads per kv head, 64-wide heads, a window of odd size with first tokens
        attn_case("attn8", B=33, Hq=64, Hkv=4, D=64, P=32, lengths="uniform", lo=1, hi=9000,
                  window=1001, first=5, sinks=True, pick=4, name="attn8_window"),
        # the window layer of a served batch: 128 tokens and the first 4
        attn_case("window", B=64, Hq=64, Hkv=8, D=128, P=16, lengths="loguniform", lo=1, hi=32768,
                  window=128, first=4, sinks=True, pick=2, name="window_layer"),
        # streaming generation far past a wide window, 4 query heads per kv head
        attn_case("window", B=32, Hq=32, Hkv=8, D=128, P=32, lengths="uniform", lo=2000, hi=60000,
                  window=4096, first=64, sinks=False, pick=5, name="window_stream"),
        # one decode step's tokens into the cache
        append_case(B=64, Hkv=8, D=128, P=16, lo=1, hi=1, before=4000, pick=6, name="append_step"),
        # a batch of prompts of ragged length, some continuing a page
        append_case(B=16, Hkv=8, D=128, P=16, lo=1, hi=2048, before=700, pick=7,
                    name="append_prompts"),
        # one request forked for four samples
        fork_case(parents=1, copies=4, Hkv=8, D=128, P=16, hi=1000, pages=512, pick=8,
                  name="fork_one"),
        # a batch forked for parallel sampling
        fork_case(parents=64, copies=4, Hkv=8, D=128, P=16, hi=4000, pages=16384, pick=9,
                  name="fork_batch"),
        # a fragmented pool, half of its pages live, moved together
        compact_case(rows=128, Hkv=8, D=128, P=16, pages=16384, hi=2000, pick=10,
                     name="compact_pool"),
        # between two steps: rejected tokens released, room for the next ones reserved
        turnover_case(rows=64, P=16, pages=16384, hi=3000, back=8, grow=9, pick=11,
                      name="turnover_step"),
    ]


def attn_case(op, **kw):
    return dict(op=op, **kw)


def append_case(**kw):
    return dict(op="append", **kw)


def fork_case(**kw):
    return dict(op="fork", **kw)


def compact_case(**kw):
    return dict(op="compact", **kw)


def turnover_case(**kw):
    return dict(op="turnover", **kw)


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn8", "attn8", "window", "window", "append", "append", "fork", "compact",
                     "turnover"])
    pick = rng.randrange(1 << 20)
    D = rng.choice([64, 128])
    P = rng.choice([16, 32])
    if op in ("attn8", "window"):
        Hkv = rng.choice([1, 2, 3, 4, 8])
        G = rng.choice([1, 2, 4, 5, 7, 8, 16])
        B = _log_int(rng, 1, 128)
        # no draw attends to more keys than the largest listed case of its cache type
        most = (1 << 20 if op == "attn8" else 1 << 17) * 8 // Hkv
        hi = max(1, min(_log_int(rng, 1, 131072), most // B))
        window = rng.choice([0, 0, _log_int(rng, 1, 5000)]) if op == "attn8" else _log_int(rng, 1, 5000)
        first = 0 if window == 0 else rng.choice([0, 1, 4, 17, 64])
        return attn_case(op, B=B, Hq=G * Hkv, Hkv=Hkv, D=D, P=P,
                         lengths=rng.choice(["uniform", "loguniform", "const"]),
                         lo=hi if rng.random() < 0.2 else max(1, hi // 50), hi=hi, window=window,
                         first=first, sinks=rng.random() < 0.5, pick=pick)
    if op == "append":
        B = _log_int(rng, 1, 128)
        hi = rng.choice([1, _log_int(rng, 2, max(3, 16384 // B))])
        return append_case(B=B, Hkv=rng.choice([1, 2, 4, 8]), D=D, P=P, lo=1, hi=hi,
                           before=_log_int(rng, 1, 2000), pick=pick)
    if op == "fork":
        parents = _log_int(rng, 1, 64)
        return fork_case(parents=parents, copies=rng.randint(1, 4), Hkv=rng.choice([1, 2, 8]), D=D,
                         P=P, hi=_log_int(rng, 20, 3000), pages=16384, pick=pick)
    if op == "compact":
        return compact_case(rows=rng.randint(8, 128), Hkv=rng.choice([1, 3, 8]), D=D, P=P,
                            pages=_log_int(rng, 2048, 16000), hi=_log_int(rng, 50, 2000), pick=pick)
    return turnover_case(rows=_log_int(rng, 1, 200), P=P, pages=_log_int(rng, 9000, 40000),
                         hi=_log_int(rng, 30, 600), back=rng.randint(0, 20),
                         grow=rng.randint(1, 40), pick=pick)


# ------------------------------------------------- sizes, fixed by the case --
def _lengths(c, n=None, lo=None, hi=None, kind=None, salt=0):
    r = random.Random(c["pick"] * 1009 + salt)
    lo, hi = c.get("lo", 1) if lo is None else lo, c["hi"] if hi is None else hi
    kind = kind or c.get("lengths", "uniform")
    n = n or c["B"]
    if kind == "const":
        return [hi] * n
    if kind == "loguniform":
        return [min(hi, max(lo, int(round(math.exp(r.uniform(0.0, math.log(hi))))))) for _ in range(n)]
    return [r.randint(lo, hi) for _ in range(n)]


def _cdiv(a, b):
    return -(-a // b)


def _visible(c, L):
    """Number of keys that the token of a request of length L sees."""
    if c["window"] <= 0:
        return L
    start = max(0, L - c["window"])
    return L - start + min(c["first"], start)


def _seen_pages(c, L):
    """Logical pages that hold a visible key."""
    P = c["P"]
    start = max(0, L - c["window"]) if c["window"] > 0 else 0
    head = range(0, _cdiv(min(c["first"], start), P))
    tail = range(max(start // P, len(head)), _cdiv(L, P))
    return [*head, *tail]


def _append_plan(c):
    """Per request: tokens already held, new tokens."""
    new = _lengths(c)
    old = _lengths(c, lo=0, hi=c["before"], kind="uniform", salt=1)
    return old, new


def work(c):
    if c["op"] in ("attn8", "window"):
        Ls = _lengths(c)
        esz = 1 if c["op"] == "attn8" else 2
        keys = sum(_visible(c, L) for L in Ls)
        pages = sum(len(_seen_pages(c, L)) for L in Ls)
        b = keys * c["Hkv"] * 2 * c["D"] * esz + pages * 4 + c["B"] * 4
        b += (pages * c["Hkv"] * 8) if esz == 1 else 0
        b += c["B"] * c["Hq"] * (2 * c["D"] * 2 + 4)
        return {"bytes": b, "flops": 4 * keys * c["Hq"] * c["D"]}
    if c["op"] == "append":
        old, new = _append_plan(c)
        T = sum(new)
        pages = sum(_cdiv(o + n, c["P"]) - o // c["P"] for o, n in zip(old, new))
        return {"bytes": T * c["Hkv"] * 2 * c["D"] * 3 + pages * (c["Hkv"] * 16 + 4),
                "flops": T * c["Hkv"] * 2 * c["D"] * 2}
    if c["op"] == "fork":
        Ls = _fork_lengths(c)
        n = c["copies"]
        copied = sum(n for L in Ls if L % c["P"])
        shared = sum(n * (L // c["P"]) for L in Ls)
        page = c["Hkv"] * (c["P"] * 2 * c["D"] + 8)
        return {"bytes": copied * 2 * page + shared * 16 + c["pages"] * 4, "flops": shared + copied}
    if c["op"] == "compact":
        live = [p for r in _compact_rows(c) for p in r]
        n = len(live)
        moves = sum(p >= n for p in live)
        page = c["Hkv"] * (c["P"] * 2 * c["D"] + 8)
        return {"bytes": moves * 2 * page + c["pages"] * 8 + n * 8, "flops": c["pages"]}
    keep, now, after = _turnover_lengths(c)
    gone = sum(_cdiv(n, c["P"]) - _cdiv(k, c["P"]) for k, n in zip(keep, now))
    come = sum(_cdiv(a, c["P"]) - _cdiv(k, c["P"]) for k, a in zip(keep, after))
    return {"bytes": c["pages"] * 4 + (gone + come) * 12 + len(now) * 24, "flops": c["pages"]}


def _fork_lengths(c):
    return _lengths(c, n=c["parents"], lo=1, kind="uniform")


def _compact_rows(c):
    """Each row's pages: a random half of the pool, at most, dealt to the rows."""
    r = random.Random(c["pick"] * 31 + 7)
    Ls = _lengths(c, n=c["rows"], lo=1, kind="uniform")
    order = r.sample(range(c["pages"]), c["pages"])
    rows, at = [], 0
    for L in Ls:
        n = _cdiv(L, c["P"])
        n = max(0, min(n, c["pages"] // 2 - at))
        rows.append(order[at:at + n])
        at += n
    return rows


def _turnover_lengths(c):
    now = _lengths(c, n=c["rows"], lo=1, kind="uniform")
    keep = [max(0, L - r) for L, r in zip(now, _lengths(c, n=c["rows"], lo=0, hi=c["back"],
                                                          kind="uniform", salt=3))]
    after = [k + g for k, g in zip(keep, _lengths(c, n=c["rows"], lo=0, hi=c["grow"],
                                                  kind="uniform", salt=4))]
    return keep, now, after


# ---------------------------------------------------------------- inputs --
def _pow2_scale(amax):
    """Smallest power of two s with amax <= 448 s (0 for 0), at least 2^-100."""
    f, e = torch.frexp(amax.float())
    e = torch.where(f <= 0.875, e - 9, e - 8).clamp(min=MIN_EXP)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(f), e), torch.zeros_like(f))


def _values(shape, g):
    """Keys and values as a model makes them: unit normal with a few wide channels and a
    magnitude that varies from page to page."""
    x = torch.randn(shape, device=DEV, generator=g)
    wide = 1 + 5 * (torch.rand(shape[-1], device=DEV, generator=g) < 0.03).float()
    size = torch.exp(0.5 * torch.randn(shape[0], shape[1], 1, 1, device=DEV, generator=g))
    return x.mul_(wide).mul_(size)


def _cache8(pages, Hkv, P, D, g):
    x = _values((pages, Hkv, P, 2 * D), g)
    s = _pow2_scale(x.view(pages, Hkv, P, 2, D).abs().amax(dim=(2, 4)))
    codes = (x.view(pages, Hkv, P, 2, D) / s[:, :, None, :, None]).to(torch.float8_e4m3fn)
    return codes.view(pages, Hkv, P, 2 * D), s.contiguous()


def _tables(rows, width, pool):
    t = torch.full((len(rows), width), -1, dtype=torch.int32)
    for i, r in enumerate(rows):
        t[i, :len(r)] = torch.tensor(r, dtype=torch.int32)
    return t


def _deal(c, counts, pool, seed):
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(pool, generator=g).tolist()
    rows, at = [], 0
    for n in counts:
        rows.append(order[at:at + n])
        at += n
    return rows


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": c}
    if c["op"] in ("attn8", "window"):
        Ls, P, D, Hkv = _lengths(c), c["P"], c["D"], c["Hkv"]
        counts = [_cdiv(L, P) for L in Ls]
        # a page is held for each visible key; the ones behind the window were given back
        seen = [_seen_pages(c, L) for L in Ls]
        pool = sum(map(len, seen)) + 3
        rows = _deal(c, [len(x) for x in seen], pool, seed)
        bt = torch.full((c["B"], max(counts)), -1, dtype=torch.int32)
        for i, (x, r) in enumerate(zip(seen, rows)):
            bt[i, torch.tensor(x, dtype=torch.int64)] = torch.tensor(r, dtype=torch.int32)
        s["bt"], s["sl"] = bt.to(DEV), _ints(Ls)
        if c["op"] == "attn8":
            s["kv"], s["sc"] = _cache8(pool, Hkv, P, D, g)
        else:
            s["kv"] = _values((pool, Hkv, P, 2 * D), g).bfloat16()
        s["q"] = torch.randn(c["B"], c["Hq"], D, device=DEV, generator=g).bfloat16()
        s["sinks"] = torch.randn(c["Hq"], device=DEV, generator=g) if c["sinks"] else None
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(c["B"], c["Hq"], device=DEV)
        s["scale"] = 1 / math.sqrt(D)
        # the (request, logical page) pairs that hold visible keys
        s["req"] = _ints([i for i, x in enumerate(seen) for _ in x]).long()
        s["page"] = _ints([j for x in seen for j in x]).long()
    elif c["op"] == "append":
        old, new = _append_plan(c)
        P, D, Hkv = c["P"], c["D"], c["Hkv"]
        Ls = [o + n for o, n in zip(old, new)]
        counts = [_cdiv(L, P) for L in Ls]
        touched = [list(range(o // P, k)) for o, k in zip(old, counts)]
        pool = sum(map(len, touched)) + 5
        rows = _deal(c, map(len, touched), pool, seed)
        bt = torch.full((c["B"], max(counts)), -1, dtype=torch.int32)
        for i, (x, r) in enumerate(zip(touched, rows)):
            bt[i, torch.tensor(x, dtype=torch.int64)] = torch.tensor(r, dtype=torch.int32)
        s["bt"], s["sl"] = bt.to(DEV), _ints(Ls)
        s["kv"], s["sc"] = _cache8(pool, Hkv, P, D, g)
        T = sum(new)
        x = _values((T, Hkv, 1, 2 * D), g).bfloat16()
        s["k"], s["v"] = x[:, :, 0, :D].contiguous(), x[:, :, 0, D:].contiguous()
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        s["cu"] = _ints(cu)
        # unit u = one touched page; where each new token goes in it
        s["req"] = _ints([i for i, x in enumerate(touched) for _ in x]).long()
        s["page"] = _ints([j for x in touched for j in x]).long()
        s["held"] = _ints([max(0, o - j * P) for o, x in zip(old, touched) for j in x])
        base, slots = 0, []
        for o, n, x in zip(old, new, touched):
            slots += [base * P + (o + i) - x[0] * P for i in range(n)]
            base += len(x)
        s["slot"] = _ints(slots).long()
    else:
        P = c["P"]
        if c["op"] == "fork":
            Ls = _fork_lengths(c)
            n = c["parents"] * c["copies"]
            rows = _deal(c, [_cdiv(L, P) for L in Ls], c["pages"], seed) + [[]] * n
            lens, width = Ls + [0] * n, _cdiv(c["hi"], P) + 1
            s["parents"] = _ints([i // c["copies"] for i in range(n)])
            s["children"] = _ints([c["parents"] + i for i in range(n)])
            s["src"], s["dst"] = _ints([-1] * n), _ints([-1] * n)
        elif c["op"] == "compact":
            rows = _compact_rows(c)
            lens, width = [len(r) * P - (len(r) > 0) for r in rows], _cdiv(c["hi"], P) + 1
            s["src"], s["dst"] = _ints([-1] * (c["pages"] // 2)), _ints([-1] * (c["pages"] // 2))
            s["moves"] = _ints([0])
        else:
            s["keep"], lens, s["after"] = _turnover_lengths(c)
            s["keep"], s["after"] = _ints(s["keep"]), _ints(s["after"])
            rows = _deal(c, [_cdiv(L, P) for L in lens], c["pages"], seed)
            width = _cdiv(c["hi"] + c["grow"], P) + 1
            s["rows"] = _ints(list(range(c["rows"])))
        if c["op"] != "turnover":
            s["kv"], s["sc"] = _cache8(c["pages"], c["Hkv"], P, c["D"], g)
        refs = torch.zeros(c["pages"], dtype=torch.int32)
        refs[torch.tensor([p for r in rows for p in r], dtype=torch.int64)] = 1
        bt = _tables(rows, width, c["pages"])
        # the tables, lengths and counts in one buffer, so that a pass can begin by putting
        # them back with one copy
        s["fresh"] = torch.cat([bt.view(-1), torch.tensor(lens, dtype=torch.int32), refs]).to(DEV)
        s["now"] = s["fresh"].clone()
        n = len(rows)
        s["bt"] = s["now"][:n * width].view(n, width)
        s["sl"], s["refs"] = s["now"][n * width:n * width + n], s["now"][n * width + n:]
    return s


# -------------------------------------------------------------------- run --
def run(s):
    op = s["case"]["op"]
    if op in ("attn8", "window"):
        return _run_attn(s)
    if op == "append":
        return _run_append(s)
    s["now"].copy_(s["fresh"])
    if op == "fork":
        return _run_fork(s)
    if op == "compact":
        return _run_compact(s)
    return _run_turnover(s)


def _run_attn(s):
    c = s["case"]
    if own:
        import paged_kv_cache_30_gb300 as pkv
        if c["op"] == "attn8":
            pkv.paged_decode_attn_fp8(s["q"], s["kv"], s["sc"], s["bt"], s["sl"], s["sinks"],
                                      c["window"], c["first"], s["scale"], c["P"], s["out"], s["lse"])
        else:
            pkv.paged_window_attn(s["q"], s["kv"], s["bt"], s["sl"], s["sinks"], c["window"],
                                  c["first"], s["scale"], c["P"], s["out"], s["lse"])
        return s["out"], s["lse"]
    B, Hq, D = s["q"].shape
    Hkv, P = s["kv"].shape[1], c["P"]
    blk = s["bt"][s["req"], s["page"]].long()
    kv = s["kv"][blk].float()
    k, v = kv[..., :D], kv[..., D:]
    if c["op"] == "attn8":
        sc = s["sc"][blk]
        k, v = k * sc[:, :, 0, None, None], v * sc[:, :, 1, None, None]
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)[s["req"]]
    x = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]  # [pages, Hkv, G, P]
    pos = s["page"][:, None] * P + torch.arange(P, device=DEV)
    L = s["sl"].long()[s["req"]][:, None]
    see = pos < L
    if c["window"] > 0:
        see = see & ((pos >= L - c["window"]) | (pos < c["first"]))
    x = x.masked_fill(~see[:, None, None, :], -math.inf)
    at = s["req"][:, None, None].expand(x.shape[:3])
    m = torch.full((B, *x.shape[1:3]), -math.inf, device=DEV).scatter_reduce_(0, at, x.amax(-1), "amax")
    p = torch.exp(x - m[s["req"]][..., None])
    l = torch.zeros(m.shape, device=DEV, dtype=torch.float64).index_add_(0, s["req"], p.sum(-1).double())
    o = torch.zeros(*m.shape, D, device=DEV, dtype=torch.float64)
    o.index_add_(0, s["req"], torch.matmul(p, v).double())
    den = l if s["sinks"] is None else l + torch.exp(s["sinks"].view(1, *m.shape[1:]) - m).double()
    out = (o / den[..., None]).view(B, Hq, D).bfloat16()
    return out, (m.double() + torch.log(l)).view(B, Hq).float()


def _run_append(s):
    c = s["case"]
    if own:
        import paged_kv_cache_30_gb300 as pkv
        pkv.gqa_kv_append_fp8(s["k"], s["v"], s["kv"], s["sc"], s["bt"], s["sl"], s["cu"], c["P"])
        return s["kv"], s["sc"]
    Hkv, P, D = c["Hkv"], c["P"], c["D"]
    blk = s["bt"][s["req"], s["page"]].long()
    n = blk.shape[0]
    x = torch.zeros(n * P, Hkv, 2, D, device=DEV)
    x[s["slot"]] = torch.stack([s["k"], s["v"]], dim=2).float()
    x = x.view(n, P, Hkv, 2, D).permute(0, 2, 1, 3, 4)  # [unit, head, slot, K|V, D]
    fresh = torch.zeros(n * P, dtype=torch.bool, device=DEV)
    fresh[s["slot"]] = True
    held = s["held"][:, None, None]
    s_old = torch.where(held > 0, s["sc"][blk], torch.zeros((), device=DEV))
    s_new = torch.maximum(s_old, _pow2_scale(x.abs().amax(dim=(2, 4))))
    div = torch.where(s_new > 0, s_new, torch.ones_like(s_new))[:, :, None, :, None]
    was = s["kv"][blk].view(n, Hkv, P, 2, D)
    kept = (was.float() * (s_old[:, :, None, :, None] / div)).clamp(-E4M3_MAX, E4M3_MAX)
    kept = kept.to(torch.float8_e4m3fn)
    code = (x / div).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    slot = torch.arange(P, device=DEV)[None, None, :, None, None]
    got = torch.where(fresh.view(n, 1, P, 1, 1), code.view(torch.uint8),
                      torch.where(slot < held[..., None, None], kept.view(torch.uint8),
                                  was.view(torch.uint8)))
    s["kv"].view(torch.uint8)[blk] = got.reshape(n, Hkv, P, 2 * D)
    s["sc"][blk] = s_new
    return s["kv"], s["sc"]


def _free_page(refs, rank):
    """The free page of each rank, lowest first, and how many there are."""
    seen = torch.cumsum(refs == 0, 0)
    return torch.searchsorted(seen, rank.long() + 1).clamp(max=refs.shape[0] - 1), seen[-1]


def _copy_pages(s):
    ok = s["dst"] >= 0
    src, dst = s["src"][ok].long(), s["dst"][ok].long()
    s["kv"].view(torch.uint8)[dst] = s["kv"].view(torch.uint8)[src]
    s["sc"][dst] = s["sc"][src]


def _run_fork(s):
    c = s["case"]
    if own:
        import paged_kv_cache_30_gb300 as pkv
        pkv.pages_fork(s["bt"], s["sl"], s["refs"], s["parents"], s["children"], c["P"], s["src"], s["dst"])
        pkv.pages_copy([s["kv"], s["sc"]], s["src"], s["dst"])
        return s["bt"], s["sl"], s["refs"], s["src"], s["dst"], s["kv"], s["sc"]
    P, par, chi = c["P"], s["parents"].long(), s["children"].long()
    L = s["sl"][par]
    full, part = (L // P).long(), L % P > 0
    page, free = _free_page(s["refs"], torch.cumsum(part, 0) - part.long())
    ok = ~part | (torch.cumsum(part, 0) <= free)
    rows = s["bt"][par]
    col = torch.arange(rows.shape[1], device=DEV)[None, :]
    share = (col < full[:, None]) & ok[:, None]
    took = part & ok
    at = (col == full[:, None]) & took[:, None]
    s["src"].copy_(torch.where(took, (rows * at).sum(1).int(), -1))
    s["dst"].copy_(torch.where(took, page.int(), -1))
    s["bt"][chi] = torch.where(share, rows, torch.where(at, page.int()[:, None], -1))
    s["sl"][chi] = torch.where(ok, L, 0)
    s["refs"].index_add_(0, rows.clamp(min=0).view(-1).long(), share.int().view(-1))
    s["refs"].index_add_(0, page, took.int())
    _copy_pages(s)
    return s["bt"], s["sl"], s["refs"], s["src"], s["dst"], s["kv"], s["sc"]


def _run_compact(s):
    c = s["case"]
    if own:
        import paged_kv_cache_30_gb300 as pkv
        pkv.pages_compact(s["bt"], s["sl"], s["refs"], c["P"], s["src"], s["dst"], s["moves"])
        pkv.pages_copy([s["kv"], s["sc"]], s["src"], s["dst"])
        return s["bt"], s["refs"], s["src"], s["dst"], s["moves"], s["kv"], s["sc"]
    refs, n = s["refs"], s["refs"].shape[0]
    live = refs > 0
    page = torch.arange(n, device=DEV)
    kept = live.sum()
    src, dst = torch.nonzero(live & (page >= kept))[:, 0], torch.nonzero(~live & (page < kept))[:, 0]
    dst = dst[:src.shape[0]]
    to = page.clone()
    to[src] = dst
    used = torch.arange(s["bt"].shape[1], device=DEV)[None, :] < ((s["sl"] + c["P"] - 1) // c["P"])[:, None]
    s["bt"].copy_(torch.where(used, to[s["bt"].clamp(min=0).long()].int(), s["bt"]))
    refs[dst] = refs[src]
    refs[src] = 0
    s["src"].fill_(-1)[:src.shape[0]] = src.int()
    s["dst"].fill_(-1)[:src.shape[0]] = dst.int()
    s["moves"].fill_(src.shape[0])
    _copy_pages(s)
    return s["bt"], s["refs"], s["src"], s["dst"], s["moves"], s["kv"], s["sc"]


def _run_turnover(s):
    c = s["case"]
    if own:
        import paged_kv_cache_30_gb300 as pkv
        pkv.pages_release(s["bt"], s["sl"], s["refs"], s["rows"], s["keep"], c["P"])
        pkv.pages_reserve(s["bt"], s["sl"], s["refs"], s["rows"], s["after"], c["P"])
        return s["bt"], s["sl"], s["refs"]
    P, rows = c["P"], s["rows"].long()
    L, keep = s["sl"][rows], torch.minimum(s["keep"], s["sl"][rows])
    table = s["bt"][rows]
    col = torch.arange(table.shape[1], device=DEV)[None, :]
    gone = (col >= ((keep + P - 1) // P)[:, None]) & (col < ((L + P - 1) // P)[:, None])
    s["refs"].index_add_(0, table.clamp(min=0).view(-1).long(), -gone.int().view(-1))
    table = torch.where(gone, -1, table)
    have = (keep + P - 1) // P
    want = torch.maximum((s["after"] + P - 1) // P, have)
    need = want - have
    first = torch.cumsum(need, 0) - need
    come = (col >= have[:, None]) & (col < want[:, None])
    page, free = _free_page(s["refs"], (first[:, None] + col - have[:, None]).clamp(min=0))
    ok = (need == 0) | (first + need <= free)
    come = come & ok[:, None]
    s["bt"][rows] = torch.where(come, page.int(), table)
    s["refs"].index_add_(0, page.view(-1), come.int().view(-1))
    s["sl"][rows] = torch.where(ok, torch.maximum(s["after"], keep), keep)
    return s["bt"], s["sl"], s["refs"]


# ------------------------------------------------------------------ exact --
def exact(c, seed):
    """The outputs from the definition, in 64 bits, request by request."""
    s = prepare(c, seed)
    if c["op"] in ("attn8", "window"):
        return _exact_attn(c, s)
    if c["op"] == "append":
        return _exact_append(c, s)
    return None  # page numbers and copied bytes: nothing is computed that could be inexact


def _exact_attn(c, s):
    B, Hq, D = s["q"].shape
    Hkv, P = c["Hkv"], c["P"]
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=DEV)
    for b, L in enumerate(s["sl"].tolist()):
        start = max(0, L - c["window"]) if c["window"] > 0 else 0
        pos = torch.cat([torch.arange(0, min(c["first"], start), device=DEV),
                         torch.arange(start, L, device=DEV)])
        if not len(pos):
            continue
        blk = s["bt"][b].long()[pos // P]
        sink = s["sinks"].double() if s["sinks"] is not None else None
        for h in range(Hkv):
            row = s["kv"].view(torch.uint8 if c["op"] == "attn8" else torch.bfloat16)[blk, h, pos % P]
            row = row.view(s["kv"].dtype).double()
            if c["op"] == "attn8":
                sc = s["sc"].double()[blk, h]
                row = torch.cat([row[:, :D] * sc[:, :1], row[:, D:] * sc[:, 1:]], dim=1)
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            x = (s["q"][b, heads].double() @ row[:, :D].T) / math.sqrt(D)
            lse[b, heads] = torch.logsumexp(x, dim=1)
            den = lse[b, heads]
            if sink is not None:
                den = torch.logaddexp(den, sink[heads])
            out[b, heads] = torch.exp(x - den[:, None]) @ row[:, D:]
    return out, lse


def _exact_append(c, s):
    """Codes and scales after the append, token by token of each page in 64 bits (the scale's
    exponent from the ratio itself, the code as the nearest multiple of its binade's step)."""
    kv, sc = s["kv"].double(), s["sc"].double()
    P, D = c["P"], c["D"]
    new = torch.stack([s["k"], s["v"]], dim=2).double()  # [T, Hkv, 2, D]
    cu, Ls, bt = s["cu"].tolist(), s["sl"].tolist(), s["bt"].tolist()
    for b, L in enumerate(Ls):
        at, n = L - (cu[b + 1] - cu[b]), cu[b + 1] - cu[b]
        for j in range(at // P, _cdiv(L, P)):
            lo, hi = max(at, j * P), min(L, (j + 1) * P)
            page, x = bt[b][j], new[cu[b] + lo - at:cu[b] + hi - at]  # [n, Hkv, 2, D]
            a = x.abs().amax(dim=(0, 3))
            need = torch.exp2(torch.ceil(torch.log2(a / E4M3_MAX) - 1e-12).clamp(min=MIN_EXP))
            need = torch.where(a > 0, need, torch.zeros_like(a))
            old = sc[page].clone() if lo > j * P else torch.zeros_like(a)
            now = torch.maximum(old, need)
            div = torch.where(now > 0, now, torch.ones_like(now))
            view = kv[page].view(c["Hkv"], P, 2, D)
            view[:, :lo - j * P] = _nearest(view[:, :lo - j * P] * (old / div)[:, None, :, None])
            view[:, lo - j * P:hi - j * P] = _nearest((x / div[None, :, :, None]).transpose(0, 1))
            sc[page] = now
    return kv, sc


def _nearest(x):
    """Nearest value with 3 fraction bits from 2^-6 on, steps of 2^-9 below, at most 448; ties
    to even."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -30))).clamp(min=-6)
    e = e - (torch.exp2(e) > x.abs()).double() * (e > -6) + (torch.exp2(e + 1) <= x.abs()).double()
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
