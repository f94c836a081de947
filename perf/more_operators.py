"""Cases and plain forms of a served batch whose requests share a prefix, and of what comes
before its attention.

Three operators of a paged-attention server, each as a user calls it:

* ``prefix``  one decode token per request where groups of requests (forked samples, a common
  system prompt) share the pages of their first tokens, over a bf16 or an e4m3 cache;
* ``rope``    queries and keys of new tokens: a norm for each head and the rotation by their
  positions, half or interleaved pairs, the whole head or its first dims, plain frequencies or
  frequencies scaled for long contexts;
* ``append``  the same on the way into the paged cache, with the values: one token for each
  request, or whole prompts.

``run`` computes them with elementary torch operations while ``own`` is false, and through the
package's entry points while it is true.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # four samples of one short prompt on one kv head: the smallest call, all latency
        prefix_case(cache="bf16", sizes="4", Hq=8, Hkv=1, D=128, P=16,
                    shared_lo=512, shared_hi=512, mine_lo=1, mine_hi=64, idle=0, sinks=False,
                    pick=1, name="prefix_tiny"),
        # a served batch behind one system prompt, answers of mixed length
        prefix_case(cache="bf16", sizes="64", Hq=64, Hkv=8, D=128, P=16,
                    shared_lo=8192, shared_hi=8192, mine_lo=1, mine_hi=2048, idle=0, sinks=True,
                    pick=2, name="prefix_system"),
        # every request of a large batch reads one very long document
        prefix_case(cache="bf16", sizes="128", Hq=64, Hkv=8, D=128, P=32,
                    shared_lo=131072, shared_hi=131072, mine_lo=1, mine_hi=300, idle=0,
                    sinks=False, pick=3, name="prefix_document"),
        # prompts of ragged length sampled a few times each, some alone, some rows idle
        prefix_case(cache="e4m3", sizes="4,8,1,2,5,16,4,7,3,4,6,1", Hq=64, Hkv=8, D=128,
                    P=16, shared_lo=500, shared_hi=32768, mine_lo=1, mine_hi=1000, idle=3,
                    sinks=False, pick=4, name="prefix_samples8"),
        # 16 query heads per kv head, 64-wide heads, an 8-bit cache
        prefix_case(cache="e4m3", sizes="20,13", Hq=64, Hkv=4, D=64, P=32,
                    shared_lo=9000, shared_hi=20000, mine_lo=1, mine_hi=700, idle=0, sinks=True,
                    pick=5, name="prefix_heads64"),
        # the queries and keys of one decode step, rotated: all latency
        rope_case(T=64, Hq=64, Hkv=8, D=128, rot=128, pairs="half", norm=False, latent=False,
                  scaled=False, hi=32768, run=1, pick=6, name="rope_step"),
        # a prefill chunk: norms of the heads and the rotation
        rope_case(T=16384, Hq=32, Hkv=4, D=128, rot=128, pairs="half", norm=True, latent=False,
                  scaled=False, hi=32768, run=4096, pick=7, name="rope_prompts"),
        # verify tokens of a latent-attention model: the last 64 dims of 128 heads of 576, and
        # of the one latent row, frequencies scaled for long contexts
        rope_case(T=128, Hq=128, Hkv=1, D=64, rot=64, pairs="interleaved", norm=False, latent=True,
                  scaled=True, hi=131072, run=4, pick=8, name="rope_latent"),
        # half of each 64-wide head is rotated, ragged count of tokens
        rope_case(T=5001, Hq=24, Hkv=3, D=64, rot=32, pairs="interleaved", norm=True, latent=False,
                  scaled=False, hi=8192, run=700, pick=9, name="rope_part"),
        # one decode step's tokens, normed, rotated and written to the cache
        write_case(B=64, Hq=64, Hkv=8, D=128, P=16, rot=128, pairs="half", norm=True, scaled=False,
                   new_lo=1, new_hi=1, before=4000, pick=10, name="append_step"),
        # a batch of prompts of ragged length, some continuing a page, scaled frequencies
        write_case(B=16, Hq=64, Hkv=8, D=128, P=16, rot=128, pairs="half", norm=True, scaled=True,
                   new_lo=1, new_hi=2048, before=700, pick=11, name="append_prompts"),
        # one long prompt's chunk, 64-wide heads, no norms, larger pages
        write_case(B=1, Hq=32, Hkv=8, D=64, P=64, rot=64, pairs="interleaved", norm=False,
                   scaled=False, new_lo=8191, new_hi=8191, before=30000, pick=12,
                   name="append_chunk"),
    ]


def prefix_case(**kw):
    return dict(op="prefix", **kw)


def rope_case(**kw):
    return dict(op="rope", **kw)


def write_case(**kw):
    return dict(op="append", **kw)


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "prefix", "rope", "rope", "append", "append"])
    pick = rng.randrange(1 << 20)
    D = rng.choice([64, 128])
    if op == "prefix":
        Hkv, G = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8, 16])
        B, groups = _log_int(rng, 2, 200), _log_int(rng, 1, 12)
        sizes = [rng.randint(1, max(1, 2 * B // groups)) for _ in range(groups)]
        B = sum(sizes)
        # no draw has more products than the largest listed case, nor more keys of its own
        hi = _log_int(rng, 16, 100000)
        hi = max(16, min(hi, 100000 * 128 * 64 * 128 // (B * Hkv * G * D), (1 << 20) // groups))
        return prefix_case(cache=rng.choice(["bf16", "e4m3"]), sizes=",".join(map(str, sizes)),
                           Hq=G * Hkv, Hkv=Hkv, D=D, P=rng.choice([16, 32, 64]),
                           shared_lo=max(1, hi // 20), shared_hi=hi, mine_lo=1,
                           mine_hi=max(1, min(_log_int(rng, 1, 3000), (1 << 17) // B)),
                           idle=rng.choice([0, 0, 1]), sinks=rng.random() < 0.5, pick=pick)
    norm, scaled = rng.random() < 0.5, rng.random() < 0.5
    rot = rng.choice([D, D, D // 2, 16, D - 16])
    Hkv, G = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 4, 5, 8, 16])
    pairs = rng.choice(["half", "interleaved"])
    T = _log_int(rng, 1, 20000)
    T = max(1, min(T, (1 << 26) // ((G + 1) * Hkv * D)))
    if op == "rope":
        latent = rng.random() < 0.2
        if latent:
            D = rot = 64
            Hkv, G, T, norm = 1, 128, min(T, 512), False
        return rope_case(T=T, Hq=G * Hkv, Hkv=Hkv, D=D, rot=rot, pairs=pairs, norm=norm,
                         latent=latent, scaled=scaled, hi=_log_int(rng, 1000, 1 << 20),
                         run=rng.choice([1, 3, _log_int(rng, 4, 5000)]), pick=pick)
    B = _log_int(rng, 1, 128)
    new = rng.choice([1, max(1, min(T // B, 4096))])
    return write_case(B=B, Hq=G * Hkv, Hkv=Hkv, D=D, P=rng.choice([16, 32, 64, 128]), rot=rot,
                      pairs=pairs, norm=norm, scaled=scaled, new_lo=1, new_hi=new,
                      before=_log_int(rng, 1, 20000), pick=pick)


# ------------------------------------------------- sizes, fixed by the case --
def _cdiv(a, b):
    return -(-a // b)


def _plan(c):
    """Per group (first row, rows, shared tokens); per row its length: the shared tokens and
    its own, of log-uniform number, or 0 for an idle row."""
    r = random.Random(c["pick"] * 1009 + 5)
    groups, Ls = [], []
    for n in map(int, c["sizes"].split(",")):
        S = r.randint(c["shared_lo"], c["shared_hi"])
        groups.append((len(Ls), n, S))
        lo, hi = c["mine_lo"], c["mine_hi"]
        Ls += [S + min(hi, max(lo, int(round(math.exp(r.uniform(0.0, math.log(hi)))))))
               for _ in range(n)]
    for b in r.sample(range(len(Ls)), min(c["idle"], len(Ls) - 1)):
        Ls[b] = 0
    return groups, Ls


def _write_plan(c):
    """Per request: tokens already held, new tokens."""
    r = random.Random(c["pick"] * 1013 + 7)
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["B"])]
    return [r.randint(0, c["before"]) for _ in range(c["B"])], new


def work(c):
    D = c["D"]
    if c["op"] == "prefix":
        groups, Ls = _plan(c)
        esz = 1 if c["cache"] == "e4m3" else 2
        keys = pairs = 0  # read; (token, key)
        for at, n, S in groups:
            mine = [L for L in Ls[at:at + n] if L]
            keys += (S if mine else 0) + sum(L - S for L in mine)
            pairs += sum(mine)
        b = keys * c["Hkv"] * 2 * D * esz
        b += _cdiv(keys, c["P"]) * (4 + (c["Hkv"] * 8 if esz == 1 else 0))
        return {"bytes": b + len(Ls) * c["Hq"] * (2 * D * 2 + 4) + len(Ls) * 4,
                "flops": 4 * pairs * c["Hq"] * D}
    T = c["T"] if c["op"] == "rope" else sum(_write_plan(c)[1])
    rows = T * (c["Hq"] + c["Hkv"])
    b, f = rows * D * 4 + T * 4, rows * (c["rot"] * 3 + (D * 4 if c["norm"] else 0))
    if c["op"] == "append":
        b += T * c["Hkv"] * D * 4
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------- inputs --
def _values(shape, g):
    """Queries, keys and values as a model makes them: unit normal with a few wide channels and
    a magnitude that varies from place to place."""
    x = torch.randn(shape, device=DEV, generator=g)
    wide = 1 + 5 * (torch.rand(shape[-1], device=DEV, generator=g) < 0.03).float()
    size = torch.randn(*shape[:2], *[1] * (len(shape) - 2), device=DEV, generator=g).mul_(0.5).exp_()
    return x.mul_(wide).mul_(size)


def _cache8(x, Hkv, P, D):
    """e4m3 codes and their scales: the least power of two that holds a page's values."""
    a = x.view(-1, Hkv, P, 2, D).abs().amax(dim=(2, 4))
    s = torch.exp2(torch.ceil(torch.log2(a / 448.0)))
    codes = (x.view(-1, Hkv, P, 2, D) / s[:, :, None, :, None]).to(torch.float8_e4m3fn)
    return codes.view(-1, Hkv, P, 2 * D), s.contiguous()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _frequencies(c):
    """Angle per position of each pair, in 64 bits; scaled: a pair that turns fewer than once
    in the first 8192 positions is slowed by 16, one that turns more than 32 times is kept,
    and those between are mixed by their turns."""
    f = 500000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])
    if c["scaled"]:
        keep = ((8192 * f / (2 * math.pi) - 1) / 31).clamp(0, 1)
        f = f * (keep + (1 - keep) / 16)
    return f


def _rotation(c, s):
    s["freq"] = _frequencies(c).to(DEV)
    s["factor"] = 0.1 * math.log(16) + 1 if c["scaled"] else 1.0
    s["eps"] = 1e-6
    if own:
        import paged_kv_cache_30_gb300 as pkv
        s["table"] = pkv.rope_table(c["rot"], base=500000.0, factor=16.0 if c["scaled"] else 1.0,
                                    original_len=8192, low=1.0, high=32.0, device=DEV)


def _weights(c, s, g):
    s["qw"] = s["kw"] = None
    if c["norm"]:
        s["qw"] = (1 + 0.2 * torch.randn(c["D"], device=DEV, generator=g)).bfloat16()
        s["kw"] = (1 + 0.2 * torch.randn(c["D"], device=DEV, generator=g)).bfloat16()


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": c}
    D, Hkv, Hq = c["D"], c["Hkv"], c["Hq"]
    if c["op"] == "prefix":
        P = c["P"]
        groups, Ls = _plan(c)
        # full pages of the shared tokens are the group's, the rest are the row's own
        rows, own_pages, pool = [None] * len(Ls), [], 0
        for at, n, S in groups:
            head = list(range(pool, pool + S // P))
            pool += S // P
            for b in range(at, at + n):
                k = max(0, _cdiv(Ls[b], P) - len(head))
                rows[b] = head + list(range(pool, pool + k)) if Ls[b] else []
                pool += k if Ls[b] else 0
                own_pages += [(b, j) for j in range(len(head), len(rows[b]))]
        perm = torch.randperm(pool + 3, generator=torch.Generator().manual_seed(seed)).int()
        bt = torch.full((len(Ls), max(map(len, rows))), -1, dtype=torch.int32)
        for b, r in enumerate(rows):
            bt[b, :len(r)] = perm[torch.tensor(r, dtype=torch.int64)] if r else bt[b, :0]
        x = _values((pool + 3, Hkv, P, 2 * D), g)
        # a partly shared page holds the same tokens for each of the group's rows
        for at, n, S in groups:
            part, live = S % P, [b for b in range(at, at + n) if Ls[b]]
            if part and live:
                pages = bt[live, S // P].long().to(DEV)
                x[pages, :, :part] = x[pages[0], :, :part].clone()
        if c["cache"] == "e4m3":
            s["kv"], s["sc"] = _cache8(x, Hkv, P, D)
            for at, n, S in groups:  # and the same codes and scales
                part, live = S % P, [b for b in range(at, at + n) if Ls[b]]
                if part and live:
                    pages = bt[live, S // P].long().to(DEV)
                    s["sc"][pages] = s["sc"][pages].amax(dim=0)
                    codes = x[pages].view(len(live), Hkv, P, 2, D)
                    codes = codes / s["sc"][pages][:, :, None, :, None]
                    s["kv"].view(torch.uint8)[pages] = codes.to(torch.float8_e4m3fn).view(
                        torch.uint8).view(len(live), Hkv, P, 2 * D)
        else:
            s["kv"] = x.bfloat16()
        del x
        s["bt"], s["sl"] = bt.to(DEV), _ints(Ls)
        s["cu"] = _ints([at for at, _, _ in groups] + [len(Ls)])
        s["shared"] = _ints([S for _, _, S in groups])
        s["groups"], s["lens"] = groups, Ls
        s["q"] = torch.randn(len(Ls), Hq, D, device=DEV, generator=g).bfloat16()
        s["sinks"] = torch.randn(Hq, device=DEV, generator=g) if c["sinks"] else None
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(len(Ls), Hq, device=DEV)
        s["scale"] = 1 / math.sqrt(D)
        s["req"] = _ints([b for b, _ in own_pages]).long()
        s["page"] = _ints([j for _, j in own_pages]).long()
        s["first"] = _ints([S for _, n, S in groups for _ in range(n)]).long()
        return s
    _rotation(c, s)
    _weights(c, s, g)
    if c["op"] == "rope":
        T = c["T"]
        r = random.Random(c["pick"] * 1019 + 11)
        pos = []
        while len(pos) < T:  # runs of neighbouring tokens, as prompts and verify tokens are
            p0 = r.randrange(c["hi"])
            pos += range(p0, p0 + min(c["run"], T - len(pos)))
        s["pos"] = _ints(pos)
        if c["latent"]:
            q, k = _values((T, Hq, 576), g).bfloat16(), _values((T, 1, 576), g).bfloat16()
            s["q"], s["k"] = q[..., 512:], k[..., 512:]
            s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        else:  # one projection's output
            x = _values((T, Hq + 2 * Hkv, D), g).bfloat16()
            s["q"], s["k"] = x[:, :Hq], x[:, Hq:Hq + Hkv]
            s["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
            s["k_out"] = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=DEV)
        return s
    P = c["P"]
    old, new = _write_plan(c)
    Ls = [o + n for o, n in zip(old, new)]
    touched = [list(range(o // P, _cdiv(L, P))) for o, L in zip(old, Ls)]
    pool = sum(map(len, touched)) + 5
    perm = torch.randperm(pool, generator=torch.Generator().manual_seed(seed)).int()
    bt = torch.full((c["B"], max(_cdiv(L, P) for L in Ls)), -1, dtype=torch.int32)
    at, slots = 0, []
    for b, x in enumerate(touched):
        bt[b, x[0]:x[0] + len(x)] = perm[at:at + len(x)]
        at += len(x)
    s["bt"], s["sl"] = bt.to(DEV), _ints(Ls)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["cu"] = None if c["new_hi"] == 1 else _ints(cu)
    T = cu[-1]
    s["req"] = _ints([b for b, n in enumerate(new) for _ in range(n)]).long()
    s["pos"] = _ints([o + i for o, n in zip(old, new) for i in range(n)])
    s["kv"] = _values((pool, Hkv, P, 2 * D), g).bfloat16()
    x = _values((T, Hq + 2 * Hkv, D), g).bfloat16()
    s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    s["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
    return s


# -------------------------------------------------------------------- run --
def run(s):
    op = s["case"]["op"]
    if op == "prefix":
        return _run_prefix(s)
    if op == "rope":
        return _run_rope(s)
    return _run_append(s)


def _run_prefix(s):
    c = s["case"]
    P, D, Hkv = c["P"], c["D"], c["Hkv"]
    if own:
        import paged_kv_cache_30_gb300 as pkv
        if c["cache"] == "e4m3":
            pkv.paged_prefix_attn_fp8(s["q"], s["kv"], s["sc"], s["bt"], s["sl"], s["cu"],
                                      s["shared"], s["sinks"], s["scale"], P, s["out"], s["lse"])
        else:
            pkv.paged_prefix_attn(s["q"], s["kv"], s["bt"], s["sl"], s["cu"], s["shared"],
                                  s["sinks"], s["scale"], P, s["out"], s["lse"])
        return s["out"], s["lse"]
    B, Hq, _ = s["q"].shape
    G = Hq // Hkv
    m = torch.full((B, Hkv, G), -math.inf, device=DEV)
    l = torch.zeros(B, Hkv, G, device=DEV, dtype=torch.float64)
    o = torch.zeros(B, Hkv, G, D, device=DEV, dtype=torch.float64)

    def pages(blk):  # [pages, Hkv, P, D] keys, values
        kv = s["kv"][blk].float()
        k, v = kv[..., :D], kv[..., D:]
        if c["cache"] == "e4m3":
            sc = s["sc"][blk]
            k, v = k * sc[:, :, 0, None, None], v * sc[:, :, 1, None, None]
        return k, v

    # the shared tokens of each group against all of its rows
    for at, n, S in s["groups"]:
        rows = [b for b in range(at, at + n) if s["lens"][b]]
        if not rows:
            continue
        sel = torch.tensor(rows, device=DEV)
        q = s["q"][sel].float().view(len(rows), Hkv, G, D).transpose(0, 1).reshape(Hkv, -1, D)
        gm, gl, go = m[sel].transpose(0, 1).reshape(Hkv, -1), 0.0, 0.0
        step = max(1, (1 << 27) // (q.shape[0] * q.shape[1] * P))  # pages at a time
        for p0 in range(0, _cdiv(S, P), step):
            blk = s["bt"][rows[0], p0:min(p0 + step, _cdiv(S, P))].long()
            k, v = pages(blk)
            keys = min(S - p0 * P, len(blk) * P)
            k = k.transpose(0, 1).reshape(Hkv, -1, D)[:, :keys]
            v = v.transpose(0, 1).reshape(Hkv, -1, D)[:, :keys]
            x = torch.matmul(q, k.transpose(1, 2)) * s["scale"]
            top = torch.maximum(gm, x.amax(-1))
            p = torch.exp(x - top[..., None])
            keep = torch.exp(gm - top).double()
            gl = gl * keep + p.sum(-1).double()
            go = go * keep[..., None] + torch.matmul(p, v).double()
            gm = top
        m[sel] = gm.view(Hkv, len(rows), G).transpose(0, 1)
        l[sel] = gl.view(Hkv, len(rows), G).transpose(0, 1)
        o[sel] = go.view(Hkv, len(rows), G, D).transpose(0, 1)
    # each row's own tokens, page by page
    req, page = s["req"], s["page"]
    k, v = pages(s["bt"][req, page].long())
    x = torch.matmul(s["q"].float().view(B, Hkv, G, D)[req], k.transpose(-1, -2)) * s["scale"]
    pos = page[:, None] * P + torch.arange(P, device=DEV)
    see = (pos < s["sl"].long()[req][:, None]) & (pos >= s["first"][req][:, None])
    x = x.masked_fill(~see[:, None, None, :], -math.inf)
    at = req[:, None, None].expand(x.shape[:3])
    top = m.clone().scatter_reduce_(0, at, x.amax(-1), "amax")
    keep = torch.where(l > 0, torch.exp(m - top).double(), 0.0)
    l, o = l * keep, o * keep[..., None]
    p = torch.exp(x - torch.where(top > -math.inf, top, 0.0)[req][..., None])
    l.index_add_(0, req, p.sum(-1).double())
    o.index_add_(0, req, torch.matmul(p, v).double())
    den = l if s["sinks"] is None else l + torch.exp(s["sinks"].view(1, Hkv, G) - top).double()
    out = torch.where(l[..., None] > 0, o / den[..., None], 0.0).view(B, Hq, D).bfloat16()
    return out, (top.double() + torch.log(l)).view(B, Hq).float()


def _normed(x, w, eps):
    x = x.float()
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()


def _rotated(x, s, pos):
    """x [T, H, D] in 32 bits, its first dims rotated by the angles of positions pos."""
    c = s["case"]
    a = pos.double()[:, None] * s["freq"]  # far positions: 64 bits
    cos, sin = (a.cos() * s["factor"]).float()[:, None], (a.sin() * s["factor"]).float()[:, None]
    r = x[..., :c["rot"]]
    if c["pairs"] == "half":
        u, v = r.chunk(2, dim=-1)
        r = torch.cat([u * cos - v * sin, v * cos + u * sin], dim=-1)
    else:
        u, v = r[..., 0::2], r[..., 1::2]
        r = torch.stack([u * cos - v * sin, v * cos + u * sin], dim=-1).flatten(-2)
    return torch.cat([r, x[..., c["rot"]:]], dim=-1)


def _run_rope(s):
    c = s["case"]
    if own:
        import paged_kv_cache_30_gb300 as pkv
        pkv.qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["eps"], s["pos"], s["table"],
                         s["factor"], c["pairs"] == "interleaved", s["q_out"], s["k_out"])
        return s["q_out"], s["k_out"]
    q = _rotated(_normed(s["q"], s["qw"], s["eps"]), s, s["pos"])
    k = _rotated(_normed(s["k"], s["kw"], s["eps"]), s, s["pos"])
    return q.bfloat16(), k.bfloat16()


def _run_append(s):
    c = s["case"]
    if own:
        import paged_kv_cache_30_gb300 as pkv
        pkv.gqa_rope_append(s["q"], s["k"], s["v"], s["qw"], s["kw"], s["eps"], None, s["table"],
                            s["factor"], c["pairs"] == "interleaved", s["kv"], s["bt"], s["sl"],
                            s["cu"], c["P"], s["q_out"])
        return s["q_out"], s["kv"]
    P = c["P"]
    q = _rotated(_normed(s["q"], s["qw"], s["eps"]), s, s["pos"])
    k = _rotated(_normed(s["k"], s["kw"], s["eps"]), s, s["pos"])
    pos = s["pos"].long()
    blk = s["bt"][s["req"], pos // P].long()
    s["kv"][blk, :, pos % P] = torch.cat([k.bfloat16(), s["v"]], dim=-1)
    return q.bfloat16(), s["kv"]


# ------------------------------------------------------------------ exact --
def exact(c, seed):
    """The outputs from the definition, in 64 bits."""
    s = prepare(c, seed)
    if c["op"] == "prefix":
        return _exact_prefix(c, s)
    out = [_exact_rope(c, s, s["q"], s["qw"])]
    if c["op"] == "rope":
        return out[0], _exact_rope(c, s, s["k"], s["kw"])
    k, v, P = _exact_rope(c, s, s["k"], s["kw"]), s["v"].double(), c["P"]
    kv, t = s["kv"].double(), 0
    old, new = _write_plan(c)
    for b, (o, n) in enumerate(zip(old, new)):
        for j in range(o // P, _cdiv(o + n, P)):
            lo, hi = max(o, j * P), min(o + n, (j + 1) * P)
            rows = slice(t + lo - o, t + hi - o)
            page = kv[int(s["bt"][b, j])]
            page[:, lo - j * P:hi - j * P, :c["D"]] = k[rows].transpose(0, 1)
            page[:, lo - j * P:hi - j * P, c["D"]:] = v[rows].transpose(0, 1)
        t += n
    return out[0], kv


def _exact_prefix(c, s):
    """Row by row over all of its keys, as if nothing were shared."""
    B, Hq, D = s["q"].shape
    P, Hkv = c["P"], c["Hkv"]
    G = Hq // Hkv
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=DEV)
    for at, n, S in s["groups"]:
        held, pages = None, None
        for b in range(at, at + n):
            L = s["lens"][b]
            if not L:
                continue
            blk = s["bt"][b, :_cdiv(L, P)].long()
            if pages is None or S // P == 0 or not torch.equal(blk[:S // P], pages):
                pages = blk[:S // P]
                held = _exact_pages(c, s, pages)
            mine = _exact_pages(c, s, blk[S // P:])
            q = s["q"][b].double().view(Hkv, G, D)
            keys = L - (S // P) * P
            x = torch.cat([q @ held[..., :D].mT, q @ mine[:, :keys, :D].mT], dim=-1) / math.sqrt(D)
            total = torch.logsumexp(x, dim=-1)
            lse[b] = total.view(Hq)
            if s["sinks"] is not None:
                total = torch.logaddexp(total, s["sinks"].double().view(Hkv, G))
            w = torch.exp(x - total[..., None])
            cut = held.shape[1]
            out[b] = (w[..., :cut] @ held[..., D:] + w[..., cut:] @ mine[:, :keys, D:]).view(Hq, D)
    return out, lse


def _exact_pages(c, s, blk):
    """[Hkv, tokens, 2D] of the pages in a row."""
    D, P = c["D"], c["P"]
    x = s["kv"].view(torch.uint8 if c["cache"] == "e4m3" else torch.bfloat16)[blk]
    x = x.view(s["kv"].dtype).double()
    if c["cache"] == "e4m3":
        x = (x.view(*x.shape[:3], 2, D) * s["sc"].double()[blk][:, :, None, :, None]).flatten(-2)
    return x.transpose(0, 1).reshape(c["Hkv"], -1, 2 * D)


def _exact_rope(c, s, x, w):
    """Each pair as a complex number, times the unit number of its angle."""
    x = x.double()
    if w is not None:
        x = w.double() * x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / c["D"] + s["eps"])
    turn = torch.polar(torch.full_like(s["freq"], s["factor"]).expand(len(x), -1),
                       torch.outer(s["pos"].double(), s["freq"]))[:, None]
    half, got = c["rot"] // 2, x.clone()
    i = torch.arange(half, device=DEV)
    re, im = (i, i + half) if c["pairs"] == "half" else (2 * i, 2 * i + 1)
    z = torch.complex(x[..., re], x[..., im]) * turn
    got[..., re], got[..., im] = z.real, z.imag
    return got
