"""Plain 64-bit implementations of the 8-bit append, decode with a window and
first tokens, and the page calls, and the error bounds that follow from the
kernels' roundings.  Written from the definitions in include/pkv.h."""
import math

import torch

E4M3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()  # 0 .. 448


# -------------------------------------------------------------- e4m3 pages --
def encode(x):
    """e4m3 values (double) of x: nearest, ties to the even code, saturating, NaN kept."""
    a = x.double().abs()
    hi = torch.searchsorted(E4M3, a.nan_to_num(0.0).clamp(max=448.0).contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    to_hi, to_lo = E4M3[hi] - a, a - E4M3[lo]
    pick = torch.where((to_hi < to_lo) | ((to_hi == to_lo) & (hi % 2 == 0)), hi, lo)
    pick = torch.where(a >= 448.0, torch.full_like(pick, 126), pick)
    y = torch.copysign(E4M3[pick], x.double())
    return torch.where(x.isnan(), x.double(), y)


def need_scale(a):
    """Smallest power of two >= 2^-100 with a <= 448 s; 0 for 0 (a: a Python float)."""
    if a == 0:
        return 0.0
    s = 2.0 ** -100
    while a > 448.0 * s:
        s *= 2.0
    return s


def append(k, v, cache, scale, table, lens, cu, P):
    """(values of the codes, scales) after the append, in double; all CPU tensors."""
    vals, sc = cache.double(), scale.double().clone()
    Hkv, D = k.shape[1], k.shape[2]
    new = torch.stack([k, v], dim=2).double()
    for b in range(len(lens)):
        r0, r1 = int(cu[b]), int(cu[b + 1])
        at = int(lens[b]) - (r1 - r0)
        pos = {}
        for r in range(r0, r1):
            if at + r - r0 >= 0:
                pos.setdefault((at + r - r0) // P, []).append(r)
        for pg, rows in pos.items():
            page = int(table[b, pg]) if pg < table.shape[1] else -1
            if not 0 <= page < cache.shape[0]:
                continue
            slot = (at + rows[0] - r0) % P
            for h in range(Hkv):
                for kv in range(2):
                    x = new[rows, h, kv]
                    old = float(sc[page, h, kv]) if slot else 0.0
                    fin = x[x.isfinite()].abs()
                    s = max(old, need_scale(float(fin.amax()) if fin.numel() else 0.0))
                    half = slice(kv * D, (kv + 1) * D)
                    if s > old and slot:
                        vals[page, h, :slot, half] = encode(vals[page, h, :slot, half] * (old / s))
                    vals[page, h, slot:slot + len(rows), half] = encode(x / (s if s > 0 else 1.0))
                    sc[page, h, kv] = s
    return vals, sc


# ------------------------------------------------------------------ decode --
def visible(L, window, first):
    start = max(L - window, 0) if window > 0 else 0
    return torch.cat([torch.arange(0, min(first, start)), torch.arange(start, L)])


def decode(q, cache, scale, table, lens, sinks, window, first, softmax_scale, P, p_eps):
    """out, lse in double, and elementwise bounds of the kernel's distance from them.

    The kernel rounds the weights once (p_eps relative: 2^-8 in bf16; 2^-11 in fp16, with an
    absolute floor of 2^-25 of the largest weight times scale there), adds up N of them and
    D products in 32 bits, and rounds the output to bf16 (2^-8)."""
    B, Hq, D = q.shape
    Hkv, cache = cache.shape[1], cache.double()
    out, tol = torch.zeros(B, Hq, D, dtype=torch.float64), torch.zeros(B, Hq, D, dtype=torch.float64)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64)
    lse_tol = torch.zeros(B, Hq, dtype=torch.float64)
    for b in range(B):
        pos = visible(int(lens[b]), window, first)
        N = len(pos)
        if N == 0:
            continue
        page = table[b].long()[pos // P]
        ok = (page >= 0) & (page < cache.shape[0])
        for h in range(Hq):
            g = h // (Hq // Hkv)
            row = cache[page.clamp(0, cache.shape[0] - 1), g, pos % P]
            k, v = row[:, :D], row[:, D:]
            vs = torch.ones(N, dtype=torch.float64)
            if scale is not None:
                sc = scale[page.clamp(0, cache.shape[0] - 1), g].double()
                k, v, vs = k * sc[:, :1], v * sc[:, 1:], sc[:, 1]
            k = torch.where(ok[:, None], k, torch.zeros(()).double())
            v = torch.where(ok[:, None], v, torch.zeros(()).double())
            vs = torch.where(ok, vs, torch.zeros(()).double())
            qd = q[b, h].double()
            x = softmax_scale * (k @ qd)
            # D products and sums, the scale and the exponent's argument, each 2^-24
            dx = (D + 4) * 2.0 ** -24 * softmax_scale * float((k.abs() @ qd.abs()).amax()) \
                + 2.0 ** -22 * (1 + float(x.abs().amax()))
            lse[b, h] = torch.logsumexp(x, 0)
            lse_tol[b, h] = dx + N * 2.0 ** -24 + 2.0 ** -22 * (1 + abs(float(lse[b, h])))
            den = lse[b, h]
            if sinks is not None:
                den = torch.logaddexp(den, sinks[h].double())
            w = torch.exp(x - den)
            out[b, h] = w @ v
            sums = p_eps + 2 * dx + (N + 16) * 2.0 ** -24
            tol[b, h] = 2.0 ** -8 * out[b, h].abs() + sums * (w @ v.abs())
            if scale is not None:
                tol[b, h] += N * 2.0 ** -25 * 448.0 * float((w * vs).amax())
    return out, lse, tol, lse_tol


# ------------------------------------------------------------------- pages --
class Pool:
    """Tables, lengths and counts as Python lists."""

    def __init__(self, rows, width, pages, P):
        self.P, self.width = P, width
        self.table = [[-1] * width for _ in range(rows)]
        self.lens, self.refs = [0] * rows, [0] * pages

    def pages_of(self, n):
        return -(-n // self.P)

    def free(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def reserve(self, rows, lens):
        free, before = self.free(), 0
        for i, (r, n) in enumerate(zip(rows, lens)):
            if not 0 <= r < len(self.lens) or r in rows[:i] or n > self.width * self.P:
                continue
            have = self.pages_of(self.lens[r])
            need = max(self.pages_of(n) - have, 0)
            if need == 0 or before + need <= len(free):
                for j in range(need):
                    self.table[r][have + j] = free[before + j]
                    self.refs[free[before + j]] = 1
                self.lens[r] = max(self.lens[r], n)
            before += need

    def release(self, rows, keep):
        for r, n in zip(rows, keep):
            if not 0 <= r < len(self.lens):
                continue
            n = max(min(n, self.lens[r]), 0)
            for j in range(self.pages_of(n), self.pages_of(self.lens[r])):
                if self.table[r][j] != -1:
                    self.refs[self.table[r][j]] -= 1
                    self.table[r][j] = -1
            self.lens[r] = n

    def trim(self, window, first):
        for r, n in enumerate(self.lens):
            for j in range(self.pages_of(first), max(n - window, 0) // self.P):
                if self.table[r][j] != -1:
                    self.refs[self.table[r][j]] -= 1
                    self.table[r][j] = -1

    def fork(self, parents, children):
        free, before, src, dst = self.free(), 0, [], []
        lens = list(self.lens)
        for i, (p, c) in enumerate(zip(parents, children)):
            src.append(-1)
            dst.append(-1)
            rows = range(len(lens))
            if p not in rows or c not in rows or c in children[:i] or c in parents or lens[c]:
                continue
            full = lens[p] // self.P
            part = lens[p] % self.P > 0 and self.table[p][full] != -1
            if part and before >= len(free):
                self.table[c] = [-1] * self.width
                before += 1
                continue
            self.table[c] = self.table[p][:full] + [-1] * (self.width - full)
            for page in self.table[c][:full]:
                if page != -1:
                    self.refs[page] += 1
            if part:
                src[i], dst[i] = self.table[p][full], free[before]
                self.table[c][full] = dst[i]
                self.refs[dst[i]] = 1
                before += 1
            self.lens[c] = lens[p]
        return src, dst

    def compact(self, most):
        live = sum(r > 0 for r in self.refs)
        src = [p for p, r in enumerate(self.refs) if r > 0 and p >= live]
        dst = [p for p, r in enumerate(self.refs) if r <= 0 and p < live]
        moves = list(zip(src, dst))[:most]
        to = dict(moves)
        for s, d in moves:
            self.refs[d], self.refs[s] = self.refs[s], 0
        for r, n in enumerate(self.lens):
            for j in range(self.pages_of(n)):
                self.table[r][j] = to.get(self.table[r][j], self.table[r][j])
        pad = [-1] * (most - len(moves))
        return [m[0] for m in moves] + pad, [m[1] for m in moves] + pad, len(moves)
