"""GPU page calls (fork, release, reserve, compact, copy) against lists in
Python: tables, lengths, counts, copy lists and copied bytes equal."""
import math
import random

import pytest
import torch

import paged_kv_cache_30_gb300 as pkv
from tests import paged_plain as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    pkv.load_library()
    pkv.init(0)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Device:
    """The same state on the device."""

    def __init__(self, m):
        self.P = m.P
        self.bt, self.sl, self.refs = ints(m.table), ints(m.lens), ints(m.refs)

    def same(self, m):
        torch.cuda.synchronize()
        return (self.bt.tolist() == m.table and self.sl.tolist() == m.lens
                and self.refs.tolist() == m.refs)

    def reserve(self, rows, lens):
        pkv.pages_reserve(self.bt, self.sl, self.refs, ints(rows), ints(lens), self.P)

    def release(self, rows, keep):
        pkv.pages_release(self.bt, self.sl, self.refs, ints(rows), ints(keep), self.P)

    def trim(self, window, first):
        pkv.pages_trim(self.bt, self.sl, self.refs, self.P, window, first)

    def fork(self, parents, children):
        src, dst = ints([7] * len(parents)), ints([7] * len(parents))
        pkv.pages_fork(self.bt, self.sl, self.refs, ints(parents), ints(children), self.P, src, dst)
        return src, dst

    def compact(self, most):
        src, dst, n = ints([7] * most), ints([7] * most), ints([7])
        pkv.pages_compact(self.bt, self.sl, self.refs, self.P, src, dst, n)
        return src, dst, n


def expect_flag(code):
    with pytest.raises(pkv.PkvError) as e:
        pkv.check_errors(0)
    assert e.value.code == code


@pytest.mark.parametrize("P,pages,rows", [(16, 300, 20), (32, 5000, 100), (1, 64, 5), (16, 9000, 700)])
def test_a_long_run_of_page_calls(P, pages, rows):
    rng = random.Random(P + pages)
    width = 12
    m = plain.Pool(rows, width, pages, P)
    d = Device(m)
    for step in range(30):
        pick = rng.sample(range(rows), rng.randint(1, rows))
        what = step % 4
        if what == 0:
            lens = [rng.randint(0, width * P) for _ in pick]
            need = sum(max(0, m.pages_of(n) - m.pages_of(m.lens[r])) for r, n in zip(pick, lens))
            if need > len(m.free()):
                lens = [min(n, P) for n in lens]
            m.reserve(pick, lens)
            d.reserve(pick, lens)
        elif what in (1, 3):
            keep = [rng.randint(-1, width * P) for _ in pick]
            if what == 3:
                keep = [0] * len(pick)
            m.release(pick, keep)
            d.release(pick, keep)
        else:
            empty = [r for r in range(rows) if m.lens[r] == 0]
            full = [r for r in range(rows) if m.lens[r] > 0]
            if empty and full:
                kids = rng.sample(empty, rng.randint(1, min(len(empty), len(m.free()) or 1)))
                par = [rng.choice(full) for _ in kids]
                src, dst = m.fork(par, kids)
                s, t = d.fork(par, kids)
                assert s.tolist() == src and t.tolist() == dst
        assert d.same(m), f"step {step}"
        if step % 3 == 2:  # then the row is never cut to where trimmed pages would be seen
            window, first = rng.randint(1, 9 * P), rng.choice([0, 0, 1, P, 2 * P + 3])
            m.trim(window, first)
            d.trim(window, first)
            assert d.same(m), f"trim after step {step}"
        if step % 5 == 4:
            most = rng.choice([pages // 2, 3, 0])
            src, dst, n = m.compact(most)
            s, t, k = d.compact(most)
            assert s.tolist() == src and t.tolist() == dst and k.tolist() == [n]
            assert d.same(m), f"compact after step {step}"
        flags = 0
        try:
            flags = pkv.check_errors(0)
        except pkv.PkvError as e:  # a pool that ran out is part of the run
            assert e.code == -8
        assert flags == 0


def test_reserve_grants_in_order_until_the_pool_runs_out():
    m = plain.Pool(6, 8, 10, 16)
    d = Device(m)
    rows, lens = [0, 1, 2, 3], [64, 100, 1, 0]  # needs 4, 7, 1, 0 of 10: the second is refused,
    m.reserve(rows, lens)                       # and with it all later ones that need a page
    d.reserve(rows, lens)
    assert m.lens == [64, 0, 0, 0, 0, 0]
    assert d.same(m)
    expect_flag(-8)


def test_fork_without_a_free_page_stays_empty():
    m = plain.Pool(5, 4, 4, 16)
    d = Device(m)
    for x in (m, d):
        x.reserve([0, 1], [20, 32])
    m.fork([1, 0], [2, 3])
    d.fork([1, 0], [2, 3])
    assert m.lens == [20, 32, 32, 0, 0]
    assert d.same(m)
    expect_flag(-8)


def test_refused_entries_change_nothing_and_are_flagged():
    m = plain.Pool(6, 4, 40, 16)
    d = Device(m)
    for x in (m, d):
        x.reserve([0, 1], [20, 32])
    assert pkv.check_errors(0) == 0
    cases = [([0, 0], [2, 2]), ([0, 1], [1, 2]), ([0, 9], [3, 4]), ([1, 0], [-1, 5]), ([2, 0], [3, 2])]
    for parents, children in cases:
        src, dst = m.fork(parents, children)
        s, t = d.fork(parents, children)
        assert s.tolist() == src and t.tolist() == dst
        assert d.same(m)
        expect_flag(-7)
        for x in (m, d):
            x.release([2, 3, 4, 5], [0, 0, 0, 0])
    for rows, lens in (([0, 0], [40, 50]), ([7, 1], [3, 40]), ([2, 3], [65, 64])):
        m.reserve(rows, lens)
        d.reserve(rows, lens)
        assert d.same(m)
        expect_flag(-7)


def test_a_row_released_twice_loses_its_pages_once():
    m = plain.Pool(3, 8, 40, 16)
    d = Device(m)
    for x in (m, d):
        x.reserve([0, 1], [128, 100])
        x.release([0, 1, 0, 0], [100, 0, 3, 50])
    assert m.lens[0] == 3
    assert d.same(m)
    assert pkv.check_errors(0) == 0


@pytest.mark.parametrize("window,first", [(1, 0), (16, 0), (17, 5), (40, 16), (100, 33), (5000, 1)])
def test_trimmed_rows_are_attended_as_before(window, first):
    """Pages that a window and first tokens hide go back to the pool, are taken by another row and
    overwritten; the row's attention stays what it was."""
    P, lens = 16, [200, 161, 160, 15, 0, 113]
    m = plain.Pool(7, 16, 70, P)
    d = Device(m)
    for x in (m, d):
        x.reserve([0, 1, 2, 3, 4, 5], lens)
    g = torch.Generator().manual_seed(window)
    kv = torch.randn(70, 2, P, 128, generator=g).bfloat16().cuda()
    q = torch.randn(7, 8, 64, generator=g).bfloat16().cuda()
    outs = [torch.zeros_like(q) for _ in range(2)]
    pkv.paged_window_attn(q, kv, d.bt, d.sl, None, window, first, 0.125, P, outs[0])
    held = sum(m.refs)
    for x in (m, d):
        x.trim(window, first)
    assert d.same(m)
    free = 70 - sum(m.refs)
    assert free >= 70 - held
    take = min(free, 16) * P
    for x in (m, d):
        x.reserve([6], [take])
    assert d.same(m)
    kv[torch.tensor([p for p in m.table[6] if p >= 0]).cuda()] = float("nan")
    pkv.paged_window_attn(q[:6], kv, d.bt[:6], d.sl[:6], None, window, first, 0.125, P, outs[1][:6])
    torch.cuda.synchronize()
    assert torch.equal(outs[0][:6], outs[1][:6])
    assert pkv.check_errors(0) == 0


def test_counts_below_zero_are_refused():
    m = plain.Pool(2, 4, 8, 16)
    d = Device(m)
    d.reserve([0], [40])
    d.refs[1] = 0
    d.release([0], [0])
    torch.cuda.synchronize()
    assert d.refs.tolist() == [0] * 8
    expect_flag(-7)


@pytest.mark.parametrize("live", ["none", "all", "front", "back"])
def test_compact_at_the_ends(live):
    m = plain.Pool(4, 16, 50, 16)
    d = Device(m)
    if live != "none":
        n = 50 if live == "all" else 20
        for x in (m, d):
            x.reserve([0, 1, 2, 3], [13 * 16, 13 * 16, 12 * 16, 12 * 16] if n == 50 else
                      [16 * 16, 4 * 16, 0, 0])
        if live == "back":
            for x in (m, d):
                x.release([0], [0])
    src, dst, n = m.compact(25)
    s, t, k = d.compact(25)
    assert s.tolist() == src and t.tolist() == dst and k.tolist() == [n]
    assert d.same(m)
    assert pkv.check_errors(0) == 0


def test_many_pages_one_row_and_odd_counts():
    m = plain.Pool(1, 4500, 70001, 16)
    m.refs = [1 if (i * 2654435761 >> 5) % 3 else 0 for i in range(70001)]
    d = Device(m)
    m.reserve([0], [4500 * 16 - 5])
    d.reserve([0], [4500 * 16 - 5])
    assert d.same(m)
    src, dst, n = m.compact(35000)
    s, t, k = d.compact(35000)
    assert s.tolist() == src and t.tolist() == dst and k.tolist() == [n]
    assert d.same(m)
    assert pkv.check_errors(0) == 0


@pytest.mark.parametrize("shape,dtype", [((50, 2, 16, 256), torch.bfloat16), ((50, 1, 16, 128), torch.float8_e4m3fn),
                                         ((50, 3, 2), torch.float32), ((50, 1, 1), torch.int32),
                                         ((50, 8, 32, 256), torch.bfloat16), ((50,), torch.float32)])
def test_copied_bytes(shape, dtype):
    g = torch.Generator().manual_seed(1)
    n = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
    raw = torch.randint(0, 256, (n,), generator=g, dtype=torch.uint8).cuda()
    t = raw.view(dtype).view(shape)
    src, dst = ints([3, 4, 4, -1, 49, 7, -1]), ints([0, 1, 2, 5, 48, -1, -1])
    want = raw.view(50, -1).clone()
    want[torch.tensor([0, 1, 2, 48])] = want[torch.tensor([3, 4, 4, 49])]
    pkv.pages_copy(t, src, dst)
    torch.cuda.synchronize()
    assert torch.equal(raw.view(50, -1), want)
    assert pkv.check_errors(0) == 0


def test_copies_of_several_caches_with_strides_and_bad_indices():
    g = torch.Generator().manual_seed(2)
    wide = torch.randn(30, 2, 4, 16, 64, generator=g).cuda()
    nhd = torch.randn(30, 16, 4, 32, generator=g).bfloat16().cuda()
    sc = torch.randn(20, 4, 2, generator=g).cuda()
    tensors = [wide[:, 1], nhd.transpose(1, 2), sc] + [torch.randn(30, 9, generator=g).cuda() for _ in range(10)]
    want = [t.clone() for t in tensors]
    for w in want:
        w[5], w[6] = w[1].clone(), w[19].clone()
        if w.shape[0] > 25:
            w[7] = w[25].clone()
    other = wide[:, 0].clone()
    pkv.pages_copy(tensors, ints([1, 19, 25, 40]), ints([5, 6, 7, 8]))
    torch.cuda.synchronize()
    for t, w in zip(tensors, want):
        assert torch.equal(t, w)
    assert torch.equal(wide[:, 0], other)
    expect_flag(-7)


def test_many_copies():
    t = torch.arange(4000 * 1000, dtype=torch.int32, device="cuda").view(4000, 1000)
    want = t.clone()
    want[:2000] = want[2000:]
    pkv.pages_copy([t], ints(list(range(2000, 4000))), ints(list(range(2000))))
    torch.cuda.synchronize()
    assert torch.equal(t, want)


def test_serving_run_in_a_captured_graph():
    """Reserve, append, decode, fork, copy, append, decode, release, compact, copy, decode:
    eagerly and as a replayed graph, against the definitions."""
    P, Hkv, G, D, pages, width = 16, 2, 4, 64, 64, 8
    gen = torch.Generator().manual_seed(5)
    m = plain.Pool(6, width, pages, P)
    cache = torch.zeros(pages, Hkv, P, 2 * D, dtype=torch.float8_e4m3fn)
    scale = torch.zeros(pages, Hkv, 2)
    d = Device(m)
    dc, ds = cache.cuda(), scale.cuda()
    src, dst, moves = ints([-1] * 32), ints([-1] * 32), ints([0])
    fsrc, fdst = ints([-1] * 2), ints([-1] * 2)
    prompts = [50, 33]
    k1, v1 = (torch.randn(sum(prompts), Hkv, D, generator=gen).bfloat16() for _ in range(2))
    k2, v2 = (torch.randn(4, Hkv, D, generator=gen).bfloat16() for _ in range(2))
    q = torch.randn(6, Hkv * G, D, generator=gen).bfloat16()
    cu1, cu2 = [0, 50, 83, 83, 83, 83, 83], [0, 1, 2, 3, 4, 4, 4]
    outs = [(torch.zeros_like(q, device="cuda"), torch.zeros(6, Hkv * G, device="cuda")) for _ in range(3)]
    lists = {n: ints(v) for n, v in dict(r01=[0, 1], p=prompts, par=[0, 1], kid=[2, 3], r4=[0, 1, 2, 3],
                                         l4=[51, 34, 51, 34], r0=[0], zero=[0], cu1=cu1, cu2=cu2).items()}
    dk = [t.cuda() for t in (k1, v1, k2, v2, q)]
    args = (d.bt, d.sl, d.refs)

    def step():
        a = lists
        pkv.pages_reserve(*args, a["r01"], a["p"], P)
        pkv.gqa_kv_append_fp8(dk[0], dk[1], dc, ds, d.bt, d.sl, a["cu1"], P)
        pkv.paged_decode_attn_fp8(dk[4], dc, ds, d.bt, d.sl, None, 0, 0, 0.125, P, *outs[0])
        pkv.pages_fork(*args, a["par"], a["kid"], P, fsrc, fdst)
        pkv.pages_copy([dc, ds], fsrc, fdst)
        pkv.pages_reserve(*args, a["r4"], a["l4"], P)
        pkv.gqa_kv_append_fp8(dk[2], dk[3], dc, ds, d.bt, d.sl, a["cu2"], P)
        pkv.paged_decode_attn_fp8(dk[4], dc, ds, d.bt, d.sl, None, 20, 3, 0.125, P, *outs[1])
        pkv.pages_release(*args, a["r0"], a["zero"], P)
        pkv.pages_compact(*args, P, src, dst, moves)
        pkv.pages_copy([dc, ds], src, dst)
        pkv.paged_decode_attn_fp8(dk[4], dc, ds, d.bt, d.sl, None, 0, 0, 0.125, P, *outs[2])

    def expect():
        c, s = cache.double(), scale.double()

        def copy(a, b):
            for x, y in zip(a, b):
                if x >= 0:
                    c[y], s[y] = c[x].clone(), s[x].clone()

        def attend(window, first):
            t = torch.tensor(m.table, dtype=torch.int32)
            return plain.decode(q, c, s, t, torch.tensor(m.lens), None, window, first, 0.125, P, 2.0 ** -11)

        got = []
        m.reserve([0, 1], prompts)
        c, s = plain.append(k1, v1, c, s, torch.tensor(m.table), m.lens, cu1, P)
        got.append(attend(0, 0))
        copy(*m.fork([0, 1], [2, 3]))
        m.reserve([0, 1, 2, 3], [51, 34, 51, 34])
        c, s = plain.append(k2, v2, c, s, torch.tensor(m.table), m.lens, cu2, P)
        got.append(attend(20, 3))
        m.release([0], [0])
        a, b, _ = m.compact(32)
        copy(a, b)
        got.append(attend(0, 0))
        return got, c, s

    def compare(want):
        torch.cuda.synchronize()
        assert pkv.check_errors(0) == 0
        assert d.same(m)
        for (o, l), (wo, wl, tol, ltol) in zip(outs, want[0]):
            assert ((o.cpu().double() - wo).abs() <= tol).all()
            fin = wl > -math.inf
            assert torch.equal(l.cpu() > -math.inf, fin)
            assert ((l.cpu().double() - wl)[fin].abs() <= ltol[fin]).all()
        owned = [p for r, n in enumerate(m.lens) for p in m.table[r][:m.pages_of(n)]]
        assert torch.equal(ds.cpu().double()[owned], want[2][owned])
        assert torch.equal(dc.cpu().double()[owned], want[1][owned])

    step()
    want = expect()
    compare(want)
    for _ in range(2):  # the same run captured, from the same start
        d.bt.fill_(-1), d.sl.zero_(), d.refs.zero_()
        dc.view(torch.uint8).zero_(), ds.zero_()
        if _ == 0:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        graph.replay()
        compare(want)


def test_bf16_decode_right_after_a_page_call():
    """The attention kernels that read tables and lengths before their dependency wait see
    what a page call just wrote, call after call."""
    P, Hkv, pages = 16, 1, 4096
    kv = torch.randn(pages, Hkv, P, 256, device="cuda").bfloat16()
    q = torch.randn(2, 8, 128, device="cuda").bfloat16()
    bt = torch.full((2, 200), -1, dtype=torch.int32, device="cuda")
    sl, refs = ints([0, 0]), ints([0] * pages)
    rows, zero = ints([0, 1]), ints([0, 0])
    outs = [torch.zeros_like(q) for _ in range(2)]
    for i in range(1, 40):
        n = ints([i * 70, 3000 - i * 70])
        pkv.pages_release(bt, sl, refs, rows, zero, P)
        pkv.pages_reserve(bt, sl, refs, rows, n, P)
        pkv.paged_decode_attn(q, kv, bt, sl, None, 0, 0.09, P, 0, outs[0])
        torch.cuda.synchronize()
        pkv.paged_decode_attn(q, kv, bt, sl, None, 0, 0.09, P, 0, outs[1])
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1])
    assert pkv.check_errors(0) == 0
    assert pkv.check_counters(0) == 0


def test_bf16_append_and_decode_after_copied_pages_in_a_graph():
    """A copied page, a token appended to it and the decode that reads it, captured: the decode
    kernel's early reads see the copy."""
    P = 16
    kv = torch.randn(64, 1, P, 256, device="cuda").bfloat16()
    q = torch.randn(1, 8, 128, device="cuda").bfloat16()
    k, v = (torch.randn(1, 1, 128, device="cuda").bfloat16() for _ in range(2))
    bt = torch.arange(32, 64, dtype=torch.int32, device="cuda").view(1, 32)
    sl = ints([32 * P])
    src, dst = ints(list(range(32))), ints(list(range(32, 64)))
    out = torch.zeros_like(q)

    def step():
        pkv.pages_copy(kv, src, dst)
        pkv.paged_decode_attn(q, kv, bt, sl, None, 0, 0.09, P, 0, out)
        pkv.pages_copy(kv, src, dst)
        pkv.gqa_kv_append(k, v, kv, bt, sl, P)
        pkv.paged_decode_attn(q, kv, bt, sl, None, 0, 0.09, P, 0, out)

    step()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for i in range(20):
        kv[:32] = torch.randn(32, 1, P, 256, device="cuda").bfloat16()
        kv[32:] = float("nan")
        graph.replay()
        want = kv.clone()
        want[32:] = want[:32]
        want[63, 0, 15] = torch.cat([k[0, 0], v[0, 0]])
        ref = torch.zeros_like(q)
        torch.cuda.synchronize()
        pkv.paged_decode_attn(q, want, bt, sl, None, 0, 0.09, P, 0, ref)
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    assert pkv.check_errors(0) == 0
