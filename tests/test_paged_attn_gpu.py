"""GPU decode over an e4m3 cache with a scale per (page, kv head), and over a
bf16 cache with a window and first tokens (pkv_paged_decode_attn_fp8,
pkv_paged_window_attn), against the 64-bit definition, element by element
within the bounds of the kernel's roundings."""
import math

import pytest
import torch

import paged_kv_cache_30_gb300 as pkv
from tests import paged_plain as plain

pytestmark = pytest.mark.gpu

EDGE_LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 300, 1000]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    pkv.load_library()
    pkv.init(0)


def problem(seed, lens, Hkv, G, D, P, fp8, window=0, first=0, sinks=False, nhd=False, spread=3.0,
            wide=False):
    """Seeded CPU tensors.  Every slot that no request sees holds NaN (keys and values), and
    so do the scales of pages that hold no visible key; unused table entries are -1."""
    g = torch.Generator().manual_seed(seed)
    lens = torch.tensor(lens, dtype=torch.int32)
    # a wide table (requests could be long) rules out a cluster of blocks for each request
    B, width = len(lens), max(1, -(-int(lens.max()) // P)) + (9000 if wide else 1)
    see = [plain.visible(int(L), window, first) for L in lens]
    pages = [sorted(set((s // P).tolist())) for s in see]
    pool = sum(map(len, pages)) + 4
    order = torch.randperm(pool, generator=g)
    table = torch.full((B, width), -1, dtype=torch.int32)
    seen = torch.zeros(pool, P, dtype=torch.bool)
    used = torch.zeros(pool, dtype=torch.bool)
    at = 0
    for b, (s, pg) in enumerate(zip(see, pages)):
        for j in pg:
            table[b, j] = int(order[at])
            used[order[at]] = True
            at += 1
        if len(s):
            seen[table[b].long()[s // P], s % P] = True
    x = torch.randn(pool, Hkv, P, 2 * D, generator=g)
    if fp8:
        size = torch.exp2(torch.randint(-3, 4, (pool, Hkv, 2), generator=g).float()) \
            if spread else torch.ones(pool, Hkv, 2)
        codes = (x * 60).to(torch.float8_e4m3fn)
        codes = torch.where(seen[:, None, :, None], codes.view(torch.uint8),
                            torch.tensor(0x7f, dtype=torch.uint8)).view(torch.float8_e4m3fn)
        scale = torch.where(used[:, None, None], size / 60, torch.tensor(math.nan))
    else:
        codes = torch.where(seen[:, None, :, None], x, torch.tensor(math.nan)).bfloat16()
        scale = None
    if nhd:  # [pool, P, Hkv, 2D] storage seen as [pool, Hkv, P, 2D]
        codes = codes.view(torch.uint8 if fp8 else torch.bfloat16).transpose(1, 2).contiguous() \
            .transpose(1, 2).view(codes.dtype)
    q = torch.randn(B, Hkv * G, D, generator=g).bfloat16()
    sink = torch.randn(Hkv * G, generator=g) * 2 if sinks else None
    return dict(q=q, kv=codes, sc=scale, bt=table, sl=lens, sinks=sink, window=window, first=first,
                scale=1 / math.sqrt(D), P=P, fp8=fp8)


def run(pr, stream=None, lse=True, d=None):
    d = d or {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in pr.items()}
    if pr["kv"].stride(2) != pr["kv"].shape[3]:
        u = torch.uint8 if pr["fp8"] else torch.bfloat16
        d["kv"] = pr["kv"].view(u).transpose(1, 2).contiguous().cuda().transpose(1, 2).view(pr["kv"].dtype)
    out = torch.full_like(d["q"], math.nan)
    lse_t = torch.full(d["q"].shape[:2], math.nan, device="cuda") if lse else None
    call(d, out, lse_t, stream)
    torch.cuda.synchronize()
    return out.cpu(), lse_t.cpu() if lse else None


def call(d, out, lse, stream=None):
    if d["fp8"]:
        pkv.paged_decode_attn_fp8(d["q"], d["kv"], d["sc"], d["bt"], d["sl"], d["sinks"],
                                  d["window"], d["first"], d["scale"], d["P"], out, lse, stream)
    else:
        pkv.paged_window_attn(d["q"], d["kv"], d["bt"], d["sl"], d["sinks"], d["window"],
                              d["first"], d["scale"], d["P"], out, lse, stream)


def check(pr, out, lse):
    want, want_lse, tol, lse_tol = plain.decode(
        pr["q"], pr["kv"], pr["sc"], pr["bt"], pr["sl"], pr["sinks"], pr["window"], pr["first"],
        pr["scale"], pr["P"], 2.0 ** -11 if pr["fp8"] else 2.0 ** -8)
    far = (out.double() - want).abs() - tol
    assert out.isfinite().all()
    assert (far <= 0).all(), f"{far.max():.3e} past the bound at {far.argmax()}"
    if lse is not None:
        empty = want_lse == -math.inf
        assert torch.equal(lse == -math.inf, empty)
        far = (lse.double() - want_lse).abs()[~empty] - lse_tol[~empty]
        assert (far <= 0).all(), f"lse {far.max():.3e} past the bound"
    assert pkv.check_errors(0) == 0
    assert pkv.check_counters(0) == 0


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,Hkv,P", [(1, 3, 16), (4, 2, 32), (8, 1, 16), (8, 2, 64), (5, 2, 128),
                                     (16, 1, 32), (9, 2, 16)])
@pytest.mark.parametrize("wide", [False, True])
def test_head_layouts_and_edge_lengths(fp8, D, G, Hkv, P, wide):
    pr = problem(G * 100 + P + D, EDGE_LENS, Hkv, G, D, P, fp8, sinks=(G % 2 == 0), wide=wide)
    check(pr, *run(pr))


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("window,first", [(1, 0), (1, 1), (7, 3), (16, 4), (33, 17), (100, 64),
                                          (128, 128), (5000, 9), (64, 1000)])
@pytest.mark.parametrize("P", [16, 32])
def test_windows_and_first_tokens(fp8, window, first, P):
    pr = problem(window * 7 + first, EDGE_LENS, 2, 8, 128, P, fp8, window, first, sinks=True)
    check(pr, *run(pr))


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("window,first,D,G", [(1, 1, 128, 8), (20, 3, 64, 4), (100, 70, 128, 2)])
def test_windows_of_more_pairs_than_blocks_run_at_once(fp8, window, first, D, G):
    pr = problem(window, EDGE_LENS * 20, 2, G, D, 16, fp8, window, first, sinks=True)
    check(pr, *run(pr))


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("window,first,D,G", [(1, 1, 128, 8), (20, 3, 64, 4), (100, 70, 128, 2),
                                              (33, 17, 128, 16), (300, 9, 64, 12)])
def test_windows_of_more_pairs_than_two_waves(fp8, window, first, D, G):
    pr = problem(window + 3, EDGE_LENS * 40, 2, G, D, 16, fp8, window, first, sinks=True)
    check(pr, *run(pr))


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("B,L", [(1, 100), (1, 4000), (3, 2000), (40, 600), (57, 500), (100, 300), (228, 40)])
def test_parts_of_one_to_eight_blocks_a_pair(fp8, B, L):
    """Batches whose pairs get clusters of every size, lengths from none to the table's width."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, L + 1, (B,), generator=g).tolist()
    lens[-1] = L
    pr = problem(B, lens, 1 if B > 60 else 2, 8, 64, 16, fp8, sinks=True)
    check(pr, *run(pr))


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("D,G", [(128, 8), (64, 16)])
def test_long_and_ragged_batches_split_over_many_blocks(fp8, D, G):
    pr = problem(5, [5000, 1, 0, 4097, 16, 12001], 2, G, D, 16, fp8)
    check(pr, *run(pr))


@pytest.mark.parametrize("fp8", [True, False])
def test_many_short_requests(fp8):
    g = torch.Generator().manual_seed(9)
    lens = torch.randint(0, 70, (700,), generator=g).tolist()
    pr = problem(9, lens, 1, 4, 64, 16, fp8, sinks=True)
    check(pr, *run(pr))


MANY = [n for i in range(27) for n in EDGE_LENS]  # with 3 kv heads more pairs than two waves


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,P", [(1, 16), (5, 32), (8, 128), (16, 64)])
def test_head_layouts_of_many_requests(fp8, D, G, P):
    pr = problem(G + P, MANY, 3, G, D, P, fp8, sinks=(G % 2 == 0))
    check(pr, *run(pr))


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("D,G", [(128, 8), (64, 12)])
@pytest.mark.parametrize("lens,Hkv", [
    (MANY, 3),                                                     # more than two waves
    ([180 + i % 21 for i in range(300)], 1),                       # whole pairs, one a block
    ([180 + i % 21 if i % 50 else 0 for i in range(300)], 2),      # two a block, some of no key
    ([3000] + [200] * 299, 1)])                                    # one that is cut
def test_tables_wider_than_the_lengths(fp8, D, G, lens, Hkv):
    """The lengths, not the width of the table, choose how the work is cut."""
    pr = problem(28, lens, Hkv, G, D, 16, fp8, sinks=True, wide=True)
    check(pr, *run(pr))


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("D,G", [(128, 8), (64, 16)])
def test_long_requests_among_many_of_one_key(fp8, D, G):
    """The long ones are cut into dozens of parts, which one warp merges."""
    lens = [1] * 400 + [1000, 0, 990] + [1, 2] * 100 + [1008] + [1] * 100
    pr = problem(23, lens, 2, G, D, 16, fp8, sinks=True)
    check(pr, *run(pr))


@pytest.mark.parametrize("fp8", [True, False])
def test_many_requests_strided_and_without_lse(fp8):
    pr = problem(24, MANY, 3, 5, 128, 16, fp8, nhd=True)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in pr.items()}
    B, Hq, D = pr["q"].shape
    hold = torch.full((B, Hq + 1, D + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, 2 * Hq), 7.0, device="cuda")
    call(d, hold[:, :Hq, :D], lse[:, ::2])
    torch.cuda.synchronize()
    check(pr, hold[:, :Hq, :D].cpu(), lse[:, ::2].cpu())
    assert (hold[:, Hq:] == 7).all() and (hold[:, :, D:] == 7).all() and (lse[:, 1::2] == 7).all()
    first = hold[:, :Hq, :D].clone()
    hold.fill_(7.0)
    call(d, hold[:, :Hq, :D], None)
    torch.cuda.synchronize()
    assert torch.equal(hold[:, :Hq, :D], first)


@pytest.mark.parametrize("fp8", [True, False])
def test_many_requests_replayed_beside_eager_calls(fp8):
    """Every run gives the same bits, a captured one with new lengths gives theirs, and the
    counters that the parts of a request share are back at zero."""
    pr = problem(25, MANY, 3, 8, 64, 16, fp8, sinks=True)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in pr.items()}
    want = run(pr, d=d)
    check(pr, *want)
    out, lse = torch.empty_like(d["q"]), torch.empty(d["q"].shape[:2], device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(d, out, lse, torch.cuda.current_stream())
    for _ in range(10):
        out.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want[0]) and torch.equal(lse.cpu(), want[1])
        again = run(pr, d=d)
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
    pr["sl"] = pr["sl"] // 2
    d["sl"].copy_(pr["sl"])
    graph.replay()
    torch.cuda.synchronize()
    check(pr, out.cpu(), lse.cpu())


@pytest.mark.parametrize("fp8", [True, False])
def test_bad_entries_among_many_requests(fp8):
    pr = problem(26, MANY, 3, 4, 128, 16, fp8, sinks=True)
    want = run(pr)
    rows = [b for b, n in enumerate(MANY) if n >= 300][::5]
    for i, b in enumerate(rows):
        pr["bt"][b, 3] = pr["kv"].shape[0] if i % 2 else -7
    out, lse = run(pr)
    with pytest.raises(pkv.PkvError) as e:
        pkv.check_errors(0)
    assert e.value.code == -7
    check(pr, out, lse)
    rest = [b for b in range(len(MANY)) if b not in rows]
    assert torch.equal(out[rest], want[0][rest]) and torch.equal(lse[rest], want[1][rest])


def test_many_requests_in_a_small_workspace():
    """No room for the partials of every warp: blocks share the work, in fewer places."""
    pr = problem(27, MANY, 3, 8, 128, 16, True, sinks=True)
    torch.cuda.synchronize()
    pkv.shutdown()
    try:
        pkv.init(0, 100 * 2 * (8 * 128 + 24) * 4)
        check(pr, *run(pr))
    finally:
        pkv.shutdown()
        pkv.init(0)
    check(pr, *run(pr))


def test_largest_batch_and_one_request_of_no_key():
    pr = problem(2, [1 + i % 3 for i in range(2048)], 1, 1, 64, 16, True)
    check(pr, *run(pr))
    pr = problem(3, [0], 1, 8, 128, 16, True, sinks=True)
    out, lse = run(pr)
    assert (out == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("fp8", [True, False])
def test_token_stride_of_an_nhd_cache(fp8):
    pr = problem(4, EDGE_LENS, 3, 8, 128, 32, fp8, 40, 5, nhd=True)
    check(pr, *run(pr))


@pytest.mark.parametrize("fp8", [True, False])
def test_strided_query_output_tables_and_scales(fp8):
    pr = problem(6, EDGE_LENS, 2, 4, 128, 16, fp8)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in pr.items()}
    B, Hq, D = pr["q"].shape
    wide = torch.full((B, Hq + 3, D + 16), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:, 1:Hq + 1, 8:D + 8] = d["q"]
    d["q"] = wide[:, 1:Hq + 1, 8:D + 8]
    table = torch.full((B, pr["bt"].shape[1] + 5), 1 << 30, dtype=torch.int32, device="cuda")
    table[:, :-5] = d["bt"]
    d["bt"] = table[:, :-5]
    if fp8:
        sc = torch.full((pr["sc"].shape[0], 5, 4), math.nan, device="cuda")
        sc[:, 1:3, 2:] = d["sc"]
        d["sc"] = sc[:, 1:3, 2:]
    hold = torch.full((B, Hq + 1, D + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, 2 * Hq), 7.0, device="cuda")
    call(d, hold[:, :Hq, :D], lse[:, ::2])
    torch.cuda.synchronize()
    check(pr, hold[:, :Hq, :D].cpu(), lse[:, ::2].cpu())
    assert (hold[:, Hq:] == 7).all() and (hold[:, :, D:] == 7).all() and (lse[:, 1::2] == 7).all()


def test_without_lse():
    pr = problem(7, EDGE_LENS, 2, 8, 128, 16, True)
    out, _ = run(pr, lse=False)
    check(pr, out, None)


def test_scales_far_apart_between_pages():
    """Values of one page 2^40 times another's: the large page's weight is small, the output is
    right relative to its own bound; a page of scale 0 adds nothing to the output."""
    pr = problem(8, [200, 33, 64], 1, 8, 128, 16, True, spread=0)
    pr["sc"][int(pr["bt"][0, 2]), 0, 1] *= 2.0 ** 20
    pr["sc"][int(pr["bt"][0, 5]), 0, 1] *= 2.0 ** -20
    pr["sc"][int(pr["bt"][0, 7]), 0, 0] = 0.0
    pr["sc"][int(pr["bt"][1, 1]), 0, 1] = 0.0
    pr["sc"][:, :, 0] *= 3.7  # no power of two
    check(pr, *run(pr))
    pr["sc"][:, :, 1] = 0.0
    pr["sc"][torch.isnan(pr["sc"])] = 0.0
    out, lse = run(pr)
    assert (out == 0).all() and lse.isfinite().all()


def test_queries_of_any_magnitude():
    """The query enters scaled to fp16's range by a power of two: rows of 2^60 and of 2^-60
    next to ordinary ones, and a row of zeros."""
    pr = problem(10, [70, 70, 70, 70], 1, 4, 128, 16, True)
    size = torch.tensor([2.0 ** 60, 2.0 ** -60, 0.0, 1.0])[:, None, None]
    pr["q"] = (pr["q"].float() * size).bfloat16()
    pr["sc"][pr["bt"][0, :5].long(), 0, 0] *= 2.0 ** -62
    check(pr, *run(pr))


@pytest.mark.parametrize("fp8", [True, False])
def test_bad_entries_read_as_zero_pages_and_are_flagged(fp8):
    pr = problem(11, [50, 40], 1, 8, 128, 16, fp8)
    pr["bt"][0, 1] = -1
    pr["bt"][1, 0] = 1 << 20
    out, lse = run(pr)
    with pytest.raises(pkv.PkvError) as e:
        pkv.check_errors(0)
    assert e.value.code == -7
    check(pr, out, lse)


def test_lengths_past_the_table_are_clamped_and_flagged():
    pr = problem(12, [64, 40], 1, 8, 128, 16, True)
    want = run(pr)
    pr["bt"] = pr["bt"][:, :4].contiguous()
    pr["sl"][0] = 100000
    out, lse = run(pr)
    with pytest.raises(pkv.PkvError):
        pkv.check_errors(0)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_same_results_every_time_and_on_another_stream():
    pr = problem(13, [9000, 3000, 17, 700], 2, 8, 128, 16, True, sinks=True)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in pr.items()}
    first = run(pr, d=d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        a, b = run(pr, d=d), run(pr, stream=side, d=d)
        for o in (a, b):
            assert torch.equal(o[0], first[0]) and torch.equal(o[1], first[1])
    check(pr, *first)


def test_agrees_with_the_bf16_decode_call():
    """Without first tokens the window call computes what pkv_paged_decode_attn does: both
    within the bound of the definition, and so within twice that of each other."""
    pr = problem(14, EDGE_LENS, 2, 8, 128, 16, False, window=50, sinks=True)
    out, lse = run(pr)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in pr.items()}
    o2, l2 = torch.empty_like(d["q"]), torch.empty(d["q"].shape[:2], device="cuda")
    pkv.paged_decode_attn(d["q"], d["kv"], d["bt"], d["sl"], d["sinks"], 50, d["scale"], 16, 0, o2, l2)
    torch.cuda.synchronize()
    check(pr, out, lse)
    check(pr, o2.cpu(), l2.cpu())


def test_captured_graphs_share_the_workspace_and_see_new_lengths():
    a = problem(15, [4000, 900, 33], 2, 8, 128, 16, True)
    b = problem(16, [2500, 1, 800, 64], 1, 8, 128, 16, False, 300, 4)
    da, db = ({k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in p.items()} for p in (a, b))
    outs = [(torch.zeros_like(d["q"]), torch.zeros(d["q"].shape[:2], device="cuda")) for d in (da, db)]
    run(a)
    graphs = []
    for d, (o, l) in zip((da, db), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(d, o, l)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    check(a, outs[0][0].cpu(), outs[0][1].cpu())
    check(b, outs[1][0].cpu(), outs[1][1].cpu())
    da["sl"].copy_(torch.tensor([37, 0, 20], dtype=torch.int32))
    graphs[0].replay()
    torch.cuda.synchronize()
    short = dict(a, sl=torch.tensor([37, 0, 20], dtype=torch.int32))
    check(short, outs[0][0].cpu(), outs[0][1].cpu())


def far_cache(fp8):
    """A cache of more than 2^32 bytes (and scales) of which a few pages, near its end, are used."""
    P, Hkv, D = 32, 8, 128
    pool = (5 << 30) // (Hkv * P * 2 * D * (1 if fp8 else 2))
    pr = problem(21, [300, 77, 310], Hkv, 2, D, P, fp8, sinks=True)
    n = pr["kv"].shape[0]
    kv = torch.empty(pool, Hkv, P, 2 * D, dtype=pr["kv"].dtype, device="cuda")
    kv[-n:] = pr["kv"].cuda()
    d = {k: v.cuda() if isinstance(v, torch.Tensor) and k != "kv" else v for k, v in pr.items()}
    d["kv"] = kv
    d["bt"] = torch.where(d["bt"] >= 0, d["bt"] + (pool - n), d["bt"])
    if fp8:
        d["sc"] = torch.zeros(pool, Hkv, 2, device="cuda")
        d["sc"][-n:] = pr["sc"].cuda()
    return pr, d, pool, n


@pytest.mark.parametrize("fp8", [True, False])
def test_offsets_past_32_bits(fp8):
    pr, d, pool, n = far_cache(fp8)
    out = torch.full_like(d["q"], math.nan)
    lse = torch.full(d["q"].shape[:2], math.nan, device="cuda")
    call(d, out, lse)
    torch.cuda.synchronize()
    check(pr, out.cpu(), lse.cpu())
    # pages moved to the front of the pool, and there attended
    src = torch.arange(pool - n, pool, dtype=torch.int32, device="cuda")
    dst = torch.arange(n, dtype=torch.int32, device="cuda")
    pkv.pages_copy([d["kv"], d["sc"]] if fp8 else d["kv"], src, dst)
    d["bt"] = torch.where(d["bt"] >= 0, d["bt"] - (pool - n), d["bt"])
    out2 = torch.full_like(out, math.nan)
    call(d, out2, lse)
    torch.cuda.synchronize()
    assert torch.equal(out, out2)


def test_append_past_32_bits():
    pr, d, pool, n = far_cache(True)
    T = 5
    k, v = (torch.randn(T, 8, 128, device="cuda").bfloat16() for _ in range(2))
    sl = torch.tensor([2 * T], dtype=torch.int32, device="cuda")
    d["sc"][-1] = 2.0 ** -9
    bt = torch.tensor([[pool - 1]], dtype=torch.int32, device="cuda")
    before = d["kv"][:-1].view(torch.uint8)[::997].clone()
    pkv.gqa_kv_append_fp8(k, v, d["kv"], d["sc"], bt, sl, None, 32)
    torch.cuda.synchronize()
    got = d["kv"][-1, :, T:2 * T].float() * d["sc"][-1][:, None, :].repeat_interleave(128, 2)
    want = torch.cat([k, v], 2).transpose(0, 1).float()
    # e4m3 of x / s is within 2^-4 of x, or 2^-10 s where x / s is below 2^-6
    far = (got - want).abs() - want.abs() * 2.0 ** -4 \
        - 2.0 ** -10 * d["sc"][-1][:, None, :].repeat_interleave(128, 2)
    assert (far <= 0).all()
    assert torch.equal(d["kv"][:-1].view(torch.uint8)[::997], before)


def test_host_memory_is_refused():
    pr = problem(30, [20, 3], 1, 8, 64, 16, True)
    out = torch.empty_like(pr["q"])
    with pytest.raises(pkv.PkvError):
        call(pr, out, None)
    with pytest.raises(pkv.PkvError) as e:
        call(pr, out, None, torch.cuda.current_stream())
    assert e.value.code == -1


def test_a_small_workspace_runs_on_fewer_blocks():
    """Room for partials of a dozen blocks, then for none: the first is slower and right, the
    second refused; a cluster launch needs none."""
    pr = problem(31, [3000, 1, 900, 0, 64, 2222], 2, 8, 128, 16, True, sinks=True, wide=True)
    few = problem(32, [100, 300, 0], 1, 8, 128, 16, True)
    torch.cuda.synchronize()
    pkv.shutdown()
    try:
        pkv.init(0, 12 * 2 * (8 * 128 + 24) * 4)
        check(pr, *run(pr))
        pkv.shutdown()
        pkv.init(0, 1024)
        with pytest.raises(pkv.PkvError) as e:
            run(pr)
        assert e.value.code == -4
        check(few, *run(few))
    finally:
        pkv.shutdown()
        pkv.init(0)
    check(pr, *run(pr))
