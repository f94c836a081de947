"""GPU decode of groups of requests that share their first tokens (pkv_paged_prefix_attn,
pkv_paged_prefix_attn_fp8) against the 64-bit definition on each request's own row, element by
element within the bounds of the kernels' roundings."""
import math
import threading

import pytest
import torch

import paged_kv_cache_30_gb300 as pkv
from tests import prefix_plain as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    pkv.load_library()
    pkv.init(0)


def upload(pr):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in pr.items()}


def call(d, out, lse, stream=None):
    if d["fp8"]:
        pkv.paged_prefix_attn_fp8(d["q"], d["kv"], d["sc"], d["bt"], d["sl"], d["cu"], d["shared"],
                                  d["sinks"], d["scale"], d["P"], out, lse, stream)
    else:
        pkv.paged_prefix_attn(d["q"], d["kv"], d["bt"], d["sl"], d["cu"], d["shared"], d["sinks"],
                              d["scale"], d["P"], out, lse, stream)


def run(pr, stream=None, d=None):
    d = d or upload(pr)
    out = torch.full_like(d["q"], math.nan)
    lse = torch.full(d["q"].shape[:2], math.nan, device="cuda")
    call(d, out, lse, stream)
    torch.cuda.synchronize()
    return out, lse


def check(pr, out, lse, flags=0):
    want, want_lse, tol, lse_tol = plain.decode(pr, "cuda")
    rows = slice(pr["lead"], len(pr["sl"]) - pr["tail"])
    for pad in (slice(0, pr["lead"]), slice(len(pr["sl"]) - pr["tail"], None)):
        assert out[pad].isnan().all()  # not written
        assert lse is None or lse[pad].isnan().all()
    if flags:
        with pytest.raises(pkv.PkvError, match=f"0x{flags:x}"):
            pkv.check_errors(0)
    else:
        assert pkv.check_errors(0) == 0
    assert pkv.check_counters(0) == 0
    far = ((out.double() - want).abs() - tol)[rows]
    assert out[rows].isfinite().all()
    assert (far <= 0).all(), f"{int((far > 0).sum())} of {far.numel()}, {far.max():.3e} past the bound"
    if lse is not None:
        empty = (want_lse == -math.inf)[rows]
        assert torch.equal(lse[rows] == -math.inf, empty)
        far = (lse.double() - want_lse).abs()[rows][~empty] - lse_tol[rows][~empty]
        assert (far <= 0).all(), f"lse {far.max():.3e} past the bound"


BOTH = pytest.mark.parametrize("fp8", [False, True])


@BOTH
@pytest.mark.parametrize("D", [128, 64])
def test_one_tile(fp8, D):
    pr = plain.problem(1, [(128, [130, 140, 129, 150])], 1, 4, D, 16, fp8)
    check(pr, *run(pr))


@BOTH
@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("G,Hkv,P,shared", [(1, 3, 16, 200), (4, 2, 32, 1000), (8, 1, 16, 257),
                                            (8, 2, 64, 96), (5, 2, 128, 700), (16, 1, 32, 2049),
                                            (9, 2, 16, 31), (7, 1, 16, 16)])
def test_head_layouts(fp8, D, G, Hkv, P, shared):
    own = [1, 2, 15, 16, 17, 40, 130]
    pr = plain.problem(G + P + D, [(shared, [shared + n for n in own])], Hkv, G, D, P, fp8,
                       sinks=G % 2 == 0)
    check(pr, *run(pr))


@BOTH
@pytest.mark.parametrize("n,G", [(16, 8), (17, 8), (32, 8), (33, 8), (70, 8), (40, 5), (33, 16), (150, 7)])
def test_blocks_of_rows(fp8, n, G):
    """Up to 128 rows a group, up to 256, and several blocks of them."""
    pr = plain.problem(n + G, [(900, [901 + i % 50 for i in range(n)])], 2, G, 128, 16, fp8, sinks=True)
    check(pr, *run(pr))


@BOTH
@pytest.mark.parametrize("boxes", range(1, 20, 3))
def test_shared_tokens_that_end_inside_a_tile(fp8, boxes):
    S = 16 * boxes
    pr = plain.problem(boxes, [(S + 5, [S + 5, S + 6, S + 20]), (S, [S + 1] * 20)], 2, 8, 64, 32, fp8)
    check(pr, *run(pr))


@BOTH
@pytest.mark.parametrize("D,Hkv,S", [(128, 1, 30000), (64, 2, 41000), (128, 8, 9000)])
def test_long_prefixes_cut_among_many_blocks(fp8, D, Hkv, S):
    pr = plain.problem(S, [(S, [S + 1, S + 700, S + 33, S + 4])], Hkv, 8, D, 16, fp8, sinks=True)
    check(pr, *run(pr))
    pr = plain.problem(S + 1, [(S // 4, [S // 4 + 1 + i for i in range(40)])], Hkv, 8, D, 16, fp8)
    check(pr, *run(pr))


@BOTH
@pytest.mark.parametrize("D,P", [(64, 16), (128, 32), (64, 128)])
def test_long_shares_of_many_blocks_of_rows(fp8, D, P):
    """Shares of more than 32 tiles, cut elsewhere for each block of rows: their tiles come in
    turned order, with the unit's last tile, which is cut short, among them."""
    pr = plain.problem(P, [(11237, [11238 + 3 * i for i in range(100)]), (6100, [6101 + i for i in range(70)])],
                       8, 16, D, P, fp8)
    check(pr, *run(pr))


GROUPS = [(500, [0, 510, 501, 700]), (0, [40, 30]), (1000, [1300]), (64, [0, 0]), (300, []),
          (256, [257] * 9), (90, [20, 95, 200]), (48, [48, 48, 48]), (5, [6, 9]), (33, [0, 35, 0])]


@BOTH
@pytest.mark.parametrize("lead,tail", [(0, 0), (3, 2)])
def test_groups_of_all_kinds(fp8, lead, tail):
    """Idle requests, nobody to share with, nothing shared, requests shorter than what is
    shared or as long, empty groups, padding rows."""
    for seed, (D, Hkv, G, P) in enumerate([(128, 2, 8, 16), (64, 1, 5, 32)]):
        pr = plain.problem(seed, GROUPS, Hkv, G, D, P, fp8, sinks=True, lead=lead, tail=tail)
        check(pr, *run(pr))


@BOTH
def test_many_groups(fp8):
    g = torch.Generator().manual_seed(5)
    n = torch.randint(1, 5, (300,), generator=g).tolist()
    S = torch.randint(0, 600, (300,), generator=g).tolist()
    pr = plain.problem(6, [(s, [s + 1 + (7 * i + s) % 90 for i in range(k)]) for s, k in zip(S, n)], 4, 2,
                       64, 16, fp8)
    check(pr, *run(pr))


@BOTH
def test_the_largest_batch(fp8):
    pr = plain.problem(7, [(64, [65 + i % 30 for i in range(1000)]), (0, [1 + i % 9 for i in range(48)]),
                           (128, [130] * 1000)], 2, 2, 64, 16, fp8)
    check(pr, *run(pr))


@BOTH
def test_many_short_requests_of_their_own(fp8):
    """More pairs than two waves of blocks: the part behind the shared tokens is dealt to warps."""
    for D, G in ((128, 8), (64, 4), (128, 16)):
        pr = plain.problem(8, [(300, [301 + (13 * i) % 200 for i in range(90)]) for _ in range(3)], 8, G, D,
                           16, fp8, sinks=True)
        check(pr, *run(pr))


@BOTH
def test_shared_pages_are_read_through_the_first_row_alone(fp8):
    pr = plain.problem(9, [(320, [0, 330, 400, 321, 500])], 2, 8, 128, 16, fp8)
    d = upload(pr)
    d["bt"][2:, :20] = -1  # entries that would be flagged if they were read
    d["bt"][0] = -1
    check(pr, *run(pr, d=d))


@BOTH
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1.7])
def test_scales_of_any_sign(fp8, scale):
    pr = plain.problem(10, [(400, [401, 420, 500])], 2, 8, 64, 16, fp8)
    pr["scale"] = scale
    check(pr, *run(pr))


@BOTH
@pytest.mark.parametrize("scale", [0.0, -0.0, 0.75 * 2.0 ** -126, 2.0 ** -120])
def test_small_scales_of_large_products(fp8, scale):
    """Products of up to 2^125: a scale of 0 makes equal weights of them, one below the smallest
    normal value the weights that it should."""
    pr = plain.problem(46, [(500, [501, 520, 700]), (130, [131] * 20)], 2, 8, 128, 16, fp8)
    pr["scale"] = scale
    if fp8:
        pr["q"] *= 2.0 ** 100
        pr["sc"][..., 0] *= 2.0 ** 15
    else:
        pr["q"] *= 2.0 ** 59
        pr["kv"][..., :128] *= 2.0 ** 59
    out, lse = run(pr)
    check(pr, out, lse)
    d = upload(pr)
    d["q"][1, 3, 7] = math.inf  # times 0 is no number
    bad, _ = run(pr, d=d)
    if scale == 0:
        assert bad[1, 3].isnan().all()
    bad[1, 3] = out[1, 3]
    assert torch.equal(bad, out)


def test_scales_far_apart_between_pages():
    """One page's keys outweigh the others', or its values do, by factors up to 2^40."""
    for seed in range(4):
        pr = plain.problem(20 + seed, [(640, [641, 700, 900] * 7)], 2, 4, 128, 16, True, spread=6)
        page = pr["bt"][0, 3 + seed].long()
        pr["sc"][page, :, 1] *= 2.0 ** 40 if seed % 2 else 2.0 ** -40
        pr["sc"][pr["bt"][0, 30].long(), :, 0] = 0.0
        check(pr, *run(pr))


def test_weights_of_any_size_keep_their_bits():
    """A first token outweighs all others by 2^60 and has no value: what the others add is
    right relative to itself."""
    for fp8 in (False, True):
        pr = plain.problem(30, [(2000, [2001, 2050, 2300])], 1, 8, 128, 16, fp8, spread=0)
        pr["q"][..., 0] = 64
        kv, page = pr["kv"].float(), int(pr["bt"][0, 0])
        kv[..., 0] = torch.where(kv[..., 0].isnan(), kv[..., 0], 0.0)
        kv[page, :, 0, 0] = 448 if fp8 else 7.5
        kv[page, :, 0, 128:] = 0
        pr["kv"] = kv.to(pr["kv"].dtype)
        check(pr, *run(pr))


@BOTH
def test_nan_of_one_query_stays_in_its_row(fp8):
    pr = plain.problem(11, [(500, [501 + i for i in range(20)])], 2, 8, 128, 16, fp8)
    d = upload(pr)
    good, _ = run(pr, d=d)
    d["q"][3, 5, 7] = math.nan
    bad, lse = run(pr, d=d)
    assert bad[3, 5].isnan().all() and lse[3, 5].isnan()
    bad[3, 5] = good[3, 5]
    assert torch.equal(bad, good)


@BOTH
def test_strides_and_no_lse(fp8):
    pr = plain.problem(12, [(200, [201, 230, 300]), (90, [100, 95])], 2, 4, 64, 16, fp8, sinks=True)
    want, _ = run(pr)
    d = upload(pr)
    q = torch.zeros(5, 16, 72, dtype=torch.bfloat16, device="cuda")[:, ::2, :64]
    q.copy_(d["q"])
    u = torch.uint8 if fp8 else torch.bfloat16
    d["kv"] = pr["kv"].view(u).transpose(1, 2).contiguous().cuda().transpose(1, 2).view(pr["kv"].dtype)
    bt = torch.full((5, d["bt"].shape[1] + 3), -1, dtype=torch.int32, device="cuda")[:, :-3]
    d["q"], d["bt"] = q, bt.copy_(d["bt"])
    if fp8:
        sc = torch.zeros(*pr["sc"].shape[:2], 4, device="cuda")[..., :2]
        d["sc"] = sc.copy_(d["sc"])
    out = torch.full((5, 8, 136), math.nan, dtype=torch.bfloat16, device="cuda")
    call(d, out[..., :64], None)
    torch.cuda.synchronize()
    assert torch.equal(out[..., :64], want) and out[..., 64:].isnan().all()
    pkv.check_errors(0)


@BOTH
def test_bad_entries_lengths_and_offsets_are_flagged(fp8):
    pr = plain.problem(13, [(320, [330, 400, 321])], 2, 8, 128, 16, fp8)
    for entry in (-1, pr["kv"].shape[0]):
        for b in range(3):
            pr["bt"][b, 4] = entry  # a shared page: reads as zeros
        check(pr, *run(pr), flags=1)
    pr = plain.problem(14, [(320, [330, 400, 321])], 2, 8, 128, 16, fp8)
    pr["sl"][1] = 5000
    d = upload(pr)
    pr["sl"][1] = pr["bt"].shape[1] * 16
    pr["kv"] = pr["kv"].view(torch.uint8).clone().view(pr["kv"].dtype)
    hole = pr["kv"].view(torch.uint8 if fp8 else torch.int16)
    hole[torch.where(pr["kv"].float().isnan())] = 0
    d["kv"] = pr["kv"].cuda()
    if fp8:
        pr["sc"] = pr["sc"].nan_to_num(0.0)
        d["sc"] = pr["sc"].cuda()
    check(pr, *run(pr, d=d), flags=2)
    for cu in ([0, 3, 2], [-1, 2, 3], [0, 2, 4]):
        pr = plain.problem(15, [(320, [330, 400]), (16, [321])], 2, 8, 128, 16, fp8)
        d = upload(pr)
        d["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        check(pr, *run(pr, d=d), flags=64)


@BOTH
def test_agrees_with_the_calls_that_share_nothing(fp8):
    pr = plain.problem(16, [(1024, [1030, 1500, 2000, 1025]), (0, [800, 3])], 4, 8, 128, 16, fp8, sinks=True)
    got, lse = run(pr)
    d = upload(pr)
    out, lse2 = torch.empty_like(d["q"]), torch.empty_like(lse)
    if fp8:
        pkv.paged_decode_attn_fp8(d["q"], d["kv"], d["sc"], d["bt"], d["sl"], d["sinks"], 0, 0, d["scale"],
                                  16, out, lse2)
    else:
        pkv.paged_window_attn(d["q"], d["kv"], d["bt"], d["sl"], d["sinks"], 0, 0, d["scale"], 16, out, lse2)
    check(pr, out, lse2)
    check(pr, got, lse)


@pytest.mark.parametrize("D,rows", [(128, 8), (64, 8), (128, 48), (64, 136)])
def test_units_of_one_tile_with_queries_of_every_size(D, rows):
    """An e4m3 query row's power of two lies where the second slot leaves its m and l, which comes
    right behind in a unit of one step; the next unit's scales come there too.  Units of up to 128
    rows and of more, one tile each, several a block; rows of sizes 2^-20 to 2^6, whose weights go
    wrong with another row's power of two."""
    G = 8
    n = max(2, rows // G)
    groups = [(16 * (1 + i % 8), [16 * (1 + i % 8) + 1 + (i + j) % 5 for j in range(n)])
              for i in range(min(2000 // n, 300))]
    pr = plain.problem(45, groups, 4, G, D, 16, True, sinks=True)
    size = torch.arange(len(pr["sl"]) * 4 * G).view(len(pr["sl"]), 4 * G, 1) * 7 % 27 - 20
    pr["q"] = (pr["q"].float() * torch.exp2(size.float())).bfloat16()
    d = upload(pr)
    outs = [torch.empty_like(d["q"]) for _ in range(40)]
    for out in outs:
        call(d, out, None)
    torch.cuda.synchronize()
    assert all(torch.equal(out, outs[0]) for out in outs)
    # Where a sink passes a row's largest score by 128 (log2), 2^(sink - m) is an infinity in 32 bits
    # and the output 0, where it is sum_j 2^(x_j - sink) v_j <= 133 keys 2^-128 60 < 2^-115: values
    # are below 448 2^3 / 60 < 60.  (Outputs below 2^-126 lose bits as well.)
    want, _, tol, _ = plain.decode(pr, "cuda")
    far = (outs[0].double() - want).abs() - tol - 2.0 ** -115
    assert (far <= 0).all(), f"{int((far > 0).sum())} of {far.numel()}, {far.max():.3e} past the bound"
    assert pkv.check_errors(0) == 0 and pkv.check_counters(0) == 0


def test_captured_graphs_share_the_workspace_and_see_new_lengths():
    a = plain.problem(17, [(700, [701, 730, 900, 710]), (90, [95, 99])], 2, 8, 128, 16, True)
    b = plain.problem(18, [(1500, [1501 + i for i in range(40)])], 2, 8, 64, 32, False)
    da, db = upload(a), upload(b)
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
    check(a, *outs[0])
    check(b, *outs[1])
    for lens, shared in (([701, 0, 703, 705, 0, 0], [700, 90]), ([30, 20, 17, 700, 95, 1], [16, 0])):
        for d, pr in ((da, a),):
            pr["sl"], pr["shared"] = torch.tensor(lens).int(), torch.tensor(shared).int()
            d["sl"].copy_(pr["sl"])
            d["shared"].copy_(pr["shared"])
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        check(a, *outs[0])
        check(b, *outs[1])


@BOTH
def test_same_bits_every_time_back_to_back_and_on_another_stream(fp8):
    pr = plain.problem(19, [(3000, [3001 + 9 * i for i in range(36)]), (400, [420, 500])], 2, 8, 128, 16, fp8)
    d = upload(pr)
    outs = [torch.empty_like(d["q"]) for _ in range(8)]
    for o in outs:  # each call's first grid may start under the one before it
        call(d, o, None)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs.append(torch.empty_like(d["q"]))
    call(d, outs[-1], None, s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, outs[0]) for o in outs)
    check(pr, outs[0], None)


def test_calls_of_three_threads():
    """Each on a stream of its own, with parts, counters and the counter of shares in the one
    workspace: every result is what the call gives alone."""
    jobs = []
    for seed, fp8, groups in ((41, False, [(5000, [5001 + 7 * i for i in range(20)]), (0, [3000])]),
                              (42, True, [(700, [710, 900, 3000]), (9000, [9001, 9500])]),
                              (43, False, [(33, [40] * 50), (128, [129, 4000])])):
        d = upload(plain.problem(seed, groups, 2, 8, 128, 16, fp8))
        want = torch.empty_like(d["q"])
        call(d, want, None)
        outs = [torch.full_like(d["q"], math.nan) for _ in range(40)]
        jobs.append((d, want, outs, torch.cuda.Stream()))
    torch.cuda.synchronize()
    failed, start = [], threading.Barrier(len(jobs))

    def work(d, want, outs, stream):
        try:
            start.wait()
            for out in outs:
                call(d, out, None, stream)
        except Exception as e:  # noqa: BLE001 (shown below)
            failed.append(e)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for _, want, outs, _ in jobs:
        assert all(torch.equal(out, want) for out in outs)
    assert pkv.check_errors(0) == 0
    assert pkv.check_counters(0) == 0


@BOTH
def test_one_request_of_many_own_tokens_beside_short_ones(fp8):
    """Own tokens of very unequal length: blocks that begin early take several shares in turn."""
    pr = plain.problem(44, [(160, [161, 20000, 170, 162]), (64, [65, 66, 6000])], 4, 4, 128, 16, fp8,
                       sinks=True)
    check(pr, *run(pr))


@BOTH
def test_offsets_past_32_bits(fp8):
    pr = plain.problem(21, [(300, [301, 377, 310])], 8, 2, 128, 32, fp8, sinks=True)
    pool = (5 << 30) // (8 * 32 * 256 * (1 if fp8 else 2))
    n, d = pr["kv"].shape[0], upload(pr)
    kv = torch.empty(pool, *pr["kv"].shape[1:], dtype=pr["kv"].dtype, device="cuda")
    kv[-n:] = d["kv"]
    d["kv"], d["bt"] = kv, torch.where(d["bt"] >= 0, d["bt"] + (pool - n), d["bt"])
    if fp8:
        sc = torch.zeros(pool, 8, 2, device="cuda")
        sc[-n:] = d["sc"]
        d["sc"] = sc
    check(pr, *run(pr, d=d))


def test_a_small_workspace():
    pr = plain.problem(31, [(3000, [3001, 3002, 4000, 3100])], 2, 8, 128, 16, True, sinks=True)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    need = 4 * 16 + 4 * 16 * (2 * 128 * 4 + 24) + sms * 256 * (128 * 4 + 8)
    torch.cuda.synchronize()
    pkv.shutdown()
    try:
        pkv.init(0, need + 3 * 2 * (8 * 128 + 24) * 4 + 256)
        check(pr, *run(pr))
        pkv.shutdown()
        pkv.init(0, need)
        with pytest.raises(pkv.PkvError) as e:
            run(pr)
        assert e.value.code == -4
    finally:
        pkv.shutdown()
        pkv.init(0)
    check(pr, *run(pr))


def test_a_prompt_forked_and_continued():
    """The calls of a served prompt together: pages reserved, the prompt normed, rotated and
    appended, forked, each sample's next token appended, all samples attended to at once."""
    from tests import rope_plain
    g = torch.Generator().manual_seed(40)
    Hq, Hkv, D, P, L, n = 16, 2, 128, 16, 333, 5
    rows, W, pool = n + 1, 30, 80
    bt = torch.full((rows, W), -1, dtype=torch.int32, device="cuda")
    sl = torch.zeros(rows, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pool, dtype=torch.int32, device="cuda")
    kv = torch.full((pool, Hkv, P, 2 * D), math.nan, dtype=torch.bfloat16, device="cuda")
    table = pkv.rope_table(D)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")

    def tokens(T):
        return [torch.randn(T, h, D, generator=g).bfloat16() for h in (Hq, Hkv, Hkv)]
    w = torch.rand(2, D, generator=g) + 0.5
    qw, kw = w[0].cuda(), w[1].cuda()
    pkv.pages_reserve(bt, sl, refs, ints([0]), ints([L]), P)
    q0, k0, v0 = tokens(L)
    q_out = torch.empty(L, Hq, D, dtype=torch.bfloat16, device="cuda")
    pkv.gqa_rope_append(q0.cuda(), k0.cuda(), v0.cuda(), qw, kw, 1e-6, None, table, 1.0, False, kv, bt[:1],
                        sl[:1], ints([0, L]), P, q_out)
    src, dst = ints([-1] * n), ints([-1] * n)
    pkv.pages_fork(bt, sl, refs, ints([0] * n), ints(list(range(1, rows))), P, src, dst)
    pkv.pages_copy(kv, src, dst)
    pkv.pages_reserve(bt, sl, refs, ints(list(range(1, rows))), ints([L + 1] * n), P)
    q1, k1, v1 = tokens(n)
    q = torch.empty(n, Hq, D, dtype=torch.bfloat16, device="cuda")
    pkv.gqa_rope_append(q1.cuda(), k1.cuda(), v1.cuda(), qw, kw, 1e-6, None, table, 1.0, False, kv, bt[1:],
                        sl[1:], None, P, q)
    out = torch.empty_like(q)
    lse = torch.empty(n, Hq, device="cuda")
    pkv.paged_prefix_attn(q, kv, bt[1:], sl[1:], ints([0, n]), ints([L]), None, D ** -0.5, P, out, lse)
    torch.cuda.synchronize()
    assert pkv.check_errors(0) == 0
    # the definition on the tokens themselves
    freq = rope_plain.frequencies(D)
    keys, _ = rope_plain.norm_rope(k0, w[1], 1e-6, torch.arange(L), freq, 1.0, False)
    mine, _ = rope_plain.norm_rope(k1, w[1], 1e-6, torch.full((n,), L), freq, 1.0, False)
    qs, _ = rope_plain.norm_rope(q1, w[0], 1e-6, torch.full((n,), L), freq, 1.0, False)
    for b in range(n):
        for h in range(Hq):
            K = torch.cat([keys[:, h // 8], mine[b:b + 1, h // 8]])
            V = torch.cat([v0[:, h // 8], v1[b:b + 1, h // 8]]).double()
            x = K @ qs[b, h] * D ** -0.5
            want = torch.softmax(x, 0) @ V
            # q and k each rounded to bf16: scores off by 2^-7 of their terms' sizes
            dx = 2.0 ** -7 * float((K.abs() @ qs[b, h].abs()).amax()) * D ** -0.5
            spread = float((torch.softmax(x, 0) @ V.abs()).amax())
            tol = 2.0 ** -8 * want.abs() + (2 * dx + 2.0 ** -7) * spread
            assert ((out[b, h].cpu().double() - want).abs() <= tol).all()
            assert abs(float(lse[b, h]) - float(torch.logsumexp(x, 0))) <= dx + 1e-4
    # and bit by bit what the call on the same rows without sharing says within its bounds
    pr = dict(q=q.cpu(), kv=kv.cpu(), sc=None, bt=bt[1:].cpu(), sl=sl[1:].cpu(), sinks=None,
              scale=D ** -0.5, P=P, fp8=False, lead=0, tail=0)
    check(pr, out, lse)
