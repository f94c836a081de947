"""GPU norm and rotation of queries and keys (pkv_qk_norm_rope), and the same on the way into
the paged cache (pkv_gqa_rope_append), against the 64-bit definitions, element by element
within the bounds of the kernel's roundings."""
import math

import pytest
import torch

import paged_kv_cache_30_gb300 as pkv
from tests import rope_plain as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    pkv.load_library()
    pkv.init(0)


def heads(g, T, H, D):
    return (torch.randn(T, H, D, generator=g) * torch.exp(torch.randn(T, H, 1, generator=g))).bfloat16()


def weight(g, D, kind):
    if kind is None:
        return None
    w = 1 + 0.3 * torch.randn(D, generator=g)
    return w.bfloat16() if kind == "bf16" else w


def up(t):
    return None if t is None else t.cuda()


def close(got, want, tol, what=""):
    got = got.double().cpu()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, worst " \
        f"{float(((got - want).abs() / tol).nan_to_num(math.inf).max())} of the bound"


def check(T, Hq, Hkv, D, rot, interleaved, qw=None, kw=None, seed=0, scaled=False, far=1 << 20,
          in_place=False, fused=True, pad=()):
    g = torch.Generator().manual_seed(seed)
    q, k = heads(g, T, Hq, D), heads(g, T, Hkv, D)
    wq, wk = weight(g, D, qw), weight(g, D, kw)
    pos = torch.randint(0, far, (T,), generator=g, dtype=torch.int64).int()
    for t in pad:
        pos[t] = -1 - t
    kind = dict(base=500000.0, factor=8.0, original=4096, low=1.0, high=4.0) if scaled else {}
    freq = plain.frequencies(rot, **kind) if rot else None
    table = None
    if rot:
        if scaled:
            kind["original_len"] = kind.pop("original")
        table = pkv.rope_table(rot, **kind)
    factor = 1.25 if scaled else 1.0
    whole = torch.cat([q, k, heads(g, T, 2, D)], dim=1) if fused else None
    dq, dk = (whole.cuda()[:, :Hq], None) if fused else (q.cuda(), k.cuda())
    if fused:
        base = whole.cuda()
        dq, dk = base[:, :Hq], base[:, Hq:Hq + Hkv]
    qo = dq if in_place else torch.full_like(q, math.nan).cuda()
    ko = dk if in_place else torch.full_like(k, math.nan).cuda()
    pkv.qk_norm_rope(dq, dk, up(wq), up(wk), 1e-5, pos.cuda(), table, factor, interleaved, qo, ko)
    torch.cuda.synchronize()
    live = torch.tensor([t not in pad for t in range(T)])
    for got, x, w, name in ((qo, q, wq, "q"), (ko, k, wk, "k")):
        want, tol = plain.norm_rope(x, w, 1e-5, pos, freq, factor, interleaved)
        close(got[live.cuda()], want[live], tol[live], name)
        for t in pad:  # not written
            rest = x[t] if in_place else torch.full_like(x[t], math.nan)
            assert torch.equal(got[t].cpu().view(torch.int16), rest.view(torch.int16))
    if fused and in_place:  # the heads beside them stay
        assert torch.equal(base[:, Hq + Hkv:].cpu(), whole[:, Hq + Hkv:])
    elif fused:
        assert torch.equal(base.cpu(), whole)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (128, 112), (128, 16), (64, 64), (64, 32),
                                   (64, 48), (64, 16)])
def test_pairs_and_parts_of_a_head(D, rot, interleaved):
    check(T=37, Hq=5, Hkv=3, D=D, rot=rot, interleaved=interleaved, qw="bf16", kw="f32", seed=rot)


@pytest.mark.parametrize("qw,kw", [(None, None), ("bf16", "bf16"), ("f32", None), (None, "f32")])
@pytest.mark.parametrize("D", [64, 128])
def test_norms(D, qw, kw):
    check(T=19, Hq=8, Hkv=2, D=D, rot=D, interleaved=False, qw=qw, kw=kw, seed=1)
    check(T=19, Hq=7, Hkv=1, D=D, rot=D, interleaved=True, qw=qw, kw=kw, seed=2, fused=False)


@pytest.mark.parametrize("T", [1, 2, 7, 64, 609, 1300, 2500])
@pytest.mark.parametrize("Hq,Hkv", [(64, 8), (1, 1), (13, 3)])
def test_counts_of_tokens(T, Hq, Hkv):
    check(T=T, Hq=Hq, Hkv=Hkv, D=128, rot=128, interleaved=False, qw="bf16", kw="bf16", seed=T)
    check(T=T, Hq=Hq, Hkv=Hkv, D=64, rot=32, interleaved=True, seed=T, in_place=True)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("T", [5, 2600])
def test_padding_is_not_written(T, in_place):
    check(T=T, Hq=6, Hkv=2, D=64, rot=64, interleaved=False, seed=3, in_place=in_place,
          pad=[0, 3, T - 1])
    check(T=T, Hq=6, Hkv=2, D=128, rot=64, interleaved=True, qw="f32", kw="f32", seed=4,
          in_place=in_place, pad=[0, 3, T - 1])


@pytest.mark.parametrize("far", [1, 2, 1 << 24, (1 << 31) - 1])
def test_far_positions_and_scaled_frequencies(far):
    check(T=50, Hq=4, Hkv=1, D=128, rot=128, interleaved=False, scaled=True, far=far, seed=far % 97)
    # 64-bit angles of the plain form: 2^31 radians are off by 2^-22, less than is allowed
    check(T=50, Hq=4, Hkv=1, D=64, rot=64, interleaved=True, far=far, seed=5)


def test_norms_without_a_rotation():
    g = torch.Generator().manual_seed(6)
    q, w = heads(g, 33, 6, 128), weight(g, 128, "bf16")
    out = torch.empty_like(q).cuda()
    pkv.qk_norm_rope(q.cuda(), None, w.cuda(), None, 1e-6, None, None, 1.0, False, out, None)
    close(out, *plain.norm_rope(q, w, 1e-6, None, None, 1.0, False))


def test_the_rotated_part_of_latent_rows():
    g = torch.Generator().manual_seed(7)
    q, row = heads(g, 12, 128, 576), heads(g, 12, 1, 576)
    pos = torch.randint(0, 1 << 17, (12,), generator=g).int()
    dq, dr = q.cuda(), row.cuda()
    pkv.qk_norm_rope(dq[..., 512:], dr[..., 512:], None, None, 0.0, pos.cuda(), pkv.rope_table(64),
                     1.0, True, dq[..., 512:], dr[..., 512:])
    for got, x in ((dq, q), (dr, row)):
        close(got[..., 512:], *plain.norm_rope(x[..., 512:], None, 0, pos, plain.frequencies(64), 1.0,
                                               True))
        assert torch.equal(got[..., :512].cpu(), x[..., :512])


def test_zeros_infinities_and_nan_stay_in_their_heads():
    g = torch.Generator().manual_seed(8)
    q = heads(g, 6, 4, 128)
    q[1, 2] = 0
    q[2, 0, 5] = math.nan
    q[3, 1, 100] = math.inf
    w, pos = weight(g, 128, "f32"), torch.arange(6).int()
    out = torch.empty_like(q).cuda()
    pkv.qk_norm_rope(q.cuda(), None, w.cuda(), None, 1e-6, pos.cuda(), pkv.rope_table(128), 1.0, False,
                     out, None)
    want, tol = plain.norm_rope(q, w, 1e-6, pos, plain.frequencies(128), 1.0, False)
    fine = torch.ones(6, 4, dtype=torch.bool)
    fine[2, 0] = fine[3, 1] = False
    close(out[fine.cuda()], want[fine], tol[fine])
    assert out[1, 2].eq(0).all() and out[2, 0].isnan().all() and out[3, 1].isnan().any()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_heads_whose_squares_overflow_are_normed_to_zero(D, interleaved):
    g = torch.Generator().manual_seed(34)
    q, k = heads(g, 8, 5, D), heads(g, 8, 2, D)
    big = torch.tensor([2.0 ** 66, 2.0 ** 100, 2.0 ** 127, -3.3e38])
    q[2, 1, ::7], q[3, 4] = big[3], big[0]
    q[5, 0, :4], k[6, 1, D - 4:] = big, big
    w = 1 + 3 * torch.rand(D, generator=g)  # weights above 1
    pos, freq = torch.arange(8).int() * 1000, plain.frequencies(D // 2)
    qo, ko = torch.empty_like(q).cuda(), torch.empty_like(k).cuda()
    pkv.qk_norm_rope(q.cuda(), k.cuda(), w.cuda(), w.cuda(), 1e-6, pos.cuda(), pkv.rope_table(D // 2), 1.5,
                     interleaved, qo, ko)
    for got, x, zero in ((qo, q, [(2, 1), (3, 4), (5, 0)]), (ko, k, [(6, 1)])):
        fine = torch.ones(x.shape[:2], dtype=torch.bool)
        for t, h in zero:
            assert got[t, h].eq(0).all()
            fine[t, h] = False
        want, tol = plain.norm_rope(x, w, 1e-6, pos, freq, 1.5, interleaved)
        close(got[fine.cuda()], want[fine], tol[fine])


def test_rotation_captured_and_replayed_at_other_positions():
    g = torch.Generator().manual_seed(33)
    q, k, freq = heads(g, 5, 4, 128), heads(g, 5, 2, 128), plain.frequencies(128)
    dq, dk, table = q.cuda(), k.cuda(), pkv.rope_table(128)
    pos, qo, ko = torch.zeros(5, dtype=torch.int32, device="cuda"), torch.empty_like(dq), torch.empty_like(dk)

    def call():
        pkv.qk_norm_rope(dq, dk, None, None, 0.0, pos, table, 1.0, False, qo, ko)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
    torch.cuda.synchronize()
    for at in ([0, 1, 2, 3, 4], [(1 << 31) - 1, 70000, 5, 0, 123456789]):
        pos.copy_(torch.tensor(at, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for got, x in ((qo, q), (ko, k)):
            close(got, *plain.norm_rope(x, None, 0.0, pos.cpu(), freq, 1.0, False))


def test_given_frequencies():
    g = torch.Generator().manual_seed(9)
    freq = torch.rand(16, generator=g, dtype=torch.float64) * 7 - 1  # also more than a turn, negative
    q, pos = heads(g, 20, 2, 64), torch.randint(0, 50000, (20,), generator=g).int()
    out = torch.empty_like(q).cuda()
    pkv.qk_norm_rope(q.cuda(), None, None, None, 0.0, pos.cuda(), pkv.rope_table(32, inv_freq=freq),
                     -0.5, False, out, None)
    close(out, *plain.norm_rope(q, None, 0, pos, freq, -0.5, False))


# ----------------------------------------------------------------- append --
def problem(seed, lens, new, Hq, Hkv, D, P, rot, lead=0, tail=0, norm=True, one_each=False):
    """Requests of `lens` tokens, the last `new` of them fresh, padding rows around theirs."""
    g = torch.Generator().manual_seed(seed)
    T = lead + sum(new) + tail
    cu = [lead]
    for n in new:
        cu.append(cu[-1] + n)
    width = max(1, max(-(-L // P) for L in lens))
    pool = sum(-(-max(L, 0) // P) for L in lens) + 3
    order, at = torch.randperm(pool, generator=g).int(), 0
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    for b, L in enumerate(lens):
        n = -(-max(L, 0) // P)
        table[b, :n] = order[at:at + n]
        at += n
    return dict(q=heads(g, T, Hq, D), k=heads(g, T, Hkv, D), v=heads(g, T, Hkv, D),
                qw=weight(g, D, "bf16") if norm else None, kw=weight(g, D, "f32") if norm else None,
                kv=torch.randn(pool, Hkv, P, 2 * D, generator=g).bfloat16(), bt=table,
                sl=torch.tensor(lens, dtype=torch.int32),
                cu=None if one_each else torch.tensor(cu, dtype=torch.int32), P=P, rot=rot,
                pos=None, interleaved=False)


def run(pr, kv=None, stream=None, flags=0):
    d = {n: up(pr[n]) for n in ("q", "k", "v", "qw", "kw", "bt", "sl", "cu", "pos")}
    kv = pr["kv"].cuda() if kv is None else kv
    out = torch.full_like(d["q"], math.nan)
    table = pkv.rope_table(pr["rot"]) if pr["rot"] else None
    pkv.gqa_rope_append(d["q"], d["k"], d["v"], d["qw"], d["kw"], 1e-5, d["pos"], table, 1.0,
                        pr["interleaved"], kv, d["bt"], d["sl"], d["cu"], pr["P"], out, stream=stream)
    torch.cuda.synchronize()
    if flags:
        with pytest.raises(pkv.PkvError, match=f"0x{flags:x}"):
            pkv.check_errors(0)
    else:
        pkv.check_errors(0)
    return out, kv


def verify(pr, out, kv):
    T, D = pr["q"].shape[0], pr["q"].shape[2]
    at = plain.places(pr["sl"], pr["cu"], T, pr["bt"], pr["P"], pr["kv"].shape[0], pr["pos"])
    live = [t for t in range(T) if at[t][0] is not None]
    pos = torch.tensor([at[t][0] for t in live], dtype=torch.int64)
    freq = plain.frequencies(pr["rot"]) if pr["rot"] else None
    want, tol = plain.norm_rope(pr["q"][live], pr["qw"], 1e-5, pos, freq, 1.0, pr["interleaved"])
    close(out[torch.tensor(live, dtype=torch.long).cuda()], want, tol, "q_out")
    rest = [t for t in range(T) if at[t][0] is None]
    assert out[torch.tensor(rest, dtype=torch.long).cuda()].isnan().all()
    key, ktol = plain.norm_rope(pr["k"][live], pr["kw"], 1e-5, pos, freq, 1.0, pr["interleaved"])
    want, tol = pr["kv"].double(), torch.zeros(pr["kv"].shape, dtype=torch.float64)
    for i, t in enumerate(live):
        _, page, slot = at[t]
        if page is None:
            continue
        want[page, :, slot, :D], tol[page, :, slot, :D] = key[i], ktol[i]
        want[page, :, slot, D:] = pr["v"][t].double()
    close(kv, want, tol, "cache")


@pytest.mark.parametrize("D,Hq,Hkv,P,rot,norm", [
    (128, 64, 8, 16, 128, True), (64, 4, 4, 32, 32, False), (128, 5, 1, 64, 16, True),
    (64, 14, 2, 128, 64, True), (128, 8, 2, 16, 0, True), (64, 3, 1, 16, 0, False)])
def test_one_token_each(D, Hq, Hkv, P, rot, norm):
    lens = [1, 16, 17, 300, 0, 33, 2, 1024]
    pr = problem(D + P, lens, [1] * 8, Hq, Hkv, D, P, rot, norm=norm, one_each=True)
    verify(pr, *run(pr))


@pytest.mark.parametrize("D,P,interleaved", [(128, 16, False), (64, 64, True), (128, 128, True)])
def test_ragged_prompts_between_padding_rows(D, P, interleaved):
    new = [40, 0, 1, 333, 17, 0, 0, 128, 5]
    lens = [40, 12, 9, 600, 17, 0, 3, 129, 3]  # the last request's first tokens have no place
    pr = problem(P, lens, new, 6, 2, D, P, D, lead=3, tail=5)
    pr["interleaved"] = interleaved
    verify(pr, *run(pr))


def test_lengths_of_any_size_below_the_new_tokens():
    for one in (True, False):
        new = [1, 1, 1, 1] if one else [3, 1, 0, 5]
        pr = problem(23, [-(1 << 31), 0, -(1 << 31) + 5, 7], new, 4, 2, 64, 16, 64, one_each=one)
        verify(pr, *run(pr))


def test_many_requests_and_long_prompts():
    pr = problem(11, [3 + b % 7 for b in range(1500)], [b % 3 for b in range(1500)], 4, 2, 64, 16, 64)
    verify(pr, *run(pr))
    pr = problem(12, [5000, 1, 700], [4000, 1, 650], 4, 2, 128, 32, 128, norm=False)
    verify(pr, *run(pr))


def test_several_tokens_each_without_offsets():
    pr = problem(13, [4, 9, 100, 2], [4] * 4, 4, 2, 64, 16, 64, one_each=True)
    verify(pr, *run(pr))


def test_positions_of_their_own():
    pr = problem(14, [30, 8, 50], [30, 8, 20], 4, 2, 64, 16, 64, tail=2)
    g = torch.Generator().manual_seed(1)
    pr["pos"] = torch.randint(0, 100000, (60,), generator=g).int()
    pr["pos"][7] = -1
    verify(pr, *run(pr))


def test_bad_pages_and_tables_are_flagged():
    pr = problem(15, [30, 40, 64], [30, 10, 64], 4, 2, 64, 16, 64)
    pr["bt"][0, 1] = pr["kv"].shape[0]
    pr["bt"][2, 0] = -1
    verify(pr, *run(pr, flags=1))
    pr = problem(16, [30, 64], [30, 64], 4, 2, 64, 16, 64)
    pr["bt"] = pr["bt"][:, :2].contiguous()
    verify(pr, *run(pr, flags=2))


def test_strided_views_of_one_projection_and_an_nhd_cache():
    pr = problem(17, [30, 40], [30, 10], 4, 2, 64, 16, 64)
    base = torch.cat([pr["q"], pr["k"], pr["v"]], dim=1).cuda()
    q, k, v = base[:, :4], base[:, 4:6], base[:, 6:]
    kv = pr["kv"].transpose(1, 2).contiguous().cuda().transpose(1, 2)
    pkv.gqa_rope_append(q, k, v, up(pr["qw"]), up(pr["kw"]), 1e-5, None, pkv.rope_table(64), 1.0, False,
                        kv, up(pr["bt"]), up(pr["sl"]), up(pr["cu"]), 16, q)
    torch.cuda.synchronize()
    verify(pr, q, kv)
    assert torch.equal(k.cpu(), pr["k"]) and torch.equal(v.cpu(), pr["v"])


def test_queries_and_keys_in_place_side_by_side_in_each_head():
    pr = problem(24, [30, 40], [30, 10], 3, 3, 64, 16, 64)
    base = torch.stack([pr["q"], pr["k"], pr["v"]], dim=2).cuda()  # [T, H, 3, D]
    q, k, v = base.unbind(2)
    kv, table = pr["kv"].cuda(), pkv.rope_table(64)
    pkv.gqa_rope_append(q, k, v, up(pr["qw"]), up(pr["kw"]), 1e-5, None, table, 1.0, False, kv,
                        up(pr["bt"]), up(pr["sl"]), up(pr["cu"]), 16, q)
    torch.cuda.synchronize()
    verify(pr, q, kv)
    assert torch.equal(k.cpu(), pr["k"]) and torch.equal(v.cpu(), pr["v"])
    base = torch.stack([pr["q"], pr["k"], pr["v"]], dim=2).cuda()
    q, k, v = base.unbind(2)
    pos = torch.arange(40).int() * 77
    pkv.qk_norm_rope(q, k, up(pr["qw"]), up(pr["kw"]), 1e-5, pos.cuda(), table, 1.0, False, q, k)
    for got, x, w in ((q, pr["q"], pr["qw"]), (k, pr["k"], pr["kw"])):
        close(got, *plain.norm_rope(x, w, 1e-5, pos, plain.frequencies(64), 1.0, False))
    assert torch.equal(v.cpu(), pr["v"])


def test_captured_and_replayed_with_other_lengths():
    pr = problem(18, [17, 30, 16], [1, 1, 1], 4, 2, 64, 16, 64, one_each=True)
    d = {n: up(pr[n]) for n in ("q", "k", "v", "qw", "kw", "bt", "sl")}
    kv, out, table = pr["kv"].cuda(), torch.full_like(d["q"], math.nan), pkv.rope_table(64)

    def call():
        pkv.gqa_rope_append(d["q"], d["k"], d["v"], d["qw"], d["kw"], 1e-5, None, table, 1.0, False,
                            kv, d["bt"], d["sl"], None, 16, out)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
    torch.cuda.synchronize()
    for lens in ([17, 30, 16], [5, 0, 1]):
        pr["sl"] = torch.tensor(lens, dtype=torch.int32)
        d["sl"].copy_(pr["sl"])
        kv.copy_(pr["kv"])
        out.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        verify(pr, out, kv)


def test_prompts_then_a_decode_call_that_reads_ahead():
    """The decode kernel asks for its first pages before it waits; after an append of whole
    prompts it must not, on the next launch of the stream."""
    g = torch.Generator().manual_seed(19)
    B, Hq, Hkv, P, L = 4, 16, 2, 16, 2000
    pages = -(-L // P)
    table = torch.randperm(B * pages, generator=g).int().view(B, pages).cuda()
    q, k, v = (heads(g, B * L, h, 128).cuda() for h in (Hq, Hkv, Hkv))
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    cu = (torch.arange(B + 1, dtype=torch.int32) * L).cuda()
    rope, kv = pkv.rope_table(128), torch.zeros(B * pages, Hkv, P, 256, dtype=torch.bfloat16, device="cuda")
    q_out, outs = torch.empty_like(q), []
    for wait in (True, False, False):
        kv.fill_(math.nan)
        out = torch.empty(B, Hq, 128, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        pkv.gqa_rope_append(q, k, v, None, None, 0.0, None, rope, 1.0, False, kv, table, lens, cu, P, q_out)
        if wait:
            torch.cuda.synchronize()
        pkv.paged_decode_attn(q_out[L - 1::L], kv, table, lens, None, 0, 0.09, P, 0, out)
        torch.cuda.synchronize()
        outs.append(out)
    assert outs[0].isfinite().all()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    pkv.check_errors(0)


def test_cache_offsets_past_32_bits():
    pool, P, Hkv, D = 9000, 128, 8, 128  # 2.4 * 10^9 elements
    kv = torch.empty(pool, Hkv, P, 2 * D, dtype=torch.bfloat16, device="cuda")
    kv[-1].zero_()
    pr = problem(20, [40], [40], 4, Hkv, D, P, D)
    pr["bt"] = torch.tensor([[pool - 1]], dtype=torch.int32)
    out, _ = run(pr, kv=kv)
    pr["bt"][0, 0] = 0
    pr["kv"] = torch.zeros(1, Hkv, P, 2 * D).bfloat16()
    verify(pr, out, kv[-1:])


def test_another_stream_and_same_bits_every_time():
    pr = problem(21, [300, 40, 64], [300, 10, 64], 8, 2, 128, 16, 128)
    a = run(pr)
    s = torch.cuda.Stream()
    b = run(pr, stream=s)
    assert torch.equal(a[0].cpu().view(torch.int16), b[0].cpu().view(torch.int16))
    assert torch.equal(a[1].cpu(), b[1].cpu())


def test_host_memory_is_refused():
    pr = problem(22, [30], [30], 4, 2, 64, 16, 64)
    with pytest.raises(pkv.PkvError):
        pkv.gqa_rope_append(pr["q"], pr["k"], pr["v"], None, None, 0.0, None, None, 1.0, False,
                            pr["kv"], pr["bt"], pr["sl"], pr["cu"], 16, torch.empty_like(pr["q"]))
    with pytest.raises(pkv.PkvError):
        pkv.qk_norm_rope(pr["q"], None, None, None, 0.0, None, None, 1.0, False,
                         torch.empty_like(pr["q"]), None, stream=0)
