"""GPU append to an e4m3 cache with a scale per (page, kv head)
(pkv_gqa_kv_append_fp8): codes and scales equal to the definition's."""
import math

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


def problem(seed, old, new, Hkv, D, P, pad=0, size=1.0):
    """Requests that hold `old` tokens and get `new` ones; `pad` rows of padding behind them."""
    g = torch.Generator().manual_seed(seed)
    lens = torch.tensor([o + n for o, n in zip(old, new)], dtype=torch.int32)
    B, width = len(old), max(1, -(-int(lens.max()) // P)) + 1
    counts = [-(-int(L) // P) for L in lens]
    pool = sum(counts) + 3
    order = torch.randperm(pool, generator=g).int()
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    scale = torch.exp2(torch.randint(-12, -3, (pool, Hkv, 2), generator=g).float())
    cache = (torch.randn(pool, Hkv, P, 2 * D, generator=g) * 100).to(torch.float8_e4m3fn)
    T = sum(new) + pad
    kv = torch.randn(T, Hkv, 2, D, generator=g) * size
    kv *= torch.exp2(torch.randint(-6, 7, (T, 1, 2, 1), generator=g).float())
    cu = torch.tensor([0] + [sum(new[:i + 1]) for i in range(B)], dtype=torch.int32)
    return dict(k=kv[:, :, 0].bfloat16(), v=kv[:, :, 1].bfloat16(), cache=cache, scale=scale,
                bt=table, sl=lens, cu=cu, P=P)


def run(pr, cu="cu"):
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in pr.items()}
    pkv.gqa_kv_append_fp8(d["k"], d["v"], d["cache"], d["scale"], d["bt"], d["sl"],
                          d["cu"] if cu else None, pr["P"])
    torch.cuda.synchronize()
    return d["cache"].cpu(), d["scale"].cpu()


def check(pr, got, flags=0):
    want, scale = plain.append(pr["k"], pr["v"], pr["cache"], pr["scale"], pr["bt"],
                               pr["sl"].tolist(), pr["cu"].tolist(), pr["P"])
    codes = got[0].double()
    same = (codes == want) | (codes.isnan() & want.isnan())
    assert same.all(), f"{int((~same).sum())} codes differ"
    assert torch.equal(got[1].double(), scale)
    if not flags:
        assert pkv.check_errors(0) == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("Hkv", [1, 3, 8])
def test_one_token_each(D, P, Hkv):
    old = [0, 1, P - 1, P, P + 1, 2 * P - 1, 100, 5]
    pr = problem(D + P + Hkv, old, [1] * len(old), Hkv, D, P)
    check(pr, run(pr))
    check(pr, run(pr, cu=None))


@pytest.mark.parametrize("D,P", [(64, 16), (128, 16), (128, 32), (64, 128)])
def test_ragged_prompts(D, P):
    old = [0, 3, P - 1, P, 0, 40, 0, 1]
    new = [1, P, 2 * P + 1, 5, 0, 3 * P, 200, P - 1]
    pr = problem(D * 3 + P, old, new, 2, D, P)
    check(pr, run(pr))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [32, 64, 128])
def test_large_pages_in_pieces_held_and_continued(D, P):
    """Pages whose rows several warps share: whole, begun, continued twice in one batch, with bad
    pages between good ones of a request."""
    old = [0, 5, P - 3, 2 * P, 17, 0]
    new = [3 * P + 7, P, 3, 4 * P, 2 * P - 17, 1]
    pr = problem(D + 5 * P, old, new, 3, D, P)
    check(pr, run(pr))
    pr["bt"][0, 1], pr["bt"][3, 3] = -1, 10 ** 7
    got = run(pr)
    with pytest.raises(pkv.PkvError):
        pkv.check_errors(0)
    check(pr, got)


def test_negative_lengths_take_no_row_of_the_next_request():
    pr = problem(14, [0, 3, 0], [5, 6, 20], 2, 64, 16)
    pr["sl"][0], pr["sl"][1] = -3, 2
    check(pr, run(pr))


def test_one_long_prompt_among_single_tokens():
    pr = problem(15, [9] * 40, [1] * 20 + [300] + [1] * 19, 2, 128, 64)
    check(pr, run(pr))


def test_many_requests_of_one_token_and_of_none():
    g = torch.Generator().manual_seed(3)
    new = torch.randint(0, 3, (500,), generator=g).tolist()
    old = torch.randint(0, 40, (500,), generator=g).tolist()
    pr = problem(3, old, new, 2, 64, 16)
    check(pr, run(pr))


def test_more_rows_than_one_wave_of_warps():
    pr = problem(4, [5, 0, 700], [3000, 1, 1500], 4, 64, 16)
    check(pr, run(pr))


def test_padding_rows_are_ignored():
    pr = problem(5, [4, 0], [7, 20], 2, 128, 16, pad=9)
    check(pr, run(pr))
    # a first row above 0: the rows before it are padding too
    pr["cu"] = pr["cu"] + 4
    pr["k"], pr["v"] = pr["k"].roll(4, 0), pr["v"].roll(4, 0)
    check(pr, run(pr))


def test_scales_zero_tiny_huge_and_the_border_of_a_binade():
    """448 s exactly keeps s; one bf16 step more doubles it; zeros give scale 0; 2^-126 gives
    the smallest scale; the largest bf16 value."""
    P = 16
    pr = problem(6, [0] * 6, [1] * 6, 1, 64, P)
    vals = [448.0 * 2 ** -7, 450.0 * 2 ** -7, 0.0, 2.0 ** -126, 3.3895e38, 2.0 ** -133]
    for i, x in enumerate(vals):
        pr["k"][i] = 0
        pr["k"][i, 0, 3] = x
        pr["v"][i] = -pr["k"][i]
    got = run(pr)
    check(pr, got)
    s = [float(got[1][int(pr["bt"][i, 0]), 0, 0]) for i in range(6)]
    assert s[0] == 2.0 ** -7 and s[1] == 2.0 ** -6 and s[2] == 0.0 and s[3] == 2.0 ** -100
    assert s[5] == 2.0 ** -100


def test_infinities_saturate_and_nan_stays():
    pr = problem(7, [3, 0], [4, 2], 1, 128, 16)
    pr["k"][0, 0, 5], pr["k"][1, 0, 6], pr["v"][2, 0, 7] = math.inf, -math.inf, math.nan
    pr["v"][4:, 0] = math.nan
    got = run(pr)
    check(pr, got)
    page = int(pr["bt"][0, 0])
    assert got[0].double()[page, 0, 3, 5] == 448 and got[0].double()[page, 0, 4, 6] == -448
    assert got[0].double()[page, 0, 5, 128 + 7].isnan()


def test_held_tokens_are_encoded_again_when_the_scale_grows():
    pr = problem(8, [15, 31, 20], [1, 1, 20], 2, 128, 32, size=2.0 ** 14)
    got = run(pr)
    assert (got[1] > pr["scale"]).any()
    check(pr, got)


def test_scales_that_are_no_power_of_two():
    pr = problem(9, [10, 3], [2, 30], 2, 64, 16)
    pr["scale"] *= 1.37
    # quotients and products rounded to 32 bits first: restate them so
    vals, sc = pr["cache"].double(), pr["scale"].double()
    got = run(pr)
    assert pkv.check_errors(0) == 0
    b, page = 0, int(pr["bt"][0, 0])
    for h in range(2):
        for kv, x in ((0, pr["k"]), (1, pr["v"])):
            old = pr["scale"][page, h, kv]
            a = float(x[:2, h].abs().amax())
            s = torch.maximum(old, torch.tensor(plain.need_scale(a), dtype=torch.float32))
            assert got[1][page, h, kv] == s
            half = slice(kv * 64, kv * 64 + 64)
            new = plain.encode(x[:2, h].float() / s)
            assert torch.equal(got[0].double()[page, h, 10:12, half], new)
            held = vals[page, h, :10, half]
            if s > old:
                held = plain.encode(held.float() * (old / s))
            assert torch.equal(got[0].double()[page, h, :10, half], held)


def test_bad_pages_are_skipped_and_flagged_and_negative_positions_dropped():
    pr = problem(10, [0, 30, 40], [5, 5, 5], 1, 64, 16)
    pr["bt"][1, 2] = -1           # 30..34: slots of page 1 and of page 2
    pr["bt"][2, 2] = 10 ** 6
    got = run(pr)
    with pytest.raises(pkv.PkvError):
        pkv.check_errors(0)
    check(pr, got)
    pr = problem(11, [0, 0], [5, 5], 1, 64, 16)
    pr["sl"][0] = 3               # five tokens of three: the first two are dropped
    pr["sl"][1] = 0
    check(pr, run(pr))
    pr = problem(12, [0], [40], 1, 64, 16)
    pr["bt"] = pr["bt"][:, :2].contiguous()  # the third page is past the table
    got = run(pr)
    with pytest.raises(pkv.PkvError):
        pkv.check_errors(0)
    check(pr, got)


def test_strided_sources_and_caches():
    pr = problem(13, [7, 16], [3, 40], 2, 128, 16)
    T, Hkv, D = pr["k"].shape
    both = torch.zeros(T, Hkv + 1, 2 * D + 8, dtype=torch.bfloat16, device="cuda")
    both[:, :Hkv, :D], both[:, :Hkv, D:2 * D] = pr["k"].cuda(), pr["v"].cuda()
    n, _, P, W = pr["cache"].shape
    store = torch.zeros(n, P, Hkv, W, dtype=torch.uint8, device="cuda")
    store.copy_(pr["cache"].view(torch.uint8).transpose(1, 2))
    cache = store.transpose(1, 2).view(torch.float8_e4m3fn)
    sc = torch.zeros(n, Hkv + 1, 2, device="cuda")
    sc[:, :Hkv] = pr["scale"].cuda()
    pkv.gqa_kv_append_fp8(both[:, :Hkv, :D], both[:, :Hkv, D:2 * D], cache, sc[:, :Hkv],
                          pr["bt"].cuda(), pr["sl"].cuda(), pr["cu"].cuda(), 16)
    torch.cuda.synchronize()
    check(pr, (cache.cpu(), sc[:, :Hkv].cpu()))
    assert (sc[:, Hkv] == 0).all()
