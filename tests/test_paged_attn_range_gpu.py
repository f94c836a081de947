"""GPU decode over an e4m3 cache where one key outweighs all others by far and adds little or
nothing to the output: what the others add stays right relative to itself.  The bound has no
absolute floor: each weight is rounded once, by 2^-11 of itself, however small it is beside
the largest."""
import math

import pytest
import torch

import paged_kv_cache_30_gb300 as pkv
from tests import paged_plain as plain
from tests.test_paged_attn_gpu import call

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    pkv.load_library()
    pkv.init(0)


def problem(seed, lens, Hkv, G, D, P, window=0, first=0, wide=False):
    """Seeded CPU tensors, values positive.  Dim 0 of the queries is 128 and of the keys 0, so
    a key's code there sets its logit; the cache holds no page twice."""
    g = torch.Generator().manual_seed(seed)
    lens = torch.tensor(lens, dtype=torch.int32)
    B, width = len(lens), -(-int(lens.max()) // P) + (9000 if wide else 0)
    need = [-(-int(n) // P) for n in lens]
    order, at = torch.randperm(sum(need), generator=g).int(), 0
    table = torch.full((B, width), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    x = torch.randn(sum(need), Hkv, P, 2 * D, generator=g)
    x[..., D:] = x[..., D:].abs()
    x[..., 0] = 0
    q = torch.randn(B, Hkv * G, D, generator=g)
    q[..., 0] = 128
    scale = torch.full((sum(need), Hkv, 2), 1 / 64)
    scale[..., 1] *= torch.exp2(torch.randint(-2, 3, (sum(need), Hkv), generator=g).float())
    return dict(q=q.bfloat16(), kv=(x * 60).to(torch.float8_e4m3fn), sc=scale, bt=table, sl=lens,
                sinks=None, window=window, first=first, scale=1 / math.sqrt(D), P=P, fp8=True)


def put(pr, b, j, nats, value):
    """Key j of request b: its logit `nats` above (below) the others', its value codes `value`."""
    D = pr["q"].shape[2]
    page, slot = int(pr["bt"][b, j // pr["P"]]), j % pr["P"]
    codes = pr["kv"][page, :, slot].float()
    codes[:, 0] = nats * math.sqrt(D) / 2  # times 128 / 64 and the softmax scale
    codes[:, D:] = value
    pr["kv"].view(torch.uint8)[page, :, slot] = codes.to(torch.float8_e4m3fn).view(torch.uint8)


def check(pr):
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in pr.items()}
    out = torch.full_like(d["q"], math.nan)
    lse = torch.full(d["q"].shape[:2], math.nan, device="cuda")
    call(d, out, lse)
    torch.cuda.synchronize()
    D = pr["q"].shape[2]
    cache = pr["kv"].double()
    cache[..., :D] *= pr["sc"].double()[:, :, None, :1]
    cache[..., D:] *= pr["sc"].double()[:, :, None, 1:]
    want, want_lse, tol, lse_tol = plain.decode(
        pr["q"], cache, None, pr["bt"], pr["sl"], pr["sinks"], pr["window"], pr["first"],
        pr["scale"], pr["P"], 2.0 ** -11)
    far = (out.cpu().double() - want).abs() - tol
    assert out.isfinite().all()
    assert (far <= 0).all(), f"off by {(far + tol).max():.3e} of {want.abs().max():.3e}"
    assert ((lse.cpu().double() - want_lse).abs() <= lse_tol).all()
    assert pkv.check_errors(0) == 0
    assert pkv.check_counters(0) == 0


@pytest.mark.parametrize("nats", [9, 14, 18, 22, 40])
@pytest.mark.parametrize("D,G", [(128, 8), (64, 4), (128, 16), (64, 16)])
@pytest.mark.parametrize("wide", [False, True])
def test_first_token_far_above_the_others_without_a_value(nats, D, G, wide):
    """From requests of one tile, where the others share the first key's, to long ones."""
    lens = [2, 9, 16, 17, 40, 300] + ([6000] if wide else [])
    pr = problem(nats + D + G, lens, 1, G, D, 16, wide=wide)
    for b in range(len(lens)):
        put(pr, b, 0, nats, 0.0)
    check(pr)


@pytest.mark.parametrize("D,G", [(128, 8), (64, 16)])
@pytest.mark.parametrize("nats", [14, 22])
def test_many_requests_with_such_a_first_token(nats, D, G):
    lens = [5 + i % 60 for i in range(400)]
    pr = problem(nats + D, lens, 3, G, D, 16)
    for b in range(len(lens)):
        put(pr, b, 0, nats, 0.0)
    check(pr)


@pytest.mark.parametrize("nats", [12, 20])
def test_such_keys_at_the_end_and_in_every_page(nats):
    pr = problem(nats, [1000, 1000, 333], 2, 8, 128, 32, window=700, first=5)
    put(pr, 0, 999, nats, 0.0)
    for j in list(range(7, 1000, 32)) + [0]:
        put(pr, 1, j, nats, 0.0)
    put(pr, 2, 150, nats, 2.0 ** -9)
    check(pr)


@pytest.mark.parametrize("power,nats", [(12, -9), (24, -18), (40, -30)])
@pytest.mark.parametrize("D,G", [(128, 8), (64, 16)])
def test_page_of_a_large_scale_that_nobody_attends_to(power, nats, D, G):
    """One outlier sets the value scale of its page, in which all other codes are 0."""
    pr = problem(power, [3000, 64, 16], 1, G, D, 16)
    for b, j in ((0, 1600), (1, 32), (2, 0)):
        page = int(pr["bt"][b, j // 16])
        pr["sc"][page, :, 1] *= 2.0 ** power
        pr["kv"].view(torch.uint8)[page, :, :, D:] = 0
        put(pr, b, j + 3, nats, 2.0 ** -4)
    check(pr)
