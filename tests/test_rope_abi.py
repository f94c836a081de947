"""CPU-side checks of the rotation calls: what is refused, with its code, before any CUDA call;
the table of frequencies; and the plain implementation that the GPU tests compare with."""
import math
from fractions import Fraction

import pytest
import torch

import paged_kv_cache_30_gb300 as pkv
from paged_kv_cache_30_gb300 import build as pkv_build
from tests import rope_plain as plain
from tests.test_paged_abi import BF16, F32, FP8, I32, ref
from tests.test_abi import _t

NAMES = ["q", "k", "v", "qw", "kw", "pos", "rope", "qo", "ko", "kv", "bt", "sl", "cu"]
PTR = {n: 0x10000000 * (i + 1) for i, n in enumerate(NAMES)}


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return pkv.load_library()


def tensor(name, shape, dtype, strides=None, ptr=None):
    return _t(shape, dtype, strides, PTR[name] if ptr is None else ptr)


def args(T=4, Hq=4, Hkv=2, D=128, B=2):
    return dict(q=tensor("q", [T, Hq, D], BF16), k=tensor("k", [T, Hkv, D], BF16),
                v=tensor("v", [T, Hkv, D], BF16), qw=tensor("qw", [D], BF16),
                kw=tensor("kw", [D], F32), eps=1e-6, pos=tensor("pos", [T], I32),
                rope=tensor("rope", [D // 2, 2], I32), factor=1.0,
                qo=tensor("qo", [T, Hq, D], BF16), ko=tensor("ko", [T, Hkv, D], BF16),
                kv=tensor("kv", [64, Hkv, 16, 2 * D], BF16), bt=tensor("bt", [B, 8], I32),
                sl=tensor("sl", [B], I32), cu=tensor("cu", [B + 1], I32), P=16)


def call(lib, a, cache=False):
    if cache:
        return lib.pkv_gqa_rope_append(
            ref(a["q"]), ref(a["k"]), ref(a["v"]), ref(a["qw"]), ref(a["kw"]), a["eps"], ref(a["pos"]),
            ref(a["rope"]), a["factor"], 0, ref(a["kv"]), ref(a["bt"]), ref(a["sl"]), ref(a["cu"]),
            a["P"], ref(a["qo"]), None)
    return lib.pkv_qk_norm_rope(ref(a["q"]), ref(a["k"]), ref(a["qw"]), ref(a["kw"]), a["eps"],
                                ref(a["pos"]), ref(a["rope"]), a["factor"], 0, ref(a["qo"]),
                                ref(a["ko"]), None)


BOTH = [
    (dict(q=None), -1), (dict(qo=None), -1), (dict(eps=-1.0), -1), (dict(eps=math.nan), -1),
    (dict(factor=math.inf), -1), (dict(k=None), -1),
    (dict(q=tensor("q", [4, 4, 128], F32)), -1), (dict(q=tensor("q", [4, 512], BF16)), -1),
    (dict(q=tensor("q", [4, 4, 96], BF16), qo=tensor("qo", [4, 4, 96], BF16)), -2),
    (dict(q=tensor("q", [4, 0, 128], BF16), qo=tensor("qo", [4, 0, 128], BF16)), -1),
    (dict(q=tensor("q", [4, 4, 128], BF16, ptr=PTR["q"] + 8)), -3),
    (dict(q=tensor("q", [4, 4, 128], BF16, [600, 130, 1])), -3),
    (dict(q=tensor("q", [4, 4, 128], BF16, [2048, 256, 2])), -1),
    (dict(k=tensor("k", [3, 2, 128], BF16)), -1), (dict(k=tensor("k", [4, 2, 64], BF16)), -1),
    (dict(qw=tensor("qw", [64], BF16)), -1), (dict(qw=tensor("qw", [128], I32)), -1),
    (dict(kw=tensor("kw", [128], F32, [2])), -1), (dict(kw=tensor("kw", [128], F32, ptr=PTR["kw"] + 2)), -3),
    (dict(pos=tensor("pos", [5], I32)), -1), (dict(pos=tensor("pos", [4], F32)), -1),
    (dict(pos=tensor("pos", [4], I32, [2])), -1),
    (dict(rope=tensor("rope", [64], I32)), -1), (dict(rope=tensor("rope", [64, 2], I32, [4, 1])), -1),
    (dict(rope=tensor("rope", [60, 2], I32)), -2), (dict(rope=tensor("rope", [72, 2], I32)), -2),
    (dict(rope=tensor("rope", [0, 2], I32)), -2),
    (dict(rope=tensor("rope", [64, 2], I32, ptr=PTR["rope"] + 4)), -3),
    (dict(qo=tensor("qo", [4, 4, 128], BF16, [0, 128, 1])), -1),
    (dict(qo=tensor("qo", [4, 4, 128], BF16, ptr=PTR["q"] + 256)), -1),
    (dict(qo=tensor("qo", [4, 4, 128], BF16, ptr=PTR["k"])), -1),
    (dict(qo=tensor("qo", [4, 4, 128], BF16, ptr=PTR["rope"])), -1),
    (dict(qo=tensor("qo", [4, 4, 64], BF16)), -1),
    # the same memory in another order is not q itself
    (dict(qo=tensor("qo", [4, 4, 128], BF16, [128, 512, 1], ptr=PTR["q"])), -1),
    # side by side, but heads of q_out reach into k's place
    (dict(q=tensor("q", [4, 4, 128], BF16, [1024, 128, 1]),
          k=tensor("k", [4, 2, 128], BF16, [1024, 128, 1], ptr=PTR["q"] + 3 * 256),
          qo=tensor("qo", [4, 4, 128], BF16, [1024, 128, 1], ptr=PTR["q"])), -1),
]


@pytest.mark.parametrize("cache", [False, True])
@pytest.mark.parametrize("change,code", BOTH)
def test_refusals(lib, cache, change, code):
    assert call(lib, {**args(), **change}, cache) == code
    assert pkv.last_error()


@pytest.mark.parametrize("change,code", [
    (dict(pos=None), -1), (dict(ko=None), -1), (dict(k=None, kw=None), -1),
    (dict(ko=tensor("ko", [4, 2, 64], BF16)), -1),
    (dict(ko=tensor("ko", [4, 2, 128], BF16, ptr=PTR["ko"] + 2)), -3),
    (dict(ko=tensor("ko", [4, 2, 128], BF16, ptr=PTR["qo"])), -1),
    (dict(ko=tensor("ko", [4, 2, 128], BF16, ptr=PTR["q"] + 512)), -1),
    (dict(ko=tensor("ko", [4, 2, 128], BF16, ptr=PTR["pos"])), -1),
    (dict(ko=tensor("ko", [4, 2, 128], BF16, [256, 0, 1])), -1),
])
def test_refusals_without_a_cache(lib, change, code):
    assert call(lib, {**args(), **change}) == code


@pytest.mark.parametrize("change,code", [
    (dict(v=None), -1), (dict(kv=None), -1), (dict(bt=None), -1), (dict(sl=None), -1), (dict(P=24), -2),
    (dict(P=32), -1), (dict(v=tensor("v", [4, 2, 64], BF16)), -1),
    (dict(v=tensor("v", [4, 2, 128], BF16, ptr=PTR["v"] + 2)), -3),
    (dict(kv=tensor("kv", [64, 2, 16, 256], FP8)), -1), (dict(kv=tensor("kv", [64, 3, 16, 256], BF16)), -1),
    (dict(kv=tensor("kv", [64, 2, 16, 256], BF16, [0, 4096, 256, 1])), -1),
    (dict(kv=tensor("kv", [64, 2, 16, 256], BF16, ptr=PTR["q"])), -1),
    (dict(qo=tensor("qo", [4, 4, 128], BF16, ptr=PTR["v"])), -1),
    (dict(qo=tensor("qo", [4, 4, 128], BF16, ptr=PTR["kv"])), -1),
    (dict(cu=tensor("cu", [4], I32)), -1), (dict(cu=tensor("cu", [3], I32, [2])), -1),
    (dict(cu=None, sl=tensor("sl", [3], I32), bt=tensor("bt", [3, 8], I32)), -1),
    (dict(bt=tensor("bt", [3, 8], I32)), -1), (dict(sl=tensor("sl", [2], I32, [2])), -1),
])
def test_append_refusals(lib, change, code):
    assert call(lib, {**args(), **change}, True) == code


def test_views_side_by_side_are_told_from_views_that_cross(lib):
    """Queries and keys in place inside the rows of a projection, next to one another in each token
    or in each head."""
    def refused(cache, heads, q, k, v):
        views = {n: tensor(n, [4, heads, 128], BF16, s, PTR["q"] + 2 * at)
                 for n, (s, at) in (("q", q), ("k", k), ("v", v))}
        a = {**args(Hq=heads, Hkv=heads), **views, "qo": views["q"], "ko": views["k"]}
        return call(lib, a, cache) == -1 and "overlaps" in pkv.last_error()
    for cache in (False, True):
        token, head = [6 * 128, 128, 1], [6 * 128, 3 * 128, 1]
        assert not refused(cache, 2, (token, 0), (token, 256), (token, 512))
        assert not refused(cache, 2, (head, 0), (head, 128), (head, 256))
        assert not refused(cache, 2, (head, 256), (head, 0), (head, 128))
        assert refused(cache, 2, (head, 0), (head, 64), (head, 256))  # half a head further
        assert refused(cache, 2, (token, 0), (head, 128), (token, 512))
        odd = [5 * 128, 2 * 128, 1]  # a token's row is no whole number of heads
        assert refused(cache, 2, (odd, 0), (odd, 128), (odd, 8192))


def test_no_tokens_are_no_ops(lib):
    for cache in (False, True):
        a = args(T=0)
        for n in ("q", "k", "v", "pos", "qo", "ko"):
            a[n].data = None
        assert call(lib, a, cache) == 0


@pytest.mark.parametrize("kind", [dict(), dict(base=500000.0), dict(factor=4.0),
                                  dict(factor=16.0, original_len=8192, low=1.0, high=32.0),
                                  dict(inv_freq=[0.3 * i - 1 for i in range(32)])])
def test_table_holds_turns_per_position(lib, kind):
    table = pkv.rope_table(64, device="cpu", **kind)
    words = table.view(torch.uint8).reshape(32, 8)
    plain_kind = {k: v for k, v in kind.items() if k not in ("original_len", "inv_freq")}
    freq = plain.frequencies(64, original=kind.get("original_len", 0), **plain_kind).tolist()
    freq = kind.get("inv_freq", freq)
    two_pi = Fraction(314159265358979323846264338327950288, 10 ** 35) * 2
    for i in range(32):
        got = Fraction(int.from_bytes(bytes(words[i].tolist()), "little"), 1 << 64)
        turns = Fraction(freq[i]) / two_pi
        off = (got - turns) % 1
        off = min(off, 1 - off)
        # a few roundings to 53 bits of the frequency, and one of the fraction
        assert off <= abs(turns) * Fraction(6, 1 << 53) + Fraction(1, 1 << 53)


@pytest.mark.parametrize("kw", [dict(rot_dim=24), dict(rot_dim=0), dict(rot_dim=144), dict(base=0.0),
                                dict(base=math.nan), dict(factor=0.0), dict(factor=math.inf),
                                dict(original_len=-1.0), dict(inv_freq=[1.0]),
                                dict(factor=2.0, original_len=4096, low=4.0, high=4.0),
                                dict(inv_freq=[math.inf] * 32)])
def test_table_refusals(lib, kw):
    with pytest.raises(pkv.PkvError):
        pkv.rope_table(**{"rot_dim": 64, "device": "cpu", **kw})
    assert lib.pkv_rope_table(None, 64, 1e4, 1.0, 0.0, 1.0, 4.0, None) == -1


def test_the_plain_form_keeps_what_a_rotation_keeps():
    """Lengths of pairs, and products of two rows by the difference of their positions."""
    g = torch.Generator().manual_seed(0)
    x, y = torch.randn(2, 1, 1, 64, generator=g, dtype=torch.float64)
    freq = plain.frequencies(64)
    for inter in (False, True):
        a = [plain.norm_rope(x, None, 0, torch.tensor([n]), freq, 1.0, inter)[0] for n in (0, 9, 100)]
        b = [plain.norm_rope(y, None, 0, torch.tensor([n]), freq, 1.0, inter)[0] for n in (5, 14, 105)]
        dots = [float((u * v).sum()) for u, v in zip(a, b)]
        assert max(dots) - min(dots) < 1e-9
        assert torch.equal(a[0], x) and abs(float(a[2].norm() - x.norm())) < 1e-9
    n, _ = plain.norm_rope(x, torch.ones(64), 0.0, torch.tensor([0]), None, 1.0, False)
    assert abs(float((n ** 2).mean()) - 1) < 1e-12
