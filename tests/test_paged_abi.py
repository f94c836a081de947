"""CPU-side checks of the 8-bit append, decode with a window and first tokens and the page
calls: what is refused, with its code, before any CUDA call; and the plain implementations the
GPU tests compare with."""
import ctypes

import pytest
import torch

import oracle
import paged_kv_cache_30_gb300 as pkv
from paged_kv_cache_30_gb300 import build as pkv_build
from tests import paged_plain as plain
from tests.test_abi import _t

BF16, F32, I32, FP8 = pkv.DTYPE_BF16, pkv.DTYPE_F32, pkv.DTYPE_I32, pkv.DTYPE_FP8
PTR = {n: 0x10000000 * (i + 1) for i, n in enumerate(
    ["q", "kv", "sc", "bt", "sl", "sinks", "out", "lse", "k", "v", "cu", "refs", "a", "b", "c", "d"])}


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return pkv.load_library()


def tensor(name, shape, dtype, strides=None, ptr=None):
    return _t(shape, dtype, strides, PTR[name] if ptr is None else ptr)


def attn(B=2, Hq=16, Hkv=2, D=128, P=16, nb=64, W=8, fp8=True):
    return dict(q=tensor("q", [B, Hq, D], BF16),
                kv=tensor("kv", [nb, Hkv, P, 2 * D], FP8 if fp8 else BF16),
                sc=tensor("sc", [nb, Hkv, 2], F32), bt=tensor("bt", [B, W], I32),
                sl=tensor("sl", [B], I32), sinks=None, window=0, first=0, scale=0.1, P=P,
                out=tensor("out", [B, Hq, D], BF16), lse=tensor("lse", [B, Hq], F32))


def ref(t):
    return None if t is None else ctypes.byref(t)


def call_attn(lib, a, fp8=True):
    if fp8:
        return lib.pkv_paged_decode_attn_fp8(
            ref(a["q"]), ref(a["kv"]), ref(a["sc"]), ref(a["bt"]), ref(a["sl"]), ref(a["sinks"]),
            a["window"], a["first"], a["scale"], a["P"], ref(a["out"]), ref(a["lse"]), None)
    return lib.pkv_paged_window_attn(
        ref(a["q"]), ref(a["kv"]), ref(a["bt"]), ref(a["sl"]), ref(a["sinks"]), a["window"],
        a["first"], a["scale"], a["P"], ref(a["out"]), ref(a["lse"]), None)


ATTN = [
    (dict(q=None), -1), (dict(kv=None), -1), (dict(bt=None), -1), (dict(sl=None), -1),
    (dict(out=None), -1), (dict(first=-1), -1), (dict(scale=float("nan")), -1), (dict(P=24), -2),
    (dict(P=32), -1),
    (dict(q=tensor("q", [2, 16, 128], F32)), -1),
    (dict(q=tensor("q", [2, 15, 128], BF16)), -1),
    (dict(q=tensor("q", [2, 34, 128], BF16), out=tensor("out", [2, 34, 128], BF16)), -2),
    (dict(q=tensor("q", [2, 16, 96], BF16), out=tensor("out", [2, 16, 96], BF16)), -2),
    (dict(q=tensor("q", [3, 16, 128], BF16)), -1),
    (dict(q=tensor("q", [2, 16, 128], BF16, ptr=PTR["q"] + 2)), -3),
    (dict(q=tensor("q", [2, 16, 128], BF16, [16 * 132, 132, 1])), -3),
    (dict(q=tensor("q", [2, 16, 128], BF16, [4096, 256, 2])), -1),
    (dict(out=tensor("out", [2, 16, 128], BF16, [0, 128, 1])), -1),
    (dict(out=tensor("out", [2, 16, 128], BF16, ptr=PTR["kv"])), -1),
    (dict(lse=tensor("lse", [2, 16], F32, [1, 1])), -1),
    (dict(lse=tensor("lse", [2, 8], F32)), -1),
    (dict(sinks=tensor("sinks", [8], F32)), -1),
    (dict(bt=tensor("bt", [2, 8], I32, [16, 2])), -1),
    (dict(bt=tensor("bt", [2, 1 << 27], I32, [0, 1])), -1),
    (dict(sl=tensor("sl", [2], I32, [2])), -1),
]


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("change,code", ATTN)
def test_attention_refusals(lib, fp8, change, code):
    assert call_attn(lib, {**attn(fp8=fp8), **change}, fp8) == code
    assert pkv.last_error()


@pytest.mark.parametrize("change,code", [
    (dict(sc=None), -1), (dict(sc=tensor("sc", [64, 2], F32)), -1),
    (dict(sc=tensor("sc", [63, 2, 2], F32)), -1),
    (dict(sc=tensor("sc", [64, 2, 2], F32, [4, 1, 2])), -1),
    (dict(sc=tensor("sc", [64, 2, 2], F32, [5, 2, 1])), -3),
    (dict(sc=tensor("sc", [64, 2, 2], F32, ptr=PTR["sc"] + 4)), -3),
    (dict(kv=tensor("kv", [64, 2, 16, 256], BF16)), -1),
    (dict(kv=tensor("kv", [64, 2, 16, 256], FP8, [8200, 4096, 256, 1])), -3),
    (dict(kv=tensor("kv", [0, 2, 16, 256], FP8)), -1),
])
def test_8_bit_cache_refusals(lib, change, code):
    assert call_attn(lib, {**attn(), **change}) == code


def test_empty_batches_are_no_ops(lib):
    for fp8 in (True, False):
        a = attn(B=0, fp8=fp8)
        for n in ("q", "bt", "sl", "out", "lse"):
            a[n].data = None
        assert call_attn(lib, a, fp8) == 0


def append(T=4, B=4, Hkv=2, D=128, P=16):
    return dict(k=tensor("k", [T, Hkv, D], BF16), v=tensor("v", [T, Hkv, D], BF16),
                kv=tensor("kv", [64, Hkv, P, 2 * D], FP8), sc=tensor("sc", [64, Hkv, 2], F32),
                bt=tensor("bt", [B, 8], I32), sl=tensor("sl", [B], I32),
                cu=tensor("cu", [B + 1], I32), P=P)


def call_append(lib, a):
    return lib.pkv_gqa_kv_append_fp8(ref(a["k"]), ref(a["v"]), ref(a["kv"]), ref(a["sc"]),
                                     ref(a["bt"]), ref(a["sl"]), ref(a["cu"]), a["P"], None)


@pytest.mark.parametrize("change,code", [
    (dict(k=None), -1), (dict(kv=tensor("kv", [64, 2, 16, 256], BF16)), -1), (dict(P=20), -2),
    (dict(v=tensor("v", [4, 2, 64], BF16)), -1),
    (dict(v=tensor("v", [4, 2, 128], BF16, [512, 128, 1])), -1),
    (dict(kv=tensor("kv", [64, 3, 16, 256], FP8), sc=tensor("sc", [64, 3, 2], F32)), -1),
    (dict(kv=tensor("kv", [64, 2, 16, 256], FP8, [0, 4096, 256, 1])), -1),
    (dict(sc=tensor("sc", [64, 2, 2], F32, [2, 2, 1])), -1),
    (dict(cu=tensor("cu", [4], I32)), -1), (dict(cu=tensor("cu", [5], I32, [2])), -1),
    (dict(cu=tensor("cu", [5], F32)), -1),
    (dict(k=tensor("k", [5, 2, 128], BF16), v=tensor("v", [5, 2, 128], BF16), cu=None), -1),
    (dict(k=tensor("k", [4, 2, 128], BF16, ptr=PTR["k"] + 8)), -3),
    (dict(k=tensor("k", [4, 2, 128], BF16, ptr=PTR["kv"])), -1),
    (dict(bt=tensor("bt", [3, 8], I32)), -1),
])
def test_append_refusals(lib, change, code):
    assert call_append(lib, {**append(), **change}) == code


def test_append_of_nothing_is_a_no_op(lib):
    assert call_append(lib, append(T=0)) == 0
    a = append(T=0, B=0)
    a["cu"] = None
    assert call_append(lib, a) == 0


def pages(rows=4, W=8, n=3, num=50):
    return dict(bt=tensor("bt", [rows, W], I32), sl=tensor("sl", [rows], I32),
                refs=tensor("refs", [num], I32), a=tensor("a", [n], I32), b=tensor("b", [n], I32),
                c=tensor("c", [n], I32), d=tensor("d", [n], I32), one=tensor("q", [1], I32), P=16)


def call_pages(lib, what, x):
    r = {k: t if k in ("P", "window", "first") else ref(t) for k, t in x.items()}
    if what == "fork":
        return lib.pkv_pages_fork(r["bt"], r["sl"], r["refs"], r["a"], r["b"], r["P"], r["c"], r["d"], None)
    if what == "trim":
        return lib.pkv_pages_trim(r["bt"], r["sl"], r["refs"], r["P"], x.get("window", 5), x.get("first", 2), None)
    if what == "compact":
        return lib.pkv_pages_compact(r["bt"], r["sl"], r["refs"], r["P"], r["a"], r["b"], r["one"], None)
    return getattr(lib, "pkv_pages_" + what)(r["bt"], r["sl"], r["refs"], r["a"], r["b"], r["P"], None)


@pytest.mark.parametrize("what", ["fork", "release", "trim", "reserve", "compact"])
@pytest.mark.parametrize("change,code", [
    (dict(bt=None), -1), (dict(sl=tensor("sl", [3], I32)), -1), (dict(refs=None), -1),
    (dict(bt=tensor("bt", [4, 8], I32, [4, 1])), -1), (dict(bt=tensor("bt", [4, 8], I32, [8, 2])), -1),
    (dict(bt=tensor("bt", [4, 8], F32)), -1), (dict(P=0), -1),
    (dict(refs=tensor("refs", [0], I32)), -1), (dict(refs=tensor("refs", [50], I32, [2])), -1),
    (dict(refs=tensor("refs", [50], I32, ptr=PTR["bt"])), -1),
    (dict(bt=tensor("bt", [9000, 8], I32), sl=tensor("sl", [9000], I32)), -2),
])
def test_table_refusals(lib, what, change, code):
    assert call_pages(lib, what, {**pages(), **change}) == code


@pytest.mark.parametrize("change", [dict(window=0), dict(window=-3), dict(first=-1)])
def test_trim_refusals(lib, change):
    assert call_pages(lib, "trim", {**pages(), **change}) == -1
    assert call_pages(lib, "trim", pages(rows=0)) == 0


@pytest.mark.parametrize("what", ["fork", "release", "reserve", "compact"])
@pytest.mark.parametrize("change,code", [
    (dict(b=tensor("b", [2], I32)), -1), (dict(a=tensor("a", [3], I32, [2])), -1),
    (dict(a=tensor("a", [3], F32)), -1), (dict(b=tensor("b", [3], I32, ptr=PTR["bt"])), -1),
])
def test_page_call_refusals(lib, what, change, code):
    assert call_pages(lib, what, {**pages(), **change}) == code


def test_page_calls_on_empty_lists_are_no_ops(lib):
    x = pages(n=0)
    for k in "abcd":
        x[k].data = None
    for what in ("fork", "release", "reserve"):
        assert call_pages(lib, what, x) == 0


@pytest.mark.parametrize("t,code", [
    (_t([8, 4, 4], BF16, [16, 4, 1], 0x1000002), -3), (_t([8, 3], BF16, None, 0x1000000), -3),
    (_t([8, 4, 4], F32, [32, 8, 1], 0x1000000), -1), (_t([8, 4, 4], F32, [8, 4, 1], 0x1000000), -1),
    (_t([0, 4], F32, None, 0x1000000), -1), (_t([8, 4], F32, None, PTR["a"]), -1),
    (_t([8, 4], F32, None, 0), -1),
])
def test_copy_refusals(lib, t, code):
    one = (ctypes.POINTER(pkv.PkvTensor) * 2)(ctypes.pointer(t), ctypes.pointer(t))
    a, b = tensor("a", [3], I32), tensor("b", [3], I32)
    assert lib.pkv_pages_copy(ctypes.cast(one, ctypes.c_void_p), 1, ref(a), ref(b), None) == code


def test_copy_refuses_lists_and_counts(lib):
    t = _t([8, 4], F32, None, 0x1000000)
    two = (ctypes.POINTER(pkv.PkvTensor) * 2)(ctypes.pointer(t), ctypes.pointer(t))
    p = ctypes.cast(two, ctypes.c_void_p)
    a, b, short = tensor("a", [3], I32), tensor("b", [3], I32), tensor("c", [2], I32)
    assert lib.pkv_pages_copy(None, 1, ref(a), ref(b), None) == -1
    assert lib.pkv_pages_copy(p, 0, ref(a), ref(b), None) == -1
    assert lib.pkv_pages_copy(p, 65, ref(a), ref(b), None) == -1
    assert lib.pkv_pages_copy(p, 1, ref(a), ref(short), None) == -1
    assert lib.pkv_pages_copy(p, 2, ref(a), ref(b), None) == -1  # the same cache twice
    with pytest.raises(pkv.PkvError):
        pkv.pages_copy([], torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


# ------------------------------------------------- the plain implementations --
def test_plain_encoder_is_the_oracles():
    g = torch.Generator().manual_seed(0)
    x = torch.cat([torch.randn(3000, generator=g) * 50, torch.randn(500, generator=g) * 1e-3,
                   (plain.E4M3[1:] + plain.E4M3[:-1]).float() / 2, plain.E4M3.float(),
                   torch.tensor([464.0, 465.0, 1e9, 0.0])])
    x = torch.cat([x, -x])
    lib = oracle.load()
    want = [lib.pkv_oracle_e4m3_to_f64(lib.pkv_oracle_f32_to_e4m3(float(v))) for v in x]
    assert torch.equal(plain.encode(x), torch.tensor(want, dtype=torch.float64))


def test_plain_decode_is_the_oracles_without_first_tokens():
    from paged_kv_cache_30_gb300 import workloads as W
    pr = W.gqa_problem(1, B=5, Hq=16, Hkv=2, page_size=16, lengths="uniform", Lmin=0, Lmax=90,
                       sinks=True, window=20)
    scale = ctypes.c_float(pr.scale).value  # as the C ABI takes it
    out, lse, tol, _ = plain.decode(pr.q, pr.kv_cache, None, pr.block_table, pr.seq_lens, pr.sinks,
                                    20, 0, scale, 16, 2.0 ** -8)
    want, want_lse = oracle.gqa_decode(pr.q, pr.kv_cache, pr.block_table, pr.seq_lens, pr.sinks, 20,
                                       pr.scale, 16)
    assert torch.allclose(out.view(-1), torch.from_numpy(want).view(-1), atol=1e-12, rtol=1e-12)
    fin = torch.isfinite(lse.view(-1))
    assert torch.allclose(lse.view(-1)[fin], torch.from_numpy(want_lse).view(-1)[fin], atol=1e-12)
    assert (tol[pr.seq_lens > 0] > 0).all()


def test_plain_visibility():
    assert plain.visible(10, 3, 2).tolist() == [0, 1, 7, 8, 9]
    assert plain.visible(10, 0, 2).tolist() == list(range(10))
    assert plain.visible(4, 3, 2).tolist() == [0, 1, 2, 3]
    assert plain.visible(0, 3, 2).tolist() == []
