"""CPU-side checks of the decode calls with shared tokens: what is refused, with its code, before
any CUDA call; and the plain implementation that the GPU tests compare with."""
import math

import pytest
import torch

import paged_kv_cache_30_gb300 as pkv
from paged_kv_cache_30_gb300 import build as pkv_build
from tests import paged_plain
from tests import prefix_plain as plain
from tests.test_paged_abi import ATTN, BF16, F32, FP8, I32, attn, ref, tensor


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return pkv.load_library()


def args(fp8=True, **kw):
    return dict(attn(fp8=fp8, **kw), cu=tensor("cu", [2], I32), shared=tensor("a", [1], I32))


def call(lib, a, fp8=True):
    tail = (ref(a["bt"]), ref(a["sl"]), ref(a["cu"]), ref(a["shared"]), ref(a["sinks"]), a["scale"],
            a["P"], ref(a["out"]), ref(a["lse"]), None)
    if fp8:
        return lib.pkv_paged_prefix_attn_fp8(ref(a["q"]), ref(a["kv"]), ref(a["sc"]), *tail)
    return lib.pkv_paged_prefix_attn(ref(a["q"]), ref(a["kv"]), *tail)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("change,code", [(c, k) for c, k in ATTN if "first" not in c] + [
    (dict(cu=None), -1), (dict(shared=None), -1), (dict(cu=tensor("cu", [3], I32)), -1),
    (dict(cu=tensor("cu", [2], F32)), -1), (dict(cu=tensor("cu", [2], I32, [2])), -1),
    (dict(shared=tensor("a", [1], F32)), -1), (dict(shared=tensor("a", [1, 1], I32)), -1),
    (dict(shared=tensor("a", [2], I32, [2]), cu=tensor("cu", [3], I32)), -1),
    (dict(shared=tensor("a", [2049], I32), cu=tensor("cu", [2050], I32)), -1),
    (dict(out=tensor("cu", [2, 16, 128], BF16)), -1), (dict(lse=tensor("a", [2, 16], F32)), -1),
    (dict(kv=tensor("kv", [64, 2, 16, 256], F32)), -1),
])
def test_refusals(lib, fp8, change, code):
    assert call(lib, {**args(fp8), **change}, fp8) == code
    assert pkv.last_error()


def test_nothing_to_do_is_a_no_op(lib):
    for fp8 in (True, False):
        a = args(fp8, B=0)
        for n in ("q", "bt", "sl", "out", "lse"):
            a[n].data = None
        assert call(lib, a, fp8) == 0
        a = {**args(fp8), "cu": tensor("cu", [1], I32), "shared": tensor("a", [0], I32)}
        a["shared"].data = None
        assert call(lib, a, fp8) == 0


@pytest.mark.parametrize("fp8", [True, False])
def test_plain_forms_agree(fp8):
    groups = [(40, [50, 0, 41]), (33, [60, 35]), (0, [5])]
    pr = plain.problem(1, groups, 2, 3, 64, 16, fp8, sinks=True)
    out, lse, _, _ = plain.decode(pr)
    o2, l2, _, _ = paged_plain.decode(pr["q"], pr["kv"], pr["sc"], pr["bt"], pr["sl"], pr["sinks"], 0, 0,
                                      pr["scale"], 16, 2.0 ** -8)
    assert torch.allclose(out, o2, rtol=1e-12, atol=1e-14)
    assert torch.equal(lse == -math.inf, l2 == -math.inf)
    assert torch.allclose(lse[lse > -math.inf], l2[l2 > -math.inf], rtol=1e-12)
    # requests of a group hold the same first tokens
    for at, (S, Ls) in zip(pr["cu"].tolist(), groups):
        rows = [at + i for i, L in enumerate(Ls) if L]
        pos = torch.arange(S)
        got = [pr["kv"].float()[pr["bt"][b].long()[pos // 16], :, pos % 16] for b in rows]
        if fp8:
            got = [x * pr["sc"][pr["bt"][b].long()[pos // 16]].repeat_interleave(64, 2)
                   for x, b in zip(got, rows)]
        assert all(torch.equal(x, got[0]) and x.isfinite().all() for x in got)
