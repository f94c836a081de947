"""GPU page calls in a pool that keeps running out: the error word names that exactly after the
calls that refused an entry for want of pages, and is clear after all others."""
import random

import pytest
import torch

import paged_kv_cache_30_gb300 as pkv
from tests import paged_plain as plain
from tests.test_pages_gpu import Device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    pkv.load_library()
    pkv.init(0)


class Pool(plain.Pool):
    """`refused`: the last call left out an entry for want of pages (rows valid, named once)."""

    refused = False

    def reserve(self, rows, lens):
        super().reserve(rows, lens)
        self.refused = any(self.lens[r] < n for r, n in zip(rows, lens))

    def fork(self, parents, children):
        out = super().fork(parents, children)
        self.refused = any(self.lens[c] < self.lens[p] for p, c in zip(parents, children))
        return out

    def release(self, rows, keep):
        super().release(rows, keep)
        self.refused = False

    def trim(self, window, first):
        super().trim(window, first)
        self.refused = False

    def compact(self, most):
        self.refused = False
        return super().compact(most)


def flag():
    try:
        return pkv.check_errors(0)
    except pkv.PkvError as e:
        return e.code


@pytest.mark.parametrize("P,pages,rows,width", [(16, 40, 20, 12), (32, 150, 100, 12), (1, 30, 9, 40),
                                                (16, 2500, 300, 80)])
def test_the_flag_is_raised_when_the_pool_runs_out_and_only_then(P, pages, rows, width):
    rng = random.Random(P + pages)
    m = Pool(rows, width, pages, P)
    d = Device(m)
    seen = {"reserve": set(), "fork": set()}
    for step in range(80):
        pick = rng.sample(range(rows), rng.randint(1, rows))
        what = rng.choice(["reserve", "reserve", "release", "fork", "fork", "trim", "compact"])
        if what == "reserve":
            most = rng.choice([P, 3 * P, width * P])
            lens = [rng.randint(0, most) for _ in pick]
            m.reserve(pick, lens)
            d.reserve(pick, lens)
        elif what == "release":
            keep = [rng.choice([0, 0, rng.randint(0, width * P)]) for _ in pick]
            m.release(pick, keep)
            d.release(pick, keep)
        elif what == "fork":
            kids = [r for r in pick if m.lens[r] == 0][:rng.randint(1, 30)]
            full = [r for r in range(rows) if m.lens[r] > 0]
            if not kids or not full:
                continue
            par = [rng.choice(full) for _ in kids]
            src, dst = m.fork(par, kids)
            s, t = d.fork(par, kids)
            assert s.tolist() == src and t.tolist() == dst
        elif what == "trim":
            window = rng.randint(1, width * P)
            m.trim(window, 0)
            d.trim(window, 0)
        else:
            m.compact(pages // 2)
            d.compact(pages // 2)
        assert d.same(m), f"step {step}: {what}"
        assert flag() == (-8 if m.refused else 0), f"step {step}: {what}"
        if what in seen:
            seen[what].add(m.refused)
    assert seen["reserve"] == {True, False}
    assert P == 1 or seen["fork"] == {True, False}  # a page of one token is never partly filled
