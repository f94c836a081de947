"""GPU calls that share the workspace, made by several threads on streams of their own at once:
each result is what the same call gives alone."""
import threading

import pytest
import torch

import paged_kv_cache_30_gb300 as pkv
from tests.test_paged_attn_gpu import call, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    pkv.load_library()
    pkv.init(0)


def cuda(pr):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in pr.items()}


def test_attention_of_three_threads():
    """Requests that are cut into parts: their partials and counters lie in the workspace."""
    jobs = []
    for seed, fp8 in ((1, True), (2, False), (3, True)):
        d = cuda(problem(seed, [9000 + seed, 5000, 33, 7000], 2, 8, 128, 16, fp8))
        want = torch.empty_like(d["q"])
        call(d, want, None)
        torch.cuda.synchronize()
        outs = [torch.full_like(d["q"], float("nan")) for _ in range(60)]
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
    for d, want, outs, _ in jobs:
        for out in outs:
            assert torch.equal(out, want)
    assert pkv.check_errors(0) == 0
    assert pkv.check_counters(0) == 0


def test_page_calls_of_two_threads():
    """Forks and reservations plan in the workspace."""
    P, rows, width, n = 16, 64, 300, 40

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    jobs = []
    for seed in (1, 2):
        s = dict(bt=torch.full((rows, width), -1, dtype=torch.int32, device="cuda"), sl=ints([0] * rows),
                 refs=ints([0] * 20000), rows=ints(list(range(rows))), zero=ints([0] * rows),
                 lens=ints([(37 * i * seed) % (width * P) for i in range(rows)]))
        s["held"] = torch.empty(n, rows, width, dtype=torch.int32, device="cuda")
        jobs.append((s, torch.cuda.Stream()))
    torch.cuda.synchronize()
    failed, start = [], threading.Barrier(len(jobs))

    def step(s, stream, i):
        args = s["bt"], s["sl"], s["refs"], s["rows"]
        pkv.pages_reserve(*args, s["lens"], P, stream)
        with torch.cuda.stream(stream):
            s["held"][i].copy_(s["bt"])
        pkv.pages_release(*args, s["zero"], P, stream)

    def work(s, stream):
        try:
            start.wait()
            for i in range(n):
                step(s, stream, i)
        except Exception as e:  # noqa: BLE001 (shown below)
            failed.append(e)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for s, stream in jobs:
        got = s["held"].clone()
        torch.cuda.synchronize()
        step(s, stream, 0)
        torch.cuda.synchronize()
        assert (got == s["held"][0]).all()
        assert not s["refs"].any()
    assert pkv.check_errors(0) == 0
