"""GPU attention calls that read tables early, right behind page calls: with a capture begun in
between, and with the page call on another stream of the capture."""
import ctypes

import pytest
import torch

import paged_kv_cache_30_gb300 as pkv

pytestmark = pytest.mark.gpu

P, PAGES = 16, 4096


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    pkv.load_library()
    pkv.init(0)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def state():
    g = torch.Generator(device="cuda").manual_seed(3)
    return dict(kv=torch.randn(PAGES, 1, P, 256, device="cuda", generator=g).bfloat16(),
                q=torch.randn(2, 8, 128, device="cuda", generator=g).bfloat16(),
                bt=torch.full((2, 200), -1, dtype=torch.int32, device="cuda"), sl=ints([0, 0]),
                refs=ints([0] * PAGES), rows=ints([0, 1]), zero=ints([0, 0]),
                outs=[torch.zeros(2, 8, 128, device="cuda").bfloat16() for _ in range(3)])


def change(s, lens):
    pkv.pages_release(s["bt"], s["sl"], s["refs"], s["rows"], s["zero"], P)
    pkv.pages_reserve(s["bt"], s["sl"], s["refs"], s["rows"], lens, P)


def attend(s, out):
    pkv.paged_decode_attn(s["q"], s["kv"], s["bt"], s["sl"], None, 0, 0.09, P, 0, out)


def test_eager_calls_around_a_capture():
    """Page calls, a capture that records an attention call, an attention call."""
    s = state()
    stream = torch.cuda.Stream()
    lens = [ints([i * 70, 3000 - i * 70]) for i in range(1, 40)]
    attend(s, s["outs"][2])
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for n in lens:
            graph = torch.cuda.CUDAGraph()
            change(s, n)
            graph.capture_begin(capture_error_mode="thread_local")
            attend(s, s["outs"][2])
            graph.capture_end()
            attend(s, s["outs"][0])
            torch.cuda.synchronize()
            attend(s, s["outs"][1])
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(s["outs"][0], s["outs"][1])
            assert torch.equal(s["outs"][0], s["outs"][2])
    assert pkv.check_errors(0) == 0
    assert pkv.check_counters(0) == 0


def test_captured_page_calls_on_another_stream():
    s = state()
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    lens = ints([0, 0])
    attend(s, s["outs"][2])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(main):
        graph.capture_begin(capture_error_mode="thread_local")
        attend(s, s["outs"][2])
        side.wait_stream(main)
        with torch.cuda.stream(side):
            change(s, lens)
        main.wait_stream(side)
        attend(s, s["outs"][0])
        graph.capture_end()
    for i in range(1, 40):
        lens.copy_(ints([i * 70, 3000 - i * 70]))
        graph.replay()
        torch.cuda.synchronize()
        attend(s, s["outs"][1])
        torch.cuda.synchronize()
        assert torch.equal(s["outs"][0], s["outs"][1])
    assert pkv.check_errors(0) == 0
    assert pkv.check_counters(0) == 0


def test_a_stream_for_each_page_call():
    """More streams than are remembered."""
    s = state()
    cudart = torch.cuda.cudart()
    handles = [ctypes.c_void_p() for _ in range(100)]
    for h in handles:
        assert int(cudart.cudaStreamCreate(ctypes.addressof(h))) == 0
    streams = [torch.cuda.ExternalStream(h.value) for h in handles]
    torch.cuda.synchronize()
    for i, stream in enumerate(streams):
        with torch.cuda.stream(stream):
            change(s, ints([i * 20 + 1, 2500 - i * 20]))
            torch.cuda.synchronize()
    for i, stream in enumerate(streams[::-1]):
        lens = ints([i * 20 + 5, 2400 - i * 20])
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            change(s, lens)
            attend(s, s["outs"][0])
            torch.cuda.synchronize()
            attend(s, s["outs"][1])
            torch.cuda.synchronize()
            assert torch.equal(s["outs"][0], s["outs"][1])
    attend(s, s["outs"][1])  # the library's last stream is one that stays
    torch.cuda.synchronize()
    for h in handles:
        assert int(cudart.cudaStreamDestroy(h.value)) == 0
    assert pkv.check_errors(0) == 0


def test_a_call_on_another_stream_while_the_last_one_is_captured():
    """The capture of the last call's stream records nothing of it: it runs at once."""
    s = state()
    with torch.cuda.stream(torch.cuda.Stream()):
        change(s, ints([700, 900]))
        torch.cuda.synchronize()
    last, other = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(last):
        attend(s, s["outs"][0])
        torch.cuda.synchronize()
        graph.capture_begin(capture_error_mode="relaxed")
        attend(s, s["outs"][2])
        with torch.cuda.stream(other):
            attend(s, s["outs"][1])
        other.synchronize()
        graph.capture_end()
    assert torch.equal(s["outs"][0], s["outs"][1])
    assert not s["outs"][2].any()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(s["outs"][0], s["outs"][2])
    assert pkv.check_errors(0) == 0
