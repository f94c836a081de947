"""CPU test of the host's note of page calls (csrc/page_order.h): which attention call gets a
memset before it, in streams and in captures."""
import ctypes
import shutil
import subprocess

import pytest

from paged_kv_cache_30_gb300 import build as pkv_build

CODE = """
#include "page_order.h"
static pkv::PageOrder* o = nullptr;
extern "C" void fresh() { delete o; o = new pkv::PageOrder(); }
extern "C" int wrote(long s, unsigned long long c) { return o->wrote((const void*)s, c); }
extern "C" int settle(long s, unsigned long long c) { return o->settle((const void*)s, c); }
extern "C" int due(long s, unsigned long long c) { return o->due((const void*)s, c); }
extern "C" void settled(long s, unsigned long long c) { o->settled((const void*)s, c); }
extern "C" int size() { return o->size(); }
"""
S, T = 0x1000, 0x2000  # streams


@pytest.fixture(scope="module")
def built(tmp_path_factory):
    d = tmp_path_factory.mktemp("page_order")
    (d / "t.cpp").write_text(CODE)
    subprocess.run([shutil.which("g++") or "c++", "-std=c++17", "-shared", "-fPIC", "-I", pkv_build.CSRC,
                    str(d / "t.cpp"), "-o", str(d / "t.so")], check=True)
    lib = ctypes.CDLL(str(d / "t.so"))
    for f in (lib.wrote, lib.settle, lib.due, lib.settled):
        f.argtypes = [ctypes.c_long, ctypes.c_ulonglong]
    return lib


@pytest.fixture
def o(built):
    built.fresh()
    return built


def test_the_first_attention_call_after_a_page_call(o):
    assert not o.settle(S, 0)
    assert not o.wrote(S, 0) and not o.wrote(S, 0)
    assert not o.settle(T, 0)  # another stream: events order it
    assert o.settle(S, 0) and not o.settle(S, 0)
    assert o.size() == 0


def test_a_capture_settles_nothing_of_the_stream(o):
    assert not o.wrote(S, 0)
    assert not o.settle(S, 7)  # recorded, not run
    assert o.settle(S, 0)


def test_a_captured_page_call_concerns_its_capture_alone(o):
    assert not o.wrote(S, 7)
    assert not o.settle(S, 0)
    assert not o.settle(S, 8)
    assert o.settle(S, 7) and not o.settle(S, 7)
    assert not o.wrote(S, 7) and o.settle(S, 7)


def test_both_at_once(o):
    assert not o.wrote(S, 0) and not o.wrote(S, 7)
    assert o.settle(S, 7) and not o.settle(S, 7)
    assert o.settle(S, 0) and not o.settle(S, 0)


def test_page_calls_of_another_stream_in_the_capture(o):
    """Joined by an event at any time: every call of the other stream is ordered."""
    assert not o.settle(T, 7)
    assert not o.wrote(S, 7)
    assert o.settle(T, 7) and o.settle(T, 7)
    assert o.settle(S, 7) and not o.settle(S, 7)
    assert o.settle(T, 7)


def test_a_later_capture_takes_the_streams_place(o):
    for c in range(1, 500):
        assert not o.wrote(S, c)
        assert not o.settle(T, c - 1)  # the capture before is over
    assert o.size() == 1
    assert o.settle(S, 499)


def test_no_more_than_64_streams_are_kept(o):
    for i in range(64):
        assert not o.wrote(0x1000 + 16 * i, 0)
    for i in range(64, 500):
        assert o.wrote(0x1000 + 16 * i, 0)  # the memset goes in at once
        assert not o.settle(0x1000 + 16 * i, 0)
    assert o.size() == 64
    for i in range(64):
        assert o.settle(0x1000 + 16 * i, 0)
    assert o.size() == 0


def test_the_default_streams_handles(o):
    assert not o.wrote(0, 0) and o.settle(1, 0)  # two names of one stream
    assert not o.wrote(1, 0) and o.settle(0, 0)
    assert o.wrote(2, 0) and not o.settle(2, 0)  # one name of a stream for each thread


@pytest.mark.parametrize("c", [0, 7])
def test_a_call_that_fails_settles_nothing(o, c):
    """It asks what is due; only what is in the stream settles it."""
    assert not o.wrote(S, c)
    assert o.due(S, c) and o.due(S, c)
    o.settled(T, c)
    o.settled(S, 9)
    assert o.due(S, c)
    o.settled(S, c)
    assert not o.due(S, c)
    o.settled(S, c)
    assert not o.wrote(S, c) and o.due(S, c)
