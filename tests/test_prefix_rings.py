"""CPU model of the barriers of csrc/prefix_attn.cu: its roles (TMA producers, MMA issuers, softmax
threads, e4m3 converters) as coroutines in any order, copies and products that end any time later,
and barriers that tell two phases apart and no more, as an mbarrier's parity does.  Memory holds
who wrote it; it is an error to write what is still to be read, to read what is not there, and to
wait for ever.  Places, phases and the order of operands are those of csrc/prefix_ring.h."""
import ctypes
import random
import shutil
import subprocess

import pytest

from paged_kv_cache_30_gb300 import build as pkv_build

CODE = """
#include "prefix_ring.h"
#define RING(NAME, OPS, EXTRA) \\
  extern "C" void* NAME() { return new pkv::OpRing<OPS, EXTRA>(); } \\
  extern "C" void NAME##_begin(void* r, int dual) { ((pkv::OpRing<OPS, EXTRA>*)r)->begin(dual); } \\
  extern "C" int NAME##_place(void* r, int n) { return ((pkv::OpRing<OPS, EXTRA>*)r)->place(n); } \\
  extern "C" int NAME##_phase(void* r, int n) { return ((pkv::OpRing<OPS, EXTRA>*)r)->phase(n); } \\
  extern "C" void NAME##_end(void* r, int n) { ((pkv::OpRing<OPS, EXTRA>*)r)->end(n); } \\
  extern "C" void NAME##_gone(void* r) { delete (pkv::OpRing<OPS, EXTRA>*)r; }
RING(ring8, 8, false) RING(ring4, 4, false) RING(ring6, 6, false) RING(ring3, 3, true)
extern "C" int keys(int by, int T, int t) { return pkv::OperandOrder{by != 0, T}.keys(t); }
extern "C" int values(int by, int T, int t) { return pkv::OperandOrder{by != 0, T}.values(t); }
extern "C" int are_values(int by, int T, int n) { return pkv::OperandOrder{by != 0, T}.are_values(n); }
extern "C" int tile_of(int by, int T, int n) { return pkv::OperandOrder{by != 0, T}.tile_of(n); }
"""
# cache, head dim: operand places, raw places, ring
CONFIGS = {"bf16-64": (8, 0, "ring8"), "bf16-128": (4, 0, "ring4"), "e4m3-64": (6, 6, "ring6"),
           "e4m3-128": (3, 3, "ring3")}
SCALES = 8


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    d = tmp_path_factory.mktemp("rings")
    (d / "t.cpp").write_text(CODE)
    subprocess.run([shutil.which("g++") or "c++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    pkv_build.CSRC, str(d / "t.cpp"), "-o", str(d / "t.so")], check=True)
    lib = ctypes.CDLL(str(d / "t.so"))
    for r in ("ring8", "ring4", "ring6", "ring3"):
        getattr(lib, r).restype = ctypes.c_void_p
        for f in ("_begin", "_place", "_phase", "_end", "_gone"):
            getattr(lib, r + f).argtypes = [ctypes.c_void_p] + [ctypes.c_int] * (f != "_gone")
    return lib


class Wrong(Exception):
    pass


def must(ok, *what):
    if not ok:
        raise Wrong(what)


class Bar:
    def __init__(self, count):
        self.count = self.left = count
        self.tx = self.phase = 0

    def step(self, arrive=0, tx=0):
        self.left -= arrive
        self.tx += tx
        must(self.left >= 0, "an arrival too many")
        if self.left == 0 and self.tx == 0:
            self.phase += 1
            self.left = self.count

    def done(self, parity):
        return (self.phase & 1) != (parity & 1)


class Cell:  # an operand's place, or a query tile's
    what, parts, reads = None, 0, 0

    def write(self, what, reads):
        if self.what != what:
            must(self.reads == 0, "written over", self.what, "by", what)
            self.what, self.parts, self.reads = what, 0, reads

    def read(self, what, parts):
        must(self.what == what and self.parts == parts and self.reads > 0, "read", what, "found", self.what,
             self.parts)
        self.reads -= 1


class Model:
    def __init__(self, code, config, units, seed, mistake):
        self.code, self.units, self.rnd, self.mistake = code, units, random.Random(seed), mistake
        self.ops, self.raws, self.ring_name = CONFIGS[config]
        self.fp8 = self.raws > 0
        bars = lambda n, count: [Bar(count) for _ in range(n)]  # noqa: E731
        self.op_full, self.op_empty = bars(8, 1 if self.fp8 else 2), bars(8, 2)
        self.raw_full, self.raw_empty = bars(6, 1), bars(6, 1)
        self.s_full, self.p_ready, self.o_done = bars(2, 1), bars(2, 1), bars(2, 1)
        self.p_half, self.turn, self.scale_full = bars(2, 1), bars(2, 1), bars(SCALES, 1)
        self.q_full, self.q_free = Bar(2), Bar(2)
        self.cell = [Cell() for _ in range(self.ops)]
        self.q = [Cell(), Cell()]
        self.cell.append(self.q[1])  # the extra place is the other query tile's
        self.raw = [Cell() for _ in range(6)]
        self.scale = [None] * SCALES
        self.s, self.o = [None, None], [None, None]  # in tensor memory
        self.scratch = [None, None]  # rows' powers of two, or slot 1's m and l
        self.named = {1: 0, 2: 0}
        self.copies, self.queue = [], ([], [])

    def ring(self):
        r = getattr(self.code, self.ring_name)()
        f = lambda name: lambda *a: getattr(self.code, self.ring_name + name)(r, *a)  # noqa: E731
        return f("_begin"), f("_place"), f("_phase"), f("_end"), f("_gone")

    def order(self, T, dual):
        by = int(self.fp8 or dual)
        return [lambda x, f=f: f(by, T, x) for f in (self.code.keys, self.code.values, self.code.are_values,
                                                     self.code.tile_of)]

    def wait(self, bar, parity):
        while not bar.done(parity):
            yield

    def rendezvous(self, name):  # of both slots' threads
        self.named[name] += 1
        target = (self.named[name] + 1) // 2 * 2
        while self.named[name] < target:
            yield

    def copy(self, cell, what, bar, reads):
        cell.write(what, reads)
        self.copies.append((cell, what, bar))

    def producer(self, half):
        begin, place, phase, end, gone = self.ring()
        op = tiles = 0
        for k, (T, dual) in enumerate(self.units):
            _, _, are_values, tile_of = self.order(T, dual)
            begin(dual)
            for n in range(2 * T):
                if self.mistake == "a producer of keys and one of values" and are_values(n) != half:
                    op += 1
                    continue
                if self.fp8:
                    e = op % self.raws
                    yield from self.wait(self.raw_empty[e], op // self.raws ^ 1)
                    cell, bar = self.raw[e], self.raw_full[e]
                else:
                    e = place(n)
                    yield from self.wait(self.op_empty[e], phase(n) ^ 1)
                    cell, bar = self.cell[e], self.op_full[e]
                split = self.mistake != "a producer of keys and one of values"
                for _ in range(1 if split else 2):
                    bar.step(arrive=1, tx=1)
                    self.copy(cell, (k, n), bar, 1 if self.fp8 or not dual else 2)
                if self.fp8 and not are_values(n):
                    at = (tiles + tile_of(n)) % SCALES
                    self.scale[at] = (k, tile_of(n))
                    self.scale_full[at].step(arrive=1)
                op += 1
                yield
            tiles += T
            end(2 * T)
        gone()

    def converter(self):
        begin, place, phase, end, gone = self.ring()
        op = 0
        for k, (T, dual) in enumerate(self.units):
            begin(dual)
            for n in range(2 * T):
                er, eo = op % self.raws, place(n)
                yield from self.wait(self.raw_full[er], op // self.raws)
                self.raw[er].read((k, n), 1)
                yield from self.wait(self.op_empty[eo], phase(n) ^ 1)
                self.cell[eo].write((k, n), 2 if dual else 1)
                yield
                self.cell[eo].parts = 2
                self.raw_empty[er].step(arrive=1)
                self.op_full[eo].step(arrive=1)
                op += 1
                yield
            end(2 * T)
        gone()

    # what the tensor cores do when they come to it
    def products(self, slot, k, n, cell, q, j):
        def s():
            must(self.s[slot] is None or self.s[slot][0] == "used", "scores over", self.s[slot])
            self.q[q].read(("q", k), 2)
            cell.read((k, n), 2)
            self.s[slot] = ("scores", k, j)

        def pv():
            must(self.s[slot] == ("weights", k, j), "weights", k, j, "found", self.s[slot])
            cell.read((k, n), 2)
            must(j > 1 or self.o[slot] is None, "sums over", self.o[slot])
            self.o[slot] = ("sums", k)
            self.s[slot] = ("used",)
        return s if q is not None else pv

    def issuer(self, slot):
        begin, place, phase, end, gone = self.ring()
        before = ready = turns = 0
        queue = self.queue[slot]
        commit = lambda bar: queue.append(lambda: bar.step(arrive=1))  # noqa: E731
        for k, (T, dual) in enumerate(self.units):
            steps = 2 * T if dual else T
            keys, values, _, _ = self.order(T, dual)
            begin(dual)
            yield from self.wait(self.q_full, k)

            def release(n):
                for _ in range(1 if dual or self.mistake == "given back once" else 2):
                    commit(self.op_empty[place(n)])

            def wait_op(n):
                yield from self.wait(self.op_full[place(n)], phase(n))
            tile = lambda j: j >> 1 if dual else j  # noqa: E731
            if slot >= steps:
                self.q_free.step(arrive=1)
            for j in range(slot - 2, steps, 2):
                first, more = j < 0, j + 2 < steps
                if first and not more:
                    continue
                kn = keys(tile(j + 2)) if more else 0
                vn = 0 if first else values(tile(j))
                early = not self.fp8 or dual or first
                if more and early:
                    yield from wait_op(kn)
                if not first:
                    yield from wait_op(vn)
                    yield from self.wait(self.p_half[slot], ready)
                if (slot == 1 or before == 1) if first else steps > 1:
                    yield from self.wait(self.turn[slot], turns)
                    turns += 1
                if not first:
                    yield from self.wait(self.p_ready[slot], ready)
                    queue.append(self.products(slot, k, vn, self.cell[place(vn)], None, j))
                    ready += 1
                    release(vn)
                    if not more:
                        commit(self.o_done[slot])
                    yield
                    if more and not early:
                        yield from wait_op(kn)
                if more:
                    queue.append(self.products(slot, k, kn, self.cell[place(kn)], slot if dual else 0, j + 2))
                if slot == 1 or (steps > 1 if first else j + 1 < steps):
                    self.turn[slot ^ 1].step(arrive=1)
                yield
                if more:
                    commit(self.s_full[slot])
                    release(kn)
                    if j + 4 >= steps:
                        commit(self.q_free)
            before = (steps - 1) & 1
            end(2 * T)
        gone()

    def softmax(self, slot):
        got, tiles, done = 0, 0, [0, 0]
        for k, (T, dual) in enumerate(self.units):
            steps = 2 * T if dual else T
            if k > 0:
                yield from self.wait(self.q_free, k - 1)
            q = self.q[slot if dual else 0]
            q.write(("q", k), T)
            q.parts += 2 if dual else 1
            if self.fp8:
                self.scratch[slot] = ("scale", k)
            yield
            self.q_full.step(arrive=1)
            if self.fp8:
                yield from self.rendezvous(1)
                yield
                must(self.scratch == [("scale", k)] * 2, "powers of two of", k, "found", self.scratch)
                if self.mistake != "powers of two written over":
                    yield from self.rendezvous(1)
            for j in range(slot, steps, 2):
                yield from self.wait(self.s_full[slot], got)
                got += 1
                t = j >> 1 if dual else j
                if self.fp8:
                    at = (tiles + t) % SCALES
                    yield from self.wait(self.scale_full[at], (tiles + t) // SCALES)
                    must(self.scale[at] == (k, t), "scales of", k, t, "found", self.scale[at])
                must(self.s[slot] == ("scores", k, j), "scores", k, j, "found", self.s[slot])
                yield
                if self.fp8:
                    must(self.scale[at] == (k, t), "scales of", k, t, "found", self.scale[at])
                self.p_half[slot].step(arrive=1)
                yield
                self.s[slot] = ("weights", k, j)
                self.p_ready[slot].step(arrive=1)
                yield
            both = steps > 1
            if not dual:
                if slot == 1:
                    self.scratch = [("ml", k)] * 2
                yield from self.rendezvous(1)
                if slot == 0:
                    must(self.scratch == [("ml", k)] * 2, "m and l of", k, "found", self.scratch)
            if slot == 0 or dual:
                yield from self.wait(self.o_done[slot], done[slot])
            if not dual and slot == 0 and both:
                yield from self.wait(self.o_done[1], done[1])
            done[0] += 1
            done[1] += both
            yield
            for o in ([slot] if dual else [0, 1][:1 + both] if slot == 0 else []):
                must(self.o[o] == ("sums", k), "sums of", k, "found", self.o[o])
                self.o[o] = None
            if not dual:
                yield from self.rendezvous(2)
            tiles += T

    def run(self):
        roles = [self.producer(0), self.issuer(0), self.issuer(1), self.softmax(0), self.softmax(1)]
        roles.append(self.converter() if self.fp8 else self.producer(1))
        bars = [b for v in vars(self).values() if isinstance(v, list) for b in v if isinstance(b, Bar)]
        bars += [self.q_full, self.q_free]
        idle, last = 0, None
        while roles:
            what = self.rnd.randrange(len(roles) + 3)
            if what >= len(roles) + 1:
                queue = self.queue[what - len(roles) - 1]
                if queue:
                    queue.pop(0)()
            elif what == len(roles):
                if self.copies:
                    cell, which, bar = self.copies.pop(self.rnd.randrange(len(self.copies)))
                    must(cell.what == which, "a copy of", which, "came to", cell.what)
                    cell.parts += 1
                    bar.step(tx=-1)
            else:
                try:
                    next(roles[what])
                except StopIteration:
                    del roles[what]
            idle += 1
            if idle % 500 == 0:  # long enough for all to move that can
                state = ([(b.phase, b.left, b.tx) for b in bars], len(self.copies), len(roles),
                         [len(q) for q in self.queue], dict(self.named))
                must(state != last, "nothing moves")
                last = state


def units_of(seed):
    r = random.Random(seed)
    return [(r.choice([1, 1, 2, 3, r.randint(1, 12)]), r.randrange(2)) for _ in range(r.randint(1, 9))]


@pytest.mark.parametrize("config", CONFIGS)
def test_units_in_any_order_at_any_speed(code, config):
    for seed in range(60):
        Model(code, config, units_of(seed), seed, None).run()
    Model(code, config, [(1, 0)] * 30 + [(1, 1)] * 30, 1, None).run()
    Model(code, config, [(40, 0), (40, 1)], 2, None).run()


@pytest.mark.parametrize("config,mistake", [
    ("bf16-128", "a producer of keys and one of values"), ("e4m3-64", "powers of two written over"),
    ("e4m3-128", "powers of two written over"), ("bf16-64", "given back once")])
def test_the_model_sees_mistakes(code, config, mistake):
    with pytest.raises(Wrong):
        for seed in range(20):
            Model(code, config, units_of(seed), seed, mistake).run()


def test_the_model_has_the_kernel_s_rings():
    """Places and raw places of the configurations above, from the kernel's source."""
    with open(f"{pkv_build.CSRC}/prefix_attn.cu") as f:
        text = f.read()
    assert "kOps = D == 64 ? (kFp8 ? 6 : 8) : (kFp8 ? 3 : 4);" in text
    assert "kRaws = D == 64 ? 6 : 3;" in text
    assert "kExtraOp = kOps == 3;" in text
    assert f"kScaleTiles = {SCALES};" in text
