"""The chunk entry points' refusals and launch plans, on the host: td_chunks.cpp built with
stand-ins for the CUDA runtime and the kernels (tests/chunk_host.cpp)."""
from __future__ import annotations

import ctypes as C
import os
import random
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def td():
    from collective_kv_cache_gb300 import build
    build.build()
    from collective_kv_cache_gb300 import td as _td
    return _td


@pytest.fixture(scope="module")
def lib(td, tmp_path_factory):
    from collective_kv_cache_gb300 import build
    out = str(tmp_path_factory.mktemp("chunk_host") / "libchunk_host.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-Wall",
                    # its own stand-ins, not a CUDA runtime that the process has loaded
                    "-Wl,-Bsymbolic", "-I", build.INC, "-I",
                    build.CSRC, "-I", os.path.join(build.CUDA_HOME, "include"),
                    os.path.join(build.CSRC, "td_chunks.cpp"),
                    os.path.join(ROOT, "tests", "chunk_host.cpp"), "-o", out], check=True)
    h = C.CDLL(out)
    h.fake_ctx.restype = C.c_void_p
    h.fake_ctx.argtypes = [C.POINTER(td.td_shape), C.c_int, C.c_int]
    h.fake_floats.restype = C.c_int64
    P, I32, VP = C.POINTER, C.c_int32, C.c_void_p
    h.td_quantise_append.argtypes = [VP, P(td.td_chunks), P(td.td_paged8), VP, VP, I32, I32, VP]
    h.td_dequantise_read.argtypes = [VP, P(td.td_chunks), P(td.td_paged8), I32, I32, VP, VP, VP]
    for f, pool in ((h.td_chunk_attention, td.td_paged), (h.td_chunk_attention_q8, td.td_paged8)):
        f.argtypes = [VP, P(td.td_chunks), P(pool), I32, I32, VP, I32, C.c_float, I32, I32, VP, VP,
                      VP]
    return h


A = 0x10000    # a 16-byte aligned address that nothing reads


class Call:
    """One call with arguments that are right unless a test changes them."""

    def __init__(self, td, lib, H=4, D=128, P=16, L=3, max_agents=8, sms=152):
        self.td, self.lib, self.H, self.D, self.P = td, lib, H, D, P
        self.ctx = lib.fake_ctx(C.byref(td.td_shape(L, H, D, P, 16, 1e6)), max_agents, sms)
        lib.fake_state(0, 0, 0)

    def pages(self, q8, **kw):
        a = dict(base=A, scale=A, num_pages=1000, table=A, width=1 << 20, format=0)
        a.update(kw)
        if q8:
            return self.td.td_paged8(a["base"], a["scale"], a["num_pages"], a["table"], a["width"],
                                     a["format"])
        return self.td.td_paged(a["base"], a["num_pages"], a["table"], a["width"])

    def run(self, op, chunks=((0, 5, 1),), ctx=True, layers=(0, 1), k=A, v=A, q=A, nq=28, scale=0.1,
            window=0, sinks=0, out=A, lse=A, null_pages=False, null_chunks=False, n=None, **pages):
        td, lib = self.td, self.lib
        lib.fake_reset()
        ch = chunks if isinstance(chunks, td.td_chunks) else td.make_chunks(*zip(*chunks)) \
            if chunks else td.make_chunks([], [], [])
        if n is not None:
            ch.n = n
        pg = self.pages(op != "attend", **pages)
        pp = None if null_pages else C.byref(pg)
        cc = None if null_chunks else C.byref(ch)
        c = self.ctx if ctx else None
        if op == "write":
            return lib.td_quantise_append(c, cc, pp, k, v, *layers, None)
        if op == "read":
            return lib.td_dequantise_read(c, cc, pp, *layers, k, v, None)
        f = lib.td_chunk_attention_q8 if op == "attend8" else lib.td_chunk_attention
        return f(c, cc, pp, *layers, q, nq, scale, window, sinks, out, lse, None)

    def launches(self):
        res = []
        for i in range(self.lib.fake_launches()):
            v = (C.c_int64 * 14)()
            self.lib.fake_launch(i, v)
            keys = ("what kind rows n direct span tok0 tokens per_cta lane_shift head_mul "
                    "box whole_units join_from").split()
            d = dict(zip(keys, v))
            arr = [np.zeros(300, np.int32) for _ in range(7)]
            self.lib.fake_list(i, *(a.ctypes.data_as(C.c_void_p) for a in arr))
            d.update(zip(("agent", "start", "row", "base", "nsplit", "tok", "whole"), arr))
            res.append(d)
        return res


EVERY = ("write", "read", "attend", "attend8")
BAD = {
    "no context": (EVERY, dict(ctx=False)),
    "no pages": (EVERY, dict(null_pages=True)),
    "no chunks": (EVERY, dict(null_chunks=True)),
    "a negative count": (EVERY, dict(n=-1)),
    "an agent below 0": (EVERY, dict(chunks=[(-1, 0, 1)])),
    "an agent past the context's": (EVERY, dict(chunks=[(0, 0, 1), (8, 0, 1)])),
    "a start below 0": (EVERY, dict(chunks=[(0, -1, 2)])),
    "a length below 0": (EVERY, dict(chunks=[(0, 4, -1)])),
    "past the block table": (EVERY, dict(chunks=[(0, 160, 1)], width=10)),
    "across the block table's end": (EVERY, dict(chunks=[(0, 150, 11)], width=10)),
    "a position past 31 bits": (EVERY, dict(chunks=[(0, 2**31 - 1, 1)], width=2**31 - 1)),
    "layers out of order": (EVERY, dict(layers=(1, 1))),
    "a layer too many": (EVERY, dict(layers=(0, 4))),
    "a layer below 0": (EVERY, dict(layers=(-1, 1))),
    "no base": (EVERY, dict(base=None)),
    "a base off 16 bytes": (EVERY, dict(base=A + 8)),
    "no block table": (EVERY, dict(table=None)),
    "no page": (EVERY, dict(num_pages=0)),
    "pages past 31 bits of rows": (EVERY, dict(num_pages=2**27)),
    "a table without columns": (EVERY, dict(width=0)),
    "no scales": (("write", "read", "attend8"), dict(scale=None, q=A)),
    "a format that is none": (("write", "read", "attend8"), dict(format=2)),
    "no K": (("write", "read"), dict(k=None)),
    "no V": (("write", "read"), dict(v=None)),
    "K off 16 bytes": (("write", "read"), dict(k=A + 2)),
    "V off 16 bytes": (("write", "read"), dict(v=A + 4)),
    "chunks of an agent that overlap": (("write",), dict(chunks=[(1, 5, 4), (0, 0, 9), (1, 8, 2)])),
    "the same chunk twice": (("write",), dict(chunks=[(1, 5, 1), (1, 5, 1)])),
    "no queries": (("attend", "attend8"), dict(q=None)),
    "queries off 16 bytes": (("attend", "attend8"), dict(q=A + 8)),
    "no output": (("attend", "attend8"), dict(out=None)),
    "an output off 16 bytes": (("attend", "attend8"), dict(out=A + 2)),
    "lse off 4 bytes": (("attend", "attend8"), dict(lse=A + 2)),
    "heads that do not divide": (("attend", "attend8"), dict(nq=30)),
    "fewer query heads than kv heads": (("attend", "attend8"), dict(nq=2)),
    "no query head": (("attend", "attend8"), dict(nq=0)),
    "a negative window": (("attend", "attend8"), dict(window=-1)),
    "negative sinks": (("attend", "attend8"), dict(window=5, sinks=-1)),
    "a scale that is infinite": (("attend",), dict(scale=float("inf"))),
    "a scale that is NaN": (("attend",), dict(scale=float("nan"))),
    "a scale past float32 in base 2": (("attend",), dict(scale=3e38)),
    "more rows than 31 bits": (("attend", "attend8"), dict(chunks=[(0, 0, 10**8)] * 2, nq=28)),
}


@pytest.mark.parametrize("why", list(BAD))
def test_refused_without_a_launch(td, lib, why):
    ops, kw = BAD[why]
    for op in ops:
        call = Call(td, lib)
        kw2 = dict(kw)
        if "scale" in kw and op in ("write", "read", "attend8") and kw["scale"] is None:
            kw2 = {"null": None}
            pg = call.pages(True)
            pg.scale = None
            lib.fake_reset()
            ch = td.make_chunks([0], [5], [1])
            f = {"write": lambda: lib.td_quantise_append(call.ctx, C.byref(ch), C.byref(pg), A, A, 0, 1, None),
                 "read": lambda: lib.td_dequantise_read(call.ctx, C.byref(ch), C.byref(pg), 0, 1, A, A, None),
                 "attend8": lambda: lib.td_chunk_attention_q8(call.ctx, C.byref(ch), C.byref(pg), 0, 1, A, 28,
                                                              0.1, 0, 0, A, A, None)}[op]
            assert f() == td.TD_ERR_INVALID_ARG
        else:
            assert call.run(op, **kw2) == td.TD_ERR_INVALID_ARG, op
        assert lib.fake_launches() == 0


def test_refused_head_dims_devices_and_captures(td, lib):
    for D in (16, 32, 48, 96, 256):
        assert Call(td, lib, H=2, D=D).run("attend", nq=4) == td.TD_ERR_INVALID_ARG
        assert Call(td, lib, H=2, D=D).run("write") == td.TD_OK
    for op in ("write", "read"):
        assert Call(td, lib, H=1, D=272).run(op) == td.TD_ERR_INVALID_ARG
    for op in EVERY:
        call = Call(td, lib)
        lib.fake_state(1, 0, 0)                      # another device is current
        assert call.run(op) == td.TD_ERR_INVALID_ARG and lib.fake_launches() == 0
    call = Call(td, lib)
    long = [(0, 100000, 1)]
    lib.fake_state(0, 1, 0)                          # in a capture: no allocation
    assert call.run("attend", chunks=long) == td.TD_ERR_INVALID_ARG and lib.fake_launches() == 0
    assert call.run("attend", chunks=[(0, 5, 1)]) == td.TD_OK       # needs none
    lib.fake_state(0, 0, 1)                          # no memory left
    assert call.run("attend", chunks=long) == td.TD_ERR_CUDA and lib.fake_launches() == 0
    lib.fake_state(0, 0, 0)
    assert call.run("attend", chunks=long) == td.TD_OK
    lib.fake_state(0, 1, 0)
    assert call.run("attend", chunks=long) == td.TD_OK
    lib.fake_state(0, 0, 0)


def test_empty_batches_launch_nothing(td, lib):
    for op in EVERY:
        for chunks in ([], [(0, 3, 0)], [(0, 0, 0), (7, 9, 0)]):
            call = Call(td, lib)
            assert call.run(op, chunks=chunks, k=None, v=None, q=None, out=None, lse=None) == td.TD_OK
            assert lib.fake_launches() == 0


def test_plans_of_the_quantising_kernels(td, lib):
    for H, D in ((4, 128), (1, 16), (128, 16), (3, 48), (8, 256), (2, 64), (7, 112)):
        for T in (1, 31, 32, 4000):
            call = Call(td, lib, H=H, D=D)
            for op in ("write", "read"):
                assert call.run(op, chunks=[(0, 3, T)]) == td.TD_OK
                (l,) = call.launches()
                lanes = 1 << l["lane_shift"]
                need = D // (16 if op == "write" else 8)       # elements a lane
                assert need <= lanes <= 32 and lanes < 2 * need
                assert 1 <= l["per_cta"] <= 32
                rows = np.arange(l["per_cta"] * H, dtype=np.int64)
                prod = rows * l["head_mul"]
                assert prod.max(initial=0) < 2**32
                assert np.array_equal(prod >> 20, rows // H)      # the division it stands for


def _steps(what, s, t, G, R, tile, window, sinks):
    """Steps that the kernel takes for a tile: visible positions, or KV tiles of 128."""
    first = s + tile * R // G
    last = s + min(tile * R + R - 1, t * G - 1) // G
    lo = max(0, first - window + 1) if window else 0
    kept = min(sinks, lo) if window else 0
    if what == 2:
        return last + 1 - lo + kept
    tiles = set(range(lo // 128, last // 128 + 1)) | set(range(-(-kept // 128)))
    return len(tiles)


def _check_attention(lib, call, H, D, P, nq, chunks, window, sinks, nl, q8):
    G = nq // H
    at, tok, tails = {}, 0, 0
    for i, (a, s, t) in enumerate(chunks):
        if t:
            at[tok] = (a, s, t)
        tok += t
    for l in call.launches():
        if l["what"] == 3:
            continue
        n, R, tc = int(l["n"]), int(l["rows"]), l["what"] == 4
        assert R in ((128, 256) if tc else (8, 16)) and 0 < n <= 256
        assert tc or l["span"] % 16 == 0
        split = l["direct"] == 0 and l["whole_units"] == 0
        assert not tc or q8 or (P % 8 == 0 and P % l["box"] == 0 and 8 <= l["box"] <= 128)
        for x in range(n):
            a, s, t = at.pop(int(l["tok"][x]))
            assert (l["agent"][x], l["start"][x], l["row"][x + 1] - l["row"][x]) == (a, s, t)
            assert not tc or t * G > 16
            assert tc or t * G <= 16 or (not q8 and P % 8)
            tiles = -(-t * G // R)
            ns = int(l["nsplit"][x])
            whole = int(l["whole"][x])             # tiles from the last one down, a unit each
            assert 0 <= whole <= tiles and (tc or whole == 0)
            assert l["base"][x + 1] - l["base"][x] == whole + (tiles - whole) * ns
            assert ns == 1 or not l["direct"]
            split |= whole < tiles
            if not split:                          # whole ones come first, and are not joined
                assert l["direct"] or l["join_from"] >= l["row"][x + 1]
            elif whole:
                assert l["whole_units"] == l["base"][x] + whole and l["join_from"] == l["row"][x]
            tails += whole > 0
            for tile in range(tiles - whole):
                assert ns * int(l["span"]) >= _steps(l["what"], s, t, G, R, tile, window, sinks)
        units = int(l["base"][n]) * H * nl
        assert not l["direct"] or l["whole_units"] == l["join_from"] == 0
        if not l["direct"]:
            parts = units - l["whole_units"] * H * nl
            assert parts > 0 and parts * R * (D + 2) <= lib.fake_floats()
        assert units < 2**31
    assert not at                                   # every sequence in one launch
    return tails


def test_plans_cover_every_visible_position(td, lib):
    rng = random.Random(7)
    tails = 0
    for i in range(400):
        H, D, G = rng.choice((1, 2, 3, 8)), rng.choice((64, 128)), rng.choice((1, 2, 5, 7, 8, 16, 40))
        P, nl = rng.choice((1, 5, 8, 16, 24, 32, 256)), rng.choice((1, 2))
        n = rng.choice((1, 2, 9, 300, 600))
        hi = rng.choice((1, 2, 40, 700))
        chunks = [(i % 8, rng.randint(0, rng.choice((1, 50, 20000))), rng.randint(0, hi)) for i in range(n)]
        window = rng.choice((0, 0, 1, 64, 1000))
        sinks = rng.choice((0, 4, 300))
        call = Call(td, lib, H=H, D=D, P=P, sms=rng.choice((152, 8)))
        op = rng.choice(("attend", "attend8"))
        assert call.run(op, chunks=chunks, nq=H * G, window=window, sinks=sinks,
                        layers=(1, 1 + nl)) == td.TD_OK
        tails += _check_attention(lib, call, H, D, P, H * G, chunks, window, sinks, nl,
                                  op == "attend8")
    assert tails > 3


def test_long_chunks_over_8bit_pages_are_unfolded_once(td, lib):
    """Every KV tile that a query tile takes has a place of its own in the copy that its launch
    reads; the copy stays within its limit, and the scratch holds all of it."""
    rng = random.Random(11)
    unfolded = 0
    for i in range(300):
        H, D, G = rng.choice((1, 2, 8)), rng.choice((64, 128)), rng.choice((1, 5, 8))
        nl = rng.choice((1, 2, 28))
        n = rng.choice((1, 3, 300))
        chunks = [(j % 8, rng.randint(0, rng.choice((1, 300, 30000))), rng.randint(0, 900))
                  for j in range(n)]
        window, sinks = rng.choice((0, 0, 1, 130, 1000)), rng.choice((0, 4, 300, 2000))
        call = Call(td, lib, H=H, D=D, L=29)
        assert call.run("attend8", chunks=chunks, nq=H * G, window=window, sinks=sinks,
                        layers=(1, 1 + nl)) == td.TD_OK
        launches = call.launches()
        seen = set()
        for u in range(lib.fake_unfolds()):
            base, out = np.zeros(257, np.int32), np.zeros(6, np.int64)
            lib.fake_unfold(u, base.ctypes.data_as(C.c_void_p), out.ctypes.data_as(C.c_void_p))
            at, m, rows, same, scales, parts = (int(v) for v in out)
            l = launches[at]
            assert same and rows == 128 * base[m] and at not in seen
            seen.add(at)
            floats = nl * 2 * rows * H * D // 2
            assert scales == floats and parts == floats + nl * 2 * rows * H
            assert 4 * parts <= 2**30 and parts % 4 == 0 and scales % 4 == 0
            units = (int(l["base"][m]) - int(l["whole_units"])) * H * nl
            assert parts + (0 if l["direct"] else units * 256 * (D + 2)) <= lib.fake_floats()
            for x in range(m):
                s, t = int(l["start"][x]), int(l["row"][x + 1] - l["row"][x])
                assert t * G > 512
                span = np.zeros(3, np.int32)
                lib.fake_span(s, t, window, sinks, span.ctypes.data_as(C.c_void_p))
                first, t0, tiles = (int(v) for v in span)
                assert base[x + 1] - base[x] == tiles
                have = list(range(first)) + list(range(t0, t0 + tiles - first))
                assert len(set(have)) == len(have) and have[-1] <= (s + t - 1) // 128
                for tile in range(-(-t * G // 256)):
                    p0, p1 = s + tile * 256 // G, s + min(tile * 256 + 255, t * G - 1) // G
                    lo = max(0, p0 - window + 1) if window else 0
                    kept = min(sinks, lo) if window else 0
                    need = set(range(lo // 128, p1 // 128 + 1)) | set(range(-(-kept // 128)))
                    assert need <= set(have)
                    for kt in need:                      # the kernel's place of a tile
                        assert have[kt if kt < first else first + kt - t0] == kt
                unfolded += 1
        for k, l in enumerate(launches):
            if l["what"] == 4 and k not in seen:         # converted in the kernel: short, or long
                for x in range(int(l["n"])):
                    s, t = int(l["start"][x]), int(l["row"][x + 1] - l["row"][x])
                    tiles = -(-(s + t) // 128)
                    assert t * G <= 512 or nl * 2 * 128 * tiles * H * (2 * D + 4) > 2**30
    assert unfolded > 1000


def test_the_last_wave_is_cut_where_it_pays(td, lib):
    """372 units on 152 SMs: the last 68 in parts; 128, 152 and 304 stay as they are."""
    call = Call(td, lib, H=4, D=128)
    for chunks, cut in (([(0, 4200, 1500), (1, 3900, 1300), (2, 3700, 160)], 17),
                        ([(0, 4000, 1216)], 0), ([(0, 4000, 2432)], 0), ([(0, 4000, 1000)], 0)):
        assert call.run("attend", chunks=chunks, nq=32) == td.TD_OK
        l = [x for x in call.launches() if x["what"] == 4][0]
        n = int(l["n"])
        tiles = sum(-(-8 * t // 256) for _, _, t in chunks)
        assert cut == (0 if l["direct"] else tiles - int(l["whole"][:n].sum()))
        _check_attention(lib, call, 4, 128, 16, 32, chunks, 0, 0, 1, False)


def test_scratch_that_cannot_double_takes_what_is_needed(td, lib):
    call = Call(td, lib, H=2, D=128)
    lib.fake_room.argtypes = [C.c_int64]
    try:
        assert call.run("attend", chunks=[(0, 9000, 1)], nq=14) == td.TD_OK
        first = lib.fake_floats()
        assert call.run("attend", chunks=[(i, 9000, 1) for i in range(4)], nq=14) == td.TD_OK
        assert lib.fake_floats() >= 2 * first
        second = lib.fake_floats()
        # long chunks over 8-bit pages: 7 tiles of 128 positions unfolded, K and V, over 2 layers
        need = 2 * 2 * 7 * 128 * (2 * 128 // 2 + 2)
        assert second < need < 2 * second
        lib.fake_room(need * 4)
        assert call.run("attend8", chunks=[(0, 0, 800)], nq=14, layers=(0, 2)) == td.TD_OK
        assert need == lib.fake_floats()
        lib.fake_room(need * 4 - 4)
        call = Call(td, lib, H=2, D=128)
        assert call.run("attend8", chunks=[(0, 0, 800)], nq=14, layers=(0, 2)) == td.TD_ERR_CUDA
    finally:
        lib.fake_room(2**62)
