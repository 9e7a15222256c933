"""The calls over 4-bit pages and device lengths at the ends of their ranges: sizes, scales and
queries where index arithmetic or precision could give out."""
from __future__ import annotations

import math
import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import cache4kit as k4
from tests import chunkkit as ck

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def td():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from collective_kv_cache_gb300 import build
    build.build()
    from collective_kv_cache_gb300 import td as _td
    return _td


def _ctx(td, H=1, D=64, P=16, L=1, rows=8):
    return td.Context(td.td_shape(L, H, D, P, 16, 1e6), rows, 1, 1)


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _errors(td, ctx):
    return td.td_get_error(ctx.handle, _stream())


def _dev(a):
    return torch.tensor(np.asarray(a, dtype=np.int32), device="cuda")


# ------------------------------------------------------------------------------ tables
@pytest.mark.parametrize("met", [True, False])
@pytest.mark.parametrize("max_slots", [2 ** 31 - 1, 2 ** 31 - 155000])
def test_the_largest_slot_map(td, max_slots, met):
    """Every slot past the tokens' is -1, in a call that is met and in one that is not; nothing before
    or behind the map is written."""
    guard = 1 << 18
    if torch.cuda.mem_get_info()[0] < 4.5 * max_slots:
        pytest.skip("the slot map does not fit this GPU's free memory")
    mem = torch.full((max_slots + 2 * guard,), 7, dtype=torch.int32, device="cuda")
    slots = mem[guard:guard + max_slots]
    ctx = _ctx(td, P=1, rows=2)
    lens, bt = _dev([2, 0]), torch.full((2, 8), -1, dtype=torch.int32, device="cuda")
    bt[0, :2] = _dev([5, 3])
    pages, count = _dev([0, 1, 2, 4]), _dev([4])
    start = torch.full((3,), -5, dtype=torch.int32, device="cuda")
    add = _dev([1, 2 if met else 4])
    td.td_update_tables(ctx.handle, td.make_requests(lens), add.data_ptr(), bt.data_ptr(), 8,
                        td.make_page_list(pages, count, 6), start.data_ptr(), slots.data_ptr(), max_slots,
                        _stream())
    e = 0 if met else td.TD_ERR_CAPACITY
    assert _errors(td, ctx) == (e, 1 << e if e else 0)
    assert bool((mem[:guard] == 7).all()) and bool((mem[guard + max_slots:] == 7).all())
    tokens = [4, 2, 1] if met else [-1, -1, -1]
    assert slots[:3].tolist() == tokens
    assert start.tolist() == ([0, 1, 3] if met else [0, 0, 0])
    assert lens.tolist() == ([3, 2] if met else [2, 0])
    for part in slots[3:].split(1 << 28):
        assert bool((part == -1).all())


@pytest.mark.parametrize("P", [2 ** 30 + 7, 2 ** 31 - 1])
def test_pages_past_2_to_30_positions(td, P):
    """One page holds whatever a request may hold: the second call takes none, the last gives it back."""
    ctx = _ctx(td, P=P, rows=1)
    lens, bt = _dev([0]), _dev([[-1, -1]])
    mem, count = _dev([-9, -9, 0, -9, -9]), _dev([1])
    slots = torch.empty(5, dtype=torch.int32, device="cuda")
    held = 0
    for add, free in ((3, 0), (2, 0), (-1, 0), (-4, 1)):
        a = _dev([add])
        td.td_update_tables(ctx.handle, td.make_requests(lens), a.data_ptr(), bt.data_ptr(), 2,
                            td.make_page_list(mem[2:3], count, 1), None, slots.data_ptr(), 5, _stream())
        assert _errors(td, ctx) == (0, 0)
        new = list(range(held, held + add))
        held += add
        assert slots.tolist() == new + [-1] * (5 - len(new))
        assert lens.tolist() == [held] and count.tolist() == [free] and mem.tolist() == [-9, -9, 0, -9, -9]
        assert bt.tolist() == [[-1 if free else 0, -1]]


@pytest.mark.parametrize("what", ["sizes", "threads"])
def test_many_requests_in_a_process_of_their_own(td, what):
    """Whatever sizes came before, and whatever another thread asks for (tests/tables_many.py)."""
    done = subprocess.run([sys.executable, "-m", "tests.tables_many", what], cwd=ROOT, capture_output=True,
                          text=True, timeout=300)
    assert done.returncode == 0 and done.stdout.strip() == "ok", done.stdout + done.stderr


# --------------------------------------------------------------------------- slots: reading
@pytest.mark.parametrize("D", [64, 128])
def test_a_quarter_that_is_nan_reads_back_as_nan_and_the_others_do_not(td, D):
    """e2m1: a byte 255 stands for NaN in its own quarter; the other quarters have their values."""
    H, P, pages = 3, 5, 8
    ctx = _ctx(td, H, D, P)
    gen = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, 256, (1, 2, pages, H, P, D // 2), generator=gen, device="cuda",
                          dtype=torch.uint8)
    byte = torch.randint(120, 130, (1, 2, pages, H, P, 4), generator=gen, device="cuda")
    byte[torch.rand(byte.shape, generator=gen, device="cuda") < 0.3] = 255
    word = k4.words(byte, "e2m1")
    bt = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    T = pages * P
    slots = torch.randperm(T, generator=gen, device="cuda").int()
    ko, vo = (torch.empty((1, T, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    td.td_dequantise_slots(ctx.handle, slots.data_ptr(), T, td.make_paged4(codes, word, bt, "e2m1"), 0, 1,
                           ko.data_ptr(), vo.data_ptr(), _stream())
    assert _errors(td, ctx) == (0, 0)
    grid = torch.tensor(k4.E2M1 + tuple(-x for x in k4.E2M1), dtype=torch.float64, device="cuda")
    want = grid[k4.unpack(codes).long()].unflatten(-1, (4, -1)) * 2.0 ** (byte[..., None].double() - 127)
    want = torch.where(byte[..., None] == 255, math.nan, want).flatten(-2)[0]    # [2][pages][H][P][D]
    s = slots.long()
    for got, val in zip((ko, vo), want):
        val = val[s // P, :, s % P]
        assert bool((got.isnan() == val.isnan()[None]).all()) and bool(got.isnan().any(-1).any())
        assert torch.equal(got.nan_to_num(9.0), val.to(torch.bfloat16)[None].nan_to_num(9.0))


# --------------------------------------------------------------------------------- attention
def _attend(td, b, codes, word, fmt, q, scale, decode=False):
    """Output and log-sum-exp of the batch's chunks (decode: its tokens) over all layers."""
    ctx = _ctx(td, b.H, b.D, b.P, b.L, rows=b.n_agents)
    out = torch.full(q.shape, math.nan, dtype=torch.bfloat16, device="cuda")
    z = torch.full(q.shape[:3], math.nan, device="cuda")
    pages = td.make_paged4(codes, word, b.bt_t, fmt)
    tail = (0, b.L, q.data_ptr(), q.shape[2], scale, 0, 0, out.data_ptr(), z.data_ptr(), _stream())
    if decode:
        td.td_decode_attention_q4(ctx.handle, td.make_requests(_dev([s + 1 for s in b.starts])), pages, *tail)
    else:
        td.td_chunk_attention_q4(ctx.handle, td.make_chunks(b.agents, b.starts, b.lens), pages, *tail)
    assert _errors(td, ctx) == (0, 0)
    return out, z


@pytest.mark.parametrize("fmt", k4.FORMATS)
def test_elements_of_a_query_far_below_its_largest(td, fmt):
    """Elements of 8 bits keep them down to 2^-19 of their row's largest (e2m1 2^-23), and count for
    something over 2^-27 (2^-31) of it: a query row a head, one small element each at another dim, its
    largest where K is zero. Of one position the log-sum-exp is the score, q_small * k * scale."""
    D, G, edge, last = 128, 40, 19 if fmt == "int4" else 23, 27 if fmt == "int4" else 31
    b = k4.Batch([0], [1], 1, D, 16, seed=31)
    code = torch.zeros(b.shape((D,)), dtype=torch.uint8, device="cuda")
    code[..., :G] = 2                                  # int4: 2; e2m1: 1
    if fmt == "int4":
        word = k4.words(torch.ones(b.shape(), device="cuda"), fmt, torch.zeros(b.shape(), device="cuda"))
        k = 2.0
    else:
        word, k = k4.words(torch.full(b.shape((4,)), 127, device="cuda"), fmt), 1.0
    codes = k4.pack(code)
    for small, low, high in ((255 / 128 * 2.0 ** -edge, 1 - 2.0 ** -12, 1 + 2.0 ** -12),
                             (1.5 * 2.0 ** -last, 2.0 ** -8, 2.0)):
        q = torch.zeros((1, 1, G, D), device="cuda")
        i = torch.arange(G, device="cuda")
        q[0, 0, i, i] = small
        q[0, 0, i, G + i] = torch.where(i % 2 == 0, 1.0, -1.0)
        scale = 2.0 ** edge
        for decode in (False, True):
            _, z = _attend(td, b, codes, word, fmt, q.to(torch.bfloat16), scale, decode)
            ratio = z.double()[0, 0] / (small * k * scale)
            assert bool(((ratio >= low) & (ratio <= high)).all()), ratio.tolist()


SUMS = {
    # name: (starts, lens, H, G, D, P, decode)
    "tokens": ([5000, 1, 700], [1, 1, 1], 2, 7, 128, 16, True),
    "tokens_d64": ([3000, 64, 127, 128], [1] * 4, 4, 3, 64, 24, True),
    "one_long_token": ([12000], [1], 8, 8, 128, 16, True),
    "drafts": ([4000, 300], [2, 3], 2, 7, 128, 16, False),
    "drafts_d64": ([4000, 300], [5, 2], 2, 8, 64, 5, False),
    "converted": ([3000, 90], [20, 30], 2, 7, 128, 16, False),
    "converted_d64": ([2000], [70], 3, 7, 64, 16, False),
    "unfolded": ([900, 30], [150, 90], 1, 7, 128, 16, False),
    "unfolded_d64": ([2000, 500], [520, 600], 8, 2, 64, 24, False),
    "unfolded_256": ([500, 0], [600, 700], 8, 4, 128, 16, False),
}


@pytest.mark.parametrize("fmt", k4.FORMATS)
@pytest.mark.parametrize("name", list(SUMS))
def test_sums_of_thousands_of_positions(td, name, fmt):
    """Weights and scales that are powers of two, which no way of the kernels rounds: 2^0 to 2^3 by one
    element of K (a query head has one dim of its own, and the softmax scale is ln 2, 2^-24 off at
    most), V's scales 2^-1 to 2^1. A product of weight, scale and code is a multiple of 2^-2 up to
    15 * 2^4 (a weight can be 2^-16 of that where the reference lags: the factor is common), and the sums
    of 12001 of them stay under 2^24 such steps, so float32 adds them exactly, cut or rounded. What is
    left: the exponential's 2^-21 of a weight with its exponent's 3 * 2^-23, the parts' and the last
    scalings' few 2^-24, under 2^-18 of sum w |v| in all; and the output's rounding, 2^-8 of it. An
    output is near 4 / sqrt(C), far above the former."""
    starts, lens, H, G, D, P, decode = SUMS[name]
    b = k4.Batch(starts, lens, H, D, P, seed=32)
    codes, _, _, _ = b.random_pages(fmt)
    code = k4.unpack(codes)
    dims = torch.arange(D, device="cuda") < G
    n = torch.randint(0, 4, code[:, 0].shape, generator=b.gen, device="cuda").to(torch.uint8)
    if fmt == "int4":
        zero = torch.randint(0, 12, b.shape(), generator=b.gen, device="cuda")
        zero[:, 1] = torch.randint(0, 16, zero[:, 1].shape, generator=b.gen, device="cuda")
        power = torch.randint(-1, 2, b.shape(), generator=b.gen, device="cuda")
        power[:, 0] = 0
        word = k4.words(2.0 ** power.float(), fmt, zero)
        code[:, 0] = torch.where(dims, n + zero[:, 0, ..., None].to(torch.uint8), code[:, 0])
    else:
        power = torch.randint(126, 129, b.shape((4,)), generator=b.gen, device="cuda")
        power[:, 0] = 128                              # (a code n is n / 2 up to 2, and 3 is 1.5)
        word = k4.words(power, fmt)
        code[:, 0] = torch.where(dims, n, code[:, 0])
    codes = k4.pack(code)
    val = k4.values(codes, word, fmt).transpose(3, 4)
    q = torch.zeros((1, b.T, H, G, D), device="cuda")
    i = torch.arange(G, device="cuda")
    q[:, :, :, i, i] = 1.0
    q = q.flatten(2, 3).to(torch.bfloat16)
    out, z = _attend(td, b, codes, word, fmt, q, math.log(2.0), decode)
    want, lse, mag, _ = ck.attend(b, val[:, 0], val[:, 1], q, scale=math.log(2.0))
    err, tol = (out.double() - want).abs(), want.abs() * 2.0 ** -8 + mag * 2.0 ** -18
    assert bool((err <= tol).all()), float((err / tol).max())
    assert float((z.double() - lse).abs().max()) <= 2.0 ** -17 + 2.0 ** -23 * float(lse.abs().max())


KINDS = {
    # name: (starts, lens, H, G, D, P)
    "token": ([700], [1], 1, 3, 128, 16),
    "few": ([300, 90], [3, 2], 2, 7, 64, 16),
    "converted": ([400, 90], [20, 30], 2, 7, 128, 16),
    "converted_d64": ([700], [60], 2, 3, 64, 24),
    "unfolded": ([300, 30], [150, 90], 1, 7, 128, 16),
    "unfolded_d64": ([900], [520], 2, 2, 64, 24),
    "unfolded_256": ([100, 0], [600, 500], 8, 4, 64, 16),
}


def _apart(b, gen, kv, base, most, word):
    """Bytes of every row's quarters: base less 0 to most, one of them base itself."""
    d = torch.randint(0, most + 1, b.shape((4,))[:1] + b.shape((4,))[2:], generator=gen, device="cuda")
    d.scatter_(-1, torch.randint(0, 4, d.shape[:-1] + (1,), generator=gen, device="cuda"), 0)
    word[:, kv] = k4.words(base - d, "e2m1")
    return d


@pytest.mark.parametrize("base", [127, 60, 235])
@pytest.mark.parametrize("name", list(KINDS))
def test_quarters_of_v_up_to_2_to_40_apart(td, name, base):
    """Rows of V whose quarters lie 2^0 to 2^40 apart, around 1, from 2^-67 down to 2^-107, and from 2^108
    down: chunks of up to 48 query rows count a quarter of 2^-27 of its row's largest or less as 0; the
    others nothing."""
    starts, lens, H, G, D, P = KINDS[name]
    b = k4.Batch(starts, lens, H, D, P, seed=33)
    codes, word, _, _ = b.random_pages("e2m1")
    d = _apart(b, b.gen, 1, base, 40, word)
    val = k4.values(codes, word, "e2m1").transpose(3, 4)
    q = b.rows(1, b.T, H * G, D)
    scale = D ** -0.5
    got = _attend(td, b, codes, word, "e2m1", q, scale)
    want = ck.attend(b, val[:, 0], val[:, 1], q)
    few = max(lens) * G <= 48
    tol, tol_lse = k4.bounds(want, q, word, "e2m1", scale, few, 0)
    tol = tol - 1e-30 + 2.0 ** -132                     # (the bound's floor would hide the small ones)
    if few:
        # the quarters left out; and weights below f16's normal range, 2^-31 of every row's largest scale
        off = (d >= 27)[..., None].expand(d.shape + (D // 4,)).flatten(-2).transpose(2, 3)
        tol = tol + ck.attend(b, val[:, 0], torch.where(off, val[:, 1], 0.0), q)[2]
        C = max(s + t for s, t in zip(starts, lens))
        tol = tol + C * 2.0 ** -31 * ck.attend(b, val[:, 0], val[:, 1], q, scale=0.0)[2]
    err = (got[0].double() - want[0]).abs()
    assert bool((err <= tol).all()), (float((err - tol).max()), float((err / tol).max()))
    assert bool(((got[1].double() - want[1]).abs() <= tol_lse).all())


@pytest.mark.parametrize("base,up", [(26, 100), (235, -106), (228, -100), (40, 88)])
@pytest.mark.parametrize("name", [n for n in KINDS if n != "few"])
def test_quarters_of_k_at_the_ends_of_their_bytes(td, name, base, up):
    """Rows of K whose bytes are at, or reach below, the least ones that an unfolded copy holds multiplied
    out, or above the largest, up to 2^20 apart, under queries that bring the scores back to order 1."""
    starts, lens, H, G, D, P = KINDS[name]
    b = k4.Batch(starts, lens, H, D, P, seed=34)
    codes, word, _, _ = b.random_pages("e2m1")
    _apart(b, b.gen, 0, base, 20, word)
    val = k4.values(codes, word, "e2m1").transpose(3, 4)
    q = (b.rows(1, b.T, H * G, D).float() * 2.0 ** up).to(torch.bfloat16)
    scale = D ** -0.5
    got = _attend(td, b, codes, word, "e2m1", q, scale)
    want = ck.attend(b, val[:, 0], val[:, 1], q)
    assert float(want[3].max()) > 2.0 ** -6             # (the scores differ)
    few = max(lens) * G <= 48
    tol, tol_lse = k4.bounds(want, q, word, "e2m1", scale, few, max(s + t for s, t in zip(starts, lens)))
    err = (got[0].double() - want[0]).abs()
    assert bool((err <= tol).all()), (float((err - tol).max()), float((err / tol).max()))
    assert bool(((got[1].double() - want[1]).abs() <= tol_lse).all())


@pytest.mark.parametrize("name", [n for n in KINDS if n not in ("token", "few")])
def test_quarters_of_v_as_far_apart_as_they_count(td, name):
    """Chunks of more query rows: quarters up to 2^126 apart have their values; in an unfolded copy one of
    2^-127 of its row's largest counts as 0."""
    starts, lens, H, G, D, P = KINDS[name]
    b = k4.Batch(starts, lens, H, D, P, seed=35)
    codes, word, _, _ = b.random_pages("e2m1")
    _apart(b, b.gen, 1, 235, 126, word)
    q = b.rows(1, b.T, H * G, D)
    scale = D ** -0.5
    val = k4.values(codes, word, "e2m1").transpose(3, 4)
    got = _attend(td, b, codes, word, "e2m1", q, scale)
    want = ck.attend(b, val[:, 0], val[:, 1], q)
    tol = k4.bounds(want, q, word, "e2m1", scale, False, 0)[0] - 1e-30 + 2.0 ** -132
    err = (got[0].double() - want[0]).abs()
    assert bool((err <= tol).all()), (float((err - tol).max()), float((err / tol).max()))
    if not name.startswith("unfolded"):
        return
    word[:, 1] = k4.words(torch.tensor([235, 108, 235, 107], device="cuda").expand(b.shape((4,))[:1] +
                                                                               b.shape((4,))[2:]), "e2m1")
    out = _attend(td, b, codes, word, "e2m1", q, scale)[0].unflatten(-1, (4, -1))
    assert bool((out[..., 1::2, :] == 0).all()) and bool((out[..., 0::2, :] != 0).any())


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("D,G", [(128, 7), (64, 16)])
def test_scores_over_int4_pages_are_float32(td, D, G, decode):
    """Requests of one position, whose log-sum-exp is the score. Elements of the queries have 8 bits and
    lie at most 2^5 below the row's largest, so that products with codes of 0 to 15 are multiples of 2^-12
    of the largest's power of two and their sums stay under 2^24 such steps: t = sum q u and sum q are
    exact in float32. (q, q and K's zero point: t - z sum q is then rounded once, multiplied three times by
    scales, one of them rounded itself, and by ln 2: 6 times 2^-24, under 2^-21 of the score.)"""
    n, H = 40, 2
    b = k4.Batch([0] * n, [1] * n, H, D, 16, seed=36)
    codes, _, _, _ = b.random_pages("int4")
    zero = torch.randint(0, 16, b.shape(), generator=b.gen, device="cuda")
    power = torch.rand(b.shape(), generator=b.gen, device="cuda") + 0.5
    word = k4.words(power, "int4", zero)
    val = k4.values(codes, word, "int4").transpose(3, 4)
    shape = (1, n, H * G, D)
    rand = lambda lo, hi: torch.randint(lo, hi, shape, generator=b.gen, device="cuda")  # noqa: E731
    q = rand(128, 256).float() * 2.0 ** -(7 + rand(0, 6)).float() * (2 * rand(0, 2) - 1)
    q[..., 5] = 1.0
    q = q.to(torch.bfloat16)
    _, z = _attend(td, b, codes, word, "int4", q, D ** -0.5, decode)
    want = ck.attend(b, val[:, 0], val[:, 1], q)[1]
    err = (z.double() - want).abs()
    assert bool((err <= want.abs() * 2.0 ** -21 + 1e-30).all()), float((err / want.abs()).max())
