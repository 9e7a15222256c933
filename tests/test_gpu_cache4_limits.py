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
