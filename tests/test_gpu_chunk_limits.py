"""Chunks of new tokens over paged caches: values, scales and ranges at their limits, on each
of the attention's ways (a few rows, many, and many over 8-bit pages unfolded first)."""
from __future__ import annotations

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import chunkkit as ck
from tests.test_gpu_chunks import _chunks, _close, _ctx, _errors, _run_attention, _stream, _weight_step, td

pytestmark = pytest.mark.gpu


def _pages8(td, b, kv, fmt):
    """Values kv as 8-bit pages: the pages, their codes and scales, the values they stand for."""
    val, s = ck.quantise(kv, fmt)
    codes, scale = ck.code_bytes(val, fmt).contiguous(), s.float().contiguous()
    return td.make_paged8(codes, scale, b.bt_t, fmt), codes, scale, val * s[..., None]


# ------------------------------------------------------- values that are not finite, in sight
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("at", [20, 199])
@pytest.mark.parametrize("n", [2, 40, 300])
def test_a_value_in_sight_counts_whatever_its_weight(td, n, at, value):
    """V of a position whose weight is under the least float32 (its score is 128 below the
    others', e^-128 = 2^-184) holds a NaN or an infinity: every row sees it, so no row's element
    is finite, in a step that masks something (at 199, beside the chunk) as in one that does
    not (at 20)."""
    b = ck.Batch([200], [n], 1, 128, 16, seed=61)
    pool, q = b.rows(*b.pool_shape()), torch.zeros((1, n, 3, 128), dtype=torch.bfloat16, device="cuda")
    pool[:, 0] = 0
    pool[:, 0, ..., 0] = 8.0
    q[..., 0] = 8.0
    pg, sl = b.place(0, np.array([at]))
    pool[0, 0, pg, sl, 0, 0] = -8.0
    pool[0, 1, pg, sl, 0, 5] = value
    out, z = _run_attention(td, b, td.make_paged(pool, b.bt_t), q, scale=1.0)
    assert not bool(torch.isfinite(out[..., 5]).any())
    if math.isnan(value):
        assert bool(torch.isnan(out[..., 5]).all())
    rest = torch.cat([out[..., :5], out[..., 6:]], -1)
    assert bool(torch.isfinite(rest).all()) and bool(torch.isfinite(z).all())


@pytest.mark.parametrize("n", [2, 40, 300])
def test_a_scale_in_sight_counts_at_a_score_of_minus_infinity(td, n):
    """8-bit pages: K's scale of a position is infinite, so that its score is -infinity and its
    weight 0, and V's scale is a NaN: the rows see it, and are NaN."""
    b = ck.Batch([200], [n], 1, 128, 16, seed=62)
    kv, q = b.rows(*b.pool_shape()), torch.zeros((1, n, 3, 128), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    pg, sl = b.place(0, np.array([199]))
    kv[0, 0, pg, sl, 0] = 0
    kv[0, 0, pg, sl, 0, 0] = -1.0
    pages, codes, scale, _ = _pages8(td, b, kv, "int8")
    scale[0, 0, pg, sl, 0] = math.inf
    scale[0, 1, pg, sl, 0] = math.nan
    out, z = _run_attention(td, b, pages, q, q8=True)
    assert bool(torch.isnan(out).all())


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("case", [(2, 3, 128, 0), (40, 3, 128, 0), (170, 2, 64, 60), (300, 7, 128, 0),
                                  (300, 7, 128, 90), (40, 8, 64, 0)])
def test_a_value_of_v_changes_its_element_of_the_rows_that_see_it_alone(td, case, value):
    """Bit for bit: every other element of those rows, and every other row, is as without it."""
    n, G, D, W = case
    b = ck.Batch([150, 40], [n, 20], 2, D, 16, seed=63)
    pool, q = b.rows(*b.pool_shape()), b.rows(1, b.T, 2 * G, D)
    clean, zc = _run_attention(td, b, td.make_paged(pool, b.bt_t), q, W, 3)
    keep = torch.ones(clean.shape, dtype=torch.bool, device="cuda")
    pos = 150 + torch.arange(n, device="cuda")
    # in the chunk, before it, and among the kept first tokens; two of them in one page
    for at, d in ((150 + n // 2, 5), (149, D - 1), (148, 5), (1, 17)):
        pg, sl = b.place(0, np.array([at]))
        pool[0, 1, pg, sl, 1, d] = value
        sees = (pos >= at) & ((pos < at + W) | (at < 3) if W else pos >= 0)
        keep[0, :n, G:, d] &= ~sees[:, None]
    dirty, zd = _run_attention(td, b, td.make_paged(pool, b.bt_t), q, W, 3)
    assert torch.equal(zc, zd)
    assert bool((clean == dirty)[keep].all())
    assert not bool(torch.isfinite(dirty[~keep]).any())
    if math.isnan(value):
        assert bool(torch.isnan(dirty[~keep]).all())


def test_a_value_of_v_in_one_part_of_a_tile(td):
    """The same where the tile's positions are several units, joined afterwards."""
    b = ck.Batch([6000], [60], 1, 128, 16, seed=64)
    pool, q = b.rows(*b.pool_shape()), b.rows(1, b.T, 3, 128)
    clean, zc = _run_attention(td, b, td.make_paged(pool, b.bt_t), q)
    pg, sl = b.place(0, np.array([6031, 6050]))
    pool[0, 1, pg, sl, 0, 9] = torch.tensor([math.inf, -math.inf], device="cuda").to(torch.bfloat16)
    dirty, zd = _run_attention(td, b, td.make_paged(pool, b.bt_t), q)
    keep = torch.ones(clean.shape, dtype=torch.bool, device="cuda")
    keep[0, 31:, :, 9] = False
    assert torch.equal(zc, zd) and bool((clean == dirty)[keep].all())
    assert not bool(torch.isfinite(dirty[~keep]).any())
    assert bool((dirty[0, 31:50, :, 9] == math.inf).all())
    assert bool(torch.isnan(dirty[0, 50:, :, 9]).all())


# ---------------------------------------------- 8-bit pages: scales and queries far from one
def _far(td, fmt, n, q_log2, k_log2, seed):
    b = ck.Batch([150], [n], 2, 128, 16, seed=seed)
    kv = b.rows(*b.pool_shape()).float()
    kv[:, 0] *= 2.0 ** k_log2
    pages, codes, scale, val = _pages8(td, b, kv.to(torch.bfloat16), fmt)
    q = (b.rows(1, b.T, 6, 128).float() * 2.0 ** q_log2).to(torch.bfloat16)
    got = _run_attention(td, b, pages, q, q8=True)
    _close(got, ck.attend(b, val[:, 0], val[:, 1], q), _weight_step(b, 3))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n", [2, 100, 300])
def test_large_scales_meet_small_queries(td, n, fmt):
    """K's scales around 2^106 and queries around 2^-104: scores of some hundreds. A score before
    its scales reaches 2^25 and more, which times K's scale alone is past float32."""
    _far(td, fmt, n, -104, 112, 65)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n", [2, 100, 300])
def test_the_smallest_queries(td, n, fmt):
    """Queries around 2^-115, next to the least normal numbers, and K's scales around 2^109. The
    query row's power of two times the softmax scale is then a subnormal of 20 bits or more: 2^-21 of a
    score, within the bound's 2^-16."""
    _far(td, fmt, n, -115, 115, 66)


@pytest.mark.parametrize("scale", [1e-38, -1e-38, 0.0])
@pytest.mark.parametrize("n", [2, 100])
def test_the_smallest_softmax_scales(td, n, scale):
    """q . k around 2^126 times a softmax scale next to the least float32: scores around 1; and a
    scale of 0, where every position counts alike."""
    b = ck.Batch([150], [n], 2, 128, 16, seed=67)
    pool, q = b.rows(*b.pool_shape()).float(), b.rows(1, b.T, 6, 128).float()
    pool[:, 0] *= 2.0 ** 61
    pool, q = pool.to(torch.bfloat16), (q * 2.0 ** 60).to(torch.bfloat16)
    # what the calls take: the scale as a float32 in base 2, a subnormal of 2^-149 steps
    s2 = float(np.float32(np.float32(scale) * np.float32(1.4426950408889634)))
    got = _run_attention(td, b, td.make_paged(pool, b.bt_t), q, scale=scale)
    out, lse, mag, dot = ck.attend(b, pool[:, 0].double(), pool[:, 1].double(), q,
                                   scale=s2 * math.log(2.0))
    _close(got, (out, lse, mag, dot.abs()), _weight_step(b, 3))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n", [2, 100, 300])
def test_a_large_scale_of_a_row_of_zero_codes(td, n, fmt):
    """Codes of zero under a scale of 2^100, queries around 2^60, the other rows' scales around
    2^-60: that position's score is 0, not infinity times 0."""
    b = ck.Batch([150], [n], 2, 128, 16, seed=68)
    kv = b.rows(*b.pool_shape()).float()
    kv[:, 0] *= 2.0 ** -60
    pg, sl = b.place(0, np.array([7, 131, 150]))
    kv[0, 0, pg, sl] = 0
    _, codes, scale, val = _pages8(td, b, kv.to(torch.bfloat16), fmt)
    scale[0, 0, pg, sl] = 2.0 ** 100
    q = (b.rows(1, b.T, 6, 128).float() * 2.0 ** 60).to(torch.bfloat16)
    got = _run_attention(td, b, td.make_paged8(codes, scale, b.bt_t, fmt), q, q8=True)
    _close(got, ck.attend(b, val[:, 0], val[:, 1], q), _weight_step(b, 3))


# ----------------------------------------------------------------- large values under the sums
@pytest.mark.parametrize("fmt", ["", "int8", "e4m3"])
@pytest.mark.parametrize("n", [2, 40, 300])
def test_weights_stay_at_one_or_less(td, n, fmt):
    """A later tile's score is 7.5 (in base 2) over all before it, and its V next to the largest
    float32 in half of its dims: weights over 1 would make its term infinite, where the row's
    value is 181 / (200 + 181) of it or less."""
    b = ck.Batch([200], [n], 1, 128, 16, seed=69)
    kv = b.rows(*b.pool_shape())
    q = torch.zeros((1, n, 3, 128), dtype=torch.bfloat16, device="cuda")
    kv[:, 0] = 0
    q[..., 0] = 1.0
    pg, sl = b.place(0, np.array([140]))
    kv[0, 0, pg, sl, 0, 0] = 7.5
    kv[0, 1, pg, sl, 0] = 0
    kv[0, 1, pg, sl, 0, :64] = 2e38
    if fmt:
        pages, _, _, val = _pages8(td, b, kv, fmt)
    else:
        pages, val = td.make_paged(kv, b.bt_t), kv.double()
    got = _run_attention(td, b, pages, q, scale=math.log(2.0), q8=bool(fmt))
    _close(got, ck.attend(b, val[:, 0], val[:, 1], q, scale=math.log(2.0)), _weight_step(b, 3))


# ------------------------------------------------------------------------------ 8-bit codes
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_every_code_is_read_as_the_value_it_stands_for(td, fmt):
    """All 256 bytes, the two that e4m3 reads as NaN and int8's -128 among them."""
    b = ck.Batch([5], [9], 2, 128, 16, seed=70)
    codes = torch.arange(int(np.prod(b.pool_shape())), device="cuda").to(torch.int8)
    codes = codes.view(b.pool_shape()).contiguous()
    scale = torch.rand(b.pool_shape()[:-1], generator=b.gen, device="cuda") * 3 + 0.01
    ctx = _ctx(td, b)
    k, v = (torch.zeros((1, b.T, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    td.td_dequantise_read(ctx.handle, _chunks(td, b), td.make_paged8(codes, scale, b.bt_t, fmt), 0, 1,
                          k.data_ptr(), v.data_ptr(), _stream())
    assert _errors(td, ctx) == (0, 0)
    pg, sl = b.place(0, np.arange(5, 14))
    want = (ck.code_values(codes, fmt).float() * scale[..., None]).to(torch.bfloat16)
    for kv, got in enumerate((k, v)):
        w = want[:, kv, pg, sl]
        assert torch.equal(torch.isnan(got), torch.isnan(w))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(w))


# --------------------------------------------- 8-bit pages: layer ranges, far offsets, holes
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("lens", [[2, 1], [100, 31], [300, 2]])
def test_layers_of_a_range_over_8bit_pages(td, lens, fmt):
    """Layers 2 and 3 of 4, on each way through the attention."""
    b = ck.Batch([200, 31], lens, 2, 64, 16, 4, seed=71)
    pages, _, _, val = _pages8(td, b, b.rows(*b.pool_shape()), fmt)
    q = b.rows(2, b.T, 6, 64)
    ctx = _ctx(td, b)
    out, z = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    td.td_chunk_attention_q8(ctx.handle, _chunks(td, b), pages, 2, 4, q.data_ptr(), 6, 0.125, 0, 0,
                             out.data_ptr(), z.data_ptr(), _stream())
    assert _errors(td, ctx) == (0, 0)
    b.L = 2
    _close((out, z), ck.attend(b, val[2:, 0], val[2:, 1], q), _weight_step(b, 3))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_8bit_pages_beyond_32_bit_offsets(td, fmt):
    """A pool of more than 2^32 bytes of codes: the same bits as from a small one."""
    H, D, P, L = 8, 128, 16, 2
    pages = 70000                                # 2 layers: 4.6e9 codes
    codes = torch.zeros((L, 2, pages, P, H, D), dtype=torch.int8, device="cuda")
    scale = torch.zeros((L, 2, pages, P, H), device="cuda")
    for lens in ([1, 1], [130, 40], [300, 40]):
        b = ck.Batch([400, 90], lens, H, D, P, L, seed=72)
        near, c, s, _ = _pages8(td, b, b.rows(*b.pool_shape()), fmt)
        far = torch.where(b.bt_t >= 0, pages - 1 - b.bt_t, -1).to(torch.int32).contiguous()
        codes[:, :, pages - b.pages:] = c.flip(2)
        scale[:, :, pages - b.pages:] = s.flip(2)
        q = b.rows(L, b.T, H * 2, D)
        one = _run_attention(td, b, near, q, q8=True)
        two = _run_attention(td, b, td.make_paged8(codes, scale, far, fmt), q, q8=True)
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
        assert bool(torch.isfinite(one[0]).all())


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n", [2, 100])
def test_a_scale_that_is_not_finite_in_the_middle_of_a_chunk(td, n, fmt):
    """K's or V's scale of a token within the chunk is a NaN: the rows that see it are NaN, the
    tokens before it and the other kv head keep to float64."""
    b = ck.Batch([150], [n], 2, 128, 16, seed=73)
    pages, codes, scale, val = _pages8(td, b, b.rows(*b.pool_shape()), fmt)
    q = b.rows(1, b.T, 4, 128)
    want = ck.attend(b, val[:, 0], val[:, 1], q)
    at = n // 2
    pg, sl = b.place(0, np.array([150 + at]))
    for half in (0, 1):
        dirty = scale.clone()
        dirty[0, half, pg, sl, 1] = math.nan
        out, z = _run_attention(td, b, td.make_paged8(codes, dirty, b.bt_t, fmt), q, q8=True)
        step = _weight_step(b, 2)
        _close((out[:, :at], z[:, :at]), [t[:, :at] for t in want], step)
        _close((out[:, :, :2], z[:, :, :2]), [t[:, :, :2] for t in want], step)
        assert bool(torch.isnan(out[0, at:, 2:]).all())
