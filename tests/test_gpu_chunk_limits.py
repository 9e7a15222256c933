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
