"""Chunks of new tokens over paged caches: td_quantise_append, td_dequantise_read,
td_chunk_attention and td_chunk_attention_q8 against float64 references (tests/chunkkit.py)."""
from __future__ import annotations

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import chunkkit as ck

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def td():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from collective_kv_cache_gb300 import build
    build.build()
    from collective_kv_cache_gb300 import td as _td
    return _td


def _ctx(td, b, max_agents=None):
    return td.Context(td.td_shape(b.L, b.H, b.D, b.P, 16, 1e6), max_agents or b.n_agents, 1, 1)


def _chunks(td, b):
    return td.make_chunks(b.agents, b.starts, b.lens)


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _errors(td, ctx):
    return td.td_get_error(ctx.handle, _stream())


# ------------------------------------------------------------------- 8-bit pages: writing
WRITES = {
    # name: (starts, lens, H, D, P, L)
    "one_token": ([37], [1], 2, 64, 16, 1),
    "ragged": ([0, 15, 16, 200], [1, 17, 33, 100], 4, 128, 16, 3),
    "no_tokens_between": ([5, 9, 3], [4, 0, 7], 1, 64, 24, 2),
    "narrow_d16": ([3, 8], [19, 5], 8, 16, 8, 2),
    "odd_d48": ([1, 30], [31, 12], 3, 48, 5, 1),
    "wide_d256": ([2], [40], 2, 256, 32, 1),
    "heads_128x16": ([7], [9], 128, 16, 16, 1),
    "page_of_one": ([0, 2], [6, 11], 2, 64, 1, 1),
    "many_tokens": ([11, 0], [3000, 1717], 4, 128, 16, 2),
}


def _special_rows(x):
    """Rows where rounding and scaling can go wrong, put over the first tokens of x."""
    T, H, D = x.shape[1:]
    f = x.view(-1, D)
    cases = [torch.zeros(D), torch.full((D,), 3.0e38), torch.full((D,), 1e-40),
             torch.arange(D).float() - D / 2, torch.full((D,), -2.0 ** -133),
             (torch.arange(D).float() % 255 - 127.0),           # exact codes of amax 127
             (torch.arange(D).float() % 255 - 127.0) / 2.0,     # ties where amax = 63.5
             1.75 * 2.0 ** (torch.arange(D).float() % 20),      # up to a power of two times 448
             1.7578125 * 2.0 ** -(torch.arange(D).float() % 20)]
    for i, c in enumerate(cases[:f.shape[0] // 2]):
        f[2 * i] = c.to(x.device).to(torch.bfloat16)
    return x


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("name", list(WRITES))
def test_append_writes_the_exact_codes_and_nothing_else(td, name, fmt):
    starts, lens, H, D, P, L = WRITES[name]
    b = ck.Batch(starts, lens, H, D, P, L + 2, seed=3)       # layers 1 .. L of L + 2
    ctx = _ctx(td, b)
    k, v = _special_rows(b.rows(L, b.T, H, D)), b.rows(L, b.T, H, D, scale=17.0)
    codes = torch.full(b.pool_shape(), 0x55, dtype=torch.int8, device="cuda")
    scale = torch.full(b.pool_shape()[:-1], -7.0, dtype=torch.float32, device="cuda")
    want_c, want_s = codes.clone(), scale.clone()
    for kv, x in enumerate((k, v)):
        val, s = ck.quantise(x, fmt)
        for i in range(len(lens)):
            pg, sl = b.place(i, np.arange(starts[i], starts[i] + lens[i]))
            want_c[1:L + 1, kv, pg, sl] = ck.code_bytes(val[:, b.chunk_rows(i)], fmt)
            want_s[1:L + 1, kv, pg, sl] = s[:, b.chunk_rows(i)].float()
    td.td_quantise_append(ctx.handle, _chunks(td, b), td.make_paged8(codes, scale, b.bt_t, fmt),
                          k.data_ptr(), v.data_ptr(), 1, L + 1, _stream())
    assert _errors(td, ctx) == (0, 0)
    assert torch.equal(scale, want_s)
    # a negative value that rounds to zero keeps its sign in e4m3: compare values there
    assert torch.equal(ck.code_values(codes, fmt), ck.code_values(want_c, fmt))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_places_every_quotient_next_to_a_border(td, fmt):
    """Rows of every bf16 significand under many maxima: the codes are those of the exact
    quotients, ties to even included."""
    D, P, T = 128, 16, 1024
    b = ck.Batch([0], [T], 1, D, P, seed=4)
    ctx = _ctx(td, b)
    i = torch.arange(T * D, device="cuda").view(1, T, 1, D)
    x = ((i * 37 % 256).float() + 0.0) * torch.where(i % 2 == 0, 1.0, -1.0)
    x[..., 0] = (128 + torch.arange(T, device="cuda") % 128).float().view(1, T, 1)
    x = x.clamp(-255, 255).to(torch.bfloat16).contiguous()
    x = torch.where(x.abs() > x[..., :1], x[..., :1], x).contiguous()
    codes = torch.zeros(b.pool_shape(), dtype=torch.int8, device="cuda")
    scale = torch.zeros(b.pool_shape()[:-1], device="cuda")
    td.td_quantise_append(ctx.handle, _chunks(td, b), td.make_paged8(codes, scale, b.bt_t, fmt),
                          x.data_ptr(), x.data_ptr(), 0, 1, _stream())
    val, s = ck.quantise(x, fmt)
    pg, sl = b.place(0, np.arange(T))
    assert torch.equal(scale[0, 0, pg, sl], s[0].float())
    assert torch.equal(ck.code_values(codes, fmt)[0, 0, pg, sl], val[0])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_marks_rows_that_are_not_finite(td, fmt):
    b = ck.Batch([3], [6], 2, 64, 16, seed=5)
    ctx = _ctx(td, b)
    k, v = b.rows(1, 6, 2, 64), b.rows(1, 6, 2, 64)
    k[0, 2, 1, 63] = math.nan
    v[0, 4, 0, 0] = -math.inf
    codes = torch.ones(b.pool_shape(), dtype=torch.int8, device="cuda")
    scale = torch.ones(b.pool_shape()[:-1], device="cuda")
    pages = td.make_paged8(codes, scale, b.bt_t, fmt)
    td.td_quantise_append(ctx.handle, _chunks(td, b), pages, k.data_ptr(), v.data_ptr(), 0, 1,
                          _stream())
    assert _errors(td, ctx) == (td.TD_ERR_NONFINITE, 1 << td.TD_ERR_NONFINITE)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    td.td_dequantise_read(ctx.handle, _chunks(td, b), pages, 0, 1, ko.data_ptr(), vo.data_ptr(),
                          _stream())
    bad_k, bad_v = torch.isnan(ko).all(-1)[0], torch.isnan(vo).all(-1)[0]
    assert bad_k.nonzero().tolist() == [[2, 1]] and bad_v.nonzero().tolist() == [[4, 0]]
    assert int(torch.isnan(ko).sum()) == 64 and int(torch.isnan(vo).sum()) == 64


# ------------------------------------------------------------------ 8-bit pages: reading
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("name", list(WRITES))
def test_read_gives_the_values_the_pages_stand_for(td, name, fmt):
    starts, lens, H, D, P, L = WRITES[name]
    b = ck.Batch(starts, lens, H, D, P, L + 1, seed=6)       # layers 1 .. L of L + 1
    ctx = _ctx(td, b)
    # every byte but the ones no write produces (-128; the NaNs 0x7F and 0xFF)
    codes = torch.randint(-127, 127, b.pool_shape(), dtype=torch.int8, device="cuda")
    codes = torch.where((codes == 127) | (codes == -1), 1, codes).to(torch.int8)
    scale = torch.rand(b.pool_shape()[:-1], device="cuda") * 3 + 2.0 ** -9
    ko = torch.full((L, b.T + 2, H, D), 9.0, dtype=torch.bfloat16, device="cuda")[:, :b.T].contiguous()
    guard = torch.full((2, L * b.T * H * D + 64,), 9.0, dtype=torch.bfloat16, device="cuda")
    ko, vo = (g[:L * b.T * H * D].view(L, b.T, H, D) for g in guard)
    td.td_dequantise_read(ctx.handle, _chunks(td, b), td.make_paged8(codes, scale, b.bt_t, fmt), 1,
                          L + 1, ko.data_ptr(), vo.data_ptr(), _stream())
    assert _errors(td, ctx) == (0, 0)
    val = ck.code_values(codes, fmt).float() * scale[..., None]
    for i in range(len(lens)):
        pg, sl = b.place(i, np.arange(starts[i], starts[i] + lens[i]))
        for kv, got in enumerate((ko, vo)):
            want = val[1:, kv, pg, sl].to(torch.bfloat16)
            assert torch.equal(got[:, b.chunk_rows(i)], want)
    assert bool((guard[:, L * b.T * H * D:] == 9.0).all())      # rows past the last: left alone


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_unmapped_pages_of_a_write_and_a_read(td, fmt):
    b = ck.Batch([10, 0], [30, 20], 2, 64, 16, seed=7)
    hole = int(b.bt[0, 1])
    b.bt_t[0, 1] = -1
    b.bt_t[1, 0] = b.pages                                  # out of range
    ctx = _ctx(td, b)
    k, v = b.rows(1, 50, 2, 64), b.rows(1, 50, 2, 64)
    codes = torch.full(b.pool_shape(), 3, dtype=torch.int8, device="cuda")
    scale = torch.full(b.pool_shape()[:-1], 0.5, device="cuda")
    pages = td.make_paged8(codes, scale, b.bt_t, fmt)
    td.td_quantise_append(ctx.handle, _chunks(td, b), pages, k.data_ptr(), v.data_ptr(), 0, 1,
                          _stream())
    assert _errors(td, ctx)[0] == td.TD_ERR_UNMAPPED_PAGE
    assert bool((codes[:, :, hole] == 3).all()) and bool((scale[:, :, hole] == 0.5).all())
    ko, vo = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    td.td_dequantise_read(ctx.handle, _chunks(td, b), pages, 0, 1, ko.data_ptr(), vo.data_ptr(),
                          _stream())
    assert _errors(td, ctx)[0] == td.TD_ERR_UNMAPPED_PAGE
    pos = torch.cat([torch.arange(10, 40), torch.arange(20)])
    out = torch.cat([(pos[:30] >= 16) & (pos[:30] < 32), pos[30:] < 16])
    assert bool((ko[0, out.cuda()] == 0).all()) and bool((vo[0, out.cuda()] == 0).all())
    val, s = ck.quantise(k[0, :6], fmt)
    assert torch.equal(ko[0, :6], (val.float() * s.float()[..., None]).to(torch.bfloat16))


# -------------------------------------------------------------------------- attention
ATTEND = {
    # name: (starts, lens, H, G, D, P, window, sinks)
    "first_token": ([0], [1], 1, 1, 64, 16, 0, 0),
    "one_token": ([33], [1], 2, 3, 64, 16, 0, 0),
    "one_token_g8": ([700, 5, 129], [1, 1, 1], 2, 8, 128, 16, 0, 0),
    "tokens_and_none": ([7, 40, 300], [1, 0, 2], 2, 7, 128, 24, 0, 0),
    "few_tokens_g5": ([100, 3], [3, 2], 2, 5, 128, 16, 0, 0),
    "prompt_alone": ([0], [65], 2, 2, 64, 16, 0, 0),
    "chunk_g7": ([130, 0, 1000], [100, 19, 37], 2, 7, 128, 16, 0, 0),
    "chunk_g1": ([500], [300], 3, 1, 128, 32, 0, 0),
    "chunk_g16": ([64], [33], 1, 16, 64, 16, 0, 0),
    "chunk_g40": ([10], [9], 1, 40, 128, 16, 0, 0),
    "page_of_one": ([9], [12], 2, 2, 64, 1, 0, 0),
    "page_of_five": ([131], [140], 1, 3, 128, 5, 0, 0),
    "page_of_24": ([100, 255], [257, 30], 2, 3, 128, 24, 0, 0),
    "page_of_8_d64": ([77], [200], 2, 4, 64, 8, 0, 0),
    "page_of_256": ([300], [300], 1, 2, 128, 256, 0, 0),
    "long_context": ([5000], [3], 2, 7, 128, 16, 0, 0),
    "chunk_long_context": ([3000, 2500], [70, 130], 2, 7, 128, 16, 0, 0),
    "window_token": ([900], [1], 2, 7, 128, 16, 100, 4),
    "window_of_one": ([50], [20], 2, 2, 64, 16, 1, 0),
    "window_no_sinks": ([200, 0], [150, 90], 2, 3, 128, 24, 65, 0),
    "window_sinks": ([400, 2], [300, 150], 2, 7, 128, 16, 130, 4),
    "window_sinks_d64": ([1000], [520], 1, 8, 64, 16, 256, 7),
    "window_beyond": ([30], [40], 2, 2, 128, 16, 5000, 3),
    "sinks_beyond_window": ([600], [40], 2, 2, 128, 16, 16, 300),
}


def _run_attention(td, b, pages, q, window=0, sinks=0, scale=None, q8=False, ctx=None, lse=True,
                   expect=(0, 0)):
    ctx = ctx or _ctx(td, b)
    out = torch.full(q.shape, math.nan, dtype=torch.bfloat16, device="cuda")
    z = torch.full(q.shape[:3], math.nan, device="cuda")
    call = td.td_chunk_attention_q8 if q8 else td.td_chunk_attention
    call(ctx.handle, _chunks(td, b), pages, 0, b.L, q.data_ptr(), q.shape[2],
         1.0 / math.sqrt(b.D) if scale is None else scale, window, sinks, out.data_ptr(),
         z.data_ptr() if lse else None, _stream())
    assert _errors(td, ctx) == expect
    return out, z


def _close(got, want, weight_step):
    out, z = got
    o, lse, mag, dot = want
    tol, tol_lse = ck.bounds(o, mag, dot, weight_step)
    err = (out.double() - o).abs()
    assert bool((err <= tol).all()), (float((err - tol).max()), float((err / tol).max()))
    e2 = (z.double() - lse).abs()
    both = (z == -math.inf) & (lse == -math.inf)
    assert bool((both | (e2 <= tol_lse)).all()), float(e2.max())


def _weight_step(b, G):
    """Chunks of at most 16 query rows keep 16 bits of a weight, longer ones bf16's 8."""
    return 2.0 ** -16 if max(b.lens) * G <= 16 else 2.0 ** -8


@pytest.mark.parametrize("name", list(ATTEND))
def test_chunk_attention_over_bf16_pages(td, name):
    starts, lens, H, G, D, P, window, sinks = ATTEND[name]
    b = ck.Batch(starts, lens, H, D, P, 2, seed=11)
    pool, q = b.rows(*b.pool_shape()), b.rows(2, b.T, H * G, D)
    got = _run_attention(td, b, td.make_paged(pool, b.bt_t), q, window, sinks)
    want = ck.attend(b, pool[:, 0].double(), pool[:, 1].double(), q, window, sinks)
    _close(got, want, _weight_step(b, G))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("name", list(ATTEND))
def test_chunk_attention_over_8bit_pages(td, name, fmt):
    starts, lens, H, G, D, P, window, sinks = ATTEND[name]
    b = ck.Batch(starts, lens, H, D, P, 1, seed=12)
    val, s = ck.quantise(b.rows(*b.pool_shape()), fmt)
    codes, scale = ck.code_bytes(val, fmt).contiguous(), s.float().contiguous()
    q = b.rows(1, b.T, H * G, D)
    got = _run_attention(td, b, td.make_paged8(codes, scale, b.bt_t, fmt), q, window, sinks, q8=True)
    kv = val * s[..., None]
    want = ck.attend(b, kv[:, 0], kv[:, 1], q, window, sinks)
    _close(got, want, _weight_step(b, G))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("lens", [[1, 2], [40, 150]])
def test_places_out_of_sight_hold_anything(td, lens, q8):
    """NaN in every place that no token of its sequence sees, pages out of the window
    unmapped: the results are those of clean pages, and no error is recorded."""
    b = ck.Batch([500, 301], lens, 2, 128, 16, seed=13)
    W, sinks, G = 70, 4, 3
    pool, q = b.rows(*b.pool_shape()), b.rows(1, b.T, 6, 128)
    want = ck.attend(b, pool[:, 0].double(), pool[:, 1].double(), q, W, sinks)
    seen = torch.zeros(b.pool_shape()[2:4], dtype=torch.bool, device="cuda")
    for x in range(2):
        lo = b.starts[x] - W + 1
        vis = np.concatenate([np.arange(sinks), np.arange(lo, b.starts[x] + lens[x])])
        pg, sl = b.place(x, vis)
        seen[pg, sl] = True
        b.bt_t[x, sinks // 16 + 1: lo // 16] = -1
    if q8:
        val, s = ck.quantise(pool, "e4m3")
        kv = val * s[..., None]
        want = ck.attend(b, kv[:, 0], kv[:, 1], q, W, sinks)
        codes, scale = ck.code_bytes(val, "e4m3").contiguous(), s.float().contiguous()
        codes[:, :, ~seen] = 0x7F
        scale[:, :, ~seen] = math.nan
        pages = td.make_paged8(codes, scale, b.bt_t, "e4m3")
    else:
        pool[:, :, ~seen] = math.nan
        pages = td.make_paged(pool, b.bt_t)
    got = _run_attention(td, b, pages, q, W, sinks, q8=q8)
    _close(got, want, _weight_step(b, G))


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("case", [(2, 3, 128), (40, 3, 128), (170, 2, 64), (300, 7, 128)])
def test_a_value_of_a_later_token_does_not_reach_earlier_ones(td, case, which, value):
    """K or V of a token in the middle of the chunk holds a NaN or an infinity: the tokens
    before it, and under the window those that have lost it, keep their results: bit for bit
    where K holds it, and within the bounds against float64 where V does (such rows may be
    computed by other arithmetic)."""
    n, G, D = case
    b = ck.Batch([150], [n], 2, D, 16, seed=14)
    W = 0 if n != 170 else 60
    pool, q = b.rows(*b.pool_shape()), b.rows(1, n, 2 * G, D)
    clean, zc = _run_attention(td, b, td.make_paged(pool, b.bt_t), q, W, 0)
    want = ck.attend(b, pool[:, 0].double(), pool[:, 1].double(), q, W, 0)
    at = 150 + n // 2
    pg, sl = b.place(0, np.array([at]))
    pool[0, 0 if which == "k" else 1, pg, sl, 1, 5] = value
    dirty, zd = _run_attention(td, b, td.make_paged(pool, b.bt_t), q, W, 0)
    pos = 150 + torch.arange(n, device="cuda")
    blind = (pos < at) | (pos >= at + W if W else pos < 0)
    assert torch.equal(clean[0, :, :G], dirty[0, :, :G]) and torch.equal(zc[0, :, :G], zd[0, :, :G])
    if which == "k":
        assert torch.equal(clean[0, blind], dirty[0, blind]) and torch.equal(zc[0, blind], zd[0, blind])
    else:
        _close((dirty[:, blind], zd[:, blind]), [t[:, blind] for t in want], _weight_step(b, G))
    sees = dirty[0, ~blind][:, G:]
    if which == "v":
        col = sees[..., 5]
        assert not bool(torch.isfinite(col).any())
        rest = torch.cat([sees[..., :5], sees[..., 6:]], -1)
        assert bool(torch.isfinite(rest).all())
    elif math.isnan(value):
        assert bool(torch.isnan(sees).all())


def test_rows_that_see_only_unmapped_pages_are_zeros(td):
    for lens in ([1, 3], [30, 200]):
        b = ck.Batch([100, 64], lens, 2, 128, 16, seed=15)
        b.bt_t[0] = -1
        b.bt_t[1, 1] = -1
        pool, q = b.rows(*b.pool_shape()), b.rows(1, b.T, 4, 128)
        got = _run_attention(td, b, td.make_paged(pool, b.bt_t), q,
                             expect=(td.TD_ERR_UNMAPPED_PAGE, 1 << td.TD_ERR_UNMAPPED_PAGE))
        assert bool((got[0][:, :lens[0]] == 0).all())
        assert bool((got[1][:, :lens[0]] == -math.inf).all())
        want = ck.attend(b, pool[:, 0].double(), pool[:, 1].double(), q)
        _close(got, want, _weight_step(b, 2))


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
@pytest.mark.parametrize("lens", [[2], [90]])
def test_other_scales(td, lens, scale):
    b = ck.Batch([200], lens, 1, 128, 16, seed=16)
    pool, q = b.rows(*b.pool_shape()), b.rows(1, b.T, 3, 128)
    got = _run_attention(td, b, td.make_paged(pool, b.bt_t), q, scale=scale)
    out, lse, mag, dot = ck.attend(b, pool[:, 0].double(), pool[:, 1].double(), q, scale=scale)
    _close(got, (out, lse, mag, dot.abs()), _weight_step(b, 3))


@pytest.mark.parametrize("lens", [[1, 3], [100, 40]])
def test_windows_and_sinks_of_any_size(td, lens):
    """A window past every position is none, whatever the sinks; sinks past it keep all."""
    b = ck.Batch([300, 7], lens, 2, 64, 16, seed=35)
    pool, q = b.rows(*b.pool_shape()), b.rows(1, b.T, 4, 64)
    pages, ctx = td.make_paged(pool, b.bt_t), _ctx(td, b)
    want = ck.attend(b, pool[:, 0].double(), pool[:, 1].double(), q)
    for window, sinks in ((2**31 - 1, 0), (2**31 - 1, 2**31 - 1), (2**30, 5), (1, 2**31 - 1)):
        _close(_run_attention(td, b, pages, q, window, sinks, ctx=ctx), want, _weight_step(b, 2))


def test_three_hundred_sequences_span_two_launches(td):
    rng = np.random.RandomState(1)
    for lens in ([1] * 300, list(rng.randint(0, 40, 300))):
        starts = list(rng.randint(0, 90, 300))
        b = ck.Batch(starts, lens, 1, 64, 16, seed=17)
        pool, q = b.rows(*b.pool_shape()), b.rows(1, b.T, 2, 64)
        got = _run_attention(td, b, td.make_paged(pool, b.bt_t), q)
        want = ck.attend(b, pool[:, 0].double(), pool[:, 1].double(), q)
        _close(got, want, _weight_step(b, 2))
        ctx = _ctx(td, b)
        k, v = b.rows(1, b.T, 1, 64), b.rows(1, b.T, 1, 64)
        codes = torch.zeros(b.pool_shape(), dtype=torch.int8, device="cuda")
        sc = torch.zeros(b.pool_shape()[:-1], device="cuda")
        pages = td.make_paged8(codes, sc, b.bt_t, "int8")
        td.td_quantise_append(ctx.handle, _chunks(td, b), pages, k.data_ptr(), v.data_ptr(), 0, 1,
                              _stream())
        ko, vo = torch.empty_like(k), torch.empty_like(v)
        td.td_dequantise_read(ctx.handle, _chunks(td, b), pages, 0, 1, ko.data_ptr(),
                              vo.data_ptr(), _stream())
        for x, o in ((k, ko), (v, vo)):
            val, s = ck.quantise(x, "int8")
            assert torch.equal(o, (val.float() * s.float()[..., None]).to(torch.bfloat16))


def test_one_agent_listed_twice(td):
    """Two chunks of one agent: the same rows as a batch with each alone."""
    b = ck.Batch([20, 61, 20], [3, 40, 3], 2, 128, 16, agents=[1, 1, 1], n_agents=3, seed=18)
    pool, q = b.rows(*b.pool_shape()), b.rows(1, b.T, 4, 128)
    q[:, 43:] = q[:, :3]
    got = _run_attention(td, b, td.make_paged(pool, b.bt_t), q)
    assert torch.equal(got[0][:, 43:], got[0][:, :3])
    want = ck.attend(b, pool[:, 0].double(), pool[:, 1].double(), q)
    _close(got, want, 2.0 ** -8)


def test_same_bits_twice_and_without_lse(td):
    for lens in ([1] * 6, [300, 7, 0, 64, 1, 33]):
        b = ck.Batch([900, 5, 3, 640, 77, 2000], lens, 2, 128, 16, seed=19)
        pool, q = b.rows(*b.pool_shape()), b.rows(1, b.T, 14, 128)
        pages, ctx = td.make_paged(pool, b.bt_t), _ctx(td, b)
        one = _run_attention(td, b, pages, q, ctx=ctx)
        two = _run_attention(td, b, pages, q, ctx=ctx)
        bare = _run_attention(td, b, pages, q, ctx=ctx, lse=False)
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
        assert torch.equal(one[0], bare[0]) and bool(torch.isnan(bare[1]).all())


def test_layers_of_a_range(td):
    b = ck.Batch([200, 31], [20, 1], 2, 64, 16, 4, seed=20)
    pool, q = b.rows(*b.pool_shape()), b.rows(2, b.T, 4, 64)
    ctx = _ctx(td, b)
    out = torch.empty_like(q)
    z = torch.empty(q.shape[:3], device="cuda")
    td.td_chunk_attention(ctx.handle, _chunks(td, b), td.make_paged(pool, b.bt_t), 2, 4,
                          q.data_ptr(), 4, 0.125, 0, 0, out.data_ptr(), z.data_ptr(), _stream())
    b.L = 2
    want = ck.attend(b, pool[2:, 0].double(), pool[2:, 1].double(), q)
    _close((out, z), want, 2.0 ** -8)


@pytest.mark.parametrize("lens", [[1, 1], [130, 40]])
def test_pages_beyond_32_bit_offsets(td, lens):
    """A pool of more than 2^32 bytes and 2^31 elements: rows are found by 64-bit offsets."""
    H, D, P, L = 8, 128, 16, 2
    pages = 70000                                # 2 layers: 4.6e9 elements, 9.2 GB
    b = ck.Batch([400, 90], lens, H, D, P, L, seed=21)
    far = torch.where(b.bt_t >= 0, pages - 1 - b.bt_t, -1).to(torch.int32).contiguous()
    near = b.rows(L, 2, b.pages, P, H, D)
    pool = torch.empty((L, 2, pages, P, H, D), dtype=torch.bfloat16, device="cuda")
    pool[:, :, pages - b.pages:] = near.flip(2)
    q = b.rows(L, b.T, H * 2, D)
    one = _run_attention(td, b, td.make_paged(near, b.bt_t), q)
    two = _run_attention(td, b, td.make_paged(pool, far), q)
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    del pool
    codes = torch.empty((L, 2, pages, P, H, D), dtype=torch.int8, device="cuda")
    sc = torch.empty((L, 2, pages, P, H), device="cuda")
    k, v = b.rows(L, b.T, H, D), b.rows(L, b.T, H, D)
    ctx = _ctx(td, b)
    pg = td.make_paged8(codes, sc, far, "int8")
    td.td_quantise_append(ctx.handle, _chunks(td, b), pg, k.data_ptr(), v.data_ptr(), 0, L, _stream())
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    td.td_dequantise_read(ctx.handle, _chunks(td, b), pg, 0, L, ko.data_ptr(), vo.data_ptr(),
                          _stream())
    for x, o in ((k, ko), (v, vo)):
        val, s = ck.quantise(x, "int8")
        assert torch.equal(o, (val.float() * s.float()[..., None]).to(torch.bfloat16))


# --------------------------------------------------------------- streams, graphs, together
@pytest.mark.parametrize("lens", [[1, 1, 1], [200, 33, 64]])
def test_on_another_stream_and_in_a_captured_graph(td, lens):
    b = ck.Batch([2000, 10, 333], lens, 2, 128, 16, seed=22)
    pool, q = b.rows(*b.pool_shape()), b.rows(1, b.T, 14, 128)
    pages, ctx = td.make_paged(pool, b.bt_t), _ctx(td, b)
    want = _run_attention(td, b, pages, q, ctx=ctx)
    ch, scale = _chunks(td, b), 1.0 / math.sqrt(128)
    out, z = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")

    def call(s):
        td.td_chunk_attention(ctx.handle, ch, pages, 0, 1, q.data_ptr(), 14, scale, 0, 0,
                              out.data_ptr(), z.data_ptr(), s)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side.cuda_stream)
    side.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(z, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        call(side.cuda_stream)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0])
    # a larger call grows the scratch; the graph's buffer stays valid, and new values are read
    big = ck.Batch([30000], [1], 2, 128, 16, seed=23)
    bp, bq = big.rows(*big.pool_shape()), big.rows(1, 1, 14, 128)
    big.n_agents = b.n_agents
    _run_attention(td, big, td.make_paged(bp, big.bt_t), bq, ctx=ctx)
    q.copy_(b.rows(*q.shape))
    fresh = _run_attention(td, b, pages, q)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, fresh[0]) and torch.equal(z, fresh[1])


def test_a_capture_that_would_allocate_is_refused(td):
    b = ck.Batch([9000], [1], 2, 128, 16, seed=24)
    pool, q = b.rows(*b.pool_shape()), b.rows(1, 1, 14, 128)
    pages, ctx, ch = td.make_paged(pool, b.bt_t), _ctx(td, b), _chunks(td, b)
    out = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    x = torch.zeros(4, device="cuda")
    with torch.cuda.graph(g):
        x += 1
        s = td.td_chunk_attention(ctx.handle, ch, pages, 0, 1, q.data_ptr(), 14, 0.1, 0, 0,
                                  out.data_ptr(), None, _stream(), check=False)
    assert s == td.TD_ERR_INVALID_ARG
    g.replay()
    torch.cuda.synchronize()
    _run_attention(td, b, pages, q, ctx=ctx)


def test_contexts_on_two_streams_at_once(td):
    """Two contexts have their own scratch: their calls may overlap."""
    runs = []
    for i, st in enumerate((torch.cuda.Stream(), torch.cuda.Stream())):
        b = ck.Batch([4000 + i, 17], [1, 1 + i], 4, 128, 16, seed=25 + i)
        pool, q = b.rows(*b.pool_shape()), b.rows(1, b.T, 28, 128)
        pages, ctx = td.make_paged(pool, b.bt_t), _ctx(td, b)
        want = _run_attention(td, b, pages, q, ctx=ctx)
        runs.append((b, pool, q, pages, ctx, _chunks(td, b), torch.zeros_like(q), want, st))
    torch.cuda.synchronize()
    for _ in range(20):
        for b, pool, q, pages, ctx, ch, out, want, st in runs:
            td.td_chunk_attention(ctx.handle, ch, pages, 0, 1, q.data_ptr(), 28,
                                  1.0 / math.sqrt(128), 0, 0, out.data_ptr(), None, st.cuda_stream)
    torch.cuda.synchronize()
    for r in runs:
        assert torch.equal(r[6], r[7][0])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_a_sequence_grown_chunk_by_chunk(td, fmt):
    """As a server runs it: chunks of new tokens are written into 8-bit pages and attend to
    everything before them; the rows equal one attention over the whole prompt, and reading
    back gives what the attention saw."""
    H, G, D, P = 2, 3, 128, 16
    steps = [[40, 7], [1, 1], [90, 1], [1, 30], [1, 1]]
    total = [sum(s[i] for s in steps) for i in range(2)]
    whole = ck.Batch([0, 0], total, H, D, P, seed=31)
    ctx = _ctx(td, whole)
    k, v = whole.rows(1, whole.T, H, D), whole.rows(1, whole.T, H, D)
    q = whole.rows(1, whole.T, H * G, D)
    codes = torch.zeros(whole.pool_shape(), dtype=torch.int8, device="cuda")
    scale = torch.zeros(whole.pool_shape()[:-1], device="cuda")
    pages = td.make_paged8(codes, scale, whole.bt_t, fmt)
    got_o, got_z = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    pos = [0, 0]
    for s in steps:
        pick = torch.cat([whole.chunk_rows(i).start + torch.arange(pos[i], pos[i] + s[i])
                          for i in range(2)]).cuda()
        ch = td.make_chunks([0, 1], pos, s)
        kk, vv, qq = (t[:, pick].contiguous() for t in (k, v, q))
        o, z = torch.empty_like(qq), torch.empty(qq.shape[:3], device="cuda")
        td.td_quantise_append(ctx.handle, ch, pages, kk.data_ptr(), vv.data_ptr(), 0, 1, _stream())
        td.td_chunk_attention_q8(ctx.handle, ch, pages, 0, 1, qq.data_ptr(), H * G,
                                 1.0 / math.sqrt(D), 0, 0, o.data_ptr(), z.data_ptr(), _stream())
        got_o[:, pick], got_z[:, pick] = o, z
        pos = [pos[0] + s[0], pos[1] + s[1]]
    assert _errors(td, ctx) == (0, 0)
    val = ck.code_values(codes, fmt) * scale.double()[..., None]
    want = ck.attend(whole, val[:, 0], val[:, 1], q)
    _close((got_o, got_z), want, 2.0 ** -8)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    td.td_dequantise_read(ctx.handle, _chunks(td, whole), pages, 0, 1, ko.data_ptr(),
                          vo.data_ptr(), _stream())
    for x, o in ((k, ko), (v, vo)):
        c, s = ck.quantise(x, fmt)
        assert torch.equal(o, (c.float() * s.float()[..., None]).to(torch.bfloat16))


def test_after_a_restored_round(td):
    """The pages of a restored round read by a one-token chunk give what td_paged_attention
    gives over them (its float32 output rounded to bf16), and a recomputed span attends to
    the same pages."""
    import oracle
    from collective_kv_cache_gb300 import runner as R
    from collective_kv_cache_gb300 import synth
    from tests import roundkit as rk
    cfg = synth.RoundConfig(name="mini", n_agents=4, n_layers=2, n_kv_heads=2, head_dim=128,
                            page_size=16, block_lens=(20, 37, 16, 9), hist_range=(3, 45),
                            check_layer=1, recompute_pct=15, perturb_mode="runs",
                            perturb_frac=(0.10, 0.20), seed=101)
    nq = 6
    ch = rk.run_oracle_chain(rk.make_inputs(cfg, map_history=True), restore=False)
    rnd = ch.rnd
    pool = oracle.new_pool(cfg, rnd.num_pages, fill=ck.NAN16)
    rk.fill_history(cfg, rnd, pool)
    assert oracle.get().fused_restore(cfg, ch.desc, ch.master, ch.store, np.arange(4), pool,
                                      rnd.num_pages, rnd.block_table, frame=0) == 0
    rr = R.RoundRunner(cfg, rnd.block_len, rnd.hist_len, rnd.perm, rnd.block_table, rnd.num_pages)
    rr.pool_t.copy_(R.to_device_bf16(pool, "cuda").reshape(rr.pool_t.shape))
    agents = [2, 0, 3, 1]
    q = torch.randn((2, 4, nq, 128), device="cuda").to(torch.bfloat16)
    scale = 1.0 / math.sqrt(128)
    o32 = torch.empty(q.shape, device="cuda")
    z32 = torch.empty(q.shape[:3], device="cuda")
    td.td_paged_attention(rr.ctx.handle, rr.round, rr.pool, agents, 0, 2, q.data_ptr(), nq, scale,
                          o32.data_ptr(), z32.data_ptr(), rr.s)
    out, z = torch.empty_like(q), torch.empty_like(z32)
    last = [int(rnd.hist_len[a]) + cfg.n_shared - 1 for a in agents]
    td.td_chunk_attention(rr.ctx.handle, td.make_chunks(agents, last, [1] * 4), rr.pool, 0, 2,
                          q.data_ptr(), nq, scale, 0, 0, out.data_ptr(), z.data_ptr(), rr.s)
    torch.cuda.synchronize()
    assert rr.get_error() == (0, 0)
    assert torch.allclose(out.float(), o32, rtol=2.0 ** -7, atol=1e-5)
    assert torch.allclose(z, z32, atol=1e-4)
    # a span of each agent: its last token is the one above when given the same query
    n = 5
    qs = torch.randn((2, 4 * n, nq, 128), device="cuda").to(torch.bfloat16)
    qs[:, n - 1::n] = q
    os_ = torch.empty_like(qs)
    td.td_chunk_attention(rr.ctx.handle, td.make_chunks(agents, [p - n + 1 for p in last], [n] * 4),
                          rr.pool, 0, 2, qs.data_ptr(), nq, scale, 0, 0, os_.data_ptr(), None, rr.s)
    torch.cuda.synchronize()
    assert rr.get_error() == (0, 0)
    assert torch.allclose(os_[:, n - 1::n].float(), o32, rtol=2.0 ** -6, atol=2.0 ** -7)


def test_a_wait_that_runs_out_is_reported_and_the_context_recovers(td):
    """td_inject_attention_wait_fault makes every tile's barrier expect bytes that never come:
    the bounded waits run out, the error word says so and nothing faults; the next call on the
    context is right."""
    b = ck.Batch([300, 20], [50, 30], 1, 128, 16, seed=34)
    pool, q = b.rows(*b.pool_shape()), b.rows(1, b.T, 4, 128)
    ctx, pages = _ctx(td, b), td.make_paged(pool, b.bt_t)
    td.td_inject_attention_wait_fault(ctx.handle, 16)
    bit = 1 << td.TD_ERR_DEVICE_TIMEOUT
    _run_attention(td, b, pages, q, ctx=ctx, expect=(td.TD_ERR_DEVICE_TIMEOUT, bit))
    td.td_inject_attention_wait_fault(ctx.handle, 0)
    got = _run_attention(td, b, pages, q, ctx=ctx)
    want = ck.attend(b, pool[:, 0].double(), pool[:, 1].double(), q)
    _close(got, want, _weight_step(b, 4))


def test_batches_without_tokens_write_nothing(td):
    b = ck.Batch([3, 4], [0, 0], 2, 64, 16, seed=33)
    ctx = _ctx(td, b, 2)
    pool = torch.full(b.pool_shape(), 2.0, dtype=torch.bfloat16, device="cuda")
    codes = torch.full(b.pool_shape(), 3, dtype=torch.int8, device="cuda")
    sc = torch.full(b.pool_shape()[:-1], 0.5, device="cuda")
    for ch in (_chunks(td, b), td.make_chunks([], [], [])):
        td.td_chunk_attention(ctx.handle, ch, td.make_paged(pool, b.bt_t), 0, 1, None, 2, 0.1, 0, 0,
                              None, None, _stream())
        td.td_quantise_append(ctx.handle, ch, td.make_paged8(codes, sc, b.bt_t, "int8"), None, None,
                              0, 1, _stream())
        td.td_dequantise_read(ctx.handle, ch, td.make_paged8(codes, sc, b.bt_t, "int8"), 0, 1, None,
                              None, _stream())
    assert _errors(td, ctx) == (0, 0)
    assert bool((codes == 3).all()) and bool((sc == 0.5).all()) and bool((pool == 2.0).all())


# ------------------------------------------------- long chunks over 8-bit pages, unfolded first
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D,window,sinks", [(64, 0, 0), (128, 0, 0), (128, 210, 150), (64, 33, 3)])
def test_long_chunks_over_scales_of_any_kind(td, fmt, D, window, sinks):
    """Powers of two (which the unfolded values take in) up to some position, then scales of
    both signs, zeros and large ones; an unmapped page within sight of all tokens."""
    b = ck.Batch([400, 37, 900, 3], [150, 300, 2, 40], 2, D, 16, seed=41)
    val, s = ck.quantise(b.rows(*b.pool_shape()), fmt)
    codes, scale = ck.code_bytes(val, fmt).contiguous(), s.float().contiguous()
    if fmt == "e4m3":
        scale[:, 1] *= 2.0 ** -90                      # (still a power of two)
    pick = torch.randint(0, 6, scale.shape, generator=b.gen, device="cuda")
    odd = torch.zeros_like(scale, dtype=torch.bool)
    for x, first in ((0, 256), (1, 130)):
        pg, sl = b.place(x, np.arange(first, b.starts[x] + b.lens[x]))
        odd[:, :, pg, sl] = True
    other = torch.where(pick == 0, -0.7 * scale, torch.where(pick == 1, scale * 0, scale * 1.3))
    scale = torch.where(odd & (pick < 3), other, scale).contiguous()
    scale[:, 1] = torch.where(odd[:, 1] & (pick[:, 1] == 5), 2.0 ** 9, scale[:, 1])
    hole = int(b.bt[0, 24]), int(b.bt[1, 3])           # positions 384 and 48 on
    b.bt_t[0, 24] = b.bt_t[1, 3] = -1
    codes[:, :, list(hole)] = 0x7F
    scale[:, :, list(hole)] = math.nan
    q = b.rows(1, b.T, 8, D)
    hit = (td.TD_ERR_UNMAPPED_PAGE, 1 << td.TD_ERR_UNMAPPED_PAGE)
    got = _run_attention(td, b, td.make_paged8(codes, scale, b.bt_t, fmt), q, window, sinks, q8=True,
                         expect=hit)
    kv = torch.nan_to_num(ck.code_values(codes, fmt) * scale.double()[..., None])
    want = ck.attend(b, kv[:, 0], kv[:, 1], q, window, sinks)
    _close(got, want, 2.0 ** -8)
    again = _run_attention(td, b, td.make_paged8(codes, scale, b.bt_t, fmt), q, window, sinks,
                           q8=True, expect=hit)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def test_a_scale_that_is_not_finite_stays_with_the_rows_that_see_it(td):
    """K's or V's scale of a token in the middle of a long chunk is a NaN."""
    b = ck.Batch([150], [300], 2, 128, 16, seed=42)
    val, s = ck.quantise(b.rows(*b.pool_shape()), "e4m3")
    codes, scale = ck.code_bytes(val, "e4m3").contiguous(), s.float().contiguous()
    q = b.rows(1, b.T, 4, 128)
    clean, zc = _run_attention(td, b, td.make_paged8(codes, scale, b.bt_t, "e4m3"), q, q8=True)
    pg, sl = b.place(0, np.array([290]))
    for half in (0, 1):
        dirty_scale = scale.clone()
        dirty_scale[0, half, pg, sl, 1] = math.nan
        out, z = _run_attention(td, b, td.make_paged8(codes, dirty_scale, b.bt_t, "e4m3"), q, q8=True)
        # (a tile with such a scale applies its scales to the scores and weights instead: other
        # roundings, so the bounds rather than the same bits)
        kv = val * s[..., None]
        want = ck.attend(b, kv[:, 0], kv[:, 1], q)
        blind = torch.arange(300, device="cuda") < 140
        _close((out[:, blind], z[:, blind]), [t[:, blind] for t in want], 2.0 ** -8)
        _close((out[:, :, :2], z[:, :, :2]), [t[:, :, :2] for t in want], 2.0 ** -8)
        assert bool(torch.isnan(out[0, ~blind, 2:]).all())


def test_unfolded_copies_past_their_limit_take_several_launches(td):
    """Three sequences over 28 layers, whose copies together pass 2^30 bytes."""
    b = ck.Batch([4700, 3300, 4000], [300, 280, 290], 8, 128, 16, 28, seed=43)
    codes = torch.randint(-127, 128, b.pool_shape(), generator=b.gen, device="cuda",
                          dtype=torch.int8)
    scale = torch.rand(b.pool_shape()[:-1], generator=b.gen, device="cuda") * 0.01 + 0.001
    q = b.rows(28, b.T, 16, 128)
    got = _run_attention(td, b, td.make_paged8(codes, scale, b.bt_t, "int8"), q, q8=True)
    kv = codes.double() * scale.double()[..., None]
    _close(got, ck.attend(b, kv[:, 0], kv[:, 1], q), 2.0 ** -8)


def test_long_chunks_over_8bit_pages_in_a_captured_graph(td):
    """Unfolding, attention and join replayed over new pages and queries."""
    b = ck.Batch([2000, 90], [200, 150], 2, 128, 16, seed=44)
    q = b.rows(1, b.T, 6, 128)
    ctx = _ctx(td, b)
    val, s = ck.quantise(b.rows(*b.pool_shape()), "int8")
    codes, scale = ck.code_bytes(val, "int8").contiguous(), s.float().contiguous()
    pages = td.make_paged8(codes, scale, b.bt_t, "int8")
    _run_attention(td, b, pages, q, q8=True, ctx=ctx)
    out = torch.full(q.shape, math.nan, dtype=torch.bfloat16, device="cuda")
    z = torch.full(q.shape[:3], math.nan, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        td.td_chunk_attention_q8(ctx.handle, _chunks(td, b), pages, 0, 1, q.data_ptr(), 6, 0.09, 0,
                                 0, out.data_ptr(), z.data_ptr(), _stream())
    for _ in range(2):
        val, s = ck.quantise(b.rows(*b.pool_shape()), "int8")
        codes.copy_(ck.code_bytes(val, "int8"))
        scale.copy_(s.float())
        q.copy_(b.rows(1, b.T, 6, 128))
        graph.replay()
        kv = val * s[..., None]
        _close((out, z), ck.attend(b, kv[:, 0], kv[:, 1], q, scale=0.09), 2.0 ** -8)


def test_a_wait_that_runs_out_over_unfolded_pages(td):
    b = ck.Batch([300], [140], 1, 128, 16, seed=45)
    val, s = ck.quantise(b.rows(*b.pool_shape()), "e4m3")
    codes, scale = ck.code_bytes(val, "e4m3").contiguous(), s.float().contiguous()
    pages, q, ctx = td.make_paged8(codes, scale, b.bt_t, "e4m3"), b.rows(1, b.T, 4, 128), _ctx(td, b)
    td.td_inject_attention_wait_fault(ctx.handle, 64)
    _run_attention(td, b, pages, q, q8=True, ctx=ctx,
                   expect=(td.TD_ERR_DEVICE_TIMEOUT, 1 << td.TD_ERR_DEVICE_TIMEOUT))
    td.td_inject_attention_wait_fault(ctx.handle, 0)
    got = _run_attention(td, b, pages, q, q8=True, ctx=ctx)
    kv = val * s[..., None]
    _close(got, ck.attend(b, kv[:, 0], kv[:, 1], q), 2.0 ** -8)


# ------------------------------------------- more tiles than SMs: the last wave's tiles in parts
TAIL = ([4200, 3900, 3700], [1500, 1300, 160], 4, 8)     # (47 + 41 + 5) x 4 units


@pytest.mark.parametrize("D,fmt,window,sinks", [(128, "", 0, 0), (64, "", 0, 0),
                                                (128, "e4m3", 0, 0), (64, "int8", 2500, 4)])
def test_a_last_wave_in_parts(td, D, fmt, window, sinks):
    starts, lens, H, G = TAIL
    b = ck.Batch(starts, lens, H, D, 16, seed=51)
    pool, q = b.rows(*b.pool_shape()), b.rows(1, b.T, H * G, D)
    if fmt:
        val, s = ck.quantise(pool, fmt)
        kv = val * s[..., None]
        pages = td.make_paged8(ck.code_bytes(val, fmt).contiguous(), s.float().contiguous(), b.bt_t,
                               fmt)
    else:
        kv, pages = pool.double(), td.make_paged(pool, b.bt_t)
    got = _run_attention(td, b, pages, q, window, sinks, q8=bool(fmt))
    _close(got, ck.attend(b, kv[:, 0], kv[:, 1], q, window, sinks), 2.0 ** -8)
    again = _run_attention(td, b, pages, q, window, sinks, q8=bool(fmt))
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def test_a_last_wave_in_parts_with_a_nan_in_v(td):
    """In the part of a tile that some of its rows see and others do not."""
    starts, lens, H, G = TAIL
    b = ck.Batch(starts, lens, H, 128, 16, seed=52)
    pool, q = b.rows(*b.pool_shape()), b.rows(1, b.T, H * G, 128)
    want = ck.attend(b, pool[:, 0].double(), pool[:, 1].double(), q)
    at = starts[2] + 11
    pg, sl = b.place(2, np.array([at]))
    pool[0, 1, pg, sl, 1, 5] = math.nan
    out, z = _run_attention(td, b, td.make_paged(pool, b.bt_t), q)
    keep = torch.ones(out.shape, dtype=torch.bool, device="cuda")
    keep[0, b.T - lens[2] + 11:, G:2 * G, 5] = False
    assert bool(torch.isnan(out[~keep]).all())
    o = torch.where(keep, out, want[0].to(torch.bfloat16))
    _close((o, z), want, 2.0 ** -8)
