"""Decode attention over a round's pages in captured graphs: its scratch stays where a graph
has it, and a capture never allocates."""
from __future__ import annotations

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def test_a_graph_outlives_larger_calls_and_a_capture_does_not_allocate():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from collective_kv_cache_gb300 import build
    build.build()
    import oracle
    from collective_kv_cache_gb300 import runner as R
    from collective_kv_cache_gb300 import synth, td
    from tests import roundkit as rk
    cfg = synth.RoundConfig(name="mini", n_agents=6, n_layers=2, n_kv_heads=2, head_dim=128,
                            page_size=16, block_lens=(20, 37, 16, 9), hist_range=(3, 45),
                            check_layer=1, recompute_pct=15, perturb_mode="runs",
                            perturb_frac=(0.10, 0.20), seed=101)
    ch = rk.run_oracle_chain(rk.make_inputs(cfg, map_history=True), restore=False)
    rnd = ch.rnd
    pool = oracle.new_pool(cfg, rnd.num_pages, fill=0x3F80)
    rk.fill_history(cfg, rnd, pool)
    assert oracle.get().fused_restore(cfg, ch.desc, ch.master, ch.store, np.arange(6), pool,
                                      rnd.num_pages, rnd.block_table, frame=0) == 0
    rr = R.RoundRunner(cfg, rnd.block_len, rnd.hist_len, rnd.perm, rnd.block_table, rnd.num_pages)
    rr.pool_t.copy_(R.to_device_bf16(pool, "cuda").reshape(rr.pool_t.shape))
    nq, agents = 6, [2, 0, 5, 3, 1, 4]
    q = torch.randn((2, 6, nq, 128), device="cuda").to(torch.bfloat16)

    q1 = q[:, :1].contiguous()

    def call(n, out, stream, check=True):
        return td.td_paged_attention(rr.ctx.handle, rr.round, rr.pool, agents[:n], 0, 2,
                                     (q if n == 6 else q1).data_ptr(), nq, 1.0 / math.sqrt(128),
                                     out.data_ptr(), None, stream, check=check)

    small = torch.zeros((2, 1, nq, 128), device="cuda")
    large = torch.zeros((2, 6, nq, 128), device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    call(1, small, side.cuda_stream)
    side.synchronize()
    want = small.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        call(1, small, side.cuda_stream)
    # the larger call in a capture is refused, and the capture goes on
    g2 = torch.cuda.CUDAGraph()
    x = torch.zeros(4, device="cuda")
    with torch.cuda.graph(g2, stream=side):
        x += 1
        status = call(6, large, side.cuda_stream, check=False)
    assert status == td.TD_ERR_INVALID_ARG
    # outside it grows the scratch; the graph's buffer stays
    call(6, large, side.cuda_stream)
    side.synchronize()
    filler = torch.full((1 << 20,), math.nan, device="cuda")   # what a freed buffer may become
    small.zero_()
    g.replay()
    g2.replay()
    torch.cuda.synchronize()
    assert torch.equal(small, want) and bool(torch.isnan(filler).all())
    assert torch.equal(large[:, :1], want)
    assert rr.get_error() == (0, 0)
