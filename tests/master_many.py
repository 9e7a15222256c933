"""td_pick_master of many agents, in a process where nothing has asked for more shared memory before:
sizes at which the kernel's static shared memory makes the difference. For tests/test_gpu_edges_many.py."""
import numpy as np
import torch

from collective_kv_cache_gb300 import td


def check(N, S, k, seed):
    nb = -(-S // 16)
    r = np.random.RandomState(seed)
    sel = np.sort(np.stack([r.choice(S, k, replace=False) for _ in range(N)]), 1).astype(np.int32)
    has = np.zeros((N, nb), np.float64)
    has[np.arange(N)[:, None], sel // 16] = 1
    n = has.sum(1)
    union = n[:, None] + n[None, :] - has @ has.T        # blocks of either of two agents
    want = union.sum(1) - n                              # (an agent with itself does not count)
    ctx = td.Context(td.td_shape(1, 1, 64, 16, 16, 1e6), N, 1, S)
    rnd = td.make_round([S], [0] * N, [[0]] * N)
    sel_t = torch.from_numpy(sel).cuda()
    cost = torch.full((N,), -1, dtype=torch.int64, device="cuda")
    master = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    m = td.td_pick_master(ctx.handle, rnd, sel_t.data_ptr(), k, cost.data_ptr(), master.data_ptr())
    assert cost.cpu().numpy().tolist() == want.astype(np.int64).tolist(), (N, S)
    assert m == int(master) == int(want.argmin()), (N, S)
    assert td.td_get_error(ctx.handle, 0) == (0, 0)


if __name__ == "__main__":
    # masks and costs: 48 KiB less 8, and just 48 KiB, of 1, 4 and 6 words a mask; then less and more
    for N, S in ((4095, 500), (4096, 512), (2048, 2000), (1536, 2880), (100, 700), (4096, 800)):
        check(N, S, 20, N)
    print("ok")
