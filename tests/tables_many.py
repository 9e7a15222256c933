"""td_update_tables for many requests, in a process where nothing has asked for more shared memory
before: rising sizes around those where the kernel's static shared memory makes the difference, then two
contexts' calls of different sizes from two threads. For tests/test_gpu_cache4_limits.py."""
import sys
import threading

import torch

from collective_kv_cache_gb300 import td


class Calls:
    def __init__(self, n, rows):
        self.n = n
        self.ctx = td.Context(td.td_shape(1, 1, 64, 16, 16, 1e6), rows, 1, 1)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.len, self.add = torch.zeros(n, **i32), torch.ones(n, **i32)
        self.bt = torch.full((rows, 1), -1, **i32)
        self.pages, self.count = torch.arange(n, **i32), torch.full((1,), n, **i32)
        self.start, self.slots = torch.zeros(n + 1, **i32), torch.zeros(n, **i32)
        self.req = td.make_requests(self.len)
        self.list = td.make_page_list(self.pages, self.count, n)

    def update(self, stream=0):
        td.td_update_tables(self.ctx.handle, self.req, self.add.data_ptr(), self.bt.data_ptr(), 1, self.list,
                            self.start.data_ptr(), self.slots.data_ptr(), self.n, stream)

    def check(self, held):
        n = self.n
        want = torch.arange(n - 1, -1, -1, device="cuda", dtype=torch.int32)
        assert torch.equal(self.slots, want * 16 + held - 1) and torch.equal(self.bt[:n, 0], want)
        assert bool((self.len == held).all()) and int(self.count) == 0
        assert td.td_get_error(self.ctx.handle, 0) == (0, 0)


def sizes():
    for n, rows in ([(n, 4096) for n in range(3029, 3042)] + [(n, n) for n in range(3038, 3050)] +
                    [(4096, 4096), (3040, 3040), (5, 4096)]):
        c = Calls(n, rows)
        try:
            c.update()
        except Exception as e:
            sys.exit(f"{n} requests of {rows} rows: {e}")
        c.check(1)


def threads():
    calls = [Calls(n, 4096) for n in (4096, 3300)]
    torch.cuda.synchronize()
    failed = []

    def run(c, stream):
        try:
            for _ in range(16):
                c.update(stream)
        except Exception as e:
            failed.append(e)

    streams = [torch.cuda.Stream() for _ in calls]
    for turn in range(20):
        for c in calls:
            c.add.fill_(1 if turn == 0 else 0)
        torch.cuda.synchronize()
        if turn == 0:
            for c in calls:
                c.update()
                c.check(1)
            continue
        t = [threading.Thread(target=run, args=(c, s.cuda_stream)) for c, s in zip(calls, streams)]
        for x in t:
            x.start()
        for x in t:
            x.join()
    torch.cuda.synchronize()
    if failed:
        sys.exit(f"{len(failed)} calls of two threads: {failed[0]}")
    for c in calls:
        assert bool((c.len == 1).all()) and td.td_get_error(c.ctx.handle, 0) == (0, 0)


if __name__ == "__main__":
    {"sizes": sizes, "threads": threads}[sys.argv[1]]()
    print("ok")
