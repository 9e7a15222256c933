"""Operators over the paged KV cache, as a serving program calls them: new tokens' K/V written
into 8-bit pages and read back, and attention of a chunk of new tokens over bf16 or 8-bit
pages, over the whole context or a sliding window with the first tokens kept visible.

`run` computes a case in elementary torch operations, or, with `own` set, through the
library's entry points. A case's sequence lengths are drawn from its own "lens" number, so
that they are a part of the case; the tensors' values come from the seed.
"""
from __future__ import annotations

import math
import random

import torch

own = False

FORMATS = ("int8", "e4m3")
CODE_MAX = {"int8": 127.0, "e4m3": 448.0}
SCALE_MIN = 2.0 ** -100


# ---------------------------------------------------------------------------- the cases
def _case(name, op, layers, heads, dim, page, seqs, ctx, new, lens, group=0, fmt="", window=0,
          sinks=0):
    return dict(name=name, op=op, layers=layers, heads=heads, dim=dim, page=page, seqs=seqs,
                ctx_min=ctx[0], ctx_max=ctx[1], new_min=new[0], new_max=new[1], lens=lens,
                group=group, fmt=fmt, window=window, sinks=sinks)


def listed():
    return [
        # a decode step of a 10-agent round: one token an agent, every layer, 4 x 128 heads
        _case("write_step_int8", "write", 28, 4, 128, 16, 10, (3060, 6560), (1, 1), 1, fmt="int8"),
        # the agents' outputs after a round: ragged chunks of every layer
        _case("write_chunk_e4m3", "write", 28, 4, 128, 16, 10, (500, 4000), (300, 1100), 2,
              fmt="e4m3"),
        # two small layers read back, 2 x 64 heads, odd lengths and positions
        _case("read_small_int8", "read", 2, 2, 64, 24, 3, (5, 40), (17, 131), 3, fmt="int8"),
        # whole shared spans of a 10-agent round read back, 8 x 128 heads
        _case("read_span_e4m3", "read", 8, 8, 128, 32, 10, (1000, 8000), (5120, 5120), 4,
              fmt="e4m3"),
        # one token over a short context: the smallest call
        _case("token_small", "attend", 1, 2, 64, 16, 1, (33, 33), (1, 1), 5, group=3),
        # a decode step of one layer of the 10-agent round
        _case("token_round", "attend", 1, 4, 128, 16, 10, (3060, 6560), (1, 1), 6, group=7),
        # recomputed spans of uneven length over long contexts, 8 x 128 heads, 24-token pages
        _case("spans_ragged", "attend", 1, 8, 128, 24, 32, (6000, 13000), (1, 301), 7, group=5),
        # long prompt chunks over a long context
        _case("chunk_long", "attend", 1, 4, 128, 16, 2, (8192, 8192), (2048, 2048), 8, group=7),
        # one token of 64 agents, long contexts, a window with four tokens kept
        _case("token_window", "attend", 1, 4, 128, 16, 64, (8192, 24576), (1, 1), 9, group=7,
              window=1024, sinks=4),
        # a prompt chunk under a short window, 64-wide heads
        _case("chunk_window", "attend", 1, 8, 64, 16, 4, (1000, 9000), (1500, 4097), 10, group=8,
              window=1024, sinks=4),
        # one token of 64 agents over 8-bit pages
        _case("token_int8", "attend", 1, 4, 128, 16, 64, (8192, 24576), (1, 1), 11, group=7,
              fmt="int8"),
        # prompt chunks over 8-bit pages
        _case("chunk_e4m3", "attend", 1, 8, 128, 16, 4, (4096, 8192), (500, 700), 12, group=5,
              fmt="e4m3"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("write", "read", "attend", "attend", "attend"))
    heads, dim = rng.choice((1, 2, 3, 4, 8)), rng.choice((64, 128))
    page = rng.choice((8, 16, 16, 24, 32))
    lens = rng.randrange(1 << 30)
    if op != "attend":
        seqs, layers = _log_int(rng, 1, 64), _log_int(rng, 1, 28)
        most = max(1, min(5120, 160_000_000 // (seqs * layers * heads * dim * 2)))
        hi = _log_int(rng, 1, most)
        ctx = rng.randrange(0, 4000)
        c = _case("", op, layers, heads, dim, page, seqs, (ctx, ctx + rng.randrange(0, 4000)),
                  (rng.randint(1, hi), hi), lens, fmt=rng.choice(FORMATS))
    else:
        group = rng.choice((1, 2, 3, 5, 7, 8))
        seqs = _log_int(rng, 1, 64)
        # tokens a chunk: half of the draws single tokens or a few, half up to long prompts
        hi = 1 if rng.random() < 0.35 else _log_int(rng, 2, max(2, 4096 // seqs))
        most = min(24576, 200_000_000 // (seqs * hi * heads * group), 40_000_000 // (seqs * heads))
        c_hi = _log_int(rng, 1, max(2, most))
        window = rng.choice((0, 0, 0, 64, 1000, 4096))
        c = _case("", "attend", 1, heads, dim, page, seqs, (rng.randint(0, c_hi), c_hi),
                  (rng.randint(1, hi), hi), lens, group=group, fmt=rng.choice(("", "") + FORMATS),
                  window=window, sinks=rng.choice((0, 4, 7)) if window else 0)
    del c["name"]
    return c


def _lengths(c):
    """First position and token count of every sequence's chunk."""
    r = random.Random(c["lens"])
    start = [r.randint(c["ctx_min"], c["ctx_max"]) for _ in range(c["seqs"])]
    new = [r.randint(c["new_min"], c["new_max"]) for _ in range(c["seqs"])]
    return start, new


def _seen(c, start, u):
    """How many positions token u of a chunk sees, and how many of them are kept first tokens
    outside the window."""
    pos = start + u
    if not c["window"]:
        return pos + 1
    lo = max(0, pos - c["window"] + 1)
    return pos + 1 - lo + min(c["sinks"], lo)


def work(case):
    c = case
    start, new = _lengths(c)
    L, H, D, T = c["layers"], c["heads"], c["dim"], sum(new)
    if c["op"] != "attend":
        rows = L * 2 * T * H   # bf16 on one side, codes and a scale on the other
        return {"bytes": rows * (3 * D + 4), "flops": rows * D * 2}
    nq = H * c["group"]
    per_pos = 2 * H * (D + 4 if c["fmt"] else 2 * D)
    read = pairs = 0
    for s, n in zip(start, new):
        last = s + n - 1
        if not c["window"]:
            read += last + 1
        else:
            lo = max(0, s - c["window"] + 1)
            read += last + 1 - lo + min(c["sinks"], lo)
        pairs += sum(_seen(c, s, u) for u in range(n))
    return {"bytes": L * (read * per_pos + T * nq * (4 * D + 4)),
            "flops": L * pairs * nq * D * 4}


# ---------------------------------------------------------------------------- the inputs
def _power_of_two(k):
    """2^k, exactly (the device's exp2 and pow may be off by an ulp)."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _quantise(x, fmt):
    """Codes and scales of rows x[..., D]: float64, so that quotients next to a border fall on
    the right side of it."""
    x = x.double()
    top = x.abs().amax(-1, keepdim=True)
    if fmt == "int8":
        # the scale is a float32: the quotient by it is what is rounded
        s = (top / 127.0).float().double().clamp_min(SCALE_MIN)
        return torch.round(x / s).to(torch.int8), s.squeeze(-1).float()
    # the least power of two that brings the row's largest magnitude to 448 or less, 2^-100 at
    # least
    m, e = torch.frexp(top)            # top = m 2^e, m in [0.5, 1)
    k = e - 9 + (m > 0.875).to(e.dtype)
    s = torch.where(top > 0, _power_of_two(k), 0.0).clamp_min(SCALE_MIN)
    return (x / s).float().to(torch.float8_e4m3fn), s.squeeze(-1).float()


def prepare(case, seed):
    c = case
    start, new = _lengths(c)
    g = torch.Generator(device="cuda").manual_seed(seed)
    L, H, D, P, n, T = c["layers"], c["heads"], c["dim"], c["page"], c["seqs"], sum(new)
    pages = [-(-(s + t) // P) for s, t in zip(start, new)]
    width, total = max(pages), sum(pages)
    order = torch.randperm(total, generator=g, device="cuda").int()
    bt = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, k in enumerate(pages):
        bt[i, :k] = order[at:at + k]
        at += k
    st = dict(case=c, start=start, new=new, bt=bt, T=T, pages=total)
    # sequence and position of every new token, in chunk order
    cnt = torch.tensor(new, device="cuda")
    beg = torch.tensor(start, device="cuda")
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), cnt)
    idx = torch.arange(T, device="cuda") - torch.repeat_interleave(cnt.cumsum(0) - cnt, cnt)
    st.update(cnt=cnt, beg=beg, seq=seq, idx=idx)

    def rows(shape):
        out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        flat = out.view(-1)
        for i in range(0, flat.numel(), 1 << 28):
            k = min(1 << 28, flat.numel() - i)
            flat[i:i + k] = torch.randn(k, generator=g, device="cuda").to(torch.bfloat16)
        return out

    code_t = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}.get(c["fmt"])
    shape = (L, 2, total, P, H, D)
    if c["op"] == "write":
        st["k"], st["v"] = rows((L, T, H, D)), rows((L, T, H, D))
        st["codes"] = torch.zeros(shape, dtype=torch.int8, device="cuda").view(code_t)
        st["scale"] = torch.zeros(shape[:-1], dtype=torch.float32, device="cuda")
    elif c["fmt"]:
        st["codes"] = torch.empty(shape, dtype=torch.int8, device="cuda").view(code_t)
        st["scale"] = torch.empty(shape[:-1], dtype=torch.float32, device="cuda")
        for l in range(L):
            for kv in range(2):
                st["codes"][l, kv], st["scale"][l, kv] = _quantise(rows(shape[2:]), c["fmt"])
    else:
        st["pool"] = rows(shape)
    if c["op"] == "read":
        st["k_out"] = torch.empty((L, T, H, D), dtype=torch.bfloat16, device="cuda")
        st["v_out"] = torch.empty_like(st["k_out"])
    if c["op"] == "attend":
        nq = H * c["group"]
        st["q"] = rows((L, T, nq, D))
        st["out"] = torch.empty((L, T, nq, D), dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.empty((L, T, nq), dtype=torch.float32, device="cuda")
    if own:
        from collective_kv_cache_gb300 import td
        st["ctx"] = td.Context(td.td_shape(L, H, D, P, 16, 1e6), n, 1, 1)
        st["chunks"] = td.make_chunks(list(range(n)), start, new)
        if c["fmt"]:
            st["paged"] = td.make_paged8(st["codes"], st["scale"], bt, c["fmt"])
        else:
            st["paged"] = td.make_paged(st["pool"], bt)
    return st


# ---------------------------------------------------------------------------- one pass
def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    return (_write if op == "write" else _read if op == "read" else _attend)(state)


def _run_own(st):
    from collective_kv_cache_gb300 import td
    c = st["case"]
    stream = torch.cuda.current_stream().cuda_stream
    h, L, ch, pg = st["ctx"].handle, c["layers"], st["chunks"], st["paged"]
    if c["op"] == "write":
        td.td_quantise_append(h, ch, pg, st["k"].data_ptr(), st["v"].data_ptr(), 0, L, stream)
        return st["codes"], st["scale"]
    if c["op"] == "read":
        td.td_dequantise_read(h, ch, pg, 0, L, st["k_out"].data_ptr(), st["v_out"].data_ptr(),
                              stream)
        return st["k_out"], st["v_out"]
    call = td.td_chunk_attention_q8 if c["fmt"] else td.td_chunk_attention
    call(h, ch, pg, 0, L, st["q"].data_ptr(), c["heads"] * c["group"], 1.0 / math.sqrt(c["dim"]),
         c["window"], c["sinks"], st["out"].data_ptr(), st["lse"].data_ptr(), stream)
    return st["out"], st["lse"]


def _places(st):
    """Page and slot of every new token."""
    P = st["case"]["page"]
    pos = st["beg"][st["seq"]] + st["idx"]
    return st["bt"][st["seq"], pos // P].long(), pos % P


def _write(st):
    c = st["case"]
    page, slot = _places(st)
    kc, ks = _quantise(st["k"], c["fmt"])
    st["codes"].view(torch.int8)[:, 0, page, slot] = kc.view(torch.int8)
    st["scale"][:, 0, page, slot] = ks
    del kc, ks
    vc, vs = _quantise(st["v"], c["fmt"])
    st["codes"].view(torch.int8)[:, 1, page, slot] = vc.view(torch.int8)
    st["scale"][:, 1, page, slot] = vs
    return st["codes"], st["scale"]


def _read(st):
    page, slot = _places(st)
    codes = st["codes"].view(torch.int8)[:, :, page, slot].view(st["codes"].dtype)
    rows = (codes.float() * st["scale"][:, :, page, slot].unsqueeze(-1)).to(torch.bfloat16)
    return rows[:, 0].contiguous(), rows[:, 1].contiguous()


def _visible(c, pos_q, pos_k):
    ok = pos_k <= pos_q
    if c["window"]:
        ok = ok & ((pos_k > pos_q - c["window"]) | (pos_k < c["sinks"]))
    return ok


def _attend(st):
    """Chunks and contexts padded to the longest, all heads in one product, in float32."""
    c = st["case"]
    L, H, D, P, G, n = c["layers"], c["heads"], c["dim"], c["page"], c["group"], c["seqs"]
    N, C = max(st["new"]), max(s + t for s, t in zip(st["start"], st["new"]))
    pos = torch.arange(C, device="cuda")
    page = st["bt"][:, pos // P].long().clamp_min(0)                     # [n][C]
    if c["fmt"]:
        kv = (st["codes"].view(torch.int8)[:, :, page, pos % P].view(st["codes"].dtype).float()
              * st["scale"][:, :, page, pos % P].unsqueeze(-1))
    else:
        kv = st["pool"][:, :, page, pos % P].float()                     # [L][2][n][C][H][D]
    kv = torch.where((pos < (st["beg"] + st["cnt"])[:, None])[:, :, None, None], kv, 0.0)
    k, v = kv[:, 0].permute(0, 1, 3, 4, 2), kv[:, 1].permute(0, 1, 3, 2, 4)
    q = torch.zeros((L, n, N, H, G, D), dtype=torch.float32, device="cuda")
    q[:, st["seq"], st["idx"]] = st["q"].float().view(L, -1, H, G, D)
    q = q.permute(0, 1, 3, 2, 4, 5).reshape(L, n, H, N * G, D)
    s = torch.matmul(q, k) * (1.0 / math.sqrt(D))                        # [L][n][H][N*G][C]
    pos_q = (st["beg"][:, None] + torch.arange(N, device="cuda")).repeat_interleave(G, 1)
    s = s.masked_fill_(~_visible(c, pos_q[:, :, None], pos)[:, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    s = s.sub_(top).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s, v) / total
    lse = (top + total.log()).squeeze(-1)
    o = o.view(L, n, H, N, G, D).permute(0, 1, 3, 2, 4, 5)[:, st["seq"], st["idx"]]
    lse = lse.view(L, n, H, N, G).permute(0, 1, 3, 2, 4)[:, st["seq"], st["idx"]]
    return o.reshape(L, -1, H * G, D).to(torch.bfloat16), lse.reshape(L, -1, H * G)


# ---------------------------------------------------------------------------- in 64 bits
def _exact_codes(x, fmt):
    x = x.to(torch.float64)
    top = x.abs().max(dim=-1).values
    if fmt == "int8":
        s = torch.maximum((top / 127).to(torch.float32).to(torch.float64),
                          torch.tensor(SCALE_MIN, dtype=torch.float64, device=x.device))
        return torch.round(x / s[..., None]), s
    # the powers of two that are candidates, as a table: the first with amax / s <= 448
    table = torch.tensor([2.0 ** e for e in range(-100, 122)], dtype=torch.float64,
                         device=x.device)
    s = table[torch.searchsorted(table, top / 448.0)]
    y = x / s[..., None]
    # e4m3: three fraction bits, least exponent -6; round half to even on that grid
    steps = torch.tensor([2.0 ** e for e in range(-6, 10)], dtype=torch.float64, device=x.device)
    step = steps[torch.searchsorted(steps, y.abs(), right=True).clamp_(min=1) - 1] / 8.0
    return torch.round(y / step) * step, s


def exact(case, seed):
    st = _prepare_plain(case, seed)
    c = case
    L, H, D, P = c["layers"], c["heads"], c["dim"], c["page"]
    bt, at = st["bt"].tolist(), 0
    if c["op"] == "write":
        codes = torch.zeros(st["codes"].shape, dtype=torch.float32, device="cuda")
        scale = torch.zeros(st["scale"].shape, dtype=torch.float64, device="cuda")
        for i, (s, t) in enumerate(zip(st["start"], st["new"])):
            where = [(bt[i][p // P], p % P) for p in range(s, s + t)]
            pg = torch.tensor([w[0] for w in where], device="cuda")
            sl = torch.tensor([w[1] for w in where], device="cuda")
            for kv, x in enumerate((st["k"], st["v"])):
                for l in range(L):
                    y, sc = _exact_codes(x[l, at:at + t], c["fmt"])
                    codes[l, kv, pg, sl], scale[l, kv, pg, sl] = y.float(), sc
            at += t
        return (None if c["fmt"] == "int8" else codes), scale
    outs = []
    for i, (s, t) in enumerate(zip(st["start"], st["new"])):
        p = torch.arange(0 if c["op"] == "attend" else s, s + t, device="cuda")
        pg, sl = st["bt"][i].long()[torch.div(p, P, rounding_mode="floor")], p % P
        if c["op"] == "read":
            rows = (st["codes"].view(torch.int8)[:, :, pg, sl].view(st["codes"].dtype).double()
                    * st["scale"][:, :, pg, sl].double()[..., None])
            outs.append((rows[:, 0].float(), rows[:, 1].float()))
            continue
        o = torch.empty((L, t, H * c["group"], D), dtype=torch.float64, device="cuda")
        z = torch.empty((L, t, H * c["group"]), dtype=torch.float64, device="cuda")
        pq = torch.arange(s, s + t, device="cuda")[:, None]
        dark = p[None, :] > pq
        if c["window"]:
            dark |= (p[None, :] <= pq - c["window"]) & (p[None, :] >= c["sinks"])
        for l in range(L):
            for h in range(H):
                if c["fmt"]:
                    k, v = (st["codes"].view(torch.int8)[l, kv, pg, sl, h]
                            .view(st["codes"].dtype).double()
                            * st["scale"][l, kv, pg, sl, h].double()[:, None] for kv in (0, 1))
                else:
                    k, v = (st["pool"][l, kv, pg, sl, h].double() for kv in (0, 1))
                for j in range(h * c["group"], (h + 1) * c["group"]):
                    x = st["q"][l, at:at + t, j].double() @ k.T / math.sqrt(D)
                    x = x.masked_fill(dark, -math.inf)
                    z[l, :, j] = torch.logsumexp(x, -1)
                    o[l, :, j] = torch.exp(x - z[l, :, j, None]) @ v
        at += t
        outs.append((o, z))
    return tuple(torch.cat(x, dim=1) for x in zip(*outs))


def _prepare_plain(case, seed):
    global own
    kept, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = kept
