"""Inputs and float64 references for the operators over chunks of new tokens: 8-bit pages
written and read back, attention of the chunks over bf16 or 8-bit pages."""
from __future__ import annotations

import math

import numpy as np
import torch

NAN16 = 0x7FC0


class Batch:
    """Chunks over a paged cache: a block table with scattered pages, spare pages left over."""

    def __init__(self, starts, lens, H, D, P, L=1, agents=None, n_agents=None, seed=0, spare=3,
                 device="cuda"):
        self.starts, self.lens = list(starts), list(lens)
        self.agents = list(range(len(self.lens))) if agents is None else list(agents)
        self.n_agents = n_agents or max(self.agents, default=0) + 1
        self.H, self.D, self.P, self.L, self.T = H, D, P, L, sum(self.lens)
        rng = np.random.RandomState(seed)
        need = [0] * self.n_agents
        for a, s, t in zip(self.agents, self.starts, self.lens):
            need[a] = max(need[a], -(-(s + t) // P))
        self.width = max(max(need), 1) + 1
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages)
        bt = np.full((self.n_agents, self.width), -1, np.int32)
        at = 0
        for a, k in enumerate(need):
            bt[a, :k] = order[at:at + k]
            at += k
        self.bt = bt
        self.device = device
        self.bt_t = torch.from_numpy(bt).to(device)
        self.gen = torch.Generator(device=device).manual_seed(seed + 1)

    def rows(self, *shape, scale=1.0):
        x = torch.randn(shape, generator=self.gen, device=self.device) * scale
        return x.to(torch.bfloat16)

    def pool_shape(self):
        return (self.L, 2, self.pages, self.P, self.H, self.D)

    def place(self, x, positions):
        """Pages and slots of positions of chunk x's agent."""
        p = torch.as_tensor(positions, device=self.device)
        row = self.bt_t[self.agents[x]].long()
        return row[torch.div(p, self.P, rounding_mode="floor")], p % self.P

    def chunk_rows(self, x):
        r0 = sum(self.lens[:x])
        return slice(r0, r0 + self.lens[x])


def power_of_two(k):
    """2^k, exactly (the device's exp2 and pow may be off by an ulp)."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def e4m3_grid(y):
    """y rounded to the e4m3 grid, ties to even (|y| <= 448), in float64."""
    e = torch.frexp(y.abs().clamp_min(2.0 ** -6))[1] - 1
    step = power_of_two(e - 3)
    return torch.round(y / step) * step


def quantise(x, fmt):
    """(values of the codes, scales), float64, of finite rows x[..., D]."""
    x = x.double()
    top = x.abs().amax(-1)
    low = torch.full_like(top, 2.0 ** -100)
    if fmt == "int8":
        s = torch.maximum((top / 127.0).float().double(), low)
        return torch.round(x / s[..., None]), s
    m, e = torch.frexp(top)
    k = e - 9 + (m > 0.875).to(e.dtype)
    s = torch.where(top > 0, power_of_two(k), low)
    s = torch.maximum(s, low)
    return e4m3_grid(x / s[..., None]), s


def code_values(codes, fmt):
    """Bytes (int8 tensor) -> values."""
    return codes.double() if fmt == "int8" else codes.view(torch.float8_e4m3fn).double()


def code_bytes(values, fmt):
    return values.to(torch.int8) if fmt == "int8" else (
        values.float().to(torch.float8_e4m3fn).view(torch.int8))


def attend(b: Batch, K, V, q, window=0, sinks=0, scale=None, mapped=None):
    """K, V: float64 [L][2 halves gone: pages][P][H][D] values of the pages; q bf16
    [L][T][nq][D]. Returns out, lse, sum_p softmax |v| and scale |q| max |k|, float64."""
    nq = q.shape[2]
    G, D = nq // b.H, b.D
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    mag = torch.zeros_like(out)
    lse = torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device=q.device)
    dot = torch.zeros_like(lse)
    for x, (s, t) in enumerate(zip(b.starts, b.lens)):
        if t == 0:
            continue
        p = torch.arange(s + t, device=q.device)
        row = b.bt_t[b.agents[x]].long()[torch.div(p, b.P, rounding_mode="floor")]
        pq = torch.arange(s, s + t, device=q.device)[:, None]
        seen = p <= pq
        if window:
            seen = seen & ((p > pq - window) | (p < sinks))
        seen = seen & (row >= 0)
        k, v = (z[:, row.clamp_min(0), p % b.P] for z in (K, V))     # [L][C][H][D]
        rs = b.chunk_rows(x)
        for l in range(b.L):
            for h in range(b.H):
                kk, vv = k[l, :, h], v[l, :, h]
                any_seen = seen.any(0)
                kk = torch.where(any_seen[:, None], kk, 0.0)
                for g in range(h * G, (h + 1) * G):
                    qq = q[l, rs, g].double()
                    sc = (qq @ kk.T * scale).masked_fill(~seen, -math.inf)
                    z = torch.logsumexp(sc, -1)
                    w = torch.exp(sc - z[:, None])
                    w = torch.where(seen & torch.isfinite(z)[:, None], w, 0.0)
                    # 0 * NaN must not count: sum over the seen positions only
                    bad = ~torch.isfinite(vv)
                    o = w @ torch.where(bad, 0.0, vv)
                    if bad.any():
                        hit = seen.double() @ bad.double() > 0
                        o = torch.where(hit, math.nan, o)
                    out[l, rs, g] = o
                    mag[l, rs, g] = w @ torch.where(bad, 0.0, vv).abs()
                    lse[l, rs, g] = z
                    dot[l, rs, g] = scale * qq.norm(dim=-1) * kk.nan_to_num(0.0).norm(dim=-1).max()
    return out, lse, mag, dot


def bounds(out, mag, dot, weight_step):
    """Elementwise bounds of the output and the log-sum-exp.

    A score is a sum of D <= 128 exact products added in float32, on tensor cores that may cut
    instead of round: off by at most 128 * 2^-23 of sum |q_d k_d| <= |q| |k|, so by delta =
    2^-16 scale |q| |k|, which covers the float32 scalings too (a few 2^-24). A weight moves by
    2 delta (its own score and the sum's), by the exponential's 2^-21 and the sums' rounding
    (2^-14: at most a thousand float32 additions one after the other), and by its own rounding
    before the second product, `weight_step`: half a step of bf16, 2^-8, or two bf16 parts,
    2^-16. All of these are relative to sum_p w_p |v_p|. The output is rounded to bf16: 2^-8
    of its value."""
    delta = dot * 2.0 ** -16
    rel = 2 * delta[..., None] + 2.0 ** -14 + weight_step
    return mag * rel + out.abs() * 2.0 ** -8 + 1e-30, delta + 2.0 ** -14
