"""Small ragged batches on a paged pool, and 64-bit formulas of the attention-side operators."""
from __future__ import annotations

import math

import numpy as np
import torch

import paged_kv_cache_lmkv_gb300 as pkg

DEV = torch.device("cuda:0")
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


class Batch:
    """Requests of new[r] new and kv[r] cached tokens (the new ones last) in a pool
    of shuffled pages, behind a shared prefix.  Page slots that hold no token
    are NaN."""

    def __init__(self, new, kv, heads, kv_heads, dim, dtype, prefix=0, page=16, seed=0, extra_rows=0, spread=1.5,
                 device=DEV, layers=2, layer=1):
        g = torch.Generator().manual_seed(seed)
        self.new, self.kv, self.prefix, self.page = list(new), list(kv), prefix, page
        self.heads, self.kv_heads, self.dim, self.dtype = heads, kv_heads, dim, dtype
        self.group = heads // kv_heads
        self.layer = layer
        need = [-(-n // page) for n in self.kv] + [-(-prefix // page)]
        total = sum(need)
        self.num_blocks = total + 3
        ids = torch.randperm(self.num_blocks, generator=g)
        cols = max(1, max(need[:-1], default=1)) + 1
        self.table = torch.full((len(self.kv), cols), -1, dtype=torch.int32)
        at = 0
        for r, n in enumerate(need[:-1]):
            self.table[r, :n] = ids[at:at + n]
            at += n
        self.prefix_table = torch.full((need[-1] + 1,), -1, dtype=torch.int32)
        self.prefix_table[:need[-1]] = ids[at:at + need[-1]]
        row = kv_heads * dim
        pool = torch.full((layers, 2, self.num_blocks, page, row), float("nan"))
        flat = pool[layer].view(2, -1, row)
        for slots in [self.slots(r) for r in range(len(self.kv))] + [self.prefix_slots()]:
            flat[:, slots] = torch.randn((2, len(slots), row), generator=g)
        self.pool_cpu = pool.to(dtype)
        self.q_start = torch.tensor(np.concatenate([[0], np.cumsum(self.new)]), dtype=torch.int32)
        self.kv_len = torch.tensor(self.kv, dtype=torch.int32)
        self.tokens = int(self.q_start[-1]) + extra_rows
        self.q_cpu = (torch.randn((self.tokens, heads, dim), generator=g) * spread).to(dtype)
        self.scale = 1.0 / math.sqrt(dim)
        self.device = device
        if device is not None:
            self.pool = pkg.Pool(list(self.pool_cpu.to(device)), kv_heads, dim)
            for n in ("table", "prefix_table", "q_start", "kv_len"):
                setattr(self, n + "_d", getattr(self, n).to(device))
            self.q = self.q_cpu.to(device)
            self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def _slots(self, table, n):
        j = torch.arange(n)
        return (table.long()[j // self.page] * self.page + j % self.page) if n else j

    def slots(self, r):
        return self._slots(self.table[r], self.kv[r])

    def prefix_slots(self):
        return self._slots(self.prefix_table, self.prefix)

    def rows64(self, slots, h, kv):
        d = self.dim
        return self.pool_cpu[self.layer, kv].view(-1, self.kv_heads * d)[slots, h * d:(h + 1) * d].double()

    def visible(self, r):
        """[new, kv]: which own tokens each new token sees."""
        n, m = self.new[r], self.kv[r]
        return torch.arange(m)[None] <= (m - n + torch.arange(n))[:, None]

    def attend(self, hide=None):
        """(out, lse, tolerance of out, of lse) in 64 bits; hide(r or None, tokens) -> bool mask of unseen."""
        t, hq, d = self.tokens, self.heads, self.dim
        out = torch.zeros((t, hq, d), dtype=torch.float64)
        lse = torch.full((t, hq), -math.inf, dtype=torch.float64)
        tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
        step, tiny = HALF_STEP[self.dtype], TINY[self.dtype]
        ps = self.prefix_slots()
        for r in range(len(self.new)):
            lo, n = int(self.q_start[r]), self.new[r]
            if n == 0:
                continue
            own = self.slots(r)
            seen = torch.cat((torch.ones((n, self.prefix), dtype=torch.bool), self.visible(r)), 1)
            if hide is not None:
                seen = seen & ~torch.cat((hide(None, self.prefix), hide(r, self.kv[r])))[None]
            for h in range(self.kv_heads):
                k = torch.cat((self.rows64(ps, h, 0), self.rows64(own, h, 0)))
                v = torch.cat((self.rows64(ps, h, 1), self.rows64(own, h, 1)))
                for a in range(h * self.group, (h + 1) * self.group):
                    q = self.q_cpu[lo:lo + n, a].double()
                    if k.shape[0] == 0:
                        continue
                    x = (q @ k.T * self.scale).masked_fill(~seen, -math.inf)
                    top = x.amax(1, keepdim=True).clamp(min=-1e300)
                    w = torch.exp(x - top)
                    total = w.sum(1, keepdim=True)
                    some = total[:, 0] > 0
                    p = torch.where(total > 0, w / total, 0.0)
                    o = p @ torch.where(seen.any(0)[:, None], v, 0.0)
                    out[lo:lo + n, a] = o
                    lse[lo:lo + n, a] = torch.where(some, (top + total.log())[:, 0], -math.inf)
                    # A product of d terms in fp32, in any order, is off by at most d 2^-23 of the
                    # sum of magnitudes (truncating adders included), an fp32 sum of n weights or of n weighted values by
                    # (n + 16) 2^-23 likewise, 2^x by 2^-22; the weights round to the type by half a step (fp16
                    # weights below 2^-14 by 2^-25 of the largest), the result by half a step.
                    keys = k.shape[0]
                    dx = (d + 8) * 2.0 ** -23 * (q.abs() @ k.abs().T).amax(1, keepdim=True) * abs(self.scale)
                    mag = p @ torch.where(seen.any(0)[:, None], v.abs(), 0.0)
                    vmax = torch.where(seen.any(0)[:, None], v.abs(), 0.0).amax()
                    f32 = 2 * dx + (keys + 16) * 2.0 ** -23 + 2.0 ** -21
                    tol_o[lo:lo + n, a] = (1.01 * step + f32) * mag + step * 1.01 * o.abs() + tiny + \
                        (keys * 2.0 ** -25 * vmax if self.dtype == torch.float16 else 0.0)
                    tol_l[lo:lo + n, a] = (dx[:, 0] + (keys + 16) * 2.0 ** -23 +
                                           2.0 ** -21 * (1 + lse[lo:lo + n, a].abs().nan_to_num(posinf=0.0)))
        return out, lse, tol_o, tol_l

    def weigh(self, lse, scores, decay):
        """(scores_out, tolerance) in 64 bits."""
        out = scores.double().clone()
        tol = torch.zeros_like(out)
        for r in range(len(self.new)):
            lo, n, m = int(self.q_start[r]), self.new[r], self.kv[r]
            own = self.slots(r)
            for h in range(self.kv_heads):
                total = torch.zeros(m, dtype=torch.float64)
                bound = torch.zeros(m, dtype=torch.float64)
                k = self.rows64(own, h, 0)
                for a in range(h * self.group, (h + 1) * self.group):
                    if n == 0 or m == 0:
                        continue
                    q = self.q_cpu[lo:lo + n, a].double()
                    e = lse[lo:lo + n, a].double()
                    x = q @ k.T * self.scale - e[:, None]
                    w = torch.where(self.visible(r) & (e > -math.inf)[:, None], torch.exp(x), 0.0)
                    dx = (self.dim + 8) * 2.0 ** -23 * (q.abs() @ k.abs().T) * abs(self.scale)
                    # x itself is rounded: 3 roundings of numbers up to |scale q.k| + |lse|
                    near = 4 * 2.0 ** -24 * 1.45 * (x.abs() + 2 * e[:, None].abs().nan_to_num(posinf=0.0))
                    total += w.sum(0)
                    bound += torch.where(w > 0, w * (dx + near + 2.0 ** -21), 0.0).sum(0)
                old = scores[r, h, :m].double()
                out[r, h, :m] = (decay * old if decay else 0.0) + total
                tol[r, h, :m] = bound + (n * self.group + 8) * 2.0 ** -23 * out[r, h, :m].abs() + 2.0 ** -140
        return out, tol


def within(got, want, tol, what=""):
    got = got.detach().double().cpu()
    same = (got == want) | (got.isnan() & want.isnan())
    off = torch.where(same, 0.0, (got - want).abs())
    bad = ~(off <= tol) & ~same
    if bool(bad.any()):
        i = tuple(int(x[0]) for x in bad.nonzero(as_tuple=True))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {float(got[i])} for "
                             f"{float(want[i])}, tolerance {float(tol[i])}")


def rotate64(x, pos, inv_freq, interleaved, magnitude=1.0):
    """x [tokens, heads, d] (64 bits) at positions pos [tokens]: (turned, |a| + |b| of each pair's element)."""
    # fractions of a turn from whole-number arithmetic: exact for any position
    frac = torch.empty((len(pos), len(inv_freq)), dtype=torch.float64)
    scaled = [int(round(float(f) / (2 * math.pi) * 2 ** 80)) for f in inv_freq]
    for i, p in enumerate(pos.tolist()):
        for j, f in enumerate(scaled):
            frac[i, j] = ((p * f) % 2 ** 80) / 2 ** 80
    c, s = torch.cos(2 * math.pi * frac)[:, None], torch.sin(2 * math.pi * frac)[:, None]
    h = len(inv_freq)
    y, mag = x.clone(), torch.zeros_like(x)
    a_at = slice(0, 2 * h, 2) if interleaved else slice(0, h)
    b_at = slice(1, 2 * h, 2) if interleaved else slice(h, 2 * h)
    a, b = x[..., a_at], x[..., b_at]
    y[..., a_at], y[..., b_at] = magnitude * (a * c - b * s), magnitude * (a * s + b * c)
    mag[..., a_at] = mag[..., b_at] = (a.abs() + b.abs()) * abs(magnitude)
    return y, mag
