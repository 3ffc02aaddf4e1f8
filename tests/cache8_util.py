"""Small ragged batches on 16-bit pools and pools of e4m3 codes, and 64-bit formulas of the
8-bit cache's operators."""
from __future__ import annotations

import math

import numpy as np
import torch

import paged_kv_cache_lmkv_gb300 as pkg
from operator_util import DEV, HALF_STEP, TINY, rotate64

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
LOWEST, HIGHEST = -60, 60


def exponent(amax):
    """Least e with amax <= 448 * 2^e, in -60 .. 60 (amax 0: -60); exact."""
    m, e = torch.frexp(amax.double() / 448.0)
    e = torch.where(m > 0.5, e, e - 1)
    return torch.where(amax > 0, e, LOWEST).clamp(LOWEST, HIGHEST)


def codes_of(x):
    """Values as codes, to nearest even, saturating; what is not finite as NaN."""
    c = x.double().clamp(-448, 448).float().to(E4M3)
    return torch.where(x.isfinite(), c.view(torch.uint8), 0x7F).to(torch.uint8)


class Cache:
    """Requests of new[r] new and kv[r] cached tokens (the new ones last) in shuffled pages of one
    layer of a pool; page slots that hold no token are NaN.  wide: a 16-bit pool of the rows' type."""

    def __init__(self, new, kv, heads, kv_heads, dim, dtype, wide=False, page=16, seed=0, extra_rows=0, spread=1.5,
                 exps=(-9, -3), layers=2, layer=1, spare=3, device=DEV):
        g = torch.Generator().manual_seed(seed)
        self.new, self.kv, self.page, self.wide = list(new), list(kv), page, wide
        self.heads, self.kv_heads, self.dim, self.dtype = heads, kv_heads, dim, dtype
        self.group, self.layer = heads // kv_heads, layer
        need = [-(-max(n, 0) // page) for n in self.kv]
        self.num_blocks = sum(need) + spare
        ids = torch.randperm(self.num_blocks, generator=g)
        cols = max(1, max(need, default=1)) + 1
        self.table = torch.full((len(self.kv), cols), -1, dtype=torch.int32)
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = ids[at:at + n]
            at += n
        shape = (layers, 2, self.num_blocks, page, kv_heads, dim)
        rows = torch.randn(shape, generator=g)
        if wide:
            pool, self.scales_cpu = rows.to(dtype), None
        else:
            e = torch.randint(exps[0], exps[1] + 1, (layers, 2, self.num_blocks, kv_heads), generator=g)
            pool = codes_of(rows * 100.0).view(shape)
            self.scales_cpu = (e + 127).to(torch.uint8)
        nan = torch.full((), float("nan"), dtype=dtype) if wide else torch.tensor(0x7F, dtype=torch.uint8)
        there = torch.zeros(self.num_blocks, page, dtype=torch.bool)
        for r in range(len(self.kv)):
            s = self.slots(r)
            there.view(-1)[s] = True
        self.pool_cpu = torch.where(there[None, None, :, :, None, None], pool, nan).flatten(-2).contiguous()
        self.q_start = torch.tensor(np.concatenate([[0], np.cumsum(self.new)]), dtype=torch.int32)
        self.kv_len = torch.tensor(self.kv, dtype=torch.int32)
        self.tokens = int(self.q_start[-1]) + extra_rows
        self.q_cpu = (torch.randn((self.tokens, heads, dim), generator=g) * spread).to(dtype)
        self.scale = 1.0 / math.sqrt(dim)
        self.to(device)

    def to(self, device):
        self.device = device
        scales = None
        if not self.wide:
            self.scales_d = self.scales_cpu.to(device)
            scales = list(self.scales_d)
        pool = self.pool_cpu.to(device)
        self.pool = pkg.Pool(list(pool if self.wide else pool.view(E4M3)), self.kv_heads, self.dim, scales=scales)
        for n in ("table", "q_start", "kv_len"):
            setattr(self, n + "_d", getattr(self, n).to(device))
        self.q = self.q_cpu.to(device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def slots(self, r):
        j = torch.arange(max(self.kv[r], 0))
        return self.table[r].long()[j // self.page] * self.page + j % self.page

    def rows64(self, slots, h, kv):
        """Rows of head h, values in 64 bits."""
        d = self.dim
        x = self.pool_cpu[self.layer, kv].view(-1, self.kv_heads * d)[slots, h * d:(h + 1) * d]
        if self.wide:
            return x.double()
        byte = self.scales_cpu[self.layer, kv, slots // self.page, h].double()
        power = torch.where(byte == 255, math.nan, torch.exp2(byte - 127))
        return x.contiguous().view(E4M3).double() * power[:, None]

    def sizes(self, slots, h, kv):
        """448 times the scale of each token's page (16 bits: 1)."""
        if self.wide:
            return torch.ones(len(slots), dtype=torch.float64)
        return 448.0 * torch.exp2(self.scales_cpu[self.layer, kv, slots // self.page, h].double() - 127)

    def seen(self, r, window, sinks):
        n, m = self.new[r], max(self.kv[r], 0)
        t = self.kv[r] - n + torch.arange(n)[:, None]
        j = torch.arange(m)[None]
        s = j <= t
        return s & ((j > t - window) | (j < sinks)) if window else s

    def attend(self, window=0, sinks=0, hide=None, scale=None):
        """(out, lse, tolerance of out, of lse) in 64 bits; hide(r, tokens): bool mask of tokens that are not there."""
        scale = self.scale if scale is None else scale
        t, hq, d = self.tokens, self.heads, self.dim
        out = torch.zeros((t, hq, d), dtype=torch.float64)
        lse = torch.full((t, hq), -math.inf, dtype=torch.float64)
        tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
        # weights are rounded to fp16 beside codes, else to the rows' type
        step, tiny = HALF_STEP[self.dtype], TINY[self.dtype]
        weight = HALF_STEP[torch.float16] if not self.wide else step
        for r in range(len(self.new)):
            lo, n = int(self.q_start[r]), self.new[r]
            if n == 0 or self.kv[r] <= 0:
                continue
            slots = self.slots(r)
            seen = self.seen(r, window, sinks)
            if hide is not None:
                seen = seen & ~hide(r, self.kv[r])[None]
            some_row = seen.any(0)
            for h in range(self.kv_heads):
                k, v = self.rows64(slots, h, 0), self.rows64(slots, h, 1)
                k, v = (torch.where(some_row[:, None], x, 0.0) for x in (k, v))
                size = torch.where(some_row, self.sizes(slots, h, 1), 0.0).amax()
                for a in range(h * self.group, (h + 1) * self.group):
                    q = self.q_cpu[lo:lo + n, a].double()
                    raw = q @ k.T * scale
                    x = raw.masked_fill(~seen, -math.inf)
                    top = x.amax(1, keepdim=True).clamp(min=-1e300)
                    w = torch.exp(x - top)
                    total = w.sum(1, keepdim=True)
                    some = total[:, 0] > 0
                    p = torch.where(total > 0, w / total, 0.0)
                    o = p @ v
                    out[lo:lo + n, a] = o
                    lse[lo:lo + n, a] = torch.where(some, (top + total.log())[:, 0], -math.inf)
                    # A product of d terms in fp32, in any order, is off by at most d 2^-23 of the sum of magnitudes
                    # (truncating adders included); a score in powers of 2 (up to |x| / ln 2 and the scale's
                    # exponent, 70 at most here) is rounded twice, its factor twice; an fp32 sum of n weights or of n weighted
                    # values is off by (n + 16) 2^-23, 2^x by 2^-22.  Weights are rounded by half a step of
                    # their type, or, below 2^-14, by 2^-25, where the largest is 2^6 at least: 2^-31 of that for each key, times
                    # the largest value that a page holds.  The result is rounded by half a step.
                    keys = k.shape[0]
                    far = raw.abs().masked_fill(~seen, 0.0).nan_to_num(0.0).amax(1, keepdim=True)
                    dx = (d + 8) * 2.0 ** -23 * (q.abs() @ k.abs().T).nan_to_num(0.0).amax(1, keepdim=True) * abs(scale) + \
                        4 * 2.0 ** -24 * (far + 70)
                    mag = p @ v.abs()
                    f32 = 2 * dx + (keys + 16) * 2.0 ** -23 + 2.0 ** -21
                    tol_o[lo:lo + n, a] = (1.01 * weight + f32) * mag + step * 1.01 * o.abs() + tiny
                    if weight == HALF_STEP[torch.float16]:
                        tol_o[lo:lo + n, a] += keys * 2.0 ** -31 * size * (4.0 if self.wide else 1.0)
                    tol_l[lo:lo + n, a] = (dx[:, 0] + (keys + 16) * 2.0 ** -23 +
                                           2.0 ** -21 * (1 + lse[lo:lo + n, a].abs().nan_to_num(posinf=0.0)))
        return out, lse, tol_o, tol_l


def normed64(x, w, eps):
    x = x.double()
    return x if w is None else x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()


def turned64(x, pos, rotary):
    """(x turned, |a| + |b| of each element's pair)."""
    if rotary is None:
        return x, x.abs()
    y, mag = rotate64(x, pos, rotary.inv_freq, rotary.interleaved, rotary.magnitude)
    mag[..., rotary.rot_dim:] = x[..., rotary.rot_dim:].abs()
    return y, mag
