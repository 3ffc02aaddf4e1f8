"""What the operators of the 8-bit cache are measured on: append with norms of queries and keys,
attention with a sliding window and sinks, and forking, freeing and compacting of pages.

``run`` computes an operator from elementary torch operations, or, with ``own`` set, through
this package.  Shapes follow the package's workloads (Llama-3.1-8B: 32 query and 8 KV heads
of 128; 70B: 64 and 8; Qwen2.5-32B: 40 and 8; the tiny shape: 2 KV heads of 64; 16-token pages).

An 8-bit pool holds e4m3 codes; scales[kv][page][head], e8m0, is the power of two that a page's
codes of one head are multiplied by.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
_E4M3, _E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
_EPS = 1e-6
_LOWEST, _HIGHEST = -60, 60          # exponents that an append gives


# ---- cases --------------------------------------------------------------

def _append(name, requests, new_lo, new_hi, ctx, hq, hkv, d, rot, interleaved, norms, dtype, cache, page=16):
    c = dict(op="append", requests=requests, new_lo=new_lo, new_hi=new_hi, ctx=ctx, hq=hq, hkv=hkv, d=d, rot=rot,
             interleaved=interleaved, norms=norms, dtype=dtype, cache=cache, page=page)
    return dict(c, name=name) if name else c


def _attend(name, requests, new_lo, new_hi, ctx_lo, ctx_hi, window, sinks, hq, hkv, d, dtype, cache, page=16):
    c = dict(op="attend", requests=requests, new_lo=new_lo, new_hi=new_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi,
             window=window, sinks=sinks, hq=hq, hkv=hkv, d=d, dtype=dtype, cache=cache, page=page)
    return dict(c, name=name) if name else c


def _beams(name, groups, beams, ctx_lo, ctx_hi, layers, hkv, d, cache, page=16):
    c = dict(op="beams", groups=groups, beams=beams, ctx_lo=ctx_lo, ctx_hi=ctx_hi, layers=layers, hkv=hkv, d=d,
             cache=cache, page=page)
    return dict(c, name=name) if name else c


def _shrink(name, requests, ctx_lo, ctx_hi, keep, layers, hkv, d, cache, page=16):
    c = dict(op="shrink", requests=requests, ctx_lo=ctx_lo, ctx_hi=ctx_hi, keep=keep, layers=layers, hkv=hkv, d=d,
             cache=cache, page=page)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode step of a small batch into the 8-bit cache: latency
        _append("append8-decode", 8, 1, 1, 20000, 32, 8, 128, 128, False, True, "bf16", "e4m3"),
        # the prompts of a prefill step, 70B heads, ragged
        _append("append8-prefill", 6, 300, 2700, 9000, 64, 8, 128, 128, False, True, "bf16", "e4m3"),
        # a model that norms its heads and turns half of each, on a 16-bit cache
        _append("append16-norms", 5, 37, 411, 3000, 16, 4, 64, 32, True, True, "fp16", "wide"),
        # a few users, tiny heads: latency
        _attend("attend8-small", 4, 1, 1, 5, 600, 0, 0, 8, 2, 64, "bf16", "e4m3"),
        # a decode step over long contexts, which the cache's bytes bound
        _attend("attend8-decode", 64, 1, 1, 1000, 9000, 0, 0, 32, 8, 128, "bf16", "e4m3"),
        # a few drafted tokens each to verify
        _attend("attend8-verify", 12, 2, 5, 700, 7000, 0, 0, 64, 8, 128, "fp16", "e4m3"),
        # prompts behind earlier turns of a conversation
        _attend("attend8-prompts", 4, 65, 1200, 1500, 8000, 0, 0, 64, 8, 128, "bf16", "e4m3"),
        # a decode step of layers that see a window and the first tokens, 16-bit cache
        _attend("window-decode", 48, 1, 1, 300, 16000, 4096, 4, 40, 8, 128, "bf16", "wide"),
        # whole prompts in such layers
        _attend("window-prompts", 2, 4100, 6000, 4100, 6000, 1024, 4, 32, 8, 128, "bf16", "wide"),
        # beams of a few requests go on from the best ones: fork, then room for the next token
        _beams("beams-small", 2, 4, 20, 300, 4, 2, 64, "e4m3"),
        _beams("beams-batch", 16, 8, 300, 3000, 32, 8, 128, "e4m3"),
        # requests were evicted down or ended: free their pages, then close the gaps of the pool
        _shrink("shrink-pool", 24, 500, 3000, 0.45, 16, 8, 128, "e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "beams", "shrink"])
    hkv, d = rng.choice([(2, 64), (8, 128), (4, 128), (1, 128), (8, 64)])
    group = rng.choice([1, 4, 5, 8])
    dtype = rng.choice(["bf16", "fp16"])
    cache = rng.choice(["e4m3", "e4m3", "wide"])
    page = rng.choice([16, 16, 32, 64, 8])
    if op == "append":
        requests = _log(rng, 1, 64)
        lo = rng.choice([1, _log(rng, 2, 300)])
        hi = min(lo if lo == 1 else _log(rng, lo, 2700), max(1, 9000 // requests))
        return _append(None, requests, min(lo, hi), hi, _log(rng, 300, 20000), hkv * group, hkv, d,
                       rng.choice([d, d, d // 2, 0]), rng.choice([False, True]), rng.choice([True, True, False]),
                       dtype, cache, page)
    if op == "attend":
        if rng.random() < 0.6:
            requests, new_lo = _log(rng, 1, 64), 1
            new_hi = rng.choice([1, 1, 5])
        else:
            requests, new_lo = _log(rng, 1, 4), _log(rng, 2, 300)
            new_hi = _log(rng, new_lo, 1000)
        lo = max(new_lo, _log(rng, 1, 2000))
        window = rng.choice([0, 0, _log(rng, 16, 4096)])
        return _attend(None, requests, new_lo, new_hi, lo, max(new_hi, _log(rng, lo, 6000)), window,
                       rng.choice([0, 1, 4, 37]) if window else 0, hkv * group, hkv, d, dtype, cache, page)
    if op == "beams":
        lo = _log(rng, 3, 1000)
        return _beams(None, _log(rng, 1, 16), rng.choice([2, 3, 4, 8]), lo, _log(rng, lo, 3000), _log(rng, 1, 16), hkv,
                      d, cache, page)
    lo = _log(rng, 30, 1000)
    return _shrink(None, _log(rng, 1, 24), lo, _log(rng, lo, 3000), rng.choice([0.1, 0.3, 0.6]), _log(rng, 1, 12), hkv,
                   d, cache, page)


# ---- sizes and inputs ---------------------------------------------------

def _spread(n, lo, hi):
    """n whole numbers spread over lo..hi, the same for every seed."""
    f = (np.arange(1, n + 1) * 0.6180339887498949) % 1.0
    return (lo + np.floor(f * (hi - lo + 1))).astype(np.int64)


def _lens(c):
    """(new tokens, cached tokens with them) of each request."""
    new = _spread(c["requests"], c["new_lo"], c["new_hi"])
    if c["op"] == "append":
        return new, new + _spread(c["requests"], 0, c["ctx"])
    return new, np.maximum(new, _spread(c["requests"], c["ctx_lo"], c["ctx_hi"])[::-1])


def _inv_freq(rot):
    """Radians per position of each rotated pair: long wavelengths 8 times longer, short ones kept, a ramp between."""
    f = 500000.0 ** (-2.0 * np.arange(rot // 2, dtype=np.float64) / max(rot, 1))
    ramp = np.clip((8192.0 * f / (2 * math.pi) - 1.0) / (4.0 - 1.0), 0.0, 1.0)
    return f * (ramp + (1 - ramp) / 8.0)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _exponent(amax):
    """The least e with amax <= 448 * 2^e, within what an append gives (amax 0: the lowest)."""
    m, e = torch.frexp(amax.double() / 448.0)
    e = torch.where(m > 0.5, e, e - 1)
    return torch.where(amax > 0, e, _LOWEST).clamp(_LOWEST, _HIGHEST)


def _pool(g, layers, num_blocks, page, hkv, d, cache, dtype):
    """(pool, scales or None): rows of N(0, 1) whose heads' sizes differ from page to page."""
    shape = (layers, 2, num_blocks, page, hkv, d)
    if cache == "wide":
        return _randn(g, shape, dtype).flatten(-2), None
    pool = torch.empty(shape, dtype=_E4M3, device="cuda")
    scales = torch.empty((layers, 2, num_blocks, hkv), dtype=_E8M0, device="cuda")
    for layer in range(layers):
        x = _randn(g, shape[1:], torch.float32)
        x *= torch.exp2(0.7 * torch.randn((2, num_blocks, 1, hkv, 1), generator=g, device="cuda"))
        e = _exponent(x.abs().amax((2, 4)))
        pool[layer] = (x * torch.exp2(-e.float())[:, :, None, :, None]).to(_E4M3)
        scales[layer] = (e + 127).to(torch.uint8).view(_E8M0)
    return pool.flatten(-2), scales


def _tables(g, lens, page, num_blocks):
    """int32 [requests][columns] block table of distinct shuffled ids, -1 where unused."""
    need = torch.from_numpy(-(-np.asarray(lens) // page)).cuda()
    cols = max(1, int(-(-int(max(lens, default=1)) // page)))
    ids = torch.randperm(num_blocks, generator=g, device="cuda")
    first = torch.cumsum(need, 0) - need
    col = torch.arange(cols, device="cuda")
    at = (first[:, None] + col).clamp(max=num_blocks - 1)
    return torch.where(col < need[:, None], ids[at], -1).to(torch.int32).contiguous()


def _prepare_pages(c, g, s):
    """Block tables with shared pages, and how often each page is held."""
    page = c["page"]
    if c["op"] == "beams":
        lens = np.repeat(_spread(c["groups"], c["ctx_lo"], c["ctx_hi"]), c["beams"])
        rows = len(lens)
        full = lens // page
        shared = (full * 3 // 4)                        # pages that the beams of a request have in common
        cols = int((lens // page).max()) + 2            # room for the next token
        own_pages = -(-lens // page) - shared
        need = int(own_pages.sum() + shared[::c["beams"]].sum())
        num_blocks = need + rows + max(8, need // 8)
        ids = torch.randperm(num_blocks, generator=g, device="cuda").cpu().numpy()
        table = np.full((rows, cols), -1, np.int32)
        at = 0
        for r in range(rows):
            if r % c["beams"] == 0:
                table[r, :shared[r]] = ids[at:at + shared[r]]
                at += shared[r]
            else:
                table[r, :shared[r]] = table[r - r % c["beams"], :shared[r]]
            table[r, shared[r]:shared[r] + own_pages[r]] = ids[at:at + own_pages[r]]
            at += own_pages[r]
        # the best beams of a request go on, some of them more than once
        pick = torch.randint(0, c["beams"], (rows,), generator=g, device="cuda")
        base = torch.arange(rows, device="cuda") // c["beams"] * c["beams"]
        s["parents"] = (base + pick).to(torch.int32)
    else:
        lens = _spread(c["requests"], c["ctx_lo"], c["ctx_hi"])
        rows = c["requests"]
        pages = -(-lens // page)
        cols = int(pages.max())
        num_blocks = int(pages.sum()) + max(8, int(pages.sum()) // 16)
        ids = torch.randperm(num_blocks, generator=g, device="cuda").cpu().numpy()
        table = np.full((rows, cols), -1, np.int32)
        at = 0
        for r in range(rows):
            table[r, :pages[r]] = ids[at:at + pages[r]]
            at += pages[r]
        keep = np.floor(lens * c["keep"]).astype(np.int32)
        keep[2::5] = 0                                  # every fifth request has ended
        s["kept_len"] = torch.from_numpy(keep).cuda()
        s["page_map"] = torch.empty(num_blocks, dtype=torch.int32, device="cuda")
    s["table"] = torch.from_numpy(table).cuda()
    s["kv_len"] = torch.from_numpy(lens.astype(np.int32)).cuda()
    held = np.bincount(table[table >= 0], minlength=num_blocks).astype(np.int32)
    s["refs"] = torch.from_numpy(held).cuda()
    s["table_out"], s["refs_out"] = torch.empty_like(s["table"]), torch.empty_like(s["refs"])
    s["len_out"] = torch.empty_like(s["kv_len"])
    s["pool"], s["scales"] = _pool(g, c["layers"], num_blocks, page, c["hkv"], c["d"], c["cache"], torch.bfloat16)


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    page, d, hkv = c["page"], c["d"], c["hkv"]
    s = {"case": c}
    if c["op"] in ("beams", "shrink"):
        _prepare_pages(c, g, s)
    else:
        dt = _DTYPES[c["dtype"]]
        new, lens = _lens(c)
        q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        s["q_start"] = torch.from_numpy(q_start).cuda()
        s["kv_len"] = torch.from_numpy(lens.astype(np.int32)).cuda()
        s["max_new"], s["tokens"], s["max_len"] = int(new.max()), int(q_start[-1]), int(lens.max())
        pages = int((-(-lens // page)).sum())
        num_blocks = pages + max(8, pages // 8)
        s["pool"], s["scales"] = _pool(g, 1, num_blocks, page, hkv, d, c["cache"], dt)
        s["table"] = _tables(g, lens, page, num_blocks)
        t = s["tokens"]
        if c["op"] == "append":
            qkv = _randn(g, (t, c["hq"] + 2 * hkv, d), dt, 1.5)
            s["q"], s["k"], s["v"] = qkv[:, :c["hq"]], qkv[:, c["hq"]:c["hq"] + hkv], qkv[:, c["hq"] + hkv:]
            s["q_out"] = torch.empty((t, c["hq"], d), dtype=dt, device="cuda")
            s["q_norm"] = s["k_norm"] = None
            if c["norms"]:
                s["q_norm"] = 1.0 + 0.3 * torch.randn(d, generator=g, device="cuda")
                s["k_norm"] = 1.0 + 0.3 * torch.randn(d, generator=g, device="cuda")
            # positions run ahead of the cache index by what was evicted before
            req = np.searchsorted(q_start, np.arange(t), side="right") - 1
            index = np.arange(t) - q_start[req] + (lens - new)[req]
            ahead = torch.randint(0, 80000, (c["requests"],), generator=g, device="cuda")
            s["positions"] = torch.from_numpy(index).cuda() + ahead[torch.from_numpy(req).cuda()]
            s["inv_freq"] = torch.from_numpy(_inv_freq(c["rot"])).cuda()
        else:
            s["q"] = _randn(g, (t, c["hq"], d), dt, 1.5)
            s["scale"] = 1.0 / math.sqrt(d)
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty((t, c["hq"]), dtype=torch.float32, device="cuda")
    if own:
        import paged_kv_cache_lmkv_gb300 as pkg
        s["pkg"] = pkg
        scales = None if s["scales"] is None else list(s["scales"])
        s["handle"] = pkg.Pool(list(s["pool"]), hkv, d, scales=scales)
        if c["op"] == "append" and c["rot"]:
            s["rotary"] = pkg.Rotary(c["rot"], base=500000.0, interleaved=c["interleaved"], scaling="bands", factor=8.0,
                                     low=1.0, high=4.0, original=8192)
        if c["op"] == "attend":
            n = pkg.attend_window_workspace_bytes(s["handle"], c["hq"], s["tokens"], c["requests"], s["max_new"],
                                                  s["max_len"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        if c["op"] in ("beams", "shrink"):
            n = pkg.pages_workspace_bytes(s["handle"], s["table"].shape[0])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


# ---- one pass -----------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _outputs(s, **more):
    """What an operator wrote, with the cache: codes, and scales where it has them."""
    more["pool"] = s["pool"]
    if s["scales"] is not None:
        more["scales"] = s["scales"]
    return more


def _run_own(s):
    c, pkg = s["case"], s["pkg"]
    if c["op"] == "append":
        pkg.check(pkg.append_layer_normed(s["handle"], 0, s["table"], s["q"], s["k"], s["v"], s["q_out"], s["q_start"],
                                          s["kv_len"], rotary=s.get("rotary"), q_norm=s["q_norm"], k_norm=s["k_norm"],
                                          eps=_EPS, positions=s["positions"]), "append_layer_normed")
        return _outputs(s, q=s["q_out"])
    if c["op"] == "attend":
        pkg.check(pkg.attend_layer_window(s["handle"], 0, s["q"], s["out"], s["q_start"], s["kv_len"], s["table"],
                                          s["scale"], s["workspace"], window=c["window"], sinks=c["sinks"],
                                          lse=s["lse"], max_new=s["max_new"], max_kv_len=s["max_len"]),
                  "attend_layer_window")
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "beams":
        pkg.check(pkg.fork_pages(s["handle"], s["table"], s["kv_len"], s["parents"], s["refs"], s["table_out"],
                                 s["len_out"], s["refs_out"], s["workspace"]), "fork_pages")
        pkg.check(pkg.resize_pages(s["handle"], s["table_out"], s["len_out"], s["len_out"] + 1, s["refs_out"],
                                   s["table_out"], s["refs_out"], s["workspace"]), "resize_pages")
        return _outputs(s, table=s["table_out"], lens=s["len_out"], refs=s["refs_out"])
    pkg.check(pkg.resize_pages(s["handle"], s["table"], s["kv_len"], s["kept_len"], s["refs"], s["table_out"],
                               s["refs_out"], s["workspace"]), "resize_pages")
    pkg.check(pkg.compact_pages(s["handle"], s["table_out"], s["kept_len"], s["refs_out"], s["table_out"],
                                s["refs_out"], s["page_map"], s["workspace"]), "compact_pages")
    return _outputs(s, table=s["table_out"], refs=s["refs_out"], map=s["page_map"])


def _normed(x, w):
    x = x.float()
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS) * w


def _rotated(x, angle, interleaved):
    """x [..., tokens, heads, d] rotated by angle [tokens, rot / 2] (64 bits), in 32 bits."""
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    half = angle.shape[-1]
    turn, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = turn[..., 0::2], turn[..., 1::2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = turn[..., :half], turn[..., half:]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((turned, rest), dim=-1)


def _plain_append(s):
    c, page = s["case"], s["case"]["page"]
    t = torch.arange(s["tokens"], device="cuda")
    start, lens = s["q_start"].long(), s["kv_len"].long()
    req = torch.searchsorted(start, t, right=True) - 1
    index = lens[req] - start[req + 1] + t
    blk = s["table"].long()[req, index // page]
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    s["q_out"].copy_(_rotated(_normed(s["q"], s["q_norm"]), angle, c["interleaved"]))
    kv = torch.stack((_rotated(_normed(s["k"], s["k_norm"]), angle, c["interleaved"]), s["v"].float()))
    pool = s["pool"][0].unflatten(-1, (c["hkv"], c["d"]))             # [2, pages, page, heads, d]
    if s["scales"] is None:
        pool[:, blk, index % page] = kv.to(pool.dtype)
        return
    exps = s["scales"][0].view(torch.uint8).int() - 127               # [2, pages, heads]
    amax = torch.zeros(exps.shape, device="cuda").index_reduce_(1, blk, kv.abs().amax(-1), "amax")
    # a request's first page may hold earlier tokens
    first = lens - (start[1:] - start[:-1])
    page0, held = s["table"].long()[torch.arange(len(lens), device="cuda"), first // page], first % page
    before = torch.full_like(exps, _LOWEST)
    before[:, page0] = torch.where((held > 0)[None, :, None], exps[:, page0], _LOWEST)
    now = torch.maximum(before, _exponent(amax).int())
    old = torch.exp2((before - now)[:, page0].float())[:, :, None, :, None]
    codes = pool[:, page0].float()
    kept = torch.arange(page, device="cuda")[None, :, None, None] < held[:, None, None, None]
    pool[:, page0] = torch.where(kept, codes * old, codes).to(_E4M3)
    pool[:, blk, index % page] = (kv * torch.exp2(-now[:, blk].float())[..., None]).to(_E4M3)
    touched = torch.zeros(exps.shape[1], dtype=torch.bool, device="cuda").index_fill_(0, blk, True)
    now = torch.where(touched[None, :, None], now, exps)
    s["scales"][0].copy_((now + 127).to(torch.uint8).view(_E8M0))


def _plain_attend(s):
    c, page = s["case"], s["case"]["page"]
    r, group = c["requests"], c["hq"] // c["hkv"]
    new, lens = (s["q_start"][1:] - s["q_start"][:-1]).long(), s["kv_len"].long()
    m = s["max_len"]
    if c["window"]:
        # the first tokens, then those from the first new token's window on
        behind = min(m, c["window"] + s["max_new"] - 1)
        begin = (lens - new + 1 - c["window"]).clamp(min=c["sinks"])
        index = torch.cat((torch.arange(c["sinks"], device="cuda").expand(r, -1),
                           begin[:, None] + torch.arange(behind, device="cuda")), dim=1)
    else:
        index = torch.arange(m, device="cuda").expand(r, m)
    there = index < lens[:, None]
    at = index.clamp(max=s["table"].shape[1] * page - 1)
    blk = s["table"].long().gather(1, at // page).clamp(min=0)
    rows = s["pool"][0].unflatten(-1, (c["hkv"], c["d"]))[:, blk, at % page].float()    # [2, r, keys, heads, d]
    if s["scales"] is not None:
        rows = rows * s["scales"][0][:, blk].float()[..., None]
    k, v = torch.where(there[..., None, None], rows, 0.0).unbind()
    t = torch.arange(s["tokens"], device="cuda")
    req = torch.searchsorted(s["q_start"].long(), t, right=True) - 1
    i = t - s["q_start"].long()[req]
    q = torch.zeros((r, s["max_new"], c["hkv"], group, c["d"]), device="cuda")
    q[req, i] = s["q"].float().view(-1, c["hkv"], group, c["d"])
    q = q.permute(0, 2, 1, 3, 4).flatten(2, 3)                                          # [r, heads, new * group, d]
    x = (q @ k.permute(0, 2, 3, 1)).mul_(s["scale"])
    last = ((lens - new)[:, None] + torch.arange(s["max_new"], device="cuda")).repeat_interleave(group, dim=1)
    seen = (index[:, None] <= last[..., None]) & there[:, None]
    if c["window"]:
        seen &= (index[:, None] > last[..., None] - c["window"]) | (index[:, None] < c["sinks"])
    x.masked_fill_(~seen[:, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = x @ v.transpose(1, 2)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (top + total.log())[..., 0]
    o = o.unflatten(2, (s["max_new"], group))[req, :, i].flatten(1, 2)
    lse = lse.unflatten(2, (s["max_new"], group))[req, :, i].flatten(1)
    return {"out": o.to(s["q"].dtype), "lse": lse}


def _held(table, lens, page):
    """Which columns of a table hold pages of rows of these lengths."""
    return torch.arange(table.shape[1], device="cuda") < ((lens.long() + page - 1) // page)[:, None]


def _count(refs, table, on, by):
    return refs.scatter_add(0, table[on].long(), torch.full((), by, dtype=torch.int32, device="cuda").expand(
        int(on.sum())))


def _resized(table, lens, new_lens, refs, page):
    had, has = _held(table, lens, page), _held(table, new_lens, page)
    refs = _count(refs, table, had & ~has, -1)
    table = torch.where(had & has, table, -1)
    want = has & ~had
    free = (refs == 0).nonzero()[:int(want.sum()), 0].int()           # the lowest ones, row by row
    table[want] = free
    return table, _count(refs, table, want, 1)


def _plain_beams(s):
    c, page, table = s["case"], s["case"]["page"], s["table"]
    rows = table.shape[0]
    lens = s["kv_len"][s["parents"].long()]
    after = table[s["parents"].long()]
    refs = _count(s["refs"], table, _held(table, s["kv_len"], page), -1)
    full = torch.arange(table.shape[1], device="cuda") < (lens.long() // page)[:, None]
    refs = _count(refs, after, full, 1)
    # a page that is not full goes on with the first row that wants it, if nobody else holds it
    r = torch.arange(rows, device="cuda")
    last = (lens.long() // page).clamp(max=table.shape[1] - 1)
    part = lens % page > 0
    src = after[r, last].long().clamp(min=0)
    first = torch.full((len(refs),), rows, dtype=torch.long, device="cuda")
    first.scatter_reduce_(0, src[part], r[part], "amin")
    stays = part & (first[src] == r) & (refs[src] == 0)
    refs[src[stays]] = 1
    copied = part & ~stays
    fresh = (refs == 0).nonzero()[:int(copied.sum()), 0]
    refs[fresh] = 1
    after = torch.where(_held(after, lens, page), after, -1)
    after[r[copied], last[copied]] = fresh.int()
    slot = torch.arange(page, device="cuda")[None] < (lens % page)[copied][:, None]
    pages = s["pool"]
    old = pages[:, :, src[copied]]
    pages[:, :, fresh] = torch.where(slot[None, None, ..., None], old.view(_bits(old)),
                                     pages[:, :, fresh].view(_bits(old))).view(old.dtype)
    if s["scales"] is not None:
        s["scales"][:, :, fresh] = s["scales"][:, :, src[copied]]
    s["len_out"].copy_(lens)
    table, refs = _resized(after, lens, lens + 1, refs, page)
    s["table_out"].copy_(table)
    s["refs_out"].copy_(refs)


def _bits(t):
    return torch.uint8 if t.element_size() == 1 else torch.int16


def _plain_shrink(s):
    page = s["case"]["page"]
    table, refs = _resized(s["table"], s["kv_len"], s["kept_len"], s["refs"], page)
    # the lowest gaps take the highest pages
    gaps, used = (refs == 0).nonzero()[:, 0], (refs > 0).nonzero()[:, 0].flip(0)
    n = min(len(gaps), len(used))
    move = gaps[:n] < used[:n]
    to, src = gaps[:n][move], used[:n][move]
    s["pool"][:, :, to] = s["pool"][:, :, src]
    if s["scales"] is not None:
        s["scales"][:, :, to] = s["scales"][:, :, src]
    page_map = torch.arange(len(refs), dtype=torch.int32, device="cuda")
    page_map[src] = to.int()
    held = refs[src]
    refs[src] = 0
    refs[to] = held
    s["page_map"].copy_(page_map)
    s["table_out"].copy_(torch.where(table >= 0, page_map[table.long().clamp(min=0)], -1))
    s["refs_out"].copy_(refs)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "append":
        _plain_append(s)
        return _outputs(s, q=s["q_out"])
    if c["op"] == "attend":
        return _plain_attend(s)
    if c["op"] == "beams":
        _plain_beams(s)
        return _outputs(s, table=s["table_out"], lens=s["len_out"], refs=s["refs_out"])
    _plain_shrink(s)
    return _outputs(s, table=s["table_out"], refs=s["refs_out"], map=s["page_map"])


# ---- what a pass cannot do without --------------------------------------

def work(case):
    c, page = case, case["page"]
    row = c["hkv"] * c["d"] * (1 if c["cache"] == "e4m3" else 2)
    scale = c["hkv"] if c["cache"] == "e4m3" else 0             # bytes of a page's scales, of K or V
    if c["op"] == "append":
        new, lens = _lens(c)
        t = int(new.sum())
        pages = int((-(-lens // page) - (lens - new) // page).sum())
        return {"bytes": t * (2 * 2 * c["hq"] * c["d"] + 2 * c["hkv"] * c["d"] * 2 + 2 * row) + 2 * pages * scale,
                "flops": t * (c["hq"] + c["hkv"]) * (4 * c["d"] + 3 * c["rot"])}
    if c["op"] == "attend":
        new, lens = _lens(c)
        pairs = keys = 0
        for n, m in zip(new.tolist(), lens.tolist()):
            last = np.arange(m - n, m)
            seen = last + 1
            lo = 0
            if c["window"]:
                begin = np.maximum(last + 1 - c["window"], 0)
                seen = last + 1 - begin + np.minimum(begin, c["sinks"])
                lo = max(0, int(begin[0]) - c["sinks"])
            pairs += int(seen.sum())
            keys += m - lo
        return {"bytes": 2 * keys * row + 2 * (keys // page) * scale + int(new.sum()) * c["hq"] * (4 * c["d"] + 4),
                "flops": 4 * c["d"] * c["hq"] * pairs}
    if c["op"] == "beams":
        # of the rows of a request that go on, about a third share the parent of an earlier one
        lens = np.repeat(_spread(c["groups"], c["ctx_lo"], c["ctx_hi"]), c["beams"])
        copied = int((lens % page).sum() * 0.34)
        return {"bytes": 4 * copied * c["layers"] * row + int((-(-lens // page)).sum()) * 16, "flops": 0}
    lens = _spread(c["requests"], c["ctx_lo"], c["ctx_hi"])
    keep = np.floor(lens * c["keep"]).astype(np.int64)
    keep[2::5] = 0
    before, after = int((-(-lens // page)).sum()), int((-(-keep // page)).sum())
    blocks = before + max(8, before // 16)
    moved = int(after * (1 - after / blocks))
    return {"bytes": 4 * moved * c["layers"] * (page * row + scale) + blocks * 12, "flops": 0}


# ---- 64 bits ------------------------------------------------------------

def _turn64(x, pos, c):
    """x [tokens, heads, d] in 64 bits turned as complex numbers; pos [tokens]."""
    h = c["rot"] // 2
    f = torch.from_numpy(_inv_freq(c["rot"])).to(x.device)
    unit = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), pos.double()[:, None, None] * f)
    y = x.clone()
    a = slice(0, 2 * h, 2) if c["interleaved"] else slice(0, h)
    b = slice(1, 2 * h, 2) if c["interleaved"] else slice(h, 2 * h)
    z = torch.complex(x[..., a], x[..., b]) * unit
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _norm64(x, w):
    x = x.double()
    return x if w is None else w.double() * x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + _EPS)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] in ("beams", "shrink"):
        return None                   # copies and choices: nothing is computed
    page, hkv, d = c["page"], c["hkv"], c["d"]
    begin, lens = s["q_start"].tolist(), s["kv_len"].tolist()
    table = s["table"].cpu().numpy()
    pool = s["pool"][0].double().view(2, -1, page, hkv, d)
    if c["op"] == "append":
        q = _turn64(_norm64(s["q"], s["q_norm"]), s["positions"], c)
        k = _turn64(_norm64(s["k"], s["k_norm"]), s["positions"], c)
        for r in range(c["requests"]):
            old = lens[r] - (begin[r + 1] - begin[r])
            at = begin[r]
            for col in range(old // page, -(-lens[r] // page)):
                lo, hi = max(old, col * page), min(lens[r], col * page + page)
                new = torch.stack((k[at:at + hi - lo], s["v"][at:at + hi - lo].double()))     # [2, n, heads, d]
                at += hi - lo
                where = pool[:, int(table[r, col])]
                if s["scales"] is not None:
                    # codes are multiples of the page's power of two
                    e = torch.ceil(torch.log2(new.abs().amax((1, 3)) / 448.0)).clamp(_LOWEST, _HIGHEST)
                    if lo > col * page:
                        was = s["scales"][0][:, int(table[r, col])].double().log2()
                        e = torch.maximum(e, was)
                        where[:, :lo - col * page] *= torch.exp2(was - e)[:, None, :, None]
                    new = new / torch.exp2(e)[:, None, :, None]
                where[:, lo - col * page:hi - col * page] = new
        out = {"q": q, "pool": pool.view(s["pool"].shape)}
        if s["scales"] is not None:
            out["scales"] = None
        return out
    if s["scales"] is not None:
        pool = pool * s["scales"][0].double()[:, :, None, :, None]
    group = c["hq"] // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    for r in range(c["requests"]):
        lo, hi, n = begin[r], begin[r + 1], lens[r]
        ids = torch.from_numpy(table[r, :-(-n // page)].astype(np.int64)).cuda()
        k, v = pool[:, ids].flatten(1, 2)[:, :n].unbind()                                  # [n, heads, d]
        j, i = torch.arange(n, device="cuda"), torch.arange(n - (hi - lo), n, device="cuda")[:, None]
        seen = j <= i
        if c["window"]:
            seen = seen & ((i - j < c["window"]) | (j < c["sinks"]))
        for h in range(hkv):
            heads = slice(h * group, (h + 1) * group)
            x = s["q"][lo:hi, heads].double().transpose(0, 1) @ k[:, h].T * s["scale"]       # [group, new, n]
            x = torch.where(seen, x, float("-inf"))
            lse[lo:hi, heads] = torch.logsumexp(x, -1).T
            out[lo:hi, heads] = (torch.softmax(x, -1) @ v[:, h]).transpose(0, 1)
    return {"out": out, "lse": lse}
