"""What the cache's attention-side operators are measured on: rotary append, rotary-shifted
retrieve, shared-prefix attention, attention weights and eviction on a paged KV pool.

``run`` computes an operator from elementary torch operations, or, with ``own`` set, through
this package.  Shapes follow the package's workloads (Llama-3.1-8B: 32 query and 8 KV heads
of 128; 70B: 64 and 8; the tiny shape: 2 KV heads of 64; 16-token pages, 256-token chunks).
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---- cases --------------------------------------------------------------

def _append(name, requests, new_lo, new_hi, ctx, hq, hkv, d, rot, interleaved, scaling, dtype, page=16):
    c = dict(op="append", requests=requests, new_lo=new_lo, new_hi=new_hi, ctx=ctx, hq=hq, hkv=hkv, d=d,
             rot=rot, interleaved=interleaved, scaling=scaling, dtype=dtype, page=page)
    return dict(c, name=name) if name else c


def _shifted(name, requests, tok_lo, tok_hi, layers, hkv, d, rot, interleaved, scaling, dtype, one_layer,
             page=16, chunk=256):
    c = dict(op="shifted", requests=requests, tok_lo=tok_lo, tok_hi=tok_hi, layers=layers, hkv=hkv, d=d,
             rot=rot, interleaved=interleaved, scaling=scaling, dtype=dtype, one_layer=one_layer,
             page=page, chunk=chunk)
    return dict(c, name=name) if name else c


def _attend(name, requests, new_lo, new_hi, prefix, ctx_lo, ctx_hi, hq, hkv, d, dtype, page=16):
    c = dict(op="attend", requests=requests, new_lo=new_lo, new_hi=new_hi, prefix=prefix, ctx_lo=ctx_lo,
             ctx_hi=ctx_hi, hq=hq, hkv=hkv, d=d, dtype=dtype, page=page)
    return dict(c, name=name) if name else c


def _weigh(name, requests, new_lo, new_hi, ctx_lo, ctx_hi, hq, hkv, d, dtype, page=16):
    c = dict(op="weigh", requests=requests, new_lo=new_lo, new_hi=new_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi,
             hq=hq, hkv=hkv, d=d, dtype=dtype, page=page)
    return dict(c, name=name) if name else c


def _evict(name, requests, ctx_lo, ctx_hi, budget, sinks, recent, hkv, d, dtype, page=16):
    c = dict(op="evict", requests=requests, ctx_lo=ctx_lo, ctx_hi=ctx_hi, budget=budget, sinks=sinks,
             recent=recent, hkv=hkv, d=d, dtype=dtype, page=page)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode step of a small batch, 8B heads: latency
        _append("append-decode", 8, 1, 1, 40000, 32, 8, 128, 128, False, "bands", "bf16"),
        # the prompts of a prefill step, 70B heads, ragged
        _append("append-prefill", 6, 300, 2700, 12000, 64, 8, 128, 128, False, "bands", "bf16"),
        # prompts of a model that rotates half of each head in interleaved pairs, odd token counts
        _append("append-partial", 5, 37, 411, 3000, 16, 4, 128, 64, True, "linear", "fp16"),
        # one layer of the 10240-token retrieve at another position (layer-wise pipeline)
        _shifted("shifted-layer", 1, 10240, 10240, 4, 8, 128, 128, False, "bands", "bf16", True),
        # several documents, all layers in one call, partial last chunks
        _shifted("shifted-batch", 5, 1500, 9000, 16, 8, 128, 128, False, "plain", "bf16", False),
        # a few users behind a short system prompt, tiny heads: latency
        _attend("attend-small", 4, 1, 1, 512, 5, 90, 8, 2, 64, "bf16"),
        # decode of 64 users that share a long document, 8B heads
        _attend("attend-decode", 64, 1, 1, 16384, 33, 900, 32, 8, 128, "bf16"),
        # new questions (prompts) of 12 users on a shared document, 70B heads
        _attend("attend-extend", 12, 65, 400, 8192, 65, 700, 64, 8, 128, "fp16"),
        # a decode step's weights, long own contexts
        _weigh("weigh-decode", 24, 1, 1, 1000, 9000, 32, 8, 128, "bf16"),
        # an observation window of 64 queries at the end of each prompt
        _weigh("weigh-window", 4, 64, 64, 5000, 16000, 32, 8, 128, "bf16"),
        # one short request over its budget: latency
        _evict("evict-small", 2, 700, 1100, 512, 4, 64, 2, 64, "bf16"),
        # a batch of long requests cut to a quarter, some still below the budget
        _evict("evict-batch", 12, 3500, 20000, 4096, 4, 512, 8, 128, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "shifted", "attend", "attend", "weigh", "evict"])
    hkv, d = rng.choice([(2, 64), (8, 128), (4, 128), (1, 128), (8, 64)])
    group = rng.choice([1, 4, 5, 8])
    dtype = rng.choice(["bf16", "fp16"])
    page = rng.choice([16, 16, 32, 64, 8])
    scaling = rng.choice(["plain", "linear", "bands"])
    rot = rng.choice([d, d, d // 2])
    if op == "append":
        requests = _log(rng, 1, 64)
        lo = rng.choice([1, _log(rng, 2, 300)])
        hi = min(lo if lo == 1 else _log(rng, lo, 2700), max(1, 9000 // requests))
        return _append(None, requests, min(lo, hi), hi, _log(rng, 300, 40000), hkv * group, hkv, d, rot,
                       rng.choice([False, True]), scaling, rng.choice(["bf16", "fp16", "fp32"]), page)
    if op == "shifted":
        requests = _log(rng, 1, 4)
        lo = _log(rng, 20, 4000)
        return _shifted(None, requests, lo, _log(rng, lo, 9000), _log(rng, 1, 6), hkv, d, rot,
                        rng.choice([False, True]), scaling, rng.choice(["bf16", "fp16", "fp32"]),
                        rng.choice([False, True]), page)
    if op == "attend":
        if rng.random() < 0.5:
            requests, new_lo, new_hi = _log(rng, 1, 150), 1, 1
        else:
            requests, new_lo = _log(rng, 1, 12), _log(rng, 2, 65)
            new_hi = _log(rng, new_lo, 130)
        ctx_lo = max(new_lo, _log(rng, 1, 300))
        return _attend(None, requests, new_lo, new_hi, rng.choice([0, _log(rng, 100, 16384)]), ctx_lo,
                       max(new_hi, _log(rng, ctx_lo, 2000)), hkv * group, hkv, d, dtype, page)
    if op == "weigh":
        new = rng.choice([1, 1, _log(rng, 2, 64)])
        requests = _log(rng, 1, 24 if new == 1 else 4)
        lo = max(new, _log(rng, 64, 5000))
        return _weigh(None, requests, new, new, lo, _log(rng, lo, 9000), hkv * group, hkv, d, dtype, page)
    lo = _log(rng, 64, 4000)
    hi = _log(rng, lo, 16000)
    budget = _log(rng, 32, hi)
    sinks = min(rng.choice([0, 4]), budget)
    return _evict(None, _log(rng, 1, 12), lo, hi, budget, sinks, rng.randint(0, (budget - sinks) // 2), hkv, d,
                  rng.choice(["bf16", "fp16", "fp32"]), page)


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


def _inv_freq(rot, scaling):
    """Radians per position of each rotated pair."""
    f = 500000.0 ** (-2.0 * np.arange(rot // 2, dtype=np.float64) / rot)
    if scaling == "linear":
        return f / 4.0
    if scaling == "bands":         # long wavelengths 8 times longer, short ones kept, a ramp between
        turns = 8192.0 * f / (2 * math.pi)
        ramp = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        return f * (ramp + (1 - ramp) / 8.0)
    return f


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _tables(g, lens, page, num_blocks):
    """int32 [requests][columns] block table of distinct shuffled ids, -1 where unused."""
    need = torch.from_numpy(-(-np.asarray(lens) // page)).cuda()
    cols = max(1, int(-(-int(max(lens, default=1)) // page)))
    ids = torch.randperm(num_blocks, generator=g, device="cuda")
    first = torch.cumsum(need, 0) - need
    col = torch.arange(cols, device="cuda")
    at = (first[:, None] + col).clamp(max=num_blocks - 1)
    return torch.where(col < need[:, None], ids[at], -1).to(torch.int32).contiguous()


def _rotary_handle(c):
    import paged_kv_cache_lmkv_gb300 as pkg
    kw = {"plain": {}, "linear": dict(scaling="linear", factor=4.0),
          "bands": dict(scaling="bands", factor=8.0, low=1.0, high=4.0, original=8192)}[c["scaling"]]
    return pkg.Rotary(c["rot"], base=500000.0, interleaved=c["interleaved"], **kw)


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    dt, page, d, hkv = _DTYPES[c["dtype"]], c["page"], c["d"], c["hkv"]
    s = {"case": c}
    if c["op"] == "shifted":
        lens = _spread(c["requests"], c["tok_lo"], c["tok_hi"])
    elif c["op"] == "evict":
        lens = _spread(c["requests"], c["ctx_lo"], c["ctx_hi"])
    else:
        new, lens = _lens(c)
        q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        s["q_start"] = torch.from_numpy(q_start).cuda()
        s["kv_len"] = torch.from_numpy(lens.astype(np.int32)).cuda()
        s["max_new"], s["tokens"] = int(new.max()), int(q_start[-1])
    s["max_len"] = int(lens.max())
    prefix = c.get("prefix", 0)
    pages = int((-(-lens // page)).sum()) + -(-prefix // page)
    num_blocks = pages + max(8, pages // 8)
    layers = c.get("layers", 1)
    if c["op"] == "shifted":
        pool = torch.zeros((layers, 2, num_blocks, page, hkv * d), dtype=dt, device="cuda")
    else:
        pool = _randn(g, (layers, 2, num_blocks, page, hkv * d), dt)
    s["pool"] = pool
    rows = _tables(g, list(lens) + [prefix], page, num_blocks)
    cols = -(-s["max_len"] // page)
    s["table"] = rows[:-1, :cols].contiguous()
    s["prefix_table"] = rows[-1, :max(1, -(-prefix // page))].contiguous()

    if c["op"] == "append":
        t = s["tokens"]
        qkv = _randn(g, (t, c["hq"] + 2 * hkv, d), dt)
        s["q"], s["k"], s["v"] = qkv[:, :c["hq"]], qkv[:, c["hq"]:c["hq"] + hkv], qkv[:, c["hq"] + hkv:]
        s["q_out"] = torch.empty((t, c["hq"], d), dtype=dt, device="cuda")
        # positions run ahead of the cache index by what was evicted before
        req = np.searchsorted(q_start, np.arange(t), side="right") - 1
        index = np.arange(t) - q_start[req] + (lens - new)[req]
        ahead = torch.randint(0, 80000, (c["requests"],), generator=g, device="cuda")
        s["positions"] = torch.from_numpy(index).cuda() + ahead[torch.from_numpy(req).cuda()]
    elif c["op"] == "shifted":
        n_l = layers
        cuts = [min(c["chunk"], int(n) - a) for n in lens for a in range(0, int(n), c["chunk"])]
        s["chunks"] = [_randn(g, (2, n_l, n, hkv * d), dt) for n in cuts]
        s["start"], s["end"] = np.zeros(len(lens), np.int64), lens
        s["shift"] = np.random.default_rng(seed).integers(-100000, 100000, len(lens))
        s["shift_gpu"] = torch.from_numpy(s["shift"]).cuda()
        s["ends_gpu"] = torch.from_numpy(np.cumsum(lens)).cuda()
        s["tokens"] = int(lens.sum())
    elif c["op"] in ("attend", "weigh"):
        t = s["tokens"]
        s["q"] = _randn(g, (t, c["hq"], d), dt, 1.5)
        s["scale"] = 1.0 / math.sqrt(d)
        if c["op"] == "attend":
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty((t, c["hq"]), dtype=torch.float32, device="cuda")
        else:
            seen = torch.from_numpy(np.repeat(lens, new).astype(np.float32)).cuda()
            noise = torch.randn((t, c["hq"]), generator=g, device="cuda") * 0.05
            s["lse"] = seen.log()[:, None] + 0.5 * 1.5 ** 2 + noise
            s["scores"] = torch.rand((c["requests"], hkv, s["max_len"]), generator=g, device="cuda")
            s["scores_out"] = torch.zeros_like(s["scores"])
    else:
        shape = (c["requests"], hkv, s["max_len"])
        # accumulated softmax weight is heavy-tailed; tokens never looked at tie at zero
        w = torch.exp(3 * torch.randn(shape, generator=g, device="cuda") - 6)
        s["scores"] = torch.where(torch.rand(shape, generator=g, device="cuda") < 0.2, 0.0, w)
        s["kv_len"] = torch.from_numpy(lens.astype(np.int32)).cuda()
        s["keep"] = torch.empty((c["requests"], hkv, c["budget"]), dtype=torch.int32, device="cuda")
        s["new_len"] = torch.empty(c["requests"], dtype=torch.int32, device="cuda")
        s["kept_scores"] = torch.empty((c["requests"], hkv, c["budget"]), dtype=torch.float32, device="cuda")
    if own:
        import paged_kv_cache_lmkv_gb300 as pkg
        s["pkg"] = pkg
        s["handle"] = pkg.Pool(list(pool), hkv, d)
        if c["op"] in ("append", "shifted"):
            s["rotary"] = _rotary_handle(c)
        if c["op"] == "shifted":
            s["chunk_ptrs"] = pkg.pointer_array(s["chunks"], "cuda")
        if c["op"] == "attend":
            n = pkg.attend_workspace_bytes(s["handle"], c["hq"], s["tokens"], c["requests"], s["max_new"],
                                            prefix, s["max_len"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    if c["op"] in ("append", "shifted"):
        s["inv_freq"] = torch.from_numpy(_inv_freq(c["rot"], c["scaling"])).cuda()
    return s


# ---- one pass -----------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    c, pkg = s["case"], s["pkg"]
    if c["op"] == "append":
        pkg.check(pkg.append_layer(s["handle"], 0, s["table"], s["q"], s["k"], s["v"], s["q_out"], s["q_start"],
                                   s["kv_len"], s["rotary"], positions=s["positions"]), "append_layer")
        return {"q": s["q_out"], "pool": s["pool"]}
    if c["op"] == "shifted":
        a = (s["handle"], s["table"], s["start"], s["end"], c["chunk"], True, s["chunk_ptrs"], s["shift"],
             s["rotary"])
        if c["one_layer"]:
            pkg.check(pkg.scatter_layer_shifted(*a, 0), "scatter_layer_shifted")
            return {"pool": s["pool"][0]}
        pkg.check(pkg.scatter_chunks_shifted(*a), "scatter_chunks_shifted")
        return {"pool": s["pool"]}
    if c["op"] == "attend":
        pkg.check(pkg.attend_layer(s["handle"], 0, s["q"], s["out"], s["q_start"], s["kv_len"], s["table"],
                                   s["scale"], s["workspace"], prefix_table=s["prefix_table"],
                                   prefix_len=c["prefix"], lse=s["lse"], max_new=s["max_new"],
                                   max_kv_len=s["max_len"]), "attend_layer")
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "weigh":
        pkg.check(pkg.weigh_layer(s["handle"], 0, s["q"], s["lse"], s["q_start"], s["kv_len"], s["table"],
                                  s["scale"], s["scores"], s["scores_out"], decay=0.75, max_new=s["max_new"],
                                  max_kv_len=s["max_len"]), "weigh_layer")
        return {"scores": s["scores_out"]}
    pkg.check(pkg.evict_layer(s["handle"], 0, s["table"], s["kv_len"], s["scores"], c["sinks"], c["recent"],
                              s["keep"], s["new_len"], kept_scores=s["kept_scores"],
                                  max_kv_len=s["max_len"]), "evict_layer")
    return {"keep": s["keep"], "new_len": s["new_len"], "kept_scores": s["kept_scores"], "pool": s["pool"]}


def _rotated(x, angle, interleaved):
    """x [..., tokens, heads, d] rotated by angle [tokens, rot / 2] (64 bits), in 32 bits."""
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    half = angle.shape[-1]
    x = x.float()
    turn, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = turn[..., 0::2], turn[..., 1::2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = turn[..., :half], turn[..., half:]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((turned, rest), dim=-1)


def _slots(table, index, page):
    """Row of the flattened pool for each cached index of each request of the table."""
    return table.long().clamp(min=0).gather(-1, index // page) * page + index % page


def _own_rows(s, kv):
    """Own K (0) or V (1) padded to the longest request, [requests, keys, heads, d], 32 bits."""
    c = s["case"]
    r, m = c["requests"], s["max_len"]
    index = torch.arange(m, device="cuda").expand(r, m)
    at = _slots(s["table"], index, c["page"])
    flat = s["pool"][0].view(2, -1, c["hkv"], c["d"])
    there = (index < s["kv_len"].long()[:, None])[:, :, None, None]
    return torch.where(there, flat[kv][at].float(), 0.0)


def _padded_queries(s):
    """q [requests, kv heads, new * group, d] in 32 bits, and (request, new index) of each token."""
    c = s["case"]
    t = torch.arange(s["tokens"], device="cuda")
    req = torch.searchsorted(s["q_start"].long(), t, right=True) - 1
    i = t - s["q_start"].long()[req]
    group = c["hq"] // c["hkv"]
    q = torch.zeros((c["requests"], s["max_new"], c["hkv"], group, c["d"]), device="cuda")
    q[req, i] = s["q"].float().view(-1, c["hkv"], group, c["d"])
    return q.permute(0, 2, 1, 3, 4).flatten(2, 3), req, i


def _hidden(s, rows_per_new):
    """[requests, 1, new * group, keys]: own keys that a query may not see."""
    new = (s["q_start"][1:] - s["q_start"][:-1]).long()
    i = torch.arange(s["max_new"], device="cuda").repeat_interleave(rows_per_new)
    last = (s["kv_len"].long() - new)[:, None] + i
    hidden = torch.arange(s["max_len"], device="cuda") > last[:, :, None]
    return hidden[:, None]


def _run_plain(s):
    c = s["case"]
    group = c["hq"] // c["hkv"] if "hq" in c else 1
    if c["op"] == "append":
        t = torch.arange(s["tokens"], device="cuda")
        req = torch.searchsorted(s["q_start"].long(), t, right=True) - 1
        index = s["kv_len"].long()[req] - s["q_start"].long()[req + 1] + t
        at = _slots(s["table"][req], index[:, None], c["page"])[:, 0]
        angle = s["positions"].double()[:, None] * s["inv_freq"]
        dt = s["q"].dtype
        flat = s["pool"][0].view(2, -1, c["hkv"], c["d"])
        flat[0][at] = _rotated(s["k"], angle, c["interleaved"]).to(dt)
        flat[1][at] = s["v"]
        return {"q": _rotated(s["q"], angle, c["interleaved"]).to(dt), "pool": s["pool"]}
    if c["op"] == "shifted":
        lo, hi = (0, 1) if c["one_layer"] else (0, c["layers"])
        rows = torch.cat([x[:, lo:hi] for x in s["chunks"]], dim=2)
        t = torch.arange(s["tokens"], device="cuda")
        req = torch.searchsorted(s["ends_gpu"], t, right=True)
        before = torch.cat((s["ends_gpu"].new_zeros(1), s["ends_gpu"]))[req]
        at = _slots(s["table"][req], (t - before)[:, None], c["page"])[:, 0]
        angle = s["shift_gpu"].double()[req][:, None] * s["inv_freq"]
        flat = s["pool"].view(c["layers"], 2, -1, c["hkv"] * c["d"])
        k = rows[0].unflatten(-1, (c["hkv"], c["d"]))
        flat[lo:hi, 0, at] = _rotated(k, angle, c["interleaved"]).to(rows.dtype).flatten(-2)
        flat[lo:hi, 1, at] = rows[1]
        return {"pool": s["pool"][0] if c["one_layer"] else s["pool"]}
    if c["op"] == "attend":
        k, v = _own_rows(s, 0), _own_rows(s, 1)
        q, req, i = _padded_queries(s)
        a = (q @ k.permute(0, 2, 3, 1)) * s["scale"]
        a = a.masked_fill(_hidden(s, group), float("-inf"))
        a = a.unflatten(2, (s["max_new"], group))[req, :, i]             # [tokens, kv heads, group, keys]
        p = c["prefix"]
        index = torch.arange(p, device="cuda")
        at = _slots(s["prefix_table"][None], index[None], c["page"])[0]
        flat = s["pool"][0].view(2, -1, c["hkv"], c["d"])
        pk, pv = flat[0][at].float(), flat[1][at].float()
        qt = s["q"].float().view(-1, c["hkv"], group, c["d"]).transpose(0, 1).flatten(1, 2)
        b = (qt @ pk.permute(1, 2, 0)) * s["scale"]                      # [kv heads, tokens * group, prefix]
        b = b.unflatten(1, (-1, group)).transpose(0, 1)
        x = torch.cat((b, a), dim=-1)
        del a, b
        top = x.amax(-1, keepdim=True)
        top = torch.where(top == float("-inf"), 0.0, top)
        x = (x - top).exp_()
        total = x.sum(-1, keepdim=True)
        o = (x[..., :p].transpose(0, 1).flatten(1, 2) @ pv.transpose(0, 1)).unflatten(1, (-1, group)).transpose(0, 1)
        w = torch.zeros((c["requests"], s["max_new"], c["hkv"], group, s["max_len"]), device="cuda")
        w[req, i] = x[..., p:]
        u = w.permute(0, 2, 1, 3, 4).flatten(2, 3) @ v.transpose(1, 2)
        o = o + u.unflatten(2, (s["max_new"], group))[req, :, i]
        o = torch.where(total > 0, o / total, 0.0)
        lse = (top + total.log())[..., 0]
        return {"out": o.flatten(1, 2).to(s["q"].dtype), "lse": lse.flatten(1)}
    if c["op"] == "weigh":
        k = _own_rows(s, 0)
        q, req, i = _padded_queries(s)
        a = (q @ k.permute(0, 2, 3, 1)) * s["scale"]
        lse = torch.full((c["requests"], s["max_new"], c["hkv"], group), float("inf"), device="cuda")
        lse[req, i] = s["lse"].view(-1, c["hkv"], group)
        a = (a - lse.permute(0, 2, 1, 3).flatten(2)[..., None]).exp_()
        a = a.masked_fill(_hidden(s, group), 0.0).sum(2)
        there = torch.arange(s["max_len"], device="cuda") < s["kv_len"][:, None]
        old = s["scores"]
        s["scores_out"].copy_(torch.where(there[:, None], 0.75 * old + a, s["scores_out"]))
        return {"scores": s["scores_out"]}
    n, m = c["budget"], s["max_len"]
    length = s["kv_len"].long()[:, None]
    j = torch.arange(m, device="cuda")
    w = s["scores"]
    w = torch.where(((j < c["sinks"]) | (j >= length - c["recent"]))[:, None], float("inf"), w)
    w = torch.where((j < length)[:, None], w, float("-inf"))
    order = w.sort(dim=-1, descending=True, stable=True).indices[..., :n]
    kept = torch.minimum(length, length.new_tensor(n))
    slot = torch.arange(n, device="cuda")
    pad = n - order.shape[-1]
    order = torch.nn.functional.pad(order, (0, pad), value=m)
    order = torch.where((slot < kept)[:, None], order, m).sort(dim=-1).values
    there = order < m
    src = order.clamp(max=m - 1)
    heads = torch.arange(c["hkv"], device="cuda")[None, :, None]
    flat = s["pool"][0].view(2, -1, c["hkv"], c["d"])
    table = s["table"][:, None].expand(-1, c["hkv"], -1)
    at = _slots(table, src, c["page"])
    to = _slots(table, slot.clamp(max=m - 1).expand_as(src), c["page"])
    heads = heads.expand_as(src)
    rows = flat[:, at[there], heads[there]]
    flat[:, to[there], heads[there]] = rows
    return {"keep": torch.where(there, order, -1).int(), "new_len": kept[:, 0].int(),
            "kept_scores": torch.where(there, s["scores"].gather(-1, src), 0.0), "pool": s["pool"]}


# ---- what a pass cannot do without --------------------------------------

def work(case):
    c, e = case, _BYTES[case["dtype"]]
    row = c["hkv"] * c["d"] * e
    if c["op"] == "append":
        new, _ = _lens(c)
        t = int(new.sum())
        return {"bytes": 2 * t * (c["hq"] + 2 * c["hkv"]) * c["d"] * e,
                "flops": 3 * t * (c["hq"] + c["hkv"]) * c["rot"]}
    if c["op"] == "shifted":
        t = int(_spread(c["requests"], c["tok_lo"], c["tok_hi"]).sum())
        n_l = 1 if c["one_layer"] else c["layers"]
        return {"bytes": 4 * n_l * t * row, "flops": 3 * n_l * t * c["hkv"] * c["rot"]}
    if c["op"] == "evict":
        lens = _spread(c["requests"], c["ctx_lo"], c["ctx_hi"])
        cut = int((lens > c["budget"]).sum())
        kept = int(np.minimum(lens, c["budget"]).sum())
        return {"bytes": 4 * int(lens.sum()) * c["hkv"] + 8 * kept * c["hkv"]
                + 4 * cut * (c["budget"] - c["sinks"]) * row, "flops": int(lens.sum()) * c["hkv"]}
    new, lens = _lens(c)
    t = int(new.sum())
    pairs = int((new * (lens - new) + new * (new + 1) // 2).sum())
    if c["op"] == "weigh":
        return {"bytes": int(lens.sum()) * (row + 8 * c["hkv"]) + t * c["hq"] * (c["d"] * e + 4),
                "flops": 2 * c["d"] * c["hq"] * pairs}
    return {"bytes": 2 * (c["prefix"] + int(lens.sum())) * row + t * c["hq"] * (2 * c["d"] * e + 4),
            "flops": 4 * c["d"] * c["hq"] * (pairs + t * c["prefix"])}


# ---- 64 bits ------------------------------------------------------------

def _turn64(x, pos, c):
    """x [tokens, heads, d] in 64 bits turned as complex numbers; pos [tokens]."""
    h = c["rot"] // 2
    f = torch.from_numpy(_inv_freq(c["rot"], c["scaling"])).to(x.device)
    unit = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), pos.double()[:, None, None] * f)
    y = x.clone()
    first = slice(0, 2 * h, 2) if c["interleaved"] else slice(0, h)
    second = slice(1, 2 * h, 2) if c["interleaved"] else slice(h, 2 * h)
    z = torch.complex(x[..., first], x[..., second]) * unit
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _rows_of(table, n, page):
    ids = table[: -(-n // page)].long()
    return (ids[:, None] * page + torch.arange(page, device=ids.device)).flatten()[:n]


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    pool = s["pool"]
    if c["op"] == "evict":
        return None                   # copies and choices: nothing is computed
    if c["op"] == "shifted":
        lens, a = s["end"], 0
        n_l = 1 if c["one_layer"] else c["layers"]
        rows = torch.cat(s["chunks"], dim=2)[:, :n_l].double()
        out = pool[:n_l].double().view(n_l, 2, -1, c["hkv"] * c["d"])
        for r, n in enumerate(int(x) for x in lens):
            at = _rows_of(s["table"][r], n, c["page"])
            pos = torch.full((n,), int(s["shift"][r]), device="cuda")
            for layer in range(n_l):
                k = rows[0, layer, a:a + n].view(n, c["hkv"], c["d"])
                out[layer, 0, at] = _turn64(k, pos, c).view(n, -1)
                out[layer, 1, at] = rows[1, layer, a:a + n]
            a += n
        out = out.view(n_l, 2, -1, c["page"], c["hkv"] * c["d"])
        return {"pool": out[0] if c["one_layer"] else out}
    begin = s["q_start"].tolist()
    lens = s["kv_len"].tolist()
    flat = pool[0].view(2, -1, c["hkv"], c["d"])
    if c["op"] == "append":
        out = flat.double()
        for r in range(c["requests"]):
            lo, hi = begin[r], begin[r + 1]
            at = _rows_of(s["table"][r], lens[r], c["page"])[lens[r] - (hi - lo):]
            out[0, at] = _turn64(s["k"][lo:hi].double(), s["positions"][lo:hi], c)
            out[1, at] = s["v"][lo:hi].double()
        q = _turn64(s["q"].double(), s["positions"], c)
        return {"q": q, "pool": out.view(pool.shape)}
    group = c["hq"] // c["hkv"]
    scores = None
    if c["op"] == "weigh":
        scores = torch.zeros_like(s["scores"], dtype=torch.float64)
    else:
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    shared = _rows_of(s["prefix_table"], c.get("prefix", 0), c["page"])
    for h in range(c["hkv"]):
        heads = slice(h * group, (h + 1) * group)
        pk, pv = flat[0, shared, h].double(), flat[1, shared, h].double()
        for r in range(c["requests"]):
            lo, hi, n = begin[r], begin[r + 1], lens[r]
            at = _rows_of(s["table"][r], n, c["page"])
            q = s["q"][lo:hi, heads].double().transpose(0, 1)                       # [group, new, d]
            x = q @ torch.cat((pk, flat[0, at, h].double())).T * s["scale"]
            p = len(shared)
            seen = torch.arange(n, device="cuda") <= n - (hi - lo) + torch.arange(hi - lo, device="cuda")[:, None]
            x[..., p:].masked_fill_(~seen, float("-inf"))
            if c["op"] == "weigh":
                w = torch.exp(x - s["lse"][lo:hi, heads].T.double()[..., None]).sum((0, 1))
                scores[r, h, :n] = 0.75 * s["scores"][r, h, :n].double() + w
            else:
                lse[lo:hi, heads] = torch.logsumexp(x, -1).T
                o[lo:hi, heads] = (torch.softmax(x, -1) @ torch.cat((pv, flat[1, at, h].double()))).transpose(0, 1)
    return {"scores": scores} if c["op"] == "weigh" else {"out": o, "lse": lse}
