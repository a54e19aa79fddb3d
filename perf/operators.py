"""The operators of the quantised KV cache, as they are measured.

A cache of 8-bit floating-point codes (e4m3) with one fp32 scale per (token, KV head) takes 132
bytes where bf16 takes 256.  Four operators make it usable beside the bf16 pool:

  store   new tokens' bf16 K and V are quantised into their pool slots:
            scale = max(amax |x| / 448, 2^-126) over a row's 128 values, code = e4m3(x / scale)
          (a row with an infinity or a NaN: scale NaN, codes 0)
  load    slots are read back as bf16 rows: x = code * scale
  decode  one query per request over all of its keys, straight from the codes
  extend  a chunk of new tokens over the cached prefix and, causally, over themselves

`listed()` names the measured cases, `draw()` gives more of the same ranges; `run()` computes one
pass in plain torch operations in 32 bits, or, with `own` set, with this library's calls.
"""
import math

import numpy as np
import torch

own = False

D = 128          # head dimension
E4M3_MAX = 448.0
TINY = 2.0 ** -126


# ---- cases ------------------------------------------------------------------------------------

def listed():
    return [
        # a decode step's new tokens: 40 requests, 32 KV heads; launch latency counts
        dict(name="store-step", op="store", tokens=40, hkv=32, pool=32768),
        # the new tokens of a mixed prefill and decode step (16 extends, 8 cache misses, 40 decodes)
        dict(name="store-prompt", op="store", tokens=13064, hkv=32, pool=32768),
        # a 1,000-token system prompt of a grouped-query model read back, e.g. to move it elsewhere
        dict(name="load-prompt", op="load", tokens=1000, hkv=8, pool=71680),
        # most of a pool read back (a cache handed to another instance), an odd count
        dict(name="load-pool", op="load", tokens=32003, hkv=32, pool=32768),
        # four requests on one 1,000-token prompt: the smallest batch of a running server
        dict(name="decode-tiny", op="decode", hq=8, hkv=2, groups=1, members=4, prefix=1000,
             own_lo=1, own_hi=48, alone=0, alone_lo=1, alone_hi=1, lens=11),
        # one request with a long context and nothing to share: only splitting its keys fills a GPU
        dict(name="decode-single", op="decode", hq=32, hkv=8, groups=0, members=0, prefix=0,
             own_lo=1, own_hi=1, alone=1, alone_lo=16411, alone_hi=16411, lens=12),
        # 61 unrelated requests of very different lengths, grouped-query heads
        dict(name="decode-ragged", op="decode", hq=32, hkv=8, groups=0, members=0, prefix=0,
             own_lo=1, own_hi=1, alone=61, alone_lo=1, alone_hi=8191, lens=13),
        # 16 groups of 16 requests on 2,000-token prefixes, one query head per KV head
        dict(name="decode-shared", op="decode", hq=32, hkv=32, groups=16, members=16, prefix=2000,
             own_lo=100, own_hi=500, alone=0, alone_lo=1, alone_hi=1, lens=14),
        # 16 groups of 16 requests on 16,000-token prefixes, four query heads per KV head
        dict(name="decode-gqa", op="decode", hq=32, hkv=8, groups=16, members=16, prefix=16000,
             own_lo=200, own_hi=1000, alone=0, alone_lo=1, alone_hi=1, lens=15),
        # four users' 40-token questions on a 1,000-token system prompt
        dict(name="extend-tiny", op="extend", hq=8, hkv=2, groups=1, members=4, prefix=1000,
             own_lo=0, own_hi=0, new_lo=40, new_hi=40, lens=16),
        # 4 groups of 16 requests on 2,000-token prefixes, 40 to 200 new tokens each
        dict(name="extend-shared", op="extend", hq=32, hkv=32, groups=4, members=16, prefix=2000,
             own_lo=0, own_hi=0, new_lo=40, new_hi=200, lens=17),
        # the last chunk of a long prompt prefilled 2,048 tokens at a time, grouped-query heads
        dict(name="extend-chunk", op="extend", hq=32, hkv=8, groups=1, members=1, prefix=1024,
             own_lo=4096, own_hi=4096, new_lo=2048, new_hi=2048, lens=18),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["store", "load", "decode", "decode", "extend", "extend"])
        hkv = rng.choice([1, 2, 3, 4, 5, 8, 8, 12, 16, 32])
        if op in ("store", "load"):
            tokens = _log(rng, 1, 32003)
            if op == "store":
                tokens = min(tokens, 13064)
            return dict(op=op, tokens=tokens, hkv=hkv, pool=tokens + rng.randint(0, 20000))
        gq = rng.choice([1, 2, 4, 8])
        if hkv * gq > 64:
            continue
        case = dict(op=op, hq=hkv * gq, hkv=hkv, groups=rng.randint(0, 8),
                    members=_log(rng, 1, 24), prefix=_log(rng, 1, 16000),
                    lens=rng.randint(0, 1 << 30))
        if op == "decode":
            case.update(own_lo=1, own_hi=_log(rng, 1, 1000), alone=rng.randint(1, 40), alone_lo=1,
                        alone_hi=_log(rng, 1, 16411))
        else:
            case.update(groups=max(1, case["groups"]), own_lo=0, own_hi=_log(rng, 1, 300),
                        new_lo=1, new_hi=_log(rng, 1, 2048))
        w, n = work(case), _lengths(case)
        most = work(listed()[8 if op == "decode" else 10])
        padded = n["total"].size * int(n["total"].max()) * hkv
        rows = n["total"].size * int(n["new"].max()) * int(n["total"].max()) * case["hq"]
        if w["flops"] > most["flops"] or w["bytes"] > 2 * most["bytes"]:
            continue
        if padded > 256 * 17000 * 8 or (op == "extend" and rows > 64 * 200 * 2200 * 32):
            continue  # the plain forms pad their requests to the longest
        return case


def _lengths(case):
    """The lengths of a case's requests: shared and own cached tokens, new tokens, group."""
    r = np.random.default_rng(case["lens"])
    n_grp, extend = case["groups"] * case["members"], case["op"] == "extend"
    alone = 0 if extend else case["alone"]
    shared = np.concatenate([np.full(n_grp, case["prefix"]), np.zeros(alone, np.int64)])
    mine = np.concatenate([r.integers(case["own_lo"], case["own_hi"] + 1, n_grp),
                           r.integers(case["alone_lo"], case["alone_hi"] + 1, alone)
                           if alone else np.zeros(0, np.int64)])
    new = r.integers(case["new_lo"], case["new_hi"] + 1, n_grp) if extend else np.ones_like(mine)
    total = shared + mine + (new if extend else 0)  # a decode's own keys hold its current token
    group = np.concatenate([np.repeat(np.arange(case["groups"]), case["members"]),
                            np.full(alone, -1)])
    row = r.permutation(shared.size)  # the table row of each request
    return dict(shared=shared, mine=total - shared, new=new, total=total, group=group, row=row)


def work(case):
    """Codes, scales and slots of the distinct tokens once, queries and outputs once; the products
    of the unmasked (query, key) pairs."""
    if case["op"] in ("store", "load"):
        return {"bytes": case["tokens"] * (case["hkv"] * 2 * (2 * D + D + 4) + 4), "flops": 0}
    n = _lengths(case)
    tokens = case["groups"] * case["prefix"] + int(n["mine"].sum())
    rows = int(n["new"].sum())
    pairs = int((n["new"] * (n["total"] - n["new"]) + n["new"] * (n["new"] + 1) // 2).sum())
    return {"bytes": tokens * (case["hkv"] * 2 * (D + 4) + 4) + rows * case["hq"] * (4 * D + 4),
            "flops": 4 * D * case["hq"] * pairs}


# ---- inputs -----------------------------------------------------------------------------------

def _quantised(x):
    """Codes (as bytes) and scales of rows x [..., 128]."""
    amax = x.abs().amax(-1)
    scale = torch.clamp_min(amax / E4M3_MAX, TINY)
    scale = torch.where(torch.isfinite(amax), scale, torch.full_like(scale, math.nan))
    y = torch.clamp(x / scale[..., None], -E4M3_MAX, E4M3_MAX)
    y = torch.where(torch.isfinite(scale)[..., None], y, torch.zeros_like(y))
    return y.to(torch.float8_e4m3fn).view(torch.uint8), scale


def _rows(n, hkv, g, keys):
    """fp32 K or V rows [n, hkv, 128]: normal values; tokens differ in size, and a few of a head's
    key channels stand out."""
    x = torch.randn((n, hkv, D), generator=g, device="cuda")
    if keys:
        gain = torch.ones((hkv, D), device="cuda")
        gain[:, ::37] = 3.0
        return x * gain
    return x * torch.exp(0.5 * torch.randn((n, hkv, 1), generator=g, device="cuda"))


def _pool(case, pool, g):
    out = {}
    for name in ("k", "v"):
        codes, scales = [], []
        for at in range(0, pool, 65536):
            c, s = _quantised(_rows(min(65536, pool - at), case["hkv"], g, name == "k"))
            codes.append(c)
            scales.append(s)
        out[name + "_code"], out[name + "_scale"] = torch.cat(codes), torch.cat(scales)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"op": case["op"]}
    if case["op"] in ("store", "load"):
        s["slots"] = torch.randperm(case["pool"], generator=g, device="cuda")[:case["tokens"]].int()
        if case["op"] == "store":
            for name in ("k", "v"):
                s[name + "_new"] = _rows(case["tokens"], case["hkv"], g, name == "k").bfloat16()
                s[name + "_code"] = torch.zeros((case["pool"], case["hkv"], D), dtype=torch.uint8,
                                                device="cuda")
                s[name + "_scale"] = torch.zeros((case["pool"], case["hkv"]), device="cuda")
        else:
            s.update(_pool(case, case["pool"], g))
            for name in ("k", "v"):
                s[name + "_out"] = torch.empty((case["tokens"], case["hkv"], D),
                                               dtype=torch.bfloat16, device="cuda")
        pool = case["pool"]
        hq, table = case["hkv"], torch.zeros((1, 16), dtype=torch.int32, device="cuda")
    else:
        n = _lengths(case)
        b, width = n["total"].size, int(n["total"].max())
        starts = case["groups"] * case["prefix"] + np.cumsum(n["mine"]) - n["mine"]
        pool = int(case["groups"] * case["prefix"] + n["mine"].sum()) + 64
        perm = torch.randperm(pool, generator=g, device="cuda")
        dev = {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in
               dict(n, starts=starts).items()}
        j = torch.arange(width, device="cuda")[None]
        at = torch.where(j < dev["shared"][:, None], dev["group"][:, None] * case["prefix"] + j,
                         dev["starts"][:, None] + j - dev["shared"][:, None])
        at = torch.where(j < dev["total"][:, None], perm[at.clamp(0, pool - 1)], 0)
        table = torch.zeros((b, width), dtype=torch.int32, device="cuda")
        table[dev["row"]] = at.int()
        s.update(_pool(case, pool, g))
        rows, hq = int(n["new"].sum()), case["hq"]
        s["q"] = torch.randn((rows, hq, D), generator=g, device="cuda").bfloat16()
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((rows, hq), device="cuda")
        s["table"], s["row"], s["total"], s["new"] = table, dev["row"], dev["total"], dev["new"]
        s["width"], s["most_new"] = width, int(n["new"].max())
        s["of"] = torch.from_numpy(np.repeat(np.arange(b), n["new"])).cuda()  # a query's request
        s["nth"] = torch.from_numpy(np.concatenate([np.arange(e) for e in n["new"]])).cuda()
    if own:
        from prefix_shared_kv_gb300 import rx
        s["desc"] = rx.kv_desc(hq, case["hkv"], pool, table)
        s["kv"] = rx.kv_q8(s["k_code"], s["v_code"], s["k_scale"], s["v_scale"])
        if case["op"] in ("decode", "extend"):
            s["plan"] = plan = rx.Plan()
            plan.set_kv_type(rx.RX_KV_E4M3)
            prefixes = np.full(case["groups"], case["prefix"])
            if case["op"] == "decode":
                rx.decode_plan(plan, s["desc"], n["row"], n["total"], n["group"], prefixes)
            else:
                rx.extend_plan(plan, s["desc"], n["row"], n["total"] - n["new"], n["new"],
                               n["group"], prefixes)
            s["ws"] = torch.empty(max(256, plan.workspace_size()), dtype=torch.uint8,
                                  device="cuda")
            plan.upload(s["ws"])
    return s


# ---- one pass ---------------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"store": _store, "load": _load, "decode": _decode, "extend": _extend}[s["op"]](s)


def _run_own(s):
    from prefix_shared_kv_gb300 import rx
    if s["op"] == "store":
        rx.store_kv_q8(s["desc"], s["kv"], s["k_new"], s["v_new"], s["slots"])
        return _stored(s)
    if s["op"] == "load":
        rx.load_kv_q8(s["desc"], s["kv"], s["slots"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    attn = rx.decode_attn_q8 if s["op"] == "decode" else rx.extend_attn_q8
    attn(s["plan"], s["desc"], s["kv"], s["q"], s["o"], s["lse"], s["ws"])
    return {"o": s["o"], "lse": s["lse"]}


def _stored(s):
    return {"k_code": s["k_code"].view(torch.float8_e4m3fn), "k_scale": s["k_scale"],
            "v_code": s["v_code"].view(torch.float8_e4m3fn), "v_scale": s["v_scale"]}


def _store(s):
    at = s["slots"].long()
    s["k_code"][at], s["k_scale"][at] = _quantised(s["k_new"].float())
    s["v_code"][at], s["v_scale"][at] = _quantised(s["v_new"].float())
    return _stored(s)


def _values(s, name, at):
    codes = s[name + "_code"][at].view(torch.float8_e4m3fn).float()
    return codes.mul_(s[name + "_scale"][at][..., None])


def _load(s):
    at = s["slots"].long()
    return {"k": _values(s, "k", at).bfloat16(), "v": _values(s, "v", at).bfloat16()}


def _attend(s, q, limit):
    """q [B, E, hq, 128] fp32 over each request's table row; query e of request b sees the key
    positions below limit [B, E]."""
    at = s["table"][s["row"]].long()
    b, e, hq, hkv = q.shape[0], q.shape[1], q.shape[2], s["k_code"].shape[1]
    q = q.view(b, e, hkv, hq // hkv, D)
    scores = torch.einsum("behgd,blhd->bhgel", q, _values(s, "k", at)) * D ** -0.5
    seen = torch.arange(s["width"], device="cuda") < limit[..., None]
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgel,blhd->bhged", p, _values(s, "v", at)) / total
    lse = (top + torch.log(total))[..., 0]
    return (o.permute(0, 3, 1, 2, 4).reshape(b, e, hq, D),
            lse.permute(0, 3, 1, 2).reshape(b, e, hq))


def _decode(s):
    o, lse = _attend(s, s["q"].float()[:, None], s["total"][:, None])
    return {"o": o[:, 0].bfloat16(), "lse": lse[:, 0].contiguous()}


def _extend(s):
    b, e = s["total"].shape[0], s["most_new"]
    q = torch.zeros((b, e, *s["q"].shape[1:]), device="cuda")
    q[s["of"], s["nth"]] = s["q"].float()
    limit = (s["total"] - s["new"])[:, None] + 1 + torch.arange(e, device="cuda")
    o, lse = _attend(s, q, torch.minimum(limit, s["total"][:, None]))
    return {"o": o[s["of"], s["nth"]].bfloat16(), "lse": lse[s["of"], s["nth"]]}


# ---- the definition in 64 bits ----------------------------------------------------------------

def _e4m3(y):
    """The nearest e4m3 value of y (float64, |y| <= 448), ties to the even code."""
    size = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -30))).clamp_min(-6)
    step = torch.exp2(size - 3)
    return torch.round(y / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "store":
        out = {}
        for name in ("k", "v"):
            x = s[name + "_new"].double()
            scale = (x.abs().amax(-1) / E4M3_MAX).clamp_min(TINY)
            codes = s[name + "_code"].double()
            scales = s[name + "_scale"].double()
            codes[s["slots"].long()] = _e4m3(x / scale[..., None])
            scales[s["slots"].long()] = scale
            out[name + "_code"], out[name + "_scale"] = codes, scales
        return out

    def rows(name, at):
        return (s[name + "_code"][at].view(torch.float8_e4m3fn).double()
                * s[name + "_scale"][at].double()[..., None])

    if s["op"] == "load":
        return {name: rows(name, s["slots"].long()) for name in ("k", "v")}
    total, new, row = (s[k].tolist() for k in ("total", "new", "row"))
    hq, hkv = s["q"].shape[1], s["k_code"].shape[1]
    o = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    first = 0
    for b in range(len(total)):
        at = s["table"][row[b], :total[b]].long()
        k, v = rows("k", at).transpose(0, 1), rows("v", at).transpose(0, 1)  # [hkv, L, 128]
        for e0 in range(0, new[b], 256):
            e1 = min(new[b], e0 + 256)
            q = s["q"][first + e0:first + e1].double().view(e1 - e0, hkv, hq // hkv, D)
            z = (q.permute(1, 2, 0, 3).reshape(hkv, -1, D) @ k.transpose(1, 2)) / math.sqrt(D)
            z = z.view(hkv, hq // hkv, e1 - e0, total[b])
            last = total[b] - new[b] + torch.arange(e0, e1, device="cuda")
            hidden = torch.arange(total[b], device="cuda") > last[:, None]
            z = z.masked_fill(hidden, -math.inf)
            ls = torch.logsumexp(z, -1)
            w = torch.exp(z - ls[..., None]).reshape(hkv, -1, total[b]) @ v
            o[first + e0:first + e1] = w.view(hkv, hq // hkv, e1 - e0, D).permute(
                2, 0, 1, 3).reshape(e1 - e0, hq, D)
            lse[first + e0:first + e1] = ls.permute(2, 0, 1).reshape(e1 - e0, hq)
        first += new[b]
    return {"o": o, "lse": lse}
