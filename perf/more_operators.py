"""The block-scaled cache: its cases, its plain forms and the framework's calls.

The cache holds e4m3 codes and one power-of-two scale for each block of tokens and KV head, an exponent byte e: a code
c stands for c * 2^(e - 127). Four operators. ``write`` quantises keys and values as they are appended; a block that
already holds tokens keeps the larger scale, and its old codes are moved to it. ``read`` brings requests' tokens back
as bf16 rows. ``decode`` is attention of a few query tokens a request over the cache, ``prompt`` attention of ragged
chunks of a prompt over what is cached of it, the chunk itself among it.
"""

import math

import numpy as np
import torch

own = False

BIAS, LOW, HIGH = 127, 95, 159  # exponent bytes: 2^-32 .. 2^32


# ------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one token for one user, in the middle of a block: nothing but latency
        dict(name="write 1 token 8 heads", kind="write", B=1, lo=1, hi=1, ctx=1000, h_k=8, d=128, page=16, block=16, pad=0),
        # a decode step of 64 requests, each at its own place of its block
        dict(name="write 64 tokens 8 heads", kind="write", B=64, lo=1, hi=1, ctx=600, h_k=8, d=128, page=16, block=16, pad=0),
        # ragged prompt chunks that begin and end inside blocks, head 256, every 9th token a padding token
        dict(name="write 11 ragged chunks", kind="write", B=11, lo=3, hi=701, ctx=300, h_k=4, d=256, page=64, block=32, pad=9),
        # the whole prompts of a batch at once
        dict(name="write 4 x 4096 8 heads", kind="write", B=4, lo=4096, hi=4096, ctx=0, h_k=8, d=128, page=16, block=16, pad=0),
        # a short shared prefix brought back for one request
        dict(name="read 333 tokens", kind="read", B=1, lo=333, hi=333, h_k=8, d=128, page=16, block=16),
        # the cached part of a batch, ragged, for a pass that wants it as rows
        dict(name="read 12 ragged", kind="read", B=12, lo=500, hi=16384, h_k=8, d=128, page=64, block=64),
        # the smallest attention: two short requests that end inside a page
        dict(name="decode 2 short requests", kind="decode", B=2, lo=37, hi=100, q_len=1, h_q=32, h_k=8, d=128, page=16,
             block=16, pad=0, append=False),
        # the 64 x 4096 batch of the decode step with the 32/8 heads of the Qwen3-8B-shaped one
        dict(name="decode 64 x 4096", kind="decode", B=64, lo=4096, hi=4096, q_len=1, h_q=32, h_k=8, d=128, page=16,
             block=16, pad=0, append=False),
        # one request of 131072 tokens: split over the whole GPU and joined
        dict(name="decode 1 x 131072", kind="decode", B=1, lo=131072, hi=131072, q_len=1, h_q=32, h_k=8, d=128, page=64,
             block=64, pad=0, append=False),
        # speculative verify of ragged requests: four query tokens each, written first, then read by the attention; padding requests
        dict(name="verify 4, ragged, written", kind="decode", B=40, lo=200, hi=16384, q_len=4, h_q=32, h_k=8, d=128, page=32,
             block=32, pad=6, append=True),
        # short ragged chunks of several prompts, head 256, nothing cached for some of them
        dict(name="prompt 5 ragged chunks", kind="prompt", B=5, lo=20, hi=700, ctx=1500, h_q=16, h_k=8, d=256, page=64, block=16,
             pad=0, append=True),
        # one long chunk with 12288 tokens before it: the matrix rate bounds it
        dict(name="prompt 4096 after 12288", kind="prompt", B=1, lo=4096, hi=4096, ctx=-12288, h_q=32, h_k=8, d=128, page=16,
             block=16, pad=0, append=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["write", "write", "read", "decode", "decode", "decode", "prompt", "prompt"])
    page = rng.choice([16, 32, 64, 128])
    c = dict(kind=kind, h_k=rng.choice([1, 2, 4, 8]), d=rng.choice([128, 128, 256]), page=page,
             block=rng.choice([b for b in (16, 32, 64, 128) if b <= page]))
    if kind == "write":
        hi = _log(rng, 1, 8192)
        lo = rng.choice([hi, max(1, hi // 7)])
        B = max(1, min(_log(rng, 1, 300), 30000 * 8 * 128 // ((lo + hi) * c["h_k"] * c["d"])))
        return dict(c, B=B, lo=lo, hi=hi, ctx=rng.choice([0, 200, 1000]), pad=rng.choice([0, 0, 5, 17]))
    if kind == "read":
        hi = _log(rng, 1, 32768)
        lo = rng.choice([hi, max(1, hi // 9)])
        return dict(c, B=max(1, min(_log(rng, 1, 100), 160000 * 8 * 128 // ((lo + hi) * c["h_k"] * c["d"]))), lo=lo, hi=hi)
    c["h_q"] = c["h_k"] * rng.choice([1, 2, 4, 5, 8])
    if kind == "decode":
        c["q_len"] = rng.choice([1, 1, 1, 2, 3, 6])
        hi = _log(rng, max(64, c["q_len"]), 131072)
        lo = max(c["q_len"], _log(rng, max(1, hi // 50), hi))
        c.update(B=max(1, min(_log(rng, 1, 200), 800000 // (lo + hi))), lo=lo, hi=hi, append=rng.random() < 0.3)
        c["pad"] = rng.choice([0, 0, 1]) if c["B"] > 2 else 0
        while work(c)["bytes"] > 5.5e8 and c["B"] > 1 + c["pad"]:
            c["B"] -= 1
        return c
    hi = _log(rng, 2, 4096)
    c.update(lo=rng.choice([hi, max(1, hi // 20)]), hi=hi, ctx=rng.choice([0, 0, 100, _log(rng, 1, 30000)]),
             append=rng.random() < 0.3, pad=0)
    c["B"] = max(1, min(_log(rng, 1, 30), 6000 // hi))
    while work(c)["flops"] > 9e11 or _area(c) > 2.2e9:  # no more than the long chunk's, and logits that fit the plain form
        if c["B"] > 1:
            c["B"] -= 1
        else:
            c["ctx"], c["hi"], c["lo"] = c["ctx"] // 2, max(2, c["hi"] * 3 // 4), max(1, c["lo"] * 3 // 4)
    return c


def _lens(c):
    """(tokens cached before the call's own, the call's own tokens) of each request; the same for every seed.
    decode: the new ones are q_len of the length; padding requests, the last, have none."""
    r = np.random.default_rng(c["B"] * 1000003 + c["lo"] * 101 + c["hi"])
    n = r.integers(c["lo"], c["hi"] + 1, c["B"])
    if c["B"] == 2:
        n[:] = c["lo"], c["hi"]
    if c["kind"] == "decode":
        if c["pad"]:
            n[-c["pad"]:] = 0
        new = np.minimum(n, c["q_len"])
        return (n - new).astype(np.int64), new.astype(np.int64)
    ctx = c.get("ctx", 0)
    before = np.full(c["B"], -ctx) if ctx < 0 else r.integers(0, ctx + 1, c["B"])
    if c["kind"] == "prompt" and ctx > 0 and c["B"] > 1:
        before[::3] = 0
    if c["kind"] == "read":
        before[:] = 0
    return before.astype(np.int64), n.astype(np.int64)


def _area(c):
    """Elements of the plain form's logits."""
    before, new = _lens(c)
    return float(c["B"]) * c["h_q"] * float(new.max()) * float((before + new).max())


def work(c):
    before, new = _lens(c)
    row = c["h_k"] * c["d"] * 2  # codes of a token's keys and values
    blocks = 2 * c["h_k"] / c["block"]  # exponent bytes a token
    if c["kind"] == "write":
        T = int(new.sum())
        live = T - (T // c["pad"] if c["pad"] else 0)
        return {"bytes": live * row * 3 + 8 * T + int(live * blocks), "flops": 2 * live * row}
    if c["kind"] == "read":
        T = int(new.sum())
        return {"bytes": T * row * 3 + int(T * blocks) + 4 * T // c["page"], "flops": T * row}
    keys = int((before + new).sum())
    T = int(new.sum())
    b = keys * row + int(keys * blocks) + T * c["h_q"] * c["d"] * 4
    if c["append"]:
        b += T * row * 3
    pairs = int((new * before + new * (new + 1) // 2).sum())
    return {"bytes": b, "flops": 4 * c["h_q"] * c["d"] * pairs}


# ------------------------------------------------------------------------------------------------- the inputs
def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    before, new = _lens(c)
    total = before + new
    B, h_k, d, page, block = c["B"], c["h_k"], c["d"], c["page"], c["block"]
    s = {"c": c, "before": before, "new": new, "total": total}
    per = (total + page - 1) // page
    pages = int(per.sum()) + 2
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    first = torch.from_numpy(np.concatenate([[0], np.cumsum(per)])[:-1]).cuda()
    cols = int(per.max()) + 1
    col = torch.arange(cols, device="cuda")[None]
    table = ids[(first[:, None] + col).clamp(max=pages - 1)]
    s["table"] = torch.where(col < torch.from_numpy(per).cuda()[:, None], table, -1).contiguous()
    s["lens"] = torch.from_numpy(total.astype(np.int32)).cuda()
    # pools as [page, head, token, channel], seen as [page, token, head, channel]; blocks a few binades apart in size
    for name in "kv":
        codes = (rn(pages, h_k, page, d) * 75).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        s[name + "_cache"] = codes.transpose(1, 2)
        s[name + "_exp"] = torch.randint(BIAS - 9, BIAS - 5, (pages, h_k, page // block), generator=g, device="cuda",
                                         dtype=torch.uint8)
    # what lies behind the end of a request's cached tokens is of no value: NaN codes, and any exponent
    at = torch.arange(cols * page, device="cuda")[None]
    held = torch.from_numpy(before if c["kind"] == "write" or c.get("append") else total).cuda()[:, None]
    tail = (at >= held) & (at // page < torch.from_numpy(per).cuda()[:, None])
    pg, row = s["table"][:, :, None].expand(-1, -1, page).reshape(B, -1)[tail].long(), (at % page).expand(B, -1)[tail]
    for name in "kv":
        s[name + "_cache"][pg, row] = 0x7F
        fresh = row % block == 0
        s[name + "_exp"][pg[fresh], :, row[fresh] // block] = 255
    # the call's own tokens: request after request, keys and values strided parts of one projection's output
    T = int(new.sum())
    s["T"] = T
    req = torch.from_numpy(np.repeat(np.arange(B), new)).cuda()
    start = np.concatenate([[0], np.cumsum(new)])
    s["starts"] = torch.from_numpy(start.astype(np.int32)).cuda()
    pos = torch.arange(T, device="cuda") - s["starts"].long()[req] + torch.from_numpy(before).cuda()[req]
    s["req"], s["pos"] = req, pos
    if c["kind"] == "write" or c.get("append"):
        # tokens differ in size, and a few channels stand out, as keys' do
        size = torch.exp2(rn(T, 1, 1) * 0.7) * (1 + 7 * (torch.arange(d, device="cuda") % 61 == 5))
        qkv = (rn(T, 2 * h_k, d) * size).to(torch.bfloat16)
        s["k"], s["v"] = qkv[:, :h_k], qkv[:, h_k:]
        s["slots"] = s["table"][req, pos // page].long() * page + pos % page
        if c["pad"] and c["kind"] == "write":
            s["slots"][c["pad"] - 1::c["pad"]] = -1
    if c["kind"] == "read":
        s["k_rows"] = torch.zeros(T, h_k, d, dtype=torch.bfloat16, device="cuda")
        s["v_rows"] = torch.zeros(T, h_k, d, dtype=torch.bfloat16, device="cuda")
    if c["kind"] in ("decode", "prompt"):
        rows = B * c["q_len"] if c["kind"] == "decode" else T
        s["q"] = (rn(rows, c["h_q"], d) * 1.5).to(torch.bfloat16)
        s["out"] = torch.zeros(rows, c["h_q"], d, dtype=torch.bfloat16, device="cuda")
        s["scale"] = d ** -0.5
    if own:
        _own_args(s)
    return s


def _own_args(s):
    import paged_fp8_decode_gb300 as mj

    c = s["c"]
    kv = mj.BlockKV(s["k_cache"], s["v_cache"], s["k_exp"], s["v_exp"])
    if "slots" in s:
        s["write"] = mj.block_write_args(s["k"], s["v"], s["slots"], kv)
    if c["kind"] == "read":
        s["read"] = mj.block_read_args(kv, s["table"], s["starts"], s["k_rows"], s["v_rows"])
    if c["kind"] == "decode":
        step = mj.BlockStep(max_num_seqs=c["B"], q_len=c["q_len"], h_q=c["h_q"], h_k=c["h_k"], d=c["d"])
        step.plan(s["total"].astype(np.int32), c["B"])
        s["step"], s["attend"] = step, step.args(s["q"], s["out"], kv, s["table"], s["lens"], c["B"], s["scale"])
    if c["kind"] == "prompt":
        step = mj.PromptStep(max_tokens=s["T"], max_num_seqs=c["B"], max_q_len=int(s["new"].max()),
                             max_len=int(s["total"].max()), h_q=c["h_q"], h_k=c["h_k"], d=c["d"])
        s["step"], s["attend"] = step, step.args(s["q"], s["out"], kv, s["table"], s["lens"], s["starts"], c["B"], s["scale"])


# ------------------------------------------------------------------------------------------------- one pass
def _cache_out(s):
    return dict(k=s["k_cache"].view(torch.float8_e4m3fn), v=s["v_cache"].view(torch.float8_e4m3fn), k_exp=s["k_exp"],
                v_exp=s["v_exp"])


def run(s):
    kind = s["c"]["kind"]
    if own:
        import paged_fp8_decode_gb300 as mj

        if "slots" in s:
            mj.mj_block_write_kv(s["write"])
        if kind == "read":
            mj.mj_block_read_kv(s["read"])
        if kind == "decode":
            mj.mj_block_attention(s["attend"])
        if kind == "prompt":
            mj.mj_block_prompt(s["attend"])
    else:
        if "slots" in s:
            _plain_write(s, "k")
            _plain_write(s, "v")
        if kind == "read":
            at = s["table"][s["req"], s["pos"] // s["c"]["page"]].long(), s["pos"] % s["c"]["page"]
            s["k_rows"].copy_(_values(s, "k", *at))
            s["v_rows"].copy_(_values(s, "v", *at))
        if kind == "decode":
            _plain_decode(s)
        if kind == "prompt":
            _plain_prompt(s)
    if kind == "read":
        return dict(k=s["k_rows"], v=s["v_rows"])
    return dict(**({"out": s["out"]} if kind != "write" else {}), **(_cache_out(s) if "slots" in s else {}))


def _plain_write(s, name):
    c, x, cache, exp = s["c"], s[name], s[name + "_cache"], s[name + "_exp"]
    page, block, h_k = c["page"], c["block"], c["h_k"]
    live = s["slots"] >= 0
    slot, x = s["slots"][live], x[live].float()
    blk, which = torch.unique(slot // block, return_inverse=True)  # the blocks that the call writes into
    n = blk.numel()
    big = torch.zeros(n, h_k, device="cuda").scatter_reduce(0, which[:, None].expand(-1, h_k), x.abs().amax(-1), "amax")
    first = torch.full((n,), block, device="cuda").scatter_reduce(0, which, slot % block, "amin")
    m, e = torch.frexp(big)  # big = m 2^e, m in [1/2, 1): the smallest e' with big <= 448 2^e', 448 = 0.875 2^9
    need = torch.where(big > 0, e - 9 + (m > 0.875), -1000).clamp(LOW - BIAS, HIGH - BIAS) + BIAS
    pg, sub = blk * block // page, blk * block % page // block
    old = exp[pg, :, sub].int().clamp(LOW, HIGH)
    now = torch.where(first[:, None] > 0, torch.maximum(old, need), need)  # a block that begins anew forgets
    # the tokens before the call's first in a block move to the larger scale
    row = torch.arange(block, device="cuda")
    rows = (sub * block)[:, None] + row
    codes = cache[pg[:, None], rows]  # [n, block, h_k, d]
    shift = torch.exp2((old - now).float())[:, None, :, None]
    moved = (codes.view(torch.float8_e4m3fn).float() * shift).to(torch.float8_e4m3fn).view(torch.uint8)
    kept = (row < first[:, None])[:, :, None, None] & (now > old)[:, None, :, None]
    cache[pg[:, None], rows] = torch.where(kept, moved, codes)
    exp[pg, :, sub] = now.to(torch.uint8)
    y = x * torch.exp2((BIAS - now).float())[which][:, :, None]
    cache[slot // page, slot % page] = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _values(s, name, pg, row):
    """The values of cached tokens, 32 bits: [..., h_k, d] of pages and rows."""
    e = s[name + "_exp"][pg, :, row // s["c"]["block"]].int().clamp(LOW, HIGH) - BIAS
    return s[name + "_cache"][pg, row].view(torch.float8_e4m3fn).float() * torch.exp2(e.float())[..., None]


def _dense(s, name, n):
    """[B, h_k, n, d]: every request's first n tokens, zeros past its end."""
    key = torch.arange(n, device="cuda")
    pg = s["table"][:, key // s["c"]["page"]].clamp(min=0).long()
    x = _values(s, name, pg, (key % s["c"]["page"])[None].expand_as(pg))
    return torch.where((key[None] < s["lens"][:, None])[:, :, None, None], x, torch.zeros((), device="cuda")).transpose(1, 2)


def _attend(s, q, last):
    """q [B, h_k, m, d] in 32 bits over the cache; row i of request b sees the keys up to last[b, i]."""
    n = int(s["total"].max())
    logit = torch.matmul(q * s["scale"], _dense(s, "k", n).transpose(2, 3))
    see = torch.arange(n, device="cuda") <= last[:, None, :, None]
    logit.masked_fill_(~see, -math.inf)
    top = logit.amax(dim=-1, keepdim=True)
    p = logit.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    weight = p.sum(dim=-1, keepdim=True)
    return torch.matmul(p, _dense(s, "v", n)) / torch.where(weight > 0, weight, torch.ones_like(weight))


def _plain_decode(s):
    c = s["c"]
    B, q_len, h_k, d = c["B"], c["q_len"], c["h_k"], c["d"]
    r = c["h_q"] // h_k
    q = s["q"].float().view(B, q_len, h_k, r, d).transpose(1, 2).reshape(B, h_k, q_len * r, d)
    last = s["lens"].long()[:, None] - q_len + torch.arange(q_len, device="cuda")[None]
    o = _attend(s, q, last.repeat_interleave(r, 1)).view(B, h_k, q_len, r, d).transpose(1, 2)
    old = s["out"].view(B, q_len, h_k, r, d)  # padding requests' rows stay as they were
    s["out"].copy_(torch.where((s["lens"] > 0)[:, None, None, None, None], o.to(torch.bfloat16), old).reshape(s["out"].shape))


def _plain_prompt(s):
    c = s["c"]
    B, h_k, d, T = c["B"], c["h_k"], c["d"], s["T"]
    r, m = c["h_q"] // h_k, int(s["new"].max())
    at = torch.arange(T, device="cuda") - s["starts"].long()[s["req"]]
    q = torch.zeros(B, m, h_k, r, d, device="cuda")
    q[s["req"], at] = s["q"].float().view(T, h_k, r, d)
    last = torch.full((B, m), -1, device="cuda")
    last[s["req"], at] = s["pos"]
    q = q.transpose(1, 2).reshape(B, h_k, m * r, d)
    o = _attend(s, q, last.repeat_interleave(r, 1)).view(B, h_k, m, r, d).transpose(1, 2)
    s["out"].copy_(o[s["req"], at].reshape(T, c["h_q"], d))


# ------------------------------------------------------------------------------------------------- in 64 bits
def _exact_write(s, name):
    """(codes before their rounding as numbers, exponents): block after block on the host's list of them."""
    c = s["c"]
    page, block = c["page"], c["block"]
    want = s[name + "_cache"].view(torch.float8_e4m3fn).double()
    exps = s[name + "_exp"].clone()
    slots = s["slots"].cpu().numpy()
    live = np.nonzero(slots >= 0)[0]
    of = slots[live] // block
    edges = np.concatenate([[0], np.nonzero(np.diff(of))[0] + 1, [live.size]])
    x = s[name].double()
    size = x.abs().amax(-1).cpu().numpy()  # [T, h_k]
    old = exps.cpu().numpy().astype(np.int64).clip(LOW, HIGH)
    new = exps.cpu().numpy()
    moves = []
    for a, b in zip(edges[:-1], edges[1:]):
        t = live[a:b]
        pg, sub, first = slots[t[0]] // page, slots[t[0]] % page // block, int((slots[t] % block).min())
        amax = size[t].max(0)
        with np.errstate(divide="ignore"):
            need = np.where(amax > 0, np.ceil(np.log2(amax / 448)), -1000).clip(LOW - BIAS, HIGH - BIAS).astype(np.int64) + BIAS
        now = np.maximum(need, old[pg, :, sub]) if first else need
        if first and (now > old[pg, :, sub]).any():
            moves.append((int(pg), int(sub) * block, first, old[pg, :, sub] - now))
        new[pg, :, sub] = now
    for pg, at, first, by in moves:
        want[pg, at:at + first] *= torch.from_numpy(2.0 ** np.minimum(by, 0)).cuda()[None, :, None]
    now = torch.from_numpy(new).cuda()
    t = torch.from_numpy(live).cuda()
    sl = s["slots"][t]
    e = now[sl // page, :, sl % page // block].double() - BIAS
    want[sl // page, sl % page] = (x[t] / torch.pow(2.0, e)[:, :, None]).clamp(-448.0, 448.0)
    return want, now


def exact(c, seed):
    s = prepare(c, seed)
    page, block, h_k = c["page"], c["block"], c["h_k"]
    given = {}
    held = {}
    for name in "kv":
        codes, exps = s[name + "_cache"].view(torch.float8_e4m3fn), s[name + "_exp"]
        if "slots" in s:
            given[name], exps = _exact_write(s, name)
            given[name + "_exp"] = exps
            codes = given[name].to(torch.float32).to(torch.float8_e4m3fn)  # the attention reads what was rounded
        held[name] = codes.view(torch.uint8), exps

    def rows(name, b, n):
        at = torch.arange(n, device="cuda")
        pg = s["table"][b].long()[at // page]
        codes, exps = held[name]
        e = exps[pg, :, at % page // block].double().clamp(LOW, HIGH) - BIAS
        return codes[pg, at % page].view(torch.float8_e4m3fn).double() * torch.pow(2.0, e)[..., None]

    if c["kind"] == "write":
        return given
    if c["kind"] == "read":
        whole = [[rows(name, b, int(s["total"][b])) for b in range(c["B"])] for name in "kv"]
        return dict(k=torch.cat(whole[0]), v=torch.cat(whole[1]))
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    r = c["h_q"] // h_k
    start = s["starts"].cpu().numpy() if c["kind"] == "prompt" else np.arange(c["B"]) * c["q_len"]
    for b in range(c["B"]):
        n, m = int(s["total"][b]), int(s["new"][b])
        if not n:
            continue
        k, v = rows("k", b, n), rows("v", b, n)
        skip = c["q_len"] - m if c["kind"] == "decode" else 0  # query tokens that no key reaches
        hidden = torch.arange(n, device="cuda")[None] > (torch.arange(m, device="cuda") + n - m)[:, None]
        q = s["q"][start[b] + skip:start[b] + skip + m].double()
        for h in range(c["h_q"]):
            logit = (q[:, h] @ k[:, h // r].t() * s["scale"]).masked_fill(hidden, -math.inf)
            out[start[b] + skip:start[b] + skip + m, h] = torch.softmax(logit, dim=-1) @ v[:, h // r]
    return dict(out=out, **given)
