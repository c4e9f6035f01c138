"""The rotated cache writes and the latent-cache attention: their cases, their plain forms and the framework's calls.

Three operators. ``rope_write`` rotates the new tokens' queries and keys by their positions and appends keys and
values to the paged cache that the decode step reads. ``latent_write`` appends one latent row a token (512 latent
codes and 64 rotated ones) and rotates the queries' rotary part. ``latent`` is decode attention over those rows, in
the absorbed form: every query head reads the same 576-wide key, and the first 512 channels of it are the value.
"""

import math

import numpy as np
import torch

own = False

LAT, ROPE = 512, 64
ROW = LAT + ROPE


# ------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one token for one user: the smallest append there is, nothing but latency
        dict(name="append 1 token 32/8", kind="rope_write", T=1, h_q=32, h_k=8, d=128, rot=128, axes=1, inter=False,
             per_head=True, page=16, pad=0, far=4096),
        # a decode step of 64 requests with the 32/8 heads of the Qwen3-8B-shaped step, one scale per KV head
        dict(name="append 64 tokens 32/8", kind="rope_write", T=64, h_q=32, h_k=8, d=128, rot=128, axes=1, inter=False,
             per_head=True, page=16, pad=0, far=8192),
        # a prompt chunk with positions of three axes (time, height, width), head 256, half of it rotated, adjacent
        # pairs, an odd number of tokens, every 7th a padding token
        dict(name="append 1501 image tokens", kind="rope_write", T=1501, h_q=16, h_k=8, d=256, rot=128, axes=3, inter=True,
             per_head=False, page=64, pad=7, far=40000),
        # a whole prompt of a batch at once, positions up to a million
        dict(name="append 16384 tokens 32/8", kind="rope_write", T=16384, h_q=32, h_k=8, d=128, rot=128, axes=1,
             inter=False, per_head=True, page=16, pad=0, far=1000000),
        # one decode step of 40 requests (8 of them padding), 128 heads
        dict(name="latent append 40 tokens", kind="latent_write", T=40, H=128, axes=1, inter=True, page=64, pad=5, far=163840),
        # a prompt chunk, 16 heads, odd length
        dict(name="latent append 8191 tokens", kind="latent_write", T=8191, H=16, axes=1, inter=True, page=64, pad=0,
             far=131072),
        # the smallest attention: two short requests that end inside a page
        dict(name="latent 2 short requests", kind="latent", B=2, lo=37, hi=100, q_len=1, H=8, page=16, pad=0, append=False),
        # the 64 x 4096 batch with 16 heads a GPU: the cache stream bounds it
        dict(name="latent 64 x 4096, 16 heads", kind="latent", B=64, lo=4096, hi=4096, q_len=1, H=16, page=64, pad=0,
             append=False),
        # one request of 131072 tokens: split over the whole GPU and joined
        dict(name="latent 131072, 16 heads", kind="latent", B=1, lo=131072, hi=131072, q_len=1, H=16, page=64, pad=0,
             append=False),
        # all 128 heads on one GPU, ragged lengths: the matrix rate bounds it
        dict(name="latent ragged, 128 heads", kind="latent", B=48, lo=1024, hi=16384, q_len=1, H=128, page=64, pad=0,
             append=False),
        # speculative verify: four query tokens each, causal, 32 requests and 8 padding ones, page 32
        dict(name="latent verify 4 x 16 heads", kind="latent", B=40, lo=1024, hi=16384, q_len=4, H=16, page=32, pad=8,
             append=False),
        # the two as one step: the new token's row is written, then read by the attention
        dict(name="latent step, 32 heads", kind="latent", B=96, lo=300, hi=5000, q_len=1, H=32, page=128, pad=0,
             append=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope_write", "latent_write", "latent", "latent"])
    if kind == "rope_write":
        d = rng.choice([128, 256])
        h_k = rng.choice([1, 2, 4, 8])
        h_q = h_k * rng.choice([1, 2, 4, 5, 8])
        T = min(_log(rng, 1, 16384), 16000 * (32 * 4 + 8 * 6) * 128 // ((h_q * 4 + h_k * 6) * d))
        axes = rng.choice([1, 1, 2, 3])
        return dict(kind=kind, T=T, h_q=h_q, h_k=h_k, d=d, rot=rng.choice([d, d // 2, 32, d - 16]), axes=axes,
                    inter=rng.random() < 0.5, per_head=rng.random() < 0.5, page=rng.choice([16, 32, 64, 128]),
                    pad=rng.choice([0, 0, 3, 11]), far=_log(rng, 64, 1000000))
    if kind == "latent_write":
        H = rng.randint(1, 128)
        return dict(kind=kind, T=min(_log(rng, 1, 8192), 8192 * 40 // (24 + H)), H=H, axes=rng.choice([1, 1, 3]),
                    inter=rng.random() < 0.7, page=rng.choice([16, 32, 64, 128]), pad=rng.choice([0, 0, 4]),
                    far=_log(rng, 64, 200000))
    q_len = rng.choice([1, 1, 1, 2, 3, 5])
    H = rng.choice([rng.randint(1, 16), rng.randint(1, 64), rng.randint(1, 128), 128])
    if q_len * H > 128:
        q_len = max(1, 128 // H)
    hi = _log(rng, max(64, q_len), 131072)
    lo = max(q_len, _log(rng, max(1, hi // 50), hi))
    B = max(1, min(_log(rng, 1, 200), 800000 // (lo + hi)))
    c = dict(kind=kind, B=B, lo=lo, hi=hi, q_len=q_len, H=H, page=rng.choice([16, 32, 64, 128]),
             pad=rng.choice([0, 0, 1]) if B > 2 else 0, append=rng.random() < 0.3)
    while work(c)["flops"] > 1.07e11:  # no more than the ragged 128-head case's
        c["B"] -= 1
    return c


def _lens(c):
    """The requests' lengths (the last `pad` are padding requests of length 0); the same for every seed."""
    r = np.random.default_rng(c["B"] * 1000003 + c["lo"] * 101 + c["hi"])
    n = c["B"] - c["pad"]
    if c["B"] == 2 and c["pad"] == 0:
        live = np.array([c["lo"], c["hi"]])
    else:
        live = r.integers(c["lo"], c["hi"] + 1, n)
    return np.concatenate([live, np.zeros(c["pad"], np.int64)]).astype(np.int32)


def work(c):
    if c["kind"] == "rope_write":
        live = c["T"] if not c["pad"] else c["T"] - len(range(c["pad"] - 1, c["T"], c["pad"]))
        return {"bytes": c["T"] * (c["h_q"] * c["d"] * 4 + 8 * (c["axes"] + 1)) + live * 2 * c["h_k"] * c["d"] * 3,
                "flops": 3 * c["T"] * (c["h_q"] + c["h_k"]) * c["rot"]}
    if c["kind"] == "latent_write":
        live = c["T"] if not c["pad"] else c["T"] - len(range(c["pad"] - 1, c["T"], c["pad"]))
        return {"bytes": c["T"] * (c["H"] * ROPE * 4 + 8 * (c["axes"] + 1)) + live * ROW * 3,
                "flops": 3 * c["T"] * (c["H"] + 1) * ROPE}
    lens = _lens(c).astype(np.int64)
    rows = c["q_len"] * c["H"]
    n = int((lens > 0).sum())
    b = int(lens.sum()) * ROW + n * rows * (ROW + LAT) * 2
    if c["append"]:
        b += n * (ROW * 3 + rows * ROPE * 2)
    return {"bytes": b, "flops": 2 * rows * int(lens.sum()) * (ROW + LAT)}


# ------------------------------------------------------------------------------------------------- the inputs
def _inv_freq(rot, base=1000000.0):
    """The usual geometric frequencies, 64 bits, on the host (a program makes them once)."""
    return torch.pow(torch.tensor(base, dtype=torch.float64), -torch.arange(0, rot, 2, dtype=torch.float64) / rot)


def _axis_table(n, axes):
    """The axis of each frequency: contiguous sections, the first the longest where they do not divide."""
    return torch.tensor([min(axes - 1, i * axes // n) for i in range(n)], dtype=torch.uint8)


def _positions(g, axes, T, far):
    p = torch.randint(0, far, (axes, T), generator=g, device="cuda")
    return p[0].contiguous() if axes == 1 else p


def _slots(g, T, pad, slots):
    s = torch.randperm(slots, generator=g, device="cuda")[:T]
    if pad:
        s[pad - 1::pad] = -1
    return s


def _old_codes(g, *shape):
    """Cache contents before the call: codes of normal values."""
    return (torch.randn(*shape, generator=g, device="cuda") * 64).to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rn(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    s = {"c": c}
    if c["kind"] == "rope_write":
        T, h_q, h_k, d, page = c["T"], c["h_q"], c["h_k"], c["d"], c["page"]
        pages = (T + page - 1) // page + 3
        qkv = rn(T, h_q + 2 * h_k, d)  # one projection's output: q, k and v are strided views of it
        s["q"], s["k"], s["v"] = qkv[:, :h_q], qkv[:, h_q:h_q + h_k], qkv[:, h_q + h_k:]
        s["inv"] = _inv_freq(c["rot"])
        s["axis"] = _axis_table(c["rot"] // 2, c["axes"]).cuda()
        s["pos"] = _positions(g, c["axes"], T, c["far"])
        s["slots"] = _slots(g, T, c["pad"], pages * page)
        s["k_scale"] = (torch.rand(h_k if c["per_head"] else 1, generator=g, device="cuda") + 0.5) * (5 / 448)
        s["v_scale"] = (torch.rand(h_k if c["per_head"] else 1, generator=g, device="cuda") + 0.5) * (5 / 448)
        s["q_out"] = torch.zeros(T, h_q, d, dtype=torch.bfloat16, device="cuda")
        s["k_cache"], s["v_cache"] = _old_codes(g, pages, h_k, page, d), _old_codes(g, pages, h_k, page, d)
        s["scale"] = 1.0 if c["axes"] == 1 else 1.0625
        s["inv_dev"] = s["inv"].cuda()
        if own:
            import paged_fp8_decode_gb300 as mj

            s["args"] = mj.rope_write_args(
                s["q"], s["k"], s["v"], s["pos"], mj.mj_rope_turns(s["inv"]).cuda(), s["slots"], s["k_cache"],
                s["v_cache"], (h_k * page * d, d, page * d), page, pages, mj.MJ_KV_E4M3, s["k_scale"], s["v_scale"],
                q_out=s["q_out"], freq_axis=s["axis"] if c["axes"] > 1 else None, interleaved=c["inter"],
                rope_scale=s["scale"], scale_per_head=c["per_head"])
    elif c["kind"] == "latent_write":
        T, H, page = c["T"], c["H"], c["page"]
        pages = (T + page - 1) // page + 3
        kv = rn(T, ROW)  # the down-projection's output: latent and rotary part side by side
        _latent_inputs(s, g, kv[:, :LAT], kv[:, LAT:], T, H, c["axes"], c["far"], rn)
        s["slots"] = _slots(g, T, c["pad"], pages * page)
        s["cache"] = _old_codes(g, pages, page, ROW)
        if own:
            s["args"] = _latent_write_args(s, c["inter"])
    else:
        B, q_len, H, page = c["B"], c["q_len"], c["H"], c["page"]
        lens = _lens(c)
        per = [(int(n) + page - 1) // page for n in lens]
        pages = sum(per) + 2
        ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((B, max(per) + 1), -1, dtype=torch.int32, device="cuda")
        edge = np.concatenate([[0], np.cumsum(per)])
        col = torch.arange(max(per) + 1, device="cuda")[None]
        n = torch.tensor(per, device="cuda")[:, None]
        first = torch.tensor(edge[:-1], device="cuda")[:, None]
        table = torch.where(col < n, ids[(first + col).clamp(max=pages - 1)], table)
        s["table"], s["lens"], s["host_lens"] = table.contiguous(), torch.from_numpy(lens).cuda(), lens
        s["max_len"] = int(lens.max())
        s["descale"] = torch.tensor([6 / 448, 9 / 448], device="cuda")
        s["cache"] = (torch.randn(pages, page, ROW, generator=g, device="cuda") * 75).clamp(-448, 448).to(
            torch.float8_e4m3fn).view(torch.uint8)
        # the unwritten end of each request's last page holds NaN codes
        last = torch.tensor([max(0, e - 1) for e in edge[1:]], device="cuda")
        used = torch.from_numpy(lens.astype(np.int64)).cuda() % page
        tail = (torch.arange(page, device="cuda")[None] >= used[:, None]) & (used[:, None] > 0)
        at = ids[last].long()[:, None].expand(B, page)[tail], torch.arange(page, device="cuda")[None].expand(B, page)[tail]
        s["cache"][at] = 0x7F
        s["q"] = rn(B * q_len, H, ROW)
        s["out"] = torch.zeros(B * q_len, H, LAT, dtype=torch.bfloat16, device="cuda")
        s["softmax_scale"] = 192 ** -0.5
        if c["append"]:
            # the newest q_len tokens of every request are written by the call
            T = B * q_len
            kv = rn(T, ROW)
            _latent_inputs(s, g, kv[:, :LAT], kv[:, LAT:], T, H, 1, 0, rn)
            p = (s["lens"].long()[:, None] - q_len + torch.arange(q_len, device="cuda")[None])
            s["pos"] = p.clamp(min=0).reshape(-1).contiguous()
            pg = torch.gather(table.long(), 1, (p.clamp(min=0) // page))
            s["slots"] = torch.where(p >= 0, pg * page + p.clamp(min=0) % page, -1).reshape(-1).contiguous()
            s["q_out"] = s["q"][:, :, LAT:]
        if own:
            import paged_fp8_decode_gb300 as mj

            step = mj.LatentStep(max_num_seqs=B, q_len=q_len, h=H)
            step.plan(lens, B)
            kv = mj.PagedLatent(cache=s["cache"], descale=s["descale"], block_table=s["table"], seq_lens=s["lens"])
            s["step"], s["args"] = step, step.args(s["q"], s["out"], kv, B, s["softmax_scale"])
            if c["append"]:
                s["write_args"] = _latent_write_args(s, True)
    return s


def _latent_inputs(s, g, latent, pe, T, H, axes, far, rn):
    s["latent"], s["pe"] = latent, pe
    s["q_pe"] = rn(T, H, 128 + ROPE)[:, :, 128:]  # the query projection's heads: a part without positions, then this
    s["inv"] = _inv_freq(ROPE, 10000.0)
    s["inv_dev"] = s["inv"].cuda()
    s["axis"] = _axis_table(ROPE // 2, axes).cuda()
    if far:
        s["pos"] = _positions(g, axes, T, far)
    s["axes"] = axes
    if "descale" not in s:
        s["descale"] = torch.tensor([6 / 448, 9 / 448], device="cuda")
    if "q_out" not in s:
        s["q"] = torch.zeros(T, H, ROW, dtype=torch.bfloat16, device="cuda")  # the absorbed query: its last 64 are written
        s["q_out"] = s["q"][:, :, LAT:]


def _latent_write_args(s, inter):
    import paged_fp8_decode_gb300 as mj

    return mj.latent_write_args(s["q_pe"], s["latent"], s["pe"], s["pos"], mj.mj_rope_turns(s["inv"]).cuda(), s["slots"],
                                s["cache"], s["descale"], q_out=s["q_out"],
                                freq_axis=s["axis"] if s["axes"] > 1 else None, interleaved=inter)


# ------------------------------------------------------------------------------------------------- one pass
def run(s):
    if own:
        return _run_own(s)
    kind = s["c"]["kind"]
    if kind == "rope_write":
        return _plain_rope_write(s)
    if kind == "latent_write":
        return _plain_latent_write(s, s["c"]["inter"])
    if s["c"]["append"]:
        _plain_latent_write(s, True)
    return dict(out=_plain_latent(s), **({"cache": s["cache"].view(torch.float8_e4m3fn)} if s["c"]["append"] else {}))


def _run_own(s):
    import paged_fp8_decode_gb300 as mj

    kind = s["c"]["kind"]
    if kind == "rope_write":
        mj.mj_rope_write_kv(s["args"])
        return dict(q=s["q_out"], k=s["k_cache"].view(torch.float8_e4m3fn), v=s["v_cache"].view(torch.float8_e4m3fn))
    if kind == "latent_write":
        mj.mj_latent_write(s["args"])
        return dict(q=s["q_out"], cache=s["cache"].view(torch.float8_e4m3fn))
    if s["c"]["append"]:
        mj.mj_latent_write(s["write_args"])
    mj.mj_latent_attention(s["args"])
    return dict(out=s["out"], **({"cache": s["cache"].view(torch.float8_e4m3fn)} if s["c"]["append"] else {}))


def _cos_sin(pos, inv, axis):
    """Cosine and sine [T, rot / 2] of position times frequency, the product in 64 bits (far positions)."""
    p = pos if pos.dim() == 2 else pos[None]
    a = p.double()[axis.long()].t() * inv[None]
    return torch.cos(a).float(), torch.sin(a).float()


def _rotate(x, cos, sin, inter, scale):
    """x [T, heads, d]: its first 2 * n channels rotated, in 32 bits."""
    n = cos.shape[1]
    x = x.float()
    r, rest = x[..., :2 * n], x[..., 2 * n:]
    c, s = cos[:, None] * scale, sin[:, None] * scale
    if inter:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    else:
        a, b = r[..., :n], r[..., n:]
        r = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    return torch.cat([r, rest], dim=-1)


def _codes(x, scale):
    """e4m3 codes of x / scale, saturating."""
    return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_rope_write(s):
    c = s["c"]
    cos, sin = _cos_sin(s["pos"], s["inv_dev"], s["axis"])
    s["q_out"].copy_(_rotate(s["q"], cos, sin, c["inter"], s["scale"]))
    k = _codes(_rotate(s["k"], cos, sin, c["inter"], s["scale"]), s["k_scale"][None, :, None])
    v = _codes(s["v"].float(), s["v_scale"][None, :, None])
    live = s["slots"] >= 0
    page, row = s["slots"][live] // c["page"], s["slots"][live] % c["page"]
    s["k_cache"][page, :, row] = k[live]
    s["v_cache"][page, :, row] = v[live]
    return dict(q=s["q_out"], k=s["k_cache"].view(torch.float8_e4m3fn), v=s["v_cache"].view(torch.float8_e4m3fn))


def _plain_latent_write(s, inter):
    cos, sin = _cos_sin(s["pos"], s["inv_dev"], s["axis"])
    s["q_out"].copy_(_rotate(s["q_pe"], cos, sin, inter, 1.0))
    pe = _rotate(s["pe"][:, None], cos, sin, inter, 1.0)[:, 0]
    row = torch.cat([_codes(s["latent"].float(), s["descale"][0]), _codes(pe, s["descale"][1])], dim=1)
    live = s["slots"] >= 0
    at = s["slots"][live]
    page = s["cache"].shape[1]
    s["cache"][at // page, at % page] = row[live]
    return dict(q=s["q_out"], cache=s["cache"].view(torch.float8_e4m3fn))


def _visible(s, n):
    """[B, q_len, n]: which keys each query token of each request sees."""
    c = s["c"]
    lens = s["lens"].long()
    key = torch.arange(n, device="cuda")
    last = lens[:, None] - c["q_len"] + torch.arange(c["q_len"], device="cuda")[None]
    return (key[None, None] <= last[:, :, None]) & (key[None, None] < lens[:, None, None])


def _plain_latent(s):
    c = s["c"]
    B, q_len, H = c["B"], c["q_len"], c["H"]
    n, page = s["max_len"], s["cache"].shape[1]
    key = torch.arange(n, device="cuda")
    pg = s["table"][:, key // page].clamp(min=0).long()  # [B, n]
    held = key[None] < s["lens"][:, None]
    rows = s["cache"][pg, key[None] % page].view(torch.float8_e4m3fn).float()
    rows = torch.where(held[:, :, None], rows, torch.zeros((), device="cuda"))
    lat, pe = rows[..., :LAT] * s["descale"][0], rows[..., LAT:] * s["descale"][1]
    q = s["q"].float().view(B, q_len * H, ROW)
    logit = (torch.bmm(q[..., :LAT], lat.transpose(1, 2)) + torch.bmm(q[..., LAT:], pe.transpose(1, 2))) * s["softmax_scale"]
    see = _visible(s, n)[:, :, None].expand(B, q_len, H, n).reshape(B, q_len * H, n)
    logit = torch.where(see, logit, torch.full((), -math.inf, device="cuda"))
    top = logit.amax(dim=-1, keepdim=True)
    p = torch.exp(logit - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = p.sum(dim=-1, keepdim=True)
    o = torch.bmm(p, lat) / torch.where(total > 0, total, torch.ones_like(total))
    live = (s["lens"] > 0)[:, None, None, None]  # padding requests: their rows stay as they were
    new = o.view(B, q_len, H, LAT).to(torch.bfloat16)
    s["out"].copy_(torch.where(live, new, s["out"].view(B, q_len, H, LAT)).view(B * q_len, H, LAT))
    return s["out"]


# ------------------------------------------------------------------------------------------------- in 64 bits
def _exact_turn(x, pos, inv, axis, inter, scale):
    """The rotation as a product of complex numbers: x [T, heads, d] in 64 bits."""
    p = pos if pos.dim() == 2 else pos[None]
    n = inv.numel()
    T = x.shape[0]
    angle = torch.empty(T, n, dtype=torch.float64, device="cuda")
    for a in range(p.shape[0]):
        mine = (axis == a).nonzero()[:, 0]
        angle[:, mine] = torch.outer(p[a].double(), inv[mine])
    w = torch.polar(torch.full_like(angle, scale), angle)[:, None]
    x = x.double().clone()
    if inter:
        z = torch.view_as_complex(x[..., :2 * n].reshape(T, x.shape[1], n, 2).contiguous()) * w
        x[..., :2 * n] = torch.view_as_real(z).reshape(T, x.shape[1], 2 * n)
    else:
        z = torch.complex(x[..., :n].contiguous(), x[..., n:2 * n].contiguous()) * w
        x[..., :n], x[..., n:2 * n] = z.real, z.imag
    return x


def exact(c, seed):
    s = prepare(c, seed)
    if c["kind"] == "rope_write":
        q = _exact_turn(s["q"], s["pos"], s["inv_dev"], s["axis"], c["inter"], s["scale"])
        k = _exact_turn(s["k"], s["pos"], s["inv_dev"], s["axis"], c["inter"], s["scale"])
        caches = []
        for x, sc, cache in ((k, s["k_scale"], s["k_cache"]), (s["v"].double(), s["v_scale"], s["v_cache"])):
            want = cache.view(torch.float8_e4m3fn).double()
            per = sc.double() if sc.numel() > 1 else sc.double().expand(c["h_k"])
            val = torch.clamp(x / per[None, :, None], -448.0, 448.0)
            hold = s["slots"] >= 0
            flat = want.transpose(1, 2).reshape(-1, c["h_k"], c["d"])  # one row a slot
            flat[s["slots"][hold]] = val[hold]
            caches.append(flat.view(want.shape[0], c["page"], c["h_k"], c["d"]).transpose(1, 2).contiguous())
        return dict(q=q, k=caches[0], v=caches[1])
    q_all, cache = s["q"].double(), None
    if c["kind"] == "latent_write" or c["append"]:
        inter = c.get("inter", True)
        q_pe = _exact_turn(s["q_pe"], s["pos"], s["inv_dev"], s["axis"], inter, 1.0)
        pe = _exact_turn(s["pe"][:, None], s["pos"], s["inv_dev"], s["axis"], inter, 1.0)[:, 0]
        row = torch.cat([s["latent"].double() / s["descale"][0].double(), pe / s["descale"][1].double()], dim=1)
        cache = s["cache"].view(torch.float8_e4m3fn).double().reshape(-1, ROW)
        hold = s["slots"] >= 0
        cache[s["slots"][hold]] = row[hold].clamp(-448.0, 448.0)
        cache = cache.view(s["cache"].shape)
        if c["kind"] == "latent_write":
            return dict(q=q_pe, cache=cache)
        # the attention reads what the write rounded: bf16 queries and the codes held in the cache
        q_all[..., LAT:] = q_pe.to(torch.bfloat16).double()
    # the attention, request by request
    B, q_len, H, page = c["B"], c["q_len"], c["H"], c["page"]
    held = (cache.to(torch.float32).to(torch.float8_e4m3fn) if cache is not None else s["cache"].view(torch.float8_e4m3fn))
    held = held.view(torch.uint8).reshape(-1, ROW)
    out = torch.zeros(B * q_len, H, LAT, dtype=torch.float64, device="cuda")
    fold = torch.cat([s["descale"][:1].double().expand(LAT), s["descale"][1:].double().expand(ROPE)])
    for b in range(B):
        n = int(s["host_lens"][b])
        if not n:
            continue
        at = torch.arange(n, device="cuda")
        slot = s["table"][b].long()[at // page] * page + at % page
        key = held[slot].view(torch.float8_e4m3fn).double() * fold
        for t in range(q_len):
            seen = max(0, n - q_len + t + 1)
            if seen:
                logit = q_all[b * q_len + t] @ key[:seen].t() * s["softmax_scale"]
                out[b * q_len + t] = torch.softmax(logit, dim=-1) @ key[:seen, :LAT]
    return dict(out=out, **({"cache": cache} if c["append"] else {}))
