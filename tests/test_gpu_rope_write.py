"""The rotated cache writes on the GPU against float64 (oracle.rope).

Tolerances. A rotated value y = m (x0 cos a - x1 sin a) is formed in float32
from exact bf16 x0, x1: cos and sin (of an angle below 2^-31 half turns off)
are within 2^-23 of their size or so, times m one more rounding, two products
and a sum: below 2^-20 m (|x0| + |x1|) in all. Queries add bf16's half step,
2^-8 of the value. A key's code must be a nearest one of the exact quotient up
to that slack (over the scale) and the division's 2^-24. Values are not
rotated: bit-exact, like every byte that the call must leave alone."""

import numpy as np
import pytest
import torch

from oracle import formats as F
from oracle import kvwrite as OW
from oracle import rope as OR

pytestmark = pytest.mark.gpu

SLACK = 2.0 ** -20


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_fp8_decode_gb300.build import build

    build()


def grid_values(fmt):
    decode, codes = {"fp8": (F.e4m3_decode, range(256)), "e2m3": (F.e2m3_decode, range(64)),
                     "e3m2": (F.e3m2_decode, range(64)), "e2m1": (F.e2m1_decode, range(16))}[fmt]
    v = decode(np.array(list(codes), np.uint8)).astype(np.float64)
    return np.sort(v[np.isfinite(v)])


def unpack(rows, fmt):
    if fmt == "fp8":
        return F.e4m3_decode(rows).astype(np.float64)
    if fmt == "e2m1":
        return F.e2m1_decode(F.fp4_unpack_rows(rows)).astype(np.float64)
    return (F.e2m3_decode if fmt == "e2m3" else F.e3m2_decode)(F.fp6_unpack_rows(rows)).astype(np.float64)


def nearest_gap(y, grid):
    """Distance of each y to the nearest value of the grid."""
    i = np.clip(np.searchsorted(grid, y), 1, len(grid) - 1)
    return np.minimum(np.abs(y - grid[i - 1]), np.abs(y - grid[i]))


def bf16(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16)


CASES = [
    dict(T=1, h_q=1, h_k=1, d=128, rot=16, inter=False, fmt="fp8"),
    dict(T=1, h_q=32, h_k=8, d=128, rot=128, inter=False, fmt="fp8"),
    dict(T=67, h_q=8, h_k=2, d=128, rot=128, inter=False, fmt="fp8", pad=5, head_scale=True),
    dict(T=67, h_q=8, h_k=2, d=128, rot=64, inter=True, fmt="fp8", axes=3, nhd=True),
    dict(T=130, h_q=5, h_k=1, d=256, rot=240, inter=False, fmt="fp8", axes=2, head_scale=True, inplace=True),
    dict(T=33, h_q=0, h_k=3, d=256, rot=256, inter=True, fmt="fp8", pad=2),
    dict(T=1000, h_q=1, h_k=1, d=128, rot=112, inter=True, fmt="fp8", axes=4),  # several tokens a CTA
    dict(T=700, h_q=40, h_k=8, d=256, rot=256, inter=False, fmt="fp8", nhd=True),
    dict(T=41, h_q=4, h_k=2, d=128, rot=128, inter=False, fmt="e2m3"),
    dict(T=41, h_q=4, h_k=2, d=128, rot=32, inter=True, fmt="e3m2", pad=3),
    dict(T=41, h_q=4, h_k=2, d=128, rot=96, inter=False, fmt="e2m1", nhd=True),
    dict(T=21, h_q=2, h_k=2, d=256, rot=64, inter=True, fmt="e2m1", scale=0.5),
    dict(T=19, h_q=2, h_k=2, d=256, rot=256, inter=False, fmt="e2m3", axes=3),
]


def make(c, seed):
    rng = np.random.default_rng(seed)
    T, h_q, h_k, d, fmt = c["T"], c["h_q"], c["h_k"], c["d"], c["fmt"]
    axes, ps = c.get("axes", 1), 16
    pages = T // ps + 3
    rb = OW.row_bytes(d, {"fp8": 0, "e2m3": 1, "e3m2": 2, "e2m1": 3}[fmt])
    strides = (ps * h_k * rb, h_k * rb, rb) if c.get("nhd") else (h_k * ps * rb, rb, ps * rb)
    w = dict(c, pages=pages, ps=ps, strides=strides, rb=rb)
    qkv = bf16(rng, T, h_q + 2 * h_k, d)
    w["q"], w["k"], w["v"] = qkv[:, :h_q], qkv[:, h_q:h_q + h_k], qkv[:, h_q + h_k:]
    w["inv"] = 500000.0 ** (-np.arange(0, c["rot"], 2) / c["rot"])
    pos = rng.integers(0, [100, 40000, 2 ** 40][seed % 3], size=(axes, T))
    pos[:, 0] = 0
    pos[:, T // 2] = -7  # a negative position turns backwards
    w["pos"] = pos if axes > 1 else pos[0]
    w["axis"] = rng.integers(0, axes, size=c["rot"] // 2).astype(np.uint8)
    if axes > 1:
        w["axis"][-1] = 200  # past the last axis: the last
    slots = rng.permutation(pages * ps)[:T].astype(np.int64)
    if c.get("pad"):
        slots[::c["pad"]] = -1
    w["slots"] = slots
    n = h_k * d if fmt != "fp8" else (h_k if c.get("head_scale") else 1)
    top = {"fp8": 448, "e2m3": 7.5, "e3m2": 28, "e2m1": 6}[fmt]
    shape = (h_k, d) if fmt != "fp8" else (n,)
    # some values saturate
    w["ks"], w["vs"] = ((rng.uniform(1.5, 5, n) / top).astype(np.float32).reshape(shape) for _ in range(2))
    w["kp"], w["vp"] = (rng.integers(0, 256, pages * ps * h_k * rb).astype(np.uint8) for _ in range(2))
    return w


def call(w, status=None, stream=None):
    import paged_fp8_decode_gb300 as mj

    dev = "cuda"
    T, h_q, h_k = w["T"], w["h_q"], w["h_k"]
    qkv = torch.cat([w["q"], w["k"], w["v"]], dim=1).to(dev)  # q, k, v: strided views of one buffer
    q, k, v = qkv[:, :h_q], qkv[:, h_q:h_q + h_k], qkv[:, h_q + h_k:]
    big = torch.full((T, h_q + 1, w["d"] + 8), 7.0, dtype=torch.bfloat16, device=dev)
    q_out = None if h_q == 0 else (q if w.get("inplace") else big[:, :h_q, :w["d"]])
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    kp, vp = up(w["kp"]), up(w["vp"])
    a = mj.rope_write_args(q if h_q else None, k, v, up(w["pos"]), mj.mj_rope_turns(w["inv"]).to(dev), up(w["slots"]),
                           kp, vp, w["strides"], w["ps"], w["pages"], mj.KV_FORMATS[w["fmt"]], up(w["ks"]), up(w["vs"]),
                           q_out=q_out, freq_axis=up(w["axis"]) if w.get("axes", 1) > 1 else None,
                           interleaved=w["inter"], rope_scale=w.get("scale", 1.0),
                           scale_per_head=bool(w.get("head_scale")), status=status)
    mj.mj_rope_write_kv(a, stream)
    torch.cuda.synchronize()
    if h_q and not w.get("inplace"):  # nothing outside q_out was written
        assert bool((big[:, h_q:] == 7).all()) and bool((big[:, :, w["d"]:] == 7).all())
    return (q_out.double().cpu().numpy() if h_q else None), kp.cpu().numpy(), vp.cpu().numpy()


def amplitude(x, ang, inter, scale):
    """|x0| + |x1| of each channel's pair (its own |x| where it is not rotated), times the scale."""
    one = np.abs(OR.rotate(np.abs(x), np.zeros_like(ang), inter))
    n = ang.shape[1]
    amp = one.copy()
    if inter:
        s = one[..., 0:2 * n:2] + one[..., 1:2 * n:2]
        amp[..., 0:2 * n:2], amp[..., 1:2 * n:2] = s * scale, s * scale
    else:
        s = one[..., :n] + one[..., n:2 * n]
        amp[..., :n], amp[..., n:2 * n] = s * scale, s * scale
    return amp


def check_rotated(w, q_out, kp, vp):
    scale = w.get("scale", 1.0)
    ang = OR.angles(w["pos"], w["inv"], w["axis"] if w.get("axes", 1) > 1 else None)
    if w["h_q"]:
        x = w["q"].double().numpy()
        want = OR.rotate(x, ang, w["inter"], scale)
        tol = 2.0 ** -8 * np.abs(want) + SLACK * amplitude(x, ang, w["inter"], scale)
        assert np.all(np.abs(q_out - want) <= tol)
    fmt, h_k, d, ps = w["fmt"], w["h_k"], w["d"], w["ps"]
    code = {"fp8": 0, "e2m3": 1, "e3m2": 2, "e2m1": 3}[fmt]
    # values, and every byte that no live slot covers: exact (keys are checked below)
    okp, ovp = w["kp"].copy(), w["vp"].copy()
    OW.write_kv(w["k"].float().numpy(), w["v"].float().numpy(), okp, ovp, w["slots"], ps, w["strides"], w["strides"], code,
                w["ks"], w["vs"])
    assert np.array_equal(vp, ovp)
    x = w["k"].double().numpy()
    want = OR.rotate(x, ang, w["inter"], scale)
    amp = amplitude(x, ang, w["inter"], scale)
    grid = grid_values(fmt)
    touched = np.zeros(kp.size, bool)
    for t, s in enumerate(w["slots"]):
        if s < 0:
            continue
        for h in range(h_k):
            off = (s // ps) * w["strides"][0] + (s % ps) * w["strides"][1] + h * w["strides"][2]
            touched[off:off + w["rb"]] = True
            got = unpack(kp[off:off + w["rb"]][None], fmt)[0]
            sc = (w["ks"][h] if w["ks"].ndim == 2 else w["ks"][h if w["ks"].size > 1 else 0]).astype(np.float64)
            y = np.clip(want[t, h] / sc, grid[0], grid[-1])
            slack = SLACK * amp[t, h] / sc + 2.0 ** -24 * np.abs(y)
            assert np.all(np.abs(got - y) <= nearest_gap(y, grid) + 2 * slack)
    assert np.array_equal(kp[~touched], w["kp"][~touched])


@pytest.mark.parametrize("i", range(len(CASES)))
def test_rope_write(i):
    w = make(CASES[i], i)
    check_rotated(w, *call(w))


def test_zero_positions_equal_the_plain_write():
    import paged_fp8_decode_gb300 as mj

    w = make(CASES[2], 5)
    w["pos"][:] = 0
    _, kp, vp = call(w)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    k2, v2 = up(w["kp"]), up(w["vp"])
    mj.mj_write_kv(w["k"].cuda(), w["v"].cuda(), up(w["slots"]), k2, v2, w["strides"], w["ps"], w["pages"], 0, up(w["ks"]),
                   up(w["vs"]), scale_per_head=True)
    assert np.array_equal(kp, k2.cpu().numpy()) and np.array_equal(vp, v2.cpu().numpy())


def test_slot_past_the_pool_is_skipped_and_reported():
    w = make(CASES[2], 6)
    w["slots"][4] = w["pages"] * w["ps"]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = call(w, status)
    w["slots"][4] = -1
    check_rotated(w, *out)
    assert int(status.item()) == 1


def test_no_tokens_and_no_live_token():
    import paged_fp8_decode_gb300 as mj

    w = make(CASES[2], 9)
    w["slots"][:] = -1
    check_rotated(w, *call(w))  # queries rotated, caches as they were
    z = torch.zeros(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(0, dtype=torch.int64, device="cuda")
    pool = torch.full((4096,), 9, dtype=torch.uint8, device="cuda")
    one = torch.ones(1, device="cuda")
    mj.mj_rope_write_kv(mj.rope_write_args(z, z, z, i, mj.mj_rope_turns([1.0] * 8).cuda(), i, pool, pool,
                                           (4096, 128, 2048), 16, 1, 0, one, one))
    torch.cuda.synchronize()
    assert bool((pool == 9).all())


def test_nan_and_infinite_inputs_stay_in_their_pairs():
    w = make(CASES[1], 7)
    w["q"][0, 3, 5] = float("inf")
    w["q"][0, 4, 9] = float("nan")
    w["slots"][:] = 0
    q_out, _, _ = call(w)
    bad = ~np.isfinite(q_out[0])
    assert set(zip(*np.nonzero(bad))) <= {(3, 5), (3, 69), (4, 9), (4, 73)}
    assert bad[4, 9] and bad[4, 73]


def test_captured_and_replayed_on_another_stream():
    import paged_fp8_decode_gb300 as mj

    w = make(CASES[2], 8)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    q, k, v = (w[n].cuda().contiguous() for n in "qkv")
    pos, kp, vp = up(w["pos"]), up(w["kp"]), up(w["vp"])
    q_out = torch.empty_like(q)
    a = mj.rope_write_args(q, k, v, pos, mj.mj_rope_turns(w["inv"]).cuda(), up(w["slots"]), kp, vp, w["strides"], w["ps"],
                           w["pages"], 0, up(w["ks"]), up(w["vs"]), q_out=q_out, scale_per_head=True)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        mj.mj_rope_write_kv(a)
    for step in range(3):
        w["pos"] = w["pos"] + step
        pos.copy_(torch.from_numpy(w["pos"]))
        g.replay()
        torch.cuda.synchronize()
        check_rotated(w, q_out.double().cpu().numpy(), kp.cpu().numpy(), vp.cpu().numpy())


# ---------------------------------------------------------------- latent rows
@pytest.mark.parametrize("T,h,inter,axes,pad,pitch,ps", [
    (1, 1, True, 1, 0, 576, 16), (1, 128, True, 1, 0, 576, 64), (130, 16, True, 1, 7, 640, 64), (77, 0, False, 3, 0, 576, 32),
    (400, 3, False, 2, 0, 592, 128), (900, 128, True, 1, 0, 576, 64)])
def test_latent_write(T, h, inter, axes, pad, pitch, ps):
    import paged_fp8_decode_gb300 as mj

    rng = np.random.default_rng(T + h)
    pages = T // ps + 2
    kv = bf16(rng, T, 576)
    q = bf16(rng, T, h, 192)
    inv = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    pos = rng.integers(0, 200000, size=(axes, T))
    axis = rng.integers(0, axes, 32).astype(np.uint8)
    slots = rng.permutation(pages * ps)[:T].astype(np.int64)
    if pad:
        slots[::pad] = -1
    pool = rng.integers(0, 256, (pages, ps, pitch)).astype(np.uint8)
    scale = np.array([3.0 / 448, 2.5 / 448], np.float32)  # some values saturate
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    cache = up(pool)
    kvd, qd = kv.cuda(), q.cuda()
    q576 = torch.full((T, h, 576), 3.0, dtype=torch.bfloat16, device="cuda")
    posd = up(pos if axes > 1 else pos[0])
    a = mj.latent_write_args(qd[:, :, 128:] if h else None, kvd[:, :512], kvd[:, 512:], posd, mj.mj_rope_turns(inv).cuda(),
                             up(slots), cache[:, :, :576], up(scale), q_out=q576[:, :, 512:] if h else None,
                             freq_axis=up(axis) if axes > 1 else None, interleaved=inter)
    mj.mj_latent_write(a)
    torch.cuda.synchronize()
    ang = OR.angles(pos if axes > 1 else pos[0], inv, axis if axes > 1 else None)
    if h:
        x = q[:, :, 128:].double().numpy()
        want = OR.rotate(x, ang, inter)
        tol = 2.0 ** -8 * np.abs(want) + SLACK * amplitude(x, ang, inter, 1.0)
        assert np.all(np.abs(q576[:, :, 512:].double().cpu().numpy() - want) <= tol)
        assert bool((q576[:, :, :512] == 3).all())
    got = cache.cpu().numpy()
    live = np.nonzero(slots >= 0)[0]
    rows = got.reshape(pages * ps, pitch)[slots[live]]
    lat = F.e4m3_encode((kv[:, :512].float().numpy() / scale[0]).astype(np.float32))
    assert np.array_equal(rows[:, :512], lat[live])
    x = kv[:, None, 512:].double().numpy()
    grid = grid_values("fp8")
    y = np.clip(OR.rotate(x, ang, inter)[live, 0] / float(scale[1]), -448, 448)
    slack = SLACK * amplitude(x, ang, inter, 1.0)[live, 0] / float(scale[1]) + 2.0 ** -24 * np.abs(y)
    assert np.all(np.abs(F.e4m3_decode(rows[:, 512:576]) - y) <= nearest_gap(y, grid) + 2 * slack)
    rest = got.reshape(pages * ps, pitch).copy()
    rest[slots[live], :576] = pool.reshape(pages * ps, pitch)[slots[live], :576]
    assert np.array_equal(rest, pool.reshape(pages * ps, pitch))
