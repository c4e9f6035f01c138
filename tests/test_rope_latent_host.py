"""The rotated writes and the latent attention on the host: the turns, the
latent plan, the refusals (no call here reaches a launch), and the pins of
their oracle."""

import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_fp8_decode_gb300 as mj
from oracle import rope as OR


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_fp8_decode_gb300.build import build

    build()


# ---------------------------------------------------------------- the oracle's pins
def test_angles_against_float64_products():
    inv = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    pos = np.array([0, 1, 7, 4095, 123456])
    got = OR.angles(pos, inv)
    want = pos[:, None] * inv[None]
    # the float64 product is off by 2^-53 of itself, the reduction by less
    assert np.allclose(np.cos(got), np.cos(want), rtol=0, atol=1e-10)
    assert np.allclose(np.sin(got), np.sin(want), rtol=0, atol=1e-10)


def test_rotation_keeps_lengths_and_relative_positions():
    rng = np.random.default_rng(3)
    inv = 100.0 ** (-np.arange(0, 32, 2) / 32)
    q, k = rng.normal(size=(1, 1, 48)), rng.normal(size=(1, 1, 48))
    for inter in (False, True):
        dots = []
        for a, b in ((5, 2), (1005, 1002)):
            x = OR.rotate(q, OR.angles([a], inv), inter)
            y = OR.rotate(k, OR.angles([b], inv), inter)
            assert np.isclose((x ** 2).sum(), (q ** 2).sum())
            assert np.array_equal(x[..., 32:], q[..., 32:])
            dots.append((x * y).sum())
        assert np.isclose(dots[0], dots[1], rtol=0, atol=1e-9)


def test_rotation_by_hand():
    x = np.arange(1.0, 5.0).reshape(1, 1, 4)
    ang = np.array([[np.pi / 2, np.pi]])
    assert np.allclose(OR.rotate(x, ang, False)[0, 0], [-3, -2, 1, -4])
    assert np.allclose(OR.rotate(x, ang, True)[0, 0], [-2, 1, -3, -4])
    assert np.allclose(OR.rotate(x, ang, True, 2.0)[0, 0], [-4, 2, -6, -8])


def test_angles_take_their_axis():
    pos = np.array([[1, 2], [10, 20]])
    got = OR.angles(pos, [0.01, 0.02, 0.03], freq_axis=[1, 0, 7])
    assert np.allclose(got, [[0.1, 0.02, 0.3], [0.2, 0.04, 0.6]])


def test_latent_oracle_by_hand():
    # two keys, one aligned with the query: weights e^2 : 1
    rows = np.zeros((2, 576))
    rows[0, 512], rows[0, 0], rows[1, 0] = 2.0, 1.0, -1.0
    q = np.zeros((2, 1, 576))
    q[:, :, 512] = 1.0
    out, lse = OR.latent_attention(q, rows, 1.0, 2, True)
    e2 = np.exp(2.0)
    assert np.isclose(out[1, 0, 0], (e2 - 1) / (e2 + 1)) and np.isclose(lse[1, 0], np.log(e2 + 1))
    assert np.isclose(out[0, 0, 0], 1.0) and np.isclose(lse[0, 0], 2.0)  # the first token sees one key
    out, lse = OR.latent_attention(np.repeat(q, 2, axis=0), rows, 1.0, 2, True)
    assert not out[:2].any() and np.all(np.isneginf(lse[:2]))  # four tokens, two keys: two see none


# ---------------------------------------------------------------- turns
def test_turns_are_the_nearest_fractions():
    rng = np.random.default_rng(0)
    f = np.concatenate([10.0 ** rng.uniform(-9, 6, 300), [1.0, 0.0, -1.0, -0.37, 1e-300, 5e-324, 1048576.0, 2 * np.pi]])
    got = mj.mj_rope_turns(f).numpy().view(np.uint64)
    for a, t in zip(f, got):
        v = Fraction(abs(float(a))) / (2 * OR.PI) * 2 ** 64
        want = int(v + Fraction(1, 2)) % 2 ** 64
        if a < 0:
            want = -want % 2 ** 64
        assert int(t) == want, a


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan, 2097152.0])
def test_turns_refuse(bad):
    with pytest.raises(mj.MjError) as e:
        mj.mj_rope_turns([1.0, bad])
    assert e.value.status == mj.MJ_ERR_INVALID_ARG


# ---------------------------------------------------------------- the plan
def plan_parts(plan, slots, max_num_seqs):
    split_words = (2 * max_num_seqs + 3) // 4 * 4
    table = plan[:4 * slots].reshape(-1, 4)
    splits = plan[4 * slots:4 * slots + 2 * max_num_seqs].reshape(-1, 2)
    work = plan[4 * slots + split_words:4 * slots + split_words + 4 * (slots + max_num_seqs)].reshape(-1, 4)
    # the slots' rows follow each other; a slot's entry repeats its first row's request and tile
    off = [0]
    for first, end, b, tile in table:
        if end > first:
            assert first == off[-1] and (b, tile) == tuple(work[first][:2])
        else:
            assert not (first or end or b or tile)
        off.append(max(off[-1], int(end)))
    return np.array(off), splits, work


def check_plan(lens, slots, max_num_seqs, margin, plan):
    off, splits, work = plan_parts(plan, slots, max_num_seqs)
    assert off[0] == 0 and np.all(np.diff(off) >= 0) and off[-1] <= len(work)
    rows = work[:off[-1]]
    at, parts = 0, []
    for b, n in enumerate(lens):
        tiles = -(-(int(n) + margin) // 128) if n > 0 else 0
        mine = []
        while at < len(rows) and rows[at][0] == b:
            mine.append(rows[at])
            at += 1
        # contiguous pieces, none empty, that cover the tiles
        edges = [0] + [int(w[2]) for w in mine]
        assert [int(w[1]) for w in mine] == edges[:-1] and edges[-1] == tiles
        assert all(w[2] > w[1] for w in mine)
        if len(mine) > 1:
            assert splits[b][1] == len(mine)
            assert [int(w[3]) for w in mine] == list(range(splits[b][0], splits[b][0] + len(mine)))
            parts += [int(w[3]) for w in mine]
        else:
            assert splits[b][1] == 0 and all(w[3] == -1 for w in mine)
    assert at == len(rows)
    assert sorted(parts) == list(range(len(parts))) and len(parts) <= 2 * slots
    return off, rows


@pytest.mark.parametrize("seed", range(60))
def test_plan_covers_every_tile_once(seed):
    rng = np.random.default_rng(seed)
    n = int(rng.integers(0, 60))
    lens = rng.integers(0, [300, 5000, 200000][seed % 3], size=n).astype(np.int32)
    lens[rng.random(n) < 0.1] = 0
    slots, margin = int(rng.choice([1, 2, 9, 38, 76, 152])), int(rng.integers(0, 4))
    extra = int(rng.integers(0, 5))
    h, cost = [(16, 1), (32, 3), (128, 5)][seed // 3 % 3]
    plan = mj.mj_latent_plan(lens, n, n + extra, slots, 1, h, margin)
    off, rows = check_plan(lens, slots, n + extra, margin, plan)
    # balance: no slot holds more than what an even cut of all rows would give, and a row's cost
    held = [sum(int(w[2] - w[1]) + cost for w in rows[off[s]:off[s + 1]]) for s in range(slots)]
    tiles = sum(-(-(int(x) + margin) // 128) for x in lens if x)
    if tiles:
        assert max(held) <= (tiles + cost * (int((lens > 0).sum()) + slots)) / slots + 2 + cost


def test_plan_of_one_long_request_fills_the_slots():
    plan = mj.mj_latent_plan(np.array([131072], np.int32), 1, 1, 152, 1, 16)
    off, rows = check_plan([131072], 152, 1, 0, plan)
    assert len(rows) >= 140 and max(int(w[2] - w[1]) for w in rows) == 7


def test_plan_refusals():
    with pytest.raises(mj.MjError):
        mj.mj_latent_plan(np.array([5, -1], np.int32), 2, 2, 4, 1, 16)
    with pytest.raises(mj.MjError):
        mj.mj_latent_plan(np.array([5, 1], np.int32), 2, 1, 4, 1, 16)
    with pytest.raises(mj.MjError):
        mj.mj_latent_plan(np.array([5], np.int32), 1, 1, 0, 1, 16)
    for q_len, h in ((0, 16), (1, 0)):
        with pytest.raises(mj.MjError):
            mj.mj_latent_plan(np.array([5], np.int32), 1, 1, 4, q_len, h)
    with pytest.raises(ValueError):
        mj.mj_latent_plan(np.array([5], np.int32), 1, 1, 4, 1, 16, plan_out=np.zeros(8, np.int32))
    with pytest.raises(ValueError):
        mj.mj_latent_plan(np.array([5], np.int32), 2, 2, 4, 1, 16)
    lib, lens, out = mj.load_library(), np.array([5], np.int32), np.zeros(64, np.int32)
    assert lib.mj_latent_plan(lens.ctypes.data, 1, 1, 4, 1, 16, 0, out.ctypes.data, 8) == mj.MJ_ERR_CAPACITY
    # a length that its margin takes past 32 bits
    lens[0] = 2 ** 31 - 2
    assert lib.mj_latent_plan(lens.ctypes.data, 1, 1, 4, 1, 16, 5, out.ctypes.data, 64) == mj.MJ_ERR_INVALID_ARG


def test_slots_and_sizes():
    assert mj.mj_latent_slots(152, 1, 16) == 152
    assert mj.mj_latent_slots(152, 1, 64) == 152
    assert mj.mj_latent_slots(152, 1, 128) == 76
    assert mj.mj_latent_slots(152, 5, 128) == 15
    assert mj.mj_latent_slots(4, 8, 128) == 1
    assert mj.mj_latent_plan_size(152, 10) % 4 == 0
    assert mj.mj_latent_workspace_size(10, 2, 3) == 256 + 2 * 10 * 16 * 514 * 4
    assert mj.mj_latent_workspace_size(10, 5, 13) == 256 + 2 * 10 * 128 * 514 * 4


# ---------------------------------------------------------------- refusals of the C calls
BASE = 1 << 40  # fake, never dereferenced


def rope(a, rot):
    a.positions, a.axis_stride, a.num_axes, a.turns, a.rot_dim, a.scale = BASE, 0, 1, BASE + 0x100, rot, 1.0


def rope_write():
    a = mj.mj_rope_write_kv_args()
    rope(a.rope, 128)
    a.h_q, a.q, a.q_tok_stride, a.q_head_stride = 8, BASE + 0x1000, 1024, 128
    a.q_out, a.q_out_tok_stride, a.q_out_head_stride = BASE + 0x9000, 1024, 128
    w = a.kv
    w.num_tokens, w.h_k, w.d = 3, 2, 128
    w.key, w.value, w.slot_mapping = BASE + 0x11000, BASE + 0x12000, BASE + 0x13000
    w.key_tok_stride, w.key_head_stride, w.value_tok_stride, w.value_head_stride = 256, 128, 256, 128
    w.kv_format, w.page_size, w.num_pages = 0, 16, 4
    w.k_cache, w.v_cache = BASE + 0x20000, BASE + 0x30000
    w.k_stride_page, w.k_stride_token, w.k_stride_head = 4096, 128, 2048
    w.v_stride_page, w.v_stride_token, w.v_stride_head = 4096, 128, 2048
    w.k_scale, w.v_scale = BASE + 0x14000, BASE + 0x14100
    return a


def latent_write():
    a = mj.mj_latent_write_args()
    rope(a.rope, 64)
    a.num_tokens, a.h = 3, 8
    a.q_pe, a.q_tok_stride, a.q_head_stride = BASE + 0x1000, 512, 64
    a.q_out, a.q_out_tok_stride, a.q_out_head_stride = BASE + 0x9000, 512, 64
    a.latent, a.latent_tok_stride, a.k_pe, a.k_pe_tok_stride = BASE + 0x11000, 576, BASE + 0x11400, 576
    a.slot_mapping, a.page_size, a.num_pages = BASE + 0x13000, 16, 4
    a.cache, a.stride_page, a.stride_token, a.scale = BASE + 0x20000, 9216, 576, BASE + 0x14000
    return a


def latent():
    a = mj.mj_latent_args()
    a.num_seqs, a.max_num_seqs, a.q_len, a.h, a.causal, a.softmax_scale = 2, 2, 1, 8, 1, 0.07
    a.q, a.q_tok_stride, a.q_head_stride = BASE, 4608, 576
    a.cache, a.stride_page, a.stride_token, a.page_size, a.num_pages = BASE + 0x20000, 9216, 576, 16, 4
    a.descale, a.block_table, a.block_table_stride, a.seq_lens = BASE + 0x10000, BASE + 0x11000, 8, BASE + 0x12000
    a.block_table_len = 8
    a.plan, a.slots = BASE + 0x13000, 4
    a.out, a.out_tok_stride, a.out_head_stride, a.out_dtype = BASE + 0x14000, 4096, 512, 0
    a.workspace, a.workspace_bytes = BASE + 0x40000, mj.mj_latent_workspace_size(4, 1, 8)
    return a


def set_path(a, path, value):
    *outer, last = path.split(".")
    for p in outer:
        a = getattr(a, p)
    setattr(a, last, value)


I, U, A, C = mj.MJ_ERR_INVALID_ARG, mj.MJ_ERR_UNSUPPORTED, mj.MJ_ERR_ALIGNMENT, mj.MJ_ERR_CAPACITY
ROPE_BAD = [("rope.positions", None, I), ("rope.turns", None, I), ("rope.num_axes", 0, I), ("rope.num_axes", 5, I),
            ("rope.num_axes", 2, I), ("rope.rot_dim", 0, U), ("rope.rot_dim", 24, U), ("rope.rot_dim", 272, U),
            ("rope.scale", float("nan"), I), ("rope.positions", BASE + 4, A), ("rope.turns", BASE + 4, A),
            ("rope.axis_stride", -1, I), ("q_tok_stride", 12, A), ("q_out_head_stride", 4, A), ("q_out", BASE + 8, A),
            ("q_out", None, I), ("q_head_stride", -8, I)]


@pytest.mark.parametrize("path,value,status", ROPE_BAD + [
    ("h_q", -1, I), ("q", None, I), ("q", BASE + 2, A), ("kv.key", None, I), ("kv.d", 64, U), ("kv.page_size", 8, U),
    ("kv.kv_format", 4, U), ("kv.k_stride_token", 24, A), ("kv.value_tok_stride", 4, A), ("kv.num_tokens", -1, I),
    ("kv.slot_mapping", None, I), ("kv.v_scale", None, I), ("rope.rot_dim", 144, U)])
def test_rope_write_refusals(path, value, status):
    a = rope_write()
    set_path(a, path, value)
    assert mj.load_library().mj_rope_write_kv(ctypes.byref(a), None) == status


@pytest.mark.parametrize("path,value,status", ROPE_BAD + [
    ("h", -1, I), ("q_pe", None, I), ("q_pe", BASE + 2, A), ("latent", None, I), ("k_pe", None, I), ("cache", None, I),
    ("scale", None, I), ("slot_mapping", None, I), ("latent", BASE + 8, A), ("k_pe_tok_stride", 4, A),
    ("stride_token", 584, A), ("stride_page", -16, I), ("page_size", 48, U), ("num_tokens", -1, I), ("rope.rot_dim", 80, U),
    ("status", BASE + 2, A)])
def test_latent_write_refusals(path, value, status):
    a = latent_write()
    set_path(a, path, value)
    assert mj.load_library().mj_latent_write(ctypes.byref(a), None) == status


@pytest.mark.parametrize("path,value,status", [
    ("num_seqs", -1, I), ("num_seqs", 3, I), ("q_len", 0, I), ("h", 0, I), ("slots", 0, I), ("page_size", 256, U),
    ("num_pages", 0, I), ("num_pages", 1 << 31, I), ("softmax_scale", 0.0, I), ("softmax_scale", float("inf"), I),
    ("softmax_scale", float("nan"), I), ("out_dtype", 2, U), ("q", None, I), ("cache", None, I), ("descale", None, I),
    ("block_table", None, I), ("seq_lens", None, I), ("plan", None, I), ("out", None, I), ("workspace", None, I),
    ("q", BASE + 8, A), ("cache", BASE + 8, A), ("out", BASE + 2, A), ("workspace", BASE + 4, A), ("lse", BASE + 2, A),
    ("q_tok_stride", 12, A), ("out_head_stride", 4, A), ("stride_token", 560, I), ("stride_token", 584, A),
    ("stride_page", 0, I), ("workspace_bytes", 256, C), ("block_table_stride", -1, I), ("block_table_len", -1, I)])
def test_latent_attention_refusals(path, value, status):
    a = latent()
    set_path(a, path, value)
    assert mj.load_library().mj_latent_attention(ctypes.byref(a), None) == status


@pytest.mark.parametrize("path,value", [("stride_token", 560), ("stride_token", 0), ("stride_page", 560), ("stride_page", 0)])
def test_latent_write_refuses_rows_that_overlap(path, value):
    a = latent_write()
    set_path(a, path, value)
    a.rope.scale = 1.0
    a.latent_tok_stride = 4  # (stops a call that passed the check, by another status)
    assert mj.load_library().mj_latent_write(ctypes.byref(a), None) == I


def test_more_tokens_than_a_launch_indexes_are_refused():
    lib = mj.load_library()
    a, b = rope_write(), latent_write()
    a.kv.num_tokens, a.kv.h_k, b.num_tokens = (1 << 30) + 1, 1, (1 << 30) + 1
    a.kv.slot_mapping = b.slot_mapping = None  # (a call that passed the limit would stop here, by another status)
    a.rope.rot_dim = b.rope.rot_dim = 24
    assert lib.mj_rope_write_kv(ctypes.byref(a), None) == mj.MJ_ERR_CAPACITY
    assert lib.mj_latent_write(ctypes.byref(b), None) == mj.MJ_ERR_CAPACITY


def test_workspace_of_more_rows_than_the_attention_takes_is_refused():
    lib, n = mj.load_library(), ctypes.c_size_t(0)
    assert lib.mj_latent_workspace_size(152, 8192, 128, ctypes.byref(n)) == mj.MJ_OK
    assert lib.mj_latent_workspace_size(152, 8193, 128, ctypes.byref(n)) == I
    assert lib.mj_latent_workspace_size(2**31 - 1, 2**31 - 1, 2**31 - 1, ctypes.byref(n)) == I


def test_nothing_to_do_is_ok():
    lib = mj.load_library()
    a, b, c = rope_write(), latent_write(), latent()
    a.kv.num_tokens, b.num_tokens, c.num_seqs = 0, 0, 0
    assert lib.mj_rope_write_kv(ctypes.byref(a), None) == mj.MJ_OK
    assert lib.mj_latent_write(ctypes.byref(b), None) == mj.MJ_OK
    assert lib.mj_latent_attention(ctypes.byref(c), None) == mj.MJ_OK
    for fn in (lib.mj_rope_write_kv, lib.mj_latent_write, lib.mj_latent_attention):
        assert fn(None, None) == mj.MJ_ERR_INVALID_ARG


# ---------------------------------------------------------------- refusals of the binding
def test_builders_refuse_host_tensors():
    T = 2
    key = torch.zeros(T, 1, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="key"):
        mj.rope_write_args(None, key, key, torch.zeros(T, dtype=torch.int64), mj.mj_rope_turns([1.0] * 8),
                           torch.zeros(T, dtype=torch.int64), key, key, (0, 0, 0), 16, 1, 0, key, key)
    with pytest.raises(ValueError, match="latent"):
        mj.latent_write_args(None, torch.zeros(T, 512, dtype=torch.bfloat16), key, key, key, key, key, key)


def test_a_launch_on_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for fn, a in ((mj.mj_rope_write_kv, rope_write()), (mj.mj_latent_write, latent_write()),
                  (mj.mj_latent_attention, latent())):
        a.device_index = 1
        with pytest.raises(ValueError, match="cuda:1"):
            fn(a)
