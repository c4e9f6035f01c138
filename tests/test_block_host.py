"""The block-scaled cache on the host: what the calls refuse before they touch the device, what the
plan covers, what the argument builders check."""

import ctypes

import numpy as np
import pytest
import torch

import paged_fp8_decode_gb300 as mj
from tests.test_latent_calls_host import on_gpu

BASE = 1 << 40  # never dereferenced

# (a call that passed the checks would stop at the launch, which needs a GPU; on one it must not get there)
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are not real")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_fp8_decode_gb300.build import build

    build()


def cache(c):
    c.h_k, c.d, c.page_size, c.block, c.num_pages = 2, 128, 32, 16, 4
    c.k_cache, c.v_cache, c.k_exp, c.v_exp = BASE, BASE + (1 << 20), BASE + (2 << 20), BASE + (3 << 20)
    for w in "kv":
        for n, x in (("stride_page", 8192), ("stride_token", 128), ("stride_head", 4096), ("exp_stride_page", 4), ("exp_stride_head", 2)):
            setattr(c, f"{w}_{n}", x)


def write():
    a = mj.mj_block_write_args()
    cache(a.cache)
    a.num_tokens, a.key, a.value, a.slot_mapping = 5, BASE + (4 << 20), BASE + (5 << 20), BASE + (6 << 20)
    a.key_tok_stride = a.value_tok_stride = 256
    a.key_head_stride = a.value_head_stride = 128
    return a


def read():
    a = mj.mj_block_read_args()
    cache(a.cache)
    a.num_seqs, a.num_rows, a.block_table, a.block_table_stride, a.block_table_len = 2, 7, BASE + (7 << 20), 4, 4
    a.starts, a.k_out, a.v_out = BASE + (8 << 20), BASE + (9 << 20), BASE + (10 << 20)
    a.k_tok_stride = a.v_tok_stride = 256
    a.k_head_stride = a.v_head_stride = 128
    return a


def attend(q_len=1):
    a = mj.mj_block_args()
    cache(a.cache)
    a.num_seqs, a.max_num_seqs, a.q_len, a.h_q, a.causal, a.softmax_scale = 2, 3, q_len, 8, 1, 0.1
    a.q, a.q_tok_stride, a.q_head_stride = BASE + (11 << 20), 1024, 128
    a.block_table, a.block_table_stride, a.block_table_len, a.seq_lens = BASE + (7 << 20), 4, 4, BASE + (12 << 20)
    a.plan, a.slots = BASE + (13 << 20), 5
    a.out, a.out_tok_stride, a.out_head_stride = BASE + (14 << 20), 1024, 128
    a.workspace, a.workspace_bytes = BASE + (15 << 20), mj.mj_block_workspace_size(5, q_len, 8, 2, 128)
    return a


def prompt(splits=2):
    a = mj.mj_block_prompt_args()
    cache(a.cache)
    a.num_seqs, a.num_tokens, a.max_q_len, a.splits, a.h_q, a.causal, a.softmax_scale = 2, 9, 6, splits, 8, 1, 0.1
    a.q, a.q_tok_stride, a.q_head_stride, a.q_starts = BASE + (11 << 20), 1024, 128, BASE + (16 << 20)
    a.block_table, a.block_table_stride, a.block_table_len, a.seq_lens = BASE + (7 << 20), 4, 4, BASE + (12 << 20)
    a.out, a.out_tok_stride, a.out_head_stride = BASE + (14 << 20), 1024, 128
    a.workspace, a.workspace_bytes = BASE + (15 << 20), mj.mj_block_prompt_workspace_size(9, 8, 128, splits)
    return a


CALLS = {"mj_block_write_kv": write, "mj_block_read_kv": read, "mj_block_attention": attend, "mj_block_prompt": prompt}


def call(fn, a):
    return getattr(mj.load_library(), fn)(ctypes.byref(a), None)


def with_(a, path, value):
    o = a
    *way, last = path.split(".")
    for p in way:
        o = getattr(o, p)
    setattr(o, last, value)
    return a


@no_gpu
@pytest.mark.parametrize("fn", list(CALLS))
def test_valid_arguments_pass_the_checks(fn):
    # past every check: no GPU to launch on (the attentions: no driver to describe the cache to)
    assert call(fn, CALLS[fn]()) in (mj.MJ_ERR_CUDA, mj.MJ_ERR_UNSUPPORTED)
    assert getattr(mj.load_library(), fn)(None, None) == mj.MJ_ERR_INVALID_ARG


@no_gpu
@pytest.mark.parametrize("fn", list(CALLS))
@pytest.mark.parametrize("field,value,status", [
    ("h_k", 0, mj.MJ_ERR_INVALID_ARG), ("num_pages", 0, mj.MJ_ERR_INVALID_ARG), ("num_pages", 1 << 31, mj.MJ_ERR_UNSUPPORTED),
    ("d", 64, mj.MJ_ERR_UNSUPPORTED), ("d", 192, mj.MJ_ERR_UNSUPPORTED), ("page_size", 24, mj.MJ_ERR_UNSUPPORTED),
    ("block", 8, mj.MJ_ERR_UNSUPPORTED), ("block", 64, mj.MJ_ERR_INVALID_ARG), ("k_cache", None, mj.MJ_ERR_INVALID_ARG),
    ("v_exp", None, mj.MJ_ERR_INVALID_ARG), ("v_cache", BASE + 8, mj.MJ_ERR_ALIGNMENT), ("k_stride_token", 136, mj.MJ_ERR_ALIGNMENT),
    ("v_stride_page", -8192, mj.MJ_ERR_INVALID_ARG), ("k_exp_stride_head", -1, mj.MJ_ERR_INVALID_ARG)])
def test_caches_are_refused(fn, field, value, status):
    assert call(fn, with_(CALLS[fn](), "cache." + field, value)) == status


@no_gpu
@pytest.mark.parametrize("field,value", [("k_stride_token", 112), ("v_stride_head", 128), ("k_stride_page", 4096), ("v_stride_page", 0),
                                         ("k_exp_stride_head", 1), ("v_exp_stride_page", 2), ("k_exp_stride_page", 0)])
def test_writes_refuse_rows_and_exponents_that_overlap(field, value):
    assert call("mj_block_write_kv", with_(write(), "cache." + field, value)) == mj.MJ_ERR_INVALID_ARG


@no_gpu
@pytest.mark.parametrize("fn,field,value,status", [
    ("mj_block_write_kv", "num_tokens", -1, mj.MJ_ERR_INVALID_ARG), ("mj_block_write_kv", "num_tokens", (1 << 30) + 1, mj.MJ_ERR_CAPACITY),
    ("mj_block_write_kv", "key", None, mj.MJ_ERR_INVALID_ARG), ("mj_block_write_kv", "value", BASE + 2, mj.MJ_ERR_ALIGNMENT),
    ("mj_block_write_kv", "key_tok_stride", 260, mj.MJ_ERR_ALIGNMENT), ("mj_block_write_kv", "slot_mapping", None, mj.MJ_ERR_INVALID_ARG),
    ("mj_block_write_kv", "slot_mapping", BASE + 4, mj.MJ_ERR_ALIGNMENT), ("mj_block_write_kv", "status", BASE + 2, mj.MJ_ERR_ALIGNMENT),
    ("mj_block_read_kv", "num_seqs", -1, mj.MJ_ERR_INVALID_ARG), ("mj_block_read_kv", "starts", None, mj.MJ_ERR_INVALID_ARG),
    ("mj_block_read_kv", "k_tok_stride", 128, mj.MJ_ERR_INVALID_ARG), ("mj_block_read_kv", "v_head_stride", 64, mj.MJ_ERR_INVALID_ARG),
    ("mj_block_read_kv", "out_dtype", 2, mj.MJ_ERR_UNSUPPORTED), ("mj_block_read_kv", "block_table", None, mj.MJ_ERR_INVALID_ARG),
    ("mj_block_read_kv", "block_table_len", -1, mj.MJ_ERR_INVALID_ARG), ("mj_block_read_kv", "num_rows", 1 << 40, mj.MJ_ERR_CAPACITY),
    ("mj_block_attention", "num_seqs", 4, mj.MJ_ERR_INVALID_ARG), ("mj_block_attention", "h_q", 7, mj.MJ_ERR_INVALID_ARG),
    ("mj_block_attention", "softmax_scale", float("nan"), mj.MJ_ERR_INVALID_ARG), ("mj_block_attention", "slots", 0, mj.MJ_ERR_INVALID_ARG),
    ("mj_block_attention", "plan", BASE + 8, mj.MJ_ERR_ALIGNMENT), ("mj_block_attention", "workspace_bytes", 4096, mj.MJ_ERR_CAPACITY),
    ("mj_block_attention", "out_head_stride", 64, mj.MJ_ERR_INVALID_ARG), ("mj_block_attention", "out_tok_stride", 128, mj.MJ_ERR_INVALID_ARG),
    ("mj_block_attention", "q", BASE + 8, mj.MJ_ERR_ALIGNMENT), ("mj_block_attention", "lse", BASE + 2, mj.MJ_ERR_ALIGNMENT),
    ("mj_block_attention", "q_len", 1 << 30, mj.MJ_ERR_CAPACITY), ("mj_block_attention", "seq_lens", None, mj.MJ_ERR_INVALID_ARG),
    ("mj_block_prompt", "splits", 0, mj.MJ_ERR_INVALID_ARG), ("mj_block_prompt", "splits", 65, mj.MJ_ERR_INVALID_ARG),
    ("mj_block_prompt", "workspace_bytes", 4096, mj.MJ_ERR_CAPACITY), ("mj_block_prompt", "q_starts", None, mj.MJ_ERR_INVALID_ARG),
    ("mj_block_prompt", "out_tok_stride", 512, mj.MJ_ERR_INVALID_ARG), ("mj_block_prompt", "num_seqs", 65536, mj.MJ_ERR_UNSUPPORTED),
    ("mj_block_prompt", "h_q", 9, mj.MJ_ERR_INVALID_ARG), ("mj_block_prompt", "max_q_len", -1, mj.MJ_ERR_INVALID_ARG),
    ("mj_block_prompt", "softmax_scale", 0.0, mj.MJ_ERR_INVALID_ARG), ("mj_block_prompt", "out_dtype", 5, mj.MJ_ERR_UNSUPPORTED)])
def test_arguments_are_refused(fn, field, value, status):
    assert call(fn, with_(CALLS[fn](), field, value)) == status


def test_empty_calls_do_nothing():
    for fn, fields in (("mj_block_write_kv", ["num_tokens"]), ("mj_block_read_kv", ["num_rows"]), ("mj_block_read_kv", ["num_seqs"]),
                       ("mj_block_attention", ["num_seqs"]), ("mj_block_prompt", ["num_seqs"]), ("mj_block_prompt", ["num_tokens"]),
                       ("mj_block_prompt", ["max_q_len"])):
        a = CALLS[fn]()
        for f in fields:
            setattr(a, f, 0)
        assert call(fn, a) == mj.MJ_OK


@no_gpu
def test_neither_output_of_a_read():
    assert call("mj_block_read_kv", with_(with_(read(), "k_out", None), "v_out", None)) == mj.MJ_ERR_INVALID_ARG
    assert call("mj_block_read_kv", with_(read(), "k_out", None)) == mj.MJ_ERR_CUDA


# ------------------------------------------------------------------------------------------------- the plan
@pytest.mark.parametrize("seed", range(40))
def test_plan_covers_every_tile_once(seed):
    rng = np.random.default_rng(seed)
    slots, B = int(rng.integers(1, 300)), int(rng.integers(0, 80))
    most = B + int(rng.integers(0, 5))
    lens = rng.integers(0, [200, 5000, 200000][seed % 3], B).astype(np.int32)
    if B:
        lens[rng.random(B) < 0.2] = 0
        lens[rng.integers(0, B)] = 131072 if seed % 4 == 0 else lens[0]
    margin = int(rng.integers(0, 200)) * (seed % 2)
    p = mj.mj_block_plan(lens, B, most, slots, margin)
    rows = slots + most
    assert p.size == 4 * (rows + most) == mj.mj_block_plan_size(slots, most)
    work, req = p[:4 * rows].reshape(rows, 4), p[4 * rows:].reshape(most, 4)
    live = work[work[:, 2] > work[:, 1]]
    assert np.array_equal(work[:len(live)], live)  # the empty ones last
    n = live[:, 2] - live[:, 1]
    assert np.all(np.diff(n) <= 0)  # the longest first
    part = 0
    for b in range(B):
        t = -(-(int(lens[b]) + margin) // 128) if lens[b] else 0
        mine = live[live[:, 0] == b]
        mine = mine[np.argsort(mine[:, 3])]
        assert req[b, 3] == t and req[b, 1] == len(mine)
        if t == 0:
            assert len(mine) == 0
            continue
        assert np.array_equal(mine[:, 3], np.arange(len(mine)))
        assert mine[0, 1] == 0 and mine[-1, 2] == t and np.array_equal(mine[1:, 1], mine[:-1, 2])
        assert np.array_equal(mine[:, 1], np.arange(len(mine)) * req[b, 2])
        if len(mine) > 1:
            assert req[b, 0] == part
            part += len(mine)
    assert part <= 4 * slots and not req[B:].any()
    bytes_ = mj.mj_block_workspace_size(slots, 2, 8, 4, 128)
    assert bytes_ == 256 + 4 * slots * 4 * 4 * 130 * 4


def test_plan_splits_a_long_request_among_short_ones():
    p = mj.mj_block_plan(np.array([131072] + [100] * 63, np.int32), 64, 64, 38)
    assert p[4 * (38 + 64)][()] == 0 and p[4 * (38 + 64) + 1] >= 19  # pieces of request 0
    whole = mj.mj_block_plan(np.full(64, 4096, np.int32), 64, 64, 38)
    assert np.all(whole[4 * (38 + 64):].reshape(64, 4)[:, 1] == 1)


def test_plan_refusals():
    for args, status in (((np.array([-1], np.int32), 1, 1, 4), mj.MJ_ERR_INVALID_ARG), ((np.array([5, 5], np.int32), 2, 1, 4), mj.MJ_ERR_INVALID_ARG),
                         ((np.array([5], np.int32), 1, 1, 0), mj.MJ_ERR_INVALID_ARG), ((np.array([5], np.int32), 1, 1, 4, -1), mj.MJ_ERR_INVALID_ARG)):
        with pytest.raises(mj.MjError) as e:
            mj.mj_block_plan(*args)
        assert e.value.status == status
    with pytest.raises(ValueError):
        mj.mj_block_plan(np.array([5], np.int32), 1, 1, 4, plan_out=np.zeros(8, np.int32))


def test_slots_and_splits():
    assert mj.mj_block_slots(152, 1, 32, 8, 128) == 38      # two CTAs an SM
    assert mj.mj_block_slots(152, 4, 32, 8, 128) == 19      # by rows: one
    assert mj.mj_block_slots(152, 2, 16, 4, 256) == 76 and mj.mj_block_slots(152, 9, 16, 4, 256) == 38
    assert mj.mj_block_slots(152, 100, 64, 64, 128) == 2    # 100 rows in one tile
    assert mj.mj_block_slots(0, 1, 32, 8, 128) == 1
    assert mj.mj_block_prompt_splits(152, 1, 8192, 8192, 32, 8, 128) == 1
    assert mj.mj_block_prompt_splits(152, 1, 64, 100000, 32, 8, 128) == 19
    assert mj.mj_block_prompt_splits(152, 1, 64, 3000, 32, 8, 128) == 9
    assert mj.mj_block_prompt_splits(152, 1, 1, 10 ** 6, 1, 1, 128) == 64


# ------------------------------------------------------------------------------------------------- the builders
def kv(pages=4, page=32, h_k=2, d=128, block=16):
    u8 = torch.uint8
    return mj.BlockKV(on_gpu(pages, page, h_k, d, dtype=u8), on_gpu(pages, page, h_k, d, dtype=u8),
                      on_gpu(pages, h_k, page // block, dtype=u8), on_gpu(pages, h_k, page // block, dtype=u8))


def test_builders_take_views_and_say_the_block():
    c = kv()
    a = mj.block_write_args(on_gpu(3, 2, 128), on_gpu(3, 2, 128), on_gpu(3, dtype=torch.int64), c)
    assert (a.cache.block, a.cache.page_size, a.cache.k_stride_page, a.cache.k_stride_head) == (16, 32, 8192, 128)
    c.k_cache = on_gpu(4, 2, 32, 128, dtype=torch.uint8).transpose(1, 2)
    a = mj.block_write_args(on_gpu(3, 2, 128), on_gpu(3, 2, 128), on_gpu(3, dtype=torch.int64), c)
    assert (a.cache.k_stride_token, a.cache.k_stride_head) == (128, 4096)


@pytest.mark.parametrize("field,value", [
    ("k_cache", torch.zeros(4, 32, 2, 128, dtype=torch.uint8)), ("v_cache", on_gpu(4, 32, 2, 256, dtype=torch.uint8)),
    ("k_exp", on_gpu(4, 2, 3, dtype=torch.uint8)), ("v_exp", on_gpu(4, 2, 1, dtype=torch.uint8)), ("k_exp", on_gpu(3, 2, 2, dtype=torch.uint8)),
    ("k_cache", on_gpu(4, 32, 2, 128)), ("v_cache", on_gpu(4, 32, 128, 2, dtype=torch.uint8).transpose(2, 3))])
def test_builders_refuse_caches(field, value):
    c = kv()
    setattr(c, field, value)
    with pytest.raises(ValueError):
        mj.block_write_args(on_gpu(3, 2, 128), on_gpu(3, 2, 128), on_gpu(3, dtype=torch.int64), c)


def test_builders_refuse_tensors():
    c, key, slots = kv(), on_gpu(3, 2, 128), on_gpu(3, dtype=torch.int64)
    table, starts = on_gpu(2, 4, dtype=torch.int32), on_gpu(3, dtype=torch.int32)
    for bad in (lambda: mj.block_write_args(key, on_gpu(4, 2, 128), slots, c), lambda: mj.block_write_args(key, key, on_gpu(3, dtype=torch.int32), c),
                lambda: mj.block_write_args(on_gpu(3, 2, 128, dtype=torch.float16), key, slots, c),
                lambda: mj.block_write_args(key, key, slots, c, status=on_gpu(1, dtype=torch.int64)),
                lambda: mj.block_read_args(c, table, starts), lambda: mj.block_read_args(c, table, starts, key, on_gpu(4, 2, 128)),
                lambda: mj.block_read_args(c, table, starts, on_gpu(3, 2, 128, dtype=torch.float32)),
                lambda: mj.block_read_args(c, table[:1], starts, key), lambda: mj.block_read_args(c, table, starts, key, first=starts)):
        with pytest.raises(ValueError):
            bad()
    a = mj.block_read_args(c, table, starts, v_out=key)
    assert a.num_seqs == 2 and a.num_rows == 3 and a.k_out is None and a.block_table_len == 4


def test_steps_refuse_what_they_were_not_made_for():
    c, table, lens, starts = kv(), on_gpu(2, 4, dtype=torch.int32), on_gpu(2, dtype=torch.int32), on_gpu(3, dtype=torch.int32)
    s = mj.BlockStep.__new__(mj.BlockStep)
    s.max_num_seqs, s.q_len, s.h_q, s.h_k, s.d, s.causal, s.evict_first, s.slots, s.lse = 2, 2, 8, 2, 128, True, True, 5, None
    s.plan_dev, s.workspace, s.ws_bytes = on_gpu(64, dtype=torch.int32), on_gpu(1024, dtype=torch.uint8), 1024
    q, out = on_gpu(4, 8, 128), on_gpu(4, 8, 128)
    assert s.args(q, out, c, table, lens, 2, 0.1).q_len == 2
    p = mj.PromptStep.__new__(mj.PromptStep)
    p.max_tokens, p.max_num_seqs, p.max_q_len, p.h_q, p.h_k, p.d, p.causal, p.splits, p.lse = 4, 2, 3, 8, 2, 128, True, 1, None
    p.workspace, p.ws_bytes = on_gpu(1024, dtype=torch.uint8), 1024
    assert p.args(q, out, c, table, lens, starts, 2, 0.1).num_tokens == 4
    for bad in (lambda: s.args(q, out, c, table, lens, 3, 0.1), lambda: s.args(q[:3], out, c, table, lens, 2, 0.1),
                lambda: s.args(q, out, kv(h_k=1), table, lens, 2, 0.1), lambda: s.args(q, out, c, table, lens[:1], 2, 0.1),
                lambda: s.args(on_gpu(4, 6, 128), out, c, table, lens, 2, 0.1), lambda: s.args(q, on_gpu(4, 8, 128, dtype=torch.float32), c, table, lens, 2, 0.1),
                lambda: p.args(on_gpu(5, 8, 128), on_gpu(5, 8, 128), c, table, lens, starts, 2, 0.1),
                lambda: p.args(q, out[:3], c, table, lens, starts, 2, 0.1), lambda: p.args(q, out, c, table, lens, starts[:2], 2, 0.1),
                lambda: p.args(q, out, kv(d=256), table, lens, starts, 2, 0.1), lambda: p.args(q, out, c, table[:1], lens, starts, 2, 0.1)):
        with pytest.raises(ValueError):
            bad()
