"""The rotated writes and the latent attention on the host, beside
test_rope_latent_host.py: what the plan says of its lengths, refusals."""

import ctypes
import types

import numpy as np
import pytest
import torch

import paged_fp8_decode_gb300 as mj
from tests import test_rope_latent_host as H


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_fp8_decode_gb300.build import build

    build()


@pytest.mark.parametrize("margin", [0, 1, 130])
def test_plan_states_the_tiles_of_every_request(margin):
    lens = np.array([1, 0, 128, 129, 131072, 127], np.int32)
    plan = mj.mj_latent_plan(lens, 6, 9, 12, 1, 16, margin)
    words = (9 + 3) // 4 * 4
    assert len(plan) == mj.mj_latent_plan_size(12, 9) and len(plan) % 4 == 0
    tiles = plan[-words:]
    assert tiles[:6].tolist() == [-(-(int(n) + margin) // 128) if n else 0 for n in lens] and not tiles[6:].any()


def test_a_plan_on_another_device_is_refused(monkeypatch):
    # its default stream would be the current device's, in no order with the attention
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    step = mj.LatentStep.__new__(mj.LatentStep)
    step.plan_dev = types.SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="cuda:1"):
        step.plan(np.array([5], np.int32), 1)


class OnGpu(torch.Tensor):
    """A host tensor that says it is on a GPU: what the argument builders look at, without one."""

    is_cuda = True


def on_gpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


def rope_args(fmt=0, T=3, h_k=2, d=128, k_bytes=None, v_bytes=None, page=16, pages=4, strides=None, pools=None):
    row = d * {0: 8, 1: 6, 2: 6, 3: 4}[fmt] // 8
    strides = strides or (h_k * page * row, row, page * row)
    full = pages * page * h_k * row
    k, v = pools or (on_gpu(k_bytes or full, dtype=torch.uint8), on_gpu(v_bytes or full, dtype=torch.uint8))
    n = 1 if fmt == 0 else h_k * d
    scale = on_gpu(n, dtype=torch.float32)
    x = on_gpu(T, h_k, d)
    return mj.rope_write_args(x, x.clone(), x.clone(), on_gpu(T, dtype=torch.int64), mj.mj_rope_turns([1.0] * 64).as_subclass(OnGpu),
                              on_gpu(T, dtype=torch.int64), k, v, strides, page, pages, fmt, scale, scale)


@pytest.mark.parametrize("fmt", [0, 1, 2, 3])
def test_caches_that_end_before_their_pages_are_refused(fmt):
    row = 128 * {0: 8, 1: 6, 2: 6, 3: 4}[fmt] // 8
    full = 4 * 16 * 2 * row
    a = rope_args(fmt)
    assert (a.kv.k_stride_page, a.kv.k_stride_token, a.kv.k_stride_head) == (32 * row, row, 16 * row)
    for bad in (dict(k_bytes=full - 1), dict(v_bytes=full - 1), dict(k_bytes=full, v_bytes=full, pages=5),
                dict(k_bytes=full, v_bytes=full, page=32), dict(strides=(32 * row, row, 64 * row)),
                dict(strides=(64 * row, row, 16 * row))):
        with pytest.raises(ValueError, match="_cache"):
            rope_args(fmt, **bad)


def test_caches_may_be_views_of_one_pool():
    # keys and values side by side in each page: a view's extent ends with its own last row
    pool = on_gpu(4, 2, 2, 16, 128, dtype=torch.uint8)
    k, v = pool[:, 0], pool[:, 1]
    rope_args(pools=(k, v), strides=(8192, 128, 2048))
    with pytest.raises(ValueError, match="v_cache"):
        rope_args(pools=(k, v[:3]), strides=(8192, 128, 2048))
    rope_args(pools=(on_gpu(0, dtype=torch.uint8), on_gpu(0, dtype=torch.uint8)), pages=0)


def set_all(a, **fields):
    for path, value in fields.items():
        H.set_path(a, path.replace("__", "."), value)
    return a


# (a call that passed the check would stop at the launch, which needs a GPU; on one it must not get there)
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are not real")


@no_gpu
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("page,token,head", [(4096, 112, 2048), (4096, 128, 112), (4096, 128, 128), (4096, 128, 1024),
                                             (2048, 128, 4096), (0, 128, 2048), (4096, 0, 2048), (4096, 128, 0)])
def test_rope_write_refuses_cache_rows_that_overlap(which, page, token, head):
    a = H.rope_write()  # 4 pages of 16 tokens, 2 heads of 128 bytes
    set_all(a, **{f"kv__{which}_stride_page": page, f"kv__{which}_stride_token": token, f"kv__{which}_stride_head": head})
    assert mj.load_library().mj_rope_write_kv(ctypes.byref(a), None) == mj.MJ_ERR_INVALID_ARG


@no_gpu
def test_cache_rows_in_any_order_of_strides_are_taken():
    # past every check, the call fails at the launch: there is no GPU
    for page, token, head in ((4096, 128, 2048), (4096, 256, 128), (2048, 128, 8192), (256, 1024, 128), (8192, 144, 2560)):
        a = set_all(H.rope_write(), **{f"kv__{w}_stride_{n}": x for w in "kv" for n, x in
                                       (("page", page), ("token", token), ("head", head))})
        assert mj.load_library().mj_rope_write_kv(ctypes.byref(a), None) == mj.MJ_ERR_CUDA
    one = set_all(H.rope_write(), kv__h_k=1, kv__num_pages=1, kv__k_stride_head=0, kv__v_stride_head=0, kv__k_stride_page=0)
    assert mj.load_library().mj_rope_write_kv(ctypes.byref(one), None) == mj.MJ_ERR_CUDA
    six = set_all(H.rope_write(), kv__kv_format=1, **{f"kv__{w}_stride_{n}": x for w in "kv" for n, x in
                                                      (("page", 4096), ("token", 96), ("head", 2048))})
    assert mj.load_library().mj_rope_write_kv(ctypes.byref(six), None) == mj.MJ_ERR_CUDA


@no_gpu
@pytest.mark.parametrize("page,token,ok", [(9216, 576, True), (576, 2304, True), (9200, 576, False), (576, 576, False),
                                           (1152, 2304, False)])
def test_latent_write_refuses_pages_that_overlap(page, token, ok):
    a = set_all(H.latent_write(), stride_page=page, stride_token=token)  # 4 pages of 16 tokens
    assert mj.load_library().mj_latent_write(ctypes.byref(a), None) == (mj.MJ_ERR_CUDA if ok else mj.MJ_ERR_INVALID_ARG)


@no_gpu
@pytest.mark.parametrize("fn,make,d,q", [("mj_rope_write_kv", H.rope_write, 128, "q"), ("mj_latent_write", H.latent_write, 64, "q_pe")])
def test_queries_written_over_each_other_are_refused(fn, make, d, q):
    call = getattr(mj.load_library(), fn)
    for tok, head in ((8 * d, 0), (0, d), (8 * d, d - 8), (8 * d - 8, d), (d, d), (d, 2 * d)):  # 3 tokens of 8 heads
        a = set_all(make(), q_out_tok_stride=tok, q_out_head_stride=head)
        assert call(ctypes.byref(a), None) == mj.MJ_ERR_INVALID_ARG
        a = set_all(make(), q_out_tok_stride=tok, q_out_head_stride=head, q_tok_stride=tok, q_head_stride=head)
        a.q_out = getattr(a, q)  # in place
        assert call(ctypes.byref(a), None) == mj.MJ_ERR_INVALID_ARG
    a = set_all(make(), q_out_tok_stride=16 * d)
    a.q_out = getattr(a, q)  # in place, at other strides
    assert call(ctypes.byref(a), None) == mj.MJ_ERR_INVALID_ARG
    for tok, head in ((d, 3 * d), (9 * d + 8, d + 8)):
        assert call(ctypes.byref(set_all(make(), q_out_tok_stride=tok, q_out_head_stride=head)), None) == mj.MJ_ERR_CUDA
    # queries read twice are no fault
    assert call(ctypes.byref(set_all(make(), q_tok_stride=0, q_head_stride=0)), None) == mj.MJ_ERR_CUDA


@no_gpu
def test_an_expanded_query_is_not_rotated_in_place():
    x = on_gpu(1, 2, 128).expand(3, 2, 128)
    pool = on_gpu(16384, dtype=torch.uint8)
    i, one = on_gpu(3, dtype=torch.int64), on_gpu(1, dtype=torch.float32)
    key = on_gpu(3, 2, 128)
    a = mj.rope_write_args(x, key, key, i, mj.mj_rope_turns([1.0] * 8).as_subclass(OnGpu), i, pool, pool,
                           (4096, 128, 2048), 16, 4, 0, one, one)
    assert mj.load_library().mj_rope_write_kv(ctypes.byref(a), None) == mj.MJ_ERR_INVALID_ARG


@no_gpu
def test_attention_rows_written_over_each_other_are_refused():
    lib = mj.load_library()
    for tok, head in ((4096, 0), (0, 512), (4096, 504), (4088, 512), (512, 512), (512, 768)):  # 2 requests of 8 heads
        a = set_all(H.latent(), out_tok_stride=tok, out_head_stride=head)
        a.workspace_bytes = 256  # (stops a call that passed the check, by another status)
        assert lib.mj_latent_attention(ctypes.byref(a), None) == mj.MJ_ERR_INVALID_ARG
    for tok, head in ((4096, 512), (512, 1024), (4800, 600)):
        a = set_all(H.latent(), out_tok_stride=tok, out_head_stride=head, workspace_bytes=256)
        assert lib.mj_latent_attention(ctypes.byref(a), None) == mj.MJ_ERR_CAPACITY
