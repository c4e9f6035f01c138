"""The block-scaled cache's calls at their limits, without a GPU: the index bounds that the kernels take from
headers, compiled here for the host, and what the calls refuse."""

import ctypes
import subprocess
import types

import numpy as np
import pytest
import torch

import paged_fp8_decode_gb300 as mj
from tests import test_block_host as H
from tests.test_latent_calls_host import on_gpu

no_gpu = H.no_gpu

HOST = """
#include "mj_block.h"
extern "C" int prefetch_pages(int begin, int end, int depth, int ppt, long long len) {
  return mj::prefetch_pages(begin, end, depth, ppt, len);
}
extern "C" int plan_entry_ok(int first, int pieces, int each, long long cap) {
  return mj::plan_entry_ok(first, pieces, each, cap);
}
"""


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_fp8_decode_gb300.build import build

    build()


@pytest.fixture(scope="module")
def bounds(tmp_path_factory):
    """The kernels' bounds as a host library."""
    from paged_fp8_decode_gb300 import build as B

    at = tmp_path_factory.mktemp("bounds")
    (at / "bounds.cu").write_text(HOST)
    subprocess.run([B._nvcc(), "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-I", B.INCLUDE, "-I", B.CSRC] + B.ARCH +
                   ["-o", str(at / "bounds.so"), str(at / "bounds.cu")], check=True, capture_output=True, text=True)
    lib = ctypes.CDLL(str(at / "bounds.so"))
    lib.prefetch_pages.argtypes = [ctypes.c_int] * 4 + [ctypes.c_longlong]
    lib.plan_entry_ok.argtypes = [ctypes.c_int] * 3 + [ctypes.c_longlong]
    return lib


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_pages_looked_up_ahead_lie_inside_the_table(bounds, page):
    """Every work row of plans with and without a margin, over tables that end at the longest request's last page, before it and
    after it: the entries that the decode kernel looks up before it knows the lengths."""
    rng = np.random.default_rng(page)
    ppt, ends = 128 // page, 0
    for _ in range(20):
        lens = rng.integers(1, [100, 3000, 70000][rng.integers(3)], rng.integers(1, 20)).astype(np.int32)
        slots, margin = int(rng.integers(1, 60)), int(rng.choice([0, 1, 500]))
        plan = mj.mj_block_plan(lens, len(lens), len(lens), slots, margin)
        pages = -(-int(lens.max()) // page)
        for b, begin, end, _ in plan[:4 * (slots + len(lens))].reshape(-1, 4):
            for table in (pages, pages - 1, pages + 9, 0):
                for depth in (4, 8, 16):
                    n = bounds.prefetch_pages(int(begin), int(end), depth, ppt, table)
                    want = [e for e in range(begin * ppt, min(end, begin + depth) * ppt) if e < table]
                    assert n == len(want)
                    ends += n < min(end - begin, depth) * ppt and n > 0
    assert ends or page == 128  # tiles that reach past the table were among them


def test_pages_looked_up_ahead_of_rows_that_are_no_plan(bounds):
    for begin, end in ((-3, 5), (-2 ** 31, 2 ** 31 - 1), (7, 7), (9, 2), (2 ** 31 - 2, 2 ** 31 - 1)):
        assert bounds.prefetch_pages(begin, end, 16, 8, 1000) == 0
    assert bounds.prefetch_pages(0, 2 ** 31 - 1, 16, 8, 2 ** 40) == 128


def test_decode_refuses_a_block_table_that_ends_inside_its_last_row():
    """mj_decode_attention has no table length: a request's pages are looked up within block_table_stride entries."""
    step = mj.DecodeStep.__new__(mj.DecodeStep)
    step.plan_info, step.q_mode = None, "fp8"
    whole, x = on_gpu(5, 12, dtype=torch.int32), on_gpu(4)

    def kv(table):
        return types.SimpleNamespace(block_table=table, k_cache=x, v_cache=x, k_descale=x, v_descale=x, seq_lens=x, q_mul=None, o_mul=None)

    for table, n in ((whole[:, 4:], 5), (whole[1:, 1:], 4), (whole[4:, :1].expand(1, 1)[:, :1], 2)):
        with pytest.raises(ValueError, match="block_table"):
            step.args(kv(table), x, n, 0.1)
    for table, n in ((whole, 5), (whole[:, 4:], 4), (whole[:, :3], 5), (whole[2:], 3), (whole[:1].expand(5, 12), 5)):
        with pytest.raises((TypeError, AttributeError)):  # past the check: the step has no shape
            step.args(kv(table), x, n, 0.1)


def test_plan_entries_whose_partials_the_workspace_does_not_hold(bounds):
    for slots in (1, 7, 304):
        cap = 4 * slots
        for lens in ([131072], [9000] * 5 + [20], [1, 0, 3]):
            plan = mj.mj_block_plan(np.array(lens, np.int32), len(lens), len(lens), slots)
            for first, pieces, each, _ in plan[4 * (slots + len(lens)):].reshape(-1, 4):
                assert bounds.plan_entry_ok(int(first), int(pieces), int(each), cap)
        big = 2 ** 31 - 1
        for first, pieces, each in ((-1, 2, 1), (cap - 1, 2, 1), (0, cap + 1, 1), (0, big, 1), (big, 2, 1), (big, big, 1), (0, 2, 0), (0, 2, -5)):
            assert not bounds.plan_entry_ok(first, pieces, each, cap)
        assert bounds.plan_entry_ok(big, 1, 0, cap) and bounds.plan_entry_ok(cap - 2, 2, 1, cap)


def token_of_row(row, h_r):
    """The prompt kernel's quotient, as it takes it."""
    f = np.float32
    return int((f(row) + f(0.5)) * (f(1) / f(h_r)))


def test_the_quotient_that_finds_a_rows_token():
    # exact up to 2^21 heads a KV head; past that it is not, and a row would be read in front of its token's
    for h_r in list(range(1, 300)) + [2 ** 20 - 1, 2 ** 20, 2 ** 21]:
        for row in {0, 1, h_r - 1, h_r, h_r + 1, h_r + 255, 2 * h_r - 1 if h_r < 256 else 0}:
            assert token_of_row(row, h_r) == row // h_r
    assert any(token_of_row(h_r - 1, h_r) != 0 for h_r in range(2 ** 23, 2 ** 23 + 100))


@no_gpu
def test_prompts_refuse_more_heads_a_kv_head_than_the_quotient_takes():
    a = H.prompt(splits=1)
    a.cache.h_k, a.num_tokens, a.max_q_len, a.num_seqs = 1, 1, 1, 1
    for h_q, status in ((2 ** 20, (mj.MJ_ERR_CUDA, mj.MJ_ERR_UNSUPPORTED)), (2 ** 20 + 1, (mj.MJ_ERR_INVALID_ARG,)),
                        (2 ** 23 + 2, (mj.MJ_ERR_INVALID_ARG,))):
        a.h_q = h_q
        a.q_tok_stride = a.out_tok_stride = h_q * 128
        assert H.call("mj_block_prompt", a) in status
