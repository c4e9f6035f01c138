"""The block-scaled cache's calls at their limits on the GPU, against oracle.block (float64).

Tolerances as in test_gpu_block.py and test_gpu_block_prompt.py where nothing else is said."""

import numpy as np
import pytest
import torch

from oracle import block as OB
from tests import test_gpu_block as D
from tests import test_gpu_block_prompt as P
from tests._block import SENTINEL, Batch, bf16, up

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_fp8_decode_gb300.build import build

    build()


# ------------------------------------------------------------------------------------------------- block tables
@pytest.mark.parametrize("h_q", [8, 32])
def test_a_block_table_inside_a_larger_one(h_q):
    # columns 4 .. of a wider buffer whose other entries are no pages, the last request's last tile ends inside its first page
    b = Batch([4000, 130, 2 * 128 + 5], seed=20)
    kv = b.kv()
    wide = torch.full((4, b.table.shape[1] + 11), 2 ** 30, dtype=torch.int32, device="cuda")
    wide[:3, 4:4 + b.table.shape[1]] = b.table_dev
    q = D.queries(b, 3, h_q)
    want = D.decode(b, q, 1, h_q)
    for pages in (b.table.shape[1], -(-4000 // 16)):
        b.table_dev = wide[:3, 4:4 + pages]
        for kw in ({}, {"margin": 3000}):
            out, lse, status = D.decode(b, q, 1, h_q, **kw)
            assert status == 0
            D.check_decode(b, q, out, lse, 1, h_q)
    assert torch.equal(D.decode(b, q, 1, h_q)[0], want[0])


@pytest.mark.parametrize("h_q", [8, 32])
def test_one_row_of_a_block_table_for_all_requests(h_q):
    b = Batch([700], seed=21)
    kv = b.kv()
    b.B, b.lens = 3, np.array([700, 16, 333], np.int32)
    b.table = np.repeat(b.table, 3, 0)
    b.table_dev, b.lens_dev = b.table_dev.expand(3, -1), up(b.lens)
    q = D.queries(b, 3, h_q)
    out, lse, status = D.decode(b, q, 1, h_q)
    assert status == 0
    D.check_decode(b, q, out, lse, 1, h_q)


# ------------------------------------------------------------------------------------------------- plans that are not this step's
@pytest.mark.parametrize("h_q", [8, 32])
@pytest.mark.parametrize("word,value", [(0, -1), (0, "cap"), (0, 2 ** 31 - 1), (1, 2 ** 31 - 1), (2, 0), (2, -7)])
def test_a_plan_whose_partials_lie_outside_the_workspace(h_q, word, value):
    """An entry of a split request that mj_block_plan does not make: the request is left out by the attention and by the join,
    and reported."""
    import paged_fp8_decode_gb300 as mj

    b = Batch([20000, 300, 17], seed=22, page=64, block=32)
    kv = b.kv()
    q = D.queries(b, 3, h_q)
    step = mj.BlockStep(max_num_seqs=3, q_len=1, h_q=h_q, h_k=2, d=128, with_lse=True)
    plan = step.plan(b.lens, 3).clone()
    at = 4 * (step.slots + 3)
    assert plan[at + 1] > 1
    plan[at + word] = 4 * step.slots - 1 if value == "cap" else value
    step.plan_dev.copy_(plan)
    out = torch.full((5, h_q, 128), SENTINEL, dtype=torch.bfloat16, device="cuda")
    step.lse.fill_(SENTINEL)
    step.run(q, out, kv, b.table_dev, b.lens_dev, 3, 128 ** -0.5)
    assert mj.mj_workspace_status(step.workspace) == 4
    assert (out[0] == SENTINEL).all() and (step.lse[0] == SENTINEL).all()
    step.plan(b.lens, 3)  # and the step is as it was
    step.run(q, out, kv, b.table_dev, b.lens_dev, 3, 128 ** -0.5)
    assert mj.mj_workspace_status(step.workspace) == 0
    D.check_decode(b, q, out, step.lse, 1, h_q)
