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


# ------------------------------------------------------------------------------------------------- chunks past the call's rows
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("past", [1, 7, 40])
def test_a_chunk_that_reaches_past_the_rows_keeps_its_limits(past, splits):
    """q_starts names more query tokens than q has rows: those that there are see what they would in the whole call, and
    the others are reported."""
    import paged_fp8_decode_gb300 as mj

    b = Batch([90, 200], seed=past)
    kv = b.kv()
    q = D.queries(b, 30 + 60, 8)
    starts = up(np.array([0, 30, 90], np.int32))
    outs, lses, codes = [], [], []
    for T in (90, 90 - past):
        step = mj.PromptStep(max_tokens=90, max_num_seqs=2, max_q_len=60, max_len=200, h_q=8, h_k=2, d=128, splits=splits, with_lse=True)
        out = torch.full((90, 8, 128), SENTINEL, dtype=torch.bfloat16, device="cuda")
        step.lse.fill_(SENTINEL)
        mj.mj_block_prompt(step.args(q[:T], out, kv, b.table_dev, b.lens_dev, starts, 2, 128 ** -0.5))
        outs.append(out)
        lses.append(step.lse)
        codes.append(mj.mj_workspace_status(step.workspace))
    assert codes == [0, 4]
    T = 90 - past
    assert torch.equal(outs[0][:T], outs[1][:T]) and torch.equal(lses[0][:T], lses[1][:T])
    assert (outs[1][T:] == SENTINEL).all() and (lses[1][T:] == SENTINEL).all()


@pytest.mark.parametrize("splits", [1, 2])
def test_a_request_that_begins_past_the_rows_is_reported(splits):
    import paged_fp8_decode_gb300 as mj

    b = Batch([20, 50], seed=2)
    kv = b.kv()
    q = D.queries(b, 20, 8)
    step = mj.PromptStep(max_tokens=20, max_num_seqs=2, max_q_len=20, max_len=50, h_q=8, h_k=2, d=128, splits=splits, with_lse=True)
    out = torch.full((20, 8, 128), SENTINEL, dtype=torch.bfloat16, device="cuda")
    mj.mj_block_prompt(step.args(q, out, kv, b.table_dev, b.lens_dev, up(np.array([0, 20, 29], np.int32)), 2, 128 ** -0.5))
    assert mj.mj_workspace_status(step.workspace) == 4
    want, want_lse = OB.attention(q.double().cpu().numpy(), b.rows("k", 0), b.rows("v", 0), 128 ** -0.5, True)
    D.check_rows(out.double().cpu().numpy(), step.lse.cpu().numpy(), want, want_lse, b.vmax(0), rel=0.0025, elem=0.003, lse_tol=6e-4)


# ------------------------------------------------------------------------------------------------- small softmax scales
@pytest.mark.parametrize("scale", [1e-12, 1e-20, 1e-30, 1e-38])
@pytest.mark.parametrize("d", [128, 256])
def test_small_softmax_scales_and_queries_of_zero(scale, d):
    """The logits are 0 to within 1e-8: a row's output is the mean of the V that it sees, its LSE the log of their number. Hidden
    keys stay hidden, also for queries of zero over the smallest scales."""
    import paged_fp8_decode_gb300 as mj

    new = [70, 33]
    b = Batch([300, 33], d=d, seed=4)
    live = (b.exps["k"] > 0) & (b.exps["k"] < 255)
    b.exps["k"][live] = 95
    kv = b.kv()
    q = D.queries(b, 103, 8)
    q[::2] = 0
    starts = up(np.array([0, 70, 103], np.int32))
    for h_q, splits in ((8, 1), (8, 2), (2, 1)):
        qh = q[:, :h_q].contiguous()
        step = mj.PromptStep(max_tokens=103, max_num_seqs=2, max_q_len=70, max_len=300, h_q=h_q, h_k=2, d=d, splits=splits, with_lse=True)
        out = torch.empty(103, h_q, d, dtype=torch.bfloat16, device="cuda")
        mj.mj_block_prompt(step.args(qh, out, kv, b.table_dev, b.lens_dev, starts, 2, scale))
        got, lse = out.double().cpu().numpy(), step.lse.cpu().numpy()
        for i, s in enumerate((slice(0, 70), slice(70, 103))):
            want, want_lse = OB.attention(qh[s].double().cpu().numpy(), b.rows("k", i), b.rows("v", i), scale, True)
            D.check_rows(got[s], lse[s], want, want_lse, b.vmax(i), rel=0.0025, elem=0.003, lse_tol=6e-4)
    for h_q, q_len in ((8, 1), (8, 4), (40, 4)):  # 4, 16 and 80 rows
        qd = D.queries(b, 2 * q_len, h_q)
        qd[::2] = 0
        step = mj.BlockStep(max_num_seqs=2, q_len=q_len, h_q=h_q, h_k=2, d=d, with_lse=True)
        step.plan(b.lens, 2)
        out = torch.full((2 * q_len + 2, h_q, d), SENTINEL, dtype=torch.bfloat16, device="cuda")
        step.run(qd, out, kv, b.table_dev, b.lens_dev, 2, scale)
        got = out[:2 * q_len].double().cpu().numpy().reshape(2, q_len, h_q, d)
        lse = step.lse.cpu().numpy().reshape(2, 2, q_len, h_q // 2).transpose(0, 2, 1, 3).reshape(2, q_len, h_q)
        for i in range(2):
            want, want_lse = OB.attention(qd.double().cpu().numpy().reshape(2, q_len, h_q, d)[i], b.rows("k", i), b.rows("v", i), scale, True)
            D.check_rows(got[i], lse[i], want, want_lse, b.vmax(i))


@pytest.mark.parametrize("by", [-100, -60, 60])
def test_small_and_large_queries_with_the_scale_that_makes_up_for_them(by):
    """Queries of 2^by times the usual size, the softmax scale 2^-by times: the same logits, and as exact."""
    import paged_fp8_decode_gb300 as mj

    b = Batch([300, 33], seed=23)
    kv = b.kv()
    scale = 128 ** -0.5 * 2.0 ** -by
    q = D.queries(b, 103, 8, size=2.0 ** by)
    for h_q in (8, 2):
        qh = q[:, :h_q].contiguous()
        step = mj.PromptStep(max_tokens=103, max_num_seqs=2, max_q_len=70, max_len=300, h_q=h_q, h_k=2, d=128, with_lse=True)
        out = torch.empty(103, h_q, 128, dtype=torch.bfloat16, device="cuda")
        mj.mj_block_prompt(step.args(qh, out, kv, b.table_dev, b.lens_dev, up(np.array([0, 70, 103], np.int32)), 2, scale))
        for i, s in enumerate((slice(0, 70), slice(70, 103))):
            want, want_lse = OB.attention(qh[s].double().cpu().numpy(), b.rows("k", i), b.rows("v", i), scale, True)
            D.check_rows(out[s].double().cpu().numpy(), step.lse[s].cpu().numpy(), want, want_lse, b.vmax(i), rel=0.0025, elem=0.003,
                         lse_tol=6e-4)
    for h_q, q_len in ((8, 1), (8, 4)):
        qd = D.queries(b, 2 * q_len, h_q, size=2.0 ** by)
        step = mj.BlockStep(max_num_seqs=2, q_len=q_len, h_q=h_q, h_k=2, d=128, with_lse=True)
        step.plan(b.lens, 2)
        out = torch.empty(2 * q_len, h_q, 128, dtype=torch.bfloat16, device="cuda")
        step.run(qd, out, kv, b.table_dev, b.lens_dev, 2, scale)
        lse = step.lse.cpu().numpy().reshape(2, 2, q_len, h_q // 2).transpose(0, 2, 1, 3).reshape(2, q_len, h_q)
        for i in range(2):
            s = slice(i * q_len, (i + 1) * q_len)
            want, want_lse = OB.attention(qd[s].double().cpu().numpy(), b.rows("k", i), b.rows("v", i), scale, True)
            D.check_rows(out[s].double().cpu().numpy(), lse[i], want, want_lse, b.vmax(i))


# ------------------------------------------------------------------------------------------------- layouts
def one_head(b, order):
    """The caches of a batch of one KV head, K's rows as ``phtd``, V's as ``order``, each with its own stride of the one head."""
    import paged_fp8_decode_gb300 as mj

    def side(c, order):
        axes = {"p": 0, "t": 1, "h": 2}
        perm = [axes[x] for x in order[:3]] + [3]
        return up(c.transpose(perm)).permute(*[perm.index(i) for i in range(4)])

    wide = torch.zeros(b.pages, b.page, 3, b.d, dtype=torch.uint8, device="cuda")  # (one of three heads, as a slice)
    if order == "slice":
        wide[:, :, 1:2] = up(b.codes["v"])
        v = wide[:, :, 1:2]
    else:
        v = side(b.codes["v"], order)
    b.table_dev, b.lens_dev = up(b.table), up(b.lens)
    return mj.BlockKV(side(b.codes["k"], "phtd"), v, up(b.exps["k"]), up(b.exps["v"]))


@pytest.mark.parametrize("order", ["phtd", "pthd", "slice"])
@pytest.mark.parametrize("d", [128, 256])
def test_one_head_whatever_its_stride(order, d):
    b = Batch([300, 77], h_k=1, d=d, page=32, block=32, seed=5)
    b._dev = one_head(b, order)
    for h_q, q_len in ((8, 1), (8, 4)):
        q = D.queries(b, 2 * q_len, h_q)
        out, lse, status = D.decode(b, q, q_len, h_q)
        assert status == 0
        D.check_decode(b, q, out, lse, q_len, h_q)
    out, lse, status, q = P.run(b, [100, 77], 4)
    assert status == 0
    P.check(b, [100, 77], out, lse, q)


@pytest.mark.parametrize("order", ["tphd", "hptd"])
@pytest.mark.parametrize("d", [128, 256])
def test_attention_over_tokens_or_heads_outermost(order, d):
    b = Batch([5, 700, 64], page=32, block=16, order=order, d=d, seed=6)
    for h_q in (8, 32):
        q = D.queries(b, 3, h_q)
        out, lse, status = D.decode(b, q, 1, h_q)
        assert status == 0
        D.check_decode(b, q, out, lse, 1, h_q)
    out, lse, status, q = P.run(b, [5, 200, 33], 4)
    assert status == 0
    P.check(b, [5, 200, 33], out, lse, q)


def test_k_and_v_in_different_orders_are_written_and_read_but_not_attended_to():
    import paged_fp8_decode_gb300 as mj

    b, k, v, slots = D.make_write([(3, 60)], seed=7)
    kv = b.kv()
    kv.v_cache = kv.v_cache.contiguous()  # V's heads inside its tokens, K's outside
    D.check_write(b, k, v, slots)
    rows = torch.empty(60, 2, 128, dtype=torch.bfloat16, device="cuda")
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    mj.mj_block_read_kv(mj.block_read_args(kv, table, up(np.array([0, 60], np.int32)), v_out=rows, first=up(np.array([3], np.int32))))
    b.reload()
    assert torch.equal(rows.double().cpu(), torch.from_numpy(OB.values(b.codes["v"], b.exps["v"])[:4].reshape(64, 2, 128)[3:63]))
    lens = up(np.array([63], np.int32))
    for h_q in (8, 32):
        q, out = D.queries(b, 1, h_q), torch.empty(1, h_q, 128, dtype=torch.bfloat16, device="cuda")
        step = mj.BlockStep(max_num_seqs=1, q_len=1, h_q=h_q, h_k=2, d=128)
        step.plan(np.array([63], np.int32), 1)
        with pytest.raises(mj.MjError) as e:
            step.run(q, out, kv, table, lens, 1, 0.1)
        assert e.value.status == mj.MJ_ERR_UNSUPPORTED
    step = mj.PromptStep(max_tokens=1, max_num_seqs=1, max_q_len=1, max_len=63, h_q=8, h_k=2, d=128)
    with pytest.raises(mj.MjError) as e:
        step.run(q[:, :8].contiguous(), out[:, :8].contiguous(), kv, table, lens, up(np.array([0, 1], np.int32)), 1, 0.1)
    assert e.value.status == mj.MJ_ERR_UNSUPPORTED
