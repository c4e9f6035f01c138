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


# ------------------------------------------------------------------------------------------------- steps kept for larger batches
@pytest.mark.parametrize("h_q,q_len", [(8, 1), (16, 1), (8, 3), (80, 1)])
@pytest.mark.parametrize("extra", [1, 30, 500])
def test_decode_of_fewer_requests_than_the_step_was_made_for(h_q, q_len, extra):
    b = Batch([3000, 0, 17, 300], seed=extra, page=32, block=32)
    q = D.queries(b, 4 * q_len, h_q)
    out, lse, status = D.decode(b, q, q_len, h_q, extra=extra)
    assert status == 0
    assert (lse[4:] == SENTINEL).all()
    D.check_decode(b, q, out, lse[:4], q_len, h_q)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("splits", [None, 1, 3])
def test_prompt_of_fewer_and_shorter_chunks_than_the_step_was_made_for(splits, d):
    import paged_fp8_decode_gb300 as mj

    new = [5, 64, 1]
    b = Batch([900, 64, 400], d=d, seed=9)
    kv = b.kv()
    step = mj.PromptStep(max_tokens=500, max_num_seqs=40, max_q_len=400, max_len=3000, h_q=8, h_k=2, d=d, splits=splits, with_lse=True)
    step.lse.fill_(SENTINEL)
    q = D.queries(b, 70 + 9, 8)
    out = torch.full((79, 8, d), SENTINEL, dtype=torch.bfloat16, device="cuda")
    step.run(q, out, kv, b.table_dev, b.lens_dev, up(np.array([0, 5, 69, 70], np.int32)), 3, d ** -0.5)
    assert mj.mj_workspace_status(step.workspace) == 0
    P.check(b, new, out, step.lse, q)


# ------------------------------------------------------------------------------------------------- rows by themselves
@pytest.mark.parametrize("h_q,q_len,lens", [(2, 2, [65, 33]), (4, 2, [65, 33]), (2, 4, [66, 34])])  # 4, 8 and 8 rows a KV head
@pytest.mark.parametrize("d", [128, 256])
def test_small_decode_rows_whose_unseen_keys_have_a_large_scale(h_q, q_len, lens, d):
    # the first query tokens do not see the last block's keys, whose V is 2^20 times the others'
    b = Batch(lens, h_k=1, d=d, seed=10, spread=(-20, -20))
    for i, n in enumerate(b.lens):
        b.exps["v"][b.table[i, (n - 1) // 16]] = 127
    q = D.queries(b, 2 * q_len, h_q)
    out, lse, status = D.decode(b, q, q_len, h_q)
    assert status == 0
    got = out[:2 * q_len].double().cpu().numpy().reshape(2, q_len, h_q, d)
    qd = q.double().cpu().numpy().reshape(2, q_len, h_q, d)
    for i in range(2):
        want, _ = OB.attention(qd[i], b.rows("k", i), b.rows("v", i), d ** -0.5, True)
        assert np.abs(want[0]).max() < 1e-3 < np.abs(want[-1]).max()
        err = np.linalg.norm(got[i] - want, axis=2) / np.linalg.norm(want, axis=2)
        assert err.max() <= 2 * D.REL, err


def peaked(b, rows, h_q, limit, rng):
    """Queries that each look at one key of their request: a logit of 30, where others' are normal with 30 / sqrt(d) at most."""
    q = np.zeros((rows.shape[0], h_q, b.d))
    r = h_q // b.h_k
    for t, i in enumerate(rows):
        k = b.rows("k", i)
        for h in range(h_q):
            x = k[rng.integers(0, limit[t]), h // r]
            q[t, h] = x * 30 * b.d ** 0.5 / (x @ x)
    return bf16(q).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [128, 256])
def test_peaked_rows_one_by_one(d, dtype):
    """One key has nearly all of a row's weight, so that the weight's own error is the row's: within 2^-8 (two e4m3 terms; the sum
    takes it unrounded) or 2^-11 (fp16) of itself, the logit 4e-4. The output's rounding, half a step at most, is uniform in it:
    2^-8 / sqrt(3) of the values' power of two (fp16: 2^-11), 2^-9 of the values in the 2-norm of a row of 128 (2^-12)."""
    half = 2.0 ** -9 if dtype == torch.bfloat16 else 2.0 ** -12
    rng = np.random.default_rng(d)
    b = Batch([3000, 700, 130], d=d, seed=11, spread=(-5, -5), page=32, block=32)
    for h_q, q_len in ((8, 1), (4, 3), (16, 1), (8, 4), (40, 2)):
        rows = np.repeat(np.arange(3), q_len)
        limit = np.array([int(b.lens[i]) - q_len + 1 for i in rows])
        q = peaked(b, rows, h_q, limit, rng)
        out, lse, status = D.decode(b, q, q_len, h_q, dtype=dtype)
        assert status == 0
        got = out[:3 * q_len].double().cpu().numpy().reshape(3, q_len, h_q, d)
        qd = q.double().cpu().numpy().reshape(3, q_len, h_q, d)
        weight = 2.0 ** -8 if q_len * h_q // 2 <= 8 else 2.0 ** -11
        for i in range(3):
            want, _ = OB.attention(qd[i], b.rows("k", i), b.rows("v", i), d ** -0.5, True)
            err = np.linalg.norm(got[i] - want, axis=2) / np.linalg.norm(want, axis=2)
            assert err.max() <= weight + half + 4e-4, (h_q, q_len, err.max())
    new = [200, 70, 130]
    rows = np.repeat(np.arange(3), new)
    limit = np.concatenate([int(b.lens[i]) - n + 1 + np.arange(n) for i, n in enumerate(new)])
    q = peaked(b, rows, 8, limit, rng)
    for splits in (1, 3):
        out, lse, status, _ = P.run(b, new, 8, q=q, extra=0, splits=splits, dtype=dtype)
        assert status == 0
        got, qd, at = out.double().cpu().numpy(), q.double().cpu().numpy(), 0
        for i, n in enumerate(new):
            want, _ = OB.attention(qd[at:at + n], b.rows("k", i), b.rows("v", i), d ** -0.5, True)
            err = np.linalg.norm(got[at:at + n] - want, axis=2) / np.linalg.norm(want, axis=2)
            assert err.max() <= 2.0 ** -11 + half + 4e-4, (splits, err.max())
            at += n


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("rows,exact,below", [(4, 13, 21), (8, 13, 21), (16, 9, 17), (40, 9, 17)])
def test_channels_far_below_the_largest_of_a_query(rows, exact, below, d):
    """A query's largest value, 225 times a power of two, is the worst for its other channels. It meets zeros of K: the logits
    are the other channels' alone. Those of 2^-exact of the largest and more are exact, the smaller within 2^-below of it."""
    rng = np.random.default_rng(rows + d)
    b = Batch([400], h_k=1, d=d, seed=12, spread=(0, 0))
    b.codes["k"][..., 0] = 0
    k = b.rows("k", 0)
    for down, off in ((exact, 0.0), (below - 7, 2.0 ** -below), (below - 3, 2.0 ** -below)):
        q = rng.uniform(1.0, 2.0, (1, rows, d)) * rng.choice([-1.0, 1.0], (1, rows, d))
        q[..., 0] = 1.0
        q = bf16(q * 225 * 2.0 ** -down)
        q[..., 0] = 225.0
        qd = q.double().numpy()
        scale = 4.0 / np.abs(qd[..., 1:] @ k[:, 0, 1:].T).max()  # logits within 4 nats
        kv = b.kv()
        import paged_fp8_decode_gb300 as mj

        tol = 4e-4 + off * 225 * np.abs(k).sum(2).max() * scale
        want, want_lse = OB.attention(qd, b.rows("k", 0), b.rows("v", 0), scale, True)
        step = mj.BlockStep(max_num_seqs=1, q_len=1, h_q=rows, h_k=1, d=d, with_lse=True)
        step.plan(b.lens, 1)
        out = torch.empty(1, rows, d, dtype=torch.bfloat16, device="cuda")
        step.run(q.cuda(), out, kv, b.table_dev, b.lens_dev, 1, float(scale))
        assert np.abs(step.lse.cpu().numpy().reshape(rows) - want_lse[0]).max() <= tol, (down, tol)


# ------------------------------------------------------------------------------------------------- a step in one graph
@pytest.mark.parametrize("h_q", [8, 32])  # 4 and 16 rows a KV head
@pytest.mark.parametrize("splits", [1, 2])
def test_a_batch_written_prompted_and_decoded_in_one_captured_graph(h_q, splits):
    """write, prompt (and join), write, decode, join, captured once and replayed with other slots, chunks, lengths, tokens and plans,
    nothing waited for between."""
    import paged_fp8_decode_gb300 as mj

    B, T = 3, 60
    b = Batch([400, 300, 200], seed=13, spread=(-10, -6))
    kv = b.kv()
    held = [130, 0, 77]  # tokens of each request so far
    i32 = dict(dtype=torch.int32, device="cuda")
    slots, slots1 = torch.full((T,), -1, dtype=torch.int64, device="cuda"), torch.full((B,), -1, dtype=torch.int64, device="cuda")
    lens, lens1, starts = torch.zeros(B, **i32), torch.zeros(B, **i32), torch.zeros(B + 1, **i32)
    x, x1 = D.queries(b, T, 4, 1), D.queries(b, B, 4, 2)
    q, q1 = D.queries(b, T, h_q, 3), D.queries(b, B, h_q, 4)
    out = torch.empty(T, h_q, 128, dtype=torch.bfloat16, device="cuda")
    out1 = torch.empty(B + 2, h_q, 128, dtype=torch.bfloat16, device="cuda")
    chunks = mj.PromptStep(max_tokens=T, max_num_seqs=B, max_q_len=T, max_len=400, h_q=h_q, h_k=2, d=128, splits=splits, with_lse=True)
    step = mj.BlockStep(max_num_seqs=B, q_len=1, h_q=h_q, h_k=2, d=128, with_lse=True)
    write, write1 = mj.block_write_args(x[:, :2], x[:, 2:], slots, kv), mj.block_write_args(x1[:, :2], x1[:, 2:], slots1, kv)
    attend = chunks.args(q, out, kv, b.table_dev, lens, starts, B, 128 ** -0.5)
    attend1 = step.args(q1, out1, kv, b.table_dev, lens1, B, 128 ** -0.5)

    def calls():
        mj.mj_block_write_kv(write)
        mj.mj_block_prompt(attend)
        mj.mj_block_write_kv(write1)
        mj.mj_block_attention(attend1)

    step.plan(np.zeros(B, np.int32), B)
    calls()  # nothing to do: no slots, no chunks, no lengths
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()

    def write_on_host(t, at):
        for name, part in (("k", t[:, :2]), ("v", t[:, 2:])):
            b.codes[name], b.exps[name] = OB.write(part.double().cpu().numpy(), at, b.codes[name], b.exps[name])
        if hasattr(b, "_vals"):
            del b._vals

    for turn, new in enumerate(([20, 33, 7], [1, 0, 40], [3, 5, 1], [0, 0, 60], [10, 10, 10])):
        x.copy_(D.queries(b, T, 4, 10 + turn, size=1.25 ** turn))  # (later tokens are larger: earlier codes move)
        x1.copy_(D.queries(b, B, 4, 20 + turn, size=2.0))
        q.copy_(D.queries(b, T, h_q, 30 + turn, size=0.7))
        q1.copy_(D.queries(b, B, h_q, 40 + turn, size=0.7))
        pos = [held[i] + np.arange(new[i]) for i in range(B)]
        at = np.full(T, -1, np.int64)
        at[:sum(new)] = np.concatenate([b.table[i][p // 16] * 16 + p % 16 for i, p in enumerate(pos)])
        after = np.array([held[i] + new[i] for i in range(B)], np.int32)
        at1 = np.array([b.table[i][n // 16] * 16 + n % 16 if n else -1 for i, n in enumerate(after)], np.int64)
        last = np.where(after > 0, after + 1, 0).astype(np.int32)
        slots.copy_(up(at))
        slots1.copy_(up(at1))
        lens.copy_(up(after))
        lens1.copy_(up(last))
        starts.copy_(up(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)))
        for t in (out, out1, chunks.lse, step.lse):
            t.fill_(SENTINEL)
        step.plan(last, B)
        g.replay()
        torch.cuda.synchronize()
        write_on_host(x, at)
        b.lens = after
        P.check(b, new, out, chunks.lse, q)
        write_on_host(x1, at1)
        b.lens = last
        D.check_decode(b, q1, out1, step.lse, 1, h_q)
        held = [int(n) for n in last]
    assert mj.mj_workspace_status(chunks.workspace) == 0 and mj.mj_workspace_status(step.workspace) == 0
    for name, codes, exps in (("k", kv.k_cache, kv.k_exp), ("v", kv.v_cache, kv.v_exp)):
        nan = (b.codes[name] & 0x7F) == 0x7F
        got = codes.cpu().numpy()
        assert np.array_equal(got[~nan], b.codes[name][~nan]) and np.array_equal(exps.cpu().numpy(), b.exps[name])
