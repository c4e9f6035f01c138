"""The latent attention's calls as programs make them: plans that no longer hold
the lengths, a step made on a busy stream, and what the kernel reads before it
waits for the preceding one."""

import numpy as np
import pytest
import torch

from tests.test_gpu_latent import SENTINEL, Case

pytestmark = pytest.mark.gpu

BAD_PLAN = 4


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_fp8_decode_gb300.build import build

    build()


def attend(c, plan_lens, planned_seqs=None, **kw):
    import paged_fp8_decode_gb300 as mj

    step = c.step(**kw)
    step.lse.fill_(SENTINEL)
    step.plan(plan_lens, len(plan_lens) if planned_seqs is None else planned_seqs)
    out = c.outputs()
    step.run(c.q.cuda(), out, c.device(), c.B, c.scale)
    torch.cuda.synchronize()
    return out, step.lse[:c.B], mj.mj_workspace_status(step.workspace)


@pytest.mark.parametrize("h", [16, 128])
@pytest.mark.parametrize("sms", [1, 40, None])
def test_length_past_the_plan_is_reported(h, sms):
    c = Case([300, 1281, 0, 5], 1, h, 64, seed=1)
    # 1281 tokens reach into an eleventh tile: a plan for ten drops the newest one
    assert attend(c, np.array([300, 1280, 0, 5], np.int32), sm_count=sms)[2] == BAD_PLAN
    # growth inside the last planned tile is served
    out, lse, status = attend(c, np.array([257, 1281, 0, 1], np.int32), sm_count=sms)
    assert status == 0
    c.check(out, lse)
    # a margin that covers it
    out, lse, status = attend(c, np.array([300, 1280, 0, 5], np.int32), sm_count=sms, margin=1)
    assert status == 0
    c.check(out, lse)


@pytest.mark.parametrize("planned", [[300, 700, 0], [300, 700]])
def test_live_request_without_a_plan_is_reported(planned):
    c = Case([300, 700, 90], 1, 16, 64, seed=2)
    out, _, status = attend(c, np.array(planned, np.int32))
    assert status == BAD_PLAN
    assert bool((out[2] == SENTINEL).all())


def test_step_made_on_a_busy_stream_and_used_on_another():
    """The buffers of a new step are ready when it is: work that is still queued
    on the stream where it was made does not clear its plan later."""
    c = Case([700, 2000], 1, 16, 64, seed=3)
    kv, q, out, s = c.device(), c.q.cuda(), c.outputs(), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # a tenth of a second
    step = c.step()
    step.plan(c.lens, c.B, stream=s)
    torch.cuda.synchronize()
    step.lse.fill_(SENTINEL)
    torch.cuda.synchronize()
    step.run(q, out, kv, c.B, c.scale, stream=s)
    torch.cuda.synchronize()
    c.check(out, step.lse)


@pytest.mark.parametrize("h,q_len,sms", [(16, 1, None), (16, 1, 2), (32, 1, None), (128, 1, None), (16, 4, None)])
def test_inputs_rewritten_right_before_the_attention(h, q_len, sms):
    """Before the kernel waits for the preceding one it reads plan, lengths' owner
    and block table to aim prefetches. Here the kernels right before each call
    rewrite the table (to a second copy of the pages; the copy that it leaves holds
    NaN codes), the plan (cut finely, or not at all), the lengths and the queries."""
    import paged_fp8_decode_gb300 as mj

    long, short = np.array([3000, 700, 1290], np.int32), np.array([140, 0, 900], np.int32)
    c = Case(long, q_len, h, 64, seed=4)
    kv = c.device()
    P, pool = c.pages, kv.cache.contiguous()
    both = torch.cat([pool, pool]).contiguous()
    kv.cache = both
    tables = [kv.block_table.clone(), torch.where(kv.block_table >= 0, kv.block_table + P, kv.block_table)]
    step = c.step(sm_count=sms)
    lens = [torch.from_numpy(x).cuda() for x in (long, short)]
    plans = []
    for x in (long, short):
        step.plan(x, c.B)
        torch.cuda.synchronize()
        plans.append(step.plan_dev.clone())
    q, out = c.q.cuda(), c.outputs()
    qs = [q.clone(), (-q).contiguous()]
    aa = step.args(q, out, kv, c.B, c.scale)
    wants = []
    for x, sign in ((long, 1), (short, -1)):
        c.q = c.q * sign
        wants.append(c.expected(x))
        c.q = c.q * sign
    for i in range(6):
        use = i % 2
        out.fill_(SENTINEL)
        step.lse.fill_(SENTINEL)
        stale = both[:P] if use else both[P:]
        stale.fill_(0x7F)
        q.copy_(qs[use])
        kv.seq_lens.copy_(lens[use])
        step.plan_dev.copy_(plans[use])
        kv.block_table.copy_(tables[use])  # the last kernel before the attention
        mj.mj_latent_attention(aa)
        torch.cuda.synchronize()
        assert mj.mj_workspace_status(step.workspace) == 0
        c.check(out, step.lse, lens=(long, short)[use], want=wants[use])
        stale.copy_(pool)
