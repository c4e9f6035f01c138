"""Prompt attention over the block-scaled cache on the GPU against oracle.block (float64).

Tolerance. Queries are exact down to 2^-10 of their row's largest value and within 2^-17 of it
below, keys exact: a logit is off by at most 2^-17 |q|max sum|k| scale, below 4e-4 here, in the
sum at random far less; float32 sums as in the decode attention: LSE within 6e-4. Weights in fp16:
2^-12 rms of themselves; the output's rounding 0.0017 rms (bf16), 0.0002 (fp16): 0.0025 in the 2-norm for bf16, 0.0006 for
fp16. Elementwise: a weight within 2^-11 of itself, the rounding 2^-9 (2^-12 fp16): 0.003 of the
largest V that the codes could stand for."""

import numpy as np
import pytest
import torch

from oracle import block as OB
from tests._block import SENTINEL, Batch, bf16, up
from tests.test_gpu_block import check_rows, queries

pytestmark = pytest.mark.gpu

REL = {torch.bfloat16: 0.0025, torch.float16: 0.0006}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_fp8_decode_gb300.build import build

    build()


def run(b, new, h_q, *, causal=True, dtype=torch.bfloat16, q=None, splits=None, max_q_len=None, extra=3, seed=0):
    """The last new[i] tokens of each request as query tokens. (out, lse, status, q)"""
    import paged_fp8_decode_gb300 as mj

    kv = b.kv()
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(starts[-1])
    q = queries(b, T + extra, h_q, seed) if q is None else q
    step = mj.PromptStep(max_tokens=T + extra, max_num_seqs=b.B, max_q_len=max(new) if max_q_len is None else max_q_len,
                         max_len=int(b.lens.max()), h_q=h_q, h_k=b.h_k, d=b.d, causal=causal, splits=splits, with_lse=True)
    step.lse.fill_(SENTINEL)
    out = torch.full((T + extra, h_q, b.d), SENTINEL, dtype=dtype, device="cuda")
    step.run(q, out, kv, b.table_dev, b.lens_dev, up(starts), b.B, b.d ** -0.5)
    return out, step.lse, mj.mj_workspace_status(step.workspace), q


def check(b, new, out, lse, q, causal=True, dtype=torch.bfloat16, elem=0.003):
    starts = np.concatenate([[0], np.cumsum(new)])
    got, lse, qd = out.double().cpu().numpy(), lse.cpu().numpy(), q.double().cpu().numpy()
    assert np.all(got[starts[-1]:] == SENTINEL) and np.all(lse[starts[-1]:] == SENTINEL)
    for i in range(b.B):
        s = slice(starts[i], starts[i + 1])
        if new[i] == 0:
            continue
        if b.lens[i] == 0:
            assert np.all(got[s] == 0) and np.all(np.isneginf(lse[s]))
            continue
        want, want_lse = OB.attention(qd[s], b.rows("k", i), b.rows("v", i), b.d ** -0.5, causal)
        check_rows(got[s], lse[s], want, want_lse, b.vmax(i), rel=REL[dtype], elem=elem, lse_tol=6e-4)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("h_q,h_k", [(4, 1), (8, 8), (16, 2), (10, 2), (3, 1), (64, 1)])
def test_short_and_odd_chunks(h_q, h_k, d):
    new = [1, 0, 5, 64, 65, 3, 1]
    b = Batch([1, 7, 5, 64, 300, 129, 128], h_k=h_k, d=d, seed=h_q + d)
    for dtype in (torch.bfloat16, torch.float16):
        out, lse, status, q = run(b, new, h_q, dtype=dtype)
        assert status == 0
        check(b, new, out, lse, q, dtype=dtype)


@pytest.mark.parametrize("page,block", [(16, 16), (32, 16), (32, 32), (64, 64), (128, 128), (128, 16), (128, 64)])
@pytest.mark.parametrize("order", ["phtd", "pthd"])
@pytest.mark.parametrize("d", [128, 256])
def test_pages_blocks_and_layouts(page, block, order, d):
    new = [200, 33]
    b = Batch([777, 33], page=page, block=block, order=order, d=d, seed=page + block)
    out, lse, status, q = run(b, new, 4)
    assert status == 0
    check(b, new, out, lse, q)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("splits", [1, 2, 3, 7, 64])
def test_keys_in_pieces(splits, d):
    new = [100, 1, 300]
    b = Batch([3000, 500, 300], d=d, seed=splits)
    out, lse, status, q = run(b, new, 4, splits=splits)
    assert status == 0
    check(b, new, out, lse, q)


@pytest.mark.parametrize("d", [128, 256])
def test_a_longer_chunk(d):
    new = [1500]
    b = Batch([4100], d=d, page=64, block=32, seed=1)
    out, lse, status, q = run(b, new, 8)
    check(b, new, out, lse, q)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("h_q,longest", [(2, 9), (2, 33), (4, 30), (4, 70)])
def test_rows_of_every_tile_shape(h_q, longest, d):
    # the longest chunk's rows choose the kernel: up to 32 rows, up to 128, more
    new = [longest, 1, longest // 2, 0]
    b = Batch([900, 1, longest // 2, 50], h_k=1, d=d, page=32, block=32, seed=longest)
    for splits in (1, 3):
        out, lse, status, q = run(b, new, h_q, splits=splits)
        assert status == 0
        check(b, new, out, lse, q)


def test_without_a_causal_limit():
    new = [40, 7]
    b = Batch([333, 7], seed=2)
    for splits in (1, 3):
        out, lse, status, q = run(b, new, 4, causal=False, splits=splits)
        check(b, new, out, lse, q, causal=False)


@pytest.mark.parametrize("splits", [1, 3])
def test_rows_that_see_no_key(splits):
    # more query tokens than the request has keys, and a request without any
    new = [20, 6, 200]
    b = Batch([5, 0, 130], seed=3)
    out, lse, status, q = run(b, new, 4, splits=splits)
    assert status == 0
    check(b, new, out, lse, q)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("spread", [(-32, 32), (20, 32), (-32, -32)])
def test_scales_far_apart(spread, d):
    b = Batch([900, 300], seed=5, spread=(-6, -3), d=d)
    rng = np.random.default_rng(0)
    live = (b.exps["v"] > 0) & (b.exps["v"] < 255)
    b.exps["v"][live] = rng.integers(127 + spread[0], 128 + spread[1], live.sum())
    out, lse, status, q = run(b, [150, 300], 4)
    starts = [0, 150, 450]
    got, qd = out.double().cpu().numpy(), q.double().cpu().numpy()
    for i in range(2):  # every row by itself: as exact where it sees small values alone
        s = slice(starts[i], starts[i + 1])
        want, want_lse = OB.attention(qd[s], b.rows("k", i), b.rows("v", i), d ** -0.5, True)
        err = np.linalg.norm(got[s] - want, axis=2) / np.linalg.norm(want, axis=2)
        assert err.max() <= 2 * REL[torch.bfloat16], err.max()
        assert np.abs(lse.cpu().numpy()[s] - want_lse).max() <= 6e-4


def test_logits_that_rise_and_fall():
    # keys that grow towards the end move every row's reference often; then the same the other way round
    for up_hill in (True, False):
        b = Batch([2000], seed=6, h_k=1)
        n = np.arange(2000) // 16 * 16
        size = np.round(n / 2000 * 9 if up_hill else (2000 - n) / 2000 * 9).astype(int)
        pages, rows = b.table[0][np.arange(2000) // 16], np.arange(2000) % 16
        b.exps["k"][pages, 0, 0] = 127 - 9 + size
        out, lse, status, q = run(b, [500], 4)
        check(b, [500], out, lse, q, elem=0.004)


def test_queries_that_are_not_finite_and_zeros():
    b = Batch([300, 140], seed=8)
    out0, lse0, _, q = run(b, [200, 140], 4)
    bad = q.clone()
    bad[3, 1, 9], bad[250, 2, 0] = float("inf"), float("nan")
    bad[17, 3] = 0
    for splits in (1, 2):
        out, lse, status, _ = run(b, [200, 140], 4, q=bad, splits=splits)
        assert torch.isnan(out[3, 1]).all() and torch.isnan(out[250, 2]).all()
        ref = bad.clone()
        ref[3, 1], ref[250, 2] = 0, 0
        out[3, 1], out[250, 2] = run(b, [200, 140], 4, q=ref, splits=splits)[0][[3, 250], [1, 2]]
        lse[3, 1], lse[250, 2] = run(b, [200, 140], 4, q=ref, splits=splits)[1][[3, 250], [1, 2]]
        check(b, [200, 140], out, lse, ref)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("new", [2, 9, 40])  # 32, 144 and 640 rows
def test_any_channel_that_is_not_finite(new, d):
    """Each place of a 16-byte piece, in every second row: that row is NaN, the others keep their bits."""
    b = Batch([50], h_k=1, d=d, seed=16)
    out0, lse0, _, q = run(b, [new], 16, extra=0)
    bad = q.clone()
    n = 0
    for t in range(new):
        for h in range(t % 2, 16, 2):
            bad[t, h, (n * 9) % d] = [float("inf"), float("-inf"), float("nan")][n % 3]
            n += 1
    out, lse, status, _ = run(b, [new], 16, q=bad, extra=0)
    hit = ~torch.isfinite(bad).all(2)
    assert status == 0 and int(hit.sum()) == 8 * new
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(out[~hit], out0[~hit]) and torch.equal(lse[~hit], lse0[~hit])


@pytest.mark.parametrize("d", [128, 256])
def test_hundreds_of_heads_a_kv_head(d):
    b = Batch([70, 20], h_k=1, d=d, seed=17)
    out, lse, status, q = run(b, [3, 2], 300)
    assert status == 0
    check(b, [3, 2], out, lse, q)


def test_rows_of_very_different_size():
    b = Batch([400], h_k=1, seed=9)
    q = queries(b, 103, 4)
    q *= torch.exp2(-torch.arange(103, device="cuda") * 1.2)[:, None, None].to(torch.bfloat16)
    out, lse, status, _ = run(b, [100], 4, q=q)
    check(b, [100], out, lse, q)


def test_more_query_tokens_than_announced():
    b = Batch([500, 100], seed=10)
    for splits in (1, 2):
        out, lse, status, q = run(b, [300, 20], 4, max_q_len=128, splits=splits)
        assert status == 4
        assert (out[128:300] == SENTINEL).all() and (lse[128:300] == SENTINEL).all()
        full, _, _, _ = run(b, [300, 20], 4, q=q, splits=splits)
        want, want_lse = OB.attention(q[:300].double().cpu().numpy(), b.rows("k", 0), b.rows("v", 0), 128 ** -0.5, True)
        check_rows(out[:128].double().cpu().numpy(), lse[:128].cpu().numpy(), want[:128], want_lse[:128], b.vmax(0), rel=0.0025,
                   elem=0.003, lse_tol=6e-4)
        assert torch.equal(out[300:320], full[300:320])


def test_bad_pages():
    b = Batch([200, 90], seed=11)
    b.kv()
    b.table_dev[0, 2], b.table_dev[1, 0] = b.pages + 5, -3
    out, lse, status, q = run(b, [50, 90], 4)
    assert status == 1 and torch.isfinite(out[:140].float()).all()


def test_a_captured_call_replayed_with_other_chunks():
    import paged_fp8_decode_gb300 as mj

    b = Batch([900, 400, 70], seed=12)
    kv = b.kv()
    q = queries(b, 400, 8)
    out = torch.empty(400, 8, 128, dtype=torch.bfloat16, device="cuda")
    for splits in (1, 3):
        step = mj.PromptStep(max_tokens=400, max_num_seqs=3, max_q_len=300, max_len=900, h_q=8, h_k=2, d=128, splits=splits, with_lse=True)
        starts = up(np.array([0, 300, 340, 400], np.int32))
        args = step.args(q, out, kv, b.table_dev, b.lens_dev, starts, 3, 128 ** -0.5)
        mj.mj_block_prompt(args)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mj.mj_block_prompt(args)
        for new, lens in (([300, 40, 60], [900, 400, 70]), ([0, 1, 200], [5, 17, 70]), ([7, 0, 0], [899, 0, 0])):
            b.lens = np.array(lens, np.int32)
            b.lens_dev.copy_(up(b.lens))
            starts.copy_(up(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)))
            out.fill_(SENTINEL)
            step.lse.fill_(SENTINEL)
            g.replay()
            torch.cuda.synchronize()
            check(b, new, out, step.lse, q)
        b.lens = np.array([900, 400, 70], np.int32)
        b.lens_dev.copy_(up(b.lens))


def test_chunk_written_then_attended_to():
    # prefill in two chunks: each is written, then attends to what is cached by then
    import paged_fp8_decode_gb300 as mj

    lens = [150, 70]
    b = Batch(lens, seed=13, h_k=2)
    kv = b.kv()
    x = queries(b, 220, 4, seed=4, size=2.0)
    at = [0, 150]
    q = queries(b, 220, 8, seed=5)
    done = [0, 0]
    for chunk in ([100, 30], [50, 40]):
        starts = np.concatenate([[0], np.cumsum(chunk)]).astype(np.int32)
        idx = np.concatenate([at[i] + done[i] + np.arange(chunk[i]) for i in range(2)])
        pos = [done[i] + np.arange(chunk[i]) for i in range(2)]
        slots = np.concatenate([b.table[i][pos[i] // 16] * 16 + pos[i] % 16 for i in range(2)]).astype(np.int64)
        kx = x[idx]
        qx = q[idx].contiguous()
        b.lens = np.array([done[i] + chunk[i] for i in range(2)], np.int32)
        b.lens_dev.copy_(up(b.lens))
        step = mj.PromptStep(max_tokens=len(idx), max_num_seqs=2, max_q_len=max(chunk), max_len=150, h_q=8, h_k=2, d=128, with_lse=True)
        out = torch.empty(len(idx), 8, 128, dtype=torch.bfloat16, device="cuda")
        mj.mj_block_write_kv(mj.block_write_args(kx[:, :2], kx[:, 2:], up(slots), kv))
        step.run(qx, out, kv, b.table_dev, b.lens_dev, up(starts), 2, 128 ** -0.5)
        torch.cuda.synchronize()
        b.reload()
        check(b, chunk, out, step.lse, qx)
        done = [done[i] + chunk[i] for i in range(2)]


def test_the_same_bits_twice():
    b = Batch([3000, 700], seed=14)
    for splits in (1, 4):
        one, _, _, q = run(b, [600, 100], 8, splits=splits)
        assert torch.equal(one, run(b, [600, 100], 8, q=q, splits=splits)[0])


@pytest.mark.parametrize("d", [128, 256])
def test_many_calls_in_a_row(d):
    # every wait of every CTA ends by itself, whatever the order in which its warps come to it
    import paged_fp8_decode_gb300 as mj

    new = [40, 300, 130, 200, 7]
    b = Batch([900, 669, 130, 777, 7], d=d, h_k=8, seed=15)
    kv = b.kv()
    starts = up(np.concatenate([[0], np.cumsum(new)]).astype(np.int32))
    q = queries(b, sum(new), 16)
    out = torch.empty(sum(new), 16, d, dtype=torch.bfloat16, device="cuda")
    step = mj.PromptStep(max_tokens=sum(new), max_num_seqs=5, max_q_len=300, max_len=900, h_q=16, h_k=8, d=d, splits=1)
    args = step.args(q, out, kv, b.table_dev, b.lens_dev, starts, 5, d ** -0.5)
    mj.mj_block_prompt(args)
    first = out.clone()
    for _ in range(300):
        mj.mj_block_prompt(args)
    assert mj.mj_workspace_status(step.workspace) == 0 and torch.equal(out, first)
