"""The block-scaled cache on the GPU against oracle.block (float64): the write (bit for bit), reading
back (bit for bit) and decode attention.

Tolerance of the attention. A query enters exactly (bf16 as two e4m3 terms), so logits are
float32 sums of at most 256 exact products: off by at most 256 * 2^-24 times the sum of their
sizes, some 1e-4 of a nat here, and 2^-19 for the exponent's addition: LSE within 4e-4. A weight
is within 2^-8 of itself, uniform in a step that shrinks with its residual: 0.0015 rms; the output's
rounding (bf16) within 2^-9, 0.0017 rms: 0.0023 in the 2-norm, which random errors add up in -> 0.004.
Elementwise: a row's weights below 2^-10 of its largest (pair A alone, up to 1024 keys) are off by 2^-18 of it each, so
2^-8 together; the others by 2^-8 of themselves; the rounding 2^-9: 0.01 of the largest V that the
codes could stand for."""

import numpy as np
import pytest
import torch

from oracle import block as OB
from tests._block import SENTINEL, Batch, bf16, up

pytestmark = pytest.mark.gpu

REL, ELEM, LSE_TOL = 0.004, 0.01, 4e-4


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_fp8_decode_gb300.build import build

    build()


# ------------------------------------------------------------------------------------------------- the write
def make_write(runs, *, h_k=2, d=128, page=16, block=16, pages=40, seed=0, pad=(), values=None, order="phtd", special=False):
    """runs: (first slot, tokens); pad: positions of the call at which a padding token is put in."""
    rng = np.random.default_rng(seed)
    slots = np.concatenate([np.arange(a, a + n) for a, n in runs]).astype(np.int64)
    for at in sorted(pad):
        slots = np.insert(slots, at, -1 - at)
    T = len(slots)
    x = rng.standard_normal((2, T, h_k, d)) * 2.0 ** rng.integers(-8, 9, (2, T, 1, 1))
    if special:
        flat = x.reshape(-1)
        at = rng.permutation(flat.size)[:flat.size // 50]
        flat[at] = rng.choice([np.inf, -np.inf, np.nan, 0.0, -0.0, 3e38, -1e-39, 1e-20], at.size)
    b = Batch([1], h_k=h_k, d=d, page=page, block=block, extra=pages - 1, seed=seed, order=order)
    for name in "kv":  # any codes but NaN, any exponents
        c = rng.integers(0, 127, b.codes[name].shape).astype(np.uint8) | (rng.integers(0, 2, b.codes[name].shape) << 7).astype(np.uint8)
        b.codes[name] = c
        b.exps[name] = rng.integers(110, 140, b.exps[name].shape).astype(np.uint8)
    qkv = torch.cat([bf16(x[0]), bf16(x[1])], 1).cuda()  # one projection's output
    return b, qkv[:, :h_k], qkv[:, h_k:], slots


def check_write(b, k, v, slots, **kw):
    import paged_fp8_decode_gb300 as mj

    kv = b.kv()
    want = [OB.write(x.double().cpu().numpy(), slots, b.codes[n], b.exps[n]) for x, n in ((k, "k"), (v, "v"))]
    mj.mj_block_write_kv(mj.block_write_args(k, v, up(slots), kv, **kw))
    torch.cuda.synchronize()
    for (c, e), gc, ge in zip(want, (kv.k_cache, kv.v_cache), (kv.k_exp, kv.v_exp)):
        gc, ge = gc.cpu().numpy(), ge.cpu().numpy()
        assert np.array_equal(ge, e), np.argwhere(ge != e)[:5]
        nan = (c & 0x7F) == 0x7F
        assert np.array_equal((gc & 0x7F) == 0x7F, nan)
        assert np.array_equal(gc[~nan], c[~nan]), np.argwhere((gc != c) & ~nan)[:5]


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("page,block", [(16, 16), (32, 16), (32, 32), (64, 64), (128, 16), (128, 32), (128, 64), (128, 128)])
def test_write_of_ragged_runs(page, block, d):
    b, k, v, slots = make_write([(5, 1), (page, block - 1), (3 * page + block // 2, 2 * block + 3), (7 * page + 3, 4),
                                 (9 * page, 1), (12 * page + 1, page)], d=d, page=page, block=block, pad=(0, 3, 40))
    check_write(b, k, v, slots)


@pytest.mark.parametrize("h_k", [1, 3, 8, 20])
def test_write_of_one_token_and_of_many(h_k):
    for runs in ([(37, 1)], [(0, 1)], [(15, 1)], [(16 * i + i % 16, 1) for i in range(40)], [(0, 640)]):
        check_write(*make_write(runs, h_k=h_k, seed=h_k))


def test_write_of_a_long_call():
    # more windows than resident CTAs, runs off the windows' edges
    check_write(*make_write([(7, 9000), (9100, 7001)], h_k=2, pages=1010, seed=3))


def test_write_in_any_order_inside_a_block():
    b, k, v, slots = make_write([(3, 13), (32, 16), (53, 6)], seed=5)
    by = np.concatenate([np.random.default_rng(0).permutation(13), 13 + np.random.default_rng(1).permutation(16), [29, 31, 30, 34, 33, 32]])
    check_write(b, k[by], v[by], slots[by])


@pytest.mark.parametrize("gap", [1, 31, 32, 33, 127, 128])
def test_padding_inside_a_run(gap):
    check_write(*make_write([(20, 9)], pad=range(4, 4 + gap), seed=gap))
    check_write(*make_write([(0, 40)], pad=range(21, 21 + gap), seed=gap, page=128, block=128))


@pytest.mark.parametrize("gap", [129, 255, 256, 257, 289, 1000, 5000])
def test_far_padding_inside_a_run(gap):
    check_write(*make_write([(20, 9)], pad=range(4, 4 + gap), seed=gap))
    check_write(*make_write([(0, 40), (60, 70)], pad=range(21, 21 + gap), seed=gap, page=128, block=128))


def test_padding_before_and_behind():
    check_write(*make_write([(20, 40)], pad=list(range(700)) + list(range(740, 1500)), seed=1))
    check_write(*make_write([(20, 3), (39, 2)], pad=list(range(3, 400)) + list(range(402, 1500)), seed=2, block=16))


def test_rows_left_out_inside_a_run():
    b, k, v, slots = make_write([(18, 10)], seed=6)
    keep = [0, 1, 4, 5, 9]
    check_write(b, k[keep], v[keep], slots[keep])


def test_write_of_infinities_nan_and_extremes():
    check_write(*make_write([(3, 200)], special=True, seed=8))
    check_write(*make_write([(3, 100)], special=True, seed=9, page=64, block=64, d=256))


@pytest.mark.parametrize("order", ["ptht", "tphd", "hptd", "pthd"])
def test_write_into_other_layouts(order):
    order = {"ptht": "phtd"}.get(order, order)
    check_write(*make_write([(3, 100), (200, 7)], order=order, page=32, block=16, seed=10))


def test_write_skips_and_reports_slots_past_the_pool():
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    b, k, v, slots = make_write([(3, 30)], seed=11)
    slots[[4, 20]] = [40 * 16, 2 ** 40]
    check_write(b, k, v, slots, status=status)
    assert status.item() == 1
    b, k, v, slots = make_write([(3, 30)], seed=11, pad=(2,))
    status.zero_()
    check_write(b, k, v, slots, status=status)
    assert status.item() == 0


def test_growing_block_token_by_token():
    import paged_fp8_decode_gb300 as mj

    b, k, v, slots = make_write([(16, 16)], seed=12)
    kv = b.kv()
    codes, exps = b.codes["k"], b.exps["k"]
    for t in range(16):
        codes, exps = OB.write(k[t:t + 1].double().cpu().numpy(), slots[t:t + 1], codes, exps)
        mj.mj_block_write_kv(mj.block_write_args(k[t:t + 1], v[t:t + 1], up(slots[t:t + 1]), kv))
    assert np.array_equal(kv.k_cache.cpu().numpy(), codes) and np.array_equal(kv.k_exp.cpu().numpy(), exps)


def test_write_of_nothing():
    import paged_fp8_decode_gb300 as mj

    b, k, v, slots = make_write([(3, 5)], seed=13)
    check_write(b, k[:0], v[:0], slots[:0])
    check_write(b, k, v, np.full(5, -1))
    assert mj.MJ_OK == 0


def test_write_into_a_cache_past_32_bits():
    # a pool of over 2^32 bytes: the last pages' offsets need 64 bits
    import paged_fp8_decode_gb300 as mj

    pages, page, h_k, d = 140000, 128, 2, 128
    kv = mj.BlockKV.empty(pages, page, h_k, d, 128)
    assert kv.k_cache.numel() > 2 ** 32
    k, v = torch.randn(2, 4, h_k, d, device="cuda").to(torch.bfloat16)
    slots = torch.arange(4, device="cuda") + (pages - 1) * page + 60
    mj.mj_block_write_kv(mj.block_write_args(k, v, slots, kv))
    kr = torch.empty(4, h_k, d, dtype=torch.bfloat16, device="cuda")
    table = torch.full((1, 1), pages - 1, dtype=torch.int32, device="cuda")
    mj.mj_block_read_kv(mj.block_read_args(kv, table, torch.tensor([0, 4], dtype=torch.int32, device="cuda"), kr,
                                           first=torch.tensor([60], dtype=torch.int32, device="cuda")))
    assert ((kr.float() - k.float()).abs() <= k.float().abs() / 16 + 1e-2).all()


# ------------------------------------------------------------------------------------------------- reading back
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,page,block,h_k", [(128, 16, 16, 8), (256, 64, 16, 3), (128, 128, 128, 1), (256, 32, 32, 2)])
def test_read(d, page, block, h_k, dtype):
    import paged_fp8_decode_gb300 as mj

    lens = [1, 0, 77, 300, 0, 33, 64]
    b = Batch(lens, h_k=h_k, d=d, page=page, block=block, seed=d + page)
    kv = b.kv()
    first = np.array([0, 0, 5, 131, 0, 1, 0], np.int32)
    n = np.array(lens) - first
    starts = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    for f, st in ((first, starts), (None, np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))):
        rows = int(st[-1])
        buf = torch.full((rows + 9, 2, h_k, d + 8), SENTINEL, dtype=dtype, device="cuda")
        k_out, v_out = buf[:, 0, :, :d], buf[:, 1, :, :d]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        mj.mj_block_read_kv(mj.block_read_args(kv, b.table_dev, up(st), k_out, v_out, first=None if f is None else up(f), status=status))
        for name, out in (("k", k_out), ("v", v_out)):
            want = np.concatenate([b.rows(name, i)[0 if f is None else f[i]:] for i in range(len(lens))])
            want = torch.from_numpy(want).to(dtype).cuda()
            assert torch.equal(out[:rows], want)
            assert (out[rows:] == SENTINEL).all() and (buf[..., d:] == SENTINEL).all()
        assert status.item() == 0
        one = torch.full((rows, h_k, d), SENTINEL, dtype=dtype, device="cuda")
        mj.mj_block_read_kv(mj.block_read_args(kv, b.table_dev, up(st), v_out=one, first=None if f is None else up(f)))
        assert torch.equal(one, v_out[:rows])


def test_read_of_bad_pages_and_of_fewer_rows():
    import paged_fp8_decode_gb300 as mj

    b = Batch([40, 20], seed=2)
    kv = b.kv()
    b.table_dev[0, 1] = b.pages
    b.table_dev[1, 0] = -5
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((60, 2, 128), SENTINEL, dtype=torch.bfloat16, device="cuda")
    st = up(np.array([0, 40, 70], np.int32))  # more than the outputs' rows
    mj.mj_block_read_kv(mj.block_read_args(kv, b.table_dev, st, out, status=status))
    want = np.concatenate([b.rows("k", 0, 40), b.rows("k", 1, 20)])
    want[16:32] = 0
    want[40:56] = 0
    assert torch.equal(out.double().cpu(), torch.from_numpy(want)) and status.item() == 1
    status.zero_()  # past the block table
    mj.mj_block_read_kv(mj.block_read_args(kv, b.table_dev[:1, :2], up(np.array([0, 33], np.int32)), out[:33], status=status))
    assert status.item() == 1 and (out[32] == 0).all()


# ------------------------------------------------------------------------------------------------- decode attention
def queries(b, rows, h_q, seed=0, size=1.0):
    return bf16(np.random.default_rng(seed).standard_normal((rows, h_q, b.d)) * size).cuda()


def check_rows(got, lse, want, want_lse, vmax, rel=REL, elem=ELEM, lse_tol=LSE_TOL):
    err = np.abs(got - want)
    assert np.all(np.isfinite(got)) and err.max(initial=0) <= elem * vmax, (err.max(), vmax)
    assert np.linalg.norm(err) <= rel * np.linalg.norm(want) + 1e-30, np.linalg.norm(err) / np.linalg.norm(want)
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(lse), empty) and np.all(got[empty] == 0)
    assert np.abs(lse[~empty] - want_lse[~empty]).max(initial=0) <= lse_tol, np.abs(lse[~empty] - want_lse[~empty]).max()


def decode(b, q, q_len, h_q, *, causal=True, dtype=torch.bfloat16, lens=None, extra=0, **kw):
    import paged_fp8_decode_gb300 as mj

    kv = b.kv()
    step = mj.BlockStep(max_num_seqs=b.B + extra, q_len=q_len, h_q=h_q, h_k=b.h_k, d=b.d, causal=causal, with_lse=True, **kw)
    step.lse.fill_(SENTINEL)
    step.plan(b.lens if lens is None else lens, b.B)
    out = torch.full((b.B * q_len + 2, h_q, b.d), SENTINEL, dtype=dtype, device="cuda")
    step.run(q, out, kv, b.table_dev, b.lens_dev, b.B, b.d ** -0.5)
    status = mj.mj_workspace_status(step.workspace)
    return out, step.lse, status


def check_decode(b, q, out, lse, q_len, h_q, causal=True, **kw):
    got = out.double().cpu().numpy()
    assert np.all(got[b.B * q_len:] == SENTINEL)
    r = h_q // b.h_k
    lse = lse.cpu().numpy().reshape(-1, b.h_k, q_len, r).transpose(0, 2, 1, 3).reshape(-1, q_len, h_q)
    got = got[:b.B * q_len].reshape(b.B, q_len, h_q, b.d)
    qd = q.double().cpu().numpy().reshape(-1, q_len, h_q, b.d)
    for i in range(b.B):
        if b.lens[i] == 0:
            assert np.all(got[i] == SENTINEL) and np.all(lse[i] == SENTINEL)
            continue
        want, want_lse = OB.attention(qd[i], b.rows("k", i), b.rows("v", i), b.d ** -0.5, causal)
        check_rows(got[i], lse[i], want, want_lse, b.vmax(i), **kw)


@pytest.mark.parametrize("h_q,h_k,q_len,d", [(4, 1, 1, 128), (8, 8, 1, 128), (32, 8, 1, 128), (16, 2, 1, 128), (10, 2, 1, 256),
                                             (32, 2, 1, 256), (40, 1, 1, 128), (8, 2, 3, 128), (32, 8, 4, 128), (16, 1, 5, 256)])
def test_decode_of_short_and_odd_lengths(h_q, h_k, q_len, d):
    b = Batch([1, 0, 2, 15, 16, 17, 127, 128, 129, 300, 0], h_k=h_k, d=d, seed=h_q + q_len)
    q = queries(b, b.B * q_len, h_q)
    out, lse, status = decode(b, q, q_len, h_q)
    assert status == 0
    check_decode(b, q, out, lse, q_len, h_q)


@pytest.mark.parametrize("page,block", [(32, 16), (64, 32), (128, 128), (128, 16)])
@pytest.mark.parametrize("order", ["phtd", "pthd"])
def test_decode_of_pages_blocks_and_layouts(page, block, order):
    b = Batch([5, 700, 64, 2000], page=page, block=block, order=order, seed=page + block)
    q = queries(b, b.B, 8)
    for dtype in (torch.bfloat16, torch.float16):
        out, lse, status = decode(b, q, 1, 8, dtype=dtype)
        assert status == 0
        check_decode(b, q, out, lse, 1, 8)


@pytest.mark.parametrize("lens,h_k,h_q,q_len", [([20000], 2, 8, 1), ([9000, 40, 3000], 1, 16, 2), ([30000], 8, 64, 4),
                                                ([4000] * 3 + [10] * 60, 8, 32, 1), ([16000] + [100] * 90, 4, 16, 1)])
def test_decode_of_split_requests(lens, h_k, h_q, q_len):
    b = Batch(lens, h_k=h_k, page=64, block=32, seed=len(lens))
    q = queries(b, b.B * q_len, h_q)
    out, lse, status = decode(b, q, q_len, h_q)
    assert status == 0
    check_decode(b, q, out, lse, q_len, h_q)


def test_decode_without_a_causal_limit():
    b = Batch([1, 3, 200], seed=4)
    q = queries(b, b.B * 4, 8)
    out, lse, status = decode(b, q, 4, 8, causal=False)
    check_decode(b, q, out, lse, 4, 8, causal=False)


@pytest.mark.parametrize("spread", [(-32, 32), (-25, -24), (20, 32), (-32, -32)])
def test_decode_of_scales_far_apart(spread):
    # blocks of one request 2^64 apart: small logits from small queries, every weight counts
    b = Batch([40, 900, 5000], seed=5, spread=(-6, -3))
    rng = np.random.default_rng(0)
    live = b.exps["v"] > 0
    live &= b.exps["v"] < 255
    b.exps["v"][live] = rng.integers(127 + spread[0], 128 + spread[1], live.sum())
    q = queries(b, b.B, 8)
    out, lse, status = decode(b, q, 1, 8)
    assert status == 0
    check_decode(b, q, out, lse, 1, 8)


def test_decode_where_the_seen_keys_are_the_small_ones():
    # query tokens 0 and 1 do not see the last keys, whose V is 2^20 times the others': their rows are as exact as any
    b = Batch([66, 34], page=16, seed=6, spread=(-20, -20))
    for i, n in enumerate(b.lens):
        e = b.exps["v"]
        e[b.table[i, (n - 1) // 16]] = 127
    q = queries(b, b.B * 4, 8)
    out, lse, status = decode(b, q, 4, 8)
    got = out.double().cpu().numpy()[:8].reshape(2, 4, 8, 128)
    qd = q.double().cpu().numpy().reshape(2, 4, 8, 128)
    for i in range(2):
        want, _ = OB.attention(qd[i], b.rows("k", i), b.rows("v", i), 128 ** -0.5, True)
        for t in range(4):
            assert np.linalg.norm(got[i, t] - want[t]) <= REL * np.linalg.norm(want[t])


def test_decode_of_one_dominant_key_and_of_equal_keys():
    b = Batch([3000, 500], seed=7)
    q = queries(b, 2, 8)
    for i in range(2):  # a key that every head looks at
        pg, row = b.table[i, 7], 3
        b.codes["k"][pg, row] = np.abs(b.codes["k"][pg, row].view(np.int8)).view(np.uint8)
    q[0] = q[0].abs() * 3
    q[1] = 0
    out, lse, status = decode(b, q, 1, 8)
    check_decode(b, q, out, lse, 1, 8)


def test_queries_that_are_not_finite_stay_in_their_rows():
    b = Batch([300, 40], h_k=2, seed=8)
    q = queries(b, 2 * 2, 8)
    q[1, 5, 3], q[2, 0, 100] = float("inf"), float("nan")
    out, lse, status = decode(b, q, 2, 8)
    assert torch.isnan(out[1, 5]).all() and torch.isnan(out[2, 0]).all()
    ok = q.clone()
    ok[1, 5, 3], ok[2, 0, 100] = 0, 0
    want, _, _ = decode(b, ok, 2, 8)
    keep = torch.ones(4, 8, dtype=torch.bool)
    keep[1, 5] = keep[2, 0] = False
    assert torch.equal(out[:4][keep], want[:4][keep])


def test_query_rows_of_very_different_size():
    b = Batch([400], h_k=1, seed=9)
    q = queries(b, 1, 8)
    q *= torch.tensor([2.0 ** -i for i in range(0, 24, 3)], device="cuda")[None, :, None].to(torch.bfloat16)
    out, lse, status = decode(b, q, 1, 8)
    check_decode(b, q, out, lse, 1, 8)


def test_lengths_shorter_and_longer_than_planned():
    b = Batch([1000, 300, 50], seed=10)
    q = queries(b, 3, 8)
    out, lse, status = decode(b, q, 1, 8, lens=np.array([5000, 4000, 700], np.int32))  # an upper bound
    assert status == 0
    check_decode(b, q, out, lse, 1, 8)
    out, lse, status = decode(b, q, 1, 8, lens=np.array([1000, 128, 0], np.int32))
    assert status == 4


def test_pages_outside_the_pool_and_past_the_table():
    import paged_fp8_decode_gb300 as mj

    b = Batch([200, 90], seed=11)
    kv = b.kv()
    b.table_dev[0, 2], b.table_dev[1, 0] = b.pages + 5, -3
    q = queries(b, 2, 8)
    out, lse, status = decode(b, q, 1, 8)
    assert status == 1 and torch.isfinite(out[:2].float()).all()
    step = mj.BlockStep(max_num_seqs=2, q_len=1, h_q=8, h_k=2, d=128)
    step.plan(b.lens, 2)
    good = Batch([200, 90], seed=11)
    good.kv()
    step.run(q, out, kv, good.table_dev[:, :4], good.lens_dev, 2, 0.1)  # 64 tokens of table
    assert mj.mj_workspace_status(step.workspace) == 1


def test_a_plan_captured_in_a_graph_and_replayed_with_others():
    import paged_fp8_decode_gb300 as mj

    b = Batch([3000, 0, 130, 20], seed=12)
    kv = b.kv()
    q = queries(b, 4, 8)
    step = mj.BlockStep(max_num_seqs=4, q_len=1, h_q=8, h_k=2, d=128, with_lse=True)
    out = torch.full((4 + 2, 8, 128), SENTINEL, dtype=torch.bfloat16, device="cuda")
    args = step.args(q, out, kv, b.table_dev, b.lens_dev, 4, 128 ** -0.5)
    step.plan(b.lens, 4)
    mj.mj_block_attention(args)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mj.mj_block_attention(args)
    for lens in ([3000, 0, 130, 20], [1, 0, 17, 20], [2999, 0, 129, 0], [700, 0, 1, 5]):
        b.lens = np.array(lens, np.int32)
        b.lens_dev.copy_(up(b.lens))
        step.plan(b.lens, 4)
        out.fill_(SENTINEL)
        step.lse.fill_(SENTINEL)
        g.replay()
        torch.cuda.synchronize()
        check_decode(b, q, out, step.lse, 1, 8)


def test_write_then_attend_then_read_on_a_side_stream():
    # a decode step: the newest tokens are written, attended to and read back, nothing waited for between
    import paged_fp8_decode_gb300 as mj

    b = Batch([33, 300, 1, 160], seed=13, spread=(-9, -8))
    kv = b.kv()
    before = b.lens - 1
    stream = torch.cuda.Stream()
    x = queries(b, 4, 4, seed=3, size=2.0)
    k, v = x[:, :2], x[:, 2:]
    slots = up((b.table[np.arange(4), before // 16] * 16 + before % 16).astype(np.int64))
    want = [OB.write(t.double().cpu().numpy(), slots.cpu().numpy(), b.codes[n], b.exps[n]) for t, n in ((k, "k"), (v, "v"))]
    q = queries(b, 4, 8)
    out = torch.full((6, 8, 128), SENTINEL, dtype=torch.bfloat16, device="cuda")
    step = mj.BlockStep(max_num_seqs=4, q_len=1, h_q=8, h_k=2, d=128, with_lse=True)
    starts = up(np.concatenate([[0], np.cumsum(b.lens)]).astype(np.int32))
    rows = torch.empty(int(b.lens.sum()), 2, 128, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        step.plan(b.lens, 4)
        mj.mj_block_write_kv(mj.block_write_args(k, v, slots, kv))
        step.run(q, out, kv, b.table_dev, b.lens_dev, 4, 128 ** -0.5)
        mj.mj_block_read_kv(mj.block_read_args(kv, b.table_dev, starts, v_out=rows))
    stream.synchronize()
    b.reload()
    for n, (c, e) in zip("kv", want):
        live = (c & 0x7F) != 0x7F
        assert np.array_equal(b.exps[n], e) and np.array_equal(b.codes[n][live], c[live])
    check_decode(b, q, out, step.lse, 1, 8)
    assert torch.equal(rows.cpu(), torch.from_numpy(np.concatenate([b.rows("v", i) for i in range(4)])).to(torch.bfloat16))


def test_two_steps_of_one_batch_give_the_same_bits():
    b = Batch([5000, 300], seed=14)
    q = queries(b, 2, 8)
    one, _, _ = decode(b, q, 1, 8)
    two, _, _ = decode(b, q, 1, 8)
    assert torch.equal(one, two)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("q_len", [1, 2, 4])  # 8, 16 and 32 rows
def test_any_channel_of_a_query_that_is_not_finite(q_len, d):
    b = Batch([40, 300, 17], h_k=1, d=d, seed=21)
    q = queries(b, 3 * q_len, 8)
    out0, lse0, _ = decode(b, q, q_len, 8, causal=False)
    bad = q.clone()
    for n in range(3 * q_len * 4):
        bad[n // 4, 2 * (n % 4), (n * 9) % d] = [float("inf"), float("-inf"), float("nan")][n % 3]
    out, lse, status = decode(b, bad, q_len, 8, causal=False)
    hit = ~torch.isfinite(bad).all(2)
    rows = hit.view(3, 1, q_len * 8)  # (query token, head), as the sums of weights
    assert status == 0 and torch.isnan(out[:3 * q_len][hit]).all() and torch.isfinite(out[:3 * q_len][~hit]).all()
    assert torch.isnan(lse[rows]).all() and torch.isfinite(lse[~rows]).all()
    if q_len > 1:  # (a row's own scale: the others keep their bits)
        assert torch.equal(out[:3 * q_len][~hit], out0[:3 * q_len][~hit]) and torch.equal(lse[~rows], lse0[~rows])


def test_a_query_of_nan_over_split_requests():
    b = Batch([9000, 40], h_k=1, page=64, block=32, seed=15)
    q = queries(b, 2, 8)
    q[0, 2, 7], q[1, 6, 0] = float("nan"), float("-inf")
    out, lse, status = decode(b, q, 1, 8)
    nan = torch.zeros(2, 8, dtype=torch.bool)
    nan[0, 2] = nan[1, 6] = True
    assert torch.equal(torch.isnan(out[:2]).all(2).cpu(), nan) and torch.equal(torch.isnan(out[:2]).any(2).cpu(), nan)
    assert torch.equal(torch.isnan(step_lse(lse, 2, 8)).cpu(), nan)


def step_lse(lse, B, h_q):
    return lse.reshape(B, h_q)


@pytest.mark.parametrize("h_q,h_k,q_len,d", [(36, 1, 1, 128), (128, 1, 1, 128), (43, 1, 3, 128), (64, 1, 5, 128), (40, 1, 1, 256), (43, 1, 3, 256)])
def test_decode_of_many_rows(h_q, h_k, q_len, d):
    # 33 rows and more a KV head: one row tile, one of 256 rows, several
    b = Batch([1, 0, 2, 130, 900, 5000], h_k=h_k, d=d, page=32, block=16, seed=h_q)
    q = queries(b, b.B * q_len, h_q)
    for causal in (True, False):
        out, lse, status = decode(b, q, q_len, h_q, causal=causal)
        assert status == 0
        check_decode(b, q, out, lse, q_len, h_q, causal=causal)


@pytest.mark.parametrize("h_q", [8, 32])
def test_a_request_that_was_not_planned_is_reported(h_q):
    b = Batch([300, 200], seed=16)
    q = queries(b, 2, h_q)
    out, lse, status = decode(b, q, 1, h_q, lens=np.array([300, 0], np.int32))
    assert status == 4 and (out[1] == SENTINEL).all() and (out[0] != SENTINEL).all()
    b.lens[1] = 0
    b.lens_dev.copy_(up(b.lens))
    out, lse, status = decode(b, q, 1, h_q)
    assert status == 0
    check_decode(b, q, out, lse, 1, h_q)


@pytest.mark.parametrize("h_q", [8, 32])
def test_two_steps_at_once_on_two_streams(h_q):
    import paged_fp8_decode_gb300 as mj

    batches = [Batch([20000, 300], h_k=2, page=64, block=32, seed=17), Batch([50, 9000, 1], h_k=2, page=64, block=32, seed=18)]
    qs = [queries(b, b.B, h_q, seed=i) for i, b in enumerate(batches)]
    want = [decode(b, q, 1, h_q)[0][:b.B].clone() for b, q in zip(batches, qs)]
    steps, args, outs = [], [], []
    for b, q in zip(batches, qs):
        step = mj.BlockStep(max_num_seqs=b.B, q_len=1, h_q=h_q, h_k=2, d=128)
        step.plan(b.lens, b.B)
        outs.append(torch.zeros(b.B, h_q, 128, dtype=torch.bfloat16, device="cuda"))
        args.append(step.args(q, outs[-1], b.kv(), b.table_dev, b.lens_dev, b.B, 128 ** -0.5))
        steps.append(step)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in batches]
    for _ in range(20):
        for s, a in zip(streams, args):
            mj.mj_block_attention(a, s)
    torch.cuda.synchronize()
    for o, w, st in zip(outs, want, steps):
        assert torch.equal(o, w) and mj.mj_workspace_status(st.workspace) == 0


def test_the_plan_lengths_and_table_rewritten_right_before():
    # what the call reads early is only a guess: the batch before it lies in other pages, with other lengths
    import paged_fp8_decode_gb300 as mj

    for h_q in (8, 32):
        b = Batch([4000, 130, 0, 77], h_k=2, seed=19)
        kv = b.kv()
        q = queries(b, 4, h_q)
        step = mj.BlockStep(max_num_seqs=4, q_len=1, h_q=h_q, h_k=2, d=128, with_lse=True)
        out = torch.full((4 + 2, h_q, 128), SENTINEL, dtype=torch.bfloat16, device="cuda")
        table, lens = torch.zeros_like(b.table_dev), torch.zeros_like(b.lens_dev)
        args = step.args(q, out, kv, table, lens, 4, 128 ** -0.5)
        step.plan(np.array([50, 3000, 900, 0], np.int32), 4)
        mj.mj_block_attention(args)
        out.fill_(SENTINEL)
        step.lse.fill_(SENTINEL)
        step.plan(b.lens, 4)
        new = step.plan_dev.clone()
        step.plan(np.array([50, 3000, 900, 0], np.int32), 4)
        mj.mj_workspace_status(step.workspace)
        table.copy_(b.table_dev)
        lens.copy_(b.lens_dev)
        step.plan_dev.copy_(new)
        mj.mj_block_attention(args)
        torch.cuda.synchronize()
        assert mj.mj_workspace_status(step.workspace) == 0
        check_decode(b, q, out, step.lse, 1, h_q)
