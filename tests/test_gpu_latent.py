"""Latent-cache attention on the GPU against float64 (oracle.rope).

Tolerance. Elementwise: 2e-2 max|V| at most and 2e-3 max|V| on average, the
bound of every decode path here. And in the 2-norm, which random errors add up
in: a weight is within 2^-7 of itself, uniform in a step that shrinks with its
residual: 0.0015 rms; a query value within 2^-8, 0.0013 rms, so a logit is off
by 0.0013 of its own spread (softmax_scale |q| |k|, the logits' standard
deviation sigma for independent inputs, below 1.8 here) and the output by at
most twice that (numerator and denominator); the output's rounding 2^-8 at
most, 0.0017 rms (bf16):
  sqrt(0.0015^2 + (2 * 1.8 * 0.0013)^2 + 0.0017^2) = 0.0052 -> 0.0065.
The LSE: a weight sum in float32 over weights whose logits are off by
0.0013 * 1.8 each at random; at least one key, so 5 sigma: 0.012."""

import numpy as np
import pytest
import torch

from oracle import rope as OR

pytestmark = pytest.mark.gpu

SENTINEL = -12288.0
REL, LSE_TOL = 0.0065, 0.012


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_fp8_decode_gb300.build import build

    build()


def e4m3(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.float8_e4m3fn)


class Case:
    """A batch: codes, block table, queries. Every byte that no token holds is a NaN code."""

    def __init__(self, lens, q_len, h, page, seed=0, pitch=576, causal=True, sink=None, table_len=None, dtype=torch.bfloat16):
        rng = np.random.default_rng(seed)
        self.lens, self.q_len, self.h, self.page, self.causal = np.array(lens, np.int32), q_len, h, page, causal
        self.B, self.dtype = len(lens), dtype
        self.descale = np.array([4 / 448, 5 / 448], np.float32)
        per = [-(-int(n) // page) for n in lens]
        self.pages = sum(per) + 3
        ids = rng.permutation(self.pages)
        self.table = np.full((self.B, table_len or max(per + [1]) + 1), -1, np.int32)
        self.cache = np.full((self.pages, page, pitch), 0x7F, np.uint8)
        at = 0
        self.rows = []
        for b, n in enumerate(lens):
            self.table[b, :per[b]] = ids[at:at + per[b]]
            v = rng.standard_normal((int(n), 576)) * 112  # one unit of the latent is 112 codes
            if sink is not None and n:
                v[sink % int(n)] *= 3.0
            codes = e4m3(np.clip(v, -448, 448)).view(torch.uint8).numpy()
            full = np.full((per[b] * page, 576), 0x7F, np.uint8)
            full[:int(n)] = codes
            self.cache[ids[at:at + per[b]], :, :576] = full.reshape(per[b], page, 576)
            at += per[b]
            f = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
            f[:, :512] *= float(self.descale[0])
            f[:, 512:] *= float(self.descale[1])
            self.rows.append(f)
        self.q = torch.from_numpy(rng.standard_normal((self.B * q_len, h, 576)).astype(np.float32)).to(torch.bfloat16)
        self.scale = 192 ** -0.5
        if sink is not None:
            # queries partly along the sink's key: its logit is some 11 above the others, give or take 5 a head
            for b, n in enumerate(lens):
                if n:
                    k = self.rows[b][sink % int(n)]
                    u = torch.from_numpy((k / np.linalg.norm(k)).astype(np.float32))
                    self.q[b * q_len:(b + 1) * q_len] += (u * 2.2).to(torch.bfloat16)

    def device(self):
        import paged_fp8_decode_gb300 as mj

        up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        pool = up(self.cache)
        return mj.PagedLatent(cache=pool[:, :, :576], descale=up(self.descale), block_table=up(self.table),
                              seq_lens=up(self.lens))

    def step(self, **kw):
        import paged_fp8_decode_gb300 as mj

        kw = dict(dict(max_num_seqs=self.B, q_len=self.q_len, h=self.h, causal=self.causal, with_lse=True), **kw)
        return mj.LatentStep(**kw)

    def expected(self, lens=None):
        lens = self.lens if lens is None else lens
        q = self.q.double().numpy().reshape(self.B, self.q_len, self.h, 576)
        return [OR.latent_attention(q[b], self.rows[b][:int(lens[b])], self.scale, int(lens[b]), self.causal)
                if lens[b] else None for b in range(self.B)]

    def check(self, out, lse, lens=None, want=None, rel=REL, lse_tol=LSE_TOL):
        lens = self.lens if lens is None else lens
        want = self.expected(lens) if want is None else want
        out = out.double().cpu().numpy().reshape(-1, self.q_len, self.h, 512)
        lse = lse.cpu().numpy().reshape(-1, self.q_len, self.h)
        for b in range(self.B):
            if lens[b] == 0:
                assert np.all(out[b] == SENTINEL) and np.all(lse[b] == SENTINEL)
                continue
            o, l = want[b]
            vmax = np.abs(self.rows[b][:int(lens[b]), :512]).max()
            err = np.abs(out[b] - o)
            assert np.all(np.isfinite(out[b])), f"request {b}"
            assert err.max() <= 2e-2 * vmax and err.mean() <= 2e-3 * vmax, (b, err.max(), err.mean(), vmax)
            empty = np.isneginf(l)
            assert np.array_equal(np.isneginf(lse[b]), empty) and np.all(out[b][empty] == 0)
            if not empty.all():
                assert np.linalg.norm(err) <= rel * np.linalg.norm(o), (b, np.linalg.norm(err) / np.linalg.norm(o))
                assert np.abs(lse[b][~empty] - l[~empty]).max() <= lse_tol, np.abs(lse[b][~empty] - l[~empty]).max()

    def outputs(self, extra=0):
        big = torch.full((self.B * self.q_len + extra, self.h, 512), SENTINEL, dtype=self.dtype, device="cuda")
        return big

    def run(self, plan_lens=None, **kw):
        import paged_fp8_decode_gb300 as mj

        step = self.step(**kw)
        step.lse.fill_(SENTINEL)
        step.plan(self.lens if plan_lens is None else plan_lens, self.B)
        out = self.outputs(extra=2)
        step.run(self.q.cuda(), out, self.device(), self.B, self.scale)
        torch.cuda.synchronize()
        assert mj.mj_workspace_status(step.workspace) == 0
        assert bool((out[self.B * self.q_len:] == SENTINEL).all())
        return out[:self.B * self.q_len], step.lse[:self.B]


LENS = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 385, 1000]


@pytest.mark.parametrize("h,q_len", [(1, 1), (8, 1), (16, 1), (17, 1), (32, 1), (33, 1), (64, 1), (65, 1), (128, 1), (130, 1),
                                     (4, 3), (16, 4), (40, 5)])
@pytest.mark.parametrize("page", [16, 64])
def test_lengths_and_rows(h, q_len, page):
    c = Case(LENS, q_len, h, page, seed=h * 8 + q_len)
    c.check(*c.run())


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("sms", [1, 3, 37, 152])
def test_splits(page, sms):
    # from one CTA that runs through every request to requests in many pieces
    c = Case([700, 0, 5000, 3, 1290, 0], 1, 16, page, seed=page + sms)
    c.check(*c.run(sm_count=sms))


@pytest.mark.parametrize("h", [16, 32, 128])
def test_split_rows_of_every_tile(h):
    c = Case([4000, 130, 2049], 2 if h < 128 else 1, h, 64, seed=h)
    c.check(*c.run(sm_count=40))


def test_one_long_request():
    c = Case([131072], 1, 16, 64, seed=3)
    c.check(*c.run())


@pytest.mark.parametrize("causal", [True, False])
def test_query_tokens_before_the_first_key(causal):
    # 5 query tokens over 1 to 6 keys: causal rows that see nothing write 0
    c = Case([1, 2, 3, 4, 5, 6, 0, 131], 5, 7, 16, seed=9, causal=causal)
    c.check(*c.run())


@pytest.mark.parametrize("causal", [True, False])
def test_causal_limit_inside_a_split(causal):
    # the last tiles hold keys that only the later query tokens see
    c = Case([130, 257, 258, 386, 513], 4, 16, 32, seed=10, causal=causal)
    c.check(*c.run(sm_count=64))


@pytest.mark.parametrize("sink,n", [(0, 3000), (1700, 3000), (2999, 3000), (0, 20000)])
@pytest.mark.parametrize("h", [16, 128])
def test_attention_sink(sink, n, h):
    """One key far above the others, whose weights are tiny but many: they must
    keep their share (the reference moves when the sink comes late). The sink's
    row is three times as long as the others', and its logit off by 0.0013 *
    0.0722 |q| |k| = 0.007 rms, the output by up to as much again: 3 sigma and
    the rest, 0.022. The LSE follows that logit, 5 sigma: 0.035."""
    c = Case([n], 1, h, 64, seed=11, sink=sink)
    want = c.expected()
    # the case tells: without the other keys the output would be the sink's row, beyond the tolerance
    off = np.abs(want[0][0][0] - c.rows[0][sink, :512][None]).max()
    assert off > 4e-2 * np.abs(c.rows[0][:, :512]).max()
    out, lse = c.run(sm_count=8)
    c.check(out, lse, want=want, rel=0.022, lse_tol=0.035)


def test_rows_of_very_different_sizes():
    c = Case([500, 90], 1, 24, 16, seed=12)
    c.q *= torch.logspace(-4, 0.3, 24)[None, :, None].to(torch.bfloat16)
    c.q[:, 5] = 0
    c.check(*c.run())


def test_fp16_output_and_strides():
    import paged_fp8_decode_gb300 as mj

    c = Case([300, 77, 0], 2, 5, 64, seed=13, pitch=640, dtype=torch.float16)
    step = c.step()
    step.lse.fill_(SENTINEL)
    step.plan(c.lens, c.B)
    qbig = torch.full((c.B * 2, 7, 600), float("nan"), dtype=torch.bfloat16, device="cuda")
    q = qbig[:, 1:6, 16:592]
    q.copy_(c.q)
    big = torch.full((c.B * 2, 8, 544), SENTINEL, dtype=torch.float16, device="cuda")
    out = big[:, 2:7, 8:520]
    step.run(q, out, c.device(), c.B, c.scale)
    torch.cuda.synchronize()
    assert mj.mj_workspace_status(step.workspace) == 0
    c.check(out.contiguous(), step.lse)
    big[:, 2:7, 8:520] = SENTINEL
    assert bool((big == SENTINEL).all())


def test_lengths_below_the_plan():
    """A plan from upper bounds: device lengths mask, requests that became
    padding write nothing, pieces past the end count nothing."""
    c = Case([900, 5000, 640, 3000], 1, 16, 64, seed=14)
    real = np.array([10, 2000, 0, 3000], np.int32)
    planned = c.lens.copy()
    c.lens = real
    out, lse = c.run(plan_lens=planned, sm_count=30)
    c.check(out, lse, lens=real)


def test_padding_alone_and_no_requests():
    import paged_fp8_decode_gb300 as mj

    c = Case([0, 0, 0], 2, 16, 64, seed=25)
    out, lse = c.run()
    c.check(out, lse)
    step = c.step()
    step.plan(c.lens, 0)
    step.run(c.q.cuda(), out, c.device(), 0, c.scale)
    torch.cuda.synchronize()
    assert bool((out == SENTINEL).all()) and mj.mj_workspace_status(step.workspace) == 0


def test_other_shapes_than_the_step_was_made_for_are_refused():
    c = Case([100, 200], 1, 16, 64, seed=26)
    kv, q, out = c.device(), c.q.cuda(), c.outputs()
    step = c.step()
    with pytest.raises(ValueError, match="requests"):
        step.args(q, out, kv, 3, c.scale)
    with pytest.raises(ValueError, match="rows"):
        step.args(q[:1], out, kv, 2, c.scale)
    with pytest.raises(ValueError, match="q"):
        step.args(q[:, :8], out, kv, 2, c.scale)
    with pytest.raises(ValueError, match="out"):
        step.args(q, out.float(), kv, 2, c.scale)
    with pytest.raises(ValueError, match="seq_lens"):
        kv.seq_lens = kv.seq_lens.long()
        step.args(q, out, kv, 2, c.scale)


def test_bad_page_is_reported():
    import paged_fp8_decode_gb300 as mj

    c = Case([300, 300], 1, 8, 64, seed=15)
    for bad in (-1, c.pages, 2 ** 31 - 1):
        kv = c.device()
        kv.block_table[0, 2] = bad
        step = c.step()
        step.lse.fill_(SENTINEL)
        step.plan(c.lens, c.B)
        out = c.outputs()
        step.run(c.q.cuda(), out, kv, c.B, c.scale)
        torch.cuda.synchronize()
        assert mj.mj_workspace_status(step.workspace) == 1
        # the other request is not touched by it
        want = c.expected()[1][0]
        assert np.linalg.norm(out[1].double().cpu().numpy() - want[0]) <= REL * np.linalg.norm(want[0])


def test_table_shorter_than_the_length_is_reported():
    import paged_fp8_decode_gb300 as mj

    c = Case([300], 1, 8, 64, seed=16)
    kv = c.device()
    kv.block_table = kv.block_table[:, :3].contiguous()
    step = c.step()
    step.plan(c.lens, c.B)
    step.run(c.q.cuda(), c.outputs(), kv, c.B, c.scale)
    torch.cuda.synchronize()
    assert mj.mj_workspace_status(step.workspace) == 1


def test_nan_query_stays_in_its_row():
    c = Case([400], 1, 20, 64, seed=17)
    c.q[0, 3, 100] = float("nan")
    c.q[0, 4, 575] = float("inf")
    out, _ = c.run()
    bad = ~torch.isfinite(out[0]).all(dim=1).cpu()
    assert bad.nonzero()[:, 0].tolist() == [3, 4]


@pytest.mark.parametrize("n,h", [(1, 8), (37, 20), (200, 16), (70, 128)])
def test_nan_query_of_a_request_that_ends_inside_a_tile(n, h):
    """Masked keys beside NaN logits: the row is not taken for one without a key."""
    c = Case([n], 1, h, 64, seed=31)
    c.q[0, 3, 100] = float("nan")
    out, lse = c.run(sm_count=1)
    bad = torch.isnan(out[0]).all(dim=1).cpu()
    assert bad.nonzero()[:, 0].tolist() == [3]
    assert torch.isnan(lse[0]).nonzero()[:, 0].tolist() == [3]
    assert bool(torch.isfinite(out[0][~bad.cuda()]).all())


def test_nan_code_of_the_only_token():
    c = Case([1], 1, 8, 16, seed=32)
    c.cache[c.table[0, 0], 0, 5] = 0x7F
    out, lse = c.run()
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())


def test_offsets_past_32_bits():
    """Pages at the far end of a pool larger than 4 GiB."""
    c = Case([130, 500], 1, 16, 64, seed=18)
    pages = (5 << 30) // (64 * 576)
    pool = torch.zeros(pages, 64, 576, dtype=torch.uint8, device="cuda")
    kv = c.device()
    pool[pages - c.pages:] = kv.cache
    kv.cache = pool
    kv.block_table = torch.where(kv.block_table >= 0, kv.block_table + (pages - c.pages), kv.block_table)
    step = c.step()
    step.lse.fill_(SENTINEL)
    step.plan(c.lens, c.B)
    out = c.outputs()
    step.run(c.q.cuda(), out, kv, c.B, c.scale)
    torch.cuda.synchronize()
    c.check(out, step.lse)


def test_same_page_twice():
    # two requests share their prefix's pages
    c = Case([128, 300], 1, 16, 64, seed=19)
    c.table[1, :2] = c.table[0, :2]
    c.rows[1][:128] = c.rows[0][:128]
    c.check(*c.run())


def test_same_bits_every_time():
    c = Case([3000, 50, 700], 1, 64, 64, seed=20)
    a, la = c.run()
    for _ in range(3):
        b, lb = c.run()
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_two_steps_at_once():
    cases = [Case([2000, 130], 1, 16, 64, seed=21), Case([900, 3000], 1, 64, 32, seed=22)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    held = []
    for c in cases:
        step = c.step()
        step.lse.fill_(SENTINEL)
        step.plan(c.lens, c.B)
        held.append((c, step, c.outputs(), c.q.cuda(), c.device()))
    torch.cuda.synchronize()
    for _ in range(20):
        for (c, step, out, q, kv), s in zip(held, streams):
            step.run(q, out, kv, c.B, c.scale, stream=s)
    torch.cuda.synchronize()
    for c, step, out, _, _ in held:
        c.check(out, step.lse)


def test_captured_step_with_growing_lengths():
    """The step as a program runs it: append the new token's row, attend; one
    graph, replayed with new plans, lengths, slots and positions."""
    import paged_fp8_decode_gb300 as mj

    rng = np.random.default_rng(23)
    B, h, page, steps = 3, 16, 16, 5
    first = np.array([126, 14, 2000], np.int32)
    c = Case(first + steps, 1, h, page, seed=24)
    kv = c.device()
    step = c.step(sm_count=20)
    inv = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    new = torch.zeros(B, 576, dtype=torch.bfloat16, device="cuda")
    q_pe = torch.zeros(B, h, 64, dtype=torch.bfloat16, device="cuda")
    q, out = c.q.cuda(), c.outputs()
    pos = torch.zeros(B, dtype=torch.int64, device="cuda")
    slots = torch.zeros(B, dtype=torch.int64, device="cuda")
    wa = mj.latent_write_args(q_pe, new[:, :512], new[:, 512:], pos, mj.mj_rope_turns(inv).cuda(), slots, kv.cache,
                              kv.descale, q_out=q[:, :, 512:])
    aa = step.args(q, out, kv, B, c.scale)
    step.plan(first, B)
    kv.seq_lens.copy_(torch.from_numpy(first))
    mj.mj_latent_attention(aa)  # the first call of a row tile comes before the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mj.mj_latent_write(wa)
        mj.mj_latent_attention(aa)
    for k in range(steps):
        lens = first + k + 1
        x = torch.from_numpy(rng.standard_normal((B, 576)).astype(np.float32)).to(torch.bfloat16)
        qp = torch.from_numpy(rng.standard_normal((B, h, 64)).astype(np.float32)).to(torch.bfloat16)
        p = lens.astype(np.int64) - 1
        new.copy_(x)
        q_pe.copy_(qp)
        pos.copy_(torch.from_numpy(p))
        slots.copy_(torch.from_numpy(np.array([c.table[b, p[b] // page] * page + p[b] % page for b in range(B)])))
        kv.seq_lens.copy_(torch.from_numpy(lens.astype(np.int32)))
        step.plan(lens, B)
        g.replay()
        torch.cuda.synchronize()
        assert mj.mj_workspace_status(step.workspace) == 0
        # what the write put there, from the cache; what it should be is test_latent_write's
        codes = kv.cache.view(torch.float8_e4m3fn).double().cpu().numpy()
        ang = OR.angles(p, inv)
        want_pe = OR.rotate(x[:, None, 512:].double().numpy(), ang, True)[:, 0]
        for b in range(B):
            row = codes[c.table[b, p[b] // page], p[b] % page]
            c.rows[b][p[b], :512] = row[:512] * float(c.descale[0])
            c.rows[b][p[b], 512:] = row[512:] * float(c.descale[1])
            assert np.abs(c.rows[b][p[b], 512:] - want_pe[b]).max() <= 2.0 ** -4 * np.abs(want_pe[b]).max() + 5 / 448 * 2.0 ** -9
        c.q = q.cpu()
        want_q = OR.rotate(qp.double().numpy(), ang, True)
        assert np.abs(c.q[:, :, 512:].double().numpy() - want_q).max() <= 2.0 ** -8 * np.abs(want_q).max() * 1.01
        c.check(out, step.lse, lens=lens)
