"""The latent attention's two 8-bit terms where they could go wrong: many equal
small weights below a few large ones in one piece, and queries whose logits are
large. tests/test_latent_arithmetic.py has the terms' own properties."""

import numpy as np
import pytest
import torch

from oracle import rope as OR

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_fp8_decode_gb300.build import build

    build()


def attend(codes, q, descale, scale, sm_count, page=64):
    """One request over `codes` [n, 576] (uint8, on the GPU), q [1, h, 576]; the output and the LSE."""
    import paged_fp8_decode_gb300 as mj

    n, h = codes.shape[0], q.shape[1]
    pages = -(-n // page)
    cache = torch.full((pages * page, 576), 0x7F, dtype=torch.uint8, device="cuda")
    cache[:n] = codes
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(n)).cuda()
    pool = torch.empty(pages, page, 576, dtype=torch.uint8, device="cuda")
    pool[order] = cache.view(pages, page, 576)
    kv = mj.PagedLatent(cache=pool, descale=descale, block_table=order.to(torch.int32)[None].contiguous(),
                        seq_lens=torch.tensor([n], dtype=torch.int32, device="cuda"))
    step = mj.LatentStep(max_num_seqs=1, q_len=1, h=h, with_lse=True, sm_count=sm_count)
    step.plan(np.array([n], np.int32), 1)
    out = torch.zeros(1, h, 512, dtype=torch.bfloat16, device="cuda")
    step.run(q, out, kv, 1, scale)
    torch.cuda.synchronize()
    assert mj.mj_workspace_status(step.workspace) == 0
    return out[0].double().cpu(), step.lse[0].double().cpu()


N = 131000  # ends inside a tile


@pytest.fixture(scope="module")
def values():
    g = torch.Generator(device="cuda").manual_seed(4)
    v = 1.0 + 0.25 * torch.randn(N, 512, generator=g, device="cuda")  # a mean of their own: their share shows
    return (v * 112).to(torch.float8_e4m3fn).view(torch.uint8)


@pytest.mark.parametrize("h", [16, 32, 64])
@pytest.mark.parametrize("high", [[0], [70000], [N - 1], [0, 32, 64, 96]])
@pytest.mark.parametrize("n,sms", [(N, 1), (N, None), (16384, 1)])
def test_many_equal_keys_far_below_a_few(values, n, sms, high, h):
    """Every key but those of `high` has the logit 0, those of `high` one of g
    binades, all exactly (one channel decides, its query is 1). In one piece the
    equal weights are 2^(4 - g) (or 2^(6 - g)), rounded alike but for their keys'
    dither: an error of half a step of the second term at most, at random, so
    5 sqrt(n) step / 2 of the row's sum; a weight from 2^-6 on is off by 2^-7.8
    of itself, which moves at most 1/4 of that from one side to the other, values
    4 apart; 2^-25 a weight for float16; 2^-10 for the sums' own 8192 roundings
    of 2^-23; the output's half step 2^-8."""
    codes = torch.zeros(n, 576, dtype=torch.uint8, device="cuda")
    codes[:, :512] = values[:n]
    at = torch.tensor([k % n for k in high], device="cuda")
    codes[at, :512] = torch.tensor([-224.0], device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    codes[at, 512] = torch.tensor([448.0], device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    descale = torch.tensor([1 / 112, 3 / 448], device="cuda")
    q = torch.zeros(1, h, 576, dtype=torch.bfloat16, device="cuda")
    q[:, :, 512] = 1.0
    v = codes[:, :512].view(torch.float8_e4m3fn).float() * descale[0]
    vmax = float(v.abs().max())
    low = v.sum(0, dtype=torch.float64) - v[at].sum(0, dtype=torch.float64)
    low, top = low.cpu(), v[at].sum(0, dtype=torch.float64).cpu()
    logit = float(descale[1].double() * 448)
    for gap in (8.3, 10.3, 11.7, 12.6, 14.8, 16.8, 18.4, 19.3, 20.6, 22.5):
        scale = float(np.float32(gap * np.log(2) / logit))
        w = np.exp(scale * logit)
        want = (w * top + low) / (w * len(high) + n - len(high))
        lse = np.log(w * len(high) + n - len(high))
        out, got_lse = attend(codes, q, descale, scale, sms)
        p, total = 2.0 ** (4 - gap), 16.0 * len(high) + 2.0 ** (4 - gap) * n
        step = 0.0 if p >= 2.0 ** -6 else (2.0 ** -12 if p >= 2.0 ** -10 else max(2.0 ** -16, 2.0 ** (np.floor(np.log2(p)) - 2)))
        tol = vmax * (2.0 ** -7.8 + 2.0 ** -10 + (5 * np.sqrt(n) * step / 2 + n * 2.0 ** -25) / total) + 2.0 ** -8 * want.abs()
        err = (out - want[None]).abs()
        assert bool((err <= tol[None]).all()), (gap, float(err.max()) / vmax, float(tol.max()) / vmax)
        assert float((got_lse - lse).abs().max()) <= 1e-3, gap


@pytest.mark.parametrize("h", [7, 32, 64])
@pytest.mark.parametrize("descale", [(4 / 448, 5 / 448), (-4 / 448, 5 / 448), (0.75 / 448, 5 / 448)])
def test_large_logits_of_exact_queries(h, descale):
    """Queries without a rotary part: bf16 has 8 bits, the two terms 4 each, so
    the logits (6 nats rms) are as exact as their sums: 18 products of a row, each
    rounded to 2^-22 of the terms' sum of sizes, some 20 times the logit's rms:
    18 * 2^-22 * 120 = 5e-4 nats; the LSE as much, and its own 2^-18. Values of a
    thousandth of the row's largest are exact too."""
    n = 700
    rng = np.random.default_rng(h)
    codes = torch.from_numpy(rng.standard_normal((n, 576)) * 112).clamp(-448, 448).float().to(torch.float8_e4m3fn)
    f = codes.double().numpy()
    rows = np.concatenate([f[:, :512] * np.float32(descale[0]), f[:, 512:] * np.float32(descale[1])], axis=1)
    x = rng.standard_normal((1, h, 576)) * 2.0 ** rng.uniform(-8, 0, (1, h, 576))
    x[:, :, 512:] = 0
    q = torch.from_numpy(x).to(torch.bfloat16)
    t = q[0].double().numpy() @ rows.T
    scale = float(np.float32(6 / t.std()))
    want, lse = OR.latent_attention(q.double().numpy(), rows, scale, n, True)
    out, got = attend(codes.view(torch.uint8).cuda(), q.cuda(), torch.tensor(descale, dtype=torch.float32).cuda(), scale, 1)
    assert np.abs(got.numpy() - lse[0]).max() <= 1e-3
    # weights within 2^-7.8 (0.0016 rms), few of them large; bf16
    assert np.linalg.norm(out.numpy() - want[0]) <= 0.0045 * np.linalg.norm(want[0])


@pytest.mark.parametrize("descale", [(0.0, 5 / 448), (4 / 448, 0.0), (0.0, 0.0), (2.0 ** -90, 1.0), (1.0, 2.0 ** -90)])
def test_descales_of_zero_and_far_apart(descale):
    n, h = 300, 16
    rng = np.random.default_rng(8)
    codes = torch.from_numpy(rng.standard_normal((n, 576)) * 112).clamp(-448, 448).float().to(torch.float8_e4m3fn)
    f = codes.double().numpy()
    rows = np.concatenate([f[:, :512] * np.float32(descale[0]), f[:, 512:] * np.float32(descale[1])], axis=1)
    q = torch.from_numpy(rng.standard_normal((1, h, 576))).to(torch.bfloat16)
    spread = (q[0].double().numpy() @ rows.T).std()
    scale = float(np.float32(1 / spread)) if spread else 1.0
    want, lse = OR.latent_attention(q.double().numpy(), rows, scale, n, True)
    out, got = attend(codes.view(torch.uint8).cuda(), q.cuda(), torch.tensor(descale, dtype=torch.float32).cuda(), scale, 1)
    # a logit (1 nat rms) off by 2^-8 of a query value at most, 0.0013 rms: 5 sigma
    assert np.abs(got.numpy() - lse[0]).max() <= 0.0065
    assert np.linalg.norm(out.numpy() - want[0]) <= 0.0065 * np.linalg.norm(want[0])


@pytest.mark.parametrize("descale", [(2.0 ** -30, 1.0), (2.0 ** -60, 1.0), (2.0 ** -17, 1.0), (2.0 ** -16, 1.0), (1.0, 2.0 ** -60)])
def test_queries_of_zero_and_tiny_beside_descales_far_apart(descale):
    """A row's factor is largest where its queries are 0, and may meet the ratio of the descales there."""
    n, h = 200, 16
    rng = np.random.default_rng(9)
    codes = torch.from_numpy(rng.standard_normal((n, 576)) * 112).clamp(-448, 448).float().to(torch.float8_e4m3fn)
    f = codes.double().numpy()
    rows = np.concatenate([f[:, :512] * descale[0], f[:, 512:] * descale[1]], axis=1)
    q = torch.from_numpy(rng.standard_normal((1, h, 576)))
    q[0, 0] = 0
    q[0, 1] *= 2.0 ** -110
    q[0, 2, 512:] = 0
    q = q.to(torch.bfloat16)
    scale = float(np.float32(1 / (q[0].double().numpy() @ rows.T).std()))
    want, lse = OR.latent_attention(q.double().numpy(), rows, scale, n, True)
    out, got = attend(codes.view(torch.uint8).cuda(), q.cuda(), torch.tensor(descale, dtype=torch.float32).cuda(), scale, 1)
    # as above: logits of 1 nat rms, 5 sigma of 0.0013
    assert np.abs(got.numpy() - lse[0]).max() <= 0.0065
    assert np.linalg.norm(out.numpy() - want[0]) <= 0.0065 * np.linalg.norm(want[0])
