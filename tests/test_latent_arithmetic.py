"""The number formats under the latent attention's products, emulated on the CPU
bit by bit (float16 by numpy, e4m3 by the oracle's codec, e5m2 as a float16's
upper byte). Properties that the kernel's accuracy contract (include/mj.h) is
made of; tests/test_gpu_latent_far.py checks the kernel itself.

* A softmax weight p, at most 2^8.5, enters as hi = e4m3(p) and lo, the rest in
  e5m2, by way of float16: within 2^-11 of p, or 2^-25, for that step, and
  - p >= 2^-6: lo to nearest, within 2^-7.8 of p in all;
  - p < 2^-6: lo is rounded up where the key's dither (8 bits of a hash of its
    index) says so. Over the dither's 256 values the two terms add up to the
    float16 weight exactly, so the errors of many equal weights cancel; one
    weight is within max(2^-12, where it holds no hi term its own 2^-2).
* A query value q * 2^k, its row's largest put between 224 and 448, as two e4m3
  terms is exact from 1/4 on (bf16 has 8 bits, the terms 4 each), else within
  2^-10; a rotary value times the descales' ratio within max(2^-8, 2^-10).
"""

import numpy as np
import pytest
import torch

from oracle import formats as F


def e4(x):
    return F.e4m3_decode(F.e4m3_encode(np.asarray(x, np.float32))).astype(np.float64)


def e5m2_of_byte(b):
    return (b.astype(np.uint16) << 8).view(np.float16).astype(np.float64)


def dither(key):
    """The kernel's 8 bits of a key index."""
    u = np.asarray(key, np.uint64) * 0x9E3779B1 & 0xFFFFFFFF
    u ^= u >> 16
    return ((u * 0x9E3779B1 & 0xFFFFFFFF) >> 24).astype(np.uint16)


def weight(p, r):
    """The value that the two terms of p stand for; r: the key's dither."""
    h = np.asarray(p, np.float32).astype(np.float16)
    hi = e4(h.astype(np.float32))
    d = (h - hi.astype(np.float16)).astype(np.float16)  # exact
    assert np.array_equal(d.astype(np.float64), h.astype(np.float64) - hi)
    add = np.where(h < np.float16(2.0 ** -6), np.asarray(r, np.uint16), np.uint16(0x80))
    return hi + e5m2_of_byte((d.view(np.uint16) + add) >> 8)


def nearest_weight(p):
    """Both terms to nearest (hi e4m3, lo e5m2): what a fixed rounding of lo gives."""
    return weight(p, np.uint16(0x80))


def test_dither_takes_every_value_alike():
    # whole tiles, and every 2nd, 3rd, ... key of them: each of 16 bins near its share (5 sigma of a random draw)
    for n, step in ((1 << 17, 1), (1 << 17, 2), (1 << 17, 3), (1 << 17, 16), (1 << 17, 128), (4096, 1)):
        for start in (0, 5):
            c = np.bincount(dither(np.arange(start, n, step)) >> 4, minlength=16)
            share = c.sum() / 16
            assert np.abs(c - share).max() <= 5 * np.sqrt(share)


def test_large_weights():
    p = (2.0 ** np.linspace(-6, 8.5, 200001)).astype(np.float32)
    p[0] = 2.0 ** -6
    err = np.abs(nearest_weight(p) - p)
    assert np.all(err <= 2.0 ** -7.8 * p)
    for r in (0, 77, 255):  # no dither there
        assert np.array_equal(weight(p, r), nearest_weight(p))
    assert np.sqrt(np.mean((err / p) ** 2)) <= 0.0016


def test_small_weights_are_right_on_average():
    p = (2.0 ** np.linspace(-30, -6, 20001)[:-1]).astype(np.float32)
    h = p.astype(np.float16).astype(np.float64)
    assert np.all(np.abs(h - p) <= np.maximum(2.0 ** -11 * p, 2.0 ** -25))
    r = np.arange(256, dtype=np.uint16)
    w = weight(p[:, None], r[None])
    assert np.array_equal(w.mean(axis=1), h)
    err = np.abs(w - h[:, None]).max(axis=1)
    assert np.all(err <= np.maximum(2.0 ** -12, np.where(p < 2.0 ** -10, p / 4, 0)))
    assert np.all(err[p < 2.0 ** -10] <= np.maximum(2.0 ** -16, p[p < 2.0 ** -10] / 4))
    # a fixed rounding would not be: equal weights are off together
    assert np.abs(nearest_weight(p) / p - 1)[(p > 2.0 ** -14) & (p < 2.0 ** -10)].max() > 0.1


def test_no_weight_where_there_is_none():
    assert np.all(weight(np.zeros(256, np.float32), np.arange(256, dtype=np.uint16)) == 0)


@pytest.mark.parametrize("base", [4.0, 6.0])
@pytest.mark.parametrize("n", [16384, 131072])
@pytest.mark.parametrize("gap", [10.3, 12.6, 14.8, 16.8, 18.4, 19.3, 20.6, 22.5])
def test_many_equal_weights_far_below_one(gap, n, base):
    """One key `gap` binades above n - 1 equal ones, whose values have a mean of
    their own: the output with the kernel's weights, the sum with the exact ones.
    A small weight's error has a standard deviation of half its second term's
    step at most; the worst case here, 2^-10.8 (step 2^-13) 131072 times beside
    2^4: 5 sqrt(131072) 2^-14 / 90 = 1.2e-3 of a value."""
    rng = np.random.default_rng(5)
    v = 1.0 + 0.25 * rng.standard_normal((n, 8))
    v[0] = -2.0
    p = np.full(n, 2.0 ** (base - gap), np.float32)
    p[0] = 2.0 ** base
    exact = (p[:, None].astype(np.float64) * v).sum(0) / p.sum(dtype=np.float64)
    got = (weight(p, dither(np.arange(n)))[:, None] * v).sum(0) / p.sum(dtype=np.float64)
    assert np.abs(got - exact).max() <= 1.5e-3 * np.abs(v).max()


def test_query_terms_are_exact_for_bf16():
    rng = np.random.default_rng(1)
    q = torch.from_numpy((rng.standard_normal(200000) * 2.0 ** rng.uniform(-14, 0, 200000)).astype(np.float32))
    q = q.to(torch.bfloat16).double().numpy()
    for top in (1.0, 1.74, 1.75, 1.7578125, 1.9921875, 3e5, 7e-12):
        x = np.append(q / np.abs(q).max(), 0) * top
        x = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
        am = np.float32(np.abs(x).max())
        k = 8 - int(np.frexp(np.float32(am * np.float32(8 / 7)))[1] - 1)
        y = x * 2.0 ** k
        assert 223.9 <= np.abs(y).max() <= 448
        hi = e4(y)
        err = np.abs(hi + e4(y - hi) - y)
        assert np.all(err[np.abs(y) >= 0.25] == 0) and err.max() <= 2.0 ** -10
        z = y * 0.8137  # a rotary value: times the descales' ratio
        hi = e4(z)
        assert np.all(np.abs(hi + e4(z - hi) - z) <= np.maximum(2.0 ** -8 * np.abs(z), 2.0 ** -10))
