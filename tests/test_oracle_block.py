"""Pins of oracle.block: the block-scaled cache's write and attention against
properties fixed by its definition, and worked examples."""

import numpy as np
import pytest

from oracle import block as OB
from oracle.formats import e4m3_decode


def test_need_is_the_smallest_scale():
    assert OB.need(448.0) == 127 and OB.need(np.nextafter(448.0, 500)) == 128 and OB.need(224.0) == 126
    assert OB.need(0.0) == 95 and OB.need(1e-30) == 95 and OB.need(1e30) == 159
    for x in np.exp(np.random.default_rng(0).uniform(-18, 18, 200)):
        e = OB.need(x)
        assert x <= 448 * 2.0 ** (e - 127) and (e == 95 or x > 448 * 2.0 ** (e - 128))


def empty(pages=3, page=32, h=2, d=4, block=16):
    rng = np.random.default_rng(1)
    return rng.integers(0, 256, (pages, page, h, d)).astype(np.uint8), rng.integers(0, 256, (pages, h, page // block)).astype(np.uint8)


def test_worked_example():
    codes, exps = empty(h=1)
    x = np.zeros((2, 1, 4))
    x[0, 0] = [448.0, 1.0, -2.0 ** -9, 0.0]
    c1, e1 = OB.write(x[:1], [16], codes, exps)       # page 0, block 1, row 0
    assert e1[0, 0, 1] == 127 and e4m3_decode(c1[0, 16, 0]).tolist() == [448.0, 1.0, -2.0 ** -9, 0.0]
    x[1, 0] = [900.0, 3.0, 1.0, 1.0]                  # needs 2^2: 900 / 448 > 2
    c2, e2 = OB.write(x[1:], [17], c1, e1)
    assert e2[0, 0, 1] == 129
    # 448 / 4 exact; 2^-9 / 4 = 2^-11 is a quarter of the smallest subnormal: 0
    assert e4m3_decode(c2[0, 16, 0]).tolist() == [112.0, 0.25, -0.0, 0.0]
    assert e4m3_decode(c2[0, 17, 0]).tolist() == [224.0, 0.75, 0.25, 0.25]  # 225 lies between 224 and 240
    c3, e3 = OB.write(x[:1] / 1024, [16], c2, e2)     # the block begins anew, its scale falls
    assert e3[0, 0, 1] == 117 and np.array_equal(c3[0, 17], c2[0, 17])
    c4, e4 = OB.write(x[:1] / 1024, [18], c2, e2)     # and stays where earlier tokens do
    assert e4[0, 0, 1] == 129 and np.array_equal(c4[0, 16:18], c2[0, 16:18])


@pytest.mark.parametrize("seed", range(5))
def test_write_touches_its_rows_alone_and_forgets_its_order(seed):
    rng = np.random.default_rng(seed)
    codes, exps = empty(4, 64, 2, 8, 16)
    slots = np.concatenate([np.arange(5, 41), [-1, -7], np.arange(130, 133)])
    x = rng.standard_normal((len(slots), 2, 8)) * 2.0 ** rng.integers(-6, 6, (len(slots), 1, 1))
    c, e = OB.write(x, slots, codes, exps)
    by = rng.permutation(len(slots))
    c2, e2 = OB.write(x[by], slots[by], codes, exps)
    assert np.array_equal(c, c2) and np.array_equal(e, e2)
    rows = np.ones((4, 64), bool).reshape(-1)
    rows[0:41] = rows[128:133] = False                # written, or earlier tokens of a block written into
    assert np.array_equal(c.reshape(256, 2, 8)[rows], codes.reshape(256, 2, 8)[rows])
    blocks = np.ones((4, 4), bool)
    blocks[0, :3] = blocks[2, 0] = False
    assert np.array_equal(e.transpose(0, 2, 1)[blocks], exps.transpose(0, 2, 1)[blocks])
    v = OB.values(c, e).reshape(256, 2, 8)
    live = slots >= 0
    top = np.repeat(2.0 ** (e.astype(int) - 127), 16, axis=2).transpose(0, 2, 1).reshape(256, 2)[slots[live]][..., None]
    err = np.abs(v[slots[live]] - x[live])
    assert np.all(err <= np.maximum(np.abs(x[live]) * 2.0 ** -4, top * 2.0 ** -10))


def test_values_that_are_not_finite():
    codes, exps = empty(h=1)
    x = np.array([[[np.inf, -np.inf, np.nan, 3.0]]])
    c, e = OB.write(x, [0], codes, exps)
    assert e[0, 0, 0] == 120 and e4m3_decode(c[0, 0, 0])[:2].tolist() == [448.0, -448.0]
    assert np.isnan(e4m3_decode(c[0, 0, 0])[2]) and e4m3_decode(c[0, 0, 0])[3] == 384.0


def test_attention_is_softmax_over_what_is_seen():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((3, 4, 8)), rng.standard_normal((5, 2, 8)), rng.standard_normal((5, 2, 8))
    out, lse = OB.attention(q, k, v, 0.3, True)
    for t in range(3):
        for h in range(4):
            w = np.exp(0.3 * k[:3 + t, h // 2] @ q[t, h])
            assert np.allclose(out[t, h], w @ v[:3 + t, h // 2] / w.sum()) and np.isclose(lse[t, h], np.log(w.sum()))
    out, lse = OB.attention(q, k[:2], v[:2], 0.3, True)
    assert np.all(out[0] == 0) and np.all(np.isneginf(lse[0])) and np.allclose(out[1], v[:1].repeat(2, 1)[0])
    assert np.allclose(OB.attention(q, k, v, 0.3, False)[0][2], OB.attention(q, k, v, 0.3, True)[0][2])
