"""The rotated appends with more CTAs than are resident at once: there a thread
takes up to six slots and a CTA more tokens (the split of every real prompt). The
checks are test_gpu_rope_write's; token counts that leave the last CTA a part of
its tokens."""

import pytest
import torch

from tests import test_gpu_rope_write as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_fp8_decode_gb300.build import build

    build()


def tokens_a_cta(T, slots, d):
    """The launch's split: (more than one wave, tokens a CTA)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    lanes_cta = 128 // (d // 16)

    def group(per_thread):
        lanes = 1
        while lanes < lanes_cta and lanes * per_thread < slots:
            lanes *= 2
        return lanes_cta // lanes

    many = -(-T // group(2)) > 7 * sms
    return many, group(6 if many else 2)


@pytest.mark.parametrize("case", [
    dict(T=1501, h_q=32, h_k=8, d=128, rot=128, inter=False, fmt="fp8", head_scale=True),
    dict(T=1201, h_q=12, h_k=4, d=256, rot=96, inter=True, fmt="fp8", pad=7, axes=3),
    dict(T=4501, h_q=0, h_k=4, d=128, rot=64, inter=False, fmt="fp8", nhd=True),
    dict(T=1301, h_q=24, h_k=4, d=128, rot=112, inter=False, fmt="fp8", inplace=True),
    dict(T=1301, h_q=24, h_k=4, d=128, rot=128, inter=False, fmt="e2m3"),
    dict(T=1301, h_q=24, h_k=4, d=128, rot=48, inter=True, fmt="e2m1", pad=4, nhd=True),
    dict(T=1201, h_q=12, h_k=4, d=256, rot=240, inter=False, fmt="e3m2"),
])
def test_rope_write(case):
    many, group = tokens_a_cta(case["T"], case["h_q"] + 2 * case["h_k"], case["d"])
    assert many and group > 1 and case["T"] % group
    w = W.make(case, case["T"])
    W.check_rotated(w, *W.call(w))


@pytest.mark.parametrize("T,h,inter,axes,pad,pitch,ps", [(5001, 16, True, 1, 7, 576, 64), (1403, 60, False, 2, 0, 640, 16)])
def test_latent_write(T, h, inter, axes, pad, pitch, ps):
    many, group = tokens_a_cta(T, h + 9, 64)
    assert many and group > 1 and T % group
    W.test_latent_write(T, h, inter, axes, pad, pitch, ps)
