"""The rotated writes and the latent attention on the host, beside
test_rope_latent_host.py: what the plan says of its lengths, refusals."""

import types

import numpy as np
import pytest
import torch

import paged_fp8_decode_gb300 as mj


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_fp8_decode_gb300.build import build

    build()


@pytest.mark.parametrize("margin", [0, 1, 130])
def test_plan_states_the_tiles_of_every_request(margin):
    lens = np.array([1, 0, 128, 129, 131072, 127], np.int32)
    plan = mj.mj_latent_plan(lens, 6, 9, 12, 1, 16, margin)
    words = (9 + 3) // 4 * 4
    assert len(plan) == mj.mj_latent_plan_size(12, 9) and len(plan) % 4 == 0
    tiles = plan[-words:]
    assert tiles[:6].tolist() == [-(-(int(n) + margin) // 128) if n else 0 for n in lens] and not tiles[6:].any()


def test_a_plan_on_another_device_is_refused(monkeypatch):
    # its default stream would be the current device's, in no order with the attention
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    step = mj.LatentStep.__new__(mj.LatentStep)
    step.plan_dev = types.SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="cuda:1"):
        step.plan(np.array([5], np.int32), 1)
