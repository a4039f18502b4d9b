"""What a caller passes as a workspace: one block of memory on the device. An expanded tensor counts
bytes that it does not have, a host tensor's address is not the device's."""
import pytest
import torch

import draft_block_verification_amd as sd
from draft_block_verification_amd import _lib


def test_no_tensor_and_host_tensor():
    for bad in ([0] * 4096, 4096, None):
        with pytest.raises(TypeError):
            _lib._space(bad)
    with pytest.raises(ValueError):
        _lib._space(torch.empty(4096, dtype=torch.uint8))


def calls():
    """Each call that takes a workspace, as a function of it."""
    B, g, d, V = 2, 3, 128, 96
    hidden = torch.ones((B, g + 1, d), dtype=torch.bfloat16, device="cuda")
    lm = torch.ones((V, d), dtype=torch.bfloat16, device="cuda")
    drafts = torch.zeros((B, g), dtype=torch.int32, device="cuda")
    q = torch.zeros((B, g, V), dtype=torch.bfloat16, device="cuda")
    z = torch.zeros((B * (g + 1), V), device="cuda")
    stats = torch.zeros((B * (g + 1), 4), dtype=torch.int64, device="cuda")
    ua, ur = torch.full((B, g), 0.5, device="cuda"), torch.full((B, g + 1), 0.5, device="cuda")
    params = sd.SamplingParams([1.0] * B, [4] * B, None, None)
    rows = hidden.view(-1, d)
    u = torch.full((B,), 0.5, device="cuda")
    heads = sd.Mxfp4Weights.from_tensor(lm), sd.Mxfp8Weights.from_tensor(lm), sd.W4Weights.from_tensor(lm)
    return {
        "verify": lambda w: sd.sd_verify_logits(hidden, lm, drafts, workspace=w),
        "contraction": lambda w: sd.sd_verify_contraction(hidden, lm, workspace=w),
        "greedy": lambda w: sd.sd_verify_greedy(hidden, lm, drafts, workspace=w),
        "rejection": lambda w: sd.sd_accept_rejection(z, stats, q, drafts, None, None, ua, ur, 1.0, workspace=w),
        "mxfp4": lambda w: sd.sd_mxfp4_logits(rows, heads[0], workspace=w),
        "mxfp8": lambda w: sd.sd_mxfp8_logits(rows, heads[1], workspace=w),
        "w4": lambda w: sd.sd_w4_logits(rows, heads[2], workspace=w),
        "sample": lambda w: sd.sd_sample(z[:B], u, params, workspace=w),
        "filtered": lambda w: sd.sd_accept_filtered(z, q, drafts, None, None, ua, ur, params, workspace=w),
    }


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["verify", "contraction", "greedy", "rejection", "mxfp4", "mxfp8", "w4", "sample", "filtered"])
def test_refused_by_each_call(name):
    f = calls()[name]
    one = torch.empty(1, dtype=torch.uint8, device="cuda")
    for bad in (one.expand(1 << 24), torch.empty((2, 1 << 24), dtype=torch.uint8, device="cuda").t(),
                torch.empty(1 << 24, dtype=torch.uint8)):
        with pytest.raises(ValueError):
            f(bad)
    with pytest.raises(TypeError):
        f([0] * 4096)
