"""Sizes past 32 bits: the library takes sizes as 32-bit integers, and a larger one, cut to them, would
be a call on a few rows or columns that says nothing of the rest."""
import pytest
import torch

import draft_block_verification_amd as sd

FAR = 2 ** 32 + 128


@pytest.mark.parametrize("d", [FAR, 2 ** 31, -2 ** 32 + 128, 0, 12])
def test_columns(d):
    with pytest.raises(ValueError):
        sd.mxfp4_columns(d)


def test_workspace_bytes():
    assert sd.mxfp8_logits_workspace_bytes(4, 128) > 0 and sd.w4_logits_workspace_bytes(4, 128, 32) > 0
    for far in (FAR, 2 ** 31, -2 ** 32 + 128):
        for f in (sd.mxfp4_logits_workspace_bytes, sd.mxfp8_logits_workspace_bytes, sd.sample_workspace_bytes):
            assert f(far, 128) == 0 and f(4, far) == 0
        assert sd.accept_filtered_workspace_bytes(far, 4, 128) == 0 and sd.accept_filtered_workspace_bytes(4, 4, far) == 0
        for a in ((far, 128, 32), (4, far, 32), (4, 128, far)):
            assert sd.w4_logits_workspace_bytes(*a) == 0


@pytest.mark.gpu
def test_far_rows_and_columns_are_refused():
    """2^32 + 128 rows, and as many columns."""
    x = torch.empty(FAR, dtype=torch.bfloat16, device="cuda")
    for t in (x.view(FAR, 1), x.view(1, FAR)):
        for f in (sd.sd_rms_norm, sd.sd_rms_norm_mxfp8, sd.sd_mxfp8_quantize, sd.sd_mxfp4_quantize, sd.sd_w4_quantize,
                  sd.Mxfp8Weights.from_tensor, sd.W4Weights.from_tensor):
            with pytest.raises(ValueError):
                f(t)
        with pytest.raises(ValueError):
            sd.sd_rms_norm(t, residual=t, total=t)
        with pytest.raises(ValueError):
            sd.sd_sample(t, torch.zeros(1, device="cuda"), sd.SamplingParams([1.0], None, None, None))
    head = sd.W4Weights.from_tensor(torch.ones((8, 128), device="cuda"))
    for rows in (x.view(FAR, 1), x.view(1, FAR)):
        with pytest.raises(ValueError):
            sd.sd_w4_logits(rows, head)
    del x, rows, t
    codes = torch.zeros((1, FAR // 2), dtype=torch.uint8, device="cuda")
    scales = torch.ones((1, FAR // 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        sd.sd_w4_dequantize(codes, scales, None, FAR)
    with pytest.raises(ValueError):
        sd.W4Weights(codes, scales, None, FAR)
    with pytest.raises(ValueError):
        sd.sd_mxfp8_dequantize(codes[:, :128].contiguous(), torch.zeros((1, 4), dtype=torch.uint8, device="cuda"), FAR)
    del codes, scales
    torch.cuda.empty_cache()
