"""Ends of the accepted ranges on the host: what is past them is refused before any launch."""
import ctypes

import pytest
import torch

import draft_block_verification_amd as sd

lib = ctypes.CDLL(sd.LIB_PATH)
FAKE = ctypes.c_void_p(0x10000)          # aligned, never dereferenced on the host
i64, sz = ctypes.c_int64, ctypes.c_size_t


@pytest.mark.parametrize("rows,d", [((1 << 27) - 7, 1024), (1 << 17, 1 << 20), (1 << 18, 1 << 20),
                                    (2 ** 31 - 1, 128)])
def test_mxfp4_rows_past_a_launch(rows, d):
    """A launch has under 2^32 threads, of 32 columns each at the most: 2^37 columns and more
    are a shape error, not a failed launch."""
    for f, a in ((lib.sd_mxfp4_quantize, [FAKE, 1, rows, d, i64(d), FAKE, FAKE, None]),
                 (lib.sd_mxfp4_dequantize, [FAKE, FAKE, rows, d, FAKE, 1, i64(d), None])):
        assert f(*a) == 2


def test_mxfp4_tiles_past_a_launch():
    """2^24 tiles of 64 rows by 128 columns are 2^32 threads."""
    size = lib.sd_mxfp4_head_bytes
    size.restype = ctypes.c_size_t
    rows, d = 1 << 17, 1 << 20               # 2^11 groups of 2^13 steps
    assert size(rows, d) == 0 and size(rows - 64, d) == ((1 << 24) - (1 << 13)) * 4352
    assert sd.mxfp4_logits_workspace_bytes(rows, d) == 0 < sd.mxfp4_logits_workspace_bytes(rows - 64, d)
    assert lib.sd_mxfp4_head(FAKE, FAKE, rows, d, FAKE, sz(1 << 62), None) == 2
    logits = lambda M, V: lib.sd_mxfp4_logits(FAKE, 1, M, 128, i64(128), FAKE, V, FAKE, 1, i64(V), FAKE,
                                              sz(1 << 62), None)
    assert logits(1 << 17, 1 << 21) == 2     # 2^10 by 2^14 output tiles
    assert logits(2 ** 31 - 1, 1 << 21) == 2


@pytest.mark.parametrize("bad", [dict(temperature=1e39), dict(temperature=[1.0, 3.5e38]), dict(top_k=float("inf")),
                                 dict(top_k=[1, float("-inf")]), dict(temperature=torch.tensor([1e300], dtype=torch.float64))])
def test_settings_past_their_type(bad):
    """A finite temperature that fp32 holds as infinity would count as 0, the greedy choice."""
    with pytest.raises(ValueError):
        sd.SamplingParams(device="cpu", **bad)


def test_settings_at_the_end_of_their_type():
    big = torch.finfo(torch.float32).max
    p = sd.SamplingParams(big, 2 ** 31 - 1, float("inf"), float("inf"), device="cpu")
    assert p.temperature.tolist() == [big] and p.top_k.tolist() == [2 ** 31 - 1]
