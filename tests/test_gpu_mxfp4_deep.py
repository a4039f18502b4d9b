"""MXFP4 logits over many 128-column steps, on the GPU against a 64-bit product on the device.

Each tiling of the product (ids x rows of a tile) keeps its operands in 4 LDS stages (256 x 64: in
3) that are written again every so many steps; the depths here pass each stage at least twice, with
odd and even numbers of steps. The sizes name a tiling through the rule that picks one: the
cheapest by rounds of its tiles over 256 compute units.

Tolerance: every product of two values is exact in fp32, and the sum of d of them, in any order,
is off by at most (d - 1) 2^-24 sum |terms|; rounding to bf16 adds eps / 2 of the result."""
import numpy as np
import pytest
import torch

import draft_block_verification_amd as sd
import _filtered as F

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    yield


def values(codes, scales):
    """fp64 values of codes and scales [rows][d / 2], [rows][d / 32] on their device."""
    grid = torch.tensor(np.concatenate([F.GRID, -F.GRID]), dtype=torch.float64, device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], 2).flatten(1).int()
    return grid[c] * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,V,d", [
    (500, 32001, 1152), (500, 32001, 1280), (500, 32001, 7168),      # 256 x 256: 9, 10, 56 steps
    (257, 40000, 1152), (130, 32000, 1280), (130, 32000, 7168),      # 256 x 128
    (100, 65700, 1152), (300, 2049, 1280), (300, 2049, 7296),        # 128 x 128: 9, 10, 57
    (64, 65600, 896), (40, 70001, 928), (64, 33000, 7168),           # 256 x 64: 7, 8 (in part), 56
    (32, 2000, 7296), (16, 2000, 7168), (1, 2000, 1664)])            # streamed: 57, 56, 13
def test_many_steps(M, V, d, out):
    g = torch.Generator("cuda").manual_seed(M + V + d)
    codes = torch.randint(0, 256, (V, d // 2), generator=g, device="cuda").to(torch.uint8)
    scales = torch.randint(122, 130, (V, d // 32), generator=g, device="cuda").to(torch.uint8)
    h = torch.randn((M, d), generator=g, device="cuda").to(torch.bfloat16)
    head = sd.Mxfp4Weights(codes, scales, d)
    got = sd.sd_mxfp4_logits(h, head, dtype=out).double()
    hv = torch.from_numpy(F.mx_values(*F.mx_quantize(h.double().cpu().numpy()), d)).cuda()
    wv = values(codes, scales)
    want, size = hv @ wv.t(), hv.abs() @ wv.abs().t()
    tol = d * 2.0 ** -24 * size
    if out != torch.float32:
        tol = tol + (want.abs() + tol) * torch.finfo(out).eps / 2
    assert bool(((got - want).abs() <= tol).all()), float(((got - want).abs() / tol).max())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_every_code_and_scale_back(dtype):
    """All 16 codes under all 256 scales: the value rounded once to the type, subnormal and past
    its largest (infinite) included; a scale byte of 255 is NaN."""
    codes = np.tile(np.array([(2 * i + 1) << 4 | 2 * i for i in range(8)], dtype=np.uint8), (256, 8))
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 4, axis=1)
    got = sd.sd_mxfp4_dequantize(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), 128, dtype).cpu()
    with np.errstate(over="ignore"):
        want = torch.from_numpy(F.mx_values(codes, scales, 128)).to(dtype)
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and bool(torch.isnan(got[255]).all())
    assert torch.equal(got[:255], want[:255])
    assert torch.equal(torch.signbit(got[:255]), torch.signbit(want[:255]))
