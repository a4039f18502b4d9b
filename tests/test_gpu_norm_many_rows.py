"""The norms' launch shapes of many rows (from 2048 on: 64, 128, 256 and 512 threads a row with two chunks
each; 64 threads with one, 1024 with two and four as for few rows) with everything that a call may ask
for. Tolerance: the norm is formed in fp64 (some 1e-15 off), rounded to fp32 (2^-24 relative) and to its
type (eps / 2 relative); sums and MXFP8 codes are equal."""
import numpy as np
import pytest
import torch

import _narrow as N
import draft_block_verification_amd as sd

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]
SHAPES = [(2100, 40), (2049, 504), (2050, 1000), (2048, 1024), (2049, 1496), (2051, 4008), (2048, 7168), (2048, 9000)]


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    yield


def inputs(rows, d, dtype, residual):
    return N.rand(rows, d, dtype, rows + d), N.rand(rows, d, residual, d), 1 + 0.2 * N.rand(1, d, torch.float32, 3)[0]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,d", SHAPES + [(2048, 20000)])
def test_residual_sum_weight(rows, d, dtype):
    """A residual of both types, its sum kept, weights with an offset, both results in place."""
    for kind in {dtype, torch.float32}:
        x, r, w = inputs(rows, d, dtype, kind)
        s, y = N.norm(x, w, r, 1e-5, 0.5)
        total = torch.empty_like(r, device="cuda")
        got = sd.sd_rms_norm(x.cuda(), w.cuda(), r.cuda(), 1e-5, 0.5, total=total)
        N.check_rounded(got, y, dtype)
        assert torch.equal(total.cpu(), s)
        a, b = x.cuda(), r.cuda()
        sd.sd_rms_norm(a, w.cuda(), b, 1e-5, 0.5, out=a, total=b)
        assert torch.equal(a, got) and torch.equal(b, total)
        a, b = x.cuda(), r.cuda()
        if kind == dtype:
            sd.sd_rms_norm(a, w.cuda(), b, 1e-5, 0.5, out=b, total=a)
            assert torch.equal(b, got) and torch.equal(a, total)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,d", SHAPES)
def test_mxfp8(rows, d, dtype):
    for kind in {dtype, torch.float32}:
        x, r, w = inputs(rows, d, dtype, kind)
        s, y = N.norm(x, w, r)
        rc, rs = N.mx8_quantize(y.astype(np.float32).astype(np.float64))
        b = r.cuda()
        codes, scales = sd.sd_rms_norm_mxfp8(x.cuda(), w.cuda(), b, total=b)
        assert np.array_equal(scales.cpu().numpy(), rs) and np.array_equal(codes.cpu().numpy(), rc)
        assert torch.equal(b.cpu(), s)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,d", [(2049, 503), (2050, 1001), (2048, 1495), (2051, 4001), (2048, 7167)])
def test_rows_of_wider_tensors(rows, d, dtype):
    """Odd offsets and widths: elements one by one; what lies between the rows and behind them stays."""
    x, r, w = inputs(rows, d, dtype, dtype)
    s, y = N.norm(x, w, r)
    a, b = (torch.full((rows + 1, d + 9), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    a[:rows, 3:3 + d], b[:rows, 5:5 + d] = x.cuda(), r.cuda()
    out = torch.full((rows + 1, d + 11), 5.0, dtype=dtype, device="cuda")
    sd.sd_rms_norm(a[:rows, 3:3 + d], w.cuda(), b[:rows, 5:5 + d], out=out[:rows, 7:7 + d], total=b[:rows, 5:5 + d])
    N.check_rounded(out[:rows, 7:7 + d], y, dtype)
    assert torch.equal(b[:rows, 5:5 + d].cpu(), s)
    assert bool((out[:, :7] == 5).all()) and bool((out[:, 7 + d:] == 5).all()) and bool((out[rows] == 5).all())
    assert bool((b[:, :5] == 7).all()) and bool((b[:, 5 + d:] == 7).all()) and bool((b[rows] == 7).all())
    assert torch.equal(a[:rows, 3:3 + d].cpu(), x) and bool((a[rows] == 7).all())


def test_not_finite_rows():
    """NaN and infinities stay in their rows."""
    rows, d = 2051, 1496
    x = N.rand(rows, d, torch.bfloat16, 1)
    x[5, 7], x[1000, 1495], x[2050, 0] = float("nan"), float("inf"), -float("inf")
    x[7] = 0
    _, y = N.norm(x, None, None, 0.0)
    N.check_rounded(sd.sd_rms_norm(x.cuda(), eps=0.0), y, torch.bfloat16)
    rc, rs = N.mx8_quantize(y.astype(np.float32).astype(np.float64))
    codes, scales = sd.sd_rms_norm_mxfp8(x.cuda(), eps=0.0)
    assert np.array_equal(scales.cpu().numpy(), rs) and np.array_equal(codes.cpu().numpy(), rc)
