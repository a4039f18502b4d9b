"""The RMS norms on the GPU against the 64-bit statement. Tolerance: the norm is formed in fp64
(some 1e-15 off), rounded to fp32 (2^-24 relative) and to its type (eps / 2 relative); sums are
one fp32 addition and one rounding and are equal, and so are the MXFP8 codes of the fp32 value."""
import numpy as np
import pytest
import torch

import _narrow as N
import draft_block_verification_amd as sd

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]
# every launch shape: one wave a row, four waves, sixteen, rows that are read twice
WIDTHS = [1, 2, 7, 8, 33, 511, 512, 513, 1024, 1025, 2048, 2049, 4096, 5000, 7168, 8192, 8200, 16385, 32768, 40001]


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    yield


def cuda(t):
    return None if t is None else t.cuda()


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("dtype", TYPES)
def test_norm(d, dtype):
    rows = 5 if d < 10000 else 2
    x = N.rand(rows, d, dtype, d)
    w = N.rand(1, d, dtype, d + 1)[0]
    for residual, wt, out in ((None, None, dtype), (N.rand(rows, d, dtype, d + 2), w, dtype),
                              (N.rand(rows, d, torch.float32, d + 3), w.float(), torch.bfloat16),
                              (N.rand(rows, d, dtype, d + 4), w.to(torch.float16), torch.float32)):
        s, y = N.norm(x, wt, residual, 1e-5)
        total = None if residual is None else torch.empty_like(residual, device="cuda")
        got = sd.sd_rms_norm(x.cuda(), cuda(wt), cuda(residual), eps=1e-5, dtype=out, total=total)
        N.check_rounded(got, y, out)
        if total is not None:
            assert torch.equal(total.cpu(), s)


@pytest.mark.parametrize("d", [8, 24, 128, 136, 520, 1024, 2048, 2056, 7168, 8200, 33000])
@pytest.mark.parametrize("dtype", TYPES)
def test_norm_mxfp8(d, dtype):
    rows = 6 if d < 10000 else 2
    x, r = N.rand(rows, d, dtype, d, spread=True), N.rand(rows, d, torch.float32, d + 1)
    w = N.rand(1, d, dtype, d + 2)[0]
    for residual, weight in ((None, None), (r, w)):
        _, y = N.norm(x, weight, residual)
        rc, rs = N.mx8_quantize(y.astype(np.float32).astype(np.float64))
        codes, scales = sd.sd_rms_norm_mxfp8(x.cuda(), cuda(weight), cuda(residual))
        assert np.array_equal(scales.cpu().numpy(), rs)
        assert np.array_equal(codes.cpu().numpy(), rc)


@pytest.mark.parametrize("d", [96, 1000, 4096, 36864])
@pytest.mark.parametrize("dtype", TYPES)
def test_in_place(d, dtype):
    """The sum over the residual or over x, the output over x or the residual."""
    x, r = N.rand(3, d, dtype, 1), N.rand(3, d, dtype, 2)
    w = N.rand(1, d, dtype, 3)[0].cuda()
    y = sd.sd_rms_norm(x.cuda(), w, r.cuda())
    s = N.norm(x, None, r)[0]
    a, b = x.cuda(), r.cuda()
    assert torch.equal(sd.sd_rms_norm(a, w, b, total=b), y)
    assert torch.equal(b.cpu(), s) and torch.equal(a.cpu(), x)
    a, b = x.cuda(), r.cuda()
    assert torch.equal(sd.sd_rms_norm(a, w, b, total=a), y)
    assert torch.equal(a.cpu(), s) and torch.equal(b.cpu(), r)
    a, b = x.cuda(), r.cuda()
    sd.sd_rms_norm(a, w, b, total=b, out=a)
    assert torch.equal(a, y) and torch.equal(b.cpu(), s)
    a, b = x.cuda(), r.cuda()
    sd.sd_rms_norm(a, w, b, total=a, out=b)
    assert torch.equal(b, y) and torch.equal(a.cpu(), s)
    a, b = x.cuda(), r.cuda()
    sd.sd_rms_norm(a, w, b, out=b)
    assert torch.equal(b, y) and torch.equal(a.cpu(), x)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [40, 1032, 9000])
def test_strided_rows(d, dtype):
    """Rows of wider tensors at odd offsets; what lies between them stays."""
    wide = [N.rand(6, d + 24, dtype, i).cuda() for i in range(2)]
    x, r = wide[0][::2, 3:3 + d], wide[1][1::2, 5:5 + d]
    want = sd.sd_rms_norm(x.contiguous(), None, r.contiguous())
    total = torch.full((3, d + 9), 7.0, dtype=dtype, device="cuda")
    out = torch.full((3, d + 11), 5.0, dtype=dtype, device="cuda")
    sd.sd_rms_norm(x, None, r, total=total[:, 1:1 + d], out=out[:, 7:7 + d])
    assert torch.equal(out[:, 7:7 + d], want)
    assert torch.equal(total[:, 1:1 + d], (x.float() + r.float()).to(dtype))
    assert bool((out[:, :7] == 5).all()) and bool((out[:, 7 + d:] == 5).all())
    assert bool((total[:, :1] == 7).all()) and bool((total[:, 1 + d:] == 7).all())


@pytest.mark.parametrize("d", [64, 1024, 40000])
def test_offset_zeros_and_not_finite(d):
    x = N.rand(6, d, torch.float32, 4)
    w = N.rand(1, d, torch.float32, 5)[0]
    x[0] = 0
    x[1, 7], x[2, 9], x[3, 11] = float("nan"), float("inf"), -float("inf")
    x[4] *= 1e30                       # squares far past fp32
    x[5] *= 1e-30
    for eps, offset in ((1e-6, 1.0), (0.0, 0.5)):
        _, y = N.norm(x, w, None, eps, offset)
        got = sd.sd_rms_norm(x.cuda(), w.cuda(), eps=eps, weight_offset=offset)
        N.check_rounded(got, y, torch.float32)
        rc, rs = N.mx8_quantize(y.astype(np.float32).astype(np.float64))
        codes, scales = sd.sd_rms_norm_mxfp8(x.cuda(), w.cuda(), eps=eps, weight_offset=offset)
        assert np.array_equal(scales.cpu().numpy(), rs) and np.array_equal(codes.cpu().numpy(), rc)


@pytest.mark.parametrize("rows,d", [(2048, 500), (20011, 264), (2050, 1000), (2049, 1500), (2051, 4001), (2048, 7168)])
def test_many_rows_repeat(rows, d):
    """The launch shapes of many rows; the same bytes from call to call."""
    x = N.rand(rows, d, torch.bfloat16, 6)
    _, y = N.norm(x)
    got = sd.sd_rms_norm(x.cuda(), dtype=torch.float32)
    N.check_rounded(got, y, torch.float32)
    assert torch.equal(got, sd.sd_rms_norm(x.cuda(), dtype=torch.float32))


def test_rows_past_one_launch_axis():
    """More than 2^22 workgroups: they go along two axes of the grid."""
    n = (1 << 22) + 5
    x = torch.ones((n, 1), dtype=torch.bfloat16, device="cuda")
    x[-3:] = -2
    y = sd.sd_rms_norm(x, eps=0.0)
    assert bool((y[:-3] == 1).all()) and bool((y[-3:] == -1).all())


@pytest.mark.parametrize("T", [0.0, 1.0])
def test_verify_round_with_norm(T):
    """The norm in front of a verify round: the round on hidden rows that are made beforehand."""
    B, g, d, V = 3, 4, 256, 1500
    gen = torch.Generator().manual_seed(1)
    x = torch.randn((B, g + 1, d), generator=gen).to(torch.bfloat16).cuda()
    res = torch.randn((B, g + 1, d), generator=gen).cuda()
    w = (1 + 0.1 * torch.randn(d, generator=gen)).to(torch.bfloat16).cuda()
    head = torch.randn((V, d), generator=gen).to(torch.bfloat16).cuda()
    drafts = torch.randint(0, V, (B, g), generator=gen, dtype=torch.int32).cuda()
    conf = torch.rand((B, g), generator=gen).sort(dim=1, descending=True)[0].cuda()
    q = torch.randn((B, g, V), generator=gen).to(torch.bfloat16).cuda()
    ua, ur = torch.rand((B, g), generator=gen).cuda(), torch.rand((B, g + 1), generator=gen).cuda()
    for residual in (res, None):
        flat = None if residual is None else residual.view(-1, d)
        hidden = sd.sd_rms_norm(x.view(-1, d), w, flat, eps=1e-5, weight_offset=0.5).view(B, g + 1, d)
        a = sd.VerifyRound(B, g, d, V, T, True)
        b = sd.VerifyRound(B, g, d, V, T, True, norm=sd.RmsNorm(w, 1e-5, 0.5))
        want = a.run(hidden, head, drafts, conf, q, ua, ur)
        got = b.run(x, head, drafts, conf, q, ua, ur, residual=residual)
        assert torch.equal(b.hidden, hidden)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    with pytest.raises(ValueError):
        b.run(x[:2], head, drafts, conf, q, ua, ur)
    with pytest.raises(ValueError):
        b.run(x, head, drafts, conf, q, ua, ur, residual=res[:, :2])
    with pytest.raises(ValueError):
        a.run(hidden, head, drafts, conf, q, ua, ur, residual=res)
