"""MXFP8 logits of every size and output type are sums of exact products in fp32.

Tolerance of the sums: products of two MXFP8 values are exact in fp32, d of them added in fp32 in any
order are off by at most (d - 1) 2^-24 sum |terms|; an output in bf16 or fp16 adds its one rounding
(eps / 2 relative). Logits in 16 bits are the fp32 logits of the same call, rounded."""
import numpy as np
import pytest
import torch

import _narrow as N
import draft_block_verification_amd as sd

pytestmark = pytest.mark.gpu
HALVES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    yield


def given(h, coded):
    return sd.sd_mxfp8_quantize(h.cuda()) if coded else h.cuda()


# from the rows of one tile over those of several, of few ids and of more than a workgroup a unit
ROWS = [1, 16, 17, 32, 33, 64, 65, 128, 129, 200, 256, 300, 513]


@pytest.mark.parametrize("coded", [False, True])
@pytest.mark.parametrize("out", HALVES)
@pytest.mark.parametrize("M", ROWS)
def test_products_far_below_their_neighbours(M, out, coded):
    """Large products that cancel, one in each eight columns, and small ones beside them that make
    the whole sum: 224 and -224 in turn against 7 of 0.01171875 each."""
    d, V = 256, 515
    h, w = torch.full((M, d), 0.125), torch.full((V, d), 0.09375)
    h[:, ::8] = 224.0
    w[:, ::16], w[:, 8::16] = 1.0, -1.0
    head = sd.Mxfp8Weights.from_tensor(w.cuda())
    want = 224 * 0.01171875                              # 2.625, of 32 groups
    size = 32 * 224 + want
    got = sd.sd_mxfp8_logits(given(h, coded), head, dtype=out).double().cpu()
    tol = d * 2.0 ** -24 * size                          # 0.11; without the small products 2.625 is missing
    tol += (want + tol) * torch.finfo(out).eps / 2
    assert bool(((got - want).abs() <= tol).all()), (float(got.min()), float(got.max()))


def stream_rows(M, d, seed):
    """Hidden rows with a few columns far larger than the rest, as residual streams have them."""
    h = N.rand(M, d, torch.bfloat16, seed)
    g = torch.Generator().manual_seed(seed + 1)
    h[:, torch.randperm(d, generator=g)[:max(4, d // 100)]] *= 100
    return h


@pytest.mark.parametrize("coded", [False, True])
@pytest.mark.parametrize("M,V,d", [(16, 1001, 512), (17, 1000, 512), (40, 70001, 136), (64, 777, 2048), (100, 33000, 264),
                                   (128, 9000, 1152), (256, 1536, 4096), (300, 2049, 768), (520, 32001, 256)])
def test_16_bits_are_the_fp32_logits_rounded(M, V, d, coded):
    h, w = stream_rows(M, d, M), N.rand(V, d, torch.bfloat16, V) * 2.0 ** -6
    head = sd.Mxfp8Weights.from_tensor(w.cuda())
    rows = given(h, coded)
    full = sd.sd_mxfp8_logits(rows, head)
    for out in HALVES:
        assert torch.equal(sd.sd_mxfp8_logits(rows, head, dtype=out), full.to(out)), out
    at = torch.randperm(V, generator=torch.Generator().manual_seed(1))[:64]
    hv = torch.from_numpy(N.mx8_values(*N.mx8_quantize(h.double().numpy()), d))
    wv = torch.from_numpy(N.mx8_values(*N.mx8_quantize(w[at].double().numpy()), d))
    tol = d * 2.0 ** -24 * (hv.abs() @ wv.abs().t())
    assert bool(((full.cpu()[:, at].double() - hv @ wv.t()).abs() <= tol).all())


@pytest.mark.parametrize("M", [64, 128, 300])
def test_size_of_the_error(M):
    """On normal data, fp16 logits less their own rounding. A sum of d terms has at most d roundings,
    each uniform within 2^-24 of a partial sum no larger (rms) than the logits: together a standard
    deviation of at most sqrt(d / 3) 2^-24 of their rms, 1.1e-6 here. Six of them are allowed."""
    V, d = 900, 1024
    h, w = N.rand(M, d, torch.bfloat16, 5), N.rand(V, d, torch.bfloat16, 6)
    head = sd.Mxfp8Weights.from_tensor(w.cuda())
    got = sd.sd_mxfp8_logits(h.cuda(), head, dtype=torch.float16).cpu()
    hv = torch.from_numpy(N.mx8_values(*N.mx8_quantize(h.double().numpy()), d))
    wv = torch.from_numpy(N.mx8_values(*N.mx8_quantize(w.double().numpy()), d))
    want = hv @ wv.t()
    slack = 6 * (d / 3) ** 0.5 * 2.0 ** -24 * float(want.square().mean().sqrt())
    half = want.abs() * torch.finfo(torch.float16).eps / 2 + 2.0 ** -25
    assert bool(((got.double() - want).abs() <= half + slack).all())


@pytest.mark.parametrize("M", [16, 247])
@pytest.mark.parametrize("swap", [False, True])
def test_every_code_under_every_scale(M, swap):
    """Logits of one product each: every e4m3 code under scale bytes 3 .. 246, whose values are bf16
    numbers, subnormal ones among them, times 2^60 (below byte 127) or 2^-60, exact in fp32; as LM head
    and as hidden rows."""
    B = 247
    d = 32 * B
    kp = N.padded(d)
    codes, scales = np.zeros((256, kp), np.uint8), np.zeros((256, kp // 32), np.uint8)
    codes[:, :d:32] = np.arange(256)[:, None]
    codes[127] = codes[255] = 0                          # NaN codes would fill every logit of their id
    scales[:, :B] = np.arange(B)[None]
    value = N.mx8_values(codes, scales, d)[:, ::32]      # [code][byte]
    ones, by = np.zeros((B, kp), np.uint8), np.zeros((B, kp // 32), np.uint8)
    power = np.where(np.arange(B) < 127, 60, -60)
    ones[np.arange(B), 32 * np.arange(B)] = 0x38         # 1.0, in a block of its own for each byte
    by[np.arange(B), np.arange(B)] = 127 + power
    dev = lambda a: torch.from_numpy(a).cuda()
    head = sd.Mxfp8Weights(dev(ones), dev(by), d) if swap else sd.Mxfp8Weights(dev(codes), dev(scales), d)
    h, s = (codes, scales) if swap else (ones, by)
    got = torch.cat([sd.sd_mxfp8_logits((dev(h[i:i + M].copy()), dev(s[i:i + M].copy())), head) for i in range(0, len(h), M)])
    want = value * 2.0 ** power
    want = want if swap else want.T
    got = got.cpu().double().numpy()
    keep = np.arange(B) >= 3
    assert np.array_equal(got[:, keep], want[:, keep]) if swap else np.array_equal(got[keep], want[keep])


@pytest.mark.parametrize("M", [3, 100])
@pytest.mark.parametrize("dtype,tiny", [(torch.float16, 2.0 ** -24), (torch.bfloat16, 2.0 ** -130)])
def test_subnormal_hidden_rows_under_4_bits(M, dtype, tiny):
    """Hidden values under the type's smallest normal number count in full."""
    h = torch.zeros((M, 128), dtype=dtype)
    h[:, 0], h[:, 5] = tiny, 3 * tiny
    w = torch.zeros((64, 128))
    w[:, 0], w[:, 5], w[:, 9] = torch.arange(64) % 15 - 7.0, 7.0 - torch.arange(64) % 15, 7.0
    codes, scales, _ = sd.sd_w4_quantize(w.cuda(), 128, True)
    v = sd.sd_w4_dequantize(codes, scales, None, 128).cpu().double()
    got = sd.sd_w4_logits(h.cuda(), sd.W4Weights(codes, scales, None, 128)).cpu().double()
    assert torch.equal(got, h.double() @ v.t())
