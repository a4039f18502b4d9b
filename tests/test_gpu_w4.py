"""4-bit integers with group scales on the GPU against the 64-bit statement: codes, scales, zeros
and values exactly, logits within the fp32 accumulation's rounding.

Logit tolerance: a group's sums of code products (exact in fp32) and of hidden values are each off
by at most group 2^-24 sum |terms|, their combination and the sum over the groups add a rounding
an operation: with the terms scale (code + zero) |hidden|, (d + 8) 2^-24 of their sum bounds all
of it. An output rounded once to bf16 or fp16 adds half a step (eps / 2 relative)."""
import numpy as np
import pytest
import torch

import _narrow as N
import draft_block_verification_amd as sd

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]
HALF = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    yield


def same_form(got, want):
    codes, scales, zeros = got
    assert np.array_equal(codes.cpu().numpy(), want[0])
    a, b = scales.cpu().float(), want[1].float()
    assert bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())
    assert (zeros is None) == (want[2] is None)
    if zeros is not None:
        assert np.array_equal(zeros.cpu().numpy(), want[2])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("symmetric", [False, True])
@pytest.mark.parametrize("rows,d,group", [(1, 32, 32), (3, 96, 32), (2, 64, 64), (5, 320, 64), (1, 128, 128), (7, 640, 128),
                                          (130, 2048, 32), (33, 7168, 128), (1030, 2112, 64)])
def test_quantise_and_back(rows, d, group, symmetric, dtype):
    x = N.rand(rows, d, dtype, rows * d + group, spread=True)
    for kind in HALF:
        got = sd.sd_w4_quantize(x.cuda(), group, symmetric, kind)
        want = N.w4_quantize(x.double().numpy(), group, symmetric, kind)
        same_form(got, want)
        c, s, _ = N.w4_parts(want[0], want[1], want[2])
        for out in TYPES:
            back = sd.sd_w4_dequantize(*got, d, out).cpu()
            ref = torch.from_numpy(c * s).float().to(out)
            assert bool(((back == ref) | (torch.isnan(back) & torch.isnan(ref))).all())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("symmetric", [False, True])
def test_ties_zeros_signs_and_ends(group, symmetric):
    """Quotients halfway between codes, groups of one sign, of zeros, of one value, of the largest
    and the smallest numbers, with a NaN or an infinity."""
    base = np.zeros((14, group), dtype=np.float32)
    ramp = np.arange(group, dtype=np.float32)
    base[0] = ramp % 16 - 7.5                         # ties of a scale of 1
    base[1] = (ramp % 29) / 2 - 7                     # halves: symmetric scale 1
    base[2], base[3] = ramp + 1, -(ramp + 1)
    base[5] = -0.0
    base[6], base[7] = 3.25, -3.25
    base[8] = np.where(ramp % 2 == 0, 3e38, -3e38)
    base[9], base[10] = 1e-37, 2.0 ** -149
    base[11, 3], base[12, group - 1], base[13, 0] = np.nan, np.inf, -np.inf
    with np.errstate(all="ignore"):
        for dtype in TYPES:
            x = torch.from_numpy(base).to(dtype)
            for kind in HALF:
                same_form(sd.sd_w4_quantize(x.cuda(), group, symmetric, kind),
                          N.w4_quantize(x.double().numpy(), group, symmetric, kind))


@pytest.mark.parametrize("dtype", TYPES)
def test_strided_rows(dtype):
    d = 192
    x = N.rand(6, 250, dtype, 9).cuda()[::2, 3:3 + d]
    got, want = sd.sd_w4_quantize(x, 64), sd.sd_w4_quantize(x.contiguous(), 64)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = torch.full((3, 300), 77.0, dtype=dtype, device="cuda")
    sd.sd_w4_dequantize(*got, d, out=out[:, 5:5 + d])
    assert torch.equal(out[:, 5:5 + d], sd.sd_w4_dequantize(*got, d, dtype))
    assert bool((out[:, :5] == 77).all()) and bool((out[:, 5 + d:] == 77).all())


def logits_case(M, V, d, group, symmetric, dtype, out, seed, kind=torch.bfloat16, hidden=None, spread=False):
    h = N.rand(M, d, dtype, seed) if hidden is None else hidden
    w = N.rand(V, d, torch.bfloat16, seed + 1, spread)
    codes, scales, zeros = N.w4_quantize(w.double().numpy(), group, symmetric, kind)
    head = sd.W4Weights(torch.from_numpy(codes).cuda(), scales.cuda(),
                        None if zeros is None else torch.from_numpy(zeros).cuda(), d)
    got = sd.sd_w4_logits(h.cuda(), head, dtype=out).cpu().double()
    c, s, both = N.w4_parts(codes, scales, zeros)
    hv = h.double()
    want = hv @ torch.from_numpy(c * s).t()
    tol = (d + 8) * 2.0 ** -24 * (hv.abs() @ torch.from_numpy(both * s).t())
    if out != torch.float32:
        tol = tol + (want.abs() + tol) * torch.finfo(out).eps / 2
    return got, want, tol


SHAPES = [(1, 1, 32, 32), (1, 15, 64, 64), (2, 17, 128, 128), (3, 64, 160, 32), (16, 100, 256, 64), (17, 1000, 512, 128),
          (5, 257, 2048, 32), (33, 515, 640, 64), (64, 1023, 384, 128), (65, 300, 1152, 32), (129, 777, 1024, 64),
          (256, 1536, 512, 128), (300, 2049, 768, 128), (1, 5003, 4096, 128), (1, 300, 4096, 32), (40, 333, 192, 64),
          (1, 16385, 160, 32), (16, 20003, 1216, 64), (32, 17001, 1152, 128), (17, 20001, 96, 32)]


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("symmetric", [False, True])
@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("M,V,d,group", SHAPES)
def test_logits(M, V, d, group, out, symmetric, dtype):
    kind = HALF[(M + V) % 2]
    got, want, tol = logits_case(M, V, d, group, symmetric, dtype, out, 7 * M + V + d, kind)
    assert bool(((got - want).abs() <= tol).all()), float(((got - want).abs() / tol).max())


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,V,d,group", [(40, 70001, 160, 32), (64, 65600, 256, 128), (130, 32000, 320, 64),
                                         (500, 32001, 256, 128), (257, 40000, 384, 128), (1030, 140, 128, 64),
                                         (17, 66000, 384, 32), (32, 70001, 128, 128), (20, 65537, 1152, 64), (300, 65600, 384, 64)])
def test_logits_many_ids(M, V, d, group, out):
    got, want, tol = logits_case(M, V, d, group, False, torch.bfloat16, out, 3)
    assert bool(((got - want).abs() <= tol).all())


@pytest.mark.parametrize("M", [2, 20, 140])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_logits_scales_apart(M, group):
    """Groups of very different scales and zeros: each is applied to its own."""
    got, want, tol = logits_case(M, 333, 640, group, False, torch.bfloat16, torch.float32, 8, spread=True)
    assert bool(((got - want).abs() <= tol).all())


@pytest.mark.parametrize("M", [4, 40, 200])
@pytest.mark.parametrize("symmetric", [False, True])
def test_logits_not_finite(M, symmetric):
    """A hidden row with a NaN or an infinity gives NaN in that row alone, a NaN scale in that id."""
    h = N.rand(M, 256, torch.bfloat16, 1)
    h[1, 200], h[2, 3] = float("nan"), float("inf")
    got, want, tol = logits_case(M, 130, 256, 64, symmetric, torch.bfloat16, torch.float32, 1, hidden=h)
    assert bool(torch.isnan(got[1:3]).all())
    rest = [0] + list(range(3, M))
    assert bool(((got - want)[rest].abs() <= tol[rest]).all())
    codes, scales, zeros = sd.sd_w4_quantize(N.rand(130, 256, torch.bfloat16, 2).cuda(), 64, symmetric)
    scales[100, 2] = float("nan")
    got = sd.sd_w4_logits(N.rand(M, 256, torch.bfloat16, 3).cuda(), sd.W4Weights(codes, scales, zeros, 256))
    assert bool(torch.isnan(got[:, 100]).all()) and int(torch.isnan(got).sum()) == M


@pytest.mark.parametrize("M", [1, 6, 40, 100])
@pytest.mark.parametrize("out", TYPES)
def test_strided_hidden_and_logits(M, out):
    """Hidden rows at an odd offset and stride, logits into every third row of an odd vocabulary;
    what lies between, and rows behind the last, stay."""
    g, V, d = 3, 203, 256
    wide = N.rand(2 * M, d + 13, torch.bfloat16, 4).cuda()
    h = wide[::2, 5:5 + d]
    head = sd.W4Weights.from_tensor(N.rand(V, d, torch.bfloat16, 5).cuda(), 64)
    plain = sd.sd_w4_logits(h.contiguous(), head, dtype=out)
    block = torch.full((M + 2, g, V), 7.0, dtype=out, device="cuda")
    sd.sd_w4_logits(h, head, block[:M, 1])
    assert torch.equal(block[:M, 1], plain)
    assert bool((block[:, 0] == 7).all()) and bool((block[:, 2] == 7).all()) and bool((block[M:] == 7).all())


@pytest.mark.parametrize("M,d", [(1, 512), (48, 512), (272, 512), (5, 544)])
def test_logits_repeat_and_graph(M, d):
    """The same bytes from call to call, and from two captured graphs that share a workspace,
    replayed in turn with eager work and new inputs in between."""
    V = 1500
    heads = [sd.W4Weights.from_tensor(N.rand(V, d, torch.bfloat16, 2).cuda(), 32, sym) for sym in (False, True)]
    hs = [N.rand(M, d, torch.bfloat16, 20 + i).cuda() for i in range(3)]
    eager = [[sd.sd_w4_logits(h, head) for h in hs] for head in heads]
    h = hs[0].clone()
    outs = [torch.empty((M, V), device="cuda") for _ in range(2)]
    ws = sd.new_workspace(sd.w4_logits_workspace_bytes(M, d, 32), "cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for k in (0, 1):
            sd.sd_w4_logits(h, heads[k], outs[k], workspace=ws)
    torch.cuda.current_stream().wait_stream(st)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for k in (0, 1):
        with torch.cuda.graph(graphs[k]):
            sd.sd_w4_logits(h, heads[k], outs[k], workspace=ws)
    for i in (1, 2, 0, 1):
        h.copy_(hs[i])
        for k in (0, 1):
            outs[k].zero_()
            graphs[k].replay()
            assert torch.equal(outs[k], eager[k][i])
        assert torch.equal(sd.sd_w4_logits(hs[i], heads[0]), eager[0][i])
        torch.cuda.synchronize()


def test_workspace_header_stays():
    """A workspace that other calls keep flags in: the products leave its header alone."""
    M, d, V = 5, 160, 300
    ws = sd.new_workspace(1 << 20, "cuda")
    ws[:256] = 0xa5
    h = N.rand(M, d, torch.bfloat16, 1).cuda()
    lm = N.rand(V, d, torch.bfloat16, 2).cuda()
    a = sd.sd_w4_logits(h, sd.W4Weights.from_tensor(lm, 32), workspace=ws)
    b = sd.sd_mxfp8_logits(h, sd.Mxfp8Weights.from_tensor(lm), workspace=ws)
    assert bool((ws[:256] == 0xa5).all())
    assert torch.equal(a, sd.sd_w4_logits(h, sd.W4Weights.from_tensor(lm, 32)))
    assert torch.equal(b, sd.sd_mxfp8_logits(h, sd.Mxfp8Weights.from_tensor(lm)))


@pytest.mark.parametrize("handle", [False, True])
def test_given_stream(handle):
    d, V, M = 160, 3000, 70
    w = N.rand(V, d, torch.bfloat16, 1).cuda()
    h = N.rand(M, d, torch.bfloat16, 2).cuda()
    form = sd.sd_w4_quantize(w, 32)
    want = sd.sd_w4_logits(h, sd.W4Weights(*form, d))
    back = sd.sd_w4_dequantize(*form, d)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    s = st.cuda_stream if handle else st
    big = torch.randn(4096, 4096, device="cuda")
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(st):
            late = torch.zeros_like(w)
            for _ in range(4):
                big @ big
            late.copy_(w)
        form = sd.sd_w4_quantize(late, 32, stream=s)
        got = sd.sd_w4_logits(h, sd.W4Weights(*form, d, stream=s), stream=s)
        val = sd.sd_w4_dequantize(*form, d, stream=s)
        junk = [torch.full((V, d), 9.0, device="cuda") for _ in range(4)]
        st.synchronize()
        assert torch.equal(got, want) and torch.equal(val, back)
        del junk
