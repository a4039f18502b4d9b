"""MXFP4 on the GPU against the 64-bit statement: codes and scales exactly, logits within the
fp32 accumulation's rounding.

Logit tolerance: a product of two MXFP4 values is exact in fp32, and the sum of d of them in
fp32, in any order, is off by at most (d - 1) 2^-24 sum |terms|; an output rounded once to
bf16 or fp16 adds half a step, 2^-9 or 2^-12 of the largest binade (eps / 2 relative)."""
import numpy as np
import pytest
import torch

import draft_block_verification_amd as sd
import _filtered as F

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    yield


def rand(rows, d, dtype, seed, spread=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, d), generator=g)
    if spread:      # blocks of very different size
        x = x * torch.exp2(torch.randint(-12, 12, (rows, d // 8), generator=g).float()).repeat_interleave(8, 1)
        if dtype == torch.float16:
            x = x.clamp(-60000, 60000)
    return x.to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,d", [(1, 8), (3, 32), (2, 40), (5, 96), (7, 136), (1, 256), (130, 2048), (33, 7168)])
def test_quantise_and_back(rows, d, dtype):
    x = rand(rows, d, dtype, rows * d)
    codes, scales = sd.sd_mxfp4_quantize(x.cuda())
    rc, rs = F.mx_quantize(x.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(codes.cpu().numpy(), rc)
    for out in TYPES:
        got = sd.sd_mxfp4_dequantize(codes, scales, d, out).cpu()
        want = torch.from_numpy(F.mx_values(rc, rs, d)).to(out)
        assert torch.equal(got, want), out


def test_borders_zeros_and_extremes():
    """Every tie between neighbouring magnitudes, zeros of both signs, the smallest and the
    largest scales, subnormal blocks."""
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    around = [np.nextafter(np.float32(t), np.float32(s)) for t in ties for s in (0, 10)]
    vals = np.array([4.0, 7.999, -6.5] + ties + [-t for t in ties] + around, dtype=np.float32)
    block = np.zeros(32, dtype=np.float32)
    block[:31] = vals[:31]
    rows = [block * np.float32(2.0 ** e) for e in (0, 1, -3, 60, -100, 124)]
    rows.append(np.zeros(32, dtype=np.float32))
    rows.append(np.full(32, -0.0, dtype=np.float32))
    rows.append(np.full(32, np.finfo(np.float32).max, dtype=np.float32))
    rows.append(np.full(32, np.finfo(np.float32).tiny, dtype=np.float32))
    rows.append(np.full(32, np.float32(1e-42), dtype=np.float32))
    x = np.stack(rows)
    codes, scales = sd.sd_mxfp4_quantize(torch.from_numpy(x).cuda())
    rc, rs = F.mx_quantize(x.astype(np.float64))
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(codes.cpu().numpy(), rc)
    got = sd.sd_mxfp4_dequantize(codes, scales, 32).cpu().numpy()
    assert np.array_equal(got, F.mx_values(rc, rs, 32).astype(np.float32))


def test_not_finite_blocks():
    x = rand(4, 128, torch.float32, 3)
    x[0, 5], x[1, 40], x[2, 127] = float("nan"), float("inf"), float("-inf")
    codes, scales = sd.sd_mxfp4_quantize(x.cuda())
    rc, rs = F.mx_quantize(x.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), rs) and (rs == 255).sum() == 3
    got = sd.sd_mxfp4_dequantize(codes, scales, 128).cpu().numpy()
    assert np.array_equal(np.isnan(got), np.repeat(rs == 255, 32, axis=1))


@pytest.mark.parametrize("dtype", TYPES)
def test_strided_rows(dtype):
    """Rows of a wider tensor at an odd offset, into rows of a wider one, neighbours untouched."""
    d = 136
    wide = rand(6, 160, dtype, 9).cuda()
    x = wide[::2, 3:3 + d]
    codes, scales = sd.sd_mxfp4_quantize(x)
    c2, s2 = sd.sd_mxfp4_quantize(x.contiguous())
    assert torch.equal(codes, c2) and torch.equal(scales, s2)
    out = torch.full((3, 200), 77.0, dtype=dtype, device="cuda")
    sd.sd_mxfp4_dequantize(codes, scales, d, out=out[:, 5:5 + d])
    assert torch.equal(out[:, 5:5 + d], sd.sd_mxfp4_dequantize(codes, scales, d, dtype))
    assert bool((out[:, :5] == 77).all()) and bool((out[:, 5 + d:] == 77).all())


def logits_case(M, V, d, dtype, out, seed, hidden=None):
    h = rand(M, d, dtype, seed, spread=False) if hidden is None else hidden
    w = rand(V, d, torch.bfloat16, seed + 1, spread=False)
    head = sd.Mxfp4Weights.from_tensor(w.cuda())
    got = sd.sd_mxfp4_logits(h.cuda(), head, dtype=out).cpu().double()
    hv = torch.from_numpy(F.mx_values(*F.mx_quantize(h.double().numpy()), d))
    wv = torch.from_numpy(F.mx_values(*F.mx_quantize(w.double().numpy()), d))
    want, size = hv @ wv.t(), hv.abs() @ wv.abs().t()
    tol = d * 2.0 ** -24 * size
    if out != torch.float32:
        tol = tol + (want.abs() + tol) * torch.finfo(out).eps / 2
    return got, want, tol


SHAPES = [(1, 1, 8), (1, 15, 32), (2, 17, 128), (3, 64, 136), (16, 100, 256), (17, 1000, 512),
          (5, 257, 2048), (33, 515, 640), (64, 1023, 384), (65, 300, 1152), (129, 777, 1024),
          (256, 1536, 512), (300, 2049, 768), (1, 5003, 4096)]


@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("M,V,d", SHAPES)
def test_logits(M, V, d, out):
    got, want, tol = logits_case(M, V, d, torch.bfloat16, out, 7 * M + V + d)
    assert bool(((got - want).abs() <= tol).all()), float(((got - want).abs() / tol).max())


@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("M,V,d", [(40, 70001, 136), (64, 65600, 256), (130, 32000, 264), (100, 65700, 128),
                                   (500, 32001, 256), (257, 40000, 384), (33, 300, 640), (1030, 140, 128)])
def test_logits_many_ids(M, V, d, out):
    """Sizes at which every tiling is taken, whole and cut at both edges."""
    got, want, tol = logits_case(M, V, d, torch.bfloat16, out, 3)
    assert bool(((got - want).abs() <= tol).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("M", [1, 20, 140])
def test_logits_hidden_types(M, dtype):
    got, want, tol = logits_case(M, 333, 256, dtype, torch.float32, 5)
    assert bool(((got - want).abs() <= tol).all())


@pytest.mark.parametrize("d", [32, 160, 992])
def test_unpadded_weights(d):
    """Codes and scales as checkpoints hold them, d no multiple of 128."""
    w = rand(77, d, torch.bfloat16, d, spread=False)
    rc, rs = F.mx_quantize(w.double().numpy())
    h = rand(3, d, torch.bfloat16, d + 1, spread=False).cuda()
    head = sd.Mxfp4Weights(torch.from_numpy(rc[:, :d // 2].copy()).cuda(),
                           torch.from_numpy(rs[:, :d // 32].copy()).cuda(), d)
    assert torch.equal(sd.sd_mxfp4_logits(h, head),
                       sd.sd_mxfp4_logits(h, sd.Mxfp4Weights.from_tensor(w.cuda())))


@pytest.mark.parametrize("M", [4, 40, 200])
def test_logits_not_finite_row(M):
    """A hidden row with a NaN or an infinity gives NaN in that row alone."""
    h = rand(M, 256, torch.bfloat16, 1, spread=False)
    h[1, 200], h[2, 3] = float("nan"), float("inf")
    got, want, tol = logits_case(M, 130, 256, torch.bfloat16, torch.float32, 1, hidden=h)
    assert bool(torch.isnan(got[1:3]).all())
    rest = [0] + list(range(3, M))
    assert bool(((got - want)[rest].abs() <= tol[rest]).all())


@pytest.mark.parametrize("M", [1, 6, 100])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_logits_into_strided_columns(M, out):
    """A drafter's use: position j of every request's block of logits, rows gamma V apart,
    at an odd vocabulary; the other positions stay."""
    g, V, d = 3, 203, 256
    h = rand(2 * M, d, torch.bfloat16, 4, spread=False).cuda()
    head = sd.Mxfp4Weights.from_tensor(rand(V, d, torch.bfloat16, 5, spread=False).cuda())
    plain = sd.sd_mxfp4_logits(h[::2].contiguous(), head, dtype=out)
    block = torch.full((M, g, V), 7.0, dtype=out, device="cuda")
    sd.sd_mxfp4_logits(h[::2], head, block[:, 1])
    assert torch.equal(block[:, 1], plain)
    assert bool((block[:, 0] == 7).all()) and bool((block[:, 2] == 7).all())


@pytest.mark.parametrize("M", [1, 48, 272])
def test_logits_repeat_and_graph(M):
    """The same bytes from call to call, and from a captured graph replayed with eager work
    and new inputs in between."""
    V, d = 1500, 512
    head = sd.Mxfp4Weights.from_tensor(rand(V, d, torch.bfloat16, 2, spread=False).cuda())
    hs = [rand(M, d, torch.bfloat16, 20 + i, spread=False).cuda() for i in range(3)]
    eager = [sd.sd_mxfp4_logits(h, head) for h in hs]
    h = hs[0].clone()
    out = torch.empty((M, V), device="cuda")
    ws = sd.new_workspace(sd.mxfp4_logits_workspace_bytes(M, d), "cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        sd.sd_mxfp4_logits(h, head, out, workspace=ws)
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sd.sd_mxfp4_logits(h, head, out, workspace=ws)
    for i in (1, 2, 0, 1):
        h.copy_(hs[i])
        out.zero_()
        graph.replay()
        assert torch.equal(out, eager[i])
        assert torch.equal(sd.sd_mxfp4_logits(hs[i], head), eager[i])
        torch.cuda.synchronize()


@pytest.mark.parametrize("handle", [False, True])
def test_given_stream(handle):
    """Everything a call makes for itself (padding, codes, workspace, results) is made on the
    stream it is given, behind work that is still on it."""
    d, V, M = 160, 3000, 70
    w = rand(V, d, torch.bfloat16, 1, spread=False).cuda()
    h = rand(M, d, torch.bfloat16, 2, spread=False).cuda()
    codes, scales = sd.sd_mxfp4_quantize(w)
    want = sd.sd_mxfp4_logits(h, sd.Mxfp4Weights(codes, scales, d))
    back = sd.sd_mxfp4_dequantize(codes, scales, d)
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
        c, e = sd.sd_mxfp4_quantize(late, stream=s)
        head = sd.Mxfp4Weights(c, e, d, stream=s)
        got = sd.sd_mxfp4_logits(h, head, stream=s)
        val = sd.sd_mxfp4_dequantize(c, e, d, stream=s)
        junk = [torch.full((V, d), 9.0, device="cuda") for _ in range(4)]
        st.synchronize()
        assert torch.equal(got, want) and torch.equal(val, back)
        del junk
