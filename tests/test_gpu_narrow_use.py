"""The norm, MXFP8 and 4-bit calls in use: more than 2^31 elements a call, far strides, two calls at
once on two streams, everything between residual and token captured in one graph."""
import numpy as np
import pytest
import torch

import _narrow as N
import draft_block_verification_amd as sd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    yield
    torch.cuda.empty_cache()


def forms(V, d, seed):
    lm = N.rand(V, d, torch.bfloat16, seed).cuda()
    return sd.Mxfp8Weights.from_tensor(lm), sd.W4Weights.from_tensor(lm, 32), sd.W4Weights.from_tensor(lm, 128, True)


def logits(h, head, **kw):
    return (sd.sd_mxfp8_logits if isinstance(head, sd.Mxfp8Weights) else sd.sd_w4_logits)(h, head, **kw)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_logits_past_2_31_elements(out):
    """Every row of a long call is the row that a short call gives: rows are independent, and
    both calls take tiles of the same kernel."""
    M, V, d = 34000, 65700, 128
    h = N.rand(M, d, torch.bfloat16, 1).cuda()
    for head in forms(V, d, 2):
        z = logits(h, head, dtype=out)
        assert z.numel() > 2 ** 31
        for at in (0, 16000, M - 600):
            assert torch.equal(z[at:at + 600], logits(h[at:at + 600], head, dtype=out))
        del z


@pytest.mark.parametrize("M", [3, 40])
def test_far_strides(M):
    """Hidden rows and logit rows 2^26 elements apart and more: byte offsets far past 32 bits."""
    V, d, step = 999, 256, (1 << 26) + 24
    flat = torch.empty((M - 1) * step + d, dtype=torch.bfloat16, device="cuda")
    far = flat.as_strided((M, d), (step, 1))
    h = N.rand(M, d, torch.bfloat16, 3).cuda()
    far.copy_(h)
    zf = torch.empty((M - 1) * step + V, dtype=torch.bfloat16, device="cuda")
    z = zf.as_strided((M, V), (step, 1))
    for head in forms(V, d, 4):
        logits(far, head, logits=z)
        assert torch.equal(z, logits(h, head, dtype=torch.bfloat16))
    assert torch.equal(sd.sd_rms_norm(far, residual=far), sd.sd_rms_norm(h, residual=h))
    assert torch.equal(sd.sd_mxfp8_quantize(far)[0], sd.sd_mxfp8_quantize(h)[0])
    assert torch.equal(sd.sd_w4_quantize(far, 64)[0], sd.sd_w4_quantize(h, 64)[0])
    out = sd.sd_mxfp8_dequantize(*sd.sd_mxfp8_quantize(h), d, torch.bfloat16)
    sd.sd_mxfp8_dequantize(*sd.sd_mxfp8_quantize(h), d, out=far)
    assert torch.equal(far, out)


def test_large_quantisations():
    """2.2e9 values a call: the last rows are those of a call of their own."""
    rows, d = 134300, 16384
    x = torch.empty((rows, d), dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    c, s = sd.sd_mxfp8_quantize(x)
    tail = x[-3:].clone()
    a, b = sd.sd_mxfp8_quantize(tail)
    assert torch.equal(c[-3:], a) and torch.equal(s[-3:], b)
    back = sd.sd_mxfp8_dequantize(c, s, d, torch.bfloat16)
    assert torch.equal(back[-3:], sd.sd_mxfp8_dequantize(a, b, d, torch.bfloat16))
    del c, s, back
    got, want = sd.sd_w4_quantize(x, 32), sd.sd_w4_quantize(tail, 32)
    assert all(torch.equal(p[-3:], q) for p, q in zip(got, want))
    assert torch.equal(sd.sd_w4_dequantize(*got, d, torch.bfloat16)[-3:], sd.sd_w4_dequantize(*want, d, torch.bfloat16))
    del got
    y = sd.sd_rms_norm(x, residual=x, total=x)
    assert torch.equal(x[-3:], tail * 2) and torch.equal(y[-3:], sd.sd_rms_norm(tail, residual=tail))


def test_two_streams_at_once():
    """Calls on two streams that overlap, each with a workspace of its own."""
    M, V, d = 80, 30000, 1024
    hs = [N.rand(M, d, torch.bfloat16, 5 + i).cuda() for i in range(2)]
    for head in forms(V, d, 7):
        want = [logits(h, head) for h in hs]
        outs = [[torch.empty_like(w) for _ in range(6)] for w in want]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        for j in range(6):
            for i, st in enumerate(streams):
                logits(hs[i], head, logits=outs[i][j], stream=st)
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(o, want[i]) for o in outs[i])


@pytest.mark.parametrize("M", [1, 40])
def test_drafter_step_in_one_graph(M):
    """Residual, norm, logits and draw captured without buffers of the caller's, replayed with new
    inputs, eager work and synchronisations between the replays."""
    V, d = 3000, 384
    heads = forms(V, d, 11)
    x, res = (N.rand(M, d, torch.bfloat16, 12 + i).cuda() for i in range(2))
    w = N.rand(1, d, torch.bfloat16, 14)[0].cuda()
    u = torch.rand(M, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    params = sd.SamplingParams([0.8] * M, [20] * M, [0.9] * M, None)

    def step():
        out = []
        for head in heads:
            if isinstance(head, sd.Mxfp8Weights):
                z = sd.sd_mxfp8_logits(sd.sd_rms_norm_mxfp8(x, w, res), head, dtype=torch.bfloat16)
            else:
                z = sd.sd_w4_logits(sd.sd_rms_norm(x, w, res), head)
            out += [z, sd.sd_sample(z, u, params)[0]]
        return out

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        x.copy_(N.rand(M, d, torch.bfloat16, 20 + i).cuda())
        u.uniform_()
        graph.replay()
        got = [t.clone() for t in held]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_verify_round_with_norm_in_a_graph():
    """VerifyRound(norm=...) replayed from a graph, residual in fp32."""
    B, g, d, V = 2, 3, 128, 700
    gen = torch.Generator().manual_seed(3)
    x = torch.randn((B, g + 1, d), generator=gen).to(torch.bfloat16).cuda()
    res = torch.randn((B, g + 1, d), generator=gen).cuda()
    w = (1 + 0.1 * torch.randn(d, generator=gen)).cuda()
    head = torch.randn((V, d), generator=gen).to(torch.bfloat16).cuda()
    drafts = torch.randint(0, V, (B, g), generator=gen, dtype=torch.int32).cuda()
    vr = sd.VerifyRound(B, g, d, V, 0.0, False, norm=sd.RmsNorm(w))
    plain = sd.VerifyRound(B, g, d, V, 0.0, False)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        vr.run(x, head, drafts, residual=res)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vr.run(x, head, drafts, residual=res)
    for i in range(3):
        x.copy_(torch.randn((B, g + 1, d), generator=gen).to(torch.bfloat16))
        hidden = sd.sd_rms_norm(x.view(-1, d), w, res.view(-1, d)).view(B, g + 1, d)
        # the drafts of the first request are the target's own tokens: all are kept
        z = (hidden[0].float() @ head.float().t()).argmax(1)
        drafts[0].copy_(z[:g].int())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(vr.hidden, hidden)
        want = plain.run(hidden, head, drafts)
        assert torch.equal(vr.accept_len, want[0]) and torch.equal(vr.next_token, want[1])
        assert int(vr.accept_len[0]) == g


def test_refusals_of_device_tensors():
    """Scalars for matrices, rows in more or fewer parts than two, inputs that are no tensors or have
    another shape."""
    scalar = torch.zeros((), dtype=torch.uint8, device="cuda")
    scale = torch.zeros((1, 1), dtype=torch.bfloat16, device="cuda")
    head = sd.Mxfp8Weights.from_tensor(torch.ones(8, 128, device="cuda"))
    codes, scales = sd.sd_mxfp8_quantize(torch.ones(2, 128, device="cuda"))
    for f in (lambda: sd.Mxfp8Weights(scalar, scalar, 128), lambda: sd.sd_mxfp8_dequantize(scalar, scalar, 128),
              lambda: sd.W4Weights(scalar, scale, None, 64), lambda: sd.sd_w4_dequantize(scalar, scale, None, 64),
              lambda: sd.sd_mxfp8_logits((scalar, scalar), head), lambda: sd.sd_mxfp8_logits((codes,), head),
              lambda: sd.sd_mxfp8_logits((codes, scales, scales), head),
              lambda: sd.sd_mxfp8_logits((codes, scales[:1]), head)):
        with pytest.raises(ValueError):
            f()
    vr = sd.VerifyRound(1, 1, 128, 8, 0.0, False, norm=sd.RmsNorm())
    x = torch.ones((1, 2, 128), dtype=torch.bfloat16, device="cuda")
    lm, drafts = torch.ones((8, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    for hidden, residual in ((None, None), ([1.0], None), (x, [1.0])):
        with pytest.raises(TypeError):
            vr.run(hidden, lm, drafts, residual=residual)
    for hidden, residual in ((x[:, :1], None), (x, x.view(1, 1, 256))):
        with pytest.raises(ValueError):
            vr.run(hidden, lm, drafts, residual=residual)
