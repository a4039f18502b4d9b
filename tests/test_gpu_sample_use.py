"""Filtered sampling, filtered acceptance and MXFP4 logits in the ways a server calls them: captured
without buffers of their own, on a given stream, with one workspace for everything, and through
VerifyRound with truncated blocks and other LM-head forms. Whole numbers are compared with the
64-bit statement or with an eager call, and must be equal."""
import ctypes

import numpy as np
import pytest
import torch

import draft_block_verification_amd as sd
import _filtered as F
from test_gpu_sample import f32, head_logits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    yield


def block(B, g, V, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    z = 1.5 * torch.randn((B * (g + 1), V), device="cuda", generator=gen)
    zq = (z.view(B, g + 1, V)[:, :g] + 0.3 * torch.randn((B, g, V), device="cuda", generator=gen)).bfloat16().contiguous()
    x = z.view(B, g + 1, V)[:, :g].argmax(2).int()
    x[:, g // 2:] = torch.randint(0, V, (B, g - g // 2), device="cuda", generator=gen, dtype=torch.int32)
    ua = 0.1 * torch.rand((B, g), device="cuda", generator=gen)
    return [z, zq, x, ua, torch.rand((B, g + 1), device="cuda", generator=gen)]


def operators(R, V, d=256):
    """name -> (call(inputs, **kw) giving a list of tensors, inputs of seed)."""
    params = sd.SamplingParams(temperature=0.9, top_k=40, top_p=0.9, n=R)
    nucleus = sd.SamplingParams(top_p=0.8, n=R)
    head = sd.Mxfp4Weights.from_tensor(torch.randn((V, d), device="cuda", generator=torch.Generator("cuda").manual_seed(0)).bfloat16())
    gen = lambda s: torch.Generator("cuda").manual_seed(s)
    rows = lambda s: [3 * torch.randn((R, V), device="cuda", generator=gen(s)), torch.rand(R, device="cuda", generator=gen(s + 50))]
    accept = lambda p: lambda a, **k: list(sd.sd_accept_filtered(a[0], a[1], a[2], None, None, a[3], a[4], p, **k))
    return {
        "sample": (lambda a, **k: list(sd.sd_sample(*a, params, **k)), rows),
        "sample top-p": (lambda a, **k: list(sd.sd_sample(*a, nucleus, **k)), rows),
        "accept": (accept(params), lambda s: block(R, 4, V, s)),
        "accept top-p": (accept(nucleus), lambda s: block(R, 4, V, s)),
        "logits": (lambda a, **k: [sd.sd_mxfp4_logits(a[0], head, **k)],
                   lambda s: [torch.randn((3 * R, d), device="cuda", generator=gen(s)).bfloat16()]),
    }


@pytest.mark.parametrize("R,V", [(3, 2003), (2, 40009), (25, 20700)])
def test_captured_without_buffers(R, V):
    """Results and workspaces made inside the capture; replays between eager calls."""
    for name, (call, make) in operators(R, V).items():
        inputs = [make(s) for s in (1, 2, 3)]
        eager = [[t.clone() for t in call(a)] for a in inputs]
        live = [t.clone() for t in inputs[0]]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call(live)
        for i in (1, 2, 0, 2):
            for a, b in zip(live, inputs[i]):
                a.copy_(b)
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(out, eager[i])), name
            assert all(torch.equal(a, b) for a, b in zip(call(inputs[i]), eager[i])), name
            torch.cuda.synchronize()


@pytest.mark.parametrize("R,V", [(3, 2003), (2, 40009)])
def test_one_workspace_for_everything(R, V):
    """Calls in turn on one workspace, eagerly and from two graphs that share it: a call leaves
    nothing there that the next one minds."""
    ops = operators(R, V)
    nbytes = max(sd.sample_workspace_bytes(R, V), sd.accept_filtered_workspace_bytes(R, 4, V),
                 sd.mxfp4_logits_workspace_bytes(3 * R, 256))
    ws = sd.new_workspace(nbytes, "cuda")
    inputs = {n: make(7) for n, (_, make) in ops.items()}
    want = {n: [t.clone() for t in call(inputs[n])] for n, (call, _) in ops.items()}
    order = list(ops) * 2 + list(ops)[::-1]
    for n in order:
        assert all(torch.equal(a, b) for a, b in zip(ops[n][0](inputs[n], workspace=ws), want[n])), n
    torch.cuda.synchronize()
    graphs = {}
    for n in ("sample top-p", "accept"):
        graphs[n] = torch.cuda.CUDAGraph(), []
        with torch.cuda.graph(graphs[n][0]):
            graphs[n][1].extend(ops[n][0](inputs[n], workspace=ws))
    for n in ("accept", "sample top-p", "sample top-p", "accept"):
        for t in graphs[n][1]:
            t.zero_()
        graphs[n][0].replay()
        assert all(torch.equal(a, b) for a, b in zip(graphs[n][1], want[n])), n
        ops["logits"][0](inputs["logits"], workspace=ws)
        torch.cuda.synchronize()
    assert sd.device_flags(ws) == 0


@pytest.mark.parametrize("handle", [False, True])
def test_sampling_on_a_given_stream(handle):
    """Behind work that is still on the stream, with memory of that stream."""
    for name, (call, make) in operators(3, 3001).items():
        a = make(5)
        want = [t.clone() for t in call(a)]
        torch.cuda.synchronize()
        st = torch.cuda.Stream()
        big = torch.randn(4096, 4096, device="cuda")
        st.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            with torch.cuda.stream(st):
                late = [torch.zeros_like(t) for t in a]
                for _ in range(4):
                    big @ big
                for t, s in zip(late, a):
                    t.copy_(s)
            got = call(late, stream=st.cuda_stream if handle else st)
            junk = [torch.full((1 << 20,), 9, dtype=torch.int32, device="cuda") for _ in range(4)]
            st.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(got, want)), name
            del junk


@pytest.mark.parametrize("head", ["rows", "blocked", "w12"])
@pytest.mark.parametrize("T", [0.0, 1.0])
@pytest.mark.parametrize("cut", ["whole", "threshold", "scheduler"])
def test_round_with_truncation(cut, T, head):
    """VerifyRound(sampling=...) after either truncation, at any verify temperature and LM-head
    form: accepted lengths and tokens are the statement's on the logits that the round left."""
    B, g, V, d = 5, 6, 1501, 256
    r = np.random.default_rng(17)
    W = torch.from_numpy(r.standard_normal((V, d)).astype(np.float32) / 8).to(torch.bfloat16)
    hid = torch.from_numpy(r.standard_normal((B, g + 1, d)).astype(np.float32)).to(torch.bfloat16).cuda()
    sets = [dict(temperature=0.8, top_k=50, top_p=0.95), dict(top_p=0.8), dict(temperature=1.2, min_p=0.05),
            dict(temperature=0.0), dict()]
    settings = [f32(s) for s in sets]
    params = sd.SamplingParams(*[[s[i] for s in settings] for i in range(4)])
    lm = {"rows": lambda: W.cuda(), "blocked": lambda: sd.BlockedWeights(W.cuda()),
          "w12": lambda: sd.W12Weights.from_bf16(W.view(torch.int16).numpy().view(np.uint16))}[head]()
    conf = torch.from_numpy(r.random((B, g)).astype(np.float32)).cuda()
    extra = dict(scheduler=sd.SCHED_EARLY_STOP, sps=torch.linspace(2.0, 1.0, B * (g + 1) + 1).cuda()) if cut == "scheduler" else {}
    vr = sd.VerifyRound(B, g, d, V, T, cut != "whole", device="cuda", sampling=params, **extra)
    zq = torch.from_numpy(np.stack([head_logits(g, V, 40 + b) for b in range(B)])).to(torch.bfloat16)
    x = torch.from_numpy(r.integers(0, V, (B, g)).astype(np.int32))
    top = (hid.float() @ W.cuda().float().t()).argmax(2).int().cpu()
    x[:, :2] = top[:, :2]
    ua = torch.from_numpy(0.2 * r.random((B, g), dtype=np.float32))
    ur = torch.from_numpy(r.random((B, g + 1), dtype=np.float32))
    a, t = vr.run(hid, lm, x.cuda(), conf=conf, draft_logits=zq.cuda(), u_accept=ua.cuda(), u_resample=ur.cuda())
    lens = [g] * B if cut == "whole" else vr.verify_len.cpu().tolist()
    offs = np.arange(B + 1) * (g + 1) if cut == "whole" else vr.row_offsets.cpu().numpy()
    want = F.accept(vr.logits.double().cpu().numpy(), zq.double().numpy(), x.numpy(), lens, offs, ua.numpy(), ur.numpy(), settings)
    assert a.tolist() == want[0].tolist() and t.tolist() == want[1].tolist()
    assert vr.counters.tolist() == [sum(lens), int(want[0].sum())]
    assert sd.device_flags(vr.ws_accept) == 0


def test_a_workspace_between_kinds_is_prepared_anew():
    """The verify calls keep state behind a workspace's header that the other calls write over:
    sd_workspace_init makes it a verify workspace again."""
    lib = ctypes.CDLL(sd.LIB_PATH)
    B, g, V, d = 2, 3, 2003, 256
    r = np.random.default_rng(3)
    W = torch.from_numpy(r.standard_normal((V, d)).astype(np.float32)).to(torch.bfloat16).cuda()
    hid = torch.from_numpy(r.standard_normal((B, g + 1, d)).astype(np.float32)).to(torch.bfloat16).cuda()
    x = torch.from_numpy(r.integers(0, V, (B, g)).astype(np.int32)).cuda()
    x[:, 0] = (hid[:, 0].float() @ W.float().t()).argmax(1).int()
    want = [t.clone() for t in sd.sd_verify_greedy(hid, W, x)[1:]]
    ops = operators(B, V)
    nbytes = max(sd.verify_workspace_bytes(B, g, d, V), sd.accept_filtered_workspace_bytes(B, 4, V),
                 sd.sample_workspace_bytes(B, V), sd.mxfp4_logits_workspace_bytes(3 * B, d))
    ws = sd.new_workspace(nbytes, "cuda")
    for n, (call, make) in ops.items():
        a = make(1)
        call(a, workspace=ws)
        assert lib.sd_workspace_init(ctypes.c_void_p(ws.data_ptr()), ctypes.c_size_t(nbytes), None) == 0
        got = sd.sd_verify_greedy(hid, W, x, workspace=ws)[1:]
        assert all(torch.equal(p, q) for p, q in zip(got, want)), n
        assert sd.device_flags(ws) == 0
