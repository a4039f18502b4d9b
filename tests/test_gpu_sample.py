"""Filtered sampling and filtered acceptance on the GPU against the 64-bit statement.

Tokens, accepted lengths and sizes of kept sets are whole numbers and must be equal. The
library's weights are fp64 to about 1e-14 and its sums are rounded to units of 2^-46 of the
largest weight, so a decision can differ only where u times the total (or p times it, or
min_p) lies within V 2^-47 of a step of the running sum: V = 1e5 gives 1e-9. The seeded
cases are checked to lie outside that (`near_border`), so equality is asserted.
Log-probabilities: one rounding to fp32, 2^-24 relative, on an fp64 logarithm whose argument
is good to 1e-9: |error| <= 2^-24 |logprob| + 2e-9."""
import numpy as np
import pytest
import torch

import draft_block_verification_amd as sd
import _filtered as F

pytestmark = pytest.mark.gpu
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    yield


def head_logits(rows, V, seed, peaks=12):
    g = np.random.default_rng(seed)
    z = 1.5 * g.standard_normal((rows, V))
    for r in range(rows):
        ids = g.integers(0, V, min(peaks, V))
        z[r, ids] += 3 + 6 * g.random(len(ids)) ** 2
    return z.astype(np.float32)


def check_rows(z, u, settings, params, dtype=torch.float32, tokens=None):
    zt = torch.from_numpy(z).to(dtype)
    x, kept, lp = sd.sd_sample(zt.cuda(), torch.from_numpy(u).cuda(), params, tokens=tokens)
    x, kept, lp = x.cpu().numpy(), kept.cpu().numpy(), lp.cpu().numpy().astype(np.float64)
    zd = zt.double().numpy()
    for r in range(len(z)):
        w, n = F.filtered(zd[r], *settings[r])
        assert not F.near_border(w, float(u[r]), 1e-9), ("choose another seed", r)
        assert kept[r] == n, (r, kept[r], n, settings[r])
        want = F.draw(w, float(u[r]))
        assert x[r] == want, (r, x[r], want, settings[r])
        if want < 0:
            assert lp[r] == -np.inf
        else:
            ref = np.log(w[want] / w.sum())
            assert abs(lp[r] - ref) <= 2.0 ** -24 * abs(ref) + 2e-9, (r, lp[r], ref)
    return x


SETTINGS = {
    "plain": dict(),
    "temperature": dict(temperature=0.7),
    "hot": dict(temperature=3.0, top_p=0.98),
    "greedy": dict(temperature=0.0, top_k=50, top_p=0.9),
    "top_k": dict(temperature=0.9, top_k=40),
    "top_1": dict(top_k=1),
    "top_k_cold": dict(temperature=0.05, top_k=500),
    "top_p": dict(top_p=0.9),
    "top_p_long": dict(top_p=0.999),
    "top_p_none": dict(top_p=0.0),
    "min_p": dict(min_p=0.05),
    "min_p_one": dict(min_p=1.0),
    "usual": dict(temperature=0.8, top_k=50, top_p=0.95),
    "all": dict(temperature=1.2, top_k=3000, top_p=0.97, min_p=0.001),
    "wide_k": dict(temperature=1.5, top_k=20000, top_p=0.9),
}


def as_tuple(s):
    return (s.get("temperature", 1.0), s.get("top_k", 0), float(np.float32(s.get("top_p", 1.0))),
            float(np.float32(s.get("min_p", 0.0))))


def f32(s):
    t = as_tuple(s)
    return (float(np.float32(t[0])),) + t[1:]


@pytest.mark.parametrize("name", list(SETTINGS))
@pytest.mark.parametrize("V", [1, 2, 5, 63, 64, 1000, 4099, 50257, 151936])
def test_sample_settings(name, V):
    rows = 3 if V > 10000 else 9
    z = head_logits(rows, V, V + len(name))
    u = np.random.default_rng(V).random(rows, dtype=np.float32)
    s = SETTINGS[name]
    check_rows(z, u, [f32(s)] * rows, sd.SamplingParams(**s))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("V", [7, 1001, 32768, 129281])
def test_sample_types_and_mixed_settings(V, dtype):
    """Each request its own settings; 16-bit logits tie often."""
    rows = 12
    g = np.random.default_rng(V)
    z = head_logits(rows, V, V)
    t = g.choice([0.0, 0.6, 1.0, 1.3], rows).astype(np.float32)
    k = g.choice([0, 1, 20, 700, 10 ** 6], rows).astype(np.int32)
    p = g.choice([1.0, 0.5, 0.9, 0.99], rows).astype(np.float32)
    m = g.choice([0.0, 0.0, 0.02, 0.3], rows).astype(np.float32)
    params = sd.SamplingParams(*[torch.from_numpy(a).cuda() for a in (t, k, p, m)])
    settings = [(float(t[r]), int(k[r]), float(p[r]), float(m[r])) for r in range(rows)]
    check_rows(z, g.random(rows, dtype=np.float32), settings, params, TYPES[dtype])


@pytest.mark.parametrize("name", ["plain", "top_k", "top_p", "min_p", "usual", "all"])
def test_sample_hard_rows(name):
    """Masked rows: nothing left, one id left, NaN among them, the type's lowest value, +inf,
    rows of one value, two values, both zeros, and a huge spread."""
    V = 6001
    g = np.random.default_rng(5)
    base = head_logits(14, V, 11)
    z = base.copy()
    z[0] = -np.inf
    z[1] = np.nan
    z[2] = -np.inf
    z[2, 4321] = -3.0
    z[3, g.random(V) < 0.99] = -np.inf
    z[4, g.random(V) < 0.99] = np.finfo(np.float32).min
    z[5] = np.finfo(np.float32).min
    z[6, [17, 5000]] = np.inf
    z[7] = 0.25
    z[8] = np.where(np.arange(V) % 3 == 0, 1.0, 0.0)
    z[9] = np.where(np.arange(V) % 2 == 0, 0.0, -0.0)
    z[10] = base[10] * 1e30
    z[11, ::2] = np.nan
    z[12] = np.where(np.arange(V) < 5000, 2.0, 2.0 + 1e-6 * np.arange(V)).astype(np.float32)
    z[13] = np.linspace(-100, 100, V).astype(np.float32)
    u = g.random(14, dtype=np.float32)
    s = SETTINGS[name]
    ws = sd.new_workspace(sd.sample_workspace_bytes(14, V), "cuda")
    x = check_rows(z, u, [f32(s)] * 14, sd.SamplingParams(**s))
    assert x[0] == x[1] == -1 and x[2] == 4321 and x[6] in (17, 5000)
    sd.sd_sample(torch.from_numpy(z).cuda(), torch.from_numpy(u).cuda(), sd.SamplingParams(**s),
                 workspace=ws)
    assert sd.device_flags(ws) == sd.FLAG_EMPTY_ROW


@pytest.mark.parametrize("V", [20000, 151936])
def test_sample_many_ties(V):
    """More equal logits at the cut than are ranked at once: the lowest ids stay."""
    g = np.random.default_rng(V)
    z = np.zeros((4, V), dtype=np.float32)
    z[1, g.random(V) < 0.5] = 1.0
    z[2, g.random(V) < 0.3] = -1.0
    z[2, :100] = 2.0
    z[3] = np.round(g.standard_normal(V) * 2) / 2
    u = g.random(4, dtype=np.float32)
    for s in (dict(top_k=9000), dict(top_p=0.6), dict(top_k=17000, top_p=0.7), dict(top_k=V - 1)):
        check_rows(z, u, [f32(s)] * 4, sd.SamplingParams(**s))


def test_sample_uniform_ends():
    """u = 0 takes the first kept id, the largest u the last; values outside count as those."""
    z = np.tile(head_logits(1, 3000, 1), (6, 1))
    u = np.array([0.0, np.nextafter(np.float32(1), np.float32(0)), 1.0, -5.0, 7.0, np.nan], dtype=np.float32)
    x, _, _ = sd.sd_sample(torch.from_numpy(z).cuda(), torch.from_numpy(u).cuda(), sd.SamplingParams(top_k=10))
    ids = np.sort(np.argsort(-z[0], kind="stable")[:10])
    assert x.cpu().tolist() == [ids[0], ids[-1], ids[-1], ids[0], ids[-1], ids[0]]


def test_sample_bad_settings_raise_a_flag():
    z = head_logits(5, 500, 2)
    nan = float("nan")
    t = torch.tensor([nan, -1.0, float("inf"), 1.0, 1.0], device="cuda")
    p = torch.tensor([1.0, 1.0, 1.0, nan, 1.0], device="cuda")
    m = torch.tensor([0.0, 0.0, 0.0, 0.0, nan], device="cuda")
    ws = sd.new_workspace(sd.sample_workspace_bytes(5, 500), "cuda")
    u = torch.full((5,), 0.5, device="cuda")
    x, kept, _ = sd.sd_sample(torch.from_numpy(z).cuda(), u, sd.SamplingParams(t, None, p, m), workspace=ws)
    assert sd.device_flags(ws) == sd.FLAG_SAMPLING
    assert kept.cpu().tolist() == [1, 1, 1, 500, 500]
    assert x.cpu().tolist()[:3] == z[:3].argmax(1).tolist()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("V", [129, 5003])
def test_sample_strided(V, dtype):
    """Logits of one position of every block, tokens into a column, settings shared by rows."""
    B, g = 4, 3
    z = torch.from_numpy(head_logits(B * g, V, 8)).to(TYPES[dtype]).view(B, g, V).cuda()
    u = torch.rand(B, generator=torch.Generator().manual_seed(1)).cuda()
    params = sd.SamplingParams(temperature=[0.9, 1.1], top_k=[30, 0], top_p=[0.9, 0.8])
    block = torch.full((B, g), -7, dtype=torch.int32, device="cuda")
    for j in range(g):
        sd.sd_sample(z[:, j], u, params, tokens=block[:, j])
        x, _, _ = sd.sd_sample(z[:, j].contiguous(), u, params)
        assert torch.equal(block[:, j], x)
        assert bool((block[:, j + 1:] == -7).all())


def accept_case(B, g, V, seed, noise=0.4, lens=None):
    r = np.random.default_rng(seed)
    base = head_logits(B * g, V, seed)
    zq = torch.from_numpy(base + noise * r.standard_normal(base.shape).astype(np.float32)).to(torch.bfloat16).view(B, g, V)
    lens = [g] * B if lens is None else lens
    offs = np.concatenate([[0], np.cumsum(np.array(lens) + 1)]).astype(np.int32)
    z = np.full((B * (g + 1), V), 99.0, dtype=np.float32)
    for b in range(B):
        for j in range(lens[b]):
            z[offs[b] + j] = base[b * g + j] + noise * r.standard_normal(V).astype(np.float32)
        z[offs[b] + lens[b]] = head_logits(1, V, seed + 100 + b)[0]
    ua = r.random((B, g), dtype=np.float32)
    ur = r.random((B, g + 1), dtype=np.float32)
    return z, zq, np.array(lens, dtype=np.int32), offs, ua, ur


def draft_by_sampling(zq, settings, seed):
    r = np.random.default_rng(seed)
    B, g, _ = zq.shape
    return np.array([[F.draw(F.filtered(zq[b, j], *settings[b])[0], r.random()) for j in range(g)]
                     for b in range(B)], dtype=np.int32)


MIXES = [dict(), dict(temperature=0.8, top_k=50, top_p=0.95), dict(top_p=0.9), dict(top_k=3),
         dict(temperature=0.0), dict(min_p=0.05, temperature=1.3)]


@pytest.mark.parametrize("mix", range(len(MIXES)))
@pytest.mark.parametrize("B,g,V", [(1, 1, 50), (2, 4, 1000), (3, 16, 5003), (2, 64, 333)])
def test_accept_filtered(B, g, V, mix):
    s = f32(MIXES[mix])
    lens = [min(g, 3 * b + 1) for b in range(B)] if B > 1 else None
    z, zq, lens, offs, ua, ur = accept_case(B, g, V, 10 * mix + V, lens=lens)
    zqd = zq.double().numpy()
    x = draft_by_sampling(zqd, [s] * B, mix)
    want = F.accept(z.astype(np.float64), zqd, x, lens, offs, ua, ur, [s] * B)
    params = sd.SamplingParams(**MIXES[mix], n=B)
    counters = torch.zeros(2, dtype=torch.int64, device="cuda")
    ws = sd.new_workspace(sd.accept_filtered_workspace_bytes(B, g, V), "cuda")
    c = lambda a: torch.from_numpy(a).cuda()
    a, t = sd.sd_accept_filtered(c(z), zq.cuda(), c(x), c(lens), c(offs), c(ua), c(ur), params,
                                 counters=counters, workspace=ws)
    assert np.array_equal(a.cpu().numpy(), want[0])
    assert np.array_equal(t.cpu().numpy(), want[1])
    assert counters.cpu().tolist() == [int(lens.sum()), int(want[0].sum())]
    assert sd.device_flags(ws) == 0


def test_accept_filtered_own_settings_and_hard_rows():
    """Requests with settings of their own; a token outside the target's kept set, a token out
    of range, a masked target row, equal target and drafter rows (never rejected)."""
    B, g, V = 6, 4, 2000
    sets = [dict(top_k=5), dict(top_p=0.8), dict(temperature=0.0), dict(), dict(min_p=0.1), dict(top_k=20, top_p=0.9)]
    settings = [f32(s) for s in sets]
    z, zq, lens, offs, ua, ur = accept_case(B, g, V, 77)
    x = draft_by_sampling(zq.double().numpy(), settings, 3)
    x[0, 1] = int(np.argmin(z[offs[0] + 1]))        # not kept by the target
    x[1, 0] = V + 5                                 # out of range
    x[3, 2] = -1
    z[offs[4] + 1] = -np.inf                        # masked out
    zq[5] = torch.from_numpy(z[offs[5]:offs[5] + g]).to(torch.bfloat16)
    z[offs[5]:offs[5] + g] = zq[5].float().numpy()
    x[5] = draft_by_sampling(zq[5:6].double().numpy(), settings[5:6], 4)[0]
    zqd = zq.double().numpy()
    want = F.accept(z.astype(np.float64), zqd, x, lens, offs, ua, ur, settings)
    assert want[0][5] == g
    arr = lambda i, dt: torch.tensor([s[i] for s in settings], dtype=dt, device="cuda")
    params = sd.SamplingParams(arr(0, torch.float32), arr(1, torch.int32), arr(2, torch.float32), arr(3, torch.float32))
    c = lambda a: torch.from_numpy(a).cuda()
    a, t = sd.sd_accept_filtered(c(z), zq.cuda(), c(x), None, None, c(ua), c(ur), params)
    assert np.array_equal(a.cpu().numpy(), want[0])
    assert np.array_equal(t.cpu().numpy(), want[1])


def test_accept_filtered_flags():
    """Lengths out of range are clamped, rows past the capacity skipped, each with its flag;
    equal rows whose drafted token is rejected by a uniform of 1 draw from the target."""
    B, g, V = 3, 2, 300
    z, zq, lens, offs, ua, ur = accept_case(B, g, V, 5)
    x = draft_by_sampling(zq.double().numpy(), [f32({})] * B, 1)
    c = lambda a: torch.from_numpy(a).cuda()
    ws = sd.new_workspace(sd.accept_filtered_workspace_bytes(B, g, V), "cuda")
    params = sd.SamplingParams(n=B)
    sd.sd_accept_filtered(c(z), zq.cuda(), c(x), c(np.array([g, g + 9, g], np.int32)), c(offs),
                          c(ua), c(ur), params, workspace=ws)
    assert sd.device_flags(ws) == sd.FLAG_VERIFY_LEN
    bad = offs.copy()
    bad[2] = B * (g + 1) - 1
    a, t = sd.sd_accept_filtered(c(z), zq.cuda(), c(x), c(lens), c(bad), c(ua), c(ur), params, workspace=ws)
    assert sd.device_flags(ws) == sd.FLAG_ROW_OFFSETS
    assert a.cpu()[2] == 0 and t.cpu()[2] == -1
    z[:g] = zq[0].float().numpy()
    ua[0] = 1.0
    a, t = sd.sd_accept_filtered(c(z), zq.cuda(), c(x), None, None, c(ua), c(ur), params, workspace=ws)
    assert sd.device_flags(ws) == sd.FLAG_NO_RESIDUAL
    assert a.cpu()[0] == 0 and t.cpu()[0] == F.draw(F.filtered(z[0].astype(np.float64))[0], float(ur[0, 0]))


def test_unfiltered_agrees_with_accept_rejection():
    """With every filter off the rule is sd_accept_rejection's."""
    B, g, V, d = 4, 6, 3001, 128
    r = np.random.default_rng(3)
    W = torch.from_numpy(r.standard_normal((V, d)).astype(np.float32) / 6).to(torch.bfloat16).cuda()
    h = torch.from_numpy(r.standard_normal((B, g + 1, d)).astype(np.float32)).to(torch.bfloat16).cuda()
    x = torch.from_numpy(r.integers(0, V, (B, g)).astype(np.int32)).cuda()
    logits, stats = sd.sd_verify_logits(h, W, x, temperature=0.9, logits=True)
    zq = (logits.view(B, g + 1, V)[:, :g] + 0.1 * torch.randn((B, g, V), device="cuda", generator=torch.Generator("cuda").manual_seed(1))).to(torch.bfloat16).contiguous()
    ua = torch.from_numpy(r.random((B, g), dtype=np.float32)).cuda()
    ur = torch.from_numpy(r.random((B, g + 1), dtype=np.float32)).cuda()
    a0, t0 = sd.sd_accept_rejection(logits, stats, zq, x, None, None, ua, ur, 0.9)
    a1, t1 = sd.sd_accept_filtered(logits, zq, x, None, None, ua, ur, sd.SamplingParams(temperature=0.9, n=B))
    assert torch.equal(a0, a1) and torch.equal(t0, t1)


def test_drafter_step_verify_and_accept_together():
    """A whole round as a server runs it: the drafter's 4-bit LM head, filtered draws of each
    position into the block, verification at the bf16 LM head, filtered acceptance -- eagerly
    and replayed from a captured graph with new hidden states and uniforms."""
    B, g, V, d = 3, 4, 2003, 256
    r = np.random.default_rng(9)
    dev = "cuda"
    W = torch.from_numpy(r.standard_normal((V, d)).astype(np.float32) / 8).to(torch.bfloat16).to(dev)
    head = sd.Mxfp4Weights.from_tensor(W)
    sets = [dict(temperature=0.8, top_k=50, top_p=0.95), dict(top_p=0.8), dict(temperature=1.2, min_p=0.05)]
    settings = [f32(s) for s in sets]
    params = sd.SamplingParams([s[0] for s in settings], [s[1] for s in settings],
                               [s[2] for s in settings], [s[3] for s in settings])
    vr = sd.VerifyRound(B, g, d, V, 1.0, False, device=dev, sampling=params)
    hid = torch.empty((B, g + 1, d), dtype=torch.bfloat16, device=dev)
    u = torch.empty((3, B, g + 1), device=dev)
    zq = torch.empty((B, g, V), dtype=torch.bfloat16, device=dev)
    x = torch.empty((B, g), dtype=torch.int32, device=dev)
    wl = sd.new_workspace(sd.mxfp4_logits_workspace_bytes(B, d), dev)
    wsm = sd.new_workspace(sd.sample_workspace_bytes(B, V), dev)
    u_col = [torch.empty(B, device=dev) for _ in range(g)]
    ua = torch.empty((B, g), device=dev)

    def step():
        for j in range(g):
            sd.sd_mxfp4_logits(hid[:, j], head, zq[:, j], workspace=wl)
            sd.sd_sample(zq[:, j], u_col[j], params, tokens=x[:, j], workspace=wsm)
        vr.run(hid, W, x, draft_logits=zq, u_accept=ua, u_resample=u[2])

    def load(i):
        q = np.random.default_rng(i)
        hid.copy_(torch.from_numpy(q.standard_normal((B, g + 1, d)).astype(np.float32)))
        u.copy_(torch.from_numpy(q.random((3, B, g + 1), dtype=np.float32)))
        for j in range(g):
            u_col[j].copy_(u[0, :, j])
        ua.copy_(u[1, :, :g])

    def expect():
        z, q = vr.logits.double().cpu().numpy(), zq.double().cpu().numpy()
        offs = np.arange(B + 1) * (g + 1)
        for b in range(B):
            for j in range(g):
                assert int(x[b, j]) == F.draw(F.filtered(q[b, j], *settings[b])[0], float(u[0, b, j]))
        return F.accept(z, q, x.cpu().numpy(), [g] * B, offs, ua.cpu().numpy(), u[2].cpu().numpy(), settings)

    load(0)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda.synchronize()
    want = expect()
    assert np.array_equal(vr.accept_len.cpu().numpy(), want[0])
    assert np.array_equal(vr.next_token.cpu().numpy(), want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in (1, 2, 3):
        load(i)
        graph.replay()
        torch.cuda.synchronize()
        want = expect()
        assert np.array_equal(vr.accept_len.cpu().numpy(), want[0])
        assert np.array_equal(vr.next_token.cpu().numpy(), want[1])


def test_sample_many_rows():
    """More rows than are dealt to several workgroups, each with settings of its own."""
    rows, V = 520, 20611
    z = head_logits(rows, V, 1)
    z[7] = -np.inf
    z[8, 1:] = -np.inf
    z[9] = np.round(z[9])
    z[10] = 0.0
    u = np.random.default_rng(2).random(rows, dtype=np.float32)
    settings = [f32(list(SETTINGS.values())[r % len(SETTINGS)]) for r in range(rows)]
    col = lambda i, dt: torch.tensor([s[i] for s in settings], dtype=dt, device="cuda")
    params = sd.SamplingParams(col(0, torch.float32), col(1, torch.int32), col(2, torch.float32), col(3, torch.float32))
    check_rows(z, u, settings, params)


@pytest.mark.parametrize("name", ["top_k", "usual", "all", "top_p", "min_p"])
@pytest.mark.parametrize("V", [9001, 40009])
def test_sample_misleading_rows(V, name):
    """Rows of which a part says little about the rest: sorted, a likely block, likely (or
    unlikely) ids at evenly spread places alone, ties, a few ids in one place."""
    g = np.random.default_rng(V)
    rows = 9
    z = (1.5 * g.standard_normal((rows, V))).astype(np.float32)
    z[0] = np.linspace(0, -20, V)
    z[1] = np.linspace(-20, 0, V)
    z[2, :V // 256] += 9
    for r, up in ((3, 12.0), (4, -12.0)):
        head = (-(r * V)) % 4
        off = head - 4 if head else 0
        nv = (V - off + 3) // 4
        for c in range(128):
            a = off + 4 * (c * (nv - 8) // 127)
            z[r, max(a, 0):max(a + 32, 0)] += up
    z[5] = 1.25
    z[6] = -np.inf
    z[6, V // 2 + 40:V // 2 + 100] = g.standard_normal(60)
    z[7] = -np.inf
    z[7, V - 1] = -3.0
    z[8, ::2] = -np.inf
    u = g.random(rows, dtype=np.float32)
    s = SETTINGS[name]
    check_rows(z, u, [f32(s)] * rows, sd.SamplingParams(**s))


@pytest.mark.parametrize("mix", range(len(MIXES)))
@pytest.mark.parametrize("B,g,V", [(1, 5, 70003), (3, 2, 30011), (37, 7, 20603)])
def test_accept_filtered_long_rows(B, g, V, mix):
    s = f32(MIXES[mix])
    lens = [min(g, b % (g + 1)) for b in range(B)] if B > 1 else None
    z, zq, lens, offs, ua, ur = accept_case(B, g, V, 10 * mix + V, lens=lens)
    zqd = zq.double().numpy()
    x = draft_by_sampling(zqd, [s] * B, mix)
    want = F.accept(z.astype(np.float64), zqd, x, lens, offs, ua, ur, [s] * B)
    c = lambda a: torch.from_numpy(a).cuda()
    a, t = sd.sd_accept_filtered(c(z), zq.cuda(), c(x), c(lens), c(offs), c(ua), c(ur),
                                 sd.SamplingParams(**MIXES[mix], n=B))
    assert np.array_equal(a.cpu().numpy(), want[0])
    assert np.array_equal(t.cpu().numpy(), want[1])


@pytest.mark.parametrize("mix", [dict(top_p=0.9), dict(top_p=0.7, min_p=0.01), dict(top_k=30, top_p=0.95), dict(min_p=0.02)])
@pytest.mark.parametrize("B,g,V", [(3, 64, 700), (2, 6, 24001)])
def test_accept_filtered_tokens_at_the_border(B, g, V, mix):
    """Equal target and drafter rows: the last kept id is accepted whatever the uniform, up to
    a whole block of 64 and the bonus row; the next id in rank is rejected."""
    s = f32(mix)
    z, zq, lens, offs, ua, ur = accept_case(B, g, V, 4)
    z = z.reshape(B, g + 1, V)
    z[:, :g] = zq.float().numpy()
    z = z.reshape(B * (g + 1), V)
    zqd = zq.double().numpy()
    x = np.zeros((B, g), dtype=np.int32)
    for b in range(B):
        for j in range(g):
            n = F.filtered(zqd[b, j], *s)[1]
            order = np.lexsort((np.arange(V), -zqd[b, j]))
            x[b, j] = order[n - 1 if b < B - 1 or j != g // 2 else n]
    want = F.accept(z.astype(np.float64), zqd, x, lens, offs, ua, ur, [s] * B)
    assert want[0].tolist() == [g] * (B - 1) + [g // 2]
    c = lambda a: torch.from_numpy(a).cuda()
    a, t = sd.sd_accept_filtered(c(z), zq.cuda(), c(x), None, None, c(ua), c(ur), sd.SamplingParams(**mix, n=B))
    assert np.array_equal(a.cpu().numpy(), want[0])
    assert np.array_equal(t.cpu().numpy(), want[1])


@pytest.mark.parametrize("B,g,V", [(1, 3, 30000), (4, 5, 3000), (40, 7, 20600)])
def test_accept_filtered_graph_and_two_streams(B, g, V):
    """A captured call replayed with new inputs between eager ones, and two calls at once on
    streams and workspaces of their own."""
    params = sd.SamplingParams(top_p=0.9, temperature=0.9, n=B)
    cases = []
    for seed in (1, 2, 3):
        gen = torch.Generator("cuda").manual_seed(seed)
        z = 1.5 * torch.randn((B * (g + 1), V), device="cuda", generator=gen)
        zq = (z.view(B, g + 1, V)[:, :g] + 0.3 * torch.randn((B, g, V), device="cuda", generator=gen)).to(torch.bfloat16).contiguous()
        x = torch.randint(0, V, (B, g), device="cuda", generator=gen, dtype=torch.int32)
        x[:, :g // 2] = z.view(B, g + 1, V)[:, :g // 2].argmax(2).int()
        ua = 0.1 * torch.rand((B, g), device="cuda", generator=gen)
        ur = torch.rand((B, g + 1), device="cuda", generator=gen)
        cases.append((z, zq, x, ua, ur))
    call = lambda s, **k: sd.sd_accept_filtered(s[0], s[1], s[2], None, None, s[3], s[4], params, **k)
    eager = [[t.clone() for t in call(s)] for s in cases]
    nbytes = sd.accept_filtered_workspace_bytes(B, g, V)
    live = [t.clone() for t in cases[0]]
    ws = sd.new_workspace(nbytes, "cuda")
    out = (torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda"))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        call(live, accept_len=out[0], next_token=out[1], workspace=ws)
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(live, accept_len=out[0], next_token=out[1], workspace=ws)
    for i in (1, 2, 0, 2):
        for a, b in zip(live, cases[i]):
            a.copy_(b)
        graph.replay()
        assert torch.equal(out[0], eager[i][0]) and torch.equal(out[1], eager[i][1])
        again = call(cases[i])
        assert torch.equal(again[0], eager[i][0]) and torch.equal(again[1], eager[i][1])
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [sd.new_workspace(nbytes, "cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        got = []
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got.append(call(cases[k], workspace=spaces[k]))
        torch.cuda.synchronize()
        for k in range(2):
            assert torch.equal(got[k][0], eager[k][0]) and torch.equal(got[k][1], eager[k][1])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V,rows", [(1000, 24), (40009, 24), (20611, 560)])
def test_sample_three_filters(V, rows, dtype):
    """Top-k, top-p and min-p together, each of them the shortest run in some rows: the share of
    top-p is one of the top-k run, whatever min-p leaves of it."""
    g = np.random.default_rng(rows + V)
    z = head_logits(rows, V, rows)
    z[::4, g.random(V) < 0.98] = -np.inf
    settings = [(float(np.float32(t)), int(k), float(np.float32(p)), float(np.float32(m)))
                for t, k, p, m in zip(g.choice([0.6, 0.8, 1.1], rows), g.choice([15, 80, 320], rows),
                                      g.choice([0.8, 0.9, 0.95], rows), g.choice([0.01, 0.03, 0.07], rows))]
    col = lambda i, dt: torch.tensor([s[i] for s in settings], dtype=dt, device="cuda")
    params = sd.SamplingParams(col(0, torch.float32), col(1, torch.int32), col(2, torch.float32), col(3, torch.float32))
    check_rows(z, g.random(rows, dtype=np.float32), settings, params, TYPES[dtype])


@pytest.mark.parametrize("B,g,V", [(3, 5, 2000), (2, 4, 30011)])
def test_accept_filtered_three_filters(B, g, V):
    mix = dict(temperature=0.8, top_k=90, top_p=0.9, min_p=0.04)
    s = f32(mix)
    z, zq, lens, offs, ua, ur = accept_case(B, g, V, 21)
    zqd = zq.double().numpy()
    x = draft_by_sampling(zqd, [s] * B, 2)
    want = F.accept(z.astype(np.float64), zqd, x, lens, offs, ua, ur, [s] * B)
    c = lambda a: torch.from_numpy(a).cuda()
    a, t = sd.sd_accept_filtered(c(z), zq.cuda(), c(x), None, None, c(ua), c(ur), sd.SamplingParams(**mix, n=B))
    assert np.array_equal(a.cpu().numpy(), want[0])
    assert np.array_equal(t.cpu().numpy(), want[1])


@pytest.mark.parametrize("B,g,V", [(60, 3, 1200), (60, 2, 21000)])
def test_accept_filtered_short_runs(B, g, V):
    """Top-k runs that end before min-p's: what min-p alone would keep has no probability."""
    r = np.random.default_rng(V)
    settings = [(float(np.float32(0.8 + 0.4 * r.random())), int(r.integers(2, 9)), 1.0,
                 float(np.float32(0.002 + 0.02 * r.random()))) for _ in range(B)]
    z, zq, lens, offs, ua, ur = accept_case(B, g, V, 8)
    zqd = zq.double().numpy()
    r2 = np.random.default_rng(1)
    x = np.array([[F.draw(F.filtered(zqd[b, j], *settings[b])[0], r2.random()) for j in range(g)] for b in range(B)], dtype=np.int32)
    col = lambda i, dt: torch.tensor([s[i] for s in settings], dtype=dt, device="cuda")
    params = sd.SamplingParams(col(0, torch.float32), col(1, torch.int32), col(2, torch.float32), col(3, torch.float32))
    c = lambda a: torch.from_numpy(a).cuda()
    for seed in range(4):
        ur = np.random.default_rng(seed).random((B, g + 1), dtype=np.float32)
        want = F.accept(z.astype(np.float64), zqd, x, lens, offs, ua, ur, settings)
        a, t = sd.sd_accept_filtered(c(z), zq.cuda(), c(x), None, None, c(ua), c(ur), params)
        assert np.array_equal(a.cpu().numpy(), want[0])
        assert np.array_equal(t.cpu().numpy(), want[1])
